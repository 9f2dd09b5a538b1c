"""The plain calls' way from Python to the library takes exact CUDA tensors alone (CPU: everything else is left to the
functions of the binding, without an exception)."""
import pytest
import torch

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def quick():
    from kda_state_gb300 import _build
    _build.build()
    import kda_state_gb300.binding as binding
    binding.lib()
    return binding._quick


def test_is_loaded_with_the_library(quick):
    assert quick.__file__.endswith("_quick.so")


CALLS = [
    ("add_rmsnorm", lambda t: (t(3, 64, BF), t(3, 64, BF), t(64, BF), 1e-5, 1, None)),
    ("append_rope", lambda t: (t(3, 4, 64, BF), t(3, 2, 64, BF), t(3, 2, 64, BF), t(9, 64, torch.float32), t(3, I32), t(2, I32), t(2, 5, I32),
                               t(8, 2, 1, 1152, U8), False, 1.0, 1.0, None, None)),
    ("bounds", lambda t: (t(3, I32), t(2, I32), 3, t(2, 5, I32), t(8, 2, 1, 1152, U8), t(8, 2, 144, torch.int8), None)),
    ("pick", lambda t: (t(3, 4, 64, BF), t(3, I32), 2, t(2, I32), t(2, 5, I32), t(8, 2, 144, torch.int8), 16, 3, 1, 1, t(4096, U8), None)),
    ("attention_picked", lambda t: (t(3, 4, 64, BF), t(3, I32), 2, t(2, I32), t(2, 5, I32), t(3, 2, 3, I32), t(8, 2, 1, 1152, U8), None, 1.0, 1.0,
                                    t(4096, U8), None)),
    ("append", lambda t: (t(3, 2, 64, BF), t(3, 2, 64, BF), t(3, I32), t(2, I32), t(2, 5, I32), t(8, 2, 1, 1152, U8), 1.0, 1.0, None)),
    ("gather", lambda t: (t(3, I32), t(2, I32), 3, t(2, 5, I32), t(8, 2, 1, 1152, U8), BF, 1.0, 1.0, None)),
    ("attention", lambda t: (t(3, 4, 64, BF), t(3, I32), 2, t(2, I32), t(2, 5, I32), t(8, 2, 1, 1152, U8), 0.1, 0, 1.0, 1.0, t(4096, U8), None)),
]


def cpu(*spec):
    return torch.zeros(spec[:-1], dtype=spec[-1])


@pytest.mark.parametrize("name,args", CALLS, ids=[n for n, _ in CALLS])
def test_what_is_not_plain_is_left(quick, name, args):
    call = getattr(quick, name)
    assert call(*args(cpu)) is None                              # not on a GPU
    assert call() is None and call(*args(cpu)[:-1]) is None
    for i in range(len(args(cpu))):
        for other in (None, 3, "x", 1e300, 2 ** 70, [1], object()):
            a = list(args(cpu))
            a[i] = other
            assert call(*a) is None


def test_addresses_are_needed(quick):
    with pytest.raises(TypeError):
        quick.bind(1, 2)
    with pytest.raises(ValueError):
        quick.bind(*[0] * 8)
    with pytest.raises(TypeError):
        quick.bind(*["x"] * 8)
