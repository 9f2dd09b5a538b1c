"""Calls on another stream than the current one that make their own workspaces and results, while the
current stream allocates, writes and frees memory of the same sizes."""
import numpy as np
import pytest
import torch

from kv4_testutil import cu_of, make_cache, packed_q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


def kda():
    import kda_state_gb300
    return kda_state_gb300


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def churn(sizes):
    """The current stream takes blocks of these sizes, fills them and gives them back."""
    for n in sizes:
        torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("news", [[1, 1, 1], [70, 90, 64]])
def test_attention_and_gather(news, handle):
    lens, D, P, H, Hq = [6000, 95, 700], 128, 16, 2, 8
    pool, table = make_cache(lens, H, D, P, 90)
    q = packed_q(news, Hq, D, torch.bfloat16, 91).to(DEV)
    args = (q, cu_of(news).to(DEV), max(news), i32(lens), i32(table), torch.as_tensor(pool).to(DEV))
    where = (args[1], i32([a - n for a, n in zip(lens, news)]), sum(news), *args[4:])
    want, want_lse = kda().kda_kv4_attention(*args)
    want_k, want_v = kda().kda_kv4_gather(*where)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        s.wait_stream(torch.cuda.current_stream())
        on = s.cuda_stream if handle else s
        o, lse = kda().kda_kv4_attention(*args, stream=on)
        churn([kda().kv4_workspace_bytes(), o.numel() * 2, lse.numel() * 4])
        k, v = kda().kda_kv4_gather(*where, stream=on)
        churn([k.numel() * 2, kda().kv4_workspace_bytes()])
        torch.cuda.current_stream().wait_stream(s)
        for x, y in ((o, want), (lse, want_lse), (k, want_k), (v, want_v)):
            assert torch.equal(x, y)


def test_forks_and_compaction():
    N, P, rows, M, layers = 400, 16, 24, 12, 4
    rng = np.random.default_rng(5)
    data = [torch.from_numpy(rng.integers(0, 256, (N, 64, 1024), dtype=np.uint8)).to(DEV) for _ in range(layers)]
    s = torch.cuda.Stream()

    def step(stream):
        pools = [x.clone() for x in data]
        refs, table, lens = i32([0] * N), i32([[-1] * M] * rows), i32([0] * rows)
        grow = i32([37 + 3 * b if b < 12 else 0 for b in range(rows)])
        src, dst, gone = i32(range(12)), i32(range(12, 24)), i32(range(0, 12, 2))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kda().kda_page_alloc(refs, table, lens, grow, P, stream=stream)
        kda().kda_page_fork(pools, refs, table, lens, src, dst, P, stream=stream)
        churn([96, 192] * 4)
        kda().kda_page_free(refs, table, lens, gone, P, stream=stream)
        live = kda().kda_page_compact(pools, refs, table, stream=stream)
        churn([(3 * N + 16) * 4, 4] * 4)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return [live, refs, table, lens] + pools

    want = step(None)
    torch.cuda.synchronize()
    for _ in range(10):
        for x, y in zip(step(s), want):
            assert torch.equal(x, y)
