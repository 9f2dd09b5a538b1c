"""Kernels that are launched early wait for the ones ahead before anything else: what they read before it may not be written
yet, whatever was launched directly ahead (CPU: the sources are read)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_state_gb300", "csrc")


def test_every_early_kernel_waits_before_it_reads():
    sources = {p: open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))}
    early = set()
    for text in sources.values():
        early |= set(re.findall(r"\b(\w+_kernel)<", " ".join(re.findall(r"launch_early\(([^;]*);", text))))
    early |= {"append_rope_kernel"}                              # (by a pointer)
    assert early == {"add_rmsnorm_kernel", "append_rope_kernel", "bounds_kernel", "score_one_kernel", "score_kernel", "pick_kernel",
                     "decode_attention_kernel"}
    for name in early:
        body = [t.split(name + "(const ", 1)[1] for t in sources.values() if re.search(r"__global__[^;{]*\b%s\(const " % name, t)]
        assert len(body) == 1, name
        before = body[0].split("{", 1)[1].split("wait_for_earlier_kernels()")[0]
        for word in ("a.cu", "a.q", "a.k", "a.start", "a.page_table", "a.x", "load8", "owner_with", "__ldg"):
            assert not re.search(r"(?<!\w)%s\b" % re.escape(word), before), (name, word)
