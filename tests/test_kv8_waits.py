"""Waits that run out: read from the source, since no test may make a GPU hang."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "turboquant_compressed_kv_tq_gb300", "csrc")


def test_chunk_kernel_gives_up_a_warp_at_a_time():
    """A lane whose wait ran out may not leave its warp before tensor-memory loads and shuffles of all its lanes. Softmax
    warps wait through arrived_warp, which has one answer for all lanes; a converter's lane goes on with its warp, without
    waiting again; the MMAs' single thread waits for itself."""
    text = open(os.path.join(CSRC, "kv8_prefill.cu")).read()
    softmax, convert, mma = (text.index(f"// ================================================= {w}\n") for w in ("softmax", "convert", "mma"))
    assert re.search(r"bool arrived_warp\(.*\) \{ return __all_sync\(0xffffffffu, arrived\(bar, parity\)\); \}", text)
    assert not re.search(r"(?<![_\w])arrived\(", text[softmax:convert]) and text[softmax:convert].count("arrived_warp(") >= 4
    warps = text[convert:mma]
    assert re.findall(r".*(?<![_\w])arrived\(.*", warps) == re.findall(r" *if \(i > 0 && ok\) ok = .*", warps)
    assert not re.search(r"!ok\) *(break|return)|&& ok; \+\+i", warps)
    single = text[mma:text.index("\ntemplate", mma)]
    assert "if (lane == 0 && n_tiles > 0) {" in single and "arrived_warp(" not in single


def test_split_kernel_votes_on_its_waits():
    text = open(os.path.join(CSRC, "kv8_decode.cu")).read()
    i = text.index("dead = !arrived(")
    assert "if (__any_sync(0xffffffffu, dead)) {" in text[i:i + 200]
