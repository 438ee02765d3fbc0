"""The bytes that the Python calls hand to the library are those of the C structs."""
import ctypes

import turboquant_compressed_kv_tq_gb300 as tq
from turboquant_compressed_kv_tq_gb300 import _lib


def as_bytes(s):
    return ctypes.string_at(ctypes.addressof(s), ctypes.sizeof(s))


def test_rows():
    values = (0x123456789ABC0, 1 << 40, -3, 77)
    assert tq._pack_rows(*values) == as_bytes(_lib.tq_rows(*values))


def test_scores():
    rope = _lib.tq_rope(0x1000, 64, 1, 0.5)
    packed = tq._pack_scores(0.25, 50.0, 0x2000, 4096, 0x3000, 0x4000, ctypes.addressof(rope), 0x5000)
    s = _lib.tq_kv8_scores.from_buffer_copy(packed)
    assert ctypes.sizeof(s) == len(packed)
    assert (s.scale, s.softcap, s.slopes, s.window, s.prefix_lens, s.doc_starts, s.positions) == (0.25, 50.0, 0x2000, 4096, 0x3000, 0x4000, 0x5000)
    assert s.rope.contents.rot_dim == 64 and s.rope.contents.inv_freq == 0x1000 and s.rope.contents.scale == 0.5
    empty = _lib.tq_kv8_scores()
    assert tq._pack_scores(0.0, 0.0, 0, 0, 0, 0, 0, 0) == as_bytes(empty)
