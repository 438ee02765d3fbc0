"""Argument checks of the 8-bit cache's C entries: host only, no device is touched before they pass."""
import ctypes

import pytest

from turboquant_compressed_kv_tq_gb300 import _lib, build

FAKE = 0x10000   # never looked at


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def cache(**kw):
    d = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, code_layer_stride=0, scale_layer_stride=0, num_layers=1, num_blocks=8, block_tokens=16,
             num_kv_heads=2, head_dim=64, format=0)
    d.update(kw)
    return _lib.tq_kv8_cache(**d)


def rows(**kw):
    d = dict(data=FAKE, stride_batch=1024, stride_head=512, stride_token=64)
    d.update(kw)
    return _lib.tq_rows(**d)


def append(lib, c=None, layer=0, k=None, v=None, dtype=1, batch=1, n=4, seq=FAKE, table=FAKE, width=4, rope=None):
    c, k, v = c or cache(), k or rows(), v or rows()
    return lib.tq_kv8_append(ctypes.byref(c), layer, ctypes.byref(k), ctypes.byref(v), dtype, batch, n, seq, None, table, width,
                             ctypes.byref(rope) if rope else None, None, None)


def attention(lib, c=None, layer=0, q=None, dtype=1, batch=1, heads=4, L=1, seq=FAKE, table=FAKE, width=4, max_seq=64, scores=None, out=None):
    c, q, out = c or cache(), q or rows(), out or rows(data=2 * FAKE)
    return lib.tq_kv8_attention(ctypes.byref(c), layer, ctypes.byref(q), dtype, batch, heads, L, seq, None, table, width, max_seq,
                                ctypes.byref(scores) if scores else None, ctypes.byref(out), None, 0, None)


INVALID, UNSUPPORTED, CAPACITY = _lib.TQ_ERR_INVALID_ARG, _lib.TQ_ERR_UNSUPPORTED, _lib.TQ_ERR_CAPACITY


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=96), UNSUPPORTED), (dict(block_tokens=8), UNSUPPORTED), (dict(block_tokens=48), UNSUPPORTED),
    (dict(block_tokens=512), UNSUPPORTED), (dict(format=2), UNSUPPORTED), (dict(num_blocks=0), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(num_layers=0), INVALID), (dict(k_codes=None), INVALID),
    (dict(v_scales=None), INVALID), (dict(k_codes=FAKE + 8), INVALID), (dict(num_layers=2, code_layer_stride=16, scale_layer_stride=16), INVALID),
    (dict(num_layers=2, code_layer_stride=8 * 2 * 16 * 64, scale_layer_stride=15), INVALID),
    (dict(num_layers=2, code_layer_stride=8 * 2 * 16 * 64 + 8, scale_layer_stride=16), INVALID),
])
def test_caches(lib, kw, want):
    assert append(lib, c=cache(**kw)) == want
    assert attention(lib, c=cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(layer=1), INVALID), (dict(layer=-1), INVALID), (dict(dtype=3), INVALID), (dict(batch=-1), INVALID),
    (dict(batch=32768), INVALID), (dict(width=0), INVALID), (dict(seq=None), INVALID), (dict(table=None, batch=3), CAPACITY),
])
def test_common(lib, kw, want):
    assert append(lib, **kw) == want
    assert attention(lib, **kw) == want


@pytest.mark.parametrize("r", [rows(data=None), rows(data=FAKE + 2), rows(stride_token=68), rows(stride_head=4), rows(stride_batch=-4)])
def test_rows(lib, r):
    assert append(lib, k=r) == INVALID
    assert append(lib, v=r) == INVALID
    assert attention(lib, q=r) == INVALID
    assert attention(lib, out=r) == INVALID


def test_append_only(lib):
    assert append(lib, n=-1) == INVALID
    assert append(lib, n=65) == CAPACITY
    for rot, want in ((24, UNSUPPORTED), (80, UNSUPPORTED), (-16, UNSUPPORTED), (32, INVALID)):
        assert append(lib, rope=_lib.tq_rope(None, rot, 0, 1.0)) == want
    assert append(lib, rope=_lib.tq_rope(FAKE, 32, 0, float("inf"))) == INVALID
    assert append(lib, n=0) == 0 and append(lib, batch=0) == 0


def test_attention_only(lib):
    assert attention(lib, dtype=_lib.TQ_F32) == UNSUPPORTED
    for kw in (dict(heads=3), dict(heads=0), dict(L=-1), dict(max_seq=-1), dict(max_seq=(1 << 30) + 1), dict(L=1 << 30), dict(out=rows())):
        assert attention(lib, **kw) == INVALID
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")), dict(scale=float("inf"))):
        assert attention(lib, scores=_lib.tq_kv8_scores(**kw)) == INVALID
    assert attention(lib, L=0) == 0 and attention(lib, batch=0) == 0
    n = ctypes.c_size_t(7)
    assert lib.tq_kv8_workspace_bytes(ctypes.byref(cache()), 1, 4, 1, 64, None) == INVALID
    assert lib.tq_kv8_workspace_bytes(ctypes.byref(cache()), 1, 3, 1, 64, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.tq_kv8_workspace_bytes(ctypes.byref(cache(head_dim=32)), 1, 4, 1, 64, ctypes.byref(n)) == UNSUPPORTED
    assert lib.tq_kv8_workspace_bytes(ctypes.byref(cache()), 0, 4, 1, 64, ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("name", ["tq_kv8_cache", "tq_rows", "tq_rope", "tq_kv8_scores"])
def test_struct_layout_matches_header(tmp_path, name):
    import os
    import subprocess
    s = getattr(_lib, name)
    fields = [f for f, _ in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "tq.h"\nint main(void) {\n  printf("%zu\\n", sizeof(' + name + '));\n'
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-I", inc, str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(s)] + [getattr(s, f).offset for f in fields]
