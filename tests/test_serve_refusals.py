"""Argument checks of the calls around the caches': host only, no device is touched before they pass."""
import ctypes

import pytest

import turboquant_compressed_kv_tq_gb300 as tq
from turboquant_compressed_kv_tq_gb300 import _lib, build

FAKE = 0x10000   # never looked at
INVALID, UNSUPPORTED = _lib.TQ_ERR_INVALID_ARG, _lib.TQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def blocks(**kw):
    return _lib.tq_blocks(**(dict(table=FAKE, free_blocks=FAKE, n_used=FAKE, n_free=8, max_blocks=4, block_tokens=16, num_blocks=8) | kw))


def reserve(lib, b=None, batch=2, seq=FAKE, news=None, n=1, places=None):
    b = b or blocks()
    return lib.tq_blocks_reserve(ctypes.addressof(b), batch, seq, news, n, ctypes.addressof(places) if places else None, None)


def release(lib, b=None, batch=2, keep=FAKE):
    b = b or blocks()
    return lib.tq_blocks_release(ctypes.addressof(b), batch, keep, None)


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), INVALID), (dict(n_used=None), INVALID), (dict(free_blocks=None), INVALID), (dict(n_free=-1), INVALID),
    (dict(max_blocks=0), INVALID), (dict(num_blocks=0), INVALID), (dict(block_tokens=8), UNSUPPORTED), (dict(block_tokens=48), UNSUPPORTED),
    (dict(block_tokens=0), UNSUPPORTED), (dict(max_blocks=1 << 27), INVALID),
])
def test_block_tables(lib, kw, want):
    assert reserve(lib, blocks(**kw)) == want
    assert release(lib, blocks(**kw)) == want


def test_blocks_calls(lib):
    assert lib.tq_blocks_reserve(None, 1, FAKE, None, 1, None, None) == INVALID
    assert lib.tq_blocks_release(None, 1, FAKE, None) == INVALID
    assert reserve(lib, batch=-1) == INVALID and release(lib, batch=-1) == INVALID
    assert reserve(lib, seq=None) == INVALID and release(lib, keep=None) == INVALID
    assert reserve(lib, n=-1) == INVALID
    assert reserve(lib, batch=(1 << 24) + 1, n=0) == INVALID and release(lib, batch=(1 << 24) + 1) == INVALID
    assert reserve(lib, places=_lib.tq_places(max_tokens=-1)) == INVALID
    assert reserve(lib, places=_lib.tq_places(slots=FAKE, max_tokens=4)) == INVALID          # maps without starts
    # 2^31 places: rows that can be given 2^20 each
    assert reserve(lib, blocks(max_blocks=1 << 16), batch=1 << 11, n=1 << 20) == INVALID
    assert reserve(lib, batch=0) == 0 and release(lib, batch=0) == 0


def rows(**kw):
    return _lib.tq_rows(**(dict(data=FAKE, stride_batch=8 * 64, stride_head=64, stride_token=16 * 8 * 64) | kw))


def rope(lib, r=None, back=0, dtype=1, D=64, batch=2, n=3, q=None, qh=8, qo=None, k=None, kh=2, ko=None):
    r = r or _lib.tq_rope(FAKE, 32, 0, 1.0)
    q, qo = q or rows(), qo or rows(data=FAKE << 8)
    a = ctypes.addressof
    return lib.tq_rope_apply(a(r), back, dtype, D, batch, n, a(q), qh, a(qo), a(k) if k else None, kh, a(ko) if ko else None, None, None, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=1040), UNSUPPORTED), (dict(r=_lib.tq_rope(FAKE, 24, 0, 1.0)), UNSUPPORTED),
    (dict(r=_lib.tq_rope(FAKE, 80, 0, 1.0)), UNSUPPORTED), (dict(r=_lib.tq_rope(FAKE, -16, 0, 1.0)), UNSUPPORTED),
    (dict(r=_lib.tq_rope(None, 32, 0, 1.0)), INVALID), (dict(r=_lib.tq_rope(FAKE, 32, 0, float("nan"))), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(batch=-1), INVALID), (dict(n=-1), INVALID), (dict(batch=1 << 16, n=1 << 15), INVALID),
    (dict(qh=0), INVALID), (dict(qh=65536), INVALID), (dict(k=rows(data=FAKE << 10), ko=rows(data=FAKE << 12), kh=0), INVALID),
    (dict(q=rows(data=None)), INVALID), (dict(q=rows(data=FAKE + 2)), INVALID), (dict(qo=rows(data=(FAKE << 8) + 8)), INVALID),
    (dict(q=rows(stride_token=68)), INVALID), (dict(qo=rows(stride_head=4)), INVALID), (dict(k=rows(data=FAKE << 10)), INVALID),
])
def test_rope(lib, kw, want):
    assert rope(lib, **kw) == want


def test_rope_of_nothing(lib):
    assert rope(lib, batch=0) == 0 and rope(lib, n=0) == 0
    assert lib.tq_rope_apply(None, 0, 1, 64, 1, 1, None, 1, None, None, 0, None, None, None, None, None) == INVALID


def token_major(data, heads, of, n, D=64, dtype_bytes=2):
    """Heads `of`.. of a fused [batch][n][heads][D]."""
    return _lib.tq_rows(data + of * D * dtype_bytes, n * heads * D, D, heads * D)


def test_rope_outputs_that_overlap(lib):
    n, H = 3, 12
    q, k = token_major(FAKE, H, 0, n), token_major(FAKE, H, 8, n)
    size = 2 * n * H * 64 * 2
    far = FAKE << 8

    def call(qo, ko, q=q, k=k, qh=8, kh=2):
        return rope(lib, q=q, qo=qo, k=k, ko=ko, qh=qh, kh=kh)

    # refused: an output over the other's input or output, a row over its neighbour, another layout over the same memory
    assert call(token_major(FAKE, H, 2, n), token_major(far, H, 8, n)) == INVALID          # q's rows, two heads on
    assert call(token_major(far, H, 0, n), token_major(FAKE, H, 6, n)) == INVALID          # k into q's last heads
    assert call(token_major(far, H, 0, n), token_major(far, H, 7, n)) == INVALID           # the outputs over one another
    assert call(_lib.tq_rows(far, n * 8 * 64, 32, 8 * 64), token_major(far << 4, H, 8, n)) == INVALID   # heads half a row apart
    assert call(_lib.tq_rows(far, 0, 64, H * 64), token_major(far << 4, H, 8, n)) == INVALID            # one row for both sequences
    assert call(_lib.tq_rows(FAKE, 8 * n * 64, n * 64, 64), token_major(far, H, 8, n)) == INVALID       # head-major over the projection
    assert call(token_major(FAKE + size - 3 * 128, H, 0, n), token_major(far, H, 8, n)) == INVALID      # its first row over k's last
    wrong = _lib.tq_rows(far + 8, n * 8 * 64, 64, 8 * 64)
    assert call(q, wrong) == INVALID and call(wrong, k) == INVALID


def drafts(**kw):
    return _lib.tq_drafts(**(dict(target=FAKE, target_stride_batch=300, target_stride_row=100, draft=FAKE, draft_tokens=FAKE, uniforms=FAKE, noise=FAKE,
                                  noise_stride=100, target_dtype=1, draft_dtype=0) | kw))


def verify(lib, d=None, batch=1, K=2, V=100, acc=FAKE, tokens=FAKE, logs=None, keep=None):
    d = d or drafts()
    return lib.tq_verify_drafts(ctypes.addressof(d), batch, K, V, acc, tokens, logs, keep, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INVALID), (dict(batch=(1 << 24) + 1), INVALID), (dict(V=(1 << 28) + 1), INVALID), (dict(K=-1), INVALID), (dict(K=65), UNSUPPORTED), (dict(V=0), INVALID), (dict(acc=None), INVALID), (dict(tokens=None), INVALID),
    (dict(keep=FAKE), INVALID), (dict(d=drafts(target=None)), INVALID), (dict(d=drafts(target=FAKE + 1)), INVALID), (dict(d=drafts(draft=FAKE + 2)), INVALID),
    (dict(d=drafts(target_dtype=3)), INVALID), (dict(d=drafts(draft_dtype=7)), INVALID), (dict(d=drafts(draft_tokens=None)), INVALID),
    (dict(d=drafts(uniforms=None)), INVALID),
])
def test_verify(lib, kw, want):
    assert verify(lib, **kw) == want


def test_verify_of_nothing(lib):
    assert verify(lib, batch=0) == 0
    assert lib.tq_verify_drafts(None, 1, 0, 10, FAKE, FAKE, None, None, None) == INVALID


@pytest.mark.parametrize("name", ["tq_blocks", "tq_places", "tq_drafts"])
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


def test_packed_drafts_are_the_struct():
    values = [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16]
    s = _lib.tq_drafts.from_buffer_copy(tq._pack_drafts(*values))
    assert [getattr(s, f) for f, _ in s._fields_] == values[:13] + [14, 15, 16]
