"""The 8-bit cache on the GPU: appending with rotation and attention over it, against their definitions in 64 bits."""
import math

import pytest
import torch

import kv8_util as ref
import turboquant_compressed_kv_tq_gb300 as tq

pytestmark = pytest.mark.gpu
E4M3, INT8, BF16, F16, F32 = ref.E4M3, ref.INT8, ref.BF16, ref.F16, ref.F32
DEV = "cuda"


@pytest.fixture(autouse=True)
def no_device_error():
    tq_errors()
    yield
    torch.cuda.synchronize()
    assert tq_errors() == 0


def tq_errors():
    try:
        return tq.tq_device_error()
    except tq.TQError:
        return -1


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def dirty_cache(blocks, H, BT, D, fmt, seed, layers=1):
    """A cache whose unwritten bytes are anything at all, NaN codes among them."""
    c = tq.KV8Cache(layers, blocks, BT, H, D, fmt)
    g = gen(seed)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(torch.randint(64, 191, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


def filled_cache(blocks, H, BT, D, fmt, seed, spread=1):
    """A cache of plausible contents: no NaN code, scales 2^-6 .. 2^(spread - 7)."""
    c = dirty_cache(blocks, H, BT, D, fmt, seed)
    g = gen(seed + 1)
    for t in (c.k_codes, c.v_codes):
        if fmt == E4M3:
            t.copy_(torch.where((t & 0x7F) == 0x7F, torch.zeros_like(t), t))
            t.copy_((torch.randn(t.shape, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            t.copy_((torch.randn(t.shape, generator=g, device=DEV) * 40).round().clamp(-127, 127).to(torch.int8).view(torch.uint8))
    for t in (c.k_scales, c.v_scales):
        t.copy_(127 - 6 + torch.randint(0, spread, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


def shuffled_table(B, width, blocks, seed):
    return torch.randperm(blocks, generator=gen(seed), device=DEV)[: B * width].to(torch.int32).view(B, width)


# ------------------------------------------------------------------ append

def check_append(c, before, k, v, lens, news, table, rope, positions=None):
    """Every byte of layer 0 against the definition; `before`: clones of the cache's tensors."""
    fmt, BT = c.format, c.block_tokens
    touched = torch.zeros((c.num_blocks, BT), dtype=torch.bool, device=DEV)
    for b, (N, n) in enumerate(zip(lens, news)):
        for lb in range(N // BT, -(-(N + n) // BT) if n else 0):
            id = int(table[b, lb])
            s0, s1 = max(N - lb * BT, 0), min(N + n - lb * BT, BT)
            touched[id, :s1] = True
            for x, codes, scales, oc, ox, turn in ((k, c.k_codes, c.k_scales, before[0], before[2], True),
                                                   (v, c.v_codes, c.v_scales, before[1], before[3], False)):
                i0 = lb * BT + s0 - N
                y = x[b, :, i0:i0 + s1 - s0].double()
                size = torch.zeros_like(y)
                if turn and rope is not None:
                    pos = positions[b, i0:i0 + s1 - s0] if positions is not None else torch.arange(N + i0, N + i0 + s1 - s0, device=DEV)
                    inter = bool(rope.desc.interleaved)
                    size = ref.rotated(y.abs(), pos * 0, rope.inv_freq, inter, rope.desc.scale)
                    rot = 2 * rope.inv_freq.numel()
                    if rot:   # |x1| + |x2| of each pair, in both places
                        z = size[..., :rot]
                        z = (z[..., 0::2] + z[..., 1::2]).repeat_interleave(2, -1) if inter else (z[..., :rot // 2] + z[..., rot // 2:]).repeat(1, 1, 2)
                        size = torch.cat((z, torch.zeros_like(size[..., rot:])), -1)
                    y = ref.rotated(y, pos, rope.inv_freq, inter, rope.desc.scale)
                # fp32 rotation: cos and sin within 2^-22, three roundings of 2^-24 each
                err = size * 2.0 ** -21
                for h in range(c.num_kv_heads):
                    e = int(scales[0, id, h]) - 127
                    tops = [float(y[h].abs().max()), float((y[h].abs() + err[h]).max()), max(float((y[h].abs() - err[h]).max()), 0.0)]
                    want = {ref.exponent(t, fmt) for t in tops}
                    if s0 > 0:
                        want = {max(w, int(ox[0, id, h]) - 127) for w in want}
                    assert e in want
                    got = ref.values(codes[0, id, h, s0:s1], fmt) * 2.0 ** e
                    z = y[h] * 2.0 ** -e
                    off = (ref.nearest(z, fmt) - z).abs() * 2.0 ** e
                    assert ((got - y[h]).abs() <= off + err[h]).all()
                    if s0 > 0:   # the earlier tokens, at the scale they have now
                        if e == int(ox[0, id, h]) - 127:   # which they had
                            assert torch.equal(oc[0, id, h, :s0], codes[0, id, h, :s0])
                            continue
                        old = ref.values(oc[0, id, h, :s0], fmt) * 2.0 ** (int(ox[0, id, h]) - 127 - e)
                        fine = ~old.isnan()
                        assert torch.equal(ref.nearest(old, fmt)[fine], ref.values(codes[0, id, h, :s0], fmt)[fine])
    for codes, old in ((c.k_codes, before[0]), (c.v_codes, before[1])):
        same = (codes[0] == old[0]) | touched[:, None, :, None]
        assert same.all()   # bytes behind the last token, and other blocks, stay
    for scales, old in ((c.k_scales, before[2]), (c.v_scales, before[3])):
        assert torch.equal(scales[0][~touched.any(1)], old[0][~touched.any(1)])
    for t, o in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), before):
        assert torch.equal(t[1:], o[1:])


def tensors(c):
    return [t.clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("D,BT,H,n,lens,news,rot,inter,dtype,major", [
    (128, 16, 3, 1, [0, 15, 16, 37], None, 128, False, BF16, "token"),
    (128, 64, 2, 200, [0, 63, 130], None, 128, False, BF16, "head"),
    (64, 32, 2, 77, [5, 0, 31, 64], [77, 0, 1, 40], 32, True, F16, "token"),
    (256, 128, 1, 129, [127, 3], None, 256, False, F32, "head"),
    (256, 256, 2, 700, [0, 255], [700, 513], 64, False, BF16, "token"),
    (64, 16, 1, 33, [1], None, 0, False, F32, "head"),
    (128, 256, 1, 2, [255, 254], None, 96, True, F16, "head"),
])
def test_append(fmt, D, BT, H, n, lens, news, rot, inter, dtype, major):
    B = len(lens)
    width = max(lens) // BT + (n - 1) // BT + 2
    blocks = B * width + 3
    c = dirty_cache(blocks, H, BT, D, fmt, 1, layers=2)
    c.k_scales.clamp_(100, 125)
    c.v_scales.clamp_(100, 125)
    table = shuffled_table(B, width, blocks, 2)
    g = gen(3)
    shape = (B, n, H, D) if major == "token" else (B, H, n, D)
    k, v = ((torch.randn(shape, generator=g, device=DEV) * torch.exp2(torch.randint(-4, 5, shape[:3] + (1,), generator=g, device=DEV).float())).to(dtype)
            for _ in "kv")
    if major == "token":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    rope = tq.Rope.of_base(rot, 10000.0, interleaved=inter) if rot else None
    before = tensors(c)
    c.append(0, k, v, i32(lens), table, width, new_lens=None if news is None else i32(news), rope=rope)
    check_append(c, before, k, v, lens, news or [n] * B, table, rope)


def test_append_without_table_and_with_layers():
    c = dirty_cache(6, 2, 16, 64, E4M3, 4, layers=3)
    c.k_scales.fill_(110), c.v_scales.fill_(110)
    before = tensors(c)
    k, v = (torch.randn(2, 2, 20, 64, generator=gen(s), device=DEV) for s in (5, 6))
    c.append(1, k, v, i32([0, 9]), None, 3)
    one = tq.KV8Cache.wrap(c.k_codes[1:2].clone(), c.v_codes[1:2].clone(), c.k_scales[1:2].clone(), c.v_scales[1:2].clone())
    check_append(one, [t[1:2] for t in before], k, v, [0, 9], [20, 20], torch.arange(6).view(2, 3), None)
    for t, o in zip(tensors(c), before):
        assert torch.equal(t[0], o[0]) and torch.equal(t[2], o[2])


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_append_token_by_token(fmt):
    """Each token is a thousandth to a thousand times the last ones: scales grow on the way, never shrink."""
    D, BT, n = 64, 16, 40
    c = tq.KV8Cache(1, 3, BT, 1, D, fmt)
    g = gen(7)
    x = torch.randn(1, 1, n, D, generator=g, device=DEV) * torch.exp2(torch.randint(-10, 11, (1, 1, n, 1), generator=g, device=DEV).float())
    table = i32([[2, 0, 1]])
    for t in range(n):
        before = tensors(c)
        y = x[:, :, t:t + 1]
        c.append(0, y, -y, i32([t]), table, 3)
        check_append(c, before, y, -y, [t], [1], table, None)


@pytest.mark.parametrize("inter", [False, True])
def test_append_far_positions(inter):
    """Angles of positions up to 2^30 (float64 holds them to 2^-22 of a radian or so: 1e9 * 2^-53 * a few)."""
    D, n = 128, 64
    c = tq.KV8Cache(1, 4, 16, 1, D)
    k = torch.randn(1, 1, n, D, generator=gen(8), device=DEV)
    pos = torch.randint(0, 1 << 30, (1, n), generator=gen(9), device=DEV, dtype=torch.int32)
    pos[0, :3] = i32([0, 1, (1 << 30) - 1])
    rope = tq.Rope.of_base(D, 500000.0, interleaved=inter, scale=1.25)
    before = tensors(c)
    c.append(0, k, k, i32([0]), None, 4, rope=rope, positions=pos)
    check_append(c, before, k, k, [0], [n], torch.arange(4).view(1, 4), rope, pos)


@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_append_keeps_nan_and_infinity_out(fmt):
    c = tq.KV8Cache(1, 1, 16, 1, 64, fmt)
    k = torch.randn(1, 1, 4, 64, generator=gen(10), device=DEV)
    k[0, 0, 1, 3], k[0, 0, 2, 5], k[0, 0, 2, 6] = math.nan, math.inf, -math.inf
    clean = k.clone()
    clean[0, 0, 1, 3] = 0
    clean[0, 0, 2, 5:7] = 0
    c.append(0, k, clean, i32([0]), None, 1)
    assert tq.tq_device_error() == tq._lib.TQ_DEVERR_NONFINITE
    kc, vc = (ref.values(t[0, 0, 0], fmt) for t in (c.k_codes, c.v_codes))
    assert torch.equal(c.k_scales, c.v_scales)
    assert kc[1, 3] == 0 and kc[2, 5] == ref.TOP[fmt] and kc[2, 6] == -ref.TOP[fmt]
    kc[2, 5:7] = 0
    assert torch.equal(kc, vc)


def test_append_extremes():
    """Zeros, and magnitudes beyond the scales' range."""
    c = tq.KV8Cache(1, 4, 16, 1, 64)
    x = torch.zeros(4, 1, 1, 64, device=DEV)
    x[1] = 2.0 ** -90
    x[2] = 3e38
    x[3] = 2.0 ** -60
    c.append(0, x, x, i32([0, 0, 0, 0]), None, 1)
    assert c.k_scales[0, :, 0].tolist() == [64, 64, 190, 64]
    assert ref.values(c.k_codes[0, :, 0, 0, 0], E4M3).tolist() == [0.0, 0.0, 448.0, 8.0]


def test_append_violations_are_flagged_and_skipped():
    c = dirty_cache(4, 1, 16, 64, E4M3, 11)
    before = tensors(c)
    x = torch.randn(1, 1, 20, 64, generator=gen(12), device=DEV)
    for lens, news, table, width, flag in (([-1], None, [[0, 1]], 2, tq.TQ_DEVERR_SEQLEN), ([0], [21], [[0, 1]], 2, tq.TQ_DEVERR_SEQLEN),
                                           ([0], [-2], [[0, 1]], 2, tq.TQ_DEVERR_SEQLEN), ([40], None, [[0, 1]], 2, tq.TQ_DEVERR_CAPACITY),
                                           ([0], None, [[-1, 4]], 2, tq.TQ_DEVERR_BLOCK)):
        c.append(0, x, x, i32(lens), i32(table), width, new_lens=None if news is None else i32(news))
        assert tq.tq_device_error() == flag
        for t, o in zip(tensors(c), before):
            assert torch.equal(t, o)
    c.append(0, x, x, i32([20]), i32([[0, 1]]), 2)   # 12 of the 20 fit
    assert tq.tq_device_error() == tq.TQ_DEVERR_CAPACITY
    check_append(c, before, x, x, [20], [12], i32([[0, 1]]), None)
    assert not torch.equal(c.k_codes, before[0])


# ------------------------------------------------------------------ attention

def see_of(N, nq, window=0, prefix=0, docs=None):
    p = torch.arange(N - nq, N, device=DEV)
    t = torch.arange(N, device=DEV)
    see = t <= p[:, None]
    if window:
        see &= p[:, None] - t < window
    if docs is not None:
        see &= t >= docs[:, None]
    return p, see | (t < prefix)


def check_attention(c, q, out, before, lens, news, table, scale=0.0, cap=0.0, slopes=None, window=0, prefixes=None, docs=None,
                    rope=None, positions=None):
    fmt, BT, D = c.format, c.block_tokens, c.head_dim
    B, Hq, L, _ = q.shape
    for b, (N, nq) in enumerate(zip(lens, news)):
        assert torch.equal(out[b, :, nq:], before[b, :, nq:])
        if nq == 0:
            continue
        ids = table[b, :-(-N // BT)].long()
        ids = ids.clamp(0, c.num_blocks - 1)   # entries of blocks that nobody sees
        k, v = ((ref.values(codes[0, ids], fmt) * torch.exp2(scales[0, ids].double() - 127)[..., None, None]).transpose(0, 1).reshape(c.num_kv_heads, -1, D)[:, :N]
                for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)))
        p, see = see_of(N, nq, window, prefixes[b] if prefixes else 0, docs[b, :nq] if docs is not None else None)
        qq = q[b, :, :nq].double()
        if rope is not None:
            qq = ref.rotated(qq, positions[b, :nq] if positions is not None else p, rope.inv_freq, bool(rope.desc.interleaved), rope.desc.scale)
        sc = scale or 1 / math.sqrt(D)
        seen = see.any(0)
        k = torch.where(seen[:, None], k, 0.0)
        v = torch.where(seen[:, None], v, 0.0)
        want, wv, size = ref.attention(qq, k, v, p, see, sc, cap, slopes)
        tol = ref.bound(want, wv, size, q.dtype, N, float(v.abs().max()) if N else 0.0, D, cap, float(slopes.max()) if slopes is not None else 0.0)
        got = out[b, :, :nq].double()
        assert torch.isfinite(got).all()
        off = ((got - want).abs() / tol).max()
        assert off <= 1, (b, float(off))
        empty = ~see.any(1)
        assert (got[:, empty] == 0).all()


def attend(c, q, lens, table, max_seq=None, q_lens=None, out=None, **kw):
    return c.attention(0, q, i32(lens), table, table.shape[1], max(lens) if max_seq is None else max_seq,
                       q_lens=None if q_lens is None else i32(q_lens), out=out, **kw)


CASES = [
    # D, BT, H, G, L, lens, q_lens, options
    (128, 16, 2, 4, 1, [1, 16, 17, 300], None, {}),
    (128, 256, 1, 8, 2, [5000, 257], None, {"rope": 128}),
    (128, 32, 2, 1, 1, [0, 1, 2], None, {}),
    (64, 16, 3, 5, 3, [3, 33, 100, 1025], None, {"cap": 20.0}),
    (256, 64, 1, 2, 4, [4, 777], None, {"bias": True, "rope": 64}),
    (64, 128, 2, 8, 1, [640, 129], None, {"window": 100, "prefix": [3, 0]}),
    (128, 16, 1, 16, 4, [900, 64], [4, 2], {"window": 33, "cap": 50.0, "rope": 128, "inter": True}),
    (128, 64, 2, 3, 7, [7, 70, 2000], [7, 0, 3], {"prefix": [7, 65, 1999]}),
    (64, 16, 1, 2, 50, [50, 333], [50, 49], {"docs": 20}),
    (128, 32, 2, 4, 65, [65, 1000], None, {"docs": 33, "prefix": [10, 500], "bias": True, "cap": 30.0, "rope": 128}),
    (256, 16, 2, 1, 130, [130, 190], [130, 1], {"rope": 256}),
    (64, 64, 1, 4, 257, [300, 257], None, {"window": 50}),
    (128, 128, 1, 8, 300, [300, 1111], [299, 300], {"rope": 128, "scale": 0.3}),
    (128, 16, 2, 2, 513, [513, 2049], None, {"empty": True}),
    (256, 256, 1, 8, 40, [40, 600], None, {"cap": 10.0, "prefix": [40, 1]}),
    # more than 16 rows behind long sequences: still split over the tokens
    (128, 64, 2, 4, 16, [20000, 9001], None, {"rope": 128}),
    (64, 32, 4, 8, 12, [4000, 100, 33], [12, 5, 0], {"docs": 700, "prefix": [3999, 2, 0]}),
    (64, 16, 4, 8, 12, [3000, 12, 13, 2999, 16, 1500, 600, 29], None, {"cap": 25.0, "bias": True}),
    (256, 64, 1, 8, 50, [6000], None, {"window": 3000, "rope": 256}),
]


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, BF16), (E4M3, F16), (INT8, F16)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, fmt, dtype):
    D, BT, H, G, L, lens, news, o = CASES[case]
    B, width = len(lens), max(lens) // BT + 2
    blocks = B * width + 2
    c = filled_cache(blocks, H, BT, D, fmt, 20 + case, spread=4)
    table = shuffled_table(B, width, blocks, 21)
    # behind the last token: anything, NaN codes among it; behind the last block: no block at all
    junk = dirty_cache(blocks, H, BT, D, fmt, 22)
    for b, N in enumerate(lens):
        for lb in range(width):
            id, used = int(table[b, lb]), min(max(N - lb * BT, 0), BT)
            c.k_codes[0, id, :, used:] = junk.k_codes[0, id, :, used:]
            c.v_codes[0, id, :, used:] = 0x7F
            if used == 0:
                table[b, lb] = -1 - lb
    g = gen(23)
    q = torch.randn(B, L, H * G, D, generator=g, device=DEV).to(dtype).transpose(1, 2)
    out = torch.randn(B, L, H * G, D, generator=g, device=DEV).to(dtype).transpose(1, 2)
    before = out.clone()
    kw, ck = {}, {}
    if "rope" in o:
        kw["rope"] = ck["rope"] = tq.Rope.of_base(o["rope"], interleaved=o.get("inter", False))
    if "cap" in o:
        kw["softcap"] = ck["cap"] = o["cap"]
    if "scale" in o:
        kw["scale"] = ck["scale"] = o["scale"]
    if "window" in o:
        kw["window"] = ck["window"] = o["window"]
    if "bias" in o:
        kw["slopes"] = ck["slopes"] = torch.rand(H * G, generator=g, device=DEV) * 0.5
    if "prefix" in o:
        ck["prefixes"] = o["prefix"]
        kw["prefix_lens"] = i32(o["prefix"])
    if "docs" in o or "empty" in o:
        n = i32(news or [L] * B)[:, None]
        p = i32(lens)[:, None] - n + torch.arange(L, device=DEV, dtype=torch.int32)
        d = p // o["docs"] * o["docs"] if "docs" in o else torch.where(p % 3 == 0, p + 1, p - p % 7)   # every third row sees nothing
        kw["doc_starts"] = ck["docs"] = d.to(torch.int32).contiguous()
    got = attend(c, q, lens, table, q_lens=news, out=out, **kw)
    assert got is out
    check_attention(c, q, out, before, lens, news or [L] * B, table, **ck)


@pytest.mark.parametrize("L", [1, 6, 300])
def test_attention_scales_apart(L):
    """Blocks whose scales differ by 2^40, values that matter in the small ones, zeros at the smallest scale."""
    D, BT, H, G, N = 128, 16, 1, 2, 700
    width = N // BT + 1
    c = filled_cache(width, H, BT, D, E4M3, 30)
    e = torch.randint(0, 41, (1, width, 1), generator=gen(31), device=DEV)
    c.v_scales.copy_((101 + e).to(torch.uint8))
    c.v_codes[0, 3] = 0
    c.v_scales[0, 3] = 64
    c.k_scales.copy_((121 - e % 7).to(torch.uint8))
    q = torch.randn(1, H * G, L, D, generator=gen(32), device=DEV).to(BF16)
    table = torch.arange(width, dtype=torch.int32, device=DEV).view(1, width)
    out = attend(c, q, [N], table)
    check_attention(c, q, out, out, [N], [L], table)
    # keys of one hot block with a small value scale: the large blocks' weights vanish next to it
    c.k_codes[0, 5] = c.k_codes[0, 5, :, :1]
    out = attend(c, q * 8, [N], table)
    check_attention(c, q * 8, out, out, [N], [L], table)


@pytest.mark.parametrize("L", [1, 4, 200])
def test_attention_queries_of_any_size(L):
    """bf16 queries far outside fp16's range, scaled back by the softmax scale."""
    c = filled_cache(8, 1, 16, 64, INT8, 33)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8)
    n = min(L, 128)
    q = torch.randn(1, 2, n, 64, generator=gen(34), device=DEV)
    for x in (1e30, 1e-30):
        big = (q * x).to(BF16)
        out = attend(c, big, [128], table, scale=0.125 / x)
        check_attention(c, big, out, out, [128], [n], table, scale=0.125 / x)


@pytest.mark.parametrize("L", [1, 2, 256])
def test_attention_far_into_the_pool(L):
    """Codes behind 2^32 bytes, a long table, a window that skips most of it."""
    D, BT, H = 128, 256, 4
    blocks = (1 << 32) // (BT * H * D) + 40
    c = tq.KV8Cache(1, blocks, BT, H, D)
    N = 39 * BT + 17
    ids = torch.arange(blocks - 40, blocks, device=DEV)
    for t in (c.k_codes, c.v_codes):
        t[0, blocks - 40:] = (torch.randn((40, H, BT, D), generator=gen(35), device=DEV) * 60).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_scales.fill_(121), c.v_scales.fill_(121)
    table = ids.flip(0).to(torch.int32).view(1, 40).contiguous()
    q = torch.randn(1, H, L, D, generator=gen(36), device=DEV).to(BF16)
    out = attend(c, q, [N], table)
    check_attention(c, q, out, out, [N], [L], table)
    x = torch.randn(1, H, 300, D, generator=gen(37), device=DEV).to(BF16)
    before = [t[:, blocks - 40:].clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]
    c.append(0, x, x, i32([N - 250]), table, 40)
    tail = tq.KV8Cache.wrap(*(t[:, blocks - 40:].clone() for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)))
    check_append(tail, before, x, x, [N - 250], [250 + 17 + 33], table - (blocks - 40), None)


@pytest.mark.parametrize("L", [1, 300])
def test_attention_unseen_blocks_may_be_gone(L):
    """A window's earlier blocks are freed: their table entries are anything."""
    D, BT, N, W = 64, 16, 2000, 130
    width = N // BT + 1
    c = filled_cache(width, 2, BT, D, E4M3, 40)
    table = torch.arange(width, dtype=torch.int32, device=DEV).view(1, width)
    first = (N - L - W + 1) // BT
    table[0, 1:first] = 1 << 30
    q = torch.randn(1, 4, L, D, generator=gen(41), device=DEV).to(F16)
    out = attend(c, q, [N], table, window=W, prefix_lens=i32([4]))
    check_attention(c, q, out, out, [N], [L], table, window=W, prefixes=[4])


@pytest.mark.parametrize("L", [1, 200])
def test_attention_violations_are_flagged(L):
    c = filled_cache(16, 1, 16, 64, E4M3, 42)
    table = torch.arange(16, dtype=torch.int32, device=DEV).view(1, 16)
    q = torch.randn(1, 2, L, 64, generator=gen(43), device=DEV).to(BF16)
    for n in (-5, 257, 1 << 30):
        out = attend(c, q, [n], table, max_seq=256)
        assert tq.tq_device_error() == tq.TQ_DEVERR_SEQLEN
        assert (out == 0).all()
    out = attend(c, q, [200], table, max_seq=199)
    assert tq.tq_device_error() == tq.TQ_DEVERR_SEQLEN and (out == 0).all()
    for nq in (-1, L + 1):
        out = torch.ones_like(q)
        attend(c, q, [256], table, q_lens=[nq], out=out)
        assert tq.tq_device_error() == tq.TQ_DEVERR_SEQLEN
        check_attention(c, q, out, torch.ones_like(q), [256], [min(max(nq, 0), L)], table)
    # a block id outside the pool: a block that nobody sees
    bad = table.clone()
    bad[0, 2], bad[0, 5] = -1, 16
    out = attend(c, q, [256], bad)
    assert tq.tq_device_error() == tq.TQ_DEVERR_BLOCK
    k, v = ((ref.values(t[0, :, 0], E4M3) * torch.exp2(s[0].double() - 127)[..., None]).reshape(1, 256, 64) for t, s in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)))
    p, see = see_of(256, L)
    see[:, 32:48] = False
    see[:, 80:96] = False
    want, wv, size = ref.attention(q[0].double(), k, v, p, see, 0.125)
    assert ((out[0].double() - want).abs() <= ref.bound(want, wv, size, BF16, 256, float(v.abs().max()), 64)).all()


@pytest.mark.parametrize("L,G", [(1, 1), (3, 4), (60, 1), (60, 4)])
@pytest.mark.parametrize("inter", [False, True])
def test_attention_rotation_positions(L, G, inter):
    """Queries rotated to positions of the caller's, far ones among them; part of the head, and a scale."""
    D, BT, N = 128, 32, 200
    c = filled_cache(8, 2, BT, D, E4M3, 100)
    table = shuffled_table(1, 8, 8, 101)
    pos = torch.randint(0, 1 << 29, (1, L), generator=gen(102), device=DEV, dtype=torch.int32)
    rope = tq.Rope.of_base(96, 1e6, interleaved=inter, scale=0.75)
    for dtype in (BF16, F16):
        q = torch.randn(1, 2 * G, L, D, generator=gen(103), device=DEV).to(dtype)
        out = attend(c, q, [N], table, rope=rope, positions=pos)
        check_attention(c, q, out, out, [N], [L], table, rope=rope, positions=pos)


@pytest.mark.parametrize("L", [1, 5, 70])
def test_attention_of_a_layer_and_with_a_negative_scale(L):
    D, BT, N = 64, 16, 150
    c = tq.KV8Cache(3, 10, BT, 1, D)
    one = filled_cache(10, 1, BT, D, E4M3, 110)
    for t, o in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), (one.k_codes, one.v_codes, one.k_scales, one.v_scales)):
        t[1] = o[0]
    table = torch.arange(10, dtype=torch.int32, device=DEV).view(1, 10)
    q = torch.randn(1, 4, L, D, generator=gen(111), device=DEV).to(BF16)
    for scale in (0.2, -0.2):
        out = c.attention(1, q, i32([N]), table, 10, N, scale=scale)
        check_attention(one, q, out, out, [N], [L], table, scale=scale)
        assert torch.equal(out, attend(one, q, [N], table, scale=scale))
    # without a table, the blocks in order
    assert torch.equal(c.attention(1, q, i32([N]), None, 10, N), attend(one, q, [N], table))


@pytest.mark.parametrize("L", [1, 9, 300])
def test_attention_over_nothing(L):
    c = filled_cache(4, 2, 16, 128, INT8, 120)
    q = torch.randn(3, 4, L, 128, generator=gen(121), device=DEV).to(F16)
    out = torch.ones_like(q)
    c.attention(0, q, i32([0, 0, 0]), None, 1, 0, out=out)
    assert (out == 0).all()
    out = torch.ones_like(q)
    c.attention(0, q, i32([0, 16, 0]), None, 1, 16, out=out, q_lens=i32([L, 0, 1]))
    assert (out[0] == 0).all() and (out[1] == 1).all() and (out[2, :, :1] == 0).all() and (out[2, :, 1:] == 1).all()


# ------------------------------------------------------------------ together, as a program uses them

def serve(c, table, k, v, q, steps, rope, L0, **kw):
    """A prompt of L0 tokens, then `steps` single tokens; returns the outputs."""
    B, width = table.shape
    outs = []
    at, n = 0, L0
    for _ in range(steps + 1):
        lens = i32([at] * B)
        c.append(0, k[:, :, at:at + n], v[:, :, at:at + n], lens, table, width, rope=rope)
        outs.append(c.attention(0, q[:, :, at:at + n], lens + n, table, width, at + n, rope=rope, **kw))
        at, n = at + n, 1
    return outs


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("D,G,BT,L0", [(128, 4, 16, 70), (64, 8, 64, 33), (256, 2, 32, 129)])
def test_prompt_then_tokens(fmt, D, G, BT, L0):
    B, H, steps = 2, 2, 6
    T = L0 + steps
    width = T // BT + 1
    c = dirty_cache(B * width, H, BT, D, fmt, 50)
    table = shuffled_table(B, width, B * width, 51)
    g = gen(52)
    qkv = torch.randn(B, T, H * G + 2 * H, D, generator=g, device=DEV).to(BF16)   # one projection, token-major
    q, k, v = qkv[:, :, :H * G].transpose(1, 2), qkv[:, :, H * G:H * G + H].transpose(1, 2), qkv[:, :, H * G + H:].transpose(1, 2)
    rope = tq.Rope.of_base(D)
    outs = serve(c, table, k, v, q, steps, rope, L0)
    # against attention over the unrounded keys and values: their 8-bit rounding is off by at most half a step
    p, see = see_of(T, T)
    kr = ref.rotated(k.double(), p, rope.inv_freq)
    at = 0
    for o in outs:
        n = o.shape[2]
        for b in range(B):
            pp = p[at:at + n]
            qq = ref.rotated(q[b, :, at:at + n].double(), pp, rope.inv_freq)
            want, wv, size = ref.attention(qq, kr[b, :, :at + n], v[b, :, :at + n].double(), pp, see[at:at + n, :at + n], D ** -0.5)
            # e4m3: half a step is 2^-4 of a value (and 2^-10 of the scale below); int8: half a unit of scales up to
            # 2^-4 (magnitudes up to 127 / 16). A value may be rounded twice (its block's scale grew).
            half = 2 * 2.0 ** -4 if fmt == E4M3 else 0.0
            unit = 2 * 2.0 ** -5 if fmt == INT8 else 2 * 2.0 ** -10 * 2.0 ** -5
            qn = qq.abs().sum(-1, keepdim=True) * D ** -0.5
            d = half * size + unit * qn
            tol = ref.bound(want, wv, size, BF16, at + n, 8.0, D) + 2 * d.clamp(max=20).exp() * d * wv + half * wv + unit
            assert ((o[b].double() - want).abs() <= tol).all()
        at += n
    # and exactly: the cache's own values
    last = outs[-1]
    check_attention(c, q[:, :, T - 1:], last, last, [T] * B, [1] * B, table, rope=rope)


def test_captured_and_replayed_with_other_inputs():
    B, H, G, D, BT, N = 2, 2, 4, 128, 16, 900
    width = N // BT + 2
    c = filled_cache(B * width, H, BT, D, E4M3, 60)
    table = shuffled_table(B, width, B * width, 61)
    rope = tq.Rope.of_base(D)
    lens = i32([N - 7, N])
    q, k, v = (torch.randn(B, n, 1, D, generator=gen(62 + n), device=DEV).to(BF16) for n in (H * G, H, H))
    ws = [torch.empty(c.workspace_bytes(B, H * G, 1, N + 20), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]

    def step(i):
        c.append(0, k, v, lens, table, width, rope=rope)
        grown = lens + 1
        c.attention(0, q, grown, table, width, N + 20, out=outs[i], workspace=ws[i], rope=rope)

    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(1)
    for s in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen(70 + s), device=DEV).to(BF16))
        lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        now = [int(x) + 1 for x in lens]
        check_attention(c, q, outs[1], outs[1], now, [1] * B, table, rope=rope)


def test_two_calls_at_once_on_two_streams():
    D, BT, H, G, N = 128, 64, 2, 4, 40000
    width = N // BT + 1
    c = filled_cache(width, H, BT, D, INT8, 80)
    table = torch.arange(width, dtype=torch.int32, device=DEV).view(1, width)
    qs = [torch.randn(1, H * G, n, D, generator=gen(81 + n), device=DEV).to(BF16) for n in (1, 2, 130)]
    want = [attend(c, q, [N], table).clone() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[] for _ in qs]
    for _ in range(5):
        for i, (q, s) in enumerate(zip(qs, streams)):
            with torch.cuda.stream(s):
                got[i].append(attend(c, q, [N], table))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for o in many:
            assert torch.equal(w, o)   # the same bits every time: joins have a fixed order


def test_next_to_the_compressed_cache():
    """One block table and one set of lengths address the 8-bit cache and a compressed cache."""
    D, BT, H, G, N = 128, 16, 2, 4, 100
    kc, vc = tq.Codec(D, 4, tq.TQ_MODE_MSE, 0), tq.Codec(D, 4, tq.TQ_MODE_MSE, 1)
    width = N // BT + 1
    comp = tq.CompressedKVCache(kc, vc, 1, width, BT, H)
    c = tq.KV8Cache(1, width, BT, H, D)
    table = shuffled_table(1, width, width, 90)
    k, v = (torch.randn(1, H, N, D, generator=gen(s), device=DEV).to(BF16) for s in (91, 92))
    q = torch.randn(1, H * G, 1, D, generator=gen(93), device=DEV).to(BF16)
    zero, n = i32([0]), i32([N])
    comp.append(0, k, v, zero, table, width)
    c.append(0, k, v, zero, table, width)
    out4 = torch.empty(1, H * G, 1, D, device=DEV)
    ws = torch.empty(comp.workspace_bytes(1, H * G, 1, N), dtype=torch.uint8, device=DEV)
    comp.decode(0, q, n, table, width, N, out4, ws)
    out8 = c.attention(0, q, n, table, width, N)
    p, see = see_of(N, 1)
    want, _, _ = ref.attention(q[0].double(), k[0].double(), v[0].double(), p, see, D ** -0.5)
    e4, e8 = ((o[0].double() - want).norm() / want.norm() for o in (out4, out8))
    assert e8 < e4 and e8 < 2.0 ** -4   # at most half a step of e4m3 a value


# ------------------------------------------------------------------ refusals of the Python entry points

def test_refusals():
    c = tq.KV8Cache(1, 8, 16, 2, 64)
    x = torch.zeros(1, 2, 4, 64, device=DEV, dtype=BF16)
    n0 = i32([0])
    ok = dict(block_table=None, max_blocks=8)
    with pytest.raises(ValueError):
        c.append(0, x[:, :1], x, n0, **ok)
    with pytest.raises(ValueError):
        c.append(0, x, x.half(), n0, **ok)
    with pytest.raises(ValueError):
        c.append(0, x, x.cpu(), n0, **ok)
    with pytest.raises(ValueError):
        c.append(0, x, x, n0.long(), **ok)
    with pytest.raises(ValueError):
        c.append(0, x, x, i32([0, 0]), **ok)
    with pytest.raises(ValueError):
        c.append(0, x, torch.zeros(1, 2, 64, 4, device=DEV, dtype=BF16).transpose(2, 3), n0, **ok)
    with pytest.raises(tq.TQError):   # rows that do not start on 16 bytes
        c.append(0, torch.zeros(1, 2, 4, 72, device=DEV, dtype=BF16)[..., 4:68], x, n0, **ok)
    with pytest.raises(tq.TQError):
        c.append(1, x, x, n0, **ok)
    with pytest.raises(TypeError):
        c.append(0, x.double(), x.double(), n0, **ok)
    with pytest.raises(tq.TQError):
        c.append(0, x, x, n0, rope=tq.Rope.of_base(72, 10.0), **ok)
    with pytest.raises(tq.TQError):
        c.append(0, x, x, n0, rope=tq.Rope.of_base(24, 10.0), **ok)
    with pytest.raises(tq.TQError):
        c.attention(0, x.float(), n0, None, 8, 16)
    with pytest.raises(tq.TQError):
        c.attention(0, x[:, :1].expand(1, 3, 4, 64), n0, None, 8, 16)
    with pytest.raises(tq.TQError):
        c.attention(0, x, n0, None, 8, 16, out=x)
    with pytest.raises(tq.TQError):
        c.attention(0, x, n0, None, 8, 16, window=-1)
    with pytest.raises(tq.TQError):
        c.attention(0, x, n0, None, 8, 16, softcap=-1.0)
    with pytest.raises(ValueError):
        c.attention(0, x, n0, None, 8, 16, slopes=torch.zeros(3, device=DEV))
    with pytest.raises(ValueError):
        c.attention(0, x, n0, None, 8, 16, doc_starts=i32([[0]]))
    big = tq.KV8Cache(1, 64, 256, 2, 64)
    need = big.workspace_bytes(1, 2, 1, 16384)
    assert need > 0
    with pytest.raises(tq.TQError):
        big.attention(0, x[:, :, :1], n0, None, 64, 16384, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        tq.KV8Cache.wrap(c.k_codes, c.v_codes[:, :4], c.k_scales, c.v_scales)
    # nothing to do is done
    c.append(0, x[:, :, :0], x[:, :, :0], n0, **ok)
    c.append(0, x[:0], x[:0], n0[:0], **ok)
    assert c.attention(0, x[:, :, :0], n0, None, 8, 16).shape == (1, 2, 0, 64)
