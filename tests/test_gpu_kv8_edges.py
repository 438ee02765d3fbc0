"""The 8-bit cache's attention where it can go wrong: the chunk kernel's own forms, scales far apart, caps of any size,
windows of any size, against the definition in 64 bits with a bound for each row."""
import math

import pytest
import torch

import kv8_util as ref
import test_gpu_kv8 as base
import turboquant_compressed_kv_tq_gb300 as tq
from test_gpu_kv8 import BF16, DEV, E4M3, F16, F32, INT8, gen, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    base.tq_errors()
    yield
    torch.cuda.synchronize()
    assert base.tq_errors() == 0


def kernel_of(c, B, Hq, L, max_seq):
    """"chunk" or "few": the chunk kernel takes no workspace, and the sizes here are beyond the eight tiles that few rows do without."""
    H = c.num_kv_heads
    assert B * H * -(-(Hq // H * L) // 16) * -(-max_seq // 16) > 8
    return "few" if c.workspace_bytes(B, Hq, L, max_seq) else "chunk"


def check(c, q, out, lens, news, table, kernel, scale=0.0, cap=0.0, slopes=None, window=0, prefixes=None, docs=None, rope=None):
    """Every row against the definition, within what the roundings of its own visible keys may do:

    scores, d: the queries' fp16 (2^-11 of each product if they were rotated and go in one part, else 2^-22; 2^-25 of the
    row's largest coordinate for the small ones), the rotation in fp32 (2^-21), fp32 sums ((D + 8) 2^-24), the cap (2^-19
    of the capped score), the bias (3 roundings of slope x distance), score plus scale exponent less reference in fp32
    (2^-22 of the largest). An error d of every score moves the output by at most (e^2d - 1) sum w |v|.
    weights: fp16 (2^-11) of weight x value scale, for which the chunk kernel takes the tile's largest up to 2^6 apart;
    below 2^-14 of the reference an absolute 2^-25 of it (the reference is at most the row's largest such product), or all
    of a smaller one; fp32 sums in steps of 16 keys (2^-22 each).
    output: half a step."""
    fmt, BT, D, H = c.format, c.block_tokens, c.head_dim, c.num_kv_heads
    Hq = q.shape[1]
    G = Hq // H
    two = rope is None or (q.dtype == F16 and (kernel == "few" or D == 64))
    tile = 16 if kernel == "few" else 64 if D == 256 else 128
    limit = 0 if kernel == "few" else 6
    sc = scale or 1 / math.sqrt(D)
    worst = 0.0
    for b, (N, nq) in enumerate(zip(lens, news)):
        ids = table[b, :-(-N // BT)].long().clamp(0, c.num_blocks - 1)
        p, see = base.see_of(N, nq, window, prefixes[b] if prefixes else 0, docs[b, :nq] if docs is not None else None)
        seen = see.any(0)
        k, v = (ref.values(codes[0, ids], fmt).transpose(0, 1).reshape(H, -1, D)[:, :N] for codes in (c.k_codes, c.v_codes))
        ek, ev = (s[0, ids].double().sub(127).transpose(0, 1).repeat_interleave(BT, 1)[:, :N] for s in (c.k_scales, c.v_scales))   # [H, N]
        k, v = (torch.where(seen[:, None], x * torch.exp2(e)[..., None], 0.0) for x, e in ((k, ek), (v, ev)))
        x0 = q[b, :, :nq].double()
        qq, rsize = x0, torch.zeros_like(x0)
        if rope is not None:
            inter = bool(rope.desc.interleaved)
            qq = ref.rotated(x0, p, rope.inv_freq, inter, rope.desc.scale)
            rot = 2 * rope.inv_freq.numel()
            z = x0[..., :rot].abs() * abs(rope.desc.scale)
            z = (z[..., 0::2] + z[..., 1::2]).repeat_interleave(2, -1) if inter else (z[..., :rot // 2] + z[..., rot // 2:]).repeat(1, 1, 2)
            rsize[..., :rot] = z
        k_, v_, ev_ = (t.repeat_interleave(G, 0) for t in (k, v, ev))
        kt = k_.transpose(1, 2)
        s = (qq @ kt) * sc
        size = (qq.abs() @ kt.abs()) * abs(sc)
        d = size * ((2.0 ** -22 if two else 2.0 ** -11) + (D + 8) * 2.0 ** -24) + 2.0 ** -25 * qq.abs().amax(-1, keepdim=True) * kt.abs().sum(1, keepdim=True) * abs(sc)
        d = d + (rsize @ kt.abs()) * abs(sc) * 2.0 ** -21
        if cap:
            s = cap * torch.tanh(s / cap)
            d = d + 2.0 ** -19 * size.clamp(max=cap)
        if slopes is not None:
            far = slopes.double()[:, None, None] * (p[:, None] - torch.arange(N, device=DEV)).abs()
            s = s - far
            d = d + 3 * 2.0 ** -24 * far
        d = d + 2.0 ** -22 * (s.abs() + ev_.abs()[:, None])
        d = d.masked_fill(~see, 0.0).amax(-1, keepdim=True)
        empty = ~see.any(1)
        w = torch.softmax(s.masked_fill(~see, -math.inf).masked_fill(empty[:, None], 0.0), -1).masked_fill(empty[:, None], 0.0)
        want, wv = w @ v_, w @ v_.abs()
        T = -(-N // tile) * tile
        top = torch.full((Hq, T), -1000.0, device=DEV, dtype=torch.float64)
        top[:, :N] = torch.where(seen, ev_, -1000.0)
        top = top.view(Hq, -1, tile).amax(-1).repeat_interleave(tile, 1)[:, :N]
        ev0 = torch.where(seen, ev_, 0.0)
        most = (w * torch.exp2(torch.where(seen, torch.minimum(top, ev_ + limit), 0.0))[:, None]).amax(-1, keepdim=True)
        small = torch.minimum(w * torch.exp2(ev0)[:, None], 2.0 ** -25 * most) @ (v_.abs() * torch.exp2(-ev0)[..., None])
        tol = want.abs() * (torch.finfo(q.dtype).eps / 2) + wv * (2.0 ** -11 + torch.expm1(2 * d) * 1.01 + (N / 16 + 16) * 2.0 ** -22) + small
        tol = tol + (2.0 ** -25 if q.dtype == F16 else 2.0 ** -134)
        got = out[b, :, :nq].double()
        assert torch.isfinite(got).all(), b
        assert (got[:, empty] == 0).all(), b
        worst = max(worst, float(((got - want).abs() / tol).max()))
    assert worst <= 1, worst


def call(c, q, lens, table, max_seq=None, **kw):
    return base.attend(c, q, lens, table, max_seq=max_seq, **kw)


def straight(c, B=1):
    """Sequences over the pool's blocks in order."""
    return torch.arange(c.num_blocks, dtype=torch.int32, device=DEV).view(B, -1)


# ------------------------------------------------------------------ the chunk kernel's forms

FORMS = {
    "plain": {},
    "rotated": {"rope": 1.0},
    "half rotated": {"rope": 0.5, "inter": True},
    "cap": {"cap": 20.0},
    "bias": {"bias": True},
    "cap, bias, rotated": {"cap": 5.0, "bias": True, "rope": 1.0},
    "prefix": {"prefix": [70, 333]},
    "window, prefix, blocks gone": {"window": 50, "prefix": [5, 40], "gone": True},
    "documents, prefix, cap": {"docs": 57, "prefix": [1, 200], "cap": 30.0},
    "documents, bias": {"docs": 100, "bias": True, "rope": 1.0},
    "uneven scales": {"spread": 14},
    "uneven scales, cap, window": {"spread": 14, "cap": 8.0, "window": 200},
}


@pytest.mark.parametrize("fmt,dtype", [(E4M3, BF16), (INT8, F16)])
@pytest.mark.parametrize("D,BT", [(64, 16), (128, 32), (128, 256), (256, 16)])
@pytest.mark.parametrize("form", FORMS)
def test_chunk_forms(form, D, BT, fmt, dtype):
    o = FORMS[form]
    B, H, G, L, lens, news = 2, 2, 4, 300, [600, 411], [300, 277]
    width = -(-600 // BT) + 1
    blocks = B * width + 2
    c = base.filled_cache(blocks, H, BT, D, fmt, 200, spread=o.get("spread", 3))
    table = base.shuffled_table(B, width, blocks, 201)
    g = gen(202)
    q = torch.randn(B, H * G, L, D, generator=g, device=DEV).to(dtype)
    kw, ck = {}, {}
    if "rope" in o:
        kw["rope"] = ck["rope"] = tq.Rope.of_base(int(D * o["rope"]), interleaved=o.get("inter", False))
    if "cap" in o:
        kw["softcap"] = ck["cap"] = o["cap"]
    if "bias" in o:
        kw["slopes"] = ck["slopes"] = torch.rand(H * G, generator=g, device=DEV) * 0.2
    if "window" in o:
        kw["window"] = ck["window"] = o["window"]
    if "prefix" in o:
        kw["prefix_lens"], ck["prefixes"] = i32(o["prefix"]), o["prefix"]
    if "docs" in o:
        p = i32(lens)[:, None] - i32(news)[:, None] + torch.arange(L, device=DEV, dtype=torch.int32)
        kw["doc_starts"] = ck["docs"] = (p // o["docs"] * o["docs"]).to(torch.int32).contiguous()
    if "gone" in o:   # blocks between the prefix and the first window: no block at all
        for b in range(B):
            for lb in range(-(-o["prefix"][b] // BT), (lens[b] - news[b] - o["window"] + 1) // BT):
                table[b, lb] = -7
    assert kernel_of(c, B, H * G, L, max(lens)) == "chunk"
    out = call(c, q, lens, table, q_lens=news, **kw)
    check(c, q, out, lens, news, table, "chunk", **ck)
    assert (out[1, :, news[1]:] == 0).all()


@pytest.mark.parametrize("L", [1, 4, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotated_fp16_queries(D, L):
    """In two parts for few rows and at head_dim 64: one would be 2^-11 of each product off."""
    H, G, N, BT = 2, 4, 500, 64
    c = base.filled_cache(8, H, BT, D, E4M3, 210)
    q = (torch.randn(1, H * G, L, D, generator=gen(211), device=DEV) * 4).to(F16)
    rope = tq.Rope.of_base(D)
    kernel = kernel_of(c, 1, H * G, L, N)
    assert kernel == ("chunk" if L == 300 else "few")
    out = call(c, q, [N], straight(c), rope=rope)
    check(c, q, out, [N], [L], straight(c), kernel, rope=rope)


def test_chunk_far_into_the_pool():
    """Codes behind 2^32 bytes, for the chunk kernel."""
    D, BT, H, G, L, N = 128, 256, 4, 4, 600, 2400
    blocks = (1 << 32) // (BT * H * D) + 10
    c = tq.KV8Cache(1, blocks, BT, H, D)
    few = base.filled_cache(10, H, BT, D, E4M3, 220)
    for t, o in zip((c.k_codes, c.v_codes, c.k_scales, c.v_scales), (few.k_codes, few.v_codes, few.k_scales, few.v_scales)):
        t[:, blocks - 10:] = o
    q = torch.randn(1, H * G, L, D, generator=gen(221), device=DEV).to(BF16)
    order = torch.randperm(10, generator=gen(222), device=DEV).to(torch.int32).view(1, 10)
    assert kernel_of(c, 1, H * G, L, N) == "chunk"
    out = call(c, q, [N], order + (blocks - 10))
    check(few, q, out, [N], [L], order, "chunk")


# ------------------------------------------------------------------ windows of any size

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 300, 2 ** 30 + 5, 2 ** 30])
@pytest.mark.parametrize("N,L", [(10, 64), (600, 700), (1, 300), (300, 300)])
def test_windows_wider_than_everything(N, L, window):
    """As no window, also for sequences shorter than the queries' padded length."""
    H, G, D, BT = 2, 4, 128, 16
    c = base.filled_cache(40, H, BT, D, E4M3, 230)
    table = straight(c)
    q = torch.randn(1, H * G, L, D, generator=gen(231), device=DEV).to(BF16)
    assert kernel_of(c, 1, H * G, L, max(N, 8)) == "chunk"
    out = call(c, q, [N], table, max_seq=max(N, 8), window=window)
    assert torch.equal(out, call(c, q, [N], table, max_seq=max(N, 8)))
    check(c, q, out, [N], [L], table, "chunk")


# ------------------------------------------------------------------ scales far apart

@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("cap", [0.0, 12.0])
@pytest.mark.parametrize("D,BT", [(64, 32), (128, 64), (128, 16), (256, 32)])
def test_masked_neighbours_of_other_scales(D, BT, cap, fmt):
    """Documents of one block: a row sees one block only, whose scale may be 2^46 below its neighbours' in the same tile."""
    H, G, N = 2, 4, 384
    c = base.filled_cache(N // BT, H, BT, D, fmt, 240)
    g = gen(241)
    up = torch.randint(-8, -4, (2, N // BT, H), generator=g, device=DEV)
    ek, ev = (u + torch.where(torch.arange(N // BT, device=DEV)[:, None] % 3 == i, 0, -42) for i, u in enumerate(up))
    c.k_scales[0], c.v_scales[0] = (ek + 127).to(torch.uint8), (ev + 127).to(torch.uint8)
    table = straight(c)
    q = torch.randn(1, H, G, N, D, generator=g, device=DEV)
    q = q * torch.exp2(-6.0 - ek.float()).T.repeat_interleave(BT, 1)[None, :, None, :, None]   # scores of size 1 with their own block
    q = q.reshape(1, H * G, N, D).to(BF16)
    docs = (torch.arange(N, device=DEV, dtype=torch.int32) // BT * BT).view(1, N)
    assert kernel_of(c, 1, H * G, N, N) == "chunk"
    out = call(c, q, [N], table, doc_starts=docs, softcap=cap)
    check(c, q, out, [N], [N], table, "chunk", cap=cap, docs=docs)
    small = out[0].double().abs().amax((0, 2)).view(-1, BT).amax(1)   # of each block's rows
    assert (small > torch.exp2(ev.double().amax(1) - 4)).all()        # nothing vanished


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("apart", [3, 6, 7, 14, 23])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_values_next_to_seen_ones(D, apart, fmt):
    """Most rows see the first block and their own; the first one's neighbours, of larger values, are masked. Their scale may not
    cost the rows' own values, 2^-9 below the first block's, their digits."""
    H, G, N, L, BT = 2, 4, 600, 300, 16
    c = base.filled_cache(38, H, BT, D, fmt, 248)
    c.v_scales[0] = 127 - 15
    c.v_scales[0, 0] = 127 - 6
    c.v_scales[0, 1:8] = 127 - 6 + apart
    c.v_codes[0, 0, ..., ::2] = 0   # half the coordinates are the rows' own alone
    q = (torch.randn(1, H * G, L, D, generator=gen(249), device=DEV) * 0.1).to(BF16)
    assert kernel_of(c, 1, H * G, L, N) == "chunk"
    p = torch.arange(N - L, N, dtype=torch.int32, device=DEV)
    docs = torch.where(p % 20 == 0, 0, p - 15).to(torch.int32).view(1, L)   # a few rows see everything: nothing is skipped
    out = call(c, q, [N], straight(c), doc_starts=docs, prefix_lens=i32([16]))
    check(c, q, out, [N], [L], straight(c), "chunk", docs=docs, prefixes=[16])


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("L", [1, 5, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_seen_blocks_of_other_scales(D, L, fmt):
    """Rows that see blocks of all scales; one block's keys are liked by every row, so that its small values count."""
    H, G, N, BT, hot = 2, 4, 500, 16, 9
    c = base.filled_cache(32, H, BT, D, fmt, 250)
    g = gen(251)
    ev = torch.randint(-45, -35, (32, H), generator=g, device=DEV)
    ev[5] = ev[10] = ev[20] = -6
    ev[hot] = -50
    ev[12], c.v_codes[0, 12] = -63, 0
    c.v_scales[0] = (ev + 127).to(torch.uint8)
    one = torch.where(torch.rand(D, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    c.k_codes[0, hot] = ((one * 64).to(torch.float8_e4m3fn).view(torch.uint8) if fmt == E4M3 else (one * 64).to(torch.int8).view(torch.uint8))
    q = (torch.randn(1, H * G, L, D, generator=g, device=DEV) * 0.2 + one * 60 / math.sqrt(D)).to(BF16)
    table = straight(c)
    kernel = kernel_of(c, 1, H * G, L, 512)
    assert L == 5 or kernel == ("chunk" if L == 300 else "few")
    out = call(c, q, [N], table, max_seq=512)
    check(c, q, out, [N], [L], table, kernel)


@pytest.mark.parametrize("kind", ["keys", "values"])
@pytest.mark.parametrize("fmt,apart", [(E4M3, 14), (E4M3, 15), (E4M3, 16), (INT8, 23), (INT8, 24), (INT8, 25)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_at_the_edge_of_one_tile(D, fmt, apart, kind):
    """The furthest apart that a tile's codes go to one scale, and the next: codes of every size, down to the smallest."""
    H, G, N, BT = 2, 4, 384, 32
    c = base.filled_cache(N // BT, H, BT, D, fmt, 245)
    g = gen(246)
    every = torch.arange(256, device=DEV, dtype=torch.int32).to(torch.uint8)
    every = every[(every & 0x7F) != 0x7F] if fmt == E4M3 else every[every != 128]
    low = torch.arange(N // BT, device=DEV) % 2 == 1
    codes, exps = (c.k_codes, c.k_scales) if kind == "keys" else (c.v_codes, c.v_scales)
    codes[0] = every[torch.randint(0, len(every), codes[0].shape, generator=g, device=DEV)]
    exps[0] = (127 - 8 - low * apart)[:, None].to(torch.uint8)
    q = torch.randn(1, H * G, N, D, generator=g, device=DEV)
    if kind == "keys":   # scores of size 1 with their own block
        q = q * torch.exp2(low.float() * apart).repeat_interleave(BT)[:, None]
    q = q.to(BF16)
    docs = (torch.arange(N, device=DEV, dtype=torch.int32) // BT * BT).view(1, N)
    assert kernel_of(c, 1, H * G, N, N) == "chunk"
    out = call(c, q, [N], straight(c), doc_starts=docs)
    check(c, q, out, [N], [N], straight(c), "chunk", docs=docs)


@pytest.mark.parametrize("L", [1, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_zeros_next_to_the_largest_values(order, D, L):
    """A block of zeros has the smallest scale, 2^-63; next to values of 2^70 its keys still take their share of the weights."""
    H, G, BT = 2, 4, 256
    N = 40 * BT if L == 1 else 2 * BT
    c = base.filled_cache(N // BT, H, BT, D, E4M3, 260)
    half = N // BT // 2
    zero, large = (slice(0, half), slice(half, None))[order[0]], (slice(0, half), slice(half, None))[order[1]]
    c.v_codes[0, zero], c.v_scales[0, zero] = 0, 127 - 63
    c.v_scales[0, large] = 127 + 62
    one = torch.where(torch.rand(D, generator=gen(261), device=DEV) < 0.5, -1.0, 1.0)
    c.k_codes[0] = (one * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_codes[0, large] = (one * 96).to(torch.float8_e4m3fn).view(torch.uint8)
    c.k_scales.fill_(127 - 6)
    q = (one * (4 / math.sqrt(D)) * torch.ones(1, H * G, L, 1, device=DEV)).to(BF16)   # scores of 4 and 6
    table = straight(c)
    assert kernel_of(c, 1, H * G, L, N) == ("chunk" if L == 300 else "few")
    out = call(c, q, [N], table)
    check(c, q, out, [N], [L], table, kernel_of(c, 1, H * G, L, N))


# ------------------------------------------------------------------ caps of any size

@pytest.mark.parametrize("cap", [1e-42, 1e-3, 0.3, 3.0, 50.0, 256.0, 1e4, 1e6, 1e8, 1e20, 3e38])
@pytest.mark.parametrize("D,L", [(64, 1), (128, 7), (256, 2), (64, 300), (128, 300), (256, 300)])
def test_caps(D, L, cap):
    """cap tanh(score / cap) to a relative error, whatever the cap."""
    H, G, N, BT = 2, 4, 500, 64
    c = base.filled_cache(8, H, BT, D, E4M3, 270)
    q = (torch.randn(1, H * G, L, D, generator=gen(271), device=DEV) * 3).to(F16)
    table = straight(c)
    kernel = kernel_of(c, 1, H * G, L, 512)
    assert kernel == ("chunk" if L == 300 else "few")
    out = call(c, q, [N], table, max_seq=512, softcap=cap)
    check(c, q, out, [N], [L], table, kernel, cap=float(torch.tensor(cap, dtype=torch.float32)))


# ------------------------------------------------------------------ scores and queries at their ends

@pytest.mark.parametrize("L", [1, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_any_size(D, L):
    """The first row of a sequence sees one key: its output is that key's value, however low the score."""
    H, G, BT = 2, 4, 256
    N = L if L > 1 else 1
    c = base.filled_cache(2, H, BT, D, E4M3, 280)
    c.k_codes[0] = torch.where(torch.arange(BT, device=DEV) % 3 == 1, 0x3B, 0x3D).to(torch.uint8)[:, None]   # 1.375 or 1.625
    c.k_scales.fill_(127)
    q = 1 + torch.rand(1, H * G, L, D, generator=gen(281), device=DEV).to(BF16)
    table = straight(c)
    v = (ref.values(c.v_codes[0, 0, :, 0], E4M3) * torch.exp2(c.v_scales[0, 0].double() - 127)[:, None]).repeat_interleave(G, 0)
    for scale in (1e5, -1e5, 1e7, -1e7, 1e20, -1e20, 1e34, -1e34):
        out = call(c, q, [N], table, max_seq=512, scale=scale)
        assert out.isfinite().all()
        assert ((out[0, :, 0].double() - v).abs() <= v.abs() * 2.0 ** -8 + 2.0 ** -20).all(), scale   # 2^-9 by weight and sum, half a step


@pytest.mark.parametrize("L", [1, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_values_under_large_scores(D, L):
    """Every second block's values are of the smallest scales; all keys have one score. And the newest block alone, under
    scores of any size.

    The exponent of a weight is one fp32 number, score x log2(e) + the value scale's exponent. At the larger of the first
    scores, 1e4 (2^13.8 in log2 units), it is rounded by up to 2^-11, next to half a step of bf16 (2^-9) and the weights'
    2^-11; from 2^24 on by more than 1, so that the scales of different blocks are not told apart: no case for that."""
    H, G, BT, N = 2, 4, 16, 512
    c = base.filled_cache(32, H, BT, D, E4M3, 284)
    c.k_codes[0], c.k_scales[0] = 0x38, 127
    c.v_scales[0, ::2] = 127 - 50
    q = torch.ones(1, H * G, L, D, device=DEV).to(BF16)
    table = straight(c)
    docs = torch.arange(N - L, N, dtype=torch.int32, device=DEV).view(1, L)
    for scale in (0.01, 1e4 / D, 1e6, 1e20):
        if scale < 1e3:
            out = call(c, q, [N], table, scale=scale)
            if scale == 0.01:
                check(c, q, out, [N], [L], table, kernel_of(c, 1, H * G, L, N), scale=scale)
                want = out.double()
            assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -7 + 2.0 ** -12).all(), scale
        # the newest block alone, of small values
        out = call(c, q, [N - BT], table, max_seq=N, scale=scale, doc_starts=docs - BT)
        v = (ref.values(c.v_codes[0, 30].transpose(0, 1), E4M3) * 2.0 ** -50)[-min(L, BT):].repeat_interleave(G, 1)   # [n, heads, D]
        assert ((out[0, :, L - len(v):].double() - v.transpose(0, 1)).abs() <= v.transpose(0, 1).abs() * 2.0 ** -8 + 2.0 ** -134).all(), scale


@pytest.mark.parametrize("L", [1, 300])
def test_biases_of_any_size(L):
    """Rows that see the sequence's first two keys only, so far away that the bias is beyond 2^24."""
    D, H, G, BT, N = 128, 2, 4, 256, 512
    c = base.filled_cache(2, H, BT, D, E4M3, 283)
    c.k_codes[0] = 0x38
    q = torch.ones(1, H * G, L, D, device=DEV).to(BF16)
    v = (ref.values(c.v_codes[0, 0, :, :2], E4M3) * torch.exp2(c.v_scales[0, 0].double() - 127)[:, None, None]).repeat_interleave(G, 0)
    for slope, want in ((0.0, v.mean(1)), (3e7, v[:, 1]), (1e12, v[:, 1])):   # the nearer key
        slopes = torch.full((H * G,), slope, device=DEV)
        docs = torch.full((1, L), N, dtype=torch.int32, device=DEV)
        out = call(c, q, [N], straight(c), slopes=slopes, doc_starts=docs, prefix_lens=i32([2]))
        w = want[:, None].expand(-1, L, -1)
        assert ((out[0].double() - w).abs() <= w.abs() * 2.0 ** -8 + v.abs().amax() * 2.0 ** -11).all(), slope


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("L,row", [(2, 1), (300, 17), (300, 299)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_that_are_no_numbers(D, L, row, bad):
    """A NaN in a query makes its own row NaN, as the formula has it, and no other."""
    H, G, N, BT = 2, 4, 500, 64
    c = base.filled_cache(8, H, BT, D, E4M3, 290)
    c.k_codes[..., 5] = 0x38          # infinite scores of one sign but for one key's
    c.k_codes[0, 0, :, 0, 5] = 0xB8
    q = torch.randn(1, H * G, L, D, generator=gen(291), device=DEV).to(BF16)
    table = straight(c)
    kernel = kernel_of(c, 1, H * G, L, 512)
    assert kernel == ("chunk" if L == 300 else "few")
    fine = call(c, q, [N], table, max_seq=512)
    odd = q.clone()
    odd[0, 2, row, 5] = bad
    out = call(c, odd, [N], table, max_seq=512)
    assert out[0, 2, row].isnan().all()
    out[0, 2, row] = fine[0, 2, row]
    check(c, q, out, [N], [L], table, kernel)


# ------------------------------------------------------------------ appends of every block size

@pytest.mark.parametrize("D,BT,n", [(64, 256, 150), (64, 256, 152), (64, 256, 153), (64, 256, 154), (128, 128, 84), (128, 128, 85), (128, 256, 86),
                                    (256, 64, 44), (256, 64, 45), (256, 128, 46)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_appends_whose_angles_fill_48_kb(D, BT, n, dtype):
    c = base.dirty_cache(2, 1, BT, D, E4M3, 300)
    k, v = (torch.randn(1, 1, n, D, generator=gen(s), device=DEV).to(dtype) for s in (301, 302))
    rope = tq.Rope.of_base(D)
    before = base.tensors(c)
    c.append(0, k, v, i32([0]), straight(c), 2, rope=rope)
    base.check_append(c, before, k, v, [0], [n], straight(c), rope)


# ------------------------------------------------------------------ another stream than the current one

@pytest.mark.parametrize("raw", [False, True])
def test_outputs_and_workspaces_belong_to_the_calls_stream(raw):
    """The output (zeroed behind q_lens) and the workspace are made on the stream that the call names."""
    c = base.filled_cache(64, 2, 64, 128, E4M3, 310)
    table = straight(c)
    q = torch.randn(1, 8, 3, 128, generator=gen(311), device=DEV).to(BF16)
    n, nq = i32([4000]), i32([2])
    want = c.attention(0, q, n, table, 64, 4096, q_lens=nq)
    side = torch.cuda.Stream()
    for _ in range(2):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)   # about 10 ms of the current stream
        out = c.attention(0, q, n, table, 64, 4096, q_lens=nq, stream=side.cuda_stream if raw else side)
        side.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del out


# ------------------------------------------------------------------ outputs between the queries

@pytest.mark.parametrize("L", [1, 3, 300])
def test_outputs_in_the_queries_tensor(L):
    """Next to the queries, in a slot of its own of one tensor: every layout whose rows are apart."""
    B, H, G, D, BT, N = 2, 2, 4, 64, 64, 400
    c = base.filled_cache(16, H, BT, D, E4M3, 320)
    table = straight(c, B)
    both = torch.randn(B, L, 2, H * G, D, generator=gen(321), device=DEV).to(BF16)
    q, out = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    want = call(c, q.clone(), [N, N], table, max_seq=512)
    before = both.clone()
    assert call(c, q, [N, N], table, max_seq=512, out=out) is out
    assert torch.equal(out, want) and torch.equal(both[:, :, 0], before[:, :, 0])
    # one after the other, and heads of the two in turn
    flat = torch.empty(2, B, H * G, L, D, device=DEV, dtype=BF16)
    turn = torch.empty(B, H * G, 2, L, D, device=DEV, dtype=BF16)
    for q1, out1 in ((flat[0], flat[1]), (flat[1], flat[0]), (turn[:, :, 0], turn[:, :, 1]), (turn[:, :, 1], turn[:, :, 0])):
        q1.copy_(before[:, :, 0].transpose(1, 2))
        assert torch.equal(call(c, q1, [N, N], table, max_seq=512, out=out1), want)
    with pytest.raises(tq.TQError):
        call(c, q[:, :4], [N, N], table, max_seq=512, out=q[:, 1:5])


@pytest.mark.parametrize("L", [3, 300])
def test_rows_behind_the_queries_may_lie_over_others(L):
    """Sequences packed one after another, each shorter than q_len: rows behind q_lens lie over the next sequence's."""
    H, G, D, BT, N = 2, 4, 64, 64, 400
    c = base.filled_cache(24, H, BT, D, E4M3, 330)
    table = straight(c, 3)
    n = L // 2 + 1
    packed = torch.randn(2 * n + L, H * G, D, generator=gen(331), device=DEV).to(BF16)
    result = torch.zeros_like(packed)
    q, out = (t.as_strided((3, H * G, L, D), (n * H * G * D, D, H * G * D, 1)) for t in (packed, result))
    want = torch.cat([call(c, q[b:b + 1, :, :n].contiguous(), [N], table[b:b + 1], max_seq=512)[0].transpose(0, 1) for b in range(3)])
    call(c, q, [N] * 3, table, max_seq=512, q_lens=[n] * 3, out=out)
    assert ((result[:3 * n].double() - want.double()).abs() <= want.double().abs() * 2.0 ** -7 + 2.0 ** -9).all()   # (another choice of kernel: two roundings, and the weights')
    assert (result[3 * n:] == 0).all()


class RawStream:
    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("kind", ["torch", "object", "number", "default"])
def test_streams_of_every_kind(kind):
    c = base.filled_cache(64, 2, 64, 128, E4M3, 340)
    q = torch.randn(1, 8, 3, 128, generator=gen(341), device=DEV).to(BF16)
    n = i32([4000])
    want = c.attention(0, q, n, straight(c), 64, 4096)
    torch.cuda.synchronize()
    s = torch.cuda.default_stream() if kind == "default" else torch.cuda.Stream()
    given = {"torch": s, "object": RawStream(s), "number": s.cuda_stream, "default": 0}[kind]
    out = c.attention(0, q, n, straight(c), 64, 4096, stream=given)
    s.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ the chunk kernel in graphs and on several streams

def test_chunks_captured_replayed_and_at_once():
    """Chunks with and without wide tiles: the same bits from two streams at once, and from a graph with other inputs."""
    H, G, L, N, BT, D = 2, 4, 300, 600, 32, 128
    caches = [base.filled_cache(19, H, BT, D, E4M3, 350 + i) for i in range(2)]
    caches[1].k_scales[0, ::2] -= 30
    caches[1].v_scales[0, 1::2] -= 30
    table = straight(caches[0])
    lens = i32([N])
    qs = [torch.randn(1, H * G, L, D, generator=gen(352 + i), device=DEV).to(BF16) for i in range(2)]
    assert kernel_of(caches[0], 1, H * G, L, 600) == "chunk"
    want = [c.attention(0, q, lens, table, 19, 600) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in qs], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(caches[i].attention(0, qs[i], lens, table, 19, 600))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)
    outs = [torch.empty_like(q) for q in qs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, q, o in zip(caches, qs, outs):
            c.attention(0, q, lens, table, 19, 600, out=o)
    for n in (600, 431):
        lens.fill_(n)
        for q in qs:
            q.copy_(torch.randn(q.shape, generator=gen(360 + n), device=DEV).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        for c, q, o in zip(caches, qs, outs):
            assert torch.equal(o, c.attention(0, q, lens, table, 19, 600))
            check(c, q, o, [n], [L], table, "chunk")
