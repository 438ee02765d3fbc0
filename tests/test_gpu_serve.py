"""The calls around the caches' on the GPU: position rotation, block tables and slot maps, verification of drafts, and a run
of them together, against their definitions."""
import math
import random

import pytest
import torch

import serve_util as ref
import turboquant_compressed_kv_tq_gb300 as tq
from turboquant_compressed_kv_tq_gb300 import speculative

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"
WORDS = {"capacity": tq.TQ_DEVERR_CAPACITY, "block": tq.TQ_DEVERR_BLOCK, "seqlen": tq.TQ_DEVERR_SEQLEN}


@pytest.fixture(autouse=True)
def no_device_error():
    tq.tq_device_error()
    yield
    torch.cuda.synchronize()
    assert tq.tq_device_error() == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ rotation

def laid_out(B, heads, n, D, order, dtype, seed, gap=0):
    """Random rows [B, heads, n, D] in memory in `order` of their axes, `gap` elements between rows."""
    dims = {"b": B, "h": heads, "t": n}
    x = torch.randn([dims[a] for a in order] + [D + gap], generator=gen(seed), device=DEV).to(dtype)[..., :D]
    return x.permute(*[order.index(a) for a in "bht"], 3)


def check_rotation(x, out, pos, r, freq, back=False, news=None, before=None):
    inter, scale = bool(r.desc.interleaved), float(r.desc.scale)
    want = ref.rotated(x.double(), pos, freq, inter, scale, back)
    bound = ref.rotation_bound(x.double(), want, pos, freq, x.dtype, inter, scale)
    bad = (out.double() - want).abs() > bound
    n = x.shape[2]
    if news is not None:
        behind = (torch.arange(n, device=DEV) >= news[:, None])[:, None, :, None].expand_as(out)
        assert torch.equal(out[behind], before[behind])
        bad &= ~behind
    assert not bool(bad.any()), (out.double() - want).abs().max()
    rot = 2 * freq.numel()
    if rot < x.shape[3] and news is None:
        raw = torch.int32 if x.dtype == F32 else torch.int16
        assert torch.equal(out.contiguous().view(raw)[..., rot:], x.contiguous().view(raw)[..., rot:])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (128, 64, True), (64, 64, True), (64, 16, False), (256, 256, False), (80, 32, False), (16, 16, True),
                                         (1024, 1024, False), (208, 48, True)])
@pytest.mark.parametrize("B,n,Hq,Hk", [(1, 1, 8, 2), (3, 7, 5, 1), (2, 130, 3, 3)])
def test_rotation(dtype, D, rot, inter, B, n, Hq, Hk):
    r = tq.Rope.of_base(rot, interleaved=inter, scale=1.25)
    starts = i32([17 + 100003 * b for b in range(B)])
    q, k = laid_out(B, Hq, n, D, "bth", dtype, 1), laid_out(B, Hk, n, D, "bht", dtype, 2)
    out, k_out = r.apply(q, k, starts=starts)
    assert out.is_contiguous() and k_out.is_contiguous()
    pos = starts[:, None] + torch.arange(n, device=DEV)
    for x, y in ((q, out), (k, k_out)):
        check_rotation(x, y, pos, r, r.inv_freq)
    out, none = r.apply(k, starts=starts, transposed=True)
    assert none is None
    check_rotation(k, out, pos, r, r.inv_freq, back=True)


@pytest.mark.parametrize("order_in", ["bth", "htb", "tbh"])
@pytest.mark.parametrize("order_out", ["bht", "bth", "thb"])
def test_rotation_layouts(order_in, order_out):
    B, H, n, D = 3, 6, 37, 128
    r = tq.Rope.of_base(D)
    q, k = laid_out(B, H, n, D, order_in, BF16, 3, gap=8), laid_out(B, 2, n, D, order_in, BF16, 4, gap=24)
    out, k_out = laid_out(B, H, n, D, order_out, BF16, 5, gap=16), laid_out(B, 2, n, D, order_out, BF16, 6)
    pos = torch.randint(-5, 1 << 30, (B, n), generator=gen(7), device=DEV, dtype=torch.int32)
    r.apply(q, k, out, k_out, positions=pos)
    check_rotation(q, out, pos, r, r.inv_freq)
    check_rotation(k, k_out, pos, r, r.inv_freq)


@pytest.mark.parametrize("first", ["q", "k"])
@pytest.mark.parametrize("dtype,D,rot", [(BF16, 128, 64), (F32, 64, 64)])
def test_rotation_in_place_in_a_projection(first, dtype, D, rot):
    B, n, Hq, Hk = 2, 19, 8, 2
    whole = laid_out(B, Hq + 2 * Hk, n, D, "bth", dtype, 8)
    before = whole.clone()
    q0, k0 = (0, Hq) if first == "q" else (Hk, 0)
    q, k = whole[:, q0:q0 + Hq], whole[:, k0:k0 + Hk]
    r = tq.Rope.of_base(rot)
    news = i32([n, 4])
    r.apply(q, k, q, k, new_lens=news)
    pos = torch.arange(n, device=DEV).expand(B, n)
    for at, h, x in ((q0, Hq, q), (k0, Hk, k)):
        check_rotation(before[:, at:at + h], x, pos, r, r.inv_freq, news=news, before=before[:, at:at + h])
    others = [h for h in range(Hq + 2 * Hk) if not (q0 <= h < q0 + Hq or k0 <= h < k0 + Hk)]
    assert torch.equal(whole[:, others], before[:, others])


def test_rotation_of_rows_behind_lengths_and_broadcast_inputs():
    B, H, n, D = 4, 3, 9, 64
    r = tq.Rope.of_base(32, scale=0.5)
    q = laid_out(1, H, n, D, "bht", F16, 9).expand(B, H, n, D)
    out = laid_out(B, H, n, D, "bht", F16, 10)
    before = out.clone()
    news = i32([9, 0, 1, 5])
    starts = i32([0, 5, 1 << 20, 3])
    r.apply(q, out=out, new_lens=news, starts=starts)
    check_rotation(q, out, starts[:, None] + torch.arange(n, device=DEV), r, r.inv_freq, news=news, before=before)
    assert not r.apply(q, new_lens=news)[0][1].any()
    r.apply(q, out=out, new_lens=i32([9, -1, 10, 2]))
    torch.cuda.synchronize()
    assert tq.tq_device_error() == tq.TQ_DEVERR_SEQLEN
    assert torch.equal(out[1], before[1])
    check_rotation(q[2:3], out[2:3], torch.arange(n, device=DEV)[None], r, r.inv_freq)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rotation_of_what_is_no_number(dtype):
    # a pair's own; what passes, passes bit for bit
    B, H, n, D, rot = 1, 2, 3, 128, 64
    q = laid_out(B, H, n, D, "bht", dtype, 11).clone()
    q[0, 0, 1, 5] = math.nan
    q[0, 1, 2, 40] = math.inf
    raw = torch.int32 if dtype == F32 else torch.int16
    q.view(raw)[0, 1, 0, 100] = 0x7FC01234 if dtype == F32 else 0x7FD5   # a NaN with something in it
    r = tq.Rope.of_base(rot)
    out, _ = r.apply(q)
    assert torch.equal(out.view(raw)[..., rot:], q.view(raw)[..., rot:])
    odd = torch.zeros_like(q, dtype=torch.bool)
    odd[0, 0, 1, [5, 37]] = True
    odd[0, 1, 2, [8, 40]] = True
    assert bool((~out.isfinite()[..., :rot] == odd[..., :rot]).all())
    pos = torch.arange(n, device=DEV)[None]
    clean = torch.where(odd, 0.0, q)
    check_rotation(clean, torch.where(odd, r.apply(clean)[0], out), pos, r, r.inv_freq)


def test_rotation_gradient():
    B, H, n, D, rot = 2, 3, 5, 64, 48
    r = tq.Rope.of_base(rot, interleaved=True, scale=1.5)
    pos = torch.randint(0, 5000, (B, n), generator=gen(12), device=DEV, dtype=torch.int32)
    x, g = laid_out(B, H, n, D, "bht", F32, 13), laid_out(B, H, n, D, "bht", F32, 14)
    y, _ = r.apply(x, positions=pos)
    dx, _ = r.apply(g, positions=pos, transposed=True)
    # the formula's, by autograd in 64 bits
    leaf = x.double().requires_grad_()
    ref.rotated(leaf, pos, r.inv_freq, True, 1.5).backward(g.double())
    bound = ref.rotation_bound(g.double(), leaf.grad, pos, r.inv_freq, F32, True, 1.5)
    assert bool(((dx.double() - leaf.grad).abs() <= bound).all())
    # differences: the map is linear, so a step of any size gives them; x and the two sums of n numbers are off by 2^-21 of their terms
    step = laid_out(B, H, n, D, "bht", F32, 15)
    moved, _ = r.apply(x + step, positions=pos)
    by_steps = (g.double() * (moved.double() - y.double())).sum()
    by_gradient = (dx.double() * step.double()).sum()
    terms = 1.5 * (g.abs().double() * (x.abs() + step.abs()).double()).sum() * 4 + 1.5 * (g.abs().double() * step.abs().double()).sum() * 4
    assert abs(float(by_steps - by_gradient)) <= float(terms) * 2.0 ** -20
    back, _ = tq.Rope.of_base(rot, interleaved=True).apply(tq.Rope.of_base(rot, interleaved=True).apply(x, positions=pos)[0], positions=pos, transposed=True)
    assert float((back - x).abs().max()) < 2.0 ** -19 * float(x.abs().max())


def test_rotation_scaled_frequencies():
    rot, factor, base, original = 64, 8.0, 500000.0, 4096
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    assert torch.allclose(tq.Rope.linear(rot, factor, base).inv_freq.cpu(), f / factor, rtol=1e-14, atol=0)
    ntk = tq.Rope.ntk(rot, factor, base).inv_freq.cpu()
    assert torch.allclose(ntk, (base * factor ** (rot / (rot - 2))) ** (-i / rot), rtol=1e-13, atol=0)
    assert abs(float(ntk[-1] * factor / f[-1]) - 1) < 1e-12 and float(ntk[0]) == 1.0
    parts = tq.Rope.by_parts(rot, factor, original, low=1.0, high=4.0, base=base).inv_freq.cpu()
    for got, x in zip(parts.tolist(), f.tolist()):
        turns = original * x / (2 * math.pi)
        want = x if turns > 4 else x / factor if turns < 1 else ((turns - 1) / 3) * x + (1 - (turns - 1) / 3) * x / factor
        assert abs(got / want - 1) < 1e-12
    with pytest.raises(ValueError):
        tq.Rope.by_parts(rot, factor, original, low=4.0, high=4.0)
    with pytest.raises(ValueError):
        tq.Rope.ntk(2, factor)


def test_rotation_captured_on_another_stream():
    B, H, n, D = 2, 4, 3, 128
    r = tq.Rope.of_base(D)
    q, out = laid_out(B, H, n, D, "bht", BF16, 16), torch.zeros(B, H, n, D, dtype=BF16, device=DEV)
    pos = torch.zeros(B, n, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.apply(q, out=out, positions=pos)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r.apply(q, out=out, positions=pos)
    for seed in (17, 18):
        pos.copy_(torch.randint(0, 1 << 20, pos.shape, generator=gen(seed), device=DEV))
        q.copy_(laid_out(B, H, n, D, "bht", BF16, seed))
        graph.replay()
        check_rotation(q, out, pos, r, r.inv_freq)
    other = torch.cuda.Stream()
    made, _ = r.apply(q, positions=pos, stream=other)   # the current stream waits for it
    torch.cuda.current_stream().wait_stream(other)
    check_rotation(q, made, pos, r, r.inv_freq)


def test_rotation_of_far_rows():
    # rows more than 2^31 elements apart
    B, H, n, D = 2, 2, 3, 64
    r = tq.Rope.of_base(D)
    hold = torch.zeros((1 << 31) + 4096, dtype=BF16, device=DEV)
    q = torch.as_strided(hold, (B, H, n, D), (1 << 31, 64 * n, 64, 1))
    x = laid_out(B, H, n, D, "bht", BF16, 19)
    q.copy_(x)
    out, _ = r.apply(q)
    check_rotation(x, out, torch.arange(n, device=DEV).expand(B, n), r, r.inv_freq)
    r.apply(q, out=q)
    assert torch.equal(q, out)


def test_rotation_refusals():
    r = tq.Rope.of_base(64)
    q = laid_out(1, 2, 3, 64, "bht", BF16, 20)
    for kw in (dict(out=q[:, :1]), dict(out=q.float()), dict(starts=torch.zeros(1, dtype=torch.int64, device=DEV)), dict(starts=i32([0, 0])),
               dict(positions=i32([[0, 1]])), dict(new_lens=torch.zeros(1, dtype=torch.int32)), dict(k_out=q)):
        with pytest.raises(ValueError):
            r.apply(q, **kw)
    with pytest.raises(TypeError):
        r.apply(q.double())
    with pytest.raises(ValueError):
        r.apply(q.cpu())
    with pytest.raises(ValueError):
        r.apply(q.transpose(2, 3))
    whole = torch.zeros(1, 2, 4, 64, dtype=BF16, device=DEV)
    for kw in (dict(out=whole[:, :, 1:]), dict(k=whole[:, :, :3], out=whole[:, :, 1:].clone(), k_out=whole[:, :, 1:]),
               dict(out=torch.zeros(3, dtype=BF16, device=DEV).new_zeros(1, 2, 1, 64).expand(1, 2, 3, 64))):
        with pytest.raises(tq.TQError):
            r.apply(whole[:, :, :3], **kw)
    with pytest.raises(tq.TQError):
        r.apply(torch.zeros(1, 2, 3, 32, dtype=BF16, device=DEV))   # fewer coordinates than are to turn
    with pytest.raises(tq.TQError):
        r.apply(torch.zeros(1, 2, 3, 72, dtype=BF16, device=DEV)[..., 4:68])


# ------------------------------------------------------------------ block tables

def blocks_case(seed, B, width, BT, n_new, most_len, spare, ragged=True, missing=False):
    """A table whose rows hold their lengths' blocks, and a shuffled free list of the others (spare < 0: too few)."""
    rnd = random.Random(seed)
    lens = [rnd.randint(0, most_len) for _ in range(B)]
    news = [rnd.randint(0, n_new) for _ in range(B)] if ragged else None
    held = [-(-N // BT) for N in lens]
    extra = sum(-(-(N + (n_new if news is None else news[b])) // BT) - held[b] for b, N in enumerate(lens))
    n_free = max(0, extra + spare)
    total = sum(held) + n_free
    ids = list(range(total))
    rnd.shuffle(ids)
    table = []
    for h in held:
        table.append([ids.pop() for _ in range(h)] + [-1] * (width - h))
    if missing and B > 1:   # a block that was taken away
        b = max(range(B), key=lambda b: held[b])
        if held[b]:
            ids.append(table[b][held[b] - 1])
            table[b][held[b] - 1] = -1
    return table, ids, lens, news, max(1, total)


def on_device(table, free, used, BT, num_blocks, width):
    return tq.BlockTable.wrap(torch.tensor(table, dtype=torch.int32, device=DEV).view(len(table), width), i32(free), i32([used]), BT, num_blocks)


def errors(words):
    torch.cuda.synchronize()
    want = 0
    for w in words:
        want |= WORDS[w]
    assert tq.tq_device_error() == want, (words, want)


def check_reserve(bt, table, free, used, lens, news, n_new, BT, num_blocks, max_tokens):
    places = tq.Places(len(lens), max_tokens)
    for t in (places.granted, places.starts, places.seq_ids, places.positions, places.slots):
        t.fill_(-7)
    bt.reserve(i32(lens), None if news is None else i32(news), n_new, places)
    used, granted, starts, seqs, pos, slots, err = ref.reserve(table, free, used, lens, news, n_new, BT, num_blocks, max_tokens)
    errors(err)
    assert places.granted.tolist() == granted and places.starts.tolist() == starts
    assert bt.table.tolist() == table and bt.free_blocks.tolist() == free
    assert bt.n_used.tolist() == [used]
    assert places.seq_ids.tolist() == seqs and places.positions.tolist() == pos and places.slots.tolist() == slots
    return used


def check_release(bt, table, free, used, keeps, BT, num_blocks):
    bt.release(i32(keeps))
    used, err = ref.release(table, free, used, keeps, BT, num_blocks)
    errors(err)
    assert bt.table.tolist() == table and bt.free_blocks.tolist() == free and bt.n_used.tolist() == [used]
    return used


@pytest.mark.parametrize("B,width,BT,n_new,most_len,spare", [
    (1, 1, 16, 1, 0, 0), (1, 4, 16, 1, 63, 5), (7, 9, 16, 5, 100, 0), (33, 20, 32, 100, 500, 3), (300, 8, 64, 9, 400, 11), (1025, 3, 16, 7, 30, 0),
    (2500, 6, 16, 40, 30, 100), (3, 700, 16, 11000, 50, 9), (64, 130, 16, 2000, 17, -40), (7, 9, 16, 5, 100, -2), (1500, 4, 32, 30, 90, -300), (5, 3, 256, 600, 100, 0),
    (40, 10, 16, 0, 100, 4), (4097, 3, 16, 7, 30, 0), (9001, 3, 16, 2, 30, 50), (20000, 8, 16, 100, 20, -5000), (33, 70, 16, 1000, 90, 20), (9, 4, 16, 900, 60, -3), (20, 40, 16, 130, 500, -4)])
@pytest.mark.parametrize("ragged", [True, False])
def test_blocks_reserve_and_release(B, width, BT, n_new, most_len, spare, ragged):
    table, free, lens, news, total = blocks_case(B * 31 + width, B, width, BT, n_new, min(most_len, width * BT), spare, ragged, missing=spare > 5)
    bt = on_device(table, free, 0, BT, total, width)
    asked = sum(n_new if news is None else news[b] for b in range(B))
    for max_tokens in (asked + 13, asked, max(0, asked - 3)):   # the second and third time there is nothing left to take
        used = check_reserve(bt, table, free, bt.n_used.item(), lens, news, n_new, BT, total, max_tokens)
    rnd = random.Random(5)
    keeps = [min(N + rnd.randint(0, n_new), width * BT) for N in lens]
    used = check_release(bt, table, free, used, keeps, BT, total)
    used = check_release(bt, table, free, used, keeps, BT, total)            # nothing more
    used = check_reserve(bt, table, free, used, lens, news, n_new, BT, total, asked)
    used = check_release(bt, table, free, used, lens, BT, total)
    held = sum(x >= 0 for row in table for x in row)
    assert held + len(free) - used <= total


def test_blocks_that_cannot_be():
    BT, width = 16, 4
    table = [[0, 1, -1, -1], [2, 99, -1, -1], [-1] * 4, [3, -1, -1, -1], [4, 5, 6, 7], [8, -1, -1, -1]]
    free = [9, 50, 10, 11, 12, 13]
    lens, news = [32, 30, -1, 65, 60, 16], [1, 5, 3, 2, 9, 40]
    bt = on_device(table, free, 0, BT, 16, width)
    used = check_reserve(bt, table, free, 0, lens, news, 20, BT, 16, 64)
    assert tq.tq_device_error() == 0
    used = check_release(bt, table, free, used, [-3, 10, 0, 1 << 30, 48, 0], BT, 16)
    check_release(bt, table, free, used, [0] * 6, BT, 16)     # more than were taken
    for bad in (-1, 7):
        bt = on_device([[-1, -1]], [0, 1, 2], bad, BT, 4, 2)
        check_reserve(bt, [[-1, -1]], [0, 1, 2], bad, [0], None, 3, BT, 4, 3)
        bt = on_device([[0, -1]], [3, 1, 2], bad, BT, 4, 2)
        check_release(bt, [[0, -1]], [3, 1, 2], bad, [0], BT, 4)


def test_blocks_of_no_sequences_or_maps():
    bt = tq.BlockTable(4, 3, 12, 16)
    places = tq.Places(0, 5)
    places.starts.fill_(9)
    places.slots.fill_(9)
    bt.reserve(i32([]), None, 4, places)
    assert places.starts.tolist() == [0] and places.slots.tolist() == [-1] * 5
    bt.release(i32([]))
    bt.reserve(i32([0, 20]), None, 2)          # no places asked for
    assert bt.table.tolist() == [[0, -1, -1], [-1, 1, -1], [-1] * 3, [-1] * 3] and bt.n_used.tolist() == [2]
    empty = tq.BlockTable.wrap(bt.table, i32([]), i32([0]), 16, 12)
    empty.reserve(i32([0]), None, 2)           # an empty list, and nothing needed
    errors([])
    empty.reserve(i32([14]), None, 9)
    errors(["capacity"])
    for call in (lambda: bt.reserve(torch.zeros(5, dtype=torch.int32, device=DEV)), lambda: bt.reserve(i32([0, 0]), places=tq.Places(3)),
                 lambda: bt.reserve(i32([0]), new_lens=i32([0, 0])), lambda: bt.release(torch.zeros(2, device=DEV)),
                 lambda: tq.BlockTable.wrap(bt.table.long(), bt.free_blocks, bt.n_used, 16, 12),
                 lambda: tq.BlockTable.wrap(bt.table, bt.free_blocks, i32([0, 0]), 16, 12)):
        with pytest.raises(ValueError):
            call()


def test_blocks_of_far_rows():
    # entries more than 2^31 behind the table's start, positions near 2^31, slots beyond it
    width, BT, rows = (1 << 27) - 1, 16, 17
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    near_end = width * BT - 5
    table[rows - 1, near_end // BT - 1] = 3
    bt = tq.BlockTable.wrap(table, i32([(1 << 30) + 7, 9, 11]), i32([0]), BT, (1 << 30) + 9)
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    lens[rows - 1] = near_end - near_end % BT - 2
    news = torch.zeros(rows, dtype=torch.int32, device=DEV)
    news[rows - 1] = 20
    places = tq.Places(rows, 21)
    bt.reserve(lens, news, 20, places)
    assert places.granted.tolist() == [0] * (rows - 1) + [18]          # what the row has left
    at = int(lens[rows - 1])
    id = (1 << 30) + 7
    want = [(3 * BT + p % BT) if p // BT == near_end // BT - 1 else id * BT + p % BT for p in range(at, at + 18)]
    assert places.slots.tolist() == want + [-1] * 3 and places.positions.tolist()[:18] == list(range(at, at + 18))
    assert tq.tq_device_error() == tq.TQ_DEVERR_CAPACITY
    lens[rows - 1] = at - BT + 2
    bt.release(torch.where(torch.arange(rows, device=DEV) == rows - 1, lens, 0).to(torch.int32))
    errors(["capacity"])   # block 3 was not taken from the list
    assert bt.n_used.item() == 0 and bt.free_blocks.tolist() == [id, 9, 11] and int(table.max()) == -1


def test_blocks_captured_and_replayed():
    B, width, BT = 5, 40, 16
    bt = tq.BlockTable(B, width, B * width, BT)
    lens, places = torch.zeros(B, dtype=torch.int32, device=DEV), tq.Places(B, B * 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bt.reserve(lens, None, 7, places)
        bt.release(lens)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bt.reserve(lens, None, 7, places)
        lens += places.granted - torch.arange(B, device=DEV, dtype=torch.int32)   # row b gives b of its tokens back
        bt.release(lens)
    table, free, used, host = bt.table.tolist(), bt.free_blocks.tolist(), 0, [0] * B
    for _ in range(20):
        graph.replay()
        used, granted, _, _, _, slots, err = ref.reserve(table, free, used, host, None, 7, BT, B * width, B * 7)
        assert not err
        host = [h + g - b for b, (h, g) in enumerate(zip(host, granted))]
        used, err = ref.release(table, free, used, host, BT, B * width)
        assert not err
        assert bt.table.tolist() == table and bt.free_blocks.tolist() == free and bt.n_used.item() == used and lens.tolist() == host
        assert places.slots.tolist() == slots


@pytest.mark.parametrize("cut", [0, 1, 2])
def test_blocks_large_maps_captured(cut):
    # maps of a launch of their own, into arrays that begin anywhere; every replay goes on from the last
    B, width, BT, n = 70, 200, 16, 701
    bt = tq.BlockTable(B, width, B * width, BT)
    lens, places = torch.zeros(B, dtype=torch.int32, device=DEV), tq.Places(B, B * n + 8)
    hold = [torch.zeros(B * n + 16, dtype=d, device=DEV) for d in (torch.int32, torch.int32, torch.int64)]
    maps = [h[cut:cut + B * n + 8] for h in hold]
    for name, m in zip(("seq_ids", "positions", "slots"), maps):
        setattr(places, name, m)
        setattr(places.desc, name, m.data_ptr())
    news = i32([(37 * b) % (n + 1) for b in range(B)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bt.reserve(lens, news, n, places)
        bt.release(lens)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bt.reserve(lens, news, n, places)
        lens += places.granted
    table, free, used, host = bt.table.tolist(), bt.free_blocks.tolist(), 0, [0] * B
    for _ in range(4):
        graph.replay()
        used, granted, starts, seqs, pos, slots, err = ref.reserve(table, free, used, host, news.tolist(), n, BT, B * width, B * n + 8)
        assert not err and places.starts.tolist() == starts
        assert [m.tolist() for m in maps] == [seqs, pos, slots]
        host = [h + g for h, g in zip(host, granted)]
    assert all(not h[:cut].any() and not h[cut + B * n + 8:].any() for h in hold)


def test_blocks_share_the_batch_calls_free_list():
    kc, vc = tq.Codec(64, 3, tq.TQ_MODE_PROD, seed=0), tq.Codec(64, 3, tq.TQ_MODE_MSE, seed=1)
    cache, other = (tq.CompressedKVCache(kc, vc, 1, 32, 16, 1) for _ in "ab")
    bt = tq.BlockTable(4, 6, 32, 16)
    lens = i32([40, 5, 0, 0])
    bt.reserve(torch.zeros_like(lens[:2]), lens[:2].clone(), 64)
    src = tq.Batch(other, 1, 6, table=i32([[7, 3, -1, -1, -1, -1]]), lens=i32([20]), batch=1)
    dst = bt.batch(cache, lens, 2)
    tq.tq_batch_extend(dst, src, bt.free_blocks, bt.n_used)
    assert dst.batch == 3 and bt.n_used.item() == 6 and bt.table[2].tolist() == [4, 5, -1, -1, -1, -1] and lens[2].item() == 20
    bt.release(i32([40, 0, 20]))
    assert bt.n_used.item() == 5 and bt.free_blocks[5].item() == 3


# ------------------------------------------------------------------ verification

def verify_case(seed, B, K, V, dtype=BF16, draft=F32, temps="mixed", lens=False, probs=False, spread=3.0):
    g = gen(seed)
    common = spread * torch.randn((B, K + 1, V), generator=g, device=DEV)
    guess = (common + torch.randn((B, K + 1, V), generator=g, device=DEV))[:, :K]
    x = common + torch.randn((B, K + 1, V), generator=g, device=DEV)
    t = None
    if temps == "mixed":
        t = torch.where(torch.rand(B, generator=g, device=DEV) < 0.3, 0.0, 0.3 + 1.5 * torch.rand(B, generator=g, device=DEV))
    target = (torch.softmax(x, -1) if probs else x).to(dtype)
    q = torch.softmax(guess, -1)
    e = torch.empty_like(q).exponential_(generator=g)
    tokens = (q / e).argmax(-1).to(torch.int32) if K else None
    return dict(target=target, draft_tokens=tokens, draft_probs=None if draft is None or not K else q.to(draft),
                uniforms=torch.rand((B, K), generator=g, device=DEV) if K else None,
                noise=torch.empty((B, V), device=DEV).exponential_(generator=g).clamp_(min=2.0 ** -100), temperatures=t,
                draft_lens=torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if lens else None,
                seq_lens=torch.randint(0, 1000, (B,), generator=g, device=DEV, dtype=torch.int32), target_probs=probs)


def check(c):
    got = tq.tq_verify_drafts(**c)
    again = tq.tq_verify_drafts(**c)
    for x, y in zip(got, again):
        assert x is None or torch.equal(x, y)
    ref.check_verified(c["target"], c["draft_tokens"], c["draft_probs"], c["uniforms"], c["noise"], c["temperatures"], c["draft_lens"], c["target_probs"],
                       c["seq_lens"], got)
    return got


@pytest.mark.parametrize("dtype,draft", [(BF16, F32), (F16, F16), (F32, BF16), (F32, None)])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 0, 2), (5, 3, 31), (40, 4, 1000), (3, 8, 4097), (2, 64, 333), (4, 2, 50021), (2, 1, 131072), (1, 2, 200003)])
def test_verification(dtype, draft, B, K, V):
    got = check(verify_case(B + V, B, K, V, dtype, draft, lens=B > 3))
    if B == 40:
        assert 0 < int(got.accepted.sum()) < 40 * K


@pytest.mark.parametrize("B,K,V", [(30, 3, 700), (2, 1, 70001), (1, 0, 513)])
def test_verification_against_probabilities(B, K, V):
    for draft in (F32, F16, None):
        check(verify_case(V, B, K, V, F32, draft, temps=None, probs=True))
    check(verify_case(V, B, K, V, F32, F32, temps="mixed", probs=True))
    c = verify_case(V + 1, B, K, V, BF16, BF16, temps=None, probs=True)
    check(c)


@pytest.mark.parametrize("B,K,V", [(30, 3, 700), (2, 1, 70001), (9, 0, 300)])
def test_verification_greedy(B, K, V):
    c = verify_case(V, B, K, V, F16, F32, temps=None)
    c["noise"] = None
    likeliest = c["target"].float().argmax(-1).to(torch.int32)
    if K:   # half of the drafts right
        c["draft_tokens"] = torch.where(torch.rand((B, K), generator=gen(1), device=DEV) < 0.5, likeliest[:, :K], c["draft_tokens"])
    got = check(c)
    c["uniforms"] = None
    for x, y in zip(got, tq.tq_verify_drafts(**c)):
        assert torch.equal(x, y)
    for b, n in enumerate(got.accepted.tolist()):
        assert got.tokens[b, :n + 1].tolist() == likeliest[b, :n + 1].tolist()


@pytest.mark.parametrize("cut", [1, 2, 3, 5])
@pytest.mark.parametrize("V", [997, 4096, 33000])
def test_verification_of_rows_anywhere(cut, V):
    # rows that begin at any element, of strides of any size
    B, K = 4, 2
    c = verify_case(V + cut, B, K, V, BF16, F16)
    for name in ("target", "draft_probs", "noise"):
        x = c[name]
        hold = torch.full(x.shape[:-1] + (V + cut + 2,), math.nan, dtype=x.dtype, device=DEV)
        hold[..., cut:cut + V] = x
        c[name] = hold[..., cut:cut + V]
    check(c)
    c["noise"] = c["noise"][:1].expand(B, V)
    c["target"] = c["target"][:, :1].expand(B, K + 1, V)
    check(c)


@pytest.mark.parametrize("V", [300, 20000])
def test_verification_of_masked_rows(V):
    B, K = 12, 2
    for low in (-math.inf, torch.finfo(F32).min):
        c = verify_case(V, B, K, V, F32, F32)
        x = c["target"]
        x[:, :, V // 2:] = low                                      # the upper half cannot be
        x[1, 0] = low
        x[1, 0, 7] = 0.0                                            # one token left
        x[2, 1, :] = 5.0                                            # all alike
        got = check(c)
        if low == -math.inf:
            for b in range(B):
                n = int(got.accepted[b])
                assert 0 <= int(got.tokens[b, n]) < (V if (b, n) == (2, 1) else V // 2)
    errors([])
    # rows with nothing in them
    c = verify_case(V, B, K, V, BF16, F32)
    c["target"][:, :] = -math.inf
    got = check(c)
    assert tq.tq_device_error() == 16
    assert not got.accepted.any() and bool((got.tokens == -1).all()) and not got.logprobs.any()
    c = verify_case(V, B, K, V, F32, F32, temps=None, probs=True)
    c["target"][:, :] = 0.0
    got = check(c)
    assert tq.tq_device_error() == 16 and not got.accepted.any() and bool((got.tokens == -1).all())
    c["noise"] = None
    got = check(c)
    assert tq.tq_device_error() == 16 and bool((got.tokens == -1).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("K,V", [(0, 40), (0, 30011), (2, 40), (2, 30011)])
def test_verification_of_rows_of_one_value(dtype, K, V):
    # the lowest number, the largest, zero: each token alike, the lowest of equals where nothing is drawn
    B = 6
    for value in (torch.finfo(dtype).min, torch.finfo(dtype).max, 0.0, -1000.0):
        c = verify_case(V, B, K, V, dtype, F32, temps="mixed")
        c["target"][:] = value
        c["target"][:, :, 3] = -math.inf
        check(c)
        c["noise"] = None
        got = check(c)
        assert all(int(got.tokens[b, int(got.accepted[b])]) == 0 for b in range(B))
        c["target"][:, :, :5] = -math.inf
        assert check(c).tokens[:, 0].tolist() == [5] * B
        c["noise"] = torch.ones((B, V), device=DEV)   # with equal noise the lowest too
        c["temperatures"] = torch.full((B,), 0.7, device=DEV)
        if K == 0:
            assert check(c).tokens[:, 0].tolist() == [5] * B


@pytest.mark.parametrize("B,V", [(1, 1), (3, 31), (700, 1000), (5, 4097), (300, 33000), (40, 131072), (2, 200003), (160, 20000)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_drawing_one_token(dtype, B, V):
    check(verify_case(B + V, B, 0, V, dtype, None))
    c = verify_case(B + V + 1, B, 0, V, dtype, None, temps=None, probs=True)
    check(c)
    check(c | {"noise": None})
    # equals stand apart: the lowest of them, whatever the largest logit was when either came by
    c = verify_case(B + V + 2, B, 0, V, dtype, None, temps=None)
    if V > 30:
        lo, hi = V // 5, V - 2
        for at in (lo, hi):
            c["target"][:, 0, at] = 12.25
            c["noise"][:, at] = 2.0 ** -20
        assert check(c).tokens[:, 0].tolist() == [lo] * B


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V", [50, 9001])
def test_verification_of_what_is_no_number(dtype, V):
    B = 10
    for K, odd in ((2, math.nan), (2, math.inf), (0, math.nan), (0, math.inf)):
        c = verify_case(V + 3, B, K, V, dtype, F32)
        c["target"][::2, 0, 11] = odd
        c["target"][::2, 0, V - 1] = odd
        c["noise"][:, 12] = 0.0
        c["noise"][3, 13] = math.nan
        check(c)
        assert tq.tq_device_error() == 16
        c["noise"] = None
        check(c)
        assert tq.tq_device_error() == 16
    c = verify_case(V + 4, B, 2, V, dtype, F32)
    c["draft_probs"][0, 0, int(c["draft_tokens"][0, 0])] = math.nan   # not kept
    c["uniforms"][1, 0] = math.nan
    c["temperatures"][0:2] = 1.0
    got = tq.tq_verify_drafts(**c)
    assert got.accepted[:2].tolist() == [0, 0]


def test_verification_ties_go_to_the_lowest():
    B, V = 6, 40001
    x = torch.zeros((B, 2, V), device=DEV)
    tops = [(5, 40000), (1023, 1024), (0, 1), (31, 32), (20000, 20001), (8191, 39999)]
    for b, (i, j) in enumerate(tops):
        x[b, :, i] = x[b, :, j] = 9.0
    drafts = i32([[i] for i, _ in tops])
    got = tq.tq_verify_drafts(x, drafts)
    assert got.accepted.tolist() == [1] * B and got.tokens[:, 1].tolist() == [i for i, _ in tops]
    drafts = i32([[j] for _, j in tops])
    got = tq.tq_verify_drafts(x, drafts)
    assert got.accepted.tolist() == [0] * B and got.tokens.tolist() == [[i, -1] for i, _ in tops]
    noise = torch.ones((B, V), device=DEV)
    got = tq.tq_verify_drafts(x[:, :1], noise=noise)
    assert got.tokens[:, 0].tolist() == [i for i, _ in tops]
    for dtype in (BF16, F16):
        assert torch.equal(tq.tq_verify_drafts(x[:, :1].to(dtype), noise=noise).tokens, got.tokens)


def test_verification_of_drafts_that_cannot_be():
    B, K, V = 5, 3, 100
    c = verify_case(1, B, K, V, F32, F32, temps=None)
    c["draft_tokens"][0, 0], c["draft_tokens"][1, 0], c["draft_tokens"][2, 1] = -1, V, 1 << 30
    c["uniforms"].zero_()
    check(c)
    c["draft_probs"] = None
    check(c)
    c["draft_lens"] = i32([-4, 9, 0, 2, 3])
    check(c)
    assert tq.tq_device_error() == tq.TQ_DEVERR_SEQLEN
    c = verify_case(2, B, K, V, F32, F32, temps=None)
    c["target"] = c["draft_probs"].log()[:, [0, 1, 2, 2]].contiguous()   # the drafting model's own: nearly all stand
    c["uniforms"].fill_(1 - 2.0 ** -10)
    got = check(c)
    assert got.accepted.tolist() == [K] * B
    c["target_probs"], c["target"] = True, c["draft_probs"][:, [0, 1, 2, 2]].contiguous()
    c["uniforms"].fill_(1.0)   # outside its range: no residual is left, the row itself is
    got = check(c)
    assert got.accepted.tolist() == [0] * B


@pytest.mark.parametrize("T", [1e-40, 1e-30, 1e-3, 100.0, 1e30, 3e38, math.inf, math.nan, -1.0])
def test_verification_temperatures(T):
    B, K, V = 4, 2, 600
    for dtype in (F32, BF16):
        c = verify_case(3, B, K, V, dtype, F32, temps=None)
        c["target"][:, :, 100:200] = -math.inf
        c["temperatures"] = torch.full((B,), T, device=DEV)
        if T == T and abs(T) != math.inf:
            check(c)
        got = tq.tq_verify_drafts(**c)
        for b in range(B):
            n = int(got.accepted[b])
            assert not 100 <= int(got.tokens[b, n]) < 200


def test_verification_looks_at_no_row_behind_the_drafts():
    B, K, V = 9, 4, 3001
    c = verify_case(71, B, K, V, BF16, F32)
    c["draft_lens"] = i32([b % (K + 1) for b in range(B)])
    want = check(c)
    spoilt = c | {name: c[name].clone() for name in ("target", "draft_probs", "draft_tokens", "uniforms")}
    for b in range(B):
        k = b % (K + 1)
        spoilt["target"][b, k + 1:] = math.nan
        for name in ("draft_probs", "uniforms"):
            spoilt[name][b, k:] = math.nan
        spoilt["draft_tokens"][b, k:] = 1 << 30
    for x, y in zip(tq.tq_verify_drafts(**spoilt), want):
        assert torch.equal(x, y)
    errors([])


def test_verification_draws_the_targets_distribution():
    # 60000 sequences of one draft over 6 tokens, one row of p and one of q for all: the first token is distributed as p, the
    # second as its row. A count is off by five deviations once in a million.
    B, V = 60000, 6
    g = gen(21)
    p = torch.tensor([[0.05, 0.3, 0.2, 0.0, 0.35, 0.1], [0.5, 0.1, 0.1, 0.1, 0.1, 0.1]], device=DEV)
    q = torch.tensor([0.3, 0.1, 0.2, 0.2, 0.1, 0.1], device=DEV)
    x = (p.log() * 0.7).expand(B, 2, V)
    drafts = (q / torch.empty((B, V), device=DEV).exponential_(generator=g)).argmax(-1).to(torch.int32)[:, None]
    noise = torch.empty((B, V), device=DEV).exponential_(generator=g)
    got = tq.tq_verify_drafts(x, drafts, q.expand(B, 1, V), torch.rand((B, 1), generator=g, device=DEV), noise, torch.full((B,), 0.7, device=DEV))
    first = torch.bincount(got.tokens[:, 0].long(), minlength=V).double().cpu()
    kept = got.accepted == 1
    second = torch.bincount(got.tokens[kept, 1].long(), minlength=V).double().cpu()
    for count, row, n in ((first, p[0], B), (second, p[1], int(kept.sum()))):
        row = row.double().cpu()
        assert bool(((count - n * row).abs() <= 5 * (n * row * (1 - row)).sqrt() + 1e-9).all()), (count / n, row)


def test_verification_captured_and_on_two_streams():
    cases = [verify_case(s, 7, 3, 5003, BF16, F32) for s in (31, 32, 33)]
    want = [tq.tq_verify_drafts(**c) for c in cases]
    s = torch.cuda.Stream()
    live = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in cases[0].items()}
    out = tq.Verified(*(torch.zeros_like(x) for x in want[0]))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tq.tq_verify_drafts(**live, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tq.tq_verify_drafts(**live, out=out)
    for c, w in zip(cases, want):
        for k, v in live.items():
            if isinstance(v, torch.Tensor):
                v.copy_(c[k])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, w):
            assert torch.equal(x, y)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[tq.tq_verify_drafts(**c, stream=st) for c, st in zip(cases, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for round_ in got:
        for x, w in zip(round_, want):
            assert all(torch.equal(a, b) for a, b in zip(x, w))


@pytest.mark.parametrize("K", [0, 2])
@pytest.mark.parametrize("dtype,V", [(BF16, 33003), (F32, 33003), (F16, 65536)])
def test_verification_of_infinities_between_ctas(dtype, V, K):
    # two tokens of +inf are equally likely, wherever one of them lies: the smaller noise decides
    B = 48
    c = verify_case(V + K, B, K, V, dtype, None, temps=None)
    c["draft_tokens"] = None if K == 0 else torch.zeros((B, K), dtype=torch.int32, device=DEV)
    at = torch.arange(B, device=DEV)
    ends = [(i * V) // 8 + j for i in (1, 2, 3, 4, 5, 6) for j in range(-4, 4)]   # where the shares of eight CTAs may end
    places = torch.tensor([ends[b % len(ends)] for b in range(B)], device=DEV)
    c["target"][at, :, places] = math.inf
    c["target"][:, :, 77] = math.inf
    c["noise"][:, 77], c["noise"][at, places] = 0.5, 0.75
    got = check(c)
    errors_word = tq.tq_device_error()
    assert errors_word == tq.TQ_DEVERR_NONFINITE and not got.accepted.any() and bool((got.tokens[:, 0] == 77).all())
    c["noise"][:, 77] = 1.0
    got = check(c)
    assert tq.tq_device_error() == tq.TQ_DEVERR_NONFINITE and torch.equal(got.tokens[:, 0].long(), places)


@pytest.mark.parametrize("K", [0, 1])
def test_verification_of_far_rows(K):
    B, V = 2, 999
    c = verify_case(41, B, K, V, BF16, F32)
    hold = torch.zeros((1 << 31) + 4 * V, dtype=BF16, device=DEV)
    x = torch.as_strided(hold, (B, K + 1, V), (1 << 31, V, 1))
    x.copy_(c["target"])
    c["target"] = x
    check(c)


def test_verification_lengths_in_place():
    c = verify_case(61, 6, 2, 700)
    want = tq.tq_verify_drafts(**c)
    lens = c["seq_lens"].clone()
    out = tq.Verified(*(torch.zeros_like(x) for x in want))._replace(keep_lens=lens)
    tq.tq_verify_drafts(**(c | {"seq_lens": lens}), out=out)
    for x, y in zip(out, want):
        assert torch.equal(x, y)
    quiet = tq.tq_verify_drafts(**(c | {"seq_lens": None}), out=out._replace(keep_lens=None, logprobs=None))
    assert quiet.keep_lens is None and torch.equal(quiet.tokens, want.tokens)


FIRST_IN_A_GRAPH = """
import torch, turboquant_compressed_kv_tq_gb300 as tq
f = dict(device="cuda")
bt, lens, places = tq.BlockTable(3, 4, 12, 16), torch.zeros(3, dtype=torch.int32, **f), tq.Places(3, 6)
rope, q = tq.Rope.of_base(64), torch.randn(3, 4, 2, 64, **f)
x, d, u, e = torch.randn(3, 9, 5000, **f), torch.zeros(3, 8, dtype=torch.int32, **f), torch.rand(3, 8, **f), torch.rand(3, 5000, **f) + 0.1
def calls():
    bt.reserve(lens, None, 2, places)
    bt.release(lens)
    return rope.apply(q, starts=lens)[0], tq.tq_verify_drafts(x, d, None, u, e), tq.tq_verify_drafts(x[:, :1], noise=e), tq.tq_verify_drafts(x[:, :1])
s = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    got = calls()
g.replay()
torch.cuda.synchronize()
want = calls()
assert torch.equal(got[0], want[0]) and all(torch.equal(a.tokens, b.tokens) for a, b in zip(got[1:], want[1:])) and tq.tq_device_error() == 0
print("same")
"""


def test_first_calls_of_a_process_in_a_graph():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", (r.stdout[-500:], r.stderr[-2000:])


def test_verification_refusals():
    c = verify_case(51, 2, 2, 50)
    bad = [("target", c["target"][0]), ("target", c["target"].cpu()), ("target", c["target"].transpose(1, 2)), ("draft_tokens", None), ("draft_tokens", c["draft_tokens"].long()),
           ("draft_probs", c["draft_probs"][:, :1]), ("uniforms", c["uniforms"].double()), ("noise", c["noise"][:1]), ("temperatures", c["temperatures"][:1]),
           ("draft_lens", i32([1])), ("seq_lens", i32([1]))]
    for name, x in bad:
        with pytest.raises(ValueError):
            tq.tq_verify_drafts(**(c | {name: x}))
    for name, x in (("target", c["target"].double()), ("draft_probs", c["draft_probs"].double()), ("noise", c["noise"].double())):
        with pytest.raises(TypeError):
            tq.tq_verify_drafts(**(c | {name: x}))
    out = tq.tq_verify_drafts(**c)
    with pytest.raises(ValueError):
        tq.tq_verify_drafts(**(c | {"seq_lens": None}), out=out)
    with pytest.raises(tq.TQError):
        tq.tq_verify_drafts(torch.zeros(1, 66, 4, device=DEV), torch.zeros(1, 65, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("graphed", [False, True])
def test_drafted_steps(graphed):
    """Steps of 3 tokens for 4 sequences over the compressed cache: every call of the loop, against the same loop on
    contiguous lengths that the host keeps."""
    B, Hq, Hk, D, V, K, BT, width, layers = 4, 8, 2, 128, 500, 2, 16, 12, 2
    kc, vc = tq.Codec(D, 3, tq.TQ_MODE_PROD, seed=0), tq.Codec(D, 3, tq.TQ_MODE_MSE, seed=1)
    cache = tq.CompressedKVCache(kc, vc, layers, 40, BT, Hk, exact_encode=True)
    plain = tq.CompressedKVCache(kc, vc, layers, B * width, BT, Hk, exact_encode=True)
    bt = tq.BlockTable(B, width, 40, BT)
    bt.free_blocks.copy_(torch.randperm(40, generator=gen(1), device=DEV))
    rope = tq.Rope.of_base(D)
    lens0 = i32([5, 33, 0, 16])
    bt.reserve(torch.zeros_like(lens0), lens0, 64)
    for layer in range(layers):   # prompts
        k, v = laid_out(B, Hk, 33, D, "bht", BF16, 60 + layer), laid_out(B, Hk, 33, D, "bht", BF16, 70 + layer)
        for b, n in enumerate(lens0.tolist()):
            if n:
                kb, vb = (x[b:b + 1, :, :n].contiguous() for x in (k, v))
                cache.append(layer, kb, vb, i32([0]), bt.table[b:b + 1], width)
                plain.append(layer, kb, vb, i32([0]), (torch.arange(width, device=DEV, dtype=torch.int32) + b * width)[None], width)
    loop = speculative.DraftedBatch(bt, lens0.clone())
    n, most = K + 1, width * BT
    qkv = torch.zeros(B, n, Hq + 2 * Hk, D, dtype=BF16, device=DEV)
    logits, drafts = torch.zeros(B, n, V, device=DEV), torch.zeros(B, K, dtype=torch.int32, device=DEV)
    uniforms, noise = torch.zeros(B, K, device=DEV), torch.ones(B, V, device=DEV)
    q_rot, k_rot = torch.empty(B, Hq, n, D, dtype=BF16, device=DEV), torch.empty(B, Hk, n, D, dtype=BF16, device=DEV)
    outs = [torch.empty(B, Hq, n, D, device=DEV) for _ in range(layers)]
    want_outs = [torch.empty_like(x) for x in outs]
    ws = torch.empty(cache.workspace_bytes(B, Hq, n, most), dtype=torch.uint8, device=DEV)
    seen = tq.Verified(i32([0] * B), torch.zeros(B, n, dtype=torch.int32, device=DEV), i32([0] * B), torch.zeros(B, n, device=DEV))
    q, k, v = (x.transpose(1, 2) for x in qkv.split((Hq, Hk, Hk), dim=2))

    def step():
        loop.begin(n)
        for layer in range(layers):
            loop.rotate(rope, q, k, q_rot, k_rot)
            loop.attend(cache, layer, k_rot, v.contiguous(), q_rot, most, outs[layer], ws)
        loop.finish(logits, drafts, None, uniforms, noise, out=seen)

    def draw(seed):
        g = gen(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
        logits.copy_(4 * torch.randn(logits.shape, generator=g, device=DEV))
        drafts.copy_(logits[:, :K].argmax(-1))
        uniforms.copy_(torch.rand(uniforms.shape, generator=g, device=DEV))
        noise.copy_(torch.empty_like(noise).exponential_(generator=g))

    graph = None
    if graphed:
        table, free, used = bt.table.clone(), bt.free_blocks.clone(), bt.n_used.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        draw(99)
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        # as before the step (its appended records are behind the lengths, and are written again)
        for x, y in ((bt.table, table), (bt.free_blocks, free), (bt.n_used, used), (loop.seq_lens, lens0)):
            x.copy_(y)
    lens = lens0.tolist()
    for i in range(8):
        draw(100 + i)
        graph.replay() if graph else step()
        before = i32(lens)
        pos = before[:, None] + torch.arange(n, device=DEV)
        qr, kr = (rope.apply(x, positions=pos.to(torch.int32))[0] for x in (q, k))
        for layer in range(layers):
            plain.decode_step(layer, kr, v.contiguous(), qr, before, None, width, most, want_outs[layer], ws)
            assert torch.equal(outs[layer], want_outs[layer]), (i, layer)
        ref.check_verified(logits, drafts, None, uniforms, noise, None, None, False, before, seen)
        lens = [N + a + 1 for N, a in zip(lens, seen.accepted.tolist())]
        assert loop.seq_lens.tolist() == lens
        held = [sum(x >= 0 for x in row) for row in bt.table.tolist()]
        assert held == [-(-N // BT) for N in lens]
        ids = [x for row in bt.table.tolist() for x in row if x >= 0] + bt.free_blocks[bt.n_used.item():].tolist()
        assert sorted(ids) == list(range(40))
    assert lens != [N + 8 for N in lens0.tolist()]   # some drafts stood
