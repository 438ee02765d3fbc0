"""Verification and drawing against the precision that include/tq.h states, where it is nearest to being missed."""
import math

import pytest
import torch

import turboquant_compressed_kv_tq_gb300 as tq
from test_gpu_serve import BF16, DEV, F16, F32, gen, i32, no_device_error, verify_case  # noqa: F401 (no_device_error: fixture)

pytestmark = pytest.mark.gpu
LOG2E = 1 / math.log(2)


def of_weight(d):
    """A weight 2^-d: ex2 is good to 2^-22; the exponent to d 2^-24 by the scale's rounding and as much by its own, times ln 2."""
    return 2.0 ** -22 + d * 2.0 ** -23


def of_draft(d):
    """The exponent's own rounding put back: what is left is that of (x - largest), d 2^-24 ln 2, and three roundings."""
    return 2.0 ** -21 + d * 2.0 ** -24


def of_sum(V):
    """Weights are off by 2^-22 + d 2^-23.5, d at most log2(V) on average; 29 roundings of a sum and its joins, one for each 4096
    tokens, and where the largest rises there 2^-22 + 2^-24: 2^-18 + V 2^-33."""
    return 2.0 ** -18 + V * 2.0 ** -33


QUOTIENT = 2.0 ** -22   # a reciprocal to 2^-23, a product to 2^-24


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T", [1.0, 0.3, 7.0])
@pytest.mark.parametrize("drafted", [False, True])
def test_two_tokens_of_nearly_one_score(dtype, T, drafted):
    # far below the largest, which is not to be drawn; everything else has infinite noise
    B, V = 4000, 1024
    g = gen(1)
    x = torch.full((B, 2, V), -30.0 * T, device=DEV)
    x[:, :, 3] = (torch.rand((B, 1), generator=g, device=DEV) * 40 - 20).to(dtype).float()
    far = torch.rand((B, 2), generator=g, device=DEV).double() * 85 / LOG2E * T
    at = torch.stack((torch.randint(10, V // 2, (B,), generator=g, device=DEV), torch.randint(V // 2, V, (B,), generator=g, device=DEV)), 1)
    row = torch.arange(B, device=DEV)
    for i in range(2):
        x[row, :, at[:, i]] = (x[:, 0, 3].double() - far[:, i]).float()[:, None]
    x = x.to(dtype)
    top = x[:, 0].double().amax(1)
    temps = torch.full((B,), T, device=DEV)
    Td = float(temps[0])
    d = (top[:, None] - torch.gather(x[:, 0], 1, at).double()) / Td * LOG2E
    least = of_weight(d).sum(1) + 2 * QUOTIENT
    gap = least * (1 + torch.rand(B, generator=g, device=DEV, dtype=torch.float64)) * torch.where(torch.rand(B, generator=g, device=DEV) < 0.5, 1.0, -1.0)
    noise = torch.full((B, V), math.inf, device=DEV)
    weight = torch.exp2(-d)
    noise[row, at[:, 0]] = (weight[:, 0]).float()
    noise[row, at[:, 1]] = (weight[:, 1] * (1 + gap)).float()
    # as they count: weights below 2^-126 not, noise below 2^-100 as that (where the largest is one of the others, far off)
    score = torch.where(d < 126, weight, 0.0) / torch.gather(noise, 1, at).double().clamp(min=2.0 ** -100)
    ratio = score[:, 0] / score[:, 1] - 1
    none = (score == 0).all(1)
    clear = ((ratio.abs() > least) | none) & ((d - 126).abs() > 0.01).all(1)   # (noise is rounded: a few are nearer than asked)
    assert bool((clear.double().mean() > 0.9))
    want = torch.where(none, -1, torch.where(ratio > 0, at[:, 0], at[:, 1]))
    if drafted:
        got = tq.tq_verify_drafts(x, i32([[0]] * B), None, torch.zeros(B, 1, device=DEV), noise, temps, draft_lens=i32([0] * B))
    else:
        got = tq.tq_verify_drafts(x[:, :1], noise=noise, temperatures=temps)
    torch.cuda.synchronize()
    assert tq.tq_device_error() == (tq.TQ_DEVERR_NONFINITE if bool((got.tokens[:, 0] < 0).any()) else 0)
    bad = clear & (got.tokens[:, 0].long() != want)
    assert not bool(bad.any()), (int(bad.sum()), d[bad][:4].tolist(), ratio[bad][:4].tolist())


def rows_of(kind, B, V, dtype, seed):
    g = gen(seed)
    if kind == "random":
        return (4 * torch.randn((B, 2, V), generator=g, device=DEV)).to(dtype)
    if kind == "flat":   # one likely token, all others alike and together likelier than it
        x = -(torch.rand((B, 1, 1), generator=g, device=DEV) * 11).expand(B, 2, V).contiguous()
        x[:, :, V // 3] = 0.0
        return x.to(dtype)
    step = torch.rand((B, 1, 1), generator=g, device=DEV) * 20 / V   # rising from the first to the last
    return (step * torch.arange(V, device=DEV)).expand(B, 2, V).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["random", "flat", "rising"])
@pytest.mark.parametrize("B,V", [(6, 131072), (700, 9000), (160, 65536)])
def test_logs_and_drafts_at_the_border(dtype, kind, B, V):
    x = rows_of(kind, B, V, dtype, V)
    g = gen(2)
    T = 0.25 + 1.5 * torch.rand(B, generator=g, device=DEV)
    drafts = torch.randint(0, V, (B, 1), generator=g, device=DEV, dtype=torch.int32)
    drafts[::3] = x[::3, :1].float().argmax(-1).to(torch.int32)
    near = 2.0 ** -30
    chances, tops = [], []
    for b in range(B):   # (a row at a time: 64 bits)
        z = x[b].double() / T[b].double()
        tops.append((z.amax(-1, keepdim=True) - z) * LOG2E)
        chances.append(torch.log_softmax(z, -1))
        tops[-1] = torch.gather(tops[-1], 1, drafts[b].long().expand(2)[:, None])[:, 0]
    log_p = torch.stack([c[0, int(t)] for c, t in zip(chances, drafts[:, 0])])
    d = torch.stack(tops)[:, 0]
    p = log_p.exp()
    # a draft is kept below the border and not above it; the drafts' probabilities lie so that u is about a half
    least = of_draft(d) + of_sum(V) + 2.0 ** -22   # (two products)
    side = torch.where(torch.rand(B, generator=g, device=DEV) < 0.5, 1.0, -1.0)
    q = torch.full((B, 1, V), near, device=DEV)
    q[torch.arange(B, device=DEV), 0, drafts[:, 0].long()] = (1.9 * p).float()
    u = (p * (1 + side * least * 1.5) / (1.9 * p).float().double()).float()[:, None]
    limit = u[:, 0].double() * (1.9 * p).float().double()
    clear = (limit / p - 1).abs() > least
    assert bool(clear.double().mean() > 0.9)
    noise = torch.empty((B, V), device=DEV).exponential_(generator=g)
    got = tq.tq_verify_drafts(x, drafts, q, u, noise, T)
    bad = clear & ((limit < p) != (got.accepted == 1))
    assert not bool(bad.any()), (int(bad.sum()), (limit / p - 1)[bad][:4].tolist(), least[bad][:4].tolist())
    drawn = tq.tq_verify_drafts(x[:, :1], noise=noise, temperatures=T)
    likeliest = tq.tq_verify_drafts(x[:, :1])
    for b in range(B):
        c = chances[b]
        n = int(got.accepted[b])
        for i in range(n + 1):
            want = float(c[i, int(got.tokens[b, i])])
            assert abs(float(got.logprobs[b, i]) - want) <= of_sum(V) + 2.0 ** -22 * abs(want)
        want = float(c[0, int(drawn.tokens[b, 0])])
        assert abs(float(drawn.logprobs[b, 0]) - want) <= of_sum(V) + 2.0 ** -22 * abs(want)
        want = float(torch.log_softmax(x[b, 0].double(), -1)[int(likeliest.tokens[b, 0])])
        assert abs(float(likeliest.logprobs[b, 0]) - want) <= of_sum(V) + 2.0 ** -22 * abs(want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("close", [0.0, 0.99, 0.9999])
def test_next_tokens_of_residuals(dtype, close):
    # the drafts' probabilities near the target's: a residual is off by a part of p
    B, V = 60, 5000
    c = verify_case(9, B, 1, V, dtype, F32, temps=None)
    p = torch.softmax(c["target"].double(), -1)
    c["draft_probs"] = (close * p[:, :1] + (1 - close) * c["draft_probs"].double()).float()
    c["uniforms"] = torch.ones_like(c["uniforms"])   # (most of them not kept)
    got = tq.tq_verify_drafts(**c)
    some = 0
    for b in range(B):
        n = int(got.accepted[b])
        t = int(got.tokens[b, n])
        pn = p[b, n]
        q = c["draft_probs"][b, 0].double() if n == 0 else torch.zeros_like(pn)
        d = torch.log2(pn.amax() / pn)
        off = (of_weight(d) + of_sum(V)) * pn
        e = c["noise"][b].double()
        rest = (pn - q).clamp(min=0)
        least, most = (pn - q - off).clamp(min=0) / e, ((pn - q + off) / e).clamp(min=0)
        if bool((rest > 0).any()):
            some += n == 0
            assert float(most[t]) * (1 + 2 * QUOTIENT) >= float(least.max())
    assert some > 5
