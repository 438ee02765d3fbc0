"""The calls around the caches' where they can go wrong: masked rows with a NaN in them, lengths where nothing is drafted, noise that
leaves no token, the largest rotation."""
import math

import pytest
import torch

import serve_util as ref
import turboquant_compressed_kv_tq_gb300 as tq
from test_gpu_serve import BF16, DEV, F16, F32, check, check_rotation, errors, gen, i32, no_device_error, verify_case  # noqa: F401 (no_device_error: fixture)

pytestmark = pytest.mark.gpu


def nonfinite():
    torch.cuda.synchronize()
    return bool(tq.tq_device_error() & tq.TQ_DEVERR_NONFINITE)


@pytest.mark.parametrize("form", ["drafts", "greedy", "draw"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V", [300, 50021, 131072])
def test_nan_among_masked_tokens_is_told(dtype, V, form):
    # few tokens allowed, one of them NaN; or a row that begins with NaNs: nothing else in the lanes that see them
    B, K = 4, 2 if form == "drafts" else 0
    rows = {"one": [V // 2 + 1], "first": list(range(min(V // 3, 9000))), "last": [V - 1]}
    for name, at in rows.items():
        c = verify_case(V + K, B, K, V, dtype, F32, temps=None)
        x = c["target"]
        if name == "first":
            x[2, 0, at] = math.nan
        else:
            x[2, 0] = -math.inf
            x[2, 0, V // 4] = 1.5
            x[2, 0, at] = math.nan
        if form == "greedy":
            c["noise"] = None
        got = check(c)
        assert nonfinite(), name
        if name != "first":
            assert int(got.tokens[2, int(got.accepted[2])]) == V // 4 or int(got.accepted[2]) > 0
        # masked alike without a NaN: nothing to tell
        x[2, 0, at] = -math.inf
        check(c)
        assert not nonfinite(), name


@pytest.mark.parametrize("noise", [True, False])
def test_lengths_where_nothing_is_drafted(noise):
    c = verify_case(3, 4, 0, 700, F32, None, temps=None)
    if not noise:
        c["noise"] = None
    want = check(c)
    for bad in ([0, 0, 1, 0], [0, -1, 0, 0]):
        got = tq.tq_verify_drafts(**(c | {"draft_lens": i32(bad)}))
        errors(["seqlen"])
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    check(c | {"draft_lens": i32([0] * 4)})
    errors([])


@pytest.mark.parametrize("V", [900, 40000])
def test_noise_that_leaves_no_token(V):
    # what is likely has infinite noise, what is left counts as 0: no token, whether or not the call has drafts
    B = 3
    for dtype in (F32, BF16):
        x = torch.full((B, 2, V), -200.0, dtype=dtype, device=DEV)
        x[:, :, :V // 2] = 0.0
        e = torch.ones(B, V, device=DEV)
        e[:, :V // 2] = math.inf
        drawn = tq.tq_verify_drafts(x[:, :1], noise=e)
        assert nonfinite()
        drafted = tq.tq_verify_drafts(x, i32([[0]] * B), None, torch.zeros(B, 1, device=DEV), e, draft_lens=i32([0] * B))
        assert nonfinite()
        for got in (drawn, drafted):
            assert got.tokens[:, 0].tolist() == [-1] * B and not got.logprobs.any() and not got.accepted.any()


@pytest.mark.parametrize("K", [0, 2])
@pytest.mark.parametrize("noise", [True, False])
def test_probabilities_that_are_no_numbers_are_not_taken(K, noise):
    # greedy, of probabilities: no logits, nothing to tell
    B, V = 4, 3001
    c = verify_case(17, B, K, V, F32, F32, temps=None, probs=True)
    if noise:
        c["temperatures"] = torch.zeros(B, device=DEV)
    else:
        c["noise"] = None
    c["target"][1, 0, 5:900] = math.nan
    got = check(c)
    errors([])
    assert not bool(((got.tokens[1] >= 5) & (got.tokens[1] < 900))[0])


def test_the_largest_rotation():
    # 2^31 - 1 tokens, the most that a call takes, in place
    n, D = (1 << 31) - 1, 16
    x = torch.zeros(1, 1, n, D, dtype=BF16, device=DEV)
    ends = [slice(0, 40), slice(n // 2 - 20, n // 2 + 20), slice(n - 40, n)]
    before = []
    for i, s in enumerate(ends):
        x[:, :, s] = torch.randn((1, 1, 40, D), generator=gen(i), device=DEV).to(BF16)
        before.append(x[:, :, s].clone())
    r = tq.Rope.of_base(D)
    r.apply(x, out=x)
    for s, y in zip(ends, before):
        pos = torch.arange(s.start, s.stop, device=DEV)[None]
        check_rotation(y, x[:, :, s], pos, r, r.inv_freq)
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("Hq,Hk", [(8, 1), (1, 4), (1, 1)])
def test_rotation_of_a_single_head_in_place(Hq, Hk):
    # queries or keys of one head in a fused projection: its stride says nothing
    B, n, D = 3, 7, 64
    whole = torch.randn((B, n, Hq + 2 * Hk, D), generator=gen(5), device=DEV).to(BF16).transpose(1, 2)
    before = whole.clone()
    q, k = whole[:, :Hq], whole[:, Hq:Hq + Hk]
    r = tq.Rope.of_base(D)
    r.apply(q, k, q, k)
    pos = torch.arange(n, device=DEV).expand(B, n)
    check_rotation(before[:, :Hq], q, pos, r, r.inv_freq)
    check_rotation(before[:, Hq:Hq + Hk], k, pos, r, r.inv_freq)
    assert torch.equal(whole[:, Hq + Hk:], before[:, Hq + Hk:])
    with pytest.raises(tq.TQError):   # one head over the others
        r.apply(q, k, out=q, k_out=whole[:, Hq - 1:Hq - 1 + Hk])


@pytest.mark.parametrize("B,n", [(5, 7), (300, 40), (2500, 60)])
def test_new_lengths_that_become_the_granted_ones(B, n):
    width, BT = 6, 16
    news = [(7 * b) % (n + 1) for b in range(B)]
    lens = [(5 * b) % 50 for b in range(B)]
    table, free = [[-1] * width for _ in range(B)], list(range(B * 2))
    bt = tq.BlockTable.wrap(torch.tensor(table, dtype=torch.int32, device=DEV), i32(free), i32([0]), BT, B * 2)
    places = tq.Places(B, sum(news))
    places.granted.copy_(i32(news))
    bt.reserve(i32(lens), places.granted, n, places)
    used, granted, starts, seqs, pos, slots, err = ref.reserve(table, free, 0, lens, news, n, BT, B * 2, sum(news))
    errors(err)
    assert places.granted.tolist() == granted and places.starts.tolist() == starts and bt.table.tolist() == table and bt.n_used.item() == used
    assert places.seq_ids.tolist() == seqs and places.positions.tolist() == pos and places.slots.tolist() == slots
