"""Drafted steps for which the free list, or a sequence's row of the table, has not blocks enough."""
import pytest
import torch

import serve_util as ref
import turboquant_compressed_kv_tq_gb300 as tq
from test_gpu_serve import BF16, DEV, gen, i32, laid_out, no_device_error  # noqa: F401 (no_device_error: fixture)
from turboquant_compressed_kv_tq_gb300 import speculative

pytestmark = pytest.mark.gpu


class Run:
    """4 sequences over a pool of few blocks, and beside them the same ones in rows of their own."""
    B, Hq, Hk, D, V, K, BT, width = 4, 8, 2, 128, 300, 2, 16, 5
    n = K + 1

    def __init__(self, lens, blocks):
        B, BT, width = self.B, self.BT, self.width
        kc, vc = tq.Codec(self.D, 3, tq.TQ_MODE_PROD, seed=0), tq.Codec(self.D, 3, tq.TQ_MODE_MSE, seed=1)
        self.cache = tq.CompressedKVCache(kc, vc, 1, blocks, BT, self.Hk, exact_encode=True)
        self.plain = tq.CompressedKVCache(kc, vc, 1, B * width, BT, self.Hk, exact_encode=True)
        self.bt, self.blocks, self.lens = tq.BlockTable(B, width, blocks, BT), blocks, list(lens)
        self.bt.free_blocks.copy_(torch.randperm(blocks, generator=gen(1), device=DEV))
        self.bt.reserve(i32([0] * B), i32(lens), width * BT)
        for b, n in enumerate(lens):
            self.prompt(b, n, 40 + b)
        self.loop = speculative.DraftedBatch(self.bt, i32(lens))
        self.table, self.free = self.bt.table.tolist(), self.bt.free_blocks.tolist()
        self.used = self.bt.n_used.item()
        n, Hq, Hk, D, V, K = self.n, self.Hq, self.Hk, self.D, self.V, self.K
        self.qkv = torch.zeros(B, n, Hq + 2 * Hk, D, dtype=BF16, device=DEV)
        self.logits, self.drafts = torch.zeros(B, n, V, device=DEV), torch.zeros(B, K, dtype=torch.int32, device=DEV)
        self.uniforms, self.noise = torch.zeros(B, K, device=DEV), torch.ones(B, V, device=DEV)
        self.out, self.want = torch.empty(B, Hq, n, D, device=DEV), torch.empty(B, Hq, n, D, device=DEV)
        self.ws = torch.empty(self.cache.workspace_bytes(B, Hq, n, width * BT), dtype=torch.uint8, device=DEV)
        self.seen = tq.Verified(i32([0] * B), torch.zeros(B, n, dtype=torch.int32, device=DEV), i32([0] * B), torch.zeros(B, n, device=DEV))

    def prompt(self, b, n, seed):
        if n:
            k, v = (laid_out(1, self.Hk, n, self.D, "bht", BF16, seed + d) for d in (0, 500))
            self.cache.append(0, k, v, i32([0]), self.bt.table[b:b + 1], self.width)
            self.plain.append(0, k, v, i32([0]), torch.arange(self.width, device=DEV, dtype=torch.int32)[None] + b * self.width, self.width)

    def step(self, stream=None):
        q, k, v = (x.transpose(1, 2) for x in self.qkv.split((self.Hq, self.Hk, self.Hk), dim=2))
        k, v, q = (x.contiguous() for x in (k, v, q))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(1 << 22)   # 2 ms of the current stream: what is not on the named one comes late
        self.loop.begin(self.n, stream)
        self.loop.attend(self.cache, 0, k, v, q, self.width * self.BT, self.out, self.ws, stream=stream)
        seen = self.loop.finish(self.logits, self.drafts, None, self.uniforms, self.noise, out=self.seen, stream=stream)
        if stream is not None:
            stream.synchronize()   # (q, k and v are the other stream's)
        return seen

    def draw(self, seed):
        g = gen(seed)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device=DEV))
        self.logits.copy_(4 * torch.randn(self.logits.shape, generator=g, device=DEV))
        self.drafts.copy_(self.logits[:, :self.K].argmax(-1))
        self.uniforms.copy_(torch.rand(self.uniforms.shape, generator=g, device=DEV) * 0.6)
        self.noise.copy_(torch.empty_like(self.noise).exponential_(generator=g))

    def check(self, call):
        """One step by `call` against the definition: rows that have all their places, and the others (returned)."""
        B, n, BT, width = self.B, self.n, self.BT, self.width
        before = list(self.lens)
        call()
        # the append and the attention flag what has no block
        torch.cuda.synchronize()
        word = tq.tq_device_error()
        self.used, granted, _, _, _, _, err = ref.reserve(self.table, self.free, self.used, before, None, n, BT, self.blocks, 0)
        short = [b for b in range(B) if granted[b] < n]
        assert bool(word & tq.TQ_DEVERR_CAPACITY) == bool(short) and (short or word == 0)
        q, k, v = (x.transpose(1, 2).contiguous() for x in self.qkv.split((self.Hq, self.Hk, self.Hk), dim=2))
        self.plain.decode_step(0, k, v, q, i32(before), None, width, width * BT, self.want, self.ws)
        torch.cuda.synchronize()
        tq.tq_device_error()   # (rows at their end)
        whole = [b for b in range(B) if b not in short]
        assert torch.equal(self.out[whole], self.want[whole])
        accepted, tokens = self.seen.accepted.tolist(), self.seen.tokens.tolist()
        got = tq.Verified(*(x[whole] for x in self.seen))
        if whole:
            ref.check_verified(self.logits[whole], self.drafts[whole], None, self.uniforms[whole], self.noise[whole], None, None, False, i32(before)[whole], got)
        for b in whole:
            self.lens[b] += accepted[b] + 1
        for b in short:   # as it was
            assert accepted[b] == 0 and tokens[b] == [-1] * n and self.seen.logprobs[b].tolist() == [0.0] * n
        assert self.loop.seq_lens.tolist() == self.lens and self.seen.keep_lens.tolist() == self.lens
        self.used, err = ref.release(self.table, self.free, self.used, self.lens, BT, self.blocks)
        assert not err
        assert self.bt.table.tolist() == self.table and self.bt.free_blocks.tolist() == self.free and self.bt.n_used.item() == self.used
        assert [sum(x >= 0 for x in row) for row in self.table] == [-(-N // BT) for N in self.lens]
        return short

    def empty(self, b):
        """Sequence b is done: its blocks go back, and another begins in its row with nothing."""
        self.lens[b] = 0
        self.loop.seq_lens[b] = 0
        self.bt.release(self.loop.seq_lens)
        self.used, err = ref.release(self.table, self.free, self.used, self.lens, self.BT, self.blocks)
        assert not err


@pytest.mark.parametrize("graphed", [False, True])
def test_steps_that_run_out_of_blocks(graphed):
    # 14 + 3 tokens take the last block; 30 + 3 find none, and wait until another sequence has ended
    r = Run([14, 30, 5, 33], 8)
    call = r.step
    if graphed:
        s = torch.cuda.Stream()
        kept = [x.clone() for x in (r.bt.table, r.bt.free_blocks, r.bt.n_used, r.loop.seq_lens)]
        s.wait_stream(torch.cuda.current_stream())
        r.draw(99)
        with torch.cuda.stream(s):
            r.step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r.step()
        for x, y in zip((r.bt.table, r.bt.free_blocks, r.bt.n_used, r.loop.seq_lens), kept):
            x.copy_(y)
        torch.cuda.synchronize()
        tq.tq_device_error()
        call = graph.replay
    waited = []
    for i in range(6):
        r.draw(100 + i)
        waited.append(r.check(call))
    assert waited[0] == [1] and r.lens[1] == 30
    r.empty(3)
    more = []
    for i in range(6):
        r.draw(200 + i)
        more.append(r.check(call))
    assert 1 not in more[0] and r.lens[1] > 30
    for b in range(4):
        r.empty(b)
    assert r.bt.n_used.item() == 0 and sorted(r.bt.free_blocks.tolist()) == list(range(8))


def test_steps_at_the_end_of_a_row():
    # a row of 5 blocks holds 80 tokens: 79 + 3 do not fit, shorter steps do
    r = Run([79, 10, 77, 3], 20)
    r.draw(7)
    assert r.check(r.step) == [0]
    r.draw(8)
    assert r.check(r.step) == ([0, 2] if r.lens[2] > 77 else [0])
    seen = []

    def one():
        r.loop.begin(1)
        seen.append(r.loop.finish(r.logits[:, :1], noise=r.noise))
    before = list(r.lens)
    one()
    torch.cuda.synchronize()
    tq.tq_device_error()
    grown = [N + (N < 80) for N in before]
    assert r.loop.seq_lens.tolist() == grown and seen[0].keep_lens.tolist() == grown
    assert [t[0] >= 0 for t in seen[0].tokens.tolist()] == [N < 80 for N in before]
    kept = seen[0].keep_lens.clone()
    one()
    torch.cuda.synchronize()
    tq.tq_device_error()
    assert torch.equal(seen[0].keep_lens, kept)   # what was returned stays


def test_steps_on_a_named_stream():
    r = Run([14, 30, 5, 33], 8)
    s = torch.cuda.Stream()
    for i in range(3):
        r.draw(400 + i)
        assert 1 in r.check(lambda: r.step(s))


def test_steps_whose_kept_lengths_go_in_place():
    r = Run([14, 30, 5, 33], 8)
    r.seen = r.seen._replace(keep_lens=r.loop.seq_lens)
    for i in range(3):
        r.draw(300 + i)
        assert 1 in r.check(r.step)


def test_a_verification_of_more_rows_than_were_asked_for():
    r = Run([14, 30, 5, 33], 12)
    r.loop.begin(2)
    with pytest.raises(ValueError):
        r.loop.finish(r.logits, r.drafts)
    r.loop.finish(r.logits[:, :2], r.drafts[:, :1].contiguous())
