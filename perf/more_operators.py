"""What a serving loop does around the caches' calls, as it is measured: rotary positions ahead of an append or an
attention call, block tables and slot maps from request lengths, and the verification of drafted tokens.

`own` chooses between the plain torch form and the framework's calls."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _rope(name, **kw):
    return {"name": name, "op": "rope", "rot": kw["D"], "inter": False, "source": "fused", "at": "starts", "ragged": False, "scaling": "none", "back": False, **kw}


def _blocks(name, **kw):
    return {"name": name, "op": "blocks", "ragged": False, "keep": "none", "short": False, **kw}


def _verify(name, **kw):
    return {"name": name, "op": "verify", "draft": None, "probs": False, "temp": "one", "ragged": False, **kw}


def listed():
    return [
        # one decoding step of a continuous batch: queries and keys taken out of a fused projection, rotated and laid out as decode wants them
        _rope("rope step", dtype="bf16", B=32, Hq=32, Hk=8, D=128, n=1, lo=4096, hi=65536),
        # a chunk of a long prompt at the far end of a stretched context
        _rope("rope chunk", dtype="bf16", B=1, Hq=64, Hk=8, D=128, n=8192, lo=253952, hi=253952, scaling="parts"),
        # a padded batch of prompts, half of each head rotated in neighbouring pairs, positions of the caller's own
        _rope("rope ragged", dtype="f16", B=12, Hq=12, Hk=4, D=64, rot=32, n=777, lo=3, hi=500, inter=True, ragged=True, at="positions", source="head"),
        # the gradient of a rotation, in 32 bits, wide heads
        _rope("rope gradient", dtype="f32", B=6, Hq=8, Hk=4, D=256, n=1999, lo=0, hi=130, scaling="ntk", back=True, source="head"),
        # one decoding step of a continuous batch: a place for one token each
        _blocks("blocks step", B=32, BT=16, lo=4096, hi=65536, n=1),
        # a step of drafted tokens: places for all, and the blocks behind the kept ones back to the free list
        _blocks("blocks drafts", B=300, BT=16, lo=17, hi=32749, n=5, ragged=True, keep="part"),
        # many prompts admitted at once
        _blocks("blocks prompts", B=512, BT=64, lo=0, hi=0, n=4096, ragged=True),
        # two drafted-for rows of one sequence
        _verify("verify pair", dtype="bf16", B=1, K=1, V=32000, draft="f32"),
        # continuous batching with four drafts each
        _verify("verify batch", dtype="bf16", B=64, K=4, V=131072, draft="f32"),
        # sequences with temperatures of their own, some greedy, of fewer drafts than others, an odd vocabulary
        _verify("verify mixed", dtype="f16", B=24, K=3, V=50021, draft="f16", temp="mixed", ragged=True),
        # probabilities that the caller has filtered, drafts that were looked up and have no probabilities
        _verify("verify filtered", dtype="f32", B=16, K=7, V=65537, probs=True),
        # no drafts: the next token of each sequence
        _verify("verify none", dtype="f32", B=200, K=0, V=131072, temp="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges, no dearer than the largest listed one."""
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["rope", "blocks", "verify"])
        if op == "rope":
            D = rng.choice([64, 64, 128, 128, 256, 80, 96, 192])
            Hk = rng.choice([1, 2, 4, 8])
            lo = _log(rng, 1, 1 << 20) - 1
            c = _rope("", dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), B=_log(rng, 1, 128), Hq=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, D=D,
                      n=rng.choice([1, 1, 2, 5, _log(rng, 3, 8192)]), lo=lo, hi=lo + rng.randrange(0, 5000))
            c |= {"rot": rng.choice([D, D, D // 32 * 16, 16]), "inter": rng.random() < 0.3, "source": rng.choice(["fused", "head"]),
                  "at": rng.choice(["starts", "positions"]), "ragged": rng.random() < 0.3, "scaling": rng.choice(["none", "linear", "ntk", "parts"]),
                  "back": rng.random() < 0.3}
        elif op == "blocks":
            lo = rng.choice([0, _log(rng, 1, 30000)])
            c = _blocks("", B=_log(rng, 1, 1500), BT=rng.choice([16, 32, 64, 128, 256]), lo=lo, hi=lo + rng.randrange(0, 1 + lo),
                        n=rng.choice([1, 1, 2, 5, 9, _log(rng, 3, 8192)]))
            c |= {"ragged": rng.random() < 0.5, "keep": rng.choice(["none", "part", "part", "all"]), "short": rng.random() < 0.2}
            if c["B"] * (c["hi"] // c["BT"] + 1) > 4e6:
                continue
        else:
            c = _verify("", dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), B=_log(rng, 1, 256), K=rng.choice([0, 0, 1, 2, 3, 4, 5, 7, 8]),
                        V=_log(rng, 500, 200000))
            c |= {"draft": rng.choice([None, "f32", "f32", "bf16", "f16"]) if c["K"] else None, "probs": rng.random() < 0.25,
                  "temp": rng.choice(["one", "mixed", "mixed", "greedy"]), "ragged": c["K"] > 0 and rng.random() < 0.4}
            if c["probs"]:
                c |= {"temp": "one", "dtype": "f32"}
        del c["name"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _spread(lo, hi, n):
    """n lengths between lo and hi, the longest among them, in no order."""
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(n)]


def _news(c):
    """Tokens (or drafts) of each sequence in this call."""
    n = c["K"] if c["op"] == "verify" else c["n"]
    least = 0 if c["op"] == "verify" else 1
    return [n if not c["ragged"] or b == 0 else max(least, int((n + 1) * ((b * 0.7548776662) % 1.0))) for b in range(c["B"])]


def work(c):
    news = _news(c)
    if c["op"] == "rope":
        values, turned = (sum(news) * (c["Hq"] + c["Hk"]) * d for d in (c["D"], c["rot"]))
        return {"bytes": 2 * values * DTYPES[c["dtype"]].itemsize, "flops": 3 * turned}
    if c["op"] == "blocks":
        lens = _spread(c["lo"], c["hi"], c["B"])
        touched = sum(-(-(N + n) // c["BT"]) - N // c["BT"] for N, n in zip(lens, news))
        # lengths in, counts and starts out; each touched entry read and written, and again where it is given back; 16 bytes of maps a token
        return {"bytes": 20 * c["B"] + touched * (8 if c["keep"] == "none" else 16) + 16 * sum(news), "flops": 0}
    size, V = DTYPES[c["dtype"]].itemsize, c["V"]
    rows = c["B"] if c["probs"] else sum(news) + c["B"]   # of probabilities, only the row that the next token comes from is read whole
    q = DTYPES[c["draft"]].itemsize if c["draft"] else 0  # and one row of the drafts'
    return {"bytes": (rows * size + c["B"] * (4 + q)) * V, "flops": (4 * rows + 3 * c["B"]) * V}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


ORIGINAL, FACTOR, LOW, HIGH = 8192, 32.0, 1.0, 32.0   # of a stretched context: trained length, stretch, and the turns between which it sets in


def _freq(c):
    """Angles a position adds to each pair, and what the rotated coordinates are multiplied by."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
    base = 10000.0
    if c["scaling"] == "ntk":
        base *= FACTOR ** (c["rot"] / (c["rot"] - 2))
    f = base ** (-i / c["rot"])
    if c["scaling"] == "linear":
        f = f / FACTOR
    if c["scaling"] == "parts":
        ramp = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * ((1 - ramp) / FACTOR + ramp)
        return f, 1.0 + 0.1 * math.log(FACTOR)
    return f, 1.0


def _rows_of(c, g, heads):
    """[B, heads, n, D] in 32 bits, token-major or head-major."""
    if c["source"] == "head":
        return torch.randn((c["B"], heads, c["n"], c["D"]), generator=g, device="cuda")
    return torch.randn((c["B"], c["n"], heads, c["D"]), generator=g, device="cuda").transpose(1, 2)


def _prepare_rope(c, s, g):
    dt = DTYPES[c["dtype"]]
    if c["source"] == "fused":  # queries, keys and values of one projection, as it leaves them
        whole = _rows_of(c, g, c["Hq"] + 2 * c["Hk"]).to(dt)
        s["q"], s["k"] = whole[:, :c["Hq"]], whole[:, c["Hq"]:c["Hq"] + c["Hk"]]
    else:
        s["q"], s["k"] = (_rows_of(c, g, h).to(dt) for h in (c["Hq"], c["Hk"]))
    for t in "qk":
        s[t + "_out"] = torch.randn(s[t].shape, generator=g, device="cuda").to(dt)
    starts = _spread(c["lo"], c["hi"], c["B"])
    s["starts"] = _i32(starts)
    s["positions"] = None
    if c["at"] == "positions":  # the same place twice among them, as where a prompt's parts share positions
        s["positions"] = s["starts"][:, None] + torch.randint(0, c["n"], (c["B"], c["n"]), generator=g, device="cuda", dtype=torch.int32)
    s["news"] = _i32(_news(c)) if c["ragged"] else None
    s["freq"], s["scale"] = _freq(c)
    if own:
        import turboquant_compressed_kv_tq_gb300 as tq
        if c["scaling"] == "parts":
            s["rope"] = tq.Rope.by_parts(c["rot"], FACTOR, ORIGINAL, low=LOW, high=HIGH, scale=s["scale"], interleaved=c["inter"])
        elif c["scaling"] == "none":
            s["rope"] = tq.Rope.of_base(c["rot"], interleaved=c["inter"])
        else:
            s["rope"] = (tq.Rope.linear if c["scaling"] == "linear" else tq.Rope.ntk)(c["rot"], FACTOR, interleaved=c["inter"])


def _prepare_blocks(c, s, g):
    B, BT = c["B"], c["BT"]
    lens, news = _spread(c["lo"], c["hi"], B), _news(c)
    width = max(-(-(N + c["n"]) // BT) for N in lens) + 1
    held = _i32([-(-N // BT) for N in lens])
    need = sum(-(-(N + n) // BT) - -(-N // BT) for N, n in zip(lens, news))
    free = max(1, (need * 9 // 10) if c["short"] else need + need // 4 + 7)
    total = int(held.sum()) + free
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    s["table"][torch.arange(width, device="cuda") < held[:, None]] = ids[free:]
    s["free"], s["used"] = ids[:free].contiguous(), _i32([0])
    s["lens"], s["news"], s["blocks"] = _i32(lens), _i32(news) if c["ragged"] else None, total
    s["tokens"] = sum(news)
    if c["keep"] == "part":
        s["keep"] = _i32([N + int((n + 1) * ((7 + b * 0.5698402910) % 1.0)) for b, (N, n) in enumerate(zip(lens, news))])
    else:
        s["keep"] = _i32(lens) if c["keep"] == "all" else None
    if own:
        import turboquant_compressed_kv_tq_gb300 as tq
        s["pages"] = tq.BlockTable.wrap(s["table"], s["free"], s["used"], BT, total)
        s["places"] = tq.Places(B, s["tokens"])


def _prepare_verify(c, s, g):
    B, K, V = c["B"], c["K"], c["V"]
    dt = DTYPES[c["dtype"]]
    s["temp"] = None
    t = torch.ones(B, device="cuda")
    if c["temp"] == "mixed":  # a third of the sequences greedy
        t = torch.where(torch.rand(B, generator=g, device="cuda") < 0.33, 0.0, 0.5 + torch.rand(B, generator=g, device="cuda"))
        s["temp"] = t
    elif c["temp"] == "greedy":
        t = torch.zeros(B, device="cuda")
    common = 4.0 * torch.randn((B, K + 1, V), generator=g, device="cuda")
    hot = torch.where(t > 0, t, 1.0)[:, None, None]
    guess = (common + 1.5 * torch.randn((B, K + 1, V), generator=g, device="cuda"))[:, :K]  # the drafting model's logits
    x = common + 1.5 * torch.randn((B, K + 1, V), generator=g, device="cuda")
    del common
    x[:, :, V // 3::97] = -math.inf  # tokens that the caller does not allow
    if c["probs"]:  # all but the likeliest tokens taken out, as a program that samples from few does
        x = torch.where(x >= x.topk(min(V, 64), -1).values[..., -1:], x, -math.inf)
        s["target"] = torch.softmax(x, -1).to(dt)
    else:
        s["target"] = x.to(dt)
    del x
    q = torch.softmax(guess / hot, -1)
    e = torch.empty_like(q).exponential_(generator=g).clamp_(min=1e-30)
    s["tokens"] = (q / e).argmax(-1).to(torch.int32) if K else None
    s["draft"] = q.to(DTYPES[c["draft"]]) if c["draft"] else None
    s["drafts"] = _i32(_news(c)) if c["ragged"] else None
    s["lens"] = torch.randint(10, 60000, (B,), generator=g, device="cuda", dtype=torch.int32)
    greedy = c["temp"] == "greedy"
    s["uniforms"] = torch.rand((B, K), generator=g, device="cuda") if K and not greedy else None
    s["noise"] = None if greedy else torch.empty((B, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    {"rope": _prepare_rope, "blocks": _prepare_blocks, "verify": _prepare_verify}[c["op"]](c, s, g)
    return s


# ------------------------------------------------------------------ the plain forms

def _rope_plain(s):
    c = s["case"]
    n, rot = c["n"], c["rot"]
    t = torch.arange(n, device="cuda")
    p = s["positions"] if s["positions"] is not None else s["starts"][:, None] + t
    a = p.double()[:, None, :, None] * s["freq"]  # far positions: 64 bits
    co, si = (torch.cos(a) * s["scale"]).float(), (torch.sin(a) * s["scale"]).float()
    if c["back"]:
        si = -si
    for name in "qk":
        x, out = s[name].float(), s[name + "_out"]
        y = x[..., :rot]
        u, w = (y[..., 0::2], y[..., 1::2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:])
        u, w = u * co - w * si, w * co + u * si
        y = torch.stack((u, w), -1).flatten(-2) if c["inter"] else torch.cat((u, w), -1)
        y = torch.cat((y, x[..., rot:]), -1).to(out.dtype)
        if s["news"] is not None:
            y = torch.where((t < s["news"][:, None])[:, None, :, None], y, out)
        out.copy_(y)


def _blocks_plain(s):
    c = s["case"]
    BT, table, width = c["BT"], s["table"], s["table"].shape[1]
    lens = s["lens"].long()
    news = s["news"].long() if s["news"] is not None else torch.full_like(lens, c["n"])
    first = lens // BT
    lb = first[:, None] + torch.arange((c["n"] - 1) // BT + 2, device="cuda")  # the blocks that new tokens can touch
    touched = lb < ((lens + news + BT - 1) // BT)[:, None]
    at = lb.clamp(max=width - 1)
    ids = torch.gather(table, 1, at)
    need = touched & (ids < 0)
    rank = need.flatten().long().cumsum(0).view(need.shape) - 1
    left = s["free"].numel() - s["used"].long()
    got = need & (rank < left)
    ids = torch.where(got, s["free"][(s["used"].long() + rank).clamp(0, s["free"].numel() - 1)], ids)
    table.scatter_(1, at, torch.where(touched, ids, torch.gather(table, 1, at)))
    s["used"] += got.sum().to(torch.int32)
    lack = touched & (ids < 0)
    stop = torch.where(lack, lb, width + 1).amin(1) * BT  # the first place without a block
    granted = torch.minimum(news, (stop - lens).clamp(min=0))
    starts = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), granted.cumsum(0)))
    i = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(starts[1:], i, right=True)
    there = i < starts[-1]
    b = torch.where(there, b, 0)
    pos = lens[b] + i - starts[b]
    slot = table[b, (pos // BT).clamp(0, width - 1)].long() * BT + pos % BT
    out = {"granted": granted.int(), "starts": starts.int(), "seq_ids": torch.where(there, b, -1).int(), "positions": torch.where(there, pos, 0).int(),
           "slots": torch.where(there, slot, -1)}
    if s["keep"] is not None:
        col = torch.arange(width, device="cuda")
        start = (s["keep"].long() + BT - 1) // BT
        behind = col >= start[:, None]
        gap = torch.where(behind & (table < 0), col, width).amin(1)
        back = behind & (col < gap[:, None])
        n = back.sum()
        where = s["used"].long() - n + back.flatten().long().cumsum(0).view(back.shape) - 1
        s["free"][where[back]] = table[back]
        table[back] = -1
        s["used"] -= n.to(torch.int32)
    return out | {"table": table, "free": s["free"], "used": s["used"]}


def _verify_plain(s):
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    x = s["target"].double()  # tokens are chosen where two numbers differ: 64 bits
    if c["probs"]:
        p, chance = x, x.log()
    else:
        t = torch.zeros(B, device="cuda") if s["noise"] is None else s["temp"] if s["temp"] is not None else torch.ones(B, device="cuda")
        t = t.double()[:, None, None]
        z = (x - x.amax(-1, keepdim=True)) / torch.where(t > 0, t, 1.0)
        w = torch.exp(z)
        total = w.sum(-1, keepdim=True)
        p, chance = w / total, z - total.log()  # a greedy sequence's chances are those at temperature 1
        p = torch.where(t > 0, p, (torch.arange(V, device="cuda") == x.argmax(-1, keepdim=True)).double())
    kept = torch.zeros(B, dtype=torch.long, device="cuda")
    one = torch.arange(V, device="cuda")
    if K:
        d = s["tokens"].long()
        pd = torch.gather(p[:, :K], 2, d[..., None])[..., 0]
        qd = torch.gather(s["draft"], 2, d[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(pd)
        u = s["uniforms"].double() if s["uniforms"] is not None else torch.zeros_like(pd)
        there = torch.arange(K, device="cuda") < (s["drafts"][:, None] if s["drafts"] is not None else K)
        kept = (there & (u * qd < pd)).long().cumprod(1).sum(1)
    rows = torch.arange(B, device="cuda")
    r = p[rows, kept]
    rest = r
    if K:
        last = kept >= (s["drafts"].long() if s["drafts"] is not None else K)
        at = kept.clamp(max=K - 1)
        q = s["draft"][rows, at].double() if s["draft"] is not None else (one == d[rows, at][:, None]).double()
        rest = (r - torch.where(last[:, None], 0.0, q)).clamp(min=0)
        rest = torch.where(rest.amax(1, keepdim=True) > 0, rest, r)
    nxt = (rest / (s["noise"].double() if s["noise"] is not None else 1.0)).argmax(-1)
    i = torch.arange(K + 1, device="cuda")
    tokens = torch.where(i == kept[:, None], nxt[:, None], -1)
    if K:
        tokens[:, :K] = torch.where(i[:K] < kept[:, None], d, tokens[:, :K])
    chance = torch.where(tokens >= 0, torch.gather(chance, 2, tokens.clamp(min=0)[..., None])[..., 0], 0.0)
    return {"accepted": kept.int(), "tokens": tokens.int(), "keep_lens": (s["lens"] + kept + 1).int(), "logprobs": chance.float()}


def run(s):
    c = s["case"]
    if c["op"] == "rope":
        if own:
            s["rope"].apply(s["q"], s["k"], out=s["q_out"], k_out=s["k_out"], starts=None if s["positions"] is not None else s["starts"],
                            positions=s["positions"], new_lens=s["news"], transposed=c["back"])
        else:
            _rope_plain(s)
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "blocks":
        if not own:
            return _blocks_plain(s)
        p = s["places"]
        s["pages"].reserve(s["lens"], s["news"], c["n"], places=p)
        if s["keep"] is not None:
            s["pages"].release(s["keep"])
        return {"granted": p.granted, "starts": p.starts, "seq_ids": p.seq_ids, "positions": p.positions, "slots": p.slots, "table": s["table"], "free": s["free"],
                "used": s["used"]}
    if not own:
        return _verify_plain(s)
    import turboquant_compressed_kv_tq_gb300 as tq
    accepted, tokens, keep, chances = tq.tq_verify_drafts(s["target"], s["tokens"], draft_probs=s["draft"], uniforms=s["uniforms"], noise=s["noise"], temperatures=s["temp"],
                                                 draft_lens=s["drafts"], seq_lens=s["lens"], target_probs=c["probs"])
    return {"accepted": accepted, "tokens": tokens, "keep_lens": keep, "logprobs": chances}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_rope(s):
    c = s["case"]
    rot = c["rot"]
    got = {}
    for name in "qk":
        out = s[name + "_out"].double().clone()
        for b, n in enumerate(_news(c)):
            p = s["positions"][b, :n].double() if s["positions"] is not None else int(s["starts"][b]) + torch.arange(n, device="cuda", dtype=torch.float64)
            x = s[name][b, :, :n].double()
            y = x[..., :rot]
            z = torch.complex(y[..., 0::2], y[..., 1::2]) if c["inter"] else torch.complex(y[..., :rot // 2], y[..., rot // 2:])
            turn = torch.polar(torch.full((1, 1), s["scale"], dtype=torch.float64, device="cuda"), p[:, None] * s["freq"])
            z = z * (turn.conj() if c["back"] else turn)
            y = torch.view_as_real(z).flatten(-2) if c["inter"] else torch.cat((z.real, z.imag), -1)
            out[b, :, :n] = torch.cat((y, x[..., rot:]), -1)
        got[name] = out
    return got


def _exact_blocks(s):
    """Row by row, block by block, as the definition goes."""
    c = s["case"]
    BT = c["BT"]
    table, free, used = s["table"].cpu().tolist(), s["free"].cpu().tolist(), 0
    granted, starts, seqs, places, slots = [], [0], [], [], []
    for b, (N, n) in enumerate(zip(s["lens"].tolist(), _news(c))):
        end = N + n
        for lb in range(N // BT, -(-(N + n) // BT)):
            if table[b][lb] < 0:
                if used < len(free):
                    table[b][lb] = free[used]
                    used += 1
                else:
                    end = min(end, max(N, lb * BT))
        granted.append(end - N)
        starts.append(starts[-1] + end - N)
        seqs += [b] * (end - N)
        places += range(N, end)
        slots += [table[b][p // BT] * BT + p % BT for p in range(N, end)]
    more = s["tokens"] - len(seqs)
    if s["keep"] is not None:
        back = []
        for b, k in enumerate(s["keep"].tolist()):
            lb = -(-k // BT)
            while lb < len(table[b]) and table[b][lb] >= 0:
                back.append(table[b][lb])
                table[b][lb] = -1
                lb += 1
        used -= len(back)
        free[used:used + len(back)] = back
    out = {"granted": granted, "starts": starts, "seq_ids": seqs + [-1] * more, "positions": places + [0] * more}
    return {k: _i32(v) for k, v in out.items()} | {"slots": torch.tensor(slots + [-1] * more, dtype=torch.int64, device="cuda"), "table": _i32(table),
                                                   "free": _i32(free), "used": _i32([used])}


def _exact_verify(s):
    c = s["case"]
    V = c["V"]
    accepted, tokens, logs = [], [], torch.zeros((c["B"], c["K"] + 1), dtype=torch.float64, device="cuda")
    for b, k in enumerate(_news(c)):
        T = 0.0 if s["noise"] is None else 1.0 if s["temp"] is None else float(s["temp"][b])

        def chances(i):
            x = s["target"][b, i].double()
            if c["probs"]:
                return x
            if T <= 0:
                return torch.nn.functional.one_hot(x.argmax(), V).double()
            return torch.softmax(x / T, 0)

        got = []
        for i in range(k + 1):
            p = chances(i)
            if i < k:
                d = int(s["tokens"][b, i])
                q = s["draft"][b, i].double() if s["draft"] is not None else torch.nn.functional.one_hot(torch.tensor(d, device="cuda"), V).double()
                u = 0.0 if s["uniforms"] is None else float(s["uniforms"][b, i])
                if u * float(q[d]) < float(p[d]):
                    got.append(d)
                    continue
                rest = torch.clamp(p - q, min=0)
                p = rest if bool((rest > 0).any()) else p
            break
        accepted.append(len(got))  # the next token is not one of them
        race = p if s["noise"] is None else p / s["noise"][b].double()
        got.append(int(race.argmax()))
        for i, token in enumerate(got):
            x = s["target"][b, i].double()
            logs[b, i] = x[token].log() if c["probs"] else torch.log_softmax(x / (T if T > 0 else 1.0), 0)[token]
        tokens.append(got + [-1] * (c["K"] + 1 - len(got)))
    accepted = _i32(accepted)
    return {"accepted": accepted, "tokens": _i32(tokens).view(c["B"], c["K"] + 1), "keep_lens": s["lens"] + accepted + 1, "logprobs": logs}


def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "blocks": _exact_blocks, "verify": _exact_verify}[c["op"]](s)
