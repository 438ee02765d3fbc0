"""The 8-bit cache's operators, as they are measured: appending with the position rotation, and attention over the
cache for single tokens and for chunks of a prompt.

The cache is paged. A block holds `BT` tokens of one sequence for every KV head, as 8-bit codes [block][head][token][dim]
(e4m3 or int8), keys and values apart, and one power-of-two scale 2^(x - 127) for each block and head, held as the byte x.
`own` chooses between the plain torch form and the framework's calls."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ the cases

def _append(name, **kw):
    return {"name": name, "op": "append", "fmt": "e4m3", "rot": kw["D"], "inter": False, "ragged": False, "major": "head", **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend", "fmt": "e4m3", "dtype": "bf16", "rope": False, "cap": 0.0, "bias": False, "window": 0, "prefix": 0, "doc": 0,
            "ragged": False, **kw}


def listed():
    return [
        # one decoding step's new tokens of a continuous batch, straight from a fused projection (token-major)
        _append("append step", dtype="bf16", B=32, H=8, D=128, BT=16, n=1, lo=120, hi=1000, major="token"),
        # a prompt chunk of one long sequence that does not start on a block's border
        _append("append chunk", dtype="bf16", B=1, H=8, D=128, BT=64, n=8192, lo=1001, hi=1001),
        # a padded batch of prompts of several lengths, half of each head rotated, neighbouring pairs
        _append("append ragged", dtype="f16", B=12, H=4, D=64, BT=32, n=777, lo=3, hi=500, rot=32, inter=True, ragged=True, major="token"),
        # several prompts at once with wide heads, in 32 bits
        _append("append wide", dtype="f32", B=6, H=4, D=256, BT=128, n=4096, lo=0, hi=130),
        # the smallest call: one token of one short sequence, wide heads
        _attend("decode short", B=1, H=2, G=8, D=256, BT=64, q=1, lo=512, hi=512, fmt="int8", rope=True),
        # continuous batching: ragged sequences through 16-token blocks, one token each
        _attend("decode batch", B=32, H=8, G=4, D=128, BT=16, q=1, lo=4096, hi=32768, rope=True),
        # two speculative tokens of one very long sequence
        _attend("decode long", B=1, H=8, G=8, D=128, BT=256, q=2, lo=262144, hi=262144),
        # a layer with a sliding window whose scores are capped, the first tokens kept as sinks
        _attend("decode window", dtype="f16", B=24, H=4, G=4, D=64, BT=32, q=1, lo=5000, hi=32749, window=4096, prefix=4, cap=30.0, rope=True, fmt="int8"),
        # a short prompt, wide heads, scores capped
        _attend("prompt short", B=2, H=2, G=4, D=256, BT=64, q=333, lo=333, hi=500, cap=50.0, rope=True),
        # a prompt's chunk behind what is already in the cache
        _attend("prompt chunk", B=1, H=8, G=4, D=128, BT=256, q=4096, lo=12288, hi=12288, rope=True),
        # packed documents with a bias that falls with the distance
        _attend("prompt documents", dtype="f16", B=3, H=8, G=1, D=64, BT=128, q=2111, lo=2111, hi=2111, doc=517, bias=True, fmt="int8"),
        # a padded batch of prompts that see their prefix whole
        _attend("prompt prefix", B=4, H=4, G=8, D=128, BT=16, q=700, lo=700, hi=1900, prefix=611, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges, no dearer than the largest listed one."""
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        D = rng.choice([64, 128, 128, 256])
        kind = rng.choice(["append", "decode", "prompt"])
        c = {"D": D, "BT": rng.choice([16, 32, 64, 128, 256]), "H": rng.choice([1, 2, 4, 8])}
        if kind == "append":
            n = rng.choice([1, 1, 2, 5, _log(rng, 3, 8192)])
            lo = _log(rng, 1, 3000) - 1
            c = _append("", dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), B=_log(rng, 1, 32), n=n, lo=lo, hi=lo + rng.randrange(0, 1000),
                        **c) | {"rot": rng.choice([0, D // 4, D // 2, D, D]), "inter": rng.random() < 0.3, "ragged": rng.random() < 0.3,
                                "major": rng.choice(["head", "token"])}
        else:
            few = kind == "decode"
            G = rng.choice([1, 2, 4, 8, 6] if few else [1, 2, 4, 8])
            q = rng.choice([1, 1, 1, 2, 4]) if few else _log(rng, 33, 4096)
            lo = _log(rng, max(q, 16), 100000 if few else 3 * max(q, 16))
            c = _attend("", dtype=rng.choice(["bf16", "bf16", "f16"]), B=_log(rng, 1, 32 if few else 6), G=G, q=q, lo=lo,
                        hi=lo + rng.randrange(0, 1 + (lo if few else lo // 2)), **c)
            c |= {"fmt": rng.choice(["e4m3", "int8"]), "rope": rng.random() < 0.6, "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "bias": rng.random() < 0.25,
                  "window": rng.choice([0, 0, 0, _log(rng, 100, 8192)]), "prefix": rng.choice([0, 0, rng.randrange(1, 200)]),
                  "doc": 0 if few else rng.choice([0, 0, _log(rng, 50, 2000)]), "ragged": not few and rng.random() < 0.3}
        del c["name"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and c.get("B") * c.get("q", 0) * c.get("H") * c.get("G", 0) * c["hi"] < 1.7e9 \
                and c["B"] * c["H"] * c["D"] * (c["hi"] + c.get("n", 0)) < 1.1e9:
            return c


def _spread(lo, hi, n):
    """n lengths between lo and hi, the longest among them, in no order."""
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(n)]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["B"])


def _news(c):
    """Tokens (or queries) of each sequence in this call."""
    n = c["n"] if c["op"] == "append" else c["q"]
    return [n if not c["ragged"] or b == 0 else max(1, n - (b * n) // (c["B"] + 1)) for b in range(c["B"])]


def _seen(c, N, nq):
    """How many keys the queries of a sequence see, each, by arithmetic over the positions."""
    p = torch.arange(N - nq, N, dtype=torch.int64)
    lo = torch.zeros_like(p)
    if c["window"]:
        lo = torch.maximum(lo, p - c["window"] + 1)
    if c["doc"]:
        lo = torch.maximum(lo, p // c["doc"] * c["doc"])
    P = min(c["prefix"], N)
    both = torch.minimum(p + 1, torch.full_like(p, P)) - torch.minimum(lo, torch.full_like(p, P))
    return p - lo + 1 + P - torch.clamp(both, min=0), lo, P


def work(c):
    if c["op"] == "append":
        size = DTYPES[c["dtype"]].itemsize
        values = sum(_news(c)) * c["H"] * c["D"] * 2
        return {"bytes": values * (size + 1), "flops": 3 * values}
    flops = keys = 0
    for N, nq in zip(_lens(c), _news(c)):
        seen, lo, P = _seen(c, N, nq)
        flops += 4 * int(seen.sum()) * c["D"] * c["G"] * c["H"]
        keys += N - int(lo.min()) + max(0, min(P, int(lo.min())))
    rows = sum(_news(c)) * c["G"] * c["H"]
    return {"bytes": keys * c["H"] * c["D"] * 2 + rows * c["D"] * 4, "flops": flops}


# ------------------------------------------------------------------ inputs

def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _pool(c, blocks, g):
    """A cache of normally distributed keys or values, each head with a spread of its own: codes and scale bytes."""
    codes = torch.empty((blocks, c["H"], c["BT"], c["D"]), dtype=torch.uint8, device="cuda")
    exps = torch.empty((blocks, c["H"]), dtype=torch.uint8, device="cuda")
    spread = 0.5 + 1.5 * torch.rand((1, c["H"], 1, 1), generator=g, device="cuda")
    step = max(1, (1 << 27) // (c["H"] * c["BT"] * c["D"]))
    for i in range(0, blocks, step):
        x = _normal(codes[i:i + step].shape, g) * spread
        e = _exponent(x.abs().amax((2, 3)), c["fmt"])
        exps[i:i + step] = (e + 127).to(torch.uint8)
        codes[i:i + step] = _codes(x * torch.exp2(-e.float())[:, :, None, None], c["fmt"])
    return codes, exps


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, B, H, D, BT = DTYPES[c["dtype"]], c["B"], c["H"], c["D"], c["BT"]
    lens, news = _lens(c), _news(c)
    ends = [N + n for N, n in zip(lens, news)] if c["op"] == "append" else lens
    width = max(N // BT for N in lens) + ((c["n"] - 1) // BT if c["op"] == "append" else 0) + 2
    blocks = B * width if c["op"] == "append" else sum(-(-e // BT) for e in ends)
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    if c["op"] == "append":
        table = order.view(B, width)
    else:  # entries behind a sequence's last block are unused
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, e in enumerate(ends):
            k = -(-e // BT)
            table[b, :k] = order[at:at + k]
            at += k
    s = {"case": c, "table": table, "width": width, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "ends": max(ends),
         "news": torch.tensor(news, dtype=torch.int32, device="cuda") if c["ragged"] else None}
    s["kc"], s["kx"] = _pool(c, blocks, g)
    s["vc"], s["vx"] = _pool(c, blocks, g)
    rot = c["rot"] if c["op"] == "append" else D if c["rope"] else 0
    s["rot"] = rot
    s["freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    if c["op"] == "append":
        shape = (B, c["n"], H, D) if c["major"] == "token" else (B, H, c["n"], D)
        for t in "kv":
            x = _normal(shape, g, 1.5).to(dt)
            s[t] = x.transpose(1, 2) if c["major"] == "token" else x
    else:
        s["q"] = _normal((B, c["q"], H * c["G"], D), g, 1.25).to(dt).transpose(1, 2)
        s["out"] = _normal((B, c["q"], H * c["G"], D), g).to(dt).transpose(1, 2)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H * c["G"] + 1, device="cuda") / (H * c["G"])).float() if c["bias"] else None
        s["prefix"] = torch.tensor([min(c["prefix"], N) for N in lens], dtype=torch.int32, device="cuda") if c["prefix"] else None
        if c["doc"]:
            p = s["lens"][:, None] - torch.tensor(news, dtype=torch.int32, device="cuda")[:, None] + torch.arange(c["q"], dtype=torch.int32, device="cuda")
            s["docs"] = (p // c["doc"] * c["doc"]).to(torch.int32).contiguous()
        else:
            s["docs"] = None
    if own:  # the handle that a program keeps, and its workspace
        import turboquant_compressed_kv_tq_gb300 as tq
        s["cache"] = tq.KV8Cache.wrap(s["kc"], s["vc"], s["kx"], s["vx"], tq.TQ_KV8_E4M3 if c["fmt"] == "e4m3" else tq.TQ_KV8_INT8)
        s["rope"] = tq.Rope(s["freq"], interleaved=c.get("inter", False)) if rot else None
        if c["op"] == "attend":
            s["ws"] = torch.empty(s["cache"].workspace_bytes(B, H * c["G"], c["q"], s["ends"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _exponent(top, fmt):
    """The smallest e in [-63, 63] with top / 2^e at most the format's largest code."""
    m, x = torch.frexp(top)  # top = m 2^x, m in [0.5, 1)
    limit, shift = (0.875, 9) if fmt == "e4m3" else (127 / 128, 7)
    e = x - shift + (m > limit).to(x.dtype)
    return torch.where(top > 0, e, -63).clamp(-63, 63)


def _codes(x, fmt):
    if fmt == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).to(torch.int8).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _rotated(x, pos, freq, rot, inter):
    """x [B, heads, n, D] in 32 bits, pos [B, n]."""
    if not rot:
        return x
    a = pos.double()[:, None, :, None] * freq
    co, si = torch.cos(a).float(), torch.sin(a).float()
    y = x[..., :rot]
    u, w = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :rot // 2], y[..., rot // 2:])
    u, w = u * co - w * si, w * co + u * si
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _append_one(s, x, codes, exps, rot):
    c = s["case"]
    B, H, D, BT, n, fmt = c["B"], c["H"], c["D"], c["BT"], c["n"], c["fmt"]
    lens = s["lens"].long()
    news = s["news"].long() if s["news"] is not None else torch.full_like(lens, n)
    x = _rotated(x.float(), lens[:, None] + torch.arange(n, device=x.device), s["freq"], rot, c["inter"])
    nb = (n - 1) // BT + 2
    first = lens // BT
    phys = torch.gather(s["table"].long(), 1, first[:, None] + torch.arange(nb, device=x.device))
    at = (first[:, None] * BT + torch.arange(nb * BT, device=x.device)).view(B, nb, BT)  # positions of the touched blocks' slots
    i = at - lens[:, None, None]
    new = (i >= 0) & (i < news[:, None, None])
    y = torch.gather(x, 2, i.clamp(0, n - 1).view(B, 1, nb * BT, 1).expand(B, H, nb * BT, D)).view(B, H, nb, BT, D).transpose(1, 2)
    y = torch.where(new[:, :, None, :, None], y, 0.0)
    e = _exponent(y.abs().amax((3, 4)), fmt)
    before = exps[phys].int() - 127  # [B, nb, H]
    held = (at[:, :, 0] < lens[:, None])[:, :, None]
    e = torch.where(held, torch.maximum(before, e), e)
    was = codes[phys]
    moved = _codes(_values(was, fmt) * torch.exp2((before - e).clamp(-140, 0).float())[..., None, None], fmt)
    old = (at < lens[:, None, None])[:, :, None, :, None]
    fresh = _codes(y * torch.exp2(-e.float())[..., None, None], fmt)
    touched = new.any(2)[:, :, None]
    now = torch.where(new[:, :, None, :, None], fresh, torch.where(old & touched[..., None, None], moved, was))
    x_now = torch.where(touched, (e + 127).to(torch.uint8), exps[phys])
    codes[phys] = now
    exps[phys] = x_now


def _attend_plain(s):
    c = s["case"]
    B, H, G, D, BT, L, fmt = c["B"], c["H"], c["G"], c["D"], c["BT"], c["q"], c["fmt"]
    T = s["width"] * BT
    at = s["table"].long().clamp(min=0)
    t = torch.arange(T, device=at.device)
    lens = s["lens"].long()
    inside = (t < lens[:, None])[:, None, :, None]

    def whole(codes, exps):
        x = _values(codes[at], fmt) * torch.exp2(exps[at].float() - 127.0)[..., None, None]  # [B, width, H, BT, D]
        return torch.where(inside, x.transpose(1, 2).reshape(B, H, T, D), 0.0)

    news = s["news"].long() if s["news"] is not None else torch.full_like(lens, L)
    p = (lens - news)[:, None] + torch.arange(L, device=at.device)  # [B, L]
    q = _rotated(s["q"].float(), p, s["freq"], s["rot"], False).reshape(B, H, G * L, D)
    x = torch.matmul(q, whole(s["kc"], s["kx"]).transpose(2, 3)).view(B, H, G, L, T) * (1.0 / math.sqrt(D))
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    far = p[:, :, None] - t
    if c["bias"]:
        x = x - s["slopes"].view(1, H, G, 1, 1) * far.abs().float()[:, None, None]
    see = far >= 0
    if c["window"]:
        see &= far < c["window"]
    if c["doc"]:
        see &= t >= s["docs"].long()[:, :, None]
    if c["prefix"]:
        see |= t < s["prefix"].long()[:, None, None]
    see &= t < lens[:, None, None]
    x = torch.where(see[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, H, G * L, T), whole(s["vc"], s["vx"])).view(B, H, G, L, D)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0).view(B, H * G, L, D).to(s["out"].dtype)
    rows = (torch.arange(L, device=at.device) < news[:, None])[:, None, :, None]
    s["out"].copy_(torch.where(rows, o, s["out"]))


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["cache"].append(0, s["k"], s["v"], s["lens"], s["table"], s["width"], new_lens=s["news"], rope=s["rope"])
        else:
            _append_one(s, s["k"], s["kc"], s["kx"], s["rot"])
            _append_one(s, s["v"], s["vc"], s["vx"], 0)
        f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        return {"k": s["kc"].view(f8), "k_scale": s["kx"].view(e8), "v": s["vc"].view(f8), "v_scale": s["vx"].view(e8)}
    if own:
        s["cache"].attention(0, s["q"], s["lens"], s["table"], s["width"], s["ends"], out=s["out"], workspace=s["ws"], q_lens=s["news"], softcap=c["cap"],
                             slopes=s["slopes"], window=c["window"], prefix_lens=s["prefix"], doc_starts=s["docs"], rope=s["rope"])
    else:
        _attend_plain(s)
    return s["out"]


# ------------------------------------------------------------------ from the definition, in 64 bits

def _e4m3_64(x):
    """The e4m3 value nearest to x, ties to the even one: 3 bits behind the leading one, multiples of 2^-9 below 2^-6."""
    unit = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
    return torch.round(x / unit) * unit


def _turn64(x, pos, freq, inter):
    """x [heads, n, rot] as complex pairs, turned by pos * freq."""
    half = x.shape[-1] // 2
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if inter else torch.complex(x[..., :half], x[..., half:])
    a = pos.double()[:, None] * freq
    z = z * torch.polar(torch.ones_like(a), a)
    return torch.view_as_real(z).flatten(-2) if inter else torch.cat((z.real, z.imag), -1)


def _exact_append(s):
    c = s["case"]
    BT, rot = c["BT"], s["rot"]
    lens, news = _lens(c), _news(c)
    got = {}
    for name, x, codes, exps in (("k", s["k"], s["kc"], s["kx"]), ("v", s["v"], s["vc"], s["vx"])):
        v = codes.view(torch.float8_e4m3fn).double()
        sc = torch.exp2(exps.double() - 127.0)
        for b, (N, n) in enumerate(zip(lens, news)):
            y = x[b, :, :n].double()
            if name == "k" and rot:
                y = torch.cat((_turn64(y[..., :rot], torch.arange(N, N + n, device=y.device), s["freq"], c["inter"]), y[..., rot:]), -1)
            front, back = N % BT, -(N + n) % BT
            nb = (front + n + back) // BT
            ids = s["table"][b, N // BT:N // BT + nb].long()
            y = torch.nn.functional.pad(y, (0, 0, front, back)).view(c["H"], nb, BT, -1).transpose(0, 1)
            here = torch.arange(nb * BT, device=y.device).view(nb, 1, BT, 1)
            ratio = (y.abs().amax((2, 3)) / TOP["e4m3"]).clamp(min=2.0 ** -63, max=2.0 ** 63)
            scale = torch.exp2(torch.ceil(torch.log2(ratio)))
            scale = torch.where(scale / 2 >= ratio, scale / 2, torch.where(scale < ratio, scale * 2, scale))
            if front:
                scale[0] = torch.maximum(scale[0], sc[ids[0]])
            blk = v[ids]
            blk = torch.where(here < front, _e4m3_64(blk * (sc[ids] / scale)[..., None, None]) if front else blk, blk)
            v[ids] = torch.where((here >= front) & (here < front + n), _e4m3_64(y / scale[..., None, None]), blk)
            sc[ids] = scale
        got[name], got[name + "_scale"] = v, sc
    return got


def _exact_attend(s):
    c = s["case"]
    H, G, D, BT = c["H"], c["G"], c["D"], c["BT"]
    out = s["out"].double().clone()
    kind = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8
    for b, (N, nq) in enumerate(zip(_lens(c), _news(c))):
        ids = s["table"][b, :-(-N // BT)].long()
        _, lo, P = _seen(c, N, nq)
        p = torch.arange(N - nq, N, device=ids.device)
        t = torch.arange(N, device=ids.device)
        see = ((t <= p[:, None]) & (t >= lo.to(ids.device)[:, None])) | (t < P)
        for h in range(H):
            k, v = ((codes[ids, h].view(kind).double() * torch.exp2(exps[ids, h].double() - 127.0)[:, None, None]).view(-1, D)[:N]
                    for codes, exps in ((s["kc"], s["kx"]), (s["vc"], s["vx"])))
            q = s["q"][b, h * G:(h + 1) * G, :nq].double()
            if s["rot"]:
                q = torch.cat((_turn64(q[..., :s["rot"]], p, s["freq"], False), q[..., s["rot"]:]), -1)
            x = q @ k.T / math.sqrt(D)
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if c["bias"]:
                x = x - s["slopes"][h * G:(h + 1) * G].double()[:, None, None] * (p[:, None] - t).abs()
            out[b, h * G:(h + 1) * G, :nq] = torch.softmax(x.masked_fill(~see, -math.inf), -1) @ v
    return out


def exact(c, seed):
    s = prepare(c, seed)
    return _exact_append(s) if c["op"] == "append" else _exact_attend(s)
