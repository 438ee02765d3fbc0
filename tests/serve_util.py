"""Plain definitions of the calls around the caches': block tables on Python integers, rotation and verification in 64 bits."""
import math

import torch


def reserve(table, free, used, lens, news, n_new, BT, num_blocks, max_tokens):
    """On lists, changed in place: (used, granted, starts, seq_ids, positions, slots, error words)."""
    width = len(table[0]) if table else 1
    err = set()
    if not 0 <= used <= len(free):
        err.add("capacity")
        used = len(free)
    granted, starts, seqs, pos, slots = [], [0], [], [], []
    taken = []
    for b, N in enumerate(lens):
        n = n_new if news is None else news[b]
        if not 0 <= n <= n_new:
            err.add("seqlen")
            n = min(max(n, 0), n_new)
        if not 0 <= N <= width * BT:
            err.add("seqlen")
            N, n = 0, 0
        if N + n > width * BT:
            err.add("capacity")
            n = width * BT - N
        end = N + n
        for lb in range(N // BT, -(-(N + n) // BT) if n else 0):
            if lb * BT >= end and end < N + n:
                break
            if table[b][lb] < 0:
                if used == len(free):
                    err.add("capacity")
                    end = max(N, lb * BT)
                    break
                table[b][lb] = free[used]
                used += 1
            if not 0 <= table[b][lb] < num_blocks:
                err.add("block")
        granted.append(end - N)
        starts.append(starts[-1] + end - N)
        for p in range(N, end):
            seqs.append(b)
            pos.append(p)
            id = table[b][p // BT]
            slots.append(id * BT + p % BT if 0 <= id < num_blocks else -1)
    if max_tokens and len(seqs) > max_tokens:
        err.add("capacity")
    more = max(0, max_tokens - len(seqs))
    cut = slice(0, max_tokens)
    return used, granted, starts, seqs[cut] + [-1] * more, pos[cut] + [0] * more, slots[cut] + [-1] * more, err


def release(table, free, used, keeps, BT, num_blocks):
    """(used, error words)."""
    err, back = set(), []
    if not 0 <= used <= len(free):
        err.add("capacity")
        used = min(max(used, 0), len(free))
    for b, keep in enumerate(keeps):
        if keep < 0:
            err.add("seqlen")
            continue
        for lb in range(-(-keep // BT), len(table[b])):
            if table[b][lb] < 0:
                break
            if table[b][lb] < num_blocks:
                back.append(table[b][lb])
            else:
                err.add("block")
            table[b][lb] = -1
    if len(back) > used:
        err.add("capacity")
        back = back[len(back) - used:]
    free[used - len(back):used] = back
    return used - len(back), err


def rotated(x, pos, inv_freq, inter=False, scale=1.0, back=False):
    """x [B, heads, n, D] fp64 with its first 2 len(inv_freq) coordinates turned; pos [B, n]."""
    rot = 2 * inv_freq.numel()
    if rot == 0:
        return x
    y = x[..., :rot]
    u, w = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :rot // 2], y[..., rot // 2:])
    a = pos.double()[:, None, :, None] * inv_freq
    co, si = torch.cos(a) * scale, torch.sin(a) * scale * (-1 if back else 1)
    u, w = u * co - w * si, w * co + u * si
    y = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((y, x[..., rot:]), -1)


def rotation_bound(x, ref, pos, inv_freq, dtype, inter=False, scale=1.0):
    """How far a rotated row may be from `ref`. cos and sin are off by 2^-23 and rounded with the scale (2^-24), each product and
    the sum by 2^-24: below 2^-21 scale (|u| + |w|) together; the angle by p (2^-64 + |f| 2^-54) turns, and the
    reference's own by 2^-53 of itself; the output is rounded once, by half a step (2^-25 below fp16's normal numbers)."""
    rot = 2 * inv_freq.numel()
    bound = ref.abs() * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    if rot == 0:
        return bound
    y = x[..., :rot].abs()
    m = y[..., 0::2] + y[..., 1::2] if inter else y[..., :rot // 2] + y[..., rot // 2:]
    far = pos.double().abs()[:, None, :, None] * (2 * math.pi * 2.0 ** -64 + inv_freq.abs() * (2 * math.pi * 2.0 ** -54 + 2.0 ** -53))
    e = m * scale * (2.0 ** -21 + far) * (1 + 2.0 ** -7)   # (of a value that is then rounded: half a step of it more)
    e = torch.stack((e, e), -1).flatten(-2) if inter else torch.cat((e, e), -1)
    bound[..., :rot] += e
    return bound


NEAR = 2.0 ** -18   # numbers nearer than this (relative) may be told apart either way: weights, sum and quotient are each good to 2^-20


def check_verified(target, drafts, q, u, noise, temps, lens, probs, seq_lens, got):
    """Every sequence of a verification against its definition in 64 bits; what is nearer than NEAR may go either way."""
    B, R, V = target.shape
    K = R - 1
    target = target.double().cpu()
    drafts, q, u, noise, temps, lens = (None if x is None else x.cpu() for x in (drafts, q, u, noise, temps, lens))
    accepted, tokens, logs = got.accepted.cpu(), got.tokens.cpu(), got.logprobs.double().cpu()
    if seq_lens is not None:
        assert torch.equal(got.keep_lens.cpu(), seq_lens.cpu() + accepted + 1)
    for b in range(B):
        k = K if lens is None else min(max(int(lens[b]), 0), K)
        T = 0.0 if noise is None else 1.0 if temps is None else float(temps[b])
        T = T if T > 0 else 0.0
        n = int(accepted[b])
        assert 0 <= n <= k, (b, n, k)

        def row(i):
            """(chances that decide, chances that are reported as logs)."""
            x = target[b, i]
            if probs:
                x = torch.where(x == x, x, 0.0)
                one = torch.zeros(V, dtype=torch.float64)
                if T == 0 and bool((x > 0).any()):
                    one[x.argmax()] = 1.0
                return (one if T == 0 else x), x.log()
            x = torch.where(x == x, x, -math.inf).clamp(max=torch.finfo(torch.float32).max)
            if x.max() == -math.inf:
                return torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
            z = (x - x.max()) / (min(max(T, 2.0 ** -120), 2.0 ** 100) if T else 1.0)
            z = z - torch.exp(z).sum().log()
            if T:
                return torch.exp(z), z
            one = torch.zeros(V, dtype=torch.float64)
            one[x.argmax()] = 1.0
            return one, z

        def drawn(i):
            d = int(drafts[b, i])
            if q is not None:
                return q[b, i].double()
            one = torch.zeros(V, dtype=torch.float64)
            if 0 <= d < V:
                one[d] = 1.0
            return one

        for i in range(min(n + 1, k)):
            d = int(drafts[b, i])
            assert int(tokens[b, i]) == d or i == n
            p, _ = row(i)
            if not 0 <= d < V:
                assert i == n
                continue
            limit = float(u[b, i]) * float(drawn(i)[d]) if T else 0.5
            if abs(limit - float(p[d])) > NEAR * float(p[d]):
                assert (limit < float(p[d])) == (i < n), (b, i, limit, float(p[d]))
        p, _ = row(n)
        next_ = int(tokens[b, n])
        rest = (p - drawn(n)).clamp(min=0) if n < k and T else p
        if not bool((rest > 0).any()):
            rest = p
        if not bool((rest > 0).any()):
            assert next_ == -1
        else:
            e = torch.ones(V, dtype=torch.float64) if noise is None or not T else noise[b].double()
            e = torch.where(e == e, e, 0.0).clamp(min=2.0 ** -100)
            score = rest / e
            # where a residual is small next to its p, the p's rounding counts
            slack = (rest + NEAR * p) / e
            assert slack[next_] >= score.max() * (1 - NEAR), (b, next_, int(score.argmax()))
            if not T:
                assert next_ == int(rest.argmax())
        assert tokens[b, n + 1:].eq(-1).all()
        for i in range(K + 1):
            t = int(tokens[b, i])
            if t < 0:
                assert logs[b, i] == 0
                continue
            want = float(row(i)[1][t])
            assert logs[b, i] == want or abs(float(logs[b, i]) - want) <= 2.0 ** -20 + 2.0 ** -23 * abs(want), (b, i, float(logs[b, i]), want)
