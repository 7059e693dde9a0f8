"""Plain forms of the paged-cache operators for the tests: the plan in Python
integers, the attention in fp64 on the host, with its error bound."""
import math

import torch

BF16_HALF = 2.0 ** -8      # half a step of bfloat16, relative
F32_HALF = 2.0 ** -24


def pages(tokens, page):
    return -(-tokens // page)


def plan(lens, fresh, pool, ring, table, page, max_tokens):
    """(lens, pool, starts, slots, ring, table, fault) after a step; fault is
    None, "pages" or "invalid"."""
    ring, table = list(ring), [list(r) for r in table]
    n, cap, rows = len(lens), len(ring), len(table[0])
    head, free = pool
    same = (list(lens), [head, free], [0] * (n + 1), [-1] * max_tokens, ring, table)
    tokens = sum(max(f, 0) for f in fresh)
    if not (0 <= head < cap and 0 <= free) or tokens > max_tokens:
        return (*same, "invalid")
    for i in range(n):
        if lens[i] < 0 or fresh[i] < -1 or pages(lens[i] + max(fresh[i], 0), page) > rows:
            return (*same, "invalid")
    have = [pages(x, page) for x in lens]
    need = [pages(x + max(f, 0), page) - h for x, f, h in zip(lens, fresh, have)]
    back = [h if f < 0 else 0 for h, f in zip(have, fresh)]
    if free + sum(back) > cap:
        return (*same, "invalid")
    if sum(need) > free:
        return (*same, "pages")
    tail = head + free
    for i in range(n):
        for j in range(back[i]):
            ring[tail % cap] = table[i][j]
            tail += 1
    at = head
    for i in range(n):
        for j in range(need[i]):
            table[i][have[i] + j] = ring[at % cap]
            at += 1
    starts, slots, out, fault = [0], [], [], None
    for i in range(n):
        for t in range(lens[i], lens[i] + max(fresh[i], 0)):
            p = table[i][t // page]
            good = 0 <= p < cap
            slots.append(p * page + t % page if good else -1)
            fault = fault if good else "invalid"
        starts.append(len(slots))
        out.append(0 if fresh[i] < 0 else lens[i] + fresh[i])
    slots += [-1] * (max_tokens - len(slots))
    return (out, [(head + sum(need)) % cap, free - sum(need) + sum(back)], starts, slots, ring,
            table, fault)


def decode(Q, k_pages, v_pages, table, lens):
    """fp64 attention of one token per request: (O, lse, bound of O's error,
    bound of lse's error) for a kernel that sums in fp32, with the weights
    rounded to bf16 when the tensors are bf16 and O rounded to its type."""
    Q, kp, vp = (x.detach().cpu().double() for x in (Q, k_pages, v_pages))
    half = BF16_HALF if k_pages.dtype == torch.bfloat16 else F32_HALF
    weights = BF16_HALF if k_pages.dtype == torch.bfloat16 else 0.0
    n, hq, d = Q.shape
    N, hkv, page, _ = kp.shape
    g = hq // hkv
    O = torch.zeros(n, hq, d, dtype=torch.float64)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(O), torch.zeros(n, hq, dtype=torch.float64)
    for i in range(n):
        size = min(max(int(lens[i]), 0), table.shape[1] * page)
        t = torch.arange(size)
        row = table[i].cpu().long()[t // page]
        ok = (row >= 0) & (row < N)
        t, row = t[ok], row[ok]
        if t.numel() == 0:
            continue
        k, v = kp[row, :, t % page], vp[row, :, t % page]        # [T, hkv, d]
        for h in range(hq):
            kk, vv = k[:, h // g], v[:, h // g]
            s = kk @ Q[i, h] / math.sqrt(d)
            lse[i, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[i, h])
            # a token that weighs nothing in fp64 weighs nothing in fp32, whatever its logit
            size_s = (kk[p > 0].abs() @ Q[i, h].abs() / math.sqrt(d)).max().item()
            O[i, h] = p @ vv
            A = p @ vv.abs()
            # logits: d products and sums, a scale and a base-2 logarithm's factor, each a
            # step of 2^-23 at most of a value no larger than size_s (a tensor core's sums
            # may cut instead of rounding); a weight is off by the exponential's 2^-21 more
            ds = (d + 6) * 2.0 ** -23 * size_s
            # T weights are summed, and up to 64 partial sums joined, in fp32
            sums = (t.numel() + 64) * 2.0 ** -23
            tol[i, h] = A * (weights + 2 * ds + sums + 2.0 ** -20)
            tol[i, h] += half * (O[i, h].abs() + tol[i, h]) + 1e-30
            tol_lse[i, h] = ds + sums + 2.0 ** -20 + 2.0 ** -22 * abs(lse[i, h])
    return O, lse, tol, tol_lse
