"""Cases of the paged-cache operators: plan, append and decode.

``prepare`` makes the inputs of a case on the GPU from a seed, ``run`` makes one
pass, in plain torch operations or, where ``own`` is true, through the package's
calls, and ``exact`` gives the same outputs from the definition in 64 bits.

Shared terms: a pool of ``num_pages`` pages of ``page`` tokens each holds the keys
and values of ``nseq`` requests. Row i of the block table lists the pages of
request i. A slot is page * page_size + offset. The free pages sit in a ring
whose state is (head, number of free pages).
"""
import math
import random

import torch

own = False

_BF16, _F32 = "bf16", "f32"
_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32}
_SIZE = {_BF16: 2, _F32: 4}
DEVICE = "cuda"

# Most of what a drawn case may cost: the largest listed one's.
_MOST_KV = 2 * 76800 * 24 * 128      # elements of K that a decode call reads
_MOST_APPEND = 131072 * 8 * 128      # elements of K that an append call writes
_MOST_PLAN = 64 * 16384              # tokens that a plan call maps


def listed():
    return [
        # one decode step of a small server: latency counts
        {"name": "plan step of 8", "op": "plan", "nseq": 8, "page": 16, "longest": 4096,
         "kind": "step", "spare": 0},
        # a large server's step: some requests end, the token buffer is padded for a graph
        {"name": "plan step of 1024", "op": "plan", "nseq": 1024, "page": 16, "longest": 8192,
         "kind": "mixed", "spare": 37},
        # prompts of different lengths enter an empty cache
        {"name": "plan prefill", "op": "plan", "nseq": 64, "page": 16, "longest": 16384,
         "kind": "prefill", "spare": 0},
        # the new token of each of 64 requests, as a projection lays it out
        {"name": "append step", "op": "append", "nseq": 64, "page": 16, "hkv": 8, "d": 128,
         "dtype": _BF16, "longest": 1, "source": "token", "order": "head", "spare": 0},
        # the keys and values of one 128K prompt, as the prefill attention takes them
        {"name": "append 128k prompt", "op": "append", "nseq": 1, "page": 128, "hkv": 8, "d": 128,
         "dtype": _BF16, "longest": 131072, "source": "head", "order": "head", "spare": 0},
        # ragged fp32 prompts, odd sizes, a padded batch
        {"name": "append ragged f32", "op": "append", "nseq": 7, "page": 32, "hkv": 3, "d": 64,
         "dtype": _F32, "longest": 4001, "source": "head", "order": "token", "spare": 5},
        # a single chat request: latency counts
        {"name": "decode one short", "op": "decode", "nseq": 1, "page": 16, "hq": 32, "hkv": 8,
         "d": 128, "dtype": _BF16, "longest": 517, "order": "head"},
        # one request at 128K: the cache's length is all the parallel work there is
        {"name": "decode one 128k", "op": "decode", "nseq": 1, "page": 128, "hq": 32, "hkv": 8,
         "d": 128, "dtype": _BF16, "longest": 131072, "order": "head"},
        # a server's ordinary step: many requests of very different lengths
        {"name": "decode 64 ragged", "op": "decode", "nseq": 64, "page": 16, "hq": 32, "hkv": 8,
         "d": 128, "dtype": _BF16, "longest": 8192, "order": "head"},
        # no shared heads, long
        {"name": "decode mha 76800", "op": "decode", "nseq": 2, "page": 128, "hq": 24, "hkv": 24,
         "d": 128, "dtype": _BF16, "longest": 76800, "order": "head"},
        # sixteen query heads a KV head, pages that hold a token's heads side by side
        {"name": "decode group of 16", "op": "decode", "nseq": 16, "page": 64, "hq": 32, "hkv": 2,
         "d": 128, "dtype": _BF16, "longest": 32768, "order": "token"},
        # the fp32 path, odd sizes
        {"name": "decode f32", "op": "decode", "nseq": 5, "page": 32, "hq": 6, "hkv": 3, "d": 64,
         "dtype": _F32, "longest": 4001, "order": "head"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "decode", "decode"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "plan":
        nseq = _spread(rng, 1, 2048)
        kind = rng.choice(("step", "mixed", "prefill"))
        most = max(1, min(131072, _MOST_PLAN // nseq))
        return {"op": op, "nseq": nseq, "page": page, "longest": _spread(rng, 1, most),
                "kind": kind, "spare": rng.randrange(0, 65)}
    dtype = rng.choice((_BF16, _BF16, _F32))
    d = rng.choice((64, 128) if dtype == _BF16 else (32, 64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8, 12, 24))
    order = rng.choice(("head", "token"))
    if op == "append":
        nseq = _spread(rng, 1, 256)
        most = max(1, _MOST_APPEND * 2 // _SIZE[dtype] // (nseq * hkv * d))
        source = rng.choice(("head", "token"))
        return {"op": op, "nseq": nseq, "page": page, "hkv": hkv, "d": d, "dtype": dtype,
                "longest": _spread(rng, 1, min(131072, most)), "source": source, "order": order,
                "spare": rng.randrange(0, 65)}
    nseq = _spread(rng, 1, 256)
    most = max(1, _MOST_KV * 2 // _SIZE[dtype] // (nseq * hkv * d))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16, 32))
    while group * hkv > 128:
        group //= 2
    return {"op": op, "nseq": nseq, "page": page, "hq": group * hkv, "hkv": hkv, "d": d,
            "dtype": dtype, "longest": _spread(rng, 1, min(131072, most)), "order": order}


# ---------------------------------------------------------------- lengths
# The lengths belong to the case (they set its work), not to the seed.

def _rng(case):
    return random.Random("%s %s %s %s" % (case["op"], case["nseq"], case["page"], case["longest"]))


def _ragged(rng, n, longest, least):
    """n lengths up to ``longest``, one of them ``longest`` itself."""
    v = [rng.randint(least, longest) for _ in range(n)]
    v[rng.randrange(n)] = longest
    return v


def _decode_lens(case):
    rng = _rng(case)
    lens = _ragged(rng, case["nseq"], case["longest"], 1)
    if case["nseq"] > 8:
        lens[lens.index(min(lens))] = 0          # a row of a padded batch holds nothing
    return lens


def _append_lens(case):
    return _ragged(_rng(case), case["nseq"], case["longest"], 0 if case["nseq"] > 1 else 1)


def _plan_lens(case):
    """(tokens held, new tokens; -1 where the request ends)."""
    rng, n = _rng(case), case["nseq"]
    if case["kind"] == "prefill":
        return [0] * n, _ragged(rng, n, case["longest"], 0)
    held = _ragged(rng, n, case["longest"], 1)
    if case["kind"] == "step":
        return held, [1] * n
    fresh = []
    for _ in range(n):
        x = rng.random()
        # most go on by a token, some end, some wait, some bring a piece of a prompt
        fresh.append(1 if x < 0.9 else -1 if x < 0.94 else 0 if x < 0.97
                     else rng.randint(1, max(1, min(512, case["longest"]))))
    return held, fresh


def _pages(tokens, page):
    return -(-tokens // page)


def _plan_sizes(case):
    held, fresh = _plan_lens(case)
    page = case["page"]
    have = [_pages(h, page) for h in held]
    after = [_pages(h + max(f, 0), page) for h, f in zip(held, fresh)]
    tokens = sum(max(f, 0) for f in fresh)
    popped = sum(a - h for a, h in zip(after, have))
    pushed = sum(h for h, f in zip(have, fresh) if f < 0)
    return held, fresh, have, after, tokens, popped, pushed


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _table(case, lens, perm, max_pages):
    """The rows' pages, dealt from ``perm`` in request order; -1 behind them."""
    page = case["page"]
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device=DEVICE)
    have = torch.tensor([_pages(n, page) for n in lens], device=DEVICE)
    at = torch.arange(max_pages, device=DEVICE)[None, :] < have[:, None]
    table[at] = perm[: int(have.sum())].to(torch.int32)
    return table


def _pool(case, num_pages, g, fill):
    """One cache of [num_pages, hkv, page, d], its memory in the case's order."""
    hkv, page, d, t = case["hkv"], case["page"], case["d"], _TYPES[case["dtype"]]
    shape = (num_pages, hkv, page, d) if case["order"] == "head" else (num_pages, page, hkv, d)
    x = torch.randn(shape, device=DEVICE, dtype=t, generator=g) if fill \
        else torch.zeros(shape, device=DEVICE, dtype=t)
    return x if case["order"] == "head" else x.transpose(1, 2)


def prepare(case, seed):
    g = _gen(seed)
    page, n = case["page"], case["nseq"]
    state = {"case": case}
    if case["op"] == "plan":
        held, fresh, have, after, tokens, popped, pushed = _plan_sizes(case)
        max_pages = max(after) + 1
        num_pages = sum(have) + popped + 11      # a few pages stay free
        perm = torch.randperm(num_pages, device=DEVICE, generator=g).to(torch.int32)
        free = num_pages - sum(have)
        head = int(torch.randint(0, num_pages, (1,), device=DEVICE, generator=g))
        ring = torch.full((num_pages,), -1, dtype=torch.int32, device=DEVICE)
        ring[(head + torch.arange(free, device=DEVICE)) % num_pages] = perm[sum(have):]
        state.update(lens=_i32(held), fresh=_i32(fresh), pool=_i32([head, free]), ring=ring,
                     table=_table(case, held, perm, max_pages), tokens=tokens, popped=popped,
                     pushed=pushed, max_tokens=tokens + case["spare"])
        return state
    hkv, d, t = case["hkv"], case["d"], _TYPES[case["dtype"]]
    if case["op"] == "append":
        lens = _append_lens(case)
        tokens = sum(lens)
        rows = tokens + case["spare"]
        num_pages = sum(_pages(x, page) for x in lens) + 1
        perm = torch.randperm(num_pages, device=DEVICE, generator=g)
        max_pages = max(1, max(_pages(x, page) for x in lens))
        table = _table(case, lens, perm, max_pages)
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x)
        starts = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
        seq = torch.repeat_interleave(torch.arange(n, device=DEVICE),
                                      torch.tensor(lens, device=DEVICE), output_size=tokens)
        pos = torch.arange(tokens, device=DEVICE) - starts[seq]
        slots = torch.full((rows,), -1, dtype=torch.int32, device=DEVICE)
        slots[:tokens] = table[seq, pos // page] * page + (pos % page).to(torch.int32)
        shape = (rows, hkv, d) if case["source"] == "token" else (rows * hkv, d)
        state.update(tokens=tokens, lens=lens, starts=starts, slots=slots,
                     K=torch.randn(shape, device=DEVICE, dtype=t, generator=g),
                     V=torch.randn(shape, device=DEVICE, dtype=t, generator=g),
                     k_pages=_pool(case, num_pages, g, False),
                     v_pages=_pool(case, num_pages, g, False))
        return state
    lens = _decode_lens(case)
    num_pages = sum(_pages(x, page) for x in lens) + 1
    perm = torch.randperm(num_pages, device=DEVICE, generator=g)
    max_pages = _pages(case["longest"], page) + 1
    # queries twice as long as keys: some keys stand out, as in a trained layer
    Q = torch.randn((n, case["hq"], d), device=DEVICE, dtype=torch.float32, generator=g)
    state.update(Q=(2 * Q).to(t), k_pages=_pool(case, num_pages, g, True),
                 v_pages=_pool(case, num_pages, g, True), lens=_i32(lens),
                 table=_table(case, lens, perm, max_pages))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "decode": _own_decode}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode}[op](state)


def _plain_plan(s):
    page, n = s["case"]["page"], s["case"]["nseq"]
    lens, fresh = s["lens"].long(), s["fresh"].long()
    head, free, cap = s["pool"][0].long(), s["pool"][1].long(), s["ring"].shape[0]
    grow = fresh.clamp(min=0)
    ends = fresh < 0
    have = (lens + page - 1) // page
    need = (lens + grow + page - 1) // page - have
    back = torch.where(ends, have, torch.zeros_like(have))
    rows = torch.arange(n, device=lens.device)
    zero = torch.zeros(1, dtype=torch.long, device=lens.device)
    table, ring = s["table"], s["ring"]

    # released pages go to the ring's tail, in row order
    first = torch.cumsum(back, 0) - back
    row = torch.repeat_interleave(rows, back, output_size=s["pushed"])
    j = torch.arange(s["pushed"], device=lens.device)
    ring[(head + free + j) % cap] = table[row, j - first[row]]
    # new pages come from its head, in row order
    first = torch.cumsum(need, 0) - need
    row = torch.repeat_interleave(rows, need, output_size=s["popped"])
    j = torch.arange(s["popped"], device=lens.device)
    table[row, have[row] + j - first[row]] = ring[(head + j) % cap]
    # the slot of every new token
    starts = torch.cat([zero, torch.cumsum(grow, 0)])
    row = torch.repeat_interleave(rows, grow, output_size=s["tokens"])
    pos = lens[row] + torch.arange(s["tokens"], device=lens.device) - starts[row]
    slots = torch.full((s["max_tokens"],), -1, dtype=torch.int32, device=lens.device)
    slots[: s["tokens"]] = table[row, pos // page] * page + (pos % page).to(torch.int32)
    lens_out = torch.where(ends, torch.zeros_like(lens), lens + grow).to(torch.int32)
    pool_out = torch.stack([(head + need.sum()) % cap, free - need.sum() + back.sum()])
    return {"lens": lens_out, "pool": pool_out.to(torch.int32), "starts": starts.to(torch.int32),
            "slots": slots, "table": table, "ring": ring}


def _plain_append(s):
    case, tokens = s["case"], s["tokens"]
    page, hkv = case["page"], case["hkv"]
    slot = s["slots"][:tokens].long()
    if case["source"] == "token":
        K, V = s["K"][:tokens], s["V"][:tokens]
    else:
        # request i is a [hkv, L_i, d] array; the row of (token, head) in the packed array
        starts = s["starts"].long()
        size = starts[1:] - starts[:-1]
        seq = torch.repeat_interleave(torch.arange(case["nseq"], device=slot.device), size,
                                      output_size=tokens)
        t = torch.arange(tokens, device=slot.device) - starts[seq]
        row = (starts[seq] * hkv + t)[:, None] + \
            torch.arange(hkv, device=slot.device)[None, :] * size[seq][:, None]
        K, V = s["K"][row], s["V"][row]
    s["k_pages"][slot // page, :, slot % page] = K
    s["v_pages"][slot // page, :, slot % page] = V
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    case = s["case"]
    n, hkv, d, page = case["nseq"], case["hkv"], case["d"], case["page"]
    group, used = case["hq"] // hkv, _pages(case["longest"], page)
    at = s["table"][:, :used].long().clamp(min=0)
    K = s["k_pages"][at].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, used * page, d)
    q = s["Q"].float().reshape(n, hkv, group, d) / math.sqrt(d)
    logits = torch.matmul(q, K.transpose(2, 3))
    del K
    there = torch.arange(used * page, device=at.device)[None, :] < s["lens"][:, None]
    logits = logits.masked_fill(~there[:, None, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(logits - base)
    total = e.sum(-1, keepdim=True)
    V = s["v_pages"][at].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, used * page, d)
    O = torch.matmul(e, V)
    O = torch.where(total > 0, O / total, torch.zeros_like(O))
    lse = base + torch.log(total)
    return {"O": O.reshape(n, case["hq"], d).to(s["Q"].dtype), "lse": lse.reshape(n, case["hq"])}


def _own_plan(s):
    from block_sparse_long_score_b200 import plan_buffers, xattn_paged_plan
    buf = s.get("buffers")
    if buf is None:                      # a serving loop keeps its buffers
        buf = s["buffers"] = plan_buffers(s["table"], s["max_tokens"])
    lens, pool, starts, slots = xattn_paged_plan(
        s["lens"], s["fresh"], s["pool"], s["ring"], s["table"], s["case"]["page"],
        out=(buf["lens"], buf["pool"], buf["starts"], buf["slots"]))
    return {"lens": lens, "pool": pool, "starts": starts, "slots": slots, "table": s["table"],
            "ring": s["ring"]}


def _own_append(s):
    from block_sparse_long_score_b200 import xattn_paged_append
    xattn_paged_append(s["K"], s["V"], s["slots"], s["k_pages"], s["v_pages"],
                       starts=s["starts"] if s["case"]["source"] == "head" else None)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_decode(s):
    from block_sparse_long_score_b200 import decode_buffers, xattn_paged_decode
    buf = s.get("buffers")
    if buf is None:                      # a serving loop keeps its buffers
        buf = s["buffers"] = decode_buffers(s["Q"], s["k_pages"], s["table"])
    O, lse = xattn_paged_decode(s["Q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                out=buf["out"], lse=buf["lse"], workspace=buf["ws"])
    return {"O": O, "lse": lse}


# ---------------------------------------------------------------- work, exact

def work(case):
    page, n = case["page"], case["nseq"]
    if case["op"] == "plan":
        held, fresh, have, after, tokens, popped, pushed = _plan_sizes(case)
        # an open page of a request that goes on is read from the table
        open_pages = sum(1 for h, f in zip(held, fresh) if f > 0 and h % page)
        words = 2 * n + 2 + 2 * popped + 2 * pushed + open_pages
        words += n + 2 + n + 1 + tokens + case["spare"]
        return {"bytes": 4 * words, "flops": 0}
    row = case["hkv"] * case["d"] * _SIZE[case["dtype"]]
    if case["op"] == "append":
        tokens = sum(_append_lens(case))
        extra = n + 1 if case["source"] == "head" else 0
        return {"bytes": 4 * tokens * row + 4 * (tokens + case["spare"] + extra), "flops": 0}
    lens = _decode_lens(case)
    q = n * case["hq"] * case["d"] * _SIZE[case["dtype"]]
    small = 4 * n + 4 * n * case["hq"] + 4 * sum(_pages(x, page) for x in lens)
    return {"bytes": 2 * sum(lens) * row + 2 * q + small,
            "flops": 4 * sum(lens) * case["hq"] * case["d"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                      # whole numbers: compared as they are
    page, hkv, d = case["page"], case["hkv"], case["d"]
    if case["op"] == "append":
        done = {}
        for name, src in (("k_pages", s["K"]), ("v_pages", s["V"])):
            pages = s[name].shape[0]
            flat = torch.zeros((pages * page, hkv, d), dtype=torch.float64, device=DEVICE)
            at = 0
            for size in s["lens"]:
                if case["source"] == "token":
                    x = src[at:at + size]
                else:
                    x = src[at * hkv:(at + size) * hkv].reshape(hkv, size, d).transpose(0, 1)
                flat[s["slots"][at:at + size].long()] = x.double()
                at += size
            done[name] = flat.reshape(pages, page, hkv, d).transpose(1, 2)
        return done
    group = case["hq"] // hkv
    O = torch.zeros((case["nseq"], case["hq"], d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((case["nseq"], case["hq"]), -math.inf, dtype=torch.float64, device=DEVICE)
    for i, size in enumerate(_decode_lens(case)):
        if size == 0:
            continue
        pages = s["table"][i, : _pages(size, page)].long()
        for h in range(hkv):
            k = s["k_pages"][pages, h].reshape(-1, d)[:size].double()
            v = s["v_pages"][pages, h].reshape(-1, d)[:size].double()
            mine = slice(h * group, (h + 1) * group)
            x = (s["Q"][i, mine].double() @ k.T) * (1.0 / math.sqrt(d))
            total = torch.logsumexp(x, dim=1)
            O[i, mine] = torch.exp(x - total[:, None]) @ v
            lse[i, mine] = total
    return {"O": O, "lse": lse}
