"""The paged-cache operators against their plain forms: block tables and slot
maps (exact), writes (exact), and single-token attention within an error bound
worked out from the roundings (tests/paged_ref.py)."""
import random

import pytest
import torch

from block_sparse_long_score_b200 import (PagedCache, XattnError, decode_buffers, plan_buffers,
                                          prefill_attention, xattn_get_device_status,
                                          xattn_paged_append, xattn_paged_decode,
                                          xattn_paged_plan, xattn_prefill_varlen)
from block_sparse_long_score_b200.synth import make_problem
from tests import paged_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
CANARY = 0x7F7F7F7F


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plan

def _plan_state(rng, n, page, longest, kind, spare_pages=3):
    lens = [rng.randint(0, longest) for _ in range(n)]
    fresh = []
    for x in lens:
        fresh.append({"step": 1, "prefill": rng.randint(0, longest),
                      "mixed": rng.choice((-1, 0, 1, 1, rng.randint(0, 3 * page))),
                      "end": -1}[kind])
    have = [R.pages(x, page) for x in lens]
    rows = max(max(R.pages(x + max(f, 0), page) for x, f in zip(lens, fresh)), 1)
    need = sum(R.pages(x + max(f, 0), page) - h for x, f, h in zip(lens, fresh, have))
    N = sum(have) + need + spare_pages
    ids = rng.sample(range(N), N)
    table = [[-1] * rows for _ in range(n)]
    at = 0
    for i in range(n):
        table[i][:have[i]] = ids[at:at + have[i]]
        at += have[i]
    head, free = rng.randrange(N), N - at
    ring = [-1] * N
    for j in range(free):
        ring[(head + j) % N] = ids[at + j]
    return lens, fresh, [head, free], ring, table


def _run_plan(lens, fresh, pool, ring, table, page, max_tokens, in_place=False):
    t = [_i32(x) for x in (lens, fresh, pool, ring, table)]
    n = len(lens)
    out = (t[0] if in_place else torch.full((n,), CANARY, dtype=torch.int32, device=DEV),
           t[2] if in_place else torch.full((2,), CANARY, dtype=torch.int32, device=DEV),
           torch.full((n + 1,), CANARY, dtype=torch.int32, device=DEV),
           torch.full((max_tokens,), CANARY, dtype=torch.int32, device=DEV))
    xattn_paged_plan(t[0], t[1], t[2], t[3], t[4], page, out=out)
    torch.cuda.synchronize()
    return [x.tolist() for x in out] + [t[3].tolist(), t[4].tolist()]


PLANS = [(1, 16, 1, "prefill"), (1, 16, 5000, "step"), (3, 256, 700, "mixed"),
         (7, 32, 200, "prefill"), (31, 16, 16, "step"), (33, 64, 300, "mixed"),
         (64, 16, 900, "end"), (257, 16, 120, "mixed"), (1023, 16, 40, "step"),
         (1025, 32, 100, "mixed"), (2500, 16, 60, "mixed"), (5, 16, 30000, "prefill"),
         (4099, 16, 33, "mixed"), (9000, 16, 20, "step")]


@pytest.mark.parametrize("n,page,longest,kind", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(n, page, longest, kind, in_place):
    rng = random.Random(n * 7 + longest)
    state = _plan_state(rng, n, page, longest, kind)
    max_tokens = sum(max(f, 0) for f in state[1]) + rng.choice((0, 1, 37))
    want = R.plan(*state, page, max_tokens)
    assert want[-1] is None
    got = _run_plan(*state, page, max_tokens, in_place)
    for name, g, w in zip(("lens", "pool", "starts", "slots", "ring", "table"), got, want):
        assert g == w, name
    assert xattn_get_device_status() == 0


def test_large_plan_replays_in_a_graph():
    """A step whose slots take the second kernel, captured in place and replayed
    on other lengths, one of them a step that cannot be done."""
    rng = random.Random(8)
    n, page, room = 40, 16, 50000
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    fresh, pool = torch.zeros_like(lens), torch.zeros(2, dtype=torch.int32, device=DEV)
    state = _plan_state(rng, n, page, 2000, "prefill", spare_pages=900)
    ring, table = (torch.zeros_like(_i32(x)) for x in state[3:])
    starts = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(room, dtype=torch.int32, device=DEV)
    call = lambda: xattn_paged_plan(lens, fresh, pool, ring, table, page,
                                    out=(lens, pool, starts, slots))
    call()                                     # pool says no page is free: nothing to do
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lack = [list(x) for x in state[:3]] + [state[3], state[4]]
    lack[2][1] = 10
    for s, code in ((state, 0), (lack, -6)):
        want = R.plan(*s, page, room)
        for dst, src in zip((lens, fresh, pool, ring, table), s):
            dst.copy_(_i32(src))
        slots.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        for name, g, w in zip(("lens", "pool", "starts", "slots", "ring", "table"),
                              (lens, pool, starts, slots, ring, table), want):
            assert g.tolist() == w, name
        assert xattn_get_device_status() == code


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_plan_writes_slots_at_any_alignment(offset):
    state = _plan_state(random.Random(offset), 30, 16, 3000, "prefill")
    tokens = sum(state[1])
    t = [_i32(x) for x in state]
    buf = torch.full((tokens + 9,), CANARY, dtype=torch.int32, device=DEV)
    out = (torch.empty_like(t[0]), torch.empty_like(t[2]),
           torch.empty(31, dtype=torch.int32, device=DEV), buf[offset:offset + tokens + 2])
    xattn_paged_plan(*t, 16, out=out)
    want = R.plan(*state, 16, tokens + 2)
    assert out[3].tolist() == want[3]
    assert bool((buf[:offset] == CANARY).all()) and bool((buf[offset + tokens + 2:] == CANARY).all())


@pytest.mark.parametrize("n", [5, 1500])
@pytest.mark.parametrize("what,code", [("pages", -6), ("tokens", -1), ("row", -1),
                                       ("negative", -1), ("fresh", -1), ("head", -1),
                                       ("free", -1)])
def test_plan_that_cannot_be_done_changes_nothing(n, what, code):
    rng = random.Random(3)
    lens, fresh, pool, ring, table = _plan_state(rng, n, 16, 100, "step")
    i = n // 2
    lens[i], max_tokens = 16, n
    if what == "pages":
        pool[1] = sum(R.pages(x + 1, 16) - R.pages(x, 16) for x in lens) - 1
    elif what == "tokens":
        max_tokens = n - 1
    elif what == "row":
        fresh[i] = 16 * len(table[0])
        max_tokens = 1 << 16
    elif what == "negative":
        lens[i] = -1
    elif what == "fresh":
        fresh[i] = -2
    elif what == "head":
        pool[0] = len(ring)
    else:
        pool[1] = -1
    want = R.plan(lens, fresh, pool, ring, table, 16, max_tokens)
    assert want[-1] == ("pages" if code == -6 else "invalid")
    assert xattn_get_device_status() == 0
    got = _run_plan(lens, fresh, pool, ring, table, 16, max_tokens)
    for name, g, w in zip(("lens", "pool", "starts", "slots", "ring", "table"), got, want):
        assert g == w, name
    assert xattn_get_device_status() == code
    assert xattn_get_device_status() == 0


@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_plan_reports_an_entry_that_is_no_page(bad):
    """A ring entry and a table entry that are no pages: the tokens that would
    use them have no slot, everything else is as usual."""
    state = ([16, 20, 5], [1, 1, 2], [0, 4], [9, bad, 6, 7, 8, 0, 1, 2, 3, 4],
             [[0, -1], [1, bad], [2, -1]])
    want = R.plan(*state, 16, 5)
    assert want[-1] == "invalid" and want[3] == [144, -1, 37, 38, -1]
    got = _run_plan(*state, 16, 5)
    for g, w in zip(got, want):
        assert g == w
    assert xattn_get_device_status() == -1


def test_plan_with_no_tokens_and_no_slots():
    state = ([5, 0], [0, 0], [1, 1], [0, 3, 0, 0], [[2], [-1]])
    assert _run_plan(*state, 16, 0) == list(R.plan(*state, 16, 0)[:6])


def test_plan_uses_every_free_page_and_a_full_ring_wraps():
    n, page = 8, 16
    lens, N = [16] * n, 2 * n
    table = [[i, -1] for i in range(n)]
    ring = list(range(n, N)) + [-7] * n
    ring = ring[-3:] + ring[:-3]                       # head 3
    state = (lens, [1] * n, [3, n], ring, table)
    got = _run_plan(*state, page, n)
    assert got == list(R.plan(*state, page, n)[:6]) and got[1][1] == 0
    # every request ends: all pages come back
    state = (got[0], [-1] * n, got[1], got[4], got[5])
    got = _run_plan(*state, page, n)
    assert got == list(R.plan(*state, page, n)[:6]) and got[1][1] == N
    assert sorted(got[4]) == list(range(N))


# ---------------------------------------------------------------- append

def _pool(N, hkv, page, d, dtype, order, fill=float("nan")):
    shape = {"head": (N, hkv, page, d), "token": (N, page, hkv, d), "both": (N, 2, hkv, page, d),
             "wide": (N, hkv, page, d + 64), "odd": (N, hkv, page, d + 8)}[order]
    def view(x):
        return {"head": x, "token": x.transpose(1, 2), "wide": x[..., 16:16 + d],
                "odd": x[..., 8:]}[order]
    if order == "both":
        x = torch.full(shape, fill, dtype=dtype, device=DEV)
        return x[:, 0], x[:, 1]
    return tuple(view(torch.full(shape, fill, dtype=dtype, device=DEV)) for _ in range(2))


SHAPES = [(1, 1, 128, torch.bfloat16, 16, "head"), (7, 8, 128, torch.bfloat16, 16, "token"),
          (64, 8, 128, torch.bfloat16, 128, "both"), (33, 3, 64, torch.bfloat16, 32, "wide"),
          (65, 5, 32, torch.float32, 64, "head"), (130, 2, 64, torch.float32, 256, "token"),
          (513, 4, 128, torch.float32, 32, "both")]


@pytest.mark.parametrize("tokens,hkv,d,dtype,page,order", SHAPES)
@pytest.mark.parametrize("fused", [False, True])
def test_append_token_rows(tokens, hkv, d, dtype, page, order, fused):
    g = torch.Generator(device=DEV).manual_seed(tokens)
    N = R.pages(tokens, page) + 2
    kp, vp = _pool(N, hkv, page, d, dtype, order)
    slots = torch.randperm(N * page, device=DEV, generator=g)[:tokens].to(torch.int32)
    keep = torch.rand(tokens, device=DEV, generator=g) < 0.8
    slots[~keep] = -1
    if fused:                                      # slices of one projection's rows
        x = torch.randn(tokens, 3 * hkv, d, device=DEV, generator=g).to(dtype)
        K, V = x[:, hkv:2 * hkv], x[:, 2 * hkv:]
    else:
        K, V = (torch.randn(tokens, hkv, d, device=DEV, generator=g).to(dtype)
                for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    s = slots[keep].long()
    want_k[s // page, :, s % page] = K[keep]
    want_v[s // page, :, s % page] = V[keep]
    xattn_paged_append(K, V, slots, kp, vp)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    assert torch.equal(kp.nan_to_num(nan=77.0), want_k.nan_to_num(nan=77.0))
    assert torch.equal(vp.nan_to_num(nan=77.0), want_v.nan_to_num(nan=77.0))


@pytest.mark.parametrize("lens,hkv,d,dtype,page,order,spare", [
    ([1], 1, 128, torch.bfloat16, 16, "head", 0),
    ([0, 5, 0, 0, 33, 1, 0], 2, 64, torch.bfloat16, 16, "token", 3),
    ([300, 17, 128], 8, 128, torch.bfloat16, 128, "head", 0),
    ([64, 64, 64, 64], 3, 32, torch.float32, 32, "both", 0),
    ([1000], 5, 64, torch.float32, 64, "wide", 9),
    ([3] * 90 + [0] * 20 + [211], 4, 128, torch.bfloat16, 16, "head", 31),
])
def test_append_packed_prompts(lens, hkv, d, dtype, page, order, spare):
    g = torch.Generator(device=DEV).manual_seed(len(lens))
    T = sum(lens)
    N = R.pages(T, page) + 1
    kp, vp = _pool(N, hkv, page, d, dtype, order)
    slots = torch.randperm(N * page, device=DEV, generator=g)[:T + spare].to(torch.int32)
    starts = _i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    K, V = (torch.randn((T + spare) * hkv, d, device=DEV, generator=g).to(dtype)
            for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    at = 0
    for L in lens:
        s = slots[at:at + L].long()
        for want, x in ((want_k, K), (want_v, V)):
            want[s // page, :, s % page] = \
                x[at * hkv:(at + L) * hkv].reshape(hkv, L, d).transpose(0, 1)
        at += L
    xattn_paged_append(K, V, slots, kp, vp, starts=starts)     # tokens past T are left out
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    assert torch.equal(kp.nan_to_num(nan=77.0), want_k.nan_to_num(nan=77.0))
    assert torch.equal(vp.nan_to_num(nan=77.0), want_v.nan_to_num(nan=77.0))


@pytest.mark.parametrize("slot", [-2, 64, 1 << 30])
def test_append_leaves_out_and_reports_a_bad_slot(slot):
    kp, vp = _pool(4, 2, 16, 128, torch.bfloat16, "head", 0.0)
    K = torch.ones(3, 2, 128, device=DEV, dtype=torch.bfloat16)
    xattn_paged_append(K, K + 1, _i32([5, slot, 6]), kp, vp)
    assert xattn_get_device_status() == -1
    assert kp.sum().item() == 2 * 2 * 128 and vp.sum().item() == 4 * 2 * 128


@pytest.mark.parametrize("starts", [[0, 4, 2], [0, 2, 9], [-3, 2, 3], [1, 2, 3]])
def test_append_reports_starts_that_are_no_prefix_sum(starts):
    """Rows that broken starts would place outside K are left out."""
    kp, vp = _pool(4, 1, 16, 64, torch.float32, "head", 0.0)
    K = torch.ones(3, 64, device=DEV)
    xattn_paged_append(K, K, _i32([0, 1, 2]), kp, vp, starts=_i32(starts))
    assert xattn_get_device_status() in (0, -1)
    assert kp[0, 0, 3:].abs().sum().item() == 0 and kp[1:].abs().sum().item() == 0


# ---------------------------------------------------------------- decode

def _cache(lens, hq, hkv, d, dtype, page, order="head", seed=0, extra=2, qscale=2.0):
    """Random queries and pages; what no request owns is NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = len(lens)
    have = [R.pages(max(x, 0), page) for x in lens]
    N = sum(have) + extra
    kp, vp = _pool(N, hkv, page, d, dtype, order)
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = max(max(have), 1) + 1
    table = [[-5] * rows for _ in range(n)]
    at = 0
    for i in range(n):
        table[i][:have[i]] = perm[at:at + have[i]]
        at += have[i]
        for j in range(have[i]):
            used = min(page, lens[i] - j * page)
            for p in (kp, vp):
                p[table[i][j], :, :used] = torch.randn(hkv, used, d, device=DEV,
                                                       generator=g).to(dtype)
    Q = (qscale * torch.randn(n, hq, d, device=DEV, generator=g)).to(dtype)
    return Q, kp, vp, _i32(table), _i32(lens)


def _check_decode(Q, kp, vp, table, lens, status=0):
    n, hq, d = Q.shape
    out = torch.full_like(Q, float("nan"))
    lse = torch.full((n, hq), float("nan"), device=DEV)
    ws = decode_buffers(Q, kp, table)["ws"].fill_(0x7F)
    xattn_paged_decode(Q, kp, vp, table, lens, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == status
    O, L, tol, tol_lse = R.decode(Q, kp, vp, table, lens)
    err = (out.cpu().double() - O).abs()
    assert bool((err <= tol).all()), f"{(err - tol).max().item():.3g} past its bound"
    got = lse.cpu().double()
    empty = L == -float("inf")
    assert torch.equal(got == -float("inf"), empty)
    assert bool(((got - L).abs() <= tol_lse)[~empty].all())
    assert bool((out.cpu()[empty] == 0).all())
    return out, lse


BF, F3 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("length", [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128,
                                    129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F3, 128), (F3, 64), (F3, 32)])
def test_decode_lengths(length, dtype, d):
    _check_decode(*_cache([length], 4, 1, d, dtype, 16, seed=length))


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17, 24, 31, 32, 33, 48, 64,
                                   128])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F3, 128), (F3, 32)])
def test_decode_groups(group, dtype, d):
    hkv = 2 if group < 128 else 1
    _check_decode(*_cache([77, 0, 300], group * hkv, hkv, d, dtype, 32, seed=group))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["head", "token", "both", "wide", "odd"])
@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_pages_and_strides(page, order, dtype):
    _check_decode(*_cache([page - 1, page, page + 1, 5 * page + 3, 1], 8, 2, 64, dtype, page,
                          order, seed=page))


@pytest.mark.parametrize("hq,hkv,d,dtype,page,lens", [
    (32, 8, 128, BF, 16, [1, 5000, 0, 17, 333, 2048, 4]),
    (24, 24, 128, BF, 128, [3000, 700]),
    (32, 2, 128, BF, 64, [9000, 10, 1200]),
    (8, 8, 64, BF, 32, [0, 0, 0, 5, 0]),
    (6, 3, 64, F3, 32, [4001, 3, 0, 129, 1000]),
    (40, 8, 128, F3, 16, [600] * 9),
    (4, 4, 32, F3, 256, [10000]),
    (16, 1, 128, BF, 16, [40000]),
    (12, 4, 128, BF, 16, list(range(0, 300, 3))),
])
def test_decode_batches(hq, hkv, d, dtype, page, lens):
    _check_decode(*_cache(lens, hq, hkv, d, dtype, page, seed=len(lens)))


@pytest.mark.parametrize("n", [1030, 3000])
@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_many_requests(n, dtype):
    rng = random.Random(n)
    _check_decode(*_cache([rng.choice((0, 1, 5, 17, 40)) for _ in range(n)], 2, 1, 64, dtype, 16))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F3, 128), (F3, 64), (F3, 32)])
@pytest.mark.parametrize("group", [1, 3, 8, 13, 30])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_many_short_requests(group, dtype, d, wide):
    """More units (an odd number of them) than the GPU has room for twice, none longer
    than 288 tokens: a warp takes each, and several where the table's rows could hold
    more."""
    rng = random.Random(group * d)
    longest = 270 if not wide else 280
    lens = [rng.choice((0, 1, 7, 8, 9, 15, 16, 17, 63, 65, 128, 200, longest - 1, longest))
            for _ in range(187)]
    lens[3] = longest
    case = _cache(lens, 7 * group, 7, d, dtype, 16, seed=group)
    _check_decode(*(_wide(*case, 700) if wide else case))


@pytest.mark.parametrize("dtype", [BF, F3])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("long", [1, 40, 100])
def test_decode_more_short_requests_than_warps(dtype, wide, long):
    rng = random.Random(long)
    case = _cache([rng.randint(0, long) for _ in range(1100)], 6, 3, 64, dtype, 16)
    _check_decode(*(_wide(*case, 700) if wide else case))


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_many_short_requests_with_bad_pages_and_lengths(dtype):
    Q, kp, vp, table, lens = _cache([20, 100, 33] * 63, 21, 7, 64, dtype, 16)
    table = table[:, :7].contiguous()
    table[5, 1] = -1
    table[7, 6] = 1 << 30
    table[9, 0] = kp.shape[0]
    _check_decode(Q, kp, vp, table, lens, status=-1)
    _check_decode(*_wide(Q, kp, vp, table, lens, 700), status=-1)
    kp.nan_to_num_(), vp.nan_to_num_()       # the whole row of request 188 is read
    lens[10] = -1
    lens[188] = 1 << 30
    table[188] = table[1]
    _check_decode(Q, kp, vp, table, lens, status=-1)


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_one_long_request_among_many_short_ones(dtype):
    """Far more tokens in one request than in all the others."""
    lens = [(37 * i) % 70 for i in range(220)]
    lens[100] = 20011
    _check_decode(*_cache(lens, 16, 8, 64, dtype, 64))


def _wide(Q, kp, vp, table, lens, columns):
    """The same requests in a table with room for far more tokens: the work is
    cut by tile ranges, where a narrow table's goes to CTAs or clusters by unit."""
    more = torch.full((table.shape[0], columns), 1 << 30, dtype=torch.int32, device=DEV)
    return Q, kp, vp, torch.cat([table, more], 1), lens


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1], [0, 0, 1, 0], [16], [17, 0, 15], [64], [65],
                                  [128, 1], [300, 64, 0, 129], [1000], [0, 700, 0, 0, 3, 2000],
                                  list(range(40)), [33] * 70])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F3, 128), (F3, 32)])
def test_decode_short_requests_in_a_wide_table(lens, dtype, d):
    _check_decode(*_wide(*_cache(lens, 8, 2, d, dtype, 16, seed=len(lens)), 4000))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 17, 32, 33, 64, 128])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F3, 128), (F3, 64), (F3, 32)])
def test_decode_groups_in_a_wide_table(group, dtype, d):
    """Units shared by several CTAs, for every count of heads a pass serves."""
    _check_decode(*_wide(*_cache([777, 0, 1500], group, 1, d, dtype, 32, seed=group), 3000))


@pytest.mark.parametrize("n", [1, 127, 128, 129, 400])
def test_decode_scan_of_the_lengths(n):
    """As many requests as the scan's threads, one less, one more, several each."""
    rng = random.Random(n)
    lens = [rng.choice((0, 0, 1, 40, 200)) for _ in range(n)]
    _check_decode(*_wide(*_cache(lens, 4, 2, 64, BF, 16, seed=n), 2000))


def test_decode_narrow_and_wide_tables_agree():
    """Both ways to cut the work are within the bound of the same fp64 result,
    and within twice that of each other."""
    c = _cache([500, 31, 0, 900], 16, 2, 128, BF, 16)
    a, _ = _check_decode(*c)
    b, _ = _check_decode(*_wide(*c, 4000))
    tol = R.decode(*c)[2]
    assert bool(((a.double() - b.double()).abs().cpu() <= 2 * tol).all())


def test_decode_table_of_more_than_2_to_31_entries():
    """A table whose capacity is past 2^31 tiles and whose last rows lie past
    2^31 entries: only the entries of the lengths are read."""
    n, columns = 520, (1 << 30) // 256
    Q, kp, vp, table, lens = _cache([0] * (n - 3) + [700, 0, 300], 8, 2, 128, BF, 256)
    big = torch.empty(n, columns, dtype=torch.int32, device=DEV)
    assert big.numel() > 1 << 31
    big[:, :table.shape[1]] = table
    out, lse = xattn_paged_decode(Q, kp, vp, big, lens, lse=True)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    O, L, tol, tol_lse = R.decode(Q, kp, vp, table, lens)
    assert bool(((out.cpu().double() - O).abs() <= tol).all())
    assert bool((lse[:n - 3].cpu() == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F3])
@pytest.mark.parametrize("qscale", [0.0, 30.0, 300.0])
def test_decode_flat_and_peaked_logits(dtype, qscale):
    _check_decode(*_cache([1500, 64], 8, 2, 128, dtype, 16, qscale=qscale))


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_rising_logits(dtype):
    """Each token's logit is above all before it: the running maximum moves at
    every step, by up to thousands in all."""
    Q, kp, vp, table, lens = _cache([1600], 4, 1, 64, dtype, 16)
    Q.fill_(1.0)
    ramp = torch.arange(1600, device=DEV).reshape(-1, 16).to(dtype)
    kp[table[0, :100].long(), 0] = ramp[..., None] / 4
    _check_decode(Q, kp, vp, table, lens)


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_logits_of_minus_infinity_weigh_nothing(dtype):
    Q, kp, vp, table, lens = _cache([100, 40], 4, 2, 64, dtype, 16)
    Q.abs_()
    for t in (0, 7, 50, 99):
        kp[table[0, t // 16], :, t % 16, 3] = -float("inf")
    _check_decode(Q, kp, vp, table, lens)
    low = torch.finfo(dtype).min          # finite, but its logit overflows to -inf or nearly
    for t in (1, 8):
        kp[table[0, t // 16], :, t % 16, 5] = low
    Q[..., 5] = 0.5
    _check_decode(Q, kp, vp, table, lens)


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_carries_nan_and_infinity_of_its_own_rows_only(dtype):
    Q, kp, vp, table, lens = _cache([70, 70, 70], 4, 2, 64, dtype, 16)
    kp[table[1, 2], 1, 3, 9] = float("nan")
    vp[table[2, 1], 0, 5, 7] = float("inf")
    O, lse = xattn_paged_decode(Q, kp, vp, table, lens, lse=True)
    torch.cuda.synchronize()
    assert bool(O[0].isfinite().all()) and bool(lse[0].isfinite().all())
    assert bool(O[1, 2:].isnan().all()) and bool(lse[1, 2:].isnan().all())
    assert bool(O[1, :2].isfinite().all()) and bool(O[2, 2:].isfinite().all())
    assert bool((O[2, :2, 7] == float("inf")).all())
    assert bool(lse[2].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F3])
@pytest.mark.parametrize("bad", [-1, 1 << 30, -(1 << 31)])
def test_decode_leaves_out_and_reports_bad_pages(dtype, bad):
    Q, kp, vp, table, lens = _cache([100, 600, 5], 8, 2, 64, dtype, 32)
    table[1, 3] = bad
    table[1, 18] = bad                       # the last page, partly used
    _check_decode(Q, kp, vp, table, lens, status=-1)
    table[2, 0] = bad                        # a row whose every page is bad is empty
    _check_decode(Q, kp, vp, table, lens, status=-1)


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_clamps_and_reports_bad_lengths(dtype):
    Q, kp, vp, table, lens = _cache([96, 96, 96], 4, 2, 64, dtype, 32)
    table = table[:, :3].contiguous()
    lens.copy_(_i32([96, -4, 2000000000]))
    _check_decode(Q, kp, vp, table, lens, status=-1)


def test_decode_rows_that_share_pages():
    Q, kp, vp, table, lens = _cache([100, 90, 0], 8, 2, 128, BF, 16)
    table[2], table[1, :3] = table[0], table[0, :3]
    lens[2] = 37
    _check_decode(Q, kp, vp, table, lens)


@pytest.mark.parametrize("dtype,order", [(BF, "head"), (F3, "token")])
def test_offsets_past_32_bits(dtype, order):
    """Pages whose first element is past 2^32: only their rows are filled."""
    hkv, page, d = 8, 256, 128
    N = (1 << 32) // (hkv * page * d) + 40
    shape = (N, hkv, page, d) if order == "head" else (N, page, hkv, d)
    kp, vp = (torch.empty(shape, dtype=dtype, device=DEV) for _ in range(2))
    if order == "token":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    T = 700
    table = _i32([[N - 1, 3, N - 20]])
    t = torch.arange(T, device=DEV)
    slots = (table[0, (t // page)].long() * page + t % page).to(torch.int32)
    K, V = (torch.randn(T, hkv, d, device=DEV).to(dtype) for _ in range(2))
    xattn_paged_append(K, V, slots, kp, vp)
    assert torch.equal(kp[N - 20, :, :T - 512], K[512:].transpose(0, 1))
    Q = torch.randn(1, 16, d, device=DEV).to(dtype)
    O, lse = xattn_paged_decode(Q, kp, vp, table, _i32([T]), lse=True)
    torch.cuda.synchronize()
    small_k, small_v = (x[table[0].long()].clone() for x in (kp, vp))
    small = xattn_paged_decode(Q, small_k, small_v, _i32([[0, 1, 2]]), _i32([T]), lse=True)
    assert torch.equal(O, small[0]) and torch.equal(lse, small[1])
    _check_decode(Q, small_k, small_v, _i32([[0, 1, 2]]), _i32([T]))


def test_decode_is_the_same_bits_again_and_takes_a_4d_query():
    Q, kp, vp, table, lens = _cache([5000, 17, 900, 3333], 32, 8, 128, BF, 16)
    a, la = xattn_paged_decode(Q, kp, vp, table, lens, lse=True)
    for _ in range(5):
        b, lb = xattn_paged_decode(Q.unsqueeze(2), kp, vp, table, lens, lse=True)
        assert b.shape == (4, 32, 1, 128)
        assert torch.equal(a, b.squeeze(2)) and torch.equal(la, lb)
    assert torch.equal(a, xattn_paged_decode(Q, kp, vp, table, lens))


def test_binding_refusals():
    Q, kp, vp, table, lens = _cache([20, 20], 8, 2, 128, BF, 16)
    bad = [dict(Q=Q.float()), dict(Q=Q[:, :, :64].contiguous()), dict(Q=Q[:1]),
           dict(Q=Q.transpose(0, 1)), dict(vp=vp.float()), dict(vp=vp[:-1]),
           dict(vp=vp.transpose(1, 2).contiguous().transpose(1, 2)), dict(table=table.long()),
           dict(table=table[:1]), dict(table=table[:, ::2]), dict(lens=lens[:1]),
           dict(lens=lens.cpu()), dict(lens=lens.long())]
    for kw in bad:
        a = dict(Q=Q, kp=kp, vp=vp, table=table, lens=lens)
        a.update(kw)
        with pytest.raises((ValueError, XattnError)):
            xattn_paged_decode(a["Q"], a["kp"], a["vp"], a["table"], a["lens"])
    with pytest.raises(ValueError):
        xattn_paged_decode(Q, kp, vp, table, lens, out=torch.empty_like(Q)[:1])
    with pytest.raises(ValueError):
        xattn_paged_decode(Q, kp, vp, table, lens, lse=torch.empty(2, 4, device=DEV))
    with pytest.raises(XattnError):
        xattn_paged_decode(Q, kp, vp, table, lens,
                           workspace=torch.empty(16, device=DEV, dtype=torch.uint8))
    with pytest.raises(XattnError):
        xattn_paged_decode(Q, kp[..., :7, :], vp[..., :7, :], table, lens)    # 7 tokens a page
    K = torch.zeros(3, 2, 128, device=DEV, dtype=BF)
    s = _i32([0, 1, 2])
    for args in ((K[:2], K, s, kp, vp), (K, K[:2], s, kp, vp), (K.float(), K, s, kp, vp),
                 (K, K, s.long(), kp, vp), (K, K, s, kp, vp[:-1]),
                 (K[:, :, ::2], K[:, :, ::2], s, kp, vp),
                 (K, torch.zeros(3, 4, 128, device=DEV, dtype=BF)[:, :2], s, kp, vp)):
        with pytest.raises(ValueError):
            xattn_paged_append(*args)
    with pytest.raises(XattnError):
        xattn_paged_append(K, K, s, kp, kp)
    with pytest.raises(ValueError):
        xattn_paged_append(K, K, s, kp, vp, starts=_i32([0]))
    with pytest.raises(XattnError):                       # an expanded page array
        xattn_paged_append(K, K, s, kp[:1].expand(5, -1, -1, -1), vp[:1].expand(5, -1, -1, -1))


# ------------------------------------------------- together, streams, graphs

def test_on_another_stream_than_the_default():
    Q, kp, vp, table, lens = _cache([700, 20], 8, 2, 128, BF, 16)
    want = xattn_paged_decode(Q, kp, vp, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        Q2 = Q * 1
        got = xattn_paged_decode(Q2, kp, vp, table, lens)
    side.synchronize()
    assert torch.equal(got, want)


def test_two_calls_at_once_on_two_streams():
    a = _cache([9000, 20, 600], 32, 8, 128, BF, 16, seed=1)
    b = _cache([300] * 40, 32, 8, 128, BF, 16, seed=2)
    want = [xattn_paged_decode(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(xattn_paged_decode(*x))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _steps(cache, buf, seed, n, steps, hkv, hq, d, dtype):
    """Random server steps against a plain server that keeps contiguous K, V."""
    rng = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = [[] for _ in range(n)]
    for _ in range(steps):
        fresh = [rng.choice((1, 1, 1, 0)) if rows[i] else 1 for i in range(n)]
        i = rng.randrange(n)
        if len(rows[i]) > 20:
            fresh[i] = -1
        K, V = (torch.randn(n, hkv, d, device=DEV, generator=g).to(dtype) for _ in range(2))
        Q = torch.randn(n, hq, d, device=DEV, generator=g).to(dtype)
        yield fresh, Q, K, V
        at = 0
        for i in range(n):
            if fresh[i] < 0:
                rows[i] = []
            elif fresh[i]:
                rows[i].append((K[at], V[at]))
                at += 1
        size = max(max(len(r) for r in rows), 1)
        kp, vp = (torch.zeros(n, hkv, R.pages(size, 256) * 256, d, device=DEV, dtype=dtype)
                  for _ in range(2))
        for i in range(n):
            for t, (k, v) in enumerate(rows[i]):
                kp[i, :, t], vp[i, :, t] = k, v
        O, _, tol, _ = R.decode(Q, kp, vp, torch.arange(n)[:, None], [len(r) for r in rows])
        got = buf["out"].cpu().double()
        assert bool(((got - O).abs() <= tol).all())
        assert cache.lens.tolist() == [len(r) for r in rows]
        assert xattn_get_device_status() == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F3, 64)])
def test_server_steps(captured, dtype, d):
    """Plan, append and decode together, step after step, with requests that
    end and start; the captured graph is replayed with each step's inputs."""
    n, hkv, hq = 6, 2, 8
    cache = PagedCache(n, 8, 30, 16, hkv, d, dtype, DEV)
    fresh = torch.zeros(n, dtype=torch.int32, device=DEV)
    Q = torch.zeros(n, hq, d, device=DEV, dtype=dtype)
    K, V = (torch.zeros(n, hkv, d, device=DEV, dtype=dtype) for _ in range(2))
    buf = {**plan_buffers(cache.table, n), **decode_buffers(Q, cache.k_pages, cache.table)}
    cache.step(Q, K, V, fresh, buf)                    # nothing new: also the warm-up
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.step(Q, K, V, fresh, buf)
    for f, q, k, v in _steps(cache, buf, 5, n, 60, hkv, hq, d, dtype):
        for dst, src in ((fresh, _i32(f)), (Q, q), (K, k), (V, v)):
            dst.copy_(src)
        if captured:
            graph.replay()
        else:
            cache.step(Q, K, V, fresh, buf)
        torch.cuda.synchronize()


def test_two_graphs_share_a_workspace():
    a = _cache([9000, 20, 600], 32, 8, 128, BF, 16, seed=1)
    b = _cache([300] * 40, 32, 8, 128, BF, 16, seed=2)
    want = [xattn_paged_decode(*x, lse=True) for x in (a, b)]
    bufs = [decode_buffers(x[0], x[1], x[3]) for x in (a, b)]
    ws = max((x["ws"] for x in bufs), key=lambda t: t.numel())
    graphs = []
    for x, y in zip((a, b), bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            xattn_paged_decode(*x, out=y["out"], lse=y["lse"], workspace=ws)
        graphs.append(g)
    for _ in range(10):
        for g, y, w in zip(graphs, bufs, want):
            y["out"].fill_(float("nan"))
            ws.fill_(0x5A)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y["out"], w[0]) and torch.equal(y["lse"], w[1])


def test_prefill_then_steps():
    """A sparse prefill of a batch, its keys and values into the cache, then
    new tokens: the decode reads what the prefill was given."""
    p = make_problem("c1", L=1024, hq=8, hkv=2, seed=3)
    Q, K, V = (torch.cat([x, x.flip(2)]).contiguous().to(DEV) for x in (p.Q, p.K, p.V))
    cache = PagedCache(3, 20, 40, 128, 2, 128, BF, DEV)
    # rows 0 and 2 take the prompts
    pre = plan_buffers(cache.table, 2 * 1024)
    O = cache.prefill(Q, K, V, p.B, p.S, p.tau.tolist(), p.causal, _i32([1024, 0, 1024]), pre)
    assert torch.equal(O, prefill_attention(Q, K, V, p.B, p.S, p.tau.tolist(), p.causal))
    assert cache.lens.tolist() == [1024, 0, 1024]
    for row, b in ((0, 0), (2, 1)):
        for pages, src in ((cache.k_pages, K), (cache.v_pages, V)):
            got = pages[cache.table[row, :8].long()].transpose(0, 1).reshape(2, 1024, 128)
            assert torch.equal(got, src[b])
    q = torch.randn(3, 8, 128, device=DEV).to(BF)
    buf = {**plan_buffers(cache.table, 3), **decode_buffers(q, cache.k_pages, cache.table)}
    new = torch.randn(2, 3, 2, 128, device=DEV).to(BF)
    out, lse = cache.step(q, new[0], new[1], _i32([1, 1, 1]), buf, lse=True)
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [1025, 1, 1025]
    ref, L, tol, tol_lse = R.decode(q, cache.k_pages, cache.v_pages, cache.table, cache.lens)
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    assert bool(((lse.cpu().double() - L).abs() <= tol_lse).all())
    # the middle row has one token: its attention is that token's value
    assert torch.equal(out[1].view(2, 4, 128), new[1][1].unsqueeze(1).expand(2, 4, 128))


def test_varlen_prefill_into_the_cache():
    lens = [1024, 520, 2048]
    probs = [make_problem("c1", L=L, hq=2, hkv=1, seed=30 + i) for i, L in enumerate(lens)]
    pack = lambda attr: torch.cat([getattr(p, attr)[0].reshape(-1, 128)
                                   for p in probs]).contiguous().to(DEV)
    Q, K, V = pack("Q"), pack("K"), pack("V")
    tau = probs[0].tau.tolist()
    cache = PagedCache(3, 20, 40, 128, 1, 128, BF, DEV)
    buf = plan_buffers(cache.table, sum(lens))
    O = cache.prefill_varlen(Q, K, V, lens, 2, 128, 8, tau, True, _i32(lens), buf)
    assert torch.equal(O, xattn_prefill_varlen(Q, K, V, lens, 2, 1, 128, 8, True, tau))
    at = 0
    for i, L in enumerate(lens):
        got = cache.k_pages[cache.table[i].long().clamp(min=0), 0].reshape(-1, 128)[:L]
        assert torch.equal(got, K[at:at + L])
        at += L
