"""The paged cache as a server holds it: rows that wait between the busy ones, entries
that are no pages, and calls that are refused or captured."""
import pytest
import torch

from block_sparse_long_score_b200 import (PagedCache, XattnError, decode_buffers, plan_buffers,
                                          prefill_attention, xattn_get_device_status,
                                          xattn_paged_append, xattn_paged_decode,
                                          xattn_paged_plan)
from block_sparse_long_score_b200.synth import make_problem
from tests import paged_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F3 = torch.bfloat16, torch.float32


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _us(call, times=5):
    """Least device time of a call, in microseconds."""
    call()
    best = float("inf")
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000)
    return best


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("bad", [-1, 10, 1 << 20, -(1 << 31)])
def test_plan_reports_what_an_ended_request_gives_back(n, bad):
    """Request 0 ends with an entry that is no page: it goes to the ring as it is, and the
    step reports it."""
    fill = n - 3
    lens, fresh = [20, 16, 5] + [0] * fill, [-1, 0, 1] + [0] * fill
    table = [[3, bad], [1, -1], [2, -1]] + [[-1, -1]] * fill
    t = [_i32(x) for x in (lens, fresh, [8, 3], [6, 0, 0, 0, 0, 0, 0, 0, 4, 5], table)]
    out = (t[0], t[2], _i32([7] * (n + 1)), _i32([7] * 2))
    assert xattn_get_device_status() == 0
    xattn_paged_plan(*t, 16, out=out)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == -1
    assert out[0].tolist() == [0, 16, 6] + [0] * fill and out[1].tolist() == [8, 5]
    assert out[2].tolist() == [0, 0, 0, 1] + [1] * fill and out[3].tolist() == [37, -1]
    assert t[3].tolist() == [6, 3, bad, 0, 0, 0, 0, 0, 4, 5] and t[4].tolist() == table


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("starts,kept", [([0, 4, 2], []), ([0, 2, 9], [0, 1]), ([-3, 2, 3], [2]),
                                         ([1, 2, 3], [1, 2])])
def test_append_leaves_out_what_broken_starts_misplace(starts, kept):
    """Tokens of a request whose starts are no prefix sum over K's rows are reported and left
    out; the others land where they belong."""
    kp, vp = (torch.full((4, 1, 16, 64), -9.0, device=DEV) for _ in range(2))
    K = torch.arange(3.0 * 64, device=DEV).reshape(3, 64)
    want_k, want_v = kp.clone(), vp.clone()
    for t in kept:
        want_k[0, 0, 5 + t], want_v[0, 0, 5 + t] = K[t], K[t] + 1000
    xattn_paged_append(K, K + 1000, _i32([5, 6, 7]), kp, vp, starts=_i32(starts))
    torch.cuda.synchronize()
    assert xattn_get_device_status() == -1
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def _prompts(n, rows, lens, hkv, d, dtype):
    """K, V, slots, starts and pages of prompts that enter the given rows of n."""
    T, page = sum(lens), 16
    g = torch.Generator(device=DEV).manual_seed(T)
    N = R.pages(T, page) + 1
    slots = torch.randperm(N * page, device=DEV, generator=g)[:T].to(torch.int32)
    K, V = (torch.randn(T * hkv, d, device=DEV, generator=g).to(dtype) for _ in range(2))
    grow = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    for r, L in zip(rows, lens):
        grow[r + 1] = L
    kp, vp = (torch.zeros(N, hkv, page, d, device=DEV, dtype=dtype) for _ in range(2))
    return K, V, slots, grow.cumsum(0).to(torch.int32), kp, vp


@pytest.mark.parametrize("n,rows,lens", [
    (65536, (0, 65535), (601, 1200)), (65536, (7, 8, 40000), (1000, 1, 999)),
    (5000, (0, 1, 2, 3, 4997, 4999), (1, 300, 2, 1700, 33, 1201)), (33, (31, 32), (5000, 4100)),
    (1 << 20, (3, (1 << 20) - 1), (4001, 6001))])
def test_append_finds_its_rows_among_idle_ones(n, rows, lens):
    hkv, d = 2, 64
    K, V, slots, starts, kp, vp = _prompts(n, rows, lens, hkv, d, BF)
    want_k, want_v, at, page = kp.clone(), vp.clone(), 0, 16
    for L in lens:
        s = slots[at:at + L].long()
        for want, x in ((want_k, K), (want_v, V)):
            want[s // page, :, s % page] = \
                x[at * hkv:(at + L) * hkv].reshape(hkv, L, d).transpose(0, 1)
        at += L
    xattn_paged_append(K, V, slots, kp, vp, starts=starts)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_append_does_not_walk_the_idle_rows():
    """Two prompts in the first and last of 65536 rows take about the time that they take
    in the first two; a CTA holds tokens of both (the first prompt's length is odd)."""
    n = 65536
    near, far = (_prompts(n, rows, (1201, 2000), 2, 64, BF) for rows in ((0, 1), (0, n - 1)))
    us = [_us(lambda: xattn_paged_append(x[0], x[1], x[2], x[4], x[5], starts=x[3]))
          for x in (near, far)]
    assert us[1] < 3 * us[0] + 20, us


# ---------------------------------------------------------------- decode

def _busy(n, rows, lens, hq, hkv, d, dtype, width):
    g = torch.Generator(device=DEV).manual_seed(n)
    page = 16
    have = [R.pages(x, page) for x in lens]
    N = sum(have) + 1
    kp, vp = (torch.randn(N, hkv, page, d, device=DEV, generator=g).to(dtype) for _ in range(2))
    perm = torch.randperm(N, device=DEV, generator=g).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    L, at = torch.zeros(n, dtype=torch.int32, device=DEV), 0
    for r, size, h in zip(rows, lens, have):
        table[r, :h] = perm[at:at + h]
        L[r] = size
        at += h
    return torch.randn(n, hq, d, device=DEV, generator=g).to(dtype), kp, vp, table, L


@pytest.mark.parametrize("n,rows,lens", [
    (20000, (0, 19999), (9000, 9000)), (4096, (0, 31, 32, 33, 64, 97, 4000), (700,) * 7),
    (4096, tuple(range(5, 4096, 61)), tuple(range(1, 69))), (130, (0, 129), (3000, 1)),
    (3000, (2999,), (5000,)), (100, (1, 34, 67, 99), (2000, 90, 700, 1))])
@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF, 8, 2, 64), (BF, 32, 2, 128), (F3, 4, 2, 32)])
def test_decode_of_few_busy_rows_among_idle_ones(n, rows, lens, dtype, hq, hkv, d):
    Q, kp, vp, table, L = _busy(n, rows, lens, hq, hkv, d, dtype, 600)
    O, lse = xattn_paged_decode(Q, kp, vp, table, L, lse=True)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    busy = torch.tensor(rows, device=DEV)
    want, L64, tol, tol_lse = R.decode(Q[busy], kp, vp, table[busy], L[busy])
    assert bool(((O[busy].cpu().double() - want).abs() <= tol).all())
    assert bool(((lse[busy].cpu().double() - L64).abs() <= tol_lse).all())
    idle = L == 0
    assert bool((O[idle] == 0).all()) and bool((lse[idle] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_of_many_short_busy_rows_far_apart(dtype):
    """Enough short requests for the split by warps, idle rows between them."""
    n = 20000
    rows = list(range(3, n, 29))
    lens = [1 + (11 * i) % 60 for i in range(len(rows))]
    Q, kp, vp, table, L = _busy(n, rows, lens, 8, 4, 64, dtype, 40)
    O, lse = xattn_paged_decode(Q, kp, vp, table, L, lse=True)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == 0
    busy = torch.tensor(rows, device=DEV)
    want, L64, tol, tol_lse = R.decode(Q[busy], kp, vp, table[busy], L[busy])
    assert bool(((O[busy].cpu().double() - want).abs() <= tol).all())
    assert bool(((lse[busy].cpu().double() - L64).abs() <= tol_lse).all())
    assert bool((O[L == 0] == 0).all()) and bool((lse[L == 0] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F3])
def test_decode_does_not_walk_the_idle_rows(dtype):
    """Requests spread over 65536 rows take about the time that they take in the first ones;
    their lengths put ends of units inside CTAs' ranges. A CTA's range crosses one gap of 8190 rows
    at most, and two walks of it, 128 rows a step, are 2 x 64 dependent reads of 1 us at the
    very most; row by row they are 2 x 8190 reads, 800 us as measured. (The scan of the lengths,
    512 rows a thread, differs by up to 50 us itself.)"""
    n, lens = 65536, [14000 + 331 * i for i in range(9)]
    near, far = (_busy(n, rows, lens, 8, 2, 64, dtype, 1100)
                 for rows in (range(9), range(0, n, n // 8 - 1)))
    us = [_us(lambda: xattn_paged_decode(*x)) for x in (near, far)]
    assert us[1] < us[0] + 128 + 50, us


# ----------------------------------------------------- refusals, capture

def _state(c):
    return [x.clone() for x in (c.lens, c.pool, c.table, c.ring)]


def _unchanged(c, before):
    torch.cuda.synchronize()
    return all(torch.equal(x, y) for x, y in zip(_state(c), before))


def test_a_refused_step_enters_nothing():
    c = PagedCache(2, 4, 8, 16, 2, 128, BF, DEV)
    Q = torch.randn(2, 8, 128, device=DEV).to(BF)
    K, V = (torch.randn(2, 2, 128, device=DEV).to(BF) for _ in range(2))
    buf = {**plan_buffers(c.table, 2), **decode_buffers(Q, c.k_pages, c.table)}
    fresh = _i32([1, 1])
    c.step(Q, K, V, fresh, buf)
    before = _state(c)
    shifted = torch.empty(2 * 2 * 128 + 4, device=DEV, dtype=BF)[4:].view(2, 2, 128)
    stride = torch.empty(2, 2 * 128 + 4, device=DEV, dtype=BF)[:, :256].unflatten(1, (2, 128))
    odd_q = torch.empty(2 * 8 * 128 + 4, device=DEV, dtype=BF)[4:].view(2, 8, 128)
    for q, k, v, b in ((Q, K[:1], V, buf), (Q, K.float(), V, buf), (Q, K, V.cpu(), buf),
                       (Q[:1], K, V, buf), (Q.float(), K, V, buf), (Q[..., :64], K, V, buf),
                       (Q, shifted, V, buf), (Q, K, shifted, buf), (Q, stride, stride, buf),
                       (odd_q, K, V, buf), (Q, K, V, {**buf, "out": buf["out"][:1]}),
                       (Q, K, V, {**buf, "out": odd_q}), (Q, K, V, {**buf, "ws": buf["ws"][:64]}),
                       (Q, K, V, {**buf, "ws": buf["ws"][8:]}),
                       (Q, K, V, {**buf, "lse": buf["lse"][:, :4]}),
                       (torch.zeros(2, 7, 128, device=DEV, dtype=BF), K, V,
                        {**buf, "out": torch.zeros(2, 7, 128, device=DEV, dtype=BF),
                         "lse": buf["lse"][:, :7].contiguous()})):
        with pytest.raises((ValueError, XattnError)):
            c.step(q, k, v, fresh, b, lse=True)
        assert _unchanged(c, before)
    c.step(Q, K, V, fresh, buf)
    assert c.lens.tolist() == [2, 2] and xattn_get_device_status() == 0


def test_a_refused_prefill_enters_nothing():
    p = make_problem("c1", L=1024, hq=8, hkv=2, seed=3)
    Q, K, V = (x.contiguous().to(DEV) for x in (p.Q, p.K, p.V))
    tau = p.tau.tolist()
    c = PagedCache(2, 20, 40, 128, 2, 128, BF, DEV)
    before, fresh = _state(c), _i32([1024, 0])
    buf, large = plan_buffers(c.table, 1024), plan_buffers(c.table, 2048)
    for q, k, v, B, t, b in ((Q, K, V, p.B, tau, large), (Q, K, V[:, :1], p.B, tau, buf),
                             (Q, K, V, 100, tau, buf), (Q, K, V, p.B, [2.0] * 8, buf),
                             (Q, K, V, p.B, tau[:3], buf), (Q[:, :7], K, V, p.B, tau, buf),
                             (Q, K.float(), V.float(), p.B, tau, buf)):
        with pytest.raises((ValueError, XattnError)):
            c.prefill(q, k, v, B, p.S, t, p.causal, fresh, b)
        assert _unchanged(c, before)
    flat = [x[0].reshape(-1, 128) for x in (Q, K, V)]
    for seqlens, t, b in (([1024], tau, large), ([1000], tau, buf), ([1024], [0.0] * 8, buf)):
        with pytest.raises((ValueError, XattnError)):
            c.prefill_varlen(*flat, seqlens, 8, p.B, p.S, t, p.causal, fresh, b)
        assert _unchanged(c, before)
    c.prefill(Q, K, V, p.B, p.S, tau, p.causal, fresh, buf)
    assert c.lens.tolist() == [1024, 0] and xattn_get_device_status() == 0


def test_a_captured_prefill_takes_new_prompts():
    """A prefill captured with thresholds on the device and replayed: other prompts into other
    rows, the first ones ended in between."""
    p = make_problem("c1", L=1024, hq=8, hkv=2, seed=3)
    Q, K, V = (x.contiguous().to(DEV) for x in (p.Q, p.K, p.V))
    tau = torch.from_numpy(p.tau).to(DEV)
    c = PagedCache(3, 9, 20, 128, 2, 128, BF, DEV)
    fresh = _i32([0, 0, 0])
    buf = plan_buffers(c.table, 1024)
    c.prefill(Q, K, V, p.B, p.S, tau, p.causal, fresh, buf)      # nothing new: the warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = c.prefill(Q, K, V, p.B, p.S, tau, p.causal, fresh, buf)
    end = plan_buffers(c.table, 0)
    for turn, (row, ended) in enumerate(((1, None), (0, 1), (2, 0), (1, 2))):
        if ended is not None:
            c.plan(_i32([-1 if i == ended else 0 for i in range(3)]), end)
        for dst in (Q, K, V):
            dst.copy_(dst.flip(2))
        fresh.copy_(_i32([1024 if i == row else 0 for i in range(3)]))
        graph.replay()
        torch.cuda.synchronize()
        assert xattn_get_device_status() == 0
        assert torch.equal(O, prefill_attention(Q, K, V, p.B, p.S, tau, p.causal)), turn
        assert c.lens[row].item() == 1024 and c.lens.sum().item() == 1024
        for pages, src in ((c.k_pages, K), (c.v_pages, V)):
            got = pages[c.table[row, :8].long()].transpose(0, 1).reshape(2, 1024, 128)
            assert torch.equal(got, src[0])
