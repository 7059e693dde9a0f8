"""What the decode over a paged cache keeps of its inputs: softmax weights held in
more bits than the tensors' type, values near the top of the type's range, and
every token counted once however long a request and however the work is cut.

The reference is the definition in fp64 on the GPU (``_exact``)."""
import math
import random

import pytest
import torch

from block_sparse_long_score_b200 import xattn_get_device_status, xattn_paged_decode
from tests import paged_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F3 = torch.bfloat16, torch.float32
TYPES = [(BF, 128), (BF, 64), (F3, 128), (F3, 64), (F3, 32)]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(pages, row, size):
    """[hkv, size, d] of a request whose pages are ``row``, without the tokens of
    entries that are no page."""
    page = pages.shape[2]
    t = torch.arange(size, device=DEV)
    at = row.long()[t // page]
    ok = (at >= 0) & (at < pages.shape[0])
    return pages[at[ok], :, (t % page)[ok]].transpose(0, 1)


def _exact(Q, kp, vp, table, lens):
    """O, lse, the weights' sum of |V|, and the largest sum of |q||k| / sqrt(d), in fp64."""
    n, hq, d = Q.shape
    hkv = kp.shape[1]
    O = torch.zeros(n, hkv, hq // hkv, d, dtype=torch.float64, device=DEV)
    A, lse = torch.zeros_like(O), torch.full(O.shape[:3], -math.inf, dtype=torch.float64,
                                             device=DEV)
    size_s = torch.zeros_like(lse)
    for i, size in enumerate(lens.tolist()):
        if size == 0:
            continue
        q = Q[i].double().reshape(hkv, hq // hkv, d) / math.sqrt(d)
        k, v = _rows(kp, table[i], size).double(), _rows(vp, table[i], size).double()
        s = q @ k.transpose(1, 2)
        lse[i] = torch.logsumexp(s, 2)
        p = torch.exp(s - lse[i][..., None])
        O[i], A[i] = p @ v, p @ v.abs()
        size_s[i] = (q.abs() @ k.abs().transpose(1, 2)).amax(2)
    flat = lambda x: x.reshape(n, hq, *x.shape[3:])
    return flat(O), flat(lse), flat(A), flat(size_s)


def _table(lens, page, extra=1, width=0, seed=0):
    """A table of shuffled pages, and how many pages the pool has."""
    have = [R.pages(x, page) for x in lens]
    N = sum(have) + extra
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = max(max(have), 1, width)
    table, at = [], 0
    for h in have:
        table.append(perm[at:at + h] + [-1] * (rows - h))
        at += h
    return _i32(table), N


def _decode(Q, kp, vp, table, lens, status=0):
    O, lse = xattn_paged_decode(Q, kp, vp, table, lens, lse=True)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == status
    return O.double(), lse.double()


# 21 requests of few tokens are cut by units or, in a wide table, by ranges; 140 on 8 KV
# heads by warps
@pytest.mark.parametrize("lens,hkv,width", [([2, 3, 5, 9, 17, 33, 100] * 3, 2, 0),
                                            ([2, 3, 5, 9, 17, 33, 100] * 3, 2, 600),
                                            ([2, 3, 5, 9, 17, 33, 100] * 20, 8, 0),
                                            ([2, 3, 5, 9, 17, 33, 100] * 20, 8, 600),
                                            ([700, 2500], 1, 0)])
@pytest.mark.parametrize("group", [1, 4, 8, 12, 32])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_weights_are_held_in_more_bits_than_the_tensors(dtype, d, group, lens, hkv, width):
    """The last value row cancels what the others add up to, in feature j for the
    j-th query head of the group (modulo its size), so O's own rounding hides
    nothing there: what is left of O is the error of the weights."""
    g = torch.Generator(device=DEV).manual_seed(d + group)
    page, n = 16, len(lens)
    table, N = _table(lens, page, width=width)
    kp, vp = (torch.randn(N, hkv, page, d, device=DEV, generator=g).to(dtype) for _ in range(2))
    Q = (0.5 * torch.randn(n, group * hkv, d, device=DEV, generator=g)).to(dtype)
    head = torch.arange(d, device=DEV) % group
    for i, size in enumerate(lens):
        k, v = _rows(kp, table[i], size).double(), _rows(vp, table[i], size).double()
        q = Q[i].double().reshape(hkv, group, d) / math.sqrt(d)
        p = torch.softmax(q @ k.transpose(1, 2), 2)[:, head]              # [hkv, d, size]
        last = -(p[..., :-1] * v[:, :-1].transpose(1, 2)).sum(2) / p[..., -1]
        vp[table[i, (size - 1) // page], :, (size - 1) % page] = last.to(dtype)
    L = _i32(lens)
    O, lse, A, size_s = _exact(Q, kp, vp, table, L)
    got, got_lse = _decode(Q, kp, vp, table, L)
    # O is rounded once (half a step). A weight: two terms of 8 bits hold it to 2^-8 of
    # 2^-8 in bf16, fp32 holds it as it is; a logit's d products and sums, scale and base-2
    # factor are off by a step of 2^-23 each; the exponential by 2^-21. Sums: a step for
    # each token (a tensor core may cut each of its terms) and each of up to 64 joins.
    half = R.BF16_HALF if dtype == BF else R.F32_HALF
    weight = 2.0 ** -16 if dtype == BF else 0.0
    ds = (d + 6) * 2.0 ** -23 * size_s
    sums = (L.double()[:, None] + 64) * 2.0 ** -23
    tol = A * (weight + 2 * ds + sums + 2.0 ** -20)[..., None]
    tol += half * (O.abs() + tol) + 1e-30
    err = (got - O).abs()
    assert bool((err <= tol).all()), f"{(err / tol).max().item():.3g} times its bound"
    assert bool(((got_lse - lse).abs() <= ds + sums + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all())


@pytest.mark.parametrize("n,hkv,width", [(1, 1, 0), (1, 1, 2000), (40, 8, 0), (140, 8, 0), (140, 8, 600)])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_values_near_the_top_of_the_range(dtype, d, n, hkv, width):
    """One token of 80 has two thirds of the weight, far above the tokens before it, and every
    value is 1e38: O is 1e38, although weights above 3.4 times it are no longer finite."""
    lens = [80] * n
    table, N = _table(lens, 16, width=width)
    kp = torch.zeros(N, hkv, 16, d, device=DEV, dtype=dtype)
    vp = torch.full_like(kp, 1e38)
    for i in range(n):
        kp[table[i, 70 // 16], :, 70 % 16, 3] = 5.0 * math.sqrt(d)
    Q = torch.zeros(n, 4 * hkv, d, device=DEV, dtype=dtype)
    Q[..., 3] = 1.0
    got, lse = _decode(Q, kp, vp, table, _i32(lens))
    # O: half a step, twice (of the weights' sum and of O), and 100 fp32 steps on the way
    want = vp[0, 0, 0, 0].double()
    half = R.BF16_HALF if dtype == BF else R.F32_HALF
    assert bool(((got - want).abs() <= want * (half + 2.0 ** -16 + 100 * 2.0 ** -23)).all())
    # lse: base-2 terms of up to 16 (a scale, a product, a maximum), natural ones of up to 11 and 6,
    # an exponential: some 60 steps of 2^-23 and 2^-21
    key = kp[table[0, 4], 0, 6, 3].double().item() / math.sqrt(d)
    assert bool(((lse - math.log(79 + math.exp(key))).abs() <= 2.0 ** -16).all())


@pytest.mark.parametrize("lens,hkv,width", [([1, 17, 300, 2000], 2, 0), ([1, 17, 300, 2000], 2, 900),
                                            ([90] * 140, 8, 0), ([90] * 140, 8, 600)])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_logits_that_are_all_minus_infinity(dtype, d, lens, hkv, width):
    """The second query head of each group of three sees no key at all; its neighbours do."""
    table, N = _table(lens, 16, width=width)
    g = torch.Generator(device=DEV).manual_seed(d)
    kp, vp = (torch.randn(N, hkv, 16, d, device=DEV, generator=g).to(dtype) for _ in range(2))
    kp[..., 1] = -math.inf
    Q = torch.randn(len(lens), 3 * hkv, d, device=DEV, generator=g).to(dtype)
    Q[..., 1] = 0.0
    got, lse = _decode(Q, kp, vp, table, _i32(lens))
    assert bool(got.isnan().all()) and bool(lse.isnan().all())      # 0 times an infinity
    kp[..., 1] = torch.finfo(dtype).min
    Q[:, 1::3, 1] = torch.finfo(dtype).max                          # a logit past fp32's range
    got, lse = _decode(Q, kp, vp, table, _i32(lens))
    sees = torch.arange(3 * hkv, device=DEV) % 3 != 1
    assert bool((got[:, ~sees] == 0).all()) and bool((lse[:, ~sees] == -math.inf).all())
    L = _i32(lens)
    O, want, A, size_s = _exact(Q[:, sees], kp, vp, table, L)
    half = R.BF16_HALF if dtype == BF else R.F32_HALF
    weight = 2.0 ** -16 if dtype == BF else 0.0      # the bounds of the first test
    ds = (d + 6) * 2.0 ** -23 * size_s
    sums = (L.double()[:, None] + 64) * 2.0 ** -23
    tol = A * (weight + 2 * ds + sums + 2.0 ** -20)[..., None]
    tol += half * (O.abs() + tol) + 1e-30
    assert bool(((got[:, sees] - O).abs() <= tol).all())
    assert bool(((lse[:, sees] - want).abs() <= ds + sums + 2.0 ** -20 + 2.0 ** -22 * want.abs()).all())


@pytest.mark.parametrize("n,hkv,width", [(2, 2, 0), (2, 2, 2000), (140, 8, 0), (140, 8, 600)])
@pytest.mark.parametrize("group", [3, 12, 32])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_infinite_values_of_tokens_that_weigh_next_to_nothing(dtype, d, group, n, hkv, width):
    """Token t's value is infinite in feature t and its weight falls from 1 to e^-80 or so,
    which fp32 holds: O is infinite there, with the value's sign, and finite elsewhere."""
    T = d // 2
    table, N = _table([T + 3] * n, 16, width=width)
    g = torch.Generator(device=DEV).manual_seed(d)
    kp, vp = torch.zeros(N, hkv, 16, d, device=DEV, dtype=dtype), \
        torch.randn(N, hkv, 16, d, device=DEV, generator=g).to(dtype)
    t = torch.arange(T, device=DEV)
    sign = torch.where(t % 3 == 1, -1.0, 1.0).to(dtype)
    for i in range(n):
        at = table[i].long()[t // 16]
        kp[at, :, t % 16, 3] = (-(78.0 / T) * math.sqrt(d) * t)[:, None].to(dtype)
        vp[at, :, t % 16, t] = (sign * math.inf)[:, None]
    Q = torch.zeros(n, group * hkv, d, device=DEV, dtype=dtype)
    kp[..., 5] = torch.randn(N, hkv, 16, device=DEV, generator=g).to(dtype)
    Q[..., 3], Q[..., 5] = 1.0, torch.rand(n, group * hkv, device=DEV, generator=g).to(dtype)
    got, lse = _decode(Q, kp, vp, table, _i32([T + 3] * n))
    assert bool((got[..., :T] == sign.double() * math.inf).all())
    assert bool(got[..., T:].isfinite().all()) and bool(lse.isfinite().all())


def _marked_pages(N, hkv, page, d, dtype, seed):
    """Values that mark their token's place: piece p of 8 tokens of the pool has a 1 in feature
    p % d and zeros elsewhere. With equal weights O then counts a request's pieces by feature."""
    vp = torch.zeros(N * page // 8, 8, hkv, d, device=DEV, dtype=dtype)
    piece = torch.arange(N * page // 8, device=DEV)
    mark = torch.randint(0, d, (N * page // 8,), device=DEV,
                         generator=torch.Generator(device=DEV).manual_seed(seed))
    vp[piece, :, :, mark] = 1.0
    kp = torch.randn(N, hkv, page, d, device=DEV).to(dtype)
    return kp, vp.reshape(N, page, hkv, d).transpose(1, 2).contiguous()


def _check_counts(Q, kp, vp, table, lens, status=0):
    """Q = 0: each token counts once. The sum of equal weights, a power of two, is exact, so lse
    is off by the logarithm's and the last sum's steps only; O is a count of tokens over all
    tokens, rounded once, which tells whether a piece of 8 tokens is left out or counted twice."""
    got, got_lse = _decode(Q, kp, vp, table, lens, status)
    n, hq, d = Q.shape
    hkv = kp.shape[1]
    half = R.BF16_HALF if Q.dtype == BF else R.F32_HALF
    for i, size in enumerate(lens.tolist()):
        v = _rows(vp, table[i], size)
        count, T = v.double().sum(1).repeat_interleave(hq // hkv, 0), v.shape[1]
        if T == 0:
            assert bool((got[i] == 0).all()) and bool((got_lse[i] == -math.inf).all())
            continue
        # (a base-2 logarithm below 40, its factor and the natural logarithm below 28, each off
        # by a step or two of 2^-23)
        assert bool(((got_lse[i] - math.log(T)).abs() <= 2.0 ** -23 * 2 * (28 + 28)).all()), i
        err = (got[i] * T - count).abs()
        assert bool((err <= count * (half + 2.0 ** -20)).all()), (i, err.max().item())
        assert bool((count * (half + 2.0 ** -20) < 8).all())     # less than a piece


COUNTS = [([20011], 1, 32, 0), ([20011], 3, 64, 2000), ([40000, 1, 0, 39999], 2, 16, 0),
          ([4095, 4096, 4097, 1, 0, 8, 100], 4, 16, 0), ([4095, 4096, 4097, 1, 0, 8, 100], 4, 16, 700),
          ([(97 * i) % 289 for i in range(200)], 7, 16, 0),
          ([(97 * i) % 289 for i in range(200)], 7, 16, 700),
          ([(37 * i) % 500 for i in range(150)] + [16500], 5, 16, 0)]


@pytest.mark.parametrize("lens,hkv,page,width", COUNTS)
@pytest.mark.parametrize("group", [1, 4, 9])
@pytest.mark.parametrize("dtype,d", TYPES)
def test_every_token_counts_once(dtype, d, group, lens, hkv, page, width):
    table, N = _table(lens, page, width=width, seed=len(lens))
    kp, vp = _marked_pages(N, hkv, page, d, dtype, len(lens))
    Q = torch.zeros(len(lens), group * hkv, d, device=DEV, dtype=dtype)
    _check_counts(Q, kp, vp, table, _i32(lens))


def _long_units(dtype, d, page, bad):
    """64 requests whose tokens take a CTA more than 130 tiles each, so that a warp reads page ids
    for its 65th step and beyond, again and again; ranges begin inside units. The rows share the
    pool's pages, each in an order of its own."""
    tokens = 62500 if dtype == BF else 33000
    rng = random.Random(d)
    lens = [tokens - rng.randrange(300) for _ in range(64)]
    cols = R.pages(tokens, page)
    N = cols + cols // 2
    g = torch.Generator(device=DEV).manual_seed(d)
    table = torch.stack([torch.randperm(N, device=DEV, generator=g)[:cols] for _ in lens]).int()
    for i in range(0, 64, 5) if bad else ():
        table[i, rng.randrange(cols // 3, cols)] = -1 if i % 2 else N
    return lens, table, N


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("dtype,d,group,page", [(BF, 128, 4, 64), (BF, 64, 9, 16), (F3, 64, 2, 16),
                                                (F3, 32, 8, 128), (F3, 128, 1, 32)])
def test_page_ids_of_long_units(dtype, d, group, page, bad):
    lens, table, N = _long_units(dtype, d, page, bad)
    kp, vp = _marked_pages(N, 1, page, d, dtype, 1)
    L = _i32(lens)
    _check_counts(torch.zeros(64, group, d, device=DEV, dtype=dtype), kp, vp, table, L,
                  status=-1 if bad else 0)
    g = torch.Generator(device=DEV).manual_seed(3)
    Q = torch.randn(64, group, d, device=DEV, generator=g).to(dtype)
    O, lse, A, size_s = _exact(Q, kp, vp, table, L)
    got, got_lse = _decode(Q, kp, vp, table, L, status=-1 if bad else 0)
    half = R.BF16_HALF if dtype == BF else R.F32_HALF
    weight = 2.0 ** -16 if dtype == BF else 0.0
    ds = (d + 6) * 2.0 ** -23 * size_s
    # a warp adds a CTA's every fourth chunk, of 17 terms, each of which may be cut by a step;
    # half of a unit's tokens are more than one CTA gets
    sums = (L.double()[:, None] / 8 + 64) * 2.0 ** -23
    tol = A * (weight + 2 * ds + sums + 2.0 ** -20)[..., None]
    tol += half * (O.abs() + tol)
    assert bool(((got - O).abs() <= tol).all())
    assert bool(((got_lse - lse).abs() <= ds + sums + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all())
