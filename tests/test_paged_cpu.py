"""Host checks of the paged-cache entry points (nothing is launched) and the
tests' own plain plan."""
import ctypes

import pytest
import torch

from block_sparse_long_score_b200 import build as xbuild
from block_sparse_long_score_b200 import xattn as X
from tests import paged_ref as R

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every call below fails its host checks
ODD = ctypes.c_void_p(0x10008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    xbuild.build()
    return X._lib()


def _shape(**kw):
    a = dict(nseq=2, max_pages=8, num_pages=16, page_size=16, hq=8, hkv=2, d=128,
             dtype=X.XATTN_BF16)
    a.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    d, page, hkv = a["d"], a["page_size"], a["hkv"]
    return X._Paged(*[a[k] for k in ("nseq", "max_pages", "num_pages", "page_size", "hq", "hkv",
                                     "d", "dtype")],
                    kw.get("page_stride", hkv * page * d), kw.get("head_stride", page * d),
                    kw.get("token_stride", d))


def _decode(lib, s, Q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, O=FAKE, lse=None, ws=FAKE,
            ws_bytes=BIG):
    return lib.xattn_paged_decode(Q, k, v, ctypes.byref(s) if s is not None else None, table,
                                  lens, O, lse, ws, ws_bytes, None)


def _append(lib, s, K=FAKE, V=FAKE, tokens=4, layout=0, stride=256, slots=FAKE, starts=FAKE,
            k=FAKE, v=ctypes.c_void_p(0x20000)):
    return lib.xattn_paged_append(K, V, ctypes.byref(s) if s is not None else None, tokens,
                                  layout, stride, slots, starts, k, v, None)


BAD_SHAPES = [
    (dict(nseq=0), -1), (dict(hkv=0), -1), (dict(hkv=-1), -1), (dict(num_pages=0), -1),
    (dict(page_size=0), -1), (dict(dtype=2), -1), (dict(d=0), -1),
    (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(page_size=512), -2),
    (dict(d=32), -2), (dict(d=96), -2), (dict(d=256), -2),
    (dict(d=96, dtype=X.XATTN_F32), -2),
    (dict(num_pages=1 << 27), -2), (dict(nseq=(1 << 20) + 1), -2),
    (dict(token_stride=64), -1), (dict(token_stride=132), -1), (dict(head_stride=0), -1),
    (dict(page_stride=-2048), -1), (dict(page_stride=1 << 41), -1),
]


@pytest.mark.parametrize("kw,code", BAD_SHAPES + [(dict(max_pages=0), -1), (dict(hq=0), -1),
                                                  (dict(hq=7), -1), (dict(hq=512), -2),
                                                  (dict(max_pages=(1 << 26) + 1), -2)])
def test_decode_refuses_bad_shapes(lib, kw, code):
    s = _shape(**kw)
    assert _decode(lib, s) == code
    assert X.xattn_paged_decode_workspace_bytes(s) == 0


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_append_refuses_bad_shapes(lib, kw, code):
    assert _append(lib, _shape(**kw)) == code


def test_decode_refuses_bad_pointers_and_workspaces(lib):
    s = _shape()
    need = X.xattn_paged_decode_workspace_bytes(s)
    assert need > 0
    assert _decode(lib, None) == -1
    for name in ("Q", "k", "v", "table", "lens", "O"):
        assert _decode(lib, s, **{name: None}) == -1, name
    for name in ("Q", "k", "v", "O", "ws"):
        assert _decode(lib, s, **{name: ODD}) == -1, name
    assert _decode(lib, s, lse=ctypes.c_void_p(0x10002)) == -1
    assert _decode(lib, s, ws=None) == -4
    assert _decode(lib, s, ws_bytes=need - 1) == -4


def test_append_refuses_bad_arguments(lib):
    s = _shape()
    assert _append(lib, None) == -1
    for name in ("K", "V", "slots", "k", "v"):
        assert _append(lib, s, **{name: None}) == -1, name
    for name in ("K", "V", "k", "v"):
        assert _append(lib, s, **{name: ODD}) == -1, name
    assert _append(lib, s, v=FAKE) == -1                     # K and V pages are one array
    assert _append(lib, s, tokens=-1) == -1
    assert _append(lib, s, layout=2) == -1
    assert _append(lib, s, layout=1, starts=None) == -1
    assert _append(lib, s, stride=255) == -1                 # below hkv * d
    assert _append(lib, s, stride=260) == -1                 # not a multiple of 16 bytes
    assert _append(lib, s, tokens=0, K=None, slots=None) == 0   # nothing to do, nothing launched


def _plan(lib, nseq=2, page=16, pages=16, rows=8, tokens=4, **kw):
    names = ("lens", "fresh", "pool", "ring", "table", "lens_out", "pool_out", "starts", "slots")
    return lib.xattn_paged_plan(nseq, page, pages, rows, tokens,
                                *[kw.get(n, FAKE) for n in names], None)


def test_plan_refuses_bad_arguments(lib):
    for kw, code in ((dict(nseq=0), -1), (dict(page=0), -1), (dict(page=17), -2),
                     (dict(pages=0), -1), (dict(rows=0), -1), (dict(tokens=-1), -1),
                     (dict(pages=1 << 27), -2), (dict(rows=(1 << 26) + 1), -2),
                     (dict(nseq=(1 << 20) + 1), -2)):
        assert _plan(lib, **kw) == code, kw
    for name in ("lens", "fresh", "pool", "ring", "table", "lens_out", "pool_out", "starts",
                 "slots"):
        assert _plan(lib, **{name: None}) == -1, name


def test_the_pages_error_has_a_text(lib):
    assert X.xattn_strerror(-6) == "not enough free pages"


def test_binding_refuses_host_tensors_and_wrong_shapes():
    kp = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    Q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        X.xattn_paged_decode(Q, kp, kp.clone(), t, n)
    with pytest.raises(ValueError):
        X.xattn_paged_append(Q, Q, n, kp, kp.clone())
    with pytest.raises(ValueError):
        X.xattn_paged_plan(n, n, torch.zeros(2, dtype=torch.int32), n, t, 16, 4)
    with pytest.raises(ValueError):
        X.make_paged(kp.half(), 8, 1, 4)
    with pytest.raises(ValueError):
        X.make_paged(kp.transpose(2, 3), 8, 1, 4)
    with pytest.raises(ValueError):
        X.make_paged(kp[0], 8, 1, 4)


def test_make_paged_reads_the_strides():
    kp = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)
    s = X.make_paged(kp, 8, 3, 5)
    assert (s.num_pages, s.hkv, s.page_size, s.d) == (4, 2, 16, 128)
    assert (s.page_stride, s.head_stride, s.token_stride) == (4096, 128, 256)
    both = torch.zeros(4, 2, 1, 16, 64)      # K and V of a page side by side, one head
    s = X.make_paged(both[:, 0], 1, 3, 5)
    assert (s.page_stride, s.token_stride, s.dtype) == (2048, 64, X.XATTN_F32)


def test_the_plain_plan_by_hand():
    """Two requests of 15 and 16 tokens take one token each: the second needs a
    page; a third ends and gives its two pages back at the ring's tail."""
    out = R.plan([15, 16, 17], [1, 1, -1], [4, 2], [8, 9, -1, -1, 5, 7],
                 [[0, -1], [1, -1], [2, 3]], 16, 3)
    lens, pool, starts, slots, ring, table, fault = out
    assert (lens, pool, starts, slots) == ([16, 17, 0], [5, 3], [0, 1, 2, 2], [15, 80, -1])
    assert table == [[0, -1], [1, 5], [2, 3]] and fault is None
    assert ring == [2, 3, -1, -1, 5, 7]
