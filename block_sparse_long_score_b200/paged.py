"""A paged key-value cache for serving: prefill, then token by token.

``PagedCache`` keeps the pages, the block table and the free pages of one layer
on the device and strings the calls together: ``prefill`` runs the layer's
sparse prefill attention and stores its keys and values, ``step`` attends one
new token per request. It holds no arithmetic of its own.
"""
from __future__ import annotations

from typing import Optional

import torch

from .pipeline import prefill_attention
from .xattn import (_append_call, _call_on, _decode_call, make_paged,
                    xattn_paged_decode_workspace_bytes, xattn_paged_plan, xattn_prefill_varlen)

__all__ = ["PagedCache", "plan_buffers", "decode_buffers"]


def plan_buffers(table: torch.Tensor, max_tokens: int) -> dict:
    """The outputs of xattn_paged_plan for this block table and at most
    ``max_tokens`` new tokens a step, allocated once."""
    i32 = dict(device=table.device, dtype=torch.int32)
    nseq = table.shape[0]
    return {
        "lens": torch.empty(nseq, **i32),
        "pool": torch.empty(2, **i32),
        "starts": torch.empty(nseq + 1, **i32),
        "slots": torch.empty(max_tokens, **i32),
    }


def decode_buffers(Q: torch.Tensor, k_pages: torch.Tensor, table: torch.Tensor) -> dict:
    """The outputs and the workspace of xattn_paged_decode for queries like Q,
    allocated once so that repeated calls -- a serving loop, a CUDA-graph
    capture -- allocate nothing."""
    shape = make_paged(k_pages, Q.shape[1], Q.shape[0], table.shape[1])
    return {
        "out": torch.empty_like(Q),
        "lse": torch.empty(Q.shape[0], Q.shape[1], device=Q.device, dtype=torch.float32),
        "ws": torch.empty(max(xattn_paged_decode_workspace_bytes(shape), 1), device=Q.device,
                          dtype=torch.uint8),
    }


def _aligned(*tensors: torch.Tensor) -> None:
    """The library refuses a tensor that does not start on a 16-byte boundary; here it has
    to be known before the plan is made."""
    if any(t.data_ptr() % 16 for t in tensors):
        raise ValueError("a tensor does not start on a 16-byte boundary")


class PagedCache:
    """Keys and values of up to ``nseq`` requests in ``num_pages`` pages.

    A step that would need more pages than are free enters nothing: lengths and
    tables stay as they are, the attention sees the tokens there were, and
    xattn_get_device_status returns XATTN_ERR_PAGES. A call that is refused on the host
    (ValueError, XattnError) changes nothing either.

    Attributes (device tensors, all updated in place, so a captured CUDA graph
    stays valid): ``k_pages``, ``v_pages`` [num_pages, hkv, page_size, d];
    ``table`` int32 [nseq, max_pages]; ``lens`` int32 [nseq]; ``ring``, ``pool``
    (the free pages)."""

    def __init__(self, nseq: int, max_pages: int, num_pages: int, page_size: int, hkv: int,
                 d: int, dtype=torch.bfloat16, device="cuda"):
        i32 = dict(device=device, dtype=torch.int32)
        pages = dict(device=device, dtype=dtype)
        self.page_size = page_size
        self.k_pages = torch.empty(num_pages, hkv, page_size, d, **pages)
        self.v_pages = torch.empty(num_pages, hkv, page_size, d, **pages)
        self.table = torch.full((nseq, max_pages), -1, **i32)
        self.lens = torch.zeros(nseq, **i32)
        self.ring = torch.arange(num_pages, **i32)
        self.pool = torch.tensor([0, num_pages], **i32)
        self._ws_bytes = {}     # of the decode, by query heads (the rest of its shape is fixed)

    def plan(self, fresh: torch.Tensor, buffers: dict):
        """Pages and slots for ``fresh[i]`` new tokens of request i (-1 ends
        it). ``buffers`` from plan_buffers; returns (starts, slots)."""
        xattn_paged_plan(self.lens, fresh, self.pool, self.ring, self.table, self.page_size,
                         out=(self.lens, self.pool, buffers["starts"], buffers["slots"]))
        return buffers["starts"], buffers["slots"]

    def prefill(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, B: int, S: int, tau,
                causal: bool, fresh: torch.Tensor, buffers: dict) -> torch.Tensor:
        """Sparse prefill attention of new prompts, whose keys and values enter
        the cache. Q: [batch, hq, L, d], K, V: [batch, hkv, L, d]; ``fresh`` is
        L for each of the ``batch`` rows that take a prompt, in order, and 0
        elsewhere. Inside a CUDA-graph capture ``tau`` has to be a CUDA tensor.
        Returns O."""
        append = self._append_prompts(K, V, buffers)
        O = prefill_attention(Q, K, V, B, S, tau, causal)
        self.plan(fresh, buffers)
        _call_on(*append)
        return O

    def _append_prompts(self, K, V, buffers) -> tuple:
        append = _append_call(K, V, buffers["slots"], self.k_pages, self.v_pages,
                              buffers["starts"])
        _aligned(K, V)
        return append

    def prefill_varlen(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seqlens, hq: int,
                       B: int, S: int, tau, causal: bool, fresh: torch.Tensor,
                       buffers: dict) -> torch.Tensor:
        """As ``prefill``, for prompts of different lengths packed as
        xattn_prefill_varlen takes them; ``seqlens`` are the lengths (host) of
        the rows with ``fresh`` > 0, in order."""
        append = self._append_prompts(K, V, buffers)
        O = xattn_prefill_varlen(Q, K, V, seqlens, hq, self.k_pages.shape[1], B, S, causal, tau)
        self.plan(fresh, buffers)
        _call_on(*append)
        return O

    def step(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, fresh: torch.Tensor,
             buffers: dict, lse: Optional[bool] = None):
        """One new token for each request with ``fresh[i]`` = 1: its key and
        value enter the cache, and its query attends to all of them. Q: [nseq,
        hq, d], a row per request; K, V: [tokens, hkv, d], a row per new token
        in request order (tokens = the length of the slots buffer; rows behind
        the last new token are left out). ``buffers`` holds plan_buffers' and
        decode_buffers' entries. Rows of requests without a new token attend
        to what they have. Returns O, or (O, lse)."""
        append = _append_call(K, V, buffers["slots"], self.k_pages, self.v_pages, None)
        decode, out, row_lse, ws = _decode_call(Q, self.k_pages, self.v_pages, self.table,
                                                self.lens, buffers["out"],
                                                buffers["lse"] if lse else None, buffers["ws"])
        _aligned(Q, K, V, out, ws)
        tokens, hkv, d = K.shape
        if tokens > 1 and not (hkv * d <= K.stride(0) <= 1 << 31
                               and K.stride(0) * K.element_size() % 16 == 0):
            raise ValueError("the tokens of K and V must not overlap and lie a multiple of 16 "
                             "bytes apart")
        hq = Q.shape[1]
        need = self._ws_bytes.get(hq)
        if need is None:
            need = self._ws_bytes[hq] = xattn_paged_decode_workspace_bytes(
                make_paged(self.k_pages, hq, Q.shape[0], self.table.shape[1]))
        if need == 0 or ws.nbytes < need:
            raise ValueError("the heads do not fit the cache, or the workspace is too small")
        self.plan(fresh, buffers)
        _call_on(*append)
        _call_on(*decode)
        return out if row_lse is None else (out, row_lse)
