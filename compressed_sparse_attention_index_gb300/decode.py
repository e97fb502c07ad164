"""Decode-step compositions over the C ABI (one CUDA stream, no host sync).

* Full layer: csa2_index_score over every visible entry -> csa2_topk (k=512)
  -> csa2_sparse_attn over the selected entries + the SWA window.
* Reindex layer: Full-layer scores -> csa2_topk in block mode (2,048 blocks of
  8) -> csa2_index_score over the 16,384 pool slots with the Reindex layer's
  own indexer query -> csa2_topk over the pool -> csa2_sparse_attn.
  (An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture,
  lightning-indexer note: decoder Reindex layers score only a 16,384-position
  pool picked earlier as blocks of 8; perchy.ai/models/deepseek, card "Full.
  Reindex. Reuse.": the pool feeds the top-512 that attention reads.)
* Paged cache (PagedCache): csa2_page_plan -> csa2_qk_norm_rope, which writes the
  new latents -> csa2_paged_attn, over every visible entry or a selection.
"""
from __future__ import annotations

import torch

from . import _lib as L

TOPK, POOL_BLOCKS, POOL_SLOTS, SWA = 512, 2048, 16384, 128


class DecodeBuffers:
    """Device buffers of one decode step for n_q queries over caches of n_max entries."""

    def __init__(self, n_q: int, n_max: int, pool: bool = False, out_dtype=L.CSA2_OUT_BF16, device="cuda",
                 q_group: int = 1):
        self.n_q, self.n_max, self.pool, self.out_dtype = n_q, n_max, pool, out_dtype
        self.scores = torch.empty((n_q, n_max), dtype=torch.float32, device=device)
        self.sel = torch.empty((n_q, TOPK), dtype=torch.int32, device=device)
        odt = torch.bfloat16 if out_dtype == L.CSA2_OUT_BF16 else torch.float32
        self.out = torch.empty((n_q, 64, 512), dtype=odt, device=device)
        ws_t = L.csa2_workspace_size(L.CSA2_OP_TOPK, n_q, n_max, TOPK)
        if pool:
            self.blocks = torch.empty((n_q, POOL_BLOCKS), dtype=torch.int32, device=device)
            self.pool_scores = torch.empty((n_q, POOL_SLOTS), dtype=torch.float32, device=device)
            ws_t = max(ws_t, L.csa2_workspace_size(L.CSA2_OP_TOPK, n_q, (n_max + 7) // 8, POOL_BLOCKS),
                       L.csa2_workspace_size(L.CSA2_OP_TOPK, n_q, POOL_SLOTS, TOPK))
        self.ws_topk_bytes = ws_t
        self.ws_attn_bytes = L.csa2_workspace_size(L.CSA2_OP_SPARSE_ATTN, n_q, TOPK + SWA)
        self.q_group = q_group
        self.ws_decode_bytes = L.csa2_workspace_size(L.CSA2_OP_DECODE_REINDEX, n_q, n_max, TOPK) if pool else \
            L.csa2_workspace_size(L.CSA2_OP_DECODE_MQ if q_group > 1 else L.CSA2_OP_DECODE, n_q, n_max, TOPK)
        self.ws = torch.empty(max(1, ws_t, self.ws_attn_bytes, self.ws_decode_bytes), dtype=torch.uint8,
                              device=device)


def full_decode(dw, buf: DecodeBuffers, params=None, stream=None):
    """Full-layer decode step of every query of a device workload (see gen.device)."""
    n_q = buf.n_q
    L.csa2_index_score(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib, dw.q_scale, dw.w, dw.q_seq,
                       dw.n_vis, n_q, None, buf.scores, buf.n_max, params, stream)
    L.csa2_topk(buf.scores, buf.n_max, n_q, dw.n_vis, dw.n_max, TOPK, 1, None, buf.sel, buf.ws, buf.ws_topk_bytes,
                stream)
    attend(dw, buf, params, stream)
    return buf.out


def fused_decode(dw, buf: DecodeBuffers, params=None, stream=None):
    """The same Full-layer step as full_decode, as the single call csa2_decode
    (scores stay in the workspace; buf.sel and buf.out are written)."""
    L.csa2_decode(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib, dw.q_scale, dw.w, dw.q_seq,
                  dw.n_vis, buf.n_q, dw.q, dw.kv, dw.swa, dw.swa.shape[1], dw.pos, dw.swa_first, dw.swa_cnt,
                  buf.sel, buf.out, buf.out_dtype, params, buf.ws, buf.ws_decode_bytes, stream)
    return buf.out


def mq_decode(dw, buf: DecodeBuffers, params=None, stream=None):
    """Full-layer decode of groups of buf.q_group queries per sequence (draft
    positions decoded together) as the single call csa2_decode_mq: each
    sequence's keys are scored once for its whole group."""
    L.csa2_decode_mq(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib, dw.q_scale, dw.w, dw.q_seq,
                     dw.n_vis, buf.n_q, buf.q_group, dw.q, dw.kv, dw.swa, dw.swa.shape[1], dw.pos, dw.swa_first,
                     dw.swa_cnt, buf.sel, buf.out, buf.out_dtype, params, buf.ws, buf.ws_decode_bytes, stream)
    return buf.out


def reindex_decode(dw, buf: DecodeBuffers, params=None, stream=None, build_pool: bool = True):
    """Reindex-layer decode step.  With build_pool=False the candidate pool in
    buf.blocks (chosen earlier by the Full layer) is reused as it is."""
    n_q = buf.n_q
    if build_pool:
        L.csa2_index_score(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib, dw.q_scale, dw.w,
                           dw.q_seq, dw.n_vis, n_q, None, buf.scores, buf.n_max, params, stream)
        L.csa2_topk(buf.scores, buf.n_max, n_q, dw.n_vis, dw.n_max, POOL_BLOCKS, 8, None, buf.blocks, buf.ws,
                    buf.ws_topk_bytes, stream)
    L.csa2_index_score(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib_re, dw.q_scale_re, dw.w_re,
                       dw.q_seq, dw.n_vis, n_q, buf.blocks, buf.pool_scores, POOL_SLOTS, params, stream)
    L.csa2_topk(buf.pool_scores, POOL_SLOTS, n_q, dw.n_vis, dw.n_max, TOPK, 1, buf.blocks, buf.sel, buf.ws,
                buf.ws_topk_bytes, stream)
    attend(dw, buf, params, stream)
    return buf.out


def fused_reindex_decode(dw, buf: DecodeBuffers, params=None, stream=None):
    """The Reindex-layer step over the pool in buf.blocks (chosen earlier by
    the Full layer) as the single call csa2_decode_reindex: the same selection
    and output as reindex_decode(build_pool=False); buf.sel and buf.out are
    written, the pool's scores stay in the workspace."""
    L.csa2_decode_reindex(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib_re, dw.q_scale_re, dw.w_re,
                          dw.q_seq, dw.n_vis, buf.n_q, buf.blocks, dw.q, dw.kv, dw.swa, dw.swa.shape[1], dw.pos,
                          dw.swa_first, dw.swa_cnt, buf.sel, buf.out, buf.out_dtype, params, buf.ws,
                          buf.ws_decode_bytes, stream)
    return buf.out


def attend(dw, buf: DecodeBuffers, params=None, stream=None):
    L.csa2_sparse_attn(dw.q, dw.kv, dw.n_max, dw.kv.shape[0], buf.sel, TOPK, dw.swa, dw.swa.shape[1], dw.q_seq,
                       dw.pos, dw.swa_first, dw.swa_cnt, buf.n_q, buf.out, buf.out_dtype, params, buf.ws,
                       buf.ws_attn_bytes, stream)
    return buf.out


class DecoderStep:
    """The decoder's layers in one step over the C ABI (layers as in
    gen.workloads.DECODER_LAYERS: (role, r) with role full / reindex / reuse):
    the Full layer scores every visible entry, keeps the top-512 and picks the
    pool of 2,048 blocks of 8 from the same scores; each Reindex layer r scores
    the pool with its own indexer query and keeps its top-512; every layer
    attends with its own query and window over the selection of the selecting
    layer it names (Reuse layers borrow it).  One stream, no host sync."""

    def __init__(self, n_q: int, n_max: int, layers, out_dtype=L.CSA2_OUT_F32, device="cuda"):
        self.layers, self.n_q, self.n_max = list(layers), n_q, n_max
        self.buf = DecodeBuffers(n_q, n_max, pool=True, out_dtype=out_dtype, device=device)
        n_sel = 1 + max(r for _, r in self.layers)
        self.sels = torch.empty((n_sel, n_q, TOPK), dtype=torch.int32, device=device)
        odt = torch.bfloat16 if out_dtype == L.CSA2_OUT_BF16 else torch.float32
        self.outs = torch.empty((len(self.layers), n_q, 64, 512), dtype=odt, device=device)
        self.out_dtype = out_dtype

    def run(self, dw, dl, params=None, stream=None):
        b, n_q = self.buf, self.n_q
        for l, (role, r) in enumerate(self.layers):
            if role == "full":
                L.csa2_index_score(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dw.q_nib, dw.q_scale, dw.w,
                                   dw.q_seq, dw.n_vis, n_q, None, b.scores, b.n_max, params, stream)
                L.csa2_topk(b.scores, b.n_max, n_q, dw.n_vis, dw.n_max, TOPK, 1, None, self.sels[r], b.ws,
                            b.ws_topk_bytes, stream)
                L.csa2_topk(b.scores, b.n_max, n_q, dw.n_vis, dw.n_max, POOL_BLOCKS, 8, None, b.blocks, b.ws,
                            b.ws_topk_bytes, stream)
            elif role == "reindex":
                # scoring the pool, its top-512 and the attention: one call
                L.csa2_decode_reindex(dw.key_nib, dw.key_scale, dw.n_max, dw.kv.shape[0], dl.q_nib_re[r],
                                      dl.q_scale_re[r], dl.w_re[r], dw.q_seq, dw.n_vis, n_q, b.blocks, dl.q[l], dw.kv,
                                      dl.swa[l], dl.swa.shape[2], dw.pos, dw.swa_first, dw.swa_cnt, self.sels[r],
                                      self.outs[l], self.out_dtype, params, b.ws, b.ws_decode_bytes, stream)
                continue
            L.csa2_sparse_attn(dl.q[l], dw.kv, dw.n_max, dw.kv.shape[0], self.sels[r], TOPK, dl.swa[l],
                               dl.swa.shape[2], dw.q_seq, dw.pos, dw.swa_first, dw.swa_cnt, n_q, self.outs[l],
                               self.out_dtype, params, b.ws, b.ws_attn_bytes, stream)
        return self.outs


class PagedCache:
    """A main cache in pages and a window ring for n_seq sequences, with the
    buffers of a step of up to max_tokens new tokens.  A step is plan, write,
    attend and advance, or step, which is all four.  It works on as many rows as its
    inputs have, or as plan is told (max_tokens otherwise): a step of a few tokens
    costs that of a few rows, whatever max_tokens is.  Everything stays on the
    device and on one stream (the current one, or `stream`, a torch.cuda.Stream),
    so a step can be captured into a CUDA graph and replayed: new_len and the
    inputs are read where they lie.  (write, attend and advance go with the last plan that
    the host made: a graph that plans should hold the whole step.)  A new cache is whole when its constructor returns
    (it waits for its fills); from then on the order of calls on different streams is the
    caller's, and so is the cache's life until work on other streams than the
    constructor's is over.

    Tokens are numbered in sequence order.  Pages that run out, sequences beyond
    max_len and tokens beyond max_tokens are reported by csa2_get_device_status; a
    token that got no page or no row writes nothing and is not part of its sequence
    afterwards, nor is a page taken that no token was written to.
    A token's window holds the last min(128, swa_cap) positions, and a step writes
    the window records of all its tokens before it attends: the ring has to hold the
    windows of all of them, 127 + the longest new_len records.  The default,
    127 + max_tokens, holds those of any step.  In a step of more rows than a shorter
    ring is sure to hold (swa_cap - 127), a sequence whose new tokens would overwrite
    their own windows gets none, which is reported as CSA2_ERR_BOUNDS; finding them takes
    four small launches more.
    max_tokens is at most 65,535.  Pages are taken and not returned: what ends a
    sequence, and gives its pages to others, is the caller's."""

    def __init__(self, n_seq: int, n_pages: int, page_size: int, max_len: int, max_tokens: int, swa_cap: int = None,
                 out_dtype=L.CSA2_OUT_BF16, device="cuda"):
        self.n_seq, self.n_pages, self.page_size, self.max_tokens = n_seq, n_pages, page_size, max_tokens
        swa_cap = SWA - 1 + max_tokens if swa_cap is None else swa_cap
        if not 1 <= max_tokens <= 65535 or swa_cap < 0 or n_seq * swa_cap >= 2**31:
            raise ValueError(f"max_tokens 1 .. 65535 and n_seq x swa_cap below 2^31 expected, not {max_tokens}, {n_seq} x {swa_cap}")
        self.swa_cap, self.out_dtype = swa_cap, out_dtype
        i32 = dict(dtype=torch.int32, device=device)
        self.pages = torch.zeros((n_pages, page_size, 288), dtype=torch.uint8, device=device)
        self.swa = torch.zeros((n_seq, swa_cap, 528), dtype=torch.uint8, device=device)
        self.table = torch.full((n_seq, -(-max_len // page_size)), -1, **i32)
        # the sequences' lengths and, behind them, the pages taken: what a step adds to
        self._state = torch.zeros(n_seq + 1, **i32)
        self.seq_len, self.free_head = self._state[:n_seq], self._state[n_seq:]
        self.free = torch.arange(n_pages, **i32)
        # the descriptors of a step of r rows, [7][r] (no token anywhere before the first plan), and ahead of them a row
        # that advance computes
        self._desc = torch.zeros(8 * max_tokens, **i32)
        self._desc[6 * max_tokens:] = -1
        # what advance adds to: r times free_head's place in the state, then the tokens' sequences
        self._place = torch.full((2 * max_tokens,), n_seq, **i32)
        self._added = torch.empty(2 * max_tokens, **i32)
        self._fit = (torch.empty(n_seq, **i32), torch.empty(n_seq, dtype=torch.bool, device=device),
                     torch.empty(n_seq, **i32), torch.full((n_seq,), -1, **i32), torch.full((n_seq,), swa_cap, **i32))
        self.first = torch.zeros(n_seq + 1, **i32)
        self.totals = torch.zeros(2, **i32)
        self.q = torch.empty((max_tokens, 64, 512), dtype=torch.bfloat16, device=device)
        self.latent = torch.empty((max_tokens, 512), dtype=torch.bfloat16, device=device)
        odt = torch.bfloat16 if out_dtype == L.CSA2_OUT_BF16 else torch.float32
        self.out = torch.empty((max_tokens, 64, 512), dtype=odt, device=device)
        self.lse = torch.empty((max_tokens, 64), dtype=torch.float32, device=device)
        self.ws = torch.empty(L.csa2_workspace_size(L.CSA2_OP_PAGED_ATTN, max_tokens, 0), dtype=torch.uint8,
                              device=device)
        # the fills above ran on the current stream, the steps may run on any
        if self.pages.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.pages.device).synchronize()
        self._views = {}
        self._use_rows(max_tokens)

    def _use_rows(self, rows):
        """The descriptors, buffers and counters of a step of `rows` rows."""
        v = self._views.get(rows)
        if v is None:
            at = self.max_tokens
            desc, place = self._desc[at:at + 7 * rows].view(7, rows), self._place[at - rows:at + rows]
            counted = self._desc.as_strided((2, rows), (at + 5 * rows, 1))       # the row ahead, and the slots
            added = self._added[:2 * rows]
            v = self._views[rows] = (desc, desc.unbind(), (place, place[rows:], counted, counted[0], added.view(2, rows), added),
                                     (self.out[:rows], self.lse[:rows]))
        self.rows = rows
        self.desc, self._d, self._count, self._rows = v

    def _here(self):
        """The kernels run on the current device, and read the cache there."""
        if self.pages.is_cuda and self.pages.get_device() != torch.cuda.current_device():
            raise ValueError(f"the cache is on {self.pages.device}, the current device is {torch.cuda.current_device()}")

    def _want(self, name, x, rows, cols, dtype):
        """x: rows of `cols` elements (any stride between rows), on the cache's device."""
        if x.dtype != dtype or x.device != self.seq_len.device or x.shape[0] != rows or x.numel() != rows * cols or \
                (rows > 0 and not x[0].is_contiguous()):
            raise ValueError(f"{name}: {rows} rows of {cols} contiguous {dtype} on {self.seq_len.device} expected, "
                             f"not {tuple(x.shape)} {x.dtype} on {x.device}")

    def plan(self, new_len, stream=None, rows=None):
        """Pages, slots and descriptors for new_len (device int32 [n_seq]) new tokens per sequence, in a step of `rows`
        rows (max_tokens at most, and by default)."""
        self._here()
        rows = self.max_tokens if rows is None else rows
        if not 0 <= rows <= self.max_tokens:
            raise ValueError(f"rows: 0 .. {self.max_tokens} expected, not {rows}")
        if not new_len.is_contiguous():
            raise ValueError("new_len: contiguous int32 expected")
        self._want("new_len", new_len, self.n_seq, 1, torch.int32)
        if 0 < self.swa_cap < min(SWA, self.swa_cap) - 1 + rows:
            new_len = self._that_fit(new_len, stream)
        self._use_rows(rows)
        L.csa2_page_plan(self.seq_len, new_len, self.n_seq, self.page_size, self.n_pages, self.free, self.n_pages,
                         self.free_head, self.table, self.table.shape[1], self.swa_cap, self.desc, rows, self.first,
                         self.totals, stream)

    def _that_fit(self, new_len, stream):
        """new_len, and -1, which the plan reports and gives no tokens, where the ring does not hold the records of the
        new tokens beside the first one's window, which reaches back to min(window - 1, seq_len) positions before it."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._that_fit(new_len, None)
        room, over, fit, none, cap = self._fit
        torch.clamp(self.seq_len, 0, min(SWA, self.swa_cap) - 1, out=room)
        torch.sub(cap, room, out=room)
        torch.gt(new_len, room, out=over)
        return torch.where(over, none, new_len, out=fit)

    def write(self, q, latent, q_gain=None, latent_gain=None, eps=1e-6, params=None, stream=None):
        """Norm and rotation of the planned tokens' queries (bf16 [rows][64][512]) and latents
        ([rows][512]), into self.q and self.latent, and the latents' records into the caches."""
        self._here()
        self._want("q", q, self.rows, 64 * 512, torch.bfloat16)
        self._want("latent", latent, self.rows, 512, torch.bfloat16)
        for gain in (q_gain, latent_gain):
            if gain is not None:
                self._want("gain", gain.reshape(-1, 1), 512, 1, torch.float32)
                if not gain.is_contiguous():
                    raise ValueError("gain: contiguous fp32 expected")
        # (a single row's stride may be anything)
        q_stride, stride = (q.stride(0), latent.stride(0)) if self.rows > 1 else (64 * 512, 512)
        d = self._d
        L.csa2_qk_norm_rope(q, q_stride, q_gain, self.q, latent, stride, latent_gain, self.latent, d[2], d[5], d[6],
                            self.rows, eps, self.pages, self.n_pages * self.page_size, self.swa, self.n_seq * self.swa_cap,
                            params, stream)

    def attend(self, sel=None, params=None, stream=None):
        """(output [rows][64][512], lse [rows][64]) of the planned tokens, over all that they see or over sel (device
        int32 [rows][k]); rows without a token get zeros and -inf, those behind the step's are left as they were."""
        self._here()
        if sel is not None:
            if not sel.is_contiguous():
                raise ValueError("sel: contiguous int32 expected")
            self._want("sel", sel, self.rows, sel.shape[1], torch.int32)
        d = self._d
        L.csa2_paged_attn(self.q, self.pages, self.n_pages, self.page_size, self.table, self.table.shape[1],
                          self.n_seq, sel, 0 if sel is None else sel.shape[1], self.swa, self.swa_cap, d[0], d[1],
                          d[2], d[3], d[4], self.rows, self.out, self.out_dtype, self.lse, params, self.ws,
                          self.ws.numel(), stream)
        return self._rows

    def advance(self, stream=None):
        """The tokens that were written become part of the sequences, the pages that they are on are taken."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.advance()
        # a token with a slot counts as one of its sequence; where the slot is a page's first, as a page.  (Slots end
        # within a sequence, pages of the free list within a step, so what is counted comes first in both.)
        place, seq, counted, first, added, add = self._count
        torch.clamp(self._d[0], 0, self.n_seq - 1, out=seq)            # (whatever a step of other rows has left there)
        if self.page_size > 1:
            torch.remainder(self._d[5], -self.page_size, out=first)    # 0 at a page's first place, else below
        else:
            first.copy_(self._d[5])
        torch.ge(counted, 0, out=added)
        self._state.index_add_(0, place, add)

    def step(self, new_len, q, latent, q_gain=None, latent_gain=None, eps=1e-6, sel=None, params=None, stream=None):
        """plan, write, attend and advance on as many rows as q and latent have."""
        self.plan(new_len, stream, q.shape[0])
        self.write(q, latent, q_gain, latent_gain, eps, params, stream)
        out = self.attend(sel, params, stream)
        self.advance(stream)
        return out

    def read(self, slots, out, stream=None):
        """Latents of the main cache's records `slots` (device int32, as in desc[5]) into out, bf16 or fp32 [n][512]."""
        self._here()
        if not slots.is_contiguous() or slots.dtype != torch.int32 or slots.device != self.seq_len.device or \
                not out.is_contiguous() or out.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("read: contiguous int32 slots on the cache's device and contiguous bf16 or fp32 out expected")
        self._want("out", out, slots.numel(), 512, out.dtype)
        L.csa2_cache_read(L.CSA2_KV_NVFP4, self.pages, self.n_pages * self.page_size, slots, slots.numel(), out,
                          L.CSA2_OUT_F32 if out.dtype == torch.float32 else L.CSA2_OUT_BF16, stream)
        return out
