"""One MLA decode layer over a paged latent cache, driven through the C ABI.

MLADecodeLayer owns the device state of one attention layer: the weights
W_UK, W_UV, the paged latent cache (and E4M3 scales), the RoPE tables, the
block table / sequence lengths, and reusable workspace and output buffers. A
decode step is

    append(new tokens) -> absorb_q -> decode_out_proj (decode_paged + out_proj)

on one stream, with no allocation in the step once the buffers exist; with
2 to 4 KV splits the split merge runs inside the projection kernel.

With the model-level weights attached (attach_front, attach_output), a step can
start from the hidden states of the new tokens and end in the model dimension:

    decode_front(h) -> append -> absorb_q -> decode_paged -> out_proj_fused (or out_proj, W_O)

A layer built with a window attends to the last `window` tokens and the first `sinks`
(decode_window in place of decode_paged). Its sequences live on the device: extend()
forks and grows them and gives each new token its position and cache row for the
step, evict() gives back the pages that left the window, free() those of finished
sequences, compact() moves the live pages to the front of the pool.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import capi
from .workloads import BF16, E4M3, F32, ROW, TORCH_DTYPE, Workload

CACHE_TORCH = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.uint8}


class MLADecodeLayer:
    def __init__(self, w: Workload, w_uk: torch.Tensor, w_uv: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, device="cuda", poison: bool = True, num_splits: Optional[int] = None,
                 window: int = 0, sinks: int = 0, spare_pages: int = 0, max_pos: int = 0):
        """window, sinks: sliding-window attention (0: every earlier token). spare_pages: free
        pages of the pool beyond the workload's, for extend(). max_pos: positions of the
        RoPE table beyond the workload's longest sequence. block_table may be wider than
        the workload's sequences need."""
        if window < 0 or sinks < 0:
            raise ValueError("window and sinks must not be negative")
        self.w = w
        self.device = torch.device(device)
        self.H = w.heads
        self.P = w.page_size
        self.cache_dtype = w.cache_dtype
        self.act = TORCH_DTYPE[w.act_dtype]
        self.w_uk = w_uk.to(self.device).contiguous()
        self.w_uv = w_uv.to(self.device).contiguous()
        self.block_table = block_table.to(self.device, torch.int32).contiguous()
        self.seq_lens = seq_lens.to(self.device, torch.int32).contiguous()
        self.num_pages = w.num_pages + spare_pages
        self.window, self.sinks = window, sinks
        ct = CACHE_TORCH[w.cache_dtype]
        self.cache = torch.empty(self.num_pages, self.P, ROW, dtype=ct, device=self.device)
        self.scales = (torch.empty(self.num_pages, self.P, 5, dtype=torch.float32, device=self.device)
                       if w.cache_dtype == E4M3 else None)
        if poison:
            self.poison()
        cos, sin = capi.mla_rope_table(max(w.max_pos, max_pos, 1), 64, w.rope_base)
        self.rope_cos = cos.to(self.device)
        self.rope_sin = sin.to(self.device)
        self.dev_error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.num_splits = w.num_splits if num_splits is None else num_splits
        B, Lq = w.batch, w.q_len
        # (of the table's width, by which the calls choose their splits)
        width = self.block_table.shape[1]
        if window > 0:
            args = (B, Lq, width, self.P, window, sinks, self.num_splits, self.H, self.cache_dtype)
            self.splits = capi.mla_decode_window_num_splits(*args)
            need = capi.mla_decode_window_workspace_size(*args)
        else:
            args = (B, Lq, width, self.P, self.num_splits, self.H, self.cache_dtype)
            self.splits = capi.mla_decode_num_splits(*args)
            need = capi.mla_decode_workspace_size(*args)
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=self.device)
        self.q_lat = torch.empty(B, Lq, self.H, 512, dtype=self.act, device=self.device)
        self.u = torch.empty(B, Lq, self.H, 512, dtype=self.act, device=self.device)
        self.lse = torch.empty(B, Lq, self.H, dtype=torch.float32, device=self.device)
        self.o = torch.empty(B, Lq, self.H, 128, dtype=self.act, device=self.device)
        self.softmax_scale = 1.0 / math.sqrt(128 + 64)

    def poison(self):
        """Fill the pool with NaN (values and scales) so unwritten rows are visible."""
        if self.cache_dtype == E4M3:
            self.cache.fill_(0x7F)
            self.scales.fill_(float("nan"))
        else:
            self.cache.fill_(float("nan"))

    def append(self, c_kv, k_r, positions, slots, stream=None):
        capi.mla_cache_append(c_kv, k_r, positions, slots, self.rope_cos, self.rope_sin, self.cache, self.scales,
                              self.P, self.cache_dtype, self.dev_error, stream)

    def append_chunked(self, c_kv, k_r, positions, slots, chunk: int = 1 << 18):
        """Fill a long context from host or device tensors, chunk by chunk."""
        n = c_kv.shape[0]
        for i in range(0, n, chunk):
            sl = slice(i, min(n, i + chunk))
            self.append(c_kv[sl].to(self.device, non_blocking=True).contiguous(),
                        k_r[sl].to(self.device, non_blocking=True).contiguous(),
                        positions[sl].to(self.device, non_blocking=True).contiguous(),
                        slots[sl].to(self.device, non_blocking=True).contiguous())

    def absorb(self, q_nope, stream=None):
        return capi.mla_absorb_q(q_nope, self.w_uk, self.q_lat, stream)

    def decode(self, q_lat, q_rope, stream=None):
        if self.window > 0:
            return capi.mla_decode_window(q_lat, q_rope, self.cache, self.scales, self.block_table, self.seq_lens,
                                          self.P, self.cache_dtype, self.window, self.sinks, self.softmax_scale,
                                          self.num_splits, self.workspace, self.u, self.lse, self.dev_error, stream)
        return capi.mla_decode_paged(q_lat, q_rope, self.cache, self.scales, self.block_table, self.seq_lens, self.P,
                                     self.cache_dtype, self.softmax_scale, self.num_splits, self.workspace, self.u,
                                     self.lse, self.dev_error, stream)

    def out_proj(self, u, stream=None):
        return capi.mla_out_proj(u, self.w_uv, self.o, stream)

    def decode_out_proj(self, q_lat, q_rope, stream=None):
        """decode then out_proj as one call (the KV splits merged inside the
        projection kernel where the library can); fills u, lse and o."""
        if self.window > 0:
            u, _ = self.decode(q_lat, q_rope, stream)
            return self.out_proj(u, stream)
        capi.mla_decode_out_proj(q_lat, q_rope, self.cache, self.scales, self.block_table, self.seq_lens, self.P,
                                 self.cache_dtype, self.w_uv, self.softmax_scale, self.num_splits, self.workspace,
                                 self.u, self.lse, self.o, self.dev_error, stream)
        return self.o

    def step(self, q_nope, q_rope, new_c_kv, new_k_r, new_positions, new_slots, stream=None):
        """One decode step: append the q_len new tokens, then attend. Returns o."""
        if new_c_kv is not None and new_c_kv.shape[0] > 0:
            self.append(new_c_kv, new_k_r, new_positions, new_slots, stream)
        q_lat = self.absorb(q_nope, stream)
        return self.decode_out_proj(q_lat, q_rope, stream)

    # ------------------------------------------------------------------ sequences and pages

    def prepare_pages(self, stream=None):
        """Makes the page calls' buffers on the call's stream and counts the block table's pages
        (ref_counts), once. The first page call does it; call it before capturing that one,
        since a graph would count anew at every replay. Entries outside the pool are nobody's pages."""
        if hasattr(self, "ref_counts"):
            return
        with capi.on_stream(stream):
            if self.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("prepare_pages() has to run before a page call is captured")
            i32 = dict(dtype=torch.int32, device=self.device)
            n, moves = self.block_table.shape[0], min(max(1, self.num_pages // 2), capi.MAX_LIST)
            self._lists = torch.empty(3, n, **i32)
            self._moves = torch.empty(2, moves, **i32)
            self._stats = torch.empty(2, **i32)
            self._all_seqs = torch.arange(n, **i32)
            need = max(capi.mla_cache_extend_workspace_size(n, self.num_pages),
                       capi.mla_cache_compact_workspace_size(self.num_pages),
                       capi.mla_cache_copy_workspace_size(max(n, moves), self.num_pages))
            self._page_ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            held = self.block_table[(self.block_table >= 0) & (self.block_table < self.num_pages)]
            self.ref_counts = torch.bincount(held.long(), minlength=self.num_pages).to(torch.int32)

    def extend(self, src_seqs, dst_seqs, n_new, positions, slots, stream=None):
        """Fork and grow: sequence dst_seqs[i] becomes sequence src_seqs[i] with room for
        n_new[i] more tokens (the same sequence: grows in place); int32 device lists of at
        most one entry per sequence. Fills positions (int32) and slots (int64) of the
        new tokens, request after request, as step() and append() take them, and copies
        the forks' partly filled pages in this layer's pool."""
        self.prepare_pages(stream)
        n = src_seqs.numel()
        lists = [self._lists[k][:n] for k in range(3)]
        capi.mla_cache_extend(src_seqs, dst_seqs, n_new, self.block_table, self.seq_lens, self.ref_counts, self.P,
                              *lists, positions, slots, workspace=self._page_ws, dev_error=self.dev_error,
                              stream=stream)
        capi.mla_cache_copy_pages(lists[0], lists[1], self.cache, self.scales, self.P, self.cache_dtype,
                                  n_rows=lists[2], workspace=self._page_ws, dev_error=self.dev_error, stream=stream)

    def free(self, seqs, stream=None):
        """The listed sequences end: their pages go back and their rows are empty."""
        self.prepare_pages(stream)
        capi.mla_cache_free(seqs, self.block_table, self.seq_lens, self.ref_counts, self.P, dev_error=self.dev_error,
                            stream=stream)

    def evict(self, stream=None):
        """Gives back every page that no later token's window (or the sinks) reaches. For after a
        step: with several queries per sequence, the step's own earlier ones reach further back."""
        if self.window < 1:
            raise ValueError("evict() needs a layer with a window")
        self.prepare_pages(stream)
        capi.mla_cache_free(self._all_seqs, self.block_table, self.seq_lens, self.ref_counts, self.P, self.window,
                            self.sinks, dev_error=self.dev_error, stream=stream)

    def compact(self, stream=None):
        """Moves the live pages to the front of the pool (at most 2^20 of them in a call). Returns
        the device tensor (live pages, pages at the front that hold them)."""
        self.prepare_pages(stream)
        src, dst = self._moves[0], self._moves[1]
        capi.mla_cache_compact(self.block_table, self.ref_counts, src, dst, self._stats, workspace=self._page_ws,
                               dev_error=self.dev_error, stream=stream)
        capi.mla_cache_copy_pages(src, dst, self.cache, self.scales, self.P, self.cache_dtype,
                                  workspace=self._page_ws, dev_error=self.dev_error, stream=stream)
        return self._stats

    # ------------------------------------------------------------------ model-level weights

    def attach_front(self, w_dq, w_dkv, w_kr, g_q, g_kv, w_uq, w_qr, eps: float):
        """Front-end weights (nn.Linear layouts [out, in]) and RMSNorm gains. The
        three down-projections and the two query up-projections are stacked once
        here, as mla_decode_front takes them; its workspace and outputs are
        allocated for the layer's B*Lq tokens."""
        dev = self.device
        self.w_dqkv = torch.cat([w_dq, w_dkv, w_kr], 0).to(dev).contiguous()
        self.w_uqr = torch.cat([w_uq, w_qr], 0).to(dev).contiguous()
        self.g_q = g_q.to(dev).contiguous()
        self.g_kv = g_kv.to(dev).contiguous()
        self.rms_eps = float(eps)
        n = self.w.batch * self.w.q_len
        d_model, d_cq = w_dq.shape[1], w_dq.shape[0]
        act = self.w.act_dtype
        self.front_ws = torch.empty(max(16, capi.mla_decode_front_workspace_size(n, d_model, d_cq, self.H, act)),
                                    dtype=torch.uint8, device=dev)
        mk = lambda *shape: torch.empty(*shape, dtype=self.act, device=dev)
        self.q_nope_buf, self.q_rope_buf = mk(n, self.H, 128), mk(n, self.H, 64)
        self.c_kv_buf, self.k_r_buf = mk(n, 512), mk(n, 64)

    def attach_output(self, w_o, fused: bool = True):
        """The output projection W_O [d_model, H, 128]. fused=True folds W_UV
        into it once (mla_fuse_out_weights) and a step ends with one product over
        all heads; fused=False keeps W_UV per head and applies W_O to the
        concatenated head outputs."""
        dev = self.device
        n = self.w.batch * self.w.q_len
        d_model = w_o.shape[0]
        act = self.w.act_dtype
        self.out_fused = fused
        w_o = w_o.to(dev).contiguous()
        if fused:
            self.w_out = capi.mla_fuse_out_weights(w_o, self.w_uv)
            need = capi.mla_out_proj_fused_workspace_size(n, d_model, self.H, act)
        else:
            self.w_out = w_o.view(d_model, self.H * 128)
            need = capi.mla_linear_workspace_size(n, d_model, self.H * 128, act)
        self.out_ws = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
        self.y = torch.empty(self.w.batch, self.w.q_len, d_model, dtype=self.act, device=dev)

    def front(self, h, positions, stream=None):
        """decode_front: h [B*Lq, d_model] -> (q_nope, q_rope, c_kv, k_r) in the layer's buffers."""
        return capi.mla_decode_front(h, self.w_dqkv, self.g_q, self.g_kv, self.w_uqr, positions, self.rope_cos,
                                     self.rope_sin, self.rms_eps, self.H, self.q_nope_buf, self.q_rope_buf,
                                     self.c_kv_buf, self.k_r_buf, self.front_ws, self.dev_error, stream)

    def output(self, u, stream=None):
        """u [B, Lq, H, 512] -> y [B, Lq, d_model] through the attached output projection."""
        if self.out_fused:
            return capi.mla_out_proj_fused(u, self.w_out, self.y, self.out_ws, stream)
        o = self.out_proj(u, stream)
        capi.mla_linear(o.view(-1, self.H * 128), self.w_out, self.y.view(-1, self.y.shape[-1]), self.out_ws,
                        stream)
        return self.y

    def step_from_hidden(self, h, positions, slots, stream=None):
        """One whole layer step: front end on the new tokens' hidden states, their
        rows appended at `slots`, absorbed paged decode, output projection.
        Returns y [B, Lq, d_model]."""
        B, Lq = self.w.batch, self.w.q_len
        q_nope, q_rope, c_kv, k_r = self.front(h, positions, stream)
        self.append(c_kv, k_r, positions, slots, stream)
        q_lat = self.absorb(q_nope.view(B, Lq, self.H, 128), stream)
        if self.out_fused:
            u, _ = self.decode(q_lat, q_rope.view(B, Lq, self.H, 64), stream)
            return self.output(u, stream)
        # W_UV per head (with the KV split merge inside its kernel), then W_O
        o = self.decode_out_proj(q_lat, q_rope.view(B, Lq, self.H, 64), stream)
        capi.mla_linear(o.view(-1, self.H * 128), self.w_out, self.y.view(-1, self.y.shape[-1]), self.out_ws, stream)
        return self.y

    def device_error(self) -> int:
        return capi.mla_read_device_error(self.dev_error)

    def capture(self, fn, warmup: int = 2):
        """Capture fn() (a sequence of this layer's calls on the current stream)
        into a CUDA graph. Every buffer fn touches must already exist; the
        library itself never allocates. Returns the torch.cuda.CUDAGraph."""
        side = torch.cuda.Stream(device=self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(side):
            for _ in range(warmup):
                fn()
        torch.cuda.current_stream(self.device).wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        return g


def build_layer(w: Workload, d: dict, device="cuda", fill_context: bool = True, **kw) -> MLADecodeLayer:
    """A layer for workload w with the inputs d of workloads.make_inputs, its cache
    filled with every context token except the step's new ones (when fill_context)."""
    layer = MLADecodeLayer(w, d["w_uk"], d["w_uv"], d["block_table"], d["seq_lens"], device=device, **kw)
    if fill_context:
        n = d["ctx_c_kv"].shape[0]
        keep = torch.ones(n, dtype=torch.bool)
        keep[d["new_index"]] = False
        idx = torch.nonzero(keep)[:, 0]
        layer.append_chunked(d["ctx_c_kv"][idx], d["ctx_k_r"][idx], d["ctx_positions"][idx], d["ctx_slots"][idx])
    return layer


def step_inputs(d: dict, device="cuda"):
    """Device tensors of one step's inputs (queries and the new tokens)."""
    ni = d["new_index"]
    return dict(q_nope=d["q_nope"].to(device).contiguous(), q_rope=d["q_rope"].to(device).contiguous(),
                new_c_kv=d["ctx_c_kv"][ni].to(device).contiguous(), new_k_r=d["ctx_k_r"][ni].to(device).contiguous(),
                new_positions=d["ctx_positions"][ni].to(device).contiguous(),
                new_slots=d["ctx_slots"][ni].to(device).contiguous())
