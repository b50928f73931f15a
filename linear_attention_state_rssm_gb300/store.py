"""ReplayStore: owns the device buffers of one ReplaySSM store (allocated with
PyTorch, which is used here only for device memory and streams) and forwards
calls to the C ABI with the same names. No arithmetic of the method runs here.
"""
from __future__ import annotations

import torch

from . import _lib

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class ReplayStore:
    """Checkpoint, ring and cursor of ``n_slots`` requests over ``n_layers`` layers.

    Buffers (row-major):
      state     [n_layers, n_slots, HV, dk, dv]    state_dtype
      ring_k    [n_layers, n_slots, HV, L, dk]     ring_k_dtype (one copy per value head)
      ring_d    [n_layers, n_slots, HV, L, dv]     ring_d_dtype
      ring_g    [n_layers, n_slots, HV, L] (+ [dk] for KDA)  fp32
      ring_v    [n_layers, n_slots, HV, L, dv]     in_dtype
      ring_beta [n_layers, n_slots, HV, L]         fp32
      cursor    [n_slots] int32, err_word [1] (uint32 bits in an int32 tensor)
    """

    def __init__(self, algo="gdn", n_layers=1, n_slots=1, HK=1, HV=1, dk=128, dv=128, L=16,
                 max_T=1, in_dtype="bf16", state_dtype="f32", ring_k_dtype=None,
                 ring_d_dtype="f32", commit_mode="lazy", scale=None, device="cuda"):
        self.cfg = _lib.make_config(algo, n_layers, n_slots, HK, HV, dk, dv, L, max_T, in_dtype,
                                    state_dtype, ring_k_dtype, ring_d_dtype, commit_mode, scale)
        self.algo, self.n_layers, self.n_slots = algo, n_layers, n_slots
        self.HK, self.HV, self.dk, self.dv, self.L, self.max_T = HK, HV, dk, dv, L, max_T
        self.in_dtype, self.state_dtype = in_dtype, state_dtype
        self.ring_k_dtype = ring_k_dtype or ("f16" if in_dtype == "bf16" else "f32")
        self.ring_d_dtype = ring_d_dtype
        self.commit_mode = commit_mode
        self.scale = self.cfg.scale
        self.device = torch.device(device)
        _lib.rssm_required_bytes(self.cfg)  # validates the configuration
        ls = (n_layers, n_slots)
        ng = () if algo == "gdn" else (dk,)
        dev = self.device
        self.state = torch.zeros(ls + (HV, dk, dv), dtype=_TORCH[state_dtype], device=dev)
        self.ring_k = torch.zeros(ls + (HV, L, dk), dtype=_TORCH[self.ring_k_dtype], device=dev)
        self.ring_d = torch.zeros(ls + (HV, L, dv), dtype=_TORCH[ring_d_dtype], device=dev)
        self.ring_g = torch.zeros(ls + (HV, L) + ng, dtype=torch.float32, device=dev)
        self.ring_v = torch.zeros(ls + (HV, L, dv), dtype=_TORCH[in_dtype], device=dev)
        self.ring_beta = torch.zeros(ls + (HV, L), dtype=torch.float32, device=dev)
        self.cursor = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.err_word = torch.zeros(1, dtype=torch.int32, device=dev)
        bufs = _lib.rssm_buffers(*(t.data_ptr() for t in (
            self.state, self.ring_k, self.ring_d, self.ring_g, self.ring_v, self.ring_beta,
            self.cursor, self.err_word)))
        with torch.cuda.device(dev):
            self.handle = _lib.rssm_alloc(self.cfg, bufs)

    # ---------------------------------------------------------------- calls
    def rssm_decode(self, layer, q, k, v, beta, g, slot, o, force=None, fold_out=None,
                    advance_cursor=False, stream=None):
        _lib.rssm_decode(self.handle, layer, q, k, v, beta, g, slot, force, slot.numel(), o,
                         fold_out, advance_cursor, stream)

    def rssm_verify(self, layer, q, k, v, beta, g, slot, T, o, force=None, fold_out=None,
                    stream=None):
        _lib.rssm_verify(self.handle, layer, q, k, v, beta, g, slot, force, slot.numel(), T, o,
                         fold_out, stream)

    def rssm_verify_ragged(self, layer, q, k, v, beta, g, cu_seqlens, slot, max_T, o,
                           force=None, fold_out=None, stream=None):
        """Windows of different lengths: row r's tokens are
        [cu_seqlens[r], cu_seqlens[r+1]) of the packed inputs (int32, B + 1)."""
        _lib.rssm_verify_ragged(self.handle, layer, q, k, v, beta, g, cu_seqlens, slot, force,
                                slot.numel(), max_T, o, fold_out, stream)

    def rssm_prefill(self, layer, q, k, v, beta, g, cu_seqlens, slot, o, reset_cursor=False,
                     stream=None):
        """Prompt of row r = tokens [cu_seqlens[r], cu_seqlens[r+1]); the
        checkpoint takes the state; the cursor clears on the last layer."""
        _lib.rssm_prefill(self.handle, layer, q, k, v, beta, g, cu_seqlens, slot, slot.numel(),
                          o, reset_cursor, stream)

    def rssm_native_decode(self, layer, q, k, v, beta, g, slot, o, stream=None):
        """The per-token state read/write path ReplaySSM replaces (comparison
        point): the checkpoint is the live state; ring and cursor untouched."""
        _lib.rssm_native_decode(self.handle, layer, q, k, v, beta, g, slot, slot.numel(), o,
                                stream)

    def rssm_commit(self, slot, accept_len, T, force=None, stream=None):
        _lib.rssm_commit(self.handle, slot, force, accept_len, slot.numel(), T, stream)

    def rssm_commit_ragged(self, slot, accept_len, cu_seqlens, max_T, force=None, stream=None):
        _lib.rssm_commit_ragged(self.handle, slot, force, accept_len, cu_seqlens, slot.numel(),
                                max_T, stream)

    def rssm_fold(self, slot, stream=None):
        _lib.rssm_fold(self.handle, slot, slot.numel(), stream)

    def rssm_reset_slots(self, slot, stream=None):
        _lib.rssm_reset_slots(self.handle, slot, slot.numel(), stream)

    def rssm_get_device_error(self, clear=True, stream=None) -> int:
        return _lib.rssm_get_device_error(self.handle, clear, stream)

    def rssm_set_plan(self, plan):
        """Kernel family for decode and verify: "auto", "rows" or "pipe"."""
        _lib.rssm_set_plan(self.handle, plan)

    def rssm_debug_withhold(self, barrier):
        """Test hook of the bounded waits (include/rssm.h): later launches of
        this store short-change `barrier` (-1: off)."""
        _lib.rssm_debug_withhold(self.handle, barrier)

    def close(self):
        if getattr(self, "handle", None):
            _lib.rssm_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------- helpers
    def new_output(self, B, T=1):
        return torch.empty((B * T, self.HV, self.dv), dtype=_TORCH[self.in_dtype],
                           device=self.device)

    def state_bytes_per_row_layer(self) -> int:
        return self.HV * self.dk * self.dv * (4 if self.state_dtype == "f32" else 2)


class ConvWindows:
    """Conv-state windows of ``n_slots`` requests for one convolution of width K
    over D channels, and the draft inputs of the last verify window.

    Buffers: window [n_slots, K-1, D], draft [n_slots, max_T, D] (dtype),
    err_word [1]. Taps w [D, K] and bias [D] are fp32 and passed per call.
    """

    ACT = {"none": 0, "silu": 1}

    def __init__(self, n_slots, D, K, max_T=1, dtype="bf16", device="cuda"):
        self.n_slots, self.D, self.K, self.max_T, self.dtype = n_slots, D, K, max_T, dtype
        dev = torch.device(device)
        self.window = torch.zeros((n_slots, K - 1, D), dtype=_TORCH[dtype], device=dev)
        self.draft = torch.zeros((n_slots, max_T, D), dtype=_TORCH[dtype], device=dev)
        self.err_word = torch.zeros(1, dtype=torch.int32, device=dev)

    def rssm_conv_window(self, x, w, bias, slot, T, y, act="silu", commit_now=False,
                         stream=None):
        if T > self.max_T:
            raise ValueError("window wider than the draft buffer")
        _lib.rssm_conv_window(x, w, bias, self.window, self.draft, slot, slot.numel(), T, self.D,
                              self.K, self.n_slots, self.dtype, self.ACT[act], commit_now, y,
                              self.err_word, stream)

    def rssm_conv_commit(self, slot, accept_len, T, stream=None):
        _lib.rssm_conv_commit(self.window, self.draft, slot, accept_len, slot.numel(), T, self.D,
                              self.K, self.n_slots, self.dtype, self.err_word, stream)


class RotaryTable:
    """Cosines and sines of rotary positions for KVCache.rssm_kv_append.

    table is fp32 [max_pos, 2, pairs]; sections gives how many of the pairs go
    by each position axis (one axis, or time, height, width), in blocks or
    interleaved (include/rssm.h, rssm_rope).
    """

    def __init__(self, table, sections=None, interleaved=False):
        if table.dtype != torch.float32 or table.dim() != 3 or table.shape[1] != 2 \
                or not table.is_cuda or not table.is_contiguous():
            raise ValueError("table: contiguous fp32 [max_pos, 2, pairs] on the device")
        sections = [table.shape[2]] if sections is None else list(sections)
        if not 1 <= len(sections) <= 3:
            raise ValueError("sections: one to three axes")
        self.table, self.axes = table, len(sections)
        sec = (_lib.ctypes.c_int32 * 3)(*(sections + [0] * (3 - len(sections))))
        self.struct = _lib.rssm_rope(table.data_ptr(), table.shape[0], table.shape[2], self.axes,
                                     sec, int(bool(interleaved)))

    @classmethod
    def from_base(cls, max_pos, pairs, base=10000.0, sections=None, interleaved=False,
                  device="cuda"):
        """Frequencies base^(-i / pairs), angles in 64 bits, rounded once."""
        i = torch.arange(pairs, dtype=torch.float64, device=device)
        angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] \
            * base ** (-i / pairs)
        return cls(torch.stack((angle.cos(), angle.sin()), 1).float().contiguous(), sections,
                   interleaved)


class HeadNorm:
    """Weights of the norms of queries and keys for KVCache.rssm_kv_append: fp32
    [D] each (None: those heads are left as they are). Kept, not copied."""

    def __init__(self, q_weight=None, k_weight=None, eps=1e-6):
        sizes = set()
        for w in (q_weight, k_weight):
            if w is None:
                continue
            if w.dtype != torch.float32 or w.dim() != 1 or not w.is_cuda or not w.is_contiguous():
                raise ValueError("weights: contiguous fp32 [D] on the device")
            sizes.add(w.shape[0])
        if len(sizes) > 1:
            raise ValueError("weights: one head size")
        self.D = sizes.pop() if sizes else None
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        self.struct = _lib.rssm_head_norm(*(None if w is None else w.data_ptr()
                                            for w in (q_weight, k_weight)), float(eps))


class Share:
    """A plan of shared prefixes and the attention's room for it (KVCache.new_share)."""

    def __init__(self, cache, B, T):
        self.cache, self.B, self.T = cache, B, T
        self.buffer = torch.zeros(_lib.rssm_kv_share_bytes(cache.cfg, B, T), dtype=torch.uint8,
                                  device=cache.device)


class KVCache:
    """Paged keys and values of the full-attention layers, ``n_slots`` requests.

    Buffers (row-major):
      k_pages, v_pages [n_layers, n_pages, HKV, page_size, D]  dtype, or e4m3 with
      page_scales      [n_layers, n_pages, HKV, page_size, 2] uint8 (page_dtype "e4m3":
                       quantised as they are written; else None)
      table            [n_slots, max_pages] int32 (-1: no page)
      held, length     [n_slots] int32: pages held, committed tokens
      refs             [n_pages] int32: tables that name the page
      work, err_word   scratch of the calls; error bits (_lib.DEVERR)

    q, k, v may be views whose tokens are strided (slices of one projection's
    output); outputs are contiguous. The contract of each call is that of the C
    entry point of the same name.
    """

    def __init__(self, n_layers=1, n_slots=1, HQ=1, HKV=1, D=128, n_pages=1, page_size=64,
                 max_pages=None, dtype="bf16", scale=None, device="cuda", page_dtype=None):
        if page_dtype not in (None, dtype, "e4m3"):
            raise ValueError('page_dtype: None (dtype) or "e4m3"')
        quant = page_dtype == "e4m3"
        max_pages = n_pages if max_pages is None else max_pages
        self.cfg = _lib.make_kv_config(n_layers, n_slots, HQ, HKV, D, n_pages, page_size,
                                       max_pages, dtype, scale)
        self.n_layers, self.n_slots, self.HQ, self.HKV, self.D = n_layers, n_slots, HQ, HKV, D
        self.n_pages, self.page_size, self.max_pages = n_pages, page_size, max_pages
        self.dtype, self.scale = dtype, self.cfg.scale
        self.page_dtype = "e4m3" if quant else dtype
        self._torch_dtype = _TORCH[dtype]
        self.device = torch.device(device)
        if quant:  # validates the configuration
            sizes, _ = _lib.rssm_kv_quant_required_bytes(self.cfg)
        else:
            sizes = _lib.rssm_kv_required_bytes(self.cfg)
        dev, t = self.device, torch.uint8 if quant else _TORCH[dtype]
        shape = (n_layers, n_pages, HKV, page_size, D)
        self.k_pages = torch.zeros(shape, dtype=t, device=dev)
        self.v_pages = torch.zeros(shape, dtype=t, device=dev)
        self.page_scales = None
        if quant:
            self.k_pages = self.k_pages.view(torch.float8_e4m3fn)
            self.v_pages = self.v_pages.view(torch.float8_e4m3fn)
            self.page_scales = torch.zeros(shape[:4] + (2,), dtype=torch.uint8, device=dev)
        self.table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=dev)
        self.held = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.length = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        self.work = torch.zeros(sizes.work, dtype=torch.uint8, device=dev)
        self.err_word = torch.zeros(1, dtype=torch.int32, device=dev)
        bufs = _lib.rssm_kv_buffers(*(x.data_ptr() for x in (
            self.k_pages, self.v_pages, self.table, self.held, self.length, self.refs,
            self.work, self.err_word)))
        with torch.cuda.device(dev):
            self.handle = _lib.rssm_kv_quant_alloc(self.cfg, bufs, self.page_scales) if quant \
                else _lib.rssm_kv_alloc(self.cfg, bufs)

    # ---------------------------------------------------------------- pages
    def rssm_kv_reserve(self, slot, T=1, cu_seqlens=None, stream=None):
        """Pages for the next T tokens of each row (or for its cu_seqlens)."""
        B = self._index(slot)
        self._index(cu_seqlens, B + 1)
        _lib.rssm_kv_reserve(self.handle, slot, cu_seqlens, B, T, stream)

    def rssm_kv_commit(self, slot, T=1, accept_len=None, cu_seqlens=None, stream=None):
        """length += accepted tokens (the whole window where accept_len is None)."""
        B = self._index(slot)
        self._index(accept_len, B)
        self._index(cu_seqlens, B + 1)
        _lib.rssm_kv_commit(self.handle, slot, accept_len, cu_seqlens, B, T, stream)

    def rssm_kv_fork(self, src, dst, deep=False, stream=None):
        """Slot dst[r] continues slot src[r]: full pages shared (deep: copied)."""
        B = self._index(src)
        self._index(dst, B)
        _lib.rssm_kv_fork(self.handle, src, dst, B, deep, stream)

    def rssm_kv_release(self, slot, stream=None):
        _lib.rssm_kv_release(self.handle, slot, self._index(slot), stream)

    def rssm_kv_compact(self, stream=None):
        """Pages in use move to the front of the pool."""
        _lib.rssm_kv_compact(self.handle, stream)

    # ------------------------------------------------------------ attention
    def rssm_kv_append(self, layer, q, k, v, slot, T=1, q_out=None, rope=None, positions=None,
                       cu_seqlens=None, k_out=None, stream=None, norm=None, v_out=None):
        """Norms (a HeadNorm) and rotation of q (into q_out) and k, k and v to the
        slots' pages (and, as the pages hold them, to k_out and v_out for
        rssm_attn_prefill)."""
        B = self._index(slot)
        self._index(cu_seqlens, B + 1)
        n, ks = self._tokens(k, self.HKV)
        _, vs = self._tokens(v, self.HKV, n)
        qs = self._tokens(q, self.HQ, n)[1] if q is not None else 0
        if q_out is not None:
            self._output(q_out, n)
        if k_out is not None:
            self._row("k_out", k_out, n)
        if v_out is not None:
            self._row("v_out", v_out, n)
        if norm is not None and norm.D not in (None, self.D):
            raise ValueError(f"norm: weights of {self.D} values")
        if positions is not None:
            if rope is None:
                raise ValueError("positions: with a rotary table")
            self._index(positions, rope.axes * n)
        _lib.rssm_kv_append_norm(self.handle, layer, q, k, v, qs, ks, vs,
                                 None if norm is None else norm.struct,
                                 None if rope is None else rope.struct, positions, cu_seqlens,
                                 slot, B, T, n, q_out, k_out, v_out, stream)

    def rssm_kv_gather(self, layer, slot, k_out, v_out, T=1, cu_seqlens=None, first=None,
                       stream=None):
        """Cached tokens [first[r], first[r] + T_r) of each row's slot in a row
        (k_out or v_out may be None)."""
        B = self._index(slot)
        self._index(cu_seqlens, B + 1)
        self._index(first, B)
        n = B * T if cu_seqlens is None else None
        for name, x in (("k_out", k_out), ("v_out", v_out)):
            if x is not None:
                n = x.shape[0] if n is None else n
                self._row(name, x, n)
        _lib.rssm_kv_gather(self.handle, layer, slot, first, cu_seqlens, B, T, n or 0, k_out,
                            v_out, stream)

    def rssm_attn_decode(self, layer, q, slot, T, o, lse=None, stream=None):
        """T new tokens per row over the slot's pages (their keys appended before)."""
        B = self._index(slot)
        _, qs = self._tokens(q, self.HQ, B * T)
        self._output(o, B * T, lse)
        _lib.rssm_attn_decode(self.handle, layer, q, qs, slot, B, T, o, lse, stream)

    def new_share(self, B, T=1):
        """Room for rssm_kv_share's plan of B rows of T tokens, and for what the
        attention holds between its launches."""
        return Share(self, B, T)

    def rssm_kv_share(self, slot, T, share, stream=None):
        """Which rows share a prefix's pages, into share (once for a step's layers)."""
        B = self._index(slot)
        self._shared(share, B, T)
        _lib.rssm_kv_share(self.handle, slot, B, T, share.buffer, stream)

    def rssm_attn_decode_shared(self, layer, q, slot, T, share, o, lse=None, stream=None):
        """As rssm_attn_decode, prefixes that rows share read once (rssm_kv_share's plan)."""
        B = self._index(slot)
        self._shared(share, B, T)
        _, qs = self._tokens(q, self.HQ, B * T)
        self._output(o, B * T, lse)
        _lib.rssm_attn_decode_shared(self.handle, layer, q, qs, slot, B, T, share.buffer, o, lse,
                                     stream)

    def rssm_attn_prefill(self, q, k, v, cu_seqlens, slot, o, cu_keys=None, lse=None,
                          stream=None):
        """Causal attention over packed prompts (cu_seqlens int32, B + 1)."""
        B = self._index(cu_seqlens) - 1
        self._index(slot, B)
        self._index(cu_keys, B + 1)
        n, qs = self._tokens(q, self.HQ)
        m, ks = self._tokens(k, self.HKV, n if cu_keys is None else None)
        _, vs = self._tokens(v, self.HKV, m)
        self._output(o, n, lse)
        _lib.rssm_attn_prefill(self.handle, q, k, v, qs, ks, vs, cu_seqlens, cu_keys, slot, B, n,
                               m, o, lse, stream)

    def rssm_kv_get_device_error(self, clear=True, stream=None) -> int:
        return _lib.rssm_kv_get_device_error(self.handle, clear, stream)

    def rssm_kv_debug_withhold(self, cta, unit=0):
        """Test hook of the bounded waits (include/rssm.h): later launches of this
        cache short-change a unit of CTA ``cta`` (-1: off)."""
        _lib.rssm_kv_debug_withhold(self.handle, cta, unit)

    def close(self):
        if getattr(self, "handle", None):
            _lib.rssm_kv_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------- helpers
    def _shared(self, share, B, T):
        if share.cache is not self or share.B != B or share.T != T:
            raise ValueError(f"share: of this cache, {B} rows and {T} tokens")

    @staticmethod
    def _index(x, n=None):
        """Entries of an index tensor; the kernels read it as n int32 in a run
        and cannot see where it ends."""
        if x is None:
            return 0
        m = x.numel()
        if x.dtype != torch.int32 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("index tensors: contiguous int32 on the device")
        if n is not None and m != n:
            raise ValueError(f"expected {n} entries, got {m}")
        return m

    def _tokens(self, x, heads, n=None):
        """Tokens and token stride of [n, heads, D] (heads and D contiguous)."""
        D = self.D
        try:
            m, h, d = x.shape
            s0, s1, s2 = x.stride()
        except ValueError:
            m = h = d = -1
        if h != heads or d != D or (n is not None and m != n):
            raise ValueError(f"expected {n or 'N'} x {heads} x {D}, got {tuple(x.shape)}")
        if x.dtype != self._torch_dtype or not x.is_cuda or s2 != 1 or (s1 != D and heads > 1):
            raise ValueError("the cache's dtype, on the device, with contiguous heads")
        return m, s0 if m > 1 else heads * D

    def _row(self, name, x, n):
        if x.dtype != self._torch_dtype or not x.is_contiguous() or not x.is_cuda \
                or x.numel() != n * self.HKV * self.D:
            raise ValueError(f"{name}: contiguous, the cache's dtype, [tokens, HKV, D]")

    def _output(self, o, n, lse=None):
        if o.dtype != self._torch_dtype or o.numel() != n * self.HQ * self.D \
                or not o.is_cuda or not o.is_contiguous():
            raise ValueError("outputs: contiguous, the cache's dtype, [tokens, HQ, D]")
        if lse is not None and (lse.dtype != torch.float32 or lse.numel() != n * self.HQ
                                or not lse.is_cuda or not lse.is_contiguous()):
            raise ValueError("lse: contiguous fp32 [tokens, HQ] on the device")
