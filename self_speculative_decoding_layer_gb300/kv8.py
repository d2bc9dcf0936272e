"""KVCache8: one paged 8-bit KV cache and the operators over it (ssd_kv8_* of the C ABI).

Argument checks and marshalling only.  Every call works on one layer, runs on the current torch stream of the
cache's device and returns without waiting; tensors it returns are new and belong to that stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import SSDError, KV8AttentionArgsC, KV8CacheC, KV8EvictArgsC, KV8RowsC, load_library

PAGE = 64  # slots of a page
MAX_ROWS = 64

_CAUSAL = (ctypes.c_uint64 * MAX_ROWS)(*[(2 << r) - 1 for r in range(MAX_ROWS)])
_CAUSAL_AT = ctypes.addressof(_CAUSAL)
_MASK_AT = KV8AttentionArgsC.mask.offset
_ref = ctypes.byref
_FLOAT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
# A call's time on the host is what bounds the small operators, so the current device and stream are asked for without
# the objects that torch.cuda wraps them in (1 us less a call).
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_empty = torch.empty


class KVCache8:
    """Codes k, v [n_layers, pool_pages, n_kv_heads, 64, head_dim] (torch.int8 or torch.float8_e4m3fn), fp32 scales
    k_scale, v_scale [n_layers, pool_pages, n_kv_heads, 64 / block_tokens] and the int32 block_table [n_pages]
    (logical page -> page of the pool) that every layer shares.  A slot's value is code * scale; how blocks are
    quantised, and what a block-table entry outside the pool means, stands at ssd_kv8_cache in include/ssd.h."""

    def __init__(self, n_layers: int, n_kv_heads: int, head_dim: int, max_tokens: int, dtype=None, block_tokens: int = 64,
                 device="cuda"):
        """An empty cache of ceil(max_tokens / 64) pages; dtype torch.int8 (the default) or torch.float8_e4m3fn."""
        dtype = torch.int8 if dtype is None else dtype
        if dtype not in (torch.int8, torch.float8_e4m3fn):
            raise SSDError(1, f"codes are torch.int8 or torch.float8_e4m3fn, not {dtype}")
        if min(n_layers, n_kv_heads, max_tokens) < 1 or head_dim not in (64, 128) or block_tokens not in (16, 32, 64):
            raise SSDError(1, "n_layers, n_kv_heads, max_tokens >= 1, head_dim 64 or 128, block_tokens 16, 32 or 64")
        pages = -(-max_tokens // PAGE)
        k, v = (torch.zeros((n_layers, pages, n_kv_heads, PAGE, head_dim), dtype=torch.int8, device=device).view(dtype)
                for _ in range(2))
        ks, vs = (torch.zeros((n_layers, pages, n_kv_heads, PAGE // block_tokens), dtype=torch.float32, device=device)
                  for _ in range(2))
        self._bind(k, v, ks, vs, torch.arange(pages, dtype=torch.int32, device=device))

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, block_table) -> "KVCache8":
        """A cache over existing tensors (contiguous, on one device), which it keeps alive."""
        c = cls.__new__(cls)
        c._bind(k, v, k_scale, v_scale, block_table)
        return c

    def _bind(self, k, v, k_scale, v_scale, block_table):
        if k.dtype not in (torch.int8, torch.float8_e4m3fn) or k.dim() != 5 or k.shape[3] != PAGE:
            raise SSDError(1, "k is [n_layers, pool_pages, n_kv_heads, 64, head_dim] of int8 or float8_e4m3fn")
        blocks = k_scale.shape[-1] if k_scale.dim() == 4 else 0
        if v.shape != k.shape or v.dtype != k.dtype:
            raise SSDError(1, "v has the shape and type of k")
        if blocks not in (1, 2, 4) or k_scale.shape != k.shape[:3] + (blocks,) or v_scale.shape != k_scale.shape:
            raise SSDError(1, "scales are [n_layers, pool_pages, n_kv_heads, 64 / block_tokens]")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or block_table.dtype != torch.int32:
            raise SSDError(1, "scales are float32 and the block table is int32")
        if block_table.dim() != 1 or block_table.numel() < 1 or k.shape[4] not in (64, 128) or 0 in k.shape:
            raise SSDError(1, "the block table names at least one page, head_dim is 64 or 128")
        parts = (k, v, k_scale, v_scale, block_table)
        if any(not t.is_contiguous() or t.device != k.device for t in parts) or k.device.type != "cuda":
            raise SSDError(1, "the cache's tensors are contiguous and on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.block_table = parts
        self.n_layers, self.pool_pages, self.n_kv_heads, _, self.head_dim = (int(n) for n in k.shape)
        self.n_pages, self.block_tokens = block_table.numel(), PAGE // blocks
        self.device = k.device
        self._lib = load_library()
        self._index = k.get_device()
        code = 3 if k.dtype == torch.int8 else 4
        self._layers = [KV8CacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                  block_table.data_ptr(), self.n_pages, self.pool_pages, i, self.n_kv_heads,
                                  self.head_dim, code, self.block_tokens) for i in range(self.n_layers)]
        self._scale = 1.0 / math.sqrt(self.head_dim)

    # -- plumbing
    def _call(self, fn, *args):
        """One C call on the current stream of the cache's device."""
        index = self._index
        if _device() != index:
            with torch.cuda.device(index):
                rc = fn(*args, _stream(index))
        else:
            rc = fn(*args, _stream(index))
        if rc:
            raise SSDError(rc, f"{fn.__name__} refused its arguments" if rc != 5 else fn.__name__)

    def _layer(self, layer: int) -> KV8CacheC:
        if not 0 <= layer < self.n_layers:
            raise SSDError(1, f"layer {layer} of {self.n_layers}")
        return self._layers[layer]

    def _ld(self, t, heads: int, what: str) -> int:
        """Elements between the rows of a [rows, heads, head_dim] float tensor whose rows are contiguous."""
        shape, hd = t.shape, self.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != hd or t.dtype not in _FLOAT or t.get_device() != self._index:
            raise SSDError(1, f"{what} is [rows, {heads}, {hd}] of float32, bfloat16 or float16 on {self.device}")
        ld, s1, s2 = t.stride()
        if s2 != 1 or (s1 != hd and heads > 1):
            raise SSDError(1, f"the rows of {what} are contiguous")
        return ld if shape[0] > 1 else heads * hd

    # -- API
    def append(self, layer: int, k, v, first: int) -> None:
        """Quantise rows k, v [rows, n_kv_heads, head_dim] into slots first .. first + rows - 1 (RoPE applied)."""
        ld_k, ld_v = self._ld(k, self.n_kv_heads, "k"), self._ld(v, self.n_kv_heads, "v")
        rows = k.shape[0]
        if v.dtype != k.dtype or v.shape[0] != rows:
            raise SSDError(1, "k and v have the same rows and type")
        a = KV8RowsC(k.data_ptr(), v.data_ptr(), ld_k, ld_v, _FLOAT[k.dtype], first, rows)
        self._call(self._lib.ssd_kv8_append, _ref(self._layer(layer)), _ref(a))

    def read(self, layer: int, first: int, rows: int, dtype=torch.float32):
        """The values (k, v), [rows, n_kv_heads, head_dim] each, of slots first .. first + rows - 1."""
        if dtype not in _FLOAT or rows < 1:
            raise SSDError(1, "rows >= 1 of float32, bfloat16 or float16")
        shape = (rows, self.n_kv_heads, self.head_dim)
        k, v = _empty(shape, dtype=dtype, device=self.device), _empty(shape, dtype=dtype, device=self.device)
        ld = self.n_kv_heads * self.head_dim
        a = KV8RowsC(k.data_ptr(), v.data_ptr(), ld, ld, _FLOAT[dtype], first, rows)
        self._call(self._lib.ssd_kv8_read, _ref(self._layer(layer)), _ref(a))
        return k, v

    def _attention_args(self, q, prefix, base, masks, scale, softcap) -> KV8AttentionArgsC:
        shape = q.shape
        if len(shape) != 3 or shape[1] < 1 or shape[1] % self.n_kv_heads:
            raise SSDError(1, f"q is [rows, heads, {self.head_dim}], its heads a multiple of {self.n_kv_heads}")
        rows, heads, _ = shape
        ld = self._ld(q, heads, "q")
        if not 1 <= rows <= MAX_ROWS:
            raise SSDError(1, f"{rows} rows: 1 to {MAX_ROWS}")
        a = KV8AttentionArgsC(q.data_ptr(), None, None, ld, ld, _FLOAT[q.dtype], heads, rows, prefix,
                              prefix if base is None else base, self._scale if scale is None else scale, softcap)
        if masks is None:
            ctypes.memmove(ctypes.addressof(a) + _MASK_AT, _CAUSAL_AT, 8 * rows)
        else:
            if len(masks) != rows:
                raise SSDError(1, f"{len(masks)} masks for {rows} rows")
            a.mask[:rows] = [int(m) for m in masks]
        return a

    def attention(self, layer: int, q, prefix: int, base: Optional[int] = None, masks: Optional[Sequence[int]] = None,
                  scale: Optional[float] = None, softcap: float = 0.0, out=None, return_lse: bool = False):
        """Attention of q [rows <= 64, n_q_heads, head_dim]: row r sees slots [0, prefix) and base + e for every bit e
        < rows of masks[r].  base None: the new slots continue the prefix; masks None: causal (row r sees new slots
        0 .. r); scale None: 1 / sqrt(head_dim); softcap > 0: scores become softcap * tanh(score / softcap).  Returns
        out (like q), with return_lse also the rows' log-sum-exp [rows, n_q_heads] in fp32."""
        a = self._attention_args(q, prefix, base, masks, scale, softcap)
        if out is None:
            out = _empty(q.shape, dtype=q.dtype, device=self.device)
            a.ld_out = a.n_q_heads * self.head_dim
        else:
            if out.shape != q.shape or out.dtype != q.dtype:
                raise SSDError(1, "out has the shape and type of q")
            a.ld_out = self._ld(out, a.n_q_heads, "out")
        a.out = out.data_ptr()
        lse = None
        if return_lse:
            lse = _empty((a.rows, a.n_q_heads), dtype=torch.float32, device=self.device)
            a.lse = lse.data_ptr()
        c, ra = _ref(self._layer(layer)), _ref(a)
        need = self._lib.ssd_kv8_attention_scratch_bytes(c, ra)
        if need > 256:
            # per call, from the current stream's pool: calls on other streams and captured graphs share none of it
            scratch = _empty(need, dtype=torch.uint8, device=self.device)
            self._call(self._lib.ssd_kv8_attention, c, ra, scratch.data_ptr(), need)
        else:
            self._call(self._lib.ssd_kv8_attention, c, ra, None, 0)
        return (out, lse) if return_lse else out

    def _weight_ld(self, t, slots: int) -> int:
        """Elements between the heads of a float32 [n_kv_heads, >= slots] tensor whose rows are contiguous."""
        shape = t.shape
        if len(shape) != 2 or shape[0] != self.n_kv_heads or shape[1] < slots or t.dtype != torch.float32 or \
                t.get_device() != self._index:
            raise SSDError(1, f"weights are float32 [{self.n_kv_heads}, {slots} or more] on {self.device}")
        ld, s1 = t.stride()
        if shape[0] == 1:
            ld = shape[1]
        if (s1 != 1 and shape[1] > 1) or ld < shape[1]:
            raise SSDError(1, "the rows of weights are contiguous and apart")
        return ld

    def weights(self, layer: int, q, lse, prefix: int, base: Optional[int] = None, masks: Optional[Sequence[int]] = None,
                scale: Optional[float] = None, softcap: float = 0.0, rows: Optional[Sequence[int]] = None, weight=None,
                out=None):
        """Add the attention weight that every slot drew from the given rows (None: all) of an attention call, whose
        arguments are repeated here with the lse it returned, to weight [n_kv_heads, slots] (fp32; None: zeros).
        Written to out, else into weight, else to a new tensor, which is returned; only its first
        max(prefix, base + rows) columns are touched."""
        a = self._attention_args(q, prefix, base, masks, scale, softcap)
        if lse.shape != (a.rows, a.n_q_heads) or lse.dtype != torch.float32 or not lse.is_contiguous() or \
                lse.get_device() != self._index:
            raise SSDError(1, "lse is the contiguous float32 [rows, heads] of the attention call")
        a.lse = lse.data_ptr()
        slots = max(prefix, a.base + a.rows)
        if out is None:
            out = weight if weight is not None else _empty((self.n_kv_heads, slots), dtype=torch.float32, device=self.device)
        ld = self._weight_ld(out, slots)
        if weight is not None and weight is not out and self._weight_ld(weight, slots) != ld:
            raise SSDError(1, "weight and out are laid out alike")
        take = (1 << a.rows) - 1
        if rows is not None:
            take = 0
            for r in rows:
                if not 0 <= r < a.rows:
                    raise SSDError(1, f"row {r} of {a.rows}")
                take |= 1 << r
        self._call(self._lib.ssd_kv8_weights, _ref(self._layer(layer)), _ref(a), take,
                    None if weight is None else weight.data_ptr(), out.data_ptr(), ld)
        return out

    def evict(self, layer: int, weight, keep: int, recent: int, to: "KVCache8", to_layer: int):
        """Of the slots [0, n) that weight [n_kv_heads, n] covers every KV head keeps the last `recent` and the
        keep - recent heaviest others; they move, in slot order, to slots [0, keep) of layer to_layer of `to`, whose
        first pages must be none that this layer's slots use.  Returns the kept slots [n_kv_heads, keep] (int32) and
        their weights."""
        ld = self._weight_ld(weight, 1)
        n = weight.shape[1]
        if to.device != self.device or not 1 <= keep <= n or not 0 <= recent <= keep:
            raise SSDError(1, f"0 <= recent <= keep <= {n}, keep >= 1, caches on one device")
        index = _empty((self.n_kv_heads, keep), dtype=torch.int32, device=self.device)
        kept = _empty((self.n_kv_heads, keep), dtype=torch.float32, device=self.device)
        a = KV8EvictArgsC(weight.data_ptr(), ld, index.data_ptr(), kept.data_ptr(), n, keep, recent)
        self._call(self._lib.ssd_kv8_evict, _ref(self._layer(layer)), _ref(to._layer(to_layer)), _ref(a))
        return index, kept
