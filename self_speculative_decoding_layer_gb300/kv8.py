"""KVCache8: one paged 8-bit KV cache and the operators over it (ssd_kv8_* of the C ABI).

Every call works on one layer, runs on the current torch stream of the cache's device and returns without waiting;
tensors it returns are new (unless given) and belong to that stream.  No gradients are recorded.  Arguments are checked and the library called by
lib/_kv8.so (csrc/py/kv8_ext.cpp); what it refuses is raised as SSDError.
"""
from __future__ import annotations

import importlib.util
import os
from typing import Optional, Sequence

import torch

from . import LIB_PATH, SSDError, load_library

PAGE = 64  # slots of a page
_IO = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _load():
    load_library()  # its message when nothing has been built
    path = os.path.join(os.path.dirname(LIB_PATH), "_kv8.so")
    spec = importlib.util.spec_from_file_location("_kv8", path)
    if spec is None or not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.init(SSDError)
    return mod


_ext = _load()


class KVCache8:
    """Codes k, v [n_layers, pool_pages, n_kv_heads, 64, head_dim] (torch.int8 or torch.float8_e4m3fn), fp32 scales
    k_scale, v_scale [n_layers, pool_pages, n_kv_heads, 64 / block_tokens] and the int32 block_table [n_pages]
    (logical page -> page of the pool) that every layer shares.  A slot's value is code * scale; how blocks are
    quantised, and what a block-table entry outside the pool means, stands at ssd_kv8_cache in include/ssd.h.  The
    tensors' contents may be written at any time (a new block table is copied into the old one's place)."""

    def __init__(self, n_layers: int, n_kv_heads: int, head_dim: int, max_tokens: int, dtype=torch.int8, block_tokens: int = 64,
                 device="cuda"):
        """An empty cache of ceil(max_tokens / 64) pages; dtype torch.int8 or torch.float8_e4m3fn."""
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
        if k.data_ptr() % 16 or v.data_ptr() % 16:
            raise SSDError(1, "k and v are 16-byte aligned")
        self.k, self.v, self.k_scale, self.v_scale, self.block_table = parts
        self.n_layers, self.pool_pages, self.n_kv_heads, _, self.head_dim = (int(n) for n in k.shape)
        self.n_pages, self.block_tokens, self.device = block_table.numel(), PAGE // blocks, k.device
        self._c = _ext.open(*(t.data_ptr() for t in parts), self.n_layers, self.pool_pages, self.n_kv_heads, self.head_dim,
                            self.n_pages, 3 if k.dtype == torch.int8 else 4, self.block_tokens, k.get_device())

    def append(self, layer: int, k, v, first: int) -> None:
        """Quantise rows k, v [rows, n_kv_heads, head_dim] into slots first .. first + rows - 1 (RoPE applied)."""
        _ext.append(self._c, layer, k, v, first)

    def read(self, layer: int, first: int, rows: int, dtype=torch.float32):
        """The values (k, v), [rows, n_kv_heads, head_dim] each, of slots first .. first + rows - 1."""
        io = _IO.get(dtype)
        if io is None:
            raise SSDError(1, f"values are float32, bfloat16 or float16, not {dtype}")
        return _ext.read(self._c, layer, first, rows, io)

    def attention(self, layer: int, q, prefix: int, base: Optional[int] = None, masks: Optional[Sequence[int]] = None,
                  scale: Optional[float] = None, softcap: float = 0.0, out=None, return_lse: bool = False):
        """Attention of q [rows <= 64, n_q_heads, head_dim]: row r sees slots [0, prefix) and base + e for every bit e
        < rows of masks[r].  base None: the new slots continue the prefix; masks None: causal (row r sees new slots
        0 .. r); scale None: 1 / sqrt(head_dim); softcap > 0: scores become softcap * tanh(score / softcap).  Returns
        out (like q), with return_lse also the rows' log-sum-exp [rows, n_q_heads] in fp32."""
        return _ext.attention(self._c, layer, q, prefix, base, masks, scale, softcap, out, return_lse)

    def weights(self, layer: int, q, lse, prefix: int, base: Optional[int] = None, masks: Optional[Sequence[int]] = None,
                scale: Optional[float] = None, softcap: float = 0.0, rows: Optional[Sequence[int]] = None, weight=None,
                out=None):
        """Add the attention weight that every slot drew from the given rows (None: all; each counts once) of an attention
        call, whose arguments are repeated here with the lse it returned, to weight [n_kv_heads, slots] (fp32; None: zeros).
        Written to out, else into weight, else to a new tensor, which is returned; only its first
        max(prefix, base + rows) columns are touched."""
        return _ext.weights(self._c, layer, q, prefix, base, masks, scale, softcap, lse, rows, weight, out)

    def evict(self, layer: int, weight, keep: int, recent: int, to: "KVCache8", to_layer: int):
        """Of the slots [0, n) that weight [n_kv_heads, n] covers every KV head keeps the last `recent` and the
        keep - recent heaviest others; they move, in slot order, to slots [0, keep) of layer to_layer of `to`, whose
        first pages must be none that this layer's slots use.  Returns the kept slots [n_kv_heads, keep] (int32) and
        their weights."""
        return _ext.evict(self._c, layer, weight, keep, recent, to._c, to_layer)
