"""8-bit KV cache: one scale for each block of tokens and KV head (oracle).

The pages have no counterpart; the definition is the one documented at
ssd_kv8_cache in include/ssd.h.  Scales and codes are decisions taken from
floating point, so they are taken in float32 (every operation rounded once),
like the int8 activation codes of quant.py; everything else is float64.
Slots are logical: pages and block tables are the GPU library's business.
"""
from __future__ import annotations

import math

import numpy as np

F32 = np.float32
QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3(y: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value (4 exponent bits, 3 mantissa bits, least exponent -6), ties to even, |y| <= 448."""
    y = np.asarray(y, dtype=np.float64)
    _, ex = np.frexp(np.maximum(np.abs(y), 2.0 ** -30))  # |y| = m 2^ex, m in [1/2, 1)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.rint(y / step) * step


def scale_of(x: np.ndarray, code: str) -> np.float32:
    """Scale of the block x: its largest finite magnitude over the largest code, 0 below 2^-126."""
    a = np.abs(np.asarray(x, dtype=F32)).ravel()
    a = a[np.isfinite(a)]
    with np.errstate(under="ignore"):
        s = F32(a.max() / F32(QMAX[code])) if a.size else F32(0)
    return s if s >= F32(2.0 ** -126) else F32(0)


def codes_of(x: np.ndarray, s: np.float32, code: str) -> np.ndarray:
    """Code values (float64) of x under scale s."""
    x = np.asarray(x, dtype=F32)
    if s == 0:
        return np.zeros(x.shape)
    with np.errstate(over="ignore", invalid="ignore"):
        y = (x * (F32(1) / s)).astype(F32)
    y = np.clip(np.where(np.isnan(x), F32(0), y), F32(-QMAX[code]), F32(QMAX[code])).astype(np.float64)
    return np.rint(y) if code == "int8" else e4m3(y)


class Cache8:
    """K or V of one layer: code values [slots, H, hd] and scales [blocks, H]."""

    def __init__(self, slots: int, heads: int, hd: int, code: str, block: int):
        self.code, self.block = code, block
        self.codes = np.zeros((-(-slots // block) * block, heads, hd))
        self.scale = np.zeros((-(-slots // block), heads), dtype=F32)

    def values(self, slots) -> np.ndarray:
        """float32 code * scale of the given slots, [n, H, hd]."""
        slots = np.asarray(slots)
        return (self.codes[slots].astype(F32) * self.scale[slots // self.block][:, :, None]).astype(F32)

    def append(self, x: np.ndarray, first: int) -> None:
        """Rows x [n, H, hd] into slots first ..; a block that keeps slots keeps a scale no smaller than its own."""
        T, n = self.block, x.shape[0]
        for b in range(first // T, (first + n - 1) // T + 1):
            lo, hi = max(b * T, first), min(b * T + T, first + n)
            for h in range(x.shape[1]):
                new = x[lo - first:hi - first, h]
                s = scale_of(new, self.code)
                if b * T < first:
                    kept = self.values(np.arange(b * T, first))[:, h]
                    s = max(s, self.scale[b, h])
                    self.codes[b * T:first, h] = codes_of(kept, s, self.code)
                self.codes[lo:hi, h] = codes_of(new, s, self.code)
                self.scale[b, h] = s


def scores(q, k, scale, cap):
    """[R, Hq, n] scores of q [R, Hq, hd] against k [n, H, hd] in float64."""
    group = q.shape[1] // k.shape[1]
    keys = np.repeat(k.astype(np.float64), group, 1).transpose(1, 2, 0)  # [Hq, hd, n]
    s = np.matmul(q.astype(np.float64).transpose(1, 0, 2), keys).transpose(1, 0, 2) * scale
    return cap * np.tanh(s / cap) if cap else s


def attention(q, k, v, vis, scale=None, cap=0.0):
    """(out [R, Hq, hd], lse [R, Hq]) in float64; vis bool [R, n].  A row that sees nothing: zeros and -inf."""
    scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    group = q.shape[1] // k.shape[1]
    s = np.where(vis[:, None, :], scores(q, k, scale, cap), -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    total = p.sum(-1, keepdims=True)
    v = np.where(vis.any(0)[:, None, None], v.astype(np.float64), 0.0)
    p = p / np.where(total > 0, total, 1.0)
    o = np.matmul(p.transpose(1, 0, 2), np.repeat(v, group, 1).transpose(1, 0, 2)).transpose(1, 0, 2)
    with np.errstate(divide="ignore"):
        return o, (np.where(np.isfinite(m), m, 0.0) + np.log(total))[..., 0]


def weights(q, k, vis, lse, rows, scale=None, cap=0.0):
    """[H, n] attention weight that the slots drew from the given rows."""
    scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    R, heads = q.shape[0], k.shape[1]
    s = np.where(vis[:, None, :], scores(q, k, scale, cap), -np.inf)
    with np.errstate(invalid="ignore"):
        p = np.where(np.isfinite(lse)[..., None], np.exp(s - lse[..., None]), 0.0)
    p = p.reshape(R, heads, -1, k.shape[0])
    return p[list(rows)].sum((0, 2))


def kept_slots(weight: np.ndarray, keep: int, recent: int) -> np.ndarray:
    """Slots [H, keep] that stay: the last `recent` and the heaviest others (lowest slot first among equal ones,
    NaN lightest), in slot order."""
    n = weight.shape[1]
    out = []
    for w in weight:
        order = sorted(range(n - recent), key=lambda i: (-math.inf if math.isnan(w[i]) else w[i]) * -1.0)
        nan = [i for i in order if math.isnan(w[i])]  # behind -inf, which compares equal above
        order = [i for i in order if not math.isnan(w[i])] + nan
        out.append(sorted(order[: keep - recent]) + list(range(n - recent, n)))
    return np.array(out, dtype=np.int64)


def evict(cache: Cache8, slots: np.ndarray, code: str, block: int) -> Cache8:
    """The kept slots [H, keep] of one tensor, requantised in a cache of their own."""
    heads, keep = slots.shape
    x = np.stack([cache.values(slots[h])[:, h] for h in range(heads)], 1)
    c = Cache8(keep, heads, x.shape[2], code, block)
    c.append(x, 0)
    return c
