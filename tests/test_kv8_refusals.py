"""What the 8-bit KV cache's entry points refuse (no GPU: nothing is launched), and its oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest

import self_speculative_decoding_layer_gb300 as ssd
from oracle import kv8

INVALID, CAPACITY = 1, 3
A = 0x10000  # an aligned address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return ssd.load_library()


def cache(**kw):
    c = ssd.KV8CacheC(A, A, A, A, A, 4, 4, 0, 8, 128, 3, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attn(**kw):
    a = ssd.KV8AttentionArgsC(A, A, A, 4096, 4096, 0, 0, 2, 32, 1, 100, 100, 0.1, 0.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def rows(**kw):
    r = ssd.KV8RowsC(A, A, 1024, 1024, 2, 0, 1)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def evict(**kw):
    e = ssd.KV8EvictArgsC(A, 256, A, A, 256, 64, 8)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


BAD_CACHE = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None), dict(k=A + 8),
             dict(v=A + 1), dict(k_scale=A + 2), dict(block_table=A + 1), dict(n_pages=0), dict(n_pages=-1),
             dict(n_pages=2 ** 24 + 1), dict(pool_pages=0), dict(layer=-1), dict(n_kv_heads=0), dict(n_kv_heads=4097),
             dict(head_dim=96), dict(head_dim=256), dict(dtype=0), dict(dtype=2), dict(dtype=5), dict(block_tokens=8),
             dict(block_tokens=128), dict(block_tokens=0)]


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_bad_descriptors(lib, bad):
    c = cache(**bad)
    r, a, e = rows(), attn(), evict()
    assert lib.ssd_kv8_append(ctypes.byref(c), ctypes.byref(r), None) == INVALID
    assert lib.ssd_kv8_read(ctypes.byref(c), ctypes.byref(r), None) == INVALID
    assert lib.ssd_kv8_attention_scratch_bytes(ctypes.byref(c), ctypes.byref(a)) == 0
    assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(a), A, 1 << 30, None) == INVALID
    assert lib.ssd_kv8_weights(ctypes.byref(c), ctypes.byref(a), 1, A, A, 256, None) == INVALID
    assert lib.ssd_kv8_evict(ctypes.byref(c), ctypes.byref(cache(block_table=2 * A)), ctypes.byref(e), None) == INVALID
    assert lib.ssd_kv8_evict(ctypes.byref(cache(block_table=2 * A)), ctypes.byref(c), ctypes.byref(e), None) == INVALID


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=A + 4), dict(ld_k=1023), dict(ld_v=1026), dict(dtype=3), dict(dtype=-1),
                                 dict(rows=0), dict(rows=-1), dict(first=-1), dict(first=256), dict(rows=257),
                                 dict(first=2 ** 31 - 1, rows=2 ** 31 - 1)], ids=str)
def test_bad_rows(lib, bad):
    c, r = cache(), rows(**bad)
    assert lib.ssd_kv8_append(ctypes.byref(c), ctypes.byref(r), None) == INVALID
    assert lib.ssd_kv8_read(ctypes.byref(c), ctypes.byref(r), None) == INVALID


BAD_ATTN = [dict(q=None), dict(q=A + 4), dict(ld_q=4095), dict(ld_q=4097), dict(dtype=3), dict(n_q_heads=12),
            dict(n_q_heads=0), dict(n_q_heads=8 * 4097, ld_q=8 * 4097 * 128), dict(ld_q=2 ** 62), dict(rows=0), dict(rows=65), dict(prefix=-1), dict(prefix=257), dict(base=-1), dict(base=256),
            dict(base=2 ** 31 - 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
            dict(softcap=-1.0), dict(softcap=1e-35), dict(softcap=1e31), dict(softcap=math.inf), dict(softcap=math.nan), dict(lse=A + 2), dict(ld_lse=-1),
            dict(step_lse=-4), dict(ld_lse=2 ** 50)]


@pytest.mark.parametrize("bad", BAD_ATTN, ids=str)
def test_bad_attention_arguments(lib, bad):
    c, a = cache(), attn(**bad)
    assert lib.ssd_kv8_attention_scratch_bytes(ctypes.byref(c), ctypes.byref(a)) == 0
    assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(a), A, 1 << 30, None) == INVALID
    assert lib.ssd_kv8_weights(ctypes.byref(c), ctypes.byref(a), 1, A, A, 256, None) == INVALID


def test_bad_outputs_and_scratch(lib):
    c = cache()
    for bad in (dict(out=None), dict(out=A + 8), dict(ld_out=100)):
        assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(attn(**bad)), A, 1 << 30, None) == INVALID, bad
    c = cache(n_pages=4096, pool_pages=4096, n_kv_heads=1)
    a = attn(prefix=200000, base=200000, n_q_heads=8)
    need = lib.ssd_kv8_attention_scratch_bytes(ctypes.byref(c), ctypes.byref(a))
    assert need > 256  # few heads, a long context: more key splits than a cluster holds
    assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(a), None, need, None) == INVALID
    assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(a), A + 16, need, None) == INVALID
    assert lib.ssd_kv8_attention(ctypes.byref(c), ctypes.byref(a), A, 1024, None) == CAPACITY
    c = cache()
    for w_in, w_out, ld in ((A, None, 256), (A, A + 2, 256), (A + 1, A, 256), (A, A, 100)):
        assert lib.ssd_kv8_weights(ctypes.byref(c), ctypes.byref(attn()), 1, w_in, w_out, ld, None) == INVALID
    assert lib.ssd_kv8_weights(ctypes.byref(c), ctypes.byref(attn(lse=None)), 1, A, A, 256, None) == INVALID
    for f in (lib.ssd_kv8_append, lib.ssd_kv8_read):
        assert f(None, ctypes.byref(rows()), None) == INVALID and f(ctypes.byref(c), None, None) == INVALID
    assert lib.ssd_kv8_attention(ctypes.byref(c), None, A, 1 << 30, None) == INVALID
    assert lib.ssd_kv8_evict(ctypes.byref(c), ctypes.byref(c), None, None) == INVALID


@pytest.mark.parametrize("bad", [dict(weight=None), dict(index=None), dict(weight=A + 2), dict(kept_weight=A + 1), dict(n=0),
                                 dict(n=257, ld_weight=300), dict(keep=0), dict(keep=257), dict(recent=-1), dict(recent=65),
                                 dict(ld_weight=255)], ids=str)
def test_bad_evictions(lib, bad):
    assert lib.ssd_kv8_evict(ctypes.byref(cache()), ctypes.byref(cache(layer=1)), ctypes.byref(evict(**bad)), None) == INVALID


def test_evictions_between_caches_that_differ(lib):
    e = evict()
    # onto itself
    assert lib.ssd_kv8_evict(ctypes.byref(cache(layer=1)), ctypes.byref(cache(layer=1)), ctypes.byref(e), None) == INVALID
    for other, rc in ((cache(n_kv_heads=4), INVALID), (cache(head_dim=64), INVALID), (cache(layer=1, n_pages=1), 0)):
        e.keep = 65 if rc == 0 else 64
        assert lib.ssd_kv8_evict(ctypes.byref(cache()), ctypes.byref(other), ctypes.byref(e), None) == (rc or CAPACITY)


def test_scratch_covers_every_split(lib):
    """The size that the library asks for grows with the shapes and never passes the partial results of 152 CTAs (one
    on each SM) of 256 queries."""
    c = cache(n_pages=4096, pool_pages=4096)
    for n_rows in (1, 2, 7, 64):
        for prefix in (0, 1, 100, 5000, 262000):
            got = lib.ssd_kv8_attention_scratch_bytes(
                ctypes.byref(c), ctypes.byref(attn(rows=n_rows, prefix=prefix, base=prefix)))
            assert 256 <= got <= 152 * 256 * (128 + 2) * 4 + 256, (n_rows, prefix, got)


def test_binding_structs_match_the_c_layout(lib):
    out = (ctypes.c_size_t * 9)()
    lib.ssd_abi_sizes(out, 9)
    assert list(out)[5:] == [ctypes.sizeof(c) for c in (ssd.KV8CacheC, ssd.KV8RowsC, ssd.KV8AttentionArgsC, ssd.KV8EvictArgsC)]


# ---------------------------------------------------------------- the oracle's definition


def test_e4m3_rounding_lists_every_number():
    """The positive e4m3 numbers from their definition; each is a fixed point, midpoints go to the even code."""
    nums = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    nums = [x for x in nums if x <= 448]
    assert len(nums) == 127
    assert np.array_equal(kv8.e4m3(np.array(nums)), np.array(nums))
    for i in range(len(nums) - 1):
        mid = (nums[i] + nums[i + 1]) / 2
        even = nums[i] if i % 2 == 0 else nums[i + 1]
        assert kv8.e4m3(np.array([mid]))[0] == even
        assert kv8.e4m3(np.array([-mid]))[0] == -even


def test_a_block_keeps_its_slots_and_grows_its_scale():
    rng = np.random.default_rng(0)
    for code in ("int8", "e4m3"):
        c = kv8.Cache8(64, 2, 64, code, 32)
        x = rng.standard_normal((10, 2, 64)).astype(np.float32)
        c.append(x[:5], 0)
        before = c.values(np.arange(5))
        c.append(0.25 * x[5:7], 5)  # smaller rows: nothing kept changes
        assert np.array_equal(c.values(np.arange(5)), before)
        s = c.scale[0].copy()
        c.append(8 * x[7:], 7)
        assert (c.scale[0] > s).all()
        step = c.scale[0][None, :, None] if code == "int8" else None
        got = c.values(np.arange(5))
        off = np.abs(got - before)
        lim = step / 2 * (1 + 1e-6) if code == "int8" else np.maximum(np.abs(before) * 2.0 ** -4, 2.0 ** -10 * c.scale[0][None, :, None])
        assert (off <= lim * (1 + 1e-6)).all()


def test_special_values():
    for code in ("int8", "e4m3"):
        top = kv8.QMAX[code]
        x = np.array([1.0, np.nan, np.inf, -np.inf, -2.0, 0.0], dtype=np.float32)
        s = kv8.scale_of(x, code)
        assert s == np.float32(np.float32(2.0) / np.float32(top))
        c = kv8.codes_of(x, s, code)
        assert c[1] == 0 and c[2] == top and c[3] == -top and c[4] == -top and c[5] == 0
        assert kv8.scale_of(np.full(4, 1e-40, dtype=np.float32), code) == 0
        assert not kv8.codes_of(np.full(4, 1e-40, dtype=np.float32), np.float32(0), code).any()


def test_oracle_attention_is_the_model_oracles():
    from oracle import model

    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 8, 64)), rng.standard_normal((20, 2, 64)), rng.standard_normal((20, 2, 64))
    vis = rng.random((3, 20)) < 0.6
    vis[:, 0] = True
    o, lse = kv8.attention(q, k, v, vis)
    assert np.allclose(o, model.attention(q, k, v, vis), atol=1e-12)
    w = kv8.weights(q, k, vis, lse, range(3))
    assert np.allclose(w.sum(1), 3 * 4)  # every row and head of the group spends weight 1
    assert np.allclose(w[:, ~vis.any(0)], 0)


def test_oracle_kept_slots():
    w = np.array([[3.0, 1.0, 3.0, np.nan, -np.inf, 2.0, 9.0]])
    assert kv8.kept_slots(w, 3, 1).tolist() == [[0, 2, 6]]
    assert kv8.kept_slots(w, 2, 1).tolist() == [[0, 6]]
    assert kv8.kept_slots(w, 6, 1).tolist() == [[0, 1, 2, 4, 5, 6]]
    assert kv8.kept_slots(w, 7, 0).tolist() == [[0, 1, 2, 3, 4, 5, 6]]
    assert kv8.kept_slots(w, 2, 2).tolist() == [[5, 6]]
