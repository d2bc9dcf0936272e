"""The 8-bit KV cache on the GPU against the float64 oracle (oracle/kv8.py)."""
import math

import numpy as np
import pytest

import kv8_cases as kc
from oracle import kv8

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

CODE = {"int8": "int8", "e4m3": "float8_e4m3fn"}
IO = {"fp32": "float32", "bf16": "bfloat16", "fp16": "float16"}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def garbage(shape, seed):
    """Bytes that a pool may hold before it is written, e4m3's NaN among them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    b[..., ::5] = 0x7F
    return b.view(torch.int8)


class Pair:
    """A GPU cache over pages of random order in a pool full of garbage (codes and scales), and its oracle."""

    def __init__(self, slots, heads, hd, code, block, layers=2, layer=1, seed=0, spare=2):
        import self_speculative_decoding_layer_gb300 as ssd

        pages = max(1, -(-slots // 64))
        pool = pages + spare
        dt = getattr(torch, CODE[code])
        k, v = (garbage((layers, pool, heads, 64, hd), seed + i).view(dt) for i in range(2))
        ks, vs = (torch.full((layers, pool, heads, 64 // block), float("nan"), device="cuda") for _ in range(2))
        perm = np.random.default_rng(seed).permutation(pool)[:pages]
        table = torch.tensor(perm, dtype=torch.int32, device="cuda")
        self.gpu = ssd.KVCache8.wrap(k, v, ks, vs, table)
        self.k, self.v = (kv8.Cache8(pages * 64, heads, hd, code, block) for _ in range(2))
        self.layer, self.heads, self.hd, self.code, self.block, self.perm = layer, heads, hd, code, block, perm

    def append(self, k, v, first):
        self.gpu.append(self.layer, k.cuda(), v.cuda(), first)
        self.k.append(k.float().numpy(), first)
        self.v.append(v.float().numpy(), first)

    def fill(self, rng, n, io="fp32", first=0):
        if n:
            self.append(kc.make_rows(rng, n, self.heads, self.hd, io), kc.make_rows(rng, n, self.heads, self.hd, io), first)

    def same(self, n):
        """The first n slots: codes' values and scales, bit for bit."""
        k, v = self.gpu.read(self.layer, 0, n)
        slots = np.arange(n)
        assert np.array_equal(k.cpu().numpy(), self.k.values(slots))
        assert np.array_equal(v.cpu().numpy(), self.v.values(slots))
        blocks = np.arange(-(-n // self.block)) * self.block
        for s, o in ((self.gpu.k_scale, self.k), (self.gpu.v_scale, self.v)):
            got = s[self.layer].cpu().numpy()[self.perm[blocks // 64], :, blocks % 64 // self.block]
            assert np.array_equal(got, o.scale[: len(blocks)])


# ---------------------------------------------------------------- append, read

APPENDS = [  # heads, hd, code, block, io, [(first, rows)...]
    (8, 128, "int8", 64, "fp32", [(0, 1), (1, 1), (2, 7), (9, 60), (69, 200)]),
    (2, 64, "e4m3", 16, "bf16", [(0, 16), (16, 1), (17, 15), (32, 33), (65, 1)]),
    (40, 128, "e4m3", 32, "fp16", [(0, 31), (31, 2), (33, 1), (34, 64)]),
    (1, 64, "int8", 16, "fp32", [(0, 300), (300, 1)]),
    (3, 128, "int8", 32, "bf16", [(0, 64), (63, 1), (40, 30)]),  # a rollback: slots written again
    (5, 64, "e4m3", 64, "fp32", [(0, 129)]),
]


@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_is_the_definition_bit_for_bit(case):
    heads, hd, code, block, io, steps = case
    rng = np.random.default_rng(3)
    p = Pair(max(f + n for f, n in steps), heads, hd, code, block)
    for first, n in steps:
        p.fill(rng, n, io, first)
        p.same(first + n)


def test_append_leaves_everything_else_as_it_was():
    """Other layers, other pages, and the codes of slots behind the new rows."""
    p = Pair(192, 4, 128, "int8", 32)
    before = [t.clone() for t in (p.gpu.k.view(torch.int8), p.gpu.v.view(torch.int8))]
    scales = [t.clone() for t in (p.gpu.k_scale, p.gpu.v_scale)]
    p.fill(np.random.default_rng(0), 70)
    for t, b in zip((p.gpu.k.view(torch.int8), p.gpu.v.view(torch.int8)), before):
        t = t.clone()
        for s in range(70):
            b[1, p.perm[s // 64], :, s % 64] = t[1, p.perm[s // 64], :, s % 64]
        assert torch.equal(t, b)
    for t, b in zip((p.gpu.k_scale, p.gpu.v_scale), scales):
        for s in range(0, 70, 32):
            b[1, p.perm[s // 64], :, s % 64 // 32] = t[1, p.perm[s // 64], :, s % 64 // 32]
        assert torch.equal(t.nan_to_num(-1.0), b.nan_to_num(-1.0))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_of_special_values(code):
    """Zeros, subnormals, NaN and infinities: NaN is stored as 0, an infinity as the largest code, neither sets a scale."""
    x = torch.zeros((20, 2, 64))
    x[1, 0, :4] = torch.tensor([1.0, float("nan"), float("inf"), -float("inf")])
    x[2, 0, 5] = -2.0
    x[17, 0] = 1e-41
    x[18, 1] = float("inf")
    x[3, 1, 7] = 3.0e38
    p = Pair(20, 2, 64, code, 16)
    p.append(x, -x, 0)
    k = p.k.values(np.arange(20))
    assert k[1, 0, 1] == 0 and k[1, 0, 2] == -k[1, 0, 3] > 0 and not k[17].any() and not k[18, 1].any()
    p.same(20)


def test_append_reads_rows_with_a_stride():
    """K and V as slices of one projection's output, and a single row of odd stride."""
    rng = np.random.default_rng(5)
    qkv = kc.make_rows(rng, 9, 32, 128, "bf16").cuda()  # 16 query heads, 8 K, 8 V
    a, b = Pair(9, 8, 128, "int8", 16), Pair(9, 8, 128, "int8", 16)
    a.gpu.append(1, qkv[:, 16:24], qkv[:, 24:], 0)
    b.append(qkv[:, 16:24].contiguous().cpu(), qkv[:, 24:].contiguous().cpu(), 0)
    b.same(9)
    for x, y in zip(a.gpu.read(1, 0, 9, torch.bfloat16), b.gpu.read(1, 0, 9, torch.bfloat16)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("io", ["fp32", "bf16", "fp16"])
def test_read_rounds_once(io):
    p = Pair(130, 3, 64, "int8", 32)
    p.fill(np.random.default_rng(1), 130)
    dt = getattr(torch, IO[io])
    k, v = p.gpu.read(1, 61, 69, dt)
    assert torch.equal(k.cpu(), torch.tensor(p.k.values(np.arange(61, 130))).to(dt))
    assert torch.equal(v.cpu(), torch.tensor(p.v.values(np.arange(61, 130))).to(dt))


# ---------------------------------------------------------------- attention, weights

ATTN = [  # rows, prefix, base - prefix, masks, hq, hkv, hd, code, block, io, cap
    (1, 0, 0, "causal", 4, 4, 64, "int8", 64, "fp32", 0.0),
    (1, 1, 0, "causal", 32, 8, 128, "int8", 64, "fp32", 0.0),
    (1, 700, 0, "causal", 32, 8, 128, "e4m3", 32, "bf16", 0.0),
    (1, 63, 0, "none", 8, 1, 128, "int8", 16, "fp16", 0.0),
    (1, 0, 0, "none", 8, 2, 128, "int8", 16, "fp32", 0.0),  # nothing at all to see
    (7, 301, 0, "causal", 32, 8, 128, "int8", 64, "fp32", 0.0),
    (17, 259, 0, "tree", 40, 40, 128, "e4m3", 16, "fp16", 30.0),
    (17, 300, 5, "tree", 16, 4, 64, "int8", 32, "bf16", 5.0),
    (6, 300, 0, "causal", 8, 2, 64, "int8", 16, "fp32", 0.0),  # 17 to 24 queries for a KV head
    (5, 900, 0, "tree", 8, 2, 128, "e4m3", 16, "fp32", 0.0),
    (3, 2500, 0, "causal", 16, 4, 64, "int8", 32, "fp16", 0.0),  # 9 to 16
    (8, 700, 0, "tree", 32, 8, 64, "e4m3", 64, "fp32", 0.0),  # 25 to 32
    (5, 200, 213, "own", 16, 2, 128, "e4m3", 64, "fp32", 0.0),  # the DP rows' slots, past the committed ones
    (64, 128, 0, "causal", 8, 8, 64, "int8", 32, "fp32", 0.0),
    (64, 1000, 0, "holes", 64, 8, 128, "int8", 64, "bf16", 0.0),
    (33, 1, 0, "tree", 8, 2, 128, "int8", 16, "fp16", 0.0),
    (17, 5000, 0, "tree", 40, 5, 128, "int8", 64, "fp32", 0.0),
    (31, 4000, -20, "tree", 27, 3, 128, "int8", 32, "fp32", 0.0),
    # many queries over many slots: the tcgen05 kernel, with one or two query blocks, whole and ragged
    (64, 1600, 0, "causal", 64, 64, 64, "e4m3", 32, "bf16", 0.0),
    (64, 3100, 70, "holes", 48, 8, 64, "e4m3", 16, "fp32", 30.0),
    (33, 6300, 0, "tree", 32, 8, 128, "int8", 16, "fp16", 0.0),
    (16, 6272, 0, "causal", 64, 8, 128, "int8", 64, "bf16", 50.0),
    (9, 25000, 0, "tree", 16, 4, 128, "int8", 32, "fp32", 0.0),
    (64, 4300, -20, "tree", 24, 3, 128, "e4m3", 64, "fp16", 0.0),
    (40, 100013, 0, "own", 1, 1, 64, "int8", 32, "bf16", 0.0),
    (64, 0, 3300, "holes", 40, 40, 64, "int8", 64, "fp32", 0.0),
    (17, 9000, 0, "tree", 40, 5, 128, "e4m3", 32, "fp32", 0.0),
    (17, 9000, 3, "causal", 40, 5, 128, "int8", 16, "fp32", 20.0),
    (40, 6300, 0, "tree", 40, 40, 64, "e4m3", 32, "bf16", 0.0),  # and with half a block
    (3, 0, 0, "holes", 6, 3, 64, "e4m3", 16, "fp32", 0.0),  # a row that sees nothing
    (9, 77, 40, "none", 10, 10, 128, "int8", 16, "fp16", 0.0),
    (6, 100, -10, "tree", 21, 3, 64, "int8", 32, "fp32", 50.0),  # new slots that the prefix holds already count once
    (33, 4093, 0, "tree", 8, 1, 128, "e4m3", 64, "fp32", 0.0),
    (1, 9000, 0, "causal", 64, 8, 64, "int8", 16, "fp16", 0.0),
    (2, 5000, 0, "causal", 1, 1, 128, "e4m3", 32, "fp32", 0.0),
    (1, 6000, 0, "causal", 24, 1, 128, "int8", 32, "bf16", 20.0),
]


def attention_case(case, seed=0, spare_slots=40):
    rows, prefix, gap, kind, hq, hkv, hd, code, block, io, cap = case
    rng = np.random.default_rng(seed)
    base = prefix + gap
    n = max(prefix, base + rows)
    p = Pair(n + spare_slots, hkv, hd, code, block, seed=seed)
    p.fill(rng, prefix)
    if gap <= 0:  # (otherwise the slots between stay garbage)
        p.fill(rng, n - prefix, first=prefix)
    else:
        p.fill(rng, rows, first=base)
    q = kc.make_rows(rng, rows, hq, hd, io) * (3.0 / math.sqrt(hd) * 2)
    q = q.to(getattr(torch, IO[io]))
    m = kc.masks(kind, rows, rng)
    vis = kc.visible(m, rows, prefix, base, n)
    return p, q, m, vis, n, base


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention_and_weights_match_the_oracle(case):
    rows, prefix, gap, kind, hq, hkv, hd, code, block, io, cap = case
    p, q, m, vis, n, base = attention_case(case)
    slots = np.arange(n)
    k, v = p.k.values(slots), p.v.values(slots)
    scale = 1.0 / math.sqrt(hd)
    qf = q.float().numpy()
    want, want_lse = kv8.attention(qf, k, v, vis, scale, cap)
    out, lse = p.gpu.attention(1, q.cuda(), prefix, base, masks=m, softcap=cap, return_lse=True)
    got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    blind = ~vis.any(1)
    assert not got[blind].any() and np.isneginf(got_lse[blind]).all()
    off = np.abs(got - want)
    lim = kc.out_error(qf, k, v, vis, want, scale, cap, io)
    assert (off <= lim).all(), (np.max(off / lim), np.max(off))
    ll = kc.lse_error(qf, k, vis, want_lse, scale, cap)
    assert (np.abs(got_lse[~blind] - want_lse[~blind]) <= ll[~blind]).all()
    # a second call gives the same bits: the sums have one order
    again, lse2 = p.gpu.attention(1, q.cuda(), prefix, base, masks=m, softcap=cap, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)

    take = list(range(0, rows, 2))
    w0 = np.random.default_rng(9).random((hkv, n + 3)).astype(np.float32)
    w = torch.tensor(w0).cuda()
    r = p.gpu.weights(1, q.cuda(), lse, prefix, base, masks=m, softcap=cap, rows=take, weight=w)
    assert r is w
    add = kv8.weights(qf, k, vis, got_lse, take, scale, cap)
    e = np.where(vis[:, None, :], kc.score_error(qf, k, scale, cap), 0.0)
    e = e + 2 * kc.U24 * 2 * np.abs(np.where(np.isfinite(got_lse), got_lse, 0.0))[..., None] + 2.0 ** -21
    per = np.where(vis[:, None, :] & np.isfinite(got_lse)[..., None],
                   np.exp(np.minimum(kv8.scores(qf, k, scale, cap) - np.where(np.isfinite(got_lse), got_lse, 0)[..., None], 1.0)), 0.0)
    lim = (per * 2 * e).reshape(rows, hkv, -1, n)[take].sum((0, 2)) + (len(take) * (hq // hkv) + 4) * kc.U24 * (w0[:, :n] + add)
    gw = w.cpu().numpy().astype(np.float64)
    assert (np.abs(gw[:, :n] - (w0[:, :n] + add)) <= lim + 1e-30).all()
    assert np.array_equal(gw[:, n:], w0[:, n:])  # columns behind the last slot are left alone
    fresh = p.gpu.weights(1, q.cuda(), lse, prefix, base, masks=m, softcap=cap, rows=take)
    assert fresh.shape == (hkv, max(n, 1))
    none = p.gpu.weights(1, q.cuda(), lse, prefix, base, masks=m, softcap=cap, rows=[])
    assert not none.any()


def test_causal_is_the_default_and_bits_past_the_rows_do_not_count():
    case = (9, 130, 0, "causal", 16, 2, 128, "int8", 32, "fp32", 0.0)
    p, q, m, vis, n, base = attention_case(case)
    a = p.gpu.attention(1, q.cuda(), 130)
    b = p.gpu.attention(1, q.cuda(), 130, 130, masks=[x | (1 << 9) | (1 << 63) for x in m])
    assert torch.equal(a, b)


def test_strided_queries_and_outputs():
    case = (5, 333, 0, "causal", 12, 4, 128, "e4m3", 16, "bf16", 0.0)
    p, q, m, vis, n, base = attention_case(case)
    wide = torch.full((5, 30, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:15] = q.cuda()
    room = torch.full((5, 20, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    p.gpu.attention(1, wide[:, 3:15], 333, out=room[:, 8:])
    assert torch.equal(room[:, 8:], p.gpu.attention(1, q.cuda(), 333))
    assert (room[:, :8] == 7.0).all()


def test_weights_take_any_layout_of_lse():
    case = (5, 333, 0, "causal", 12, 4, 128, "e4m3", 16, "bf16", 0.0)
    p, q, m, vis, n, base = attention_case(case)
    _, lse = p.gpu.attention(1, q.cuda(), 333, return_lse=True)
    want = p.gpu.weights(1, q.cuda(), lse, 333)
    assert torch.equal(p.gpu.weights(1, q.cuda(), lse.t().contiguous().t(), 333), want)
    wide = torch.zeros((5, 30), device="cuda")
    wide[:, 4:28:2] = lse
    assert torch.equal(p.gpu.weights(1, q.cuda(), wide[:, 4:28:2], 333), want)


def test_a_nan_query_stays_in_its_row():
    case = (4, 90, 0, "causal", 8, 2, 64, "int8", 16, "fp32", 0.0)
    p, q, m, vis, n, base = attention_case(case)
    clean = p.gpu.attention(1, q.cuda(), 90)
    q[2, 5, 7] = float("nan")
    out = p.gpu.attention(1, q.cuda(), 90)
    assert out[2, 5].isnan().all()
    out[2, 5] = clean[2, 5]
    assert torch.equal(out, clean)


def test_a_nan_query_stays_in_its_row_on_tcgen05():
    case = (16, 6272, 0, "causal", 64, 8, 64, "e4m3", 32, "bf16", 0.0)
    p, q, m, vis, n, base = attention_case(case)
    clean = p.gpu.attention(1, q.cuda(), 6272)
    q[3, 9, 7] = float("nan")
    q[12, 60, 0] = float("inf")
    out = p.gpu.attention(1, q.cuda(), 6272)
    assert out[3, 9].isnan().all() and not out[12, 60].isfinite().all()
    out[3, 9], out[12, 60] = clean[3, 9], clean[12, 60]
    assert torch.equal(out, clean)


def test_large_and_small_queries_keep_their_precision():
    """q rows of very different size: each is scaled by its own power of two."""
    rng = np.random.default_rng(2)
    p = Pair(200, 2, 128, "int8", 32)
    p.fill(rng, 200)
    q = kc.make_rows(rng, 6, 4, 128, "fp32")
    f = torch.tensor([1e-30, 1e-4, 0.1, 1.0, 1e-40, 4.0])[:, None, None]
    q = q * f
    slots = np.arange(200)
    k, v = p.k.values(slots), p.v.values(slots)
    vis = np.ones((6, 200), dtype=bool)
    scale = 1 / math.sqrt(128)
    want, _ = kv8.attention(q.numpy(), k, v, vis, scale)
    got = p.gpu.attention(1, q.cuda(), 200, 0, masks=[0] * 6).cpu().numpy()
    assert (np.abs(got - want) <= kc.out_error(q.numpy(), k, v, vis, want, scale, 0.0, "fp32")).all()


def test_scales_of_very_different_size():
    """V blocks whose scales differ by 2^20, in rising and falling order, and a block of zeros first."""
    rng = np.random.default_rng(4)
    for order in (1, -1):
        p = Pair(160, 1, 64, "int8", 16)
        k, v = kc.make_rows(rng, 160, 1, 64, "fp32"), kc.make_rows(rng, 160, 1, 64, "fp32")
        mag = 2.0 ** np.linspace(-10, 10, 160)[::order]
        v = v * torch.tensor(mag.copy(), dtype=torch.float32)[:, None, None]
        v[:16] = 0.0
        p.append(k, v, 0)
        q = kc.make_rows(rng, 3, 2, 64, "fp32")
        kk, vv = p.k.values(np.arange(160)), p.v.values(np.arange(160))
        vis = np.ones((3, 160), dtype=bool)
        want, _ = kv8.attention(q.numpy(), kk, vv, vis, 0.125)
        got = p.gpu.attention(1, q.cuda(), 160, 0, masks=[0] * 3).cpu().numpy()
        assert (np.abs(got - want) <= kc.out_error(q.numpy(), kk, vv, vis, want, 0.125, 0.0, "fp32")).all()


# ---------------------------------------------------------------- pages that are none

def test_block_table_entries_outside_the_pool():
    """Their slots are seen by nobody, read as zero, and appends to them are dropped."""
    rng = np.random.default_rng(6)
    p = Pair(256, 2, 64, "int8", 16)
    p.fill(rng, 256)
    good = p.gpu.block_table.clone()
    q = kc.make_rows(rng, 3, 4, 64, "fp32")
    keep = np.ones(256, dtype=bool)
    keep[64:128] = keep[192:] = False
    p.gpu.block_table[1], p.gpu.block_table[3] = -1, p.gpu.pool_pages
    k, v = p.gpu.read(1, 0, 256)
    assert not k.cpu().numpy()[~keep].any()
    assert np.array_equal(k.cpu().numpy()[keep], p.k.values(np.arange(256))[keep])
    vis = np.tile(keep, (3, 1))
    kk, vv = p.k.values(np.arange(256)), p.v.values(np.arange(256))
    want, _ = kv8.attention(q.numpy(), kk, vv, vis, 0.125)
    got, lse = p.gpu.attention(1, q.cuda(), 256, 0, masks=[0] * 3, return_lse=True)
    assert (np.abs(got.cpu().numpy() - want) <= kc.out_error(q.numpy(), kk, vv, vis, want, 0.125, 0.0, "fp32")).all()
    w = p.gpu.weights(1, q.cuda(), lse, 256, 0, masks=[0] * 3)
    assert not w.cpu().numpy()[:, ~keep].any() and np.allclose(w.sum(1).cpu().numpy(), 6, rtol=1e-4)
    before = [t.clone() for t in (p.gpu.k, p.gpu.v, p.gpu.k_scale, p.gpu.v_scale)]
    p.gpu.append(1, q.cuda()[:, :2].contiguous(), q.cuda()[:, :2].contiguous(), 70)
    for t, b in zip((p.gpu.k, p.gpu.v, p.gpu.k_scale, p.gpu.v_scale), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    p.gpu.block_table.fill_(-5)
    out, lse = p.gpu.attention(1, q.cuda(), 256, 0, masks=[0] * 3, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    p.gpu.block_table.copy_(good)


def test_block_table_entries_outside_the_pool_on_tcgen05():
    rng = np.random.default_rng(16)
    p = Pair(6400, 8, 64, "int8", 32)
    p.fill(rng, 6400)
    q = kc.make_rows(rng, 16, 64, 64, "fp32")
    keep = np.ones(6400, dtype=bool)
    for page, entry in ((0, -1), (17, p.gpu.pool_pages), (50, 2 ** 31 - 1), (51, -2 ** 31), (99, p.gpu.pool_pages + 5)):
        p.gpu.block_table[page] = entry
        keep[page * 64:page * 64 + 64] = False
    vis = np.tile(keep, (16, 1))
    k, v = p.k.values(np.arange(6400)), p.v.values(np.arange(6400))
    want, _ = kv8.attention(q.numpy(), k, v, vis, 0.125)
    got = p.gpu.attention(1, q.cuda(), 6400, 0, masks=[0] * 16).cpu().numpy()
    assert (np.abs(got - want) <= kc.out_error(q.numpy(), k, v, vis, want, 0.125, 0.0, "fp32")).all()


def test_offsets_past_32_bits():
    """Pages and layers that lie past 4 GB of codes: append, read, attention on both kernels, weights, eviction."""
    import self_speculative_decoding_layer_gb300 as ssd

    heads, hd, pool, layers = 8, 128, 40000, 2  # 2.6 GB of codes a layer and tensor
    k, v = (torch.empty((layers, pool, heads, 64, hd), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((layers, pool, heads, 2), device="cuda") for _ in range(2))
    pages = 100
    perm = np.random.default_rng(3).permutation(np.arange(pool - 120, pool))
    c = ssd.KVCache8.wrap(k, v, ks, vs, torch.tensor(perm[:pages], dtype=torch.int32, device="cuda"))
    d = ssd.KVCache8.wrap(k, v, ks, vs, torch.tensor(perm[pages:], dtype=torch.int32, device="cuda"))
    p = Pair(pages * 64, heads, hd, "int8", 32, layers=1, layer=0)
    rng = np.random.default_rng(5)
    n = pages * 64
    x, y = kc.make_rows(rng, n, heads, hd, "bf16").cuda(), kc.make_rows(rng, n, heads, hd, "bf16").cuda()
    c.append(1, x, y, 0)
    p.gpu.append(0, x, y, 0)
    for a, b in zip(c.read(1, 0, n), p.gpu.read(0, 0, n)):
        assert torch.equal(a, b)
    for rows in (1, 16):
        q = kc.make_rows(rng, rows, 64, hd, "bf16").cuda()
        (o, lse), (o2, lse2) = (g.attention(i, q, n - rows, return_lse=True) for g, i in ((c, 1), (p.gpu, 0)))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        w, w2 = c.weights(1, q, lse, n - rows), p.gpu.weights(0, q, lse, n - rows)
        assert torch.equal(w, w2)
    index, _ = c.evict(1, w, 1000, 10, d, 1)
    e = ssd.KVCache8(1, heads, hd, 1000, block_tokens=32)
    index2, _ = p.gpu.evict(0, w, 1000, 10, e, 0)
    assert torch.equal(index, index2)
    for a, b in zip(d.read(1, 0, 1000), e.read(0, 0, 1000)):
        assert torch.equal(a, b)


def test_two_attentions_at_once():
    """Calls on two streams with no order between them, on both kernels, over and over: no result depends on the other."""
    rng = np.random.default_rng(17)
    p = Pair(6400, 8, 64, "int8", 32)
    p.fill(rng, 6400)
    qs = [kc.make_rows(rng, r, 64, 64, "fp32").cuda() for r in (1, 16, 16, 3)]
    want = [p.gpu.attention(1, q, 6400 - q.shape[0]) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for rep in range(30):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append((q, p.gpu.attention(1, q, 6400 - q.shape[0])))
    torch.cuda.synchronize()
    for i, (q, o) in enumerate(got):
        assert torch.equal(o, want[i % 4]), i


def test_output_over_the_queries():
    rng = np.random.default_rng(18)
    p = Pair(6400, 8, 64, "int8", 32)
    p.fill(rng, 6400)
    for rows, prefix in ((1, 300), (3, 6000), (16, 6300)):
        q = kc.make_rows(rng, rows, 64, 64, "fp32").cuda()
        want = p.gpu.attention(1, q, prefix)
        assert p.gpu.attention(1, q, prefix, out=q) is q
        assert torch.equal(q, want)


# ---------------------------------------------------------------- eviction

EVICT = [  # n, keep, recent, heads, hd, code, block, to code, to block, weights
    (1, 1, 0, 1, 64, "int8", 16, "int8", 16, "normal"),
    (1, 1, 1, 3, 64, "e4m3", 32, "e4m3", 32, "normal"),
    (50, 20, 5, 2, 128, "int8", 64, "int8", 64, "normal"),
    (200, 200, 10, 2, 64, "e4m3", 16, "e4m3", 16, "normal"),   # all stay
    (200, 30, 30, 4, 128, "int8", 32, "int8", 32, "normal"),   # the last ones alone
    (300, 77, 0, 5, 64, "int8", 16, "int8", 16, "normal"),
    (1000, 130, 3, 8, 128, "e4m3", 32, "int8", 64, "ties"),
    (1000, 400, 100, 2, 64, "int8", 64, "e4m3", 16, "equal"),
    (700, 300, 7, 3, 64, "int8", 32, "int8", 32, "special"),
    (9000, 1111, 64, 2, 64, "int8", 64, "int8", 32, "normal"),
    (20001, 700, 1, 1, 64, "e4m3", 16, "e4m3", 64, "ties"),
]


@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict_matches_the_oracle(case):
    n, keep, recent, heads, hd, code, block, to_code, to_block, kind = case
    rng = np.random.default_rng(8)
    p = Pair(n, heads, hd, code, block)
    p.fill(rng, n)
    d = Pair(keep, heads, hd, to_code, to_block, seed=3)
    w = np.exp(rng.standard_normal((heads, n)) * 2).astype(np.float32)
    if kind == "ties":
        w = np.round(w)
    if kind == "equal":
        w[:] = 0.5
    if kind == "special":
        w[:, ::7], w[:, 1::7], w[:, 2::7], w[:, 3::7], w[:, 4::7] = np.nan, np.inf, -0.0, 0.0, -np.inf
        w[:, 5::7] = -1.0
    want = kv8.kept_slots(w.astype(np.float64), keep, recent)
    wide = torch.full((heads, n + 5), 1e9, device="cuda")
    wide[:, :n] = torch.tensor(w)
    index, kept = p.gpu.evict(1, wide[:, :n], keep, recent, d.gpu, 1)
    assert np.array_equal(index.cpu().numpy(), want)
    assert np.array_equal(kept.cpu().numpy(), np.take_along_axis(w, want, 1), equal_nan=True)
    d.k, d.v = (kv8.evict(c, want, to_code, to_block) for c in (p.k, p.v))
    d.same(keep)


def test_evict_within_one_pool():
    """The kept slots move to other pages of the same pool; the old pages are as they were."""
    import self_speculative_decoding_layer_gb300 as ssd

    rng = np.random.default_rng(11)
    p = Pair(500, 2, 64, "int8", 32, spare=4)
    p.fill(rng, 500)
    free = sorted(set(range(p.gpu.pool_pages)) - set(int(x) for x in p.perm))
    table = torch.tensor(free[:2], dtype=torch.int32, device="cuda")
    d = ssd.KVCache8.wrap(p.gpu.k, p.gpu.v, p.gpu.k_scale, p.gpu.v_scale, table)
    w = rng.random((2, 500)).astype(np.float32)
    index, _ = p.gpu.evict(1, torch.tensor(w).cuda(), 100, 10, d, 1)
    want = kv8.kept_slots(w, 100, 10)
    assert np.array_equal(index.cpu().numpy(), want)
    p.same(500)
    k, _ = d.read(1, 0, 100)
    assert np.array_equal(k.cpu().numpy(), kv8.evict(p.k, want, "int8", 32).values(np.arange(100)))


# ---------------------------------------------------------------- together

def test_a_long_generation_under_a_budget():
    """Prefill, then cycles of draft rows -> attention -> weights of the accepted rows -> rollback to them -> eviction
    when the budget is reached, followed step by step by the oracle."""
    heads, hq, hd, budget, keep, recent = 2, 8, 64, 200, 96, 16
    rng = np.random.default_rng(21)
    caches = [Pair(budget + 64, heads, hd, "int8", 16, seed=s) for s in (0, 1)]
    p = caches[0]
    p.fill(rng, 120)
    t = 120
    w = torch.zeros((heads, budget + 64), device="cuda")
    ow = np.zeros((heads, budget + 64))
    evictions = 0
    for cycle in range(40):
        rows = int(rng.integers(1, 8))
        new_k, new_v = kc.make_rows(rng, rows, heads, hd, "fp32"), kc.make_rows(rng, rows, heads, hd, "fp32")
        p.append(new_k, new_v, t)
        q = kc.make_rows(rng, rows, hq, hd, "fp32")
        out, lse = p.gpu.attention(1, q.cuda(), t, return_lse=True)
        vis = kc.visible(kc.masks("causal", rows, rng), rows, t, t, t + rows)
        k, v = p.k.values(np.arange(t + rows)), p.v.values(np.arange(t + rows))
        want, want_lse = kv8.attention(q.numpy(), k, v, vis)
        assert (np.abs(out.cpu().numpy() - want) <= kc.out_error(q.numpy(), k, v, vis, want, 0.125, 0.0, "fp32")).all()
        took = int(rng.integers(1, rows + 1))  # accepted rows
        ow[:, t + took:] = 0
        p.gpu.weights(1, q.cuda(), lse, t, rows=range(took), weight=w)
        ow[:, :t + rows] += kv8.weights(q.numpy(), k, vis, want_lse, range(took))
        t += took
        w[:, t:] = 0  # slots past the committed ones start anew
        assert np.allclose(w.cpu().numpy()[:, :t], ow[:, :t], rtol=1e-4, atol=1e-6)
        if t >= budget:
            evictions += 1
            other = caches[1] if p is caches[0] else caches[0]
            index, kept = p.gpu.evict(1, w[:, :t], keep, recent, other.gpu, 1)
            slots = kv8.kept_slots(w[:, :t].cpu().numpy(), keep, recent)
            assert np.array_equal(index.cpu().numpy(), slots)
            for x in ("k", "v"):
                o = kv8.evict(getattr(p, x), slots, "int8", 16)
                c = kv8.Cache8(budget + 64, heads, hd, "int8", 16)
                c.codes[: len(o.codes)], c.scale[: len(o.scale)] = o.codes, o.scale
                setattr(other, x, c)
            p, t = other, keep
            w.zero_()
            w[:, :keep] = kept
            ow[:] = 0
            ow[:, :keep] = kept.cpu().numpy()
            p.same(keep)
    assert evictions >= 1


def test_other_streams_and_graphs():
    """Calls on a side stream; two captured graphs over one cache, replayed at the same time on two streams."""
    rng = np.random.default_rng(13)
    p = Pair(4000, 8, 128, "int8", 64)
    p.fill(rng, 4000)
    qs = [kc.make_rows(rng, 7, 32, 128, "fp32").cuda() for _ in range(2)]
    want = [p.gpu.attention(1, q, 3900) for q in qs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = p.gpu.attention(1, qs[0], 3900)
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = p.gpu.attention(1, q, 3900, return_lse=True)
            w = p.gpu.weights(1, q, lse, 3900)
        graphs.append(g)
        outs.append((o, w))
    streams = [torch.cuda.Stream() for _ in qs]
    for rep in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (o, w), x in zip(outs, want):
        assert torch.equal(o, x)
        assert np.allclose(w.sum(1).cpu().numpy(), 28, rtol=1e-4)


def test_capture_of_append_and_evict():
    rng = np.random.default_rng(14)
    p, d = Pair(300, 2, 64, "int8", 16), Pair(64, 2, 64, "int8", 16, seed=1)
    p.fill(rng, 300)
    k = kc.make_rows(rng, 3, 2, 64, "fp32")
    w = torch.rand((2, 300), device="cuda")
    dk = k.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.gpu.append(1, dk, dk, 150)
        index, kept = p.gpu.evict(1, w, 64, 8, d.gpu, 1)
    g.replay()
    p.k.append(k.numpy(), 150)
    p.v.append(k.numpy(), 150)
    p.same(153)
    w.copy_(torch.rand((2, 300), device="cuda"))
    g.replay()
    assert np.array_equal(index.cpu().numpy(), kv8.kept_slots(w.cpu().numpy(), 64, 8))


# ---------------------------------------------------------------- what the binding refuses

def test_binding_refusals():
    import self_speculative_decoding_layer_gb300 as ssd

    p = Pair(128, 4, 64, "int8", 16)
    c, g = p.gpu, p.gpu
    ok = torch.zeros((2, 4, 64), device="cuda")
    q = torch.zeros((2, 8, 64), device="cuda")
    lse = torch.zeros((2, 8), device="cuda")
    w = torch.zeros((4, 128), device="cuda")
    d = Pair(64, 4, 64, "int8", 16).gpu
    bad = [
        lambda: c.append(1, ok.cpu(), ok, 0), lambda: c.append(1, ok.double(), ok.double(), 0), lambda: c.append(1, ok, ok[:1], 0),
        lambda: c.append(1, ok, ok.half(), 0), lambda: c.append(2, ok, ok, 0), lambda: c.append(-1, ok, ok, 0),
        lambda: c.append(1, ok, ok, 127), lambda: c.append(1, ok, ok, -1), lambda: c.append(1, ok[:0], ok[:0], 0),
        lambda: c.append(1, ok.transpose(1, 2).contiguous().transpose(1, 2), ok, 0), lambda: c.append(1, ok[..., :32], ok, 0),
        lambda: c.append(1, torch.zeros(2 * 4 * 64 + 1, device="cuda")[1:].view(2, 4, 64), ok, 0),
        lambda: c.read(1, 0, 0), lambda: c.read(1, 100, 29), lambda: c.read(1, 0, 4, torch.int8),
        lambda: c.attention(1, q[:, :6], 10), lambda: c.attention(1, torch.zeros((65, 8, 64), device="cuda"), 10),
        lambda: c.attention(1, q, 129), lambda: c.attention(1, q, 127), lambda: c.attention(1, q, 10, masks=[1]),
        lambda: c.attention(1, q, 10, scale=0.0), lambda: c.attention(1, q, 10, softcap=-1.0),
        lambda: c.attention(1, q, 10, out=torch.zeros_like(q).half()), lambda: c.attention(1, q, 10, out=torch.zeros((8, 2, 64), device="cuda").transpose(0, 1)),
        lambda: c.weights(1, q, lse[:1], 10), lambda: c.weights(1, q, lse.double(), 10), lambda: c.weights(1, q, lse, 10, rows=[2]),
        lambda: c.weights(1, q, lse, 10, weight=w[:, :11]), lambda: c.weights(1, q, lse, 10, weight=w.half()),
        lambda: c.weights(1, q, lse, 10, weight=w[:1].expand(4, 128)), lambda: c.weights(1, q, lse, 10, weight=w, out=w[:, :64].contiguous()),
        lambda: c.evict(1, w, 65, 0, d, 1), lambda: c.evict(1, w, 0, 0, d, 1), lambda: c.evict(1, w, 8, 9, d, 1),
        lambda: c.evict(1, w[:2], 8, 0, d, 1), lambda: c.evict(1, w, 8, 0, Pair(64, 2, 64, "int8", 16).gpu, 1),
        lambda: c.evict(1, torch.zeros((4, 129), device="cuda"), 8, 0, d, 1), lambda: c.evict(1, w, 8, 0, c, 1),
        lambda: c.attention(1, q.expand(2, 8, 64)[:1].expand(2, 8, 64), 10), lambda: c.append(1, ok, None, 0),
        lambda: c.append(1, ok, ok, 2 ** 40), lambda: c.attention(1, q, 10, softcap=1e-35),
        lambda: ssd.KVCache8(1, 4, 96, 100), lambda: ssd.KVCache8(1, 4, 64, 0), lambda: ssd.KVCache8(1, 4, 64, 64, dtype=torch.uint8),
        lambda: ssd.KVCache8(1, 4, 64, 64, block_tokens=8), lambda: ssd.KVCache8.wrap(g.k, g.v[:1], g.k_scale, g.v_scale, g.block_table),
        lambda: ssd.KVCache8.wrap(g.k, g.v, g.k_scale[..., :3], g.v_scale, g.block_table),
        lambda: ssd.KVCache8.wrap(g.k, g.v, g.k_scale, g.v_scale, g.block_table.long()),
        lambda: ssd.KVCache8.wrap(g.k, g.v, g.k_scale, g.v_scale, g.block_table[:0]),
        lambda: ssd.KVCache8.wrap(g.k.transpose(1, 2), g.v.transpose(1, 2), g.k_scale, g.v_scale, g.block_table),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ssd.SSDError):
            f()
            pytest.fail(f"call {i} was not refused")


def test_a_fresh_cache():
    import self_speculative_decoding_layer_gb300 as ssd

    for dt in (torch.int8, torch.float8_e4m3fn):
        c = ssd.KVCache8(2, 3, 64, 100, dtype=dt, block_tokens=32)
        assert c.n_pages == 2 and c.k.shape == (2, 2, 3, 64, 64) and c.k_scale.shape == (2, 2, 3, 2)
        k, v = c.read(0, 0, 128)
        assert not k.any() and not v.any()
        # magnitudes whose scale is a power of two: qmax / qmax and 2 qmax / qmax
        x = torch.full((5, 3, 64), 127.0 if dt == torch.int8 else 448.0, device="cuda")
        c.append(1, x, 2 * x, 0)
        k, v = c.read(1, 0, 5)
        assert torch.equal(k, x) and torch.equal(v, 2 * x)
        o = c.attention(1, x / 448, 0)
        assert torch.allclose(o, 2 * x, rtol=2.0 ** -20, atol=0)  # a mean of equal values


@pytest.mark.parametrize("rows,prefix,hq,hkv", [(3, 300, 16, 4), (17, 9000, 40, 5)], ids=str)
def test_a_cap_far_above_the_scores_of_fp32_queries(rows, prefix, hq, hkv):
    """tanh y = y (1 - y^2 / 3 ..), so under a cap of 1e6 a score s moves by less than s^3 / 3e12, and by its roundings:
    the product with 1 / cap, two sums of three products each, the quotient (two steps), the product with cap: ten of
    2^-24 of it at most.  A weight moves by that times e^.., twice with its sum, and the output by that times the values."""
    case = (rows, prefix, 0, "causal", hq, hkv, 128, "int8", 32, "fp32", 0.0)
    p, q, m, _, n, base = attention_case(case)
    plain = p.gpu.attention(1, q.cuda(), prefix, base, masks=m).double()
    capped = p.gpu.attention(1, q.cuda(), prefix, base, masks=m, softcap=1e6).double()
    k, v = (torch.tensor(t.values(np.arange(n))) for t in (p.k, p.v))
    s = float(q.float().norm(dim=-1).max() * k.float().norm(dim=-1).max()) / math.sqrt(128)
    move = s ** 3 / 3e12 + 10 * s * 2.0 ** -24 + 4 * s * 2.0 ** -24  # (and each call's own scores, rounded twice)
    assert move < 0.01
    limit = 2.1 * move + 2 * 2.0 ** -22  # (either call's exponentials and 22-bit weights)
    assert float((plain - capped).abs().max()) <= limit * float(v.abs().max())
