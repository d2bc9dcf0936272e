"""The 8-bit KV cache operators: what they compute, on which inputs, and how much work that is.

One layer of a paged cache of 8-bit codes with one fp32 scale for each block of T tokens and KV head:

* append     quantises new K/V rows into the cache (read back after it, so that the result comes as values);
* attention  of up to 64 rows over it, with the visibility rule of the framework's attention (a prefix, and a
             bit mask over the new slots), an optional tanh cap of the scores, and the rows' log-sum-exp;
* weights    adds the attention weight that each slot got from chosen rows to an accumulator;
* evict      keeps the last slots and the heaviest others of every KV head, compacted into other pages.

`run` computes them in plain torch operations, or with the framework's kernels where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64
QMAX = {"int8": 127.0, "e4m3": 448.0}
FLOATS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = 2.0 ** -126  # scales below the smallest normal fp32 number become zero


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one decoded token's K/V at an odd position of the 8B shape: the smallest call, one block touched
        dict(name="append token", op="append", rows=1, base=777, hkv=8, hd=128, io="fp32", code="int8", block=64),
        # the K/V of a 17-node draft tree of the 13B shape, from the middle of a block on
        dict(name="append tree", op="append", rows=17, base=523, hkv=40, hd=128, io="fp16", code="e4m3", block=16),
        # a long prompt's K/V at once
        dict(name="append prompt", op="append", rows=16384, base=0, hkv=8, hd=128, io="bf16", code="int8", block=32),
        # a draft step of the 8B shape: one row over a short context, where latency counts
        dict(name="attention token", op="attention", rows=1, prefix=640, gap=0, mask="causal", hq=32, hkv=8, hd=128, io="fp32",
             code="int8", block=64, cap=0.0),
        # a decoded token over a long context of the 70B shape, 16-bit activations
        dict(name="attention long token", op="attention", rows=1, prefix=65531, gap=0, mask="causal", hq=64, hkv=8, hd=128,
             io="bf16", code="e4m3", block=64, cap=0.0),
        # the verify pass of six drafts over a middling context
        dict(name="attention verify", op="attention", rows=7, prefix=4093, gap=0, mask="causal", hq=32, hkv=8, hd=128, io="fp32",
             code="int8", block=32, cap=0.0),
        # a draft tree's verify pass on a decoder without shared KV heads that caps its scores
        dict(name="attention tree", op="attention", rows=17, prefix=1301, gap=0, mask="tree", hq=40, hkv=40, hd=128, io="fp16",
             code="int8", block=16, cap=30.0),
        # a chunk of prefill rows behind a long context: the most arithmetic
        dict(name="attention chunk", op="attention", rows=64, prefix=16384, gap=0, mask="causal", hq=64, hkv=8, hd=128, io="bf16",
             code="int8", block=64, cap=0.0),
        # the attention weight of one decoded token over a short context
        dict(name="weights token", op="weights", rows=1, prefix=1024, gap=0, mask="causal", hq=32, hkv=8, hd=128, io="fp32",
             code="int8", block=64, cap=0.0),
        # that of a verify pass's accepted rows over a long context
        dict(name="weights verify", op="weights", rows=9, prefix=32767, gap=0, mask="causal", hq=64, hkv=8, hd=128, io="bf16",
             code="e4m3", block=32, cap=0.0),
        # a small budget on the 8B shape
        dict(name="evict short", op="evict", n=1535, keep=512, recent=64, hkv=8, hd=128, code="int8", block=64),
        # a long context down to a quarter of its slots
        dict(name="evict long", op="evict", n=65531, keep=16381, recent=1024, hkv=8, hd=128, code="int8", block=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "weights", "evict"])
    hd = rng.choice([64, 128, 128])
    code, block = rng.choice(["int8", "e4m3"]), rng.choice([16, 32, 64])
    io = rng.choice(["fp32", "bf16", "fp16"])
    hq, hkv = rng.choice([(4, 4), (32, 8), (40, 40), (64, 8), (16, 2), (8, 1), (10, 10), (21, 3)])
    if op == "append":
        rows = _log(rng, 1, 16384 * 8 // max(hkv, 8))
        return dict(op=op, rows=rows, base=rng.choice([0, rng.randrange(0, 4096)]), hkv=hkv, hd=hd, io=io, code=code,
                    block=block)
    if op == "evict":
        n = _log(rng, 2, 65531 * 8 // max(hkv, 8))
        keep = rng.randrange(1, max(2, n // 4 + 1))
        return dict(op=op, n=n, keep=keep, recent=rng.randrange(0, keep + 1), hkv=hkv, hd=hd, code=code, block=block)
    rows = _log(rng, 1, 64)
    prefix = min(_log(rng, 1, 65531 * 8 // max(hkv, 8)), 64 * 64 * 16384 // (rows * hq))
    return dict(op=op, rows=rows, prefix=prefix, gap=rng.choice([0, 0, rng.randrange(0, 100)]),
                mask=rng.choice(["causal", "tree", "own"]), hq=hq, hkv=hkv, hd=hd, io=io, code=code, block=block,
                cap=rng.choice([0.0, 0.0, 30.0]))


# ------------------------------------------------------------------------------------------------ inputs


def _codes_of(y, code):
    """Codes of values that are already divided by their scale."""
    if code == "int8":
        return torch.round(y).clamp(-127.0, 127.0).to(torch.int8)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _quantised(x, code, least=None):
    """(codes, scales) of x [..., blocks, T, hd] in fp32: one scale for each block, `least` at least."""
    s = x.abs().amax((-1, -2))
    s = s / torch.full_like(s, QMAX[code])  # by a tensor: a scalar's reciprocal would be rounded first
    s = torch.where(s < TINY, torch.zeros_like(s), s)
    if least is not None:
        s = torch.maximum(s, least)
    m = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return _codes_of(x * m[..., None, None], code), s


def _random_cache(g, slots, case, pages=None):
    """A cache whose first `slots` slots hold tokens: pages in a random order in a pool larger than the table."""
    hkv, hd, T = case["hkv"], case["hd"], case["block"]
    n_pages = pages or max(1, -(-slots // PAGE))
    pool = n_pages + 3
    dev = DEV
    dt = torch.int8 if case["code"] == "int8" else torch.float8_e4m3fn
    k = torch.zeros((1, pool, hkv, PAGE, hd), dtype=torch.int8, device=dev).view(dt)
    v = torch.zeros_like(k)
    ks = torch.zeros((1, pool, hkv, PAGE // T), dtype=torch.float32, device=dev)
    vs = torch.zeros_like(ks)
    table = torch.randperm(pool, generator=g, device=dev)[:n_pages].to(torch.int32)
    if slots:
        # keys have a few large channels, as real ones do, and tokens of different size
        gain = torch.ones(hd, device=dev)
        gain[:: max(1, hd // 4)] = 6.0
        for codes, scales, by in ((k, ks, gain), (v, vs, torch.ones(hd, device=dev))):
            x = torch.randn((n_pages, hkv, PAGE, hd), generator=g, device=dev) * by
            x *= 0.5 + torch.rand((n_pages, hkv, PAGE, 1), generator=g, device=dev)
            c, s = _quantised(x.view(n_pages, hkv, PAGE // T, T, hd), case["code"])
            codes.view(torch.int8)[0, table.long()] = c.view(torch.int8).view(n_pages, hkv, PAGE, hd)
            scales[0, table.long()] = s
    return dict(k=k, v=v, ks=ks, vs=vs, table=table)


def _masks(case, g):
    rows = case["rows"]
    if case["mask"] == "causal":
        return [(1 << (r + 1)) - 1 for r in range(rows)]
    if case["mask"] == "own":
        return [1 << r for r in range(rows)]
    up = torch.rand(rows, generator=g, device=DEV).tolist()
    anc = []
    for c in range(rows):  # each node's parent is one of those before it
        anc.append((anc[int(up[c] * c)] if c else 0) | (1 << c))
    return anc


def _visible(case, masks, n):
    """[rows, n] truth values: slots of the prefix, and the new slots of each row's mask."""
    rows, prefix, base = case["rows"], case["prefix"], case["prefix"] + case["gap"]
    vis = torch.zeros((rows, n), dtype=torch.bool)
    vis[:, :prefix] = True
    bits = torch.tensor([[(m >> e) & 1 for e in range(rows)] for m in masks], dtype=torch.bool)
    vis[:, base:base + rows] |= bits
    return vis.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    io = FLOATS.get(case.get("io"))
    hkv, hd = case["hkv"], case["hd"]
    st = dict(case=case)
    if case["op"] == "append":
        rows, base = case["rows"], case["base"]
        st["cache"] = _random_cache(g, base, case, pages=-(-(base + rows) // PAGE))
        # K and V are slices of one projection's output rows
        qkv = torch.randn((rows, 4, hkv, hd), generator=g, device=DEV).to(io)
        st["k"], st["v"] = qkv[:, 2], qkv[:, 3]
    elif case["op"] == "evict":
        n = case["n"]
        st["cache"] = _random_cache(g, n, case)
        st["kept"] = _random_cache(g, 0, case, pages=-(-case["keep"] // PAGE))
        # a few slots draw most of the weight, many little, some none at all
        w = torch.randn((hkv, n), generator=g, device=DEV).mul_(2.0).exp_()
        st["w"] = torch.where(torch.rand((hkv, n), generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
    else:
        rows, base = case["rows"], case["prefix"] + case["gap"]
        n = base + rows
        st["cache"] = _random_cache(g, n, case)
        st["q"] = torch.randn((rows, case["hq"], hd), generator=g, device=DEV).to(io)
        st["masks"] = _masks(case, g)
        st["vis"] = _visible(case, st["masks"], n)
        if case["op"] == "weights":
            st["rows"] = list(range(0, rows, 2)) if rows > 1 else [0]  # the rows that were accepted
            st["lse"] = _attend(st, torch.float64)[1].to(torch.float32)
            st["w"] = torch.rand((hkv, n), generator=g, device=DEV) * rows
            st["w_new"] = torch.empty_like(st["w"])
    return st


# ------------------------------------------------------------------------------------------------ plain forms


def _values(c, which, case, slots, ftype=torch.float32):
    """The values [slots, hkv, hd] that the first `slots` slots hold."""
    T = case["block"]
    pages = c["table"][: -(-slots // PAGE)].long()
    x = c[which][0].view(torch.int8)[pages].view(c[which].dtype).to(ftype)
    s = c[which + "s"][0][pages].to(ftype)
    x = x * s.repeat_interleave(T, -1)[..., None]
    return x.transpose(1, 2).reshape(-1, case["hkv"], case["hd"])[:slots]


def _scores(st, ftype):
    """[hkv, rows, group, n] scores of every slot (masked ones among them)."""
    case = st["case"]
    rows, hq, hkv, hd = case["rows"], case["hq"], case["hkv"], case["hd"]
    n = case["prefix"] + case["gap"] + rows
    k = _values(st["cache"], "k", case, n, ftype).permute(1, 2, 0)  # [hkv, hd, n]
    q = st["q"].to(ftype).view(rows, hkv, hq // hkv, hd).permute(1, 0, 2, 3).reshape(hkv, -1, hd)
    s = torch.matmul(q, k) * (1.0 / math.sqrt(hd))
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    return s.view(hkv, rows, hq // hkv, n)


def _attend(st, ftype):
    case = st["case"]
    rows, hq, hkv, hd = case["rows"], case["hq"], case["hkv"], case["hd"]
    s = _scores(st, ftype)
    n = s.shape[-1]
    s = s.masked_fill(~st["vis"].view(1, rows, 1, n), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    v = _values(st["cache"], "v", case, n, ftype).transpose(0, 1)  # [hkv, n, hd]
    o = torch.matmul(p.view(hkv, -1, n), v).view(hkv, rows, hq // hkv, hd)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total)).squeeze(-1)
    return o.permute(1, 0, 2, 3).reshape(rows, hq, hd), lse.permute(1, 0, 2).reshape(rows, hq)


def _weigh(st, ftype):
    case = st["case"]
    rows, hq, hkv = case["rows"], case["hq"], case["hkv"]
    lse = st["lse"].to(ftype).view(rows, hkv, hq // hkv).permute(1, 0, 2)[..., None]
    p = torch.exp(_scores(st, ftype) - lse) * st["vis"].view(1, rows, 1, -1)
    return st["w"].to(ftype) + p[:, st["rows"]].sum((1, 2))


def _append(st):
    case, c = st["case"], st["cache"]
    rows, base, hkv, hd, T = case["rows"], case["base"], case["hkv"], case["hd"], case["block"]
    b0, b1 = base // T, -(-(base + rows) // T)
    block = torch.arange(b0, b1, device=DEV)
    page, part = c["table"][block * T // PAGE].long(), block % (PAGE // T)
    slot = torch.arange(b0 * T, base + rows, device=DEV)
    spage = c["table"][slot // PAGE].long()
    out = []
    for which in ("k", "v"):
        x = torch.zeros(((b1 - b0) * T, hkv, hd), dtype=torch.float32, device=DEV)
        x[base - b0 * T: base - b0 * T + rows] = st[which].to(torch.float32)
        x = x.view(b1 - b0, T, hkv, hd).transpose(1, 2)  # [blocks, hkv, T, hd]
        least = torch.zeros((b1 - b0, hkv), dtype=torch.float32, device=DEV)
        if base % T:  # the block of slots that stay
            old = c[which + "s"][0, page[0], :, part[0]]
            first = int(base - b0 * T)
            lo = int((b0 * T) % PAGE)
            kept = c[which].view(torch.int8)[0, page[0]][:, lo:lo + first].view(c[which].dtype).to(torch.float32)
            _, fresh = _quantised(x, case["code"])
            least[0] = old
            x = x.clone()
            x[0, :, :first] = kept * old[:, None, None]
            s = torch.maximum(fresh, least)
            m = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
            codes = _codes_of(x * m[..., None, None], case["code"])
        else:
            codes, s = _quantised(x, case["code"])
        flat = codes.view(torch.int8).transpose(1, 2).reshape(-1, hkv, hd)[: base + rows - b0 * T]
        c[which].view(torch.int8)[0, spage, :, slot % PAGE] = flat
        c[which + "s"][0, page, :, part] = s
        got = (codes.to(torch.float32) * s[..., None, None]).transpose(1, 2).reshape(-1, hkv, hd)
        out.append(got[: base + rows - b0 * T].to(st[which].dtype))
    return dict(k=out[0], v=out[1], k_scale=c["ks"], v_scale=c["vs"])


def _evict(st):
    case, c, d = st["case"], st["cache"], st["kept"]
    n, keep, recent, hkv, hd, T = case["n"], case["keep"], case["recent"], case["hkv"], case["hd"], case["block"]
    order = torch.sort(st["w"][:, : n - recent], dim=1, descending=True, stable=True)[1][:, : keep - recent]
    order = torch.sort(order, dim=1)[0]
    last = torch.arange(n - recent, n, device=DEV).expand(hkv, recent)
    index = torch.cat([order, last], 1)  # [hkv, keep], in slot order
    head = torch.arange(hkv, device=DEV)[:, None]
    blocks = -(-keep // T)
    block = torch.arange(blocks, device=DEV)
    page, part = d["table"][block * T // PAGE].long(), block % (PAGE // T)
    slot = torch.arange(keep, device=DEV)
    out = []
    for which in ("k", "v"):
        from_page = c["table"][index // PAGE].long()
        raw = c[which].view(torch.int8)[0, from_page, head, index % PAGE].view(c[which].dtype).to(torch.float32)
        x = torch.zeros((hkv, blocks * T, hd), dtype=torch.float32, device=DEV)
        x[:, :keep] = raw * c[which + "s"][0, from_page, head, index % PAGE // T][..., None]
        codes, s = _quantised(x.view(hkv, blocks, T, hd), case["code"])
        flat = codes.view(torch.int8).view(hkv, -1, hd)[:, :keep].transpose(0, 1)
        d[which].view(torch.int8)[0, d["table"][slot // PAGE].long(), :, slot % PAGE] = flat
        d[which + "s"][0, page, :, part] = s.transpose(0, 1)
        got = (codes.to(torch.float32) * s[..., None, None]).view(hkv, -1, hd)[:, :keep]
        out.append(got.transpose(0, 1).contiguous())
    return dict(index=index.to(torch.int32), w=st["w"].gather(1, index), k=out[0], v=out[1], k_scale=d["ks"], v_scale=d["vs"])


def _plain(st):
    op = st["case"]["op"]
    if op == "append":
        return _append(st)
    if op == "evict":
        return _evict(st)
    if op == "attention":
        o, lse = _attend(st, torch.float32)
        return dict(out=o.to(st["q"].dtype), lse=lse)
    return dict(w=_weigh(st, torch.float32))


# ------------------------------------------------------------------------------------------------ the framework's


def _handle(st, which):
    """The cache object that a program keeps over its buffers."""
    import self_speculative_decoding_layer_gb300 as ssd

    c = st[which]
    c["handle"] = ssd.KVCache8.wrap(c["k"], c["v"], c["ks"], c["vs"], c["table"])
    return c["handle"]


def _framework(st):
    case, c = st["case"], st["cache"]
    cache = c.get("handle") or _handle(st, "cache")
    op = case["op"]
    if op == "append":
        base, T = case["base"], case["block"]
        cache.append(0, st["k"], st["v"], base)
        k, v = cache.read(0, base // T * T, base + case["rows"] - base // T * T, st["k"].dtype)
        return dict(k=k, v=v, k_scale=c["ks"], v_scale=c["vs"])
    if op == "evict":
        kept = st["kept"].get("handle") or _handle(st, "kept")
        index, w = cache.evict(0, st["w"], case["keep"], case["recent"], kept, 0)
        k, v = kept.read(0, 0, case["keep"], torch.float32)
        return dict(index=index, w=w, k=k, v=v, k_scale=st["kept"]["ks"], v_scale=st["kept"]["vs"])
    base = case["prefix"] + case["gap"]
    masks = None if case["mask"] == "causal" else st["masks"]
    if op == "attention":
        out, lse = cache.attention(0, st["q"], case["prefix"], base, masks=masks, softcap=case["cap"], return_lse=True)
        return dict(out=out, lse=lse)
    return dict(w=cache.weights(0, st["q"], st["lse"], case["prefix"], base, masks=masks, softcap=case["cap"], rows=st["rows"],
                                weight=st["w"], out=st["w_new"]))


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work and definition


def work(case):
    hkv, hd, T = case["hkv"], case["hd"], case["block"]
    size = {"fp32": 4, "bf16": 2, "fp16": 2}.get(case.get("io"), 4)
    if case["op"] == "append":
        rows = case["rows"]
        part = case["base"] % T
        vals = rows * hkv * hd * 2
        kept = part * hkv * hd * 2
        scales = 2 * hkv * (-(-(part + rows) // T)) * 4
        # rows in, codes out, the kept codes of the first block in; and the values of all of them read back
        return dict(bytes=vals * size + vals + kept + scales + (vals + kept) * size, flops=4 * (vals + kept))
    if case["op"] == "evict":
        n, keep = case["n"], case["keep"]
        vals = keep * hkv * hd * 2
        scales = 2 * hkv * (-(-keep // T)) * 4
        return dict(bytes=n * hkv * 4 + 2 * vals + 2 * scales + keep * hkv * 8 + vals * 4, flops=6 * vals)
    rows, hq = case["rows"], case["hq"]
    slots = case["prefix"] + rows
    pairs = {"causal": (rows + 1) / 2, "own": 1, "tree": math.log2(rows + 1)}[case["mask"]] + case["prefix"]
    codes = slots * hkv * hd
    scales = -(-slots // T) * hkv * 4
    if case["op"] == "attention":
        return dict(bytes=2 * (codes + scales) + 2 * rows * hq * hd * size + rows * hq * 4, flops=4 * rows * hq * hd * pairs)
    take = -(-rows // 2)
    return dict(bytes=codes + scales + take * hq * (hd * size + 4) + 2 * slots * hkv * 4, flops=2 * take * hq * hd * pairs)


def _e4m3(y):
    """The nearest e4m3 number (ties to the even one) of float64 values up to 448 in magnitude."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(y / step) * step


def _f32(x):
    return x.to(torch.float32).to(torch.float64)


def _requantised(x, keep_scale, code):
    """x [..., T, hd] float64 holding fp32 values; scales and codes are decided in fp32, so each step is rounded there."""
    s = _f32(x.abs().amax((-1, -2)) / QMAX[code])
    s = torch.where(s < TINY, torch.zeros_like(s), s)
    if keep_scale is not None:
        s = torch.maximum(s, keep_scale)
    return s


def _encoded(x, s, code):
    inv = torch.where(s > 0, _f32(1.0 / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(s))
    y = _f32(x * inv[..., None, None]).clamp(-QMAX[code], QMAX[code])
    return torch.round(y) if code == "int8" else _e4m3(y)


def exact(case, seed):
    st = prepare(case, seed)
    code, T, hkv, hd = case["code"], case["block"], case["hkv"], case["hd"]
    f64 = torch.float64
    if case["op"] in ("attention", "weights"):
        rows, hq, base = case["rows"], case["hq"], case["prefix"] + case["gap"]
        group = hq // hkv
        c, n = st["cache"], base + case["rows"]
        slot = torch.arange(n, device=DEV)
        page = c["table"].long()[slot // PAGE]
        out = torch.zeros((rows, hq, hd), dtype=f64, device=DEV)
        lse = torch.zeros((rows, hq), dtype=f64, device=DEV)
        w = st["w"].to(f64).clone() if case["op"] == "weights" else None
        for h in range(hkv):  # one KV head at a time
            kv = [c[x].view(torch.int8)[0, page, h, slot % PAGE].view(c[x].dtype).to(f64) *
                  c[x + "s"][0, page, h, slot % PAGE // T].to(f64)[:, None] for x in ("k", "v")]
            q = st["q"][:, h * group:(h + 1) * group].to(f64).reshape(-1, hd)
            s = q @ kv[0].T / math.sqrt(hd)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            seen = st["vis"][:, None, :].expand(rows, group, n).reshape(-1, n)
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            if w is not None:
                p = torch.exp(s - st["lse"][:, h * group:(h + 1) * group].to(f64).reshape(-1, 1)).view(rows, group, n)
                for r in st["rows"]:
                    w[h] += p[r].sum(0)
                continue
            some = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out[:, h * group:(h + 1) * group] = (p @ kv[1]).view(rows, group, hd)
            lse[:, h * group:(h + 1) * group] = some.view(rows, group)
        return dict(w=w) if w is not None else dict(out=out, lse=lse)
    if case["op"] == "append":
        rows, base, c = case["rows"], case["base"], st["cache"]
        b0, b1 = base // T, -(-(base + rows) // T)
        res = {}
        for x in ("k", "v"):
            scales = c[x + "s"].to(f64).clone()
            val = torch.zeros(((b1 - b0) * T, hkv, hd), dtype=f64, device=DEV)
            off = base - b0 * T
            val[off:off + rows] = st[x].to(f64)
            val = val.view(b1 - b0, T, hkv, hd).transpose(1, 2).clone()
            s = _requantised(val, None, code)
            if off:
                p0, part = int(c["table"][b0 * T // PAGE]), b0 % (PAGE // T)
                old = c[x + "s"][0, p0, :, part].to(f64)
                lo = b0 * T % PAGE
                kept = c[x].view(torch.int8)[0, p0, :, lo:lo + off].view(c[x].dtype).to(f64)
                val[0, :, :off] = _f32(kept * old[:, None, None])
                s[0] = torch.maximum(s[0], old)
            got = (_encoded(val, s, code) * s[..., None, None]).transpose(1, 2).reshape(-1, hkv, hd)
            res[x] = got[: off + rows]
            blk = torch.arange(b0, b1, device=DEV)
            scales[0, c["table"].long()[blk * T // PAGE], :, blk % (PAGE // T)] = s
            res[x + "_scale"] = scales
        return res
    n, keep, recent, c, d = case["n"], case["keep"], case["recent"], st["cache"], st["kept"]
    res = dict(index=None, w=torch.zeros((hkv, keep), dtype=f64, device=DEV))
    blocks = -(-keep // T)
    blk = torch.arange(blocks, device=DEV)
    for x in ("k", "v"):
        res[x] = torch.zeros((keep, hkv, hd), dtype=f64, device=DEV)
        res[x + "_scale"] = d[x + "s"].to(f64).clone()
    for h in range(hkv):
        w = st["w"][h].to(f64)
        # heavier first, the lower slot among equal ones
        rank = sorted(range(n - recent), key=lambda i, v=w.tolist(): (-v[i], i))[: keep - recent]
        idx = torch.tensor(sorted(rank) + list(range(n - recent, n)), device=DEV, dtype=torch.long)
        res["w"][h] = w[idx]
        page = c["table"].long()[idx // PAGE]
        for x in ("k", "v"):
            val = c[x].view(torch.int8)[0, page, h, idx % PAGE].view(c[x].dtype).to(f64)
            val = _f32(val * c[x + "s"][0, page, h, idx % PAGE // T].to(f64)[:, None])
            full = torch.zeros((blocks * T, hd), dtype=f64, device=DEV)
            full[:keep] = val
            full = full.view(blocks, T, hd)
            s = _requantised(full, None, code)
            res[x][:, h] = (_encoded(full, s, code) * s[:, None, None]).view(-1, hd)[:keep]
            res[x + "_scale"][0, d["table"].long()[blk * T // PAGE], h, blk % (PAGE // T)] = s
    return res
