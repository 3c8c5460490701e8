"""What is measured of the 8-bit key/value cache: writing it, reading it back, attending over it.

A cache holds codes [B, n_cap, Hkv, D] in e4m3 or int8 and one fp32 scale for each block of
tokens and head, [B, ceil(n_cap / block), Hkv]; a value is code * scale. A write gives every
block it touches the smallest power of two that brings its largest new value into the codes'
range, or keeps the block's scale where that is larger; rows that were in the block before
keep their values, rounded to the new scale.

``run`` with ``own`` false is the plain form (elementary torch operations in 32 bits), with
``own`` true the framework's calls. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
REAL = {"bf16": torch.bfloat16, "f32": torch.float32}
LEAST = -100            # exponent of the smallest scale


# ------------------------------------------------------------------------- cases --
def _write(name, fmt, block, dtype, batch, rows, hkv, dim, n_cap, start=-1, fused=False):
    return {"name": name, "op": "write", "fmt": fmt, "block": block, "dtype": dtype, "batch": batch, "rows": rows,
            "hkv": hkv, "dim": dim, "n_cap": n_cap, "start": start, "fused": fused}


def _read(name, fmt, block, dtype, batch, rows, hkv, dim, n_cap, start=-1):
    return {"name": name, "op": "read", "fmt": fmt, "block": block, "dtype": dtype, "batch": batch, "rows": rows,
            "hkv": hkv, "dim": dim, "n_cap": n_cap, "start": start}


def _attn(name, fmt, block, dtype, batch, lq, hq, hkv, dim, n_cap, c0, n_init, window, topk, heads=False):
    return {"name": name, "op": "attn", "fmt": fmt, "block": block, "dtype": dtype, "batch": batch, "lq": lq,
            "hq": hq, "hkv": hkv, "dim": dim, "n_cap": n_cap, "c0": c0, "n_init": n_init, "window": window,
            "topk": topk, "heads": heads}


def listed():
    """start or c0 of -1: sequences of different lengths (device lengths, see _lengths)."""
    return [
        # a decode step's new token of 16 sequences, each at its own length
        _write("write_step_b16", "e4m3", 64, "bf16", 16, 1, 8, 128, 8192),
        # one prefill chunk that begins inside a block, out of a fused projection's rows
        _write("write_chunk_ragged", "int8", 32, "bf16", 2, 509, 8, 128, 8192, start=4099, fused=True),
        # a whole prompt of a layer with 8 key/value heads
        _write("write_prompt_32k", "e4m3", 64, "bf16", 1, 32768, 8, 128, 32768, start=0),
        # a selection of the cache as a query picked it
        _read("read_selected", "int8", 64, "bf16", 4, 2048, 8, 128, 32768),
        # a prompt's cache brought back, for a step that takes plain keys and values
        _read("read_prompt_32k", "e4m3", 64, "bf16", 1, 32000, 8, 128, 32768, start=640),
        # the smallest decode step: one short sequence, fp32, a head of 64
        _attn("decode_tiny_f32", "int8", 32, "f32", 1, 1, 4, 4, 64, 2048, 2047, 16, 256, 128),
        # the decode batch: 16 sequences of 128K tokens, one list of 2048 selected tokens each
        _attn("decode_b16_128k", "e4m3", 64, "bf16", 16, 1, 32, 8, 128, 131072, 131071, 128, 4096, 2048),
        # the same with sequences of 8K to 128K tokens
        _attn("decode_varlen_b16", "int8", 64, "bf16", 16, 1, 32, 8, 128, 131072, -1, 128, 4096, 2048),
        # a list for every key/value head
        _attn("decode_heads_b16", "e4m3", 128, "bf16", 16, 1, 32, 8, 128, 131072, 131071, 128, 4096, 2048, heads=True),
        # few long sequences: offsets past 32 bits
        _attn("decode_b4_1m", "e4m3", 64, "bf16", 4, 1, 32, 8, 128, 1048576, 1048575, 128, 4096, 2048),
        # a few drafted tokens checked at once, at an odd position
        _attn("verify_5_b3", "int8", 16, "bf16", 3, 5, 32, 8, 128, 16384, 12345, 128, 4096, 2048),
        # a chunk of 512 queries of a 32K prefill
        _attn("chunk_512_32k", "e4m3", 64, "bf16", 1, 512, 32, 8, 128, 32768, 32256, 128, 4096, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    fmt, block = rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128, 128])
    op = rng.choice(["write", "read", "attn", "attn"])
    if op == "attn":
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        batch = _log(rng, 1, 24)
        lq = 1 if rng.random() < 0.6 else _log(rng, 2, 300 // batch + 2)
        n_cap = block * max(1, _log(rng, 600, 60000) // block)
        n_init, window, topk = rng.choice([0, 16, 128]), _log(rng, 64, 4096), _log(rng, 16, 2048)
        lq = min(lq, n_cap)
        c0 = -1 if lq == 1 and rng.random() < 0.4 else rng.randint((n_cap - lq) // 2, n_cap - lq)
        return {k: v for k, v in _attn("", fmt, block, dtype, batch, lq, hq, hkv, dim, n_cap, c0, n_init, window,
                                       topk, heads=rng.random() < 0.3).items() if k != "name"}
    hkv = rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    batch = _log(rng, 1, 32)
    rows = 1 if rng.random() < 0.3 else _log(rng, 2, 8192 // batch + 2)
    n_cap = block * (rows // block + 2 + _log(rng, 1, 4096 // block))
    start = -1 if rng.random() < 0.4 else rng.randint(0, n_cap - rows)
    make = _write("", fmt, block, dtype, batch, rows, hkv, dim, n_cap, start, rng.random() < 0.5) if op == "write" \
        else _read("", fmt, block, dtype, batch, rows, hkv, dim, n_cap, start)
    return {k: v for k, v in make.items() if k != "name"}


def _lengths(c):
    """Tokens that each sequence holds after the call, spread over the cache."""
    if c["op"] == "write":
        lo = c["rows"]
    else:
        lo = max(1, c["n_cap"] // 16)
    return [lo + int((c["n_cap"] - lo) * ((0.9 + 0.6180339887 * b) % 1.0)) for b in range(c["batch"])]


def _region(c, c0):
    lo = min(c0, max(c["n_init"], c0 - c["window"]))
    return lo, min(c["n_init"], lo), max(0, lo - c["n_init"])


# ----------------------------------------------------------------------- prepare --
def _normal(gen, shape, loud):
    """Keys or values of a layer: unit normal, a few louder channels in each head."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    if loud is not None:
        x *= loud
    return x


def _scale_of(amax, fmt):
    """The smallest power of two s with amax <= QMAX * s (2^LEAST at least)."""
    m, e = torch.frexp(amax)
    top, at = (0.875, 9) if fmt == "e4m3" else (127.0 / 128.0, 7)
    e = (e - at + (m > top).to(e.dtype)).clamp(min=LEAST)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, LEAST)))


def _code(y, fmt):
    return y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)


def _at(codes, *where):
    return codes.view(torch.uint8)[where].view(codes.dtype)


def _filled(gen, c, loud):
    """A whole cache of one operand: codes and scales, written block by block."""
    b, n, h, d, block, fmt = c["batch"], c["n_cap"], c["hkv"], c["dim"], c["block"], c["fmt"]
    codes = torch.empty((b, n, h, d), dtype=CODE[fmt], device=DEV)
    scale = torch.empty((b, n // block, h), dtype=torch.float32, device=DEV)
    step = max(block, (1 << 25) // (h * d) // block * block)
    for s in range(b):
        for r in range(0, n, step):
            e = min(n, r + step)
            x = _normal(gen, ((e - r) // block, block, h, d), loud)
            sc = _scale_of(x.abs().amax(dim=(1, 3)), fmt)
            scale[s, r // block:e // block] = sc
            codes[s, r:e] = _code(x / sc[:, None, :, None], fmt).view(e - r, h, d)
    return codes, scale


def _picked(gen, batch, lists, n, first, count, top):
    """`count` positions of [first, first + n) for each list, ascending, -1 behind them."""
    idx = torch.full((batch, lists, top), -1, dtype=torch.int32, device=DEV)
    for b in range(batch):
        k = count[b]
        if k:
            keys = torch.rand((lists, n[b]), generator=gen, device=DEV)
            idx[b, :, :k] = (keys.topk(k, dim=1).indices.sort(dim=1).values + first).to(torch.int32)
    return idx


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    h, d, real = c["hkv"], c["dim"], REAL[c["dtype"]]
    loud = 1.0 + 3.0 * (torch.rand((h, d), generator=gen, device=DEV) < 0.05).float()
    kc, ks = _filled(gen, c, loud)
    vc, vs = _filled(gen, c, None)
    s = {"case": c, "k": kc, "ks": ks, "v": vc, "vs": vs}
    b, n = c["batch"], c["n_cap"]
    if c["op"] == "write":
        t, w = c["rows"], h * d
        if c["fused"]:      # the key and value columns of rows that hold queries too
            x = torch.cat([_normal(gen, (b, t, h, d), None).view(b, t, w), _normal(gen, (b, t, h, d), loud).view(b, t, w),
                           _normal(gen, (b, t, h, d), None).view(b, t, w)], dim=2).to(real)
            s["new_k"], s["new_v"] = x[..., w:2 * w].unflatten(2, (h, d)), x[..., 2 * w:].unflatten(2, (h, d))
        else:
            s["new_k"], s["new_v"] = (_normal(gen, (b, t, h, d), y).to(real) for y in (loud, None))
        ends = _lengths(c) if c["start"] < 0 else [c["start"] + t] * b
        s["len"] = torch.tensor(ends, dtype=torch.int64, device=DEV)
        # what is read back: the rows of every block that the write touches, up to its end
        base = [(e - t) // c["block"] * c["block"] for e in ends]
        most = max(e - a for e, a in zip(ends, base))
        pos = torch.tensor(base, device=DEV)[:, None] + torch.arange(most, device=DEV)
        s["idx"] = torch.where(pos < s["len"][:, None], pos, -1).to(torch.int32)
    elif c["op"] == "read":
        if c["start"] < 0:
            s["idx"] = _picked(gen, b, 1, [n] * b, 0, [c["rows"]] * b, c["rows"])[:, 0].contiguous()
    else:
        lens = _lengths(c) if c["c0"] < 0 else [c["c0"] + 1] * b
        n_mid = [_region(c, x - 1)[2] for x in lens]
        lists = h if c["heads"] else 1
        count = [min(c["topk"], m) for m in n_mid]
        s["q"] = _normal(gen, (b, c["lq"], c["hq"], d), None).to(real)
        s["idx"] = _picked(gen, b, lists, n_mid, c["n_init"], count, c["topk"])
        s["count"] = torch.tensor(count, dtype=torch.int32, device=DEV)[:, None].expand(b, lists).contiguous()
        s["len"] = torch.tensor(lens, dtype=torch.int64, device=DEV)
    if own:
        import query_aware_selective_b200 as qas
        s["cache"] = qas.CacheQ8(kc, ks, vc, vs, c["block"])
        if c["op"] == "attn":
            s["p"] = qas.params(c["n_init"], c["window"], c["topk"], 0)
    return s


# --------------------------------------------------------------------- plain form --
def _plain_write(codes, scale, new, end, c):
    """Quantise rows `new` [B, T, H, D] into positions [end - T, end) of codes and scale."""
    b, t = new.shape[:2]
    block, fmt, h, d = c["block"], c["fmt"], c["hkv"], c["dim"]
    nb = min((t + block - 2) // block + 1, scale.shape[1])
    start = end - t
    first = (start // block).clamp(max=scale.shape[1] - nb)                       # first block of the window
    blk = first[:, None] + torch.arange(nb, device=DEV)                           # [B, nb]
    pos = first[:, None] * block + torch.arange(nb * block, device=DEV)           # [B, nb * block]
    rows = torch.arange(b, device=DEV)[:, None]
    fresh = ((pos >= start[:, None]) & (pos < end[:, None]))[..., None, None]
    before = ((pos < start[:, None]) & (pos // block == (start // block)[:, None]))[..., None, None]
    x_new = torch.where(fresh, new[rows, (pos - start[:, None]).clamp(0, t - 1)].float(), 0.0)
    old_codes, old_scale = _at(codes, rows, pos), scale[rows, blk]
    amax = x_new.abs().unflatten(1, (nb, block)).amax(dim=(2, 4))                 # [B, nb, H]
    touched = fresh.unflatten(1, (nb, block)).any(dim=2)[..., 0]                  # [B, nb, 1]
    holds = before.unflatten(1, (nb, block)).any(dim=2)[..., 0]
    sc = torch.maximum(_scale_of(amax, fmt), torch.where(holds, old_scale, 0.0))
    sc = torch.where(touched, sc, old_scale)
    spread = lambda z: z.repeat_interleave(block, dim=1)[..., None]               # noqa: E731
    x = torch.where(fresh, x_new, old_codes.float() * spread(old_scale))
    got = _code(x / spread(sc), fmt)
    # untouched rows keep their codes, bit for bit
    codes.view(torch.uint8)[rows, pos] = torch.where(fresh | before, got.view(torch.uint8), old_codes.view(torch.uint8))
    scale[rows, blk] = sc


def _plain_read(codes, scale, idx, block, real):
    """Rows idx [B, n] of the cache as values; a row of -1 gives zeros."""
    rows, pos = torch.arange(idx.shape[0], device=DEV)[:, None], idx.clamp(min=0).long()
    x = _at(codes, rows, pos).float() * scale[rows, pos // block][..., None]
    return torch.where((idx >= 0)[..., None, None], x, 0.0).to(real)


def _plain_attn(s):
    c = s["case"]
    b, lq, hq, h, d, block = c["batch"], c["lq"], c["hq"], c["hkv"], c["dim"], c["block"]
    lists = s["count"].shape[1]
    c0 = (s["len"] - 1)[:, None, None]                                            # the first query's position
    cnt = s["count"][..., None].long()
    lo = torch.minimum(c0, (c0 - c["window"]).clamp(min=c["n_init"]))
    ni = lo.clamp(max=c["n_init"])
    most = c["n_init"] + c["topk"] + c["window"] + lq
    t = torch.arange(most, device=DEV)
    sel = s["idx"].long().gather(2, (t - ni).clamp(0, c["topk"] - 1).expand(b, lists, most))
    pos = torch.where(t < ni, t.expand(b, lists, most), torch.where(t < ni + cnt, sel, lo + t - ni - cnt))
    keys = ni + cnt + c0 - lo + 1                                                 # that the first query attends
    seen = t < keys[..., None] + torch.arange(lq, device=DEV)[:, None]            # [B, L, Lq, T]
    pos = pos.clamp(0, c["n_cap"] - 1).expand(b, h, most)
    rows, head = torch.arange(b, device=DEV)[:, None, None], torch.arange(h, device=DEV)[:, None]
    k = _at(s["k"], rows, pos, head).float() * s["ks"][rows, pos // block, head][..., None]      # [B, H, T, D]
    v = _at(s["v"], rows, pos, head).float() * s["vs"][rows, pos // block, head][..., None]
    q = s["q"].float().view(b, lq, h, hq // h, d).permute(0, 2, 3, 1, 4)                    # [B, H, G, Lq, D]
    x = torch.matmul(q.reshape(b, h, -1, d), k.transpose(2, 3)).view(b, h, hq // h, lq, most) / math.sqrt(d)
    x = torch.where(seen[:, :, None], x, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    e = (x - top).exp()
    z = e.sum(dim=-1, keepdim=True)
    o = torch.matmul((e / z).view(b, h, -1, most), v).view(b, h, hq // h, lq, d)
    lse = (z.log() + top)[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d).to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b, lq, hq)


def run(state):
    s, c = state, state["case"]
    real = REAL[c["dtype"]]
    if own:
        import query_aware_selective_b200 as qas
        if c["op"] == "write":
            if c["start"] < 0:
                qas.cache_write_q8_varlen(s["cache"], s["new_k"], s["new_v"], s["len"])
            else:
                qas.cache_write_q8(s["cache"], s["new_k"], s["new_v"], c["start"])
            return qas.cache_read_q8(s["cache"], idx=s["idx"], dtype=real)
        if c["op"] == "read":
            if c["start"] < 0:
                return qas.cache_read_q8(s["cache"], idx=s["idx"], dtype=real)
            return qas.cache_read_q8(s["cache"], start=c["start"], rows=c["rows"], dtype=real)
        if c["c0"] < 0:
            return qas.sparse_attn_q8_varlen(s["q"], s["cache"], s["len"], s["idx"], s["count"], s["p"], want_lse=True)
        return qas.sparse_attn_q8(s["q"], s["cache"], c["c0"], s["idx"], s["count"], s["p"], want_lse=True)
    if c["op"] == "write":
        _plain_write(s["k"], s["ks"], s["new_k"], s["len"], c)
        _plain_write(s["v"], s["vs"], s["new_v"], s["len"], c)
        return (_plain_read(s["k"], s["ks"], s["idx"], c["block"], real),
                _plain_read(s["v"], s["vs"], s["idx"], c["block"], real))
    if c["op"] == "read":
        idx = s["idx"] if c["start"] < 0 else \
            torch.arange(c["start"], c["start"] + c["rows"], device=DEV, dtype=torch.int32).expand(c["batch"], c["rows"])
        return (_plain_read(s["k"], s["ks"], idx, c["block"], real),
                _plain_read(s["v"], s["vs"], idx, c["block"], real))
    return _plain_attn(s)


# ----------------------------------------------------------------------- in 64 bits --
def _near(y, fmt):
    """The representable value nearest to y (ties to even), y within the codes' range."""
    if fmt == "int8":
        return torch.round(y)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40)))
    e = e + (torch.exp2(e + 1) <= y.abs()).double() - (torch.exp2(e) > y.abs()).double() * (e > -40)
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(y / step) * step


def _exact_write(codes, scale, new, ends, c):
    """Dequantised rows of the blocks that the write touches, sequence by sequence."""
    block, fmt, t = c["block"], c["fmt"], c["rows"]
    out = []
    for b, end in enumerate(ends):
        start = end - t
        base = start // block * block
        blocks = []
        for r in range(base, end, block):
            a, e = max(r, start), min(end, r + block)
            x = new[b, a - start:e - start].double()
            need = x.abs().amax(dim=(0, 2)) / QMAX[fmt]
            power = torch.ceil(torch.log2(need.clamp(min=2.0 ** LEAST)) - 1e-9)
            power = power + (torch.exp2(power) < need).double()
            sc = torch.exp2(power.clamp(min=LEAST))
            part = []
            if a > r:
                was = scale[b, r // block].double()
                sc = torch.maximum(sc, was)
                part.append(_near(codes[b, r:a].double() * was[:, None] / sc[:, None], fmt) * sc[:, None])
            part.append(_near(x / sc[:, None], fmt) * sc[:, None])
            blocks += part
        out.append(torch.cat(blocks))
    most = max(x.shape[0] for x in out)
    return torch.stack([torch.cat([x, x.new_zeros((most - x.shape[0], *x.shape[1:]))]) for x in out])


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    block, b = c["block"], c["batch"]
    if c["op"] == "write":
        ends = _lengths(c) if c["start"] < 0 else [c["start"] + c["rows"]] * b
        return (_exact_write(s["k"], s["ks"], s["new_k"], ends, c), _exact_write(s["v"], s["vs"], s["new_v"], ends, c))

    def rows_of(x, sc, i, at):
        return _at(x, i, at).double() * sc[i, at // block].double()[..., None]

    if c["op"] == "read":
        at = [s["idx"][i].long() if c["start"] < 0 else torch.arange(c["start"], c["start"] + c["rows"], device=DEV)
              for i in range(b)]
        return tuple(torch.stack([rows_of(x, sc, i, at[i]) for i in range(b)])
                     for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    g = c["hq"] // c["hkv"]
    o = torch.zeros((b, c["lq"], c["hq"], c["dim"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, c["lq"], c["hq"]), dtype=torch.float64, device=DEV)
    lens = _lengths(c) if c["c0"] < 0 else [c["c0"] + 1] * b
    for i in range(b):
        c0 = lens[i] - 1
        lo, ni, n_mid = _region(c, c0)
        for h in range(c["hkv"]):
            picked = s["idx"][i, h if c["heads"] else 0, :min(c["topk"], n_mid)].long()
            at = torch.cat([torch.arange(ni, device=DEV), picked, torch.arange(lo, c0 + c["lq"], device=DEV)])
            k = _at(s["k"], i, at, h).double() * s["ks"][i, at // block, h].double()[:, None]
            v = _at(s["v"], i, at, h).double() * s["vs"][i, at // block, h].double()[:, None]
            q = s["q"][i, :, h * g:(h + 1) * g].double()
            x = torch.einsum("qgd,td->qgt", q, k) / math.sqrt(c["dim"])
            late = at[None, :] > c0 + torch.arange(c["lq"], device=DEV)[:, None]
            x = x.masked_fill(late[:, None, :], -math.inf)
            lse[i, :, h * g:(h + 1) * g] = torch.logsumexp(x, dim=-1)
            o[i, :, h * g:(h + 1) * g] = torch.einsum("qgt,td->qgd", torch.softmax(x, dim=-1), v)
    return o, lse


def work(case):
    c = case
    row = c["hkv"] * c["dim"]                       # codes of one token and operand
    real = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "write":
        ends = _lengths(c) if c["start"] < 0 else [c["start"] + c["rows"]] * c["batch"]
        back = sum(e - (e - c["rows"]) // c["block"] * c["block"] for e in ends)      # rows read back
        new = c["batch"] * c["rows"]
        blocks = sum((e - 1) // c["block"] - (e - c["rows"]) // c["block"] + 1 for e in ends)
        return {"bytes": 2 * (new * row * (real + 1) + back * row * real + (back - new) * row + blocks * c["hkv"] * 4),
                "flops": 2 * 3 * (new + back) * row}
    if c["op"] == "read":
        n = c["batch"] * c["rows"]
        return {"bytes": 2 * n * (row * (1 + real) + c["hkv"] * 4 // c["block"]) + (4 * n if c["start"] < 0 else 0),
                "flops": 2 * n * row}
    lens = _lengths(c) if c["c0"] < 0 else [c["c0"] + 1] * c["batch"]
    keys = pairs = listed_ = 0
    for x in lens:
        lo, ni, n_mid = _region(c, x - 1)
        first = ni + min(c["topk"], n_mid) + (x - 1 - lo) + 1
        keys += first + c["lq"] - 1
        pairs += first * c["lq"] + c["lq"] * (c["lq"] - 1) // 2
        listed_ += min(c["topk"], n_mid) * (c["hkv"] if c["heads"] else 1)
    q = c["batch"] * c["lq"] * c["hq"]
    return {"bytes": 2 * keys * row + 2 * q * c["dim"] * real + 4 * q + 4 * listed_,
            "flops": 4 * pairs * c["hq"] * c["dim"]}
