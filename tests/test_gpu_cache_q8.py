"""8-bit key/value cache on the GPU through the public calls: writing, reading back and
attending, against the oracle (oracle/cache_q8.py) and a plain attention in 64 bits.

Codes, scales and values read back are compared to the bit: the scales are powers of two,
so every step of the definition is exact but the one rounding to a code.

Attention tolerances, per output element (u(t) = finfo(t).eps / 2, half a step):
    |o - ref| <= u(out) |ref| + A (u(w) + 2 dx + 2^-19) + F max_j p_j sum_j |v_j|
A = sum_j p_j |v_j|, the size of what is summed; u(w) the relative rounding of the softmax
weights (2^-12 for three e4m3 pieces of 4 bits, 2^-11 for f16, 2^-8 for bf16 in a chunk,
2^-21 for the two f16 of fp32) and F the absolute one, in units of the largest weight, below
which a format has no more steps: int8 digits hold a weight as an integer whose largest is
2^27, so half a unit is 2^-28; the third e4m3 piece has subnormal steps of 2^-9 16^-2 under
a largest of 2^8, half of which is 2^-26; f16 has 2^-24 under a largest of 2^10 to 2^15,
half is 2^-35 at most, for two f16 too; bf16 none. dx the error
of a logit, (D + 8) 2^-24 max_j sum_d |q_d k_jd| scale for the fp32 sum of D exact products
and its three scalings, twice that for fp32 queries (split into 22 bits); 2^-19 for
the exponentials, the fp32 sums over a lane's keys and the final quotient. LSE: dx +
2^-19 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import query_aware_selective_b200 as qas
from oracle import cache_q8 as oc
from query_aware_selective_b200 import pipeline

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def _rand(shape, seed, dtype=torch.float32, spread=0.0):
    """Normal values; spread: log2 range of a factor per row, so that scales differ."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp2(spread * (torch.rand((*shape[:-1], 1), generator=g) - 0.5))
    return x.to(dtype)


def _numbers(codes):
    """Codes of the cache as the numbers they stand for (float64 on the host)."""
    return codes.cpu().double().numpy() if codes.dtype == torch.int8 else codes.cpu().float().double().numpy()


def _cache(b, n_cap, hkv, d, fmt, block, garbage=True):
    """A cache whose memory holds garbage: NaN codes (e4m3) and NaN scales."""
    c = qas.cache_q8(b, n_cap, hkv, d, DTYPE[fmt], block, device=DEV)
    if garbage:
        c.k.view(torch.uint8).fill_(0x7f)
        c.v.view(torch.uint8).fill_(0xff)
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    return c


class _Oracle:
    """The oracle's side of a cache: both operands of every sequence, and which rows count."""

    def __init__(self, b, n_cap, hkv, d, fmt, block):
        nblk = (n_cap + block - 1) // block
        self.fmt, self.block = fmt, block
        self.codes = np.zeros((2, b, n_cap, hkv, d))
        self.scale = np.zeros((2, b, nblk, hkv))
        self.len = [0] * b

    def write(self, b, k, v, start):
        for op, x in enumerate((k, v)):
            oc.write(self.codes[op, b], self.scale[op, b], x.double().numpy(), start, self.block, self.fmt)
        self.len[b] = start + k.shape[0]

    def check(self, cache):
        qas.device_status()
        for op, (codes, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
            codes, scale = _numbers(codes), scale.cpu().double().numpy()
            for b, n in enumerate(self.len):
                nb = (n + self.block - 1) // self.block
                assert np.array_equal(scale[b, :nb], self.scale[op, b, :nb])
                assert np.array_equal(codes[b, :n], self.codes[op, b, :n])
                assert np.isnan(scale[b, nb:]).all(), "a scale behind the sequence was touched"
        for codes, byte in ((cache.k, 0x7f), (cache.v, 0xff)):
            for b, n in enumerate(self.len):
                assert (codes[b, n:].view(torch.uint8) == byte).all(), "a row behind the sequence was touched"


# -------------------------------------------------------------------- write and read --
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dtype,d,hkv,b,sizes", [
    (16, torch.bfloat16, 128, 8, 2, [1, 1, 14, 1, 33, 7, 128]),     # token by token, odd, across blocks
    (32, torch.float32, 64, 3, 1, [5, 27, 1, 64, 31, 100]),
    (64, torch.bfloat16, 128, 1, 3, [63, 1, 1, 130, 61]),
    (128, torch.bfloat16, 64, 5, 1, [127, 2, 300]),
    (128, torch.float32, 128, 2, 2, [1, 128, 129]),
    (16, torch.float32, 64, 1, 1, [1, 2, 3, 4, 5, 6]),
])
def test_write_to_the_bit(fmt, block, dtype, d, hkv, b, sizes):
    n_cap = sum(sizes) + 11                        # not a multiple of the block
    cache, want = _cache(b, n_cap, hkv, d, fmt, block), _Oracle(b, n_cap, hkv, d, fmt, block)
    start = 0
    for i, t in enumerate(sizes):
        k = _rand((b, t, hkv, d), 11 + i, dtype, spread=2.0 * i)      # later rows may be louder
        v = _rand((b, t, hkv, d), 91 + i, dtype, spread=6.0)
        qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), start)
        for s in range(b):
            want.write(s, k[s], v[s], start)
        want.check(cache)
        start += t
    # back behind the end of an earlier write (rejected tokens): later rows count as empty
    back = sum(sizes[:-1]) - 1
    k, v = (_rand((b, 2, hkv, d), s, dtype) for s in (7, 8))
    qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), back)
    for s in range(b):
        want.write(s, k[s], v[s], back)
    got = qas.cache_read_q8(cache, 0, back + 2, dtype=torch.float32)
    for op in range(2):
        for s in range(b):
            ref = oc.read(want.codes[op, s], want.scale[op, s], range(back + 2), block)
            assert np.array_equal(got[op][s].cpu().double().numpy(), ref)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_range_of_magnitudes(fmt):
    # zeros, values under the smallest scale, subnormal and huge values, ties, per (block, head)
    b, t, hkv, d, block = 1, 96, 4, 64, 32
    x = _rand((b, t, hkv, d), 5, torch.float32)
    x[:, :32, 0] = 0.0
    x[:, :32, 1] *= 2.0 ** -120
    x[:, :32, 2] *= 2.0 ** -140
    x[:, :32, 3] *= 2.0 ** 125
    x[:, 32:64, 0] = torch.arange(64) / 4.0         # ties at the int8 step
    x[:, 32:64, 1] = 448.0
    x[:, 32:64, 2] = 127.0
    x[:, 32:64, 3] = 448.0 * (1 + 2.0 ** -22)
    cache, want = _cache(b, t, hkv, d, fmt, block), _Oracle(b, t, hkv, d, fmt, block)
    qas.cache_write_q8(cache, x.to(DEV), (-x).to(DEV), 0)
    want.write(0, x[0], -x[0], 0)
    want.check(cache)
    xb = x.to(torch.bfloat16)
    qas.cache_write_q8(cache, xb.to(DEV), xb.to(DEV), 0)
    want.write(0, xb[0], xb[0], 0)
    want.check(cache)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_strided_rows(dtype):
    # keys and values as columns of rows that hold queries too, of every other sequence
    b, t, hq, hkv, d = 3, 45, 4, 2, 64
    x = _rand((2 * b, t, (hq + 2 * hkv) * d), 3, dtype).to(DEV)[::2]
    k = x[..., hq * d:(hq + hkv) * d].unflatten(2, (hkv, d))
    v = x[..., (hq + hkv) * d:].unflatten(2, (hkv, d))
    a, c = (_cache(b, 100, hkv, d, "e4m3", 16, garbage=False) for _ in range(2))
    qas.cache_write_q8(a, k, v, 9)
    qas.cache_write_q8(c, k.contiguous(), v.contiguous(), 9)
    for n in ("k", "v"):
        assert torch.equal(getattr(a, n).view(torch.uint8), getattr(c, n).view(torch.uint8))
        assert torch.equal(getattr(a, n + "_scale"), getattr(c, n + "_scale"))
    # one row for every sequence (a stride of 0)
    one = _rand((1, 1, hkv, d), 4, dtype).to(DEV)
    qas.cache_write_q8(a, one.expand(b, 1, hkv, d), one.expand(b, 1, hkv, d), 54)
    qas.cache_write_q8(c, one.repeat(b, 1, 1, 1), one.repeat(b, 1, 1, 1), 54)
    assert torch.equal(a.k.view(torch.uint8), c.k.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_varlen(fmt):
    b, n_cap, hkv, d, block, t = 5, 300, 2, 128, 64, 40
    cache, want = _cache(b, n_cap, hkv, d, fmt, block), _Oracle(b, n_cap, hkv, d, fmt, block)
    ends, new = [40, 40, 0, 7, 33], [40, 40, 0, 7, 33]
    for step in range(3):
        k, v = (_rand((b, t, hkv, d), 60 + 2 * step + i, torch.bfloat16, 4.0) for i in range(2))
        qas.cache_write_q8_varlen(cache, k.to(DEV), v.to(DEV), torch.tensor(ends, device=DEV),
                                  torch.tensor(new, device=DEV))
        for s in range(b):
            if new[s]:
                want.write(s, k[s, :new[s]], v[s, :new[s]], ends[s] - new[s])
        want.check(cache)
        new = [1, 0, 40, 25, 31 + step]
        ends = [e + n for e, n in zip(ends, new)]
    # without new_len: every sequence gets all T rows
    k, v = (_rand((b, 1, hkv, d), 80 + i, torch.bfloat16) for i in range(2))
    ends = [n + 1 for n in want.len]
    qas.cache_write_q8_varlen(cache, k.to(DEV), v.to(DEV), torch.tensor(ends, device=DEV))
    for s in range(b):
        want.write(s, k[s], v[s], ends[s] - 1)
    want.check(cache)


def test_write_varlen_lengths_that_do_not_fit():
    b, n_cap, t = 4, 64, 8
    cache = _cache(b, n_cap, 1, 64, "int8", 16)
    k = _rand((b, t, 1, 64), 1, torch.bfloat16).to(DEV)
    for ends, new in (([65, 8, 8, 8], [8, 8, 8, 8]), ([8, 7, 8, 8], [8, 8, 8, 8]), ([8, 8, 20, 8], [8, 8, 9, 8]),
                      ([8, 8, 8, 8], [8, 8, 8, -1])):
        qas.cache_write_q8_varlen(cache, k, k, torch.tensor(ends, device=DEV), torch.tensor(new, device=DEV))
        with pytest.raises(qas.EsaError, match="length"):
            qas.device_status()
        bad = next(i for i, (e, n) in enumerate(zip(ends, new)) if e > n_cap or e < n or n > t or n < 0)
        assert (cache.k[bad].view(torch.uint8) == 0x7f).all() and cache.k_scale[bad].isnan().all()
        assert cache.k_scale[(bad + 1) % b, 0].isfinite().all()
        cache = _cache(b, n_cap, 1, 64, "int8", 16)
    # nothing new: any seq_len is fine, nothing is recorded
    qas.cache_write_q8_varlen(cache, k, k, torch.tensor([0, -5, 99, 8], device=DEV),
                              torch.tensor([0, 0, 0, 8], device=DEV))
    qas.device_status()
    assert cache.k_scale[:3].isnan().all() and cache.k_scale[3, 0].isfinite().all()


def test_a_write_that_does_not_fit_is_reported_as_one():
    """Not as a length that was clamped: nothing of the sequence was written."""
    cache = _cache(2, 64, 1, 64, "int8", 16)
    k = _rand((2, 8, 1, 64), 1, torch.bfloat16).to(DEV)
    good = torch.tensor([8, 8], device=DEV)
    for ends, new in (([65, 8], None), ([7, 8], None), ([8, 8], [9, 8]), ([8, 8], [-1, 8])):
        qas.cache_write_q8_varlen(cache, k, k, torch.tensor(ends, device=DEV),
                                  good if new is None else torch.tensor(new, device=DEV))
        with pytest.raises(qas.EsaError, match="left as it was") as e:
            qas.device_status()
        assert "clamped" not in str(e.value) and e.value.status == qas._abi.ESA_ERR_INVALID_ARG
        assert (cache.k[0].view(torch.uint8) == 0x7f).all() and cache.k_scale[0].isnan().all()
        qas.device_status()                        # reported once
    q = _rand((2, 1, 1, 64), 2, torch.bfloat16).to(DEV)
    cache = qas.cache_q8(2, 64, 1, 64, torch.int8, 16, device=DEV)
    zero = torch.zeros((2, 4), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    qas.sparse_attn_q8_varlen(q, cache, torch.tensor([65, 8], device=DEV), *zero, qas.params(4, 8, 4, 0))
    with pytest.raises(qas.EsaError, match="clamped"):
        qas.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_of_nan_and_infinity(fmt, dtype):
    x = _rand((1, 20, 2, 64), 2, dtype)
    bad = x.clone()
    bad[0, 3, 0, 5], bad[0, 4, 0, 6], bad[0, 5, 0, 7] = float("nan"), float("inf"), float("-inf")
    cache, clean = _cache(1, 32, 2, 64, fmt, 16), _cache(1, 32, 2, 64, fmt, 16)
    qas.cache_write_q8(cache, bad.to(DEV), x.to(DEV), 0)
    with pytest.raises(qas.EsaError, match="NaN or infinite"):
        qas.device_status()
    y = x.clone()
    y[0, 3, 0, 5] = y[0, 4, 0, 6] = y[0, 5, 0, 7] = 0.0
    qas.cache_write_q8(clean, y.to(DEV), x.to(DEV), 0)
    qas.device_status()
    a, c = _numbers(cache.k)[0, :20], _numbers(clean.k)[0, :20]
    top = 448.0 if fmt == "e4m3" else 127.0
    assert a[3, 0, 5] == 0 and a[4, 0, 6] == top and a[5, 0, 7] == -top
    a[4, 0, 6] = a[5, 0, 7] = 0.0
    assert np.array_equal(a, c) and torch.equal(cache.k_scale.cpu()[:, :2], clean.k_scale.cpu()[:, :2])
    # a block of nothing else
    qas.cache_write_q8(cache, torch.full((1, 16, 2, 64), float("inf"), dtype=dtype, device=DEV), x[:, :16].to(DEV), 0)
    with pytest.raises(qas.EsaError):
        qas.device_status()
    assert (_numbers(cache.k)[0, :16] == top).all() and (cache.k_scale[0, 0].cpu() == 2.0 ** -100).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_of_infinity_beside_the_largest_numbers(fmt, dtype):
    """qmax times the scale of the type's largest number is past fp32."""
    big = torch.finfo(dtype).max
    x = torch.zeros((1, 16, 1, 64), dtype=dtype)
    x[0, 0, 0, :4] = torch.tensor([big, -big, float("inf"), float("-inf")])
    cache, clean = _cache(1, 16, 1, 64, fmt, 16), _cache(1, 16, 1, 64, fmt, 16)
    qas.cache_write_q8(cache, x.to(DEV), x.to(DEV), 0)
    with pytest.raises(qas.EsaError, match="NaN or infinite"):
        qas.device_status()
    y = x.nan_to_num(0.0, 0.0, 0.0)
    qas.cache_write_q8(clean, y.to(DEV), y.to(DEV), 0)
    qas.device_status()
    top = 448.0 if fmt == "e4m3" else 127.0
    assert torch.equal(cache.k_scale, clean.k_scale) and torch.equal(cache.v_scale, clean.v_scale)
    for got, want in ((cache.k, clean.k), (cache.v, clean.v)):
        got, want = _numbers(got), _numbers(want)
        assert got[0, 0, 0, 2] == top and got[0, 0, 0, 3] == -top
        want[0, 0, 0, 2:4] = top, -top
        assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,n_cap,hkv,d,block", [(2, 203, 3, 64, 16), (1, 130, 8, 128, 64), (3, 77, 1, 128, 32),
                                                 (1, 700, 5, 64, 128)])
def test_read_to_the_bit(fmt, dtype, b, n_cap, hkv, d, block):
    cache = _cache(b, n_cap, hkv, d, fmt, block)
    k, v = (_rand((b, n_cap, hkv, d), 21 + i, torch.float32, 10.0) for i in range(2))
    qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), 0)
    codes = [_numbers(cache.k), _numbers(cache.v)]
    scale = [cache.k_scale.cpu().double().numpy(), cache.v_scale.cpu().double().numpy()]

    def want(op, s, positions):
        return oc.read(codes[op][s], scale[op][s], positions, block)

    for start, rows in ((0, n_cap), (0, 1), (n_cap - 1, 1), (17, 41), (5, None), (9, 0)):
        got = qas.cache_read_q8(cache, start, rows, dtype=dtype)
        n = n_cap - start if rows is None else rows
        for op in range(2):
            assert got[op].dtype == dtype and got[op].shape == (b, n, hkv, d)
            for s in range(b):
                assert np.array_equal(got[op][s].cpu().double().numpy(), want(op, s, range(start, start + n)))
    # any order, repeats, padding and positions outside the cache
    g = torch.Generator().manual_seed(3)
    idx = torch.randint(0, n_cap, (b, 61), generator=g, dtype=torch.int32)
    idx[:, 3], idx[:, 4], idx[:, 5], idx[:, 7] = -1, n_cap, 2 ** 31 - 1, idx[:, 6]
    got = qas.cache_read_q8(cache, idx=idx.to(DEV), dtype=dtype)
    for op in range(2):
        for s in range(b):
            assert np.array_equal(got[op][s].cpu().double().numpy(), want(op, s, idx[s].tolist()))
    only = qas.cache_read_q8(cache, idx=idx.to(DEV), dtype=dtype, want_k=False)
    assert only[0] is None and torch.equal(only[1], got[1])
    out = torch.empty_like(got[0])
    assert qas.cache_read_q8(cache, idx=idx.to(DEV), dtype=dtype, k_out=out, want_v=False)[0] is out
    assert torch.equal(out, got[0])
    qas.device_status()


# -------------------------------------------------------------------------- attention --
def _region(c0, n_init, window):
    lo = min(c0, max(n_init, c0 - window))
    return lo, min(n_init, lo), max(0, lo - n_init)


def _lists(c0s, lists, n_init, window, topk, seed, short=True):
    """Selections from each sequence's own middle; counts differ between lists, one is 0."""
    gen = torch.Generator().manual_seed(seed)
    idx = torch.full((len(c0s), lists, topk), -1, dtype=torch.int32)
    cnt = torch.zeros((len(c0s), lists), dtype=torch.int32)
    for b, c0 in enumerate(c0s):
        n_mid = _region(c0, n_init, window)[2]
        for g in range(lists):
            c = max(0, min(topk, n_mid) - (13 * ((b + g) % 3) if short else 0))
            if short and (b + g) % 5 == 4:
                c = 0
            idx[b, g, :c] = (torch.randperm(n_mid, generator=gen)[:c].sort().values + n_init).to(torch.int32)
            cnt[b, g] = c
    return idx, cnt


def _reference(q, kv, vv, c0s, idx, cnt, n_init, window, scale=None):
    """o, lse, A = sum p |v|, X = max_j scale sum |q k| and max p sum |v| per (sequence, query,
    head); kv, vv [B, n_cap, Hkv, D] float64 values."""
    b, lq, hq, d = q.shape
    hkv = kv.shape[2]
    grp = hq // hkv
    scale = scale or d ** -0.5
    o, big, least = (np.zeros((b, lq, hq, d)) for _ in range(3))
    lse, xmax = np.zeros((b, lq, hq)), np.zeros((b, lq, hq))
    for s in range(b):
        lo, ni, _ = _region(c0s[s], n_init, window)
        for h in range(hkv):
            g = h if cnt.shape[1] > 1 else 0
            sel = idx[s, g, :int(cnt[s, g])].long().numpy()
            at = np.concatenate([np.arange(ni), sel, np.arange(lo, c0s[s] + lq)])
            k, v = kv[s, at, h], vv[s, at, h]
            hs = slice(h * grp, (h + 1) * grp)
            qq = q[s, :, hs].double().numpy()
            x = np.einsum("igd,td->igt", qq, k) * scale
            late = at[None, None, :] > (c0s[s] + np.arange(lq))[:, None, None]
            x = np.where(late, -np.inf, x)
            m = x.max(axis=-1, keepdims=True)
            e = np.exp(x - m)
            z = e.sum(axis=-1, keepdims=True)
            o[s, :, hs] = np.einsum("igt,td->igd", e / z, v)
            big[s, :, hs] = np.einsum("igt,td->igd", e / z, np.abs(v))
            least[s, :, hs] = np.einsum("igt,td->igd", np.where(late, 0.0, 1.0 / z), np.abs(v))
            lse[s, :, hs] = (m + np.log(z))[..., 0]
            ax = np.einsum("igd,td->igt", np.abs(qq), np.abs(k)) * scale
            xmax[s, :, hs] = np.where(late, 0, ax).max(axis=-1)
    return o, lse, big, xmax, least


def _check(o, lse, ref, dtype, d, chunk=False):
    qas.device_status()
    ref_o, ref_lse, big, xmax, least = ref
    u_out = torch.finfo(dtype).eps / 2
    u_w = 2.0 ** -21 if dtype == torch.float32 else (2.0 ** -8 if chunk else 2.0 ** -11)
    dx = xmax * (d + 8) * 2.0 ** -24 * (2 if dtype == torch.float32 else 1)
    got = o.cpu().double().numpy()
    assert np.isfinite(got).all()
    floor = 0.0 if chunk else 2.0 ** -26 if dtype == torch.bfloat16 and d == 128 else 2.0 ** -35
    bound = u_out * np.abs(ref_o) + big * (u_w + 2 * dx[..., None] + 2.0 ** -19) + floor * least
    worst = float((np.abs(got - ref_o) / np.maximum(bound, 1e-300)).max())
    assert worst <= 1.0, f"{worst} times the bound"
    if lse is not None:
        err = np.abs(lse.cpu().double().numpy() - ref_lse)
        assert (err <= dx + 2.0 ** -19 * (1 + np.abs(ref_lse))).all()


def _filled(b, n_cap, hkv, d, fmt, block, upto, seed, spread=4.0):
    """A cache written up to upto[b] rows, garbage behind them; and its values."""
    cache = _cache(b, n_cap, hkv, d, fmt, block)
    k, v = (_rand((b, n_cap, hkv, d), seed + i, torch.float32, spread) for i in range(2))
    t = max(upto)
    qas.cache_write_q8_varlen(cache, k[:, :t].to(DEV), v[:, :t].to(DEV), torch.tensor(upto, device=DEV),
                              torch.tensor(upto, device=DEV))
    kv, vv = (np.nan_to_num(x.cpu().double().numpy()) for x in qas.cache_read_q8(cache, dtype=torch.float32))
    return cache, kv, vv


CASES = [
    # b, lq, n_cap, hq, hkv, d, block, lists, n_init, window, topk
    (2, 1, 3000, 32, 8, 128, 64, 1, 128, 1024, 700),      # decode, 8 KV heads
    (3, 1, 2500, 32, 8, 128, 16, 8, 64, 512, 400),        # a list per KV head
    (1, 1, 2048, 4, 4, 64, 32, 1, 16, 256, 128),          # tiny
    (1, 1, 900, 12, 4, 128, 128, 4, 16, 100, 77),         # groups of 3
    (1, 1, 800, 16, 1, 64, 64, 1, 0, 64, 200),            # 16 heads on one: two row tiles of 8
    (2, 1, 700, 10, 2, 64, 16, 2, 5, 0, 60),              # groups of 5, no window
    (1, 1, 500, 7, 7, 128, 32, 7, 500, 64, 20),           # 7 heads; all tokens initial
    (2, 5, 1500, 32, 8, 128, 64, 1, 128, 512, 300),       # 20 rows: tiles of 16 and a part
    (1, 3, 1111, 24, 3, 64, 16, 3, 32, 200, 150),         # 8 heads a group, 3 queries
    (1, 37, 600, 4, 4, 64, 64, 1, 16, 128, 100),          # more queries than a tile
    (1, 4, 800, 8, 4, 128, 32, 4, 16, 128, 100),          # 8 rows
    (2, 3, 900, 20, 4, 128, 16, 1, 16, 256, 100),         # 15 rows
    (1, 1, 400, 40, 1, 128, 64, 1, 16, 64, 33),           # 40 heads on one: two tiles of 20
    (40, 1, 300, 8, 8, 64, 16, 1, 16, 64, 50),            # more sequences than fit at once
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,lq,n_cap,hq,hkv,d,block,lists,n_init,window,topk", CASES)
def test_attention_few_queries(fmt, dtype, b, lq, n_cap, hq, hkv, d, block, lists, n_init, window, topk):
    c0 = n_cap - lq - 7
    cache, kv, vv = _filled(b, n_cap, hkv, d, fmt, block, [c0 + lq] * b, 31)
    q = _rand((b, lq, hq, d), 41, dtype)
    idx, cnt = _lists([c0] * b, lists, n_init, window, topk, 51)
    p = qas.params(n_init, window, topk, 2, 10.0)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    _check(o, lse, _reference(q, kv, vv, [c0] * b, idx, cnt, n_init, window), dtype, d)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("chunk,b,lq,n_cap,hq,hkv,block,lists,n_init,window,topk", [
    (False, 1, 64, 1500, 8, 8, 64, 1, 32, 256, 300),             # G 1
    (False, 2, 100, 1200, 8, 2, 16, 2, 16, 200, 150),            # a list per head, ragged
    (False, 1, 33, 1300, 4, 2, 128, 1, 128, 512, 100),           # G 2
    (False, 1, 8, 700, 16, 2, 32, 1, 0, 0, 64),                  # G 8, no initial tokens, no window
    (False, 1, 300, 300, 4, 1, 64, 1, 16, 64, 32),               # the first chunk: nothing before it
    (True, 1, 450, 1500, 8, 8, 64, 1, 32, 256, 300),             # the same on the chunk form
    (True, 2, 230, 1200, 8, 2, 16, 2, 16, 200, 150),
    (True, 1, 900, 1300, 4, 2, 128, 1, 128, 512, 100),
    (True, 1, 230, 700, 16, 2, 32, 1, 0, 0, 64),
    (True, 1, 900, 900, 4, 1, 64, 1, 16, 64, 32),
])
def test_attention_chunk(fmt, chunk, b, lq, n_cap, hq, hkv, block, lists, n_init, window, topk):
    d = 128
    c0 = max(0, n_cap - lq - 3)
    cache, kv, vv = _filled(b, n_cap, hkv, d, fmt, block, [c0 + lq] * b, 131)
    q = _rand((b, lq, hq, d), 141, torch.bfloat16)
    idx, cnt = _lists([c0] * b, lists, n_init, window, topk, 151)
    p = qas.params(n_init, window, topk, 2, 10.0)
    assert (qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p) > 0) == chunk
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    _check(o, lse, _reference(q, kv, vv, [c0] * b, idx, cnt, n_init, window), torch.bfloat16, d, chunk=chunk)


@pytest.mark.parametrize("b,lq,d", [(19, 1, 128), (11, 13, 128), (38, 1, 64)])
def test_attention_more_units_than_run_at_once(b, lq, d):
    """Long lists of more (sequence, KV head)s than the SMs hold: clusters in several waves. The
    reference is formed on the GPU, in 64 bits."""
    n, hq, hkv, block = 6000, 16, 8, 64
    g = torch.Generator(device=DEV).manual_seed(7)
    parts = []
    for _ in range(2):
        parts.append(torch.randint(-127, 128, (b, n, hkv, d), generator=g, device=DEV, dtype=torch.int8))
        parts.append(torch.exp2(torch.randint(-9, -5, (b, -(-n // block), hkv), generator=g, device=DEV).float()))
    cache = qas.CacheQ8(*parts, block)
    q = torch.randn((b, lq, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    p = qas.params(0, n, 1, 0)
    idx, cnt = torch.zeros((b, 1), dtype=torch.int32, device=DEV), torch.zeros(b, dtype=torch.int32, device=DEV)
    assert qas._abi.sparse_attn_q8_workspace_size(b, lq, n - lq, hq, hkv, d, 1, p) == 0
    o, lse = qas.sparse_attn_q8(q, cache, n - lq, idx, cnt, p, want_lse=True)
    blk = torch.arange(n, device=DEV) // block
    late = torch.arange(n, device=DEV)[None, :] > n - lq + torch.arange(lq, device=DEV)[:, None]
    ref = [[] for _ in range(5)]
    for s in range(b):
        k, v = (parts[i][s].double() * parts[i + 1][s, blk].double()[..., None] for i in (0, 2))
        k, v = (t.permute(1, 0, 2).repeat_interleave(hq // hkv, dim=0) for t in (k, v))           # [Hq, n, D]
        qq = q[s].double().permute(1, 0, 2)                                                       # [Hq, Lq, D]
        x = (qq @ k.transpose(1, 2) * d ** -0.5).masked_fill(late, -float("inf"))
        w, big = x.softmax(dim=2), (qq.abs() @ k.abs().transpose(1, 2) * d ** -0.5).masked_fill(late, 0.0)
        least = (~late).double() @ v.abs() * w.amax(dim=2, keepdim=True)
        for at, t in zip(ref, (w @ v, x.logsumexp(dim=2), w @ v.abs(), big.amax(dim=2), least)):
            at.append(t.transpose(0, 1).cpu().numpy())
    _check(o, lse, [np.stack(t) for t in ref], torch.bfloat16, d)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("chunk,b,lq,n_cap,hq,hkv,d,block,lists,n_init,window,topk", [
    (True, 2, 210, 1100, 10, 2, 128, 32, 2, 16, 200, 150),       # G 5, gathered queries, a list per head, ragged
    (True, 1, 65, 1000, 56, 2, 128, 64, 1, 0, 130, 64),          # G 28
    (True, 3, 9, 700, 144, 2, 128, 16, 2, 32, 64, 40),           # G 72, tiles that end inside a query's heads
    (True, 1, 160, 1500, 32, 8, 64, 64, 1, 32, 256, 300),        # heads of 64: G 4
    (True, 2, 301, 1200, 8, 8, 64, 16, 8, 16, 200, 150),         # G 1, a list per head
    (True, 2, 90, 900, 28, 4, 64, 128, 4, 128, 100, 90),         # G 7: a head at a time, a list per KV head
    (True, 1, 400, 400, 24, 2, 64, 32, 1, 16, 64, 32),           # G 12: four heads at a time, the first chunk
    (True, 3, 33, 555, 160, 2, 64, 64, 2, 8, 31, 77),            # G 80: sixteen at a time
    (False, 2, 20, 800, 28, 4, 64, 128, 4, 128, 100, 90),        # the same shapes, too few rows of a head
])
def test_attention_chunk_any_group_and_heads_of_64(fmt, chunk, b, lq, n_cap, hq, hkv, d, block, lists, n_init, window,
                                                   topk):
    c0 = max(0, n_cap - lq - 3)
    cache, kv, vv = _filled(b, n_cap, hkv, d, fmt, block, [c0 + lq] * b, 133)
    q = _rand((b, lq, hq, d), 143, torch.bfloat16)
    idx, cnt = _lists([c0] * b, lists, n_init, window, topk, 153)
    p = qas.params(n_init, window, topk, 2, 10.0)
    assert (qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p) > 0) == chunk
    guard = torch.full((b * lq * hq * d + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True,
                                out=guard[128:-128].view(b, lq, hq, d))
    _check(o, lse, _reference(q, kv, vv, [c0] * b, idx, cnt, n_init, window), torch.bfloat16, d, chunk=chunk)
    assert (guard[:128] == 7).all() and (guard[-128:] == 7).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("b,hq,hkv,d,lists", [(80, 64, 1, 128, 1), (80, 64, 1, 64, 1), (25, 128, 1, 128, 1),
                                              (25, 192, 2, 128, 2), (14, 256, 1, 128, 1), (40, 128, 2, 64, 2)])
def test_attention_single_queries_of_many_heads_on_one(fmt, b, hq, hkv, d, lists):
    """One query a sequence, but so many rows a KV head that the call takes the chunk form."""
    n_cap, n_init, window, topk = 300, 16, 64, 50
    c0 = n_cap - 4
    cache, kv, vv = _filled(b, n_cap, hkv, d, fmt, 32, [c0 + 1] * b, 137)
    q = _rand((b, 1, hq, d), 147, torch.bfloat16)
    idx, cnt = _lists([c0] * b, lists, n_init, window, topk, 157)
    p = qas.params(n_init, window, topk, 2, 10.0)
    assert qas._abi.sparse_attn_q8_workspace_size(b, 1, c0, hq, hkv, d, 1, p) > 0
    guard = torch.full((b * hq * d + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True,
                                out=guard[128:-128].view(b, 1, hq, d))
    _check(o, lse, _reference(q, kv, vv, [c0] * b, idx, cnt, n_init, window), torch.bfloat16, d, chunk=True)
    assert (guard[:128] == 7).all() and (guard[-128:] == 7).all()


@pytest.mark.parametrize("hq,hkv,d,lq", [(10, 2, 128, 210), (28, 4, 64, 140)])
def test_attention_chunk_nan_and_infinity_stay_in_their_rows(hq, hkv, d, lq):
    """A query row with a NaN or an infinity, beside rows of another head and of another query."""
    n_cap = 600
    c0 = n_cap - lq
    cache, kv, vv = _filled(2, n_cap, hkv, d, "e4m3", 32, [n_cap] * 2, 135)
    q = _rand((2, lq, hq, d), 145, torch.bfloat16)
    bad = q.clone()
    bad[0, 3, 1, d - 1], bad[0, 7, 0, 0], bad[1, lq - 1, hq - 1, 5] = float("nan"), float("inf"), float("-inf")
    idx, cnt = _lists([c0] * 2, 1, 8, 64, 50, 155)
    p = qas.params(8, 64, 50, 0)
    assert qas._abi.sparse_attn_q8_workspace_size(2, lq, c0, hq, hkv, d, 1, p) > 0
    a = (c0, idx.to(DEV), cnt.to(DEV), p)
    clean, _ = qas.sparse_attn_q8(q.to(DEV), cache, *a)
    got, _ = qas.sparse_attn_q8(bad.to(DEV), cache, *a)
    qas.device_status()
    hit = torch.zeros((2, lq, hq), dtype=torch.bool)
    hit[0, 3, 1] = hit[0, 7, 0] = hit[1, lq - 1, hq - 1] = True
    assert got.cpu()[hit].isnan().all()
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lists", [1, 2])
@pytest.mark.parametrize("dtype,hq,d", [(torch.bfloat16, 8, 128), (torch.float32, 6, 64)])
def test_attention_varlen(fmt, lists, dtype, hq, d):
    n_cap, hkv, block, n_init, window, topk = 900, 2, 32, 32, 128, 100
    lens = [900, 1, 2, 32, 33, 161, 162, 512, 899, 17]
    b = len(lens)
    cache, kv, vv = _filled(b, n_cap, hkv, d, fmt, block, lens, 231)
    q = _rand((b, 1, hq, d), 241, dtype)
    c0s = [n - 1 for n in lens]
    idx, cnt = _lists(c0s, lists, n_init, window, topk, 251)
    p = qas.params(n_init, window, topk, 2, 10.0)
    seq_len = torch.tensor(lens, device=DEV)
    o, lse = qas.sparse_attn_q8_varlen(q.to(DEV), cache, seq_len, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    ref = _reference(q, kv, vv, c0s, idx, cnt, n_init, window)
    _check(o, lse, ref, dtype, d)
    # one list as [B, topk] and [B]
    if lists == 1:
        o2, _ = qas.sparse_attn_q8_varlen(q.to(DEV), cache, seq_len, idx[:, 0].contiguous().to(DEV),
                                          cnt[:, 0].contiguous().to(DEV), p)
        assert torch.equal(o, o2)
    # a length outside the cache is clamped and reported
    qas.sparse_attn_q8_varlen(q.to(DEV), cache, torch.tensor([901] + lens[1:], device=DEV), idx.to(DEV), cnt.to(DEV),
                              p)
    with pytest.raises(qas.EsaError, match="length"):
        qas.device_status()


def test_attention_is_the_same_every_time_and_with_any_split():
    # the list split over clusters and warps differently (batch 1, 3 and 60 of the same sequence)
    n_cap, hq, hkv, d = 2000, 8, 2, 128
    cache, kv, vv = _filled(1, n_cap, hkv, d, "e4m3", 64, [n_cap], 331)
    q = _rand((1, 1, hq, d), 341, torch.bfloat16)
    idx, cnt = _lists([n_cap - 1], 1, 64, 512, 600, 351, short=False)
    p = qas.params(64, 512, 600, 2)
    ref = _reference(q, kv, vv, [n_cap - 1], idx, cnt, 64, 512)
    for b in (1, 3, 60):
        many = qas.CacheQ8(*(x.expand(b, *x.shape[1:]).contiguous() for x in
                             (cache.k, cache.k_scale, cache.v, cache.v_scale)), 64)
        args = (q.repeat(b, 1, 1, 1).to(DEV), many, n_cap - 1, idx.repeat(b, 1, 1).to(DEV), cnt.repeat(b, 1).to(DEV), p)
        o, lse = qas.sparse_attn_q8(*args, want_lse=True)
        for s in range(b):
            _check(o[s:s + 1], lse[s:s + 1], ref, torch.bfloat16, d)
            assert torch.equal(o[s], o[0])
        for _ in range(3):
            assert torch.equal(qas.sparse_attn_q8(*args)[0], o)


@pytest.mark.parametrize("lq", [1, 32, 230])
def test_attention_scale_out_and_foreign_scales(lq):
    # a softmax scale, outputs given, and a cache quantised elsewhere (scales amax / 127)
    b, n_cap, hq, hkv, d, block = 2, 400, 8, 2, 128, 32
    x = [_rand((b, n_cap, hkv, d), 400 + i, torch.float32, 3.0) for i in range(2)]
    parts = []
    for y in x:
        pad = torch.nn.functional.pad(y, (0, 0, 0, 0, 0, -n_cap % block)).unflatten(1, (-1, block))
        s = pad.abs().amax(dim=(2, 4)) / 127
        parts += [(pad / s[:, :, None, :, None]).round().to(torch.int8).flatten(1, 2)[:, :n_cap].contiguous(), s]
    cache = qas.CacheQ8(*(t.to(DEV) for t in parts), block)
    blk = np.arange(n_cap) // block
    kv, vv = (parts[i].double().numpy() * parts[i + 1].double().numpy()[:, blk][..., None] for i in (0, 2))
    c0 = n_cap - lq
    q = _rand((b, lq, hq, d), 441, torch.bfloat16)
    idx, cnt = _lists([c0] * b, 1, 16, 64, 100, 451)
    p = qas.params(16, 64, 100, 2)
    out = torch.full_like(q, float("nan"), device=DEV)
    lse = torch.full((b, lq, hq), float("nan"), device=DEV)
    got = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, scale=0.31, want_lse=True, out=out,
                             lse=lse)
    assert got[0] is out and got[1] is lse
    ref = _reference(q, kv, vv, [c0] * b, idx, cnt, 16, 64, scale=0.31)
    if lq < 230:
        _check(out, lse, ref, torch.bfloat16, d)
    else:
        # the staged bf16 values of such scales are rounded: keys add 2^-8 X to a logit, values 2^-8 A
        o, rl, big, xmax, _ = ref
        dx = xmax * (2.0 ** -8 + 136 * 2.0 ** -24)
        bound = 2.0 ** -8 * np.abs(o) + big * (2 * 2.0 ** -8 + 2 * dx[..., None] * np.exp(2 * dx[..., None]) + 2.0 ** -19)
        qas.device_status()
        assert (np.abs(out.cpu().double().numpy() - o) <= bound).all()
        assert (np.abs(lse.cpu().double().numpy() - rl) <= dx + 2.0 ** -19 * (1 + np.abs(rl))).all()


def test_attention_scales_far_apart():
    # blocks whose scales differ by 2^40: values and keys of one block dwarf the others'
    n_cap, hkv, d, block = 256, 1, 64, 16
    k, v = (_rand((1, n_cap, hkv, d), 500 + i, torch.float32) for i in range(2))
    v[:, 32:48] *= 2.0 ** 40
    v[:, 64:80] *= 2.0 ** -40
    k[:, 96:112] *= 2.0 ** -30
    q = _rand((1, 1, 4, d), 510, torch.float32)
    k[:, 32:48] = -20 * q[0, 0, 0]           # head 0 gives the loud values next to no weight
    cache = _cache(1, n_cap, hkv, d, "int8", block)
    qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), 0)
    kv, vv = (x.cpu().double().numpy() for x in qas.cache_read_q8(cache, dtype=torch.float32))
    idx, cnt = _lists([n_cap - 1], 1, 0, n_cap, 1, 1)
    p = qas.params(0, n_cap, 1, 0)
    for dtype in (torch.float32, torch.bfloat16):
        qd = q.to(dtype)
        o, lse = qas.sparse_attn_q8(qd.to(DEV), cache, n_cap - 1, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
        _check(o, lse, _reference(qd, kv, vv, [n_cap - 1], idx, cnt, 0, n_cap), dtype, d)


# What the kernels on the codes promise of a weight and of a query, by (dtype, head dim, format):
# u, the relative rounding of a weight: 2^-13 for three e4m3 pieces of 4 significant bits, 2^-17 for
#    four (up to 8 rows a KV head), none for int8 digits, 2^-11 for an f16, 2^-21 for two (fp32
#    queries);
# f, its absolute rounding in units of its tile's largest: 2^-26 (of the fourth piece 2^-30), 2^-28,
#    and 2^-35 for f16;
# e, the rounding of a query element in units of its row's largest: two e4m3 pieces end at steps
#    of 2^-9 16^-1 for a largest of 2^7 or more, so half of 2^-13 in 2^7: 2^-21; three digits
#    round to a whole number with a largest of 2^19 or more: 2^-20; an f16 has steps of 2^-24
#    for a largest of 2^13 or more: 2^-38, and no relative rounding of a bf16.
PROMISED = {(torch.bfloat16, 128, "e4m3"): (2.0 ** -13, 2.0 ** -26, 2.0 ** -21),
            (torch.bfloat16, 128, "int8"): (0.0, 2.0 ** -28, 2.0 ** -20),
            (torch.bfloat16, 64, "e4m3"): (2.0 ** -11, 2.0 ** -35, 2.0 ** -38),
            (torch.bfloat16, 64, "int8"): (2.0 ** -11, 2.0 ** -35, 2.0 ** -38),
            (torch.float32, 128, "e4m3"): (2.0 ** -21, 2.0 ** -35, 2.0 ** -38),
            (torch.float32, 64, "int8"): (2.0 ** -21, 2.0 ** -35, 2.0 ** -38)}


def _cancelling(b, hkv, d, group, dtype, fmt):
    """Four keys, all logits along dim 0 (for a query of 1 about -0.3, -2.7 and -5.5 under the
    first's), and values that cancel under the weights of each KV head's first query, each key
    finer than the one before. Returns q, k, v; the cache holds v as it is."""
    g = torch.Generator().manual_seed(17)
    n = 4
    k = torch.zeros((b, n, hkv, d))
    k[..., 0] = torch.tensor([0.0, -3.0, -30.0, -60.0])[None, :, None]
    q = torch.zeros((b, 1, group * hkv, d))
    q[..., 0] = (1.0 + torch.rand((b, 1, group * hkv), generator=g) / 4) * (d ** 0.5 / 11)
    q = q.to(dtype)
    unit = 0.5 if fmt == "e4m3" else 1.0                    # the scale of a block whose largest value is 120
    held = torch.from_numpy(oc.numbers(fmt)) * unit
    held = held[held <= 120]
    both = torch.cat([-held.flip(0), held])
    v = torch.zeros((b, n, hkv, d), dtype=torch.float64)
    some = held[held >= 60]
    v[:, 0] = some[torch.randint(len(some), (b, hkv, d), generator=g)]
    v[:, 0, :, 0] = 120.0
    x = torch.einsum("bnh,bh->bnh", k[..., 0].double(), q[:, 0, ::group, 0].double()) * d ** -0.5
    p = x.softmax(dim=1)
    rest = p[:, 0, :, None] * v[:, 0]
    for j in range(1, n):
        want = -rest / p[:, j, :, None]
        v[:, j] = both[(want[..., None] - both).abs().argmin(dim=-1)]
        rest = rest + p[:, j, :, None] * v[:, j]
    return q, k, v.float()


@pytest.mark.parametrize("group", [1, 6, 12])
@pytest.mark.parametrize("dtype,d,fmt", list(PROMISED))
def test_attention_weights_keep_their_bits(dtype, d, fmt, group):
    """What is left of an output dim is far below its values, and shows the rounding of single
    weights."""
    b, n, hkv = 16, 4, 2
    q, k, v = _cancelling(b, hkv, d, group, dtype, fmt)
    cache = qas.cache_q8(b, 16, hkv, d, DTYPE[fmt], 16, device=DEV)
    qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), 0)
    kv, vv = (y.cpu().double().numpy() for y in qas.cache_read_q8(cache, dtype=torch.float32))
    assert np.array_equal(kv[:, :n], k.double().numpy()) and np.array_equal(vv[:, :n], v.double().numpy())
    idx, cnt = torch.zeros((b, 1, 1), dtype=torch.int32), torch.zeros((b, 1), dtype=torch.int32)
    p = qas.params(0, n, 1, 0)
    o, _ = qas.sparse_attn_q8(q.to(DEV), cache, n - 1, idx.to(DEV), cnt.to(DEV), p)
    qas.device_status()
    ref_o, _, big, xmax, least = _reference(q, kv, vv, [n - 1] * b, idx, cnt, 0, n)
    u, f, e = PROMISED[dtype, d, fmt]
    if (dtype, d, fmt) == (torch.bfloat16, 128, "e4m3") and group <= 8:
        u, f = 2.0 ** -17, 2.0 ** -30
    dx = xmax[..., None] * (8 * 2.0 ** -24 + e)              # one product a logit, its scalings, the query's rounding
    bound = torch.finfo(dtype).eps / 2 * np.abs(ref_o) + big * (u + 2 * dx + 2.0 ** -19) + f * least
    # (of each KV head's first query the rounding of the output leaves room to see a weight's)
    assert np.median((bound / big)[:, :, ::group]) < 2.0 ** (-10 if u > 2.0 ** -14 else -14)
    worst = float((np.abs(o.cpu().double().numpy() - ref_o) / bound).max())
    assert worst <= 1.0, f"{worst} times the bound"


@pytest.mark.parametrize("more", [6, 10, 13, 16])
@pytest.mark.parametrize("dtype,d,fmt", list(PROMISED))
def test_attention_queries_with_a_loud_channel(dtype, d, fmt, more):
    """One channel of the queries 2^more above the others, where the keys hold nothing: the logits
    are ordinary, and of the other channels a query keeps what its format leaves."""
    n_cap, hq, hkv, lq = 400, 8, 2, 3
    k, v = (_rand((1, n_cap, hkv, d), 620 + i, torch.float32) for i in range(2))
    q = _rand((1, lq, hq, d), 630, torch.float32)
    q[..., 5] = 2.0 ** more * (1.0 + q[..., 5].abs() / 4) * q[..., 6].sign()
    k[..., 5] = 0.0
    q = q.to(dtype)
    cache = _cache(1, n_cap, hkv, d, fmt, 32)
    qas.cache_write_q8(cache, k.to(DEV), v.to(DEV), 0)
    kv, vv = (y.cpu().double().numpy() for y in qas.cache_read_q8(cache, dtype=torch.float32))
    c0 = n_cap - lq
    idx, cnt = _lists([c0], 1, 0, n_cap, 1, 1)
    p = qas.params(0, n_cap, 1, 0)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    qas.device_status()
    ref_o, ref_lse, big, xmax, least = _reference(q, kv, vv, [c0], idx, cnt, 0, n_cap)
    u, f, e = PROMISED[dtype, d, fmt]
    loud = q.double().abs().amax(dim=-1).numpy() * d ** -0.5 * float(np.abs(kv).sum(axis=-1).max())
    dx = xmax * (d + 8) * 2.0 ** -24 * (2 if dtype == torch.float32 else 1) + e * loud
    bound = torch.finfo(dtype).eps / 2 * np.abs(ref_o) + \
        big * (u + np.expm1(2 * dx[..., None]) + 2.0 ** -19) + f * least
    worst = float((np.abs(o.cpu().double().numpy() - ref_o) / bound).max())
    assert worst <= 1.0, f"{worst} times the bound"
    assert (np.abs(lse.cpu().double().numpy() - ref_lse) <= dx + 2.0 ** -19 * (1 + np.abs(ref_lse))).all()


@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** 14, 2.0 ** 60])
def test_attention_queries_of_any_range(factor):
    # queries outside f16's range against keys of the inverse one: the logits are ordinary
    n_cap, hq, hkv, d = 300, 4, 2, 128
    k, v = (_rand((1, n_cap, hkv, d), 600 + i, torch.float32) for i in range(2))
    cache = _cache(1, n_cap, hkv, d, "e4m3", 32)
    qas.cache_write_q8(cache, (k / factor).to(DEV), v.to(DEV), 0)
    kv, vv = (x.cpu().double().numpy() for x in qas.cache_read_q8(cache, dtype=torch.float32))
    idx, cnt = _lists([n_cap - 1], 1, 0, n_cap, 1, 1)
    p = qas.params(0, n_cap, 1, 0)
    for dtype in (torch.float32, torch.bfloat16):
        q = (_rand((1, 1, hq, d), 610, torch.float32) * factor).to(dtype)
        o, lse = qas.sparse_attn_q8(q.to(DEV), cache, n_cap - 1, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
        _check(o, lse, _reference(q, kv, vv, [n_cap - 1], idx, cnt, 0, n_cap), dtype, d)


def test_attention_index_list_outside_the_cache_is_clamped():
    n_cap, hq, hkv, d = 500, 4, 1, 64
    cache, kv, vv = _filled(1, n_cap, hkv, d, "e4m3", 16, [n_cap], 631)
    q = _rand((1, 1, hq, d), 641, torch.bfloat16)
    p = qas.params(8, 64, 4, 0)
    idx = torch.tensor([[-7, 100, 2 ** 31 - 1, 5000]], dtype=torch.int32)
    as_read = torch.tensor([[[0, 100, n_cap - 1, n_cap - 1]]], dtype=torch.int32)
    for count in (4, 2 ** 30, -3):
        cnt = torch.tensor([count], dtype=torch.int32)
        o, lse = qas.sparse_attn_q8(q.to(DEV), cache, n_cap - 1, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
        used = torch.tensor([[min(max(count, 0), 4)]], dtype=torch.int32)
        _check(o, lse, _reference(q, kv, vv, [n_cap - 1], as_read, used, 8, 64), torch.bfloat16, d)


@pytest.mark.parametrize("lq,hq,d", [(1, 8, 128), (2, 8, 64), (100, 8, 128), (230, 8, 128)])
def test_attention_list_longer_than_the_middle(lq, hq, d):
    """Entries that repeat: a list may hold up to topk of them however short the middle is (a
    second sequence follows the first one's, so that rows in its place would show)."""
    b, hkv, n_init, window, topk = 2, 2, 8, 32, 700
    c0 = 64
    cache, kv, vv = _filled(b, c0 + lq + 5, hkv, d, "e4m3", 16, [c0 + lq] * b, 651)
    q = _rand((b, lq, hq, d), 661, torch.bfloat16)
    gen = torch.Generator().manual_seed(671)
    idx = torch.randint(n_init, c0 - window, (b, 1, topk), generator=gen, dtype=torch.int32).sort(dim=2).values
    cnt = torch.tensor([[topk], [topk - 3]], dtype=torch.int32)
    p = qas.params(n_init, window, topk, 0)
    chunk = qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p) > 0
    assert chunk == (lq == 230)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    _check(o, lse, _reference(q, kv, vv, [c0] * b, idx, cnt, n_init, window), torch.bfloat16, d, chunk=chunk)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,d,lq", [(torch.bfloat16, 128, 1), (torch.bfloat16, 128, 3), (torch.bfloat16, 64, 3),
                                        (torch.float32, 128, 1), (torch.bfloat16, 128, 460)])
def test_attention_nan_and_infinity_stay_in_their_rows(fmt, dtype, d, lq):
    """A query row with a NaN or an infinity gives NaN there and nowhere else; so does the NaN
    scale of an attended block, in its head."""
    n_cap, hq, hkv, block = 900, 8, 2, 32
    c0 = n_cap - lq
    p = qas.params(16, 100, 40, 0)
    idx, cnt = _lists([c0], 1, 16, 100, 40, 661, short=False)
    args = (c0, idx.to(DEV), cnt.to(DEV), p)
    cache, _, _ = _filled(1, n_cap, hkv, d, fmt, block, [n_cap], 671)
    q = _rand((1, lq, hq, d), 681, dtype).to(DEV)
    good, good_lse = qas.sparse_attn_q8(q, cache, *args, want_lse=True)
    for i, h, value in ((0, 5, float("nan")), (lq - 1, 2, float("inf")), (0, 0, float("-inf"))):
        bad = q.clone()
        bad[0, i, h, 7] = value
        o, lse = qas.sparse_attn_q8(bad, cache, *args, want_lse=True)
        assert o[0, i, h].isnan().all() and lse[0, i, h].isnan()
        o[0, i, h], lse[0, i, h] = good[0, i, h], good_lse[0, i, h]
        assert torch.equal(o, good) and torch.equal(lse, good_lse)
    for scale in (cache.k_scale, cache.v_scale):
        was = scale[0, 0, 1].clone()               # the initial tokens of head 1: every query attends them
        scale[0, 0, 1] = float("nan")
        o, _ = qas.sparse_attn_q8(q, cache, *args)
        assert o[0, :, hq // 2:].isnan().all() and torch.equal(o[0, :, :hq // 2], good[0, :, :hq // 2])
        scale[0, 0, 1] = was
    qas.device_status()


def _loud_keys(layout, n, block):
    """Which of n tokens have loud values, the others zeros: whole tiles of 128 keys behind or
    ahead of quiet ones, tiles in turn, blocks inside a tile in turn, one token alone."""
    t = torch.arange(n)
    return {"behind": t >= n // 2, "ahead": t < n // 2, "tiles": t // 128 % 2 == 1, "blocks": t // block % 2 == 0,
            "one": t == n - 1, "first": t == 0}[layout]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("exponent", [27, 60, 97])
@pytest.mark.parametrize("dtype,d,lq", [(torch.bfloat16, 128, 1), (torch.bfloat16, 128, 5), (torch.float32, 128, 1),
                                        (torch.float32, 64, 3), (torch.bfloat16, 64, 1)])
def test_attention_zero_values_beside_loud_ones(fmt, exponent, dtype, d, lq):
    """A key whose values are zero (scale 2^-100) counts in the sum of the weights as much as one
    whose values are near the largest that is allowed, wherever the two lie."""
    n, block, group = 1024, 32, 4
    p = qas.params(0, n, 1, 0)
    for hkv in (1, 149):                            # a list split over a cluster, and one CTA a list
        k, v = (_rand((1, n, hkv, d), 520 + i, torch.float32) for i in range(2))
        v = v.clamp(-4, 4) * (100.0 if fmt == "e4m3" else 24.0) * 2.0 ** exponent
        q = _rand((1, lq, group * hkv, d), 530, dtype)
        idx, cnt = _lists([n - lq], 1, 0, n, 1, 1)
        for layout in ("behind", "ahead", "tiles", "blocks", "one", "first") if hkv == 1 else ("behind", "ahead", "blocks"):
            cache = _cache(1, n, hkv, d, fmt, block)
            x = torch.where(_loud_keys(layout, n, block)[None, :, None, None], v, 0.0)
            qas.cache_write_q8(cache, k.to(DEV), x.to(DEV), 0)
            s = cache.v_scale.cpu()
            assert 2.0 ** (exponent - 2) <= s.max() <= 2.0 ** exponent and s.min() == 2.0 ** -100
            kv, vv = (y.cpu().double().numpy() for y in qas.cache_read_q8(cache, dtype=torch.float32))
            o, lse = qas.sparse_attn_q8(q.to(DEV), cache, n - lq, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
            _check(o, lse, _reference(q, kv, vv, [n - lq], idx, cnt, 0, n), dtype, d)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128)])
def test_attention_nan_scale_of_a_block_that_a_query_does_not_attend(fmt, dtype, d):
    """Drafted tokens on both sides of a block's start: a NaN scale behind it is no matter of
    the queries ahead of it."""
    n, hkv, block, c0 = 320, 2, 32, 317 - 32         # queries at 285 .. 289: the last two in the block from 288
    cache, _, _ = _filled(1, n, hkv, d, fmt, block, [n], 541)
    q = _rand((1, 5, 8, d), 542, dtype).to(DEV)
    idx, cnt = _lists([c0], 1, 16, 64, 40, 543, short=False)
    args = (c0, idx.to(DEV), cnt.to(DEV), qas.params(16, 64, 40, 0))
    good, good_lse = qas.sparse_attn_q8(q, cache, *args, want_lse=True)
    for scale in (cache.k_scale, cache.v_scale):
        was = scale[0, 9, 1].clone()
        scale[0, 9, 1] = float("nan")
        o, lse = qas.sparse_attn_q8(q, cache, *args, want_lse=True)
        assert o[0, 3:, 4:].isnan().all() and lse[0, 3:, 4:].isnan().all()
        assert torch.equal(o[0, :3], good[0, :3]) and torch.equal(lse[0, :3], good_lse[0, :3])
        assert torch.equal(o[0, :, :4], good[0, :, :4])
        scale[0, 9, 1] = was
    qas.device_status()


def test_offsets_past_32_bits():
    # 3 sequences of 1M rows of 1 KB: the last ones lie past 2^31 bytes of each operand
    b, n_cap, hq, hkv, d, block = 3, 1 << 20, 32, 8, 128, 64
    cache = qas.cache_q8(b, n_cap, hkv, d, torch.float8_e4m3fn, block, device=DEV)
    n_init, window, topk = 16, 100, 50
    k, v = (_rand((b, 1, hkv, d), 700 + i, torch.bfloat16) for i in range(2))
    starts = [0, 511_111, n_cap - 200]
    for i, st in enumerate(starts):
        x, y = (_rand((b, 200, hkv, d), 710 + 2 * i + j, torch.bfloat16).to(DEV) for j in range(2))
        qas.cache_write_q8(cache, x, y, st)
    qas.cache_write_q8_varlen(cache, k.to(DEV), v.to(DEV), torch.full((b,), n_cap, device=DEV))
    at = torch.cat([torch.arange(s, s + 200) for s in starts]).to(torch.int32)
    values = qas.cache_read_q8(cache, idx=at.repeat(b, 1).to(DEV), dtype=torch.float32)
    back = qas.cache_read_q8(cache, start=n_cap - 200, rows=200, dtype=torch.float32)
    codes = [cache.k[:, n_cap - 200:], cache.v[:, n_cap - 200:]]
    for op in range(2):
        assert torch.equal(back[op], values[op][:, 400:])
        sc = (cache.k_scale, cache.v_scale)[op][:, torch.arange(n_cap - 200, n_cap, device=DEV) // block]
        assert torch.equal(back[op], codes[op].float() * sc[..., None])
    kv, vv = np.zeros((b, 600, hkv, d)), np.zeros((b, 600, hkv, d))
    for dst, src in ((kv, values[0]), (vv, values[1])):
        dst[:] = src.cpu().double().numpy()
    q = _rand((b, 1, hq, d), 720, torch.bfloat16)
    idx = torch.arange(511_111 + 60, 511_111 + 110, dtype=torch.int32).repeat(b, 1, 1)
    cnt = torch.full((b, 1), 50, dtype=torch.int32)
    p = qas.params(n_init, window, topk, 0)
    o, lse = qas.sparse_attn_q8(q.to(DEV), cache, n_cap - 1, idx.to(DEV), cnt.to(DEV), p, want_lse=True)
    # the same keys as a short list over the 600 rows read back
    keep = np.concatenate([np.arange(16), 200 + np.arange(60, 110), np.arange(400 + 99, 600)])
    zero = torch.zeros((b, 1, 1), dtype=torch.int32), torch.zeros((b, 1), dtype=torch.int32)
    n = len(keep)
    _check(o, lse, _reference(q, kv[:, keep], vv[:, keep], [n - 1] * b, *zero, 0, n), torch.bfloat16, d)


# ---------------------------------------------------------------- streams and graphs --
def _step_state(lens, n_cap=600, hq=8, hkv=2, d=128, block=64):
    b = len(lens)
    cache, _, _ = _filled(b, n_cap, hkv, d, "e4m3", block, [n - 1 for n in lens], 831)
    p = qas.params(32, 128, 64, 0)
    idx, cnt = _lists([n - 1 for n in lens], 1, 32, 128, 64, 851)
    return dict(cache=cache, p=p, idx=idx.to(DEV), cnt=cnt.to(DEV), seq_len=torch.tensor(lens, device=DEV),
                k=_rand((b, 1, hkv, d), 801, torch.bfloat16).to(DEV), v=_rand((b, 1, hkv, d), 802, torch.bfloat16).to(DEV),
                q=_rand((b, 1, hq, d), 803, torch.bfloat16).to(DEV), out=torch.empty((b, 1, hq, d), dtype=torch.bfloat16,
                                                                                    device=DEV))


def _step(s):
    """Write the new token, then attend: as a decode step uses the calls together."""
    qas.cache_write_q8_varlen(s["cache"], s["k"], s["v"], s["seq_len"])
    qas.sparse_attn_q8_varlen(s["q"], s["cache"], s["seq_len"], s["idx"], s["cnt"], s["p"], out=s["out"])
    return s["out"]


def test_write_and_attend_together_against_the_oracle():
    lens = [600, 333, 40, 1]
    s = _step_state([max(2, n) for n in lens])
    for _ in range(3):                              # the same step again: the write is idempotent
        _step(s)
    lens = s["seq_len"].tolist()
    kv, vv = (np.nan_to_num(x.cpu().double().numpy()) for x in qas.cache_read_q8(s["cache"], dtype=torch.float32))
    _check(s["out"], None, _reference(s["q"].cpu(), kv, vv, [n - 1 for n in lens], s["idx"].cpu(), s["cnt"].cpu(), 32,
                                      128), torch.bfloat16, 128)


def test_captured_step_replays_with_new_lengths():
    a, c = _step_state([300, 299]), _step_state([300, 299])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _step(a)
    _step(c)
    for i in range(4):
        for s in (a, c):
            s["seq_len"] += 1
            s["k"].mul_(1.5)
            s["q"].neg_()
        g.replay()
        _step(c)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], c["out"])
        assert torch.equal(a["cache"].k.view(torch.uint8), c["cache"].k.view(torch.uint8))
    qas.device_status()


def test_calls_by_torchs_public_entries(monkeypatch):
    """A torch without the private entries that the binding prefers: the same device and stream."""
    want = _step(_step_state([300, 299])).clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    seen = []
    monkeypatch.setattr(qas._abi, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(qas._abi, "_raw_stream",
                        lambda dev: seen.append(torch.cuda.current_stream(dev).cuda_stream) or seen[-1])
    s = _step_state([300, 299])
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = _step(s)
        assert torch.cuda.current_stream().cuda_stream == stream.cuda_stream == seen[-1]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_two_graphs_and_two_streams_at_once():
    states = [_step_state([300 + i, 200 + i]) for i in range(4)]
    want = [_step(_step_state([300 + i, 200 + i])).clone() for i in range(4)]
    torch.cuda.synchronize()
    graphs = []
    for s in states[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i].replay() if i < 2 else _step(states[i])
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert torch.equal(s["out"], w)
    qas.device_status()


def test_chunk_on_a_side_stream_and_in_a_graph():
    b, lq, n_cap, hq, hkv, d = 1, 450, 700, 8, 2, 128
    cache, kv, vv = _filled(b, n_cap, hkv, d, "int8", 32, [n_cap], 931)
    q = _rand((b, lq, hq, d), 941, torch.bfloat16)
    c0 = n_cap - lq
    idx, cnt = _lists([c0], 1, 16, 128, 100, 951)
    p = qas.params(16, 128, 100, 0)
    need = qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p)
    assert need > 0
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)       # NaN wherever it is not written
    out = torch.empty((b, lq, hq, d), dtype=torch.bfloat16, device=DEV)
    args = (q.to(DEV), cache, c0, idx.to(DEV), cnt.to(DEV), p)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qas.sparse_attn_q8(*args, out=out, workspace=ws)
    torch.cuda.synchronize()
    ref = _reference(q, kv, vv, [c0], idx, cnt, 16, 128)
    _check(out, None, ref, torch.bfloat16, d, chunk=True)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qas.sparse_attn_q8(*args, out=out, workspace=ws)
    out.zero_()
    ws.fill_(0xff)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


# ------------------------------------------------------------------------ the pipelines --
def _values(cache):
    return tuple(np.nan_to_num(x.cpu().double().numpy()) for x in qas.cache_read_q8(cache, dtype=torch.float32))


@pytest.mark.parametrize("fmt,per_head", [("e4m3", False), ("int8", True)])
def test_prefill_then_decode_over_one_cache(fmt, per_head):
    """A prefill that fills the cache chunk by chunk, then decode steps that go on with it:
    every output against the attention over the cache's own values and the selections made."""
    b, n, chunk, hq, hkv, d, dc, block = 1, 1000, 256, 16, 4, 128, 128, 32
    n_cap, n_init, window, topk = 1100, 64, 128, 200
    p = qas.params(n_init, window, topk, 2, 45.25)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((b, n_cap, h, d), generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv))
    if per_head:
        wq, wk = (pipeline.block_diagonal(torch.randn((hkv, hq // hkv * d, dc // hkv), generator=g) / 32)
                  for _ in range(2))
    else:
        wq, wk = (torch.randn((hq * d, dc), generator=g) / 32 for _ in range(2))
    wq, wk = wq.to(DEV), wk.to(DEV)
    cache = _cache(b, n_cap, hkv, d, fmt, block)
    pf = pipeline.EsaPrefill(b, n, chunk, hq, hkv, d, dc, p, per_head=per_head, cache=cache)
    plain = pipeline.EsaPrefill(b, n, chunk, hq, hkv, d, dc, p, per_head=per_head)
    qd, kd, vd = (x[:, :n].contiguous().to(DEV) for x in (q, k, v))
    out = pf.run(qd, kd, vd, wq, wk)
    ref_out = plain.run(qd, kd, vd, wq, wk)
    qas.device_status()
    assert torch.equal(pf.idx_all, plain.idx_all)                  # the selection does not see the cache
    # the chunks wrote what single writes of the same rows would have
    want = _Oracle(b, n_cap, hkv, d, fmt, block)
    for c0 in range(0, n, chunk):
        want.write(0, k[0, c0:min(n, c0 + chunk)], v[0, c0:min(n, c0 + chunk)], c0)
    want.check(cache)
    kv, vv = _values(cache)
    lists = hkv if per_head else 1
    for ci, (c0, lq) in enumerate(pf.chunks()):
        idx, cnt = pf.idx_all[ci].cpu().view(b, lists, topk), pf.count_all[ci].cpu().view(b, lists)
        ws = qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p)
        _check(out[:, c0:c0 + lq], None, _reference(q[:, c0:c0 + lq], kv, vv, [c0], idx, cnt, n_init, window),
               torch.bfloat16, d, chunk=ws > 0)
    # and stayed near the unquantised attention
    err = float((out.float() - ref_out.float()).norm() / ref_out.float().norm())
    assert err < (0.08 if fmt == "e4m3" else 0.03), err            # (2^-4 / 2^-7 a value at most, uncorrelated)

    dec = pipeline.EsaDecodeQ8(cache, hq, dc, p, per_head=per_head)
    dec.fill_cache(wk, [n + 1])
    seq_len = torch.tensor([n], device=DEV)
    for t in range(n, n + 5):
        seq_len += 1
        rows = [x[:, t].contiguous().to(DEV) for x in (k, v)]
        o = dec.step(q[:, t:t + 1].contiguous().to(DEV), *rows, wq, wk, seq_len)
        qas.device_status()
        want.write(0, k[0, t:t + 1], v[0, t:t + 1], t)
        want.check(cache)
        kv, vv = _values(cache)
        _check(o, None, _reference(q[:, t:t + 1], kv, vv, [t], dec.idx.cpu(), dec.count.cpu(), n_init, window),
               torch.bfloat16, d)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_compresses_a_row_as_given_or_as_held(fmt):
    """A step compresses the new key row as it is given, fill_cache the row as the cache holds it,
    with garbage in the rows behind a sequence."""
    b, n_cap, hq, hkv, d, dc = 3, 300, 8, 4, 128, 128
    lens = [40, 299, 130]
    g = torch.Generator().manual_seed(18)
    wq, wk = ((torch.randn((hq * d, dc), generator=g) / 32).to(DEV) for _ in range(2))
    k, v = (torch.randn((b, n_cap, hkv, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn((b, 1, hq, d), generator=g).to(torch.bfloat16).to(DEV)
    cache = _cache(b, n_cap, hkv, d, fmt, 32)
    n = torch.tensor(lens, device=DEV)
    qas.cache_write_q8_varlen(cache, k[:, :max(lens)], v[:, :max(lens)], n, n)
    dec = pipeline.EsaDecodeQ8(cache, hq, dc, qas.params(16, 64, 50, 2, 45.25))
    dec.fill_cache(wk, [x + 1 for x in lens])
    held = qas.cache_read_q8(cache)[0]
    for s, x in enumerate(lens):
        want = torch.empty((x, dc), device=DEV)
        dec.cmp.keys(held[s, :x], out=want)
        assert torch.equal(dec.k_c[s, :x], want) and not dec.k_c[s, x:].any()
    new = k[:, -1].contiguous()
    dec.step(q, new, v[:, -1].contiguous(), wq, wk, n + 1)
    want = torch.zeros_like(dec.k_c)
    qas.compress_packed_varlen(new, dec.cmp.wk_p, want, n + 1)
    qas.device_status()
    for s, x in enumerate(lens):
        assert torch.equal(dec.k_c[s, x], want[s, x]) and want[s, x].any()


def test_decode_step_in_a_graph_with_lengths_that_differ():
    b, n_cap, hq, hkv, d, dc = 3, 700, 8, 4, 128, 128
    p = qas.params(32, 64, 100, 2, 45.25)
    g = torch.Generator().manual_seed(6)
    lens = [650, 90, 300]
    wq, wk = ((torch.randn((hq * d, dc), generator=g) / 32).to(DEV) for _ in range(2))
    k, v = (torch.randn((b, n_cap, hkv, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))

    def make():
        cache = _cache(b, n_cap, hkv, d, "int8", 64)
        t = max(lens)
        n = torch.tensor(lens, device=DEV)
        qas.cache_write_q8_varlen(cache, k[:, :t], v[:, :t], n, n)
        dec = pipeline.EsaDecodeQ8(cache, hq, dc, p)
        dec.fill_cache(wk, [x + 1 for x in lens])
        return dec, n
    (a, na), (c, nc) = make(), make()
    q = torch.randn((b, 1, hq, d), generator=g).to(torch.bfloat16).to(DEV)
    kn, vn = (torch.randn((b, hkv, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    graph = pipeline.graph_of(lambda: a.step(q, kn, vn, wq, wk, na))       # (runs once: row len - 1 again)
    c.step(q, kn, vn, wq, wk, nc)
    for _ in range(4):
        for x in (na, nc):
            x += 1
        kn.neg_()
        q.mul_(1.25)
        graph.replay()
        c.step(q, kn, vn, wq, wk, nc)
        torch.cuda.synchronize()
        assert torch.equal(a.out, c.out)
        assert torch.equal(a.cache.k.view(torch.uint8), c.cache.k.view(torch.uint8))
        kv, vv = _values(c.cache)
        _check(c.out, None, _reference(q.cpu(), kv, vv, [int(x) - 1 for x in nc], c.idx.cpu(), c.count.cpu(), 32, 64),
               torch.bfloat16, d)


@pytest.mark.parametrize("dtype,hq,hkv,chunk", [(torch.bfloat16, 28, 4, 256), (torch.float32, 4, 4, 160)])
def test_prefill_over_a_cache_of_heads_of_64(dtype, hq, hkv, chunk):
    b, n, d, dc, n_init, window, topk = 2, 600, 64, 64, 32, 64, 90
    g = torch.Generator().manual_seed(15)
    q, k, v = (torch.randn((b, n, h, d), generator=g).to(dtype) for h in (hq, hkv, hkv))
    wq, wk = (torch.randn((hq * d, dc), generator=g).to(DEV) / 32 for _ in range(2))
    p = qas.params(n_init, window, topk, 2, 45.25)
    cache = _cache(b, n + 8, hkv, d, "e4m3", 16)
    pf = pipeline.EsaPrefill(b, n, chunk, hq, hkv, d, dc, p, dtype=dtype, cache=cache)
    out = pf.run(q.to(DEV), k.to(DEV), v.to(DEV), wq, wk)
    kv, vv = _values(cache)
    for ci, (c0, lq) in enumerate(pf.chunks()):
        idx, cnt = pf.idx_all[ci].cpu().view(b, 1, topk), pf.count_all[ci].cpu().view(b, 1)
        ws = qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, int(dtype == torch.bfloat16), p)
        assert (ws > 0) == (dtype == torch.bfloat16)
        _check(out[:, c0:c0 + lq], None, _reference(q[:, c0:c0 + lq], kv, vv, [c0] * b, idx, cnt, n_init, window), dtype,
               d, chunk=ws > 0)


def test_prefill_whose_last_chunk_is_one_row_of_many_heads():
    b, n, chunk, hq, hkv, d, dc, n_init, window, topk = 50, 65, 32, 64, 1, 128, 128, 4, 16, 12
    g = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn((b, n, h, d), generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv))
    wq, wk = (torch.randn((hq * d, dc), generator=g).to(DEV) / 64 for _ in range(2))
    p = qas.params(n_init, window, topk, 2, 45.25)
    cache = _cache(b, n, hkv, d, "int8", 16)
    pf = pipeline.EsaPrefill(b, n, chunk, hq, hkv, d, dc, p, cache=cache)
    assert [lq for _, lq in pf.chunks()][-1] == 1
    out = pf.run(q.to(DEV), k.to(DEV), v.to(DEV), wq, wk)
    kv, vv = _values(cache)
    for ci, (c0, lq) in enumerate(pf.chunks()):
        idx, cnt = pf.idx_all[ci].cpu().view(b, 1, topk), pf.count_all[ci].cpu().view(b, 1)
        assert qas._abi.sparse_attn_q8_workspace_size(b, lq, c0, hq, hkv, d, 1, p) > 0
        _check(out[:, c0:c0 + lq], None, _reference(q[:, c0:c0 + lq], kv, vv, [c0] * b, idx, cnt, n_init, window),
               torch.bfloat16, d, chunk=True)


def test_captured_behind_copies_and_joined_streams():
    """Each call as the first kernel behind a copy, a fill and the join of two streams: its inputs
    are those that the graph's nodes before it wrote."""
    b, n_cap, hq, hkv, d = 2, 300, 8, 2, 128
    p = qas.params(8, 64, 50, 0)
    q, k, v = (torch.randn((b, 3, h, d), device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv))
    seq_len = torch.tensor([150, 260], device=DEV)
    idx = torch.arange(8, 58, dtype=torch.int32, device=DEV).repeat(b, 1)
    cnt = torch.full((b,), 50, dtype=torch.int32, device=DEV)
    start, _, _ = _filled(b, n_cap, hkv, d, "e4m3", 32, [n_cap] * b, 971)
    work = qas.cache_q8(b, n_cap, hkv, d, torch.float8_e4m3fn, 32, device=DEV)
    qi, ki, vi, li = (torch.zeros_like(t) for t in (q, k, v, seq_len))

    def reset():
        for t, u in ((work.k, start.k), (work.v, start.v)):
            t.view(torch.uint8).copy_(u.view(torch.uint8))
        work.k_scale.copy_(start.k_scale)
        work.v_scale.copy_(start.v_scale)

    def step():
        ki.copy_(k)
        vi.copy_(v)
        li.copy_(seq_len)
        qas.cache_write_q8_varlen(work, ki, vi, li)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            qi.copy_(q)
        torch.cuda.current_stream().wait_stream(side)
        o, lse = qas.sparse_attn_q8_varlen(qi[:, :1].contiguous(), work, li, idx, cnt, p, want_lse=True)
        li.zero_()
        return o, lse, *qas.cache_read_q8(work, start=100, rows=170)
    side = torch.cuda.Stream()
    reset()
    want = [t.clone() for t in step()]
    for t in (qi, ki, vi, li):
        t.zero_()
    reset()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        reset()
        for t in (*got, qi, ki, vi, li):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    qas.device_status()
