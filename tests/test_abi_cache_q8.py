"""Host-side checks of the 8-bit cache calls that need no GPU: every bad argument is
refused before anything is launched, by the C ABI and by the binding."""
import ctypes
import itertools
import math
import os
import re
import subprocess
import sys

import pytest
import torch

import query_aware_selective_b200 as qas
from query_aware_selective_b200 import _abi
from query_aware_selective_b200 import build as qbuild

FAKE = 0x10000      # 256-byte aligned, never dereferenced on the refused paths
INVALID, UNSUPPORTED, WORKSPACE = _abi.ESA_ERR_INVALID_ARG, _abi.ESA_ERR_UNSUPPORTED, _abi.ESA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return _abi.load()


def cache(k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, n_cap=4096, batch=2, hkv=8, d=128, block=64, fmt=0):
    return _abi.EsaCacheQ8(k, ks, v, vs, n_cap, batch, hkv, d, block, fmt)


BAD_CACHES = [(dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(v=None), INVALID), (dict(vs=None), INVALID),
              (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 1), INVALID), (dict(ks=FAKE + 2), INVALID),
              (dict(n_cap=0), INVALID), (dict(n_cap=1 << 31), UNSUPPORTED), (dict(batch=0), INVALID),
              (dict(batch=65536), UNSUPPORTED), (dict(hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
              (dict(block=48), UNSUPPORTED), (dict(block=256), UNSUPPORTED), (dict(block=0), UNSUPPORTED),
              (dict(fmt=2), INVALID)]


def test_struct_layout():
    assert ctypes.sizeof(_abi.EsaCacheQ8) == 4 * 8 + 8 + 5 * 4 + 4
    assert [f[0] for f in _abi.EsaCacheQ8._fields_] == ["k", "k_scale", "v", "v_scale", "n_cap", "batch", "hkv",
                                                        "head_dim", "block", "format"]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(lib, bad, status):
    before = lib.esa_launch_count()
    c = cache(**bad)
    p = _abi.params(128, 512, 256, 2)
    assert lib.esa_cache_write_q8(FAKE, FAKE, 1, 8, 8192, 1024, 8192, 1024, c, 0, None) == status
    assert lib.esa_cache_write_q8_varlen(FAKE, FAKE, 1, 1, 1024, 1024, 1024, 1024, c, FAKE, None, None) == status
    assert lib.esa_cache_read_q8(c, 0, 8, None, FAKE, FAKE, 1, None) == status
    hq = 4 * max(1, c.hkv)
    assert lib.esa_sparse_attn_q8(FAKE, 1, c, 1, 1000, hq, FAKE, FAKE, 1, p, 0.0, FAKE, None, FAKE, 1 << 40,
                                  None) == status
    assert lib.esa_sparse_attn_q8_varlen(FAKE, 1, c, FAKE, hq, FAKE, FAKE, 1, p, 0.0, FAKE, None, None) == status
    assert lib.esa_launch_count() == before


def test_write_refusals(lib):
    before = lib.esa_launch_count()

    def w(k=FAKE, v=FAKE, dt=1, rows=8, kb=8192, kr=1024, vb=8192, vr=1024, start=0, **c):
        return lib.esa_cache_write_q8(k, v, dt, rows, kb, kr, vb, vr, cache(**c), start, None)
    assert w(k=None) == INVALID and w(v=None) == INVALID
    assert w(dt=2) == INVALID
    assert w(rows=-1) == INVALID and w(rows=4097) == INVALID
    assert w(start=-1) == INVALID and w(start=4089) == INVALID and w(start=2 ** 62) == INVALID
    assert w(k=FAKE + 8) == INVALID and w(v=FAKE + 8) == INVALID              # misaligned base
    assert w(kr=1028) == INVALID and w(vb=8196) == INVALID                    # misaligned rows
    assert w(dt=0, kr=1026) == INVALID
    assert w(kr=512) == INVALID and w(vr=0) == INVALID                        # rows would overlap
    assert w(kb=-8192) == INVALID
    assert w(rows=0, k=None) == _abi.ESA_OK                                   # nothing to write
    for shared in (dict(vs=2 * FAKE), dict(v=2 * FAKE)):                      # one buffer for keys and values
        c = cache(**shared)
        assert lib.esa_cache_write_q8(FAKE, FAKE, 1, 8, 8192, 1024, 8192, 1024, c, 0, None) == INVALID
        assert b"share a buffer" in lib.esa_last_error()
    f = lib.esa_cache_write_q8_varlen
    assert f(FAKE, FAKE, 1, 1, 1024, 1024, 1024, 1024, cache(), None, None, None) == INVALID
    assert lib.esa_launch_count() == before


def test_read_refusals(lib):
    before = lib.esa_launch_count()

    def r(start=0, rows=8, idx=None, k=FAKE, v=FAKE, dt=1):
        return lib.esa_cache_read_q8(cache(), start, rows, idx, k, v, dt, None)
    assert r(start=-1) == INVALID and r(start=4089) == INVALID and r(rows=-1) == INVALID
    assert r(rows=2 ** 62) == INVALID
    assert r(k=FAKE + 16) == INVALID and r(v=FAKE + 8) == INVALID
    assert r(dt=3) == INVALID
    assert r(rows=0) == _abi.ESA_OK and r(k=None, v=None) == _abi.ESA_OK
    assert lib.esa_launch_count() == before


def test_attention_refusals(lib):
    before = lib.esa_launch_count()
    good = _abi.params(128, 512, 256, 2)

    def a(q=FAKE, dt=1, lq=1, c0=1000, hq=32, idx=FAKE, count=FAKE, lists=1, p=good, scale=0.0, o=FAKE, ws=FAKE,
          nb=1 << 40, **c):
        return lib.esa_sparse_attn_q8(q, dt, cache(**c), lq, c0, hq, idx, count, lists, p, scale, o, None, ws, nb, None)
    assert a(q=None) == INVALID and a(o=None) == INVALID and a(idx=None) == INVALID and a(count=None) == INVALID
    assert a(q=FAKE + 8) == INVALID and a(o=FAKE + 8) == INVALID
    assert a(dt=2) == INVALID and a(lq=0) == INVALID
    assert a(c0=-1) == INVALID and a(c0=4096) == INVALID and a(lq=5, c0=4092) == INVALID
    assert a(hq=0) == INVALID and a(hq=30) == INVALID
    assert a(lists=2) == INVALID and a(lists=0) == INVALID
    assert a(scale=math.nan) == INVALID
    assert a(p=_abi.params(128, 512, 0, 2)) == INVALID and a(p=_abi.params(-1, 512, 4, 2)) == INVALID
    assert a(p=_abi.params(128, 512, 2 ** 31 - 1, 2)) == UNSUPPORTED
    assert a(lq=64, ws=None) == WORKSPACE and a(lq=64, nb=1024) == WORKSPACE and a(lq=64, ws=FAKE + 64) == WORKSPACE
    assert a(dt=0, lq=4000, c0=0, hq=8 * 300, n_cap=4096, d=64) == UNSUPPORTED   # 75000 row tiles of 16
    f = lib.esa_sparse_attn_q8_varlen
    assert f(FAKE, 1, cache(), None, 32, FAKE, FAKE, 1, good, 0.0, FAKE, None, None) == INVALID
    assert f(FAKE, 1, cache(), FAKE, 32, FAKE, FAKE, 3, good, 0.0, FAKE, None, None) == INVALID
    assert lib.esa_launch_count() == before


def test_workspace_is_for_chunks_only(lib):
    p = _abi.params(128, 4096, 2048, 2)
    size = _abi.sparse_attn_q8_workspace_size
    assert size(16, 1, 131071, 32, 8, 128, 1, p) == 0                         # decode
    assert size(1, 15, 32000, 32, 8, 128, 1, p) == 0                          # 60 rows
    assert size(1, 3, 32000, 256, 8, 128, 1, p) == 0                          # 96 rows of 8 heads: 32 units
    assert size(1, 512, 32000, 32, 8, 128, 0, p) == 0                         # fp32
    assert size(1, 16, 32000, 32, 8, 64, 1, p) == 0                           # head_dim 64: 64 rows, 32 units
    assert size(16, 16, 32000, 40, 8, 64, 1, p) == 0                          # a fifth of the heads at a time: 16 rows
    rows = 128 + 2048 + 4096 + 512                                            # 6784 = 53 * 128
    assert size(1, 512, 32000, 32, 8, 128, 1, p) == 2 * rows * 8 * 128 * 2
    assert size(1, 512, 32000, 40, 8, 128, 1, p) == 2 * rows * 8 * 128 * 2     # groups of 5
    assert size(1, 512, 32000, 32, 8, 64, 1, p) == 2 * rows * 8 * 64 * 2
    assert size(1, 512, 32000, 40, 8, 64, 1, p) == 2 * rows * 8 * 64 * 2
    assert size(1, 512, 0, 32, 8, 128, 1, p) == 2 * (2048 + 512) * 8 * 128 * 2   # a list may repeat tokens
    assert size(0, 512, 0, 32, 8, 128, 1, p) == 0


def test_binding_refuses_cpu_tensors():
    k = torch.zeros((1, 64, 2, 64), dtype=torch.int8)
    s = torch.zeros((1, 4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        qas.CacheQ8(k, s, k.clone(), s.clone(), 16)
    with pytest.raises(ValueError, match="CUDA"):
        qas.cache_q8(1, 64, 2, 64, device="cpu")


def test_kernels_set_up_under_their_producer_read_by_plain_loads():
    """The 8-bit cache's kernels start under the kernel before them and read what it wrote: no
    load of theirs takes the read-only path."""
    csrc = os.path.join(os.path.dirname(qbuild.__file__), "csrc")
    for name in ("cache_q8.cuh", "attn_q8.cuh", "attn_q8_tc.cuh", "keylist.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert "pdl_wait()" in code or name == "keylist.cuh"
        assert not re.search(r"__ldg|\.nc\b|ld_stream16|__restrict__", code), name


def _cpu_cache(b, n_cap, hkv, d):
    """A CacheQ8 on the host, for calls that are stopped before the library."""
    c = object.__new__(qas.CacheQ8)
    c._k = c._v = torch.zeros((b, n_cap, hkv, d), dtype=torch.int8)
    c._k_scale = c._v_scale = torch.zeros((b, n_cap // 16, hkv))
    c._c = _abi.EsaCacheQ8(FAKE, FAKE, FAKE, FAKE, n_cap, b, hkv, d, 16, 1)
    c._dev, c._shape = -1, (b, hkv, d)
    return c


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_binding_brings_the_workspace_that_a_call_asks_for(lib, monkeypatch, d, dtype):
    seen = {}
    monkeypatch.setattr(_abi, "_q8_call", lambda cache, where, *args: seen.update(ws=args[-2], size=args[-1]))
    p = _abi.params(16, 32, 24, 2)
    asked = set()
    for b, hkv, group, lq in itertools.product((1, 25, 64, 80), (1, 2, 8), (1, 5, 16, 24, 32, 33, 48, 49, 64, 128, 160),
                                               (1, 2, 5)):
        need = _abi.sparse_attn_q8_workspace_size(b, lq, 100, group * hkv, hkv, d, int(dtype == torch.bfloat16), p)
        q = torch.empty((b, lq, group * hkv, d), dtype=dtype)
        qas.sparse_attn_q8(q, _cpu_cache(b, 128, hkv, d), 100, torch.zeros((b, 24), dtype=torch.int32),
                           torch.zeros(b, dtype=torch.int32), p)
        assert seen["size"] >= need and (need == 0 or seen["ws"] % 256 == 0), (b, hkv, group, lq)
        if need:
            asked.add(lq)
    assert asked == ({1, 2, 5} if dtype == torch.bfloat16 else set())


def test_import_needs_no_private_name_of_torch():
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    delattr(torch._C, name)\n"
            "import query_aware_selective_b200 as qas\n"
            "from query_aware_selective_b200 import _abi, cost, pipeline, synthetic\n"
            "assert _abi._current_device is torch.cuda.current_device and callable(_abi._raw_stream)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(qas.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("block", [0, -16, 48, 256])
def test_new_caches_of_a_wrong_block_are_refused(block):
    with pytest.raises(ValueError, match="block must be"):
        qas.cache_q8(1, 64, 2, 64, block=block, device="cpu")
