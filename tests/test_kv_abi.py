"""The 4-bit cache's entry points without a GPU: sizes, refusals (nothing is launched or read),
and the plain implementation the GPU tests compare with, pinned by hand."""
import ctypes

import numpy as np
import pytest
import torch

import weight_only_quantized_int4_b200 as q
from tests import kv_plain as plain

P = ctypes.c_void_p
A, B, C_, D_ = P(0x1000), P(0x900000), P(0x1900000), P(0x2900000)     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from weight_only_quantized_int4_b200 import build
    build.build()
    return q.load()


def test_cache_sizes(lib):
    # a tile: 16 tokens x (dim bytes of K and V codes + their parameters)
    assert lib.qmm_kv_cache_size(1, 1, 128, 16, -1, 0) == 16 * (128 + 4)
    assert lib.qmm_kv_cache_size(3, 8, 128, 64, 32, 1) == 3 * 8 * 64 * (128 + 2 * 4 * 4)
    assert lib.qmm_kv_cache_size(5, 2, 64, 32, 64, 1) == 5 * 2 * 32 * (64 + 8)
    assert lib.qmm_kv_cache_size(5, 2, 256, 128, 128, 0) == 5 * 2 * 128 * (256 + 8)


@pytest.mark.parametrize("pages,heads,dim,page,group,mode,status", [
    (0, 8, 128, 64, -1, 0, -1), (4, 0, 128, 64, -1, 0, -1), (4, 8, 128, 64, -1, 7, -1),
    (4, 8, 128, 64, -1, 2, -2),                               # no table codes
    (4, 8, 96, 64, -1, 0, -2), (4, 8, 0, 64, -1, 0, -2),      # dim
    (4, 8, 128, 8, -1, 0, -2), (4, 8, 128, 48, -1, 0, -2), (4, 8, 128, 1 << 17, -1, 0, -2),   # page
    (4, 8, 128, 64, 16, 0, -2), (4, 8, 128, 64, 96, 0, -2), (4, 8, 64, 64, 128, 0, -2),   # group
    (4, 8, 128, 64, 0, 0, -2), (1 << 30, 8, 128, 64, -1, 0, -2), (4, 5000, 128, 64, -1, 0, -2),
])
def test_bad_formats(lib, pages, heads, dim, page, group, mode, status):
    assert lib.qmm_kv_cache_size(pages, heads, dim, page, group, mode) == 0
    assert lib.qmm_kv_store(A, B, 0, 1 << 20, 1 << 20, C_, 1, heads, dim, page, pages, group, mode, D_,
                            None) == status
    assert lib.qmm_kv_load(A, C_, 1, heads, dim, page, pages, group, mode, 0, B, D_, None) == status
    assert lib.qmm_kv_attend(A, 0, 1 << 20, B, C_, C_, None, 1, 1, 1, 8, heads, dim, page, pages, 4, group,
                             mode, 1.0, 0, D_, 1 << 20, None, None, 0, None) == status


def test_store_and_load_refusals(lib):
    def store(k=A, v=B, dt=0, ks=1024, vs=1024, slots=C_, tokens=3, cache=D_):
        return lib.qmm_kv_store(k, v, dt, ks, vs, slots, tokens, 8, 128, 64, 4, -1, 0, cache, None)

    assert store(dt=2) == -1 and store(tokens=-1) == -1 and store(tokens=0) == 0
    assert store(k=None) == -1 and store(v=None) == -1 and store(slots=None) == -1 and store(cache=None) == -1
    assert store(ks=1023) == -1 and store(vs=8) == -1 and store(ks=-1024) == -1
    assert store(ks=1028) == -3 and store(k=P(0x1008)) == -3 and store(cache=P(0x2900004)) == -3
    assert store(slots=P(0x1900002)) == -3

    def load(cache=A, slots=C_, tokens=3, dt=0, k=B, v=D_):
        return lib.qmm_kv_load(cache, slots, tokens, 8, 128, 64, 4, -1, 0, dt, k, v, None)

    assert load(dt=-1) == -1 and load(tokens=-5) == -1 and load(tokens=0) == 0
    assert load(cache=None) == -1 and load(slots=None) == -1 and load(k=None) == -1 and load(v=None) == -1
    assert load(k=P(0x900008)) == -3 and load(cache=P(0x1001)) == -3


def test_attend_refusals(lib):
    need = lib.qmm_kv_workspace_size(2, 1, 32, 8, 128)
    assert need > 0
    for bad in ((0, 1, 32, 8, 128), (2, 0, 32, 8, 128), (2, 1, 30, 8, 128), (2, 1, 0, 8, 128), (2, 1, 32, 8, 80)):
        assert lib.qmm_kv_workspace_size(*bad) == 0

    def attend(qp=A, dt=0, qs=4096, cache=B, table=C_, lens=C_, cu=None, batch=2, total=2, max_q=1, H=32, KV=8,
               max_pages=4, scale=0.1, window=0, out=D_, os=4096, lse=None, ws=None, wsb=0):
        return lib.qmm_kv_attend(qp, dt, qs, cache, table, lens, cu, batch, total, max_q, H, KV, 128, 64, 16,
                                 max_pages, -1, 0, scale, window, out, os, lse, ws, wsb, None)

    assert attend(batch=0) == 0 and attend(total=0) == 0           # nothing to do
    assert attend(batch=-1) == -1 and attend(total=-1, cu=C_) == -1 and attend(max_q=0, cu=C_) == -1
    assert attend(total=3) == -1 and attend(max_q=2) == -1         # without cu_q: one query each
    assert attend(dt=5) == -1 and attend(H=30) == -1 and attend(max_pages=0) == -1 and attend(window=-1) == -1
    assert attend(scale=float("nan")) == -1 and attend(scale=float("inf")) == -1
    assert attend(max_pages=1 << 26) == -2
    for name in ("qp", "cache", "table", "lens", "out"):
        assert attend(**{name: None}) == -1, name
    assert attend(qs=4095) == -1 and attend(os=8) == -1 and attend(qs=4100) == -3 and attend(os=4100) == -3
    assert attend(qp=P(0x1004)) == -3 and attend(out=P(0x2900008)) == -3 and attend(lse=P(0x3900002)) == -3
    assert attend(out=P(0x1000 + 4096)) == -1                      # overlaps q
    assert attend(ws=P(0x3900000), wsb=need - 1) == -6
    assert attend(ws=P(0x3900010), wsb=need) == -3


def test_attend_refuses_more_rows_than_32_bits_hold(lib):
    """Query heads per key head times a sequence's queries: the kernels number a tile's rows in 32
    bits.  What the bound max_q alone would allow does not count, only queries that q holds."""
    def attend(max_q, total, H):
        return lib.qmm_kv_attend(A, 0, H * 64, B, C_, C_, C_, 1, total, max_q, H, 1, 64, 64, 16, 4, -1, 0, 0.1, 0,
                                 P(1 << 56), H * 64, None, None, 0, None)

    assert attend(1 << 22, 1 << 22, 512) == -2 and attend(1 << 22, 1 << 22, 4096) == -2
    assert attend(1 << 22, 1 << 21, 1024) == -2
    assert attend((1 << 22) + 1, 1, 1) == -2
    # a loose bound over few queries is sized as before
    assert lib.qmm_kv_workspace_size(1, 1 << 22, 4096, 1, 64) > 0


def test_binding_refuses_before_the_library(lib):
    k = torch.zeros(3, 8, 128, dtype=torch.float16)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        q.kv_store(k, k, torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, 4, 2112, dtype=torch.uint8))
    with pytest.raises(q.QmmError):
        q.kv_cache(4, 8, 100, device="cpu")
    with pytest.raises(q.QmmError):
        q.kv_workspace(2, 1, 30, 8, 128, device="cpu")
    c = q.kv_cache(4, 8, 128, page=64, device="cpu")
    assert tuple(c.shape) == (4, 8, 4, 16 * 132)


# ------------------------------------------------- the plain implementation, by hand

def test_plain_quantizer_by_hand():
    x = np.zeros(64)
    x[:4] = [7.0, -3.5, 2.5, 0.5]                    # s = 1: halves go to even
    c, s, z = plain.quantize(x, -1, "sym")
    assert s[0] == 1 and list(c[:5]) == [15, 8 - 4, 8 + 2, 8, 8] and z is None
    x[:3] = [-3.0, 12.0, 4.5]                        # s = 15 / 15, z = 3
    c, s, z = plain.quantize(x, -1, "asym")
    assert s[0] == 1 and z[0] == 3 and list(c[:3]) == [0, 15, 7]
    c, s, z = plain.quantize(np.full(64, 5.0), -1, "asym")    # all of one sign: nothing clipped
    assert z[0] == 0 and np.allclose(plain.decode(c, s, z, -1), 5.0, rtol=2 ** -10)
    c, s, z = plain.quantize(np.full(64, 60000.0), -1, "sym")
    assert s[0] == 4096 and c.max() == 15
    c, s, z = plain.quantize(np.zeros(64), 32, "asym")
    assert not s.any() and not c.any() and not z.any()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_plain_layout_is_a_permutation(dim):
    for tok in range(16):
        assert sorted(plain.key_word(dim, n, tok) for n in range(dim // 8)) == list(range(dim // 8))
        assert sorted(plain.value_word(dim, n, tok) for n in range(dim // 8)) == list(range(dim // 8))


@pytest.mark.parametrize("dim,mode,group", [(64, "sym", -1), (128, "asym", 32), (256, "sym", 128)])
def test_plain_store_reads_back(dim, mode, group):
    rng = np.random.default_rng(3)
    G = 1 if group == -1 else dim // group
    cache = np.zeros((2, 3, 2, plain.tile_bytes(dim, G, mode)), np.uint8)
    k, v = (rng.standard_normal((5, 3, dim)).astype(np.float16).astype(np.float64) for _ in range(2))
    slots = [0, 17, 63, -1, 40]
    plain.store(cache, 32, k, v, slots, group, mode)
    rk, rv = plain.read_rows(cache, 32, dim, [s for s in slots if s >= 0], group, mode)
    keep = [i for i, s in enumerate(slots) if s >= 0]
    for x, r in ((k, rk), (v, rv)):
        c, s, z = plain.quantize(x[keep], group, mode)
        assert np.array_equal(plain.decode(c, s, z, group), r)
        step = np.repeat(s.astype(np.float64), dim // G, -1)
        assert np.all(np.abs(r - x[keep]) <= 0.51 * step + 8 * 2.0 ** -11 * step)


def test_workspace_stays_within_what_the_header_says(lib):
    """The header names the largest workspace of a 148-SM GPU; a sweep over the shapes comes close to
    it and never above."""
    import os
    import re
    with open(os.path.join(os.path.dirname(q.LIB_PATH), "..", "include", "qmm.h")) as f:
        said = re.search(r"at most (\d+) MB", f.read().replace("\n *", " "))
    assert said, "the header names no size"
    batches = (1, 2, 3, 5, 9, 17, 30, 37, 74, 75, 148, 300, 4096, 1 << 20)
    queries = (1, 2, 7, 8, 16, 33, 64, 100, 128, 129, 250, 511, 512, 1000, 2048, 9000, 40000, 1 << 22)
    most = 0
    for dim in (64, 128, 256):
        for kv in (1, 2, 3, 4, 8, 37, 64):
            for per in (1, 2, 3, 4, 7, 8, 16, 64):
                for b in batches:
                    for m in queries:
                        n = lib.qmm_kv_workspace_size(b, m, kv * per, kv, dim)
                        assert n > 0
                        most = max(most, n)
    assert 0.95 * int(said[1]) * 1e6 < most <= int(said[1]) * 1e6, most
