"""Attention over the 4-bit cache with many query rows per key head (the tensor-core kernel)
against the plain 64-bit implementation; needs a B200.  Bounds: tests/kv_plain.py."""
import numpy as np
import pytest
import torch

import weight_only_quantized_int4_b200 as q
from tests import kv_plain as plain
from tests.test_gpu_kv import DT, FORMATS, Values, _check as check, _expect, _f64, _ints, _setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from weight_only_quantized_int4_b200 import build
    build.build()
    q.load()


def _check(out, lse, want, dim, dtype, what=""):
    check(out, lse, (*want[:4], np.zeros_like(want[4])), dim, dtype, what, rounded_keys=True)


def _run(lens, nq, H, KV, dim, page, mode, group, dtype, seed, windows=(0,), scale=0.1, qscale=1.0):
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, KV, dim, page, mode, group, dtype, seed, qscale)
    total = int(cu[-1])
    ws = q.kv_workspace(len(lens), max(nq), H, KV, dim)
    for window in windows:
        want = _expect(qq, cu, keys, values, scale, window)
        guard = torch.full((total + 2, H, dim), 9.0, device="cuda", dtype=DT[dtype])
        lse = torch.full((total + 2, H), 5.0, device="cuda")
        q.kv_attend(qq, cache, table, _ints(lens), cu_q=torch.tensor(cu, device="cuda"), max_q=max(nq), scale=scale,
                    window=window, mode=mode, group=group, out=guard, lse=lse, ws=ws)
        q.check_error()
        _check(guard[:total], lse[:total], want, dim, dtype, f"window {window}")
        assert (guard[total:] == 9.0).all() and (lse[total:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,mode,group", FORMATS)
def test_formats(dim, mode, group, dtype):
    _run([300], [150], 2, 1, dim, 32, mode, group, dtype, dim, windows=(0, 50))


@pytest.mark.parametrize("lens,nq,H,KV", [
    ([64], [64], 1, 1), ([129], [129], 2, 2), ([256], [65], 4, 2), ([1000], [128], 2, 1), ([257, 513], [257, 90], 3, 1),
    ([70, 400, 33], [70, 1, 33], 8, 4),          # sequences of both kernels in one call
    ([100, 0, 640], [5, 70, 320], 8, 2),         # few rows; no tokens; many
    ([40], [200], 1, 1),                         # more queries than tokens
    ([900], [300], 7, 1), ([384], [384], 6, 3)])
def test_lengths(lens, nq, H, KV):
    _run(lens, nq, H, KV, 128, 16, "asym", 64, "f16", sum(lens), windows=(0, 1, 130))


@pytest.mark.parametrize("page", [16, 64, 512])
def test_pages(page):
    _run([700, 130], [100, 130], 4, 2, 64, page, "sym", -1, "bf16", page)


@pytest.mark.parametrize("scale,qscale", [(1.0, 3.0), (-0.2, 1.0), (0.0, 1.0), (0.1, 1e-20)])
def test_scales(scale, qscale):
    _run([310], [140], 2, 1, 128, 64, "sym", -1, "bf16", 5, scale=scale, qscale=qscale)


def test_rising_logits_move_the_reference():
    """Later tokens with ever larger logits: the reference and the sums are rescaled tile by tile."""
    dim, n = 128, 640
    cache = q.kv_cache(10, 1, dim, 64)
    k = torch.zeros(n, 1, dim, device="cuda")
    k[:, 0, 0] = torch.linspace(0, 60, n, device="cuda")
    k[:, 0, 1] = 8.0
    v = torch.randn(n, 1, dim, device="cuda")
    k, v = k.half(), v.half()
    q.kv_store(k, v, _ints(range(n)), cache)
    keys, values = [], Values()
    for x, to in ((k, keys), (v, values)):
        c, s, z = plain.quantize(_f64(x), -1, "sym")
        to.append(plain.decode(c, s, z, -1))
    qq = torch.zeros(100, 2, dim, device="cuda", dtype=torch.float16)
    qq[:, 0, 0], qq[:, 1, 0], qq[:, 1, 1] = 1.0, -1.0, 0.25
    cu = np.array([0, 100], np.int32)
    want = _expect(qq, cu, keys, values, 1.0, 0)
    out = q.kv_attend(qq, cache, _ints(range(10))[None], _ints([n]), cu_q=_ints(cu), max_q=100, scale=1.0,
                      ws=q.kv_workspace(1, 100, 2, 1, dim))
    _check(out, None, want, dim, "f16")


def test_nan_query_stays_in_its_row():
    lens, nq = [200], [100]
    cache, table, qq, cu, keys, values = _setup(lens, nq, 2, 1, 128, 16, "sym", -1, "bf16", 9)
    want = _expect(qq, cu, keys, values, 0.1, 0)
    bad = qq[:100].clone()
    bad[3, 1, 17] = float("nan")
    out = q.kv_attend(bad, cache, table, _ints(lens), cu_q=_ints(cu), max_q=100, scale=0.1,
                      ws=q.kv_workspace(1, 100, 2, 1, 128))
    assert torch.isnan(out[3, 1]).all()
    out[3, 1] = torch.tensor(want[0][3, 1], device="cuda").bfloat16()
    _check(out, None, want, 128, "bf16")


def test_repeats_exactly_and_without_workspace():
    lens, nq = [1200, 300], [400, 300]
    cache, table, qq, cu, keys, values = _setup(lens, nq, 4, 1, 128, 64, "asym", 128, "f16", 19)
    total = int(cu[-1])
    args = (qq[:total], cache, table, _ints(lens))
    kw = dict(cu_q=_ints(cu), max_q=400, mode="asym", group=128)
    ws = q.kv_workspace(2, 400, 4, 1, 128)
    outs = [q.kv_attend(*args, ws=ws, **kw) for _ in range(3)] + [q.kv_attend(*args, **kw)]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dim,mode,group,dtype", [(128, "sym", -1, "f16"), (64, "asym", 32, "bf16"), (256, "sym", 128, "f16")])
def test_long_sequences_are_split(dim, mode, group, dtype):
    """Few tiles of rows on long sequences: their tokens are split between CTAs through the
    workspace, the same way at every call; without a workspace nothing is split."""
    lens, nq, H, KV = [4100, 130], [70, 100], 2, 1
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, KV, dim, 128, mode, group, dtype, 29)
    total = int(cu[-1])
    ws = q.kv_workspace(2, 100, H, KV, dim)
    for window in (0, 2500):
        want = _expect(qq, cu, keys, values, 0.1, window)
        outs = []
        for w in (ws, ws, None):
            lse = torch.zeros(total, H, device="cuda")
            outs.append(q.kv_attend(qq[:total], cache, table, _ints(lens), cu_q=_ints(cu), max_q=100, scale=0.1,
                                    window=window, mode=mode, group=group, lse=lse, ws=w))
            q.check_error()
            _check(outs[-1], lse, want, dim, dtype, f"window {window} ws {w is not None}")
        assert torch.equal(outs[0], outs[1])


def test_a_wait_that_runs_out_is_reported():
    """A wait bound too short to wait for anything: the call gives up, the error is reported,
    and the next call is right."""
    lens, nq = [500], [200]
    cache, table, qq, cu, keys, values = _setup(lens, nq, 2, 1, 128, 64, "sym", -1, "f16", 23)
    want = _expect(qq, cu, keys, values, 0.1, 0)
    args = (qq[:200], cache, table, _ints(lens))
    kw = dict(cu_q=_ints(cu), max_q=200, scale=0.1)
    old = q.set_wait_limit(1)
    try:
        q.kv_attend(*args, **kw)
        with pytest.raises(q.QmmError) as e:
            q.check_error()
        assert e.value.status == -5
    finally:
        q.set_wait_limit(old)
    out = q.kv_attend(*args, **kw)
    q.check_error()
    _check(out, None, want, 128, "f16")


@pytest.mark.parametrize("nq", [[3, 1], [120, 7]])
def test_without_a_bound_on_the_queries(nq):
    """max_q left out: every query gets its output, however many a sequence has."""
    lens, H, KV, dim = [300, 90], 4, 2, 128
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, KV, dim, 32, "sym", -1, "f16", sum(nq))
    total = int(cu[-1])
    want = _expect(qq, cu, keys, values, 0.1, 0)
    lse = torch.zeros(total, H, device="cuda")
    out = q.kv_attend(qq[:total], cache, table, _ints(lens), cu_q=torch.tensor(cu, device="cuda"), scale=0.1, lse=lse,
                      ws=q.kv_workspace(2, total, H, KV, dim))
    q.check_error()
    _check(out, lse, want, dim, "f16")


@pytest.mark.parametrize("dim", [64, 256])
def test_a_bound_on_queries_far_above_them(dim):
    """max_q at its limit with 1024 query heads on one key head: the rows that the bound alone would
    give do not fit 32 bits, those of the queries do."""
    lens, nq, H = [300, 40], [3, 1], 1024
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, 1, dim, 16, "sym", -1, "f16", 5)
    want = _expect(qq, cu, keys, values, 0.1, 0)
    most = 1 << 22
    for ws in (None, q.kv_workspace(2, most, H, 1, dim)):
        lse = torch.empty(4, H, device="cuda")
        out = q.kv_attend(qq[:4], cache, table, _ints(lens), cu_q=torch.tensor(cu, device="cuda"), max_q=most, scale=0.1,
                          lse=lse, ws=ws)
        q.check_error()
        _check(out, lse, want, dim, "f16")


@pytest.mark.parametrize("dim", [128, 256])
def test_a_split_tile_that_gives_up(dim):
    """A wait that runs out while a tile's tokens are split between CTAs: the parts that gave up are
    not counted, the error is reported, and the workspace is good again once it is zero filled."""
    lens, nq, H = [4100], [70], 2
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, 1, dim, 128, "sym", -1, "f16", 31)
    want = _expect(qq, cu, keys, values, 0.1, 0)
    args = (qq[:70], cache, table, _ints(lens))
    ws = q.kv_workspace(1, 70, H, 1, dim)
    kw = dict(cu_q=_ints(cu), max_q=70, scale=0.1, ws=ws)
    q.kv_attend(*args, **kw)
    q.check_error()
    old = q.set_wait_limit(1)
    try:
        q.kv_attend(*args, **kw)
        with pytest.raises(q.QmmError) as e:
            q.check_error()
        assert e.value.status == -5
    finally:
        q.set_wait_limit(old)
    ws.zero_()
    outs = [q.kv_attend(*args, **kw) for _ in range(2)]
    q.check_error()
    for out in outs:
        _check(out, None, want, dim, "f16")
    assert torch.equal(outs[0], outs[1])
