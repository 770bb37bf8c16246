"""The 4-bit key / value cache and attention over it against the plain 64-bit implementation
(tests/kv_plain.py); needs a B200.  Stored bytes and decoded values must be equal; attention
keeps the bounds derived there."""
import numpy as np
import pytest
import torch

import weight_only_quantized_int4_b200 as q
from tests import kv_plain as plain

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from weight_only_quantized_int4_b200 import build
    build.build()
    q.load()


def _f64(t):
    return t.double().cpu().numpy()


def _ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


FORMATS = [(64, "sym", -1), (64, "asym", 32), (128, "sym", -1), (128, "asym", 32), (128, "sym", 64),
           (128, "asym", 128), (256, "sym", 32), (256, "asym", -1), (256, "sym", 128)]


# ------------------------------------------------------------------ store and load

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,mode,group", FORMATS)
def test_store_writes_the_plain_bytes(dim, mode, group, dtype):
    torch.manual_seed(dim + len(mode))
    T, H, page, pages = 37, 3, 32, 4
    qkv = torch.randn(T, 3, H, dim, device="cuda") * torch.logspace(-6, 3, T, device="cuda")[:, None, None, None]
    qkv[5, 1] = 0                                    # a row of zeros
    qkv[6, 1, 0] = qkv[6, 1, 0].abs()                # one sign only
    qkv[7, 2, 1] = torch.randint(-7, 8, (dim,), device="cuda").float() / 2   # halves: ties
    qkv[7, 2, 1, ::32] = 7.0
    qkv = qkv.to(DT[dtype])
    slots = np.random.default_rng(1).permutation(page * pages)[:T].astype(np.int64)
    slots[3], slots[11], slots[20] = -1, page * pages, 2 ** 31 - 1          # skipped
    cache = q.kv_cache(pages, H, dim, page, mode, group)
    cache.random_(0, 256, generator=torch.Generator("cuda").manual_seed(4))
    want = cache.cpu().numpy().copy()
    k, v = qkv[:, 1], qkv[:, 2]                      # strided slices
    plain.store(want, page, _f64(k), _f64(v), slots, group, mode)
    q.kv_store(k, v, _ints(slots), cache, mode, group)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"

    live = [i for i in range(T) if 0 <= slots[i] < page * pages]
    rk, rv = q.kv_load(cache, _ints(slots), dim, mode, group, dtype=DT[dtype])
    pk, pv = plain.read_rows(want, page, dim, slots[live], group, mode)
    for r, p in ((rk, pk), (rv, pv)):
        exact = torch.tensor(p, dtype=torch.float32).to(DT[dtype])   # 16-bit products are exact in fp32
        assert torch.equal(r[live].cpu(), exact)
        dead = [i for i in range(T) if i not in live]
        assert not r[dead].any()


@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (2, 5), (700, 2)])
def test_store_sizes(T, H):
    dim, page = 128, 16
    torch.manual_seed(T)
    pages = (T + page - 1) // page + 1
    k = torch.randn(T, H, dim, device="cuda", dtype=torch.float16)
    v = torch.randn(T, H, dim, device="cuda", dtype=torch.float16)
    cache = q.kv_cache(pages, H, dim, page)
    slots = np.arange(T) + 3
    q.kv_store(k, v, _ints(slots), cache)
    want = np.zeros(tuple(cache.shape), np.uint8)
    plain.store(want, page, _f64(k), _f64(v), slots, -1, "sym")
    assert np.array_equal(cache.cpu().numpy(), want)
    empty = torch.empty(0, H, dim, device="cuda", dtype=torch.float16)
    q.kv_store(empty, empty, _ints([]), cache)       # nothing to do
    rk, _ = q.kv_load(cache, _ints([]), dim)
    assert rk.shape == (0, H, dim) and np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mode", ["sym", "asym"])
def test_store_at_rounding_borders(mode, dtype):
    """Scales that are powers of two and values at and next to every border between two codes;
    the largest value and the zero-point both rounded up; scales below fp16's normals."""
    dim = 64
    rows = []
    for scale in (1.0, 2.0 ** -10, 2.0 ** -20, 2.0 ** -23, 300.0):
        for top in (7.5, 7.0, 15.0):                 # with -7.5: 15 steps; code 16 must come out as 15
            for nudge in (-1, 0, 1):
                x = torch.zeros(dim)
                x[0], x[1] = -7.5 if mode == "asym" else -7.0, top if mode == "asym" else 7.0
                x[2:32] = (torch.arange(30) - 14.5) / 2 * (1 + nudge * 2.0 ** -9)
                rows.append(x * scale)
    k = torch.stack(rows)[:, None].cuda().to(DT[dtype])
    T = k.shape[0]
    cache = q.kv_cache(4, 1, dim, 16, mode, -1)
    q.kv_store(k, k, _ints(range(T)), cache, mode, -1)
    want = np.zeros(tuple(cache.shape), np.uint8)
    plain.store(want, 16, _f64(k), _f64(k), range(T), -1, mode)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("mode", ["sym", "asym"])
def test_store_of_values_that_are_not_finite(mode):
    dim, H = 128, 2
    k = torch.randn(4, H, dim, device="cuda").bfloat16()
    k[0, 0, 5] = float("nan")
    k[1, 0, 7] = float("inf")
    k[2, 1, 9] = -float("inf")
    k[3, 1, 3] = 3e38                                # beyond the largest scale
    cache = q.kv_cache(1, H, dim, 16, mode, 64)
    q.kv_store(k, k, _ints(range(4)), cache, mode, 64)
    want = np.zeros(tuple(cache.shape), np.uint8)
    plain.store(want, 16, _f64(k), _f64(k), range(4), 64, mode)
    assert np.array_equal(cache.cpu().numpy(), want)
    for t in q.kv_load(cache, _ints(range(4)), dim, mode, 64):
        assert torch.isfinite(t).all()


# ------------------------------------------------------------------------ attention

class Values(list):
    one_scale = True      # of a format with one scale per token


def _setup(lens, nq, H, KV, dim, page, mode, group, dtype, seed, qscale=1.0, spare=3):
    """A cache filled by kv_store, unwritten places left as NaN bytes; queries; the plain K~, V~."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(1, max(need))), -7, np.int32)      # unused entries are not pages
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = q.kv_cache(pages, KV, dim, page, mode, group)
    cache.fill_(0xFF)                                # every scale a NaN
    keys, values = [], Values()
    values.one_scale = group in (-1, dim)
    for b, n in enumerate(lens):
        k = torch.randn(n, KV, dim, device="cuda", generator=gen).to(DT[dtype])
        v = torch.randn(n, KV, dim, device="cuda", generator=gen).to(DT[dtype])
        t = np.arange(n)
        slots = table[b][t // page].astype(np.int64) * page + t % page
        q.kv_store(k, v, _ints(slots), cache, mode, group)
        for x, to in ((k, keys), (v, values)):
            c, s, z = plain.quantize(_f64(x), group, mode)
            to.append(plain.decode(c, s, z, group))
    total = sum(nq)
    qq = (torch.randn(total + 2, H, dim, device="cuda", generator=gen) * qscale).to(DT[dtype])
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    return cache, torch.tensor(table, device="cuda"), qq, cu, keys, values


def _expect(qq, cu, keys, values, scale, window):
    parts = [plain.attend(_f64(qq[cu[b]:cu[b + 1]]), keys[b], values[b], scale, window) for b in range(len(keys))]
    o, l, spread, dots, step = (np.concatenate([p[i] for p in parts]) for i in range(5))
    return o, l, spread, dots, step * values.one_scale


def _check(out, lse, want, dim, dtype, what="", rounded_keys=False):
    o, l, spread, dots, step = want
    bound, lbound = plain.bounds(o, spread, dots, dim, dtype, step, rounded_keys)
    err = np.abs(_f64(out) - o)
    assert np.all(err <= bound), (f"{what}: {int((~(err <= bound)).sum())} of {err.size} over the bound, worst "
                                  f"{np.nanmax(err / bound):.3f}, nan {int(np.isnan(err).sum())}")
    if lse is not None:
        g = _f64(lse)
        seen = np.isfinite(l)
        assert np.array_equal(np.isneginf(g), ~seen), what
        assert np.all(np.abs(g - np.where(seen, l, 0))[seen] <= lbound[seen] + 2.0 ** -22 * np.abs(l[seen])), what


RAGGED = [1, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 513]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,mode,group", FORMATS)
def test_decode_of_a_ragged_batch(dim, mode, group, dtype):
    H, KV, page = (8, 2, 16) if dim == 128 else (6, 3, 32)
    nq = [1] * len(RAGGED)
    cache, table, qq, cu, keys, values = _setup(RAGGED, nq, H, KV, dim, page, mode, group, dtype, 7 * dim)
    qd = qq[:len(RAGGED)].contiguous()
    scale = dim ** -0.5
    for window in (0, 1, 40):
        want = _expect(qq, cu, keys, values, scale, window)
        ws = q.kv_workspace(len(RAGGED), 1, H, KV, dim)
        for w in (ws, ws, None):                     # twice on one workspace, then without
            lse = torch.zeros(len(RAGGED), H, device="cuda")
            out = q.kv_attend(qd, cache, table, _ints(RAGGED), window=window, mode=mode, group=group, lse=lse, ws=w)
            _check(out, lse, want, dim, dtype, f"window {window} ws {w is not None}")


@pytest.mark.parametrize("H,KV,nq", [(32, 32, [1, 2]), (1, 1, [5, 3]), (7, 1, [1, 9]), (16, 1, [1, 1]), (24, 8, [4, 4]),
                                     (40, 8, [17, 1]), (64, 8, [70, 2]), (12, 4, [200, 31])])
@pytest.mark.parametrize("dim,mode,group,dtype", [(128, "sym", -1, "bf16"), (64, "asym", 64, "f16"),
                                                  (256, "asym", 64, "f16"), (128, "asym", 32, "f16")])
def test_several_queries(H, KV, nq, dim, mode, group, dtype):
    lens = [211, 97]
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, KV, dim, 64, mode, group, dtype, H + nq[0])
    total = int(cu[-1])
    for window in (0, 33):
        want = _expect(qq, cu, keys, values, 0.11, window)
        for split in (True, False):
            ws = q.kv_workspace(2, max(nq), H, KV, dim) if split else None
            guard = torch.full((total + 2, H, dim), 9.0, device="cuda", dtype=DT[dtype])
            lse = torch.full((total + 2, H), 5.0, device="cuda")
            q.kv_attend(qq, cache, table, _ints(lens), cu_q=torch.tensor(cu, device="cuda"), max_q=max(nq), scale=0.11,
                        window=window, mode=mode, group=group, out=guard, lse=lse, ws=ws)
            _check(guard[:total], lse[:total], want, dim, dtype, f"window {window} split {split}",
                   rounded_keys=max(nq) * H // KV >= 64)   # the tensor-core kernel's
            assert (guard[total:] == 9.0).all() and (lse[total:] == 5.0).all()    # rows behind the last


def test_more_queries_than_tokens_see_nothing():
    lens, nq = [3, 0, 40], [6, 2, 1]
    cache, table, qq, cu, keys, values = _setup(lens, nq, 8, 4, 128, 16, "sym", -1, "f16", 5)
    want = _expect(qq, cu, keys, values, 0.3, 0)
    total = int(cu[-1])
    lse = torch.zeros(total, 8, device="cuda")
    out = q.kv_attend(qq[:total], cache, table, _ints(lens), cu_q=torch.tensor(cu, device="cuda"), max_q=6, scale=0.3,
                      lse=lse, ws=q.kv_workspace(3, 6, 8, 4, 128))
    _check(out, lse, want, 128, "f16")
    assert not out[:3].any() and not out[6:8].any() and torch.isneginf(lse[6:8]).all()


def test_strided_queries_and_output():
    lens, H, KV, dim = [65, 200], 8, 8, 128
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], H, KV, dim, 32, "sym", 64, "bf16", 11)
    want = _expect(qq, cu, keys, values, dim ** -0.5, 0)
    fused = torch.zeros(2, 3, H, dim, device="cuda", dtype=torch.bfloat16)
    fused[:, 0] = qq[:2]
    wide = torch.full((2, 2 * H, dim), 3.0, device="cuda", dtype=torch.bfloat16)
    q.kv_attend(fused[:, 0], cache, table, _ints(lens), group=64, out=wide[:, :H])
    _check(wide[:, :H], None, want, dim, "bf16")
    assert (wide[:, H:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_peaked_and_tiny_queries(dtype):
    """Large logits (one key takes all), and queries far below fp16's range."""
    for qscale in (30.0, 1e-6 if dtype == "f16" else 1e-30):
        lens = [1000, 130]
        cache, table, qq, cu, keys, values = _setup(lens, [1, 1], 4, 1, 128, 64, "asym", 64, dtype, 3, qscale)
        want = _expect(qq, cu, keys, values, 1.0, 0)
        lse = torch.zeros(2, 4, device="cuda")
        out = q.kv_attend(qq[:2], cache, table, _ints(lens), scale=1.0, mode="asym", group=64, lse=lse,
                          ws=q.kv_workspace(2, 1, 4, 1, 128))
        _check(out, lse, want, 128, dtype, f"q of {qscale}")


def test_nan_query_stays_in_its_row():
    lens = [100, 50]
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], 8, 1, 128, 16, "sym", -1, "bf16", 9)
    want = _expect(qq, cu, keys, values, 0.1, 0)
    bad = qq[:2].clone()
    bad[0, 3, 17] = float("nan")
    out = q.kv_attend(bad, cache, table, _ints(lens), scale=0.1, ws=q.kv_workspace(2, 1, 8, 1, 128))
    assert torch.isnan(out[0, 3]).all()
    keep = [h for h in range(8) if h != 3]
    bound, _ = plain.bounds(want[0], want[2], want[3], 128, "bf16", want[4])
    err = np.abs(_f64(out) - want[0])
    assert np.all(err[1] <= bound[1]) and np.all(err[0, keep] <= bound[0, keep])


def test_negative_and_zero_scale():
    lens = [77]
    cache, table, qq, cu, keys, values = _setup(lens, [1], 4, 2, 64, 16, "sym", 32, "f16", 13)
    for scale in (-0.2, 0.0):
        want = _expect(qq, cu, keys, values, scale, 0)
        out = q.kv_attend(qq[:1], cache, table, _ints(lens), scale=scale, group=32, ws=q.kv_workspace(1, 1, 4, 2, 64))
        _check(out, None, want, 64, "f16", f"scale {scale}")


def test_pages_and_lengths_outside_are_clamped():
    """Table entries outside the cache read as page 0, lengths stop at the table, no access outside."""
    lens, H, KV, dim, page = [64, 64], 8, 8, 128, 16
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], H, KV, dim, page, "sym", -1, "f16", 21)
    good = q.kv_attend(qq[:2], cache, table, _ints(lens), ws=q.kv_workspace(2, 1, H, KV, dim))
    t2 = table.clone()
    t2[1, 0], t2[1, 1] = 1 << 30, -3
    t0 = table.clone()
    t0[1, 0] = t0[1, 1] = 0
    cache.masked_fill_(cache == 0xFF, 0)             # page 0 may be one never written
    a = q.kv_attend(qq[:2], cache, t2, _ints([1000, 64]), ws=q.kv_workspace(2, 1, H, KV, dim))
    b = q.kv_attend(qq[:2], cache, t0, _ints([64, 64]), ws=q.kv_workspace(2, 1, H, KV, dim))
    assert torch.equal(a, b)
    e = q.kv_attend(qq[:2], cache, table, _ints([-5, 64]), ws=q.kv_workspace(2, 1, H, KV, dim))
    assert not e[0].any()
    # query ranges outside q are cut off
    out = torch.full((2, H, dim), 4.0, device="cuda", dtype=torch.float16)
    q.kv_attend(qq[:2], cache, table, _ints(lens), cu_q=_ints([0, 1, 9]), max_q=8, out=out,
                ws=q.kv_workspace(2, 8, H, KV, dim))
    assert torch.isfinite(out).all()


def test_long_sequences_are_split_and_repeat_exactly():
    lens, H, KV, dim = [9000, 3], 8, 1, 128
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], H, KV, dim, 128, "asym", 64, "bf16", 31)
    want = _expect(qq, cu, keys, values, 0.2, 0)
    ws = q.kv_workspace(2, 1, H, KV, dim)
    outs = [q.kv_attend(qq[:2], cache, table, _ints(lens), scale=0.2, mode="asym", group=64, ws=ws) for _ in range(5)]
    _check(outs[0], None, want, dim, "bf16")
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    whole = q.kv_attend(qq[:2], cache, table, _ints(lens), scale=0.2, mode="asym", group=64)
    _check(whole, None, want, dim, "bf16")


def test_many_sequences():
    """More sequences than a CTA has threads: the length scan takes several rounds."""
    rng = np.random.default_rng(2)
    lens = [int(n) for n in rng.integers(0, 40, 300)]
    cache, table, qq, cu, keys, values = _setup(lens, [1] * 300, 4, 2, 64, 16, "sym", -1, "f16", 17)
    want = _expect(qq, cu, keys, values, 0.125, 0)
    for ws in (q.kv_workspace(300, 1, 4, 2, 64), None):
        out = q.kv_attend(qq[:300], cache, table, _ints(lens), ws=ws)
        _check(out, None, want, 64, "f16")


def test_captured_graph_serves_new_lengths():
    lens, H, KV, dim = [50, 700], 8, 2, 128
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], H, KV, dim, 16, "sym", -1, "f16", 41)
    ws = q.kv_workspace(2, 1, H, KV, dim)
    ld, qd, out = _ints(lens), qq[:2].clone(), torch.empty(2, H, dim, device="cuda", dtype=torch.float16)
    kn, vn = (torch.randn(2, KV, dim, device="cuda", dtype=torch.float16) for _ in range(2))
    slots = _ints([-1, -1])

    def step():
        q.kv_store(kn, vn, slots, cache)
        q.kv_attend(qd, cache, table, ld, out=out, ws=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([50, 700], [10, 33], [0, 699]):
        ld.copy_(_ints(new))
        graph.replay()
        want = _expect(qq, cu, [keys[b][:n] for b, n in enumerate(new)],
                       Values(values[b][:n] for b, n in enumerate(new)), dim ** -0.5, 0)
        _check(out, None, want, dim, "f16", str(new))
    # a token appended inside the graph
    page = int(table[0, 10 // 16]) * 16
    slots.copy_(_ints([page + 10, -1]))
    ld.copy_(_ints([11, 33]))
    graph.replay()
    for x, full in ((kn, keys), (vn, values)):
        c, sc, z = plain.quantize(_f64(x), -1, "sym")
        full[0][10] = plain.decode(c, sc, z, -1)[0]
    want = _expect(qq, cu, [keys[0][:11], keys[1][:33]], Values([values[0][:11], values[1][:33]]), dim ** -0.5, 0)
    _check(out, None, want, dim, "f16", "appended")


def test_one_workspace_for_calls_of_all_shapes():
    """Calls of different shapes in turn on one workspace: each leaves it ready for the next."""
    shapes = [([5000, 4000, 3000], [1, 1, 1], 8, 2), ([6000], [70], 2, 1), ([900] * 20, [1] * 20, 16, 8),
              ([3000], [3], 4, 4), ([5000], [2], 64, 1)]
    sets = [(_setup(lens, nq, H, KV, 64, 64, "sym", -1, "f16", i), lens, nq, H, KV) for i, (lens, nq, H, KV) in enumerate(shapes)]
    size = max(q.kv_workspace(len(lens), max(nq), H, KV, 64).numel() for _, lens, nq, H, KV in sets)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(3):
        for i, ((cache, table, qq, cu, _, _), lens, nq, H, KV) in enumerate(sets):
            own = q.kv_workspace(len(lens), max(nq), H, KV, 64)
            args = (qq[:sum(nq)], cache, table, _ints(lens))
            kw = dict(cu_q=_ints(cu), max_q=max(nq))
            if i not in first:
                first[i] = q.kv_attend(*args, ws=own, **kw)
            assert torch.equal(q.kv_attend(*args, ws=ws, **kw), first[i]), (turn, i)


@pytest.mark.parametrize("H,KV", [(4, 2), (64, 1)])
def test_queries_past_max_q_get_no_output(H, KV):
    """... and the others keep their places in the sequence."""
    lens, nq = [300], [9]
    cache, table, qq, cu, keys, values = _setup(lens, nq, H, KV, 64, 16, "sym", -1, "f16", 61)
    want = _expect(qq, cu, keys, values, 0.1, 40)
    out = torch.full((9, H, 64), 8.0, device="cuda", dtype=torch.float16)
    q.kv_attend(qq[:9], cache, table, _ints(lens), cu_q=_ints([0, 9]), max_q=5, scale=0.1, window=40, out=out,
                ws=q.kv_workspace(1, 5, H, KV, 64))
    _check(out[:5], None, tuple(w[:5] for w in want), 64, "f16", rounded_keys=5 * H // KV >= 64)
    assert (out[5:] == 8.0).all()


def test_two_streams_at_once():
    lens, H, KV, dim = [4000, 2500], 32, 4, 128
    cache, table, qq, cu, keys, values = _setup(lens, [1, 1], H, KV, dim, 64, "sym", -1, "bf16", 51)
    ref = q.kv_attend(qq[:2], cache, table, _ints(lens), ws=q.kv_workspace(2, 1, H, KV, dim))
    ld = _ints(lens)
    ss = [torch.cuda.Stream() for _ in range(2)]
    wss = [q.kv_workspace(2, 1, H, KV, dim) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for s, ws in zip(ss, wss):
            with torch.cuda.stream(s):
                outs.append(q.kv_attend(qq[:2], cache, table, ld, ws=ws))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


def test_binding_refusals():
    c = q.kv_cache(4, 8, 128, page=64)
    k = torch.zeros(3, 8, 128, device="cuda", dtype=torch.float16)
    s = _ints([0, 1, 2])
    for bad in (lambda: q.kv_store(k, k.bfloat16(), s, c), lambda: q.kv_store(k, k[:2], s, c),
                lambda: q.kv_store(k, k, s[:2], c), lambda: q.kv_store(k, k, s.long(), c),
                lambda: q.kv_store(k.transpose(0, 1), k.transpose(0, 1), _ints(range(8)), c),
                lambda: q.kv_store(k[:, :4], k[:, :4], s, c), lambda: q.kv_store(k, k, s, c, "asym"),
                lambda: q.kv_store(k.float(), k.float(), s, c), lambda: q.kv_store(k.cpu(), k.cpu(), s, c),
                lambda: q.kv_load(c, s, 64), lambda: q.kv_load(c, s, 128, dtype=torch.float32, out=(k.float(), k)),
                lambda: q.kv_attend(k, c, _ints([0, 1, 2]), s), lambda: q.kv_attend(k, c, s[:, None], s[:2]),
                lambda: q.kv_attend(k, c, s[:, None], s, cu_q=s), lambda: q.kv_attend(k, c, s[:, None], s, out=k[:2]),
                lambda: q.kv_attend(k, c, s[:, None], s, lse=torch.zeros(3, 8, device="cuda").half())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.QmmError):
        q.kv_store(k, k, s, c, "lut")
    with pytest.raises(q.QmmError):                  # out over q
        q.kv_attend(k, c, s[:, None], s, out=k)
    with pytest.raises(q.QmmError):                  # 5 query heads on 8 key heads
        q.kv_attend(k[:, :5].contiguous(), c, s[:, None], s)
