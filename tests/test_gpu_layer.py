"""A decoder layer on 4-bit weights and a 4-bit cache, as a serving program runs it (needs a
B200): QKV product with bias, keys and values into the cache, attention over it, output product
added onto the residual stream, gated feed-forward, down product added in place.  A prompt of one
sequence and of another, then decode steps of both from one captured graph.

Every stage is checked against its plain 64-bit form on the inputs it really had (the outputs of
the stage before, read back), with the bounds of the single operators' tests."""
import numpy as np
import pytest
import torch

import oracle
import weight_only_quantized_int4_b200 as q
from tests import cases
from tests import kv_plain as plain
from weight_only_quantized_int4_b200 import synth

pytestmark = pytest.mark.gpu

HID, H, KV, DIM, FF, PAGE, GROUP = 512, 4, 2, 128, 704, 16, 64
HALF = 2.0 ** -11


def _f64(t):
    return t.double().cpu().numpy()


class Weight:
    """A SYM group-64 weight on the device and its decoded values."""

    def __init__(self, name, N, K):
        self.N, self.K = N, K
        W = synth.weights(3, name, N, K, 0.04)
        codes, scales, _ = oracle.quantize(W, "sym", 4, GROUP)
        self.values = oracle.dequant(codes, scales, None, "sym", 4, GROUP).astype(np.float64)
        self.qw, self.sc, _ = q.pack(torch.from_numpy(W).cuda(), "sym", 4, GROUP)

    def check(self, y, x, bias=None, residual=None):
        xs = _f64(x)
        s, lim = xs @ self.values.T, cases.ELEM_TOL * (np.abs(xs) @ np.abs(self.values).T)
        b = 0.0 if bias is None else _f64(bias)
        r = 0.0 if residual is None else _f64(residual)
        ref = r + s + b
        err = np.abs(_f64(y) - ref)
        assert np.all(err <= lim + 2.0 ** -20 * (np.abs(s) + np.abs(b) + np.abs(r)) + HALF * np.abs(ref) + 2.0 ** -24)


class Layer:
    def __init__(self):
        g = torch.Generator("cuda").manual_seed(1)
        self.qkv = Weight("qkv", (H + 2 * KV) * DIM, HID)
        self.o = Weight("o", HID, H * DIM)
        self.down = Weight("down", HID, FF)
        self.bias = torch.randn((H + 2 * KV) * DIM, device="cuda", generator=g).half() * 0.1
        Wg, Wu = synth.weights(3, "gate", FF, HID, 0.04), synth.weights(3, "up", FF, HID, 0.04)
        self.gated = q.pack_gated(torch.from_numpy(Wg).cuda(), torch.from_numpy(Wu).cuda(), "sym", 4, GROUP)
        dec = [oracle.dequant(*oracle.quantize(W, "sym", 4, GROUP)[:2], None, "sym", 4, GROUP) for W in (Wg, Wu)]
        self.Wg, self.Wu = (d.astype(np.float64) for d in dec)
        self.cache = q.kv_cache(24, KV, DIM, PAGE, "asym", GROUP)
        self.ws = {}

    def workspace(self, M, N, K):
        if (M, N, K) not in self.ws:
            self.ws[M, N, K] = q.workspace(M, N, K, "sym", 4, GROUP)
        return self.ws[M, N, K]

    def product(self, x, w, **kw):
        return q.qmm_epilogue(x, w.qw, w.sc, None, w.N, w.K, "sym", 4, GROUP, ws=self.workspace(x.shape[0], w.N, w.K), **kw)

    def run(self, h, slots, table, lens, cu, max_q, kws):
        """One pass; every intermediate is returned (h is updated in place)."""
        M = h.shape[0]
        qkv = self.product(h, self.qkv, bias=self.bias).view(M, H + 2 * KV, DIM)
        k, v = qkv[:, H:H + KV], qkv[:, H + KV:]
        q.kv_store(k, v, slots, self.cache, "asym", GROUP)
        att = q.kv_attend(qkv[:, :H], self.cache, table, lens, cu_q=cu, max_q=max_q, mode="asym", group=GROUP, ws=kws)
        mid = self.product(att.view(M, H * DIM), self.o, residual=h)
        ff = q.qmm_gated(mid, *self.gated[:2], None, FF, HID, "sym", 4, GROUP, ws=self.workspace(M, 2 * FF, HID))
        out = self.product(ff, self.down, residual=mid.clone(), y=h)
        return qkv, att, mid, ff, out

    def check(self, h0, parts, slots, seqs, keys, values, rounded):
        """seqs: per sequence (rows of this pass); keys / values: its decoded history, extended here."""
        qkv, att, mid, ff, out = parts
        M = h0.shape[0]
        self.qkv.check(qkv.view(M, -1), h0, bias=self.bias)
        for s, rows in enumerate(seqs):
            for x, hist in ((qkv[rows, H:H + KV], keys), (qkv[rows, H + KV:], values)):
                c, sc, z = plain.quantize(_f64(x), GROUP, "asym")
                hist[s] = np.concatenate([hist[s], plain.decode(c, sc, z, GROUP)])
            o, _, spread, dots, _ = plain.attend(_f64(qkv[rows, :H]), keys[s], values[s], DIM ** -0.5, 0)
            bound, _ = plain.bounds(o, spread, dots, DIM, "f16", np.zeros_like(dots), rounded)
            assert np.all(np.abs(_f64(att[rows]) - o) <= bound)
        self.o.check(mid, att.reshape(M, -1), residual=h0)
        xs = _f64(mid)
        a, b = xs @ self.Wg.T, xs @ self.Wu.T
        ea, eb = (cases.ELEM_TOL * (np.abs(xs) @ np.abs(W).T) for W in (self.Wg, self.Wu))
        gate = a / (1 + np.exp(-a))
        assert np.all(np.abs(_f64(ff) - gate * b) <= 1.1 * np.abs(b) * ea + np.abs(gate) * eb + 1.1 * ea * eb
                      + 2 * HALF * np.abs(gate * b) + 2.0 ** -24)
        self.down.check(out, ff, residual=mid)


def test_prompt_then_decode_steps():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from weight_only_quantized_int4_b200 import build
    build.build()
    layer = Layer()
    pages = np.random.default_rng(0).permutation(24)
    table = torch.tensor(pages.reshape(2, 12).astype(np.int32), device="cuda")
    slot = lambda s, t: int(pages.reshape(2, 12)[s, t // PAGE]) * PAGE + t % PAGE
    g = torch.Generator("cuda").manual_seed(2)
    ints = lambda a: torch.tensor(list(a), dtype=torch.int32, device="cuda")
    none = np.zeros((0, KV, DIM))
    keys, values = [none, none], [none, none]

    # prompts of 130 and 37 tokens in one pass (rows per key head: 260 and 74)
    n = [130, 37]
    h = torch.randn(sum(n), HID, device="cuda", generator=g).half()
    slots = ints(slot(s, t) for s in range(2) for t in range(n[s]))
    kws = q.kv_workspace(2, 130, H, KV, DIM)
    h0 = h.clone()
    parts = layer.run(h, slots, table, ints(n), ints([0, n[0], sum(n)]), 130, kws)
    q.check_error()
    layer.check(h0, parts, slots, [slice(0, n[0]), slice(n[0], sum(n))], keys, values, rounded=True)

    # decode: one token of each, the same graph for every step
    h, slots, lens = torch.zeros(2, HID, device="cuda", dtype=torch.float16), ints([-1, -1]), ints([0, 0])
    kws = q.kv_workspace(2, 1, H, KV, DIM)
    layer.run(h, slots, table, lens, None, 1, kws)          # warm-up on nothing: padding slots, empty sequences
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        parts = layer.run(h, slots, table, lens, None, 1, kws)
    for step in range(5):
        h0 = torch.randn(2, HID, device="cuda", generator=g).half()
        h.copy_(h0)
        slots.copy_(ints(slot(s, n[s] + step) for s in range(2)))
        lens.copy_(ints(x + step + 1 for x in n))
        graph.replay()
        layer.check(h0, parts, slots, [slice(0, 1), slice(1, 2)], keys, values, rounded=False)
    q.check_error()
