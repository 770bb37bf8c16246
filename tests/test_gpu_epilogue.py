"""qmm_epilogue, y = residual + act(x . W~^T + bias), against the oracle's 64-bit sums (needs a
B200).

Bound: the sum carries the parity tests' element bound (4e-3 sum |x||w~|, which the decode and
the tensor path keep); an activation passes an error on by at most its steepest slope (GELU 1.13,
its tanh form 1.13, SiLU 1.10, else 1); the fp32 additions and functions err by at most 2^-20 of
their terms, the store by half a step of y's type."""
import ctypes
import math

import numpy as np
import pytest
import torch

import weight_only_quantized_int4_b200 as q
from tests import cases

pytestmark = pytest.mark.gpu

SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.13, "silu": 1.1}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from weight_only_quantized_int4_b200 import build
    build.build()
    q.load()


def _act(v, act):
    t = torch.from_numpy(v)
    if act == "relu":
        t = t.clamp(min=0)
    elif act == "gelu":
        t = 0.5 * t * torch.special.erfc(-t / math.sqrt(2))
    elif act == "gelu_tanh":
        t = 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    elif act == "silu":
        t = t * torch.sigmoid(t)
    return t.numpy()


def _dev16(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def _run(p, act, bias, res, ws=True, y=None):
    tdt = TDT[p.xdtype]
    dev = dict(bias=None if bias is None else bias.to(tdt).cuda(), residual=None if res is None else res.to(tdt).cuda())
    w = q.workspace(p.M, p.N, p.K, p.mode, p.bits, p.group) if ws else None
    if y is not None:
        dev["residual"] = y.copy_(dev["residual"])
    out = q.qmm_epilogue(_dev16(p.x).view(tdt), torch.from_numpy(p.qw).cuda(), _dev16(p.sp), _dev16(p.zl), p.N, p.K,
                         p.mode, p.bits, p.group, act=act, ws=w, y=y, **dev)
    q.check_error()
    return out


def _check(out, p, act, bias, res, what):
    s, bound = cases.expected(p)
    tdt = TDT[p.xdtype]
    b = np.zeros(p.N) if bias is None else bias.to(tdt).double().numpy()
    r = np.zeros((p.M, p.N)) if res is None else res.to(tdt).double().numpy()
    ref = r + _act(s + b, act)
    lim = SLOPE[act] * bound + 2.0 ** -20 * (np.abs(s) + np.abs(b) + np.abs(r)) + HALF[p.xdtype] * np.abs(ref) + 2.0 ** -24
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= lim), f"{what}: {int((~(err <= lim)).sum())} over the bound, worst {np.nanmax(err / lim):.3f}"


def _extras(p, which, seed):
    g = torch.Generator().manual_seed(seed)
    bias = torch.randn(p.N, generator=g) if "b" in which else None
    res = torch.randn(p.M, p.N, generator=g) * 3 if "r" in which else None
    return bias, res


@pytest.mark.parametrize("act,which", [("none", "r"), ("none", "b"), ("relu", "br"), ("gelu", "b"), ("gelu_tanh", "br"),
                                       ("silu", ""), ("none", "")])
@pytest.mark.parametrize("mode,bits,group,xdtype", [("sym", 4, 128, "f16"), ("asym", 4, 64, "bf16"),
                                                    ("sym", 4, -1, "bf16"), ("lut", 4, 64, "f16")])
def test_acts_on_both_paths(mode, bits, group, xdtype, act, which):
    for M in (1, 20, 70):                            # decode tiles of 8 and 32 tokens, tensor path
        p = cases.make(mode, bits, group, M, 176, 512, xdtype, seed=M)
        bias, res = _extras(p, which, M)
        for ws in (True, False):
            _check(_run(p, act, bias, res, ws), p, act, bias, res, f"M {M} {act} {which} ws {ws}")


@pytest.mark.parametrize("mode,bits,group,M,N,K", [
    ("lut", 3, 64, 3, 272, 1024), ("lut", 2, 32, 17, 272, 1024), ("asym", 4, 32, 9, 16, 64),
    ("sym", 4, 64, 16, 9600, 1024),      # split K through the workspace
    ("sym", 4, 128, 40, 1040, 2048), ("asym", 4, 128, 129, 400, 4160), ("sym", 4, -1, 300, 272, 704),
    ("lut", 4, 64, 260, 144, 576), ("sym", 4, 128, 257, 4096, 1024)])
@pytest.mark.parametrize("xdtype", ["f16", "bf16"])
def test_odd_sizes(mode, bits, group, M, N, K, xdtype):
    if group != -1 and K % group:
        group = 64
    p = cases.make(mode, bits, group, M, N, K, xdtype, seed=N + M)
    bias, res = _extras(p, "br", N)
    _check(_run(p, "silu", bias, res), p, "silu", bias, res, f"{mode}{bits} {M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 33, 300])
def test_in_place_on_the_residual(M):
    p = cases.make("sym", 4, 128, M, 528, 1024, "f16", seed=3)
    bias, res = _extras(p, "br", 5)
    y = torch.empty(M, 528, dtype=torch.float16, device="cuda")
    out = _run(p, "none", bias, res, y=y)
    assert out.data_ptr() == y.data_ptr()
    apart = _run(p, "none", bias, res)
    assert torch.equal(out, apart)
    _check(out, p, "none", bias, res, f"in place M {M}")


@pytest.mark.parametrize("M", [1, 12, 30, 64, 200])
def test_nothing_added_is_qmm(M):
    """Without bias, activation and residual the bits are qmm's: same sums, same rounding."""
    p = cases.make("asym", 4, 128, M, 528, 1024, "bf16", seed=8)
    x, qw, sp, zl = _dev16(p.x).view(torch.bfloat16), torch.from_numpy(p.qw).cuda(), _dev16(p.sp), _dev16(p.zl)
    y = q.qmm(x, qw, sp, zl, p.N, p.K, p.mode, ws=q.workspace(M, p.N, p.K, p.mode))
    assert torch.equal(y, _run(p, "none", None, None))


def test_infinities_and_nan_stay_in_their_places():
    p = cases.make("sym", 4, 128, 2, 64, 128, "f16", seed=1)
    bias, res = _extras(p, "br", 1)
    bias[3], res[0, 5], res[1, 7], bias[9] = float("inf"), float("nan"), -float("inf"), -float("inf")
    out = _run(p, "relu", bias, res).float().cpu()
    assert torch.isposinf(out[:, 3]).all() and torch.isnan(out[0, 5]) and torch.isneginf(out[1, 7])
    assert torch.equal(out[:, 9], res.half().float()[:, 9])          # relu(-inf) = 0
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[:, 3] = ok[0, 5] = ok[1, 7] = False
    assert torch.isfinite(out[ok]).all()


def test_rows_around_y_are_untouched():
    for M in (3, 100):
        p = cases.make("sym", 4, 128, M, 272, 256, "f16", seed=2)
        bias, res = _extras(p, "br", 2)
        buf = torch.full((M + 2, 272), 7.0, dtype=torch.float16, device="cuda")
        _run(p, "gelu", bias, res, y=buf[1:M + 1])
        assert (buf[0] == 7.0).all() and (buf[M + 1] == 7.0).all()


def test_refusals():
    lib = q.load()
    P = ctypes.c_void_p
    A, Y = P(0x1000), P(0x900000)

    def call(bias=None, act=0, res=None, M=2, y=Y, mode=0, x=A):
        return lib.qmm_epilogue(x, 0, A, A, None, bias, act, res, M, 64, 64, 4, 64, mode, y, None, 0, None)

    assert call(M=0) == 0 and call(M=-1) == -1
    assert call(act=5) == -1 and call(act=-1) == -1 and call(mode=4) == -1
    assert call(bias=P(0x1001)) == -3 and call(res=P(0x1003)) == -3
    assert call(bias=P(0x900000 + 64)) == -1          # bias inside y
    assert call(res=P(0x900000 + 128)) == -1          # residual over y, not at it
    assert call(x=None) == -1 and call(y=None) == -1
    x = torch.zeros(2, 64, device="cuda", dtype=torch.float16)
    w = torch.zeros(64 * 32, device="cuda", dtype=torch.uint8)
    s = torch.zeros(64, device="cuda", dtype=torch.int16)
    for kw in (dict(act="tanh"), dict(bias=x[0, :32]), dict(bias=torch.zeros(64, device="cuda")),
               dict(residual=torch.zeros(64, 2, device="cuda", dtype=torch.float16).t()), dict(residual=x.cpu()),
               dict(y=torch.zeros(2, 32, device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            q.qmm_epilogue(x, w, s, None, 64, 64, "sym", 4, 64, **kw)


# ---- the activations by themselves: x = 0, so the sum is exactly 0 and y = act(bias)

def _act64(v, act):
    """The activation in 64 bits, its lower tail without cancellation."""
    if act == "gelu":
        return v * torch.exp(torch.special.log_ndtr(v))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v.clamp(min=0) if act == "relu" else v


def _act_bound(v, act, xdtype):
    """Half a step of the output's type around the activation's own error.  GELU: a fit off by 2^-22
    and ten fp32 operations, below 2^-19; the exponent v^2 / 2 in base 2 is rounded in three factors,
    3 2^-24 of it.  The forms v / (1 + e^w): the same 2^-19, and w is rounded in eight steps, 2^-21 of
    it; a denominator of 2^126 and more may give 0, which with |v| < 2^7 there is below 2^-119."""
    ref = _act64(v, act)
    w = {"gelu": 2.0 ** -23 * v ** 2, "silu": 2.0 ** -21 * v.abs(),
         "gelu_tanh": 2.0 ** -21 * 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3).abs()}
    own = ref.abs() * (2.0 ** -19 + w[act]) if act in w else torch.zeros_like(ref)
    return ref, own + HALF[xdtype] * (ref.abs() + own) + (2.0 ** -25 if xdtype == "f16" else 2.0 ** -134) + 2.0 ** -119


def _sweep(xdtype):
    near = torch.logspace(-7, 0, 496, dtype=torch.float64)
    far = torch.tensor([0.0, 14.0, -14.0, 20.0, -20.0, 100.0, -100.0, 1000.0, -1000.0, 6e4, -6e4] + [0.0] * 5,
                       dtype=torch.float64)
    v = torch.cat([torch.linspace(-13, 13, 2080, dtype=torch.float64), near, -near, far])
    return v.to(TDT[xdtype])


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("xdtype", ["f16", "bf16"])
def test_activation_of_the_bias_alone(xdtype, act):
    bias = _sweep(xdtype)
    N, K = bias.numel(), 128
    v = bias.double()
    ref, lim = _act_bound(v, act, xdtype)
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(1)).cuda()
    for mode, group in (("sym", 128), ("asym", -1)):
        qw, sc, ze = q.pack(W, mode, 4, group)
        for M in (1, 12, 30, 40, 200):               # decode tiles of 8, 16 and 32 tokens, tensor path
            x = torch.zeros(M, K, dtype=TDT[xdtype], device="cuda")
            y = q.qmm_epilogue(x, qw, sc, ze, N, K, mode, 4, group, bias=bias.cuda(), act=act,
                               ws=q.workspace(M, N, K, mode, 4, group))
            err = (y.double().cpu() - ref).abs()
            bad = ~(err <= lim)
            assert not bad.any(), (f"{mode} M {M}: {int(bad.sum())} over the bound, the worst "
                                   f"{float((err / lim).max()):.2f} of it at {float(v[(err / lim).max(0).values.argmax()])}")


@pytest.mark.parametrize("xdtype", ["f16", "bf16"])
def test_the_bound_tells_the_activations_apart(xdtype):
    """Each activation, rounded to the output's type, breaks every other one's bound."""
    v = _sweep(xdtype).double()
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        ref, lim = _act_bound(v, act, xdtype)
        for other in ("none", "relu", "gelu", "gelu_tanh", "silu"):
            y = _act64(v, other).to(TDT[xdtype]).double()
            assert ((y - ref).abs() <= lim).all() == (act == other), (act, other)


@pytest.mark.parametrize("M", [1, 20, 40, 129, 300])
def test_y_needs_no_alignment_beyond_its_type(M):
    """y, bias and residual that start 2 bytes past a 16-byte border, on both paths; what lies
    around y stays as it was."""
    p = cases.make("sym", 4, 128, M, 288, 1024, "f16", seed=M)
    bias, res = _extras(p, "br", M)
    want = _run(p, "silu", bias, res)

    def off(t):
        buf = torch.full((t.numel() + 17,), 7.0, dtype=torch.float16, device="cuda")
        view = buf[1:1 + t.numel()].view(t.shape)
        return buf, view.copy_(t)

    x, qw, sp = _dev16(p.x).view(torch.float16), torch.from_numpy(p.qw).cuda(), _dev16(p.sp)
    ws = q.workspace(M, p.N, p.K, p.mode)
    for w in (ws, None):
        buf, y = off(torch.zeros(M, p.N))
        kw = dict(bias=off(bias)[1], residual=off(res)[1], act="silu", y=y, ws=w)
        q.qmm_epilogue(x, qw, sp, None, p.N, p.K, p.mode, **kw)
        ref = want if w is ws else _run(p, "silu", bias, res, ws=False)
        assert torch.equal(y, ref) and (buf[0] == 7.0) and (buf[1 + y.numel():] == 7.0).all()
        buf, y = off(res)                            # and in place
        q.qmm_epilogue(x, qw, sp, None, p.N, p.K, p.mode, **dict(kw, residual=y, y=y))
        assert torch.equal(y, ref) and (buf[0] == 7.0) and (buf[1 + y.numel():] == 7.0).all()
        buf, y = off(torch.zeros(M, p.N))            # the product alone
        q.qmm(x, qw, sp, None, p.N, p.K, p.mode, y=y, ws=w)
        assert torch.equal(y, q.qmm(x, qw, sp, None, p.N, p.K, p.mode, ws=w))
        assert (buf[0] == 7.0) and (buf[1 + y.numel():] == 7.0).all()
        buf, y = off(torch.zeros(M, p.N // 2))       # and the gate's
        q.qmm_gated(x, qw, sp, None, p.N // 2, p.K, p.mode, y=y, ws=w)
        assert torch.equal(y, q.qmm_gated(x, qw, sp, None, p.N // 2, p.K, p.mode, ws=w))
        assert (buf[0] == 7.0) and (buf[1 + y.numel():] == 7.0).all()
