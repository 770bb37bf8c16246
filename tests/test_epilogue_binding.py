"""What qmm_epilogue's binding refuses before the library is reached, without a GPU: tensors on
another device, views with gaps, and buffers smaller than the format reads."""
import pytest
import torch

import weight_only_quantized_int4_b200 as q

HERE = -1            # the device number of host tensors, taken as the current device here


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


class Library:
    def __init__(self):
        self.calls = []

    def qmm_epilogue(self, *a):
        self.calls.append(a)
        return 0

    qmm_kv_attend = qmm_epilogue


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(q, "_lib", fake)
    monkeypatch.setattr(q, "_cur_dev", lambda: HERE)
    monkeypatch.setattr(q, "_stream_of", lambda dev: 0)
    return fake


def _away(t):
    return torch.Tensor._make_subclass(Elsewhere, t)


def _half(n):
    return torch.zeros(n, dtype=torch.int16)


def _parts(mode, bits, N=64, K=256, group=64):
    G = 1 if group == -1 else K // group
    zl = {"sym": None, "asym": _half(N * G), "lut": _half(2 ** bits)}[mode]
    return dict(x=torch.zeros(3, K, dtype=torch.float16), qweight=torch.zeros(N * K * bits // 8, dtype=torch.uint8),
                scales=_half(N * G), zeros_or_lut=zl, N=N, K=K, mode=mode, bits=bits, group=group,
                ws=torch.zeros(4096, dtype=torch.uint8))


FORMATS = [("sym", 4, 64), ("asym", 4, 64), ("asym", 4, -1), ("lut", 4, 64), ("lut", 3, 128), ("lut", 2, -1)]


@pytest.mark.parametrize("mode,bits,group", FORMATS)
def test_exact_sizes_are_taken(lib, mode, bits, group):
    p = _parts(mode, bits, group=group)
    y = q.qmm_epilogue(**p)
    assert len(lib.calls) == 1 and tuple(y.shape) == (3, 64)
    assert lib.calls[0][4] == (None if mode == "sym" else p["zeros_or_lut"].data_ptr())
    q.qmm_epilogue(**dict(p, ws=None))
    bigger = dict(p, scales=_half(10000), qweight=torch.zeros(1 << 16, dtype=torch.uint8))
    q.qmm_epilogue(**bigger)                        # the first part of a larger buffer
    assert len(lib.calls) == 3


@pytest.mark.parametrize("mode,bits,group", FORMATS)
@pytest.mark.parametrize("what", ["qweight", "scales", "zeros_or_lut", "ws"])
@pytest.mark.parametrize("how", ["elsewhere", "gaps", "short"])
def test_refused(lib, mode, bits, group, what, how):
    p = _parts(mode, bits, group=group)
    t = p[what]
    if t is None or (what, how) == ("ws", "short"):   # the library knows a workspace's size
        return
    bad = {"elsewhere": lambda: _away(t), "gaps": lambda: torch.stack([t, t], 1)[:, 0],
           "short": lambda: t[:-1].clone()}[how]()
    with pytest.raises(ValueError, match=what.split("_or_")[0]):
        q.qmm_epilogue(**dict(p, **{what: bad}))
    assert not lib.calls


def test_symmetric_codes_pass_no_zero_points(lib):
    """A tensor that the format does not read never reaches the library."""
    p = _parts("sym", 4)
    q.qmm_epilogue(**dict(p, zeros_or_lut=_away(_half(4))))
    assert lib.calls[0][4] is None


def test_scales_of_larger_groups_are_refused(lib):
    p = _parts("asym", 4, group=128)
    with pytest.raises(ValueError, match="scales"):
        q.qmm_epilogue(**dict(p, group=64))
    assert not lib.calls


def test_attention_refuses_a_workspace_with_gaps(lib, monkeypatch):
    monkeypatch.setattr(q, "_cache_shape", lambda *a: (4, 2, 64, 0))
    qq, one = torch.zeros(1, 4, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    args = (qq, torch.zeros(1, dtype=torch.uint8), one[None], one)
    q.kv_attend(*args, ws=torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws"):
        q.kv_attend(*args, ws=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])
    with pytest.raises(ValueError, match="ws"):
        q.kv_attend(*args, ws=_away(torch.zeros(64, dtype=torch.uint8)))
    assert len(lib.calls) == 1
