"""The layers' calls run with the layer's device current, whichever was before, and leave
that one current (no GPU: two devices are made up, and the library's calls recorded)."""

from types import SimpleNamespace

import pytest
import torch

import fp8_quantized_gemm_amd as bsq
from fp8_quantized_gemm_amd import mlp, moe

T, HD, F = 16, 32, 48


class _Buffer:
    """A tensor as far as the layers look at one."""
    dtype, shape = torch.bfloat16, (T, HD)

    def __init__(self, dev):
        self.device = dev

    data_ptr = numel = lambda self: 0
    is_contiguous = lambda self: True


@pytest.fixture
def devices(monkeypatch):
    now = SimpleNamespace(index=0, seen=[])

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now.index = now.index, self.dev.index

        def __exit__(self, *_):
            now.index = self.before

    class Lib:
        def __getattr__(self, name):
            return lambda *a: now.seen.append((name, now.index)) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now.index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: SimpleNamespace(cuda_stream=0))
    now.lib = Lib()
    return now


def _mlp(devices, fmt, optimizer):
    L = mlp.MLPLayer.__new__(mlp.MLPLayer)
    L.lib, L.dev, L.fmt, L.optimizer = devices.lib, torch.device("cuda", 1), fmt, optimizer
    L.T, L.Hd, L.F, L.it, L.rht, L.signs, L.seed, L.lr, L.xb = T, HD, F, 0, 0, 0, 0, 1e-3, {}
    b = _Buffer(L.dev)

    class Any(dict):
        def __missing__(self, key):
            return b
    L.q = {n: Any() for n in ("X", "W_gu", "H", "W_down", "dY_down", "dY_gu")}
    L.wbf, L.wamax, L.w32, L.grad, L.momentum, L.act = (Any() for _ in range(6))
    L.q_ws = L.muon_ws = b
    L.muon, L.muon_coefs, L.stack = mlp.muon_options(None), None, {"W_gu": (2, F, HD), "W_down": (1, HD, F)}
    return L, b


@pytest.mark.parametrize("optimizer", ["sgd", "muon"])
@pytest.mark.parametrize("fmt", ["int8", "nvfp4"])
@pytest.mark.parametrize("before", [0, 1])
def test_mlp_layer(devices, fmt, optimizer, before):
    L, b = _mlp(devices, fmt, optimizer)
    devices.index = before
    L.step(b, b)
    assert len(devices.seen) >= 16 and {i for _, i in devices.seen} == {1}, devices.seen
    devices.seen.clear()
    L._update("W_gu", 0.0)                                   # as the constructor does
    assert devices.seen == [("master_weight_update", 1)] and devices.index == before


def test_the_device_before_is_restored_after_an_error(devices):
    L, b = _mlp(devices, "int8", "sgd")
    with pytest.raises(ValueError):
        L.forward(SimpleNamespace(shape=(1, 1)))
    assert devices.index == 0


def test_moe_layer(devices, monkeypatch):
    L = moe.MoELayer.__new__(moe.MoELayer)
    L.dev, L.optimizer, L.lr, L.it = torch.device("cuda", 1), "sgd", 1e-3, 0
    L.w32, L.grad, L.wbf, L.wamax = {"W_gu": 0}, {"W_gu": 0}, {"W_gu": 0}, {}
    L.norm, L.saved = dict(w_pre=0), dict(r=0, o=0, rstd_pre=0, rstd_post=0, kw={})

    def call(name, **out):
        def f(*a, **k):
            devices.seen.append((name, devices.index))
            return dict(r=0, h=0, rstd_pre=0, rstd_post=0, amax=0, **out)
        monkeypatch.setattr(moe, name, f)
    for name in ("master_weight_update", "block_norm", "block_norm_backward"):
        call(name)

    def stop(name):
        def f(*a, **k):
            devices.seen.append((name, devices.index))
            raise KeyError(name)
        monkeypatch.setattr(moe, name, f)
    stop("moe_route")
    stop("moe_combine_backward")
    L.open(0, 0), L.close(0, 0), L.update(), L._update("W_gu", 0.0)
    L.k = L.bias = L.score_bias = L.y_down = 0
    L.routing, L.route = {}, dict(src=0, row_of=0, weights=0)
    for f in (lambda: L.forward(0, 0), lambda: L.backward(0)):
        with pytest.raises(KeyError):
            f()
    assert [n for n, _ in devices.seen] == ["block_norm", "block_norm_backward", "master_weight_update", "master_weight_update",
                                            "moe_route", "moe_combine_backward"]
    assert {i for _, i in devices.seen} == {1} and devices.index == 0
