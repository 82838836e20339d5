"""Refusals of the one-token products, the expert sort and rows, and the experts' products: host checks that need no
GPU. Every call fails validation before it touches the device."""
import ctypes

import pytest
import torch

from weight_only_quantization_act_b200 import awq, build

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)
ODD1 = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return awq.load_library()


def test_gemv_refusals(lib):
    def call(X=FAKE, M=1, K=256, ldx=256, codes=FAKE, steps=FAKE, zeros=FAKE, O=64, bias=None, gated=0, Y=FAKE, ldy=64):
        return lib.awq_w4a16_gemv(X, M, K, ldx, codes, steps, zeros, O, bias, gated, Y, ldy, None)

    assert call(X=None) == 1 and call(X=ODD) == 1 and call(codes=None) == 1 and call(codes=ODD) == 1
    assert call(steps=None) == 1 and call(zeros=None) == 1 and call(steps=ODD) == 1
    assert call(M=0) == 1 and call(M=-1) == 1 and call(O=0) == 1 and call(O=1 << 31) == 1
    assert call(K=200, ldx=200) == 1 and call(K=0) == 1 and call(ldx=128) == 1 and call(ldx=260) == 1
    assert call(M=9) == 1 and "awq_w4a16_gemm" in lib.awq_last_error().decode()
    assert call(Y=None) == 1 and call(Y=ODD1) == 1 and call(M=2, ldy=63) == 1
    assert call(gated=1, O=63) == 1 and call(gated=2) == 1 and call(gated=1, bias=FAKE) == 1 and call(bias=ODD1) == 1


def test_sort_refusals(lib):
    def call(ids=FAKE, size=4, n=100, E=8, ws=None, wsb=0, offsets=FAKE, order=FAKE, pos=FAKE):
        return lib.awq_expert_sort(ids, size, n, E, ws, wsb, offsets, order, pos, None)

    assert call(size=2) == 1 and call(ids=None) == 1 and call(ids=ODD) == 1
    assert call(ids=ctypes.c_void_p((1 << 20) + 4), size=8) == 1
    assert call(n=0) == 1 and call(n=1 << 31) == 1 and call(E=0) == 1 and call(E=1025) == 1
    assert call(offsets=None) == 1 and call(order=None) == 1 and call(pos=None) == 1 and call(pos=ODD) == 1
    assert call(n=5000) == 3 and call(n=5000, ws=FAKE, wsb=4) == 3
    assert call(n=5000, ws=ODD, wsb=1 << 20) == 1
    assert lib.awq_expert_sort_workspace_size(4096, 8) == 0
    assert lib.awq_expert_sort_workspace_size(4097, 8) >= 2 * 8 * 4
    assert lib.awq_expert_sort_workspace_size(0, 8) == 0 and lib.awq_expert_sort_workspace_size(1 << 20, 1025) == 0


def test_row_refusals(lib):
    def gather(X=FAKE, T=4, K=64, ldx=64, k=2, offsets=FAKE, E=8, order=FAKE, scales=None, Xs=FAKE, ldxs=64):
        return lib.awq_expert_gather(X, T, K, ldx, k, offsets, E, order, scales, Xs, ldxs, None)

    def gather_back(dXs=FAKE, T=4, K=64, ld=64, k=2, offsets=FAKE, E=8, pos=FAKE, scales=None, dX=FAKE, lddx=64):
        return lib.awq_expert_gather_backward(dXs, T, K, ld, k, offsets, E, pos, scales, dX, lddx, None)

    def combine(Ys=FAKE, T=4, O=64, ld=64, k=2, pos=FAKE, weights=FAKE, Y=FAKE, ldy=64):
        return lib.awq_expert_combine(Ys, T, O, ld, k, pos, weights, Y, ldy, None)

    def back(dY=FAKE, T=4, O=64, lddy=64, Ys=FAKE, ldys=64, k=2, pos=FAKE, weights=FAKE, dYs=FAKE, lddys=64, dw=FAKE):
        return lib.awq_expert_combine_backward(dY, T, O, lddy, Ys, ldys, k, pos, weights, dYs, lddys, dw, None)

    assert gather(X=None) == 1 and gather(X=ODD) == 1 and gather(T=0) == 1 and gather(k=0) == 1
    assert gather(K=60, ldx=64, ldxs=64) == 1 and gather(ldx=63) == 1 and gather(ldxs=56) == 1 and gather(Xs=None) == 1
    assert gather(offsets=None) == 1 and gather(order=None) == 1 and gather(E=0) == 1 and gather(E=1025) == 1
    assert gather(scales=ODD) == 1 and gather(T=1 << 30, k=2) == 1
    assert gather_back(dXs=None) == 1 and gather_back(pos=None) == 1 and gather_back(offsets=None) == 1
    assert gather_back(dX=ODD) == 1 and gather_back(scales=ODD) == 1 and gather_back(k=0) == 1
    assert combine(Ys=None) == 1 and combine(Y=None) == 1 and combine(pos=None) == 1 and combine(O=60) == 1
    assert combine(ldy=56) == 1 and combine(k=0) == 1 and combine(T=0) == 1
    assert back(dY=None) == 1 and back(Ys=None) == 1 and back(dYs=ODD) == 1 and back(dw=None) == 1
    assert back(weights=None) == 1 and back(pos=None) == 1 and back(lddys=8) == 1


def test_experts_refusals(lib):
    def call(X=FAKE, R=4, K=256, ldx=256, offsets=FAKE, E=8, codes=FAKE, steps=FAKE, zeros=FAKE, O=64, gated=0, Y=FAKE,
             ldy=64, ws=FAKE, wsb=1 << 30):
        return lib.awq_w4a16_experts(X, R, K, ldx, offsets, E, codes, steps, zeros, O, gated, Y, ldy, ws, wsb, None)

    assert call(X=None) == 1 and call(X=ODD) == 1 and call(R=0) == 1 and call(offsets=None) == 1
    assert call(E=0) == 1 and call(E=1025) == 1 and call(K=192, ldx=192) == 1 and call(ldx=200) == 1
    assert call(codes=ODD) == 1 and call(zeros=ODD) == 1 and call(O=0) == 1 and call(O=63, gated=1) == 1
    assert call(Y=None) == 1 and call(ldy=63) == 1 and call(gated=3) == 1
    assert call(ws=None) == 3 and call(wsb=8) == 3 and call(ws=ODD) == 1
    # refused before anything is launched, whichever of the two kernels would refuse it
    assert call(R=9, E=1024, O=1 << 21, ldy=1 << 21) == 1 and "too many" in lib.awq_last_error().decode()
    assert call(R=(1 << 31) - 1, E=1024, O=1 << 20, ldy=1 << 20) == 1 and "too many" in lib.awq_last_error().decode()
    assert call(O=1 << 24, ldy=1 << 24) == 1 and "too large" in lib.awq_last_error().decode()
    assert lib.awq_w4a16_experts_workspace_size(4, 8, 256, 64) >= 16
    assert lib.awq_w4a16_experts_workspace_size(4, 0, 256, 64) == 0


def test_binding_refusals():
    cpu = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes, steps = torch.zeros(8, 32, dtype=torch.int32), torch.zeros(8, 2)
    for call in (lambda: awq.w4a16_gemv(cpu, codes, steps, steps), lambda: awq.w4a16_experts(cpu, steps, codes[None], steps, steps),
                 lambda: awq.expert_sort(torch.zeros(2, 2, dtype=torch.int64), 4), lambda: awq.expert_sort([[0]], 4),
                 lambda: awq.expert_gather(cpu, None), lambda: awq.expert_combine(cpu, None),
                 lambda: awq.expert_gather_backward(cpu, None), lambda: awq.expert_combine_backward(cpu, cpu, None, steps)):
        with pytest.raises(TypeError):
            call()


class _Elsewhere(torch.Tensor):
    """A tensor that says it lives on a CUDA device."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 5))

    def get_device(self):
        return 5


def test_device_of_arguments_given_by_name(monkeypatch):
    seen = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(self.device)

        def __exit__(self, *_):
            return False

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    ids = torch.zeros(2, 2, dtype=torch.int64).as_subclass(_Elsewhere)
    call = awq._on_stream(lambda ids, n_experts: n_experts)
    for run in (lambda: call(ids, 4), lambda: call(ids, n_experts=4), lambda: call(n_experts=4, ids=ids)):
        seen.clear()
        assert run() == 4 and seen == [torch.device("cuda", 5)]


def test_workspace_refusals():
    cpu = torch.device("cpu")
    awq._on_device("workspace", torch.zeros(4), cpu)
    for bad in (torch.zeros(4, 4).t(), torch.zeros(4, device="meta"), [0], None):
        with pytest.raises(ValueError):
            awq._on_device("workspace", bad, cpu)
