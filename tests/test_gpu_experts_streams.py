"""Calls on another stream than the tensors' own."""
import pytest
import torch

from tests import _experts_plain as plain
from tests.test_gpu_experts import expert_weights, normal, picks
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


def test_arguments_freed_after_the_call_are_not_reused_before_it():
    """The stream is busy for a while when the calls are made; their arguments are dropped and as much memory is taken and
    filled on the tensors' own stream before it gets to them."""
    T, k, E, K, I = 300, 2, 4, 512, 256
    _, gate_up = expert_weights(E, 2 * I, K, 140)
    _, down = expert_weights(E, K, I, 150)
    X, ids = normal((T, K), 160), picks(T, k, E, 161)
    weights = torch.rand(T, k, generator=torch.Generator().manual_seed(162))
    scales = torch.rand(E, K, generator=torch.Generator().manual_seed(163)) + 0.5
    W = plain.packed(600, K, 164)
    block = lambda **kw: awq.w4a16_moe(X.cuda(), ids.cuda(), weights.cuda(), tuple(t.clone() for t in gate_up),  # noqa: E731
                                       tuple(t.clone() for t in down), scales=scales.cuda(), **kw)
    vector = lambda **kw: awq.w4a16_gemv(X[:5].cuda(), *(t.cuda() for t in W), **kw)  # noqa: E731

    def gather(**kw):
        sort = awq.expert_sort(ids.cuda(), E)
        torch.cuda.current_stream().synchronize()
        return awq.expert_gather_backward(awq.expert_gather(X.cuda(), sort), sort, scales=scales.cuda(), **kw)

    for call in (block, vector, gather):
        want = call()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # about 0.1 s
        got = call(stream=side)
        taken = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
                 for n in [512, 2048, 4096, 8192, 1 << 16, 1 << 18, 1 << 19, 1 << 20] * 12]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del taken
