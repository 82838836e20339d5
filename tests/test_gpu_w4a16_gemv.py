"""One-token products with packed 4-bit weights (awq.w4a16_gemv) against 64 bits."""
import pytest
import torch

from tests import _experts_plain as plain
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


def activations(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, ::97] *= 20
    return x.bfloat16()


def on_gpu(*tensors):
    return tuple(t.cuda() for t in tensors)


# K: one group (one slice), an odd number of groups, slices that end inside a ring stage, more groups than one
# chunk of X holds; O: one row, a row block and one row, ragged ends, odd
@pytest.mark.parametrize("M,K,O", [(1, 128, 1), (1, 128, 8), (8, 256, 129), (3, 640, 200), (1, 1920, 384),
                                   (5, 4224, 77), (8, 9600, 257), (2, 28672, 130), (7, 33408, 40), (4, 4096, 4096),
                                   (6, 1152, 20001)])
def test_gemv_matches_plain(M, K, O):
    X = activations(M, K, M + K)
    W = plain.packed(O, K, K + O)
    ref, err = plain.product(X, *W)
    Y = awq.w4a16_gemv(X.cuda(), *on_gpu(*W))
    assert Y.dtype == torch.bfloat16 and tuple(Y.shape) == (M, O)
    plain.assert_within(Y, ref, err)


@pytest.mark.parametrize("M,K,O", [(1, 128, 2), (8, 384, 258), (1, 4096, 2064), (5, 4224, 1030), (3, 14336, 66)])
def test_gemv_gated_matches_plain(M, K, O):
    X = activations(M, K, M + K) * 0.2
    W = plain.packed(O, K, K + O)
    Y = awq.w4a16_gemv(X.cuda(), *on_gpu(*W), gated=True)
    assert tuple(Y.shape) == (M, O // 2)
    plain.assert_within(Y, *plain.gate(*plain.product(X, *W)))


@pytest.mark.parametrize("M,K,O", [(1, 512, 100), (8, 1408, 640)])
def test_gemv_bias(M, K, O):
    X, W = activations(M, K, 5), plain.packed(O, K, 6)
    bias = (100 * torch.randn(O, generator=torch.Generator().manual_seed(7))).bfloat16()
    ref, err = plain.product(X, *W)
    Y = awq.w4a16_gemv(X.cuda(), *on_gpu(*W), bias=bias.cuda())
    ref = ref + bias.double()
    plain.assert_within(Y, ref, err + 2.0 ** -24 * (ref.abs() + err))


def test_gemv_wild_steps_and_zero_points():
    """Zero points far outside the codes' range and steps over five decades."""
    X, W = activations(4, 1280, 8), plain.packed(300, 1280, 9, wild=True)
    plain.assert_within(awq.w4a16_gemv(X.cuda(), *on_gpu(*W)), *plain.product(X, *W))


@pytest.mark.parametrize("K,O", [(128, 48), (384, 140), (4096, 24), (33408, 16)])
def test_gemv_one_hot_is_exact(K, O):
    """A token with a single power-of-two entry gets exactly bf16(x RN32((q - z) step)): every nibble, the
    operand order, the group's step and zero point, the slices. Every in-feature of the first groups and of the last."""
    W = plain.packed(O, K, K)
    deq = plain.dequantized(*W).float()  # one rounding of the exact product
    Wd = on_gpu(*W)
    features = sorted(set(list(range(min(K, 256))) + list(range(K - 128, K)) + list(range(0, K, 1027))))
    for at in range(0, len(features), 8):
        ks = features[at:at + 8]
        X = torch.zeros(len(ks), K)
        for m, k in enumerate(ks):
            X[m, k] = 2.0 ** (m - 3)
        want = torch.stack([deq[:, k] * 2.0 ** (m - 3) for m, k in enumerate(ks)]).bfloat16()
        assert torch.equal(awq.w4a16_gemv(X.bfloat16().cuda(), *Wd).cpu(), want), ks


def test_gemv_strided_rows_output_and_neighbours():
    """X rows and Y rows inside wider matrices; what lies beside and behind the output stays."""
    X, W = activations(5, 896, 10), plain.packed(203, 896, 11)
    wide = torch.zeros(5, 896 + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:904] = X.cuda()
    buf = torch.full((7, 211), 7.0, dtype=torch.bfloat16, device="cuda")
    Wd = on_gpu(*W)
    out = buf[1:6, 3:206]
    assert awq.w4a16_gemv(wide[:, 8:904], *Wd, out=out) is out
    plain.assert_within(out, *plain.product(X, *W))
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:6, 3:206] = False
    assert bool((buf[keep] == 7.0).all())
    assert torch.equal(out, awq.w4a16_gemv(X.cuda(), *Wd))
    # a column-strided X is copied
    assert torch.equal(out, awq.w4a16_gemv(X.t().contiguous().cuda().t(), *Wd))


def test_gemv_unaligned_parameters():
    """steps and zeros need 4-byte alignment only."""
    X, (codes, steps, zeros) = activations(2, 512, 12), plain.packed(40, 512, 13)
    shifted = []
    for t in (steps, zeros):
        buf = torch.zeros(t.numel() + 1, device="cuda")
        buf[1:] = t.reshape(-1).cuda()
        shifted.append(buf[1:].view(t.shape))
    Y = awq.w4a16_gemv(X.cuda(), codes.cuda(), *shifted)
    assert torch.equal(Y, awq.w4a16_gemv(X.cuda(), codes.cuda(), steps.cuda(), zeros.cuda()))


def test_gemv_same_bits_every_time_and_on_every_path():
    """Repeated calls, two calls at once on two streams, a captured and replayed call, and a token alone or among others
    give the same bits."""
    X, W = activations(8, 4096, 14).cuda(), on_gpu(*plain.packed(1500, 4096, 15))
    want = awq.w4a16_gemv(X, *W)
    for _ in range(10):
        assert torch.equal(awq.w4a16_gemv(X, *W), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [awq.w4a16_gemv(X, *W, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    out, held = torch.empty_like(want), X.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.w4a16_gemv(held, *W, out=out)
    held.copy_(X.flip(0))
    graph.replay()
    assert torch.equal(out, want.flip(0))
    for m in (0, 7):  # the slices do not depend on the number of tokens
        assert torch.equal(awq.w4a16_gemv(X[m:m + 1], *W), want[m:m + 1])


def test_gemv_agrees_with_the_few_token_gemm():
    X, W = activations(8, 2048, 16), plain.packed(512, 2048, 17)
    ref, err = plain.product(X, *W)
    plain.assert_within(awq.w4a16_gemm(X.cuda(), *on_gpu(*W)), ref, err + 2.0 ** -23 * (X.double().abs() @ plain.dequantized(*W).abs().T))
    plain.assert_within(awq.w4a16_gemv(X.cuda(), *on_gpu(*W)), ref, err)
