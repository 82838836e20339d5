"""A block of quantized experts whose down projections have scales of their own."""
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


@pytest.mark.parametrize("T", [1, 6, 300])
def test_block_with_scales_of_the_down_projections(T):
    E, k, K, I = 4, 2, 256, 384
    X = normal((T, K), 100)
    ids = picks(T, k, E, 101, unrouted=0.05)
    weights = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(102)), 1)
    g = torch.Generator().manual_seed(103)
    scales, down_scales = torch.rand(E, K, generator=g) + 0.5, torch.exp(torch.randn(E, I, generator=g))
    gp, gate_up = expert_weights(E, 2 * I, K, 104)
    dp, down = expert_weights(E, K, I, 114)
    args = (X.cuda(), ids.cuda(), weights.cuda(), gate_up, down)
    got = awq.w4a16_moe(*args, scales=scales.cuda(), down_scales=down_scales.cuda())
    ref = torch.zeros(X.shape, dtype=torch.float64)
    for e in range(E):
        a, b = (X.double() / scales[e].double() @ plain.dequantized(*gp[e]).T).chunk(2, dim=1)
        y = (a / (1 + torch.exp(-a)) * b / down_scales[e].double()) @ plain.dequantized(*dp[e]).T
        ref += (weights.double() * (ids == e)).sum(1, keepdim=True) * y
    # half steps of the roundings: the input's twice (the gate multiplies two products of it), the gate's, the division's, the
    # down product's and the sum's
    assert float((got.cpu().double() - ref).norm()) <= 6 * 2.0 ** -8 * float(ref.norm()) + 1e-30
    # each expert's rows divided as scale_columns does
    sort = awq.expert_sort(ids.cuda(), E)
    H = awq.w4a16_experts(awq.expert_gather(X.cuda(), sort, scales=scales.cuda()), sort.offsets, *gate_up, gated=True)
    edges = sort.offsets.tolist()
    for e in range(E):
        if edges[e + 1] > edges[e]:
            rows = H[edges[e]:edges[e + 1]]
            rows.copy_(awq.scale_columns(rows, down_scales[e].cuda(), divide=True))
    Ys = awq.w4a16_experts(H, sort.offsets, *down)
    assert torch.equal(got, awq.expert_combine(Ys, sort, weights=weights.cuda()))
    with pytest.raises(ValueError):
        awq.w4a16_moe(*args, down_scales=scales.cuda())


def test_block_as_the_quantizer_gives_it():
    """Both projections as quantize_experts packs them, each with its scales: closer to the float block than with the down
    projections' scales left out, which cannot be right where a channel is large."""
    T, k, E, K, I = 400, 2, 3, 256, 256
    X = normal((T, K), 120).cuda()
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(121)).cuda()
    weights = torch.rand(T, k, generator=torch.Generator().manual_seed(122)).cuda()
    W = [normal((2 * I, K), 123 + e, 0.05) for e in range(E)]
    for w in W:
        w[I + 7] *= 40  # a large channel of H
    W = [w.cuda() for w in W]
    D = [normal((K, I), 133 + e, 0.05).cuda() for e in range(E)]
    q = awq.quantize_experts(X, ids, W)
    sort = awq.expert_sort(ids, E)
    token = sort.order.long() // k
    rows = X[token].double()
    expert = ids.reshape(-1)[sort.order.long()]
    H = torch.empty(T * k, I, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = (rows[expert == e] @ W[e].double().T).chunk(2, dim=1)
        H[expert == e] = a / (1 + torch.exp(-a)) * b
    d = awq.quantize_experts(H.bfloat16(), expert[:, None], D)
    assert float((d["scales"] - 1).abs().max()) > 0.1
    ref = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        at = expert == e
        w = weights.reshape(-1)[sort.order.long()][at].double()
        ref.index_add_(0, token[at], w[:, None] * (H[at] @ D[e].double().T))
    parts = lambda p: (p["codes"], p["steps"], p["zeros"])  # noqa: E731
    off = lambda y: float((y.double() - ref).norm())  # noqa: E731
    got = awq.w4a16_moe(X, ids, weights, parts(q), parts(d), scales=q["scales"], down_scales=d["scales"])
    assert off(got) < 0.5 * off(awq.w4a16_moe(X, ids, weights, parts(q), parts(d), scales=q["scales"]))
