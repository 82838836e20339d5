"""Tokens sorted by expert and back, their gradients, the experts' products, and a block of them together."""
import numpy as np
import pytest
import torch

from oracle import awq_oracle as orc
from tests import _experts_plain as plain
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


def picks(T, k, E, seed, unrouted=0.1):
    """Expert ids with a crowded expert, empty ones, repeats within a token and ids that name no expert."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(T, k, generator=g) ** 2 * E).long().clamp(max=E - 1)
    ids[torch.rand(T, k, generator=g) < 0.2] = E // 2
    ids[torch.rand(T, k, generator=g) < unrouted] = -1
    ids[torch.rand(T, k, generator=g) < unrouted / 2] = E + 3
    return ids


def normal(shape, seed, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).bfloat16()


def sorted_on_gpu(ids, E):
    offsets, order, pos = plain.sort_slots(ids, E)
    return awq.ExpertSort(offsets.cuda(), order.cuda(), pos.cuda()), (offsets, order, pos)


# one slot; one expert; the most experts; the last size that one block sorts alone and the first of two kernels;
# blocks that end inside a tile
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 2, 8), (3, 2, 8), (33, 1, 5), (512, 8, 128), (2049, 2, 64),
                                   (4096, 1, 1024), (4097, 1, 1024), (5000, 6, 7), (40001, 8, 257)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, k, E, dtype):
    ids = picks(T, k, E, T + k + E)
    want = plain.sort_slots(ids, E)
    got = awq.expert_sort(ids.to(dtype).cuda(), E)
    for name, g, w in zip(("offsets", "order", "pos"), (got.offsets, got.order, got.pos), want):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), w), name


@pytest.mark.parametrize("T", [700, 9000])
def test_sort_extremes(T):
    for ids, E in ((torch.full((T, 1), -1), 4), (torch.full((T, 1), 3), 4), (torch.full((T, 1), 2 ** 40), 4),
                   (torch.arange(T)[:, None] % 2, 2)):
        got = awq.expert_sort(ids.cuda(), E)
        for g, w in zip((got.offsets, got.order, got.pos), plain.sort_slots(ids, E)):
            assert torch.equal(g.cpu(), w)
    # a matrix whose rows are not next to each other
    ids = picks(T, 4, 8, 1)
    got = awq.expert_sort(ids.cuda()[:, 1:3], 8)
    assert torch.equal(got.pos.cpu(), plain.sort_slots(ids[:, 1:3], 8)[2])


@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 8), (5, 3, 4, 200), (64, 2, 8, 1032), (37, 8, 16, 4096), (9, 40, 16, 136),
                                     (130, 2, 8, 9224)])
@pytest.mark.parametrize("scaled", [False, True])
def test_gather_bits_and_untouched_rows(T, k, E, K, scaled):
    ids = picks(T, k, E, T + K)
    sort, (offsets, order, _) = sorted_on_gpu(ids, E)
    X = normal((T, K), 3, 4.0)
    scales = torch.rand(E, K, generator=torch.Generator().manual_seed(4)) * 3 + 1e-3 if scaled else None
    out = torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    got = awq.expert_gather(X.cuda(), sort, scales=None if scales is None else scales.cuda(), out=out)
    assert got is out
    want = torch.full((T * k, K), 7.0, dtype=torch.bfloat16)
    R = int(offsets[-1])
    if R:
        rows = X[order[:R].long() // k]
        if scaled:  # one IEEE division, one rounding to bf16
            rows = (rows.float() / scales[plain.expert_of_rows(offsets)]).bfloat16()
        want[:R] = rows
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


def test_gather_divides_like_scale_columns():
    """Quotients at and around bf16 ties, tiny, huge and zero: the same bits as awq_scale_columns."""
    K = 1024
    X = torch.arange(0, 64 * K, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, K)
    X = torch.where(X.float().isfinite(), X, torch.tensor(1.0, dtype=torch.bfloat16))
    g = torch.Generator().manual_seed(5)
    scales = torch.exp(torch.randn(2, K, generator=g) * 4)
    scales[0, ::3] = 2.0 ** torch.randint(-100, 100, (scales[0, ::3].numel(),), generator=g)
    scales[1, ::2] = (torch.randint(1, 256, (K // 2,), generator=g) / 256)
    ids = torch.tensor([[0, 1]] * 64)
    sort, _ = sorted_on_gpu(ids, 2)
    got = awq.expert_gather(X.cuda(), sort, scales=scales.cuda())
    for e in range(2):
        want = awq.scale_columns(X.cuda(), scales[e].cuda(), divide=True)
        assert torch.equal(got[64 * e:64 * (e + 1)].view(torch.int16), want.view(torch.int16))
    want = orc.fold_columns(X.view(torch.int16).numpy().view(np.uint16), scales[1].numpy(), divide=True)
    assert np.array_equal(got[64:].cpu().view(torch.int16).numpy().view(np.uint16), want)


def plain_back(Ys, pos, weights, offsets=None, scales=None):
    """sum_j weight Ys[pos] (/ scales) in 64 bits, and the sum of the terms' sizes."""
    T, k = pos.shape
    y, size = torch.zeros(T, Ys.shape[1], dtype=torch.float64), torch.zeros(T, Ys.shape[1], dtype=torch.float64)
    expert = None if scales is None else plain.expert_of_rows(offsets)
    for t in range(T):
        for j in range(k):
            r = int(pos[t, j])
            if r >= 0:
                v = Ys[r].double() * (1.0 if weights is None else float(weights[t, j]))
                if scales is not None:
                    v = v / scales[expert[r]].double()
                y[t] += v
                size[t] += v.abs()
    return y, size


@pytest.mark.parametrize("T,k,E,O", [(1, 1, 1, 8), (6, 3, 4, 200), (65, 2, 8, 1032), (33, 8, 16, 4104), (9, 40, 16, 136)])
@pytest.mark.parametrize("kind", ["weights", "ones", "scales"])
def test_combine_and_gather_backward(T, k, E, O, kind):
    ids = picks(T, k, E, 2 * T + O)
    sort, (offsets, _, pos) = sorted_on_gpu(ids, E)
    Ys = normal((T * k, O), 6)
    R = int(offsets[-1])
    Yd = Ys.cuda()
    Yd[R:] = float("nan")  # rows behind the last are not read
    if kind == "scales":
        scales = torch.rand(E, O, generator=torch.Generator().manual_seed(7)) + 0.25
        got = awq.expert_gather_backward(Yd, sort, scales=scales.cuda())
        ref, size = plain_back(Ys, pos, None, offsets, scales)
    else:
        w = torch.randn(T, k, generator=torch.Generator().manual_seed(8)) if kind == "weights" else None
        got = awq.expert_combine(Yd, sort, weights=None if w is None else w.cuda())
        ref, size = plain_back(Ys, pos, w)
        if w is None:
            assert torch.equal(got, awq.expert_gather_backward(Yd, sort))
    plain.assert_within(got, ref, (k + 1) * 2.0 ** -24 * size)


@pytest.mark.parametrize("T,k,E,O", [(1, 1, 1, 8), (6, 3, 4, 200), (64, 2, 8, 1032), (21, 8, 16, 4104), (5, 40, 16, 136),
                                     (3, 2, 2, 14336)])
def test_combine_backward(T, k, E, O):
    ids = picks(T, k, E, 3 * T + O)
    sort, (offsets, order, pos) = sorted_on_gpu(ids, E)
    R = int(offsets[-1])
    Ys, dY = normal((T * k, O), 9), normal((T, O), 10)
    w = torch.randn(T, k, generator=torch.Generator().manual_seed(11))
    Yd = Ys.cuda()
    Yd[R:] = float("nan")
    out = torch.full((T * k, O), 7.0, dtype=torch.bfloat16, device="cuda")
    dYs, dw = awq.expert_combine_backward(dY.cuda(), Yd, sort, w.cuda(), out=out)
    assert dYs is out and bool((out[R:] == 7.0).all())
    slot = order[:R].long()
    plain.assert_within(dYs[:R], w.reshape(-1)[slot, None].double() * dY.double()[slot // k],
                        torch.zeros(R, O, dtype=torch.float64) + 2.0 ** -24 * w.abs().max())
    ref, size = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                terms = dY[t].double() * Ys[int(pos[t, j])].double()
                ref[t, j], size[t, j] = terms.sum(), terms.abs().sum()
    # a thread adds at most ceil(O / 8 / 128) * 8 products, then 5 butterfly steps and at most 8 warps
    steps = -(-O // 1024) * 8 + 13
    assert bool(((dw.cpu().double() - ref).abs() <= steps * 2.0 ** -24 * size).all())
    assert bool((dw.cpu()[pos < 0] == 0).all())


def test_gradients_against_differences():
    """Both maps are linear, so a difference over any step gives the gradient: weights and rows of combine, tokens of
    gather."""
    T, k, E, K = 7, 2, 4, 264
    ids = picks(T, k, E, 12, unrouted=0)
    sort, (offsets, order, pos) = sorted_on_gpu(ids.clamp(0, E - 1), E)
    Ys, dY, w = normal((T * k, K), 13).cuda(), normal((T, K), 14).cuda(), torch.rand(T, k).cuda() + 0.5
    dYs, dw = awq.expert_combine_backward(dY, Ys, sort, w)
    loss = lambda Y: (Y.double() * dY.double()).sum(1)  # noqa: E731  per token
    base = awq.expert_combine(Ys, sort, weights=w)
    room = lambda *ys: sum(2.0 ** -8 * (y.double().abs() * dY.double().abs()).sum(1) for y in ys)  # noqa: E731
    for j in range(k):
        step = torch.zeros_like(w)
        step[:, j] = 4.0
        moved = awq.expert_combine(Ys, sort, weights=w + step)
        # each Y is off by half a bf16 step
        assert bool((((loss(moved) - loss(base)) - 4.0 * dw[:, j].double()).abs() <= 1.01 * room(moved, base)).all())
    direction = normal((T * k, K), 15).cuda()
    moved = awq.expert_combine(direction, sort, weights=w)
    want = (dYs.double() * direction.double()).sum(1)[sort.pos.long()].sum(1)  # dYs itself is off by half a step
    slack = room(moved) + 2.0 ** -8 * (dYs.double() * direction.double()).abs().sum(1)[sort.pos.long()].sum(1)
    assert bool(((loss(moved) - want).abs() <= 1.01 * slack).all())
    scales = (torch.rand(E, K) + 0.5).cuda()
    dXs = normal((T * k, K), 16).cuda()
    dX = awq.expert_gather_backward(dXs, sort, scales=scales)
    X = normal((T, K), 17).cuda()
    Xs = awq.expert_gather(X, sort, scales=scales)
    left = (Xs.double() * dXs.double()).sum()
    right = (X.double() * dX.double()).sum()
    slack = 2.0 ** -8 * ((Xs.double() * dXs.double()).abs().sum() + (X.double() * dX.double()).abs().sum())
    assert abs(float(left - right)) <= 1.01 * float(slack)


def expert_weights(E, O, K, seed, wild=False):
    parts = [plain.packed(O, K, seed + e, wild) for e in range(E)]
    return parts, tuple(torch.stack([p[i] for p in parts]).cuda() for i in range(3))


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


FEW_ROWS = 8  # an expert with more rows takes q - z of a zero point beyond +-240 rounded to bf16


def check_experts(Xs, counts, parts, got, gated):
    """Each expert's rows against 64 bits."""
    edges = offsets_of(counts).tolist()
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        if b > a:
            ref, err = plain.product(Xs[a:b], *parts[e], rounded_far_zeros=b - a > FEW_ROWS)
            plain.assert_within(got[a:b], *(plain.gate(ref, err) if gated else (ref, err)))


# counts per expert: single rows, empty experts at either end, more rows than a pass takes, hundreds of rows for one
# expert beside experts with few, all rows in one; K and O odd in groups and rows
EXPERT_CASES = [([1], 128, 8), ([0, 1, 0], 384, 40), ([3, 0, 8, 9, 0, 17], 640, 129), ([1] * 20, 1152, 264),
                ([0, 250, 1, 0, 40], 512, 392), ([64, 65, 16, 15, 33], 896, 200), ([700], 256, 1032),
                ([257, 0, 511, 12], 1024, 256), ([5, 6, 7], 4224, 72)]


@pytest.mark.parametrize("counts,K,O", EXPERT_CASES)
@pytest.mark.parametrize("gated", [False, True])
def test_experts_match_plain(counts, K, O, gated):
    O += O % 2 if gated else 0
    E, R = len(counts), sum(counts)
    spare = 3  # rows behind the last routed one
    parts, W = expert_weights(E, O, K, K + O)
    Xs = normal((R + spare, K), 20, 0.3)
    Xs[:, ::61] *= 10
    out = torch.full((R + spare, O // 2 if gated else O), 7.0, dtype=torch.bfloat16, device="cuda")
    Xd = Xs.cuda()
    Xd[R:] = float("nan")
    ws = awq.w4a16_experts_workspace(W[0], R + spare)
    got = awq.w4a16_experts(Xd, offsets_of(counts).cuda(), *W, gated=gated, out=out, workspace=ws)
    assert got is out and bool((out[R:] == 7.0).all())
    check_experts(Xs, counts, parts, out, gated)
    again = awq.w4a16_experts(Xd, offsets_of(counts).cuda(), *W, gated=gated, workspace=ws)
    assert torch.equal(again[:R], out[:R])
    assert not bool(ws.any())  # nothing is left behind


def test_experts_without_a_row():
    _, W = expert_weights(3, 40, 256, 1)
    out = torch.full((5, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    awq.w4a16_experts(normal((5, 256), 2).cuda(), offsets_of([0, 0, 0]).cuda(), *W, out=out)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("counts", [[4, 9, 0, 30], [300, 2, 80, 0]])
def test_experts_wild_strided_streams_and_graph(counts):
    """Zero points far outside the codes, X and Y rows inside wider matrices, another stream, a captured call replayed on
    other rows and counts."""
    K, O, R = 768, 137, sum(counts)
    parts, W = expert_weights(4, O, K, 30, wild=True)
    Xs = normal((R, K), 31)
    wide = torch.zeros(R, K + 40, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + K] = Xs.cuda()
    buf = torch.full((R, O + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    offsets = offsets_of(counts).cuda()
    awq.w4a16_experts(wide[:, 16:16 + K], offsets, *W, out=buf[:, 5:5 + O])
    check_experts(Xs, counts, parts, buf[:, 5:5 + O], False)
    assert bool((buf[:, :5] == 7.0).all()) and bool((buf[:, 5 + O:] == 7.0).all())
    want = buf[:, 5:5 + O].contiguous()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [awq.w4a16_experts(Xs.cuda(), offsets, *W, stream=s) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    held, edges, out = torch.zeros_like(Xs, device="cuda"), torch.zeros_like(offsets), torch.empty_like(want)
    ws = awq.w4a16_experts_workspace(W[0], R)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.w4a16_experts(held, edges, *W, out=out, workspace=ws)
    for shift in (0, 1):
        held.copy_(Xs)
        edges.copy_(offsets_of(counts[shift:] + counts[:shift]))
        graph.replay()
        check_experts(Xs, counts[shift:] + counts[:shift], parts, out, False)


def test_sort_gather_combine_captured():
    """A captured sort, gather and combine replayed on other picks."""
    T, k, E, K = 3000, 2, 8, 136
    X = normal((T, K), 40).cuda()
    ids = picks(T, k, E, 41).cuda()
    w = torch.rand(T, k).cuda()

    def block():
        sort = awq.expert_sort(ids, E)
        return awq.expert_combine(awq.expert_gather(X, sort), sort, weights=w)

    block()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for seed in (42, 43):
        ids.copy_(picks(T, k, E, seed))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, block())
        total = (w.double() * ((ids >= 0) & (ids < E))).sum(1, keepdim=True)
        plain.assert_within(got, (X.double() * total).cpu(), (k + 1) * 2.0 ** -24 * (X.double().abs() * total).cpu())


def moe_plain(X, ids, weights, gate_up, down, scales):
    """The block in 64 bits, token by token."""
    Y = torch.zeros(X.shape, dtype=torch.float64)
    for e in range(len(gate_up)):
        wg, wd = plain.dequantized(*gate_up[e]), plain.dequantized(*down[e])
        x = X.double() / scales[e].double()
        a, b = (x @ wg.T).chunk(2, dim=1)
        y = (a / (1 + torch.exp(-a)) * b) @ wd.T
        Y += (weights.double() * (ids == e)).sum(1, keepdim=True) * y
    return Y


@pytest.mark.parametrize("T", [1, 6, 700])
def test_block_of_experts(T):
    """Sort, gather, gated products, down products and combine together: the same bits as the calls one by one, and within the
    four bf16 roundings between the products of 64 bits in the 2-norm."""
    E, k, K, I = 5, 2, 512, 384
    X = normal((T, K), 50)
    ids = picks(T, k, E, 51, unrouted=0.05)
    weights = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(52)), 1)
    scales = torch.rand(E, K, generator=torch.Generator().manual_seed(53)) + 0.5
    gp, gate_up = expert_weights(E, 2 * I, K, 54)
    dp, down = expert_weights(E, K, I, 64)
    args = (X.cuda(), ids.cuda(), weights.cuda(), gate_up, down)
    got = awq.w4a16_moe(*args, scales=scales.cuda())
    sort = awq.expert_sort(ids.cuda(), E)
    Xs = awq.expert_gather(X.cuda(), sort, scales=scales.cuda())
    H = awq.w4a16_experts(Xs, sort.offsets, *gate_up, gated=True)
    Ys = awq.w4a16_experts(H, sort.offsets, *down)
    assert torch.equal(got, awq.expert_combine(Ys, sort, weights=weights.cuda()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = awq.w4a16_moe(*args, scales=scales.cuda(), stream=side)
    side.synchronize()
    assert torch.equal(other, got)
    ref = moe_plain(X, ids, weights, gp, dp, scales)
    # half steps of the roundings that act on the result: the input's twice (the gate multiplies two products of it),
    # the gate's, the down product's and the sum's
    assert float((got.cpu().double() - ref).norm()) <= 5 * 2.0 ** -8 * float(ref.norm()) + 1e-30


def test_quantize_experts_matches_each_layer():
    """Every expert gets what quantize_layer gives on its own tokens; one without tokens is packed at scales of one; the
    result runs as a block."""
    T, k, E, K, O = 600, 2, 4, 256, 128
    X = normal((T, K), 70).cuda()
    X[:, 3] *= 30
    ids = torch.randint(0, 3, (T, k), generator=torch.Generator().manual_seed(71)).cuda()  # expert 3 gets none
    W = [normal((O, K), 72 + e, 0.02).cuda() for e in range(E)]
    out = awq.quantize_experts(X, ids, W)
    assert tuple(out["codes"].shape) == (E, O, K // 8) and tuple(out["scales"].shape) == (E, K)
    order = plain.sort_slots(ids.cpu(), E)[1]
    offsets = plain.sort_slots(ids.cpu(), E)[0].tolist()
    for e in range(3):
        rows = (order[offsets[e]:offsets[e + 1]].long() // k).cuda()
        one = awq.quantize_layer(X[rows], W[e])
        for name in ("scales", "codes", "steps", "zeros", "losses", "best_j"):
            assert torch.equal(out[name][e], one[name]), (e, name)
    assert bool((out["scales"][3] == 1).all()) and bool(out["losses"][3].isnan().all())
    assert torch.equal(out["codes"][3], awq.quantize_pack(W[3], out["scales"][3])[0])
    sort = awq.expert_sort(ids, E)
    Y = awq.w4a16_experts(awq.expert_gather(X, sort, scales=out["scales"]), sort.offsets, out["codes"], out["steps"],
                          out["zeros"])
    for e in range(3):
        a, b = offsets[e:e + 2]
        ref = X[(order[a:b].long() // k).cuda()].double() @ W[e].double().T
        mse = float(((Y[a:b].double() - ref) ** 2).mean())
        assert mse <= 1.25 * float(out["losses"][e].min()) + 2.0 ** -16 * float((ref ** 2).mean())


@pytest.mark.parametrize("counts", [[3, 8], [4, 30], [200, 5]])
@pytest.mark.parametrize("gated", [False, True])
def test_nonfinite_rows_stay_apart(counts, gated):
    """A row with an infinity or a NaN changes no other row's bits, and its own outputs say so."""
    K, O, R = 640, 136, sum(counts)
    _, W = expert_weights(2, O, K, 60)
    X = normal((R, K), 61).cuda()
    offsets = offsets_of(counts).cuda()
    clean = awq.w4a16_experts(X, offsets, *W, gated=gated)
    bad = {1: float("nan"), counts[0] - 1: float("inf"), R - 2: -float("inf")}
    for row, value in bad.items():
        X[row, 77 + row] = value
    got = awq.w4a16_experts(X, offsets, *W, gated=gated)
    others = [r for r in range(R) if r not in bad]
    assert torch.equal(got[others], clean[others])
    if not gated:  # (an infinite gate may leave silu(gate) = 0)
        assert not bool(torch.isfinite(got[list(bad)]).any())


def test_offsets_out_of_order_stay_inside():
    """Offsets that no sort gives, falling, negative and past the rows: nothing outside Y's rows and columns is written."""
    K, O, R = 256, 72, 40
    _, W = expert_weights(4, O, K, 62)
    X = normal((R, K), 63).cuda()
    for offsets in ([-5, 20, 3, 1000000000, 2], [40, 30, 20, 10, 0], [2147483647] * 5, [-2147483648, 0, 12, 7, 40]):
        buf = torch.full((R + 2, O + 2), 7.0, dtype=torch.bfloat16, device="cuda")
        awq.w4a16_experts(X, torch.tensor(offsets, dtype=torch.int32, device="cuda"), *W, out=buf[1:-1, 1:-1])
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[1:-1, 1:-1] = False
        assert bool((buf[keep] == 7.0).all())
