"""What the products' bounds alone would not show: the experts' products and the products of a few tokens at inputs where a
kernel's own way of summing could be seen."""
import pytest
import torch

from tests import _experts_plain as plain
from tests import _products_bounds as bounds
from tests.test_gpu_experts import expert_weights, normal, offsets_of
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


def by_definition(X, codes, steps, zeros, gated):
    """Products in 64 bits term by term, so that an infinity meets each weight by itself."""
    P = torch.stack([(x.double() * plain.dequantized(codes, steps, zeros)).sum(1) for x in X])
    if not gated:
        return P
    a, b = P.chunk(2, dim=1)
    return a / (1 + torch.exp(-a)) * b


# rows of the one expert: the few-token kernel up to 8, the grouped one beyond; several slices at K = 4096
@pytest.mark.parametrize("rows", [1, 3, 8, 9, 40])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [640, 4096])
def test_infinities_are_those_of_the_definition(rows, gated, K):
    """An infinity in X gives each output the sign of its weight, a NaN where the weight is zero or where two infinities
    meet; the other tokens keep their bits. The same for an expert's rows and for one layer."""
    O = 150
    parts, W = expert_weights(1, O, K, 90)
    X = normal((rows, K), 91)
    clean = awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), *W, gated=gated)
    X[0, 77] = float("inf")
    if rows > 1:
        X[1, K - 3] = -float("inf")
    if rows > 2:
        X[2, 5], X[2, K - 130] = float("inf"), float("inf")
    bad = min(rows, 3)
    ref = by_definition(X[:bad], *parts[0], gated)
    calls = [awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), *W, gated=gated)]
    if rows <= awq.GEMV_MAX_TOKENS:
        calls.append(awq.w4a16_gemv(X.cuda(), *(t[0] for t in W), gated=gated))
    for got in calls:
        assert torch.equal(got[bad:], clean[bad:])
        got = got[:bad].double().cpu()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.isinf(), ref.isinf())
        assert torch.equal(got[ref.isinf()], ref[ref.isinf()])
    assert bool(ref.isinf().any())  # the case shows it: not every output is a NaN


def weights_around_zero(O, K, seed):
    """Codes and zero points as packing gives them for normal weights."""
    codes, steps, zeros = plain.packed(O, K, seed)
    return codes, steps, torch.where(zeros > 7, 8.0, 7.0)


@pytest.mark.parametrize("M,K,O", [(1, 4096, 4096), (8, 28672, 520), (3, 33408, 1400), (5, 1408, 2000), (8, 128, 1000)])
@pytest.mark.parametrize("one_sided", [False, True])
def test_few_tokens_lose_nothing_before_the_rounding(M, K, O, one_sided):
    """Centred activations and those of a ReLU, which are all of one sign: the sums of x do not cancel there."""
    X = normal((M, K), 92).abs() if one_sided else normal((M, K), 92)
    W = weights_around_zero(O, K, 93)
    ref, err = bounds.few(X, *W)
    got = awq.w4a16_gemv(X.cuda(), *(t.cuda() for t in W))
    bounds.assert_rounds(got, ref)
    plain.assert_within(got, ref, err)


def test_few_rows_of_experts_lose_nothing_before_the_rounding():
    counts, K, O = [1, 8, 0, 5], 14336, 600
    parts = [weights_around_zero(O, K, 94 + e) for e in range(4)]
    W = tuple(torch.stack([p[i] for p in parts]).cuda() for i in range(3))
    X = normal((14, K), 95).abs()
    got = awq.w4a16_experts(X.cuda(), offsets_of(counts).cuda(), *W)
    for e, (a, b) in enumerate(((0, 1), (1, 9), (9, 9), (9, 14))):
        if b > a:
            bounds.assert_rounds(got[a:b], bounds.few(X[a:b], *parts[e])[0])


def test_few_tokens_of_any_size():
    """Powers of two in X come out as they went in; the largest and the smallest stay within the bound."""
    M, K, O = 4, 768, 300
    X, W = normal((M, K), 96), plain.packed(O, K, 97)
    Wd = tuple(t.cuda() for t in W)
    base = awq.w4a16_gemv(X.cuda(), *Wd)
    for k in (-96, -40, 60, 112):
        assert torch.equal(awq.w4a16_gemv((X.double() * 2.0 ** k).bfloat16().cuda(), *Wd).double(), base.double() * 2.0 ** k), k
    for k in (-128, -118, 117, 121):
        Xk = (X.double() * 2.0 ** k).bfloat16()
        ref, err = bounds.few(Xk, *W)
        plain.assert_within(awq.w4a16_gemv(Xk.cuda(), *Wd), ref, torch.maximum(err, bounds.term_by_term(Xk, *W)[1]))
    # one token large, the others keep their bits; one group large, the others of the token count
    X2 = X.clone()
    X2[1, 200] = 2.0 ** 119
    got = awq.w4a16_gemv(X2.cuda(), *Wd)
    assert torch.equal(got[[0, 2, 3]], base[[0, 2, 3]])
    ref, err = bounds.term_by_term(X2[1:2], *W)
    plain.assert_within(got[1:2], ref, err)


@pytest.mark.parametrize("rows", [1, 8, 12])
def test_gate_over_the_whole_range(rows):
    """silu(a) b for a from -104 to 110, where exp(-a) passes the largest float and silu becomes subnormal, and b from 2^-20
    to 2^100: 2 units each of the exponential and the quotient, 3 roundings besides, and where that is subnormal its spacing of
    2^-149, times a b."""
    a = torch.linspace(-104, 110, 1500)
    b = 2.0 ** torch.tensor([-20.0, 0, 60, 100]).repeat(375)
    K, I = 128, 1500
    codes = torch.ones(1, 2 * I, K // 8, dtype=torch.int32)  # in-feature 0 has the code 1
    steps = torch.cat((a, b)).view(1, 2 * I, 1)
    zeros = torch.zeros_like(steps)
    X = torch.zeros(rows, K, dtype=torch.bfloat16)
    X[:, 0] = 1.0
    got = awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), codes.cuda(), steps.cuda(), zeros.cuda(), gated=True)
    ref = a.double() * torch.sigmoid(a.double()) * b.double()
    err = 6 * 2.0 ** -23 * ref.abs() + 2.0 ** -149 * (a.double() * b.double()).abs()
    for row in got:
        plain.assert_within(row[None], ref[None], err[None])
    assert int(((ref.abs() > 1e-30) & (a < -88.8)).sum()) > 20  # the case shows it


# tiles of one and of several widths, two, three and four groups in flight, an odd number of groups
@pytest.mark.parametrize("rows,K,O", [(9, 384, 130), (16, 384, 264), (48, 640, 257), (96, 640, 300), (97, 1152, 200),
                                      (200, 1408, 515)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("far", [False, True])
def test_one_hot_rows_of_experts_are_exact(rows, K, O, gated, far):
    """A row with a single power of two gets exactly bf16(x RN32((q - z) step)) of each weight: every nibble, the operand's order,
    the group's step and zero point (up to +-240 they stay exact). Gated, the same two numbers through the gate."""
    O += O % 2 if gated else 0
    codes, steps, zeros = plain.packed(O, K, K + rows)
    if far:
        zeros = torch.randint(-240, 241, zeros.shape, generator=torch.Generator().manual_seed(K)).float()
        steps = steps * 0.05
    deq = plain.dequantized(codes, steps, zeros).float()  # one rounding of the exact product
    W = tuple(t[None].cuda() for t in (codes, steps, zeros))
    for first in range(0, K, rows):
        k = (first + torch.arange(rows)) % K
        scale = 2.0 ** (torch.arange(rows) % 7 - 3).float()
        X = torch.zeros(rows, K)
        X[torch.arange(rows), k] = scale
        got = awq.w4a16_experts(X.bfloat16().cuda(), offsets_of([rows]).cuda(), *W, gated=gated)
        want = deq[:, k].T * scale[:, None]
        if not gated:
            assert torch.equal(got.cpu(), want.bfloat16()), first
        else:
            a, b = want.double().chunk(2, dim=1)
            ref = a * torch.sigmoid(a) * b
            plain.assert_within(got, ref, 7 * 2.0 ** -23 * ref.abs())


@pytest.mark.parametrize("counts,K,O", [([9, 0, 70, 200], 14336, 300), ([500, 33], 1152, 700), ([12] * 8, 28672, 260)])
@pytest.mark.parametrize("one_sided", [False, True])
def test_rows_of_experts_lose_nothing_before_the_rounding(counts, K, O, one_sided):
    parts = [weights_around_zero(O, K, 170 + e) for e in range(len(counts))]
    W = tuple(torch.stack([p[i] for p in parts]).cuda() for i in range(3))
    X = normal((sum(counts), K), 180)
    X = X.abs() if one_sided else X
    got = awq.w4a16_experts(X.cuda(), offsets_of(counts).cuda(), *W)
    row = 0
    for e, n in enumerate(counts):
        if n:
            ref, err = bounds.grouped(X[row:row + n], *parts[e])
            bounds.assert_rounds(got[row:row + n], ref)
            plain.assert_within(got[row:row + n], ref, err)
        row += n


def test_rows_of_experts_with_wild_steps_and_zero_points():
    K, O, rows = 768, 300, 50
    W = plain.packed(O, K, 190, wild=True)
    X = normal((rows, K), 191)
    got = awq.w4a16_experts(X.cuda(), offsets_of([rows]).cuda(), *(t[None].cuda() for t in W))
    plain.assert_within(got, *bounds.grouped(X, *W))


@pytest.mark.parametrize("K", [1024, 28672])
@pytest.mark.parametrize("kind", ["centred", "outliers", "one-sided", "squared"])
def test_few_tokens_sum_as_fp32_does(K, kind):
    """With minus the result as the bias, the output is what the result's rounding to bf16 left, r, and the error of the sums: seen
    to 2^-9 of r. The sums may be off by 2^-17 of the result's norm: cut to fp32 at every MMA without a guard bit they are by
    4e-6 at K = 28672. Activations around zero, with channels twenty times as large, of one sign, and squared."""
    M, O = 4, 1024
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(200))
    if kind == "outliers":
        X[:, 7::200] *= 20
    if kind in ("one-sided", "squared"):
        X = X.clamp(min=0) if kind == "one-sided" else X.clamp(min=0) ** 2
    X, W = X.bfloat16(), weights_around_zero(O, K, 201)
    ref = X.double() @ plain.dequantized(*W).T
    Wd, bias = tuple(t.cuda() for t in W), -ref.bfloat16()
    left = ref + bias.double()
    got = torch.cat([awq.w4a16_gemv(X[m:m + 1].cuda(), *Wd, bias=bias[m].cuda()) for m in range(M)])
    off = float((got.double().cpu() - left).norm() / ref.norm())
    assert off <= 2.0 ** -9 * float(left.norm() / ref.norm()) + 2.0 ** -17, off
