"""How far the products may be from 64 bits: for the few-token kernel and for the experts' grouped kernel, each by its own way
of summing, and how rarely a whole output may round the other way."""
import torch

from tests import _experts_plain as plain

GROUP = 128


def _sums(X, steps, zeros):
    x = X.double()
    A = x.abs().view(x.shape[0], steps.shape[1], GROUP).sum(2)  # sum of |x| per group
    return A, steps.double(), zeros.double().abs()


def few(X, codes, steps, zeros):
    """(X deq(W)^T in 64 bits, bound of the few-token kernel before its output rounding), in units of 2^-24. Per group, S sums q x
    by 8 MMAs of 16 products and the sum so far; each of the 17 may be cut by 2 units of the largest, at most 15 A; the same for
    the sum of x, times |z|. x in fp16 is off by 2^-39 of the group's largest, less than one unit of (15 + |z|) A. Then a
    rounding of (15 + |z|) A each for z's product and the step's, and one per sum over G groups and 8 slices."""
    A, step, z = _sums(X, steps, zeros)
    G = steps.shape[1]
    coef = step * (2 * 17 * 8 * (15 + z) + (3 + G + 8) * (15 + z))
    return X.double() @ plain.dequantized(codes, steps, zeros).T, 2.0 ** -24 * (A @ coef.T)


def term_by_term(X, codes, steps, zeros):
    """The same for sums of x times the weight as an fp32 number: 2 roundings of the weight, and a lane's 4 G terms, 5 levels
    across the lanes and 8 slices one rounding each."""
    A, step, z = _sums(X, steps, zeros)
    coef = step * (15 + z) * (2 + 4 * steps.shape[1] + 13)
    return X.double() @ plain.dequantized(codes, steps, zeros).T, 2.0 ** -24 * (A @ coef.T)


def differ(got, ref):
    """||got - bf16(ref)|| / ||ref||, and the ||bf16 spacing at ref|| / ||ref|| that goes with it."""
    got, ref = got.double().cpu(), ref.double()
    spacing = 2.0 ** (torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -126))) - 7)
    norm = ref.norm()
    return float((got - ref.bfloat16().double()).norm() / norm), float(spacing.norm() / norm)


def assert_rounds(got, ref, before=2.0 ** -14):
    """got (bf16) is what ref gives with an error of `before` times its norm ahead of the last rounding. An error e_i turns the
    rounding of output i with the probability |e_i| / u_i, u_i the spacing there, and then costs u_i: the expected square is
    sum u_i |e_i| <= ||u|| ||e||; twice that, for the spread, and the errors themselves.
    2^-14: with every addend and sum of an MMA cut to fp32 without a guard bit, a group's sums of q x (or of (q - z) x) make
    4e-6 of the result at K = 28672, one-sided X included; sixteen times that. Weights or steps rounded to bf16 make 1e-3, a
    left-out in-feature K^-0.5 = 6e-3."""
    off, spacing = differ(got, ref)
    limit = (2 * spacing * before + before ** 2) ** 0.5
    assert off <= limit, (off, limit)


def grouped(X, codes, steps, zeros):
    """The same as `few` for the experts' grouped kernel: per group, (q - z) x summed by 8 MMAs of 16 products and the sum so far,
    17 addends cut by 2 units of (15 + |z|) A at most, then one rounding per group of the running sum. Where |z| > 240 a
    weight enters rounded to bf16, off by 2^-8 of its size at most."""
    A, step, z = _sums(X, steps, zeros)
    coef = step * (15 + z) * (2 * 17 * 8 + 1 + steps.shape[1])
    W = plain.dequantized(codes, steps, zeros)
    err = 2.0 ** -24 * (A @ coef.T)
    far = (z > 240).repeat_interleave(GROUP, 1)
    return X.double() @ W.T, err + 2.0 ** -8 * (X.double().abs() @ (W.abs() * far).T)
