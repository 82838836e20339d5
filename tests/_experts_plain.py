"""Plain 64-bit forms of the one-token products, the expert sort and the experts' products, and how far a
correct kernel may be from them."""
import numpy as np
import torch

from oracle import awq_oracle as orc

GROUP = 128


def packed(O, K, seed, wild=False):
    """Codes (int32), steps and zero points of a [O, K] weight, on the CPU. `wild`: every code, steps over five decades,
    and zero points far outside 0..15 (a group of nearly equal weights has those)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    words = rng.integers(0, 1 << 32, (O, K // 8), dtype=np.uint32)
    steps = np.exp(rng.uniform(np.log(1e-5), np.log(1.0), (O, K // GROUP)) if wild else
                   rng.uniform(np.log(1e-3), np.log(1e-2), (O, K // GROUP))).astype(np.float32)
    zeros = rng.integers(0, 16, (O, K // GROUP)).astype(np.float32)
    if wild:
        far = rng.random(zeros.shape) < 0.2
        zeros[far] = rng.integers(-600000, 600000, int(far.sum())).astype(np.float32)
    return (torch.from_numpy(words.view(np.int32)), torch.from_numpy(steps), torch.from_numpy(zeros))


def dequantized(codes, steps, zeros):
    """(q - z) * step in 64 bits, [O, K]."""
    O, words = codes.shape
    q = orc.unpack_codes(codes.numpy().view(np.uint32), words * 8).astype(np.float64)
    z = np.repeat(zeros.numpy().astype(np.float64), GROUP, axis=1)
    s = np.repeat(steps.numpy().astype(np.float64), GROUP, axis=1)
    return torch.from_numpy((q - z) * s)


def product(X, codes, steps, zeros, rounded_far_zeros=False):
    """(X deq(W)^T in 64 bits, bound on a kernel's fp32 error before its output rounding).

    Per group g (A_g = sum of |x| over it): S_g is 128 additions of terms up to (1024 + 15) |x|, each off by at most one
    unit 2^-23 (the tensor cores may truncate); the 1024 A_g of the constants are sums of up to 12 levels, and with them
    subtracted 15 roundings of values up to 1039 A_g; the group's sum of x has 12 more, times |z|; the product with z, the
    step and the power of two one rounding each of values up to (15 + |z|) A_g; the running sums over G groups and up to 8
    slices another G + 8 of them. x in fp16 is off by 2^-39 of the group's largest: below one more of those. (A kernel that
    sums 128 + q or q - z stays below the same bound.)
    rounded_far_zeros: q - z enters rounded to bf16, which is exact up to 256; where |z| > 240 a weight is then off by
    half a bf16 step, 2^-8 of its size."""
    x = X.double()
    W = dequantized(codes, steps, zeros)
    G = steps.shape[1]
    A = x.abs().view(x.shape[0], G, GROUP).sum(2)
    z = zeros.double().abs()
    coef = steps.double() * (2 * 128 * 1039 + 15 * 1039 + 12 * z + (G + 12) * (15 + z))
    err = 2.0 ** -24 * (A @ coef.T)
    if rounded_far_zeros:
        far = (z > 240).repeat_interleave(GROUP, 1)
        err = err + 2.0 ** -8 * (x.abs() @ (W.abs() * far).T)
    return x @ W.T, err


def gate(P, err):
    """silu(a) b of P = [a | b] and the bound after it: |silu'| < 1.1; a fast exponential is off by (2 + 1.2 |a|) units of
    2^-23 relative (its argument is scaled and rounded), the sum, a fast quotient (2 units) and the product by 4 more; an exponential
    past the largest float makes 0 of a silu below 2^-120."""
    a, b = P.chunk(2, dim=1)
    ea, eb = err.chunk(2, dim=1)
    s = a / (1 + torch.exp(-a))
    return s * b, 1.1 * ea * b.abs() + s.abs() * eb + 1.1 * ea * eb + (6 + 1.2 * a.abs()) * 2.0 ** -23 * (s * b).abs() + 2.0 ** -120 * b.abs()


def assert_within(got, ref, err):
    """got (bf16) within half a bf16 step of something within err of ref."""
    got = got.double().cpu()
    tol = err + 2.0 ** -8 * (ref.abs() + err) + 1e-38
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist(),
                           tol[bad][:4].tolist())


def sort_slots(ids, E):
    """offsets, order, pos by the definition."""
    flat = ids.reshape(-1).tolist()
    slots = [(e, s) for s, e in enumerate(flat) if 0 <= e < E]
    slots.sort()
    order = [s for _, s in slots] + [-1] * (len(flat) - len(slots))
    offsets = [sum(1 for e, _ in slots if e < i) for i in range(E + 1)] if E <= 64 else \
        np.searchsorted(np.array([e for e, _ in slots]), np.arange(E + 1)).tolist()
    pos = [-1] * len(flat)
    for r, (_, s) in enumerate(slots):
        pos[s] = r
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as_int(offsets), as_int(order), as_int(pos).view(ids.shape)


def expert_of_rows(offsets):
    """Expert of each routed row."""
    counts = (offsets[1:] - offsets[:-1]).long()
    return torch.repeat_interleave(torch.arange(len(counts)), counts)
