"""MXFP4 and the token dispatch in 64 bits, from their definitions (numpy, no library code).

Tolerances.  A product of two e2m1 values times two powers of two is exact in fp32 (bf16 operands:
16 mantissa bits), so a sum of K products differs from the exact one by its additions only: at most
K of them, each within one unit of 2^-23 of a partial sum, and no partial sum exceeds S = the sum
of the products' magnitudes.  Hence |sum - exact| <= K 2^-23 S, and rounding the result to a type
with half a step h = eps / 2 (bf16 2^-8, fp32 2^-24) adds h (|exact| + K 2^-23 S).
"""
import numpy as np

VALUES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def bf16(x):
    """fp64 -> the nearest bf16 value (ties to even), as fp64; |x| below 2^127, no subnormals."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, 8)), e - 8)


def encode(x):
    """(code of every value [..., k], scale byte of every block [..., k/32])."""
    x = np.asarray(x, np.float64)
    v = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(v).max(-1)
    finite = np.isfinite(v).all(-1)
    floor = np.frexp(np.where(finite, top, 0.0))[1] - 1  # floor(log2 top) where top > 0
    byte = np.where(finite & (top > 0), np.clip(floor - 2 + 127, 0, 254), 0)
    u = np.where(finite[..., None], v, 0.0) / np.ldexp(1.0, byte - 127)[..., None]
    a = np.minimum(np.abs(u), 6.0)
    mags = VALUES[:8]
    dist = np.abs(a[..., None] - mags)
    best = dist.min(-1, keepdims=True)
    # of two equally near codes the even one
    cand = np.where(dist == best, np.arange(8), 99)
    even = np.where((cand % 2 == 0) & (cand < 99), cand, 99).min(-1)
    code = np.where(even < 99, np.where((dist == best).sum(-1) > 1, even, cand.min(-1)), cand.min(-1))
    code = np.where(np.signbit(u), code + 8, code)
    code = np.where(finite[..., None], code, 0)
    byte = np.where(finite, byte, 255)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def values(code, byte):
    v = VALUES[code].reshape(*byte.shape, 32)
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v * scale[..., None]).reshape(code.shape)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    out = np.empty((*b.shape[:-1], 2 * b.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def product(x, w):
    """(x w^T, sum of the products' magnitudes)."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sum_bound(ref, mag, k, out):
    err = k * 2.0 ** -23 * mag
    return err + HALF[out] * (np.abs(ref) + err) + 2.0 ** -133


def gate_up_bound(g, gm, u, um, k):
    """Bound of bf16(silu(g) u): the sums' errors through the product (|silu'| <= 1.1,
    |silu(g)| <= |g|), the exponential's argument (|g| 2^-23 relative in e^-g) and a few fp32
    roundings, then the output's rounding."""
    dg, du = k * 2.0 ** -23 * gm, k * 2.0 ** -23 * um
    h = g / (1 + np.exp(-np.clip(g, -700, None))) * u
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + np.abs(h) * (8 + 2 * np.abs(g)) * 2.0 ** -23
    return h, err + HALF["bf16"] * (np.abs(h) + err) + 2.0 ** -126


def assert_within(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN at other places than expected"
    bad = ~nan & ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(got - ref) - bound, -1))), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())}/{ref.size} outside; worst at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, bound {bound[i]:.3g}")


def to_host(t):
    """A GPU tensor's values as fp64 (int16: bf16 bits)."""
    import torch

    if t.dtype == torch.int16:
        t = t.view(torch.bfloat16)
    return t.detach().double().cpu().numpy()


def weight(wq, code, byte, device="cuda"):
    """The PackedWeight of codes [E, n, k] and scale bytes [E, n, k/32]."""
    import torch

    E, n, k = code.shape
    return wq.PackedWeight(wq.FMT_MXFP4, n, k, E, 32, codes=torch.from_numpy(pack(code)).to(device),
                           qscale=torch.from_numpy(np.ascontiguousarray(byte)).to(device))


def random_codes(rng, *shape):
    """Codes and scale bytes of normal values (scales vary over a few octaves)."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-3, 4, (*shape[:-1], 1)))
    return encode(x)


def route(ids, experts):
    """(offsets, sorted pairs, positions) of the stable sort by expert; dropped ids get -1."""
    flat = ids.reshape(-1)
    keep = (flat >= 0) & (flat < experts)
    order = [p for e in range(experts) for p in np.nonzero(flat == e)[0]]
    positions = np.full(flat.size, -1, np.int32)
    positions[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=experts))]).astype(np.int32)
    return offsets, np.array(order, np.int64), positions.reshape(ids.shape)
