"""Rows in int8, the products of two int8 operands, the root-mean-square norm and the balance loss in 64 bits,
from their definitions (numpy, no library code).

Tolerances.  The sums of the products are integers, and what follows them are three fp32 roundings and one to
the output's type, so the products are compared bit for bit (gate+up: SiLU's own bound, below).  Codes are
compared as integers: quotients of bf16 values, and of their products with bf16 weights, lie half way between
two codes or at least 2^-25 from there, and fp64 carries them.  A sum of fp32 terms that a lane adds in turn
and the lanes add as a tree has at most D additions on any way: its error is at most D 2^-24 of the terms'
magnitudes' sum.  Rounding to a type is off by at most half a step, HALF (relative)."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def quantize(v):
    """(codes, a) of rows [n, k] in fp64: rint(127 v / a), half way to even; zeros for rows of zeros or rows
    that are not finite (a is then no finite number)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v).max(1)
    ok = np.isfinite(v).all(1) & (a > 0)
    safe = np.where(ok, a, 1.0)[:, None]
    codes = np.where(ok[:, None], np.round(127 * np.where(ok[:, None], v, 0.0) / safe), 0.0)
    return codes.astype(np.int8), np.where(np.isfinite(v).all(1), a, np.nan)


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32)


def bf16(x):
    """The nearest bf16 value (ties to even) as fp64, NaN kept."""
    import torch

    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def sums(codes, w_codes):
    """The products' sums: integers below 2^53, which fp64 adds exactly."""
    return codes.astype(np.float64) @ w_codes.astype(np.float64).T


def product_bits(codes, scales, w_codes, w_scales, out):
    """The product's output exactly: int sums, three fp32 roundings, one to bf16 (out 'bf16')."""
    y = sums(codes, w_codes).astype(np.float32) * scales.astype(np.float32)[:, None] * w_scales.astype(np.float32)[None]
    return bf16(y) if out == "bf16" else y.astype(np.float64)


def gate_up_bound(codes, scales, gate, gate_scales, up, up_scales):
    """(h, bound of bf16(SiLU(g) u)): g and u carry three fp32 roundings; |silu'| <= 1.1, the exponential's
    argument is off by |g| 2^-23 relative in e^-g, and a few fp32 roundings follow."""
    def exact(w, ws):
        return sums(codes, w) * scales.astype(np.float64)[:, None] * ws[None]

    g, u = exact(gate, gate_scales), exact(up, up_scales)
    dg, du = 3 * U * np.abs(g), 3 * U * np.abs(u)
    h = g / (1 + np.exp(-np.clip(g, -700, None))) * u
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + np.abs(h) * (8 + 2 * np.abs(g)) * 2 * U
    return h, err + HALF["bf16"] * (np.abs(h) + err) + 2.0 ** -126


def additions(k):
    """The longest chain of additions of a row's sum: a lane's elements, its tail, the tree over 64 lanes and
    16 waves."""
    return 64 + k // 1024 + 32


def norm(r, w, eps):
    inv = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    return r * inv * w, inv


def norm_bound(r, w, eps, out):
    """inv: half the relative error of the mean (its sum's chain, a division, an addition), and a root and a
    division; then two products."""
    y, _ = norm(r, w, eps)
    rel = ((additions(r.shape[1]) + 2) / 2 + 5) * U
    return y, np.abs(y) * (rel + HALF[out] * (1 + rel)) + 2.0 ** -133


def norm_grad(dy, r, w, eps, d_sum):
    k = r.shape[1]
    inv = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    g = dy * w
    dx = inv * (g - r * inv ** 2 * (g * r).sum(1, keepdims=True) / k) + d_sum
    return dx, (dy * r * inv).sum(0)


def norm_grad_bounds(dy, r, w, eps, d_sum, out):
    """Every factor carries inv's error or a sum's chain: (3/2 chain + 16) roundings on the magnitudes of the
    two terms, one on the last addition; d_weight adds the rows' chain."""
    n, k = r.shape
    inv = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    g = dy * w
    c = (2.5 * additions(k) + 16) * U
    terms = np.abs(inv * g) + np.abs(r) * inv ** 3 * np.abs(g * r).mean(1, keepdims=True)
    dx, dw = norm_grad(dy, r, w, eps, d_sum)
    err = c * terms + 2 * U * (terms + np.abs(d_sum))
    return (dx, err + HALF[out] * (np.abs(dx) + err) + 2.0 ** -133,
            dw, (n + additions(k) + 16) * U * np.abs(dy * r * inv).sum(0) + 2.0 ** -133)


def balance(z, ids, coefficient, d_loss=1.0, counts=None):
    """(loss, counts [E + 1], d_logits, p, real); z fp64 [t, E].  counts: of more tokens than these, for the
    gradient (the loss and the counts are of these tokens)."""
    t, E = z.shape
    inside = (ids >= 0) & (ids < E)
    real = inside.any(1)
    mine = np.append(np.bincount(ids[inside], minlength=E), real.sum()) if t else np.zeros(E + 1, np.int64)
    use = mine if counts is None else counts
    p = np.zeros((t, E))
    for i in np.nonzero(real)[0]:
        top = z[i].max()
        if top == -np.inf:
            continue
        e = np.exp(z[i] - top)
        p[i] = e / e.sum()
    pairs, tokens = use[:E].sum(), use[E]
    share = E * use[:E] / max(pairs, 1)
    own = mine[E]
    loss = coefficient * (E * mine[:E] / max(mine[:E].sum(), 1) * p.sum(0)).sum() / own if own else 0.0
    slope = d_loss * coefficient / tokens if tokens else 0.0
    dot = (share * p).sum(1, keepdims=True)
    return loss, mine.astype(np.int64), slope * p * (share - dot) * real[:, None], p, real


def balance_bounds(z, ids, coefficient, out, d_loss=1.0, counts=None):
    """A probability is off by the difference's rounding (|z - max| 2^-24), the exponential and its sum; the
    loss's sums are chains of at most t / 64 + 300 additions in fp32."""
    t, E = z.shape
    loss, mine, d, p, real = balance(z, ids, coefficient, d_loss, counts)
    rows = z[real]
    finite = rows[np.isfinite(rows)]
    span = float(finite.max() - finite.min()) if finite.size else 0.0
    rel = (span + 32) * 2 * U
    use = mine if counts is None else counts
    share = E * use[:E] / max(use[:E].sum(), 1)
    slope = abs(d_loss * coefficient) / max(use[E], 1)
    mags = slope * p * (share + (share * p).sum(1, keepdims=True))
    err = 4 * rel * mags
    return (loss, abs(loss) * (rel + (t / 64 + 310) * U), mine, d,
            err + HALF[out] * (np.abs(d) + err) + 2.0 ** -133)


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN at other places than expected"
    bad = ~np.isnan(ref) & ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(got - ref) - bound, -1))), ref.shape)
        b = np.broadcast_to(bound, ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())}/{ref.size} outside; worst at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, bound {b[i]:.3g}")


def to_host(t):
    return t.detach().double().cpu().numpy()


def random_rows(rng, n, k):
    """(codes, scales f32) of rows that fill the range of codes."""
    return rng.integers(-128, 128, (n, k)).astype(np.int8), (2.0 ** rng.uniform(-12, 3, n)).astype(np.float32)


def random_weight(rng, E, n, k):
    """(codes [E, n, k], scales bf16 as fp64 [E, n])."""
    return rng.integers(-128, 128, (E, n, k)).astype(np.int8), bf16(2.0 ** rng.uniform(-12, -4, (E, n)))


def weight(wq, codes, scales, device="cuda"):
    import torch

    E, n, k = codes.shape
    return wq.PackedWeight(wq.FMT_INT8, n, k, E, 0, codes=torch.from_numpy(codes).to(device),
                           scales=torch.from_numpy(scales).to(torch.bfloat16).to(device))


def rows(wq, codes, scales, device="cuda"):
    import torch

    return wq.Int8Rows(torch.from_numpy(codes).to(device), torch.from_numpy(scales).to(device))
