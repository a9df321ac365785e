"""MXFP4 and the gated block on MXFP4 operands in 64 bits (numpy), written from the definitions.

Tolerances of the products.  The operands' values are exact in every form, so a product differs from
the 64-bit one by the fp32 accumulation and the rounding of the stored result:
    |D - ref| <= (ceil(K / 64) + 16) 2^-23 S + u(ref),      S = sum_k |a_k| |b_k| + |bias|,
one rounding or truncation (below 2^-23 of the largest partial sum, which S bounds) for each
64-deep step of the tensor cores, for each partial sum of a split K loop, for the bias, and a few for
the sums inside a step; u(ref) is half the spacing of the stored type at ref (bf16 or fp32).

The block rounds Y, dG and dU to 4 bits from fp32.  Where such a value lies within the fp32 error of a
rounding boundary the kernel and the 64-bit reference may take different neighbours; about one value
in 10^5 does, each off by one step (a quarter of the value, typically), which moves the relative
Frobenius error of a product by about 0.25 sqrt(1e-5) = 8e-4 beside the bf16 store's 1.7e-3.  The block is
held to the framework's bf16 tolerance, 3e-3 (gpu_util.assert_close).
"""
import numpy as np

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
MIDPOINTS = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2


def quantize(x):
    """x [rows, K] (any float type) -> codes uint8 [rows, ceil(K/32)*16], scale bytes uint8 [rows, ceil(K/32)]."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    nb = -(-k // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :k] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    _, ex = np.frexp(amax)  # amax = m 2^ex, m in [1/2, 1): floor(log2) = ex - 1
    e = np.where(amax > 0, np.clip(ex - 3, -127, 125), -127)
    a = np.abs(b) * np.exp2(-e.astype(np.float64))[:, :, None]
    lo = np.searchsorted(MIDPOINTS, a.reshape(-1), side="left").reshape(a.shape)
    hi = np.searchsorted(MIDPOINTS, a.reshape(-1), side="right").reshape(a.shape)
    idx = np.where(lo % 2 == 0, lo, hi)  # at a midpoint they differ: the even code
    code = (idx + np.where(np.signbit(b), 8, 0)).astype(np.uint8).reshape(rows, nb * 16, 2)
    code = np.where(np.repeat(bad, 16, axis=1)[:, :, None], 0, code).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).astype(np.uint8), scales


def dequantize(codes, scales, k):
    """Codes and plain scale bytes -> float64 [rows, k]."""
    rows = codes.shape[0]
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(rows, -1)
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(rows, -1, 32) * s[:, :, None]).reshape(rows, -1)[:, :k]


def q(x):
    """The values that x is rounded to along its last axis."""
    return dequantize(*quantize(x), np.asarray(x).shape[1])


def tile_scales(s, rows, k, fill=0):
    """Plain scale bytes [rows, ceil(K/32)] -> the tiled layout, one byte at a time."""
    rt, kt = -(-rows // 128), -(-k // 128)
    out = np.full(rt * kt * 512, fill, dtype=np.uint8)
    for r in range(rows):
        for j in range(kt * 4):
            at = ((r // 128) * kt + j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4
            out[at] = s[r, j] if j < s.shape[1] else 0
    return out.reshape(rt, kt, 32, 4, 4)


def untile_scales(t, rows, k):
    """The tiled layout -> scale bytes [rows, 4 ceil(K/128)], padding blocks included."""
    t = np.asarray(t).reshape(-(-rows // 128), -(-k // 128), 32, 4, 4)
    return t.transpose(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, -1)[:rows]


def half_spacing(a, bits):
    """Half the spacing at |a| of numbers with `bits` significant bits (8: bf16, 24: fp32)."""
    a = np.maximum(np.abs(a), 2.0 ** -126)
    return np.ldexp(1.0, np.floor(np.log2(a)).astype(np.int64) - bits)


def assert_product(got, a, b, bias=None, bf16=True, name=""):
    """got against a b^T + bias, elementwise, with the bound derived above."""
    got = np.asarray(got, dtype=np.float64)
    ref, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        ref, size = ref + bias, size + np.abs(bias)
    tol = (-(-a.shape[1] // 64) + 16) * 2.0 ** -23 * size + half_spacing(np.maximum(np.abs(ref), np.abs(got)), 8 if bf16 else 24)
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    worst = np.max((np.abs(got - ref)) / tol) if got.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times the tolerance at {np.unravel_index(np.argmax(np.abs(got - ref) / tol), got.shape)}"


def split(h):
    """Packed columns -> (gate, up)."""
    v = np.asarray(h).reshape(h.shape[0], -1, 2, 128)
    return v[:, :, 0].reshape(h.shape[0], -1), v[:, :, 1].reshape(h.shape[0], -1)


def join(g, u):
    n = g.shape[0]
    return np.stack((g.reshape(n, -1, 128), u.reshape(n, -1, 128)), axis=2).reshape(n, -1)


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def block_fwd(x, w, b, bw=None, b2=None, rnd=q):
    """x [M,h], w [2f,h] and b [h,f] (values, packed rows) -> (Z, H).  rnd: the rounding (identity for the
    exact block)."""
    H = rnd(x) @ w.T
    if bw is not None:
        H = H + bw
    g, u = split(H)
    Z = rnd(g * sigmoid(g) * u) @ b.T
    return (Z if b2 is None else Z + b2), H


def block_bwd(x, w, b, H, dz, rnd=q):
    """w [h,2f] and b [f,h] (values) -> dX, dW [h,2f], dB [f,h], dbw, db2."""
    g, u = split(H)
    s = sigmoid(g)
    dy = rnd(dz) @ b.T
    dh = join(dy * u * s * (1 + g * (1 - s)), dy * g * s)
    y = g * s * u
    dx = rnd(dh) @ w.T
    dw = rnd(x.T) @ rnd(dh.T).T
    db = rnd(y.T) @ rnd(dz.T).T
    return dx, dw, db, dh.sum(0), dz.sum(0)
