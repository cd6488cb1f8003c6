"""Plain 64-bit forms of the calls that answer with a quantized model (numpy):
the few-token product, the rows of the 4-bit cache and the attention over it.
Written from the definitions in include/ufp4.h; tests only.

Error bounds.  A product of two operands enters exactly or within 2^-22 (an
operand kept as two FP16 values) of itself, plus 2^-38 of the largest magnitude
among the operand's row or 128 elements for what falls below FP16's normal
numbers (half a step of 2^-24 where that largest one is at least 2^14); n fp32
additions, which the tensor cores may truncate, are within n 2^-23 of the sum of
magnitudes."""
import numpy as np

U23, U24 = 2.0 ** -23, 2.0 ** -24
VALUES = {0: [0, .5, 1, 1.5, 2, 3, 4, 6], 1: [0, .5, 1, 1.5, 2, 2.5, 3, 3.5], 2: [0, .5, 1, 1.5, 2, 2, 2, 2]}
QMAX = {0: 6.0, 1: 3.5, 2: 2.0}


def half_step(dtype):
    """Relative error of a rounding to the type."""
    return 2.0 ** -8 if "bfloat16" in str(dtype) else U24


def e4m3(b):
    b = np.asarray(b, dtype=np.int64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + f / 8.0), 2.0 ** -6 * f / 8.0)
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -v, v))


def values(codes, scales, grid):
    """One code an element [.., k], one E4M3 byte a 16-block [.., k / 16]."""
    codes = np.asarray(codes, dtype=np.int64)
    v = np.array(VALUES[grid])[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(e4m3(scales), 16, axis=-1)


def unpack(b):
    b = np.asarray(b, dtype=np.uint8)
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def rotation(seed):
    """R with y = R x: (1/4) H16 diag(d)."""
    c, key, low = [0, 0, 0, 0], [seed & 0xFFFFFFFF, seed >> 32], 0xFFFFFFFF
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ key[0], b & low, (a >> 32) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    d = np.array([-1.0 if c[0] >> j & 1 else 1.0 for j in range(16)])
    h = np.array([[(-1.0) ** bin(i & j).count("1") for j in range(16)] for i in range(16)])
    return h * d / 4


def rotate(x, seed, back=False):
    r = rotation(seed)
    return (x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16)) @ (r if back else r.T)).reshape(x.shape)


def gemv(x, w, rht, seed, unit):
    """y, and the bound of its error before the result's own rounding.  x
    [t, k]; w [n, k]; unit: relative error of an element of x (0: exact)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    t, k = x.shape
    blur = np.zeros(x.shape)
    if rht:
        # four stages of fp32 additions over 16 magnitudes
        top = np.abs(x).reshape(t, k // 16, 16).sum(-1) / 4
        blur = np.repeat(top * 4 * U24, 16, axis=-1)
        x = rotate(x, seed)
    blur = blur + np.abs(x) * unit
    for a in range(0, k, 128):
        blur[:, a:a + 128] += 2.0 ** -38 * np.abs(x[:, a:a + 128]).max(-1, keepdims=True)
    adds = 2 * 128 + k / 128 + 16
    return x @ w.T, blur @ np.abs(w).T + adds * U23 * (np.abs(x) @ np.abs(w).T)


def quantize_row(x, grid, rht=False, seed=0):
    """What a row of the cache stands for (rotated where it is kept so): its
    grid values, scales and own scale, from fp32 steps as ufp4_quantize's."""
    f = np.float32
    y = np.asarray(x, np.float64)
    y = rotate(y, seed) if rht else y
    y = y.astype(f)
    top = f(448 * QMAX[grid])
    amax = np.abs(y).max()
    if not np.isfinite(amax):
        return None
    with np.errstate(over="ignore"):
        enc = f(min(top / amax, np.finfo(f).max)) if amax > 0 else f(1)
    dec = f(amax / top) if amax > 0 else f(1)
    table = np.array(VALUES[grid][:5 if grid == 2 else 8])
    # every E4M3 value, nearest with ties to the even byte
    bytes_ = np.arange(127)
    e_of = e4m3(bytes_)
    codes, scales = np.zeros(y.size, np.uint8), np.zeros(y.size // 16, np.uint8)

    def nearest(v, grid_, n):
        d = np.abs(grid_ - v)
        best = np.flatnonzero(d == d.min())
        return int(best[0] if best.size == 1 or n[best[0]] % 2 == 0 else best[1])

    for b in range(y.size // 16):
        v = y[16 * b:16 * b + 16]
        with np.errstate(over="ignore"):
            e = bytes_[nearest(min(float(f(f(np.abs(v).max() / f(QMAX[grid])) * enc)), 448.0), e_of, bytes_)]
        scales[b] = e
        if e == 0:
            continue
        r = f(enc / f(e4m3(e)))
        for i in range(16):
            q = f(v[i] * r)
            m = nearest(min(abs(float(q)), QMAX[grid]), table, np.arange(8))
            codes[16 * b + i] = m | (8 if np.signbit(q) else 0)
    return codes, scales, dec


def attn(q, k, v, rows, sees, scale, planes_exact, out_two, top_v, dim):
    """out [n, dim], lse [n] and the bounds of their errors (before out's own
    rounding) for queries q [n, dim] over k, v [L, dim] with sees [n, L].
    rows: k's and v's rotation differences are none (both in one space).
    planes_exact: q enters exactly; out_two: probabilities as two FP16 values;
    top_v: the largest row scale of v times the grid's largest value."""
    s = (q @ k.T) * scale
    mag = (np.abs(q) @ np.abs(k).T) * abs(scale)
    qtop = np.abs(q).max(-1, keepdims=True)
    blur = (0.0 if planes_exact else 2.0 ** -21) * mag + 2.0 ** -37 * abs(scale) * qtop * np.abs(k).sum(-1)[None, :]
    # sums over dim (twice: two operands), and three roundings of the factors
    ds = blur + (2 * dim + 8) * U23 * mag
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = np.where(sees, s, -np.inf)
        top = s.max(-1, keepdims=True, initial=-np.inf)
        base = np.where(np.isfinite(top), top, 0.0)
        p = np.where(sees, np.exp(s - base), 0.0)
        z = p.sum(-1, keepdims=True)
        w = np.where(z > 0, p / np.where(z > 0, z, 1), 0.0)
        out = w @ v
        lse = np.where(z[:, 0] > 0, np.log(np.where(z > 0, z, 1))[:, 0] + base[:, 0], -np.inf)
    # an exponent's error, exp2f's (2 ulp) and the argument's rounding
    de = np.where(sees, ds + (np.abs(s - base) * 2 + 4) * U24 * 2, 0.0) if sees.any() else np.zeros(s.shape)
    n = sees.sum(-1, keepdims=True) + 64.0
    rel = np.expm1(de).max(-1, keepdims=True, initial=0.0)
    w_abs = w @ np.abs(v)
    tol = w_abs * (2 * rel + (2.0 ** -21 if out_two else 2.0 ** -11) + 2 * n * U23)
    # probabilities below FP16's normal numbers: half a step of 2^-24, in units of the power of two that they are
    # multiplied by, 2^11 over the largest row's scale for fp32 results and 2^6 for bf16 ones of many queries
    tol = tol + n * 2.0 ** (-36 if out_two else -31) * top_v / np.where(z > 0, z, 1)
    lse_tol = rel[:, 0] + n[:, 0] * U23 + np.abs(np.where(np.isfinite(lse), lse, 0)) * 4 * U24 + 2.0 ** -20
    return out, lse, tol, lse_tol
