"""Plain 64-bit forms of the operators around the grouped GEMMs (numpy): the
sort, dispatch, combine and its gradients, the 8-bit checkpoint and the gated
activation with its gradients.  Written from the definitions in
include/ufp4.h; tests only."""
import numpy as np

U32, UBF = 2.0 ** -24, 2.0 ** -8     # unit roundoff of fp32 and bf16


def unit(dtype):
    return UBF if "bfloat16" in str(dtype) else 0.0


def half_step(dtype):
    """Half the spacing of the type's subnormal numbers: a rounding's error
    where the result is below the normal ones."""
    return 2.0 ** -134 if unit(dtype) else 2.0 ** -150


def sort(ids, n_experts):
    """pos, src, counts, offsets of the stable sort (dropped slots last)."""
    e = np.asarray(ids, dtype=np.int64).reshape(-1)
    e = np.where((e < 0) | (e >= n_experts), n_experts, e)
    src = np.argsort(e, kind="stable")
    pos = np.empty_like(src)
    pos[src] = np.arange(src.size)
    counts = np.bincount(e, minlength=n_experts + 1)[:n_experts]
    return pos.reshape(np.shape(ids)), src, counts, np.concatenate([[0], np.cumsum(counts)])


def dispatch(x, pos, routed):
    xs = np.zeros((pos.size, x.shape[1]))
    for t in range(pos.shape[0]):
        for p in pos[t]:
            if p < routed:
                xs[p] = x[t]
    return xs


def combine(y, pos, routed, w=None):
    """The sum and, element by element, the sum of magnitudes."""
    out, mag = np.zeros((2, pos.shape[0], y.shape[1]))
    for t in range(pos.shape[0]):
        for j, p in enumerate(pos[t]):
            if p < routed:
                v = y[p] if w is None else w[t, j] * y[p]
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def combine_bwd(dout, y, pos, routed, w):
    """dy, dw, and dw's sum of magnitudes."""
    dy = np.zeros(y.shape)
    dw, mag = np.zeros((2,) + pos.shape)
    for t in range(pos.shape[0]):
        for j, p in enumerate(pos[t]):
            if p < routed:
                dy[p] = w[t, j] * dout[t]
                dw[t, j] = np.dot(dout[t], y[p])
                mag[t, j] = np.dot(np.abs(dout[t]), np.abs(y[p]))
    return dy, dw, mag


def ckpt(x, fmt):
    """scales (bytes) and restored values of the 8-bit checkpoint."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    scales, back = np.zeros((rows, nb), np.uint8), np.zeros((rows, cols))
    for r in range(rows):
        for b in range(nb):
            v = x[r, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(v)):
                scales[r, b], back[r, 32 * b:32 * b + 32] = 255, np.nan
                continue
            top = np.max(np.abs(v))
            if top == 0:
                continue
            # top = m 2^(e - 127) with 1 <= m < 2; below fp32's normal numbers e is 0
            e = int(np.floor(np.log2(top))) + 127
            m = top / 2.0 ** (e - 127)
            e = max(e, 0)
            if fmt == 1 and m > 1.75:
                e += 1
            s = max(e - 6, 0) if fmt == 0 else min(max(e - 8, 0), 246)
            scales[r, b] = s
            u = v / 2.0 ** (s - 127)
            if fmt == 0:
                q = np.clip(np.rint(u), -127, 127)
            else:
                a = np.maximum(np.abs(u), 2.0 ** -20)
                step = 2.0 ** (np.maximum(np.floor(np.log2(a)), -6) - 3)
                q = np.clip(np.rint(u / step) * step, -448, 448)
                assert np.max(np.abs(u)) <= 448 or top > 1.75 * 2.0 ** 127
            back[r, 32 * b:32 * b + 32] = q * 2.0 ** (s - 127)
    return scales, back


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_bwd(dh, g, u):
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def swiglu_tol(g, u, h, dtype):
    """Bound of the error of h.  fp32: expf within 2 ulp, three roundings.
    bf16: __expf within 2 + 1.173 |g| ulp, __fdividef within 2, two roundings,
    and bf16's own; 0 where 1 + exp(-g) passes 2^126 (a result below 2^-118 |u|)."""
    rel = (4 + 3) * U32 if not unit(dtype) else (2 + 1.173 * np.abs(g) + 2 + 1) * 2 * U32 + UBF * 1.001
    return np.abs(h) * rel + np.abs(u) * 2.0 ** -118 + half_step(dtype)


def swiglu_bwd_tol(dh, g, u, dgate, dup, dtype):
    """The same for the gradients: es bounds the relative error of s, and
    1 - s carries the absolute error of s."""
    s = sigmoid(g)
    es = ((4 + 2) if not unit(dtype) else 2 * (2 + 1.173 * np.abs(g) * (1 - s) + 2 + 1)) * U32
    r = unit(dtype) * 1.001
    tiny = 2.0 ** -118
    mag = np.abs(dh * u)
    tol_g = mag * s * ((es + 4 * U32) * (1 + np.abs(g) * (1 - s)) + np.abs(g) * (s * es + U32)) + r * np.abs(dgate)
    tol_u = np.abs(dh * g) * s * (es + 3 * U32) + r * np.abs(dup)
    end = half_step(dtype)
    return tol_g + mag * (1 + np.abs(g)) * tiny + end, tol_u + np.abs(dh * g) * tiny + end
