"""Plain numpy fp64 forms of the operators beside the chunkwise kernels, each with an a-priori bound on what an
fp32 evaluation in any order may be off by (before the output's own rounding, see ``rounding``).

With u = 2^-24 (fp32): exp of a gate in [-1, 0] is within 3u of the true value, every product and sum within u.  In a
recurrence h_t = a_t h_{t-1} + x_t, the share of h_t that comes from row s has passed t - s decays, each at most 5u
(exp, product, sum), and at most 100 more roundings where segments are joined; W_t = sum over s of (t - s) |share| obeys
W_t = a_t (W_{t-1} + H_{t-1}) with H_t the sum of the shares' magnitudes.  The bound is u (5 W + 100 H).
"""
import numpy as np

U = 2.0 ** -24
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # unit roundoff
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half the spacing of subnormals


def rounding(ref, kind):
    """Error of rounding values near ``ref`` to a type."""
    return UNIT[kind] * np.abs(ref) + TINY[kind]


def bounds_of(B, T, cu):
    if cu is None:
        return [(n * T, (n + 1) * T) for n in range(B)]
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def scan_fwd(x, g, h0=None, cu=None):
    """x, g [B, T, D] -> h [B, T, D], ht [N, D] and their bounds."""
    B, T, D = x.shape
    x, a = x.reshape(-1, D), np.exp(g.reshape(-1, D))
    seqs = bounds_of(B, T, cu)
    h, tol = np.zeros_like(x), np.zeros_like(x)
    ht, tol_t = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    for n, (lo, hi) in enumerate(seqs):
        s = np.zeros(D) if h0 is None else h0[n].copy()
        H, W = np.abs(s), np.zeros(D)
        for r in range(lo, hi):
            W = a[r] * (W + H)
            H = a[r] * H + np.abs(x[r])
            s = a[r] * s + x[r]
            h[r], tol[r] = s, U * (5 * W + 100 * H)
        ht[n], tol_t[n] = s, U * (5 * W + 100 * H)
    return h.reshape(B, T, D), ht, tol.reshape(B, T, D), tol_t


def scan_bwd(g, h, dh, h0=None, dht=None, cu=None):
    """Gradients for L = sum(h dh) + sum(ht dht): ((dx, dg, dh0), bounds)."""
    B, T, D = g.shape
    a, h, dh = np.exp(g.reshape(-1, D)), h.reshape(-1, D), dh.reshape(-1, D)
    seqs = bounds_of(B, T, cu)
    dx, dg, tx, tg = (np.zeros_like(dh) for _ in range(4))
    d0, t0 = np.zeros((len(seqs), D)), np.zeros((len(seqs), D))
    for n, (lo, hi) in enumerate(seqs):
        mu = np.zeros(D) if dht is None else dht[n].copy()
        M, W = np.abs(mu), np.zeros(D)
        for r in range(hi - 1, lo - 1, -1):
            lam, L = dh[r] + mu, np.abs(dh[r]) + M
            prev = h[r - 1] if r > lo else (np.zeros(D) if h0 is None else h0[n])
            dx[r], tx[r] = lam, U * (5 * W + 100 * L)
            mu, M, W = a[r] * lam, a[r] * L, a[r] * (W + L)
            dg[r], tg[r] = mu * prev, U * (5 * W + 104 * M) * np.abs(prev)
        d0[n], t0[n] = mu, U * (5 * W + 100 * M)
    shape = (B, T, D)
    return (dx.reshape(shape), dg.reshape(shape), d0), (tx.reshape(shape), tg.reshape(shape), t0)


def gla_step(q, k, v, g, state, scale):
    """q, k, g [B, H, K], v [B, H, V], state [B, H, K, V] -> o, new state and their bounds (K + 16 roundings a sum)."""
    kept, put = np.exp(g)[..., None] * state, k[..., None] * v[..., None, :]
    new, size = kept + put, np.abs(kept) + np.abs(put)
    o = scale * np.einsum("bhk,bhkv->bhv", q, new)
    return o, new, (q.shape[-1] + 16) * U * scale * np.einsum("bhk,bhkv->bhv", np.abs(q), size), 5 * U * size


# A sum of squares in any order with partial sums of at most 64 terms joined by a tree: 80 roundings, halved by the
# root, and 4u of the root itself.
RSTD_TOL = 50 * U


def norm_fwd(x, res, w, eps):
    """-> y, s, rstd (bounds: 60u |y|, u |s|, RSTD_TOL rstd)."""
    s = x if res is None else x + res
    rstd = 1 / np.sqrt((s ** 2).mean(-1) + eps)
    return s * rstd[..., None] * (1 if w is None else w), s, rstd


def quant_scales(y, group):
    """-> fp64 scales [rows, groups] and the scale of every column."""
    rows, D = y.shape
    width = group or D
    starts = np.arange(0, D, width)
    scales = np.maximum(np.maximum.reduceat(np.abs(y), starts, axis=1) / 448, 1e-30)
    return scales, np.repeat(scales, width, axis=1)[:, :D]


def norm_bwd(s, rstd, w, dy, ds):
    """-> (grad, dw) and their bounds (sums over columns: 90 roundings; over rows: one for each row and 8)."""
    D = s.shape[-1]
    r, w = rstd[..., None], np.ones(D) if w is None else w
    n, wdy = s * r, w * dy
    c = (wdy * n).mean(-1, keepdims=True)
    grad = r * (wdy - n * c) + (0 if ds is None else ds)
    size = (np.abs(wdy * n)).mean(-1, keepdims=True)
    tol = U * (r * (8 * np.abs(wdy) + np.abs(n) * (100 * size)) + 2 * np.abs(0 if ds is None else ds))
    return grad, (dy * n).sum(0), tol, (s.shape[0] + 8) * U * np.abs(dy * n).sum(0)
