"""Plain numpy fp64 forms of the gated delta rule and of the group norm, token by token and value by value, and the bounds
on what the kernels may be off by.

Delta rule.  For keys of length at most 1 and strengths in [0, 2] the map S -> (1 - beta k k^T) exp(g) S does not stretch
a column of the state, so that errors made at different tokens add up at most.

  * token by token in fp32 (u = 2^-24): a token's dot products over K (or V) values are within (K + 16) u of the column's
    length, the roundings of different tokens are independent: (D + 16) u sqrt(T) with D the longer of K and V.
  * in chunks of 64 on the tensor cores: an operand in two bf16 terms is within 2^-16 of its value at worst and 2^-18 in
    the mean square (a rounding's error is spread over its half step, and a value over the steps of its binade: 2^-9 each),
    and a sum of 64 and more such errors of random sign is as large as their mean square has it.  A product of two such
    operands drops as much again (3 2^-18 in all).  k S (1), its product with the inverse (3), the state's update (1) and
    the output's product (3) make 2^-15 a chunk; chunks add up: 2^-15 (1 + chunks).  The backward reads forward's rows and
    states and walks the same chain once more, so that its products hold twice that.
    dq and dk come from operands in one 16-bit term each: ``grad_sizes``.

Both are relative to the largest value of the head (over its tokens, or of its state).  Sums over two such values
(gradients of gates and strengths) are relative to the product of the lengths.
"""
import numpy as np

U = 2.0 ** -24


def bound(kind, K, V, T, backward=False):
    """Relative bound of a head's values (kind: "scan" or "chunk")."""
    if kind == "scan":
        return (max(K, V) + 16) * U * max(T, 1) ** 0.5 * (2 if backward else 1)
    return 2.0 ** -15 * (1 + -(-T // 64)) * (2 if backward else 1)


def sequences(B, T, cu):
    return [(n * T, (n + 1) * T) for n in range(B)] if cu is None else [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def _flat(*ts):
    return [None if t is None else t.reshape(-1, *t.shape[2:]) for t in ts]


def _outer(a, b):
    return a[..., :, None] * b[..., None, :]


def delta_fwd(q, k, v, g, beta, scale, h0=None, cu=None, keep=False):
    """-> o (NaN in rows outside all sequences), ht, and with ``keep`` the states before and after each row."""
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    q, k = (np.repeat(t, HV // H, 2) for t in (q, k))
    seqs = sequences(B, T, cu)
    fq, fk, fv, fg, fb = _flat(q, k, v, g, beta)
    o, ht, states = np.full_like(fv, np.nan), np.zeros((len(seqs), HV, K, V)), {}
    for n, (lo, hi) in enumerate(seqs):
        S = np.zeros((HV, K, V)) if h0 is None else h0[n].copy()
        for r in range(lo, hi):
            old = np.exp(fg[r])[:, None, None] * S
            row = fb[r][:, None] * (fv[r] - np.einsum("hk,hkv->hv", fk[r], old))
            S = old + _outer(fk[r], row)
            o[r] = scale * np.einsum("hk,hkv->hv", fq[r], S)
            if keep:
                states[r] = (old, row, S)
        ht[n] = S
    o = o.reshape(v.shape)
    return (o, ht, states) if keep else (o, ht)


def delta_bwd(q, k, v, g, beta, do, scale, h0=None, dht=None, cu=None, keep=None):
    """-> dq, dk, dv, dg, dbeta, dh0 (zeros in rows outside all sequences).  ``keep``: a dict that gets each row's gradient of
    its update row, and of the state behind it."""
    B, T, H, K = q.shape
    HV, V = v.shape[2:]
    _, _, states = delta_fwd(q, k, v, g, beta, scale, h0, cu, keep=True)
    seqs = sequences(B, T, cu)
    fq, fk, fv, fg, fb, fo = _flat(*(np.repeat(t, HV // H, 2) for t in (q, k)), v, g, beta, do)
    dq, dk, dv, dg, db = (np.zeros_like(t) for t in (fq, fk, fv, fg, fb))
    dh0 = np.zeros((len(seqs), HV, K, V))
    for n, (lo, hi) in enumerate(seqs):
        dS = np.zeros((HV, K, V)) if dht is None else dht[n].copy()
        for r in range(hi - 1, lo - 1, -1):
            old, row, S = states[r]
            behind = dS
            dq[r] = scale * np.einsum("hkv,hv->hk", S, fo[r])
            dS = dS + scale * _outer(fq[r], fo[r])
            x = np.einsum("hk,hkv->hv", fk[r], dS)
            back = fb[r][:, None] * x
            if keep is not None:
                keep[r] = (old, row, x, behind)
            dv[r] = back
            db[r] = (x * (fv[r] - np.einsum("hk,hkv->hv", fk[r], old))).sum(-1)
            dk[r] = np.einsum("hkv,hv->hk", dS, row) - np.einsum("hkv,hv->hk", old, back)
            dold = dS - _outer(fk[r], back)
            dg[r] = (dold * old).sum((-1, -2))
            dS = np.exp(fg[r])[:, None, None] * dold
        dh0[n] = dS
    shared = lambda t: t.reshape(B, T, H, HV // H, K).sum(3)   # noqa: E731
    return shared(dq), shared(dk), dv.reshape(v.shape), dg.reshape(g.shape), db.reshape(g.shape), dh0


def grad_sizes(q, k, g, beta, do, scale, B, T, cu, keep):
    """What the terms of the chunked dq and dk add up to in magnitude, [B, T, H, K] each, from what ``delta_bwd`` kept.

    In a chunk, with G the running sum of gates and D_ij = exp(G_i - G_j),
        dq_i = scale exp(G_i) S do_i + sum over j <= i of p_ij k_j,                     p_ij = scale D_ij do_i.N_j
        dk_i = -beta_i exp(G_i) S x_i + exp(G_end - G_i) dS' N_i + sum over j of (p_ji q_j + (b_ij + b_ji) k_j),
                                                                                          b_ij = -beta_i D_ij x_i.N_j (j < i)
    Where S, dS', N, x, and then p and b are rounded to 16 bits, a term is off by at most three roundings: two of its
    factors, and p's (b's) own."""
    H, HV = q.shape[2], beta.shape[2]
    fq, fk, fg, fb, fo = _flat(*(np.repeat(np.abs(t), HV // H, 2) for t in (q, k)), g, beta, np.abs(do))
    aq, ak = np.zeros_like(fq), np.zeros_like(fk)
    for lo, hi in sequences(B, T, cu):
        for c in range(lo, hi, 64):
            rows = slice(c, min(c + 64, hi))
            G = np.cumsum(np.maximum(fg[rows], -1000), 0).T                                   # [HV, n]
            D = np.exp(np.minimum(G[:, :, None] - G[:, None, :], 0 if (fg <= 0).all() else np.inf)) * np.tril(np.ones((G.shape[1],) * 2))
            first, last = keep[rows.start], keep[rows.stop - 1]
            S = np.abs(first[0])                                                              # the state after the first row's gate
            dS, n = np.abs(last[3]), np.stack([np.abs(keep[r][1]) for r in range(c, rows.stop)], 1)
            x, d = np.stack([np.abs(keep[r][2]) for r in range(c, rows.stop)], 1), fo[rows].transpose(1, 0, 2)
            kk, qq, b = fk[rows].transpose(1, 0, 2), fq[rows].transpose(1, 0, 2), fb[rows].T[..., None]
            start, end = np.exp(G - G[:, :1])[..., None], np.exp(G[:, -1:] - G)[..., None]
            P = scale * D * (d @ n.transpose(0, 2, 1))
            A = b * D * (x @ n.transpose(0, 2, 1)) * np.tril(np.ones(D.shape[1:]), -1)
            aq[rows] = (scale * start * (d @ S.transpose(0, 2, 1)) + P @ kk).transpose(1, 0, 2)
            ak[rows] = (b * start * (x @ S.transpose(0, 2, 1)) + end * (n @ dS.transpose(0, 2, 1)) + P.transpose(0, 2, 1) @ qq +
                        (A + A.transpose(0, 2, 1)) @ kk).transpose(1, 0, 2)
    shared = lambda t: t.reshape(B, T, H, HV // H, -1).sum(3)   # noqa: E731
    return shared(aq), shared(ak)


def largest(ref, axes):
    """Largest magnitude over some axes, kept for broadcasting (NaN rows left out)."""
    return np.nan_to_num(np.abs(ref)).max(axis=axes, keepdims=True, initial=0.0)


# Group norm.  A thread adds at most 280 values one after the other in the tests, and fewer than 40 partial sums follow:
# 320 roundings, and some for the products.
SUM = 340 * U


def act_of(z, silu):
    """(act(z), act'(z))"""
    if not silu:
        return z, np.ones_like(z)
    s = 1 / (1 + np.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def _parts(x, G):
    return x.reshape(x.shape[0], -1, G, x.shape[-1] // G)


def group_norm_fwd(x, G, w, b, silu, eps):
    """-> (y, mean, rstd) and their bounds."""
    p = _parts(x, G)
    mean = p.mean((1, 3))
    d = p - mean[:, None, :, None]
    rstd = 1 / np.sqrt((d ** 2).mean((1, 3)) + eps)
    size = np.abs(p).mean((1, 3))
    n = d * rstd[:, None, :, None]
    wide = np.broadcast_to((rstd * size)[:, None, :, None], n.shape).reshape(x.shape)
    n = n.reshape(x.shape)
    w = np.ones(x.shape[-1]) if w is None else w
    b = np.zeros(x.shape[-1]) if b is None else b
    y, slope = act_of(n * w + b, silu)
    tol = 1.1 * SUM * (np.abs(w) * (np.abs(n) + wide) + np.abs(b))   # |silu'| < 1.1
    # the variance's relative error: of its own sum, and of a mean that is off by SUM size
    return (y, mean, rstd), (tol, SUM * size, rstd * (SUM + (SUM * size * rstd) ** 2))


def group_norm_bwd(x, mean, rstd, dy, w, b, silu):
    """-> (dx, dw, db) and their bounds, for the given statistics."""
    G = mean.shape[1]
    n = ((_parts(x, G) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    w = np.ones(x.shape[-1]) if w is None else w
    b = np.zeros(x.shape[-1]) if b is None else b
    z = n * w + b
    _, slope = act_of(z, silu)
    dz = dy * slope
    a, p, r = _parts(dz * w, G), _parts(n, G), rstd[:, None, :, None]
    m1, m2 = a.mean((1, 3), keepdims=True), (a * p).mean((1, 3), keepdims=True)
    dx = (r * (a - m1 - p * m2)).reshape(x.shape)
    over = tuple(range(x.ndim - 1))
    # dz: silu's slope and its argument, n off by a few u of itself and of the subtraction's operands
    off = 16 * U * (1 + np.abs(z) + np.abs(n * w) + np.abs(b) + np.abs(_spread(x, mean, rstd, w)))
    edz = np.abs(dy) * off * (1 if silu else 0) + 4 * U * np.abs(dz)
    en = 4 * U * (np.abs(n) + np.abs(_spread(x, mean, rstd, np.ones_like(w))))
    ea, size = _parts(edz * np.abs(w), G), np.abs(a)
    ep = _parts(en, G)
    e1 = (ea + SUM * size).mean((1, 3), keepdims=True)
    e2 = ((ea + SUM * size) * np.abs(p) + size * ep).mean((1, 3), keepdims=True)
    tol = r * (ea + 4 * U * size + e1 + np.abs(p) * e2 + ep * np.abs(m2) + 8 * U * (np.abs(m1) + np.abs(p * m2)))
    sums = lambda t: t.sum(over)   # noqa: E731
    return (dx, sums(dz * n), sums(dz)), \
        (tol.reshape(x.shape), sums((edz + SUM * np.abs(dz)) * np.abs(n) + np.abs(dz) * en), sums(edz + SUM * np.abs(dz)))


def _spread(x, mean, rstd, w):
    """Size of the operands of x - mean, in units of the normed value times w."""
    G = mean.shape[1]
    return ((np.abs(_parts(x, G)) + np.abs(mean)[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape) * w
