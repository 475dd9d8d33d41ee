"""Plain 64-bit forms of the attention operators and the cache layout, written
out from include/qattn.h for the tests (numpy; the Q4_0 rule is the oracle's)."""
import numpy as np

import oracle


def q4_0(x):
    """f32 rows [n, D] -> (scales f16 [n, D/32], code bytes [n, D/32, 16])."""
    n, d = x.shape
    b = np.asarray(oracle.quantize(oracle.Q4_0, np.ascontiguousarray(x, np.float32).reshape(-1))).reshape(n, d // 32, 18)
    return np.ascontiguousarray(b[:, :, :2]).view(np.float16)[:, :, 0], b[:, :, 2:]


def q4_0_values(scales, codes):
    """-> f64 [n, D]."""
    c = np.concatenate([codes & 15, codes >> 4], -1).astype(np.float64) - 8
    return (c * scales.astype(np.float64)[:, :, None]).reshape(len(c), -1)


def slot_bytes(page_size, n_kv_heads, d, slot, h):
    """Byte offsets of one row: key codes [D/32][16], value codes, key scales [D/32][2], value scales."""
    nb = d // 32
    page, r = divmod(slot, page_size)
    group = ((page * n_kv_heads + h) * (page_size // 16) + r // 16) * 18 * d
    i = r % 16
    vr = (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3)
    kc = np.empty((nb, 16), np.int64)
    vc = np.empty((nb, 16), np.int64)
    for b in range(nb):
        for j in range(16):
            kc[b, j] = i * (d // 2) + ((j // 4) * nb + b) * 4 + j % 4
            u = (j // 2) ^ (4 if vr & 2 else 0)
            vc[b, j] = 8 * d + vr * (d // 2) + (u * nb + b) * 2 + j % 2
    sc = np.array([[i * nb * 2 + 2 * b, i * nb * 2 + 2 * b + 1] for b in range(nb)])
    return group + kc, group + vc, group + 16 * d + sc, group + 17 * d + sc


def rotate(x, table, pairs, kind):
    """x [n, heads, D], table [n, rot/2, 2] of the tokens' positions; in f32
    each product and sum is rounded (numpy does)."""
    half = table.shape[1]
    x = x.astype(kind)
    c, s = table[:, None, :, 0].astype(kind), table[:, None, :, 1].astype(kind)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def attend(q, k, v, seen, scale):
    """One head in f64: q [m, D], k and v [n, D], seen [m] visible keys each.
    Returns out and what the error bounds need: sum p |v|, the largest
    scale * sum |q k| of a row's keys, and the largest |v|."""
    m, d = q.shape
    out, pv, mag, big = np.zeros((m, d)), np.zeros((m, d)), np.zeros((m, 1)), np.zeros((m, 1))
    for i in range(m):
        n = int(max(0, min(seen[i], len(k))))
        if n == 0:
            continue
        s = scale * (k[:n] @ q[i])
        p = np.exp(s - s.max())
        p /= p.sum()
        out[i], pv[i] = p @ v[:n], p @ np.abs(v[:n])
        mag[i] = abs(scale) * (np.abs(k[:n]) @ np.abs(q[i])).max()
        big[i] = np.abs(v[:n]).max()
    return out, pv, mag, big


def bound(out, pv, mag, big, d, n, q_bits, p_bits, out_f16):
    """How far a kernel's result may be from attend()'s, from its arithmetic:
    a score is off by at most (2^-q_bits + D 2^-23) of scale sum |q k| (q's
    rounding, and f32 sums that may truncate), a weight by 2^-p_bits, the
    exponential and the divisions by 2^-19 in all, sums over n keys by n
    2^-23; weights below the 16-bit parts' last place vanish, at most 2^-24 of
    the largest value each; an f16 result is rounded once more."""
    score = (2.0 ** -q_bits + d * 2.0 ** -23) * mag
    e = (2 * score + 2.0 ** -p_bits + 2.0 ** -19 + n * 2.0 ** -23) * pv + n * 2.0 ** -24 * big
    return e + (2.0 ** -11 * np.abs(out) + 2.0 ** -24 if out_f16 else 1e-37)


def tight_bound(q, k, v, scale, f16):
    """attend()'s out for rows q [m, D] that see all of k, and bound() with a smaller allowance for what 16-bit products
    lose at their last place: the largest product of a weight and a value's scale is 2^6 or more, a product is off by
    2^-25 at most where f16 ends, the codes are at most 8 and a scale is an eighth of its block's largest value: 2^-31 of
    the largest product of a weight and a token's largest value, for each token."""
    out, pv, mag, big = attend(q, k, v, [len(k)] * len(q), scale)
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(-1, keepdims=True))
    most = (p / p.sum(-1, keepdims=True) * np.abs(v).max(-1)).max(-1, keepdims=True)
    bits = (24, 10) if f16 else (20, 20)
    return out, bound(out, pv, mag, 0 * big, q.shape[1], len(k), *bits, f16) + len(k) * 2.0 ** -31 * most
