"""Plain 64-bit forms of the operators of include/qstep.h, written out from
their formulas for the tests (numpy)."""
import numpy as np

E = 2.0 ** -24  # half a step of f32


def _norm(v, err, w, b, layer, eps):
    """N(v; w, b) of rows v that are off by at most err, and how far an f32 evaluation may be from it.

    Sums of d terms take at most 16 additions (fused with the products) a thread and ten in the shuffles; 1 / d, the
    product with it and eps: 29 roundings. A mean is off by less than 34 E of the mean magnitude; what stays of v by
    that, by its own subtraction and by err; 1 / sqrt(mean square + eps) by half of the sum's 29, by its own 4 E (CUDA's
    bound of rsqrtf is 2^-22), and by the elements' errors (their root mean square beside the row's); the two products
    and the bias one rounding each: 14.5 + 4 + 2 < 22."""
    if layer:
        m = v.mean(1, keepdims=True)
        err = err + 34 * E * np.abs(v).mean(1, keepdims=True) + err.mean(1, keepdims=True)
        v = v - m
        err = err + E * np.abs(v)
    ms = (v * v).mean(1, keepdims=True)
    inv = 1.0 / np.sqrt(ms + eps)
    scale = inv * (1.0 if w is None else np.abs(w))
    y = v * inv * (1.0 if w is None else w)
    rel = 22 * E + inv * np.sqrt((err * err).mean(1, keepdims=True)) * 1.01
    off = scale * err + np.abs(y) * rel
    if b is not None:
        y = y + b
        off = off + E * np.abs(y)
    return y, off


def norm_residual(h, y, w=None, b=None, post_w=None, post_b=None, gate=None, scale=1.0, eps=1e-5, layer=False):
    """-> h', its bound, x, its bound, before any rounding to f16."""
    h = h.astype(np.float64)
    off = np.zeros_like(h)
    if y is not None:
        u = y.astype(np.float64)
        e = np.zeros_like(u)
        if post_w is not None:
            u, e = _norm(u, e, post_w.astype(np.float64), None if post_b is None else post_b.astype(np.float64), layer, eps)
        if gate is not None:
            g = gate.astype(np.float64)
            e = np.abs(g) * e + E * np.abs(g * u)
            u = g * u
        s = float(np.float32(scale))
        h = h + s * u
        off = abs(s) * e + E * np.abs(h)
    x, x_off = _norm(h, off, None if w is None else w.astype(np.float64), None if b is None else b.astype(np.float64), layer, eps)
    return h, off, x, x_off


def half(off, v):
    """A bound with one rounding to f16 more."""
    return off + 2.0 ** -11 * (np.abs(v) + off) + 2.0 ** -25


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None):
    """Tokens and probabilities, in 64 bits from sorted rows."""
    n, vocab = logits.shape
    tokens, probs = np.full(n, -1, np.int64), np.zeros(n)
    for r in range(n):
        x = logits[r].astype(np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        m = x.max()
        if m == -np.inf:
            continue
        t = 1.0 if temperature is None else float(temperature[r])
        order = np.argsort(-x, kind="stable")
        if not t >= 2.0 ** -60:
            tokens[r], probs[r] = order[0], 1.0
            continue
        if m == np.inf:
            w = (x == np.inf).astype(np.float64)
        else:
            with np.errstate(over="ignore"):
                w = np.where(x == -np.inf, 0.0, np.exp((x - m) / t))
        k = 0 if top_k is None else int(top_k[r])
        keep = order[:k] if k > 0 else order
        p = 1.0 if top_p is None else float(top_p[r])
        if p < 1:
            sums = np.cumsum(w[keep])
            before = np.concatenate([[0.0], sums[:-1]])
            keep = keep[:max(1, int((before < p * sums[-1]).sum()))]
        q = 0.0 if min_p is None else float(min_p[r])
        if q > 0:
            keep = keep[(w[keep] >= q) | (keep == order[0])]
        keep = np.sort(keep)
        sums = np.cumsum(w[keep])
        u = float(uniform[r])
        u = 0.0 if not u > 0 else u
        at = int(np.searchsorted(sums, u * sums[-1], side="right"))
        if at == len(keep):  # none passes: the last one kept that has weight
            at = int(np.nonzero(w[keep] > 2.0 ** -45)[0][-1])
        tokens[r], probs[r] = keep[at], w[keep[at]] / sums[-1]
    return tokens, probs
