"""Plain fp64 references of the calls around the recurrent layers (short convolution, selective
scan, RMS norm, sampling), written from their formulas; test infrastructure only."""
from __future__ import annotations

import numpy as np

SILU = 1


def silu(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return v / (1.0 + np.exp(-v))


def conv(x, weight, bias, act, state):
    """One request: x [n, C], state [W-1, C] (the inputs in front). Returns y, the sums of the
    terms' absolute values, and the extended line of inputs [W-1+n, C]."""
    w = weight.shape[1]
    line = np.concatenate([state, x])
    n = len(x)
    acc = np.zeros_like(x) if bias is None else np.tile(bias, (n, 1))
    mag = np.abs(acc)
    for j in range(w):
        acc = acc + line[j:j + n] * weight[:, j]
        mag = mag + np.abs(line[j:j + n] * weight[:, j])
    return (silu(acc) if act == SILU else acc), mag, line


def softplus(v):
    return np.logaddexp(v, 0.0)


def ssm(x, delta, b, c, z, a, d, delta_bias, soft, state, groups):
    """One request: x, delta, z [n, C]; b, c [n, G, N]; state [C, N]. Returns y, the states after
    every row [n + 1, C, N], and bounds of the fp32 errors of y and of the states.

    The bounds follow the recurrence. A decay exp(dt a) is off by 2^-21 of itself (the ex2
    instruction) and, through its exponent (dt off by 2^-20 of itself, three roundings more), by
    |dt a| 2^-19; an added term by 2^-20 of itself; each new state by a rounding, 2^-24. The sum
    over N states adds N roundings of its terms' absolute values."""
    n, ch = x.shape
    per = ch // groups
    v = delta + (0.0 if delta_bias is None else delta_bias)
    dt = softplus(v) if soft else v
    h, e = state.astype(np.float64), np.zeros_like(state, dtype=np.float64)
    mag = np.abs(h)
    hs, es = [h], [e]
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for t in range(n):
        bt, ct = (np.repeat(k[t], per, axis=0) for k in (b, c))
        w = dt[t][:, None] * a
        decay = np.exp(w)
        add = (dt[t] * x[t])[:, None] * bt
        e = decay * e + decay * mag * (2.0 ** -21 + np.abs(w) * 2.0 ** -19) \
            + np.abs(add) * 2.0 ** -20
        mag = decay * mag + np.abs(add)
        e = e + mag * 2.0 ** -23
        h = decay * h + add
        skip = 0.0 if d is None else d * x[t]
        y[t] = (ct * h).sum(1) + skip
        bound[t] = (np.abs(ct) * (e + mag * h.shape[1] * 2.0 ** -23)).sum(1) \
            + np.abs(skip) * 2.0 ** -22
        hs.append(h)
        es.append(e)
    if z is not None:
        g = silu(z)
        # silu in fp32: 2^-20 of itself, and the exponent's rounding
        bound = np.abs(g) * (bound + np.abs(y) * (2.0 ** -20 + np.abs(z) * 2.0 ** -22))
        y = y * g
    return y, np.stack(hs), bound, np.stack(es)


def rms_norm(x, residual, weight, offset, eps, heads, gate):
    """Rows [n, heads * dim]. Returns s, v."""
    s = x if residual is None else x + residual
    n = len(s)
    h = s.reshape(n, heads, -1)
    v = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if weight is not None:
        v = v * (weight + offset)
    v = v.reshape(n, -1)
    return s, (v if gate is None else v * silu(gate))


def sample_row(logits, temperature, top_k, top_p, min_p, u):
    """(token, its log-probability, how near the closest border was, as a share of the weight)."""
    l = np.where(np.isnan(logits), -np.inf, logits)
    top = l.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if temperature == 0:
        return int(np.argmax(l)), 0.0, 1.0
    if top == np.inf:
        w = (l == np.inf).astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((l - top) / temperature)
    order = np.lexsort((np.arange(len(l)), -l))
    near = 1.0
    if 0 < top_k < len(l):
        order = order[:top_k]
    if top_p < 1:
        part = np.cumsum(w[order])
        share = part / part[-1]
        near = min(near, np.abs(share - top_p).min())
        n = int((share < top_p).sum()) + 1
        order = order[:max(1, min(n, len(order)))]
    if min_p > 0:
        near = min(near, np.abs(w[order] - min(min_p, 1.0))[w[order] < 1].min(initial=1.0))
        order = order[w[order] >= min(min_p, 1.0)]
    order = np.sort(order[w[order] > 0])
    part = np.cumsum(w[order])
    share = part / part[-1]
    near = min(near, np.abs(share[:-1] - u).min(initial=1.0))
    at = min(int((share <= u).sum()), len(order) - 1)
    return int(order[at]), float(np.log(w[order[at]] / part[-1])), near
