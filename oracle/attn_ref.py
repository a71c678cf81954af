"""Plain reference of the full-attention layers' operators: step plan, rotary embedding, cache
append and paged attention, in Python integers and NumPy float64, written from their
definitions. It shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_EXP = -100
OK, INVALID, EXHAUSTED = 0, 1, 6


def ceil_div(a, b):
    return -(-a // b)


# ---- step plan -----------------------------------------------------------------------------

def plan(ctx, new, table, free, count, page, num_tokens, num_pages):
    """(table, cu, kv_len, positions, slots, count, status) of one step."""
    table = [list(map(int, r)) for r in table]
    max_blocks = len(table[0])
    status = OK
    if not 0 <= count <= num_pages:
        status, count = INVALID, min(max(count, 0), num_pages)
    cu, kv, positions, slots = [0], [], [0] * num_tokens, [-1] * num_tokens
    inside = lambda p: 0 <= p < num_pages  # noqa: E731
    # pages on the stack, from its top, in front of the first that is none
    usable = next((k for k in range(count) if not inside(int(free[count - 1 - k]))), count)
    row, asked, taken = 0, 0, 0
    for b, (c, m) in enumerate(zip(ctx, new)):
        c, m = int(c), int(m)
        end = row + max(m, 0)
        good = c >= 0 and m >= 0 and end <= num_tokens and c + m <= max_blocks * page
        if good and m and c % page and not inside(table[b][c // page]):
            good = False  # the page that its first new tokens go to
        if not good:
            status = max(status, INVALID)
        else:
            have = ceil_div(c, page)
            need = ceil_div(c + m, page) - have
            first = asked
            asked += need
            if need and asked > usable:
                good = False
                status = max(status, EXHAUSTED if asked > count else INVALID)
            elif need:
                taken = asked
                for j in range(need):
                    table[b][have + j] = int(free[count - 1 - first - j])
        kv.append(c + m if good else 0)
        if good:
            for i in range(m):
                pos = c + i
                positions[row + i] = pos
                slots[row + i] = table[b][pos // page] * page + pos % page
        row = end
        cu.append(min(row, num_tokens))
    return table, cu, kv, positions, slots, count - taken, status


def release(kv_len, flags, table, free, count, page, num_pages):
    table, free, status = [list(map(int, r)) for r in table], [int(x) for x in free], OK
    full = False
    for b, f in enumerate(flags):
        if not f:
            continue
        n = ceil_div(kv_len[b], page) if kv_len[b] >= 0 else -1
        pages = table[b][:n] if 0 <= n <= len(table[b]) else None
        if pages is None or any(not 0 <= p < num_pages for p in pages):
            status = INVALID
            continue
        if n and (full or count + n > num_pages):
            status, full = INVALID, True
            continue
        for j in range(n):
            free[count + j] = table[b][j]
            table[b][j] = -1
        count += n
    return table, free, count, status


# ---- rotary embedding ----------------------------------------------------------------------

def rope_axes(half, sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    for i in range(half):
        a = i % len(sections)
        if a and left[a] == 0:
            a = 0
        left[a] -= 1
        out.append(a)
    return out


def rope(x, positions, rot, sections, interleaved, adjacent, theta=None, inv_freq=None):
    """x [T][H][D] float64, positions [axes][T]."""
    half = rot // 2
    axes = rope_axes(half, sections, interleaved)
    y = np.array(x, dtype=np.float64)
    for i in range(half):
        # the angle modulo a turn in extended precision: positions reach 2^31
        wide = np.longdouble
        f = wide(theta) ** (wide(-2 * i) / wide(rot)) if inv_freq is None else wide(inv_freq[i])
        turn = 8 * np.arctan(wide(1))
        w = np.array([float(wide(int(p)) * f % turn) for p in positions[axes[i]]])
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# ---- e4m3 ----------------------------------------------------------------------------------

def e4m3_values():
    """The 256 codes' values (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else -x if c & 128 else x
    return v


def e4m3_codes(x):
    """Codes of the nearest e4m3 values, ties to the even code; beyond 448 to 448; NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    pos = e4m3_values()[:127]
    a = np.minimum(np.abs(x), E4M3_MAX)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.int64)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def scale_of(x):
    """The least power of two s >= 2^-100 with |x| <= 448 s for every finite x."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = float(np.max(a[np.isfinite(a)], initial=0.0))
    e = MIN_EXP
    while a > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(k_codes, v_codes, k_scale, v_scale, slots, k, v):
    """Codes [pages][H][P][D] and scales [pages][H] after storing k, v [T][H][D]."""
    values = e4m3_values()
    codes = [k_codes.copy(), v_codes.copy()]
    scales = [k_scale.astype(np.float64).copy(), v_scale.astype(np.float64).copy()]
    pages, heads, page, _ = k_codes.shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= pages * page:
            t += 1
            continue
        p, off, n = s // page, s % page, 1
        while t + n < len(slots) and off + n < page and slots[t + n] == s + n:
            n += 1
        for h in range(heads):
            kk, vv = np.array(k[t:t + n, h], np.float64), np.array(v[t:t + n, h], np.float64)
            bad = np.isnan(vv).any(axis=1)
            for i, x in enumerate((kk, vv)):
                sc = scale_of(x)
                if off:
                    sc = max(sc, scales[i][p, h])
                    if sc > scales[i][p, h]:
                        old = values[codes[i][p, h, :off]] * (scales[i][p, h] / sc)
                        codes[i][p, h, :off] = e4m3_codes(old)
                scales[i][p, h] = sc
                y = x / sc
                if i == 1:
                    y = np.where(np.isnan(y), 0.0, y)
                else:
                    y[bad] = np.nan
                codes[i][p, h, off:off + n] = e4m3_codes(y)
        t += n
    return codes[0], codes[1], scales[0], scales[1]


# ---- attention -----------------------------------------------------------------------------

def attention(q, k_codes, v_codes, k_scale, v_scale, table, cu, kv_len, scale, causal=True):
    """o [T][Hq][D], lse [T][Hq], and for error bounds: mean |v| under the probabilities
    [T][Hq][D], largest scale * sum |q_d k_d| a row met [T][Hq], largest |v| [T][Hq]."""
    values = e4m3_values()
    tokens, hq, d = q.shape
    pages, hkv, page, _ = k_codes.shape
    group = hq // hkv
    o, mean = np.zeros((tokens, hq, d)), np.zeros((tokens, hq, d))
    lse, size, vmax = np.full((tokens, hq), -np.inf), np.zeros((tokens, hq)), np.zeros((tokens, hq))
    for b in range(len(kv_len)):
        r0, n, kv = int(cu[b]), int(cu[b + 1] - cu[b]), int(kv_len[b])
        ids = [int(x) for x in table[b][:ceil_div(kv, page)]]
        there = np.repeat([0 <= p < pages for p in ids], page)[:kv].astype(bool)
        safe = [p if 0 <= p < pages else 0 for p in ids]
        for h in range(hkv):
            if kv == 0 or n == 0:
                continue
            k = (values[k_codes[safe, h]] * k_scale[safe, h].astype(np.float64)[:, None, None]
                 ).reshape(-1, d)[:kv]
            v = (values[v_codes[safe, h]] * v_scale[safe, h].astype(np.float64)[:, None, None]
                 ).reshape(-1, d)[:kv]
            for i in range(n):
                see = min(max(kv - n + i + 1, 0), kv) if causal else kv
                j = np.nonzero(there[:see])[0]
                if len(j) == 0:
                    continue
                for x in range(h * group, (h + 1) * group):
                    qi = q[r0 + i, x].astype(np.float64)
                    s = scale * (k[j] @ qi)
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    o[r0 + i, x] = p @ v[j] / total
                    lse[r0 + i, x] = m + np.log(total)
                    mean[r0 + i, x] = p @ np.abs(v[j]) / total
                    size[r0 + i, x] = abs(scale) * (np.abs(k[j]) @ np.abs(qi)).max()
                    vmax[r0 + i, x] = np.abs(v[j]).max()
    return o, lse, mean, size, vmax
