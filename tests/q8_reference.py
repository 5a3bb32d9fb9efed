"""Plain references of the paged 8-bit latent cache, in whole numbers and 64 bits on
the CPU, written from the definitions in ddt.h request by request."""
from __future__ import annotations

import math

import numpy as np

PAGE, HEADS, LATENT, ROPE = 64, 64, 512, 64
MIN_EXP = -40
OK, BAD_INDEX, BAD_PREFIX, BAD_LENGTH, NO_PAGES, NOT_FINITE = 0, 2, 4, 5, 7, 8


def decode_table() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f NaN."""
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[b] = math.nan if b & 0x7F == 0x7F else (-x if b & 0x80 else x)
    return v


DECODE = decode_table()


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte, ties to the even one, saturating; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    mags = DECODE[:0x7F]                       # ascending magnitudes 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 1, 0x7E)
    lo = hi - 1
    down, up = a - mags[lo], mags[hi] - a
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    out = (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), out)


def fit(amax: float) -> float:
    e = MIN_EXP
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def pages(prefix, rows, table, n_blocks, free, n_free, num_pages):
    """ddt_kv_pages on lists; returns (slots per request, status), changing the state."""
    B, width = table.shape
    st, need = [OK] * B, [0] * B
    for b in range(B):
        if rows[b] < 0:
            st[b] = BAD_LENGTH
        elif prefix[b] < 0 or prefix[b] + rows[b] > width * PAGE:
            st[b] = BAD_PREFIX
        elif not 0 <= n_blocks[b] <= width:
            st[b] = BAD_INDEX
        else:
            need[b] = -(-(prefix[b] + rows[b]) // PAGE)
    back = [(b, j) for b in range(B) if st[b] == OK for j in range(need[b], n_blocks[b])]
    if not 0 <= n_free[0] <= n_free[0] + len(back) <= num_pages:
        return [[-1] * max(0, r) for r in rows], [BAD_INDEX] * B
    for b, j in reversed(back):                # so that the first one given back is on top
        free[n_free[0]] = table[b, j]
        n_free[0] += 1
        table[b, j] = -1
    for b in range(B):
        if st[b] == OK:
            n_blocks[b] = min(n_blocks[b], need[b])
    open_ = True
    for b in range(B):
        if st[b] != OK or need[b] == n_blocks[b]:
            continue
        open_ = open_ and need[b] - n_blocks[b] <= n_free[0]
        if not open_:
            st[b] = NO_PAGES
            continue
        while n_blocks[b] < need[b]:
            n_free[0] -= 1
            table[b, n_blocks[b]] = free[n_free[0]]
            n_blocks[b] += 1
    slots = []
    for b in range(B):
        mine = []
        for i in range(max(0, rows[b])):
            pos = prefix[b] + i
            page = table[b, pos // PAGE] if st[b] == OK else -1
            mine.append(int(page) * PAGE + pos % PAGE if 0 <= page < num_pages else -1)
        slots.append(mine)
    return slots, st


def write(cache, scales, table, prefix, rows):
    """ddt_kv_write_q8: cache uint8 [pages, 64, 576], rows a list of fp64 [n, 576]."""
    status = []
    for b, x in enumerate(rows):
        n, at = len(x), 0
        need = range(prefix[b] // PAGE, -(-(prefix[b] + n) // PAGE)) if prefix[b] >= 0 else ()
        if prefix[b] < 0 or prefix[b] + n > table.shape[1] * PAGE:
            status.append(BAD_PREFIX)
            continue
        if n and any(not 0 <= table[b, k] < len(cache) for k in need):
            status.append(BAD_INDEX)
            continue
        status.append(OK if np.isfinite(x).all() else NOT_FINITE)
        while at < n:
            pos = prefix[b] + at
            page, off = table[b, pos // PAGE], pos % PAGE
            m = min(PAGE - off, n - at)
            y = x[at:at + m]
            finite = np.abs(y[np.isfinite(y)])
            scale = fit(finite.max() if finite.size else 0.0)
            if off and scales[page] >= scale:
                scale = float(scales[page])
            elif off:
                cache[page, :off] = encode(DECODE[cache[page, :off]] * (float(scales[page]) / scale))
            cache[page, off:off + m] = encode(np.where(np.isnan(y), 0.0, y) / scale)
            scales[page] = scale
            at += m
    return status


def compact(cache, scales, table, prefix, path, accept):
    """ddt_kv_compact_q8; returns (new prefixes, status)."""
    new, status = [], []
    for b, P in enumerate(prefix):
        q, alen = path.shape[1], accept[b]
        st = OK
        if not 1 <= alen <= q:
            st = BAD_LENGTH
        elif P < 0 or P + q > table.shape[1] * PAGE:
            st = BAD_PREFIX
        elif any(not 0 <= table[b, k] < len(cache) for k in range(P // PAGE, (P + q - 1) // PAGE + 1)) \
                or any(not 0 <= path[b, i] < q for i in range(alen)):
            st = BAD_INDEX
        status.append(st)
        new.append(P + (alen if st == OK else 0))
        if st != OK:
            continue
        home = [((P + i) // PAGE, (P + i) % PAGE) for i in range(alen)]
        src = [((P + int(j)) // PAGE, (P + int(j)) % PAGE) for j in path[b, :alen]]
        was = {k: float(scales[table[b, k]]) for k in range(P // PAGE, (P + q - 1) // PAGE + 1)}
        taken = [cache[table[b, k], o].copy() for k, o in src]
        now = {k: max([was[k]] + [was[s[0]] for h, s in zip(home, src) if h[0] == k]) for k in was}
        for k in was:
            if now[k] != was[k]:
                page = table[b, k]
                cache[page] = encode(DECODE[cache[page]] * (was[k] / now[k]))
                scales[page] = now[k]
        for (k, o), (ks, _), row in zip(home, src, taken):
            cache[table[b, k], o] = encode(DECODE[row] * (was[ks] / now[k]))
    return new, status


def attend(query, cache, scales, table, P, vis, scale):
    """One request of ddt_verify_attn_q8: query fp64 [Q, 64, 576], vis bool [Q, Q].
    Returns out, lse, and the terms of the error bound: the weighted mean magnitude
    sum p |c|, the bound's quantum term, and the score error (see error_bound)."""
    Q = query.shape[0]
    T = P + Q
    blocks = [int(p) for p in table[:-(-T // PAGE)]]
    step = np.repeat(np.array([float(scales[p]) if 0 <= p < len(cache) else 0.0 for p in blocks]), PAGE)[:T]
    raw = np.concatenate([DECODE[cache[p]] if 0 <= p < len(cache) else np.zeros((PAGE, 576))
                          for p in blocks])[:T]
    key = raw * step[:, None]
    seen = np.ones((Q, T), bool)
    seen[:, P:] = vis
    s = scale * (query.reshape(-1, 576) @ key.T).reshape(Q, HEADS, T)
    s = np.where(seen[:, None, :], s, -np.inf)
    top = s.max(2, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - top)
    z = e.sum(2, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        p = np.where(z > 0, e / z, 0.0)
        lse = np.where(z[..., 0] > 0, top[..., 0] + np.log(z[..., 0]), -np.inf)
    c = key[:, :LATENT]
    flat = p.reshape(-1, T)
    out = (flat @ c).reshape(Q, HEADS, LATENT)
    mean = (flat @ np.abs(c)).reshape(Q, HEADS, LATENT)
    top_w = (p * step).max(2, keepdims=True)
    quantum = 2.0 ** -14 * top_w * np.abs(raw[:, :LATENT]).sum(0)
    aq, ak = np.abs(query.reshape(-1, 576)), np.abs(key)
    off = scale * (2.0 ** -17 * aq.max(1, keepdims=True) * ak.sum(1) + 640 * 2.0 ** -24 * (aq @ ak.T))
    off = (off.max(1) + 2.0 ** -20 * (1 + np.abs(s[np.isfinite(s)]).max(initial=0.0))).reshape(Q, HEADS)
    return out, lse, mean, quantum, off


def error_bound(out, mean, quantum, off):
    """How far the call's bf16 output may be from `out`.  Each weight enters P V as two
    e4m3 terms: relative error 2^-8, or, far below the largest one, 2^-10 where the
    largest weight times its page's scale is at least 2^4 (the quantum term).  A score
    that is off by `off` (queries in two e4m3 terms: half a step, 2^-10, against a largest
    value above 224 > 2^7; 640 fp32 additions) changes weights by that factor, above and below the line.  The
    result is rounded to bf16 once: 2^-8."""
    return (2.0 ** -8 + 2.0 * off[..., None]) * mean + quantum + 2.0 ** -8 * np.abs(out) + 1e-30
