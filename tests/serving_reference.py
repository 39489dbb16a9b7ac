"""Plain references of the serving-step operators in 64 bits (numpy), written
from their definitions, for the tests."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
# e4m3 magnitudes of codes 0..0x7E (0x7F is NaN)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest_code(values, v):
    """Index of the nearest of the ascending `values`, ties to the even index, saturating."""
    lo = np.clip(np.searchsorted(values, v, side="right") - 1, 0, len(values) - 2)
    a, b = values[lo], values[lo + 1]
    up = (b - v < v - a) | ((b - v == v - a) & (lo % 2 == 1))
    return np.where(up, lo + 1, lo)


def fp4_rows(x, g):
    """Row codes [n, D] (0..15) and scale bytes [n, D/16] of finite rows."""
    n, D = x.shape
    b = x.astype(np.float64).reshape(n, D // 16, 16)
    sc = nearest_code(E4M3, np.abs(b).max(-1) / (6 * g))
    f = E4M3[sc] * g
    q = np.abs(b) / np.where(f > 0, f, 1)[..., None]
    code = nearest_code(E2M1[:8], q) + np.where(np.signbit(b), 8, 0)
    code = np.where((f > 0)[..., None], code, 0)
    return code.reshape(n, D), sc.astype(np.uint8)


def pack_page(codes, scales):
    """Bytes of one page from its rows' codes and scale bytes."""
    c = codes.astype(np.uint8)
    return np.concatenate([(c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1), scales.reshape(-1)])


def fp4_row_values(cache, loc, D, g):
    """Values [D] of the row at a cache location (cache uint8 [pages, page, D/2 + D/16])."""
    pages, ps, _ = cache.shape
    flat = cache.reshape(pages, -1)[loc // ps]
    r = loc % ps
    c = flat[r * (D // 2):(r + 1) * (D // 2)]
    s = flat[ps * (D // 2) + r * (D // 16): ps * (D // 2) + (r + 1) * (D // 16)]
    v = np.empty(D)
    v[0::2], v[1::2] = E2M1[c & 15], E2M1[c >> 4]
    return v * np.repeat(E4M3[s & 127] * np.where(s & 128, -1, 1), 16) * g


def attention(q, cache, table, row_start, ctx, scale, g, sink=None):
    """(out, lse, seen): out/lse of tokens with ctx >= 0, seen marks them."""
    T, H, D = q.shape
    ps = cache.shape[1]
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    seen = np.zeros(T, bool)
    for b in range(len(row_start) - 1):
        lo, hi = row_start[b], row_start[b + 1]
        L = max([0, *ctx[lo:hi]])
        ok = np.array([0 <= table[b][j // ps] < cache.shape[0] for j in range(L)], bool)
        k = np.array([fp4_row_values(cache, table[b][j // ps] * ps + j % ps, D, g) if ok[j] else np.zeros(D)
                      for j in range(L)]).reshape(L, D)
        for t in range(lo, hi):
            if ctx[t] < 0:
                continue
            seen[t] = True
            z = q[t].astype(np.float64) @ k[:ctx[t]].T * scale
            z[:, ~ok[:ctx[t]]] = -np.inf
            top = z.max(-1, initial=-np.inf)
            if sink is not None:
                top = np.maximum(top, sink)
            safe = np.where(np.isfinite(top), top, 0)
            e = np.exp(z - safe[:, None])
            tot = e.sum(-1) + (np.exp(sink - safe) if sink is not None else 0)
            with np.errstate(divide="ignore"):
                lse[t] = np.where(tot > 0, safe + np.log(np.where(tot > 0, tot, 1)), -np.inf)
            out[t] = np.where((tot > 0)[:, None], e @ k[:ctx[t]] / np.where(tot > 0, tot, 1)[:, None], 0)
    return out, lse, seen


def norm_rope(x, pos, table, w, R, at, interleaved, eps):
    """Rows of x [T, H, D] normed and rotated; rows of skipped tokens are None-like zeros."""
    T, H, D = x.shape
    y = np.zeros((T, H, D))
    half = R // 2
    for t in range(T):
        if pos[t] < 0:
            continue
        z = x[t].astype(np.float64)
        z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
        if w is not None:
            z = z * w.astype(np.float64)
        o = z.copy()
        for i in range(half):
            a, b = (at + 2 * i, at + 2 * i + 1) if interleaved else (at + i, at + half + i)
            c, s = float(table[pos[t], i]), float(table[pos[t], half + i])
            o[:, a] = z[:, a] * c - z[:, b] * s
            o[:, b] = z[:, b] * c + z[:, a] * s
        y[t] = o
    return y


def step_maps(seq, n, table, free, cursor, P, ps, T, tails=None):
    """All maps of one step, request by request and token by token."""
    table = table.copy()
    m = {k: np.full(T, -1, np.int64) for k in
         ("positions", "batch_ids", "slot_mapping", "cache_loc", "tail_slots", "row_positions", "ctx_rows")}
    start, at = [0], cursor
    for b in range(len(seq)):
        s, k = int(seq[b]), int(n[b])
        have, need = -(-((s - k) // P) // ps), -(-(s // P) // ps)
        for pg in range(have, need):
            table[b][pg] = free[at]
            at += 1
        for i in range(k):
            t, pos = start[-1] + i, s - k + i
            m["positions"][t], m["batch_ids"][t], m["ctx_rows"][t] = pos, b, (pos + 1) // P
            if (pos + 1) % P == 0:
                r = pos // P
                m["cache_loc"][t] = m["slot_mapping"][t] = table[b][r // ps] * ps + r % ps
                m["row_positions"][t] = pos - P + 1
            if tails is not None and tails[b] >= 0:
                m["tail_slots"][t] = tails[b] * P + pos % P
        start.append(start[-1] + k)
    m["row_start"] = np.array(start)
    if tails is None:
        del m["tail_slots"]
    return m, table, at
