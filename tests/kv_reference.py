"""Plain references of the operators around the uncompressed cache, in 64 bits and from their
definitions, for the tests."""
import torch


def seen_rows(ctx, window, first, draft_bits=None):
    """Rows that a token sees: ctx committed rows (with the token itself where there are no drafts), and
    the drafts a of draft_bits, which are rows ctx + a."""
    n = 0 if draft_bits is None else len(draft_bits)
    rows = [j for j in range(ctx) if window == 0 or j >= ctx + n - window or j < first]
    return rows + [ctx + a for a in (draft_bits or ())]


def bits_of(words):
    """Set bits of a mask's int64 words."""
    return [w * 64 + i for w, x in enumerate(words) for i in range(64) if (x >> i) & 1]


def attention(q, k, v, table, row_start, ctx, scale, window=0, first=0, mask=None, sink=None, max_rows=None):
    """(out, lse, seen, spread, slack): results of tokens with ctx >= 0 (seen marks them), sum_j w_j |v_j|,
    and sum_d |q_d k_jd| * scale at its largest, from which tolerances are formed.  k, v [pages, page_size,
    KH, D]; missing pages count as unseen."""
    T, H, D = q.shape
    pages, ps, KH, _ = k.shape
    G = H // KH
    f64 = dict(dtype=torch.float64, device=q.device)
    out, spread = torch.zeros(T, H, D, **f64), torch.zeros(T, H, D, **f64)
    lse, slack = torch.full((T, H), -torch.inf, **f64), torch.zeros(T, H, **f64)
    seen = torch.zeros(T, dtype=torch.bool)
    tab, words = table.tolist(), None if mask is None else mask.tolist()
    for b in range(len(row_start) - 1):
        for t in range(int(row_start[b]), min(int(row_start[b + 1]), T)):
            if ctx[t] < 0:
                continue
            seen[t] = True
            c = int(ctx[t]) if max_rows is None else min(int(ctx[t]), max_rows)
            rows = seen_rows(c, window, first, None if words is None else bits_of(words[t]))
            if max_rows is not None:
                rows = [j for j in rows if j < max_rows]
            rows = [j for j in rows if 0 <= tab[b][j // ps] < pages]
            if sink is not None:
                lse[t] = sink.double()
            if not rows:
                continue
            pg = torch.tensor([tab[b][j // ps] for j in rows], device=q.device)
            at = torch.tensor([j % ps for j in rows], device=q.device)
            kk, vv = k[pg, at].double(), v[pg, at].double()  # [L, KH, D]
            qq = q[t].double().view(KH, G, D)
            z = torch.einsum("kgd,lkd->kgl", qq, kk) * scale
            slack[t] = (torch.einsum("kgd,lkd->kgl", qq.abs(), kk.abs()) * abs(scale)).amax(-1).view(H)
            if sink is not None:
                z = torch.cat([z, sink.double().view(KH, G, 1)], -1)
            total = torch.logsumexp(z, -1)
            w = torch.exp(z - total[..., None])[..., :len(rows)]
            lse[t] = total.view(H)
            out[t] = torch.einsum("kgl,lkd->kgd", w, vv).reshape(H, D)
            spread[t] = torch.einsum("kgl,lkd->kgd", w, vv.abs()).reshape(H, D)
    return out, lse, seen, spread, slack


def rotate(x, pos, table, at, interleaved):
    """Rows of x [T, H, D] rotated; rows of tokens with pos < 0 are unchanged."""
    z = x.double().clone()
    R = table.shape[1]
    half = R // 2
    for t, p in enumerate(pos.tolist()):
        if p < 0:
            continue
        c, s = table[p, :half].double(), table[p, half:].double()
        i = torch.arange(half, device=x.device)
        a, b = (at + 2 * i, at + 2 * i + 1) if interleaved else (at + i, at + half + i)
        u, w = x[t][:, a].double(), x[t][:, b].double()
        z[t][:, a], z[t][:, b] = u * c - w * s, w * c + u * s
    return z


def tree(parents, row_start, ctx, words):
    """(mask bits as sets, positions) of every row; rows without a token have an empty set and -1."""
    T = len(parents)
    masks, pos = [set() for _ in range(T)], [-1] * T
    for b in range(len(row_start) - 1):
        lo, hi = row_start[b], min(row_start[b + 1], T)
        for i in range(min(hi - lo, 64 * words)):
            if ctx is not None and ctx[lo + i] < 0:
                continue
            x, chain = i, set()
            while x >= 0:
                chain.add(x)
                p = parents[lo + x]
                x = p if -1 <= p < x else -1
            masks[lo + i] = chain
            pos[lo + i] = (0 if ctx is None else ctx[lo + i]) + len(chain) - 1
    return masks, pos


def pack(masks, words):
    """int64 [T, words] of sets of bits."""
    rows = [[sum(1 << (a % 64) for a in m if a // 64 == w) for w in range(words)] for m in masks]
    return torch.tensor([[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in rows], dtype=torch.int64).view(len(masks), words)


def merge(outs, lses):
    s = torch.stack([x.double() for x in lses])
    lse = torch.logsumexp(s, 0)
    w = torch.where(s == -torch.inf, torch.zeros_like(s), torch.exp(s - torch.where(lse == -torch.inf, torch.zeros_like(lse), lse)))
    o = torch.stack([x.double() for x in outs])
    o = torch.where((w == 0)[..., None], torch.zeros_like(o), o)
    return (w[..., None] * o).sum(0), lse, (w[..., None] * o.abs()).sum(0)
