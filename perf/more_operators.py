"""Measured cases of the operators around a paged cache of uncompressed keys and values:

* append: keys and values of a step's tokens into their cache rows, keys (and queries) rotated on the way;
* attention over that cache with a sliding window and a few first rows that stay visible;
* tree masks: which drafted tokens see which, and their positions, from each token's parent;
* attention for a tree of drafted tokens over the cache;
* merge: one result of attentions over different rows (the window and the compressed rows).

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, with
`own` true, through this package.  `exact` computes it from its definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four requests, one token each: latency
        dict(name="append_few", op="append", T=4, H=16, KH=2, D=128, R=128, at=0, pairs=False, dtype="bf16", page=64,
             heads_first=False, shared=False, skip=0.0),
        # a prompt slice with an odd token count
        dict(name="append_prompt", op="append", T=8191, H=32, KH=8, D=128, R=128, at=0, pairs=False, dtype="bf16", page=64,
             heads_first=False, shared=False, skip=0.0),
        # eight requests with small drafts: latency
        dict(name="masks_few", op="masks", B=8, n_min=16, n_max=16),
        # a full batch of drafts, ragged
        dict(name="masks_many", op="masks", B=1024, n_min=1, n_max=250),
        # four short requests: latency
        dict(name="window_few", op="window", B=4, n_min=1, n_max=1, H=16, KH=2, D=128, window=128, first=4, ctx_min=1,
             ctx_max=300, page=64, heads_first=False, sink=False),
        # decode with grouped heads: long contexts of which a window and the first rows are left
        dict(name="window_decode", op="window", B=256, n_min=1, n_max=1, H=64, KH=8, D=128, window=1024, first=16, ctx_min=1,
             ctx_max=32768, page=64, heads_first=False, sink=False),
        # the last chunk of a c128 decode step: rows that are key and value of 64 heads, before they are compressed
        dict(name="window_chunk", op="window", B=1024, n_min=1, n_max=1, H=64, KH=1, D=512, window=128, first=0, ctx_min=1,
             ctx_max=32768, page=64, heads_first=False, sink=True),
        # ragged prompt slices behind their prefixes
        dict(name="window_prompt", op="window", B=9, n_min=600, n_max=3000, H=32, KH=8, D=128, window=1024, first=16, ctx_min=0,
             ctx_max=16384, page=64, heads_first=False, sink=False),
        # two requests, a small draft: latency
        dict(name="tree_few", op="tree", B=2, n_min=16, n_max=16, H=16, KH=2, D=128, window=0, first=0, ctx_min=100, ctx_max=1000,
             page=64, heads_first=False, sink=False),
        # verification of wide drafts over whole contexts
        dict(name="tree_verify", op="tree", B=128, n_min=40, n_max=64, H=32, KH=8, D=128, window=0, first=0, ctx_min=0,
             ctx_max=4096, page=64, heads_first=False, sink=False),
        # four tokens of a window and a compressed part
        dict(name="merge_few", op="merge", T=4, H=16, D=128, parts=2, empty=0.25),
        # the c128 decode step: both parts of 1024 tokens x 64 heads
        dict(name="merge_decode", op="merge", T=1024, H=64, D=512, parts=2, empty=1 / 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "masks", "window", "window", "tree", "merge"])
    if op == "masks":
        n = _log(rng, 1, 256)
        return dict(op=op, B=_log(rng, 1, 1024), n_min=rng.choice([0, n // 2, n]), n_max=n)
    D = rng.choice([128, 128, 256, 512])
    if op == "merge":
        H = rng.randint(1, 64)
        parts = rng.randint(2, 4)
        return dict(op=op, T=_log(rng, 1, 60_000_000 // (H * D * parts)), H=H, D=D, parts=parts, empty=rng.choice([0.0, 0.25]))
    KH = rng.choice([1, 1, 2, 4, 8])
    H = KH * rng.choice([1, 2, 4, 5, 8, 16] if KH > 1 else [1, 7, 16, 32, 64])
    page, heads_first = rng.choice([16, 48, 64, 100]), rng.random() < 0.3
    if op == "append":
        R = 2 * rng.randint(4, D // 2)
        return dict(op=op, T=_log(rng, 1, 40_000_000 // ((H + 2 * KH) * D)), H=H, KH=KH, D=D, R=R, at=2 * rng.randint(0, (D - R) // 2),
                    pairs=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]), page=page, heads_first=heads_first,
                    shared=rng.random() < 0.3, skip=rng.choice([0.0, 0.3]))
    more = dict(H=H, KH=KH, D=D, page=page, heads_first=heads_first, sink=rng.random() < 0.4)
    if op == "tree":
        n, B = _log(rng, 2, 130), _log(rng, 1, 64)
        window = rng.choice([0, 0, _log(rng, 130, 2048)])
        top = max(40, min(4096, 30_000_000_000 // (B * n * H * D), 200_000_000 // (B * KH * D)))
        ctx = _log(rng, 20, top + 1)
        return dict(op=op, B=B, n_min=rng.choice([1, n]), n_max=n, window=window, first=rng.choice([0, 4, 50]),
                    ctx_min=rng.choice([0, ctx // 2]), ctx_max=ctx, **more)
    window, first = rng.choice([0, _log(rng, 8, 2048), _log(rng, 8, 2048)]), rng.choice([0, 1, 4, 16, 100])
    if rng.random() < 0.6:  # single tokens or a few
        n, B = rng.choice([1, 1, 1, 4]), _log(rng, 1, 512)
        span = window + first if window else 8192
        B = max(1, min(B, 250_000_000 // (span * KH * D), 40_000_000_000 // (n * H * D * span)))
        return dict(op=op, B=B, n_min=1, n_max=n, window=window, first=first, ctx_min=0,
                    ctx_max=_log(rng, 16, 32768 if window else 8192), **more)
    B, n = rng.randint(1, 8), _log(rng, 16, 3000)
    ctx = _log(rng, 20, 16384 if window else 2000)
    n = max(16, min(n, 40_000_000_000 // (B * H * D * (window + first if window else ctx + n))))
    return dict(op=op, B=B, n_min=n // 4, n_max=n, window=window, first=first, ctx_min=0, ctx_max=ctx, **more)


# ------------------------------------------------------------------ helpers of prepare
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _host_gen(seed):
    return torch.Generator().manual_seed(seed * 7919 + 17)


def _token_counts(c):
    """Tokens of each request in this step: a batch's shape goes with its case, not with the seed."""
    n = _ints(_host_gen(c["B"] * 31 + c["n_max"]), c["n_min"], c["n_max"], c["B"])
    n[0] = max(1, int(n[0]))
    return n


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _starts(n):
    return torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])


def _blank_cache(c, pages):
    """A zeroed cache [pages, page_size, KH, D], rows or heads outermost in a page."""
    if c["heads_first"]:
        return torch.zeros(pages, c["KH"], c["page"], c["D"], dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    return torch.zeros(pages, c["page"], c["KH"], c["D"], dtype=torch.bfloat16, device=DEV)


# ------------------------------------------------------------------ append
def _cos_sin(n, R):
    """Rows of cos | sin of the angles position / 10000^(2i/R), formed in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_append(c, seed):
    g = _gen(seed)
    T, H, KH, D = c["T"], c["H"], c["KH"], c["D"]
    last = 32768
    kt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    pages = -(-T // c["page"]) + 2
    loc = torch.randperm(pages * c["page"], generator=g, device=DEV)[:T]
    live = torch.rand(T, generator=g, device=DEV) >= c["skip"]
    live[0] = True
    pos = torch.randint(0, last, (T,), generator=g, device=DEV, dtype=torch.int32)
    # queries, keys and values side by side, as a projection leaves them
    both = torch.randn(T, H + (1 if c["shared"] else 2) * KH, D, generator=g, device=DEV).to(kt)
    return dict(c=c, q=both[:, :H], k=both[:, H:H + KH], v=None if c["shared"] else both[:, H + KH:],
                loc=torch.where(live, loc, torch.full_like(loc, -1)), pos=torch.where(live, pos, torch.full_like(pos, -1)),
                table=_cos_sin(last, c["R"]), k_cache=_blank_cache(c, pages),
                v_cache=None if c["shared"] else _blank_cache(c, pages),
                q_out=torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV))


def _rotate(x, pos, c, table):
    R, at = c["R"], c["at"]
    x = x.float()
    cs = table[pos.clamp(min=0).long()][:, None, :]
    cos, sin = cs[..., :R // 2], cs[..., R // 2:]
    r = x[..., at:at + R]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :R // 2], r[..., R // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, w], -1).flatten(-2) if c["pairs"] else torch.cat([u, w], -1)
    return torch.cat([x[..., :at], r, x[..., at + R:]], -1).to(torch.bfloat16)


def _put(cache, loc, rows):
    """Rows without a location go to row loc[0] with that row's own values."""
    page = cache.shape[1]
    live = loc >= 0
    at = torch.where(live, loc, loc[0])
    cache[at // page, at % page] = torch.where(live[:, None, None], rows, rows[:1])


def _run_append(st):
    c = st["c"]
    if own:
        import compressed_kv_attention_gated_gb300 as ck

        ck.ckv_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["loc"], positions=st["pos"], cos_sin=st["table"],
                         rope_offset=c["at"], interleaved=c["pairs"], q=st["q"], q_out=st["q_out"])
        return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"] if st["v"] is not None else 0}
    _put(st["k_cache"], st["loc"], _rotate(st["k"], st["pos"], c, st["table"]))
    if st["v"] is not None:
        _put(st["v_cache"], st["loc"], st["v"].to(torch.bfloat16))
    q = _rotate(st["q"], st["pos"], c, st["table"])
    live = (st["pos"] >= 0)[:, None, None]
    return {"q": torch.where(live, q, torch.zeros_like(q)), "k": st["k_cache"], "v": st["v_cache"] if st["v"] is not None else 0}


# ------------------------------------------------------------------ tree masks
def _parents(h, n):
    """Drafts as a search leaves them: a token's parent is one of those before it, often a late one, or none (-1)."""
    out = []
    for m in n.tolist():
        i = torch.arange(m)
        u = torch.rand(m, generator=h)
        out.append((i * (1 - u * u * 0.6)).long().clamp(max=i) - 1)
    return torch.cat(out)


def _words(c):
    return max(1, -(-c["n_max"] // 64))


def _prepare_masks(c, seed):
    h = _host_gen(seed)
    n = _token_counts(c)
    ctx = torch.repeat_interleave(_ints(h, 0, 32768, c["B"]), n)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(c=c, n_max=int(n.max()), parents=_parents(h, n).to(**i32), start=_starts(n).to(**i32), ctx=ctx.to(**i32))


def _run_masks(st):
    c = st["c"]
    W = _words(c)
    if own:
        import compressed_kv_attention_gated_gb300 as ck

        mask, pos = ck.ckv_build_tree_masks(st["parents"], st["start"], st["ctx"], W)
        return {"mask": mask, "positions": pos}
    B, N, T = c["B"], st["n_max"], st["parents"].numel()
    start = st["start"].long()
    i = torch.arange(N, device=DEV)
    live = i < (start[1:] - start[:-1])[:, None]
    p = st["parents"].long()[(start[:B, None] + i).clamp(max=T - 1)]
    # token i reaches j in one step or none; squaring doubles the steps
    up = ((p[..., None] == i) & live[..., None]).float() + torch.eye(N, device=DEV)
    for _ in range(max(1, (N - 1).bit_length())):
        up = ((up @ up) > 0).float()
    bits = torch.zeros(B, N, W * 64, dtype=torch.int64, device=DEV)
    bits[..., :N] = up.long()
    word = (bits.view(B, N, W, 64) << torch.arange(64, device=DEV)).sum(-1)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:], t, right=True)
    mask = word[b, t - start[b]]
    depth = up.sum(-1).long()[b, t - start[b]] - 1
    return {"mask": mask, "positions": (st["ctx"].long() + depth).to(torch.int32)}


# ------------------------------------------------------------------ attention: window, first rows, drafts
def _prepare_attention(c, seed):
    g, h = _gen(seed), _host_gen(seed)
    B, H, KH, D, page, tree = c["B"], c["H"], c["KH"], c["D"], c["page"], c["op"] == "tree"
    n = _token_counts(c)
    before = _ints(h, c["ctx_min"], c["ctx_max"], B)  # rows of each request before this step
    total = before + n
    T, start = int(n.sum()), _starts(n)
    b = torch.repeat_interleave(torch.arange(B), n)
    i = torch.arange(T) - start[b]
    # pages that no token of the step sees have been given back
    width = -(-int(total.max()) // page)
    row0 = torch.arange(width) * page
    held = row0[None, :] < total[:, None]
    if c["window"]:
        low = (before + 1 - c["window"])[:, None]
        held &= (row0[None, :] + page > low) | (row0 < c["first"])[None, :]
    need = held.sum(1)
    pages = int(need.sum()) + 2
    perm = torch.randperm(pages, generator=h)
    order = torch.cumsum(held.flatten().long(), 0).view_as(held) - 1
    table = torch.where(held, perm[order.clamp(min=0)], -1)
    # rows that no token has written hold whatever memory held: zeros here
    k = _blank_cache(c, pages)
    v = k if D == 512 else _blank_cache(c, pages)
    k.normal_(generator=g)
    if v is not k:
        v.normal_(generator=g)
    q = torch.randn(T, H, D, generator=g, device=DEV)
    # rows that a query looks for: scores spread over several units, as after training
    q *= 1.5
    i32 = dict(dtype=torch.int32, device=DEV)
    st = dict(c=c, T=T, n_max=int(n.max()), rows_max=int(total.max()), q=q.to(torch.bfloat16), k=k, v=v, table=table.to(**i32),
              start=start.to(**i32), ctx=(before[b] if tree else before[b] + i + 1).to(**i32), scale=1.0 / math.sqrt(D),
              before=before.to(**i32), mask=None, sink=torch.randn(H, generator=g, device=DEV) if c["sink"] else None,
              out=torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV), lse=torch.empty(T, H, device=DEV))
    if tree:
        par = _parents(h, n).tolist()
        rows, at = [], start.tolist()
        for r in range(B):
            seen = []
            for x in range(at[r], at[r + 1]):
                seen.append((1 << (x - at[r])) | (seen[par[x]] if par[x] >= 0 else 0))
            rows += seen
        W = _words(c)
        words = [[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(W)] for m in rows]
        st["mask"] = torch.tensor([[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in words], dtype=torch.int64).to(DEV)
    return st


def _run_attention(st):
    c = st["c"]
    if own:
        import compressed_kv_attention_gated_gb300 as ck

        ck.ckv_kv_attention(st["q"], st["k"], st["v"], st["table"], st["start"], st["ctx"], st["rows_max"], st["scale"],
                            window=c["window"], first_rows=c["first"], tree_mask=st["mask"], sink=st["sink"], out=st["out"],
                            lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    B, H, KH, D, T, N = c["B"], c["H"], c["KH"], c["D"], st["T"], st["n_max"]
    page, window, first = c["page"], c["window"], c["first"]
    start, before = st["start"].long(), st["before"].long()
    i = torch.arange(N, device=DEV)
    token = (start[:B, None] + i).clamp(max=T - 1)
    # the rows of the window of a request's first token and all later ones, then the first rows
    if window:
        low = (before + 1 - window).clamp(min=0)
        L = min(window - 1 + N, st["rows_max"])
        j = torch.cat([low[:, None] + torch.arange(L, device=DEV), torch.arange(first, device=DEV).expand(B, first)], 1)
        twice = torch.cat([torch.zeros(B, L, dtype=torch.bool, device=DEV), j[:, L:] >= low[:, None]], 1)
    else:
        j = torch.arange(st["rows_max"], device=DEV).expand(B, -1)
        twice = torch.zeros_like(j, dtype=torch.bool)
    ctx = st["ctx"].long()[token][..., None]
    rows = j[:, None, :]
    if st["mask"] is None:
        seen = rows < ctx
        end = ctx
    else:
        m = st["mask"][token]
        bit = (rows - ctx).clamp(0, 64 * m.shape[-1] - 1)
        draft = ((torch.gather(m, 2, bit // 64) >> (bit % 64)) & 1).bool() & (rows >= ctx) & (rows - ctx < 64 * m.shape[-1])
        count = ((m[..., None] >> torch.arange(64, device=DEV)) & 1).sum((-1, -2))
        seen = rows < ctx
        end = ctx + count[..., None]
    if window:
        seen = seen & ((rows >= end - window) | (rows < first))
    if st["mask"] is not None:
        seen = seen | draft
    seen = seen & ~twice[:, None, :]
    at = st["table"].long().gather(1, (j // page).clamp(max=st["table"].shape[1] - 1)).clamp(min=0)
    k = st["k"][at, j % page].float().permute(0, 2, 3, 1)  # [B, KH, D, L]
    v = st["v"][at, j % page].float().transpose(1, 2)      # [B, KH, L, D]
    q = st["q"].float()[token].view(B, N, KH, H // KH, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = (q @ k).view(B, KH, N, H // KH, -1) * st["scale"]
    s = torch.where(seen[:, None, :, None, :], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    sink = None if st["sink"] is None else st["sink"].view(KH, 1, H // KH, 1)
    if sink is not None:
        top = torch.maximum(top, sink)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(s - safe)
    total = e.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - safe)
    o = (e.flatten(2, 3) @ v).view(B, KH, N, H // KH, D)
    o = torch.where(total > 0, o / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(o))
    lse = (safe + torch.log(total)).squeeze(-1)
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, N, H, D), lse.transpose(1, 2).reshape(B, N, H)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:], t, right=True)
    return {"out": o[b, t - start[b]].to(torch.bfloat16), "lse": lse[b, t - start[b]]}


# ------------------------------------------------------------------ merge
def _prepare_merge(c, seed):
    g = _gen(seed)
    T, H, D, n = c["T"], c["H"], c["D"], c["parts"]
    outs, lses = [], []
    for _ in range(n):
        none = torch.rand(T, 1, generator=g, device=DEV) < c["empty"]  # tokens that saw nothing of this part
        o = torch.randn(T, H, D, generator=g, device=DEV)
        outs.append(torch.where(none[..., None], torch.zeros_like(o), o).to(torch.bfloat16))
        s = 2 * torch.randn(T, H, generator=g, device=DEV) + 3
        lses.append(torch.where(none, torch.full_like(s, -math.inf), s))
    return dict(c=c, outs=outs, lses=lses, out=torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV),
                lse=torch.empty(T, H, device=DEV))


def _run_merge(st):
    if own:
        import compressed_kv_attention_gated_gb300 as ck

        ck.ckv_merge_attention(st["outs"], st["lses"], out=st["out"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    s = torch.stack(st["lses"])
    top = s.amax(0)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(s - safe)
    total = w.sum(0)
    lse = safe + torch.log(total)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    o = sum(w[i][..., None] * st["outs"][i].float() for i in range(len(st["outs"])))
    return {"out": o.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------ the interface
_PREPARE = {"append": _prepare_append, "masks": _prepare_masks, "window": _prepare_attention, "tree": _prepare_attention,
            "merge": _prepare_merge}
_RUN = {"append": _run_append, "masks": _run_masks, "window": _run_attention, "tree": _run_attention, "merge": _run_merge}


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def run(state):
    return _RUN[state["c"]["op"]](state)


def _seen_rows(c):
    """Rows that a request's tokens see together, and that one of them sees, on average over the contexts."""
    n = (c["n_min"] + c["n_max"]) / 2
    lo, hi, window, first = c["ctx_min"], c["ctx_max"], c["window"], c["first"]
    xs = [lo + (hi - lo) * (i + 0.5) / 64 for i in range(64)]
    if c["op"] == "tree":
        one = [(min(x, window + min(first, max(0, x - window))) if window else x) + 8 for x in xs]  # drafts are some eight deep
        both = [a - 8 + n for a in one]
    else:
        ends = [x + n / 2 for x in xs]
        one = [min(e, window + min(first, max(0, e - window))) if window else e for e in ends]
        both = [min(x + n, window + n - 1 + min(first, max(0, x - window))) if window else x + n for x in xs]
    return n, sum(both) / 64, sum(one) / 64


def work(case):
    c = case
    if c["op"] == "append":
        es = 4 if c["dtype"] == "f32" else 2
        live = c["T"] * (1 - c["skip"])
        rows = live * (c["H"] + (1 if c["shared"] else 2) * c["KH"])
        return {"bytes": rows * c["D"] * (es + 2) + live * c["R"] * 4 + c["T"] * 12, "flops": live * (c["H"] + c["KH"]) * c["R"] * 3}
    if c["op"] == "masks":
        T = c["B"] * (c["n_min"] + c["n_max"]) / 2
        return {"bytes": T * (12 + 8 * _words(c)), "flops": T * 8}
    if c["op"] == "merge":
        rows = c["T"] * c["H"]
        return {"bytes": rows * (c["D"] * 2 + 4) * (c["parts"] + 1), "flops": rows * c["D"] * 2 * c["parts"]}
    n, both, one = _seen_rows(c)
    T = c["B"] * n
    kv = 1 if c["D"] == 512 else 2
    return {"bytes": c["B"] * both * c["KH"] * c["D"] * 2 * kv + T * c["H"] * (c["D"] * 4 + 4), "flops": 4 * T * c["H"] * c["D"] * one}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_append(st):
    c = st["c"]
    R, at = c["R"], c["at"]
    half = R // 2
    i = torch.arange(half, device=DEV)
    ia, ib = (at + 2 * i, at + 2 * i + 1) if c["pairs"] else (at + i, at + half + i)
    turn = torch.complex(*st["table"].double()[st["pos"].clamp(min=0).long()].split(half, -1))[:, None]

    def rows(x):
        z = x.double().clone()
        pair = torch.complex(z[..., ia], z[..., ib]) * turn
        z[..., ia], z[..., ib] = pair.real, pair.imag
        return z

    def stored(cache, x):
        y = torch.zeros(cache.shape, dtype=torch.float64, device=DEV)
        live = st["loc"] >= 0
        at = st["loc"][live]
        y[at // c["page"], at % c["page"]] = x[live]
        return y

    q = rows(st["q"])
    q[st["pos"] < 0] = 0
    return {"q": q, "k": stored(st["k_cache"], rows(st["k"])), "v": stored(st["v_cache"], st["v"].double()) if st["v"] is not None else 0}


def _exact_attention(st):
    c = st["c"]
    H, KH, D, T, page, window, first = c["H"], c["KH"], c["D"], st["T"], c["page"], c["window"], c["first"]
    G = H // KH
    start, table, before = st["start"].tolist(), st["table"].tolist(), st["before"].tolist()
    ctx = st["ctx"].tolist()
    masks = None if st["mask"] is None else st["mask"].cpu()
    out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    if st["sink"] is not None:
        lse[:] = st["sink"].double()
    for b in range(c["B"]):
        lo, hi = start[b], start[b + 1]
        n = hi - lo
        if n == 0:
            continue
        if masks is None:
            end = torch.tensor(ctx[lo:hi])
            tail = torch.zeros(n, 0, dtype=torch.bool)
            old = before[b] + n
        else:
            tail = (masks[lo:hi].unsqueeze(-1) >> torch.arange(64)).bitwise_and(1).bool().flatten(1)[:, :n]
            end = before[b] + tail.sum(1)
            old = before[b]
        rows = torch.arange(old)
        see = rows[None] < torch.tensor(ctx[lo:hi])[:, None]
        if window:
            see &= (rows[None] >= end[:, None] - window) | (rows[None] < first)
        see = torch.cat([see, tail], 1)
        used = see.any(0).nonzero().flatten()
        if used.numel() == 0:
            continue
        see = see[:, used].to(DEV)
        pages = torch.tensor([table[b][r // page] for r in used.tolist()], device=DEV)
        slot = (used % page).to(DEV)
        k, v = st["k"][pages, slot].double(), st["v"][pages, slot].double()
        z = torch.einsum("tkgd,jkd->tkgj", st["q"][lo:hi].double().view(n, KH, G, D), k) * st["scale"]
        z.masked_fill_(~see[:, None, None, :], -math.inf)
        if st["sink"] is not None:
            z = torch.cat([z, st["sink"].double().view(1, KH, G, 1).expand(n, KH, G, 1)], -1)
        total = torch.logsumexp(z, -1)
        w = torch.exp(z - total[..., None].clamp(min=-1e300))[..., :used.numel()]
        out[lo:hi] = torch.einsum("tkgj,jkd->tkgd", w, v).reshape(n, H, D)
        lse[lo:hi] = total.reshape(n, H)
    return {"out": out, "lse": lse}


def _exact_merge(st):
    s = torch.stack([x.double() for x in st["lses"]])
    lse = torch.logsumexp(s, 0)
    w = torch.exp(s - lse.clamp(min=-1e300))
    return {"out": torch.einsum("nth,nthd->thd", w, torch.stack([o.double() for o in st["outs"]])), "lse": lse}


def exact(case, seed):
    if case["op"] == "masks" or (case["op"] in ("window", "tree") and work(case)["flops"] > 4e12):
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "merge":
        return _exact_merge(st)
    return _exact_attention(st)
