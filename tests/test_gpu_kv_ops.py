"""The operators around the uncompressed cache on the GPU against 64-bit references:
appending with rotation, tree masks, attention (window, first rows, drafts), merging,
and a step that runs them together with the compressed rows.

Tolerances, from the operators' arithmetic:
  * masks, positions, values stored as they are: exact
  * rotation: two fp32 products and a sum (2^-22 of |a| + |b|), then one rounding to
    bf16, 2^-8 of the value
  * attention: scores are fp32 sums of D products: e = D 2^-24 sum |q k| scale, which moves
    a weight by e of its value; exp2 and the sums another 2^-18; weights are rounded to bf16,
    2^-8 of each: (2 e + 2^-17 + 2^-8) sum w |v|, then one rounding, 2^-8 of the value;
    lse: e + 2^-18 + 2^-22 of its value
  * merging: fp32 weights (2^-18 of each), then one rounding (bf16 2^-8, fp32 2^-24)
"""
import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck():
    import compressed_kv_attention_gated_gb300 as ck

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.load()
    return ck


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _angles(n, R):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _cache(pages, ps, KH, D, layout, fill=0.0):
    """A cache [pages, ps, KH, D]: rows outermost, heads outermost, keys and values interleaved in one tensor, or rows
    that begin at odd places of 16 bytes."""
    if layout == "padded":
        return torch.full((pages, ps, KH, D + 8), fill, dtype=torch.bfloat16, device="cuda")[..., 8:]
    if layout == "heads":
        return torch.full((pages, KH, ps, D), fill, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    if layout == "halves":
        return torch.full((pages, 2, ps, KH, D), fill, dtype=torch.bfloat16, device="cuda")[:, 1]
    return torch.full((pages, ps, KH, D), fill, dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("D,H,KH,T,R,at,pairs", [
    (128, 16, 2, 4, 128, 0, False), (128, 5, 1, 37, 64, 64, False), (256, 8, 8, 3, 64, 192, True), (512, 64, 1, 9, 64, 448, True),
    (128, 4, 2, 11, 44, 24, False), (256, 3, 3, 5, 30, 98, False), (512, 7, 7, 6, 512, 0, False), (512, 2, 1, 5, 6, 2, True),
    (128, 24, 8, 700, 128, 0, False), (256, 1, 1, 1, 0, 0, False), (512, 130, 2, 3, 10, 500, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["rows", "heads", "halves", "padded"])
def test_append(ck, D, H, KH, T, R, at, pairs, dtype, layout):
    g = torch.Generator(device="cuda").manual_seed(D + T + R)
    ps, pages = (7, -(-T // 7) + 2)
    both = torch.randn(T, H + 2 * KH, D, generator=g, device="cuda").to(dtype)
    q, k, v = both[:, :H], both[:, H:H + KH], both[:, H + KH:]
    loc = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
    if T > 2:
        loc[1], pos[2] = -1, -1  # not stored; skipped
    kc, vc = _cache(pages, ps, KH, D, layout, 7.0), _cache(pages, ps, KH, D, layout, 7.0)
    table = _angles(50, R) if R else None
    err = _err()
    q_out = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    got = ck.ckv_kv_append(k, v, kc, vc, loc, positions=pos, cos_sin=table, rope_offset=at, interleaved=pairs, q=q, q_out=q_out, err_word=err)
    assert got is q_out and int(err) == 0
    tab = table if R else torch.zeros(50, 0, device="cuda")
    turned = torch.zeros(D, dtype=torch.bool, device="cuda")
    turned[at:at + R] = True

    def check(a, x):
        want = ref.rotate(x, pos, tab, at, pairs)
        size = x.double().abs()
        big = torch.where(turned, size[..., at:at + R].amax(-1, keepdim=True) * 2 if R else size, size)
        assert torch.all((a.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * big * turned)

    live = pos >= 0
    check(torch.where(live[:, None, None], q_out, q.bfloat16()), q)
    if T > 2:
        assert torch.all(q_out[2] == 3.0)
    kw, vw = torch.full((pages, ps, KH, D), 7.0, device="cuda").bfloat16(), torch.full((pages, ps, KH, D), 7.0, device="cuda").bfloat16()
    on = live & (loc >= 0)
    check(torch.where(on[:, None, None], kc[loc.clamp(min=0) // ps, loc.clamp(min=0) % ps], ref.rotate(k, pos, tab, at, pairs).bfloat16()), k)
    kw[loc[on] // ps, loc[on] % ps] = kc[loc[on] // ps, loc[on] % ps]
    vw[loc[on] // ps, loc[on] % ps] = v[on].bfloat16()
    assert torch.equal(kc, kw) and torch.equal(vc, vw)


def test_append_keys_alone_and_queries_in_place(ck):
    g = torch.Generator(device="cuda").manual_seed(1)
    for R, at, pairs in ((64, 64, False), (44, 24, False), (20, 6, True)):
        T, H, KH, D, ps = 33, 6, 2, 128, 16
        q = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
        k = torch.randn(T, KH, D, generator=g, device="cuda").bfloat16()
        pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
        loc = torch.randperm(5 * ps, generator=g, device="cuda")[:T]
        a, b = _cache(5, ps, KH, D, "rows"), _cache(5, ps, KH, D, "rows")
        table = _angles(50, R)
        apart = ck.ckv_kv_append(k, None, a, None, loc, positions=pos, cos_sin=table, rope_offset=at, interleaved=pairs, q=q)
        same = ck.ckv_kv_append(k, None, b, None, loc, positions=pos, cos_sin=table, rope_offset=at, interleaved=pairs, q=q, q_out=q)
        assert same is q and torch.equal(apart, q) and torch.equal(a, b)
    # no rotation, no positions: the rows as they are
    assert ck.ckv_kv_append(k, None, a, None, loc) is None
    assert torch.equal(a[loc // ps, loc % ps], k)


def test_append_flags_locations_and_positions(ck):
    k = torch.ones(3, 1, 128, device="cuda").bfloat16()
    c, err = _cache(2, 4, 1, 128, "rows"), _err()
    ck.ckv_kv_append(k, None, c, None, torch.tensor([8, 3, 1 << 40], device="cuda"), err_word=err)
    assert int(err) == 4 and int((c != 0).any(-1).sum()) == 1 and torch.all(c[0, 3] == 1)
    err.zero_()
    ck.ckv_kv_append(k, None, c, None, torch.tensor([0, 1, 2], device="cuda"), positions=_i32([9, 10, 11]), cos_sin=_angles(10, 64), err_word=err)
    assert int(err) == 16 and torch.all(c[0, 1] == 0) and torch.all(c[0, 2] == 0) and torch.any(c[0, 0] != 0)


# ------------------------------------------------------------------ tree masks
@pytest.mark.parametrize("B,n_lo,n_hi,words", [(1, 1, 1, 1), (8, 16, 16, 1), (5, 0, 64, 1), (3, 60, 130, 3), (2, 1000, 1024, 16), (300, 0, 9, 2),
                                               (1, 64, 64, 1), (1, 65, 65, 2)])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_tree_masks(ck, B, n_lo, n_hi, words, kind):
    rng = np.random.default_rng(B + n_hi)
    n = rng.integers(n_lo, n_hi + 1, B)
    start = np.concatenate([[0], np.cumsum(n)])
    T = int(start[-1]) + 5
    parents = np.full(T, 77)
    for b in range(B):
        i = np.arange(n[b])
        parents[start[b]:start[b + 1]] = i - 1 if kind == "chain" else -1 if kind == "star" else [rng.integers(-1, x) if x else -1 for x in i]
    ctx = rng.integers(0, 1000, T)
    ctx[start[-1] // 2] = -1
    masks, pos = ref.tree(parents.tolist(), start.tolist(), ctx.tolist(), words)
    err = _err()
    m, p = ck.ckv_build_tree_masks(_i32(parents), _i32(start), _i32(ctx), words, err_word=err)
    assert int(err) == 0
    assert torch.equal(m.cpu(), ref.pack(masks, words)) and p.tolist() == pos


def test_tree_masks_bad_parents_and_too_many_drafts(ck):
    parents, start = [0, 0, 5, -2, 2, -1], [0, 6]
    err = _err()
    m, p = ck.ckv_build_tree_masks(_i32(parents), _i32(start), None, 1, err_word=err)
    masks, pos = ref.tree(parents, start, None, 1)
    assert int(err) == 8 and torch.equal(m.cpu(), ref.pack(masks, 1)) and p.tolist() == pos
    err.zero_()
    parents = list(range(-1, 69))
    m, p = ck.ckv_build_tree_masks(_i32(parents), _i32([0, 70]), None, 1, err_word=err)
    masks, pos = ref.tree(parents, [0, 70], None, 1)
    assert int(err) == 8 and torch.equal(m.cpu(), ref.pack(masks, 1)) and p.tolist() == pos and pos[64:] == [-1] * 6


# ------------------------------------------------------------------ attention
class Step:
    """Requests with contexts in a paged cache, and tokens of a step.  Rows that no token sees are NaN,
    pages that none sees are not there."""

    def __init__(self, D, H, KH, n, before, ps=16, window=0, first=0, tree=False, layout="rows", shared=False, sink=False, words=0, seed=0,
                 spread=1.5, width_more=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(n)
        self.start = np.concatenate([[0], np.cumsum(n)]).astype(int)
        T = int(self.start[-1])
        b = np.repeat(np.arange(B), n)
        i = np.arange(T) - self.start[b]
        before = np.asarray(before)
        self.mask = None
        if tree:
            parents = np.array([rng.integers(-1, x) if x else -1 for x in i], dtype=int)
            words = words or max(1, -(-max(n) // 64))
            masks, _ = ref.tree(parents.tolist(), self.start.tolist(), None, words)
            self.mask = ref.pack(masks, words).cuda()
            self.ctx = before[b]
        else:
            self.ctx = before[b] + i + 1
        total = before + np.asarray(n)
        self.max_rows = max(1, int(total.max()))
        width = -(-self.max_rows // ps) + width_more
        seen = [set() for _ in range(B)]
        for t in range(T):
            seen[b[t]] |= set(ref.seen_rows(int(self.ctx[t]), window, first, None if self.mask is None else sorted(masks[t])))
        held = np.array([[any(r // ps == x for r in seen[y]) for x in range(width)] for y in range(B)]).reshape(B, width)
        pages = int(held.sum()) + 3
        order = iter(rng.permutation(pages).tolist())
        self.table = torch.tensor([[next(order) if held[y, x] else -1 for x in range(width)] for y in range(B)], dtype=torch.int32,
                                  device="cuda").view(B, width)
        self.k = _cache(pages, ps, KH, D, layout, float("nan"))
        self.v = self.k if shared else _cache(pages, ps, KH, D, layout, float("nan"))
        for y in range(B):
            rows = torch.tensor(sorted(seen[y]), dtype=torch.int64, device="cuda")
            if rows.numel():
                pg = self.table[y].long()[rows // ps]
                for c in ((self.k,) if shared else (self.k, self.v)):
                    c[pg, rows % ps] = torch.randn(rows.numel(), KH, D, generator=g, device="cuda").bfloat16()
        self.q = (torch.randn(T, H, D, generator=g, device="cuda") * spread).bfloat16()
        self.sink = torch.randn(H, generator=g, device="cuda") if sink else None
        self.window, self.first, self.scale = window, first, D ** -0.5

    def run(self, ck, max_rows=None, **more):
        err = _err()
        out, lse = ck.ckv_kv_attention(self.q, self.k, self.v, self.table, _i32(self.start), _i32(self.ctx), max_rows or self.max_rows,
                                       self.scale, window=self.window, first_rows=self.first, tree_mask=self.mask, sink=self.sink,
                                       err_word=err, **more)
        return out, lse, err

    def check(self, out, lse):
        want, wl, seen, spread, slack = ref.attention(self.q, self.k, self.v, self.table, self.start, self.ctx, self.scale, self.window,
                                                      self.first, self.mask, self.sink)
        close(out[seen], lse[seen], want[seen], wl[seen], spread[seen], slack[seen], self.q.shape[2])


def close(out, lse, want, wl, spread, slack, D):
    e = slack * D * 2.0 ** -24
    tol = 2.0 ** -8 * want.abs() + (2 * e[..., None] + 2.0 ** -17 + 2.0 ** -8) * spread
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(out[bad][0]), float(want[bad][0]))
    none = torch.isneginf(wl)
    assert torch.equal(torch.isneginf(lse), none)
    d = (lse.double() - wl).abs()[~none]
    assert torch.all(d <= (e + 2.0 ** -18 + 2.0 ** -22 * wl.abs())[~none]), float(d.max())


SIZES = [
    # D, H, KH, tokens of the requests, rows before them, page size
    (128, 16, 2, [1, 1, 1, 1], [0, 7, 130, 299], 16),
    (128, 5, 1, [3, 0, 1, 40], [0, 5, 127, 90], 7),
    (128, 32, 8, [200, 1, 77], [50, 600, 0], 64),
    (128, 64, 1, [1, 2], [511, 128], 48),
    (256, 8, 8, [4, 1, 150], [300, 0, 33], 16),
    (256, 24, 3, [1, 9], [255, 256], 100),
    (512, 64, 1, [1, 1, 3], [700, 0, 129], 64),
    (512, 7, 7, [2, 30], [140, 1], 5),
    (512, 130, 1, [5], [260], 32)]


@pytest.mark.parametrize("D,H,KH,n,before,ps", SIZES)
@pytest.mark.parametrize("window,first", [(0, 0), (1, 0), (100, 0), (128, 4), (37, 150), (5000, 3)])
def test_window(ck, D, H, KH, n, before, ps, window, first):
    s = Step(D, H, KH, n, before, ps, window, first, layout=("rows", "heads", "halves", "padded")[(window + n[0]) % 4], shared=D == 512 and window != 1,
             sink=first > 0, seed=D + window)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n,before,ps", SIZES)
@pytest.mark.parametrize("window,first", [(0, 0), (64, 3), (300, 0)])
def test_tree(ck, D, H, KH, n, before, ps, window, first):
    s = Step(D, H, KH, n, before, ps, window, first, tree=True, layout=("rows", "padded")[before[0] % 2], sink=window == 64, seed=D + window,
             words=5 if D == 256 else 0)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,before,window", [(128, 8, 1, 9000, 0), (512, 16, 1, 5000, 0), (256, 4, 2, 20000, 7000), (128, 128, 1, 3000, 0)])
def test_long_rows_of_few_tokens(ck, D, H, KH, before, window):
    s = Step(D, H, KH, [1, 2], [before, before // 3], 64, window, 20, sink=True, seed=before)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,tokens,before,window", [
    (128, 64, 8, 9, 40, 16), (128, 64, 8, 9, 300, 130), (128, 8, 1, 16, 20, 0), (128, 64, 8, 1, 60, 20), (256, 32, 2, 9, 100, 60),
    (512, 130, 2, 1, 90, 40), (128, 40, 8, 60, 150, 100), (512, 64, 1, 1, 150, 0), (256, 64, 8, 1, 400, 0), (128, 64, 4, 2, 200, 129)])
def test_many_short_jobs(ck, D, H, KH, tokens, before, window):
    """Hundreds of tiles of rows with one tile of keys, two or three, one after the other on an SM."""
    B = max(4, 500 // KH)
    s = Step(D, H, KH, [tokens + (i % 3 == 0) for i in range(B)], [max(0, before - i % 50) for i in range(B)], 16, window, 2 if window else 0, seed=D + before)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n,before,window", [
    (128, 64, 8, 1, 1100, 1024), (128, 64, 8, 1, 140, 100), (128, 32, 2, 2, 300, 0), (256, 32, 2, 1, 300, 200), (512, 64, 1, 1, 200, 128),
    (512, 48, 2, 2, 150, 0), (128, 64, 8, 16, 500, 400), (128, 32, 8, 40, 300, 0), (256, 32, 2, 40, 300, 0)])
def test_the_same_call_gives_the_same_bits(ck, D, H, KH, n, before, window):
    """Sums have a fixed order, and what the warps of a CTA leave one another in shared memory is not yet written over."""
    g = torch.Generator(device="cuda").manual_seed(D + before)
    B, ps = 200, 16
    width = -(-(before + n) // ps)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    k, v = (torch.randn(B * width, ps, KH, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B * n, H, D, generator=g, device="cuda").bfloat16()
    ctx = _i32([before - b % 90 + i + 1 for b in range(B) for i in range(n)])
    start = _i32(range(0, B * n + 1, n))

    def call():
        return ck.ckv_kv_attention(q, k, v, table, start, ctx, before + n, D ** -0.5, window=window)

    out, lse = call()
    for _ in range(30):
        again = call()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D,H,KH,n,B", [(128, 16, 8, 1, 100), (512, 16, 1, 1, 250), (256, 32, 4, 2, 110), (128, 32, 8, 12, 130),
                                         (128, 32, 8, 300, 9), (256, 16, 8, 70, 40)])
def test_requests_in_the_order_of_their_lengths(ck, D, H, KH, n, B):
    """Long contexts and few jobs to an SM; requests without tokens, without context and left alone among them."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 300, B)
    lens[[0, B // 2]] = 2600 - n, 1500
    tokens = [n] * B
    tokens[1], tokens[B // 3] = 0, 2 * n
    s = Step(D, H, KH, tokens, lens, 64, seed=B)
    s.ctx = np.array(s.ctx)
    s.ctx[s.start[5]:s.start[6]] = -1
    s.ctx[s.start[7]] = 0
    assert ck.ckv_kv_attention_workspace(B * n, B, H, KH, D, s.max_rows) == 4 * (2 * B + 1)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)
    s.window = s.max_rows  # which hides nothing: the same tiles as they come
    assert ck.ckv_kv_attention_workspace(B * n, B, H, KH, D, s.max_rows, s.window) == 0
    as_they_come = s.run(ck)
    on = torch.as_tensor(s.ctx >= 0).cuda()
    assert torch.equal(as_they_come[0][on], out[on]) and torch.equal(as_they_come[1][on], lse[on])


def test_rows_left_alone(ck):
    s = Step(128, 8, 2, [3, 2, 2], [20, 140, 3], seed=3)
    T = s.q.shape[0]
    s.ctx[[1, 4]] = -1
    s.start = s.start.copy()
    s.start[-1] = T - 1  # the last token belongs to nobody
    out, lse = torch.full((T, 8, 128), 5.0, device="cuda").bfloat16(), torch.full((T, 8), 5.0, device="cuda")
    got, gl, err = s.run(ck, out=out, lse=lse)
    assert got is out and gl is lse and int(err) == 0
    s.check(out, lse)
    for t in (1, 4, T - 1):
        assert torch.all(out[t] == 5) and torch.all(lse[t] == 5)


def test_tokens_that_see_nothing(ck):
    for sink in (False, True):
        s = Step(128, 8, 2, [3, 2], [20, 140], seed=4, sink=sink)
        s.ctx[0] = 0
        s.ctx[3:] = 0
        out, lse, err = s.run(ck)
        s.check(out, lse)
        assert int(err) == 0 and torch.all(out[0] == 0) and torch.all(out[3:] == 0)
        assert torch.equal(lse[0], s.sink) if sink else torch.all(torch.isneginf(lse[3:]))


def test_missing_pages_and_long_contexts_are_flagged(ck):
    for bad in (-1, 10 ** 6):
        s = Step(128, 8, 2, [3, 2], [90, 140], seed=5)
        s.table[0, 2] = bad
        out, lse, err = s.run(ck)
        assert int(err) == 4
        s.check(out, lse)
    s = Step(128, 8, 2, [3], [90], seed=6, width_more=2)
    s.ctx[1] = 10 ** 9
    s.k[torch.isnan(s.k)] = 0
    s.v[torch.isnan(s.v)] = 0
    out, lse, err = s.run(ck)
    assert int(err) == 16
    s.ctx[1] = s.max_rows
    s.check(out, lse)


def test_drafts_behind_max_rows_are_flagged(ck):
    s = Step(128, 4, 4, [10], [50], tree=True, seed=7)
    out, lse, err = s.run(ck, max_rows=55)
    assert int(err) == 16
    want = ref.attention(s.q, s.k, s.v, s.table, s.start, s.ctx, s.scale, mask=s.mask, max_rows=55)
    close(out, lse, want[0], want[1], want[3], want[4], 128)


def test_large_scores_and_constant_values(ck):
    """Rows whose weights are far apart, ascending and descending, and values that are all the same: the
    output is that value to its rounding."""
    for order in (1, -1):
        s = Step(128, 16, 2, [1, 30], [500, 400], seed=8, spread=30.0)
        out, lse, err = s.run(ck)
        s.check(out, lse)
        ramp = torch.arange(s.max_rows, device="cuda") * order + (s.max_rows if order < 0 else 0)
        for b in range(2):
            rows = torch.arange(min(int(s.start[b + 1] - s.start[b]) + (500, 400)[b], s.max_rows), device="cuda")
            pg = s.table[b].long()[rows // 16]
            s.k[pg, rows % 16] = (ramp[rows].float() / 8).bfloat16()[:, None, None]
            s.v[pg, rows % 16] = 1.75
        s.q = torch.ones_like(s.q)
        out, lse, err = s.run(ck)
        s.check(out, lse)
        assert torch.all((out.double() - 1.75).abs() <= 1.75 * (2.0 ** -8 + 2.0 ** -8))


def test_one_table_row_for_all_and_permuted_queries(ck):
    s = Step(128, 8, 2, [1, 1, 1], [80, 80, 80], seed=9)
    s.table = s.table[:1].expand(3, -1)
    s.q = s.q.transpose(0, 1).contiguous().transpose(0, 1)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n,before", [(128, 24, 3, 1, 60), (128, 40, 5, 1, 90), (128, 112, 7, 1, 30), (256, 24, 3, 2, 80), (512, 48, 3, 1, 70),
                                             (128, 200, 5, 9, 60), (256, 240, 5, 4, 90)])
def test_several_key_heads_are_looked_up_together(ck, D, H, KH, n, before):
    """Short jobs and more than 152 x 6 CTAs of them; key heads that are no power of two."""
    B = 1000 // KH
    s = Step(D, H, KH, [n] * B, [before - i % 20 for i in range(B)], 16, 32, 2, seed=KH)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n,shared", [(256, 16, 2, [1, 3], True), (256, 32, 2, [30, 1], True), (512, 64, 2, [5, 70], False), (512, 16, 1, [1, 1], False),
                                             (512, 24, 1, [1, 2], False), (128, 16, 1, [1, 5], True), (128, 32, 1, [30, 9], True)])
def test_rows_that_are_key_and_value_or_not(ck, D, H, KH, n, shared):
    s = Step(D, H, KH, n, [400, 130], 32, 300, 5, shared=shared, seed=D + H)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n", [(128, 8, 1, [1, 2]), (128, 32, 1, [20, 3]), (256, 32, 2, [20, 3]), (512, 64, 1, [2, 1])])
@pytest.mark.parametrize("tree", [False, True])
def test_a_bound_far_above_the_contexts(ck, D, H, KH, n, tree):
    """Most ranges of keys are empty, and those of one request where the other's are not."""
    s = Step(D, H, KH, n, [300, 9], 16, tree=tree, sink=True, seed=D, width_more=1000)
    assert ck.ckv_kv_attention_workspace(sum(n), 2, H, KH, D, 16000, mask_words=1 if tree else 0) > 0
    out, lse, err = s.run(ck, max_rows=16000)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n", [(128, 8, 2, [1, 2]), (128, 32, 2, [20, 3]), (256, 32, 2, [20, 3]), (512, 64, 1, [2, 1])])
def test_negative_and_zero_scale(ck, D, H, KH, n):
    for scale in (-0.07, 0.0):
        s = Step(D, H, KH, n, [200, 50], seed=11)
        s.scale = scale
        out, lse, err = s.run(ck)
        assert int(err) == 0
        s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n,before,window", [(128, 16, 2, [1, 3], [300, 20], 100), (128, 32, 2, [40, 3], [300, 20], 0), (256, 32, 2, [40, 3], [300, 20], 0),
                                                    (512, 64, 1, [2, 1], [700, 90], 0), (128, 8, 1, [1, 1], [9000, 10], 0)])
def test_nothing_is_written_beside_the_outputs(ck, D, H, KH, n, before, window):
    """Outputs and workspace lie between guards; the outputs begin on 16 bytes, not on 32."""
    s = Step(D, H, KH, n, before, 16, window, seed=D)
    T, pad = s.q.shape[0], 1024
    need = ck.ckv_kv_attention_workspace(T, len(n), H, KH, D, s.max_rows, window)
    o = torch.full((pad + 8 + T * H * D + pad,), 3.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((pad + T * H + pad,), 3.0, device="cuda")
    w = torch.full((pad + need + pad,), 77, dtype=torch.uint8, device="cuda")
    out, lse, err = s.run(ck, out=o[pad + 8:pad + 8 + T * H * D].view(T, H, D), lse=z[pad:pad + T * H].view(T, H), workspace=w[pad:pad + need])
    assert int(err) == 0
    s.check(out, lse)
    assert torch.all(o[:pad + 8] == 3) and torch.all(o[-pad:] == 3) and torch.all(z[:pad] == 3) and torch.all(z[-pad:] == 3)
    assert torch.all(w[:pad] == 77) and torch.all(w[-pad:] == 77)
    if need:
        with pytest.raises(Exception):
            s.run(ck, workspace=w[:need - 1])


@pytest.mark.parametrize("D,H,KH,n", [(128, 1024, 1, [2, 1]), (128, 1024, 1024, [1, 3]), (512, 1024, 2, [1, 1]), (256, 1000, 8, [3, 2])])
def test_a_thousand_heads(ck, D, H, KH, n):
    s = Step(D, H, KH, n, [60, 9], 16, 40, 3, sink=True, seed=H)
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("window", [0, 20])
def test_65536_requests(ck, window):
    """Requests that repeat: the first ones against the reference, the others against those."""
    B, kinds, D, H, ps = 65536, 64, 128, 4, 16
    s = Step(D, H, 2, [1] * kinds, [i for i in range(kinds)], ps, window, seed=14)
    want = s.run(ck)
    s.check(*want[:2])
    of = torch.arange(B, device="cuda") % kinds
    got = ck.ckv_kv_attention(s.q[of], s.k, s.v, s.table[of], _i32(range(B + 1)), _i32(s.ctx)[of], s.max_rows, s.scale, window=window)
    assert torch.equal(got[0], want[0][of]) and torch.equal(got[1], want[1][of])
    # most of them without tokens
    start = _i32(np.minimum(np.arange(B + 1), kinds))
    got = ck.ckv_kv_attention(s.q, s.k, s.v, s.table[of], start, _i32(s.ctx), s.max_rows, s.scale, window=window)
    s.check(*got)
    with pytest.raises(Exception):
        ck.ckv_kv_attention(s.q, s.k, s.v, s.table[of[:1]].expand(B + 1, -1), torch.zeros(B + 2, dtype=torch.int32, device="cuda"), _i32(s.ctx), s.max_rows, s.scale)


def test_no_tokens_and_no_requests(ck):
    s = Step(128, 8, 2, [1], [20], seed=15)
    out, lse = ck.ckv_kv_attention(s.q[:0], s.k, s.v, s.table, _i32([0, 0]), _i32([]), s.max_rows, s.scale)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    kept = torch.full_like(s.q, 2.0)
    ck.ckv_kv_attention(s.q, s.k, s.v, s.table[:0], _i32([0]), _i32(s.ctx), s.max_rows, s.scale, out=kept)
    assert torch.all(kept == 2)
    m, p = ck.ckv_build_tree_masks(_i32([]), _i32([0]), None, 1)
    assert m.shape == (0, 1) and p.shape == (0,)
    assert ck.ckv_kv_append(s.k[:0, 0], s.v[:0, 0], s.k, s.v, torch.zeros(0, dtype=torch.int64, device="cuda"), q=s.q[:0]).shape == (0, 8, 128)
    assert ck.ckv_merge_attention([out], [lse])[0].shape == (0, 8, 128)


@pytest.mark.parametrize("D,H,KH,n", [(128, 8, 1, [1]), (128, 32, 1, [9]), (256, 32, 1, [9]), (512, 64, 1, [1])])
def test_constant_values_over_a_long_context(ck, D, H, KH, n):
    """150,000 rows whose scores are all the same: the tensor cores cut a range's sum off towards 0 by less than 2^-23 of it
    per 16 keys, 2^17 / 16 times at most, which is 2^-10 of it; then the rounding."""
    L, ps = 150_000, 1000
    k, v = torch.zeros(L // ps, ps, KH, D, device="cuda").bfloat16(), torch.full((L // ps, ps, KH, D), 1.75, device="cuda").bfloat16()
    q = torch.ones(n[0], H, D, device="cuda").bfloat16()
    table = torch.arange(L // ps, dtype=torch.int32, device="cuda")[None]
    out, lse = ck.ckv_kv_attention(q, k, v, table, _i32([0, n[0]]), _i32([L - n[0] + i + 1 for i in range(n[0])]), L, 1.0)
    assert torch.all((out.double() - 1.75).abs() <= 1.75 * (2.0 ** -8 + 2.0 ** -10))
    want = torch.tensor([float(np.log(L - n[0] + i + 1)) for i in range(n[0])], device="cuda").double()
    assert torch.all((lse.double() - want[:, None]).abs() <= 2.0 ** -16)


def test_calls_of_two_streams_at_once(ck):
    """Each with its own tensors and workspace; results are those of calls one after the other."""
    steps = [Step(128, 8, 1, [1, 2], [9000, 3000], 64, seed=1), Step(128, 32, 8, [300, 5], [700, 100], 64, 256, 4, seed=2),
             Step(512, 64, 1, [40, 30], [500, 300], 64, seed=3)]
    alone = [s.run(ck)[:2] for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                got.append(s.run(ck)[:2])
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # named by the argument instead
    got = [s.run(ck, stream=stream)[:2] for s, stream in zip(steps, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("use_pdl", [True, False])
def test_a_captured_step_follows_its_inputs(ck, use_pdl):
    """Masks, append, attention over drafts and a merge in one graph; replayed with other lengths, parents and rows."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, n, H, KH, D, ps, pages = 5, 7, 16, 2, 128, 16, 80
    T, rows = B * n, 200
    start = _i32(range(0, T + 1, n))
    table = torch.randperm(pages, generator=g, device="cuda")[:B * 13].int().view(B, 13)
    k0, v0 = (torch.randn(pages, ps, KH, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    kc, vc = k0.clone(), v0.clone()
    cs = _angles(300, 128)
    parents, ctx = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    loc = torch.zeros(T, dtype=torch.int64, device="cuda")
    x = torch.zeros(T, H + 2 * KH, D, device="cuda")
    far = torch.randn(T, H, D, generator=g, device="cuda").bfloat16(), torch.randn(T, H, generator=g, device="cuda")
    err = _err()

    def step():
        more = dict(use_pdl=use_pdl, err_word=err)
        mask, pos = ck.ckv_build_tree_masks(parents, start, ctx, **more)
        q = ck.ckv_kv_append(x[:, H:H + KH], x[:, H + KH:], kc, vc, loc, positions=pos, cos_sin=cs, q=x[:, :H], **more)
        near = ck.ckv_kv_attention(q, kc, vc, table, start, ctx, rows, D ** -0.5, window=60, first_rows=2, tree_mask=mask, **more)
        out, lse = ck.ckv_merge_attention([near[0], far[0]], [near[1], far[1]], positions=pos, use_pdl=use_pdl)
        return mask, pos, q, *near, out, lse

    def inputs(seed):
        rng = np.random.default_rng(seed)
        parents.copy_(_i32([rng.integers(-1, i) if i else -1 for _ in range(B) for i in range(n)]))
        c = np.repeat(rng.integers(0, rows - n, B), n)
        ctx.copy_(_i32(c))
        r = torch.as_tensor(c + np.tile(np.arange(n), B)).cuda()
        loc.copy_(table.long()[torch.arange(B, device="cuda").repeat_interleave(n), r // ps] * ps + r % ps)
        x.normal_(generator=g)
        kc.copy_(k0)
        vc.copy_(v0)

    inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2, 3):
        inputs(seed)
        graph.replay()
        got = [t.clone() for t in held] + [kc.clone(), vc.clone()]
        kc.copy_(k0)
        vc.copy_(v0)
        want = list(step()) + [kc, vc]
        assert int(err) == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_caches_and_queries_beyond_32_bits(ck):
    """Pages whose first rows lie more than 2^31 elements apart, and tokens whose rows do."""
    D, KH, ps = 128, 2, 16
    stride = 150_000_000 // (ps * KH * D) * (ps * KH * D)
    pages = 20  # 3 * 10^9 elements
    flat = [torch.empty(stride * (pages - 1) + ps * KH * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (f.as_strided((pages, ps, KH, D), (stride, KH * D, D, 1)) for f in flat)
    s = Step(D, 16, KH, [3, 40], [200, 30], ps, seed=12)
    held = sorted(set(s.table.flatten().tolist()) - {-1})
    to = torch.randperm(pages, device="cuda")[:len(held)]
    assert int(to.max()) * stride > 2 ** 31
    new = {p: int(t) for p, t in zip(held, to)}
    for p, t in new.items():
        k[t], v[t] = s.k[p], s.v[p]
    table = torch.tensor([[new.get(p, -1) for p in r] for r in s.table.tolist()], dtype=torch.int32, device="cuda")
    want = s.run(ck)
    near = s.k, s.v, s.table
    s.k, s.v, s.table = k, v, table
    got = s.run(ck)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # append: rows of the highest page
    row = torch.randn(2, KH, D, device="cuda").bfloat16()
    ck.ckv_kv_append(row, row * 2, k, v, torch.tensor([(pages - 1) * ps + 3, 5], device="cuda"))
    assert torch.equal(k[pages - 1, 3], row[0]) and torch.equal(v[pages - 1, 3], row[0] * 2) and torch.equal(k[0, 5], row[1])
    del k, v, flat, got
    s.k, s.v, s.table = near
    # more than 2^31 elements of queries and outputs: a request in front without tokens of its own
    T, H, D = 33000, 130, 512
    s = Step(D, H, 1, [2], [70], ps, seed=13)
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-2:] = s.q
    ctx = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ctx[-2:] = _i32(s.ctx)
    out, lse = torch.zeros_like(q), torch.zeros(T, H, device="cuda")
    want = s.run(ck)
    ck.ckv_kv_attention(q, s.k, s.v, s.table.expand(2, -1), _i32([0, T - 2, T]), ctx, s.max_rows, s.scale, out=out, lse=lse)
    s.check(out[-2:], lse[-2:])
    assert int((out[:-2] != 0).any()) == 0 and int((lse[:-2] != 0).any()) == 0
    merged, _ = ck.ckv_merge_attention([out, out], [lse, lse], out=out, lse=lse, positions=ctx)
    s.check(out[-2:], lse[-2:] - float(np.log(2.0)))


# ------------------------------------------------------------------ merge
@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("parts", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                             (torch.bfloat16, torch.float32)])
def test_merge(ck, D, parts, dtype, out_dtype):
    g = torch.Generator(device="cuda").manual_seed(D + parts)
    T, H = 13, 5
    outs = [torch.randn(T, H, D, generator=g, device="cuda").to(dtype) for _ in range(parts)]
    lses = [4 * torch.randn(T, H, generator=g, device="cuda") for _ in range(parts)]
    for i in range(parts):  # what a part without rows holds does not count
        lses[i][i % T] = -torch.inf
        outs[i][i % T] = float("nan")
        lses[i][T - 1] = -torch.inf
    lses[0][5] = 100.0
    lses[parts - 1][6] = -300.0
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[4] = -1
    out, lse = torch.full((T, H, D), 9.0, device="cuda").to(out_dtype), torch.full((T, H), 9.0, device="cuda")
    got, gl = ck.ckv_merge_attention(outs, lses, out=out, lse=lse, positions=pos)
    assert got is out and gl is lse
    want, wl, spread = ref.merge(outs, lses)
    on = pos >= 0
    tol = (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24) * want.abs() + 2.0 ** -18 * spread
    assert torch.all(((out.double() - want).abs() <= tol)[on])
    none = torch.isneginf(wl)
    assert torch.equal(torch.isneginf(lse)[on], none[on])
    assert torch.all(((lse.double() - wl).abs() <= 2.0 ** -18 + 2.0 ** -22 * wl.abs())[on & ~none.any(1)])
    assert torch.all(out[4] == 9) and torch.all(lse[4] == 9)
    # over one of the parts
    if dtype == out_dtype:
        fresh = ck.ckv_merge_attention(outs, lses, out=torch.empty_like(out))
        same, _ = ck.ckv_merge_attention(outs, lses, out=outs[-1], lse=lses[-1])
        assert torch.equal(fresh[0], same) and torch.equal(fresh[1], lses[-1])


# ------------------------------------------------------------------ together
def test_a_step_over_the_window_and_the_compressed_rows(ck):
    """Maps, rotation and append, attention over the last rows and over the compressed ones, and their merge."""
    B, H, D, P, ps = 3, 8, 128, 4, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    seq, one = _i32([160, 3, 24]), _i32([1, 1, 1])
    err = _err()
    raw_table, raw_free, raw_cur = torch.full((B, 20), -1, dtype=torch.int32, device="cuda"), torch.randperm(60, device="cuda").int(), _i32([0, 0])
    table, free, cur = torch.full((B, 5), -1, dtype=torch.int32, device="cuda"), torch.randperm(15, device="cuda").int(), _i32([0, 0])
    cache = torch.zeros(15, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    kc = _cache(60, ps, 1, D, "rows", float("nan"))
    cs = _angles(200, 64)
    # prefix, then one token each
    for s, n in ((seq - 1, seq - 1), (seq, one)):
        T = int(n.sum())
        m = ck.ckv_build_step_maps(s, n, raw_table, raw_free, raw_cur, 1, ps, T, err_word=err)
        c = ck.ckv_build_step_maps(s, n, table, free, cur, P, ps, T, err_word=err)
        k, q = torch.randn(T, 1, D, generator=g, device="cuda"), torch.randn(T, H, D, generator=g, device="cuda")
        q = ck.ckv_kv_append(k, None, kc, None, m["cache_loc"], positions=m["positions"], cos_sin=cs, q=q, err_word=err)
        ck.ckv_fp4_store(torch.randn(T, D, generator=g, device="cuda"), cache, c["cache_loc"], cache_scale=2.0 ** -6, err_word=err)
    near = ck.ckv_kv_attention(q, kc, kc, raw_table, m["row_start"], m["ctx_rows"], 160, D ** -0.5, window=P, err_word=err)
    far = ck.ckv_fp4_attention(q, cache, table, c["row_start"], c["ctx_rows"], 40, D ** -0.5, cache_scale=2.0 ** -6, err_word=err)
    out, lse = ck.ckv_merge_attention([near[0], far[0]], [near[1], far[1]], positions=m["positions"])
    assert int(err) == 0
    wn = ref.attention(q, kc, kc, raw_table, [0, 1, 2, 3], [160, 3, 24], D ** -0.5, window=P)
    for b, rows in enumerate((40, 0, 6)):
        j = torch.arange(rows, device="cuda")
        far64 = torch.empty(rows, D, device="cuda")
        if rows:
            ck.ckv_fp4_load(cache, table[b].long()[j // ps] * ps + j % ps, far64, cache_scale=2.0 ** -6)
        z = q[b].double() @ far64.double().T * D ** -0.5
        total = torch.logsumexp(torch.cat([z, wn[1][b][:, None]], 1), 1)
        want = torch.exp(z - total[:, None]) @ far64.double() + torch.exp(wn[1][b] - total)[:, None] * wn[0][b]
        size = torch.exp(z - total[:, None]) @ far64.double().abs() + torch.exp(wn[1][b] - total)[:, None] * wn[3][b]
        # both parts' weights and outputs are rounded to bf16, then the result
        assert torch.all((out[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -10) * size)
        assert torch.all((lse[b].double() - total).abs() <= 2.0 ** -12 * (1 + total.abs()))
