"""Calls of the serving-step operators that programs make and a plain parity test does
not: outputs between guard bands, permuted and broadcast inputs, two streams at
once, graphs replayed on changed lengths, caller-owned workspaces, random shapes
against 64-bit arithmetic on the GPU.

Tolerances as in test_gpu_serving_ops.py: bf16 outputs within half a step (2^-8 of
the value) plus the weights' rounding (2^-9 of the cache's largest value)."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from test_gpu_serving_ops import _attn_check, _attn_inputs, _err, _i32, _maps_case, _rope_table

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module")
def ck():
    import compressed_kv_attention_gated_gb300 as ck

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.load()
    return ck


class Guarded:
    """A tensor between two canary bands."""

    def __init__(self, shape, dtype, fill=0):
        n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
        self.raw = torch.full((2 * GUARD + n,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)
        self.t.fill_(fill)

    def intact(self):
        r = self.raw.cpu().numpy()
        return bool(np.all(r[:GUARD] == 0xA5) and np.all(r[GUARD + self.n:] == 0xA5))


def _attn_ref64(q, cache, table, start, ctx, scale, g, sink=None):
    """float64 attention on the GPU, request by request."""
    T, H, D = q.shape
    pages, ps, _ = cache.shape
    flat = cache.view(pages, -1)
    levels = torch.tensor(ref.E2M1, dtype=torch.float64, device=q.device)
    e4 = torch.tensor(np.append(ref.E4M3, 480.0), dtype=torch.float64, device=q.device)
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -torch.inf, dtype=torch.float64, device=q.device)
    if sink is not None:
        lse[:] = sink.double()
    for b in range(len(start) - 1):
        lo, hi = int(start[b]), int(start[b + 1])
        c = ctx[lo:hi]
        L = int(c.max()) if hi > lo else 0
        if L <= 0:
            continue
        pg = flat[table[b, : -(-L // ps)].long()]
        codes = pg[:, : ps * D // 2].reshape(-1, D // 2)[:L].long()
        s = e4[pg[:, ps * D // 2:].reshape(-1, D // 16)[:L].long() & 127]
        k = torch.stack([levels[codes & 15], levels[codes >> 4]], -1).view(L, D) * s.repeat_interleave(16, 1) * g
        z = torch.einsum("thd,jd->thj", q[lo:hi].double(), k) * scale
        z.masked_fill_((torch.arange(L, device=q.device) >= c[:, None])[:, None], -torch.inf)
        if sink is not None:
            z = torch.cat([z, sink.double()[None, :, None].expand(hi - lo, H, 1)], -1)
        lse[lo:hi] = torch.logsumexp(z, -1)
        w = torch.exp(z - lse[lo:hi, :, None].clamp(min=-1e300))[..., :L]
        out[lo:hi] = torch.einsum("thj,jd->thd", w, k)
    return out, lse


def test_guard_bands(ck):
    rng = np.random.default_rng(0)
    # maps
    s, n, table, free, tails = _maps_case(rng, 37, 0, 9, 500, 4, 3, True)
    T = int(n.sum()) + 5
    tab = Guarded(table.shape, torch.int32)
    tab.t.copy_(_i32(table))
    out = {k: Guarded((38,) if k == "row_start" else (T,), torch.int64 if k == "cache_loc" else torch.int32) for k in
           ("row_start", "positions", "batch_ids", "slot_mapping", "cache_loc", "tail_slots", "row_positions", "ctx_rows")}
    cur = Guarded((2,), torch.int32)
    ck.ckv_build_step_maps(_i32(s), _i32(n), tab.t, _i32(free), cur.t, 4, 3, T, tail_blocks=_i32(tails),
                           out={k: v.t for k, v in out.items()})
    assert tab.intact() and cur.intact() and all(v.intact() for v in out.values())
    # norm + rotation
    for D in (128, 256, 512):
        for R, at, il in ((D, 0, False), (70, 6, True), (64, D - 64, True)):
            q, k = torch.randn(13, 5, D, device="cuda").bfloat16(), torch.randn(7, 1, D, device="cuda")
            qo, ko = Guarded((13, 5, D), torch.bfloat16), Guarded((7, 1, D), torch.float32)
            ck.ckv_qk_norm_rope(q, _i32(rng.integers(-1, 20, 13)), _rope_table(20, R, torch.Generator().manual_seed(0)).cuda(),
                                q_out=qo.t, k=k, k_positions=_i32(rng.integers(-1, 20, 7)), k_out=ko.t, rope_offset=at, interleaved=il)
            assert qo.intact() and ko.intact()
        # rows
        cache = Guarded((5, 6, D // 2 + D // 16), torch.uint8)
        x = torch.randn(17, D, device="cuda")
        loc = torch.from_numpy(rng.permutation(30)[:17]).cuda()
        loc[3], loc[4] = 30, 2 ** 50
        back = Guarded((17, D), torch.bfloat16)
        ck.ckv_fp4_store(x, cache.t, loc)
        ck.ckv_fp4_load(cache.t, loc, back.t)
        assert cache.intact() and back.intact()
        # attention: one CTA per tile, and split with a workspace
        for H, n, ctx in ((5, [1, 3], [40, 300, 0, -1]), (64, [2], [4000, 3990]), (16, [1], [9000])):
            ctx = np.array(ctx)
            start, T, table, cbytes, q, width = _attn_inputs(rng, np.array(n), ctx, H, D, 16)
            o, l = Guarded((T, H, D), torch.bfloat16), Guarded((T, H), torch.float32)
            need = ck.ckv_fp4_attention_workspace(T, len(n), H, D, int(ctx.max()))
            ws = Guarded((need,), torch.uint8)
            ck.ckv_fp4_attention(q.cuda(), torch.from_numpy(cbytes).cuda(), _i32(table), _i32(start), _i32(ctx), int(ctx.max()), 0.1,
                                 out=o.t, lse=l.t, workspace=ws.t)
            assert o.intact() and l.intact() and ws.intact()
            assert need > 0 or int(ctx.max()) < 4000  # the long ones are split


@pytest.mark.parametrize("D,H", [(128, 6), (128, 40), (256, 36), (512, 24)])
def test_fp4_attention_permuted_and_broadcast_queries(ck, D, H):
    """Queries as [heads, tokens, D] in memory, and one query row for all heads or all tokens."""
    rng = np.random.default_rng(1)
    ctx = np.array([100, 260, 261, 262])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 3]), ctx, H, D, 32)
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), 262, D ** -0.5)
    q = q.cuda()
    o, l = ck.ckv_fp4_attention(q, *args)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert turned.stride(0) != q.stride(0)
    o1, l1 = ck.ckv_fp4_attention(turned, *args)
    assert torch.equal(o, o1) and torch.equal(l, l1)
    for e in (q[:1].expand(T, H, D), q[:, :1].expand(T, H, D)):
        o1, l1 = ck.ckv_fp4_attention(e, *args)
        o2, l2 = ck.ckv_fp4_attention(e.contiguous(), *args)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    # a negative scale is the same as negative queries
    o1, l1 = ck.ckv_fp4_attention(q, *args[:-1], -args[-1])
    o2, l2 = ck.ckv_fp4_attention(-q, *args)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    # scale 0: the mean of the rows
    o1, l1 = ck.ckv_fp4_attention(q, *args[:-1], 0.0)
    assert torch.allclose(l1, torch.log(_i32(ctx).float())[:, None].expand(T, H), atol=1e-5)


def test_two_streams_at_once(ck):
    """Calls on two streams at the same time, each with its own outputs, keep their bits."""
    rng = np.random.default_rng(2)
    cases = []
    for D, H, n, ctx in ((512, 64, [1, 1], [3000, 2000]), (128, 64, [1, 1, 1], [5000, 100, 2500]), (256, 10, [4], [700, 701, 702, 703])):
        ctx = np.array(ctx)
        start, T, table, cache, q, width = _attn_inputs(rng, np.array(n), ctx, H, D, 64)
        args = (q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), int(ctx.max()), D ** -0.5)
        cases.append((args, ck.ckv_fp4_attention(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        got = [ck.ckv_fp4_attention(*args, stream=streams[i]) for i, (args, _) in enumerate(cases) for _ in range(2)]
        torch.cuda.synchronize()
        for i, (_, (o, l)) in enumerate(cases):
            for g in got[2 * i:2 * i + 2]:
                assert torch.equal(g[0], o) and torch.equal(g[1], l)


def test_a_captured_step_follows_its_lengths(ck):
    """Maps, store and attention in one graph, replayed while lengths grow on the device; a second
    graph captured after it runs between the replays and shares nothing with it."""
    B, H, D, P, ps, width = 4, 20, 128, 4, 4, 40
    g = torch.Generator().manual_seed(3)
    seq = torch.tensor([0, 5, 130, 260], dtype=torch.int32).cuda()
    ones = _i32(np.ones(B))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(B * width, generator=g).to(torch.int32).cuda()
    cursor, err = _i32([0, 0]), _err()
    cache = torch.zeros(B * width, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    # the rows that the prefixes closed
    pre = ck.ckv_build_step_maps(seq, seq, table, free, cursor, P, ps, int(seq.sum()), err_word=err)
    x = torch.randn(int(seq.sum()), D, generator=g).cuda()
    ck.ckv_fp4_store(x, cache, pre["cache_loc"], cache_scale=2.0 ** -6, err_word=err)
    row, q = torch.zeros(B, D, device="cuda"), torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda")

    def step(out):
        m = ck.ckv_build_step_maps(seq, ones, table, free, cursor, P, ps, B, err_word=err)
        ck.ckv_fp4_store(row, cache, m["cache_loc"], cache_scale=2.0 ** -6, err_word=err)
        ck.ckv_fp4_attention(q, cache, table, m["row_start"], m["ctx_rows"], width * ps, 0.2, cache_scale=2.0 ** -6, out=out[0], lse=out[1],
                             err_word=err)
        return m

    outs = [(torch.zeros_like(q), torch.zeros(B, H, device="cuda")) for _ in range(2)]
    graphs = []
    seq += 1
    torch.cuda.synchronize()
    for o in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            m = step(o)
            seq += 1
        graphs.append((gr, o, m))
    lens = [1, 6, 131, 261]
    for i in range(10):
        gr, o, m = graphs[i % 2]
        row.copy_(torch.randn(B, D, generator=g))
        q.copy_(torch.randn(B, H, D, generator=g))
        gr.replay()
        torch.cuda.synchronize()
        assert int(err) == 0
        ctx = torch.tensor([n // P for n in lens]).cuda()
        assert m["ctx_rows"].tolist() == ctx.tolist()
        want, wlse = _attn_ref64(q, cache, table, list(range(B + 1)), ctx, 0.2, 2.0 ** -6)
        assert bool(((o[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * 6).all())
        fin = torch.isfinite(wlse)
        assert torch.equal(fin, torch.isfinite(o[1])) and bool(((o[1].double() - wlse)[fin].abs() <= 1e-4).all())
        lens = [n + 1 for n in lens]
    # every page is held once
    held = table[table >= 0]
    assert held.unique().numel() == held.numel() == int(cursor[0])


@pytest.mark.parametrize("seed", range(24))
def test_fp4_attention_random_shapes(ck, seed):
    """Any head count, widths, pages, ragged and padded batches, split or not."""
    rng = np.random.default_rng(100 + seed)
    D = int(rng.choice([128, 256, 512]))
    H = int(rng.choice([1, 2, 3, 7, 8, 12, 16, 24, 32, 33, 48, 64, 80, 128, 200]))
    ps = int(rng.choice([2, 16, 48, 64, 100, 256]))
    B = int(rng.integers(1, 9))
    n = rng.integers(0, 2 if seed % 2 else 60, B)
    n[0] = max(1, n[0])
    top = int(rng.choice([5, 130, 700, 3000]))
    ctx = np.concatenate([np.sort(rng.integers(0, top + 1, k)) for k in n])
    ctx[rng.random(len(ctx)) < 0.1] = -1
    g = 2.0 ** int(rng.integers(-8, 3))
    start, T, table, cache, q, width = _attn_inputs(rng, n, ctx, H, D, ps)
    sink = torch.from_numpy(rng.standard_normal(H).astype(np.float32) * 3).cuda() if seed % 3 == 0 else None
    q, c, tab, cx = q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(ctx)
    scale = 1.5 * D ** -0.5 / g
    out = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 9.0, device="cuda")
    err = _err()
    ck.ckv_fp4_attention(q, c, tab, _i32(start), cx, max(1, int(ctx.max())), scale, cache_scale=g, sink=sink, out=out, lse=lse, err_word=err)
    assert int(err) == 0
    want, wlse = _attn_ref64(q, c, tab, start, cx, scale, g, sink)
    on = cx >= 0
    assert bool((out[~on] == 9).all()) and bool((lse[~on] == 9).all())
    e = (out.double() - want)[on].abs()
    assert bool((e <= 2.0 ** -8 * want[on].abs() + 2.0 ** -9 * 6 * g).all())
    fin = torch.isfinite(wlse[on])
    assert torch.equal(fin, torch.isfinite(lse[on]))
    assert bool(((lse.double() - wlse)[on][fin].abs() <= 2.0 ** -16 * (10 + wlse[on][fin].abs())).all())


@pytest.mark.parametrize("seed", range(12))
def test_step_maps_random(ck, seed):
    rng = np.random.default_rng(300 + seed)
    P, ps = int(rng.choice([1, 3, 16, 128, 1024])), int(rng.choice([1, 7, 64]))
    B = int(rng.integers(1, 60))
    s, n, table, free, tails = _maps_case(rng, B, 0, int(rng.choice([1, 5, 600])), int(rng.choice([0, 100, 5000])), P, ps, seed % 2 == 0)
    T = int(n.sum()) + int(rng.integers(0, 4))
    want, wtable, wcur = ref.step_maps(s, n, table, free, 0, P, ps, T, tails)
    tab, cur, err = _i32(table), _i32([0, 0]), _err()
    got = ck.ckv_build_step_maps(_i32(s), _i32(n), tab, _i32(free), cur, P, ps, T, tail_blocks=None if tails is None else _i32(tails),
                                 err_word=err)
    assert int(err) == 0 and cur.tolist() == [wcur, 0]
    for k in want:
        np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=k)
    np.testing.assert_array_equal(tab.cpu().numpy(), wtable)


def test_step_maps_of_a_capacity_past_the_narrow_sums(ck):
    """More than 2^21 token places: the sums are formed in two parts."""
    T = (1 << 21) + 70000
    n = np.array([T - 70001, 0, 65537, 4400])
    s = n + np.array([5, 9, 0, 100])
    P, ps, width = 16, 64, -(-(int(s.max()) // 16) // 64)
    free = np.random.default_rng(0).permutation(3 * width)
    table = np.full((4, width), -1)
    for b in range(4):
        for pg in range(-(-((int(s[b]) - int(n[b])) // P) // ps)):
            table[b, pg] = 7
    tab, cur, err = _i32(table), _i32([0, 0]), _err()
    got = ck.ckv_build_step_maps(_i32(s), _i32(n), tab, _i32(free), cur, P, ps, T, err_word=err)
    assert int(err) == 0
    start = np.concatenate([[0], np.cumsum(n)])
    assert got["row_start"].tolist() == start.tolist()
    pos = np.concatenate([np.arange(s[b] - n[b], s[b]) for b in range(4)])
    np.testing.assert_array_equal(got["positions"].cpu().numpy()[: start[-1]], pos)
    assert bool((got["positions"][int(start[-1]):] == -1).all())
    closes = (pos + 1) % P == 0
    t = tab.cpu().numpy()
    b = np.repeat(np.arange(4), n)
    want = np.where(closes, t[b, np.minimum(pos // P // ps, width - 1)] * ps + pos // P % ps, -1)
    np.testing.assert_array_equal(got["cache_loc"].cpu().numpy()[: start[-1]], want)


def test_norm_rope_large_strides(ck):
    """Rows past 2^31 elements."""
    T, H, D = 3, 2, 512
    st = (1 << 30) + 4096
    big = torch.empty((T - 1) * st + H * D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, H, D), (st, D, 1))
    x.copy_(torch.randn(T, H, D))
    y = x.contiguous()
    table = _rope_table(8, 64, torch.Generator().manual_seed(0)).cuda()
    pos = _i32([1, 2, 7])
    a, _ = ck.ckv_qk_norm_rope(x, pos, table)
    b, _ = ck.ckv_qk_norm_rope(y, pos, table)
    assert torch.equal(a, b)
    ck.ckv_qk_norm_rope(x, pos, table, q_out=x)
    assert torch.equal(x.contiguous(), b)


@pytest.mark.parametrize("D", [128, 512])
@pytest.mark.parametrize("H", [1, 2, 3, 6, 8, 12, 24, 48, 96, 160])
def test_fp4_attention_tiles_of_ragged_requests(ck, D, H):
    """Tiles are counted without room to spare: every row of requests of 0 to 5 tokens has one,
    whatever the common divisor of the heads and a tile's rows."""
    rng = np.random.default_rng(H)
    for most in (1, 2, 5):
        n = rng.integers(0, most + 1, 33)
        n[0], n[-1] = most, most
        _attn_check(ck, rng, n, rng.integers(0, 40, int(n.sum())), H, D, 16, False)


@pytest.mark.parametrize("D,H,rows", [(128, 4, 131149), (128, 40, 60000), (512, 4, 50001), (512, 70, 30000)])
def test_fp4_attention_many_ranges(ck, D, H, rows):
    """One request over so many rows that they are split into more ranges than a warp has lanes."""
    rng = np.random.default_rng(rows)
    _attn_check(ck, rng, np.array([1]), [rows], H, D, 64, True)
