"""The serving-step operators on the GPU against 64-bit references: step maps,
norm + rotation, 4-bit rows, attention over 4-bit rows, and a step that runs
them together.

Tolerances, from the operators' arithmetic:
  * maps and 4-bit codes/scales: exact
  * norm + rotation: fp32 arithmetic on D <= 512 values (errors below 2^-18 of
    the largest channel), then one rounding: bf16 2^-8 or fp32 2^-24 of the value
  * attention: keys and values are exact in the matrix products' 16-bit type, q
    keeps its 8 bits; the weights are rounded to 16 bits (2^-9 at worst for
    values that average out, at most 2^-9 of sum w |k| <= max|k|), the output to
    bf16 (2^-8 of the value); lse is fp32 arithmetic on sums of D products
    (2^-24 sqrt(D) of sum |q k| scale, bounded by 2^-16 of it)
"""
import numpy as np
import pytest
import torch

import serving_reference as ref

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


# ------------------------------------------------------------------ step maps
def _maps_case(rng, B, n_lo, n_hi, prefix, P, ps, tails):
    n = rng.integers(n_lo, n_hi + 1, B)
    s = rng.integers(0, prefix + 1, B) + n
    width = max(1, -(-((prefix + n_hi) // P) // ps))
    total = B * width + 5
    perm = rng.permutation(total)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        have = -(-((s[b] - n[b]) // P) // ps)
        table[b, :have] = perm[at:at + have]
        at += have
    return s, n, table, perm[at:], (rng.permutation(B + 3)[:B] - 1 if tails else None)


@pytest.mark.parametrize("B,n_lo,n_hi,prefix,P,ps", [
    (1, 1, 1, 0, 16, 64), (1, 1, 1, 127, 128, 1), (5, 0, 3, 40, 1, 3), (512, 4, 4, 4000, 16, 64), (64, 0, 700, 900, 128, 2),
    (3, 5000, 9000, 3, 4, 7), (1025, 0, 2, 70, 2, 5), (8192, 0, 1, 300, 16, 4), (7, 1, 5000, 100000, 1000, 48)])
@pytest.mark.parametrize("inplace", [False, True])
def test_step_maps(ck, B, n_lo, n_hi, prefix, P, ps, inplace):
    rng = np.random.default_rng(B * 7 + P)
    s, n, table, free, tails = _maps_case(rng, B, n_lo, n_hi, prefix, P, ps, P != 2)
    live = int(n.sum())
    for T in (live, live + 13):
        cur = 2
        want, wtable, wcur = ref.step_maps(s, n, table, np.concatenate([[7, 7], free]), cur, P, ps, T, tails)
        wide = torch.full((B, table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")  # a strided table
        wide[:, :table.shape[1]] = _i32(table)
        cursor, err = _i32([cur, 0]), _err()
        nxt = None if inplace else _i32([-5])
        got = ck.ckv_build_step_maps(_i32(s), _i32(n), wide[:, :table.shape[1]], _i32(np.concatenate([[7, 7], free])), cursor,
                                     P, ps, T, tail_blocks=None if tails is None else _i32(tails), cursor_out=nxt, err_word=err)
        assert int(err) == 0
        assert set(got) == set(want)
        for k in want:
            np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=k)
        np.testing.assert_array_equal(wide[:, :table.shape[1]].cpu().numpy(), wtable)
        assert bool((wide[:, table.shape[1]:] == -9).all())
        assert cursor.tolist() == ([wcur, 0] if inplace else [cur, 0])
        if not inplace:
            assert nxt.tolist() == [wcur]


def test_step_maps_of_successive_steps_and_a_replayed_graph(ck):
    """Forty decode steps in place from one captured graph: every page is taken once,
    and the maps stay those of the reference."""
    B, P, ps = 9, 4, 2
    n = np.full(B, 3)
    s = np.arange(B) + 3
    width = 40
    free = np.random.default_rng(0).permutation(B * width)
    table = np.full((B, width), -1)
    seq, nn, tab, fr, cur = _i32(s), _i32(n), _i32(table), _i32(free), _i32([0, 0])
    maps = ck.ckv_build_step_maps(seq, nn, tab.clone(), fr, cur.clone(), P, ps, 3 * B)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ckv_build_step_maps(seq, nn, tab, fr, cur, P, ps, 3 * B, out=maps)
        seq += nn
    at = 0
    # rows closed before the first step (s - n = 0 .. B - 1 positions) have their pages already
    for b in range(B):
        have = -(-((s[b] - 3) // P) // ps)
        table[b, :have] = 1000 + b
        tab[b, :have] = 1000 + b
    for _ in range(40):
        g.replay()
        torch.cuda.synchronize()
        want, table, at = ref.step_maps(s, n, table, free, at, P, ps, 3 * B)
        for k in want:
            np.testing.assert_array_equal(maps[k].cpu().numpy(), want[k], err_msg=k)
        np.testing.assert_array_equal(tab.cpu().numpy(), table)
        assert cur.tolist() == [at, 0]
        s = s + n


def test_step_maps_flags_what_it_cannot_build(ck):
    P, ps = 2, 2
    table = np.full((3, 2), -1)

    def run(s, n, free, T, cursor=0, tab=table):
        err, cur = _err(), _i32([cursor, 0])
        t = _i32(tab)
        got = ck.ckv_build_step_maps(_i32(s), _i32(n), t, _i32(free), cur, P, ps, T, err_word=err)
        return {k: v.cpu().numpy() for k, v in got.items()}, t.cpu().numpy(), int(err), cur.tolist()

    # a request that is longer than it can be counts as empty
    got, tab, err, cur = run([4, 3, 2], [4, 4, 2], range(10, 20), 7)
    assert err == 0x10 and got["row_start"].tolist() == [0, 4, 4, 6] and cur == [2, 0]
    assert got["batch_ids"].tolist() == [0] * 4 + [2] * 2 + [-1]
    assert tab.tolist() == [[10, -1], [-1, -1], [11, -1]]
    got, _, err, _ = run([4, 3, 2], [4, -1, 2], range(10, 20), 6)
    assert err == 0x10 and got["batch_ids"].tolist() == [0] * 4 + [2] * 2
    # more tokens than the maps hold
    got, _, err, _ = run([4, 3, 2], [4, 3, 2], range(10, 20), 5)
    assert err == 0x8 and got["row_start"].tolist() == [0, 4, 5, 5] and got["batch_ids"].tolist() == [0] * 4 + [1]
    # free list of one page; a table of two pages for five rows; a table without a held page
    got, tab, err, cur = run([8, 0, 0], [8, 0, 0], [10], 8)
    assert err == 0x80 and cur == [1, 0] and tab[0].tolist() == [10, -1]
    assert got["cache_loc"].tolist() == [-1, 20, -1, 21, -1, -1, -1, -1]
    got, tab, err, cur = run([10, 0, 0], [10, 0, 0], range(10, 20), 10)
    assert err == 0x80 and cur == [2, 0] and got["cache_loc"].tolist() == [-1, 20, -1, 21, -1, 22, -1, 23, -1, -1]
    got, _, err, _ = run([4, 0, 0], [1, 0, 0], range(10, 20), 1)
    assert err == 0x80 and got["cache_loc"].tolist() == [-1] and got["ctx_rows"].tolist() == [2]
    # a cursor before the list, or past it, takes nothing and stays
    for c in (-1, 40):
        got, tab, err, cur = run([2, 0, 0], [2, 0, 0], range(10, 20), 2, cursor=c)
        assert err == 0x80 and cur == [c, 0] and tab[0].tolist() == [-1, -1] and got["cache_loc"].tolist() == [-1, -1]
    # a location past 32 bits: the 64-bit map has it
    big = np.array([[2 ** 31 - 1, -1], [-1, -1], [-1, -1]])
    got, _, err, _ = run([4, 0, 0], [1, 0, 0], range(10, 20), 1, tab=big)
    assert err == 0x4 and got["slot_mapping"].tolist() == [-1] and got["cache_loc"].tolist() == [(2 ** 31 - 1) * 2 + 1]
    # no request at all
    cur, start = _i32([3]), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o = ck.ckv_build_step_maps(_i32([]), _i32([]), torch.zeros((0, 2), dtype=torch.int32, device="cuda"), _i32([5]), _i32([3]), 4, 4,
                               2, cursor_out=cur, out={"row_start": start, "ctx_rows": torch.zeros(2, dtype=torch.int32, device="cuda")})
    assert o["row_start"].tolist() == [0] and o["ctx_rows"].tolist() == [-1, -1] and cur.tolist() == [3]


# ------------------------------------------------------------------ norm + rotation
def _rope_table(n, R, g):
    a = torch.rand(n, max(1, R // 2), generator=g, dtype=torch.float64) * 6.283
    return torch.cat([a.cos(), a.sin()], 1).float()[:, :R].contiguous()


def _norm_close(got, want, what):
    got = got.double().cpu().numpy()
    half = 2.0 ** -8 if what == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(want) + 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


@pytest.mark.parametrize("D,R,at", [(128, 128, 0), (128, 64, 64), (128, 0, 0), (256, 2, 254), (256, 70, 10), (512, 64, 448),
                                    (512, 510, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Tk", [(1, 1, 0), (3, 5, 7), (33, 3, 1)])
def test_norm_rope(ck, D, R, at, interleaved, T, H, Tk):
    g = torch.Generator().manual_seed(D + R + T)
    table = _rope_table(50, R, g)
    q = (torch.randn(T, H, D, generator=g) * 3).bfloat16()
    k = torch.randn(Tk, 1, D, generator=g) * 1e-3
    qp = torch.randint(-2, 50, (T,), generator=g, dtype=torch.int32)
    kp = torch.randint(-2, 50, (Tk,), generator=g, dtype=torch.int32)
    qp[0] = 49
    q[qp < 0] = float("nan")  # rows that are skipped may hold anything
    w = torch.randn(D, generator=g)
    big = torch.zeros(T, H + 2, D + 16, dtype=torch.bfloat16, device="cuda")  # strided queries
    qs = big[:, 1:H + 1, 8:8 + D]
    qs.copy_(q)
    for odt in (torch.bfloat16, torch.float32):
        qo = torch.full((T, H, D), -7.0, dtype=odt, device="cuda")
        ko = torch.full((Tk, 1, D), -7.0, dtype=odt, device="cuda")
        err = _err()
        ck.ckv_qk_norm_rope(qs, qp.cuda(), table.cuda() if R else None, q_weight=w.cuda(), q_out=qo, k=k.cuda() if Tk else None,
                            k_positions=kp.cuda() if Tk else None, k_out=ko if Tk else None, rope_offset=at,
                            interleaved=interleaved, eps=1e-6, err_word=err)
        assert int(err) == 0
        want = ref.norm_rope(q.float().numpy(), qp.numpy(), table.numpy(), w.numpy(), R, at, interleaved, 1e-6)
        on = (qp >= 0).numpy()
        _norm_close(qo.cpu()[on], want[on], odt)
        assert bool((qo.cpu()[~on] == -7).all())
        if Tk:
            want = ref.norm_rope(k.numpy(), kp.numpy(), table.numpy(), None, R, at, interleaved, 1e-6)
            on = (kp >= 0).numpy()
            _norm_close(ko.cpu()[on], want[on], odt)
            assert bool((ko.cpu()[~on] == -7).all())
    # in place, strided: the same values, nothing beside them
    ck.ckv_qk_norm_rope(qs, qp.cuda(), table.cuda() if R else None, q_weight=w.cuda(), q_out=qs, rope_offset=at,
                        interleaved=interleaved, eps=1e-6)
    want = ref.norm_rope(q.float().numpy(), qp.numpy(), table.numpy(), w.numpy(), R, at, interleaved, 1e-6)
    on = (qp >= 0).numpy()
    _norm_close(qs.cpu()[on], want[on], torch.bfloat16)
    rest = big.clone()
    rest[:, 1:H + 1, 8:8 + D] = 0
    assert bool((rest == 0).all())


def test_norm_rope_positions_past_the_table_and_zero_rows(ck):
    table = _rope_table(4, 64, torch.Generator().manual_seed(0)).cuda()
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    err = _err()
    ck.ckv_qk_norm_rope(x, _i32([3, 4, 2 ** 31 - 1]), table, q_out=out, err_word=err)
    assert int(err) == 0x10
    assert bool((out[0] == 0).all()) and bool((out[1:] == 5).all())


# ------------------------------------------------------------------ 4-bit rows
def _fp4_inputs(rng, n, D):
    x = rng.standard_normal((n, D)) * np.exp(rng.standard_normal((n, 1)) * 2)
    x[:, ::7] = 0
    if n > 3:
        x[0] = 0
        x[1] = 1e30  # saturates
        x[2] = 1e-30  # scales round to 0
        # every rounding border of both formats, exactly and a step beside it
        b = np.concatenate([[6.0], np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0.0])])
        x[3] = np.tile(b, D // 16)
    return x


@pytest.mark.parametrize("D,ps", [(128, 2), (128, 64), (256, 1), (256, 100), (512, 1), (512, 48)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,g", [(1, 1.0), (37, 2.0 ** -6), (1000, 2.0 ** 10)])
def test_fp4_rows(ck, D, ps, dtype, n, g):
    rng = np.random.default_rng(n + D)
    x = torch.tensor(_fp4_inputs(rng, n, D), dtype=torch.float64).to(dtype)
    if n > 3:
        x[4:7] = x[4:7] * g
        if dtype == torch.float32:  # floats next to the borders
            x[7] = torch.nextafter(x[3], torch.full_like(x[3], 9.0))
            x[7, ::16] = 6.0
            x[8] = torch.nextafter(x[3], torch.full_like(x[3], -9.0))
            x[8, ::16] = 6.0
            x[7:9] *= g
        x[3] = x[3] * g
    pages = -(-n // ps) + 2
    loc = torch.from_numpy(rng.permutation(pages * ps)[:n].astype(np.int64))
    if n > 1:
        loc[rng.random(n) < 0.3] = -1
        loc[3] = max(int(loc[3]), 0) if int(loc[3]) >= 0 else -1
    cache = torch.full((pages, ps, D // 2 + D // 16), 0xA5, dtype=torch.uint8)
    want = cache.numpy().copy().reshape(pages, -1)
    codes, scales = ref.fp4_rows(x.double().numpy(), g)
    for i in range(n):
        if loc[i] >= 0:
            p, r = divmod(int(loc[i]), ps)
            row = ref.pack_page(codes[i:i + 1], scales[i:i + 1])
            want[p, r * (D // 2):(r + 1) * (D // 2)] = row[:D // 2]
            want[p, ps * (D // 2) + r * (D // 16): ps * (D // 2) + (r + 1) * (D // 16)] = row[D // 2:]
    wide = torch.full((n, D + 8), float("nan"), dtype=dtype)
    wide[:, :D] = torch.where((loc >= 0)[:, None], x, torch.full_like(x, float("nan")))  # skipped rows are not read
    c, err = cache.cuda(), _err()
    ck.ckv_fp4_store(wide.cuda()[:, :D], c, loc.cuda(), cache_scale=g, err_word=err)
    assert int(err) == 0
    np.testing.assert_array_equal(c.cpu().numpy().reshape(pages, -1), want)
    for odt in (torch.bfloat16, torch.float32):
        back = torch.full((n, D + 8), -3.0, dtype=odt, device="cuda")
        ck.ckv_fp4_load(c, loc.cuda(), back[:, :D], cache_scale=g, err_word=err)
        exact = np.array([ref.fp4_row_values(want.reshape(cache.shape), int(l), D, g) if l >= 0 else np.full(D, -3.0) for l in loc])
        np.testing.assert_array_equal(back[:, :D].double().cpu().numpy(), exact)
        assert bool((back[:, D:] == -3).all())


def test_fp4_rows_bad_locations_and_non_finite(ck):
    D, ps = 128, 4
    c0 = torch.full((2, ps, 72), 0x11, dtype=torch.uint8, device="cuda")
    x = torch.randn(4, D, device="cuda")
    for bad in (8, 2 ** 40, 2 ** 62):
        c, err = c0.clone(), _err()
        ck.ckv_fp4_store(x, c, torch.tensor([-1, bad, -2 ** 62, -7], device="cuda"), err_word=err)
        assert int(err) == 0x4 and torch.equal(c, c0)
        out = torch.full((4, D), 2.0, device="cuda")
        ck.ckv_fp4_load(c, torch.tensor([-1, bad, -2 ** 62, -7], device="cuda"), out, err_word=err)
        assert bool((out == 2).all())
    x[0, 5], x[1, 6], x[2, 7] = float("nan"), float("inf"), float("-inf")
    c = c0.clone()
    ck.ckv_fp4_store(x, c, torch.arange(4, device="cuda"))
    out = torch.zeros(4, D, device="cuda")
    ck.ckv_fp4_load(c, torch.arange(4, device="cuda"), out)
    assert bool(torch.isfinite(out).all()) and float(out[1, 6]) == 2688 and float(out[2, 7]) == -2688


# ------------------------------------------------------------------ attention
def _attn_inputs(rng, n, ctx, H, D, ps, spare=1, stride_pages=0):
    """A random cache with pages in random order; ctx gives every token's rows."""
    B = len(n)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    T = int(start[-1])
    rows = [max([0, *ctx[start[b]:start[b + 1]]]) for b in range(B)]
    width = max(1, max([-(-r // ps) for r in rows], default=1))
    need = sum(-(-r // ps) for r in rows)
    pages = need + spare
    perm = rng.permutation(pages)
    table = np.full((B, width + stride_pages), -1)
    at = 0
    for b in range(B):
        k = -(-rows[b] // ps)
        table[b, :k] = perm[at:at + k]
        at += k
    cache = rng.integers(0, 256, (pages, ps, D // 2 + D // 16), dtype=np.uint8)
    flat = cache.reshape(pages, -1)
    # scales of normalised rows: 1/8 .. 1, any byte (0x7F and 0xFF too) in the rows that no token sees
    flat[:, ps * D // 2:] = rng.integers(0x20, 0x39, (pages, ps * D // 16))
    used = {int(table[b, j // ps]) * ps + j % ps for b in range(B) for j in range(rows[b])}
    for loc in range(pages * ps):
        if loc not in used:
            flat[loc // ps, ps * D // 2 + (loc % ps) * (D // 16): ps * D // 2 + (loc % ps + 1) * (D // 16)] = rng.choice([0x7F, 0xFF, 0x7E])
    q = torch.from_numpy(rng.standard_normal((T, H, D))).bfloat16()
    return start, T, table, cache, q, width


def _attn_check(ck, rng, n, ctx, H, D, ps, sink, g=1.0, extra_tokens=0, max_rows=None, scale=None):
    ctx = np.asarray(ctx)
    start, T, table, cache, q, width = _attn_inputs(rng, n, ctx, H, D, ps, stride_pages=2)
    scale = scale if scale is not None else D ** -0.5 / g
    sk = rng.standard_normal(H).astype(np.float32) * 2 if sink else None
    Tx = T + extra_tokens
    qx = torch.full((Tx, H, D + 8), float("nan"), dtype=torch.bfloat16)
    qx[:T, :, :D] = q
    qx[:T][ctx < 0] = float("nan")
    out = torch.full((Tx, H, D), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Tx, H), -7.0, device="cuda")
    err = _err()
    ctx_x = np.concatenate([ctx, np.full(extra_tokens, 1)])
    mr = max_rows or max(1, int(ctx.max(initial=1)))
    tab = _i32(table)[:, :max(width, -(-mr // ps)) if max_rows else width]
    ck.ckv_fp4_attention(qx.cuda()[:, :, :D], torch.from_numpy(cache).cuda(), tab, _i32(start), _i32(ctx_x), mr, scale,
                         cache_scale=g, sink=None if sk is None else torch.from_numpy(sk).cuda(), out=out, lse=lse, err_word=err)
    assert int(err) == 0
    want, wlse, seen = ref.attention(q.float().numpy(), cache, table, start, ctx, scale, g, sk)
    o, s = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(o[T:] == -7) and np.all(s[T:] == -7) and np.all(o[:T][~seen] == -7) and np.all(s[:T][~seen] == -7)
    o, s, want, wlse = o[:T][seen], s[:T][seen], want[seen], wlse[seen]
    top = 6 * g  # the largest value of the cache
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * top
    assert np.all(np.abs(o - want) <= tol), np.max(np.abs(o - want) - tol)
    # the weights' roundings average out over the rows: far below the bound that holds for each value
    assert np.sqrt(np.mean((o - want) ** 2)) <= 2.0 ** -9 * max(np.sqrt(np.mean(want ** 2)), 2.0 ** -6 * top) * 1.5
    assert np.array_equal(np.isneginf(s), np.isneginf(wlse))
    fin = np.isfinite(wlse)
    size = 1 + np.abs(wlse[fin]) + D ** 0.5 * 4 * top * scale
    assert np.all(np.abs(s[fin] - wlse[fin]) <= 2.0 ** -16 * size)


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 64, 100])
@pytest.mark.parametrize("sink", [False, True])
def test_fp4_attention_decode(ck, D, H, sink):
    """One token per request: no rows, one row, around the ends of pages and tiles, long."""
    rng = np.random.default_rng(D + H)
    ctx = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0, 700]
    _attn_check(ck, rng, np.ones(len(ctx), int), ctx, H, D, 16 if H < 64 else 6, sink)


@pytest.mark.parametrize("D,H,ps", [(128, 8, 64), (128, 3, 2), (256, 24, 48), (512, 16, 1), (512, 128, 64)])
def test_fp4_attention_prompts(ck, D, H, ps):
    """Ragged requests (empty ones too) whose tokens see more and more rows, or none, or are padding."""
    rng = np.random.default_rng(H)
    n = np.array([0, 1, 37, 0, 5, 130, 2, 0])
    ctx = []
    for b, k in enumerate(n):
        first = int(rng.integers(0, 200))
        ctx += list(np.maximum(0, first + (np.arange(k) - 10) // 3))
    ctx = np.array(ctx)
    ctx[rng.random(len(ctx)) < 0.1] = -1
    ctx[rng.random(len(ctx)) < 0.1] = 0
    _attn_check(ck, rng, n, ctx, H, D, ps, True, extra_tokens=3)


@pytest.mark.parametrize("D,H,rows", [(128, 64, 9000), (256, 7, 4100), (512, 16, 2600), (512, 64, 5000)])
def test_fp4_attention_long(ck, D, H, rows):
    """Long rows of few requests: the work is split over many CTAs and joined."""
    rng = np.random.default_rng(rows)
    _attn_check(ck, rng, np.array([1, 2, 1]), [rows, 0, rows - 129, 5], H, D, 64, H == 64)
    _attn_check(ck, rng, np.array([1]), [rows], H, D, 64, False, g=2.0 ** -6)


def test_fp4_attention_bound_above_the_rows(ck):
    """max_rows is a bound only: a loose one changes nothing."""
    rng = np.random.default_rng(3)
    _attn_check(ck, rng, np.array([1, 3, 1]), [0, 0, 1, 2, 40], 16, 128, 64, False, max_rows=128)
    _attn_check(ck, rng, np.array([1, 1]), [10, 140], 16, 512, 128, True, max_rows=3 * 128)


@pytest.mark.parametrize("mult", [1e-30, 1e-4, 30.0, 3e4])
def test_fp4_attention_sizes_of_scores(ck, mult):
    """Queries from vanishing to huge (all weight on one row; scores in the thousands)."""
    rng = np.random.default_rng(5)
    D, H, ps = 256, 20, 32
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 2]), np.array([300, 299, 300]), H, D, ps)
    q = (q.float() * mult).bfloat16()
    out, lse = ck.ckv_fp4_attention(q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32([300, 299, 300]), 300, 1.0)
    want, wlse, _ = ref.attention(q.float().numpy(), cache, table, start, [300, 299, 300], 1.0, 1.0)
    # fp32 products and sums: z is off by at most 2^-24 sqrt(D) |q||k| (a random walk of D roundings, 4 deviations)
    dz = 2.0 ** -24 * 4 * np.sqrt(D) * np.linalg.norm(q.float().numpy(), axis=-1) * 6 * np.sqrt(D) / 4
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= dz + 2.0 ** -18 * (1 + np.abs(wlse)))
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + np.minimum(1, 2 * dz))[..., None] * 6
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


def test_fp4_attention_rising_scores(ck):
    """Every row scores higher than all before it, by far: the running maximum moves in every tile."""
    D, H, ps, L = 128, 16, 64, 1000
    rng = np.random.default_rng(9)
    x = rng.standard_normal((L, D)) * 0.02
    x[:, 0] = np.linspace(0.1, 4, L) ** 2  # 0.01 .. 16
    cache = torch.zeros(-(-L // ps), ps, 72, dtype=torch.uint8, device="cuda")
    ck.ckv_fp4_store(torch.tensor(x, dtype=torch.float32).cuda(), cache, torch.arange(L, device="cuda"), cache_scale=2.0 ** -6)
    q = torch.zeros(1, H, D)
    q[:, :, 0] = torch.linspace(-60, 60, H)
    q = q.bfloat16()
    table = np.arange(cache.shape[0])[None]
    out, lse = ck.ckv_fp4_attention(q.cuda(), cache, _i32(table), _i32([0, 1]), _i32([L]), L, 1.0, cache_scale=2.0 ** -6)
    want, wlse, _ = ref.attention(q.float().numpy(), cache.cpu().numpy(), table, [0, 1], [L], 1.0, 2.0 ** -6)
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= 2.0 ** -18 * (1 + np.abs(wlse)))
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * 18)


def test_fp4_attention_bad_entries(ck):
    """Page ids out of range hide their rows, rows past the bound are clamped; both are flagged."""
    rng = np.random.default_rng(2)
    D, H, ps = 128, 4, 16
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 1]), np.array([100, 100]), H, D, ps)
    table[0, 2] = cache.shape[0]
    table[1, 0] = -1
    err = _err()
    out, lse = ck.ckv_fp4_attention(q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32([100, 2 ** 31 - 1]), 100,
                                    0.1, err_word=err)
    assert int(err) == 0x4 | 0x10
    want, wlse, _ = ref.attention(q.float().numpy(), cache, table, start, [100, 100], 0.1, 1.0)
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= 2.0 ** -16 * (1 + np.abs(wlse)))
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * 6)
    # every page bad: as without rows
    out, lse = ck.ckv_fp4_attention(q.cuda(), torch.from_numpy(cache).cuda(), _i32(np.full_like(table, -1)), _i32(start),
                                    _i32([100, 100]), 100, 0.1, err_word=err)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_fp4_attention_keeps_to_its_row(ck):
    """A NaN query makes its own output NaN and no other; infinite sinks take all or nothing."""
    rng = np.random.default_rng(4)
    D, H, ps = 256, 6, 16
    ctx = np.array([50, 200, 200, 200])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 3]), ctx, H, D, ps)
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), 200, 0.06)
    o0, l0 = ck.ckv_fp4_attention(q.cuda(), *args)
    qn = q.clone()
    qn[1, 2, 7] = float("nan")
    o1, l1 = ck.ckv_fp4_attention(qn.cuda(), *args)
    assert bool(torch.isnan(o1[1, 2]).all()) and bool(torch.isnan(l1[1, 2]))
    o1[1, 2], l1[1, 2] = o0[1, 2], l0[1, 2]
    assert torch.equal(o0, o1) and torch.equal(l0, l1)
    sink = torch.full((H,), float("-inf"), device="cuda")
    o2, l2 = ck.ckv_fp4_attention(q.cuda(), *args, sink=sink)
    assert torch.equal(o0, o2) and torch.equal(l0, l2)


def test_fp4_attention_same_bits_every_time_and_in_a_graph(ck):
    rng = np.random.default_rng(6)
    D, H, ps = 512, 64, 64
    ctx = np.array([3000, 10, 2900])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 1, 1]), ctx, H, D, ps)
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), 3000, D ** -0.5)
    qd = q.cuda()
    o, l = ck.ckv_fp4_attention(qd, *args)
    for _ in range(3):
        o1, l1 = ck.ckv_fp4_attention(qd, *args)
        assert torch.equal(o, o1) and torch.equal(l, l1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = ck.ckv_fp4_attention(qd, *args, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2)
    go, gl = torch.zeros_like(o), torch.zeros_like(l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ckv_fp4_attention(qd, *args, out=go, lse=gl, use_pdl=True)
        ck.ckv_fp4_attention(qd, *args, out=go, lse=gl, use_pdl=True)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, go) and torch.equal(l, gl)


def test_fp4_attention_page_past_32_bit_offsets(ck):
    """A cache of more than 2^32 bytes with the rows at its end."""
    D, H, ps = 512, 8, 64
    page = ps * 288
    pages = (2 ** 32) // page + 40
    cache = torch.empty(pages, ps, 288, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(8)
    start, T, table, small, q, width = _attn_inputs(rng, np.array([1, 1]), np.array([500, 130]), H, D, ps)
    cache[-small.shape[0]:] = torch.from_numpy(small).cuda()
    high = np.where(table >= 0, table + pages - small.shape[0], -1)
    err = _err()
    o, l = ck.ckv_fp4_attention(q.cuda(), cache, _i32(high), _i32(start), _i32([500, 130]), 500, D ** -0.5, err_word=err)
    o1, l1 = ck.ckv_fp4_attention(q.cuda(), torch.from_numpy(small).cuda(), _i32(table), _i32(start), _i32([500, 130]), 500, D ** -0.5)
    assert int(err) == 0 and torch.equal(o, o1) and torch.equal(l, l1)
    x = torch.randn(3, D, device="cuda")
    loc = torch.tensor([pages * ps - 1, pages * ps - 64, (2 ** 32) // 288 + 5], device="cuda")
    ck.ckv_fp4_store(x, cache, loc, cache_scale=2.0 ** -6, err_word=err)
    back = torch.zeros(3, D, device="cuda")
    ck.ckv_fp4_load(cache, loc, back, cache_scale=2.0 ** -6, err_word=err)
    codes, scales = ref.fp4_rows(x.double().cpu().numpy(), 2.0 ** -6)
    vals = ref.E2M1[codes] * np.repeat(ref.E4M3[scales] * 2.0 ** -6, 16, axis=1)
    np.testing.assert_array_equal(back.double().cpu().numpy(), vals)
    assert int(err) == 0


# ------------------------------------------------------------------ together
def test_a_serving_step(ck):
    """Decode steps as a server runs them: maps -> c128 decode -> norm + rotation of the
    queries and of the rows that closed -> 4-bit store -> attention, over a growing cache."""
    B, H, D, P, ps = 6, 16, 512, 128, 2
    g, cs = torch.Generator().manual_seed(1), 2.0 ** -6
    seq = torch.tensor([128, 127, 1, 300, 256, 511], dtype=torch.int32)
    width = 4
    pages = B * width
    table = torch.full((B, width), -1, dtype=torch.int32)
    free = torch.randperm(pages, generator=g).to(torch.int32)
    cache = torch.zeros(pages, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    used = 0
    for b in range(B):  # pages and rows that the requests hold already
        rows = (int(seq[b]) - 1) // P
        for pg in range(-(-rows // ps)):
            table[b, pg] = free[used]
            used += 1
        old = torch.randn(rows, D, generator=g).bfloat16().cuda()
        at = torch.tensor([int(table[b, r // ps]) * ps + r % ps for r in range(rows)], dtype=torch.int64).cuda()
        ck.ckv_fp4_store(old, cache, at, cache_scale=cs)
    rope = _rope_table(600, 64, g)
    state = torch.rand(B, 3, D, generator=g).cuda() + 0.5
    ape = torch.randn(128, D, generator=g).cuda() * 0.1
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    ones, idx = _i32(np.ones(B)), _i32(np.arange(B))
    seq_d, table_d, free_d, cursor = seq.cuda(), table.cuda(), free.cuda(), _i32([used, 0])
    err = _err()
    for step in range(3):
        kv = torch.randn(B, 2 * D, generator=g)
        q = torch.randn(B, H, D, generator=g).bfloat16()
        m = ck.ckv_build_step_maps(seq_d, ones, table_d, free_d, cursor, P, ps, B, err_word=err)
        rows = torch.zeros(B, D, device="cuda")
        before = state.clone()
        ck.ckv_c128_online_decode(state, kv.cuda(), rows, ape, idx, seq_d, use_pdl=True, err_word=err)
        qn, kn = ck.ckv_qk_norm_rope(q.cuda(), m["positions"], rope.cuda(), k=rows.view(B, 1, D), k_positions=m["row_positions"],
                                     k_weight=w, q_weight=None, interleaved=True, use_pdl=True, err_word=err)
        ck.ckv_fp4_store(kn.view(B, D), cache, m["cache_loc"], cache_scale=cs, use_pdl=True, err_word=err)
        out, lse = ck.ckv_fp4_attention(qn, cache, table_d, m["row_start"], m["ctx_rows"], width * ps, D ** -0.5, cache_scale=cs,
                                        use_pdl=True, err_word=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        del before
        # the closed rows went through norm, rotation and storage to where the table says
        for b in range(B):
            s = int(seq[b]) + step
            if s % P:
                continue
            want = ref.norm_rope(rows[b:b + 1, None].cpu().numpy(), [s - P], rope.numpy(), w.cpu().numpy(), 64, D - 64, True, 1e-6)
            _norm_close(kn[b:b + 1], want, torch.bfloat16)
            r = s // P - 1
            at = int(table_d[b, r // ps]) * ps + r % ps
            assert int(m["cache_loc"][b]) == at
            codes, scales = ref.fp4_rows(kn[b].double().cpu().numpy(), cs)
            got = ref.fp4_row_values(cache.cpu().numpy(), at, D, cs)
            np.testing.assert_array_equal(got, (ref.E2M1[codes] * np.repeat(ref.E4M3[scales] * cs, 16, axis=1))[0])
        ctx = [(int(seq[b]) + step) // P for b in range(B)]
        want, wlse, _ = ref.attention(qn.float().cpu().numpy(), cache.cpu().numpy(), table_d.cpu().numpy(), list(range(B + 1)), ctx,
                                      D ** -0.5, cs)
        top = float(np.abs(want).max())
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * max(top, 6))
        fin = np.isfinite(wlse)
        assert np.array_equal(fin, np.isfinite(lse.cpu().numpy()))
        assert np.all(np.abs(lse.double().cpu().numpy()[fin] - wlse[fin]) <= 2.0 ** -16 * (1 + np.abs(wlse[fin])))
        seq_d += 1


@pytest.mark.parametrize("D", [128, 256, 512])
@pytest.mark.parametrize("H,n", [(8, [1, 1]), (20, [1, 2]), (50, [1, 1]), (64, [3, 2])])
def test_fp4_attention_cold_memory_and_jumping_maxima(ck, D, H, n):
    """Scores in the thousands (a row's weight sits on one key, in any tile) with the cache out
    of L2, so that loads arrive late: warps with few rows or none run far ahead of the others."""
    rng = np.random.default_rng(5)
    ctx = np.concatenate([[600 - 3 * i for i in range(k)][::-1] for k in n])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array(n), ctx, H, D, 32)
    q = (q.float() * 30).bfloat16()
    want, _, _ = ref.attention(q.float().numpy(), cache, table, start, ctx, 1.0, 1.0)
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), 600, 1.0)
    qc, flush = q.cuda(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        flush.fill_(i)
        if i % 2:
            torch.cuda.synchronize()
        out, lse = ck.ckv_fp4_attention(qc, *args)
        if first is None:
            first = (out, lse)
            # z is off by 2^-24 sqrt(D) |q| |k| at most a few times (a walk of D roundings): weights by 2^-5 of it or less
            dz = 2.0 ** -24 * 4 * np.sqrt(D) * np.linalg.norm(q.float().numpy(), axis=-1) * 6 * np.sqrt(D) / 4
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + np.minimum(1, 2 * dz))[..., None] * 6
            assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
