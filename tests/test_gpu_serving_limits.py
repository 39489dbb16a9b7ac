"""Calls of the serving-step operators at the ends of what their contracts allow, and
chains with calls that were there before them.

The tolerance of each test stands at it; a bf16 output's rounding is half a step at
most, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from test_gpu_serving_calls import _attn_ref64
from test_gpu_serving_ops import _attn_inputs, _err, _i32, _rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck():
    import compressed_kv_attention_gated_gb300 as ck

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.load()
    return ck


def _page(rows, D):
    """A cache of one page that holds the given rows (exactly: multiples of code values, scale 1)."""
    codes, scales = ref.fp4_rows(np.asarray(rows, np.float64), 1.0)
    assert np.array_equal(ref.E2M1[codes] * np.repeat(ref.E4M3[scales], 16, axis=1), rows)
    return torch.from_numpy(ref.pack_page(codes, scales).reshape(1, len(rows), D // 2 + D // 16)).cuda()


# ------------------------------------------------------------ prefill, then the step's calls
@pytest.mark.parametrize("variant", [1, 2])
@pytest.mark.parametrize("early_out", ["no_segment", "sentinels", "refused"])
def test_prefill_write_pass_without_work_orders_what_follows(ck, variant, early_out):
    """Prompts of whole chunks leave nothing to the prefill's write pass.  What follows it as a
    programmatic dependent must still see every row that the compress pass wrote."""
    B, D, n, P, ps = 32, 512, 1024, 128, 32
    T = B * n
    g = torch.Generator(device="cuda").manual_seed(0)
    inp = torch.randn(T, 2 * D, generator=g, device="cuda")
    ape = torch.randn(128, D, generator=g, device="cuda") * 0.1
    state = torch.rand(B, 3, D, generator=g, device="cuda") + 0.5
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    rope = _rope_table(n, 64, torch.Generator().manual_seed(1)).cuda()
    idx = torch.arange(B, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int64, device="cuda")
    # as a captured graph plans: entries past the segments, here all of the write pass's, are sentinels
    cp, wp, counts = ck.ckv_plan_online_prefill_device(lens, lens, T, pad_for_graph=True)
    assert bool((wp.view(torch.int32) == -1).all())
    if early_out == "no_segment":
        counts[1] = 0
    elif early_out == "refused":  # windows of no tokens, which the kernel flags and leaves
        wp.zero_()
    closing = torch.arange(T, dtype=torch.int32, device="cuda")
    rpos = torch.where(closing % P == P - 1, closing % n - (P - 1), torch.full_like(closing, -1))
    loc = torch.where(rpos >= 0, closing.long() // P, torch.full((T,), -1, device="cuda"))

    def chain(rows, kn, back, pdl):
        cache = torch.zeros(T // P // ps, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        ck.ckv_c128_online_prefill_counted(state, inp, rows, ape, idx, cp, wp, counts, use_pdl=pdl)
        ck.ckv_qk_norm_rope(rows.view(T, 1, D), rpos, rope, q_weight=w, q_out=kn, interleaved=True, use_pdl=pdl)
        ck.ckv_fp4_store(kn.view(T, D), cache, loc, use_pdl=pdl)
        ck.ckv_fp4_load(cache, loc, back, use_pdl=pdl)
        torch.cuda.synchronize()
        return cache

    def buffers():
        return (torch.full((T, D), 3.0, device="cuda"), torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"))

    prev = ck.ckv_c128_prefill_set_variant(variant)
    try:
        want = buffers()
        cache = chain(*want, False)
        assert bool((want[0][rpos >= 0] != 3).any(1).all())
        flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        got = buffers()
        for i in range(8):
            got[0].fill_(3.0), got[1].zero_(), got[2].zero_(), flush.fill_(i)
            c = chain(*got, True)
            for a, b in zip(want, got):
                assert torch.equal(a, b)
            assert torch.equal(cache, c)
    finally:
        ck.ckv_c128_prefill_set_variant(prev)


# ------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("D", [128, 512])
def test_norm_rope_outputs_with_gaps(ck, D):
    """Every other head of an odd number, every other token under heads that lie apart: rows that do
    not overlap, as outputs and in place; rows that do are refused."""
    T, g = 5, torch.Generator(device="cuda").manual_seed(0)
    rope, pos = _rope_table(9, 64, torch.Generator().manual_seed(1)).cuda(), _i32([0, 3, 8, 1, 7])
    heads = lambda: torch.zeros(T, 5, D, dtype=torch.bfloat16, device="cuda")[:, ::2]  # noqa: E731
    tokens = lambda: torch.zeros(3, 2 * T - 1, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[::2]  # noqa: E731
    flat = torch.zeros(64 * D, dtype=torch.bfloat16, device="cuda")
    for make in (heads, tokens):
        x = make().copy_(torch.randn(T, 3, D, generator=g, device="cuda"))
        want, _ = ck.ckv_qk_norm_rope(x.contiguous(), pos, rope)
        out, _ = ck.ckv_qk_norm_rope(x, pos, rope, q_out=make())
        assert torch.equal(out, want)
        base = x._base
        rest = base.clone()
        ck.ckv_qk_norm_rope(x, pos, rope, q_out=x)
        assert torch.equal(x, want)
        x.zero_()
        mask = torch.ones_like(base)
        mask.as_strided(x.shape, x.stride()).zero_()
        assert torch.equal(base, rest * mask)  # nothing beside the rows
    x = torch.zeros(T, 3, D, dtype=torch.bfloat16, device="cuda")
    for st, sh in ((2 * D, D), (D, D), (D, 2 * D), (4 * D, 2 * D), (0, D), (3 * D, D - 8), (D, 4 * D)):
        with pytest.raises(ValueError):
            ck.ckv_qk_norm_rope(x, pos, rope, q_out=flat.as_strided((T, 3, D), (st, sh, 1)))
    for st, sh in ((3 * D, D), (5 * D, 2 * D), (D, 5 * D), (2 * D, 9 * D)):
        ck.ckv_qk_norm_rope(x, pos, rope, q_out=flat.as_strided((T, 3, D), (st, sh, 1)))
    torch.cuda.synchronize()


# ------------------------------------------------------------ block tables
@pytest.mark.parametrize("D,H", [(128, 5), (128, 40), (256, 8), (512, 48), (512, 80)])
def test_fp4_attention_one_table_row_for_all_requests(ck, D, H):
    """A page list that all requests share, expanded over them: as if each had a copy."""
    rng = np.random.default_rng(0)
    n, ps = np.array([1, 3, 1, 2]), 16
    ctx = np.array([700, 5, 300, 301, 0, 699, 700])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([7]), ctx, H, D, ps)
    start = np.concatenate([[0], np.cumsum(n)])
    row, copies = _i32(table), _i32(np.repeat(table, 4, axis=0))
    c, qd, cx, st = torch.from_numpy(cache).cuda(), q.cuda(), _i32(ctx), _i32(start)
    err = _err()
    o, l = ck.ckv_fp4_attention(qd, c, copies, st, cx, 700, D ** -0.5, err_word=err)
    want, wlse, _ = ref.attention(q.float().numpy(), cache, np.repeat(table, 4, axis=0), start, ctx, D ** -0.5, 1.0)
    assert np.all(np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * 6)
    assert int(err) == 0
    for shared in (row.expand(4, width), row[0].expand(4, width), copies[:1].expand(4, width)):
        assert shared.stride(0) == 0
        o1, l1 = ck.ckv_fp4_attention(qd, c, shared, st, cx, 700, D ** -0.5, err_word=err)
        assert int(err) == 0 and torch.equal(o, o1) and torch.equal(l, l1)


def test_fp4_attention_and_maps_refuse_overlapping_table_rows(ck):
    """Rows that begin inside one another, and (where pages are written) rows that are the same."""
    q = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(4, 16, 72, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(64, dtype=torch.int32, device="cuda")
    st, cx = _i32([0, 1, 2, 3]), _i32([1, 1, 1])
    for step in (1, 7):
        with pytest.raises(ValueError):
            ck.ckv_fp4_attention(q, cache, wide.as_strided((3, 8), (step, 1)), st, cx, 128, 1.0)
    for step in (0, 1, 7):
        with pytest.raises(ValueError):
            ck.ckv_build_step_maps(cx, cx, wide.as_strided((3, 8), (step, 1)), wide, _i32([0, 0]), 4, 4, 3)
    # one request: the step to a next row does not exist; rows apart: any step
    one = [ck.ckv_fp4_attention(q[:1], cache, wide.as_strided((1, 8), (step, 1)), st[:2], cx[:1], 128, 1.0)[0] for step in (0, 1, 50)]
    assert all(bool((o == 0).all()) for o in one)
    ck.ckv_fp4_attention(q, cache, wide.as_strided((3, 8), (8, 1)), st, cx, 128, 1.0)
    ck.ckv_fp4_attention(q, cache, wide.as_strided((3, 8), (20, 1)), st, cx, 128, 1.0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("max_rows", [0, -1, 65, 2 ** 31, 2 ** 40, 160 * 2 ** 32, 2 ** 63 - 1])
def test_fp4_attention_refuses_bounds_of_its_rows(ck, max_rows):
    """max_rows past the table's pages or past 32 bits: a refusal, before any workspace is asked for."""
    for B, H in ((1, 4), (19, 16)):
        q = torch.zeros(B, H, 128, dtype=torch.bfloat16, device="cuda")
        cache = torch.zeros(4, 16, 72, dtype=torch.uint8, device="cuda")
        args = (q, cache, torch.zeros(B, 4, dtype=torch.int32, device="cuda"), _i32(np.arange(B + 1)), _i32(np.ones(B)))
        for stream in (None, torch.cuda.Stream()):
            with pytest.raises(ck.CkvError):
                ck.ckv_fp4_attention(*args, max_rows, 1.0, stream=stream)


# ------------------------------------------------------------ step maps
@pytest.mark.parametrize("T,lens", [(2 ** 31 - 1, [2 ** 31 - 1]), (2 ** 31 - 1, [5, 2 ** 30, 7]), (2 ** 31 - 152 * 1024, [3])])
def test_step_maps_of_the_most_tokens(ck, T, lens):
    """Maps of up to 2^31 - 1 tokens: each place is written once, and nothing before or behind them."""
    guard = 1 << 20
    raw = torch.full((T + 2 * guard,), -9, dtype=torch.int32, device="cuda")
    pos = raw[guard:guard + T]
    B, err = len(lens), _err()
    width = -(-max(lens) // 1024)
    ps = 1 << 16
    tab = torch.full((B, -(-width // ps)), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(100, 100 + tab.numel(), dtype=torch.int32, device="cuda")
    ck.ckv_build_step_maps(_i32(lens), _i32(lens), tab, free, _i32([0, 0]), 1024, ps, T, out={"positions": pos}, err_word=err)
    assert int(err) == 0
    assert bool((raw[:guard] == -9).all()) and bool((raw[guard + T:] == -9).all())
    at, piece = 0, 1 << 27
    for n in [*lens, None]:  # the last stretch: places without a token
        end = T if n is None else at + n
        for i in range(at, end, piece):
            j = min(i + piece, end)
            want = torch.arange(i - at, j - at, dtype=torch.int32, device="cuda") if n is not None else -1
            assert bool((pos[i:j] == want).all())
        at = end
    need = [-(-(n // 1024) // ps) for n in lens]
    assert (tab >= 0).sum(1).tolist() == need


def test_step_maps_pages_of_dropped_tokens_are_entered(ck):
    """More tokens than the maps have room for: the pages that the requests take stand in their
    block tables all the same, so that none is lost."""
    rng = np.random.default_rng(0)
    for P, ps, B in ((2, 2, 5), (4, 1, 40), (1, 3, 1500)):
        n = rng.integers(0, 30, B)
        s = n + rng.integers(0, 20, B)
        width = -(-(int(s.max()) // P) // ps)
        table = np.full((B, width), -1)
        for b in range(B):
            table[b, :-(-((s[b] - n[b]) // P) // ps)] = 5
        free = 100 + rng.permutation(B * width)
        live = int(n.sum())
        want, wtable, wcur = ref.step_maps(s, n, table, free, 0, P, ps, live)
        for T in (live - 1, live // 2, 1, 0):
            tab, cur, err = _i32(table), _i32([0, 0]), _err()
            got = ck.ckv_build_step_maps(_i32(s), _i32(n), tab, _i32(free), cur, P, ps, T, err_word=err)
            assert int(err) == 0x8 and cur.tolist() == [wcur, 0]
            for k in want:
                w = np.minimum(want[k], T) if k == "row_start" else want[k][:T]
                np.testing.assert_array_equal(got[k].cpu().numpy(), w, err_msg=k)
            np.testing.assert_array_equal(tab.cpu().numpy(), wtable)


@pytest.mark.parametrize("T", [0, 1000, (1 << 21) + 7])
def test_step_maps_pages_of_dropped_tokens_of_a_long_prompt(ck, T):
    """A prompt of more tokens than the narrow sums hold, dropped in part, with a request behind it;
    and a free list that ends inside it."""
    P, ps = 16, 1024
    n, s = np.array([3, (1 << 21) + 5, 40000]), np.array([3, (1 << 21) + 9, 50000])
    held = -(-((s - n) // P) // ps)
    need = -(-(s // P) // ps)
    for num_free in (200, 100):
        free = 1000 + np.random.default_rng(0).permutation(num_free)
        want, at = np.full((3, 130), -1), 0
        for b in range(3):
            want[b, :held[b]] = 7
        table = want.copy()
        for b in range(3):
            for pg in range(held[b], need[b]):
                if at < num_free:
                    want[b, pg] = free[at]
                at += 1
        tab, cur, err = _i32(table), _i32([0, 0]), _err()
        ck.ckv_build_step_maps(_i32(s), _i32(n), tab, _i32(free), cur, P, ps, T, err_word=err)
        assert int(err) == 0x8 | (0x80 if at > num_free else 0)
        assert cur.tolist() == [min(at, num_free), 0]
        np.testing.assert_array_equal(tab.cpu().numpy(), want)


# ------------------------------------------------------------ long rows
@pytest.mark.parametrize("D,H", [(128, 4), (128, 24), (128, 40), (256, 8), (512, 48), (512, 80)])
def test_fp4_attention_one_large_weight_over_a_long_tail(ck, D, H):
    """131,072 rows whose weights are 2^-25.1 of the first one's: together 0.36% of the sum.

    Weights are rounded by 2^-11 of their value, or by 2^-32 of the largest one's: with values up to
    6 the output is off by 6 (L 2^-32 + 2^-11) at most, and its rounding."""
    L, B = 131072, 152
    assert ck.ckv_fp4_attention_workspace(B, B, H, D, L) == 0  # not split: a range of its own would have a maximum of its own
    x = np.zeros((L, D))
    x[0, 0], x[1:, 1], x[:, 16] = 6, 6, 1.5
    cache = _page(x, D)
    z0 = 25.1 * np.log(2)
    q = torch.zeros(B, H, D)
    q[:, :, 0] = 2.875
    q = q.bfloat16()
    scale = z0 / (2.875 * 6)
    out, lse = ck.ckv_fp4_attention(q.cuda(), cache, torch.zeros(B, 1, dtype=torch.int32, device="cuda"), _i32(np.arange(B + 1)),
                                    _i32(np.full(B, L)), L, scale)
    z = np.zeros(L)
    z[0] = np.float64(np.float32(scale)) * 2.875 * 6
    p = np.exp(z - z[0])
    want = p @ x / p.sum()
    assert 0.02 < want[1] < 0.03
    tol = 2.0 ** -8 * np.abs(want) + 6 * (L * 2.0 ** -32 + 2.0 ** -11)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - (z[0] + np.log(p.sum()))) <= 2.0 ** -16 * z[0])


@pytest.mark.parametrize("D,H", [(128, 4), (128, 40), (256, 24), (512, 48), (512, 80)])
def test_fp4_attention_sums_of_long_rows(ck, D, H):
    """2^21 rows (one page again and again) for as many requests as there are SMs.  Two channels of the
    cache are constant, so the output is that constant whatever the weights.

    The accumulator cuts sums off, by 2^-9 of a value at most over the 2^17 rows of a range; weights
    are rounded to 2^-11 and the output to 2^-8: 2^-8 + 2^-9 + 2^-11 of the constants."""
    L, B, ps = 1 << 21, 152, 1 << 16
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(ps, D, generator=g, device="cuda").clamp(-5, 5)
    x[:, 0], x[:, D - 1], x[:, D - 16] = 6, -1.5, 6
    cache = torch.zeros(1, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    ck.ckv_fp4_store(x, cache, torch.arange(ps, device="cuda"))
    k = torch.empty(ps, D, device="cuda")
    ck.ckv_fp4_load(cache, torch.arange(ps, device="cuda"), k)
    assert bool((k[:, 0] == 6).all()) and bool((k[:, D - 1] == -1.5).all())
    q = torch.randn(1, H, D, generator=g, device="cuda").bfloat16()
    table = torch.zeros(1, L // ps, dtype=torch.int32, device="cuda").expand(B, -1)
    out, lse = ck.ckv_fp4_attention(q.expand(B, H, D), cache, table, _i32(np.arange(B + 1)), _i32(np.full(B, L)), L, D ** -0.5)
    tol = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11
    assert bool(((out[..., 0].double() - 6).abs() <= 6 * tol).all())
    assert bool(((out[..., D - 1].double() + 1.5).abs() <= 1.5 * tol).all())
    want = torch.logsumexp(q[0].double() @ k.double().T * D ** -0.5, -1) + np.log(L // ps)
    assert bool(((lse.double() - want).abs() <= 2.0 ** -16 * (10 + want.abs())).all())
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))


@pytest.mark.parametrize("D,H", [(128, 1), (128, 64), (512, 8), (512, 128)])
def test_fp4_attention_of_the_longest_rows(ck, D, H):
    """One request over 160 x 2^17 rows, the most that a call takes (one page again and again).
    Every row is the same, so every weight and sum is a power of two times the number of rows."""
    ps, L = 1 << 16, 160 * 2 ** 17
    row = np.tile([1.0, -2, 0.5, 6, 0, 3, -1.5, 4] * 2, D // 16)
    cache = _page(np.tile(row, (ps, 1)), D)
    table = torch.zeros(1, L // ps, dtype=torch.int32, device="cuda")
    q = torch.full((1, H, D), 0.25).bfloat16().cuda()
    out = torch.full((1, H, D), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, H), -7.0, device="cuda")
    err = _err()
    ck.ckv_fp4_attention(q, cache, table, _i32([0, 1]), _i32([L]), L, 1.0 / D, out=out, lse=lse, err_word=err)
    assert int(err) == 0
    assert bool((out.double() == torch.from_numpy(row).cuda()).all())
    want = float(row.sum()) * 0.25 / D + np.log(L)
    assert bool(((lse.double() - want).abs() <= 2.0 ** -16 * want).all())


@pytest.mark.parametrize("D,H,B", [(128, 5, 300), (128, 64, 160), (256, 24, 160), (512, 48, 160), (512, 80, 80)])
def test_fp4_attention_ranges_of_ragged_requests(ck, D, H, B):
    """Bounds past 2^17 rows split every request: those that see few rows, one more or less than a range,
    none, or are padding among those that see most."""
    ps, most = 4096, 140000
    rng = np.random.default_rng(D + H)
    half = -(-(-(-most // 128)) // 2) * 128  # two ranges
    ctx = rng.choice([0, 1, 100, half - 1, half, half + 1, 2 ** 17, most, -1], B)
    ctx[:8] = [most, half, half + 1, 0, -1, half - 1, 2 ** 17 + 1, 5]
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = torch.zeros(5, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    ck.ckv_fp4_store(torch.randn(5 * ps, D, generator=g, device="cuda"), cache, torch.arange(5 * ps, device="cuda"), cache_scale=2.0 ** -6)
    table = _i32(rng.integers(0, 5, (B, -(-most // ps))))
    q = (torch.randn(B, H, D, generator=g, device="cuda") * 2).bfloat16()
    sink = torch.randn(H, generator=g, device="cuda") + 10
    out = torch.full((B, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), 9.0, device="cuda")
    err = _err()
    ck.ckv_fp4_attention(q, cache, table, _i32(np.arange(B + 1)), _i32(ctx), most, D ** -0.5, cache_scale=2.0 ** -6, sink=sink, out=out,
                         lse=lse, err_word=err)
    assert int(err) == 0
    off = torch.from_numpy(ctx < 0).cuda()
    assert bool((out[off] == 9).all()) and bool((lse[off] == 9).all())
    for b in [*range(8), *rng.integers(8, B, 4)]:
        if ctx[b] < 0:
            continue
        want, wlse = _attn_ref64(q[b:b + 1, :6], cache, table[b:b + 1], [0, 1], torch.tensor([int(ctx[b])], device="cuda"), D ** -0.5,
                                 2.0 ** -6, sink[:6])
        assert bool(((out[b:b + 1, :6].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * 6).all())
        assert bool(((lse[b:b + 1, :6].double() - wlse).abs() <= 2.0 ** -16 * (10 + wlse.abs())).all())


# ------------------------------------------------------------ many heads, many requests
@pytest.mark.parametrize("D", [128, 256, 512])
def test_fp4_attention_of_1024_heads(ck, D):
    rng = np.random.default_rng(D)
    ctx = np.array([130, 0, 129, 7])
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1, 0, 3]), ctx, 1024, D, 16)
    c, tab = torch.from_numpy(cache).cuda(), _i32(table)
    out, lse = ck.ckv_fp4_attention(q.cuda(), c, tab, _i32(start), _i32(ctx), 130, D ** -0.5)
    want, wlse = _attn_ref64(q.cuda(), c, tab, start, _i32(ctx), D ** -0.5, 1.0)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * 6).all())
    fin = torch.isfinite(wlse)
    assert torch.equal(fin, torch.isfinite(lse)) and bool(((lse.double() - wlse)[fin].abs() <= 2.0 ** -16 * (10 + wlse[fin].abs())).all())


@pytest.mark.parametrize("D,H", [(128, 1), (128, 33), (512, 3)])
def test_fp4_attention_of_65536_requests(ck, D, H):
    """The most requests that a call takes: a token each, or a token for one in a thousand; each sees one
    row, whose values come out."""
    B, ps = 65536, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = torch.zeros(B // ps, ps, D // 2 + D // 16, dtype=torch.uint8, device="cuda")
    ck.ckv_fp4_store(torch.randn(B, D, generator=g, device="cuda"), cache, torch.arange(B, device="cuda"), cache_scale=2.0 ** -6)
    rows = torch.empty(B, D, dtype=torch.bfloat16, device="cuda")
    ck.ckv_fp4_load(cache, torch.arange(B, device="cuda"), rows, cache_scale=2.0 ** -6)
    table = torch.randint(0, B // ps, (B, 1), generator=g, dtype=torch.int32, device="cuda")
    for every in (1, 1000):
        n = (torch.arange(B) % every == every // 2).int()
        start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(n, 0).int()]).cuda()
        T = int(n.sum())
        q = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
        out, _ = ck.ckv_fp4_attention(q, cache, table, start, torch.ones(T, dtype=torch.int32, device="cuda"), 1, D ** -0.5,
                                      cache_scale=2.0 ** -6)
        want = rows[table[n.bool().cuda(), 0].long() * ps]
        assert torch.equal(out, want[:, None].expand(T, H, D))
    with pytest.raises(ck.CkvError):
        ck.ckv_fp4_attention(q[:1], cache, torch.zeros(B + 1, 1, dtype=torch.int32, device="cuda"),
                             torch.ones(B + 2, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"), 1, 1.0)


# ------------------------------------------------------------ streams
def test_outputs_and_workspaces_belong_to_the_stream_of_the_call(ck, monkeypatch):
    """What a call makes for itself on a given stream (a torch stream or its handle; the default
    stream's is 0) is allocated for that stream: another stream's pool would hand it out too early."""
    rng = np.random.default_rng(0)
    start, T, table, cache, q, width = _attn_inputs(rng, np.array([1]), np.array([9000]), 16, 128, 64)
    args = (q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32([9000]), 9000, 0.1)
    assert ck.ckv_fp4_attention_workspace(1, 1, 16, 128, 9000) > 0
    want = ck.ckv_fp4_attention(*args)
    side, made, empty = torch.cuda.Stream(), [], torch.empty

    def record(*a, **k):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **k)

    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", record)
    for current in (torch.cuda.default_stream(), side):
        for stream in (0, torch.cuda.default_stream(), side, side.cuda_stream):
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            with torch.cuda.stream(current):
                made.clear()
                got = ck.ckv_fp4_attention(*args, stream=stream)
                ck.ckv_qk_norm_rope(args[0], args[4], k=args[0], k_positions=args[4], stream=stream)
                ck.ckv_build_step_maps(_i32([5]), _i32([1]), _i32([[-1]]), _i32([3]), _i32([0, 0]), 4, 4, 1, stream=stream)
                assert torch.cuda.current_stream() == current
            torch.cuda.synchronize()
            assert len(made) == 3 + 2 + 7 and set(made) == {handle}
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
