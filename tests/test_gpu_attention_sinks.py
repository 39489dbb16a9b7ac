"""Sinks at the ends of their type, in the attention over the uncompressed cache and in the one over 4-bit rows.

A sink takes part in the sum alone: one of -infinity, or so low that its weight is 0 against every score, leaves
all as it is without one, bit for bit.  Where nothing is seen lse is the sink itself (tolerance 2^-22 of it: it goes
through units of log2 and back, four roundings of 2^-24)."""
import numpy as np
import pytest
import torch

from test_gpu_kv_ops import Step, ck  # noqa: F401
from test_gpu_serving_ops import _attn_inputs, _err, _i32

pytestmark = pytest.mark.gpu

# D, H, KH, tokens of two requests: keys on the M side, rows on the M side
FORMS = [(128, 8, 1, [1, 2]), (128, 32, 1, [20, 3]), (256, 8, 1, [1, 2]), (256, 32, 1, [20, 3]), (512, 64, 1, [2, 1])]
LOWEST = torch.finfo(torch.float32).min


def _step(D, H, KH, n, before):
    """The first and the last token see nothing."""
    s = Step(D, H, KH, n, before, 16, sink=True, seed=D, width_more=1000)
    s.ctx = np.array(s.ctx)
    s.ctx[[0, -1]] = 0
    return s


@pytest.mark.parametrize("D,H,KH,n", FORMS)
def test_minus_infinity_over_ranges_of_keys(ck, D, H, KH, n):  # noqa: F811
    """A bound far above the contexts splits the keys; what is merged behind it counts alone where nothing was seen."""
    s = _step(D, H, KH, n, [300, 9])
    s.sink[::2] = -torch.inf
    assert ck.ckv_kv_attention_workspace(sum(n), 2, H, KH, D, 16000) > 0
    out, lse, err = s.run(ck, max_rows=16000)
    assert int(err) == 0
    s.check(out, lse)
    assert torch.equal(lse[0], s.sink) and torch.equal(lse[-1], s.sink)
    g = torch.Generator(device="cuda").manual_seed(0)
    far, far_lse = torch.randn(out.shape, generator=g, device="cuda").bfloat16(), torch.randn(lse.shape, generator=g, device="cuda")
    both, total = ck.ckv_merge_attention([out, far], [lse, far_lse])
    off = torch.isneginf(lse)
    assert int(off.sum()) == H and torch.equal(both[off], far[off]) and torch.equal(total[off], far_lse[off])


@pytest.mark.parametrize("D,H,KH,n", FORMS)
@pytest.mark.parametrize("before,rows", [([40, 9], None), ([300, 9], 16000)])
def test_the_lowest_values(ck, D, H, KH, n, before, rows):  # noqa: F811
    """In one range of keys and in several."""
    s = _step(D, H, KH, n, before)
    assert (ck.ckv_kv_attention_workspace(sum(n), 2, H, KH, D, rows or s.max_rows) > 0) == (rows is not None)
    s.sink[:] = torch.tensor([LOWEST, -torch.inf, -3e38, LOWEST, -1e30, 4.0, LOWEST, -2e38], device="cuda").repeat(H // 8)
    out, lse, err = s.run(ck, max_rows=rows)
    assert int(err) == 0
    s.check(out, lse)
    ends = s.sink <= -3e38
    assert torch.equal(lse[0][ends], s.sink[ends]) and torch.equal(lse[-1][ends], s.sink[ends])
    low = s.sink < 0
    s.sink = None
    plain = s.run(ck, max_rows=rows)
    assert torch.equal(plain[0][:, low], out[:, low]) and torch.equal(plain[1][1:-1, low], lse[1:-1, low])


@pytest.mark.parametrize("D,H,n,ctx", [(256, 6, [1, 3], [50, 0, 200, 200]), (128, 8, [1, 2], [3, 0, 9000]), (512, 64, [1, 2], [0, 3, 40]),
                                       (128, 32, [60, 20], [0, 100] * 40), (256, 32, [60], [2000] * 59 + [0])])
def test_the_lowest_value_over_4_bit_rows(ck, D, H, n, ctx):  # noqa: F811
    rng = np.random.default_rng(D + H)
    ctx = np.array(ctx)
    start, T, table, cache, q, width = _attn_inputs(rng, np.array(n), ctx, H, D, 16)
    args = (q.cuda(), torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(ctx), int(ctx.max()), 0.06)
    err = _err()
    o, l = ck.ckv_fp4_attention(*args, err_word=err)
    blind = torch.from_numpy(ctx == 0).cuda()
    for low in (LOWEST, -torch.inf):
        o1, l1 = ck.ckv_fp4_attention(*args, sink=torch.full((H,), low, device="cuda"), err_word=err)
        assert int(err) == 0 and torch.equal(o, o1) and torch.equal(l[~blind], l1[~blind]) and bool((l1[blind] == low).all())


@pytest.mark.parametrize("D,H,KH,n", FORMS)
@pytest.mark.parametrize("before,rows", [([40, 9], None), ([300, 9], 16000)])
def test_infinity_takes_all(ck, D, H, KH, n, before, rows):  # noqa: F811
    s = _step(D, H, KH, n, before)
    s.sink[::2] = torch.inf
    out, lse, err = s.run(ck, max_rows=rows)
    assert int(err) == 0 and torch.all(out[:, ::2] == 0) and torch.all(lse[:, ::2] == torch.inf)
    far, far_lse = torch.ones_like(out), torch.zeros_like(lse)
    both, total = ck.ckv_merge_attention([far, out], [far_lse, lse])
    assert torch.all(both[:, ::2] == 0) and torch.all(total[:, ::2] == torch.inf)
    near, alone = out[:, 1::2].contiguous(), lse[:, 1::2].contiguous()
    want = ck.ckv_merge_attention([far[:, 1::2].contiguous(), near], [far_lse[:, 1::2].contiguous(), alone])
    assert torch.equal(both[:, 1::2], want[0]) and torch.equal(total[:, 1::2], want[1])
