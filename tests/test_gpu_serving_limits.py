"""Calls of the serving-step operators at the ends of what their contracts allow, and
chains with calls that were there before them.

The tolerance of each test stands at it; a bf16 output's rounding is half a step at
most, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from test_gpu_serving_ops import _attn_inputs, _err, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck():
    import compressed_kv_attention_gated_gb300 as ck

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.load()
    return ck


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
