"""Refusals of the serving-step operators, on the CPU: every call here returns
during argument validation."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
ONE = P(16)   # non-null, aligned, never dereferenced
ODD = P(18)


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_attention_gated_gb300 import build, ckv

    build.build()
    return ckv.load()


def _call(fn, base, **change):
    args = {**base, **change}
    return fn(*args.values())


MAPS = dict(seq=ONE, n=ONE, B=4, P=16, ps=64, table=ONE, stride=8, pages=8, free=ONE, nfree=10, cur=ONE, cur_out=ONE, tails=ONE,
            T=4, start=ONE, pos=ONE, bid=ONE, slot=ONE, loc=ONE, tail=ONE, rpos=ONE, ctx=ONE, pdl=0, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 2), (dict(B=8193), 2), (dict(P=0), 2), (dict(P=1025), 2), (dict(ps=0), 2), (dict(pages=-1), 2), (dict(stride=7), 2),
    (dict(nfree=-1), 2), (dict(nfree=2 ** 31), 2), (dict(T=-1), 2), (dict(seq=None), 1), (dict(n=None), 1), (dict(table=None), 1),
    (dict(free=None), 1), (dict(cur=None), 1), (dict(cur_out=None), 1), (dict(tails=None), 1),
    *[({k: ODD}, 4) for k in ("seq", "n", "table", "free", "cur", "cur_out", "tails", "start", "pos", "bid", "slot", "tail", "rpos",
                              "ctx", "err")], (dict(loc=P(20)), 4)])
def test_step_maps_refusals(lib, change, status):
    assert _call(lib.ckv_build_step_maps, MAPS, **change) == status


def _rows(**change):
    from compressed_kv_attention_gated_gb300.ckv import NormRows

    f = dict(x=16, out=32, weight=None, positions=16, stride_t=512, stride_h=128, out_stride_t=512, out_stride_h=128, tokens=3, heads=4,
             dtype=1, out_dtype=1, reserved=0)
    f.update(change)
    return NormRows(*f.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 2), (dict(heads=-1), 2), (dict(reserved=1), 2), (dict(dtype=2), 3), (dict(out_dtype=-1), 3), (dict(tokens=2 ** 31), 2),
    (dict(x=None), 1), (dict(out=None), 1), (dict(positions=None), 1), (dict(stride_t=-8), 2), (dict(out_stride_h=-8), 2),
    (dict(x=24), 4), (dict(out=24), 4), (dict(weight=20), 4), (dict(positions=18), 4), (dict(stride_t=516), 4),
    (dict(stride_h=4), 4), (dict(out_stride_t=4), 4), (dict(dtype=0, stride_h=2), 4), (dict(out=16, out_dtype=0), 2),
    (dict(out=16, out_stride_t=1024), 2)])
def test_norm_rope_row_set_refusals(lib, change, status):
    ok = _rows(tokens=0)
    for q, k in ((_rows(**change), None), (ok, _rows(**change))):
        assert lib.ckv_qk_norm_rope(ctypes.byref(q), None if k is None else ctypes.byref(k), ONE, 10, 128, 64, 64, 0, 1e-6, 0, None,
                                    None) == status


@pytest.mark.parametrize("D,R,at,npos,eps,status", [
    (64, 64, 0, 10, 1e-6, 2), (128, 63, 0, 10, 1e-6, 2), (128, 130, 0, 10, 1e-6, 2), (128, 64, 65, 10, 1e-6, 2), (128, 64, 66, 10, 1e-6, 2),
    (128, 64, -2, 10, 1e-6, 2), (128, -2, 0, 10, 1e-6, 2), (128, 64, 64, -1, 1e-6, 2), (128, 64, 64, 10, -1.0, 2),
    (128, 64, 64, 10, float("nan"), 2)])
def test_norm_rope_refusals(lib, D, R, at, npos, eps, status):
    q = _rows()
    assert lib.ckv_qk_norm_rope(ctypes.byref(q), None, ONE, npos, D, R, at, 0, eps, 0, None, None) == status


def test_norm_rope_nulls_and_empty(lib):
    q, none = _rows(), _rows(tokens=0, x=None, out=None, positions=None)
    assert lib.ckv_qk_norm_rope(None, None, ONE, 10, 128, 64, 64, 0, 1e-6, 0, None, None) == 1
    assert lib.ckv_qk_norm_rope(ctypes.byref(q), None, None, 10, 128, 64, 64, 0, 1e-6, 0, None, None) == 1
    assert lib.ckv_qk_norm_rope(ctypes.byref(q), None, ODD, 10, 128, 64, 64, 0, 1e-6, 0, None, None) == 4
    assert lib.ckv_qk_norm_rope(ctypes.byref(q), None, ONE, 10, 128, 64, 64, 0, 1e-6, 0, ODD, None) == 4
    assert lib.ckv_qk_norm_rope(ctypes.byref(none), ctypes.byref(none), ONE, 10, 128, 64, 64, 0, 1e-6, 0, None, None) == 0


STORE = dict(rows=ONE, dtype=1, stride=128, n=4, D=128, cache=ONE, pages=4, ps=2, loc=ONE, g=1.0, pdl=0, err=None, stream=None)
ROW_REFUSALS = [
    (dict(n=-1), 2), (dict(D=64), 2), (dict(ps=0), 2), (dict(pages=-1), 2), (dict(stride=-128), 2), (dict(dtype=2), 3),
    (dict(n=2 ** 31), 2), (dict(g=0.0), 2), (dict(g=-1.0), 2), (dict(g=0.3), 2), (dict(g=3.0), 2), (dict(g=2.0 ** -65), 2),
    (dict(g=2.0 ** 65), 2), (dict(g=float("inf")), 2), (dict(g=float("nan")), 2), (dict(rows=None), 1), (dict(cache=None), 1),
    (dict(loc=None), 1), (dict(rows=P(24)), 4), (dict(cache=P(24)), 4), (dict(loc=P(20)), 4), (dict(err=ODD), 4), (dict(stride=132), 4),
    (dict(ps=3), 4), (dict(n=0, rows=None, cache=None, loc=None), 0)]


@pytest.mark.parametrize("change,status", ROW_REFUSALS)
def test_fp4_store_and_load_refusals(lib, change, status):
    assert _call(lib.ckv_fp4_store, STORE, **change) == status
    a = {**STORE, **change}
    assert lib.ckv_fp4_load(a["cache"], a["pages"], a["ps"], a["loc"], a["n"], a["D"], a["rows"], a["dtype"], a["stride"], a["g"], 0,
                            a["err"], None) == status


def test_fp4_load_refuses_overlapping_rows(lib):
    assert lib.ckv_fp4_load(ONE, 4, 2, ONE, 4, 128, ONE, 1, 120, 1.0, 0, None, None) == 2
    assert lib.ckv_fp4_load(ONE, 4, 2, ONE, 4, 128, ONE, 1, 0, 1.0, 0, None, None) == 2


ATTN = dict(q=ONE, st=1024, sh=128, T=4, H=8, D=128, cache=ONE, pages=10, ps=64, g=1.0, table=ONE, tstride=16, mp=16, start=ONE, B=4,
            ctx=ONE, rows=1024, scale=0.1, sink=None, out=ONE, lse=ONE, ws=None, wsb=0, pdl=0, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 2), (dict(B=-1), 2), (dict(B=65537), 2), (dict(H=0), 2), (dict(H=1025), 2), (dict(D=192), 2), (dict(pages=-1), 2),
    (dict(ps=0), 2), (dict(mp=-1), 2), (dict(tstride=15), 2), (dict(g=0.7), 2), (dict(scale=float("nan")), 2),
    (dict(scale=float("inf")), 2), (dict(rows=0), 2), (dict(rows=1025), 2), (dict(T=2 ** 29), 2), (dict(st=-8), 2), (dict(sh=-8), 2),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(start=None), 1), (dict(ctx=None), 1), (dict(out=None), 1),
    (dict(q=P(24)), 4), (dict(st=1020), 4), (dict(sh=4), 4), (dict(cache=P(24)), 4), (dict(table=ODD), 4), (dict(start=ODD), 4),
    (dict(ctx=ODD), 4), (dict(sink=ODD), 4), (dict(out=P(24)), 4), (dict(lse=ODD), 4), (dict(ws=P(24)), 4), (dict(err=ODD), 4),
    (dict(ps=65), 4), (dict(T=0, q=None, out=None), 0), (dict(B=0, table=None), 0)])
def test_fp4_attention_refusals(lib, change, status):
    assert _call(lib.ckv_fp4_attention, ATTN, **change) == status


def test_fp4_attention_limits(lib):
    # ranges of cache rows are counted in 32 bits, rounded up to 128 rows per range
    wide = dict(mp=2 ** 25, tstride=2 ** 25, ps=64, ws=ONE, wsb=2 ** 62, out=P(1 << 40))
    assert _call(lib.ckv_fp4_attention, ATTN, **wide, rows=2 ** 31 - 2 ** 14) == 2
    # an output over the queries: whole, by one element at either end
    span = ((ATTN["T"] - 1) * 1024 + 7 * 128 + 128) * 2
    for q, out in ((1 << 20, 1 << 20), (1 << 20, (1 << 20) + span - 16), ((1 << 20) + 4 * 8 * 128 * 2 - 16, 1 << 20)):
        assert _call(lib.ckv_fp4_attention, ATTN, ws=ONE, wsb=2 ** 62, q=P(q), out=P(out)) == 2


def test_fp4_attention_workspace_is_asked_for(lib):
    assert lib.ckv_fp4_attention_workspace(0, 4, 8, 128, 10) == 0
    assert lib.ckv_fp4_attention_workspace(1, 1, 8, 192, 10) == 0
    big = dict(T=1, B=1, H=64, D=512, rows=10 ** 6, mp=20000, tstride=20000)
    need = lib.ckv_fp4_attention_workspace(1, 1, 64, 512, 10 ** 6)
    if need:
        assert _call(lib.ckv_fp4_attention, ATTN, **big) == 1
        assert _call(lib.ckv_fp4_attention, ATTN, **big, ws=ONE, wsb=need - 1) == 2


def test_binding_refuses_cpu_tensors(lib):
    import compressed_kv_attention_gated_gb300 as ck

    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 128)
    with pytest.raises(ValueError):
        ck.ckv_build_step_maps(i, i, i.view(4, 1), i, i, 4, 4, 4)
    with pytest.raises(ValueError):
        ck.ckv_qk_norm_rope(f.view(4, 1, 128), i)
    with pytest.raises(ValueError):
        ck.ckv_fp4_store(f, torch.zeros(1, 4, 72, dtype=torch.uint8), i.long())
    with pytest.raises(ValueError):
        ck.ckv_fp4_load(torch.zeros(1, 4, 72, dtype=torch.uint8), i.long(), f)
    with pytest.raises(ValueError):
        ck.ckv_fp4_attention(f.view(4, 1, 128).bfloat16(), torch.zeros(1, 4, 72, dtype=torch.uint8), i.view(4, 1), i, i, 4, 1.0)
