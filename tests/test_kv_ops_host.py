"""Refusals of the operators around the uncompressed cache, on the CPU: every call here returns during
argument validation."""
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


def _cache(**change):
    from compressed_kv_attention_gated_gb300.ckv import KvCache

    f = dict(k=16, v=1 << 20, k_stride_page=4096, k_stride_row=256, k_stride_head=128, v_stride_page=4096, v_stride_row=256,
             v_stride_head=128, num_pages=10, page_size=16, heads=2, D=128, reserved=0)
    assert set(change) <= set(f)
    f.update(change)
    return KvCache(*f.values())


def _rows(**change):
    from compressed_kv_attention_gated_gb300.ckv import KvRows

    f = dict(x=16, stride_t=256, stride_h=128, heads=2, dtype=1)
    f.update(change)
    return KvRows(*f.values())


def _call(fn, base, **change):
    assert set(change) <= set(base)
    args = {**base, **change}
    return fn(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args.values()])


APPEND = dict(k=_rows, v=_rows, q=_rows, q_out=P(1 << 30), st=256, sh=128, T=4, cache=_cache, loc=ONE, pos=ONE, cs=ONE, npos=10, R=64,
              at=64, pairs=0, pdl=0, err=None, stream=None)


def _append(lib, **change):
    base = {k: f() if callable(f) else f for k, f in APPEND.items()}
    return _call(lib.ckv_kv_append, base, **change)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 2), (dict(R=-2), 2), (dict(R=63), 2), (dict(R=130), 2), (dict(at=65), 2), (dict(at=66), 2), (dict(at=-2), 2),
    (dict(npos=-1), 2), (dict(T=2 ** 30), 2), (dict(st=-8), 2), (dict(sh=-8), 2), (dict(k=None), 1), (dict(cache=None), 1),
    (dict(loc=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(q_out=None), 1), (dict(loc=P(20)), 4), (dict(pos=ODD), 4),
    (dict(cs=ODD), 4), (dict(err=ODD), 4), (dict(q_out=P(24)), 4), (dict(st=260), 4), (dict(sh=4), 4), (dict(q_out=P(16), st=512), 2),
    (dict(T=0, loc=None, q_out=None), 0)])
def test_append_refusals(lib, change, status):
    assert _append(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(heads=-1), 2), (dict(heads=3), 2), (dict(stride_t=-8), 2), (dict(stride_h=-8), 2), (dict(dtype=2), 3), (dict(x=None), 1), (dict(x=24), 4),
    (dict(stride_t=260), 4), (dict(stride_h=4), 4), (dict(dtype=0), 3)])
def test_append_row_set_refusals(lib, change, status):
    for name in ("k", "v", "q"):
        if name == "q" and change == dict(heads=3):
            continue  # queries have any number of heads
        if name == "k" and change == dict(dtype=0):
            assert _append(lib, k=_rows(dtype=0)) == 3  # one type for all
            continue
        assert _append(lib, **{name: _rows(**change)}) == status
    # in place only for bf16
    f = dict(k=_rows(dtype=0), v=_rows(dtype=0), q=_rows(dtype=0))
    assert _append(lib, **f, q_out=P(16)) == 2


CACHE_REFUSALS = [
    (dict(num_pages=-1), 2), (dict(num_pages=2 ** 31), 2), (dict(page_size=0), 2), (dict(heads=0), 2), (dict(heads=1025), 2), (dict(D=64), 2),
    (dict(reserved=1), 2), (dict(k_stride_page=-8), 2), (dict(v_stride_row=-8), 2), (dict(v_stride_head=-8), 2), (dict(k=None), 1), (dict(v=None), 1),
    (dict(k=24), 4), (dict(v=24), 4), (dict(k_stride_row=132), 4), (dict(v_stride_page=4), 4), (dict(k_stride_head=2), 4)]


@pytest.mark.parametrize("change,status", CACHE_REFUSALS)
def test_cache_refusals(lib, change, status):
    assert _append(lib, cache=_cache(**change)) == status
    assert _call(lib.ckv_kv_attention, {**ATTN, "cache": _cache(**change)}) == status


def test_append_refuses_values_over_keys(lib):
    assert _append(lib, cache=_cache(v=16)) == 2


MASKS = dict(parents=ONE, start=ONE, B=4, ctx=ONE, T=10, words=1, mask=ONE, pos=ONE, pdl=0, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 2), (dict(B=65537), 2), (dict(T=-1), 2), (dict(T=2 ** 31), 2), (dict(words=0), 2), (dict(words=17), 2), (dict(parents=None), 1),
    (dict(start=None), 1), (dict(mask=None), 1), (dict(parents=ODD), 4), (dict(start=ODD), 4), (dict(ctx=ODD), 4), (dict(mask=P(20)), 4),
    (dict(pos=ODD), 4), (dict(err=ODD), 4), (dict(T=0, mask=None), 0)])
def test_tree_masks_refusals(lib, change, status):
    assert _call(lib.ckv_build_tree_masks, MASKS, **change) == status


ATTN = dict(q=P(1 << 30), st=1024, sh=128, T=4, H=8, cache=None, table=ONE, tstride=16, mp=16, start=ONE, B=4, ctx=ONE, rows=256, window=0, first=0,
            mask=None, words=0, scale=0.1, sink=None, out=ONE, lse=ONE, ws=ONE, wsb=2 ** 62, pdl=0, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), 2), (dict(B=-1), 2), (dict(B=65537), 2), (dict(H=0), 2), (dict(H=1026), 2), (dict(H=7), 2), (dict(mp=-1), 2), (dict(tstride=15), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(rows=0), 2), (dict(rows=257), 2), (dict(window=-1), 2), (dict(first=-1), 2),
    (dict(words=-1), 2), (dict(words=17, mask=ONE), 2), (dict(T=2 ** 29), 2), (dict(st=-8), 2), (dict(sh=-8), 2), (dict(q=None), 1),
    (dict(table=None), 1), (dict(start=None), 1), (dict(ctx=None), 1), (dict(out=None), 1), (dict(words=1), 1), (dict(q=P(24)), 4),
    (dict(st=1020), 4), (dict(sh=4), 4), (dict(table=ODD), 4), (dict(start=ODD), 4), (dict(ctx=ODD), 4), (dict(sink=ODD), 4), (dict(out=P(24)), 4),
    (dict(lse=ODD), 4), (dict(ws=P(24)), 4), (dict(err=ODD), 4), (dict(mask=P(20), words=1), 4), (dict(rows=20971521, mp=2 ** 22, tstride=2 ** 22), 2),
    (dict(T=0, q=None, out=None), 0), (dict(B=0, table=None), 0)])
def test_attention_refusals(lib, change, status):
    assert _call(lib.ckv_kv_attention, {**ATTN, "cache": _cache()}, **change) == status


def test_attention_refuses_an_output_over_the_queries(lib):
    span = ((ATTN["T"] - 1) * 1024 + 7 * 128 + 128) * 2
    for q, out in ((1 << 20, 1 << 20), (1 << 20, (1 << 20) + span - 16), ((1 << 20) + 4 * 8 * 128 * 2 - 16, 1 << 20)):
        assert _call(lib.ckv_kv_attention, {**ATTN, "cache": _cache()}, q=P(q), out=P(out)) == 2


def test_attention_workspace_is_asked_for(lib):
    assert lib.ckv_kv_attention_workspace(0, 4, 8, 2, 128, 10, 0, 0, 0) == 0
    assert lib.ckv_kv_attention_workspace(1, 1, 8, 3, 128, 10, 0, 0, 0) == 0
    assert lib.ckv_kv_attention_workspace(1, 1, 8, 2, 192, 10, 0, 0, 0) == 0
    need = lib.ckv_kv_attention_workspace(1, 1, 8, 2, 128, 10 ** 6, 0, 0, 0)
    if need:
        big = dict(T=1, B=1, rows=10 ** 6, mp=70000, tstride=70000)
        assert _call(lib.ckv_kv_attention, {**ATTN, "cache": _cache()}, **big, ws=None, wsb=0) == 1
        assert _call(lib.ckv_kv_attention, {**ATTN, "cache": _cache()}, **big, wsb=need - 1) == 2


def test_merge_refusals(lib):
    from compressed_kv_attention_gated_gb300.ckv import AttentionPart

    def call(parts=((16, 16), (32, 16)), n=None, dtype=1, T=3, H=4, D=128, pos=None, out=P(64), out_dtype=1, lse=None):
        arr = (AttentionPart * max(1, len(parts)))(*[AttentionPart(*p) for p in parts])
        return lib.ckv_merge_attention(arr, len(parts) if n is None else n, dtype, T, H, D, pos, out, out_dtype, lse, 0, None)

    for change, status in ((dict(n=0), 2), (dict(n=9), 2), (dict(T=-1), 2), (dict(H=0), 2), (dict(H=1025), 2), (dict(D=64), 2),
                           (dict(T=2 ** 30), 2), (dict(dtype=2), 3), (dict(out_dtype=2), 3), (dict(out=None), 1), (dict(out=P(24)), 4),
                           (dict(lse=ODD), 4), (dict(pos=ODD), 4), (dict(parts=((16, None), (32, 16))), 1), (dict(parts=((None, 16),)), 1),
                           (dict(parts=((16, 16), (24, 16))), 4), (dict(parts=((16, 18),)), 4), (dict(out=P(32), out_dtype=0), 2),
                           (dict(T=0, out=None), 0)):
        assert call(**change) == status, change
    assert lib.ckv_merge_attention(None, 1, 1, 3, 4, 128, None, ONE, 1, None, 0, None) == 1


def test_binding_refuses_cpu_tensors(lib):
    import compressed_kv_attention_gated_gb300 as ck

    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 128)
    c = torch.zeros(2, 4, 2, 128).bfloat16()
    with pytest.raises(ValueError):
        ck.ckv_kv_append(f, f, c, c.clone(), i.long())
    with pytest.raises(ValueError):
        ck.ckv_build_tree_masks(i, i)
    with pytest.raises(ValueError):
        ck.ckv_kv_attention(f.bfloat16(), c, c, i.view(4, 1), i, i, 4, 1.0)
    with pytest.raises(ValueError):
        ck.ckv_merge_attention([f], [f[..., 0]])
    with pytest.raises(ValueError):
        ck.ckv_merge_attention([], [])
