"""The ends of what the operators around the uncompressed cache accept, on the CPU: every call here returns during
argument validation."""
import os
import re

import pytest

from test_kv_ops_host import ATTN, P, _cache, _call, lib  # noqa: F401

MAX_ROWS = 160 * 2 ** 17


@pytest.mark.parametrize("T,B,KH,rows,takes", [
    (16384, 16384, 1024, MAX_ROWS, False),         # a tile of rows to a request x 160 ranges of keys x 1024 key heads
    (65536, 65536, 1024, 32 * 2 ** 17, False),     # 2^31 CTAs
    (65536, 65536, 1024, 31 * 2 ** 17, True),
    (65536, 65536, 256, MAX_ROWS, False), (65536, 65536, 128, MAX_ROWS, True),
    # requests without tokens need none
    (1, 65536, 1024, MAX_ROWS, True), (8192, 65536, 1024, MAX_ROWS, True), (16384, 65536, 1024, MAX_ROWS, False)])
def test_grids_beyond_31_bits(lib, T, B, KH, rows, takes):  # noqa: F811
    """What fits is refused for the missing queries that come next."""
    sizes = dict(T=T, B=B, H=KH, rows=rows, mp=-(-rows // 16), tstride=-(-rows // 16))
    call = {**ATTN, "cache": _cache(heads=KH, k_stride_row=128 * KH, v_stride_row=128 * KH)}
    assert _call(lib.ckv_kv_attention, call, **sizes, q=None) == (1 if takes else 2)
    need = lib.ckv_kv_attention_workspace(T, B, KH, KH, 128, rows, 0, 0, 0)
    assert need > 0 if takes else need == 0
    # the same rows behind a window, and in one request
    assert _call(lib.ckv_kv_attention, call, **sizes, window=4096, q=None) == 1
    assert _call(lib.ckv_kv_attention, call, **{**sizes, "B": 1}, q=None) == 1


@pytest.mark.parametrize("name", ["kv_attention.cu", "kv_attention_few.cu"])
def test_no_answer_of_a_wait_is_written_over(name):
    """A wait that runs out ends the kernel with an error, which no later wait may take back: an answer goes into `ok`
    together with those before it.  (From the source: on a GPU it would take a wait that does not end.)"""
    import compressed_kv_attention_gated_gb300 as ck

    text = open(os.path.join(os.path.dirname(ck.__file__), "csrc", name)).read()
    waits = re.findall(r"\bok = [^;]*mbar_wait_near\([^;]*;", text)
    assert waits and all(re.search(r"&& ok;$|= ok &&", w) for w in waits), waits
