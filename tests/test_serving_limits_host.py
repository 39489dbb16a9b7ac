"""The ends of what the serving-step operators accept, on the CPU: every call here
returns during argument validation."""
import os
import random
import subprocess
import sys

import pytest

from test_serving_ops_host import ATTN, ONE, P, _call, lib  # noqa: F401

MAX_ROWS = 160 * 2 ** 17  # cache rows that a token may see
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("stride,status", [(0, 1), (1, 2), (15, 2), (16, 1), (-16, 2)])
def test_fp4_attention_table_strides(lib, stride, status):  # noqa: F811
    """A block table's rows lie apart (stride >= 16 pages here) or are one row; with those the next
    refusal comes, that of a missing q."""
    assert _call(lib.ckv_fp4_attention, ATTN, tstride=stride, q=None) == status


@pytest.mark.parametrize("max_rows", [0, -1, -2 ** 63, MAX_ROWS + 1, 2 ** 31 - 2 ** 14, 2 ** 31, 2 ** 38, 2 ** 40, 160 * 2 ** 32, 2 ** 62, 2 ** 63 - 1])
def test_fp4_attention_workspace_of_rows_past_the_bound(max_rows):
    """Sizes that the call refuses need no workspace: the answer is 0 (in a process of its own, which a
    division by a count that wrapped to 0 would end)."""
    code = ("from compressed_kv_attention_gated_gb300 import ckv\n"
            "for T, B in ((1, 1), (19, 19), (160, 160), (65536, 65536), (7, 2)):\n"
            "    for H in (1, 16, 40, 64, 1024):\n"
            "        for D in (128, 256, 512):\n"
            f"            assert ckv.ckv_fp4_attention_workspace(T, B, H, D, {max_rows}) == 0, (T, B, H, D)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def test_fp4_attention_workspace_of_sizes_that_the_call_refuses(lib):  # noqa: F811
    for T, B, H, D in ((1, 65537, 1, 128), (2 ** 31, 1, 1, 128), (2 ** 22, 1, 1024, 128), (2 ** 62, 1, 1, 128), (1, 1, 1025, 128),
                       (1, 1, 0, 128), (-1, 1, 1, 128), (1, -1, 1, 128), (1, 1, 1, 64)):
        assert lib.ckv_fp4_attention_workspace(T, B, H, D, 2 ** 20) == 0


def test_fp4_attention_workspace_bounds(lib):  # noqa: F811
    """For sizes that the call takes: never negative, and never more than an fp32 output, a maximum and
    a sum per row for each of 160 ranges and two halves, rows rounded up to tiles of 128 per request."""
    rng = random.Random(0)
    some = 0
    assert lib.ckv_fp4_attention_workspace(1, 1, 16, 128, MAX_ROWS) > 0
    for _ in range(4000):
        B = int(2 ** rng.uniform(0, 16))
        T = min(int(B * 2 ** rng.uniform(-1, 6)) + 1, 2 ** 21 - 1)
        H, D = rng.randint(1, 1024), rng.choice([128, 256, 512])
        rows = MAX_ROWS if rng.random() < 0.1 else min(int(2 ** rng.uniform(0, 24.4)), MAX_ROWS)
        need = lib.ckv_fp4_attention_workspace(T, B, H, D, rows)
        assert 0 <= need <= (T * H + 128 * B) * 160 * 4 * (D + 4), (T, B, H, D, rows)
        some += need > 0
    assert some > 400


def test_fp4_attention_workspace_that_is_missing_or_short(lib):  # noqa: F811
    big = dict(T=1, B=1, H=64, D=512, rows=10 ** 6, mp=20000, tstride=20000, out=P(1 << 40))
    need = lib.ckv_fp4_attention_workspace(1, 1, 64, 512, 10 ** 6)
    assert need > 0
    assert _call(lib.ckv_fp4_attention, ATTN, **big) == 1
    assert _call(lib.ckv_fp4_attention, ATTN, **big, ws=ONE, wsb=need - 1) == 2


@pytest.mark.parametrize("T,B,H,D", [(1, 1, 1, 128), (1, 1, 128, 512), (152, 152, 4, 128), (152, 152, 40, 128), (3000, 9, 16, 256),
                                     (65536, 65536, 8, 512)])
def test_fp4_attention_ranges_are_of_131072_rows_at_most(lib, T, B, H, D):  # noqa: F811
    """Rows past 2^17 are split over ranges whatever that costs: the workspace holds as many outputs."""
    for rows in (2 ** 17 + 1, 2 ** 19, 10 ** 6, MAX_ROWS - 1, MAX_ROWS):
        ranges = -(-rows // 2 ** 17)
        assert lib.ckv_fp4_attention_workspace(T, B, H, D, rows) >= ranges * T * H * (D + 2) * 4


def test_fp4_attention_refuses_rows_past_the_bound(lib):  # noqa: F811
    wide = dict(mp=2 ** 25, tstride=2 ** 25, ps=64, ws=ONE, wsb=2 ** 62, out=P(1 << 40))
    for rows in (MAX_ROWS + 1, 2 ** 31 - 2 ** 14 - 1):
        assert _call(lib.ckv_fp4_attention, ATTN, **wide, rows=rows) == 2
    assert _call(lib.ckv_fp4_attention, {**ATTN, **wide}, rows=MAX_ROWS, q=None) == 1
    assert _call(lib.ckv_fp4_attention, {**ATTN, **wide}, rows=MAX_ROWS, wsb=0) == 2
