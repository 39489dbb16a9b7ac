"""The ends of what the serving-step operators accept, on the CPU: every call here
returns during argument validation."""
import pytest

from test_serving_ops_host import ATTN, _call, lib  # noqa: F401


@pytest.mark.parametrize("stride,status", [(0, 1), (1, 2), (15, 2), (16, 1), (-16, 2)])
def test_fp4_attention_table_strides(lib, stride, status):  # noqa: F811
    """A block table's rows lie apart (stride >= 16 pages here) or are one row; with those the next
    refusal comes, that of a missing q."""
    assert _call(lib.ckv_fp4_attention, ATTN, tstride=stride, q=None) == status
