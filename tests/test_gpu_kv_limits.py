"""The operators around the uncompressed cache at the ends of what their contracts allow."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_ops import _err, _i32, ck  # noqa: F401

pytestmark = pytest.mark.gpu


def test_padding_among_drafts_is_not_looked_at(ck):  # noqa: F811
    """Rows with a negative ctx_rows are no drafts: whatever parents they hold and however many they are, nothing is flagged."""
    n = [6 + 80, 0, 3]
    start = np.concatenate([[0], np.cumsum(n)])
    parents, ctx = np.full(start[-1] + 4, 2 ** 31 - 1), np.full(start[-1] + 4, -1)
    parents[1:86:2] = -2 ** 31
    parents[:6], ctx[:6] = [-1, 0, 0, 2, -1, 3], 40
    parents[86:89], ctx[86:89] = [-1, 9, 0], [7, -1, 7]
    for words in (1, 2):
        err = _err()
        mask, pos = ck.ckv_build_tree_masks(_i32(parents), _i32(start), _i32(ctx), words, err_word=err)
        masks, want = ref.tree(parents.tolist(), start.tolist(), ctx.tolist(), words)
        assert int(err) == 0 and torch.equal(mask.cpu(), ref.pack(masks, words)) and pos.tolist() == want
    ctx[7] = 40  # a draft, with a parent that is none
    mask, pos = ck.ckv_build_tree_masks(_i32(parents), _i32(start), _i32(ctx), 2, err_word=err)
    assert int(err) == 8 and pos.tolist()[7] == 40
