"""The operators around the uncompressed cache at the ends of what their contracts allow."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_ops import Step, _err, _i32, ck, close  # noqa: F401

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_merge_of_infinite_parts(ck, dtype):  # noqa: F811
    """A part whose lse is infinite (a sink of infinity) counts alone; two of them count alike; and the lowest value is a
    number like others."""
    inf, low = torch.inf, torch.finfo(torch.float32).min
    rows = [([inf, 3.0], [1.0, 0.0], inf), ([-inf, inf], [0.0, 1.0], inf), ([inf, inf], [0.5, 0.5], inf), ([low, 3.0], [0.0, 1.0], 3.0),
            ([low, -inf], [1.0, 0.0], low), ([-inf, -inf], [0.0, 0.0], -inf)]
    g = torch.Generator(device="cuda").manual_seed(1)
    for D in (128, 256, 512):
        a, b = (torch.randn(len(rows), 3, D, generator=g, device="cuda").to(dtype) for _ in range(2))
        la, lb = (torch.tensor([r[0][i] for r in rows], device="cuda")[:, None].expand(-1, 3).contiguous() for i in range(2))
        out, lse = ck.ckv_merge_attention([a, b], [la, lb], out=torch.empty_like(a))
        wa, wb = (torch.tensor([r[1][i] for r in rows], device="cuda")[:, None, None] for i in range(2))
        assert torch.equal(out, (a.float() * wa + b.float() * wb).to(dtype))
        assert torch.equal(lse, torch.tensor([r[2] for r in rows], device="cuda")[:, None].expand(-1, 3))


@pytest.mark.parametrize("D,H,KH,n,before,B", [(128, 24, 3, 1, 60, 700), (128, 40, 5, 1, 90, 800), (128, 56, 7, 4, 30, 300), (256, 56, 7, 1, 60, 300),
                                               (256, 24, 3, 2, 80, 1300), (512, 48, 3, 1, 70, 1300), (512, 80, 5, 1, 40, 400)])
@pytest.mark.parametrize("window,first", [(32, 2), (0, 0)])
def test_few_rows_of_several_key_heads(ck, D, H, KH, n, before, B, window, first):  # noqa: F811
    """Keys on the M side, and enough CTAs (2 x 6 x 152 for two, twice that for four) that each takes the jobs of two or four
    key heads from one lookup; the count of key heads is no multiple of them, so a last lookup has fewer."""
    tokens = [n + (i % 50 == 7) - (i % 50 == 9) for i in range(B)]
    s = Step(D, H, KH, tokens, [before - i % 20 for i in range(B)], 16, window, first, sink=True, seed=KH)
    s.ctx = np.array(s.ctx)
    s.ctx[[3, 11]] = -1, 0
    G = H // KH
    R = 16 if n * G <= 16 else 32
    tiles = (n * B * G + B * max(0, R - (G & -G))) // R
    assert sum(tokens) == n * B and n * G <= R and tiles * KH >= 2 * 6 * 152
    out, lse, err = s.run(ck)
    assert int(err) == 0
    s.check(out, lse)


@pytest.mark.parametrize("D,H,KH,n", [(128, 1024, 1024, 1), (128, 256, 2, 10), (256, 96, 1, 10), (512, 64, 1, 2), (128, 24, 3, 5)])
def test_a_few_tokens_among_65536_requests(ck, D, H, KH, n):  # noqa: F811
    """Requests without tokens have no tiles of rows; a bound of 160 * 2^17 rows would split every one of those into 160
    ranges of keys, one after the other on the same CTAs.  All rows of a page are its first one: a token's output is that
    value row, its lse the score and the log of the rows that it sees."""
    B, ps = 65536, 2 ** 21
    g = torch.Generator(device="cuda").manual_seed(D)
    k1, v1 = (torch.randn(4, 1, KH, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n + 1, H, D, generator=g, device="cuda").bfloat16()
    table = torch.full((B, 10), -1, dtype=torch.int32, device="cuda")
    table[777, 0], table[65535, 0] = 1, 3
    start = np.zeros(B + 1, dtype=int)
    start[778:], start[65536:] = 1, n + 1
    ctx = [70] + [300 + i for i in range(n)]
    assert ck.ckv_kv_attention_workspace(n + 1, B, H, KH, D, 10 * ps) >= 160 * (n + 1) * H * (D + 1) * 4
    err = _err()
    out, lse = ck.ckv_kv_attention(q, k1.expand(-1, ps, -1, -1), v1.expand(-1, ps, -1, -1), table, _i32(start), _i32(ctx), 10 * ps, D ** -0.5,
                                   err_word=err)
    assert int(err) == 0
    page = torch.tensor([1] + [3] * n, device="cuda")
    k, v = (x[page, 0].double().repeat_interleave(H // KH, 1) for x in (k1, v1))
    z = (q.double() * k).sum(-1) * D ** -0.5
    seen = torch.tensor(ctx, device="cuda", dtype=torch.float64).log()[:, None]
    close(out, lse, v, z + seen, v.abs(), (q.double() * k).abs().sum(-1) * D ** -0.5, D)
