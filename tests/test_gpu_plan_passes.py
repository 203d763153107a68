"""Chunk attention plans that are cut across several passes over the requests (marked gpu)."""
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.serving_reference import Batch, assert_chunk, chunk_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def chunk(b, tok_lo=0, tok_hi=-1, dtype=torch.float32, ws=None):
    out = torch.full((b.rows, b.heads, 512), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((b.rows, b.heads), 7.0, device=DEV)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale) if ws is None else ws
    S.splash_chunk_attn(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, b.heads, tok_lo, tok_hi, out, lse, ws, b.scale)
    return out, lse, ws


def splits_of(ws):
    return int(ws[:16].view(torch.int32)[2])


def test_an_even_cut_of_row_tiles_from_several_passes():
    n = 700                                # the plan looks at 512 requests a pass; most bring no token here
    q, ctx = [0] * n, [(i * 13) % 40 for i in range(n)]
    for i, tokens, c in ((5, 1, 9000), (300, 3, 4001), (511, 1, 700), (512, 2, 12345), (600, 1, 3000), (699, 1, 5000)):
        q[i], ctx[i] = tokens, c
    b = Batch(q, ctx, 128, 64, 81, DEV)
    out, lse, ws = chunk(b)
    assert S.splash_workspace_status(ws) == 0 and splits_of(ws) > 0
    assert_chunk(b, out, lse, chunk_reference(b, 0, 128), 0, 128, "even cut over two passes")


@pytest.mark.parametrize("heads", [128, 8])
def test_long_requests_cut_in_several_passes(heads):
    n = 1200                               # more row tiles than an even cut takes, and a few contexts of many
    ctx = [100 + (i * 37) % 200 for i in range(n)]          # times the others' in every pass
    for i, c in ((3, 20000), (511, 9001), (512, 30000), (700, 7777), (1150, 15000)):
        ctx[i] = c
    b = Batch([1] * n, ctx, heads, 64, 82, DEV)
    out, lse, ws = chunk(b, dtype=torch.bfloat16)
    assert S.splash_workspace_status(ws) == 0 and splits_of(ws) >= 5
    assert_chunk(b, out, lse, chunk_reference(b, 0, heads), 0, heads, "cuts in three passes")
