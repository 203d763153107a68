"""The device status word of decode and chunk calls (marked gpu)."""
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


def test_a_call_without_work_leaves_a_clean_status():
    b = Batch([1, 2], [70, 90], 16, 64, 3, DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = torch.empty(0, 16, 512, device=DEV), torch.empty(0, 16, device=DEV)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale)
    bad = b.table.clone()
    bad[0, 0] = -1
    no_tokens = dict(cu=torch.zeros(3, **i32), table=b.table, ctx=b.ctx_t)
    no_requests = dict(cu=torch.zeros(1, **i32), table=b.table[:0], ctx=b.ctx_t[:0])
    for call in (no_tokens, no_requests):
        for before in ("garbage", "flagged"):
            if before == "garbage":
                ws.fill_(0xFF)
            else:
                b2 = Batch([1, 2], [70, 90], 16, 64, 3, DEV)
                b2.table = bad
                chunk(b2, ws=ws)
                assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
            S.splash_chunk_attn(b.q[:0], b.pool, call["cu"], call["table"], call["ctx"], 0, 16, 0, -1, out, lse, ws, b.scale)
            assert S.splash_workspace_status(ws) == 0, before


def test_a_decode_without_requests_leaves_a_clean_status():
    b = Batch([1, 1], [70, 90], 16, 64, 4, DEV)
    out, lse = torch.empty(2, 16, 512, device=DEV), torch.empty(2, 16, device=DEV)
    ws = S.decode_workspace(b.q, b.pool, b.table, b.scale)
    b.table[0, 0] = -1
    S.splash_decode_attn(b.q, b.pool, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, b.scale)
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
    none = (b.q[:0], b.pool, b.table[:0], b.ctx_t[:0], 0, 16, 0, -1, out[:0], lse[:0])
    S.splash_decode_attn(*none, ws, b.scale)
    assert S.splash_workspace_status(ws) == 0
    S.splash_decode_attn_noalloc(b.q, b.pool, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, b.scale)
    assert S.splash_noalloc_status() == S.SPLASH_DEVICE_BAD_INPUT
    S.splash_decode_attn_noalloc(*none, b.scale)
    assert S.splash_noalloc_status() == 0
