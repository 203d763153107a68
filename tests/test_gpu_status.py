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


SHARES = [(0, 100), (100, 300), (37, 61), (300, -1), (130, 250), (64, 192), (399, 400)]


def share_table(b, page, lo, hi):
    """b's block table with -1 for the pages that no token of [lo, hi) lies on."""
    t = b.table.clone()
    for r, c in enumerate(b.ctx):
        end = c if hi < 0 else min(hi, c)
        for p in range(t.shape[1]):
            if p * page >= end or (p + 1) * page <= lo:
                t[r, p] = -1
    return t


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lo,hi", SHARES)
def test_pages_outside_a_share_need_not_exist(page, lo, hi):
    b = Batch([2, 30], [333, 400], 16, page, 50, DEV)
    ref = chunk_reference(b, 0, 16, lo, hi)
    b.table = share_table(b, page, lo, hi)
    out, lse, ws = chunk(b, lo, hi)
    assert_chunk(b, out, lse, ref, 0, 16, f"share [{lo}, {hi})")
    assert S.splash_workspace_status(ws) == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lo,hi", SHARES)
def test_pages_outside_a_decode_share_need_not_exist(page, lo, hi):
    b = Batch([1, 1], [333, 400], 16, page, 51, DEV)
    ref = chunk_reference(b, 0, 16, lo, hi)
    b.table = share_table(b, page, lo, hi)
    out, lse = torch.empty(2, 16, 512, device=DEV), torch.empty(2, 16, device=DEV)
    ws = S.decode_workspace(b.q, b.pool, b.table, b.scale)
    S.splash_decode_attn(b.q, b.pool, b.table, b.ctx_t, 0, 16, lo, hi, out, lse, ws, b.scale)
    assert_chunk(b, out, lse, ref, 0, 16, f"share [{lo}, {hi})")
    assert S.splash_workspace_status(ws) == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_missing_page_at_the_edge_of_a_share_is_flagged(page):
    for lo, hi in ((100, 300), (37, 161)):
        for tok in (lo, hi - 1):
            b = Batch([1, 1], [333, 400], 16, page, 52, DEV)
            b.table[1, tok // page] = -1
            out, lse, ws = chunk(b, lo, hi)
            assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT, (lo, hi, tok)
            ws = S.decode_workspace(b.q, b.pool, b.table, b.scale)
            S.splash_decode_attn(b.q, b.pool, b.table, b.ctx_t, 0, 16, lo, hi, out, lse, ws, b.scale)
            assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT, (lo, hi, tok)
