"""Causal attention of a chunk of new tokens over the paged cache (marked gpu), against the
64-bit form of tests/serving_reference.py."""
import math
import random

import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.serving_reference import Batch, assert_chunk, chunk_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def run(b, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16, ws=None, out=None, lse=None,
        stream=None):
    head_hi = b.heads if head_hi is None else head_hi
    if out is None:
        out = torch.full((b.rows, b.heads, 512), 7.0, dtype=dtype, device=b.device)
    if lse is None:
        lse = torch.full((b.rows, b.heads), 7.0, device=b.device)
    if ws is None:
        ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale, head_lo, head_hi)
    S.splash_chunk_attn(b.q, b.pool, b.cu, b.table, b.ctx_t, head_lo, head_hi, tok_lo, tok_hi, out, lse, ws,
                        b.scale, stream=stream)
    return out, lse, ws


def check(b, what, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16):
    head_hi = b.heads if head_hi is None else head_hi
    out, lse, ws = run(b, head_lo, head_hi, tok_lo, tok_hi, dtype)
    assert S.splash_workspace_status(ws) == 0, what
    assert_chunk(b, out, lse, chunk_reference(b, head_lo, head_hi, tok_lo, tok_hi), head_lo, head_hi, what)
    # what no request owns, and other heads, are left as they were
    own = int(b.cu[-1])
    assert (out[own:] == 7).all() and (lse[own:] == 7).all(), what
    assert (out[:, :head_lo] == 7).all() and (out[:, head_hi:] == 7).all() and (lse[:, head_hi:] == 7).all(), what
    return out, lse


def test_one_tile():
    check(Batch([64], [64], 2, 64, 1, DEV), "one full tile of rows, half a tile of keys")


def test_tiny():
    check(Batch([1, 4], [64, 100], 8, 16, 2, DEV), "tiny")


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [1, 8, 16, 40, 64, 128])
def test_heads_and_pages(heads, page):
    b = Batch([1, 3, 0, 17, 1], [1, 130, 77, 300, 641], heads, page, 10 + heads + page, DEV, pad_rows=3)
    check(b, f"{heads} heads, pages of {page}")


@pytest.mark.parametrize("heads", [65, 100, 129, 160, 256])
def test_odd_head_counts(heads):
    check(Batch([2, 5], [140, 259], heads, 64, heads, DEV), f"{heads} heads", dtype=torch.float32)


@pytest.mark.parametrize("lo,hi", [(0, 16), (16, 32), (112, 128), (3, 4), (5, 75), (64, 128)])
def test_head_slices(lo, hi):
    check(Batch([1, 6, 2], [90, 400, 128], 128, 64, 30, DEV, pad_rows=2), f"heads [{lo}, {hi})", lo, hi)


@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 383])
def test_whole_prompts_of_every_edge(ctx):
    for page in (16, 64, 128):
        check(Batch([ctx], [ctx], 16, page, 100 + ctx, DEV), f"prompt of {ctx}, pages of {page}")


def test_long_prompt_and_mixed_batch():
    check(Batch([513, 1, 200, 1, 64], [513, 3000, 1777, 1, 4096], 128, 64, 41, DEV), "mixed", dtype=torch.float32)


@pytest.mark.parametrize("tok_lo,tok_hi", [(0, 100), (100, -1), (128, 256), (77, 301), (300, 300), (5000, -1), (0, 0)])
def test_token_ranges(tok_lo, tok_hi):
    check(Batch([4, 40, 1], [333, 400, 90], 16, 64, 50, DEV), f"[{tok_lo}, {tok_hi})", 0, 16, tok_lo, tok_hi)


def test_shares_merge_to_the_whole():
    b = Batch([1, 9], [1000, 777], 128, 64, 51, DEV)
    whole, wl = check(b, "whole", dtype=torch.float32)
    cuts = [0, 256, 300, 2000]
    po = torch.empty(3, b.rows, 128, 512, device=DEV)
    pl = torch.empty(3, b.rows, 128, device=DEV)
    for i in range(3):
        run(b, 0, 128, cuts[i], cuts[i + 1], out=po[i], lse=pl[i])
    out, lse = torch.empty_like(whole), torch.empty_like(wl)
    S.splash_lse_merge(po, pl, out, lse)
    assert_chunk(b, out, lse, chunk_reference(b, 0, 128), 0, 128, "merged")


@pytest.mark.parametrize("q,ctx,heads", [(1, 20000, 128), (3, 9001, 16), (2, 5000, 256)])
def test_few_rows_over_a_long_context_are_split(q, ctx, heads):
    check(Batch([q], [ctx], heads, 64, q, DEV), "split", dtype=torch.float32)
    check(Batch([q], [ctx], heads, 64, q, DEV), "split")


def test_requests_past_one_batch_of_the_plan():
    n = 1100
    q = [(i * 7) % 3 for i in range(n)]
    ctx = [q[i] + (i * 37) % 150 for i in range(n)]
    check(Batch(q, ctx, 8, 16, 60, DEV), "1100 requests")


def test_growing_scores_rescale():
    b = Batch([5, 2], [900, 513], 128, 64, 61, DEV)
    for r in range(2):                    # late keys along early queries: the maximum jumps again and again
        for j, t in enumerate(range(40, b.ctx[r], 130)):
            v = b.q[int(b.cu[r]), j % 128].float().cpu() * (0.5 + 0.25 * j)
            b.keys[r][t] = v.to(torch.bfloat16)
            b.pool[b.table[r, t // 64].item(), t % 64] = b.keys[r][t].to(DEV)
    check(b, "rescale", dtype=torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_growing_scores_in_every_one_of_many_items(dtype):
    n = 320                               # several items for every pair of SMs, of three to five key tiles
    b = Batch([1] * n, [300 + (i * 29) % 260 for i in range(n)], 128, 64, 79, DEV)
    for r in range(n):
        for j, t in enumerate(range(135 + r % 7, b.ctx[r], 130)):
            b.keys[r][t] = (b.q[r, (r + 37 * j) % 128].float().cpu() * (0.5 + 0.25 * j)).to(torch.bfloat16)
            b.pool[b.table[r, t // 64].item(), t % 64] = b.keys[r][t].to(DEV)
    check(b, "rescale in every item", dtype=dtype)


def test_negative_and_zero_scale():
    for scale in (-0.1, 0.0):
        check(Batch([3], [200], 16, 64, 62, DEV, scale=scale), f"scale {scale}", dtype=torch.float32)


def test_more_new_tokens_than_context_leaves_rows_empty():
    b = Batch([5], [9], 16, 64, 63, DEV)
    b.ctx_t.fill_(3)                      # two of the five rows lie before the first position
    out, lse, ws = run(b)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    assert torch.isfinite(lse[2:]).all() and S.splash_workspace_status(ws) == 0


def test_missing_pages_are_left_out_and_flagged():
    for page in (16, 64, 128):
        b = Batch([2, 3], [400, 300], 16, page, 64, DEV)
        missing = [torch.zeros(c, dtype=torch.bool) for c in b.ctx]
        for r, pg, bad in ((0, 1, -1), (1, 0, b.pool.shape[0]), (1, 300 // page, 1 << 30)):
            b.table[r, pg] = bad
            missing[r][pg * page:(pg + 1) * page] = True
        out, lse, ws = run(b)
        assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
        assert_chunk(b, out, lse, chunk_reference(b, 0, 16, missing=missing), 0, 16, f"pages of {page}")


def test_bad_lengths_and_offsets_are_flagged():
    b = Batch([2, 3], [100, 90], 16, 64, 65, DEV)
    b.ctx_t[0] = 1 << 20
    _, _, ws = run(b)
    assert S.splash_workspace_status(ws) & S.SPLASH_DEVICE_BAD_INPUT
    b.ctx_t[0] = 100
    for cu in ([0, 9, 5], [0, 2, 50], [-3, 2, 5], [4, 1, 5]):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        _, _, ws = run(b)
        assert S.splash_workspace_status(ws) & S.SPLASH_DEVICE_BAD_INPUT, cu


@pytest.mark.parametrize("cu", [[0, 9, 5], [0, 2, 50], [-3, 2, 5], [4, 1, 5], [0, 5, 0]])
def test_offsets_out_of_order_leave_every_row_alone(cu):
    b = Batch([2, 3], [100, 90], 16, 64, 65, DEV)
    b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    out, lse, ws = run(b)
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
    assert (out == 7).all() and (lse == 7).all()


def test_empty_pool_and_empty_calls():
    b = Batch([1, 2], [1, 2], 16, 64, 66, DEV)
    b.pool = b.pool[:0]
    out, lse, ws = run(b)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
    b = Batch([0, 0], [10, 0], 16, 64, 67, DEV, pad_rows=2)
    out, lse, _ = run(b)
    assert (out == 7).all() and (lse == 7).all()


def test_same_bits_again_and_workspace_reuse():
    b = Batch([100, 7, 1], [700, 2000, 5000], 128, 64, 70, DEV)
    out, lse, ws = run(b)
    small = Batch([1], [50], 128, 64, 71, DEV)
    small.table = torch.nn.functional.pad(small.table, (0, b.table.shape[1] - small.table.shape[1]), value=-1)
    for _ in range(2):
        run(small, ws=ws)
        o2, l2, _ = run(b, ws=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_requests_that_share_their_first_pages():
    b = Batch([40, 3, 1], [500, 400, 300], 128, 64, 77, DEV)
    for r in (1, 2):
        b.table[r, :3] = b.table[0, :3]
        b.keys[r][:192] = b.keys[0][:192]
    check(b, "shared prefix")


def test_one_workspace_for_decode_and_chunk_in_turn():
    b = Batch([1, 1], [900, 2500], 128, 64, 78, DEV)
    sizes = [S.chunk_workspace(b.q, b.pool, b.table, b.scale), S.decode_workspace(b.q, b.pool, b.table, b.scale)]
    ws = torch.full((max(x.numel() for x in sizes),), 0xFF, dtype=torch.uint8, device=DEV)
    ref = chunk_reference(b, 0, 128)
    out, lse = torch.empty(2, 128, 512, device=DEV), torch.empty(2, 128, device=DEV)
    for _ in range(2):
        run(b, ws=ws, out=out, lse=lse)
        assert S.splash_workspace_status(ws) == 0
        assert_chunk(b, out, lse, ref, 0, 128, "chunk")
        S.splash_decode_attn(b.q, b.pool, b.table, b.ctx_t, 0, 128, 0, -1, out, lse, ws, b.scale)
        assert S.splash_workspace_status(ws) == 0
        assert_chunk(b, out, lse, ref, 0, 128, "decode")


def test_two_calls_at_once_on_two_streams():
    bs = [Batch([50, 1], [600, 3000], 128, 64, 72 + i, DEV) for i in range(2)]
    refs = [chunk_reference(b, 0, 128) for b in bs]
    outs = [(torch.empty(b.rows, 128, 512, dtype=torch.bfloat16, device=DEV),
             torch.empty(b.rows, 128, device=DEV), S.chunk_workspace(b.q, b.pool, b.table, b.scale)) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, (o, l, ws), s in zip(bs, outs, streams):
            run(b, out=o, lse=l, ws=ws, stream=s)
    torch.cuda.synchronize()
    for b, (o, l, ws), ref in zip(bs, outs, refs):
        assert_chunk(b, o, l, ref, 0, 128, "concurrent")
        assert S.splash_workspace_status(ws) == 0


def test_captured_and_replayed_on_new_lengths():
    b = Batch([3, 30], [500, 200], 128, 64, 74, DEV)
    out, lse, ws = run(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(b, out=out, lse=lse, ws=ws)
    for ctx in ([500, 200], [333, 64], [40, 30]):
        b.ctx = ctx
        b.ctx_t.copy_(torch.tensor(ctx, dtype=torch.int32))
        keys = b.keys
        b.keys = [k[:c] for k, c in zip(keys, ctx)]
        out.fill_(7)
        g.replay()
        assert_chunk(b, out, lse, chunk_reference(b, 0, 128), 0, 128, f"replayed {ctx}")
        b.keys = keys


def test_pages_past_two_to_the_31_bytes():
    b = Batch([2], [700], 16, 64, 75, DEV)
    n = 60000                              # 4.4 GB
    big = torch.empty(n, 64, 576, dtype=torch.bfloat16, device=DEV)
    ids = n - 1 - torch.arange(b.table.shape[1], device=DEV)
    big[ids] = b.pool[b.table[0].long()]
    b.table = ids.to(torch.int32)[None].contiguous()
    b.pool = big
    check(b, "far pages")


def test_single_tokens_agree_with_the_decode():
    b = Batch([1, 1, 1], [100, 1024, 3001], 128, 64, 76, DEV)
    out, lse = check(b, "single tokens", dtype=torch.float32)
    do, dl = torch.empty_like(out), torch.empty_like(lse)
    ws = S.decode_workspace(b.q, b.pool, b.table, b.scale)
    S.splash_decode_attn(b.q, b.pool, b.table, b.ctx_t, 0, 128, 0, -1, do, dl, ws, b.scale)
    assert_chunk(b, do, dl, chunk_reference(b, 0, 128), 0, 128, "decode")


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    r = random.Random(seed)
    heads = r.choice([1, 3, 8, 16, 24, 40, 64, 72, 128])
    lo = r.randrange(heads)
    hi = r.randint(lo + 1, heads)
    B = r.choice([1, 2, 5, 40])
    q = [r.choice([0, 1, 1, 2, r.randint(1, 200 // B + 1)]) for _ in range(B)]
    ctx = [n + r.choice([0, 0, 1, r.randint(0, 127), r.randint(0, 6000 // B)]) for n in q]
    b = Batch(q, ctx, heads, r.choice([16, 32, 64, 128]), 200 + seed, DEV, pad_rows=r.choice([0, 1, 9]),
              scale=r.choice([1 / math.sqrt(192.0), 0.3]))
    if b.rows == 0:
        pytest.skip("no rows drawn")
    tok_lo = r.choice([0, 0, r.randint(0, 300)])
    tok_hi = r.choice([-1, -1, tok_lo + r.randint(0, 3000)])
    check(b, f"seed {seed}", lo, hi, tok_lo, tok_hi, r.choice([torch.bfloat16, torch.float32]))


def test_an_infinite_or_nan_slot_past_the_context_never_shows():
    for bad in (math.nan, math.inf, -math.inf):
        for ctx in (1, 63, 65, 129, 200):
            b = Batch([min(ctx, 5)], [ctx], 16, 64, 300 + ctx, DEV)
            page, off = (ctx - 1) // 64, (ctx - 1) % 64
            b.pool[b.table[0, page].item(), off + 1:] = bad
            spare = sorted(set(range(b.pool.shape[0])) - set(b.table.flatten().tolist()))
            b.pool[spare] = bad
            check(b, f"{bad} past {ctx}")


def test_refusals():
    b = Batch([2], [70], 16, 64, 400, DEV)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale)
    out, lse = torch.empty(2, 16, 512, device=DEV), torch.empty(2, 16, device=DEV)

    def call(q=b.q, pool=b.pool, cu=b.cu, table=b.table, ctx=b.ctx_t, lo=0, hi=16, out=out, lse=lse, ws=ws):
        S.splash_chunk_attn(q, pool, cu, table, ctx, lo, hi, 0, -1, out, lse, ws, b.scale)
    call()
    for kw in (dict(q=b.q.float()), dict(pool=b.pool.float()), dict(out=out.half()), dict(lse=lse.half()),
               dict(cu=b.cu.long()), dict(table=b.table[0]), dict(ctx=b.ctx_t[:0]), dict(out=out[:1]),
               dict(q=b.q[..., :575]), dict(pool=b.pool[None]), dict(q=b.q.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(ctx=b.ctx_t.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(S.SplashError) as e:
        call(ws=ws[:256])
    assert e.value.code == S.SPLASH_ERR_WORKSPACE
    with pytest.raises(S.SplashError) as e:
        call(lo=8, hi=17)
    assert e.value.code == S.SPLASH_ERR_INVALID_ARG
    wide = torch.empty(2 * 16 * 512 + 8, dtype=torch.bfloat16, device=DEV)[8:].view(2, 16, 512)
    with pytest.raises(S.SplashError) as e:      # 16-byte aligned only
        call(out=wide)
    assert e.value.code == S.SPLASH_ERR_INVALID_ARG
