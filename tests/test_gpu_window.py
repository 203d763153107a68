"""Attention over a sliding window and some first tokens (marked gpu), against the 64-bit form of
tests/more_reference.py."""
import random

import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.more_reference import attention_reference
from tests.serving_reference import Batch, assert_chunk, chunk_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def run(b, window, sinks, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16, ws=None, stream=None):
    head_hi = b.heads if head_hi is None else head_hi
    out = torch.full((b.rows, b.heads, 512), 7.0, dtype=dtype, device=b.device)
    lse = torch.full((b.rows, b.heads), 7.0, device=b.device)
    if ws is None:
        ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale, head_lo, head_hi)
    if stream is not None:
        torch.cuda.synchronize()
    S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, head_lo, head_hi, tok_lo, tok_hi, out, lse, ws, b.scale,
                           window=window, sinks=sinks, stream=stream)
    return out, lse, ws


def leave_behind(b, window, sinks, spare=None):
    """Drops the pages that no new token sees: no page, or the id of one that holds NaN."""
    for r, (n, c) in enumerate(zip(b.q_lens, b.ctx)):
        first = c - n + 1 - window if n else c
        for j in range(-(-c // b.page)):
            if j * b.page >= sinks and (j + 1) * b.page <= first:
                b.table[r, j] = -1 if spare is None else spare


def spare_page(b):
    used = set(b.table.flatten().tolist())
    return next(i for i in range(b.pool.shape[0]) if i not in used)


def check(b, what, window, sinks, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16, behind=True):
    head_hi = b.heads if head_hi is None else head_hi
    if behind:
        leave_behind(b, window, sinks, spare_page(b) if behind == "nan" else None)
    out, lse, ws = run(b, window, sinks, head_lo, head_hi, tok_lo, tok_hi, dtype)
    assert S.splash_workspace_status(ws) == 0, what
    assert_chunk(b, out, lse, attention_reference(b, head_lo, head_hi, window, sinks, tok_lo, tok_hi), head_lo, head_hi, what)
    own = int(b.cu[-1])
    assert (out[own:] == 7).all() and (lse[own:] == 7).all(), what
    assert (out[:, :head_lo] == 7).all() and (out[:, head_hi:] == 7).all() and (lse[:, head_hi:] == 7).all(), what
    return out, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [1, 8, 16, 40, 64, 128])
def test_heads_and_pages(heads, page):
    check(Batch([1, 3, 0, 17, 1], [1, 130, 77, 300, 641], heads, page, heads + page, DEV, pad_rows=3),
          f"{heads} heads, pages of {page}", 100, 4, behind="nan")


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 192, 300, 2000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 63, 64, 65, 130, 500])
def test_windows_and_first_tokens(window, sinks):
    for page, behind in ((16, True), (64, "nan"), (128, "nan")):
        check(Batch([1, 2, 40], [700, 129, 333], 16, page, window + sinks, DEV), f"pages of {page}", window, sinks, behind=behind)


@pytest.mark.parametrize("n", [1, 64, 65, 127, 128, 129, 200, 257, 385])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (70, 4), (128, 64), (129, 3)])
def test_whole_prompts(n, window, sinks):
    check(Batch([n], [n], 16, 16, n, DEV), f"prompt of {n}", window, sinks)
    check(Batch([n], [n], 128, 64, n, DEV), f"prompt of {n}", window, sinks, dtype=torch.float32)


@pytest.mark.parametrize("heads", [65, 100, 129, 160, 256])
def test_odd_head_counts(heads):
    check(Batch([2, 5], [140, 459], heads, 64, heads, DEV), f"{heads} heads", 150, 4, dtype=torch.float32)


@pytest.mark.parametrize("lo,hi", [(0, 16), (16, 32), (112, 128), (3, 4), (5, 75), (64, 128)])
def test_head_slices(lo, hi):
    check(Batch([1, 6, 33], [90, 400, 228], 128, 64, 30, DEV, pad_rows=2), f"heads [{lo}, {hi})", 77, 5, lo, hi)


@pytest.mark.parametrize("tok_lo,tok_hi", [(0, 100), (100, -1), (64, 256), (77, 301), (300, 300), (5000, -1), (0, 0), (3, 70),
                                           (70, 80), (0, 331), (330, 332)])
@pytest.mark.parametrize("window,sinks", [(50, 4), (200, 100), (30, 0), (64, 64)])
def test_token_ranges(tok_lo, tok_hi, window, sinks):
    check(Batch([4, 40, 1], [333, 400, 90], 16, 64, 50, DEV), f"[{tok_lo}, {tok_hi})", window, sinks, 0, 16, tok_lo, tok_hi)


def test_shares_merge_to_the_whole():
    b = Batch([1, 90], [1000, 777], 128, 64, 51, DEV)
    cuts = [0, 256, 700, 2000]
    po, pl = torch.empty(3, b.rows, 128, 512, device=DEV), torch.empty(3, b.rows, 128, device=DEV)
    for i in range(3):
        po[i], pl[i], _ = run(b, 400, 70, 0, 128, cuts[i], cuts[i + 1], torch.float32)
    out, lse = torch.empty_like(po[0]), torch.empty_like(pl[0])
    S.splash_lse_merge(po, pl, out, lse)
    assert_chunk(b, out, lse, attention_reference(b, 0, 128, 400, 70), 0, 128, "merged")


@pytest.mark.parametrize("q,ctx,heads,window", [(1, 20000, 128, 15000), (3, 9001, 16, 8000), (2, 5000, 256, 4999),
                                                (300, 9000, 16, 2000)])
def test_few_rows_over_a_long_window_are_split(q, ctx, heads, window):
    check(Batch([q], [ctx], heads, 64, q, DEV), "split", window, 4, dtype=torch.float32)


def test_long_prompts_are_dealt():
    check(Batch([1100, 3], [1400, 2500], 128, 64, 41, DEV), "dealt", 333, 4)


def test_requests_past_one_batch_of_the_plan():
    n = 1100
    q = [(i * 7) % 3 for i in range(n)]
    check(Batch(q, [q[i] + (i * 37) % 150 for i in range(n)], 8, 16, 60, DEV), "1100 requests", 33, 2)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = random.Random(seed)
    heads, page = r.choice((8, 16, 24, 64, 128)), r.choice((16, 32, 64, 128))
    q = [r.choice((0, 1, 1, 5, r.randint(1, 150))) for _ in range(r.randint(1, 9))]
    ctx = [n + r.choice((0, r.randint(0, 90), r.randint(0, 1200))) for n in q]
    lo = r.choice((0, r.randint(0, heads - 1)))
    check(Batch(q, ctx, heads, page, seed, DEV), f"seed {seed}", r.choice((1, 31, 64, r.randint(1, 700))),
          r.choice((0, 1, 4, 64, r.randint(0, 300))), lo, heads, dtype=r.choice((torch.bfloat16, torch.float32)),
          behind=r.choice((True, "nan", False)))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 50), (704, 3), (10 ** 6, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_that_hide_nothing_are_the_plain_call(window, sinks):
    b = Batch([1, 30, 5], [700, 64, 129], 16, 64, 7, DEV)
    out, lse, ws = run(b, window, sinks)
    want, wl = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    S.splash_chunk_attn(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, 16, 0, -1, want, wl, ws, b.scale)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_first_tokens_that_cover_the_context():
    b = Batch([1, 30, 5], [700, 64, 129], 16, 64, 7, DEV)
    out, lse, _ = run(b, 1, 2 ** 31 - 1)
    assert_chunk(b, out, lse, chunk_reference(b, 0, 16), 0, 16)


def test_a_missing_page_is_flagged_only_where_it_is_needed():
    for page in (16, 64, 128):
        n_pages = -(-900 // page)
        for j in range(n_pages):
            b = Batch([3], [900], 16, page, 9, DEV)
            b.table[0, j] = b.pool.shape[0] + 5
            out, lse, ws = run(b, 130, 20)
            missing = [torch.zeros(900, dtype=torch.bool)]
            missing[0][j * page:(j + 1) * page] = True
            needed = j * page < 20 or (j + 1) * page > 898 - 130
            assert S.splash_workspace_status(ws) == (S.SPLASH_DEVICE_BAD_INPUT if needed else 0), (page, j)
            assert_chunk(b, out, lse, attention_reference(b, 0, 16, 130, 20, missing=missing), 0, 16, f"page {j} of {page}")


def test_growing_scores_rescale():
    b = Batch([5, 140], [900, 513], 128, 64, 61, DEV)
    for r in range(2):
        for j, t in enumerate(range(40, b.ctx[r], 130)):
            v = b.q[int(b.cu[r]), j % 128].float().cpu() * (0.5 + 0.25 * j)
            b.keys[r][t] = v.to(torch.bfloat16)
            b.pool[b.table[r, t // 64].item(), t % 64] = b.keys[r][t].to(DEV)
    check(b, "rescale", 300, 50, dtype=torch.float32)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 3.0])
def test_scales_of_every_sign(scale):
    check(Batch([3, 70], [400, 300], 16, 64, 3, DEV, scale=scale), f"scale {scale}", 100, 4)


def test_a_captured_call_replays_and_streams_run_side_by_side():
    b = Batch([1, 9, 140], [1000, 300, 500], 16, 64, 5, DEV)
    out, lse, ws = run(b, 200, 4)
    want = out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, b.scale, window=200, sinks=4)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    results = [run(b, 200, 4, stream=torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], want) and S.splash_workspace_status(r[2]) == 0 for r in results)


def test_a_workspace_serves_windowed_and_plain_calls():
    b = Batch([1, 300], [4000, 900], 128, 64, 8, DEV)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale)
    for window in (0, 100, 0, 3000):
        out, lse, _ = run(b, window, 4, ws=ws)
        assert_chunk(b, out, lse, attention_reference(b, 0, 128, window, 4), 0, 128, f"window {window}")


@pytest.mark.parametrize("page,heads", [(16, 16), (64, 128)])
def test_more_new_tokens_than_the_context_holds(page, heads):
    # the first rows lie before the first position and see nothing
    b = Batch([40, 3], [300, 90], heads, page, 21, DEV)
    b.ctx[0], b.keys[0] = 30, b.keys[0][:30]
    b.ctx_t[0] = 30
    for window, sinks in ((5, 2), (200, 0)):
        out, lse, ws = run(b, window, sinks)
        assert S.splash_workspace_status(ws) == 0 and (out[:10] == 0).all() and torch.isinf(lse[:10]).all()
        assert_chunk(b, out, lse, attention_reference(b, 0, heads, window, sinks), 0, heads, f"window {window}")


def test_refusals():
    b = Batch([1], [5], 8, 16, 1, DEV)
    for kw in (dict(window=-1, sinks=0), dict(window=5, sinks=-1)):
        with pytest.raises(S.SplashError):
            run(b, **kw)


def test_a_pool_past_32_bits():
    n = 60000                              # 4.4 GB
    b = Batch([1, 9, 130], [700, 333, 900], 16, 64, 60, DEV)
    few = b.pool.shape[0]
    pool = torch.zeros(n, 64, 576, dtype=torch.bfloat16, device=DEV)
    pool[n - few:] = b.pool
    b.pool, b.table = pool, torch.where(b.table < 0, b.table, b.table + (n - few))
    check(b, "the last pages of 4.4 GB", 200, 70)
