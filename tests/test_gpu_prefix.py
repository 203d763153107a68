"""Attention of requests that share the pages of a prefix (marked gpu), against the 64-bit form of
tests/more_reference.py, which knows nothing of groups."""
import random

import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.more_reference import attention_reference
from tests.serving_reference import Batch, assert_chunk

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def shared(groups, heads, page, seed, only_first=False, **kw):
    """A batch of groups (prefix, [(new tokens, tokens between the prefix and them), ...]); prefix 0: requests of their own.
    Whole pages of a prefix are the first request's; the page in which it ends is each request's own.
    only_first: the other requests' entries for the shared pages are missing."""
    q = [n for _, rs in groups for n, _ in rs]
    b = Batch(q, [p + past + n for p, rs in groups for n, past in rs], heads, page, seed, DEV, **kw)
    r = 0
    b.cu_groups, b.prefix = [0], []
    for p, rs in groups:
        first, whole = r, p // page
        for r in range(first + 1, first + len(rs)):
            b.keys[r][:p] = b.keys[first][:p]
            b.pool[b.table[r, :whole].long()] = float("nan")
            b.table[r, :whole] = -1 if only_first else b.table[first, :whole]
            if p % page:
                b.pool[b.table[r, whole].item(), :p % page] = b.keys[first][whole * page:p].to(DEV)
        r = first + len(rs)
        b.cu_groups.append(r)
        b.prefix.append(p)
    b.cu_groups, b.prefix = ints(b.cu_groups), ints(b.prefix)
    return b


def run(b, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16, ws=None, groups=True, stream=None):
    head_hi = b.heads if head_hi is None else head_hi
    out = torch.full((b.rows, b.heads, 512), 7.0, dtype=dtype, device=b.device)
    lse = torch.full((b.rows, b.heads), 7.0, device=b.device)
    if ws is None:
        ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale, head_lo, head_hi, num_groups=b.prefix.numel())
        ws.fill_(0xff)                             # (nothing in it is taken for granted)
    if stream is not None:
        torch.cuda.synchronize()
    S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, head_lo, head_hi, tok_lo, tok_hi, out, lse, ws, b.scale,
                           cu_groups=b.cu_groups if groups else None, prefix_lens=b.prefix if groups else None,
                           stream=stream)
    return out, lse, ws


def check(b, what, head_lo=0, head_hi=None, tok_lo=0, tok_hi=-1, dtype=torch.bfloat16):
    head_hi = b.heads if head_hi is None else head_hi
    out, lse, ws = run(b, head_lo, head_hi, tok_lo, tok_hi, dtype)
    assert S.splash_workspace_status(ws) == 0, what
    assert_chunk(b, out, lse, attention_reference(b, head_lo, head_hi, tok_lo=tok_lo, tok_hi=tok_hi), head_lo, head_hi, what)
    own = int(b.cu[-1])
    assert (out[own:] == 7).all() and (lse[own:] == 7).all(), what
    assert (out[:, :head_lo] == 7).all() and (out[:, head_hi:] == 7).all() and (lse[:, head_hi:] == 7).all(), what
    return out, lse


SINGLE = lambda m, past=5: [(1, (past + 37 * i) % 400) for i in range(m)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [1, 8, 16, 24, 40, 64, 100, 128])
def test_heads_and_pages(heads, page):
    check(shared([(1024, SINGLE(24)), (0, [(3, 100)]), (1152, SINGLE(9, 2))], heads, page, heads + page, pad_rows=3),
          f"{heads} heads, pages of {page}")


@pytest.mark.parametrize("heads,lo,hi", [(128, 16, 32), (128, 0, 8), (128, 100, 125), (128, 32, 96), (64, 63, 64), (128, 3, 128)])
def test_head_slices(heads, lo, hi):
    check(shared([(1500, SINGLE(33))], heads, 64, lo, pad_rows=2), f"heads [{lo}, {hi})", lo, hi)


@pytest.mark.parametrize("heads,lo,hi", [(16, 0, 16), (128, 16, 32), (128, 64, 96)])
def test_the_prefix_is_read_through_the_first_request(heads, lo, hi):
    # (a prefix of 8,192 keys of 64 single tokens is worth it; the other requests have no pages for it)
    check(shared([(8192, SINGLE(64))], heads, 64, 5, only_first=True), "first request's pages", lo, hi)
    check(shared([(8200, SINGLE(64))], heads, 64, 6, only_first=True), "first request's pages", lo, hi, dtype=torch.float32)


@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 127, 128, 129, 500, 640, 1000, 1023, 1025, 2049])
def test_prefixes_of_every_length(prefix):
    for page in (16, 64, 128):
        check(shared([(prefix, SINGLE(50))], 16, page, prefix, pad_rows=1), f"prefix of {prefix}, pages of {page}")


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 30])
@pytest.mark.parametrize("heads", [8, 16, 40])
def test_several_new_tokens(n, heads):
    r = random.Random(n)
    reqs = [(r.randint(1, n), r.randint(0, 300)) for _ in range(20)]
    check(shared([(1000, reqs), (2000, reqs[:7])], heads, 16, n), f"up to {n} tokens", dtype=torch.float32)


def test_nothing_between_the_prefix_and_the_new_tokens():
    check(shared([(1024, [(1, 0)] * 40), (777, [(2, 0)] * 30)], 16, 64, 3), "first step after the prefix")


def test_groups_with_requests_without_new_tokens():
    check(shared([(1024, [(0, 3), (1, 9), (0, 70), (2, 0)] * 8), (2000, [(0, 5)] * 6), (900, SINGLE(30))], 16, 16, 4), "idle requests")


def test_one_group_per_request_and_empty_ones():
    b = shared([(300, [(1, 5)]) for _ in range(40)], 16, 64, 9)
    check(b, "groups of one")
    b = shared([(1024, SINGLE(30)), (1024, SINGLE(20))], 16, 64, 10)
    b.cu_groups, b.prefix = ints([0, 0, 30, 30, 30, 50, 50]), ints([5, 1024, 9, 77, 1024, 3])
    check(b, "empty groups")
    b.cu_groups, b.prefix = ints([30, 50]), ints([1024])
    check(b, "requests before the groups")
    b.cu_groups, b.prefix = ints([0, 30]), ints([1024])
    check(b, "requests behind the groups")
    b.cu_groups, b.prefix = ints([0, 30, 50]), ints([700, 1024])
    check(b, "less than what is shared")


@pytest.mark.parametrize("tok_lo,tok_hi", [(0, 100), (100, -1), (1000, 1100), (1024, -1), (1030, -1), (0, 1024), (500, 1024),
                                           (5000, -1), (300, 300), (0, 1050), (77, 1300)])
def test_token_ranges(tok_lo, tok_hi):
    check(shared([(1024, SINGLE(40)), (0, [(5, 60)]), (1111, SINGLE(30))], 16, 64, 50), f"[{tok_lo}, {tok_hi})", 0, 16, tok_lo, tok_hi)


def test_shares_merge_to_the_whole():
    b = shared([(2000, SINGLE(40))], 16, 64, 51)
    cuts = [0, 600, 2010, 5000]
    po, pl = torch.empty(3, b.rows, 16, 512, device=DEV), torch.empty(3, b.rows, 16, device=DEV)
    for i in range(3):
        po[i], pl[i], _ = run(b, 0, 16, cuts[i], cuts[i + 1], torch.float32)
    out, lse = torch.empty_like(po[0]), torch.empty_like(pl[0])
    S.splash_lse_merge(po, pl, out, lse)
    assert_chunk(b, out, lse, attention_reference(b, 0, 16), 0, 16, "merged")


def test_many_row_tiles_are_dealt():
    # more row tiles than an even cut takes, with and without cuts of their own
    check(shared([(640, [(1, i % 50) for i in range(700)])], 8, 16, 60), "700 requests")
    check(shared([(1280, [(1, i % 50) for i in range(300)]), (1000, [(2, 7)] * 290)], 40, 64, 61), "590 requests")


def test_many_groups():
    check(shared([(700, [(1, i % 40), (1, 9), (1, 60)]) for i in range(200)], 16, 16, 62), "200 groups")
    check(shared([(512, [(1, i % 40), (1, 9)]) for i in range(600)], 8, 16, 63), "600 groups")


def test_a_long_prefix_is_cut():
    check(shared([(30000, SINGLE(20))], 16, 64, 64), "cut", dtype=torch.float32)


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    r = random.Random(seed)
    heads, page = r.choice((8, 16, 24, 40, 64, 90)), r.choice((16, 32, 64, 128))
    groups = []
    for _ in range(r.randint(1, 5)):
        n = r.choice((1, 1, 3, 12))
        groups.append((r.choice((0, r.randint(1, 300), r.randint(300, 3000))),
                       [(r.randint(0, n), r.choice((0, r.randint(0, 400)))) for _ in range(r.randint(1, 40))]))
    lo = r.choice((0, r.randint(0, heads - 1)))
    check(shared(groups, heads, page, seed), f"seed {seed}", lo, heads, dtype=r.choice((torch.bfloat16, torch.float32)))


def test_growing_scores_rescale():
    b = shared([(900, SINGLE(24))], 16, 64, 70)
    for j, t in enumerate(range(40, 900, 130)):            # in the prefix, along the queries of the first request
        b.keys[0][t] = (b.q[0, j % 16].float().cpu() * (0.5 + 0.25 * j)).to(torch.bfloat16)
        for r in range(24):
            b.keys[r][t] = b.keys[0][t]
            b.pool[b.table[r, t // 64].item(), t % 64] = b.keys[0][t].to(DEV)
    check(b, "rescale", dtype=torch.float32)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 3.0])
def test_scales_of_every_sign(scale):
    check(shared([(1000, SINGLE(40))], 16, 64, 3, scale=scale), f"scale {scale}")


# ------------------------------------------------------------------ input that does not hold together

def test_bad_groups_leave_the_call_without_work():
    b = shared([(1024, SINGLE(40))], 16, 64, 80)
    for cu in ([5, 3], [-1, 40], [0, 41], [0, 2 ** 31 - 1]):
        b.cu_groups = ints(cu)
        out, lse, ws = run(b)
        assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT and (out == 7).all() and (lse == 7).all(), cu


def test_bad_prefixes_are_flagged():
    b = shared([(1024, SINGLE(40)), (512, SINGLE(40))], 16, 64, 81)
    for p in (-1, 2 ** 31 - 1, -2 ** 31, 1030):            # (the first request has 1,029 tokens before its new one)
        b.prefix = ints([p, 512])
        out, lse, ws = run(b)
        assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT, p
        ref = attention_reference(b, 0, 16)                # the other group's rows stand
        assert_rows(b, out, lse, ref, 40)


def assert_rows(b, out, lse, ref, first):
    o, want, bound = out[first:].double(), ref[0][first:], ref[2][first:]
    assert ((o - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all()


def test_a_missing_page_of_the_prefix_is_flagged():
    b = shared([(8192, SINGLE(64))], 16, 64, 82)
    b.table[:, 3] = b.pool.shape[0]
    out, lse, ws = run(b)
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
    missing = [torch.zeros(c, dtype=torch.bool) for c in b.ctx]
    for m in missing:
        m[192:256] = True
    assert_chunk(b, out, lse, attention_reference(b, 0, 16, missing=missing), 0, 16)


# ------------------------------------------------------------------ calls around them

def test_equal_calls_give_equal_bits_captured_and_on_streams():
    b = shared([(3000, SINGLE(64)), (1000, [(3, 9)] * 20)], 16, 64, 90)
    out, lse, ws = run(b)
    want, wl = out.clone(), lse.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, b.scale,
                               cu_groups=b.cu_groups, prefix_lens=b.prefix)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    results = [run(b, stream=torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], want) for r in results)


def test_a_workspace_serves_calls_with_and_without_groups():
    b = shared([(2000, SINGLE(64)), (0, [(100, 9)])], 16, 64, 91)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale, num_groups=2)
    ref = attention_reference(b, 0, 16)
    for groups in (True, False, True, True, False):
        out, lse, _ = run(b, ws=ws, groups=groups)
        assert S.splash_workspace_status(ws) == 0
        assert_chunk(b, out, lse, ref, 0, 16, f"groups {groups}")


def test_all_heads_of_128_are_the_plain_call():
    b = shared([(1500, SINGLE(20))], 128, 64, 92)
    out, lse, ws = run(b)
    want, wl, _ = run(b, ws=ws, groups=False)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_calls_without_requests_or_tokens_clear_the_status():
    b = shared([(1024, SINGLE(40))], 16, 64, 94)
    good, ws = b.cu_groups, None
    b.cu_groups = ints([5, 3])
    _, _, ws = run(b)
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT
    S.splash_chunk_attn_ex(b.q[:0], b.pool, torch.zeros_like(b.cu), b.table, b.ctx_t, 0, 16, 0, -1,
                           torch.empty(0, 16, 512, device=DEV), torch.empty(0, 16, device=DEV), ws, b.scale, cu_groups=good,
                           prefix_lens=b.prefix)
    assert S.splash_workspace_status(ws) == 0
    S.splash_chunk_attn_ex(b.q, b.pool, b.cu[:1], b.table[:0], b.ctx_t[:0], 0, 16, 0, -1,
                           torch.empty(b.rows, 16, 512, device=DEV), torch.empty(b.rows, 16, device=DEV), ws, b.scale,
                           cu_groups=ints([0, 0]), prefix_lens=ints([64]))
    assert S.splash_workspace_status(ws) == 0


def test_as_many_groups_as_there_can_be():
    b = shared([(512, SINGLE(40)), (800, SINGLE(40, 1))], 16, 64, 95)
    b.cu_groups, b.prefix = ints([0] * 1023 + [40, 80]), ints([9] * 1022 + [512, 800])
    check(b, "1,024 groups")


def test_refusals():
    b = shared([(100, SINGLE(4))], 16, 64, 93)
    small = S.chunk_workspace(b.q, b.pool, b.table, b.scale)
    with pytest.raises(S.SplashError, match="WORKSPACE"):
        run(b, ws=small)
    out, lse, ws = run(b)
    with pytest.raises(ValueError, match="belong together"):
        S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, 1.0, cu_groups=b.cu_groups)
    call = lambda **kw: S.splash_chunk_attn_ex(b.q, b.pool, b.cu, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, 1.0, **kw)
    with pytest.raises(ValueError, match="cu_groups"):
        call(cu_groups=b.prefix, prefix_lens=b.prefix)
    with pytest.raises(ValueError, match="prefix_lens"):
        call(cu_groups=b.cu_groups, prefix_lens=b.prefix.long())
    with pytest.raises(S.SplashError, match="UNSUPPORTED"):
        call(cu_groups=b.cu_groups, prefix_lens=b.prefix, window=5)
    with pytest.raises(S.SplashError, match="UNSUPPORTED"):
        call(cu_groups=torch.zeros(1026, dtype=torch.int32, device=DEV), prefix_lens=torch.zeros(1025, dtype=torch.int32, device=DEV))


def test_a_pool_past_32_bits():
    n = 60000                              # 4.4 GB
    b = shared([(1000, SINGLE(33)), (2048, [(4, 7), (2, 90), (1, 0)])], 16, 64, 96)
    few = b.pool.shape[0]
    pool = torch.zeros(n, 64, 576, dtype=torch.bfloat16, device=DEV)
    pool[n - few:] = b.pool
    b.pool, b.table = pool, torch.where(b.table < 0, b.table, b.table + (n - few))
    check(b, "the last pages of 4.4 GB")
