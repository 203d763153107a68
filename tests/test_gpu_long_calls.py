"""Chunk attention calls that take longer than a wait inside the kernel may (marked gpu)."""
import math

import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(seed)


def test_a_call_of_seconds_reports_no_timeout():
    # A prompt of 2.2 million tokens of one head, 5.3e15 operations: 3 s at the tensor cores' rate, and no wait
    # inside it is for more than a few key tiles.  Its pages repeat, so the 64-bit form needs each distinct
    # key once, times how often a token sees it.
    n, page, distinct = 2_200_000, 64, 64
    g = gen(1, DEV)
    pool = torch.randn(distinct, page, 576, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.empty(n, 1, 576, dtype=torch.bfloat16, device=DEV)
    for a in range(0, n, 200_000):
        q[a:a + 200_000] = torch.randn(min(200_000, n - a), 1, 576, generator=g, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = (torch.arange(-(-n // page), device=DEV) % distinct).to(torch.int32)[None].contiguous()
    cu, ctx = torch.tensor([0, n], **i32), torch.tensor([n], **i32)
    out, lse = torch.empty(n, 1, 512, device=DEV), torch.empty(n, 1, device=DEV)
    scale = 1 / math.sqrt(192.0)
    ws = S.chunk_workspace(q, pool, table, scale)
    S.splash_chunk_attn(q, pool, cu, table, ctx, 0, 1, 0, -1, out, lse, ws, scale)
    assert S.splash_workspace_status(ws) == 0
    rows = torch.cat((torch.tensor([0, 1, 127, 128, 4095, 4096, n // 2, n - 2, n - 1]),
                      torch.randint(0, n, (55,), generator=gen(2)))).to(DEV)
    k = pool.view(-1, 576).double()
    x = q[rows, 0].double()
    s = x @ k.T * scale
    seen = (rows + 1)[:, None]
    times = seen // len(k) + (torch.arange(len(k), device=DEV) < seen % len(k))
    s = s + times.double().log()                          # log 0: a key that the token does not see
    l = torch.logsumexp(s, -1)
    p = torch.exp(s - l[:, None])
    A = p @ k[:, :512].abs()
    # as chunk_reference derives it, and here the long sums: a product step of 16 keys is off by at most 2^-22 of
    # the sum so far, and a tile's sum of weights joins a row's with one rounding of 2^-24
    delta = 36 * 2.0 ** -22 * (x.abs() @ k.abs().T * scale).masked_fill(times == 0, 0).amax(-1)
    steps, tiles = seen[:, 0] / 16.0 + 1, seen[:, 0] / 128.0 + 1
    bound = A * (2.0 ** -8 + 2.0 ** -12 + 2 * delta + steps * 2.0 ** -22 + tiles * 2.0 ** -24)[:, None]
    assert ((out[rows, 0].double() - p @ k[:, :512]).abs() <= bound).all()
    assert ((lse[rows, 0].double() - l).abs() <= delta + tiles * 2.0 ** -24 + 2.0 ** -20 * (1 + l.abs())).all()


def test_an_item_of_seconds_reports_no_timeout():
    # A token over 268 million keys (repeated pages) for every pair of SMs: each pair's one row tile takes 3 s, and
    # the warps that store its results wait for all of it.  So many fp32 additions leave little of out's accuracy:
    # what counts is that the call ends with a result (lse within a rounding of 2^-24 for each of the 2^21 sums).
    n, page, distinct, heads = 1 << 28, 128, 32, 8
    B = max(1, torch.cuda.get_device_properties(0).multi_processor_count // 2)
    g = gen(3, DEV)
    pool = torch.randn(distinct, page, 576, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(B, heads, 576, generator=g, device=DEV).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = (torch.arange(n // page, device=DEV) % distinct).to(torch.int32)[None].repeat(B, 1)
    cu, ctx = torch.arange(B + 1, **i32), torch.full((B,), n, **i32)
    out, lse = torch.empty(B, heads, 512, device=DEV), torch.empty(B, heads, device=DEV)
    scale = 1 / math.sqrt(192.0)
    ws = S.chunk_workspace(q, pool, table, scale)
    S.splash_chunk_attn(q, pool, cu, table, ctx, 0, heads, 0, -1, out, lse, ws, scale)
    assert S.splash_workspace_status(ws) == 0
    s = q.double().view(-1, 576) @ pool.view(-1, 576).double().T * scale
    want = (torch.logsumexp(s, -1) + math.log(n // (page * distinct))).view(B, heads)
    assert torch.isfinite(out).all()
    assert ((lse.double() - want).abs() <= 2.0 ** 21 * 2.0 ** -24 + 2.0 ** -12).all()
