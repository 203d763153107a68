"""Rotary positions, writing the paged cache (bf16 and MXFP8) and reading MXFP8 pages back
(marked gpu), against the 64-bit forms of tests/serving_reference.py; and the serving step that
uses them together with the attention."""
import math

import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests import serving_reference as R
from tests.test_gpu_chunk import run as run_chunk

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
YARN = dict(base=10000.0, scaling="yarn", factor=40.0, orig_ctx=4096.0, amplitude=1.37)
LINEAR = dict(base=500000.0, scaling="linear", factor=8.0)
NONE = dict(base=10000.0)
POSITIONS = [0, 1, 2, 511, 4096, 131071, 1 << 20, (1 << 31) - 1, -1, -(1 << 31), 77, 1000003]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_rope(x, y, positions, interleaved, rope):
    ref = R.rotate(x, positions, interleaved, **rope)
    tol = R.rotate_bound(x, x.dtype, interleaved, positions=positions, **rope)
    got = y.detach().cpu().double().numpy()
    half = torch.finfo(x.dtype).eps / 2
    err = np.abs(got - ref)
    assert (err <= tol + half * (np.abs(ref) + tol)).all(), float((err - tol - half * np.abs(ref)).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rope", [YARN, LINEAR, NONE], ids=["yarn", "linear", "none"])
@pytest.mark.parametrize("dims,width", [(64, 192), (128, 128), (2, 2), (6, 11), (64, 67), (256, 256), (32, 40)])
def test_rope(dtype, interleaved, rope, dims, width):
    T, H = len(POSITIONS), 3
    x = torch.randn(T, H, width, generator=gen(dims + width)).to(dtype).to(DEV)[..., width - dims:]
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device=DEV)
    full = torch.full((T, H, dims + 5), 3.0, dtype=dtype, device=DEV)
    desc = S.make_rope_desc(dims, interleaved=interleaved, **rope)
    for off in (0, 5):                     # aligned where dims + 5 allows, never for the second
        y = full[..., off:off + dims]
        S.splash_rope(x, pos, y, desc)
        check_rope(x, y, pos, interleaved, rope)
        assert (full[..., :off] == 3).all() and (full[..., off + dims:] == 3).all()
        full.fill_(3.0)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (7, 128), (300, 5), (33, 1000)])
def test_rope_in_place_in_a_wider_head(T, H):
    q = torch.randn(T, H, 576, generator=gen(T)).to(torch.bfloat16).to(DEV)
    q0 = q.clone()
    pos = torch.randint(0, 200000, (T,), generator=gen(H), dtype=torch.int32).to(DEV)
    desc = S.make_rope_desc(64, **YARN)
    S.splash_rope(q[..., 512:], pos, q[..., 512:], desc)
    check_rope(q0[..., 512:], q[..., 512:], pos, True, YARN)
    assert torch.equal(q[..., :512], q0[..., :512])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,dims,width", [(3001, 1, 64, 576), (5000, 5, 6, 7), (2500, 2, 256, 256), (70001, 1, 32, 32)])
def test_rope_of_many_tokens_with_few_heads(dtype, interleaved, T, H, dims, width):
    x = torch.randn(T, H, width, generator=gen(T)).to(dtype).to(DEV)
    x0 = x.clone()
    pos = torch.randint(-1000, 200000, (T,), generator=gen(H), dtype=torch.int32).to(DEV)
    v = x[..., width - dims:]
    S.splash_rope(v, pos, v, S.make_rope_desc(dims, interleaved=interleaved, **YARN))
    check_rope(x0[..., width - dims:], v, pos, interleaved, YARN)
    assert torch.equal(x[..., :width - dims], x0[..., :width - dims])


def test_rope_head_major_and_undone():
    x = torch.randn(5, 40, 128, generator=gen(3)).to(DEV).transpose(0, 1)     # [40 tokens][5 heads], heads outermost
    pos = torch.arange(40, dtype=torch.int32, device=DEV) * 30011
    y = torch.empty(5, 40, 128, device=DEV).transpose(0, 1)
    desc = S.make_rope_desc(128, interleaved=False, **LINEAR)
    S.splash_rope(x, pos, y, desc)
    check_rope(x, y, pos, False, LINEAR)
    S.splash_rope(y, -pos, y, desc)
    # two rotations, each off by at most 6 * 2^-24 of the pair's magnitudes plus its rounding
    assert float((y - x).abs().max()) <= 16 * 2.0 ** -24 * 2 * float(x.abs().max())


def test_rope_empty():
    desc = S.make_rope_desc(64)
    for T, H in ((0, 4), (4, 0)):
        x = torch.empty(T, H, 64, dtype=torch.bfloat16, device=DEV)
        S.splash_rope(x, torch.empty(T, dtype=torch.int32, device=DEV), x, desc)


def test_rope_refusals():
    desc = S.make_rope_desc(64)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    for args in ((x, pos.long(), x), (x, pos[:2], x), (x.double(), pos, x.double()), (x, pos, x.float()),
                 (x[..., :32], pos, x[..., :32]), (x[0], pos, x[0]), (x.transpose(1, 2), pos, x.transpose(1, 2)),
                 (x, pos.cpu(), x), (x, pos, x[:, :2])):
        with pytest.raises(ValueError):
            S.splash_rope(*args, desc)
    with pytest.raises(S.SplashError) as e:      # every token writes the same rows
        S.splash_rope(x, pos, x[:1].expand(3, 4, 64), desc)
    assert e.value.code == S.SPLASH_ERR_INVALID_ARG


def test_rope_many_heads_on_another_stream():
    x = torch.randn(17, 4099, 64, generator=gen(9)).to(torch.float16).to(DEV)
    pos = torch.arange(17, dtype=torch.int32, device=DEV)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    S.splash_rope(x, pos, y, S.make_rope_desc(64, interleaved=False), stream=s)
    s.synchronize()
    check_rope(x, y, pos, False, NONE)


# ------------------------------------------------------------------ the cache

def lengths(kind):
    if kind == "decode":
        return [1] * 300, [(i * 53) % 700 + 1 for i in range(300)]
    if kind == "prompts":
        return [70, 1, 0, 333], [70, 1, 9, 333]
    return [5, 0, 129, 64, 1], [40, 12, 500, 64, 257]


def batch(kind, page, seed, pad=2):
    q, ctx = lengths(kind)
    return R.Batch(q, ctx, 1, page, seed, DEV, pad_rows=pad)


def new_slots(b):
    """(row, request, position) of every new token."""
    row = 0
    for r, (n, c) in enumerate(zip(b.q_lens, b.ctx)):
        for i in range(n):
            yield row + i, r, c - n + i
        row += n


def latents(n, seed):
    x = torch.randn(n, 512, generator=gen(seed)) * torch.exp(3 * torch.randn(n, 16, generator=gen(seed + 1))).repeat_interleave(32, 1)
    x[0, :32] = 0
    x[0, 32:64] = 2.0 ** -133                                     # the least bf16
    x[0, 64:96] = torch.finfo(torch.bfloat16).max
    x[0, 96:128] = torch.arange(32) * 2.0 ** -130
    x[0, 128:160] = 448.0
    x[0, 160:192] = 450.0
    x[0, 192:224] = torch.linspace(-1, 1, 32)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("kind", ["decode", "prompts", "mixed"])
@pytest.mark.parametrize("interleaved,rope", [(True, YARN), (False, NONE), (True, None)])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_append(page, kind, interleaved, rope, fmt):
    b = batch(kind, page, 7 + page)
    n = b.rows
    wide = torch.zeros(n, 600, dtype=torch.bfloat16)
    wide[:, :512] = latents(n, page)
    wide[:, 512:576] = torch.randn(n, 64, generator=gen(5)).to(torch.bfloat16)
    wide = wide.to(DEV)
    lat, kr = wide[:, :512], wide[:, 512:576]                      # strided rows
    if fmt == "bf16":
        pool = b.pool.clone()
    else:
        pool = torch.randint(0, 255, (b.pool.shape[0], page, 656), generator=gen(6), dtype=torch.uint8).to(DEV)
    want = pool.clone().cpu()
    desc = S.make_rope_desc(64, interleaved=interleaved, **rope) if rope else None
    S.splash_kv_append(lat, kr, b.cu, b.table, b.ctx_t, pool, desc)
    got = pool.cpu()
    slots = list(new_slots(b))
    rows = torch.tensor([s[0] for s in slots])
    pos = torch.tensor([s[2] for s in slots], dtype=torch.int32)
    page_ids = torch.tensor([int(b.table[r, p // page]) for _, r, p in slots])
    off = pos.long() % page
    k = kr.cpu()[rows]
    rotated = got[page_ids, off][:, -64:] if fmt == "bf16" else got[page_ids, off][:, 528:].contiguous().view(torch.bfloat16)
    if rope:
        check_rope(k[:, None], rotated[:, None], pos, interleaved, rope)
    else:
        assert torch.equal(rotated, k)
    if fmt == "bf16":
        want[page_ids, off] = torch.cat((lat.cpu()[rows], rotated), 1)
    else:
        codes, scales = R.pack_rows(lat.cpu()[rows])
        want[page_ids, off] = torch.cat((torch.from_numpy(codes), torch.from_numpy(scales),
                                         rotated.contiguous().view(torch.uint8)), 1)
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))        # every other slot as it was


def test_append_non_finite_latents():
    b = batch("prompts", 64, 9, pad=0)
    x = latents(b.rows, 3)
    x[1, 0], x[1, 40], x[1, 41] = math.nan, math.inf, -math.inf
    x[2, 64:96] = math.nan
    pool = torch.zeros(b.pool.shape[0], 64, 656, dtype=torch.uint8, device=DEV)
    S.splash_kv_append(x.to(DEV), torch.zeros(b.rows, 64, dtype=torch.bfloat16, device=DEV), b.cu, b.table, b.ctx_t, pool)
    codes, scales = R.pack_rows(x)
    for row, r, p in new_slots(b):
        got = pool[int(b.table[r, p // 64]), p % 64].cpu().numpy()
        nan = np.isnan(x[row].double().numpy())
        assert np.array_equal(got[:512][~nan], codes[row][~nan]) and ((got[:512][nan] & 0x7F) == 0x7F).all()
        assert np.array_equal(got[512:528], scales[row])


def test_append_skips_what_it_cannot_place():
    b = batch("mixed", 64, 11, pad=0)
    pool = b.pool.clone()
    lat = torch.randn(b.rows, 512, generator=gen(1)).to(torch.bfloat16).to(DEV)
    kr = torch.randn(b.rows, 64, generator=gen(2)).to(torch.bfloat16).to(DEV)
    b.table[0].fill_(-1)
    b.table[3].fill_(pool.shape[0])
    b.ctx_t[2], b.ctx_t[4] = 1 << 30, 0
    S.splash_kv_append(lat, kr, b.cu, b.table, b.ctx_t, pool)
    assert torch.equal(pool.view(torch.int16), b.pool.view(torch.int16))


def test_append_many_requests_finds_each():
    n = 2500                                # more than 32 x 32: three steps of the search; empty requests between
    q = [(i * 5) % 4 for i in range(n)]
    b = R.Batch(q, [x + i % 9 for i, x in enumerate(q)], 1, 16, 12, DEV)
    lat = torch.randn(b.rows, 512, generator=gen(1)).to(torch.bfloat16).to(DEV)
    kr = torch.randn(b.rows, 64, generator=gen(2)).to(torch.bfloat16).to(DEV)
    pool, want = b.pool.clone(), b.pool.cpu().clone()
    S.splash_kv_append(lat, kr, b.cu, b.table, b.ctx_t, pool)
    table = b.table.cpu()
    rows = torch.cat((lat, kr), 1).cpu()
    for row, r, p in new_slots(b):
        want[table[r, p // 16], p % 16] = rows[row]
    assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("page", [16, 64, 128, 5])
def test_unpack_every_code_and_scale(page):
    n = 9
    src = torch.randint(0, 256, (n, page, 656), generator=gen(page), dtype=torch.uint8)
    flat = src.view(-1, 656)
    flat[: min(len(flat), 16), :512] = torch.arange(512).to(torch.uint8)
    flat[0, 512:528] = torch.arange(16, dtype=torch.uint8)
    flat[1, 512:528] = torch.arange(240, 256).to(torch.uint8)
    src = src.to(DEV)
    dst = torch.full((n + 2, page, 576), 5.0, dtype=torch.bfloat16, device=DEV)
    sid = torch.tensor([3, 0, 8, 1, -1, n, 2], dtype=torch.int32, device=DEV)
    did = torch.tensor([1, 10, 4, 0, 2, 3, n + 2], dtype=torch.int32, device=DEV)
    S.splash_kv_unpack(src, dst, sid, did)
    # one rounding to bf16 (exact but for values past its range): through fp32, as fp64 has no direct cast
    want = torch.full_like(dst, 5.0, device="cpu")
    ref = torch.from_numpy(R.unpack_rows(src)).float().to(torch.bfloat16)
    for s, d in ((3, 1), (0, 10), (8, 4), (1, 0)):
        want[d] = ref[s]
    got = dst.cpu()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])


def test_cache_refusals():
    b = batch("mixed", 64, 13, pad=0)
    n = b.rows
    lat, kr = torch.zeros(n, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(n, 64, dtype=torch.bfloat16, device=DEV)
    ok = dict(latent=lat, k_rope=kr, cu_q=b.cu, block_table=b.table, ctx_lens=b.ctx_t, kv_pool=b.pool)
    for kw in (dict(latent=lat.float()), dict(k_rope=kr[:-1]), dict(latent=lat[:, :511]), dict(cu_q=b.cu[:-1]),
               dict(cu_q=b.cu.long()), dict(block_table=b.table[0]), dict(kv_pool=b.pool.float()),
               dict(kv_pool=b.pool[..., :575]), dict(kv_pool=b.pool.view(torch.uint8)), dict(ctx_lens=b.ctx_t.cpu())):
        with pytest.raises(ValueError):
            S.splash_kv_append(**{**ok, **kw})
    with pytest.raises(S.SplashError):
        S.splash_kv_append(**{**ok, "kv_pool": torch.zeros(3, 48, 576, dtype=torch.bfloat16, device=DEV)})
    src = torch.zeros(2, 64, 656, dtype=torch.uint8, device=DEV)
    dst = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(1, dtype=torch.int32, device=DEV)
    for args in ((src, dst, ids.long(), ids), (src, dst, ids, ids[:0]), (dst, dst, ids, ids), (src, src, ids, ids),
                 (src, dst[:, :32], ids, ids), (src, dst.cpu(), ids, ids)):
        with pytest.raises(ValueError):
            S.splash_kv_unpack(*args)


def test_unpack_one_source_page_twice_and_bad_ids():
    src = torch.randint(0, 256, (4, 16, 656), generator=gen(5), dtype=torch.uint8).to(DEV)
    dst = torch.full((6, 16, 576), 5.0, dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    S.splash_kv_unpack(src, dst, torch.tensor([2, 2, -1, 4, 1, 0], **i32), torch.tensor([5, 0, 1, 2, 6, -1], **i32))
    want = torch.from_numpy(R.unpack_rows(src[2])).float().to(torch.bfloat16)
    for page in (0, 5):
        assert torch.equal(dst[page].cpu().nan_to_num(nan=1.0), want.nan_to_num(nan=1.0))
    assert (dst[1:5] == 5).all()


def test_unaligned_unpack_target():
    src = torch.randint(0, 256, (3, 16, 656), generator=gen(4), dtype=torch.uint8).to(DEV)
    raw = torch.zeros(3 * 16 * 576 + 8, dtype=torch.bfloat16, device=DEV)
    ids = torch.arange(3, dtype=torch.int32, device=DEV)
    a, c = raw[8:].view(3, 16, 576), torch.zeros(3, 16, 576, dtype=torch.bfloat16, device=DEV)   # 16 bytes off
    S.splash_kv_unpack(src, a, ids, ids)
    S.splash_kv_unpack(src, c, ids, ids)
    assert torch.equal(a.view(torch.int16), c.view(torch.int16)) and (raw[:8] == 0).all()


def test_pools_past_two_to_the_31_bytes():
    n = 60000
    src = torch.empty(n, 64, 656, dtype=torch.uint8, device=DEV)       # 2.5 GB
    dst = torch.empty(n, 64, 576, dtype=torch.bfloat16, device=DEV)    # 4.4 GB
    lat = latents(64, 8).to(DEV)
    kr = torch.randn(64, 64, generator=gen(2)).to(torch.bfloat16).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu, ctx, table = torch.tensor([0, 64], **i32), torch.tensor([64], **i32), torch.tensor([[n - 1]], **i32)
    S.splash_kv_append(lat, kr, cu, table, ctx, src)
    S.splash_kv_append(lat, kr, cu, table, ctx, dst)
    assert torch.equal(dst[n - 1].view(torch.int16), torch.cat((lat, kr), 1).view(torch.int16))
    S.splash_kv_unpack(src, dst, torch.tensor([n - 1], **i32), torch.tensor([n - 2], **i32))
    ref = torch.from_numpy(R.unpack_rows(src[n - 1])).float().to(torch.bfloat16)
    assert torch.equal(dst[n - 2].cpu(), ref)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_serving_step(fmt):
    """Prompt, then single tokens: rotate the queries, write the keys, attend; the quantised cache
    is migrated to a second pool and read back first.  Captured as one graph and replayed."""
    H, page, scale = 128, 64, 1 / math.sqrt(192.0)
    desc = S.make_rope_desc(64, **YARN)
    q_lens, B = [200, 37, 64], 3
    pages = 5
    table = torch.randperm(16, generator=gen(1))[:B * pages].view(B, pages).to(torch.int32).to(DEV)
    width, dt = (576, torch.bfloat16) if fmt == "bf16" else (656, torch.uint8)
    pool = torch.zeros(16, page, width, dtype=dt, device=DEV)
    held = []                                # (latent, rotated rope) per request, as the cache holds them
    ids = torch.arange(16, dtype=torch.int32, device=DEV)
    for step in range(2):
        n = q_lens if step == 0 else [1] * B
        ctx = q_lens if step == 0 else [x + 1 for x in q_lens]
        N = sum(n)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        ctx_t = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        pos = torch.cat([torch.arange(c - m, c) for m, c in zip(n, ctx)]).to(torch.int32).to(DEV)
        q0 = torch.randn(N, H, 576, generator=gen(step)).to(torch.bfloat16).to(DEV)
        kv = torch.randn(N, 576, generator=gen(10 + step)).to(torch.bfloat16).to(DEV)
        q, out = torch.empty_like(q0), torch.empty(N, H, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(N, H, device=DEV)
        plain = pool if fmt == "bf16" else torch.zeros(16, page, 576, dtype=torch.bfloat16, device=DEV)
        parked = torch.zeros_like(pool)
        ws = S.chunk_workspace(q, plain, table, scale)

        def once():
            q.copy_(q0)
            S.splash_rope(q[..., 512:], pos, q[..., 512:], desc)
            S.splash_kv_append(kv[:, :512], kv[:, 512:], cu, table, ctx_t, pool, desc)
            if fmt == "mxfp8":
                S.splash_kv_migrate(pool, parked, ids, ids)
                S.splash_kv_unpack(parked, plain, ids, ids)
            S.splash_chunk_attn(q, plain, cu, table, ctx_t, 0, H, 0, -1, out, lse, ws, scale)
        once()
        torch.cuda.synchronize()
        first = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            once()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        # the reference works on the values that the cache holds
        b = R.Batch(n, ctx, H, page, 0, DEV)
        b.q, b.cu = q, cu
        if fmt == "bf16":
            values = pool.cpu().double().numpy()
        else:
            values = R.unpack_rows(pool)
        t = table.cpu().numpy()
        b.keys = [torch.from_numpy(values[t[r]].reshape(-1, 576)[:ctx[r]]) for r in range(B)]
        R.assert_chunk(b, out, lse, R.chunk_reference(b, 0, H), 0, H, f"step {step}")
        # and the cache holds what the new tokens say
        row = 0
        for r in range(B):
            k = kv[row:row + n[r]]
            lat = k[:, :512].cpu()
            got = b.keys[r][ctx[r] - n[r]:]
            if fmt == "bf16":
                assert torch.equal(got[:, :512], lat.double())
            else:
                codes, scales = R.pack_rows(lat)
                rows = torch.cat((torch.from_numpy(codes), torch.from_numpy(scales), torch.zeros(n[r], 128, dtype=torch.uint8)), 1)
                assert np.array_equal(R.unpack_rows(rows)[:, :512], got[:, :512].numpy())
            check_rope(k[:, None, 512:].cpu(), got[:, None, 512:].to(torch.bfloat16), pos[row:row + n[r]].cpu(), True, YARN)
            row += n[r]
