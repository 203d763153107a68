"""RMS norm with rotary positions of query and key rows (marked gpu), against the same formula in 64
bits."""
import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests import serving_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def reference(x, w, positions, rope_kw, dims, eps, n, lo, offset=0.0, interleaved=True):
    """(y, bound) in 64 bits.  bound: the sum of squares adds at most 37 terms one after the other in fp32 (a lane's 32 and 5
    exchanges), half of whose relative error the root keeps: 18.5 steps of 2^-24; the products with 1 / n and the
    root (2 ulp), the sums with eps and the offset and the two products with x add under 11.  So z is off by 30 * 2^-24 of
    itself, and a rotation by that of both of its terms beside its own error."""
    x = x.detach().cpu().double()
    z = x.clone()
    p = x[..., :n].square().mean(-1, keepdim=True)
    g = torch.ones(n, dtype=torch.float64) if w is None else w.detach().cpu().double() + offset
    z[..., :n] = x[..., :n] / torch.sqrt(p + np.float32(eps).astype(np.float64)) * g
    bound = z.abs() * 30 * 2.0 ** -24
    bound[..., n:] = 0
    y, bound = z.numpy().copy(), bound.numpy()
    if dims:
        part = z[..., lo:lo + dims]
        y[..., lo:lo + dims] = R.rotate(part, positions, interleaved, **rope_kw)
        bound[..., lo:lo + dims] = R.rotate_bound(part, torch.float32, interleaved, positions=positions, **rope_kw) * 6
    return y, bound


def make(shape, dtype, seed, lead=0, pad=0):
    """Random rows inside a wider buffer: `lead` elements before the first and `pad` behind each row."""
    g = torch.Generator().manual_seed(seed)
    T, H, D = shape
    buf = (torch.randn(T * H * (D + pad) + lead, generator=g) * 2).to(dtype).to(DEV)
    return torch.as_strided(buf, shape, (H * (D + pad), D + pad, 1), lead)


def compare(y, want, bound, what=""):
    y = y.detach().cpu().double().numpy()
    step = HALF_STEP[compare.dtype]
    least = 2.0 ** -25 if compare.dtype == torch.float16 else 0.0      # half of fp16's least step
    over = np.abs(y - want) - bound - step * (np.abs(want) + bound) - least
    assert np.isfinite(y).all() and (over <= 1e-40).all(), (what, over.max())


def check(T, Hq, Hk, D, dtype, n=None, lo=0, dims=0, interleaved=True, lead=0, pad=0, seed=0, in_place=False, wdtype=None,
          offset=0.0, eps=1e-6, weights=True, x=None, stream=None, **rope_kw):
    n = D if n is None else n
    wdtype = wdtype or dtype
    q = make((T, Hq, D), dtype, seed, lead, pad) if x is None else x
    k = make((T, Hk, D), dtype, seed + 1, lead, pad) if Hk else None
    g = torch.Generator().manual_seed(seed + 2)
    qw = torch.randn(n, generator=g).to(wdtype).to(DEV) if weights else None
    kw = torch.randn(n, generator=g).to(wdtype).to(DEV) if weights and Hk else None
    pos = torch.randint(-100, 200000, (T,), generator=g, dtype=torch.int32).to(DEV)
    rope = S.make_rope_desc(dims, interleaved=interleaved, **rope_kw) if dims else None
    compare.dtype = dtype
    want = [reference(t, w, pos, rope_kw, dims, eps, n, lo, offset, interleaved)
            for t, w in ((q, qw), (k, kw)) if t is not None]
    if in_place:
        q_out, k_out = q, k
    else:
        q_out = make((T, Hq, D), dtype, 9, lead, pad)
        k_out = make((T, Hk, D), dtype, 9, lead, pad) if Hk else None
    around = q_out._base.clone()
    S.splash_norm_rope(q, qw, q_out, k, kw, k_out, pos if dims else None, rope, eps, norm_dims=n, rope_lo=lo,
                       weight_offset=offset, stream=stream)
    torch.cuda.synchronize()
    for y, (w, b) in zip((q_out, k_out), want):
        compare(y, w, b, (T, Hq, Hk, D, dtype, n, lo, dims))
    mask = torch.ones_like(around, dtype=torch.bool)
    torch.as_strided(mask, q_out.shape, q_out.stride(), q_out.storage_offset())[:] = False
    assert torch.equal(q_out._base[mask], around[mask])       # what lies between the rows is left as it was
    return q_out, k_out


DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,n,lo,dims", [
    (128, 128, 0, 128), (128, 128, 0, 64), (128, 128, 64, 64), (64, 64, 16, 32), (576, 512, 512, 64), (192, 192, 128, 64),
    (256, 256, 0, 256), (96, 96, 0, 32), (1024, 1024, 0, 64), (1024, 1000, 512, 256), (16, 16, 0, 16), (80, 80, 0, 80),
    (72, 72, 0, 72), (100, 50, 60, 40), (7, 5, 1, 6), (2, 1, 0, 2), (1023, 1023, 1, 254), (128, 8, 64, 64),
])
def test_rows_of_every_make(D, n, lo, dims, interleaved, dtype):
    check(5, 3, 2, D, dtype, n, lo, dims, interleaved, seed=D + lo)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 64, 8), (256, 16, 2), (3, 1, 1), (700, 1, 0), (5000, 1, 0), (1300, 3, 1),
                                     (2, 200, 17), (0, 4, 1), (4, 0, 3), (33, 31, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_batches(T, Hq, Hk, dtype):
    check(T, Hq, Hk, 128, dtype, dims=64, interleaved=False, seed=T, scaling="yarn", factor=40.0)


def test_latent_rows_of_many_tokens():
    check(4099, 1, 0, 576, torch.bfloat16, 512, 512, 64)


# several rows a lane, blocks of one wave and of several, runs that the angles' room ends, one and two vectors in the last unit
@pytest.mark.parametrize("T,Hq,Hk,D,n,lo,dims,interleaved", [
    (30001, 1, 0, 64, 64, 0, 64, False), (16411, 1, 1, 576, 512, 512, 64, False), (517, 33, 1, 576, 512, 512, 64, True),
    (9001, 3, 0, 192, 128, 128, 64, True), (3001, 5, 2, 256, 256, 0, 256, False), (2503, 1, 0, 1024, 1024, 0, 64, False),
    (777, 16, 3, 320, 320, 256, 64, False), (4001, 2, 1, 448, 448, 0, 0, True), (8009, 1, 1, 96, 96, 0, 32, True),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows(T, Hq, Hk, D, n, lo, dims, interleaved, dtype):
    check(T, Hq, Hk, D, dtype, n, lo, dims, interleaved, seed=T)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lead,pad", [(0, 8), (1, 0), (0, 1), (4, 4), (3, 5), (8, 24)])
def test_strides_and_alignments(lead, pad, dtype):
    check(9, 5, 2, 128, dtype, dims=128, lead=lead, pad=pad, seed=lead)
    check(9, 5, 2, 128, dtype, dims=64, lo=64, lead=lead, pad=pad, interleaved=False, in_place=True)


@pytest.mark.parametrize("wdtype", DTYPES)
def test_weights_of_every_type(wdtype):
    check(6, 4, 1, 128, torch.bfloat16, dims=64, wdtype=wdtype, offset=1.0)
    check(6, 4, 1, 128, torch.bfloat16, dims=64, weights=False, offset=1.0)


def test_without_rotation():
    check(6, 4, 1, 128, torch.float16)
    check(6, 4, 1, 33, torch.float32, n=20)


def test_tokens_first_and_heads_first():
    base = (torch.randn(3, 7, 64, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV)
    x = base.transpose(0, 1)                       # [T 7][H 3] with the heads' stride the larger one
    out = torch.empty(3, 7, 64, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    S.splash_norm_rope(x, w, out, None, None, None, None, None, 1e-6)
    compare.dtype = torch.bfloat16
    compare(out, *reference(x, w, None, {}, 0, 1e-6, 64, 0))


@pytest.mark.parametrize("size", [1e-44, 1e-30, 1e-20, 1e-14, 1e10, 1e18, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1.0])
def test_squares_outside_the_range(size, eps):
    # (weights of one: r * w stays in range; results that fp32 holds as subnormals are off by half of their step, 2^-150)
    g = torch.Generator().manual_seed(3)
    x = (torch.randint(1, 3, (4, 3, 128), generator=g) * (size / 2) * (torch.randint(0, 2, (4, 3, 128), generator=g) * 2 - 1)).float().to(DEV)
    out = torch.empty_like(x)
    S.splash_norm_rope(x, None, out, None, None, None, None, None, eps)
    want, bound = reference(x, None, None, {}, 0, eps, 128, 0)
    y = out.cpu().double().numpy()
    assert (np.abs(y - want) <= bound + 2.0 ** -24 * np.abs(want) + 2.0 ** -149).all(), (size, eps, np.abs(y / want - 1).max())


def test_rows_with_values_out_of_range_stay_alone():
    x = make((4, 3, 128), torch.bfloat16, 5).clone()
    x[1, 1, 7] = float("inf")
    x[2, 0, 9] = float("nan")
    x[3, 2] = 0
    out = torch.empty_like(x)
    S.splash_norm_rope(x, None, out, None, None, None, None, None, 1e-6)
    y = out.cpu().float()
    assert torch.isnan(y[1, 1, 7]) and torch.isnan(y[2, 0]).all() and (y[3, 2] == 0).all()
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    want, bound = reference(x, None, None, {}, 0, 1e-6, 128, 0)
    err = np.abs(y.double().numpy() - want)[keep.numpy()]
    assert (err <= (bound + 2.0 ** -8 * (np.abs(want) + bound))[keep.numpy()]).all()


def test_the_parts_behind_the_norm_are_copied():
    x = make((3, 2, 576), torch.bfloat16, 6)
    out = torch.zeros(3, 2, 576, dtype=torch.bfloat16, device=DEV)
    S.splash_norm_rope(x, None, out, None, None, None, None, None, 1e-6, norm_dims=512)
    assert torch.equal(out[..., 512:], x[..., 512:]) and not torch.equal(out[..., :512], x[..., :512])


def test_the_rotation_is_that_of_rope():
    # rows of unit power and weights of one: the norm changes them by rounding alone
    T, H = 50, 4
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=torch.Generator().manual_seed(7), dtype=torch.int32).to(DEV)
    x = (torch.randint(0, 2, (T, H, 64), generator=torch.Generator().manual_seed(8)) * 2 - 1).float().to(DEV)
    for il in (True, False):
        rope = S.make_rope_desc(64, interleaved=il, scaling="yarn", factor=40.0)
        a, b = torch.empty_like(x), torch.empty_like(x)
        S.splash_norm_rope(x, None, a, None, None, None, pos, rope, 0.0)
        S.splash_rope(x, pos, b, rope)
        assert (a - b).abs().max() < 16 * 2.0 ** -24          # rsqrtf(1) within 2 ulp, four roundings


def test_a_captured_call_replays_and_streams_run_side_by_side():
    x = make((256, 18, 128), torch.bfloat16, 11)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(256, dtype=torch.int32, device=DEV)
    rope = S.make_rope_desc(128, interleaved=False)
    out = torch.empty(256, 18, 128, dtype=torch.bfloat16, device=DEV)
    call = lambda o, s=None: S.splash_norm_rope(x[:, :16], w, o[:, :16], x[:, 16:], w, o[:, 16:], pos, rope, 1e-6, stream=s)
    call(out)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    outs, streams = [torch.empty_like(out) for _ in range(3)], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for o, s in zip(outs, streams):
        call(o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_rows_that_are_read_more_than_once():
    # a token's key for every head, and one row for every token: strides of zero
    x = make((7, 1, 128), torch.bfloat16, 12)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(7, dtype=torch.int32, device=DEV)
    rope = S.make_rope_desc(64, interleaved=False)
    compare.dtype = torch.bfloat16
    for src in (x.expand(7, 5, 128), x[2:3].expand(7, 5, 128)):
        out = torch.empty(7, 5, 128, dtype=torch.bfloat16, device=DEV)
        S.splash_norm_rope(src, w, out, None, None, None, pos, rope, 1e-6)
        compare(out, *reference(src, w, pos, {}, 64, 1e-6, 128, 0, interleaved=False))


def test_refusals_of_the_binding():
    x, out = make((4, 2, 64), torch.bfloat16, 1), make((4, 2, 64), torch.bfloat16, 2)
    w, pos = torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    rope = S.make_rope_desc(64)
    bad = [dict(q=x.double()), dict(q_out=out[:3]), dict(q_weight=w[:32]), dict(q_weight=w.double()), dict(positions=pos[:3]),
           dict(positions=None), dict(positions=pos.long()), dict(k=x), dict(k=x[:3], k_out=out[:3]), dict(norm_dims=32),
           dict(k=x, k_out=out.half()), dict(k=x, k_out=out, k_weight=w.half()), dict(q=x.transpose(1, 2)), dict(q=x[0])]
    for kw in bad:
        a = dict(q=x, q_weight=w, q_out=out, k=None, k_weight=None, k_out=None, positions=pos, rope=rope, eps=1e-6)
        a.update(kw)
        with pytest.raises(ValueError):
            S.splash_norm_rope(**a)
    for kw in (dict(rope_lo=1), dict(rope_lo=-1), dict(norm_dims=0, q_weight=None), dict(eps=-1.0), dict(eps=float("nan"))):
        a = dict(q=x, q_weight=w, q_out=out, k=None, k_weight=None, k_out=None, positions=pos, rope=rope, eps=1e-6)
        a.update(kw)
        with pytest.raises(S.SplashError):
            S.splash_norm_rope(**a)


def test_offsets_past_32_bits():
    T, H, D, apart = 3, 2, 128, 1 << 30    # the last token's rows begin 2^31 elements on
    buf = torch.empty(2 * apart + H * D, dtype=torch.bfloat16, device=DEV)
    x = make((T, H, D), torch.bfloat16, 71)
    far = torch.as_strided(buf, (T, H, D), (apart, D, 1))
    far.copy_(x)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([3, 70000, 11], dtype=torch.int32, device=DEV)
    rope = S.make_rope_desc(64, interleaved=False)
    compare.dtype = torch.bfloat16
    want = reference(x, w, pos, {}, 64, 1e-6, D, 0, interleaved=False)
    S.splash_norm_rope(far, w, far, None, None, None, pos, rope, 1e-6)
    compare(far, *want)
