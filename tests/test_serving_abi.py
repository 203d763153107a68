"""Host-side refusals of the serving entry points (rope, append, unpack, chunk attention), and pins
of the 64-bit forms their GPU tests compare with.  CPU only: no call here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import build as B
from layout_agnostic_paged_gb300 import splash as S
from tests import serving_reference as R

FAKE = 0x10000  # never dereferenced: every call below fails host validation first
INVALID, UNSUPPORTED = S.SPLASH_ERR_INVALID_ARG, S.SPLASH_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.load_library()


def desc(**kw):
    d = dict(num_reqs=2, num_heads=8, d_qk=576, d_v=512, page_size=16, num_pages=11, max_pages_per_req=7,
             scale=0.0721)
    d.update(kw)
    return S.SplashAttnDesc(**d)


# ------------------------------------------------------------------ rope

def rope(lib, r, dtype=0, x=FAKE, xt=1024, xh=128, y=FAKE << 8, yt=1024, yh=128, pos=FAKE, T=3, H=4):
    return lib.splash_rope(r, dtype, x, xt, xh, y, yt, yh, pos, T, H, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dims=0), INVALID), (dict(dims=7), INVALID), (dict(dims=-2), INVALID), (dict(dims=258), UNSUPPORTED),
    (dict(base=0.5), INVALID), (dict(base=float("nan")), INVALID), (dict(base=float("inf")), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(amplitude=float("nan")), INVALID),
    (dict(scaling="linear", factor=0.5), INVALID), (dict(scaling="linear", factor=float("nan")), INVALID),
    (dict(scaling="yarn", factor=float("inf")), INVALID), (dict(scaling="yarn", base=1.0), INVALID),
    (dict(scaling="yarn", orig_ctx=0.0), INVALID), (dict(scaling="yarn", beta_fast=-1.0), INVALID),
    (dict(scaling="yarn", beta_slow=float("nan")), INVALID),
])
def test_rope_rejects_bad_descriptions(lib, kw, code):
    args = dict(dims=64)
    args.update(kw)
    assert rope(lib, S.make_rope_desc(**args)) == code


def test_rope_rejects_a_missing_or_unknown_description(lib):
    assert rope(lib, None) == INVALID
    r = S.make_rope_desc(64)
    r.scaling = 3
    assert rope(lib, r) == INVALID
    with pytest.raises(ValueError):
        S.make_rope_desc(64, scaling="ntk")


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(T=-1), INVALID), (dict(H=-1), INVALID),
    (dict(xt=-8), INVALID), (dict(yh=-8), INVALID), (dict(x=0), INVALID), (dict(y=0), INVALID),
    (dict(pos=0), INVALID), (dict(pos=FAKE + 2), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(dtype=2, y=FAKE + 2), INVALID),
    (dict(yh=32), INVALID), (dict(yt=32), INVALID),               # head rows of y that share elements
    (dict(yt=128, yh=128), INVALID), (dict(T=1 << 16, H=1 << 16, yt=1 << 24, yh=128), UNSUPPORTED),
])
def test_rope_rejects_bad_arguments(lib, kw, code):
    assert rope(lib, S.make_rope_desc(64), **kw) == code


def test_rope_of_nothing_is_fine(lib):
    assert rope(lib, S.make_rope_desc(64), x=0, y=0, pos=0, T=0) == S.SPLASH_OK
    assert rope(lib, S.make_rope_desc(64), x=0, y=0, pos=0, H=0) == S.SPLASH_OK


# ------------------------------------------------------------------ append, unpack

def append(lib, d, r=None, fmt=0, lat=FAKE, lt=512, kr=FAKE, kt=64, cu=FAKE, n=5, table=FAKE, ctx=FAKE, pool=FAKE):
    return lib.splash_kv_append(d, r, fmt, lat, lt, kr, kt, cu, n, table, ctx, pool, None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=2), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED), (dict(n=-1), INVALID), (dict(lat=0), INVALID),
    (dict(kr=0), INVALID), (dict(cu=0), INVALID), (dict(table=0), INVALID), (dict(ctx=0), INVALID),
    (dict(pool=0), INVALID), (dict(lat=FAKE + 8), INVALID), (dict(kr=FAKE + 2), INVALID), (dict(lt=516), INVALID),
    (dict(lt=-512), INVALID), (dict(kt=65), INVALID), (dict(pool=FAKE + 8), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(table=FAKE + 1), INVALID), (dict(ctx=FAKE + 3), INVALID),
])
def test_append_rejects_bad_arguments(lib, kw, code):
    assert append(lib, desc(), **kw) == code


def test_append_rejects_bad_shapes(lib):
    assert append(lib, None) == INVALID
    assert append(lib, desc(page_size=48)) == UNSUPPORTED
    assert append(lib, desc(d_v=576)) == UNSUPPORTED
    assert append(lib, desc(num_reqs=-1)) == INVALID
    assert append(lib, desc(), S.make_rope_desc(32)) == UNSUPPORTED       # the cache's position part has 64 dims
    assert append(lib, desc(), S.make_rope_desc(64, base=0.0)) == INVALID
    for kw in (dict(num_reqs=0), dict(num_pages=0), dict(max_pages_per_req=0)):
        assert append(lib, desc(**kw), lat=0, pool=0) == S.SPLASH_OK       # nowhere to write
    assert append(lib, desc(), n=0, lat=0) == S.SPLASH_OK


def test_unpack_rejects_bad_arguments(lib):
    far = FAKE << 8
    f = lambda src=FAKE, dst=far, P=16, s=FAKE, d=FAKE, n=3, sn=8, dn=8: lib.splash_kv_unpack(src, dst, P, s, d, n, sn, dn, None)
    for kw in (dict(P=0), dict(P=-4), dict(n=-1), dict(sn=-1), dict(dn=-1), dict(src=0), dict(dst=0), dict(s=0),
               dict(d=0), dict(src=FAKE + 8), dict(dst=far + 4), dict(s=FAKE + 2), dict(dst=FAKE + 656 * 16)):
        assert f(**kw) == INVALID, kw
    assert f(n=0, src=0, dst=0) == S.SPLASH_OK


# ------------------------------------------------------------------ chunk attention

def chunk(lib, d, q=FAKE, pool=FAKE, cu=FAKE, n=6, table=FAKE, ctx=FAKE, lo=0, hi=8, tlo=0, thi=-1, dt=0, out=FAKE,
          lse=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.splash_chunk_attn(d, q, pool, cu, n, table, ctx, lo, hi, tlo, thi, dt, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(lo=3, hi=3), INVALID), (dict(lo=-1), INVALID), (dict(hi=9), INVALID),
    (dict(tlo=-1), INVALID), (dict(tlo=9, thi=4), INVALID), (dict(dt=1), UNSUPPORTED), (dict(dt=7), UNSUPPORTED),
    (dict(ws=0), INVALID), (dict(ws=FAKE + 128), INVALID), (dict(q=0), INVALID), (dict(cu=0), INVALID),
    (dict(table=0), INVALID), (dict(ctx=0), INVALID), (dict(out=0), INVALID), (dict(lse=0), INVALID),
    (dict(pool=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 16), INVALID), (dict(pool=FAKE + 2), INVALID),
    (dict(cu=FAKE + 2), INVALID), (dict(n=1 << 30), UNSUPPORTED),
])
def test_chunk_rejects_bad_arguments(lib, kw, code):
    assert chunk(lib, desc(), **kw) == code


def test_chunk_rejects_bad_shapes(lib):
    assert chunk(lib, None) == INVALID
    for kw, code in ((dict(d_qk=512), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(num_heads=0), INVALID),
                     (dict(scale=float("nan")), INVALID), (dict(num_pages=1 << 28), UNSUPPORTED),
                     (dict(page_size=16, max_pages_per_req=(1 << 27) - 63), UNSUPPORTED)):
        assert chunk(lib, desc(**kw)) == code
        assert lib.splash_chunk_workspace_size(desc(**kw), 6, 0, 1) == 0
    assert lib.splash_chunk_workspace_size(None, 6, 0, 8) == 0
    assert lib.splash_chunk_workspace_size(desc(), -1, 0, 8) == 0
    assert lib.splash_chunk_workspace_size(desc(), 6, 4, 4) == 0


# ------------------------------------------------------------------ the binding

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_rope(x, i, x, S.make_rope_desc(64))
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_kv_append(x, x, i, i, i, x)
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_kv_unpack(x, x, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_chunk_attn(x, x, i, i, i, 0, 1, 0, -1, x, x, x, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        S.chunk_workspace(x, x, i, 0.1)


# ------------------------------------------------------------------ the 64-bit forms

def test_rotation_keeps_lengths_and_adds_up():
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    p, q = torch.tensor([0, 1, 77, 4096, 131071]), torch.tensor([5, -9, 0, 12345, 7])
    for il in (True, False):
        y = R.rotate(x, p, il, scaling="yarn", factor=40.0)
        assert np.allclose(np.linalg.norm(y, axis=-1), x.norm(dim=-1).numpy(), rtol=1e-14)
        assert np.array_equal(R.rotate(x, 0 * p, il), x.numpy())
        two = R.rotate(torch.from_numpy(R.rotate(x, p, il)), q, il)
        assert np.allclose(two, R.rotate(x, p + q, il), atol=1e-9)       # angles of 1e5 radians to 1e-11


def test_rotation_of_the_two_layouts_is_one_permuted():
    x = torch.randn(3, 1, 8, generator=torch.Generator().manual_seed(2))
    p = torch.tensor([3, 1, 4])
    perm = [0, 2, 4, 6, 1, 3, 5, 7]
    assert np.allclose(R.rotate(x, p, True)[..., perm], R.rotate(x[..., perm], p, False), atol=1e-15)


def test_frequencies_of_the_scalings():
    assert np.allclose(R.frequencies(4, base=100.0), [1.0, 0.1])
    assert np.allclose(R.frequencies(4, base=100.0, scaling="linear", factor=8.0), [0.125, 0.0125])
    f, y = R.frequencies(64), R.frequencies(64, scaling="yarn", factor=40.0, orig_ctx=4096.0)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(y[turns > 40], f[turns > 40])                     # fast pairs as they are
    assert np.allclose(y[turns < 0.7], f[turns < 0.7] / 40)              # slow pairs interpolated
    assert (y <= f).all() and (y >= f / 40 - 1e-18).all()


def test_e4m3_codes_match_the_cast():
    v = torch.cat([torch.linspace(0, 448, 20001), torch.tensor(R.E4M3, dtype=torch.float32),
                   torch.exp2(torch.linspace(-12, 8, 4001))])
    assert np.array_equal(R._code(v.double().numpy()), v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_packed_rows_unpack_to_within_half_a_step():
    x = (torch.randn(6, 512, generator=torch.Generator().manual_seed(3)) * 3).to(torch.bfloat16)
    codes, scales = R.pack_rows(x)
    rows = torch.cat((torch.from_numpy(codes), torch.from_numpy(scales), torch.zeros(6, 128, dtype=torch.uint8)), 1)
    v = R.unpack_rows(rows)[:, :512]
    s = 2.0 ** (scales.astype(float) - 127).repeat(32, axis=1)
    assert (np.abs(v - x.double().numpy()) <= np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, s * 2.0 ** -10)).all()
    assert (np.abs(x.double().numpy()).reshape(6, 16, 32).max(-1) <= 448 * 2.0 ** (scales.astype(float) - 127)).all()
    assert (np.abs(x.double().numpy()).reshape(6, 16, 32).max(-1) > 448 * 2.0 ** (scales.astype(float) - 128)).all()


def test_chunk_reference_against_the_library_softmax():
    b = R.Batch([1, 7, 3], [5, 40, 3], 2, 16, 4, "cpu")
    out, lse, _, _ = R.chunk_reference(b, 0, 2)
    row = 0
    for r, (n, c) in enumerate(zip(b.q_lens, b.ctx)):
        k = b.keys[r].double()
        q = b.q[row:row + n].double().transpose(0, 1)
        mask = torch.arange(c)[None, :] <= torch.arange(c - n, c)[:, None]
        o = torch.nn.functional.scaled_dot_product_attention(q, k.expand(2, -1, -1), k[:, :512].expand(2, -1, -1),
                                                             attn_mask=mask, scale=b.scale)
        assert torch.allclose(out[row:row + n].transpose(0, 1), o, atol=1e-12)
        row += n
