"""Host-side refusals of the batch tables, the norm with rope and the attention's windows and groups.  CPU only:
no call here reaches a kernel."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from layout_agnostic_paged_gb300 import build as B
from layout_agnostic_paged_gb300 import splash as S

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


# ------------------------------------------------------------------ batch tables

def tables(lib, reqs=2, page=16, pages=11, most=7, n=6, reserved=0, past=FAKE, new=FAKE, free=FAKE, count=FAKE, table=FAKE,
           cu=FAKE, ctx=FAKE, pos=FAKE, slots=FAKE, left=FAKE):
    return lib.splash_batch_tables(S._BATCH.pack(reqs, page, pages, most, n, reserved, past, new, free, count, table, cu, ctx,
                                                 pos, slots, left), None)


@pytest.mark.parametrize("kw,code", [
    (dict(past=0), INVALID), (dict(new=0), INVALID), (dict(table=0), INVALID), (dict(free=0), INVALID),
    (dict(count=0), INVALID), (dict(cu=0), INVALID), (dict(ctx=0), INVALID), (dict(pos=0), INVALID),
    (dict(slots=0), INVALID), (dict(left=0), INVALID), (dict(n=-1), INVALID), (dict(n=(1 << 30) + 1), UNSUPPORTED),
    (dict(past=FAKE + 2), INVALID), (dict(slots=FAKE + 1), INVALID), (dict(left=FAKE + 2), INVALID), (dict(reserved=1), INVALID),
    (dict(page=48), UNSUPPORTED), (dict(page=0), UNSUPPORTED), (dict(reqs=-1), INVALID), (dict(pages=1 << 28), UNSUPPORTED),
    (dict(pages=-1), INVALID), (dict(most=-1), INVALID), (dict(most=1 << 27), UNSUPPORTED),
])
def test_tables_rejects_bad_arguments(lib, kw, code):
    assert tables(lib, **kw) == code
    assert lib.splash_batch_tables(None, None) == INVALID


def release(lib, reqs=2, page=16, pages=11, most=7, window=0, sinks=0, ctx=FAKE, keep=FAKE, table=FAKE, free=FAKE, count=FAKE):
    return lib.splash_batch_release(S._BATCH_DROP.pack(reqs, page, pages, most, window, sinks, ctx, keep, table, free, count), None)


@pytest.mark.parametrize("kw,code", [
    (dict(ctx=0), INVALID), (dict(table=0), INVALID), (dict(free=0), INVALID), (dict(count=0), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(keep=FAKE + 2), INVALID), (dict(table=FAKE + 1), INVALID),
    (dict(page=8), UNSUPPORTED), (dict(reqs=-1), INVALID), (dict(reqs=1 << 10, most=1 << 21), UNSUPPORTED),
])
def test_release_rejects_bad_arguments(lib, kw, code):
    assert release(lib, **kw) == code
    assert lib.splash_batch_release(None, None) == INVALID


def test_release_of_nothing_is_fine(lib):
    assert release(lib, reqs=0, ctx=0, table=0) == S.SPLASH_OK
    assert release(lib, most=0, ctx=0, table=0) == S.SPLASH_OK


def test_packed_structs_are_laid_out_as_in_the_header():
    """A C program states the sizes and offsets that the binding's packed structs rely on."""
    src = r"""
#include <stddef.h>
#include <stdio.h>
#include "splash.h"
int main(void) {
    printf("%zu %zu %zu %zu %zu ", sizeof(splash_batch), offsetof(splash_batch, past_lens), offsetof(splash_batch, block_table),
           offsetof(splash_batch, cu_q), offsetof(splash_batch, left));
    printf("%zu %zu %zu ", sizeof(splash_batch_drop), offsetof(splash_batch_drop, ctx_lens), offsetof(splash_batch_drop, free_count));
    printf("%zu %zu %zu %zu ", sizeof(splash_norm_rows), offsetof(splash_norm_rows, y), offsetof(splash_norm_rows, weight),
           offsetof(splash_norm_rows, heads));
    printf("%zu %zu %zu\n", sizeof(splash_chunk_ext), offsetof(splash_chunk_ext, cu_groups), offsetof(splash_chunk_ext, num_groups));
    return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "sizes.c"), os.path.join(d, "sizes")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", B.INCLUDE, c, "-o", exe], check=True)
        out = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [S._BATCH.size, 24, 56, 64, 96, S._BATCH_DROP.size, 24, 56, S._NORM_ROWS.size, 24, 48, 56,
                   ctypes.sizeof(S.SplashChunkExt), 8, 24]


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_batch_tables(i, i, t, 16, i, i, i, i, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        S.splash_batch_release(i, None, t, 16, i, i)
    with pytest.raises(ValueError, match="past_lens"):
        S._int32_arrays("x", -1, (("past_lens", i.long(), 2),))
    with pytest.raises(ValueError, match="cu_q"):
        S._int32_arrays("x", -1, (("cu_q", i, 3),))
    with pytest.raises(ValueError, match="slots"):
        S._int32_arrays("x", -1, (("slots", t[:, 0], 2),))
    with pytest.raises(ValueError, match="device"):
        S._int32_arrays("x", 0, (("slots", i, 2),))


# ------------------------------------------------------------------ norm with rope

def rows(**kw):
    d = dict(x=FAKE, x_token_stride=1024, x_head_stride=128, y=FAKE << 8, y_token_stride=1024, y_head_stride=128,
             weight=FAKE, heads=4, reserved=0)
    d.update(kw)
    return S._NORM_ROWS.pack(*d.values())


def norm(lib, n=None, r="rope", dtype=0, q="rows", k=None, pos=FAKE, T=3, **kw):
    d = dict(width=128, norm_dims=128, rope_lo=0, weight_dtype=0, eps=1e-6, weight_offset=0.0)
    d.update(n or {})
    return lib.splash_norm_rope(S.SplashNormDesc(**d), S.make_rope_desc(64) if r == "rope" else r, dtype,
                                rows() if q == "rows" else q, k, pos, T, None)


@pytest.mark.parametrize("n,code", [
    (dict(width=0), INVALID), (dict(width=1025), UNSUPPORTED), (dict(norm_dims=0), INVALID), (dict(norm_dims=129), INVALID),
    (dict(rope_lo=-1), INVALID), (dict(rope_lo=65), INVALID), (dict(weight_dtype=3), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(weight_offset=float("inf")), INVALID),
    (dict(width=32, norm_dims=32), INVALID),
])
def test_norm_rejects_bad_descriptions(lib, n, code):
    assert norm(lib, n) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNSUPPORTED), (dict(T=-1), INVALID), (dict(pos=0), INVALID), (dict(pos=FAKE + 2), INVALID),
    (dict(q=None), INVALID), (dict(r=S.make_rope_desc(7)), INVALID),
])
def test_norm_rejects_bad_arguments(lib, kw, code):
    assert norm(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), INVALID), (dict(y=0), INVALID), (dict(x=FAKE + 1), INVALID), (dict(weight=FAKE + 1), INVALID),
    (dict(heads=-1), INVALID), (dict(reserved=1), INVALID), (dict(x_token_stride=-8), INVALID), (dict(y_head_stride=64), INVALID),
    (dict(y_token_stride=64), INVALID), (dict(y_token_stride=256, y_head_stride=128), INVALID),
    (dict(heads=1 << 30, y_token_stride=1 << 40), UNSUPPORTED),
])
def test_norm_rejects_bad_rows(lib, kw, code):
    assert norm(lib, q=rows(**kw)) == code
    assert norm(lib, k=rows(**kw)) == code


def test_norm_of_nothing_is_fine(lib):
    assert norm(lib, T=0, q=rows(x=0, y=0), pos=0) == S.SPLASH_OK
    assert norm(lib, q=rows(heads=0, x=0), pos=0) == S.SPLASH_OK


# ------------------------------------------------------------------ windowed attention

def chunk_ex(lib, d, ext, n=6, lo=0, hi=8, ws_bytes=1 << 40, q=FAKE):
    return lib.splash_chunk_attn_ex(d, ext, q, FAKE, FAKE, n, FAKE, FAKE, lo, hi, 0, -1, 0, FAKE, FAKE, FAKE, ws_bytes, None)


def test_windowed_attention_rejects_bad_arguments(lib):
    for w, s in ((-1, 0), (5, -1), (0, -1), (-2 ** 31, 0)):
        assert chunk_ex(lib, desc(), S.SplashChunkExt(window=w, sinks=s)) == INVALID
        assert lib.splash_chunk_workspace_size_ex(desc(), S.SplashChunkExt(window=w, sinks=s), 6, 0, 8) == 0
    ok = S.SplashChunkExt(window=5, sinks=1)
    assert chunk_ex(lib, None, ok) == INVALID
    assert chunk_ex(lib, desc(d_qk=512), ok) == UNSUPPORTED
    assert chunk_ex(lib, desc(), ok, q=0) == INVALID
    assert chunk_ex(lib, desc(), ok, lo=4, hi=4) == INVALID
    assert chunk_ex(lib, desc(), ok, n=-1) == INVALID


def test_groups_are_checked(lib):
    good = dict(cu_groups=FAKE, prefix_lens=FAKE, num_groups=2)
    for kw, code in ((dict(num_groups=-1), INVALID), (dict(num_groups=1025), UNSUPPORTED), (dict(window=9), UNSUPPORTED),
                     (dict(cu_groups=0), INVALID), (dict(prefix_lens=0), INVALID), (dict(cu_groups=FAKE + 2), INVALID),
                     (dict(prefix_lens=FAKE + 1), INVALID), (dict(reserved=1), INVALID)):
        assert chunk_ex(lib, desc(), S.SplashChunkExt(**{**good, **kw})) == code, kw
    for kw in (dict(num_groups=-1), dict(num_groups=1025), dict(window=9), dict(reserved=7)):
        assert lib.splash_chunk_workspace_size_ex(desc(), S.SplashChunkExt(**{**good, **kw}), 6, 0, 8) == 0
