"""Norm weights far from one over rows far from one (marked gpu): every result has room in fp32, so it has to come out, whatever
the product of the row's root and a weight is."""
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.test_gpu_norm_rope import DEV, compare, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,dims", [(128, 64), (33, 0), (576, 64)])
@pytest.mark.parametrize("size,weight", [(-56, 75), (-50, 100), (56, -80), (50, -100), (-100, 90), (100, -90), (0, 100), (0, -100)])
def test_large_and_small_weights(size, weight, D, dims, dtype):
    g = torch.Generator().manual_seed(D + size)
    # magnitudes of 0.5 to 2, so that no result is subnormal
    mag = lambda *s: (torch.rand(*s, generator=g) * 1.5 + 0.5) * (torch.randint(0, 2, s, generator=g) * 2 - 1)
    x = (mag(5, 3, D).double() * 2.0 ** size).to(dtype).to(DEV)
    w = (mag(D).double() * 2.0 ** weight).to(dtype).to(DEV)
    pos = torch.tensor([0, 1, 77, 4096, 100000], dtype=torch.int32, device=DEV)
    rope = S.make_rope_desc(dims, interleaved=False) if dims else None
    out = torch.empty_like(x)
    S.splash_norm_rope(x, w, out, None, None, None, pos if dims else None, rope, 0.0)
    compare.dtype = dtype
    compare(out, *reference(x, w, pos, {}, dims, 0.0, D, 0, interleaved=False), (size, weight, D, dtype))
