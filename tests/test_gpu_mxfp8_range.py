"""The top of the MXFP8 cache's range (marked gpu)."""
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_append_and_unpack_of_the_largest_latents():
    # every bf16 from 2^124 on, in groups of one magnitude and in groups that end in bf16's maximum: what rounds
    # to 256 * 2^120 = 2^128 reads back as an infinity, and nothing else does
    bits = torch.arange(0x7D80, 0x7F80, dtype=torch.int32)
    vals = bits.to(torch.int16).view(torch.bfloat16)        # 512 of them
    alone = vals[:, None].expand(-1, 32).reshape(32, 512)
    mixed = vals.view(16, 32).repeat(1, 1).reshape(1, 512).repeat(4, 1)
    mixed[1] *= -1
    mixed[2, 31::32] = torch.finfo(torch.bfloat16).max
    x = torch.cat((alone, mixed)).contiguous()
    n = len(x)
    i32 = dict(dtype=torch.int32, device=DEV)
    src = torch.zeros(1, 64, 656, dtype=torch.uint8, device=DEV)
    dst = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device=DEV)
    S.splash_kv_append(x.to(DEV), torch.zeros(n, 64, dtype=torch.bfloat16, device=DEV), torch.tensor([0, n], **i32),
                       torch.zeros(1, 1, **i32), torch.tensor([n], **i32), src)
    S.splash_kv_unpack(src, dst, torch.zeros(1, **i32), torch.zeros(1, **i32))
    got, v = dst[0, :n, :512].cpu().double(), x.double()
    top = v.abs() >= 248 * 2.0 ** 120
    assert torch.equal(torch.isinf(got), top) and torch.equal(torch.signbit(got), torch.signbit(v))
    group = v.view(n, 16, 32).abs().amax(-1)
    step = 2.0 ** (torch.frexp(group / 448)[1].double()).repeat_interleave(32, 1)      # 2^e, or twice it
    err = (got - v).abs()[~top]
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, step * 2.0 ** -9)[~top]).all()
