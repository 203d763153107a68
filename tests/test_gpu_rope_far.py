"""Angles of far positions (marked gpu), against 60-digit arithmetic."""
import math

import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.test_rope_table import exact_turns

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FAR = [0, 1, 4096, 131071, 1 << 20, 1000003, (1 << 31) - 1, (1 << 31) - 77, 2000000011, -(1 << 31), -1999999973]


@pytest.mark.parametrize("dims", [64, 128])
@pytest.mark.parametrize("kw", [dict(base=10000.0, scaling="none"), dict(base=500000.0, scaling="linear", factor=8.0),
                                dict(base=10000.0, scaling="yarn", factor=40.0)], ids=["none", "linear", "yarn"])
def test_far_angles_are_as_exact_as_near_ones(dims, kw):
    # (1, 0) turned is (cos, sin), without a further rounding.  The angle, at most pi / 4 from a quarter turn, is rounded
    # to 2^-24 of itself, sincospi is within 1 ulp (2^-23 of the value), and the table's half unit of 2^-64 turns
    # is 2^-34 turns at 2^31.
    x = torch.zeros(len(FAR), 1, dims, device=DEV)
    x[..., 0::2] = 1
    y = torch.empty_like(x)
    S.splash_rope(x, torch.tensor(FAR, dtype=torch.int64).to(torch.int32).to(DEV), y, S.make_rope_desc(dims, **kw))
    got = y[:, 0].cpu().double().numpy()
    turns = [t / 2 ** 64 for t in exact_turns(dims, **kw)]
    part = np.array([[float((p * t) % 1) for t in turns] for p in FAR])
    c, s = np.cos(2 * math.pi * part), np.sin(2 * math.pi * part)
    far = 2 * math.pi * 2.0 ** -34 + 2.0 ** -50
    near = math.pi / 4 * 2.0 ** -24
    assert (np.abs(got[:, 0::2] - c) <= near + 2.0 ** -23 * np.abs(c) + far).all()
    assert (np.abs(got[:, 1::2] - s) <= near + 2.0 ** -23 * np.abs(s) + far).all()
