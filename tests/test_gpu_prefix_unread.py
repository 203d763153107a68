"""Groups of requests where a token's own rows fill a CTA pair's (marked gpu): nothing is shared, and the groups' arrays, good or
bad, change neither a result nor the status."""
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.test_gpu_prefix import ints, run, shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,lo,hi", [(128, 0, 128), (256, 0, 256), (200, 0, 200), (128, 0, 65), (256, 100, 200)])
def test_groups_are_not_read(heads, lo, hi):
    b = shared([(700, [(1, 5), (2, 60), (1, 0)])], heads, 64, 7)
    want, wl, ws = run(b, lo, hi, groups=False)
    for cu, prefix in (([0, 3], [700]), ([3, 0], [700]), ([-5, 2 ** 31 - 1], [700]), ([0, 3], [-1]), ([0, 3], [2 ** 31 - 1])):
        b.cu_groups, b.prefix = ints(cu), ints(prefix)
        out, lse, ws = run(b, lo, hi)
        assert torch.equal(out, want) and torch.equal(lse, wl) and S.splash_workspace_status(ws) == 0


@pytest.mark.parametrize("heads,lo,hi", [(127, 0, 127), (128, 0, 64), (128, 64, 128)])
def test_groups_are_read(heads, lo, hi):
    b = shared([(700, [(1, 5), (2, 60), (1, 0)])], heads, 64, 8)
    b.cu_groups = ints([3, 0])
    out, lse, ws = run(b, lo, hi)
    assert S.splash_workspace_status(ws) == S.SPLASH_DEVICE_BAD_INPUT and (out == 7).all() and (lse == 7).all()
