"""Numbers that do not fit the library's 32-bit arguments are refused, not cut (CPU only)."""
import pytest

from layout_agnostic_paged_gb300 import splash as S

BAD = (2 ** 32, 2 ** 32 + 5, 2 ** 31, 2 ** 63 - 1, -2 ** 31 - 1)


@pytest.mark.parametrize("v", BAD)
def test_windows_and_first_tokens(v):
    with pytest.raises(ValueError, match="window"):
        S._window_ext(v, 0)
    with pytest.raises(ValueError, match="sinks"):
        S._window_ext(5, v)
    e = S._window_ext(2 ** 31 - 1, -2 ** 31)
    assert (e.window, e.sinks) == (2 ** 31 - 1, -2 ** 31)


@pytest.mark.parametrize("v", BAD)
def test_norms(v):
    with pytest.raises(ValueError, match="rope_lo"):
        S._norm_desc(128, 128, v, 0, 1e-6, 0.0)
    with pytest.raises(ValueError, match="norm_dims"):
        S._norm_desc(128, v, 0, 0, 1e-6, 0.0)


@pytest.mark.parametrize("v", BAD + (16.5, "16"))
def test_batches(v):
    with pytest.raises(ValueError, match="splash_batch_tables"):
        S._packed("splash_batch_tables", S._BATCH, 1, v, *[0] * 14)
    with pytest.raises(ValueError, match="splash_batch_release"):
        S._packed("splash_batch_release", S._BATCH_DROP, 1, 16, 3, 4, v, *[0] * 6)
    assert S._packed("x", S._BATCH, 1, 16, *[0] * 14) == S._BATCH.pack(1, 16, *[0] * 14)
