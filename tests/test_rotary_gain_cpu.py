"""A gain that float32 holds only as infinity is refused (CPU only): 0 * inf would
turn zeros into NaN."""
import pytest

from test_paged_refusals_cpu import HAS_GPU, INVALID, NO_DEVICE, append, cache, rotate, spec, step


@pytest.mark.parametrize("gain", [1e39, -1e39, 3.5e38, 1e300])
def test_gain_beyond_float32(gain):
    assert rotate(spec(gain=gain)) == INVALID
    assert append(cache(), spec(gain=gain)) == INVALID and step(cache(), spec(gain=gain)) == INVALID


@pytest.mark.skipif(HAS_GPU, reason="checks the no-device answer")
@pytest.mark.parametrize("gain", [3.4e38, -1.0, 0.0, 1e-300])
def test_gain_within_float32(gain):
    assert rotate(spec(gain=gain)) == NO_DEVICE
