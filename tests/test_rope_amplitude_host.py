"""Host-side test of a rotation's amplitude, which the kernels take as float32.  No GPU is needed."""

import pytest

ra = pytest.importorskip("context_ring_attention_gb300")


@pytest.fixture(scope="module", autouse=True)
def _library():
    import os

    from context_ring_attention_gb300 import build
    if not os.path.exists(ra.library_path()):
        build.build()
    ra.load_library()


@pytest.mark.parametrize("amplitude", [3.5e38, 1e39, 1e300, 1e-38, 1e-46, 5e-324])
def test_amplitudes_that_float32_does_not_hold_are_refused(amplitude):
    """They would come out as infinity, as 0 or with fewer bits."""
    with pytest.raises(ra.RaError) as err:
        ra.ra_rope_plan(64, amplitude=amplitude)
    assert err.value.name == "RA_ERR_INVALID_ARG"


@pytest.mark.parametrize("amplitude", [2.0 ** -126, 0.5, 1.2079441541679836, (2 - 2.0 ** -23) * 2.0 ** 127])
def test_the_others_are_taken(amplitude):
    assert ra.ra_rope_plan(64, amplitude=amplitude).problem["amplitude"] == amplitude
