"""The sublayer's own checks of its arguments (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def test_an_mxfp8_layer_is_refused(mok):
    """Its layer would want weight copies that Params does not hold, after the norm and the router have run."""
    from mixture_experts_layer_build_gb300.sublayer import Sublayer
    with pytest.raises(ValueError, match="precision"):
        Sublayer(16, 128, 128, 4, 2, 64, cfg=mok.make_config(0, 0, precision=mok.MOK_MXFP8), device="cpu")
    assert Sublayer(16, 128, 128, 4, 2, 64, cfg=mok.make_config(128, 256), device="cpu").layer.cfg.minibatch_rows == 128
