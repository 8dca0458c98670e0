"""Products of second terms: no kernel of large tiles is compiled that no plan takes (CPU only)."""
import pytest

from test_lane_exchange import device_code, kernels


@pytest.mark.parametrize("name,outs", [("linear.hip", ["PiecesOutILb1E"]), ("cross_entropy.hip", ["GradOutILb1E", "PiecesOutILb1E"])])
def test_second_terms_have_no_large_tiles(name, outs, tmp_path):
    names = [k for k, _ in kernels(device_code(name, tmp_path), "product_tile_kernel")]
    for out in outs:
        assert [k for k in names if out in k and "Li4ELi4E" in k], (out, "tiles of 128 x 128")
        assert not [k for k in names if out in k and "Li8ELi8E" in k], (out, "tiles of 256 x 256")
