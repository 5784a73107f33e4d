"""Sizes on both sides of where the 8-bit product goes from two blocks an SM to
one, and from whole to shared K.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

from tests import test_gpu_w8a8 as product  # noqa: E402
from tests.test_gpu_w8a8 import dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# blocks: of 148 SMs five eighths are 92.5; K is cut up to 256 shares
@pytest.mark.parametrize("tiles", [23, 24, 31, 32, 46, 47, 64, 65, 92, 93, 95, 96, 128, 129, 148, 149])
@pytest.mark.parametrize("M,K", [(1, 528), (16, 1040), (20, 528), (64, 1040)])
def test_tiles_about_the_borders(dev, tiles, M, K):  # noqa: F811
    N = tiles * 128 - 3
    product.test_product_of_given_codes(dev, M, N, K, True)
    product.test_linear_is_quantizer_and_product(dev, M, N, K)
