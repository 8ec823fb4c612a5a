"""The product of few tokens where its tiles just fit the GPU four times over and their
clusters of four do not all run at once (37 and 38 tiles on 152 SMs: the contraction is
then cut in three), and one tile further on, where the kernels for whole tiles take over."""
import pytest

from tests.test_gpu_gated import test_product as product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tiles", [36, 37, 38, 39])
@pytest.mark.parametrize("M", [40, 100, 128])
def test_tiles_about_a_quarter_of_the_sms(tiles, M):
    product(M, 128 * tiles - 24, 2048, "silu")


@pytest.mark.parametrize("tiles,M", [(19, 129), (12, 300), (13, 300), (9, 500), (10, 500)])
def test_tiles_of_several_rows(tiles, M):
    product(M, 128 * tiles, 2048, "gelu")
