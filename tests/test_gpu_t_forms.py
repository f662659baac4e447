"""Forms of the grouped products' tiles that the other tile tests reach with
one case or one output type: MXFP4 in 128 x 128 tiles with every tile height
and in 256 x 256, and the input gradient in one LDS stage with FP32 outputs."""
import pytest
import torch

from tests.gpu_util import require_gpu
from tests import test_gpu_o_tiles as tiles

pytestmark = pytest.mark.gpu

HEIGHTS = [300, 257, 256, 129, 193, 1, 0, 64, 97, 33]      # 1330 rows
CASES = [("dgrad", 40, 72, 4104, 9000), ("dgrad", 30, 136, 4104, HEIGHTS * 3)]
MX_CASES = [(10, 1032, 2080, HEIGHTS), (10, 2056, 1056, HEIGHTS), (10, 4104, 4128, HEIGHTS),
            (32, 4104, 2080, [129, 144, 160, 150, 1, 32, 270, 140] * 4)]


@pytest.mark.parametrize("way,E,N,K,counts", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forms(way, E, N, K, counts, dtype):
    require_gpu()
    tiles.test_every_tile_form_is_exact(way, E, N, K, counts, dtype)


@pytest.mark.parametrize("E,N,K,counts", MX_CASES)
def test_forms_of_mxfp4(E, N, K, counts):
    require_gpu()
    tiles.test_every_tile_form_of_mxfp4_is_exact(E, N, K, counts)
