"""Each form of the grouped products' tiles in each direction, by sizes for
which it is the one taken, exact on small integers: 256 x 256 with the last
rows of groups in each lower tile, 128 x 128 with many and few steps, and both
tiles whose contraction is split over waves."""
import pytest
import torch

from tests.gpu_util import require_gpu
from tests import test_gpu_o_tiles as tiles

pytestmark = pytest.mark.gpu

GROUPS = [17, 128, 150, 200, 256, 1, 0, 400, 229, 300, 135, 184]      # 2000 rows

CASES = [
    # 256 x 256
    ("fwd", 12, 4104, 1032, GROUPS), ("dgrad", 12, 1032, 4104, GROUPS), ("wgrad", 6, 2056, 2056, 6000),
    ("wgrad", 6, 2176, 2056, [1000, 1001, 0, 1999, 1, 1999]),
    # 128 x 128, two or four workgroups a compute unit
    ("wgrad", 12, 520, 520, 5000), ("wgrad", 16, 1032, 520, 3000),
    # 64 x 64
    ("fwd", 16, 1032, 2056, 300), ("dgrad", 16, 2056, 1032, 300), ("wgrad", 8, 264, 264, 1500),
    # 32 x 64
    ("fwd", 1, 4104, 4104, [16]), ("fwd", 1, 1000, 7176, [64]), ("dgrad", 1, 7176, 264, [20]),
    ("dgrad", 1, 4104, 1032, [64]), ("dgrad", 3, 4104, 392, [1, 33, 0]), ("wgrad", 1, 264, 392, 4001),
]


@pytest.mark.parametrize("way,E,N,K,counts", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forms(way, E, N, K, counts, dtype):
    require_gpu()
    tiles.test_every_tile_form_is_exact(way, E, N, K, counts, dtype)


@pytest.mark.parametrize("E,N,K,counts", [(12, 4104, 4128, GROUPS), (16, 1032, 4128, 300), (20, 512, 7168, 1000),
                                          (3, 264, 4128, [1, 20, 0]), (1, 4104, 7200, [64]), (1, 392, 2080, [200])])
def test_forms_of_mxfp4(E, N, K, counts):
    require_gpu()
    tiles.test_every_tile_form_of_mxfp4_is_exact(E, N, K, counts)
