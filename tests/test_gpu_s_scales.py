"""MXFP4 products whose groups end with a tile of up to 32 rows, over
contractions of one to many pairs of steps: each pair's scales stay apart.
Exact on small integers under scales that differ from row to row and from
block to block."""
import pytest

from tests.gpu_util import require_gpu
from tests import test_gpu_o_tiles as tiles

pytestmark = pytest.mark.gpu

ENDS = [129, 144, 160, 150, 1, 32, 270, 140]     # 128 x 128 tiles: last ones of 1 to 32 rows


@pytest.mark.parametrize("K", [32, 256, 544, 1056, 2080, 4128])
@pytest.mark.parametrize("E,N", [(8, 2056), (32, 4104)])     # two, and up to 1056 four workgroups a compute unit
def test_last_tiles_of_few_rows(E, N, K):
    require_gpu()
    tiles.test_every_tile_form_of_mxfp4_is_exact(E, N, K, ENDS * (E // 8))
