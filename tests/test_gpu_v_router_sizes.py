"""Router sizes between those of the other router tests: the last expert of
each count of experts a lane holds and the first of the next, and 385 to 512."""
import pytest

from tests.gpu_util import require_gpu
from tests import test_gpu_k_router as router

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, k, score, bias, renorm, dtype
    (3, 64, 5, "softmax", True, False, "bf16"),
    (6, 128, 8, "sigmoid", True, True, "fp32"),
    (5, 129, 8, "softmax", False, False, "fp16"),
    (5, 256, 8, "softmax", True, True, "fp32"),
    (5, 257, 8, "sigmoid", True, False, "bf16"),
    (9, 385, 8, "sigmoid", True, True, "fp32"),
    (9, 400, 8, "softmax", False, False, "bf16"),
    (7, 448, 12, "softmax", True, False, "fp32"),
    (17, 512, 10, "softmax", False, True, "fp16"),
    (17, 512, 64, "sigmoid", True, True, "bf16"),
    (4, 1024, 9, "sigmoid", False, True, "bf16"),
    (4, 1024, 32, "softmax", True, False, "fp32"),
    (3, 2000, 16, "sigmoid", True, False, "fp16"),
]


@pytest.mark.parametrize("T,E,k,score,bias,renorm,dtype", CASES)
def test_choice_weights_and_gradient(T, E, k, score, bias, renorm, dtype):
    require_gpu()
    router.test_topk(T, E, k, score, bias, renorm, dtype)
    router.test_gradient(T, E, k, score, bias, renorm, dtype)
