"""The CUDA-core expert gradient with more row tiles than a grid's second
dimension holds (65535)."""
import pytest

import sparse_mixture_experts_topk_gb300 as moe
from test_gpu_training import check_ffn, ffn_case, run_ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mixture_experts_topk_gb300 import build
    build.build()
    moe.lib()


def test_ffn_gradient_of_many_rows():
    c = ffn_case([65535 * 64 - 63, 130], 8, 8, "gelu", True, "f32", 31)
    check_ffn(c, run_ffn(c))


def test_second_products_gradients_alone_of_many_rows():
    c = ffn_case([70, 65535 * 64], 8, 16, "gelu", False, "f32", 32)
    check_ffn(c, run_ffn(c, want=("dW2", "db2")), which=("dW2", "db2"))
