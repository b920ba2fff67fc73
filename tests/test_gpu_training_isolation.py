"""The expert gradient: an expert's NaN and infinities stay its own wherever
they come from, and the benchmark's widths against the oracle."""
import numpy as np
import pytest

import sparse_mixture_experts_topk_gb300 as moe

from harness import as_f64, to_np
from test_gpu_training import INF_BF16, NAN_BF16, check_ffn, ffn_case, run_ffn

pytestmark = pytest.mark.gpu

POISON = {"bf16": (NAN_BF16, INF_BF16), "f32": (np.nan, np.inf)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_mixture_experts_topk_gb300 import build
    build.build()
    moe.lib()


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("kind", ["bf16", "bf16_simt", "f32"])
@pytest.mark.parametrize("where", ["rows", "W1", "b1", "W2"])
def test_an_experts_non_finite_values_stay_its_own(where, kind, act):
    """Experts next to the spoilt one share its blocks of rows and, F being no
    multiple of a tile, its tiles of weight rows."""
    dtype, flags = kind[:4].rstrip("_"), moe.MOE_FLAG_SIMT_FFN if kind == "bf16_simt" else 0
    counts = [20, 33, 270, 5]
    clean = run_ffn(ffn_case(counts, 136, 200, act, True, dtype, 6), flags)
    for bad in (1, 2):
        for value in POISON[dtype]:
            c = ffn_case(counts, 136, 200, act, True, dtype, 6)
            rows, nan = slice(c["offs"][bad], c["offs"][bad + 1]), value == NAN_BF16 or value != value
            for k in ("x", "h", "dy") if where == "rows" else ():
                c[k][rows] = value
            if where == "b1":
                c["b1"][bad] = np.nan if nan else np.inf
            elif where != "rows":
                c[where][bad] = value
            dirty = run_ffn(c, flags)
            for e in set(range(4)) - {bad}:
                r = slice(c["offs"][e], c["offs"][e + 1])
                assert (to_np(clean["dx"])[r] == to_np(dirty["dx"])[r]).all(), (bad, e)
                for k in ("dW1", "db1", "dW2", "db2"):
                    assert (to_np(clean[k])[e] == to_np(dirty[k])[e]).all(), (bad, e, k)
            spoilt = "dW2" if where == "rows" else "dx"
            got = as_f64(dirty[spoilt])
            got = got[bad] if spoilt == "dW2" else got[rows]
            if where != "b1" or nan:                  # a slope at infinity may be finite
                assert not np.isfinite(got).any(), (bad, spoilt)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_ffn_gradient_at_the_benchmarks_widths(act):
    c = ffn_case([270, 0, 77], 3584, 2560, act, True, "bf16", 51)
    check_ffn(c, run_ffn(c))
