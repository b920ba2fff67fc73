"""The most rows that the expert gradient takes, refused on the host."""
import pytest

import sparse_mixture_experts_topk_gb300 as moe

A = 1 << 20          # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


class Ws(int):
    """An address with a size, as a workspace tensor has."""

    def numel(self):
        return 1 << 62


@pytest.mark.parametrize("kind,room", [("f32", 64), ("bf16_simt", 64), ("bf16", 256)])
def test_row_numbers_stay_in_32_bits(kind, room):
    """A kernel's row numbers go up to a tile past an expert's end, so the last
    rows below 2^31 are refused, whichever gradients are asked for."""
    dtype, flags = moe.MOE_F32 if kind == "f32" else moe.MOE_BF16, moe.MOE_FLAG_SIMT_FFN if kind == "bf16_simt" else 0
    for rows in (2 ** 31 - room, 2 ** 31 - 1):
        d = moe.make_desc(rows, 8, 1, 1, 8, dtype=dtype, flags=flags)
        for dx, dW1, db1, dW2, db2 in ((A, A, A, A, A), (None, None, None, A, A)):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_expert_ffn_backward(d, A, A, A, A, A, A, A, dx, dW1, db1, dW2, db2, Ws(A), stream=0)
            assert e.value.code == moe.MOE_ERR_UNSUPPORTED
