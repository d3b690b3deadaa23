"""Row lengths at the end of 32 bits, where the kernels' counts of stages and segments would
wrap: refused on the host (the pointers here are not device memory)."""
import pytest

from fp4_weight_grouped_gb300 import binding, build_lib
from test_fp4_refusals import FAKE, GEMM, INVALID, QUANT

LONGEST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


@pytest.mark.parametrize("K", [LONGEST + 32, 2 ** 31 - 512, 2 ** 31 - 32])
def test_rows_whose_counts_would_wrap(lib, K):
    assert lib.moe_fp4_quantize(*{**QUANT, "K": K, "x_stride": K, "rows": 1, "x_rows": 1}.values()) == INVALID
    assert lib.moe_fp4_grouped_gemm(*{**GEMM, "K": K, "rows": 1, "N": 1, "E": 1}.values()) == INVALID
    args = dict(ac=FAKE, asc=FAKE, a2=None, rows=1, K=K, wc=FAKE, wsc=FAKE, w2=None, fmt=0, sizes=FAKE, E=1, I=32, h2=None,
                hc=FAKE, hs=FAKE, ws=FAKE, wsb=256, stream=None)
    assert lib.moe_fp4_grouped_gemm_swiglu(*args.values()) == INVALID


def test_the_documented_limit(lib):
    """No rows: valid arguments return before a launch, or (without a GPU) at the device check."""
    for K in (32, LONGEST):
        assert lib.moe_fp4_grouped_gemm(*{**GEMM, "K": K, "rows": 0}.values()) != INVALID
        assert lib.moe_fp4_quantize(*{**QUANT, "K": K, "rows": 0}.values()) != INVALID
