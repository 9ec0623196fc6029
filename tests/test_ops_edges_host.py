"""Further refusals of the operators next to the routed half, on a machine without a GPU."""
import pytest

from tests.test_ops_host import B, matmul_args  # noqa: F401  (B is a fixture)
import ctypes as C


@pytest.mark.parametrize("cta,wait_us,frag", [(-1, 1, "cta"), (0, 2_000_001, "wait_us")])
def test_held_product_refusals(B, cta, wait_us, frag):  # noqa: F811
    st = B.lib.ts_moe_debug_fp8_matmul_held(C.byref(matmul_args(B)), cta, wait_us, None)
    assert st == 1 and frag in B.lib.ts_moe_last_error(None).decode()
