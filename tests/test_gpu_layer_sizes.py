"""Layer sizes at which a launch's shared memory passes what a kernel has without asking."""
import numpy as np
import pytest

from block_scaled_fp4_moe_gb300 import _build
from gpu_support import bf16_to_f64, check_output, random_problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("T,I", [(12, 6080), (12, 6144), (3, 6144)])
def test_inter_sizes_around_48_kb_of_sums(T, I):
    """8 I bytes of sums beside the kernel's 64 of its own: 48 KB and 64 bytes at I = 6144."""
    p = random_problem(T, 512, 4, 2, I, seed=I + T)
    got = p.forward()
    r = p.oracle_route()
    np.testing.assert_array_equal(got["ids"], r["ids"])
    check_output(got["y"], p.oracle_tokens(r, np.arange(T))["y"], f"T={T} I={I}")
    assert np.isfinite(bf16_to_f64(got["y"])).all()
