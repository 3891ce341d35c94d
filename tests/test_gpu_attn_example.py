"""examples/attention_step.py: the operators and the MoE layer together, a few
steps replayed from a graph whose lengths and free list advance on the device."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("new", [1, 3])
def test_attention_step_example(new):
    import attention_step
    out = attention_step.main(["--requests", "5", "--context", "70", "--new", str(new), "--steps", "30", "--hidden", "512"])
    assert out["finite"] and out["context"] == [70 + 30 * new] * 5
