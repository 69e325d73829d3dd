"""The plan of the products under the adapters' calls on the CPU: the sizes of the GPU tests
reach the kernels and splits that they are for."""
import pytest

import lora_paths
from test_fp8_plan import blocks, plan, product  # noqa: F401 (plan: a fixture)


@pytest.mark.parametrize("name", lora_paths.PATHS)
def test_paths(plan, name):  # noqa: F811
    (M, out, contraction, fast), want = lora_paths.PATHS[name]
    assert product(plan, M, out, blocks(contraction), fast) == want
