"""One row as torch may describe it: a stride that is not the width."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import BF16, EPS, FP32, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_row_of_a_transpose(fp4, dtype):
    n = 300
    x = rnd(n, 1, dtype=dtype).cuda().t()
    assert x.stride(0) == 1
    q, qt = fp4.Fp8Tensor(1, n), fp4.Fp8Tensor(n, 1)
    fp4.fp8_quantize(x, q, qt)
    ref.assert_quantized(q, x.cpu())
    ref.assert_quantized(qt, x.cpu().t())
    y, z, w = fp4.Fp8Tensor(1, n), fp4.Fp8Tensor(1, n), torch.ones(n, device="cuda")
    fp4.fp8_rms_norm(x, w, EPS, y)
    fp4.fp8_rms_norm(x.clone(memory_format=torch.contiguous_format).reshape(-1)[None], w, EPS, z)
    assert torch.equal(y.codes, z.codes)
    b, c = ref.put(fp4, rnd(n, n)), torch.empty(n, 1, device="cuda").t()
    fp4.fp8_gemm(q, b, c)
    d = torch.empty(1, n, device="cuda")
    fp4.fp8_gemm(q, b, d)
    assert torch.equal(c, d)
