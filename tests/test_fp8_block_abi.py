"""CPU checks of the gated block's C ABI by flags (every call fails its host-side checks)."""
import ctypes

import pytest

from test_fp8_abi import MODE, P, T, WORKSPACE, lib, m  # noqa: F401


@pytest.mark.parametrize("flags,status", [(0, WORKSPACE), (1, WORKSPACE), (2, MODE), (1 << 31, MODE)])
def test_flags(lib, flags, status):  # noqa: F811
    from nvfp4_bit_microscaled_amd.fp8 import fp8_ffn_buffers, fp8_tensor
    M, K, F = 40, 100, 260
    fprop, back = lib.fp8_ffn_fprop_flags, lib.fp8_ffn_backward_flags
    assert fprop(T(M, K), T(F, K, 1), T(F, K, 1), T(K, F, 1), T(M, F), P, P, P, K, flags, P, 0, None) == status
    bufs = ctypes.byref(fp8_ffn_buffers(*(fp8_tensor(0x100000, 0x200000, r, c, 0)
                                          for r, c in ((M, F), (M, F), (F, M), (F, M), (F, M)))))
    assert back(T(M, K), T(K, M), T(K, M), T(K, F, 1), T(K, F, 1), T(F, K, 1), P, P, bufs, P, P, P, P, flags, P, 0,
                None) == status
