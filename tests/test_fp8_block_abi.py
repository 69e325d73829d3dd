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


def test_workspaces(m):  # noqa: F811
    """Each call's own workspace: no place for the backward pass's dh (4 M F bytes) in the
    forward one, none in the fused backward step's, and never more than the common one."""
    M, K, F = 16384, 5120, 20480
    dh = 4 * M * F
    assert m.fp8_ffn_fprop_ws_bytes(M, K, F, keep=True, fast=True) < dh // 4
    assert m.fp8_ffn_fprop_ws_bytes(M, K, F, keep=True) < dh // 4
    assert dh <= m.fp8_ffn_fprop_ws_bytes(M, K, F) < 1.25 * dh  # g and u in bf16
    assert m.fp8_ffn_backward_ws_bytes(M, K, F, fast=True) < dh // 4
    assert m.fp8_ffn_backward_ws_bytes(M, K, F) >= dh
    for s in ((1, 64, 128), (8, 5120, 20480), (300, 300, 1100), (2500, 130, 4000), (1900, 130, 2205), (4100, 1030, 6100),
              (0, 10, 10), (10, 0, 10), (10, 10, 0)):
        most = m.fp8_ffn_ws_bytes(*s)
        for fast in (False, True):
            assert m.fp8_ffn_backward_ws_bytes(*s, fast=fast) <= most
            for keep in (False, True):
                assert m.fp8_ffn_fprop_ws_bytes(*s, keep=keep, fast=fast) <= most
    with pytest.raises(m.Fp4Error):
        m.fp8_ffn_fprop_ws_bytes(-1, 4, 4)
    with pytest.raises(m.Fp4Error):
        m.fp8_ffn_backward_ws_bytes(4, -1, 4)


@pytest.mark.parametrize("fast", [0, 1])
def test_workspace_refusals(lib, m, fast):  # noqa: F811
    from nvfp4_bit_microscaled_amd.fp8 import fp8_ffn_buffers, fp8_tensor
    M, K, F = 40, 2000, 2600
    for g, need in ((P, m.fp8_ffn_fprop_ws_bytes(M, K, F, True, bool(fast))),
                    (None, m.fp8_ffn_fprop_ws_bytes(M, K, F, False, bool(fast)))):
        assert need > 0
        assert lib.fp8_ffn_fprop_flags(T(M, K), T(F, K, 1), T(F, K, 1), T(K, F, 1), T(M, F), g, g, P, K, fast, P, need - 1,
                                       None) == WORKSPACE
    need = m.fp8_ffn_backward_ws_bytes(M, K, F, bool(fast))
    bufs = ctypes.byref(fp8_ffn_buffers(*(fp8_tensor(0x100000, 0x200000, r, c, 0)
                                          for r, c in ((M, F), (M, F), (F, M), (F, M), (F, M)))))
    assert lib.fp8_ffn_backward_flags(T(M, K), T(K, M), T(K, M), T(K, F, 1), T(K, F, 1), T(F, K, 1), P, P, bufs, P, P, P,
                                      P, fast, P, need - 1, None) == WORKSPACE
    # g off by 2 bytes: the fused step is not open to it, and dh needs its place
    M, K, F = 2500, 136, 4008
    need = m.fp8_ffn_backward_ws_bytes(M, K, F, True)
    assert need < 4 * M * F
    bufs = ctypes.byref(fp8_ffn_buffers(*(fp8_tensor(0x100000, 0x200000, r, c, 0)
                                          for r, c in ((M, F), (M, F), (F, M), (F, M), (F, M)))))
    assert lib.fp8_ffn_backward_flags(T(M, K), T(K, M), T(K, M), T(K, F, 1), T(K, F, 1), T(F, K, 1),
                                      ctypes.c_void_p(0x10002), P, bufs, P, P, P, P, 1, P, 4 * M * F - 1, None) == WORKSPACE
