"""CPU checks of the adapters' flag for mixed batches: where it is taken, and the workspace that
it asks for, which says nothing about the number of adapters."""
import pytest

from test_lora_abi import K, M, MODE, N, OK, P, R, T, L, lib, m  # noqa: F401 (lib, m: fixtures)

MIXED = 8


def test_flag_is_taken_by_the_adapters_calls_alone(lib, m):  # noqa: F811
    import ctypes
    n = ctypes.c_size_t()
    for flags, want in ((0, OK), (MIXED, OK), (MIXED | 1, OK), (MIXED | 2, MODE), (16, MODE)):
        assert lib.fp8_lora_fprop_ws_bytes(M, N, K, R, flags, ctypes.byref(n)) == want, flags
        assert lib.fp8_lora_backward_ws_bytes(M, N, K, R, 3, flags, ctypes.byref(n)) == want, flags
    need = m.fp8_lora_fprop_ws_bytes(100, N, K, R, mixed=True)
    short = lib.fp8_lora_fprop(T(100, K), T(N, K, 1), L(), P, None, P, N, MIXED, P, need - 1, None)
    assert short == 8  # FP4_ERR_WORKSPACE
    assert lib.fp8_gemm(T(M, K), T(N, K, 1), P, 0, N, MIXED, P, 1 << 20, None) == MODE


@pytest.mark.parametrize("fast", [False, True])
def test_workspace(m, fast):  # noqa: F811
    """A mixed batch of 65 to 512 tokens has room for the product's binary32 partials."""
    for tokens in (1, 64, 65, 300, 512, 513, 4000):
        plain, mixed = (m.fp8_lora_fprop_ws_bytes(tokens, N, K, R, fast=fast, mixed=v) for v in (False, True))
        assert (mixed >= 4 * tokens * N) if 65 <= tokens <= 512 else mixed == plain, tokens
    # as many columns as fit a launch, 16776960 / 512 groups of 256, and more, whose partials are not asked for
    assert m.fp8_lora_fprop_ws_bytes(512, 8388352, 8, 8, mixed=True) > 4 * 512 * 8388352
    assert m.fp8_lora_fprop_ws_bytes(512, 8400000, 8, 8, mixed=True) == m.fp8_lora_fprop_ws_bytes(512, 8400000, 8, 8)
