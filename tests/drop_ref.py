"""Dropout's definition on the CPU (numpy and torch), for the tests: written from
include/nvfp4_amd_fp8.h and not from the library."""
import numpy as np
import torch


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def gain(p):
    """What a kept element is multiplied by, as a binary32 value."""
    return float(np.float32(65536.0 / (65536 - threshold(p))))


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on arrays of unsigned 64-bit integers that hold 32 bits."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (q >> u(32)) ^ c1 ^ u(k0), q & low, (p >> u(32)) ^ c3 ^ u(k1), p & low
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def keep(rows, cols, p, seed, offset=0, step=0):
    """The mask of a [rows][cols] tensor (bool)."""
    groups = -(-cols // 8)
    g = np.arange(rows * groups, dtype=np.uint64)
    at = (offset + step) % 2 ** 64
    fill = lambda v: np.full_like(g, v)  # noqa: E731
    words = philox(g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), fill(at & 0xFFFFFFFF), fill(at >> 32),
                   seed & 0xFFFFFFFF, seed >> 32)
    half = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    return torch.from_numpy(half.reshape(rows, groups * 8)[:, :cols] >= threshold(p))


def dropout(x, p, mask):
    """x (binary32) dropped out, each product rounded to binary32."""
    return torch.where(mask, x.float() * gain(p), torch.zeros(()))
