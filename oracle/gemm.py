"""Matrix product of FP8 E4M3 codes with a scale for each block of 128.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The codes and scales are those of the block-128 quantizer (``oracle.fp8``);
the weight's scales are per row and block of 128, or per 128 x 128 block.
"""
from __future__ import annotations

import numpy as np

from . import fp8


def gemm_fp8_block128(a, a_scale, w, w_scale, w_scale_rows: int) -> np.ndarray:
    """out[m, n] = sum over the blocks kb of a_scale[m, kb] * w_scale[n', kb] * sum_{k in kb} a[m, k] w[n, k],
    n' = n or n // 128, in float64."""
    a, w = np.asarray(a, np.uint8), np.asarray(w, np.uint8)
    M, K = a.shape
    N = w.shape[0]
    a_scale, w_scale = np.asarray(a_scale, np.float64), np.asarray(w_scale, np.float64)
    av, wv = fp8.decode_e4m3(a), fp8.decode_e4m3(w)
    out = np.zeros((M, N), dtype=np.float64)
    for kb in range(K // 128):
        part = av[:, 128 * kb:128 * kb + 128] @ wv[:, 128 * kb:128 * kb + 128].T
        out += part * np.outer(a_scale[:, kb], w_scale[np.arange(N) // w_scale_rows, kb])
    return out


def abs_terms(a, a_scale, w, w_scale, w_scale_rows: int) -> np.ndarray:
    """sum_k |a_scale * w_scale * a * w|: what a rounding error of the sum is relative to."""
    return gemm_fp8_block128(np.asarray(a) & 0x7F, np.abs(a_scale), np.asarray(w) & 0x7F, np.abs(w_scale),
                             w_scale_rows)
