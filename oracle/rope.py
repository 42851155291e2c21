"""Norms of queries and keys for each head, and their position rotation, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

[P3] "Indexer 的结构与计算流程": the indexer norms its key (k_norm) and turns part of each query and key (rotary width
index_head_dim / 2, half-split or interleaved by indexer_rope_interleave); [P3] "稀疏 MLA 的前向路径": the latent is normed over its
kv_lora_rank 512 values and its 64 rope values are turned.
"""
from __future__ import annotations

import numpy as np


def norm(x, kind, eps, weight=None, bias=None, norm_dim=None):
    """x [..., D] float64; kind None, "rms" or "layer" over the first norm_dim dims."""
    x = np.array(x, dtype=np.float64)
    if kind is None:
        return x
    n = x.shape[-1] if norm_dim is None else norm_dim
    y = x[..., :n]
    if kind == "layer":
        y = y - y.mean(axis=-1, keepdims=True)
    y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    x[..., :n] = y
    return x


def pairs(rot_dim, rot_start, interleaved):
    """The dims (a, b) of each turned pair."""
    i = np.arange(rot_dim // 2)
    return (rot_start + 2 * i, rot_start + 2 * i + 1) if interleaved else (rot_start + i, rot_start + rot_dim // 2 + i)


def rotate(x, cos_sin_rows, rot_start, interleaved):
    """x [T, H, D] float64, cos_sin_rows [T, rot_dim] the tokens' rows of the table."""
    y = np.array(x, dtype=np.float64)
    cs = np.asarray(cos_sin_rows, np.float64)
    rot = cs.shape[1]
    a, b = pairs(rot, rot_start, interleaved)
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    p, q = y[..., a], y[..., b]
    y[..., a], y[..., b] = p * c - q * s, p * s + q * c
    return y
