"""A served attention layer over a paged KV cache and a block-quantised FP8 checkpoint, in fp64: TEST
INFRASTRUCTURE ONLY.

Only the tests use this module; the product path never imports it.  It shares nothing with the CUDA
library: numpy, straight from the definitions (block scales over 128 values; RMSNorm; the rotary
embedding of Su et al., "RoFormer", 2021; softmax attention).
"""
from __future__ import annotations

import numpy as np

from . import bf16_round, bf16_value

BLOCK = 128


def e4m3_value(codes: np.ndarray) -> np.ndarray:
    """e4m3 (finite-only) bytes -> fp64: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def block_scales(x: np.ndarray) -> np.ndarray:
    """fp64 [M][K] -> scales [M][ceil(K / 128)] = max(max |x| / 448, 2^-126) of every group."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    s = np.empty((M, kb))
    for b in range(kb):
        s[:, b] = np.maximum(np.abs(x[:, b * BLOCK:(b + 1) * BLOCK]).max(axis=1) / 448.0, 2.0 ** -126)
    return s


def spread(s: np.ndarray, K: int) -> np.ndarray:
    """Scales [M][ceil(K / 128)] -> [M][K]."""
    return np.repeat(s, BLOCK, axis=1)[:, :K]


def add_rmsnorm(x: np.ndarray, residual: np.ndarray | None, weight: np.ndarray | None, eps: float):
    """x: fp32 values [M][K] (fp64 array), residual: bf16 bits or None -> (h bf16 bits, y fp64).  The sum is
    rounded to fp32, then to bf16."""
    t = np.asarray(x, np.float32)
    if residual is not None:
        t = t + bf16_value(residual).astype(np.float32)
    h = bf16_round(t.astype(np.float64))
    v = bf16_value(h)
    y = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    return h, y


def linear_block(xq, xs, wq, ws):
    """e4m3 bytes xq [M][K], wq [N][K], fp32 scales xs [M][KB], ws [ceil(N/128)][KB] -> (y, sum |x w|)."""
    K, N = xq.shape[1], wq.shape[0]
    x = e4m3_value(xq) * spread(np.asarray(xs, np.float64), K)
    w = e4m3_value(wq) * spread(np.repeat(np.asarray(ws, np.float64), BLOCK, axis=0)[:N], K)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def norm_rope(x, weight, eps, pos, inv_freq, interleaved):
    """x: fp64 [T][H][D], pos [T] -> (rotated values, the pair magnitudes: each element's error scale)."""
    D = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(weight, np.float64)
    f = np.asarray(inv_freq, np.float64)
    half = len(f)
    a = np.asarray(pos, np.float64)[:, None, None] * f
    i = np.arange(half) * 2 if interleaved else np.arange(half)
    j = i + 1 if interleaved else i + half
    out, mag = x.copy(), np.abs(x)
    out[..., i] = x[..., i] * np.cos(a) - x[..., j] * np.sin(a)
    out[..., j] = x[..., i] * np.sin(a) + x[..., j] * np.cos(a)
    mag[..., i] = mag[..., j] = np.hypot(x[..., i], x[..., j])
    assert D >= 2 * half
    return out, mag


def paged_attention(q, k_cache, v_cache, pages, kv_len, scale, gate=None):
    """q: fp64 [S][Hq][D]; caches fp64 [n_pages][Hkv][P][D]; pages [S][max_pages]; kv_len [S].  Pages outside
    the cache are left out.  Returns (out, sum p |v| times the gate, lse, max over t of sum |q k| scale)."""
    S, Hq, D = q.shape
    n_pages, Hkv, P = k_cache.shape[:3]
    G = Hq // Hkv
    out, mag = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
    lse, dot = np.full((S, Hq), -np.inf), np.zeros((S, Hq))
    for s in range(S):
        n = int(kv_len[s])
        if n <= 0 or n > pages.shape[1] * P:
            continue
        t = np.arange(n)
        pg = pages[s][t // P]
        t = t[(pg >= 0) & (pg < n_pages)]
        if len(t) == 0:
            continue
        pg = pages[s][t // P]
        for g in range(Hkv):
            k, v = k_cache[pg, g, t % P], v_cache[pg, g, t % P]
            qq = q[s, g * G:(g + 1) * G]
            sc = scale * (qq @ k.T)
            m = sc.max(axis=1, keepdims=True)
            e = np.exp(sc - m)
            z = e.sum(axis=1, keepdims=True)
            out[s, g * G:(g + 1) * G] = e / z @ v
            mag[s, g * G:(g + 1) * G] = e / z @ np.abs(v)
            lse[s, g * G:(g + 1) * G] = (m + np.log(z))[:, 0]
            dot[s, g * G:(g + 1) * G] = abs(scale) * (np.abs(qq) @ np.abs(k).T).max(axis=1)
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-gate))
        out, mag = out * sg, mag * sg
    return out, mag, lse, dot
