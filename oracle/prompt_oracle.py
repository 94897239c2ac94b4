"""fp64 CPU oracle of the prompt side: rotary positions, the row append with
its norm and rotation, latent expansion and the expanded attention.

TEST INFRASTRUCTURE ONLY, like mla_oracle: plain numpy in float64, sharing no
code with the CUDA path and importing nothing from it.  Inputs are float64
arrays of values (bf16 and E4M3 values are exact in float64).

Pins (tests/test_prompt_oracle_pins.py): rotation against complex numbers,
norm preservation and relative positions; the scalings against their limits;
the norm against its definition by a second route; expansion and attention
against the absorbed attention of mla_oracle on the same latents, and against
hand-made cases (one key, equal keys, nothing seen).
"""
from __future__ import annotations

import math

import numpy as np


def rope_inv_freq(theta=10000.0, scaling="none", factor=1.0, original=4096, beta_fast=32.0, beta_slow=1.0):
    """Angle per position of the 32 pairs, float64 [32]."""
    inv = np.array([theta ** (-i / 32.0) for i in range(32)])
    if scaling == "none":
        return inv
    if scaling == "linear":
        return inv / factor

    def pair(beta):
        return 32.0 * math.log(original / (2.0 * math.pi * beta)) / math.log(theta)

    lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), 63)
    r = np.clip((np.arange(32) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return inv * (1.0 - r) + inv / factor * r


def rope_rotate(x, positions, inv_freq, interleaved=True, amplitude=1.0):
    """x [T, ..., 64] rotated by positions [T]."""
    x = np.asarray(x, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * inv_freq
    ang = ang.reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (32,))
    c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude
    out = np.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    ra, rb = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0::2], out[..., 1::2] = ra, rb
    else:
        out[..., :32], out[..., 32:] = ra, rb
    return out


def rms_norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * weight


def append_values(rows, positions, inv_freq, weight=None, eps=1e-6, interleaved=True, amplitude=1.0):
    """The values of new cache rows, float64 [T, 576], before their rounding to the cache's type."""
    rows = np.asarray(rows, dtype=np.float64)
    lat = rows[:, :512] if weight is None else rms_norm(rows[:, :512], weight, eps)
    return np.concatenate([lat, rope_rotate(rows[:, 512:], positions, inv_freq, interleaved, amplitude)], axis=1)


def expand_rows(latents, w_kc, w_vc):
    """latents [T, 512] -> keys [T, H, 128] and values [T, H, 128]."""
    return (np.einsum("tr,hnr->thn", latents, w_kc, optimize=True),
            np.einsum("tr,hrn->thn", latents, w_vc, optimize=True))


def prefill_attention(q, k_nope, k_rope, v, q_indptr, kv_indptr, sm_scale, causal=True):
    """Expanded attention of ragged sequences: q [Tq,H,192], k_nope and v [Tk,H,128], k_rope [Tk,64].
    Returns out [Tq,H,128], lse [Tq,H] and the weighted sum of |v| (for error bounds)."""
    Tq, H = q.shape[:2]
    out, mag = np.zeros((Tq, H, 128)), np.zeros((Tq, H, 128))
    lse = np.full((Tq, H), -np.inf)
    for b in range(len(q_indptr) - 1):
        q0, q1, k0, k1 = (int(x) for x in (q_indptr[b], q_indptr[b + 1], kv_indptr[b], kv_indptr[b + 1]))
        for i in range(q0, q1):
            n = k1 - k0 if not causal else min(k1 - k0, max(0, (i - q0) + 1 + (k1 - k0) - (q1 - q0)))
            if n == 0:
                continue
            # only the keys that the row sees are touched
            s = sm_scale * (np.einsum("hd,jhd->hj", q[i, :, :128], k_nope[k0:k0 + n]) +
                            q[i, :, 128:] @ k_rope[k0:k0 + n].T)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            t = p.sum(axis=1, keepdims=True)
            p /= t
            out[i] = np.einsum("hj,jhd->hd", p, v[k0:k0 + n])
            mag[i] = np.einsum("hj,jhd->hd", p, np.abs(v[k0:k0 + n]))
            lse[i] = (m + np.log(t))[:, 0]
    return out, lse, mag
