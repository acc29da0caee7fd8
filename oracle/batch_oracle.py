"""Plain CPU oracle of the batched path's operators, float64.

TEST INFRASTRUCTURE ONLY, like moe_oracle (whose number-format functions it
uses): nothing in the product package imports or runs this file.

  norm_quant  residual addition, root-mean-square norm, 8-bit rows
  qdense      8-bit rows times an 8-bit matrix, scales, softcap
  logits      penalties, biases, mask, greedy token
"""
from __future__ import annotations

import numpy as np

from oracle.head_oracle import softcap as cap_of
from oracle.moe_oracle import bf16_to_f64


def to_bf16(v) -> np.ndarray:
    """bf16 bits of values, infinities and NaN among them, nearest with ties to
    even.  By way of fp32, which changes no result for the sum of two bf16
    values: it is exact in fp32, or lies within 2^-16 of a bf16 value."""
    with np.errstate(over="ignore"):
        u = np.asarray(v, dtype=np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    up = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    return np.where((u & 0x7FFFFFFF) > 0x7F800000, 0x7FC0, up).astype(np.uint16)


def norm_quant(h_bits, y_bits=None, g_bits=None, eps: float = 1e-6) -> dict:
    """s (bf16 bits), q (int8), scales and x (float64, unrounded) of bf16 rows.
    A row with a non-finite s or u has codes 0 and NaN scales and x."""
    h = bf16_to_f64(h_bits)
    with np.errstate(invalid="ignore", over="ignore"):
        s_bits = np.asarray(h_bits) if y_bits is None else to_bf16(h + bf16_to_f64(y_bits))
        s = bf16_to_f64(s_bits)
        u = s if g_bits is None else s * bf16_to_f64(g_bits)
        fine = np.isfinite(u).all(axis=1) & np.isfinite(s).all(axis=1)
        m = np.abs(u).max(axis=1)
        r = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
        safe = np.where(fine & (m > 0), m, 1.0)
        q = np.rint(np.where(fine[:, None], u, 0.0) * 127.0 / safe[:, None])  # rint: ties to even
        scales = np.where(fine, m * r / 127.0, np.nan)
        x = np.where(fine[:, None], u * r[:, None], np.nan)
    return {"s": s_bits, "q": q.astype(np.int8), "scales": scales, "x": x}


def int_product(x, w) -> np.ndarray:
    """sum_k x[t, k] w[n, k] of int8 codes, exact (every sum is below 2^53), float64."""
    return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T


def qdense(x, xs, w, ws, softcap: float = 0.0) -> np.ndarray:
    """cap(xs[t] ws[n] sum_k x[t, k] w[n, k]), float64 [T, N]."""
    z = int_product(x, w) * np.asarray(xs, dtype=np.float64)[:, None] * np.asarray(ws, dtype=np.float64)[None, :]
    return cap_of(z, softcap) if softcap > 0 else z


def logits(lg, rows: list, mask=None) -> tuple[np.ndarray, np.ndarray]:
    """Processed logits (float64 [T, V]) and, per value, the sum of the
    magnitudes of the results of its operations (the scale of its rounding
    errors).  rows[t]: a dict with history, prompt (its length), repetition,
    presence, frequency, bias (list of (id, value), the last of an id
    counts); mask: bool [T, V], True where allowed."""
    v = np.asarray(lg, dtype=np.float64).copy()
    mag = np.zeros_like(v)
    T, V = v.shape
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for t, r in enumerate(rows):
            hist = [i for i in r.get("history", ())]
            made = hist[r.get("prompt", 0):]
            for i in sorted({i for i in hist if 0 <= i < V}):
                n = made.count(i)
                p = r.get("repetition", 1.0)
                v[t, i] = v[t, i] / p if v[t, i] > 0 else v[t, i] * p
                mag[t, i] += abs(v[t, i])
                if n:
                    f = r.get("frequency", 0.0) * n
                    v[t, i] -= f
                    mag[t, i] += abs(f) + abs(v[t, i])
                    v[t, i] -= r.get("presence", 0.0)
                    mag[t, i] += abs(v[t, i])
            for i, b in dict(r.get("bias", ())).items():
                if 0 <= i < V:
                    v[t, i] += b
                    mag[t, i] += abs(v[t, i])
    if mask is not None:
        v[~mask] = -np.inf
        mag[~mask] = 0.0
    return v, mag


def greedy(v) -> np.ndarray:
    """The first index of the largest finite value per row, -1 if there is none."""
    v = np.where(np.isfinite(v), v, -np.inf)
    best = v.max(axis=1)
    return np.where(best > -np.inf, v.argmax(axis=1), -1)
