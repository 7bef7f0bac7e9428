"""Inputs and tolerances shared by the attention operators' GPU tests.

Tolerances count roundings.  u is half a step of the storage type relative to the
value (finfo.eps / 2), f = 2^-24 that of fp32.

scores     an fp32 dot product of d terms in any order is off by at most
           (d + 2) f sum |q_e k_e|, the scale and the base-2 logarithm's factor add
           3 roundings of a value no larger: ds = (d + 6) f * bound, where bound is
           the largest |scale| sum |q_e k_e| of the row.
weights    exp(s - max): ds for the score, ds for the maximum, and the hardware
           exponential's 2 units: relative 2 ds + 4 f; their fp32 sum adds n f.
O          each weight enters rounded to the storage type (u) and with the relative
           error above, the sum over keys is fp32 (n f), all times terms
           A = sum w |v|; rescaling by running maxima adds one rounding a step
           (at most n of them, counted with another n f); the division 2 f; the
           final rounding u |O|.  An fp16 weight below 2^-14 is off by at most 2^-25
           instead of u of itself: n 2^-25 max|v| more.
lse        ds + (2 n + 8) f + 2 f |lse|.
mass       a weight from a given lse: ds + 2 f |lse| + 4 f relative; sums of 16 terms,
           then of at most 256 of those: 272 f; the final rounding f.
"""
from __future__ import annotations

import numpy as np
import torch

F = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def u_of(dt):
    return torch.finfo(DT[dt]).eps / 2


def host(t):
    return t.detach().to("cpu", torch.float64).numpy()


def score_err(ref_bound, d):
    return (d + 6) * F * ref_bound


def out_tol(dt, ref_O, A, bound, n, d, vmax):
    """bound broadcasts against O's leading dims."""
    ds = score_err(bound, d)[..., None]
    u = u_of(dt)
    tol = A * (u + 4 * ds + (4 * n + 16) * F) + (u + 2 * F) * np.abs(ref_O)
    if dt == "f16":
        tol = tol + n * 2.0 ** -25 * vmax + 2.0 ** -25
    return tol + 1e-30


def lse_tol(lse, bound, n, d):
    fin = np.where(np.isfinite(lse), lse, 0.0)
    return score_err(bound, d) + (2 * n + 8) * F + 2 * F * np.abs(fin)


def mass_rel(r, d):
    """Relative error of weights formed from a given lse (r: the oracle's results)."""
    if r["lse"].size == 0:
        return 0.0
    fin = np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0)).max()
    return 2 * score_err(float(r["bound"].max()), d) + 4 * F * fin + (272 + 8) * F


def close(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    both = (got == ref) | (np.isnan(got) & np.isnan(ref))
    err = np.where(both, 0.0, np.abs(got - ref))
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        t = np.broadcast_to(tol, ref.shape)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, first at {i}: "
                             f"got {got[i]!r}, want {ref[i]!r}, tolerance {t:.3e}")


def randn(gen, shape, dt, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(DT[dt])
