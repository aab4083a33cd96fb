"""Rounding bounds of the attention kernels, element by element, from the
operations that round: no tolerance here is fitted to an output.

With u the half step of the 16-bit type (bf16 2^-8, fp16 2^-11), a row's
weights p_t and A = sum_t p_t |v_t|:
* the output is rounded once:                         u |o|
* a weight enters the product rounded to the type:     u A, and, for fp16
  weights below its normal range, 2^-25 each:          2^-25 sum_t |v_t|
* a score is off by ds: fp32 sums of D products, each step 2^-23 of the
  running sum's bound X = max_t |scale| sum_d |q_d k_td|, (D + 8) steps, or
  what the caller says K's rounding adds; a weight is then off by 2 ds
  (numerator and normaliser), so is the sum:           A (e^(2 ds) - 1)
* the exponential and the fp32 sums over the keys:     A 2^-18
"""

import numpy as np
import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def score_bound(q, k, scale, q_start, kv_start):
    """X [T, Hq, 1]: the largest |scale| sum_d |q_d k_td| over the sequence."""
    G = q.shape[1] // k.shape[1]
    X = np.zeros(q.shape[:2] + (1,))
    for b in range(len(q_start) - 1):
        lo, hi, ka, kb = int(q_start[b]), int(q_start[b + 1]), int(kv_start[b]), int(kv_start[b + 1])
        if hi <= lo or kb <= ka:
            continue
        for h in range(q.shape[1]):
            kmax = np.abs(k[ka:kb, h // G])
            for i in range(lo, hi, 512):
                j = min(hi, i + 512)
                X[i:j, h, 0] = (np.abs(q[i:j, h]) @ kmax.T).max(axis=1) * abs(scale)
    return X


def bound(out, out_abs, X, D, dtype, weight_step, v_sum=None, k_step=0.0, v_step=0.0):
    ds = X * ((D + 8) * 2.0 ** -23 + k_step)
    tol = half_step(dtype) * np.abs(out) + out_abs * (weight_step + v_step + np.expm1(2 * ds) + 2.0 ** -18)
    if v_sum is not None:
        tol = tol + 2.0 ** -25 * v_sum
    return tol * (1 + 2.0 ** -7) + (2.0 ** -24 if dtype == torch.float16 else 2.0 ** -100)


def assert_within(got, want, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err - tol, -np.inf)), err.shape)
        raise AssertionError("%s: %d / %d out of bound; worst at %s: got %.6g want %.6g bound %.3g" % (
            what, bad.sum(), bad.size, i, got[i], want[i], tol[i]))
