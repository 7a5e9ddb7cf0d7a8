"""Plain 64-bit forms of the operators around the cache, and bounds of what 16-bit operands may
change, shared by their GPU tests. Tables and reconstructions come from the oracle."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle as O
import workloads as W
from gpu_util import oracle_cache, upload_cache

import kv_cache_vector_fwht_b200 as tq

OUTLIERS = list(range(1, 128, 4))


def quantizers(mode, bits, seed=7):
    outl = OUTLIERS if mode == "grouped" else None
    return (O.build_quantizer(128, bits, mode, seed, np.array(OUTLIERS) if outl else None),
            tq.tq_build_codebook(128, bits, mode, seed, outl))


def make_case(seed, mode, bits, vbits, lengths, hkv, capacity, lo=0.5, hi=2.0):
    """Oracle quantizer, library quantizer, the oracle's packed cache and the same on the GPU."""
    g = W.rng(seed)
    qo, qg = quantizers(mode, bits)
    n = max(max(lengths), 1)
    K = W.round_bf16(W.scaled_gaussian_rows(g, len(lengths) * hkv * n, lo=lo, hi=hi).reshape(len(lengths), hkv, n, 128))
    V = W.round_bf16(W.gaussian(g, (len(lengths), hkv, n, 128))) if vbits else None
    oc = oracle_cache(qo, K, V, vbits, lengths)
    cache = tq.KVCache(qg, len(lengths), hkv, capacity, value_bits=vbits, device="cuda:0")
    upload_cache(cache, oc)
    return qo, qg, oc, cache, g


def pair_planes(qo, oc, b, kv, n):
    p = dict(idx=oc["k_idx"][b, kv, :n], norms=oc["k_norms"][b, kv, :n])
    if qo.mode == "prod":
        p["signs"] = oc["k_signs"][b, kv, :n]
    return p


def score_error(qo, planes, q):
    """For every key: how far the 16-bit operands can move <q, k_hat>, in the worst case. Half a step of fp16
    is 2^-11: one for the rotated query, 2^-12 for the scaled levels (grouped: 2^-11 each for the
    group's ratio and its product with a level as well); prod: the sketch of the rounded query, the
    rounding of S q and that of r16 / n16. 1 % more for the 32-bit sums."""
    h = 2.0 ** -11
    norms = O.fp16_from_bits(planes["norms"])
    if qo.mode == "grouped":
        at, err = 0, 0.0
        for i, g in enumerate(qo.groups):
            w = O.storage_width(g.bits)
            nb = g.channels.size * w // 8
            c = np.abs(g.cent[O.unpack_bits(planes["idx"][:, at:at + nb], w, g.channels.size)])
            err = err + norms[:, i] * (3.5 * h) * (c @ np.abs(g.Pi @ q[g.channels]))
            at += nb
        return 1.01 * err
    bits = qo.bits - 1 if qo.mode == "prod" else qo.bits
    qr = np.abs(qo.Pi @ q)
    c = np.abs(qo.cent[O.unpack_bits(planes["idx"], O.storage_width(bits), 128)])
    err = norms[:, 0] * (1.5 * h) * (c @ qr)
    if qo.mode == "prod":
        sq = np.abs(qo.S @ q).sum()
        err = err + norms[:, 1] * (math.sqrt(math.pi / 2) / 128) * h * (2 * sq + (np.abs(qo.S_rot) @ qr).sum())
    return 1.01 * err


def attention64(qo, oc, query, limits, vbits, head_map=None, scale=None, keys=None):
    """query (B, H, n, 128); limits (B, n): row t of sequence b attends to positions below limits[b][t], or to
    keys[b][kv] (a list of positions, repeats counting) below it. Returns the outputs and a bound of the error
    that fp16 operands can cause: with p_i off by a factor 1 + e_i, an output is off by at most
    sum w_i e_i (|v_i| + |o|); e_i has the score's error and half a step for p_i, v_i is off by half a
    step; p below 2^-14 of the largest has an absolute error of 2^-25 of it."""
    B, H, n, _ = query.shape
    hkv = oc["k_idx"].shape[1]
    head_map = O.default_head_map(H, hkv) if head_map is None else head_map
    scale = scale or 1 / math.sqrt(128)
    out, tol = np.zeros(query.shape), np.zeros(query.shape)
    for b in range(B):
        for kv in range(hkv):
            L = int(oc["len"][b])
            heads = [h for h in range(H) if head_map[h] == kv]
            if not L or not heads:
                continue
            planes = pair_planes(qo, oc, b, kv, L)
            v = O.dequantize_values(oc["v_q"][b, kv, :L], oc["v_params"][b, kv, :L], vbits, 128)
            khat = O.reconstruct_keys(qo, planes)
            for h in heads:
                for t in range(n):
                    q = query[b, h, t].astype(np.float64)
                    at = np.arange(L) if keys is None else np.array(keys[b][kv], dtype=np.int64)
                    at = at[at < max(0, limits[b][t])]
                    if not at.size:
                        continue
                    z = scale * (khat[at] @ q)
                    p = np.exp(z - z.max())
                    w = p / p.sum()
                    va = v[at]
                    o = w @ va
                    d = scale * score_error(qo, planes, q)[at]
                    e = np.expm1(d) + 2.0 ** -11
                    out[b, h, t] = o
                    tol[b, h, t] = ((w * e) @ np.abs(va) + np.abs(o) * (w @ e) + 2.0 ** -11 * (w @ np.abs(va))
                                    + at.size * 2.0 ** -25 * (np.abs(va).max() + np.abs(o)))
    return out, tol


def check(got, ref, tol, dtype):
    """got (a tensor of `dtype`) within tol plus its own rounding (half a step of the type)."""
    g = got.detach().float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(g)), "non-finite outputs"
    half = torch.finfo(dtype).eps / 2
    bound = tol * (1 + half) + half * np.abs(ref) + 1e-6
    worst = np.max(np.abs(g - ref) / bound)
    assert worst <= 1, f"{worst:.2f} times the bound"


def causal_limits(lengths, n):
    return [[L - n + t + 1 for t in range(n)] for L in lengths]


def full_limits(lengths, n):
    return [[L] * n for L in lengths]
