"""Float64 references of the scored attention calls and of the eviction, and
the tolerances the GPU tests hold the kernels to.

The tolerances are sums of what each rounding of the kernels can do, worst
case, derived from the formats alone:
  - a score: 128 products (exact in the f32 accumulator's inputs), each
    addition off by at most 2^-23 of the running sum's bound sum |q k|, and the
    scalings, the cap's tanh (2^-22 relative) and the bias (2^-22 of its size);
  - P: rounded to f16 (2^-11 relative; below 2^-14 an absolute 2^-25 against a
    largest weight of at least 1), its exponent's error twice (once in the sum);
  - the output: rounded to bf16 (2^-8 relative);
  - the accumulated weights: ex2 and the additions, 2^-20 relative.
"""
import numpy as np
import torch

import oracle
import nvfp4_quantized_paged_quantize_gb300 as kv
from nvfp4_quantized_paged_quantize_gb300 import inputs
from gpu_util import dev, pool_host

SCALE = 1.0 / np.sqrt(128.0)


def attend(q, K, V, seen, dist, softmax_scale, softcap=0.0, slope=0.0):
    """One query head: q [128], K, V [n, 128] float64, seen [n] bool, dist [n] |p - j|.

    Returns dict(out, lse, p, tol_out, tol_lse, tol_p)."""
    out = {"out": np.zeros(V.shape[1] if len(V) else 128), "lse": -np.inf, "p": np.zeros(len(K)),
           "tol_out": np.zeros(128), "tol_lse": 0.0, "tol_p": np.zeros(len(K))}
    if not seen.any():
        return out
    x = K @ q * softmax_scale
    dx = 128 * 2.0 ** -23 * (np.abs(K) @ np.abs(q)) * softmax_scale + 2.0 ** -22 * np.abs(x)
    if softcap > 0:
        x = softcap * np.tanh(x / softcap)                     # slope at most 1: dx does not grow
        dx = dx + 2.0 ** -22 * np.abs(x)
    if slope:
        x = x - slope * dist
        dx = dx + 2.0 ** -22 * slope * dist
    dx = dx + 2.0 ** -22 * np.abs(x)
    x, dx = np.where(seen, x, -np.inf), np.where(seen, dx, 0.0)
    top = x.max()
    e = np.exp(x - top)
    total = e.sum()
    p = e / total
    d = (p * dx).sum()                                          # what the sum's error amounts to
    # (weights far below the largest carry their own dx; first order, with 10 % for the rest)
    rel = 1.1 * (dx + d) + 2.0 ** -20
    out["p"], out["lse"], out["out"] = p, top + np.log(total), p @ V
    out["tol_p"] = p * rel + 2.0 ** -100
    out["tol_lse"] = 1.1 * d + 2.0 ** -20 + 2.0 ** -22 * abs(out["lse"])
    vmax = np.abs(V[seen]).max()
    out["tol_out"] = (2.0 ** -8 * np.abs(out["out"]) + (p * (rel + 2.0 ** -11)) @ np.abs(V) * (1 + 2.0 ** -8) +
                      seen.sum() * 2.0 ** -25 * vmax / max(total, 1.0) + 2.0 ** -126)
    return out


def decode_ref(K, V, q, L, scoring, softmax_scale=SCALE, head=0):
    """A decode query over its sequence's L dequantised rows (K, V [L, 128])."""
    j = np.arange(L)
    seen = np.ones(L, bool)
    if scoring.window > 0:
        seen = (L - 1 - j < scoring.window) | (j < scoring.sinks)
    slope = 0.0 if scoring.slopes is None else float(scoring.slopes[head])
    return attend(q, K, V, seen, np.abs(L - 1 - j).astype(float), softmax_scale, scoring.softcap, slope)


def extend_seen(P, C, t, scoring, full=None, doc=None):
    """The keys chunk token t of a sequence sees, of its P + C."""
    j, p = np.arange(P + C), P + t
    high = p if full is None else max(p, min(full, P + C) - 1)
    low = 0 if doc is None else max(doc, 0)
    seen = (j >= low) & (j <= high)
    if scoring.window > 0:
        seen &= (p - j < scoring.window) | (j < low + scoring.sinks)
    return seen


def check(got, want, tol, what):
    got, want, tol = (np.asarray(a, np.float64) for a in (got, want, tol))
    assert np.isfinite(got).all(), f"{what}: non-finite"
    worst = np.max(np.abs(got - want) - tol) if got.size else 0.0
    assert worst <= 0, f"{what}: {np.max(np.abs(got - want) / np.maximum(tol, 1e-300)):.3g} times the tolerance"


def random_cache(num_pages, hkv, seed, gk=1.0, gv=1.0):
    """A cache of random codes and scales (E4M3 exponents -4 .. 0), on the GPU and in the oracle's layout."""
    rng = np.random.default_rng(seed)
    c = kv.Cache.empty(num_pages, hkv, k_global_scale=gk, v_global_scale=gv, zero=True)
    c.k_data.copy_(dev(rng.integers(0, 256, tuple(c.k_data.shape), dtype=np.uint8)))
    c.set_v_data(dev(rng.integers(0, 256, tuple(c.k_data.shape), dtype=np.uint8)))
    for s in (c.k_scale, c.v_scale):
        s.copy_(dev(inputs.fp8_bytes_by_field(rng, tuple(s.shape), 3, 7) & 0x7F))
    return c, oracle.Cache(num_pages, hkv, 128, 16, gk, gv, arrays=pool_host(c))


def sequence_rows(o, table_row, h, L):
    """Dequantised K, V [L, 128] of a sequence's KV head from the oracle's cache."""
    if L == 0:
        return np.zeros((0, 128)), np.zeros((0, 128))
    t = np.arange(L)
    rows = (table_row[t // 16].astype(np.int64) * o.num_kv_heads + h) * 16 + t % 16
    return oracle.dequantize_rows(o, "k", rows), oracle.dequantize_rows(o, "v", rows)


def page_tables(lens, seed, first=0, extra_cols=0, fill=-1):
    """Shuffled distinct pages of each sequence; unused entries hold `fill`."""
    need = [(int(n) + 15) // 16 for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need)).astype(np.int32) + first
    table = np.full((len(lens), max(1, max(need)) + extra_cols), fill, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need)


def random_q(shape, seed, size=1.0):
    """bf16 queries on the GPU and their float64 values."""
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * size).to(torch.bfloat16)
    return x.cuda(), x.double().numpy()


def on_gpu(scoring):
    """The same Scoring with its slopes as a device tensor."""
    sl = None if scoring.slopes is None else dev(np.asarray(scoring.slopes, np.float32))
    return kv.Scoring(scoring.softcap, scoring.window, scoring.sinks, sl)


def evict_ref(w, L, budget, first, recent):
    """The kept token indices of one (sequence, KV head), in order."""
    if L <= budget:
        return np.arange(L)
    j = np.arange(first, L - recent)
    key = np.where(np.isnan(w[j]), np.inf, w[j].astype(np.float64))
    nan = np.isnan(w[j])
    best = j[np.lexsort((j, -key, ~nan))][:budget - first - recent]   # NaN first, then the largest, then the lowest index
    return np.sort(np.concatenate([np.arange(first), best, np.arange(L - recent, L)]))
