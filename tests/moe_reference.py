"""Plain mixture-of-experts reference in 64 bits for the GPU tests: routing,
grouping, the expert products (through the CPU oracle) and the combination.
Numpy only."""
import numpy as np

import oracle
import q4k_synth


def route(logits, top_k, renorm):
    """ids (-1: none left), weights (float64), per-row bound of the f32 weights'
    error, of logits [t, e] (float32; NaN and -inf: not available)."""
    lg = logits.astype(np.float64)
    avail = ~np.isnan(lg) & (lg > -np.inf)
    key = np.where(avail, np.minimum(lg, np.finfo(np.float32).max), -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    val = np.take_along_axis(key, ids, 1)
    ok = val > -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.where(ok[:, :1], val[:, :1], 0.0)
        ex = np.where(ok, np.exp(val - top), 0.0)
        base = np.where(ok, val - top, 0.0) if renorm else np.where(avail, key - top, 0.0)
        total = ex.sum(1, keepdims=True) if renorm else np.where(avail, np.exp(base), 0.0).sum(1, keepdims=True)
    w = np.where(ok, ex / np.where(total > 0, total, 1.0), 0.0)
    # f32: l - top rounded (relative 2^-24, so exp's error is |l - top| 2^-24;
    # beyond |l - top| = 104 the exponential is 0 in f32 and at most 1e-45 here),
    # expf within 2 ulp, the sum of at most e terms, one division
    spread = np.minimum(np.abs(base).max(1, keepdims=True), 104.0)
    tol = w * (2 * spread + logits.shape[1] + 12) * 2.0 ** -24 + 1e-37
    return np.where(ok, ids, -1).astype(np.int32), w, tol


def group(ids, experts):
    flat = ids.reshape(-1)
    routed = np.flatnonzero(flat >= 0)
    order = np.full(flat.size, -1, np.int32)
    order[:routed.size] = routed[np.argsort(flat[routed], kind="stable")]
    counts = np.bincount(flat[routed], minlength=experts)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order


def x_row(order, per_row):
    return np.arange(order.size) if per_row == 0 else order // per_row


def random_ids(rng, tokens, experts, top_k, pad=0, skew=0.0):
    """Distinct experts per token; `pad` tokens at the end go nowhere."""
    pull = rng.standard_normal(experts) * skew
    ids = np.argsort(-(rng.standard_normal((tokens, experts)) + pull), axis=1)[:, :top_k].astype(np.int32)
    if pad:
        ids[tokens - pad:] = -1
    return ids


def expert_matrices(experts, n, k, seed):
    """[experts, n*(k/256)*144] uint8, each expert its own seeded stream."""
    return np.stack([q4k_synth.q4k_problem(n, k, 1, seed + 31 * e)[0] for e in range(experts)])


def products(fn, ws, x, offsets, order, per_row, n):
    """Per slot: fn(expert's matrices, rows of x) stacked into [slots, n] arrays
    (one per array fn returns); slots behind the last are NaN."""
    out = None
    rows = x_row(order, per_row)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        got = fn([w[e] for w in ws], np.ascontiguousarray(x[rows[a:b]]))
        if out is None:
            out = [np.full((order.size, n), np.nan) for _ in got]
        for o, v in zip(out, got):
            o[a:b] = v
    return out if out is not None else [np.full((order.size, n), np.nan) for _ in range(2)]


def swiglu(g, u, t_g, t_u):
    """silu(g) * u and its bound for g, u off by t_g, t_u (the form of
    oracle.swiglu_tolerance)."""
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    h = s * u
    tol = 1.1 * t_g * (np.abs(u) + t_u) + (np.abs(s) + 1.1 * t_g) * t_u + 1e-6 * np.abs(h) + 1e-30
    return h, tol


def gemv(ws, x, offsets, order, per_row, n, k, nthreads=1):
    """Per slot (y, bound) of q4k_moe_gemv: the q4k_gemv bound."""
    y, a = products(lambda w, xr: oracle.gemv(w[0], xr, n, k, nthreads), ws, x, offsets, order, per_row, n)
    return y, oracle.tolerance(a)


def gemm(ws, x16, offsets, order, per_row, n, k):
    """Per slot (y, bound) of q4k_moe_gemm_f16: the q4k_gemm_f16 bound."""
    y, a = products(lambda w, xr: oracle.gemm_f16(oracle.dequant_f16(w[0], n, k), xr), ws, x16, offsets, order,
                    per_row, n)
    return y, oracle.gemm_f16_tolerance(a, k)
