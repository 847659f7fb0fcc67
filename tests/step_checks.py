"""Checks of the layer's steps (RMS norm, grouped routing, key weights, eviction) against their FP64
definitions (oracle/steps.py), for any backend that takes and returns numpy arrays: the host build of the
library (tests/host_emulation/step_cases.py) and the library on a GPU (tests/test_gpu_steps.py).

Tolerances follow from the arithmetic; a rounding to BF16 is off by at most 2^-8 of the value, to E4M3 by
2^-4 (2^-10 below its normal range), an FP32 operation by 2^-24.
  norm     sums of squares of at most 16384 terms are added in chains of at most 32 + 5 + 16 terms, all of
           one sign: 2^-18 with room, for rstd (half of it) and the products after it
  dx       the two parts of dx may cancel: 2^-17 of the parts' magnitudes, and the rounding to BF16
  dweight  a chain of at most `rows of a thread` terms, then the partial rows: (rows + 64) 2^-24 of the
           terms' magnitudes, and 2^-18 of them for rstd
  route    at most eight FP32 operations on correctly chosen scores: 2^-20
  weights  a score's error: the rotated dims carry 22 bits on each side (2^-20 of the products' magnitudes
           with the angles' error, taken as 2^-19), accumulation over 320 products included; the FP32
           exponent and 2^x: 2^-22 of the magnitudes of score and lse, 2^-20 in all
"""
from __future__ import annotations

import numpy as np

from oracle import steps
from oracle.neighbors import bf16_bits_to_f64

BF16, E4M3 = 2.0 ** -8, 2.0 ** -4


def bits(x):
    return steps.f64_to_bf16_bits(np.asarray(x, dtype=np.float64))


def close(got, ref, tol, what):
    got, ref, tol = (np.asarray(a, dtype=np.float64) for a in (got, ref, tol))
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    off = ~(np.abs(got - ref) <= tol) & ~(np.isnan(got) & np.isnan(ref)) & ~((got == ref) & np.isinf(ref))
    assert not off.any(), (f"{what}: {off.sum()} of {off.size} off, first at {tuple(np.argwhere(off)[0])}: "
                           f"{got[off][0]!r} for {ref[off][0]!r}, tolerance {np.broadcast_to(tol, got.shape)[off][0]:.3g}")


# ---------------------------------------------------------------- RMS norm
def norm_inputs(T, H, seed, residual=True, w32=False):
    rng = np.random.default_rng(seed)
    x = bits(rng.standard_normal((T, H)))
    r = bits(3 * rng.standard_normal((T, H))) if residual else None
    w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    return x, r, (w if w32 else bits(w))


def weight_values(w):
    return bf16_bits_to_f64(w) if w.dtype == np.uint16 else w.astype(np.float64)


def check_norm(be, T, H, seed, residual=True, w32=False, fp8=False, both=False, eps=1e-6, x=None, r=None):
    xx, rr, w = norm_inputs(T, H, seed, residual, w32)
    x = xx if x is None else x
    r = rr if r is None else r
    got = be.rms_norm(x, w, r, eps, y=not fp8 or both, fp8=fp8)
    with np.errstate(all="ignore"):
        h, y = steps.rms_norm(x, weight_values(w), r, eps)
    if r is not None:
        nan = np.isnan(bf16_bits_to_f64(h))
        assert np.array_equal(np.where(nan, 0, got["h"]), np.where(nan, 0, h)), "h"
    if "y" in got:
        close(bf16_bits_to_f64(got["y"]), y, np.abs(y) * (BF16 + 2.0 ** -18), "y")
    if fp8:
        scale = steps.fp8_blocks(y)
        close(got["scale"], scale, scale * 2.0 ** -17, "scale")
        per = np.repeat(got["scale"].astype(np.float64), 128, -1)[:, :H]
        v = steps.fp8_values(got["codes"], got["scale"]) / per  # the codes' values
        t = y / per
        close(v, t, np.abs(t) * (E4M3 + 2.0 ** -17) + 2.0 ** -10, "codes")
    return got


def check_norm_bwd(be, T, H, seed, dh=True, w32=False, eps=1e-6):
    rng = np.random.default_rng(seed)
    h, _, w = norm_inputs(T, H, seed + 1, False, w32)
    dy = bits(rng.standard_normal((T, H)))
    d = bits(rng.standard_normal((T, H))) if dh else None
    dx, dw = be.rms_norm_bwd(h, w, dy, d, eps)
    rx, rw = steps.rms_norm_bwd(h, weight_values(w), dy, d, eps)
    hf, g = np.abs(bf16_bits_to_f64(h)), np.abs(bf16_bits_to_f64(dy) * weight_values(w))
    r = 1 / np.sqrt((hf * hf).mean(-1, keepdims=True) + eps)
    parts = r * g + r ** 3 * hf * (g * hf).sum(-1, keepdims=True) / H + (0 if d is None else np.abs(bf16_bits_to_f64(d)))
    close(bf16_bits_to_f64(dx), rx, np.abs(rx) * BF16 + parts * 2.0 ** -17, "dx")
    mag = (np.abs(bf16_bits_to_f64(dy)) * hf * r).sum(0)
    close(dw, rw, mag * (2.0 ** -18 + (T + 64) * 2.0 ** -24), "dweight")
    return dx, dw


# ---------------------------------------------------------------- routing
def route_logits(T, E, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "ties":  # a few values only: most choices are ties
        x = np.round(x).astype(np.float32)
    elif kind == "near":  # neighbours a rounding apart
        x = (1 + rng.integers(0, 4, (T, E)) * 2.0 ** -23).astype(np.float32)
    elif kind == "flat":
        x = np.zeros((T, E), dtype=np.float32)
    elif kind == "far":  # scores that underflow or saturate
        x = (x * 200).astype(np.float32)
    elif kind == "masked":  # experts switched off by the type's lowest value or -inf
        x[rng.random((T, E)) < 0.6] = np.finfo(np.float32).min
        x[rng.random((T, E)) < 0.2] = -np.inf
        x[:, 0] = 0.5  # one that is left
    return x


def check_route(be, T, E, k, groups, top_groups, softmax, normalize, bias, seed, kind="normal", scale=1.0, x=None):
    x = route_logits(T, E, seed, kind) if x is None else x
    b = None
    if bias:
        b = (0.1 * np.random.default_rng(seed + 1).standard_normal(E)).astype(np.float32)
        if kind in ("ties", "flat"):
            b = np.zeros(E, dtype=np.float32)
    ids, w = be.route(x, b, k, groups, top_groups, softmax, normalize, scale)
    with np.errstate(all="ignore"):
        rid, rw = steps.route_grouped(x, b, k, groups, top_groups, softmax, normalize, scale)
    assert np.array_equal(ids, rid), f"ids of token {np.argwhere(ids != rid)[0][0]}: {ids[ids != rid][:4]} for {rid[ids != rid][:4]}"
    close(w, rw, np.abs(rw) * 2.0 ** -20 + 2.0 ** -149, "weights")
    return ids, w


def check_route_bwd(be, T, E, k, softmax, normalize, seed, scale=1.0, kind="normal", ids=None):
    rng = np.random.default_rng(seed)
    x = route_logits(T, E, seed + 1, kind)
    if ids is None:
        ids = np.argsort(rng.random((T, E)), -1)[:, :k].astype(np.int32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    d = be.route_bwd(x, ids, g, softmax, normalize, scale)
    with np.errstate(all="ignore"):
        r = steps.route_bwd(x, ids, g, softmax, normalize, scale)
        s = steps.scores(x, softmax)
    # magnitudes of what is added: every place's |g| times its derivative, and the mean's share of it; `own` is the
    # reference's rounding, where its softmax Jacobian cancels to zero in FP64 (2^-50 of the magnitudes)
    mag, own = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        e = [(int(i), abs(scale * float(v))) for i, v in zip(ids[t], g[t]) if 0 <= i < E]
        S = sum(s[t, i] for i, _ in e) if normalize else 1.0
        S = S if S > 0 else 1.0
        mean = sum(v * s[t, i] / S for i, v in e)
        if softmax and not normalize:
            mag[t] = s[t] * mean
        if softmax and normalize:
            own[t] = s[t] * mean / S * 2.0 ** -50
        for i, v in e:
            mag[t, i] += (v + (mean if normalize else 0)) * s[t, i] / S
    close(d, r, mag * 2.0 ** -18 + own + 2.0 ** -126, "dlogits")
    return d


# ---------------------------------------------------------------- key weights, eviction
def step_batch(kv_lens, q_lens, hq, hkv, seed, spare=7):
    """A KV-cache step without V: as workloads.make_decode_inputs lays it out."""
    rng = np.random.default_rng(seed)
    total, rows = sum(kv_lens), sum(kv_lens) + spare
    q = bits(rng.standard_normal((sum(q_lens), hq, 192)))
    k = bits(rng.standard_normal((rows, hkv, 192)))
    idx = rng.permutation(rows)[:total].astype(np.int32)
    ptr = lambda n: np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return q, k, idx, ptr(kv_lens), ptr(q_lens)


def weights_tolerance(q_bits, k_bits, idx, indptr, cu_q, lse, window, base, prev):
    q, k = np.abs(bf16_bits_to_f64(q_bits)), np.abs(bf16_bits_to_f64(k_bits))
    for a in (q, k):  # a rotated value is at most its pair's norm
        n = np.hypot(a[..., :32], a[..., 32:64])
        a[..., :32] = n
        a[..., 32:64] = n
    qb, kb = bf16_bits_to_f64(q_bits), bf16_bits_to_f64(k_bits)
    hq, hkv = q.shape[1], k.shape[1]
    tol = np.zeros(len(idx))
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], indptr[b], indptr[b + 1]
        n, m = k1 - k0, q1 - q0
        pos = np.arange(n)
        off = pos[n - m:, None] - pos[None]
        may = (off >= 0) & ((off <= window) if window >= 0 else True)
        kk, qq = steps._turned(kb[idx[k0:k1]], pos, base), steps._turned(qb[q0:q1], pos[n - m:], base)
        for h in range(hq):
            g = h // (hq // hkv)
            s = qq[:, h] @ kk[:, g].T / np.sqrt(192.0)
            A = q[q0:q1, h] @ k[idx[k0:k1]][:, g].T / np.sqrt(192.0)
            l = lse[h, q0:q1, None].astype(np.float64)
            p = np.exp(s - l)
            tol[k0:k1] += np.where(may, p * (A * 2.0 ** -19 + (np.abs(s) + np.abs(l)) * 2.0 ** -22 + 2.0 ** -20), 0).sum(0)
    return tol if prev is None else tol + (np.abs(prev) + 1) * 2.0 ** -23


def check_weights(be, kv_lens, q_lens, hq, hkv, window, base, seed, sink=False, prev=False):
    q, k, idx, indptr, cu_q = step_batch(kv_lens, q_lens, hq, hkv, seed)
    rng = np.random.default_rng(seed + 1)
    s = rng.standard_normal(hq).astype(np.float32) if sink else None
    lse = steps.normaliser(q, k, idx, indptr, cu_q, window, base, s).astype(np.float32)
    p = np.abs(rng.standard_normal(len(idx))).astype(np.float32) if prev else None
    got = be.key_weights(q, k, idx, indptr, cu_q, lse, max(q_lens), max(kv_lens), window, base, p)
    ref = steps.key_weights(q, k, idx, indptr, cu_q, lse, window, base, p)
    close(got, ref, weights_tolerance(q, k, idx, indptr, cu_q, lse, window, base, p), "key weights")
    if not sink and not prev:  # every query's weights sum to one
        total = got.astype(np.float64).sum()
        assert abs(total - hq * sum(q_lens)) <= 1e-4 * hq * sum(q_lens), total
    return got


def evict_weights(total, seed, kind="spread"):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal(total)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, total).astype(np.float32)
    elif kind == "flat":
        w[:] = 1.0
    elif kind == "wild":  # NaN, infinities, both zeros, negatives, subnormals
        w *= rng.choice([1, -1], total)
        for v in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, -1e-40):
            w[rng.random(total) < 0.1] = v
    return w.astype(np.float32)


def check_evict(be, lens, budget, first, recent, seed, kind="spread"):
    total = sum(lens)
    w = evict_weights(total, seed, kind)
    idx = np.random.default_rng(seed + 1).permutation(total + 5)[:total].astype(np.int32)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    fill = -123
    gi, gw, gp, gf = be.evict(w, idx, indptr, max(lens), budget, first, recent, fill)
    ri, rw, rp, rf = steps.kv_evict(w, idx, indptr, budget, first, recent)
    assert np.array_equal(gp, rp), (gp, rp)
    n, m = len(ri), len(rf)
    assert np.array_equal(gi[:n], ri) and np.array_equal(gf[:m], rf), "rows"
    assert np.array_equal(gw[:n].view(np.uint32), rw.view(np.uint32)), "weights"
    assert np.all(gi[n:] == fill) and np.all(gf[m:] == fill) and np.all(gw[n:] == fill), "written behind the last entry"


# Cases by name: the sizes and masks where the kernels can go wrong, small enough for the host build.
CASES = {
    "norm_plain": lambda be: [check_norm(be, T, H, 10 + T + H, residual=r, w32=w32)
                              for T, H, r, w32 in ((1, 8, False, False), (3, 16, True, True), (5, 256, True, False),
                                                   (2, 264, False, True), (3, 520, True, False), (9, 1024, True, False))],
    "norm_wide": lambda be: [check_norm(be, T, H, 20 + T + H, residual=r, w32=w32)
                             for T, H, r, w32 in ((3, 1032, True, False), (2, 2048, False, True), (2, 4096, True, False),
                                                  (1, 4104, True, False), (2, 8192, False, False), (1, 16384, True, True))],
    "norm_fp8": lambda be: [check_norm(be, T, H, 30 + T + H, residual=r, fp8=True, both=b)
                            for T, H, r, b in ((1, 16, False, False), (5, 128, True, True), (3, 144, False, True),
                                               (2, 1040, True, False), (3, 4096, True, True), (1, 4112, False, False),
                                               (1, 16384, True, False))],
    "norm_values": lambda be: norm_values(be),
    "norm_bwd": lambda be: [check_norm_bwd(be, T, H, 40 + T + H, dh=d, w32=w32)
                            for T, H, d, w32 in ((1, 8, False, False), (37, 64, True, False), (5, 512, False, True),
                                                 (19, 1024, True, False), (9, 1032, True, False), (3, 4096, False, False),
                                                 (6, 4104, True, True), (3, 8192, True, False), (2, 16384, False, False))],
    "route": lambda be: [check_route(be, *c) for c in (
        (5, 256, 8, 8, 4, False, True, True, 50), (4, 256, 8, 1, 1, True, True, False, 51),
        (3, 16, 16, 1, 1, False, False, True, 52), (3, 60, 6, 4, 1, True, False, True, 53),
        (2, 512, 32, 32, 20, False, True, True, 54), (3, 160, 6, 8, 3, True, True, False, 55),
        (2, 1, 1, 1, 1, False, True, False, 56), (2, 7, 3, 7, 3, True, True, True, 57),
        (3, 72, 8, 2, 2, False, True, False, 58), (4, 128, 4, 4, 2, True, True, True, 59),
        (3, 64, 12, 8, 2, False, True, True, 60), (2, 384, 8, 1, 1, True, False, False, 61), (3, 510, 8, 17, 5, False, True, True, 62), (4, 96, 8, 3, 2, True, True, True, 63),
        (4, 224, 8, 7, 3, False, True, True, 64), (3, 256, 32, 8, 1, True, True, False, 65))],
    "route_kinds": lambda be: [check_route(be, 4, E, 8, groups, top, softmax, True, bias, 70, kind)
                               for kind in ("ties", "near", "flat", "far", "masked")
                               for E, groups, top, softmax, bias in ((256, 8, 4, False, True), (256, 1, 1, True, False),
                                                                     (128, 4, 2, False, False), (160, 1, 1, True, True))],
    # enough tokens for the kernel of four threads per token on an SM or two (and a ragged last tile)
    "route_many": lambda be: [check_route(be, T, E, k, groups, top, softmax, normalize, bias, 75 + E, kind, 2.5)
                              for T, E, k, groups, top, softmax, normalize, bias, kind in (
                                  (1111, 256, 8, 8, 4, False, True, True, "normal"), (1050, 256, 8, 1, 1, True, True, False, "normal"),
                                  (1333, 64, 6, 4, 1, True, False, True, "normal"), (1100, 128, 3, 8, 8, False, True, False, "normal"),
                                  (1100, 160, 8, 4, 2, False, True, True, "normal"), (1200, 72, 1, 3, 2, True, True, False, "normal"),
                                  (1100, 16, 8, 2, 1, False, True, True, "normal"), (1100, 256, 8, 8, 4, False, True, True, "ties"),
                                  (1100, 64, 8, 8, 4, True, True, False, "near"), (1100, 64, 8, 1, 1, False, True, False, "far"),
                                  (1100, 128, 8, 4, 2, True, True, False, "masked"), (1100, 64, 4, 8, 2, False, True, True, "flat"))],
    "route_values": lambda be: route_values(be),
    "route_far": lambda be: route_far(be, (3, 2100)),
    "route_bwd": lambda be: [check_route_bwd(be, *c) for c in (
        (5, 256, 8, False, True, 80), (5, 256, 8, True, True, 81), (5, 128, 6, True, False, 82, 2.5),
        (4, 64, 4, False, False, 83, 0.5), (3, 60, 60 // 2, True, True, 84), (2, 512, 32, False, True, 85),
        (2, 1, 1, True, False, 86), (3, 7, 3, False, True, 87), (3, 160, 8, True, False, 88),
        (3, 256, 8, False, True, 89, 1.0, "far"), (3, 256, 8, True, True, 90, 1.0, "far"),
        (3, 128, 8, True, False, 91, 1.0, "masked"), (3, 128, 8, False, True, 92, 1.0, "masked"),
        (9, 512, 8, False, True, 93), (9, 384, 8, True, True, 94), (3, 160, 8, True, False, 96, 1.0, "far"), (5, 66, 12, False, True, 97),
        (3, 64, 6, False, False, 98, 1.0, "far"), (33, 60, 5, False, True, 99))],
    "route_bwd_places": lambda be: route_bwd_places(be),
    "weights_step": lambda be: [check_weights(be, *c) for c in (
        ([5, 129, 300, 64], [1, 1, 1, 1], 8, 2, -1, 1e7, 100), ([130, 1, 257], [8, 1, 3], 8, 2, -1, 1e4, 101, False, True),
        ([300], [8], 16, 1, -1, 1e7, 102), ([128, 127], [2, 2], 6, 2, -1, 1e7, 103))],
    "weights_window": lambda be: [check_weights(be, *c) for c in (
        ([5, 129, 300, 400], [1, 8, 3, 1], 8, 2, 128, 1e4, 110, True), ([300, 260], [4, 2], 4, 1, 0, 1e4, 111, True, True),
        ([350], [1], 4, 2, 127, 1e4, 112, False, True))],
    "weights_chunk": lambda be: [check_weights(be, *c) for c in (
        ([300, 40], [36, 40], 8, 1, -1, 1e7, 120), ([260, 200], [43, 100], 6, 2, 128, 1e4, 121, True, True),
        ([150], [150], 4, 2, -1, 1e7, 122), ([200, 3], [70, 0], 12, 2, 20, 1e4, 123, True))],
    "weights_values": lambda be: weights_values(be),
    "bad_lists": lambda be: bad_lists(be),
    "evict": lambda be: [check_evict(be, lens, budget, first, recent, 130 + i, kind)
                         for i, (lens, budget, first, recent) in enumerate((
                             ([5], 3, 0, 0), ([5, 0, 9, 1], 4, 1, 2), ([300, 4, 1200], 100, 4, 20), ([64, 64], 64, 0, 0),
                             ([40], 0, 0, 0), ([1500, 2300, 30], 1024, 0, 1024), ([200], 10, 10, 0), ([1, 1, 1], 0, 0, 0),
                             ([3000], 1500, 3, 7)))
                         for kind in ("spread", "ties", "flat", "wild")],
    # eight CTAs per sequence; then more entries than their shared memory holds
    "evict_long": lambda be: [check_evict(be, *c) for c in (([17000, 5, 300], 3000, 4, 100, 160, "spread"), ([16385], 9000, 0, 1, 161, "ties"),
                                                            ([400001], 150001, 7, 1000, 162, "wild"))],
}


def norm_values(be):
    """Rows of zeros, of one value, of the type's limits, with an infinity and with a NaN; huge and tiny eps."""
    H = 256
    x = np.zeros((6, H))
    x[1] = 1.0
    x[2, 3] = 2.0 ** 100
    x[3, ::2] = 1e-30
    b = bits(x)
    b[4] = bits(np.random.default_rng(1).standard_normal(H))
    b[4, 7] = 0x7F80  # inf
    b[5] = bits(np.random.default_rng(2).standard_normal(H))
    b[5, 9] = 0x7FC0  # NaN
    for eps in (1e-6, 0.5):
        got = check_norm(be, 4, H, 1, residual=False, eps=eps, x=b[:4])
        check_norm(be, 4, H, 1, residual=False, fp8=True, eps=eps, x=b[:4])
    got = be.rms_norm(b, bits(np.ones(H)), None, 1e-6, y=True, fp8=True)
    y = bf16_bits_to_f64(got["y"])
    assert np.all(np.isnan(y[5])) and np.isnan(y[4, 7]) and np.all(np.delete(y[4], 7) == 0)  # rstd is NaN; 0 with inf 0 = NaN
    assert np.all(got["scale"][0] == 2.0 ** -126) and np.all((got["codes"][0] & 0x7F) == 0)
    assert np.all((got["codes"][5] & 0x7F) == 0x7F) and (got["codes"][4, 7] & 0x7F) == 0x7F  # E4M3 NaN


def route_values(be):
    """NaN and infinite logits and biases: ids stay distinct experts, and the rest of the batch is not touched."""
    for softmax, T in ((False, 6), (True, 6), (False, 2100), (True, 2100)):
        x = route_logits(T, 64, 3)
        x[1, 5] = np.nan
        x[2] = np.nan
        x[3, 9] = -np.inf
        x[4] = -np.inf
        clean = [0, 3, *range(5, T)]
        ids, w = be.route(x, None, 8, 8, 4, softmax, True, 1.0)
        with np.errstate(all="ignore"):
            rid, rw = steps.route_grouped(x, None, 8, 8, 4, softmax, True, 1.0)
        assert np.array_equal(ids, rid)
        close(w[clean], rw[clean], np.abs(rw[clean]) * 2.0 ** -20, "weights")
        assert np.all(np.isnan(w[2]))
        if not softmax:
            assert np.all(w[4] == 0)  # every score is zero
    b = np.zeros(64, dtype=np.float32)
    b[3], b[4], b[17] = np.nan, -np.inf, np.inf
    off = (0.1 * np.random.default_rng(5).standard_normal(64)).astype(np.float32)
    off[::3] = -1e9  # experts switched off by their bias
    off[::7] = -np.inf
    for T in (3, 2100):
        x = route_logits(T, 64, 4)
        ids, w = be.route(x, b, 8, 4, 2, False, True, 1.0)
        rid, rw = steps.route_grouped(x, b, 8, 4, 2, False, True, 1.0)
        assert np.array_equal(ids, rid) and np.all(ids[:, 0] == 17)
        close(w, rw, np.abs(rw) * 2.0 ** -20, "weights")
        ids, w = be.route(x, off, 8, 4, 2, False, True, 1.0)
        rid, rw = steps.route_grouped(x, off, 8, 4, 2, False, True, 1.0)
        assert np.array_equal(ids, rid)
        close(w, rw, np.abs(rw) * 2.0 ** -20, "weights")


def route_far(be, tokens):
    """Biases far apart: a group whose largest makes up for a second key far below all other groups' keys."""
    for T in tokens:
        for softmax in (False, True):
            for E in (64, 256):
                size = E // 8
                plain, deep = np.zeros(E, dtype=np.float32), np.full(E, -1000.0, dtype=np.float32)
                plain[:size] = -5000.0
                plain[0], plain[1], plain[2] = 1500.0, -1030.0, -np.inf
                deep[size:2 * size] = -1025.0
                deep[size] = 20.0
                x = route_logits(T, E, 6)
                for b, first in ((plain, 0), (deep, size)):
                    ids, w = be.route(x, b, 8, 8, 2, softmax, True, 1.0)
                    rid, rw = steps.route_grouped(x, b, 8, 8, 2, softmax, True, 1.0)
                    assert np.all(rid[:, 0] == first)
                    assert np.array_equal(ids, rid), f"{T} tokens, {E} experts, softmax {softmax}, group of {first}"
                    close(w, rw, np.abs(rw) * 2.0 ** -20, "weights")


def route_bwd_places(be):
    """Empty places (ids outside the experts) and the same id twice."""
    ids = np.array([[3, -1, 5, 64, 3], [-1, -1, -1, -1, -1], [7, 7, 7, 7, 7], [0, 1, 2, 3, 2 ** 30]], dtype=np.int32)
    for softmax in (False, True):
        for normalize in (False, True):
            check_route_bwd(be, 4, 64, 5, softmax, normalize, 95, ids=ids)


def weights_values(be):
    """What a query may not look at does not reach the sums: rows behind the last sequence stay as they were, and
    NaN and infinities in keys and queries stay with their own key or query's keys."""
    q, k, idx, indptr, cu_q = step_batch([200, 150], [3, 2], 8, 2, 9)
    lse = steps.normaliser(q, k, idx, indptr, cu_q, -1, 1e7).astype(np.float32)
    ref = be.key_weights(q, k, idx, indptr, cu_q, lse, 3, 200, -1, 1e7, None)
    k2 = k.copy()
    k2[idx[40]] = 0x7FC0          # a NaN key
    k2[idx[199]] = 0x7F80         # the last key of sequence 0, seen by its last query only
    got = be.key_weights(q, k2, idx, indptr, cu_q, lse, 3, 200, -1, 1e7, None, errors=True)
    other = np.delete(np.arange(350), [40, 199])
    assert np.array_equal(got[other], ref[other]) and np.isnan(got[40])
    k3 = k.copy()
    k3[np.setdiff1d(np.arange(len(k)), idx)] = 0x7FC0  # cache rows that no entry names
    assert np.array_equal(be.key_weights(q, k3, idx, indptr, cu_q, lse, 3, 200, -1, 1e7, None), ref)
    q2 = q.copy()
    q2[4] = 0x7FC0                # the last query of sequence 1
    got = be.key_weights(q2, k, idx, indptr, cu_q, lse, 3, 200, -1, 1e7, None)
    assert np.array_equal(got[:200], ref[:200]) and np.all(np.isnan(got[200:]))
    idx2 = np.concatenate([idx, np.full(9, -5, dtype=np.int32)])  # entries behind the last sequence
    got = be.key_weights(q, k, idx2, indptr, cu_q, lse, 3, 200, -1, 1e7, None, fill=7.5)
    assert np.array_equal(got[:350], ref) and np.all(got[350:] == 7.5)


BAD_RANGE, BAD_LISTS = 5, 6  # MIMO_ERR_RANGE, MIMO_ERR_BAD_SEQLENS


def bad_lists(be):
    """Index lists that only the kernels can see: reported, nothing outside the buffers is read or written, and
    the consistent sequences of the call keep their results."""
    i32 = lambda *a: np.array(a, dtype=np.int32)
    w, idx = evict_weights(20, 1), np.arange(20, dtype=np.int32)
    for bad in (i32(0, 9, 5, 20), i32(1, 9, 15, 20), i32(0, 9, 15, 21), i32(-3, 9, 15, 20), i32(0, 15, 16, 20)):
        gi, gw, _, gf = be.evict(w, idx, bad, 10, 4, 0, 0, -9, errors=True)
        assert be.status == BAD_LISTS and np.all(gi == -9) and np.all(gw == -9) and np.all(gf == -9), bad
    q, k, _, _, _ = step_batch([10, 10], [1, 2], 4, 2, 6, spare=0)
    lse = np.ones((4, 3), dtype=np.float32)
    good = dict(idx=idx, ptr=i32(0, 10, 20), cu=i32(0, 1, 3))
    ref = be.key_weights(q, k, idx, good["ptr"], good["cu"], lse, 2, 12, -1, 1e7, None)
    for bad in (dict(ptr=i32(0, 25, 20)), dict(cu=i32(0, 5, 3)), dict(ptr=i32(0, 1, 2)), dict(cu=i32(-1, 1, 3)),
                dict(ptr=i32(0, 10, 40)), dict(idx=idx + np.int32(15)), dict(idx=idx - np.int32(3))):
        a = {**good, **bad}
        got = be.key_weights(q, k, a["idx"], a["ptr"], a["cu"], lse, 2, 12, -1, 1e7, None, errors=True, fill=-1.0)
        assert be.status == BAD_LISTS, bad
        if "ptr" in bad and bad["ptr"][2] == 40:
            assert np.array_equal(got[:10], ref[:10]) and np.all(got[10:] == -1)
    big = q.copy()
    big[0, 0, 0] = bits(1e5)
    be.key_weights(big, k, idx, good["ptr"], good["cu"], lse, 2, 12, -1, 1e7, None, errors=True)
    assert be.status == BAD_RANGE
