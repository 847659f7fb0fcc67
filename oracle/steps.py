"""The steps of a decoder layer around its attention, in FP64 (numpy): RMS norm with the residual's
addition and FP8 output, its gradient; grouped expert routing and its gradient; the attention weight each
cached key receives; eviction by that weight.  Plain definitions, one row, token or sequence at a time;
test infrastructure only, sharing no code with the library."""
from __future__ import annotations

import numpy as np

from .neighbors import bf16_bits_to_f64, e4m3_to_f64, sigmoid_f64


def f64_to_bf16_bits(x: np.ndarray) -> np.ndarray:
    """Round to nearest even to BF16, from the exact value (values in BF16's normal range)."""
    x = np.asarray(x, dtype=np.float64)
    f = x.astype(np.float32)
    # round to odd in FP32 first, so that the second rounding sees on which side of the FP32 value x lies
    b = f.view(np.uint32).astype(np.uint64)
    inexact = f.astype(np.float64) != x
    toward = np.abs(f.astype(np.float64)) > np.abs(x)
    b = np.where(inexact & toward, b - 1, b)
    b = np.where(inexact, b | 1, b)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) & 0xFFFF).astype(np.uint16)


# ---------------------------------------------------------------- RMS norm
def rms_norm(x_bits, weight, residual_bits=None, eps=1e-6):
    """h = bf16(x + residual) (bits), y = h / sqrt(mean(h^2) + eps) * weight (FP64)."""
    x = bf16_bits_to_f64(x_bits)
    h_bits = np.asarray(x_bits, dtype=np.uint16)
    if residual_bits is not None:
        # the sum of two BF16 values is exact in FP64 unless their exponents are over 45 apart
        h_bits = f64_to_bf16_bits(x + bf16_bits_to_f64(residual_bits))
    h = bf16_bits_to_f64(h_bits)
    w = np.asarray(weight, dtype=np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w
    return h_bits, y


def fp8_blocks(y, block=128):
    """Scales max(max|y| / 448, 2^-126) per 1 x block, [T, ceil(H / block)]."""
    T, H = y.shape
    return np.stack([np.maximum(np.abs(y[:, j:j + block]).max(-1) / 448.0, 2.0 ** -126)
                     for j in range(0, H, block)], -1)


def fp8_values(codes, scales, block=128):
    """What codes [T, H] and scales [T, ceil(H / block)] stand for."""
    v = e4m3_to_f64(codes)
    return v * np.repeat(np.asarray(scales, dtype=np.float64), block, axis=-1)[:, :v.shape[1]]


def rms_norm_bwd(h_bits, weight, dy_bits, dh_bits=None, eps=1e-6):
    """dx [T, H] and dweight [H] by the chain rule on y = h r w, r = (mean(h^2) + eps)^(-1/2)."""
    h, dy = bf16_bits_to_f64(h_bits), bf16_bits_to_f64(dy_bits)
    w = np.asarray(weight, dtype=np.float64)
    H = h.shape[-1]
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    dr = (dy * w * h).sum(-1, keepdims=True)           # dL/dr
    dx = dy * w * r + dr * (-(r ** 3) / H) * h         # dr/dh = -r^3 h / H
    if dh_bits is not None:
        dx = dx + bf16_bits_to_f64(dh_bits)
    return dx, (dy * h * r).sum(0)


# ---------------------------------------------------------------- routing
def scores(logits, softmax):
    x = np.asarray(logits, dtype=np.float64)
    if not softmax:
        return sigmoid_f64(x)
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def route_grouped(logits, bias=None, top_k=8, num_groups=1, top_groups=1, softmax=False, normalize=True, scale=1.0):
    """ids [T, k] int32, weights [T, k] FP64; the choice on FP32 keys, ties to the lower index."""
    with np.errstate(all="ignore"):
        s = scores(logits, softmax)
        key = s.astype(np.float32)
        if bias is not None:
            key = (key + np.asarray(bias, dtype=np.float32)).astype(np.float32)
    key = np.where(np.isnan(key), np.float32(-np.inf), key)
    T, E = key.shape
    size = E // num_groups
    if num_groups > 1:
        by = np.sort(key.reshape(T, num_groups, size), -1)
        with np.errstate(all="ignore"):
            gs = (by[..., -1] + by[..., -2]).astype(np.float32) if size > 1 else by[..., -1]
        gs = np.where(np.isnan(gs), np.float32(-np.inf), gs)
        kept = np.argsort(-gs, axis=-1, kind="stable")[:, :top_groups]  # stable: ties to the lower group
        open_ = np.zeros((T, num_groups), dtype=bool)
        np.put_along_axis(open_, kept, True, -1)
        open_ = np.repeat(open_, size, -1)
    else:
        open_ = np.ones((T, E), dtype=bool)
    # experts of the kept groups first, then by key, then by index
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key.astype(np.float64), ~open_), axis=-1)
    ids = order[:, :top_k].astype(np.int32)
    w = np.take_along_axis(s, ids.astype(np.int64), -1)
    if normalize:
        total = w.sum(-1, keepdims=True)
        with np.errstate(all="ignore"):
            w = np.where(total == 0, 0.0, w / total)
    return ids, scale * w


def route_bwd(logits, ids, dweights, softmax=False, normalize=True, scale=1.0):
    """dlogits [T, E] by Jacobians: dw/dc over the chosen scores, dc/dx over the logits."""
    s = scores(logits, softmax)
    T, E = s.shape
    d = np.zeros((T, E))
    for t in range(T):
        place = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        e = [int(ids[t, j]) for j in place]
        if not e:
            continue
        c, g = s[t, e], scale * np.asarray(dweights, dtype=np.float64)[t, place]
        if normalize:
            S = c.sum()
            dc = np.zeros_like(c) if S == 0 else (np.eye(len(e)) / S - c[:, None] / S ** 2).T @ g
        else:
            dc = g
        ds = np.zeros(E)
        np.add.at(ds, e, dc)
        d[t] = s[t] * (ds - (ds * s[t]).sum()) if softmax else ds * s[t] * sigmoid_f64(-np.asarray(logits[t], dtype=np.float64))
    return d


# ---------------------------------------------------------------- key weights and eviction
def _turned(x, pos, base, rope_dims=64):
    h = rope_dims // 2
    a = np.asarray(pos, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(h) / rope_dims)
    z = (x[..., :h] + 1j * x[..., h:rope_dims]) * np.exp(1j * a)[:, None, :]
    return np.concatenate([z.real, z.imag, x[..., rope_dims:]], -1)


def key_weights(q_bits, k_bits, kv_indices, kv_indptr, cu_q, lse, window, base, prev=None):
    """[total_kv] FP64: prev + sum over heads and queries that see the key of exp(score - lse)."""
    q, k = bf16_bits_to_f64(q_bits), bf16_bits_to_f64(k_bits)
    hq, hkv = q.shape[1], k.shape[1]
    out = np.zeros(len(kv_indices)) if prev is None else np.asarray(prev, dtype=np.float64).copy()
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], kv_indptr[b], kv_indptr[b + 1]
        n, m = k1 - k0, q1 - q0
        pos = np.arange(n)
        kk = _turned(k[kv_indices[k0:k1]], pos, base)
        qq = _turned(q[q0:q1], pos[n - m:], base)
        off = pos[n - m:, None] - pos[None]
        may = (off >= 0) & ((off <= window) if window >= 0 else True)
        for h in range(hq):
            with np.errstate(all="ignore"):
                p = np.exp(qq[:, h] @ kk[:, h // (hq // hkv)].T / np.sqrt(192.0) - np.asarray(lse, dtype=np.float64)[h, q0:q1, None])
            out[k0:k1] += np.where(may, p, 0.0).sum(0)
    return out


def normaliser(q_bits, k_bits, kv_indices, kv_indptr, cu_q, window, base, sink=None):
    """lse [Hq, Tq] FP64 of the same scores."""
    q, k = bf16_bits_to_f64(q_bits), bf16_bits_to_f64(k_bits)
    hq, hkv = q.shape[1], k.shape[1]
    lse = np.zeros((hq, q.shape[0]))
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], kv_indptr[b], kv_indptr[b + 1]
        n, m = k1 - k0, q1 - q0
        pos = np.arange(n)
        kk = _turned(k[kv_indices[k0:k1]], pos, base)
        qq = _turned(q[q0:q1], pos[n - m:], base)
        off = pos[n - m:, None] - pos[None]
        may = (off >= 0) & ((off <= window) if window >= 0 else True)
        for h in range(hq):
            s = np.where(may, qq[:, h] @ kk[:, h // (hq // hkv)].T / np.sqrt(192.0), -np.inf)
            top = s.max(-1, keepdims=True)
            v = (top + np.log(np.exp(s - top).sum(-1, keepdims=True)))[:, 0]
            lse[h, q0:q1] = v if sink is None else np.logaddexp(v, float(sink[h]))
    return lse


def kv_evict(weights, kv_indices, kv_indptr, budget, keep_first=0, keep_recent=0):
    """(kept rows, kept weights, new_indptr, freed rows), by sorting."""
    idx, w, new, gone = [], [], [0], []
    for b in range(len(kv_indptr) - 1):
        at = range(kv_indptr[b], kv_indptr[b + 1])
        n = len(at)
        must = [i for j, i in enumerate(at) if j < keep_first or j >= n - keep_recent]
        rest = [i for j, i in enumerate(at) if not (j < keep_first or j >= n - keep_recent)]
        if n <= budget:
            keep = set(at)
        else:
            val = lambda i: (1, 0.0) if np.isnan(weights[i]) else (0, -float(weights[i]))
            keep = set(must) | set(sorted(rest, key=lambda i: (*val(i), i))[:budget - len(must)])
        idx += [kv_indices[i] for i in at if i in keep]
        w += [weights[i] for i in at if i in keep]
        gone += [kv_indices[i] for i in at if i not in keep]
        new.append(len(idx))
    return (np.array(idx, dtype=np.int32), np.array(w, dtype=np.float32), np.array(new, dtype=np.int32),
            np.array(gone, dtype=np.int32))
