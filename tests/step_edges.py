"""Further checks of the layer's steps, at values and sizes where they are easily wrong, for the same
backends as step_checks.py: the host build of the library (tests/host_emulation/edge_cases.py) and the
library on a GPU (tests/test_gpu_step_edges.py)."""
from __future__ import annotations

import numpy as np

from oracle import steps
from oracle.neighbors import bf16_bits_to_f64, e4m3_to_f64
from step_checks import bits, check_evict, close, evict_weights, step_batch, weights_tolerance


# ---------------------------------------------------------------- RMS norm: the FP8 codes
def e4m3_codes(q):
    """E4M3 codes of q (finite, at most 448): nearest, ties to the even code."""
    grid = e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))  # ascending
    a = np.abs(np.asarray(q, dtype=np.float64))
    up = np.searchsorted(grid, a).clip(0, 0x7E)
    down = np.maximum(up - 1, 0)
    far, near = grid[up] - a, a - grid[down]
    take = np.where((near < far) | ((near == far) & (down % 2 == 0)), down, up)
    return (take | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def fp8_codes(be):
    """codes = E4M3(y / scale), nearest even, bit for bit.  Rows of +-1 have rstd 1 exactly (the mean of their
    squares is 1, beside which eps = 1e-18 is nothing), so y is the FP32 weight with the row's sign."""
    rng = np.random.default_rng(7)
    grid = e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))
    middle = (grid[1:] + grid[:-1]) / 2
    for T, H in ((3, 128), (2, 2048), (2, 4112)):
        blocks = -(-H // 128)
        w = np.zeros(blocks * 128, dtype=np.float32)
        for b in range(blocks):
            # scales of 17 bits, so that 448 scale and scale times a midpoint (at most 5 bits) are exact in FP32
            s = float(rng.integers(2 ** 16, 2 ** 17) | 1) * 2.0 ** float(rng.integers(-30, 10))
            v = rng.choice(middle, 128) if b % 2 == 0 else rng.uniform(-448, 448, 128)
            v[rng.integers(3, 16)] = 448.0
            w[128 * b:128 * b + 128] = (v * s).astype(np.float32)
        w[1::64], w[2::64] = 0.0, -0.0  # (a code of zero keeps its sign)
        w = w[:H]
        sign = rng.choice([-1.0, 1.0], (T, H))
        got = be.rms_norm(bits(sign), w, None, 1e-18, y=False, fp8=True)
        y = (sign * w).astype(np.float32)
        most = np.stack([np.abs(y[:, j:j + 128]).max(-1) for j in range(0, H, 128)], -1)
        scale = most / np.float32(448.0)
        assert np.array_equal(got["scale"], scale)
        want = e4m3_codes(y / np.repeat(scale, 128, -1)[:, :H])
        off = got["codes"] != want
        assert not off.any(), f"{off.sum()} of {off.size} codes of {H} columns, first at {tuple(np.argwhere(off)[0])}"


def fp8_extremes(be):
    """The same at the ends of FP32: blocks of zeros, of subnormals, of values near 2^-120 and near the largest, and
    blocks with an infinite weight (scale infinite: codes 0, NaN where y is infinite)."""
    rng = np.random.default_rng(8)
    H = 128 * 6
    w = rng.standard_normal(H)
    for b, size in enumerate((0.0, 2.0 ** -140, 2.0 ** -118, 2.0 ** 126, 1.0, 2.0 ** -126)):
        w[128 * b:128 * b + 128] *= size
    w = w.astype(np.float32)
    w = np.where(np.isfinite(w), w, np.float32(3e38))
    w[128 * 4 + 9], w[128 * 4 + 40] = np.inf, -0.0
    sign = rng.choice([-1.0, 1.0], (2, H))
    got = be.rms_norm(bits(sign), w, None, 1e-18, y=False, fp8=True)
    y = (sign * w).astype(np.float32)
    scale = np.maximum(np.abs(y).reshape(2, -1, 128).max(-1) / np.float32(448.0), np.float32(2.0 ** -126)).astype(np.float32)
    assert np.array_equal(got["scale"], scale)
    with np.errstate(invalid="ignore"):
        q = y / np.repeat(scale, 128, -1)
    nan = np.isnan(q)
    assert nan.sum() == 2 and np.all((got["codes"][nan] & 0x7F) == 0x7F)
    # below about 2^-100 the remainder has no room: codes may be the neighbour's at a midpoint
    exact = np.repeat((scale >= 2.0 ** -100), 128, -1) & ~nan
    want = e4m3_codes(np.where(nan, 0, q))
    assert np.array_equal(got["codes"][exact], want[exact])
    near = ~exact & ~nan
    v = e4m3_to_f64(got["codes"][near])
    assert np.all(np.abs(v - q[near]) <= np.abs(q[near]) * 2.0 ** -4 * (1 + 2.0 ** -20) + 2.0 ** -10 * (1 + 2.0 ** -20))


# ---------------------------------------------------------------- the router's gradient where one expert dominates
def route_bwd_terms(x, ids, g, softmax, normalize, scale):
    """(dlogits, tolerance) of one token in FP64, from differences of the gradients g, so that nothing is lost where
    one expert has nearly the whole sum.  With an expert's m places taken together (g: their mean):
      normalised       d_e = scale c_e p_e sum_i p_i (g_e - g_i),   p = m s / sum m s,  c = 1 - s (sigmoid) or 1
      plain sigmoid    d_e = scale m g_e s_e c_e
      plain softmax    d_e = scale s_e (m_e g_e U + sum_i s_i (m_e g_e - m_i g_i)) for a chosen e, U the score of all
                       that are not, and -scale s_e sum_i s_i m_i g_i for those
    The tolerance counts roundings of FP32 operations, on the magnitudes of the terms with the differences taken from
    the chosen expert of the largest logit: an exponential of t = x - max is off by 2^-24 |t| (the subtraction) and
    2^-23, a sum of n terms by n 2^-24 (n 32 for the places, 512 / 32 + 5 for a row), quotients and products by a
    few; 64 + |t| in all.  Gradients of one expert's places are added in two floats: 2^-46 of their magnitude.  Below 2^-126 FP32 has its own spacing."""
    E, xd = len(x), x.astype(np.float64)
    d, tol = np.zeros(E), np.zeros(E)
    places = {}
    for i, v in zip(ids, g.astype(np.float64)):
        if 0 <= i < E:
            places.setdefault(int(i), []).append(v)
    e = np.array(sorted(places), dtype=int)
    if len(e) == 0:
        return d, tol
    m, total = np.array([len(places[i]) for i in e], dtype=float), np.array([sum(places[i]) for i in e])
    top = int(np.argmax(xd[e]))
    u = 2.0 ** -24
    with np.errstate(over="ignore", under="ignore"):
        near = np.exp(-np.abs(xd))
        s = np.where(xd >= 0, 1, near) / (1 + near)
        c = np.where(xd >= 0, near, 1) / (1 + near)
        if softmax and not normalize:
            t = np.minimum(np.abs(xd - xd.max()), 1000)  # (-inf: a score of zero)
            s = np.exp(-t) / np.exp(-t).sum()
            others = np.ones(E, dtype=bool)
            others[e] = False
            U, gm = s[others].sum(), (s[e] * total).sum()
            d, tol = -s * gm, s * (64 + t) * u * (s[e] * np.abs(total) * (1 + t[e])).sum()
            d[e] = [s[i] * (G * U + (s[e] * (G - total)).sum()) for i, G in zip(e, total)]
            dev = np.abs(total - total[top]) + np.where(m.max() > 1, np.abs(total) + np.abs(total[top]), 0) * u * 4 * u / (64 * u)
            tol[e] = s[e] * (64 + t[e] + U * t.max()) * u * (np.abs(total) * U + s[e].sum() * dev + (s[e] * dev * (1 + t[e])).sum())
        elif not normalize:
            d[e] = total * s[e] * c[e]
            tol[e] = np.abs(d[e]) * 16 * u
        else:
            t = np.maximum(xd[e] - xd[e].max(), -1000)
            if softmax:
                p = m * np.exp(t)
            else:  # s = exp(min(x, 0)) / (1 + exp(-|x|)); a common factor cancels
                p = m * np.exp(np.minimum(xd[e], 0) - min(xd[e].max(), 0)) / (1 + near[e])
            p = p / p.sum()
            G, t, k = total / m, np.abs(t), 1.0 if softmax else c[e]
            d[e] = k * p * np.array([(p * (v - G)).sum() for v in G])
            dev = np.abs(G - G[top]) + np.where(m.max() > 1, np.abs(G) + np.abs(G[top]), 0) * u * 4 * u / (64 * u)
            tol[e] = k * p * (64 + t) * u * (dev + (p * dev * (1 + t)).sum())
    return scale * d, np.abs(scale) * tol + 2.0 ** -140


def check_gradient(be, x, ids, g, softmax, normalize, scale=2.5):
    d = be.route_bwd(x, ids, g, softmax, normalize, scale)
    for t in range(len(x)):
        ref, tol = route_bwd_terms(x[t], ids[t], g[t], softmax, normalize, scale)
        close(d[t], ref, tol, f"dlogits of token {t} (softmax {softmax}, normalised {normalize}, logits of the chosen {x[t][ids[t] % len(x[t])]})")


FORMS = ((False, True), (False, False), (True, True), (True, False))


def peaked(T, E, k, gap, seed, level=0.0):
    """Logits about `level`, one chosen expert `gap` above the other chosen; gradients of like size."""
    rng = np.random.default_rng(seed)
    x = (level + rng.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(rng.random((T, E)), -1)[:, :k].astype(np.int32)
    at = np.arange(T), ids[np.arange(T), rng.integers(0, k, T)]
    x[at] = (x.max(-1) + gap).astype(np.float32)
    return x, ids, rng.standard_normal((T, k)).astype(np.float32)


def gradient_peaked(be):
    """One expert has nearly all of the chosen experts' sum (or of the softmax): the row is what the others leave."""
    for gap in (0, 4, 8, 14, 20, 45, 80):
        for E, k in ((128, 6), (60, 12), (512, 32)):
            for softmax, normalize in FORMS:
                for level in (0.0, -gap) if not softmax else (0.0,):
                    check_gradient(be, *peaked(5, E, k, gap, 200 + gap + E, level), softmax, normalize)


def gradient_levels(be):
    """Sigmoid scores far below one: chosen logits on both sides of -60 and -80, and one far above the others."""
    for level, gap in ((-30, 20), (-58, 10), (-62, 10), (-70, 5), (-70, 60), (-85, 10), (-100, 30), (-100, 100)):
        for E, k in ((64, 4), (96, 16)):
            for normalize in (True, False):
                check_gradient(be, *peaked(4, E, k, gap, 300 - level + gap, level), False, normalize)


def gradient_alike(be):
    """Chosen experts whose gradients are alike: normalised rows are zero, plain softmax rows what the others hold."""
    for softmax, normalize in FORMS:
        x, ids, g = peaked(4, 64, 8, 0, 400)
        g[:] = g[:, :1]
        x[np.arange(4)[:, None], ids[:, :2]] = 20.0  # two that share nearly the whole
        check_gradient(be, x, ids, g, softmax, normalize)
        if normalize:
            assert np.all(be.route_bwd(x, ids, g, softmax, normalize, 2.5) == 0)
    x, ids, g = peaked(3, 64, 1, 5, 401)
    for softmax in (False, True):
        assert np.all(be.route_bwd(x, ids, g, softmax, True, 1.0) == 0)  # one place: its weight is the scale


def gradient_places(be):
    """The same expert in two and more places, empty places, the dominating expert among them; switched-off experts."""
    x, _, g = peaked(6, 64, 6, 0, 500)
    ids = np.array([[3, 3, 9, 10, -1, 64], [3, 9, 3, 11, 9, 2], [5, 5, 5, 5, 6, 7], [-1, -1, -1, -1, -1, 8],
                    [-1, -7, 64, 99, -1, -1], [0, 1, 2, 3, 4, 63]], dtype=np.int32)
    for gap in (0, 14, 30):
        for at in (3, 9, 5, 63):
            z = x.copy()
            z[:, at] += np.float32(gap)
            for softmax, normalize in FORMS:
                check_gradient(be, z, ids, g, softmax, normalize)
    wild = g.copy()
    wild[(ids < 0) | (ids > 63)] = np.nan  # an empty place's gradient is not read into the others
    for softmax, normalize in FORMS:
        assert np.array_equal(be.route_bwd(x, ids, wild, softmax, normalize, 2.5), be.route_bwd(x, ids, g, softmax, normalize, 2.5))
    x[:, ::2] = -np.inf
    x[:, 1::4] = np.finfo(np.float32).min
    for softmax, normalize in FORMS:
        check_gradient(be, x, np.array([[1, 2, 3, 7, 11, 0]] * 6, dtype=np.int32), g, softmax, normalize)


# ---------------------------------------------------------------- key weights of large queries and small keys
def check_sizes(be, kv_lens, q_lens, hq, hkv, window, base, seed, q_size, k_size):
    """Queries and keys of any sizes: step_checks.weights_tolerance, and, below the 22 bits that it counts, the
    rotated values' absolute error of 2^-36 (FP16 down to 2^-14, its rest times 2^11 down to 2^-25)."""
    q, k, idx, indptr, cu_q = step_batch(kv_lens, q_lens, hq, hkv, seed)
    scaled = lambda a, f: bits(bf16_bits_to_f64(a) * f)
    q, k = scaled(q, q_size), scaled(k, k_size)
    lse = steps.normaliser(q, k, idx, indptr, cu_q, window, base).astype(np.float32)
    got = be.key_weights(q, k, idx, indptr, cu_q, lse, max(q_lens), max(kv_lens), window, base, None)
    ref = steps.key_weights(q, k, idx, indptr, cu_q, lse, window, base)
    tol = weights_tolerance(q, k, idx, indptr, cu_q, lse, window, base, None)
    # 64 dims of at most sqrt(2) 6 sizes each; a weight is at most one per query and head
    floor = 64 * 2.0 ** -36 * 9 * (q_size + k_size) / np.sqrt(192.0)
    close(got, ref, tol + ref * floor, f"key weights, queries of {q_size}, keys of {k_size}")


def weights_sizes(be):
    for q_size, k_size in ((3000.0, 3e-4), (3e-4, 3000.0), (2000.0, 1e-3), (100.0, 0.01), (8000.0, 1e-6), (1e-6, 8000.0), (0.01, 0.01)):
        check_sizes(be, [130, 40], [1, 3], 8, 2, -1, 1e7, 600, q_size, k_size)
        check_sizes(be, [200], [70], 4, 2, 128, 1e4, 601, q_size, k_size)


# ---------------------------------------------------------------- the router's weights of small scores
def route_scales(be, tokens=(3, 400)):
    """Sigmoid scores of about e^-75, chosen by biases far enough apart, and scale factors of any size: the weights
    are scale times the scores' shares (eight FP32 roundings, as in step_checks.check_route)."""
    for T in tokens:
        for E, k, groups, top in ((64, 8, 8, 4), (256, 8, 8, 4), (64, 3, 1, 1)):
            x = (-75 + np.random.default_rng(E).standard_normal((T, E))).astype(np.float32)
            b = (0.05 * np.random.default_rng(E + 1).permutation(E)).astype(np.float32)
            for scale in (1e30, 2.5, 1e-30):
                for normalize in (True, False):
                    ids, w = be.route(x, b, k, groups, top, False, normalize, scale)
                    rid, rw = steps.route_grouped(x, b, k, groups, top, False, normalize, np.float32(scale).astype(np.float64))
                    assert np.array_equal(ids, rid)
                    close(w, rw, np.abs(rw) * 2.0 ** -20 + 2.0 ** -149, f"weights, {T} tokens, {E} experts, scale {scale}, normalised {normalize}")


# ---------------------------------------------------------------- eviction by every number of CTAs to a sequence
def evict_clusters(be):
    """One, two, four and eight CTAs to a sequence (by length; by number, where there are many), with and without
    room for the weights in shared memory, and the same batch in several forms: the results agree bit for bit."""
    for lens, budget in (([8192], 1000), ([8193, 3, 0, 600], 2000), ([16384], 16383), ([16385, 40], 5000), ([65536], 100),
                         ([70001, 9], 30000), ([9000] + [5] * 80, 700), ([17000] + [3] * 40, 700), ([70000] + [1] * 15, 6000),
                         ([50000] + [2] * 80, 49999)):
        for kind in ("ties",) if sum(lens) > 40000 else ("spread", "ties", "wild"):
            check_evict(be, lens, budget, 3, 40, 700 + len(lens), kind)


def route_low(be, tokens=(3, 400)):
    """Softmax scores far below the largest, chosen by their biases: a weight is off by the roundings of one
    exponential, its sum and a quotient (2^-20), not by that of the difference x - max, which grows with it (half of
    2^-17 at 70); weights that keep the softmax's sum carry its approximate exponentials too (2^-19)."""
    for T in tokens:
        for E, k, groups, top in ((64, 8, 8, 4), (128, 8, 1, 1), (64, 3, 1, 1)):
            rng = np.random.default_rng(E + T)
            x = rng.uniform(-75, -20, (T, E)).astype(np.float32)
            x[np.arange(T), rng.integers(0, E, T)] = rng.uniform(0, 3, T).astype(np.float32)
            b = (3.0 * rng.permutation(E)).astype(np.float32)
            for normalize, tol in ((True, 2.0 ** -20), (False, 2.0 ** -19)):
                ids, w = be.route(x, b, k, groups, top, True, normalize, 2.5)
                rid, rw = steps.route_grouped(x, b, k, groups, top, True, normalize, 2.5)
                assert np.array_equal(ids, rid)
                close(w, rw, np.abs(rw) * tol + 2.0 ** -149, f"weights, {T} tokens, {E} experts, normalised {normalize}")


# ---------------------------------------------------------------- bounds that are not reached, sequences that are empty
def loose_bounds(be):
    """max_q_len, max_kv_len: bounds that no sequence reaches, as a captured graph's; sequences without new queries or
    without keys among the others."""
    for kv, q, hq, hkv, window in (([130, 0, 5, 300], [1, 0, 0, 3], 8, 2, -1), ([0, 200, 129, 0], [0, 2, 1, 0], 16, 1, -1),
                                   ([64, 0, 400], [64, 0, 2], 6, 3, 128)):
        qq, k, idx, indptr, cu_q = step_batch(kv, q, hq, hkv, 800)
        rng = np.random.default_rng(801)
        lse = (5 + rng.standard_normal((hq, sum(q)))).astype(np.float32)
        prev = np.abs(rng.standard_normal(len(idx))).astype(np.float32)
        ref = steps.key_weights(qq, k, idx, indptr, cu_q, lse, window, 1e5, prev)
        tol = weights_tolerance(qq, k, idx, indptr, cu_q, lse, window, 1e5, prev)
        for max_q, max_kv in ((max(q), max(kv)), (sum(q), sum(kv)), (max(q), sum(kv))):
            close(be.key_weights(qq, k, idx, indptr, cu_q, lse, max_q, max_kv, window, 1e5, prev), ref, tol, "key weights")
    lens = [40, 0, 300, 7, 9000]
    total = sum(lens)
    w, idx = evict_weights(total, 802), np.arange(total, dtype=np.int32)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ri, rw, rp, rf = steps.kv_evict(w, idx, indptr, 50, 3, 5)
    for most in (9000, total):
        gi, gw, gp, gf = be.evict(w, idx, indptr, most, 50, 3, 5, -1)
        assert np.array_equal(gp, rp) and np.array_equal(gi[:len(ri)], ri) and np.array_equal(gf[:len(rf)], rf)
        assert np.array_equal(gw[:len(ri)], rw)


# Cases by name.
CASES = {
    "loose_bounds": loose_bounds,
    "route_low": route_low,
    "evict_clusters": evict_clusters,
    "route_scales": route_scales,
    "weights_sizes": weights_sizes,
    "gradient_peaked": gradient_peaked,
    "gradient_levels": gradient_levels,
    "gradient_alike": gradient_alike,
    "gradient_places": gradient_places,
    "fp8_codes": fp8_codes,
    "fp8_extremes": fp8_extremes,
}
