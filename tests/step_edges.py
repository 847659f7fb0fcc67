"""Further checks of the layer's steps, at values and sizes where they are easily wrong, for the same
backends as step_checks.py: the host build of the library (tests/host_emulation/edge_cases.py) and the
library on a GPU (tests/test_gpu_step_edges.py)."""
from __future__ import annotations

import numpy as np

from oracle.neighbors import e4m3_to_f64
from step_checks import bits


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


# Cases by name.
CASES = {
    "fp8_codes": fp8_codes,
}
