"""The layer's steps through the host build of the whole library (kernels on the CPU), checked against
their FP64 definitions.  Run as a child process:

    python step_cases.py <libmimo_attn_host.so> <case> [<case> ...]
"""
import ctypes as C
import sys

import numpy as np

from library_cases import DecodeDims, Lib, vp
import step_checks  # noqa: E402  (library_cases put tests/ on the path)


class Host:
    """The library's C entry points on numpy arrays."""

    def __init__(self, path):
        H = self.H = Lib(path)
        L = self.L = H.L
        i64, f, sz = C.c_int64, C.c_float, C.c_size_t
        L.mimo_rms_norm.argtypes = [vp, vp, vp, C.c_int, i64, i64, f, vp, vp, vp, vp, vp]
        L.mimo_rms_norm_bwd.argtypes = [vp, vp, C.c_int, vp, vp, i64, i64, f, vp, vp, vp, sz, vp]
        L.mimo_rms_norm_bwd_workspace_size.argtypes = [i64, i64]
        L.mimo_rms_norm_bwd_workspace_size.restype = sz
        L.mimo_moe_route_grouped.argtypes = [vp, vp, i64] + [C.c_int] * 6 + [f, vp, vp, vp]
        L.mimo_moe_route_bwd.argtypes = [vp, vp, vp, i64] + [C.c_int] * 4 + [f, vp, vp]
        L.mimo_decode_key_weights_workspace_size.argtypes = [C.POINTER(DecodeDims)]
        L.mimo_decode_key_weights_workspace_size.restype = sz
        L.mimo_decode_key_weights.argtypes = [vp] * 7 + [C.POINTER(DecodeDims), C.c_int, C.c_int, C.c_double, C.c_int,
                                                         vp, vp, sz, vp]
        L.mimo_kv_evict.argtypes = [vp] * 3 + [C.c_int] * 6 + [vp] * 5

    def rms_norm(self, x, w, r, eps, y, fp8):
        H, (T, n) = self.H, x.shape
        blocks = (n + 127) // 128
        ph = H.empty(T * n * 2) if r is not None else None
        py = H.empty(T * n * 2) if y else None
        pc, ps = (H.empty(T * n), H.empty(T * blocks * 4)) if fp8 else (None, None)
        st = self.L.mimo_rms_norm(H.put(x), H.put(r), H.put(w), int(w.dtype == np.float32), T, n, eps, ph, py, pc, ps, None)
        out = {}
        if ph:
            out["h"] = H.get(ph, (T, n), np.uint16)
        if py:
            out["y"] = H.get(py, (T, n), np.uint16)
        if pc:
            out["codes"], out["scale"] = H.get(pc, (T, n), np.uint8), H.get(ps, (T, blocks), np.float32)
        H.finish(st)
        return out

    def rms_norm_bwd(self, h, w, dy, dh, eps):
        H, (T, n) = self.H, h.shape
        need = self.L.mimo_rms_norm_bwd_workspace_size(T, n)
        dx, dw = H.empty(T * n * 2), H.empty(n * 4)
        st = self.L.mimo_rms_norm_bwd(H.put(h), H.put(w), int(w.dtype == np.float32), H.put(dy), H.put(dh), T, n, eps, dx,
                                      dw, H.empty(need), need, None)
        out = H.get(dx, (T, n), np.uint16), H.get(dw, (n,), np.float32)
        H.finish(st)
        return out

    def route(self, x, bias, k, groups, top_groups, softmax, normalize, scale):
        H, (T, E) = self.H, x.shape
        pi, pw = H.empty(T * k * 4), H.empty(T * k * 4)
        st = self.L.mimo_moe_route_grouped(H.put(x), H.put(bias), T, E, k, groups, top_groups, int(softmax), int(normalize),
                                           scale, pi, pw, None)
        out = H.get(pi, (T, k), np.int32), H.get(pw, (T, k), np.float32)
        H.finish(st)
        return out

    def route_bwd(self, x, ids, g, softmax, normalize, scale):
        H, (T, E) = self.H, x.shape
        pd = H.empty(T * E * 4)
        st = self.L.mimo_moe_route_bwd(H.put(x), H.put(ids), H.put(g), T, E, ids.shape[1], int(softmax), int(normalize),
                                       scale, pd, None)
        out = H.get(pd, (T, E), np.float32)
        H.finish(st)
        return out

    def key_weights(self, q, k, idx, indptr, cu_q, lse, max_q, max_kv, window, base, prev, errors=False, fill=None):
        H = self.H
        n = len(idx)
        d = DecodeDims(len(cu_q) - 1, q.shape[0], n, k.shape[0], max_q, max_kv, q.shape[1], k.shape[1], 192, 128)
        need = self.L.mimo_decode_key_weights_workspace_size(C.byref(d))
        # the workspace is 256-byte aligned: the guarded block ends at a page, so its size is rounded up
        need = (need + 255) // 256 * 256
        po = H.put(np.full(n, fill if fill is not None else np.nan, dtype=np.float32))
        st = self.L.mimo_decode_key_weights(H.put(q), H.put(k), H.put(idx), H.put(indptr), H.put(cu_q), H.put(lse),
                                            H.put(prev), C.byref(d), 0 if window >= 0 else 1, window, base, 64, po,
                                            H.empty(need), need, None)
        out = H.get(po, (n,), np.float32)
        if errors:
            self.status = self.L.mimo_attn_check(None)
        H.finish(st)
        return out

    def evict(self, w, idx, indptr, max_kv, budget, first, recent, fill, errors=False):
        H, n = self.H, len(idx)
        pi, pf = (H.put(np.full(max(n, 1), fill, dtype=np.int32)) for _ in range(2))
        pw, pp = H.put(np.full(max(n, 1), fill, dtype=np.float32)), H.empty(len(indptr) * 4)
        st = self.L.mimo_kv_evict(H.put(w), H.put(idx), H.put(indptr), len(indptr) - 1, n, max_kv, budget, first, recent,
                                  pi, pw, pp, pf, None)
        out = (H.get(pi, (n,), np.int32), H.get(pw, (n,), np.float32), H.get(pp, (len(indptr),), np.int32),
               H.get(pf, (n,), np.int32))
        if errors:
            self.status = self.L.mimo_attn_check(None)
        H.finish(st)
        return out


if __name__ == "__main__":
    be = Host(sys.argv[1])
    for name in sys.argv[2:]:
        step_checks.CASES[name](be)
        print("ok", name, flush=True)
