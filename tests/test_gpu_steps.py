"""The layer's steps on a GPU: RMS norm (BF16 and FP8 output) and its gradient, grouped routing and its
gradient, key weights and cache eviction, against their FP64 definitions (tests/step_checks.py holds the
checks and where their tolerances come from)."""
import numpy as np
import pytest
import torch

import step_checks as S
from oracle import steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from global_attention_moe_b200 import mimo_attn
    return mimo_attn


def dev(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    t = torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()
    return t.view(torch.bfloat16) if a.dtype == np.uint16 else t


def host(t):
    t = t.contiguous()
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


class Gpu:
    """The Python entry points on numpy arrays."""

    def __init__(self, M):
        self.M = M

    def ok(self):
        assert self.M.check() == self.M.OK

    def rms_norm(self, x, w, r, eps, y, fp8):
        M, out = self.M, {}
        if fp8:
            codes, scale, h, *rest = M.rms_norm_fp8(dev(x), dev(w), dev(r), eps, with_bf16=y)
            out = {"codes": host(codes), "scale": host(scale), "h": host(h)}
            if y:
                out["y"] = host(rest[0])
        else:
            yy, h = M.rms_norm(dev(x), dev(w), dev(r), eps)
            out = {"y": host(yy), "h": host(h)}
        self.ok()
        return out

    def rms_norm_bwd(self, h, w, dy, dh, eps):
        dx, dw = self.M.rms_norm_bwd(dev(h), dev(w), dev(dy), dev(dh), eps)
        self.ok()
        return host(dx), host(dw)

    def route(self, x, bias, k, groups, top_groups, softmax, normalize, scale):
        ids, w = self.M.moe_route_grouped(dev(x), dev(bias), k, groups, top_groups, int(softmax), normalize, scale)
        self.ok()
        return host(ids), host(w)

    def route_bwd(self, x, ids, g, softmax, normalize, scale):
        d = self.M.moe_route_bwd(dev(x), dev(ids), dev(g), int(softmax), normalize, scale)
        self.ok()
        return host(d)

    def key_weights(self, q, k, idx, indptr, cu_q, lse, max_q, max_kv, window, base, prev, errors=False, fill=None):
        out = None if fill is None else torch.full((len(idx),), fill, device="cuda")
        w = self.M.decode_key_weights(dev(q), dev(k), dev(idx), dev(indptr), dev(cu_q), dev(lse), max_q, max_kv,
                                      0 if window >= 0 else 1, window, base, prev=dev(prev), out=out)
        self.status = self.M.check()
        assert errors or self.status == self.M.OK, self.M.status_string(self.status)
        return host(w)

    def evict(self, w, idx, indptr, max_kv, budget, first, recent, fill, errors=False):
        # through the C entry point, so that the buffers can be filled first
        n = len(idx)
        full = lambda dt: torch.full((max(n, 1),), fill, dtype=dt, device="cuda")
        gi, gf, gw = full(torch.int32), full(torch.int32), full(torch.float32)
        gp = torch.empty(len(indptr), dtype=torch.int32, device="cuda")
        dw, di, dp = dev(w), dev(idx), dev(indptr)
        st = self.M.LIB.mimo_kv_evict(dw.data_ptr(), di.data_ptr(), dp.data_ptr(), len(indptr) - 1, n, max_kv, budget,
                                      first, recent, gi.data_ptr(), gw.data_ptr(), gp.data_ptr(), gf.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
        assert st == self.M.OK
        self.status = self.M.check()
        assert errors or self.status == self.M.OK, self.M.status_string(self.status)
        return host(gi)[:n], host(gw)[:n], host(gp), host(gf)[:n]


@pytest.fixture(scope="module")
def be(M):
    return Gpu(M)


@pytest.mark.parametrize("name", sorted(S.CASES))
def test_steps_match_their_definitions(be, name):
    S.CASES[name](be)


# ---------------------------------------------------------------- larger sizes
@pytest.mark.parametrize("T,H,residual,fp8", [(300, 4096, True, True), (2049, 1024, False, False), (77, 8192, True, True),
                                              (1000, 2048, True, False)])
def test_norm_sizes(be, T, H, residual, fp8):
    S.check_norm(be, T, H, T + H, residual=residual, fp8=fp8, both=fp8)


@pytest.mark.parametrize("T,H,dh", [(3000, 256, True), (1201, 2048, True), (700, 4096, False), (333, 8192, True)])
def test_norm_bwd_sizes(be, T, H, dh):
    S.check_norm_bwd(be, T, H, T + H, dh=dh)


@pytest.mark.parametrize("T,E,k,groups,top,softmax,bias", [(3001, 256, 8, 8, 4, False, True), (2000, 256, 8, 1, 1, True, False),
                                                           (1500, 160, 6, 8, 3, True, True), (2500, 128, 8, 1, 1, False, True),
                                                           (1000, 64, 6, 4, 1, False, False), (700, 512, 10, 16, 4, True, False)])
def test_route_sizes(be, T, E, k, groups, top, softmax, bias):
    S.check_route(be, T, E, k, groups, top, softmax, True, bias, T + E, scale=2.5)
    S.check_route(be, T // 3, E, k, groups, top, softmax, True, bias, T + E + 1, "near")


@pytest.mark.parametrize("T,E,k,groups,top,softmax,bias,kind", [
    (40001, 256, 8, 8, 4, False, True, "normal"), (30011, 256, 8, 1, 1, True, False, "normal"),
    (60000, 128, 6, 4, 2, True, True, "normal"), (80001, 64, 8, 8, 4, False, True, "ties"),
    (30000, 256, 8, 8, 4, False, True, "near"), (50000, 160, 6, 4, 3, False, False, "masked")])
def test_route_many_tokens(be, T, E, k, groups, top, softmax, bias, kind):
    S.check_route(be, T, E, k, groups, top, softmax, True, bias, T + E, kind, scale=2.5)


def test_route_biases_far_apart(be):
    S.route_far(be, (3, 30000))  # the kernels of few and of many tokens


@pytest.mark.parametrize("kv,q,hq,hkv,window,sink", [([3000, 1025, 640], [1, 1, 1], 64, 4, -1, False),
                                                     ([2100, 900, 129], [8, 8, 8], 64, 4, -1, False),
                                                     ([1500, 300], [8, 1], 64, 8, 128, True),
                                                     ([900, 400], [150, 90], 16, 1, -1, False),
                                                     ([700], [300], 16, 2, 128, True)])
def test_key_weights_sizes(be, kv, q, hq, hkv, window, sink):
    S.check_weights(be, kv, q, hq, hkv, window, 1e7 if window < 0 else 1e4, sum(kv), sink=sink, prev=True)


@pytest.mark.parametrize("lens,budget,first,recent", [([70000], 5000, 4, 100), ([131072, 3, 9000], 8192, 0, 1024),
                                                      (list(range(0, 900, 7)), 300, 2, 30)])
@pytest.mark.parametrize("kind", ["spread", "ties", "wild"])
def test_evict_sizes(be, lens, budget, first, recent, kind):
    S.check_evict(be, lens, budget, first, recent, 7, kind)


# ---------------------------------------------------------------- together, as a decode step uses them
def test_a_layer_step(M):
    """norm -> FP8 weights -> fused QKV -> split -> KV-cache attention -> key weights -> eviction -> attention over
    what stayed -> projection -> norm with the residual (FP8 and BF16) -> router -> the router's and the norm's
    gradients, each checked against its definition on the tensors that came before."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    hid, hq, hkv, E = 512, 8, 2, 64
    kv_lens, q_lens = [300, 150, 41], [1, 3, 1]
    Tq = sum(q_lens)
    x, w1, w2 = rnd(Tq, hid).bfloat16(), (1 + 0.1 * rnd(hid)).bfloat16(), (1 + 0.1 * rnd(hid)).bfloat16()
    res = rnd(Tq, hid).bfloat16()
    n1, res = M.rms_norm(x, w1, res)
    wq = rnd(hq * 192 + hkv * 320, hid) / hid ** 0.5
    codes, scale, _ = M.rms_norm_fp8(wq.bfloat16(), torch.ones(hid, device="cuda"))  # any FP8 weight will do
    wq = M.fp8_dequant_blockwise(codes, scale, (1, 128)) / hid ** 0.5
    q, k, v = M.qkv_split(M.linear_proj(n1, wq), hq, hkv)
    total = sum(kv_lens)
    kc, vc = rnd(total + 9, hkv, 192).bfloat16(), rnd(total + 9, hkv, 128).bfloat16()
    idx = torch.randperm(total + 9, generator=g, device="cuda")[:total].to(torch.int32)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    indptr, cu_q = i32(np.cumsum([0] + kv_lens).tolist()), i32(np.cumsum([0] + q_lens).tolist())
    new = torch.cat([idx[e - n:e] for e, n in zip(np.cumsum(kv_lens).tolist(), q_lens)]).long()
    kc[new], vc[new] = k, v
    step = lambda ix, ptr, mx: M.decode(q, kc, vc, ix, ptr, cu_q, None, max(q_lens), mx, M.LAYER_GLOBAL, -1, 1e7)
    out, lse = step(idx, indptr, max(kv_lens))
    acc = None
    for _ in range(2):  # two steps' weights
        acc = M.decode_key_weights(q, kc, idx, indptr, cu_q, lse, max(q_lens), max(kv_lens), M.LAYER_GLOBAL, -1, 1e7, prev=acc, out=acc)
    ref = steps.key_weights(host(q), host(kc), host(idx), host(indptr), host(cu_q), host(lse), -1, 1e7)
    tol = S.weights_tolerance(host(q), host(kc), host(idx), host(indptr), host(cu_q), host(lse), -1, 1e7, None)
    S.close(host(acc), 2 * ref, 2 * tol + 2 * ref * 2.0 ** -23, "accumulated weights")
    total_w = acc.double().sum().item()
    assert abs(total_w - 2 * hq * Tq) < 2e-3 * hq * Tq  # lse is the attention's, off by about 2^-12
    idx2, acc2, indptr2, freed = M.kv_evict(acc, idx, indptr, max(kv_lens), 100, keep_first=2, keep_recent=8)
    ri, rw, rp, rf = steps.kv_evict(host(acc), host(idx), host(indptr), 100, 2, 8)
    n = int(indptr2[-1])
    assert np.array_equal(host(indptr2), rp) and np.array_equal(host(idx2)[:n], ri) and np.array_equal(host(acc2)[:n], rw)
    assert np.array_equal(host(freed)[:total - n], rf)
    out, lse = step(idx2[:n].contiguous(), indptr2, 100)
    wo = (rnd(hid, hq * 128) / (hq * 128) ** 0.5).bfloat16()
    y = M.linear_proj(out, wo)
    codes, scale, res2, n2 = M.rms_norm_fp8(y, w2, res, with_bf16=True)
    h, ref = steps.rms_norm(host(y), S.weight_values(host(w2)), host(res))
    assert np.array_equal(host(res2), h)
    S.close(S.bf16_bits_to_f64(host(n2)), ref, np.abs(ref) * (S.BF16 + 2.0 ** -18), "n2")
    back = M.fp8_dequant_blockwise(codes, scale, (1, 128)).float()
    assert (back - n2.float()).abs().max() <= 2.0 ** -3 * n2.float().abs().max()
    gate = rnd(E, hid) / hid ** 0.5
    logits = n2.float() @ gate.t()
    ids, w = M.moe_route_grouped(logits, None, 4, 8, 4, scale=2.5)
    ri, rw = steps.route_grouped(host(logits), None, 4, 8, 4, scale=2.5)
    assert np.array_equal(host(ids), ri)
    S.close(host(w), rw, rw * 2.0 ** -20, "router weights")
    dw = rnd(Tq, 4)
    dlogits = M.moe_route_bwd(logits, ids, dw, scale=2.5)
    rd = steps.route_bwd(host(logits), ri, host(dw), scale=2.5)
    assert np.abs(host(dlogits) - rd).max() <= 2.0 ** -18 * 2.5 * np.abs(host(dw)).max() * 4
    dx, dweight = M.rms_norm_bwd(res2, w2, (dlogits @ gate).bfloat16(), None)
    rx, rwt = steps.rms_norm_bwd(host(res2), S.weight_values(host(w2)), host((dlogits @ gate).bfloat16()))
    assert np.linalg.norm(S.bf16_bits_to_f64(host(dx)) - rx) <= S.BF16 * np.linalg.norm(rx)
    assert np.linalg.norm(host(dweight) - rwt) <= 2.0 ** -16 * np.linalg.norm(rwt)
    assert M.check() == M.OK


def test_ungrouped_router_agrees(M):
    """One group, sigmoid scores: moe_route's ids and weights; its gradient is the same call's."""
    x = torch.randn(999, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    b = 0.1 * torch.randn(256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    i0, w0 = M.moe_route(x, b, 8)
    i1, w1 = M.moe_route_grouped(x, b, 8)
    assert torch.equal(i0, i1) and (w0 - w1).abs().max() <= 2.0 ** -20


# ---------------------------------------------------------------- streams, graphs, repeats
def calls(M):
    """One call of each entry point on inputs of its own: (name, function of a stream -> tensors, their comparable parts)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, r, w = rnd(700, 1024).bfloat16(), rnd(700, 1024).bfloat16(), rnd(1024)
    logits, bias, many = rnd(900, 256), rnd(256), rnd(33000, 256)
    ids = torch.argsort(rnd(900, 256), -1)[:, :8].to(torch.int32).contiguous()
    dw = rnd(900, 8)
    lens = [700, 300]
    q, kc = rnd(4, 16, 192).bfloat16(), rnd(1010, 2, 192).bfloat16()
    idx = torch.randperm(1010, generator=g, device="cuda")[:1000].to(torch.int32)
    ptr, cu = torch.tensor([0, 700, 1000], dtype=torch.int32, device="cuda"), torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    lse = 5 + rnd(16, 4)
    qc, cuc = rnd(130, 16, 192).bfloat16(), torch.tensor([0, 70, 130], dtype=torch.int32, device="cuda")
    lsec = 5 + rnd(16, 130)
    kw = rnd(1000).abs()
    n = 100 + 100
    return [
        ("rms_norm", lambda s: M.rms_norm(x, w, r, stream=s)),
        ("rms_norm_fp8", lambda s: M.rms_norm_fp8(x, w, r, with_bf16=True, stream=s)),
        ("rms_norm_bwd", lambda s: M.rms_norm_bwd(x, w, r, x, stream=s)),
        ("moe_route_grouped", lambda s: M.moe_route_grouped(logits, bias, 8, 8, 4, stream=s)),
        ("moe_route_many", lambda s: M.moe_route_grouped(many, bias, 8, 8, 4, stream=s)),
        ("moe_route_softmax", lambda s: M.moe_route_grouped(logits, None, 8, score=M.ROUTE_SOFTMAX, stream=s)),
        ("moe_route_bwd", lambda s: (M.moe_route_bwd(logits, ids, dw, stream=s),)),
        ("key_weights", lambda s: (M.decode_key_weights(q, kc, idx, ptr, cu, lse, 3, 700, M.LAYER_GLOBAL, -1, 1e7, stream=s),)),
        ("key_weights_chunk", lambda s: (M.decode_key_weights(qc, kc, idx, ptr, cuc, lsec, 70, 700, M.LAYER_GLOBAL, -1, 1e7, stream=s),)),
        ("kv_evict", lambda s: tuple(t[:m] for t, m in zip(M.kv_evict(kw, idx, ptr, 700, 100, 2, 10, stream=s), (n, n, 3, 1000 - n)))),
    ]


def same(a, b):
    as_int = lambda t: t.view({4: torch.int32, 2: torch.int16, 1: torch.int8}[t.element_size()])
    return all(torch.equal(as_int(p), as_int(q)) for p, q in zip(a, b))


def test_repeats_are_bit_identical(M):
    for name, f in calls(M):
        a = [t.clone() for t in f(None)]
        for _ in range(3):
            assert same(a, f(None)), name
    assert M.check() == M.OK


def test_other_streams_and_overlapping_calls(M):
    """Each entry point on two side streams at once (workspaces and outputs of their own)."""
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for name, f in calls(M):
        ref = [t.clone() for t in f(None)]
        torch.cuda.synchronize()
        got = [[f(s) for s in (s1, s2)] for _ in range(4)]
        torch.cuda.synchronize()
        assert all(same(ref, x) for pair in got for x in pair), name
    assert M.check() == M.OK


def test_captured_and_replayed(M):
    """Two captured graphs of each entry point, replayed in turn on inputs that changed in place."""
    for name, f in calls(M):
        f(None)  # first call outside of a capture: kernel attributes are set there
        torch.cuda.synchronize()
        ref = [t.clone() for t in f(None)]
        graphs = []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                out = f(None)
            graphs.append((gr, out))
        for _ in range(2):
            for gr, out in graphs:
                for t in out:
                    t.zero_()
                gr.replay()
        torch.cuda.synchronize()
        assert all(same(ref, out) for _, out in graphs), name
    assert M.check() == M.OK


def test_replay_follows_its_inputs(M):
    """A captured eviction and routing recompute on new contents of the same buffers."""
    w = torch.rand(500, device="cuda")
    idx = torch.arange(500, dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    logits = torch.randn(64, 128, device="cuda")
    M.kv_evict(w, idx, ptr, 500, 50)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a = M.kv_evict(w, idx, ptr, 500, 50)
        b = M.moe_route_grouped(logits, None, 4)
    for _ in range(2):
        w.copy_(torch.rand(500, device="cuda"))
        logits.copy_(torch.randn(64, 128, device="cuda"))
        gr.replay()
        assert np.array_equal(host(a[0])[:50], steps.kv_evict(host(w), host(idx), host(ptr), 50)[0])
        assert np.array_equal(host(b[0]), steps.route_grouped(host(logits), None, 4)[0])


def test_in_place_forms(M):
    """h may be the residual's memory, dx dy's or dh's, and out prev's (C entry points; out= in Python)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r, w = (torch.randn(50, 2048, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = w[0].contiguous()
    y0, h0 = M.rms_norm(x, w, r)
    st, rr, y = torch.cuda.current_stream().cuda_stream, r.clone(), torch.empty_like(x)
    assert M.LIB.mimo_rms_norm(x.data_ptr(), rr.data_ptr(), w.data_ptr(), 0, 50, 2048, 1e-6, rr.data_ptr(), y.data_ptr(),
                               None, None, st) == M.OK
    assert torch.equal(rr, h0) and torch.equal(y, y0)
    dx0, dw0 = M.rms_norm_bwd(h0, w, x, r)
    for which in (0, 1):
        dy, dh, dw = x.clone(), r.clone(), torch.empty_like(dw0)
        n = M.LIB.mimo_rms_norm_bwd_workspace_size(50, 2048)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dx = (dy, dh)[which]
        assert M.LIB.mimo_rms_norm_bwd(h0.data_ptr(), w.data_ptr(), 0, dy.data_ptr(), dh.data_ptr(), 50, 2048, 1e-6,
                                       dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), n, st) == M.OK
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_empty_calls(M):
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")
    y, h = M.rms_norm(e(0, 64, dtype=torch.bfloat16), e(64))
    assert y.shape == (0, 64)
    dx, dw = M.rms_norm_bwd(e(0, 64, dtype=torch.bfloat16), e(64), e(0, 64, dtype=torch.bfloat16))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device="cuda"))
    ids, w = M.moe_route_grouped(e(0, 64))
    assert ids.shape == (0, 8)
    assert M.moe_route_bwd(e(0, 64), e(0, 8, dtype=torch.int32), e(0, 8)).shape == (0, 64)
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    idx, w, ptr, freed = M.kv_evict(e(0), e(0, dtype=torch.int32), z, 0, 5)
    assert torch.equal(ptr, z)
    # a budget beyond any length keeps everything
    a, b = torch.rand(6, device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda")
    idx, w, ptr, freed = M.kv_evict(a, b, torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda"), 4, 10 ** 12)
    assert torch.equal(idx, b) and torch.equal(w, a) and ptr.tolist() == [0, 2, 6]
    for counts in ((-10 ** 12,), (2, 2 ** 32 + 1), (2, 0, 2 ** 32), (2, -2 ** 32)):  # refused, not wrapped
        with pytest.raises(M.MimoAttnError):
            M.kv_evict(a, b, torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda"), 4, *counts)
    # no new queries: what was accumulated so far
    i = torch.arange(10, dtype=torch.int32, device="cuda")
    ptr = torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")
    p = torch.rand(10, device="cuda")
    got = M.decode_key_weights(e(0, 8, 192, dtype=torch.bfloat16), torch.zeros(10, 2, 192, dtype=torch.bfloat16, device="cuda"), i, ptr, z,
                               e(8, 0), 0, 6, M.LAYER_GLOBAL, -1, 1e7, prev=p)
    assert torch.equal(got, p) and M.check() == M.OK


def test_norm_gradient_against_differences(M):
    """dx and dweight against central differences of the FP64 definition."""
    T, H = 3, 64
    rng = np.random.default_rng(11)
    h, dy = S.bits(rng.standard_normal((T, H))), S.bits(rng.standard_normal((T, H)))
    w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    dx, dw = M.rms_norm_bwd(dev(h), dev(w), dev(dy))
    hf, g = S.bf16_bits_to_f64(h), S.bf16_bits_to_f64(dy)
    f = lambda a, b: ((a / np.sqrt((a * a).mean(-1, keepdims=True) + 1e-6) * b) * g).sum()
    step = 2.0 ** -20
    for t, j in ((0, 0), (1, 17), (2, 63)):
        d = np.zeros((T, H))
        d[t, j] = step
        num = (f(hf + d, w) - f(hf - d, w)) / (2 * step)
        assert abs(S.bf16_bits_to_f64(host(dx))[t, j] - num) <= abs(num) * S.BF16 + 2.0 ** -14
        e = np.zeros(H)
        e[j] = step
        num = (f(hf, w + e) - f(hf, w - e)) / (2 * step)
        assert abs(host(dw)[j] - num) <= abs(num) * 2.0 ** -16 + 2.0 ** -16


@pytest.mark.parametrize("softmax,normalize", [(False, True), (False, False), (True, True), (True, False)])
def test_route_gradient_against_differences(M, softmax, normalize):
    x = S.route_logits(2, 32, 21)
    ids, _ = steps.route_grouped(x, None, 5, softmax=softmax, normalize=normalize)
    g = np.random.default_rng(22).standard_normal((2, 5)).astype(np.float32)
    d = host(M.moe_route_bwd(dev(x), dev(ids), dev(g), int(softmax), normalize, 2.5))

    def f(z):
        s = np.take_along_axis(steps.scores(z, softmax), ids.astype(np.int64), 1)
        return (2.5 * (s / s.sum(-1, keepdims=True) if normalize else s) * g).sum()

    for t, e in [(0, int(ids[0, 0])), (1, int(ids[1, 4])), (0, int(np.setdiff1d(np.arange(32), ids[0])[0]))]:
        h = np.zeros(x.shape)
        h[t, e] = 2.0 ** -18
        num = (f(x + h) - f(x.astype(np.float64) - h)) / 2.0 ** -17
        assert abs(d[t, e] - num) <= 2.0 ** -16 * max(1.0, abs(num))
