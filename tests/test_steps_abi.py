"""Refusals of the layer's steps: bad arguments are rejected before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from global_attention_moe_b200 import build

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
MANY = 1 << 40


@pytest.fixture(scope="module")
def M():
    build.build()
    from global_attention_moe_b200 import mimo_attn
    return mimo_attn


@pytest.mark.parametrize("args,expect", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=-8), 1), (dict(eps=-1e-6), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1),
    (dict(H=12), 2), (dict(H=16392), 2), (dict(H=24, codes=FAKE, scale=FAKE), 2), (dict(T=1 << 31), 2),
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(codes=FAKE), 1), (dict(x=FAKE + 8), 1),
    (dict(r=FAKE + 4), 1), (dict(w=FAKE + 2), 1), (dict(h=FAKE + 8), 1), (dict(y=FAKE + 8), 1),
    (dict(codes=FAKE + 1, scale=FAKE), 1), (dict(codes=FAKE, scale=FAKE + 2), 1),
    (dict(T=0, x=None, w=None, y=None), 0),
])
def test_rms_norm(M, args, expect):
    a = dict(x=FAKE, r=None, w=FAKE, T=4, H=64, eps=1e-6, h=None, y=FAKE, codes=None, scale=None)
    a.update(args)
    assert M.LIB.mimo_rms_norm(a["x"], a["r"], a["w"], 0, a["T"], a["H"], a["eps"], a["h"], a["y"], a["codes"],
                               a["scale"], None) == expect


@pytest.mark.parametrize("args,expect", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(eps=-1.0), 1), (dict(H=4), 2), (dict(H=20000), 2), (dict(h=None), 1),
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(ws=None), 1), (dict(ws_bytes=255), 1),
    (dict(dh=FAKE + 8), 1), (dict(dx=FAKE + 2), 1), (dict(dw=FAKE + 4), 1), (dict(ws=FAKE + 8), 1),
])
def test_rms_norm_bwd(M, args, expect):
    a = dict(h=FAKE, w=FAKE, dy=FAKE, dh=None, T=4, H=64, eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE, ws_bytes=MANY)
    a.update(args)
    assert M.LIB.mimo_rms_norm_bwd(a["h"], a["w"], 0, a["dy"], a["dh"], a["T"], a["H"], a["eps"], a["dx"], a["dw"],
                                   a["ws"], a["ws_bytes"], None) == expect
    assert M.LIB.mimo_rms_norm_bwd_workspace_size(-1, 64) == 0 == M.LIB.mimo_rms_norm_bwd_workspace_size(4, 20)
    assert M.LIB.mimo_rms_norm_bwd_workspace_size(1 << 40, 64) == M.LIB.mimo_rms_norm_bwd_workspace_size(1 << 20, 64) > 0


@pytest.mark.parametrize("args,expect", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(top=0), 1), (dict(top=9), 1),
    (dict(groups=3), 1), (dict(k=33, E=64, groups=1, top=1), 2), (dict(k=9, E=64, groups=8, top=1), 1),
    (dict(E=520, groups=1, top=1), 2), (dict(E=66, groups=33, top=4, k=4), 2), (dict(score=2), 1), (dict(score=-1), 1),
    (dict(scale=float("inf")), 1), (dict(x=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(x=FAKE + 4), 1),
    (dict(bias=FAKE + 4), 1), (dict(ids=FAKE + 2), 1), (dict(w=FAKE + 1), 1), (dict(k=2 ** 31 - 1), 1),
    (dict(T=0, x=None, ids=None, w=None), 0),
])
def test_route(M, args, expect):
    a = dict(x=FAKE, bias=None, T=4, E=64, k=8, groups=8, top=4, score=0, norm=1, scale=1.0, ids=FAKE, w=FAKE)
    a.update(args)
    assert M.LIB.mimo_moe_route_grouped(a["x"], a["bias"], a["T"], a["E"], a["k"], a["groups"], a["top"], a["score"],
                                        a["norm"], a["scale"], a["ids"], a["w"], None) == expect


@pytest.mark.parametrize("args,expect", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=33), 2), (dict(E=513), 2), (dict(score=7), 1),
    (dict(scale=float("nan")), 1), (dict(x=None), 1), (dict(ids=None), 1), (dict(g=None), 1), (dict(d=None), 1),
    (dict(x=FAKE + 8), 1), (dict(d=FAKE + 8), 1), (dict(ids=FAKE + 1), 1), (dict(g=FAKE + 2), 1),
    (dict(T=0, x=None, ids=None, g=None, d=None), 0),
])
def test_route_bwd(M, args, expect):
    a = dict(x=FAKE, ids=FAKE, g=FAKE, T=4, E=64, k=8, score=0, norm=1, scale=1.0, d=FAKE)
    a.update(args)
    assert M.LIB.mimo_moe_route_bwd(a["x"], a["ids"], a["g"], a["T"], a["E"], a["k"], a["score"], a["norm"], a["scale"],
                                    a["d"], None) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(hq=6, hkv=4), 1), (dict(max_q_len=20, max_kv_len=10), 1), (dict(cache_rows=0), 1), (dict(dqk=128), 2),
    (dict(rope_dims=32), 2), (dict(rope_dims=63), 1), (dict(window=-1), 1), (dict(layer=2), 1), (dict(base=0.0), 1),
    (dict(base=float("inf")), 1), (dict(q=FAKE + 8), 1), (dict(q=None), 1), (dict(lse=None), 1), (dict(lse=FAKE + 4), 1),
    (dict(out=None), 1), (dict(out=FAKE + 2), 1), (dict(prev=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1),
    (dict(ws_bytes=100), 1), (dict(idx=None), 1), (dict(ptr=None), 1), (dict(cu=None), 1), (dict(kc=None), 1),
    (dict(max_q_len=70000, total_q=70000, max_kv_len=70000, total_kv=70000, cache_rows=70000, hq=64, hkv=4), 2),
    (dict(total_kv=2 ** 31 - 1), 2), (dict(total_kv=0x7FFFF001), 2),
    (dict(total_kv=0, max_kv_len=0, max_q_len=0, total_q=0, q=None, lse=None, kc=None, idx=None, out=None, ws=None), 0),
])
def test_key_weights(M, case, expect):
    d = dict(num_seqs=2, total_q=4, total_kv=100, cache_rows=128, max_q_len=2, max_kv_len=60, hq=8, hkv=2, dqk=192, dv=128)
    a = dict(layer=0, window=128, base=1e4, rope_dims=64, q=FAKE, kc=FAKE, idx=FAKE, ptr=FAKE, cu=FAKE, lse=FAKE, prev=None,
             out=FAKE, ws=FAKE, ws_bytes=MANY)
    for key in case:
        (d if key in d else a)[key] = case[key]
    dims = M.make_decode_dims(*(d[k] for k in ("num_seqs", "total_q", "total_kv", "cache_rows", "max_q_len", "max_kv_len",
                                               "hq", "hkv", "dqk", "dv")))
    st = M.LIB.mimo_decode_key_weights(a["q"], a["kc"], a["idx"], a["ptr"], a["cu"], a["lse"], a["prev"],
                                       ctypes.byref(dims), a["layer"], a["window"], a["base"], a["rope_dims"], a["out"],
                                       a["ws"], a["ws_bytes"], None)
    assert st == expect
    assert M.LIB.mimo_decode_key_weights_workspace_size(None) == 0


@pytest.mark.parametrize("args,expect", [
    (dict(B=0), 1), (dict(total=-1), 1), (dict(most=-1), 1), (dict(most=21), 1), (dict(first=-1), 1), (dict(recent=-1), 1),
    (dict(budget=-1), 1), (dict(budget=3, first=2, recent=2), 1), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
    (dict(w=None), 1), (dict(idx=None), 1), (dict(ptr=None), 1), (dict(ni=None), 1), (dict(nw=None), 1), (dict(np_=None), 1),
    (dict(freed=None), 1), (dict(w=FAKE + 2), 1), (dict(freed=FAKE + 1), 1),
    (dict(total=2 ** 31 - 1), 2), (dict(total=0x7FFFF001), 2), (dict(B=65537), 2),
])
def test_evict(M, args, expect):
    a = dict(w=FAKE, idx=FAKE, ptr=FAKE, B=2, total=20, most=10, budget=5, first=1, recent=1, ni=FAKE, nw=FAKE, np_=FAKE,
             freed=FAKE)
    a.update(args)
    assert M.LIB.mimo_kv_evict(a["w"], a["idx"], a["ptr"], a["B"], a["total"], a["most"], a["budget"], a["first"],
                               a["recent"], a["ni"], a["nw"], a["np_"], a["freed"], None) == expect


def test_version(M):
    assert M.version() >= (1, 6)
