"""The layer's steps (RMS norm, grouped routing, key weights, eviction) on the CPU: the library's kernels
through the host build, checked against their FP64 definitions, and those definitions against formulas and
routines of other making."""
import os
import subprocess
import sys

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
EMU = os.path.join(HERE, "host_emulation")
sys.path.insert(0, EMU)
import build_library  # noqa: E402
import step_checks  # noqa: E402
from oracle import steps  # noqa: E402


@pytest.fixture(scope="module")
def host_library(tmp_path_factory):
    # a vector load or store off its alignment, which the GPU faults on, ends the case
    return build_library.build(str(tmp_path_factory.mktemp("steps_host")),
                               flags=("-fsanitize=alignment", "-fno-sanitize-recover=alignment"))


def test_alignment_is_checked(tmp_path):
    """Planted: the lse slots of the key-weights kernel 8 bytes off (float4 reads need 16)."""
    lib = build_library.build(str(tmp_path), flags=("-fsanitize=alignment", "-fno-sanitize-recover=alignment"), mutations=[
        ("key_weights.cuh", "alignas(16) float k_cos", "float k_cos"), ("key_weights.cuh", "alignas(16) float lse2", "float lse2")])
    rc, log = run(lib, ["weights_step"])
    assert rc != 0 and "alignment" in log, log


def run(lib, names, sms=None):
    env = dict(os.environ, HEMU_SMS=str(sms)) if sms else None
    r = subprocess.run([sys.executable, os.path.join(EMU, "step_cases.py"), lib, *names], capture_output=True, text=True,
                       timeout=900, env=env)
    return r.returncode, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("name", sorted(step_checks.CASES))
def test_kernels_match_their_definitions(host_library, name):
    rc, log = run(host_library, [name])
    assert rc == 0, log


def test_with_few_sms(host_library):
    """On 1 and 3 SMs every CTA of the persistent kernels walks many rows, tokens and key tiles in turn, and the
    router takes its kernel of four threads per token."""
    for sms in (1, 3):
        rc, log = run(host_library, ["norm_bwd", "route", "route_many", "route_values", "route_far", "route_bwd", "weights_step",
                              "weights_window", "weights_chunk"], sms)
        assert rc == 0, log


# ---------------------------------------------------------------- the definitions
def test_norm_definition_against_torch():
    import torch
    rng = np.random.default_rng(0)
    h, w = rng.standard_normal((5, 48)), rng.standard_normal(48)
    hb = step_checks.bits(h)
    hf = torch.tensor(step_checks.bf16_bits_to_f64(hb), requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    y = torch.nn.functional.rms_norm(hf, (48,), wt, 1e-6)
    _, ref = steps.rms_norm(hb, w)
    assert np.abs(y.detach().numpy() - ref).max() < 1e-12
    dyb = step_checks.bits(rng.standard_normal((5, 48)))
    y.backward(torch.tensor(step_checks.bf16_bits_to_f64(dyb)))
    dx, dw = steps.rms_norm_bwd(hb, w, dyb)
    assert np.abs(hf.grad.numpy() - dx).max() < 1e-12 and np.abs(wt.grad.numpy() - dw).max() < 1e-12


def test_bf16_rounding_against_torch():
    import torch
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000), [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, 0.0, -0.0]])
    mid = np.isin(x, [1 + 2.0 ** -8 + 2.0 ** -40])
    got = steps.f64_to_bf16_bits(x)
    ref = torch.tensor(x).float().bfloat16().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got[~mid], ref[~mid]) and got[mid][0] == 0x3F81  # just above a midpoint: up, from the exact value


@pytest.mark.parametrize("softmax,normalize", [(False, True), (False, False), (True, True), (True, False)])
def test_route_definition_against_torch(softmax, normalize):
    import torch
    x = step_checks.route_logits(6, 40, 3)
    ids, w = steps.route_grouped(x, None, 5, 1, 1, softmax, normalize, 2.0)
    t = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    s = torch.softmax(t, -1) if softmax else torch.sigmoid(t)
    v, i = s.topk(5)
    assert np.array_equal(i.numpy(), ids)
    wt = 2.0 * (v / v.sum(-1, keepdim=True) if normalize else v)
    assert np.abs(wt.detach().numpy() - w).max() < 1e-12
    g = np.random.default_rng(4).standard_normal((6, 5))
    wt.backward(torch.tensor(g))
    assert np.abs(t.grad.numpy() - steps.route_bwd(x, ids, g, softmax, normalize, 2.0)).max() < 1e-12


def test_group_limit_definition():
    """Two groups of four: the pair of second-best keys outweighs the group of the single best one."""
    s = np.array([[0.9, 0.1, 0.1, 0.1, 0.6, 0.55, 0.5, 0.1]])
    x = np.log(s / (1 - s)).astype(np.float32)
    ids, w = steps.route_grouped(x, None, 3, 2, 1, normalize=False)
    assert ids.tolist() == [[4, 5, 6]] and np.allclose(w, [[0.6, 0.55, 0.5]])
    ids, _ = steps.route_grouped(x, None, 3, 2, 2)
    assert ids.tolist() == [[0, 4, 5]]
    ids, _ = steps.route_grouped(np.zeros((1, 8), np.float32), None, 3, 4, 2)  # all equal: lower group, lower expert
    assert ids.tolist() == [[0, 1, 2]]


def test_key_weights_definition_against_the_attention_oracle():
    """The normaliser of the same scores is the attention oracle's lse, and weights with V one-hot per key are the
    attention's outputs."""
    import oracle
    from decode_helpers import decode_reference
    from global_attention_moe_b200 import workloads as W
    oracle.build()
    for window, base, sink in ((128, 1e4, True), (-1, 1e7, False)):
        x = W.make_decode_inputs([150, 40], [3, 1], 4, 2, sink, 5)
        _, lse = decode_reference(x, window, base)
        mine = steps.normaliser(x.q, x.k_cache, x.kv_indices, x.kv_indptr, x.cu_q, window, base, x.sink)
        assert np.abs(lse - mine).max() < 1e-9
        w = steps.key_weights(x.q, x.k_cache, x.kv_indices, x.kv_indptr, x.cu_q, mine, window, base)
        if not sink:
            assert abs(w.sum() - 4 * 4) < 1e-9


def test_evict_definition():
    w = np.array([5, 1, np.nan, 1, 0.5, 9, -np.inf, 2], dtype=np.float32)
    idx = np.arange(10, 18, dtype=np.int32)
    kept, kw, ptr, freed = steps.kv_evict(w, idx, np.array([0, 8], np.int32), 5, 1, 1)
    assert kept.tolist() == [10, 11, 13, 15, 17] and freed.tolist() == [12, 14, 16] and ptr.tolist() == [0, 5]
    kept, _, _, _ = steps.kv_evict(w, idx, np.array([0, 8], np.int32), 4, 1, 1)
    assert kept.tolist() == [10, 11, 15, 17]  # of the two equal weights the earlier stays
