"""The layer's steps at values and sizes where they are easily wrong, on the CPU (tests/step_edges.py)."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
EMU = os.path.join(HERE, "host_emulation")
sys.path.insert(0, EMU)
import build_library  # noqa: E402
import step_edges  # noqa: E402


@pytest.fixture(scope="module")
def libraries(tmp_path_factory):
    """The host build, and one whose bounded waits have a limit of zero, compiled side by side."""
    checked = ("-fsanitize=alignment", "-fno-sanitize-recover=alignment")
    no_wait = ("mimo_attn_api.cu", "constexpr uint64_t kDefaultWaitLimitNs = 2000000000ull;",
               "constexpr uint64_t kDefaultWaitLimitNs = 0ull;")
    with ThreadPoolExecutor(2) as pool:
        jobs = [pool.submit(build_library.build, str(tmp_path_factory.mktemp("edges_host")), flags=checked),
                pool.submit(build_library.build, str(tmp_path_factory.mktemp("edges_no_wait")), mutations=[no_wait])]
        return [j.result() for j in jobs]


@pytest.fixture(scope="module")
def host_library(libraries):
    return libraries[0]


def run(lib, names, sms=None):
    env = dict(os.environ, HEMU_SMS=str(sms)) if sms else None
    r = subprocess.run([sys.executable, os.path.join(EMU, "edge_cases.py"), lib, *names], capture_output=True, text=True,
                       timeout=900, env=env)
    return r.returncode, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("name", sorted(step_edges.CASES))
def test_edges(host_library, name):
    rc, log = run(host_library, [name])
    assert rc == 0, log


def test_edges_on_one_sm(host_library):
    """On one SM the router takes its kernel of four threads per token from 192 tokens on, and CTAs walk several rows
    and tiles."""
    rc, log = run(host_library, ["gradient_places", "route_low", "route_scales", "weights_sizes"], 1)
    assert rc == 0, log


def test_e4m3_codes_against_torch():
    """The tests' own rounding to E4M3."""
    import torch
    rng = np.random.default_rng(3)
    grid = step_edges.e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))
    q = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.1, 0.1, 1000), grid, -(grid[1:] + grid[:-1]) / 2]).astype(np.float32)
    assert np.array_equal(step_edges.e4m3_codes(q), torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("softmax,normalize", step_edges.FORMS)
def test_gradient_terms_against_the_definition(softmax, normalize):
    """The gradient from differences is the chain rule's (oracle/steps.py), where that loses nothing in FP64, and
    that of torch's autograd."""
    import torch
    from oracle import steps
    for gap in (0, 4, 8):
        x, ids, g = step_edges.peaked(6, 40, 5, gap, gap)
        if gap == 4:
            ids[0, :2], ids[1, 3] = ids[0, 0], -1
        ref = steps.route_bwd(x, ids, g, softmax, normalize, 2.5)
        got = np.stack([step_edges.route_bwd_terms(x[t], ids[t], g[t], softmax, normalize, 2.5)[0] for t in range(6)])
        assert np.abs(got - ref).max() < 1e-10
        if gap != 4:
            t = torch.tensor(x, dtype=torch.float64, requires_grad=True)
            s = (torch.softmax(t, -1) if softmax else torch.sigmoid(t)).gather(1, torch.tensor(ids.astype(np.int64)))
            (2.5 * (s / s.sum(-1, keepdim=True) if normalize else s) * torch.tensor(g, dtype=torch.float64)).sum().backward()
            assert np.abs(got - t.grad.numpy()).max() < 1e-10


GAVE_UP = """
import sys
import numpy as np
from step_cases import Host
import step_checks as S
be = Host(sys.argv[1])
for q_lens in ([1, 3], [90, 40]):  # one query tile to a sequence, and several
    q, k, idx, indptr, cu_q = S.step_batch([300, 150], q_lens, 8, 2, 1)
    lse = np.ones((8, sum(q_lens)), dtype=np.float32)
    prev = np.arange(450, dtype=np.float32)
    if sys.argv[2] == "before":
        be.L.hemu_set_timeout()
    out = be.key_weights(q, k, idx, indptr, cu_q, lse, max(q_lens), 300, -1, 1e7, prev, errors=True, fill=-7.0)
    assert be.status == 4, be.status  # MIMO_ERR_TIMEOUT
    assert np.all(out == -7), out
    if sys.argv[2] == "before":  # the next call works again
        a = be.key_weights(q, k, idx, indptr, cu_q, lse, max(q_lens), 300, -1, 1e7, prev)
        S.close(a, S.steps.key_weights(q, k, idx, indptr, cu_q, lse, -1, 1e7, prev),
                S.weights_tolerance(q, k, idx, indptr, cu_q, lse, -1, 1e7, prev), "after")
"""


def gave_up(lib, *args):
    r = subprocess.run([sys.executable, "-c", GAVE_UP, lib, *args], capture_output=True, text=True, timeout=600, cwd=EMU)
    assert r.returncode == 0, (r.stdout + r.stderr)[-2000:]


def test_key_weights_after_a_timeout_leave_out_alone(host_library):
    """The status of a wait that ran out earlier is set: the product kernel does not run, and the sums that it did
    not write do not reach out."""
    gave_up(host_library, "before")


def test_key_weights_whose_wait_runs_out_leave_out_alone(libraries):
    """A wait inside the call runs out."""
    gave_up(libraries[1], "inside")
