"""The Python binding: what it needs, and arguments that it refuses itself (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from global_attention_moe_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import ctypes, sys

class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("torch is not here")

sys.meta_path.insert(0, NoTorch())
from global_attention_moe_b200 import mimo_attn as M
assert "torch" not in sys.modules
assert M.version() >= (1, 6) and M.status_string(M.OK) == "ok"
M.set_kernel(M.KERNEL_AUTO), M.set_decode_kernel(M.DECODE_AUTO), M.set_bwd_kernel(M.BWD_AUTO)
assert M.noalloc_scratch_bytes() > 0
d = M.make_dims(1, 128, 128, 8, 2)
assert M.host_workspace_size(d, True) > 0
assert M.fwd_raw(None, None, None, None, None, d, M.LAYER_GLOBAL, -1, 1e7, 64, 1.0, None, None, None) == M.ERR_INVALID_ARG
e = M.make_decode_dims(1, 1, 10, 10, 1, 10, 8, 2)
assert M.decode_raw(None, None, None, None, None, None, None, e, M.LAYER_GLOBAL, -1, 1e7, 64, 1.0, None, None, None) == M.ERR_INVALID_ARG
assert M.LIB.mimo_decode_key_weights_workspace_size(ctypes.byref(e)) > 0
assert M.LIB.mimo_rms_norm(None, None, None, 0, 1, 64, 1e-6, None, None, None, None, None) == M.ERR_INVALID_ARG
try:
    M.check()
except ImportError:
    print("fine")
"""


def run(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)


def test_raw_entry_points_do_not_need_torch():
    build.build()
    r = run(WITHOUT_TORCH)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_torch_is_bound_at_its_first_use():
    """Imported before torch, and after it."""
    build.build()
    for first in ("from global_attention_moe_b200 import mimo_attn as M; import torch",
                  "import torch; from global_attention_moe_b200 import mimo_attn as M"):
        r = run(first + "\n"
                "x = torch.zeros(2, 8)\n"
                "try:\n"
                "    M.fwd(x[:, None], x[:, None], x[:, None], None, x, 2, 1, -1, 1e7)\n"
                "except ValueError as e:\n"
                "    print('refused')\n"
                "assert M.torch is torch or not isinstance(M.torch, type(torch))\n"
                "M.torch.float32\n"
                "assert M.torch is torch and M._BF16 is torch.bfloat16 and M._I32 is torch.int32\n")
        assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]


BIG = 2 ** 32


@pytest.mark.parametrize("call", [
    dict(top_k=BIG + 8), dict(num_groups=BIG + 1), dict(top_groups=BIG + 1), dict(score=BIG), dict(score=BIG + 1),
    dict(num_groups=-BIG + 8), dict(top_k=2 ** 31)])
def test_router_counts_do_not_wrap(call):
    import torch
    build.build()
    from global_attention_moe_b200 import mimo_attn as M
    with pytest.raises(ValueError, match="32 bits"):
        M.moe_route_grouped(torch.zeros(2, 64), None, **call)
    if "score" in call:
        with pytest.raises(ValueError, match="32 bits"):
            M.moe_route_bwd(torch.zeros(2, 64), torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 8), **call)


@pytest.mark.parametrize("call", [
    dict(max_q_len=BIG + 1), dict(max_kv_len=BIG + 4), dict(layer_kind=BIG), dict(window=BIG + 128), dict(window=-BIG + 128),
    dict(rope_dims=BIG + 64)])
def test_key_weight_counts_do_not_wrap(call):
    import torch
    build.build()
    from global_attention_moe_b200 import mimo_attn as M
    i = torch.zeros(4, dtype=torch.int32)
    a = dict(max_q_len=1, max_kv_len=4, layer_kind=0, window=128, rope_base=1e4)
    with pytest.raises(ValueError, match="32 bits"):
        M.decode_key_weights(torch.zeros(1, 8, 192).bfloat16(), torch.zeros(4, 2, 192).bfloat16(), i, i[:2], i[:2], torch.zeros(8, 1),
                             **{**a, **call})
    if "max_kv_len" in call:
        with pytest.raises(ValueError, match="32 bits"):
            M.kv_evict(torch.zeros(4), i, i[:2], call["max_kv_len"], 2)
