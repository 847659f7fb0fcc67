"""The Python binding: what it needs, and arguments that it refuses itself (no GPU needed)."""
import os
import subprocess
import sys

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
