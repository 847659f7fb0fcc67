"""tests/step_edges.py through the host build of the whole library.  Run as a child process:

    python edge_cases.py <libmimo_attn_host.so> <case> [<case> ...]
"""
import sys

from step_cases import Host
import step_edges  # noqa: E402  (step_cases put tests/ on the path)

if __name__ == "__main__":
    be = Host(sys.argv[1])
    for name in sys.argv[2:]:
        step_edges.CASES[name](be)
        print("ok", name, flush=True)
