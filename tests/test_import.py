"""The package imports, and its host-side calls work, with a torch that was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
import kv_cache_pruning_gb300 as k
assert k.version() > 0
assert k.kvp_compact_block8_workspace_bytes(2, 3, 100, 8) > 0
assert k.kvp_decode_attn_workspace_bytes(1, 8, 2, 64) > 0
assert k.kvp_rope_turns([1.0, 0.5], device="cpu").numel() == 2
for call in (lambda: k.Block8PagedKV.allocate(1, 1, 64, 2, 2, device="cpu"),
             lambda: k.kvp_qk_norm_rope(torch.zeros(2, 3, 64, dtype=torch.bfloat16), None, None, None)):
    try:
        call()
    except ValueError:
        pass
    else:
        raise AssertionError("not refused")
print("fine")
"""


def test_import_with_a_torch_without_cuda():
    import __graft_entry__
    __graft_entry__._builder().build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
