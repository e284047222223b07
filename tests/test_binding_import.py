"""The binding imports, and its host checks run, on a torch build without the
CUDA parts of its C module."""
import subprocess
import sys

from block_sparse_attention_lvsa_b200 import build

CODE = """
import torch
for name in dir(torch._C):
    if name.startswith(("_cuda_", "_CudaStream", "_CudaEvent")):
        try:
            delattr(torch._C, name)
        except (AttributeError, TypeError):
            pass
assert not hasattr(torch._C, "_cuda_getCurrentRawStream")
from block_sparse_attention_lvsa_b200 import binding
assert binding.version()
assert binding.status_string(binding.BSA_ERR_ARG)
ix = binding.bsa_index()
ix.kind = binding.BSA_INDEX_LVSA_FRAMES
ix.T = 8
assert binding.workspace_bytes(binding.BSA_OP_BLOCKSPARSE_FWD, 512, 2, 64, ix) > 0
x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
for call in (lambda: binding.qk_norm_rope_fwd(x, x), lambda: binding.blocksparse_attn_fwd(x, x, x, ix)):
    try:
        call()
    except ValueError:
        continue
    raise AssertionError("a CPU tensor was taken")
"""


def test_import_without_cuda_names():
    build.build()
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
