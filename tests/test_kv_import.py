"""The package with a torch that was built without CUDA (no torch._C._cuda_*)."""
import subprocess
import sys

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import long_context_compressed_kv_b200 as v
d = v.kv_desc(8, 2, 128)
pool = torch.zeros(4, 2, 128, 128, dtype=torch.bfloat16)
x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
try:
    v.kv_append(d, k=x, v=x, k_cache=pool, v_cache=pool, q_start=torch.zeros(2, dtype=torch.int32),
                kv_len=torch.zeros(1, dtype=torch.int64),
                block_table=torch.zeros(1, 4, dtype=torch.int32),
                ws=torch.zeros(256, dtype=torch.uint8))
except ValueError as e:
    print("refused:", e)
"""


def test_import_without_cuda_functions():
    p = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    assert "refused:" in p.stdout and "one GPU" in p.stdout
