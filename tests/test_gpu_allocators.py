"""Tensors of torch's expandable segments: one address range, mapped in pieces
of 20 MB, across which a tensor may lie.  In a process of its own, since the
allocator is chosen at its start."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
import rwkv_wkv_mixing_b200 as m

gen = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(24000, 1024, generator=gen, device="cuda")         # 98 MB
y = m.group_norm(x, 16, act="silu")
for i in range(0, 24000, 4000):     # a piece at a time
    assert torch.equal(y[i:i + 4000], m.group_norm(x[i:i + 4000].clone(), 16, act="silu"))
B, T, H, D = 2, 8192, 16, 64
q = torch.nn.functional.normalize(torch.randn(B, T, H, D, generator=gen, device="cuda"), dim=-1).bfloat16()
g, beta = -torch.rand(B, T, H, device="cuda"), torch.rand(B, T, H, device="cuda")
o = m.gated_delta(q, q, q, g, beta)
grads = m.gated_delta_backward(q, q, q, g, beta, q)
for b in range(B):
    one = [t[b:b + 1].clone() for t in (q, q, q, g, beta)]
    assert torch.equal(o[b:b + 1], m.gated_delta(*one))
    for whole, part in zip(grads[:5], m.gated_delta_backward(*one, q[b:b + 1].clone())[:5]):
        assert torch.equal(whole[b:b + 1], part)
# what is not mapped is still refused
st = m.lib.group_norm(1 << 30, 1024, 16, x.data_ptr(), None, None, None, 0, 1e-5, y.data_ptr(),
                      torch.cuda.current_stream().cuda_stream)
assert st == m.WKV_ERR_INVALID_ARG and "its allocation ends" in m.wkv_last_error(), (st, m.wkv_last_error())
torch.cuda.synchronize()
print("ok")
"""


@pytest.mark.parametrize("conf", ["expandable_segments:True", "backend:cudaMallocAsync", ""])
def test_large_tensors(cuda_dev, conf):
    env = dict(os.environ, PYTORCH_CUDA_ALLOC_CONF=conf, PYTHONPATH=ROOT)
    p = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("ok"), p.stdout + p.stderr
