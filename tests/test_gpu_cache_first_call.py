"""A process whose first call of the library is one that a graph captures."""
import os
import subprocess
import sys

import pytest

from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu

_FIRST = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import quantized_attention_diffusion_gb300 as qad
what, rows, room, prefix = sys.argv[2], int(sys.argv[3]), int(sys.argv[4]), int(sys.argv[5])
g = torch.Generator().manual_seed(1)
B, H = 2, 2
cache = (torch.randint(-99, 99, (40, H, 64, 128), dtype=torch.int8, generator=g).cuda(), torch.full((40, H, 64), 0.01, device="cuda"),
         torch.randint(0, 100, (40, H, 64, 128), dtype=torch.uint8, generator=g).cuda(), torch.full((40, H, 64), 0.01, device="cuda"))
q = torch.randn((B, rows, H, 128), generator=g).to(torch.bfloat16).cuda()
table = torch.nn.functional.pad(torch.arange(6, dtype=torch.int32).view(B, 3), (0, room // 64 - 3), value=-1).cuda()
pre = torch.arange(30, 40, dtype=torch.int32).cuda()
lens, zero = (torch.full((B,), n, dtype=torch.int32, device="cuda") for n in (150, 0))


def call():
    if what == "write":
        return qad.kv_cache_write(q, q, cache, table, zero)
    if what == "read":
        return qad.kv_cache_read(cache, table, lens, 150)
    if what == "whole":
        return (qad.attn_fwd(q, q, q),)
    if prefix:
        return (qad.attn_fwd_cache_prefix(q, cache, pre, prefix, table, lens),)
    return (qad.attn_fwd_cache(q, cache, table, lens),)


def bits(out):
    torch.cuda.synchronize()
    return [t.cpu().contiguous().view(torch.uint8) for t in out]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
replayed = bits(out)
assert all(torch.equal(a, b) for a, b in zip(replayed, bits(call())))
assert qad.sync_status() == 0
print("same")
"""


@pytest.mark.parametrize("what,rows,room,prefix", [
    ("write", 3, 512, 0), ("read", 1, 512, 0), ("attend", 1, 512, 0), ("attend", 1, 20032, 0), ("attend", 10, 20032, 0),
    ("attend", 40, 20032, 0), ("attend", 1, 512, 600), ("attend", 1, 20032, 600), ("attend", 40, 20032, 600), ("whole", 256, 512, 0),
])
def test_captured_before_any_other_call(what, rows, room, prefix):
    ensure_library()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", _FIRST, root, what, str(rows), str(room), str(prefix)], capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, CUDA_MODULE_LOADING="LAZY"))
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stderr[-2000:]
