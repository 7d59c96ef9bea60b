"""A captured graph holds the first calls that a process makes: nothing is set up by an earlier one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import sparse_graph_causal_b200 as sa
B, H, Hkv, D, page, M = 5, 4, 2, 64, 16, 400
dtype, W = {dtype}, {W}
put = lambda x, t: torch.tensor(x, dtype=t, device="cuda")
quant = dtype == "e4m3"
store = dict(bf16=torch.bfloat16, fp32=torch.float32, e4m3=torch.float8_e4m3fn)[dtype]
qt = torch.float32 if dtype == "fp32" else torch.bfloat16
kv = [torch.zeros((B * M, Hkv, page, D), device="cuda").to(store) for _ in "kv"]
sc = [torch.zeros((B * M, Hkv, page), device="cuda") for _ in "kv"] if quant else [None, None]
cache = sa.PagedCache(*kv, *sc)
length, n = put([0] * B, torch.int64), put([1000, 3, 0, 1, 3000], torch.int32)
table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
stack, count = torch.arange(B * M, dtype=torch.int32, device="cuda"), put([B * M], torch.int64)
batch = sa.PagedBatch(B, 4100)
torch.manual_seed(1)
x = torch.randn((4100, H + 2 * Hkv, D), device="cuda").to(qt)
q = x[:, :H].contiguous().view(4100, H, 1, D)
g = sa.sparse_attn_graph_build_structured(M * page, W, [])

def step(l, t, s, c):
    sa.sparse_attn_paged_plan(l, n, t, s, c, page, batch)
    sa.sparse_attn_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], cache, batch.slot)
    return sa.sparse_attn_paged_decode(q, cache, t, batch.pos, g, 0.125, row=batch.row)

state = [length, table, stack, count]
mine = [t.clone() for t in state]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, lse = step(*mine)
graph.replay()
torch.cuda.synchronize()
sa.sparse_attn_check_device()
got = out.clone(), lse.clone()
want = step(*state)
assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
assert torch.isfinite(want[1][:4004]).all() and all(torch.equal(a, b) for a, b in zip(state, mine))
print("same")
"""


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("W", [64, 6400])
def test_first_calls_are_captured(dtype, W):
    p = subprocess.run([sys.executable, "-c", CODE.format(dtype=repr(dtype), W=W)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("same"), p.stderr[-2000:]
