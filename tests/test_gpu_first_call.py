"""A process's first prompt or prefix call may be one that is being captured into a graph: whatever the
library and the driver set up on first use is allowed there. Each case runs in a process of its own."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CHILD = """
import sys
import torch
import rank_latent_kv_mlra_b200 as M
import workloads as W

name, op = sys.argv[1:]
w = W.scaled(W.WORKLOADS[name], batch=3, seq_len=None, len_range=(60, 300), seed=91)
inp = W.make_workload(w, device="cuda")
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
table, lens = inp["page_table"], inp["seq_lens"]
hdl = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"])
if op == "prefix":
    q = torch.randn(2, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    out = torch.empty(2, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_decode_prefix_workspace_size(hdl, 2, 1), dtype=torch.uint8, device="cuda")
    args = (hdl, q, inp["pool"], table[:1].contiguous(), lens[:1].contiguous(), i32([0, 2]), table[1:].contiguous(),
            lens[1:].contiguous(), out)
    fn = M.mlra_decode_prefix
else:
    n = {"few": 10, "many": 60, "heads": 500}[op]
    if op == "heads":                       # whole prompts: the tables hold at most four times the query tokens
        table = table[:, :n // 64].contiguous()
        lens = torch.minimum(lens, i32([64 * table.shape[1]]))
    q = torch.randn(n, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    out = torch.empty(n, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_prefill_workspace_size(hdl, n, 3, table.shape[1]), dtype=torch.uint8, device="cuda")
    args = (hdl, q, i32([0, n // 3, n // 2, n]), inp["pool"], table, lens, out)
    fn = M.mlra_prefill
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    fn(*args, workspace=ws)
out.fill_(float("nan"))
graph.replay()
torch.cuda.synchronize()
assert M.mlra_get_status(ws) == 0
got = out.clone()
fn(*args, workspace=ws)
torch.cuda.synchronize()
assert M.mlra_get_status(ws) == 0 and not out.isnan().any() and torch.equal(got, out)
print("the first call was captured")
"""


@pytest.mark.parametrize("name,op", [("mlra4_h128_b32_n8192", "few"), ("mlra4_h128_b32_n8192", "heads"),
                                     ("mlra2_h128_b64_n4096", "many"), ("mla_h128_b128_ragged1k_32k", "prefix")])
def test_a_first_call_may_be_captured(name, op):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD, name, op], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the first call was captured" in r.stdout, r.stdout + r.stderr
