"""Workspace sizes of the operators around the decode step: one taken for the largest call serves every
smaller one on the same tables."""
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W

pytestmark = pytest.mark.gpu

NAMES = ["mlra4_h128_b32_n8192", "mlra2_h128_b64_n4096", "mla_h128_b128_ragged1k_32k", "mlra4_h8_b1_n256_f32",
         "tp4rank_mlra4_h32_b64_n8192", "mlra4fp8_h128_b32_n8192", "mlra4sum_h128_b32_n8192",
         "mlra2sum_h128_b64_n4096"]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def handle(w, w_uk=None, w_uv=None):
    if w_uk is None:
        w_uk = w_uv = torch.zeros(*((w.k,) if w.summed else ()), w.h, w.d_b, w.d_h, dtype=torch.bfloat16, device="cuda")
    return M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, w_uk, w_uv, blocks_summed=w.summed, cache_fp8=w.cache == "e4m3")


def grows(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("name", NAMES)
def test_prompt_sizes_grow_with_the_tokens(name):
    hdl = handle(W.WORKLOADS[name])
    tokens = list(range(0, 200)) + [255, 256, 257, 400, 1000, 4095, 4096, 20000]
    for batch, stride in ((1, 1), (1, 100), (8, 3), (8, 100), (300, 2)):
        assert grows([M.mlra_prefill_workspace_size(hdl, n, batch, stride) for n in tokens]), (batch, stride)


@pytest.mark.parametrize("name", [n for n in NAMES if "fp8" not in n])
def test_prefix_sizes_grow_with_sequences_and_groups(name):
    hdl = handle(W.WORKLOADS[name])
    counts = list(range(1, 140)) + [255, 256, 257, 1000]
    assert grows([M.mlra_decode_prefix_workspace_size(hdl, n, 1) for n in counts])
    assert grows([M.mlra_decode_prefix_workspace_size(hdl, 64, n) for n in counts])


def test_page_sizes_grow_with_pages_and_rows():
    hdl = handle(W.WORKLOADS["mlra4_h8_b1_n256_f32"])
    counts = list(range(1, 300)) + [8191, 8192, 8193, 10 ** 6]
    assert grows([M.mlra_pages_workspace_size(hdl, n, 7) for n in counts])
    assert grows([M.mlra_pages_workspace_size(hdl, 1000, n) for n in counts if n <= 65536])


def test_a_workspace_for_more_tokens_serves_fewer():
    """36 drafted tokens' workspace, then 32 (which the decode step's combine merges) and 1."""
    w = W.scaled(W.WORKLOADS["mlra4_h128_b32_n8192"], batch=4, seq_len=None, len_range=(300, 600), seed=81)
    inp = W.make_workload(w, device="cuda")
    hdl = handle(w, inp["w_uk"], inp["w_uv"])
    stride = inp["page_table"].shape[1]
    ws = torch.empty(M.mlra_prefill_workspace_size(hdl, 36, 4, stride), dtype=torch.uint8, device="cuda")
    q = torch.randn(36, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    for n, cu in ((36, [0, 9, 18, 27, 36]), (32, [0, 9, 16, 27, 32]), (1, [0, 0, 0, 1, 1])):
        outs = []
        for workspace in (None, ws):
            out = torch.empty(n, w.h, w.d_h, device="cuda")
            got = M.mlra_prefill(hdl, q[:n], torch.tensor(cu, dtype=torch.int32, device="cuda"), inp["pool"],
                                 inp["page_table"], inp["seq_lens"], out, workspace=workspace)
            torch.cuda.synchronize()
            assert M.mlra_get_status(got) == 0
            outs.append(out)
        assert torch.equal(*outs)


KINDS = [("mlra4_h128_b32_n8192", [3, 20], [700, 40], 0), ("mlra4_h128_b32_n8192", [33, 90, 0, 1], [10, 900, 64, 0], 0),
         ("mlra4_h128_b32_n8192", [700, 300], [0, 0], 0), ("mlra2_h128_b64_n4096", [5, 130], [900, 40], 30),
         ("mla_h128_b128_ragged1k_32k", [1] * 70, [7 * i for i in range(70)], 0),
         ("mla_h128_b128_ragged1k_32k", [300, 257], [0, 0], 0), ("mlra4fp8_h128_b32_n8192", [5, 130], [900, 40], 0),
         ("mlra4sum_h128_b32_n8192", [5, 70], [40, 300], 0)]


@pytest.mark.parametrize("name,n,past,spare", KINDS)
def test_results_do_not_depend_on_what_the_workspace_held(name, n, past, spare):
    """Prompt calls of every form in workspaces of zeros and of NaN bits: the same bits."""
    w = W.scaled(W.WORKLOADS[name], batch=len(n), seq_len=None, len_range=(1, 1), seed=82)
    lens = torch.tensor([a + b for a, b in zip(n, past)], dtype=torch.int32)
    inp = W.make_workload(w, device="cuda", seq_lens=lens)
    table = torch.nn.functional.pad(inp["page_table"], (0, spare), value=-1).contiguous()
    hdl = handle(w, inp["w_uk"], inp["w_uv"])
    q = torch.randn(sum(n), w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    cu = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device="cuda")
    size = M.mlra_prefill_workspace_size(hdl, sum(n), len(n), table.shape[1])
    outs = []
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((sum(n), w.h, w.d_h), float("nan"), device="cuda")
        lse = torch.full((sum(n), w.h * (w.k if w.summed else 1)), float("nan"), device="cuda")
        M.mlra_prefill(hdl, q, cu, inp["pool"], table, inp["seq_lens"], out, lse, workspace=ws)
        torch.cuda.synchronize()
        assert M.mlra_get_status(ws) == 0 and not out.isnan().any() and not lse.isnan().any()
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
