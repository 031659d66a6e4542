"""Decode over shared prefixes (mlra_decode_prefix) on the GPU against float64 results from the
definition: each sequence attends to its group's prefix rows, then to its own. Same tolerances as
the decode step (tests/gpu_util.py): the roundings are the same (absorbed query, probabilities,
merged latent result)."""
import ctypes

import numpy as np
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

MLRA4 = W.WORKLOADS["mlra4_h128_b32_n8192"]
MLRA2 = W.WORKLOADS["mlra2_h128_b64_n4096"]
MLA = W.WORKLOADS["mla_h128_b128_ragged1k_32k"]
TINY = W.scaled(W.WORKLOADS["mlra4_h8_b1_n256_f32"], paging="permuted")
RANK4 = W.WORKLOADS["tp4rank_mlra4_h32_b64_n8192"]
SUM4 = W.WORKLOADS["mlra4sum_h128_b32_n8192"]
SUM2 = W.WORKLOADS["mlra2sum_h128_b64_n4096"]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def make(w, offsets, pre, suf, seed=0, q_dtype=torch.bfloat16):
    """Group g = sequences offsets[g] .. offsets[g+1] - 1, behind a prefix of pre[g] rows; own rows suf."""
    G_, B = len(pre), len(suf)
    w = W.scaled(w, batch=G_ + B, seq_len=None, len_range=(1, 1), seed=seed + 300)
    inp = W.make_workload(w, device="cuda", seq_lens=torch.tensor(list(pre) + list(suf), dtype=torch.int32),
                          extra_pages=2)
    table, lens = inp["page_table"], inp["seq_lens"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    inp.update(pre_table=table[:G_].contiguous(), pre_lens=lens[:G_].contiguous(),
               suf_table=table[G_:].contiguous(), suf_lens=lens[G_:].contiguous(),
               offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
               q=torch.randn(B, w.h, w.d_h + w.d_r, generator=g, device="cuda").to(q_dtype))
    return w, inp


def handle(w, inp):
    return M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"], blocks_summed=w.summed)


def run(hdl, w, inp, out_dtype=torch.float32, **kw):
    B = inp["q"].shape[0]
    out = torch.full((B, w.h, w.d_h), float("nan"), device="cuda", dtype=out_dtype)
    lse = torch.full((B, w.h * (w.k if w.summed else 1)), float("nan"), device="cuda")
    ws = M.mlra_decode_prefix(hdl, inp["q"], inp["pool"], inp["pre_table"], inp["pre_lens"], inp["offsets"],
                              inp["suf_table"], inp["suf_lens"], out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse, M.mlra_get_status(ws)


def reference(w, inp):
    offsets, B, G_ = inp["offsets"].tolist(), inp["q"].shape[0], len(inp["pre_lens"])
    group = [next((g for g in range(G_) if offsets[g] <= b < offsets[g + 1]), None) for b in range(B)]
    q = inp["q"].to(torch.bfloat16).double()
    wuk, wuv = inp["w_uk"].double(), inp["w_uv"].double()
    blocks = w.k if w.summed else 1
    out = torch.zeros(B, w.h, w.d_h, dtype=torch.float64, device="cuda")
    lse = torch.full((B, blocks, w.h), -np.inf, dtype=torch.float64, device="cuda")
    alpha = 1.0 / np.sqrt(w.k) if w.summed else 1.0
    for b in range(B):
        parts = [W.logical_rows(inp, G_ + b).double()]
        if group[b] is not None:
            parts.insert(0, W.logical_rows(inp, group[b]).double())
        rows = torch.cat(parts)
        if len(rows) == 0:
            continue
        for h in range(w.h):
            for j in range(blocks):
                blk = j if w.summed else h // (w.h // w.k)
                uk, uv = (wuk[j, h], wuv[j, h]) if w.summed else (wuk[h], wuv[h])
                c = rows[:, blk * w.d_b:(blk + 1) * w.d_b]
                s = torch.cat([c @ uk, rows[:, w.d_c:]], dim=1) @ q[b, h] / np.sqrt(w.d_h + w.d_r)
                lse[b, j, h] = torch.logsumexp(s, 0)
                out[b, h] += alpha * (torch.softmax(s, 0) @ (c @ uv))
    return out.cpu().numpy(), lse.reshape(B, -1).cpu().numpy()


def check(w, inp, out, lse, status, what):
    assert status == 0, M.mlra_status_string(status)
    ref, rlse = reference(w, inp)
    G.assert_parity(out.float().cpu().numpy(), ref, what)
    got = lse.cpu().numpy()
    live = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(got), ~live), what
    assert np.abs(got[live] - rlse[live]).max(initial=0.0) < G.TOL_LSE_ABS, what


CASES = {
    # name: (workload, group offsets, prefix lengths, own lengths)
    "one": (MLRA4, [0, 1], [1], [0]),
    "four_samples": (MLRA4, [0, 4], [1000], [0, 1, 64, 65]),
    "no_prefix": (MLRA4, [0, 3], [0], [5, 130, 0]),
    "groups": (MLRA4, [0, 1, 4, 4, 13, 22], [63, 500, 700, 0, 129],
               [0, 3, 0, 128, 1, 1, 0, 0, 9, 300, 64, 2, 2] + [7 * i for i in range(9)]),
    "one_long": (MLRA4, [0, 2], [20000], [10, 300]),
    "some_without_group": (MLRA4, [0, 3], [200], [1, 2, 3, 4, 0, 150]),
    "mlra2": (MLRA2, [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "mla": (MLA, [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "rank4": (RANK4, [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "tiny": (TINY, [0, 70, 75], [700, 65], [(i * 13) % 200 for i in range(75)]),
    "heads3": (W.scaled(MLRA4, h=12), [0, 50, 60], [700, 65], [(i * 11) % 90 for i in range(60)]),
    "rank_heads": (W.scaled(RANK4, h=96), [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "many_members": (MLRA4, [0, 150], [300], [i % 5 for i in range(150)]),
    "sum4": (SUM4, [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "sum2": (SUM2, [0, 3, 5], [700, 65], [0, 1, 90, 0, 5]),
    "tinysum": (W.scaled(TINY, summed=True), [0, 20, 21], [300, 0], [i * 3 for i in range(21)]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_definition(name):
    w, offsets, pre, suf = CASES[name]
    w, inp = make(w, offsets, pre, suf, seed=len(name))
    hdl = handle(w, inp)
    for dt in (torch.float32, torch.bfloat16):
        check(w, inp, *run(hdl, w, inp, dt), f"{name} {dt}")


def test_large_batch_matches_decode_on_the_whole_sequences():
    """Batch 140 (the planner's block-wide path starts at 257 sequences; here several token tiles a
    group), against mlra_decode on tables whose rows list the prefix's pages, then the own ones."""
    suf = [(37 * i) % 200 for i in range(140)]
    w, inp = make(MLRA4, [0, 100, 140], [640, 1920], suf, seed=3)
    hdl = handle(w, inp)
    out, lse, status = run(hdl, w, inp)
    assert status == 0
    rows = []
    for b in range(140):
        g = 0 if b < 100 else 1
        rows.append(torch.cat([inp["pre_table"][g, :(640, 1920)[g] // 64], inp["suf_table"][b, :(suf[b] + 63) // 64]]))
    table = torch.zeros(140, max(map(len, rows)), dtype=torch.int32, device="cuda")
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    lens = inp["suf_lens"] + torch.tensor([640] * 100 + [1920] * 40, dtype=torch.int32, device="cuda")
    dout, dlse = torch.empty_like(out), torch.empty_like(lse)
    M.mlra_decode(hdl, inp["q"], inp["pool"], table, lens, dout, dlse)
    torch.cuda.synchronize()
    G.assert_parity(out.cpu().numpy(), dout.double().cpu().numpy(), "prefix against whole")
    assert (lse - dlse).abs().max() < 1e-3


def test_fp32_query_and_refusals():
    w, inp = make(MLRA4, [0, 2, 5], [600, 200], [10, 0, 64, 100, 3], seed=8, q_dtype=torch.float32)
    hdl = handle(w, inp)
    check(w, inp, *run(hdl, w, inp), "fp32 query")
    ws = torch.empty(M.mlra_decode_prefix_workspace_size(hdl, 5, 2) - 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(M.MlraError, match="WORKSPACE"):
        run(hdl, w, inp, workspace=ws)
    with pytest.raises(ValueError, match="group_offsets"):
        run(hdl, w, dict(inp, offsets=inp["offsets"][:2].contiguous()))
    e4m3 = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"], cache_fp8=True)
    with pytest.raises(M.MlraError, match="UNSUPPORTED"):
        run(e4m3, w, dict(inp, pool=torch.zeros(inp["pool"].shape, dtype=torch.uint8, device="cuda")))


def test_a_bad_row_of_one_sequence_stays_with_it():
    """NaN in one sequence's own row, and slots behind a prefix's end that hold NaN (as they do in
    every workload here), leave the others' results as they were."""
    w, inp = make(MLRA4, [0, 4], [130], [10, 20, 30, 0], seed=9)
    hdl = handle(w, inp)
    clean = run(hdl, w, inp)[0]
    inp["pool"][int(inp["suf_table"][1, 0]), 5] = float("nan")
    out = run(hdl, w, inp)[0]
    assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]]) and out[1].isnan().all()


def test_more_than_256_sequences():
    """Beyond 256 sequences the decode step plans its own rows block-wide."""
    w, inp = make(TINY, [0, 100, 300], [130, 64], [(i * 7) % 70 for i in range(300)], seed=4)
    check(w, inp, *run(handle(w, inp), w, inp), "300 sequences")


def test_runs_are_bit_identical():
    w, inp = make(MLRA4, [0, 9], [3000], list(range(9)), seed=5)
    hdl = handle(w, inp)
    a, la, _ = run(hdl, w, inp)
    b, lb, _ = run(hdl, w, inp)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_captured_graph_replays_with_new_lengths():
    w, inp = make(MLRA4, [0, 2, 5], [600, 200], [10, 0, 64, 100, 3], seed=6)
    hdl = handle(w, inp)
    out = torch.empty(5, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_decode_prefix_workspace_size(hdl, 5, 2), dtype=torch.uint8, device="cuda")
    args = (inp["q"], inp["pool"], inp["pre_table"], inp["pre_lens"], inp["offsets"], inp["suf_table"],
            inp["suf_lens"], out)
    M.mlra_decode_prefix(hdl, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mlra_decode_prefix(hdl, *args, workspace=ws)
    inp["pre_lens"].copy_(torch.tensor([333, 0], dtype=torch.int32))
    # (no sequence gets more rows than it has pages for)
    inp["suf_lens"].copy_(torch.tensor([0, 0, 1, 64, 2], dtype=torch.int32))
    inp["offsets"].copy_(torch.tensor([0, 4, 5], dtype=torch.int32))
    inp["q"].copy_(torch.randn_like(inp["q"]))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    ref, _, status = run(hdl, w, inp)
    assert status == 0 and torch.equal(got, ref)


def test_status_of_bad_lengths_offsets_and_pages():
    w, inp = make(MLRA4, [0, 2, 5], [600, 200], [10, 0, 64, 100, 3], seed=7)
    hdl = handle(w, inp)
    good = run(hdl, w, inp)[0]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    assert run(hdl, w, dict(inp, pre_lens=i32([600, 10 ** 6])))[2] == -7
    assert run(hdl, w, dict(inp, suf_lens=i32([10, 0, -1, 100, 3])))[2] == -7
    alone = run(hdl, w, dict(inp, pre_lens=i32([0, 0])))[0]
    for off in ([0, 3, 2], [1, 2, 5], [0, 2, 9]):
        out, _, status = run(hdl, w, dict(inp, offsets=i32(off)))
        assert status == -7 and torch.equal(out, alone)  # decoded without prefixes
    pt = inp["pre_table"].clone()
    pt[1, 1] = -3
    assert run(hdl, w, dict(inp, pre_table=pt))[2] == -4
    assert torch.equal(run(hdl, w, inp)[0], good)


def test_a_replayed_graph_does_not_keep_an_earlier_status():
    """Bad lengths and offsets in one replay are reported by that replay alone."""
    w, inp = make(MLRA4, [0, 2, 5], [600, 200], [10, 0, 64, 100, 3], seed=10)
    hdl = handle(w, inp)
    out = torch.empty(5, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_decode_prefix_workspace_size(hdl, 5, 2), dtype=torch.uint8, device="cuda")
    args = (inp["q"], inp["pool"], inp["pre_table"], inp["pre_lens"], inp["offsets"], inp["suf_table"],
            inp["suf_lens"], out)
    M.mlra_decode_prefix(hdl, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mlra_decode_prefix(hdl, *args, workspace=ws)

    def replay():
        graph.replay()
        return int(ws[:4].view(torch.int32)[0])

    assert replay() == 0
    good = out.clone()
    for name, at, wrong in (("pre_lens", 1, 10 ** 6), ("offsets", 1, 6), ("suf_lens", 2, -1)):
        right = int(inp[name][at])
        inp[name][at] = wrong
        assert replay() == -7
        inp[name][at] = right
        assert replay() == 0 and torch.equal(out, good)


def test_tables_wider_than_lengths_can_be_are_refused():
    """A page table whose capacity passes a 32-bit length (refused before anything is read)."""
    w, inp = make(MLRA4, [0, 2], [70], [10, 0], seed=11)
    hdl = handle(w, inp)
    lib, P = M.load_library(), ctypes.c_void_p
    call = lambda pre_stride, stride: lib.mlra_decode_prefix(
        hdl.ptr, P(16), 1, P(16), 4, P(16), pre_stride, P(16), P(16), 1, P(16), stride, P(16), 2, P(16), 1, None, P(256),
        1, None)
    assert call(2 ** 25, 1) == -1 and call(1, 2 ** 25) == -1
    assert call(1, 1) == -6  # (these sizes alone: the workspace is too small)


def widen(inp):
    """The same step with page tables wide enough that a decode kernel takes the own rows (the library
    goes by the table's capacity when it chooses; narrow tables leave them to the prefix's kernel)."""
    t = inp["suf_table"]
    return dict(inp, suf_table=torch.nn.functional.pad(t, (0, 4000 - t.shape[1]), value=-1).contiguous())


@pytest.mark.parametrize("name", ["no_prefix", "groups", "some_without_group", "mlra2", "mla", "rank4", "tiny", "heads3",
                                  "rank_heads", "sum4", "sum2", "tinysum"])
def test_wide_tables_match_the_definition(name):
    w, offsets, pre, suf = CASES[name]
    w, inp = make(w, offsets, pre, suf, seed=len(name))
    check(w, inp, *run(handle(w, inp), w, widen(inp)), name)


@pytest.mark.parametrize("wide", [False, True])
def test_bad_own_rows_of_both_forms(wide):
    """Lengths, pages and offsets that are refused, a NaN that stays with its sequence, a fp32 query."""
    w, inp = make(MLRA4, [0, 2, 5], [600, 200], [10, 0, 64, 100, 3], seed=12, q_dtype=torch.float32)
    inp = widen(inp) if wide else inp
    hdl = handle(w, inp)
    check(w, inp, *run(hdl, w, inp), "fp32 query")
    good = run(hdl, w, inp)[0]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    assert run(hdl, w, dict(inp, suf_lens=i32([10, 0, 64, 100, 10 ** 6])))[2] == -7
    table = inp["suf_table"].clone()
    table[3, 1] = inp["pool"].shape[0]
    out, _, status = run(hdl, w, dict(inp, suf_table=table))
    assert status == -4 and torch.equal(out[[0, 1, 2, 4]], good[[0, 1, 2, 4]])
    alone = run(hdl, w, dict(inp, pre_lens=i32([0, 0])))[0]
    out, _, status = run(hdl, w, dict(inp, offsets=i32([0, 6, 5])))
    assert status == -7 and torch.equal(out, alone)
    pool = inp["pool"].clone()
    pool[int(inp["suf_table"][3, 1]), 20] = float("nan")
    out = run(hdl, w, dict(inp, pool=pool))[0]
    assert torch.equal(out[[0, 1, 2, 4]], good[[0, 1, 2, 4]]) and out[3].isnan().all()


def test_rows_behind_the_groups_and_lengths_that_end_on_tiles():
    """Own lengths around page and tile ends, every sequence of a batch at the rule's largest, and a
    replayed graph that moves rows from one part to the other."""
    suf = [0, 1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 319, 320] * 4
    w, inp = make(RANK4, [0, 31, 40], [257, 128], suf, seed=13)
    hdl = handle(w, inp)
    check(w, inp, *run(hdl, w, inp), "64 sequences")
    lens, offsets = inp["suf_lens"].clone(), inp["offsets"].clone()
    out = torch.empty(64, w.h, w.d_h, device="cuda")
    args = (inp["q"], inp["pool"], inp["pre_table"], inp["pre_lens"], inp["offsets"], inp["suf_table"],
            inp["suf_lens"], out)
    ws = M.mlra_decode_prefix(hdl, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mlra_decode_prefix(hdl, *args, workspace=ws)
    for new_lens, new_offsets in ((torch.zeros_like(lens), offsets), (lens, torch.zeros_like(offsets)), (lens, offsets)):
        inp["suf_lens"].copy_(new_lens)
        inp["offsets"].copy_(new_offsets)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        ref, _, status = run(hdl, w, inp)
        assert status == 0 and torch.equal(got, ref)
    check(w, inp, *run(hdl, w, inp), "after the replays")


HALVES = {
    # many short units a CTA, so that a boundary cuts one column half's unit and leaves the other's whole
    "own_rows": (MLA, [0, 49, 63], [261, 41], [(37 * i) % 300 if i % 3 else 1 for i in range(64)]),
    "rank_of_own_rows": (W.scaled(MLA, h=16), [0, 20], [200], [(53 * i) % 300 for i in range(60)]),
    "prefixes": (MLA, list(range(0, 101)), [(29 * i) % 400 for i in range(100)], [i % 3 for i in range(100)]),
    "own_rows_mlra2": (MLRA2, [0, 49, 63], [261, 41], [(37 * i) % 300 if i % 3 else 1 for i in range(64)]),
    "own_rows_sum4": (SUM4, [0, 9], [261], [(37 * i) % 200 for i in range(40)]),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name", list(HALVES))
def test_units_of_which_one_half_is_cut(name, wide):
    """In a workspace of NaN bits, so that a result that no unit of the call has written shows."""
    w, offsets, pre, suf = HALVES[name]
    w, inp = make(w, offsets, pre, suf, seed=21)
    inp = widen(inp) if wide else inp
    hdl = handle(w, inp)
    size = M.mlra_decode_prefix_workspace_size(hdl, len(suf), len(pre))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    check(w, inp, *run(hdl, w, inp, workspace=ws), name)
