"""Prompt attention (mlra_prefill) on the GPU against the float64 oracle, token by token.

The oracle side is ``O.decode_sequence`` / ``O.decode_heads`` on the prefix of cached rows each
token may see. Tolerances: outputs of ordinary inputs (N(0,1) cache and queries) use the decode
path's parity bar (tests/gpu_util.py); the chain rounds the same quantities to bf16 (absorbed
query, probabilities, latent result, each off by at most 2^-8 / 2 relative), so the same bar holds.
"""
import numpy as np
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W
from oracle import mlra_oracle as O
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

MLRA4 = W.WORKLOADS["mlra4_h128_b32_n8192"]
MLRA2 = W.WORKLOADS["mlra2_h128_b64_n4096"]
MLA = W.WORKLOADS["mla_h128_b128_ragged1k_32k"]
TINY = W.scaled(W.WORKLOADS["mlra4_h8_b1_n256_f32"], paging="permuted")
RANK4 = W.WORKLOADS["tp4rank_mlra4_h32_b64_n8192"]
E4M3 = W.WORKLOADS["mlra4fp8_h128_b32_n8192"]
SUM4 = W.WORKLOADS["mlra4sum_h128_b32_n8192"]
SUM2 = W.WORKLOADS["mlra2sum_h128_b64_n4096"]
TINYSUM = W.scaled(TINY, summed=True)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def make(w, n_q, past, seed=0, q_dtype=torch.bfloat16, behind=0, form=None):
    """Packed queries for `n_q[b]` new tokens of sequences with `past[b]` older ones. The library
    goes by the table's capacity when it chooses a form: `form` "absorbed" widens the table past
    four times the query tokens, "heads" asserts that it is not wider."""
    total = [a + b for a, b in zip(n_q, past)]
    w = W.scaled(w, batch=len(n_q), seq_len=None, len_range=(1, 1), seed=seed + 100)
    inp = W.make_workload(w, device="cuda", seq_lens=torch.tensor(total, dtype=torch.int32), extra_pages=2)
    cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randn(int(cu[-1]) + behind, w.h, w.d_h + w.d_r, generator=g, device="cuda")
    inp["q"] = q.to(q_dtype)
    inp["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    table = inp["page_table"]
    if form == "absorbed":
        wide = 4 * q.shape[0] // (64 * len(n_q)) + 1
        if table.shape[1] < wide:
            inp["page_table"] = torch.nn.functional.pad(table, (0, wide - table.shape[1]), value=-1).contiguous()
    if form == "heads":
        assert len(n_q) * table.shape[1] * 64 <= 4 * q.shape[0]
    return w, inp


def handle(w, inp):
    fp8 = dict(cache_fp8=True, latent_scale=W.E4M3_SCALE, rope_scale=W.E4M3_SCALE) if w.cache == "e4m3" else {}
    return M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"], blocks_summed=w.summed, **fp8)


def run(hdl, w, inp, out_dtype=torch.float32, workspace=None, stream=None):
    total = inp["q"].shape[0]
    out = torch.full((total, w.h, w.d_h), float("nan"), device="cuda", dtype=out_dtype)
    lse = torch.full((total, w.h * (w.k if w.summed else 1)), float("nan"), device="cuda")
    ws = M.mlra_prefill(hdl, inp["q"], inp["cu"], inp["pool"], inp["page_table"], inp["seq_lens"], out, lse,
                        workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out, lse, M.mlra_get_status(ws)


def rows64(w, inp, b):
    rows = W.logical_rows(inp, b)
    if w.cache == "e4m3":
        return rows.view(torch.float8_e4m3fn).double() * W.E4M3_SCALE
    return rows.double()


def reference(w, inp):
    """float64 outputs and lse of every packed token (torch on the GPU, from the definition: each
    head's keys and values formed from its block of the cached rows)."""
    cu = inp["cu"].tolist()
    q = inp["q"].to(torch.bfloat16).double()
    wuk, wuv = inp["w_uk"].double(), inp["w_uv"].double()
    total = cu[-1]
    blocks = w.k if w.summed else 1
    out = torch.zeros(total, w.h, w.d_h, dtype=torch.float64, device="cuda")
    lse = torch.full((total, blocks, w.h), -np.inf, dtype=torch.float64, device="cuda")
    scale = 1.0 / np.sqrt(w.d_h + w.d_r)
    hb = w.h // w.k
    for b in range(len(cu) - 1):
        n, T = cu[b + 1] - cu[b], int(inp["seq_lens"][b])
        if n == 0 or T == 0:
            continue
        rows = rows64(w, inp, b)
        pos = torch.arange(T - n, T, device="cuda")
        mask = torch.arange(T, device="cuda")[None, :] > pos[:, None]
        for h in range(w.h):
            for j in range(blocks):
                blk = j if w.summed else h // hb
                uk, uv = (wuk[j, h], wuv[j, h]) if w.summed else (wuk[h], wuv[h])
                c = rows[:, blk * w.d_b:(blk + 1) * w.d_b]
                key = torch.cat([c @ uk, rows[:, w.d_c:]], dim=1)
                s = (q[cu[b]:cu[b + 1], h] @ key.t() * scale).masked_fill(mask, -np.inf)
                l = torch.logsumexp(s, dim=1)
                p = torch.where(mask, 0.0, torch.exp(s - torch.where(l.isinf(), 0.0, l)[:, None]))
                alpha = 1.0 / np.sqrt(w.k) if w.summed else 1.0
                out[cu[b]:cu[b + 1], h] += alpha * (p @ (c @ uv))
                lse[cu[b]:cu[b + 1], j, h] = l
    return out.cpu().numpy(), lse.reshape(total, -1).cpu().numpy()


def check(w, inp, out, lse, status, what, rows=1.0):
    """`rows`: factor of the cached rows against N(0,1). The bar's absolute parts are for N(0,1)
    rows. The rounding of the absorbed query moves a score by an amount that grows with the row
    (x rows), a probability moves by its score's error relative to itself, and the values it
    weighs are x rows too: absolute output errors grow by rows^2, those of the lse by rows. The
    relative part of the bar stays. A bf16 output's own rounding comes on top: half a step, 2^-8 of
    the value, which for the first tokens of a prompt (few keys, values of several units) is as
    large as the bar itself."""
    assert status == 0, M.mlra_status_string(status)
    ref, rlse = reference(w, inp)
    total = ref.shape[0]
    own = 2.0 ** -8 * np.abs(ref).max(initial=0.0) if out.dtype == torch.bfloat16 else 0.0
    G.assert_parity(out[:total].float().cpu().numpy(), ref, what, tol_max=G.TOL_MAX_ABS * rows ** 2 + own,
                    tol_mean=G.TOL_MEAN_ABS * rows ** 2)
    got = lse[:total].cpu().numpy()
    live = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(got), ~live), what
    assert np.abs(got[live] - rlse[live]).max(initial=0.0) < G.TOL_LSE_ABS * rows, what


CASES = {
    # name: (workload, new tokens, older tokens)
    "one_token": (MLRA4, [1], [0]),
    "one_token_long": (MLRA4, [1], [1000]),
    # few tokens (merged by the decode step's combine), each kind of handle
    "few_mla": (MLA, [3, 20], [700, 40]),
    "few_mlra2": (MLRA2, [3, 20], [700, 40]),
    "few_tiny": (TINY, [3, 20, 0, 9], [700, 40, 9, 0]),
    "few_e4m3": (E4M3, [3, 20], [700, 40]),
    "few_sum4": (SUM4, [3, 20], [700, 40]),
    "few_sum2": (SUM2, [3, 20], [700, 40]),
    "few_32": (MLRA4, [2, 30], [700, 40]),
    "not_few_33": (MLRA4, [3, 30], [700, 40]),
    "tile_edges": (MLRA4, [3, 4, 5, 8, 9, 127, 128, 129], [0, 64, 63, 0, 65, 1, 0, 127]),
    "empty_sequences": (MLRA4, [0, 7, 0, 0, 130, 0], [0, 0, 300, 0, 5, 64]),
    "ragged": (MLRA4, [333, 1, 64, 511, 20], [0, 0, 0, 77, 700]),
    "long_chunk": (MLRA4, [200], [3000]),
    "mlra2": (MLRA2, [1, 2, 3, 150, 65], [0, 63, 500, 0, 130]),
    "mla": (MLA, [1, 2, 70, 33], [0, 63, 10, 400]),
    "rank4": (RANK4, [5, 130, 1, 64], [0, 40, 200, 0]),
    "tiny": (TINY, [1, 63, 64, 65, 200, 0, 300], [0, 1, 0, 100, 0, 9, 57]),
    "e4m3": (E4M3, [5, 130, 1, 64], [0, 40, 200, 700]),
    "sum4": (SUM4, [5, 70, 1], [0, 40, 300]),
    "sum2": (SUM2, [5, 70, 1], [0, 40, 300]),
    "tinysum": (TINYSUM, [5, 70, 1, 130], [0, 40, 300, 0]),
    # whole prompts: the per-head form, and the absorbed one on a wider table
    "prompts_mlra4": (MLRA4, [300, 257, 1, 128, 129, 256, 310], [0] * 7),
    "prompts_mlra2": (MLRA2, [300, 257, 64, 0, 129], [3, 0, 0, 0, 100]),
    "prompts_mla": (MLA, [300, 257, 64, 129], [0, 0, 1, 130]),
    "prompts_rank4": (RANK4, [700, 513, 64, 300], [0, 5, 200, 0]),
    "prompt_one_odd_page": (MLRA4, [65], [0]),
    "prompt_three_units": (MLA, [700], [0]),
    "prompts_whole_units": (MLRA4, [1500, 0, 1, 900, 257, 0], [0, 0, 0, 60, 0, 5]),
    # heads of a block that do not divide a row tile, and one head a block
    "heads3": (W.scaled(MLRA4, h=12), [1, 41, 42, 43, 84, 85, 130], [0, 3, 700, 0, 64, 1, 0]),
    "heads1": (W.scaled(MLRA4, h=4), [1, 127, 300], [65, 0, 500]),
    "prompts_heads3": (W.scaled(MLRA4, h=12), [300, 41, 130], [0, 0, 0]),
    "rank_heads": (W.scaled(RANK4, h=96), [5, 130], [40, 200]),   # three chunks of 32 heads
    "mlra2_heads5": (W.scaled(MLRA2, h=10), [1, 25, 26, 130], [0, 3, 700, 0]),
}
FORMS = [(name, None) for name in CASES if not name.startswith("prompt")] + [
    (name, form) for name in CASES if name.startswith("prompt") for form in ("absorbed", "heads")]


@pytest.mark.parametrize("name,form", FORMS, ids=[f"{n}-{f}" if f else n for n, f in FORMS])
def test_matches_the_definition(name, form):
    w, n, past = CASES[name]
    w, inp = make(w, n, past, seed=len(name), form=form)
    hdl = handle(w, inp)
    for dt in (torch.float32, torch.bfloat16):
        check(w, inp, *run(hdl, w, inp, dt), f"{name} {dt}")


@pytest.mark.parametrize("n,past", [([40, 3], [0, 90]), ([300, 129], [0, 0])], ids=["chunk", "prompts"])
def test_fp32_query(n, past):
    """(An fp32 query of whole prompts takes the absorbed form in a workspace sized for both.)"""
    w, inp = make(MLRA4, n, past, seed=5, q_dtype=torch.float32)
    hdl = handle(w, inp)
    check(w, inp, *run(hdl, w, inp), "fp32 query")
    size = M.mlra_prefill_workspace_size(hdl, sum(n), len(n), inp["page_table"].shape[1])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    check(w, inp, *run(hdl, w, inp, workspace=ws), "fp32 query, own workspace")
    with pytest.raises(M.MlraError, match="WORKSPACE"):
        run(hdl, w, inp, workspace=ws[:size - 256])


def test_e4m3_cache_with_two_scales():
    """Different latent and RoPE scales, neither a power of two (outputs and lse of the same bytes)."""
    w, inp = make(E4M3, [70, 33], [0, 200], seed=15)
    lat, rope = 0.03, 0.05
    hdl = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"], cache_fp8=True, latent_scale=lat,
                        rope_scale=rope)
    out, lse, status = run(hdl, w, inp)
    # reference: a bf16-free cache of the values the bytes stand for
    plain = dict(inp)
    vals = inp["pool"].view(torch.float8_e4m3fn).double()
    plain["pool"] = torch.cat([vals[..., :w.d_c] * lat, vals[..., w.d_c:] * rope], dim=-1)
    check(W.scaled(w, cache="bf16"), plain, out, lse, status, "two scales")


def test_two_calls_at_once_on_two_streams():
    """Calls on two streams with workspaces of their own give what each gives alone."""
    runs = []
    for seed, form in ((21, "heads"), (22, "absorbed")):
        w, inp = make(MLRA4, [700, 300], [0, 0], seed=seed, form=form)
        hdl = handle(w, inp)
        runs.append((w, inp, hdl, run(hdl, w, inp)[0]))
    streams = [torch.cuda.Stream() for _ in runs]
    outs = [torch.empty_like(r[3]) for r in runs]
    torch.cuda.synchronize()
    words = []
    for _ in range(5):
        for (w, inp, hdl, _), s, out in zip(runs, streams, outs):
            words.append(M.mlra_prefill(hdl, inp["q"], inp["cu"], inp["pool"], inp["page_table"], inp["seq_lens"], out,
                                        stream=s))
    torch.cuda.synchronize()
    assert all(M.mlra_get_status(ws) == 0 for ws in words)
    for r, out in zip(runs, outs):
        assert torch.equal(out, r[3])


def test_refused_arguments():
    w, inp = make(MLRA4, [33, 90], [10, 0], seed=16)
    hdl = handle(w, inp)
    out = torch.empty(123, w.h, w.d_h, device="cuda")
    args = [inp["q"], inp["cu"], inp["pool"], inp["page_table"], inp["seq_lens"], out]

    def call(**kw):
        names = ["q", "cu", "pool", "page_table", "seq_lens", "out"]
        return M.mlra_prefill(hdl, *[kw.get(n, a) for n, a in zip(names, args)])

    with pytest.raises(ValueError, match="contiguous"):
        call(q=inp["q"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="cu_seqlens"):
        call(cu=inp["cu"][:2].contiguous())
    with pytest.raises(ValueError, match="out must be"):
        call(out=out[:100].contiguous())
    with pytest.raises(TypeError, match="seq_lens"):
        call(seq_lens=inp["seq_lens"].long())
    with pytest.raises(TypeError, match="pool"):
        call(pool=inp["pool"].float())
    with pytest.raises(ValueError, match="one device|CUDA tensor"):
        call(page_table=inp["page_table"].cpu())
    shifted = torch.empty(123 * w.h * w.d_h + 1, device="cuda")[1:].view(123, w.h, w.d_h)
    with pytest.raises(M.MlraError, match="INVALID_ARG"):  # out is not 16-byte aligned
        call(out=shifted)


def test_no_tokens():
    w, inp = make(MLRA4, [0, 0], [10, 0], seed=17)
    out, lse, status = run(handle(w, inp), w, inp)
    assert status == 0 and out.numel() == 0


BOTH = pytest.mark.parametrize("form", ["absorbed", "heads"])


@BOTH
def test_tokens_without_keys(form):
    """Sequences shorter than their query tokens: positions below 0 see nothing."""
    w, inp = make(MLRA4, [20, 26, 9], [0, 0, 3], seed=6, form=form)
    inp["seq_lens"] = torch.tensor([13, 0, 12], dtype=torch.int32, device="cuda")
    out, lse, status = run(handle(w, inp), w, inp)
    check(w, inp, out, lse, status, "short sequences")
    assert (out[:7] == 0).all() and (out[20:46] == 0).all()


@BOTH
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_behind_the_last_sequence_stay(form, dtype):
    w, inp = make(MLRA4, [30, 41], [0, 7], seed=7, behind=60, form=form)
    out, lse, status = run(handle(w, inp), w, inp, dtype)
    check(w, inp, out, lse, status, "padded batch")
    assert out[71:].isnan().all() and lse[71:].isnan().all()


@BOTH
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_cached_row_reaches_only_the_tokens_that_see_it(value, form):
    """Token 100's row holds NaN (or infinities): tokens before it keep the results they had."""
    w, inp = make(MLRA4, [360], [0], seed=8, form=form)
    hdl = handle(w, inp)
    clean, clean_lse, _ = run(hdl, w, inp)
    page = int(inp["page_table"][0, 100 // 64])
    inp["pool"][page, 100 % 64] = value
    out, lse, status = run(hdl, w, inp)
    assert status == 0
    assert torch.equal(out[:100], clean[:100]) and torch.equal(lse[:100], clean_lse[:100])
    assert out[100:].isnan().all()


@pytest.mark.parametrize("n,past", [(30, 0), (30, 900)])
def test_a_bad_cached_row_with_few_tokens(n, past):
    """The same for a call of few tokens, whose parts the decode step's combine merges."""
    w, inp = make(MLRA4, [n], [past], seed=18, form="absorbed")
    hdl = handle(w, inp)
    clean, clean_lse, _ = run(hdl, w, inp)
    inp["pool"][int(inp["page_table"][0, (past + 20) // 64]), (past + 20) % 64] = float("nan")
    out, lse, status = run(hdl, w, inp)
    assert status == 0
    assert torch.equal(out[:20], clean[:20]) and torch.equal(lse[:20], clean_lse[:20])
    assert out[20:].isnan().all() and lse[20:].isnan().all()


@BOTH
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_rows_behind_the_last_sequence_stay(form, dtype):
    w, inp = make(MLRA4, [10, 11], [0, 7], seed=19, behind=11, form=form if form == "absorbed" else None)
    out, lse, status = run(handle(w, inp), w, inp, dtype)
    check(w, inp, out, lse, status, "padded batch")
    assert out[21:].isnan().all() and lse[21:].isnan().all()


@BOTH
def test_runs_are_bit_identical_and_the_split_is_exact(form):
    """Two runs give the same bits, and a chunked prompt gives the whole prompt's results to
    within the roundings."""
    w, inp = make(MLRA4, [700], [0], seed=9, form=form)
    hdl = handle(w, inp)
    a, la, _ = run(hdl, w, inp)
    b, lb, _ = run(hdl, w, inp)
    assert torch.equal(a, b) and torch.equal(la, lb)
    pieces = []
    for lo, hi in ((0, 1), (1, 300), (300, 555), (555, 700)):
        part = dict(inp, q=inp["q"][lo:hi].contiguous(), cu=torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                    seq_lens=torch.tensor([hi], dtype=torch.int32, device="cuda"))
        pieces.append(run(hdl, w, part)[0])
    G.assert_parity(torch.cat(pieces).cpu().numpy(), a.double().cpu().numpy(), "chunks")


def test_prefill_then_decode_agree_on_the_last_token():
    w, inp = make(MLRA4, [1, 1, 1], [200, 63, 511], seed=10)
    hdl = handle(w, inp)
    out, lse, _ = run(hdl, w, inp)
    dout = torch.empty_like(out)
    dlse = torch.empty_like(lse)
    M.mlra_decode(hdl, inp["q"], inp["pool"], inp["page_table"], inp["seq_lens"], dout, dlse)
    torch.cuda.synchronize()
    G.assert_parity(out.cpu().numpy(), dout.double().cpu().numpy(), "prefill against decode")
    # The two round the absorbed query differently (the decode step scales it first). A score moves by
    # a sum of independent roundings of at most half a bf16 step, 2^-8 relative: rms at most
    # 2^-8 / sqrt(3) of a score's own rms 1; an lse moves by an average of its scores' errors, so
    # by less than the largest: 4 sigma, two sides.
    assert (lse - dlse).abs().max() < 4 * 2 ** 0.5 * 2 ** -8 / 3 ** 0.5


@BOTH
def test_large_scores_raise_the_running_maximum(form):
    """Keys whose scores grow along the sequence make the kernel raise its maximum and rescale."""
    w, inp = make(MLRA4, [260], [700], seed=11, form=form)
    ramp = torch.linspace(0.1, 6.0, 960, device="cuda")
    for t in range(960):
        page = int(inp["page_table"][0, t // 64])
        inp["pool"][page, t % 64] *= ramp[t]
    check(w, inp, *run(handle(w, inp), w, inp), "ramp", rows=6.0)


@BOTH
def test_captured_graph_replays_with_new_inputs(form):
    w, inp = make(MLRA4, [33, 90], [10, 0], seed=12, form=form)
    hdl = handle(w, inp)
    out = torch.empty(123, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_prefill_workspace_size(hdl, 123, 2, inp["page_table"].shape[1]), dtype=torch.uint8,
                     device="cuda")
    args = (inp["q"], inp["cu"], inp["pool"], inp["page_table"], inp["seq_lens"], out)
    M.mlra_prefill(hdl, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mlra_prefill(hdl, *args, workspace=ws)
    inp["q"].copy_(torch.randn_like(inp["q"]))
    inp["cu"].copy_(torch.tensor([0, 50, 123], dtype=torch.int32))
    inp["seq_lens"].copy_(torch.tensor([43, 80], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    ref, _, status = run(hdl, w, inp)
    assert status == 0 and torch.equal(got, ref)


@BOTH
def test_another_stream(form):
    w, inp = make(MLRA4, [33, 90], [10, 0], seed=13, form=form)
    hdl = handle(w, inp)
    ref, _, _ = run(hdl, w, inp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _, status = run(hdl, w, inp, stream=s)
    assert status == 0 and torch.equal(out, ref)


@BOTH
def test_status_of_bad_lengths_and_pages(form):
    """Bad device-side inputs that the kernels' own checks turn into a status."""
    w, inp = make(MLRA4, [33, 90], [10, 0], seed=14, form=form)
    hdl = handle(w, inp)
    good = run(hdl, w, inp)[0]
    bad = dict(inp, seq_lens=torch.tensor([43, 10 ** 6], dtype=torch.int32, device="cuda"))
    assert run(hdl, w, bad)[2] == -7
    for cu in ([0, 40, 33], [1, 33, 123], [0, 33, 400], [0, -5, 123]):
        bad = dict(inp, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        out, _, status = run(hdl, w, bad)
        assert status == -7 and out.isnan().all()
    pt = inp["page_table"].clone()
    pt[0, 0] = inp["pool"].shape[0]
    out, _, status = run(hdl, w, dict(inp, page_table=pt))
    assert status == -4
    assert torch.equal(run(hdl, w, inp)[0], good)


@BOTH
def test_a_replayed_graph_does_not_keep_an_earlier_status(form):
    """Bad lengths and pages in one replay are reported by that replay alone."""
    w, inp = make(MLRA4, [33, 90], [10, 0], seed=15, form=form)
    hdl = handle(w, inp)
    out = torch.empty(123, w.h, w.d_h, device="cuda")
    ws = torch.empty(M.mlra_prefill_workspace_size(hdl, 123, 2, inp["page_table"].shape[1]), dtype=torch.uint8,
                     device="cuda")
    args = (inp["q"], inp["cu"], inp["pool"], inp["page_table"], inp["seq_lens"], out)
    M.mlra_prefill(hdl, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mlra_prefill(hdl, *args, workspace=ws)

    def replay():
        graph.replay()
        return int(ws[:4].view(torch.int32)[0])

    assert replay() == 0
    good = out.clone()
    inp["seq_lens"][1] = 10 ** 6
    assert replay() == -7
    inp["seq_lens"][1] = 90
    assert replay() == 0 and torch.equal(out, good)
    page = int(inp["page_table"][0, 0])
    inp["page_table"][0, 0] = inp["pool"].shape[0]
    assert replay() == -4
    inp["page_table"][0, 0] = page
    assert replay() == 0 and torch.equal(out, good)


@BOTH
def test_offsets_past_32_bits(form):
    """More than 2^32 query and packed-query bytes and 2^31 result elements, a pool of more than 2^32
    bytes: the last sequences, whose pages lie at the pool's end, against a call of their own."""
    n, tail = 2200, 3
    w, inp = make(MLRA4, [64] * tail, [0] * tail, seed=16, form="heads")
    hdl = handle(w, inp)
    ref, ref_lse, status = run(hdl, w, inp)
    check(w, inp, ref, ref_lse, status, "alone")
    small = inp["pool"]
    pages = 60000
    pool = torch.zeros(pages, *small.shape[1:], dtype=small.dtype, device="cuda")
    pool[-small.shape[0]:] = small
    table = torch.zeros(n, 1 if form == "heads" else 5, dtype=torch.int32, device="cuda")
    table[-tail:, 0] = inp["page_table"][:, 0] + (pages - small.shape[0])
    lens = torch.full((n,), 64, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, 64 * n + 1, 64, dtype=torch.int32, device="cuda")
    q = torch.zeros(64 * n, w.h, w.d_h + w.d_r, dtype=torch.bfloat16, device="cuda")
    q[-64 * tail:] = inp["q"]
    out = torch.full((64 * n, w.h, w.d_h), float("nan"), dtype=torch.float32, device="cuda")
    lse = torch.full((64 * n, w.h), float("nan"), device="cuda")
    assert q.nbytes > 2 ** 32 and out.numel() > 2 ** 31 and pool.nbytes > 2 ** 32
    ws = M.mlra_prefill(hdl, q, cu, pool, table, lens, out, lse)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    check(w, inp, out[-64 * tail:], lse[-64 * tail:], 0, "behind others")
    assert not out[:64].any() and not out[64 * 1000:64 * 1001].any()
