"""Calls on a stream that is not the current one, without a workspace of the caller's: what they take for
themselves must not be memory that work queued on the current stream still uses. A block that such work
is about to write and read is freed, and a call on another stream made at once: it must not be handed
that block, the queued work's result must be whole, and the call's own result the usual one."""
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W

pytestmark = pytest.mark.gpu

TINY = W.scaled(W.WORKLOADS["mlra4_h8_b1_n256_f32"], batch=3, seq_len=None, len_range=(100, 200), seed=70)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def behind_queued_work(size, call):
    """call(stream) -> its workspace, made while the current stream is busy and the block of `size`
    bytes that its queued work uses has been freed."""
    busy = torch.ones(4096, 4096, device="cuda")
    prod, kept = torch.empty_like(busy), torch.zeros(size, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    block = torch.empty(size, dtype=torch.uint8, device="cuda")
    lo = block.data_ptr()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(busy, busy, out=prod)
    block.fill_(7)
    kept.copy_(block)
    del block
    ws = call(stream)
    torch.cuda.synchronize()
    assert bool((kept == 7).all())
    assert ws.data_ptr() + ws.numel() <= lo or ws.data_ptr() >= lo + size
    assert M.mlra_get_status(ws) == 0


def _tiny():
    inp = W.make_workload(TINY, device="cuda")
    hdl = M.mlra_create(TINY.h, TINY.d_h, TINY.d_c, TINY.d_r, TINY.k, inp["w_uk"], inp["w_uv"])
    return inp, hdl


def test_prefill():
    inp, hdl = _tiny()
    table = inp["page_table"]
    q = torch.randn(70, TINY.h, TINY.d_h + TINY.d_r, device="cuda").bfloat16()
    out = torch.empty(70, TINY.h, TINY.d_h, device="cuda")
    args = (hdl, q, i32([0, 30, 31, 70]), inp["pool"], table, inp["seq_lens"], out)
    M.mlra_prefill(*args)
    want = out.clone()
    out.zero_()
    behind_queued_work(M.mlra_prefill_workspace_size(hdl, 70, 3, table.shape[1]),
                       lambda s: M.mlra_prefill(*args, stream=s))
    assert torch.equal(out, want)


def test_decode_prefix():
    inp, hdl = _tiny()
    table, lens = inp["page_table"], inp["seq_lens"]
    q = torch.randn(2, TINY.h, TINY.d_h + TINY.d_r, device="cuda").bfloat16()
    out = torch.empty(2, TINY.h, TINY.d_h, device="cuda")
    args = (hdl, q, inp["pool"], table[:1].contiguous(), lens[:1].contiguous(), i32([0, 2]), table[1:].contiguous(),
            lens[1:].contiguous(), out)
    M.mlra_decode_prefix(*args)
    want = out.clone()
    out.zero_()
    behind_queued_work(M.mlra_decode_prefix_workspace_size(hdl, 2, 1), lambda s: M.mlra_decode_prefix(*args, stream=s))
    assert torch.equal(out, want)


@pytest.mark.parametrize("latent", [False, True])
def test_decode(latent):
    inp, hdl = _tiny()
    fn = M.mlra_decode_latent if latent else M.mlra_decode
    out = torch.empty(3, TINY.h, TINY.d_c // TINY.k if latent else TINY.d_h, device="cuda")
    args = (hdl, inp["q"], inp["pool"], inp["page_table"], inp["seq_lens"], out)
    fn(*args)
    want = out.clone()
    out.zero_()
    behind_queued_work(M.mlra_workspace_size(hdl, 3), lambda s: fn(*args, stream=s))
    assert torch.equal(out, want)


def test_project_append():
    inp, hdl = _tiny()
    pr = W.make_producer_inputs(TINY, inp, d_model=256)
    args = (hdl, pr["x"], pr["w_down"], pr["positions"], inp["pool"], inp["page_table"])
    M.mlra_project_append(*args)
    want = inp["pool"].clone()
    inp["pool"].zero_()
    behind_queued_work(M.mlra_project_workspace_size(hdl, 3, 256), lambda s: M.mlra_project_append(*args, stream=s))
    for b, pos in enumerate(pr["positions"].tolist()):
        page = int(inp["page_table"][b, pos // 64])
        assert torch.equal(inp["pool"][page, pos % 64], want[page, pos % 64])


def test_plan():
    """The plan's rows are cleared, filled and read in the order of the call's stream."""
    inp, hdl = _tiny()
    stride = inp["page_table"].shape[1]
    want = M.mlra_plan(hdl, inp["seq_lens"], stride)
    assert want[1] > 0
    busy = torch.ones(4096, 4096, device="cuda")
    prod, stream = torch.empty_like(busy), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(busy, busy, out=prod)
    assert M.mlra_plan(hdl, inp["seq_lens"], stride, stream=stream) == want


def test_page_operators():
    inp, hdl = _tiny()
    P = inp["pool"].shape[0]
    refs, table, lens = i32([0] * P), i32([[-1] * 2] * 3), i32([0] * 3)
    state = (refs, table, lens)
    size = M.mlra_pages_workspace_size(hdl, P, 3)
    row, other, new = i32([1]), i32([2]), i32([70])
    behind_queued_work(size, lambda s: M.mlra_reserve_pages(hdl, *state, row, new, stream=s))
    assert table.tolist() == [[-1, -1], [0, 1], [-1, -1]]
    behind_queued_work(size, lambda s: M.mlra_fork_pages(hdl, inp["pool"], *state, row, other, stream=s))
    assert table.tolist() == [[-1, -1], [0, 1], [0, 2]] and lens.tolist() == [0, 70, 70]
    behind_queued_work(size, lambda s: M.mlra_free_pages(hdl, *state, row, stream=s))
    assert lens.tolist() == [0, 0, 70] and refs.tolist()[:3] == [1, 0, 1]
    behind_queued_work(size, lambda s: M.mlra_compact_pages(hdl, inp["pool"], *state, stream=s))
    assert table[2].tolist() == [0, 1] and refs.tolist()[:3] == [1, 1, 0]


def test_different_operators_at_once():
    """Decode, prompt (both forms and few tokens), prefix and page calls on streams and workspaces of their
    own, over one pool: the bits that each gives alone."""
    w = W.scaled(W.WORKLOADS["mlra4_h128_b32_n8192"], batch=6, seq_len=None, len_range=(500, 900), seed=71)
    inp = W.make_workload(w, device="cuda", extra_pages=40)
    hdl = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"])
    pool, table, lens = inp["pool"], inp["page_table"], inp["seq_lens"]
    q = torch.randn(1200, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    size = lambda n: torch.empty(n, w.h, w.d_h, device="cuda")
    P = 500
    refs, rows, row_lens = i32([0] * P), i32([[-1] * 40] * 9), i32([0] * 9)
    ids, new = i32([3, 1, 7]), i32([2000, 70, 2560])
    part = (table[:, :3].contiguous(), torch.clamp(lens, max=192))
    calls = [
        (M.mlra_decode, (hdl, q[:6], pool, table, lens), size(6), M.mlra_workspace_size(hdl, 6)),
        (M.mlra_prefill, (hdl, q, i32([0, 200, 400, 600, 800, 1000, 1200]), pool, *part), size(1200),
         M.mlra_prefill_workspace_size(hdl, 1200, 6, 3)),
        (M.mlra_prefill, (hdl, q[:100], i32([0, 10, 20, 30, 60, 99, 100]), pool, table, lens), size(100),
         M.mlra_prefill_workspace_size(hdl, 100, 6, table.shape[1])),
        (M.mlra_prefill, (hdl, q[:20], i32([0, 1, 2, 3, 10, 19, 20]), pool, table, lens), size(20),
         M.mlra_prefill_workspace_size(hdl, 20, 6, table.shape[1])),
        (M.mlra_decode_prefix, (hdl, q[:5], pool, table[:1].contiguous(), lens[:1].contiguous(), i32([0, 5]),
                                table[1:].contiguous(), lens[1:].contiguous()), size(5),
         M.mlra_decode_prefix_workspace_size(hdl, 5, 1)),
    ]
    workspaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for *_, n in calls]
    pages_ws = torch.empty(M.mlra_pages_workspace_size(hdl, P, 9), dtype=torch.uint8, device="cuda")
    want = []
    for (fn, args, out, _), ws in zip(calls, workspaces):
        fn(*args, out, workspace=ws)
        want.append(out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(len(calls) + 1)]
    for _ in range(20):
        for (fn, args, out, _), ws, s in zip(calls, workspaces, streams):
            fn(*args, out, workspace=ws, stream=s)
        M.mlra_reserve_pages(hdl, refs, rows, row_lens, ids, new, workspace=pages_ws, stream=streams[-1])
        M.mlra_free_pages(hdl, refs, rows, row_lens, ids, workspace=pages_ws, stream=streams[-1])
    torch.cuda.synchronize()
    for (_, _, out, _), ws, ref in zip(calls, workspaces, want):
        assert M.mlra_get_status(ws) == 0 and torch.equal(out, ref)
    assert M.mlra_get_status(pages_ws) == 0 and not refs.any() and not row_lens.any()
