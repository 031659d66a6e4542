"""Softmax and output scales of a handle, in the prompt and prefix calls: a power of two moved from the
queries to the scale, or from one output scale to another, changes no bit but the exponents."""
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def setup(name, batch):
    w = W.scaled(W.WORKLOADS[name], batch=batch, seq_len=None, len_range=(100, 300), seed=95)
    inp = W.make_workload(w, device="cuda")
    return w, inp, lambda **kw: M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, inp["w_uk"], inp["w_uv"],
                                              blocks_summed=w.summed, **kw)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prompt(w, inp, hdl, q, few):
    n = q.shape[0]
    out = torch.empty(n, w.h, w.d_h, device="cuda")
    lse = torch.empty(n, w.h * (w.k if w.summed else 1), device="cuda")
    table, lens = inp["page_table"], inp["seq_lens"]
    if not few:                 # whole prompts' form: tables of at most four times the query tokens
        table = table[:, :n // 64].contiguous()
        lens = torch.minimum(lens, i32([64 * table.shape[1]]))
    ws = M.mlra_prefill(hdl, q, i32([0, n // 2, n]), inp["pool"], table, lens, out, lse)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    return out, lse


def prefix(w, inp, hdl, q, few):
    out = torch.empty(1, w.h, w.d_h, device="cuda")
    lse = torch.empty(1, w.h * (w.k if w.summed else 1), device="cuda")
    table, lens = inp["page_table"], inp["seq_lens"]
    ws = M.mlra_decode_prefix(hdl, q[:1], inp["pool"], table[:1].contiguous(), lens[:1].contiguous(), i32([0, 1]),
                              table[1:].contiguous(), lens[1:].contiguous(), out, lse)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("call", [prompt, prefix])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("name", ["mlra4_h128_b32_n8192", "mlra2_h128_b64_n4096", "mla_h128_b128_ragged1k_32k",
                                  "mlra4sum_h128_b32_n8192"])
def test_a_softmax_scale_of_the_callers(name, few, call):
    w, inp, make = setup(name, 2)
    q = torch.randn(20 if few else 340, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    scale = (w.d_h + w.d_r) ** -0.5
    want = call(w, inp, make(), q, few)
    same = call(w, inp, make(softmax_scale=scale), q, few)
    moved = call(w, inp, make(softmax_scale=2 * scale), q / 2, few)
    other = call(w, inp, make(softmax_scale=2 * scale), q, few)
    # (the default is a 32-bit quotient, this one a 64-bit one rounded once: they may differ by a step,
    # which moves a score, of a few units, by as many steps of 2^-23)
    assert torch.allclose(same[0], want[0], rtol=0, atol=1e-2) and torch.allclose(same[1], want[1], rtol=0, atol=1e-2)
    assert all(torch.equal(a, b) for a, b in zip(moved, same))
    assert not torch.equal(other[0], same[0])


@pytest.mark.parametrize("call", [prompt, prefix])
@pytest.mark.parametrize("name", ["mlra4sum_h128_b32_n8192", "mlra2sum_h128_b64_n4096"])
def test_an_output_scale_of_the_callers(name, call):
    w, inp, make = setup(name, 2)
    q = torch.randn(20, w.h, w.d_h + w.d_r, device="cuda").bfloat16()
    one, two = (call(w, inp, make(attn_scale=a), q, True) for a in (0.25, 0.5))
    assert torch.equal(2 * one[0], two[0]) and torch.equal(one[1], two[1])
