"""The operators together as a serving loop uses them: reserve pages, append a prompt's rows, attend
over the prompt, fork samples, decode them (each on its own, and as one shared prefix), free,
compact. Every attention result is checked against float64 on the host's own copy of the rows."""
import numpy as np
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W
from oracle import mlra_oracle as O
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def oracle(w, q, w_uk, w_uv, rows):
    """Heads' outputs [h][d_h] of one query over cached rows (numpy float64)."""
    out, _, _ = O.decode_heads(q.double().cpu().numpy(), w_uk.double().cpu().numpy(), w_uv.double().cpu().numpy(),
                               rows.double().cpu().numpy(), list(range(w.h)), w.k, w.d_r)
    return np.stack(out)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_prompt_fork_decode_compact(cache):
    w = W.scaled(W.WORKLOADS["mlra4_h128_b32_n8192"], cache=cache)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    w_uk = (randn(w.h, w.d_b, w.d_h) / w.d_b ** 0.5).bfloat16()
    w_uv = (randn(w.h, w.d_b, w.d_h) / w.d_b ** 0.5).bfloat16()
    fp8 = dict(cache_fp8=True, latent_scale=W.E4M3_SCALE, rope_scale=W.E4M3_SCALE) if cache == "e4m3" else {}
    hdl = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, w_uk, w_uv, **fp8)
    P, R, S = 80, 8, 12
    pool = torch.full((P, 64, w.d_c + w.d_r), float("nan"), device="cuda").bfloat16()
    if fp8:
        pool = torch.full((P, 64, w.d_c + w.d_r), 0x7F, dtype=torch.uint8, device="cuda")
    refs, table, lens = i32([0] * P), i32([[-1] * S] * R), i32([0] * R)
    state = (refs, table, lens)
    kept = {}                                   # row -> the values its cached rows stand for

    def value(rows):
        if fp8:
            return (rows.float() / W.E4M3_SCALE).to(torch.float8_e4m3fn).float() * W.E4M3_SCALE
        return rows.bfloat16().float()

    def append(row, n):
        new = randn(n, w.d_c + w.d_r)
        old = len(kept[row]) if row in kept else 0
        M.mlra_reserve_pages(hdl, *state, i32([row]), i32([old + n]))
        M.mlra_append_cache(hdl, pool, table, i32([row] * n), torch.arange(old, old + n, dtype=torch.int32, device="cuda"),
                            new[:, :w.d_c].contiguous(), new[:, w.d_c:].contiguous())
        kept[row] = torch.cat([kept[row], value(new)]) if row in kept else value(new)

    def decode(rows):
        q = randn(len(rows), w.h, w.d_h + w.d_r).bfloat16()
        out = torch.empty(len(rows), w.h, w.d_h, device="cuda")
        M.mlra_decode(hdl, q, pool, table[rows].contiguous(), lens[rows].contiguous(), out)
        torch.cuda.synchronize()
        for i, r in enumerate(rows):
            G.assert_parity(out[i].cpu().numpy(), oracle(w, q[i], w_uk, w_uv, kept[r]), f"decode row {r}")
        return q

    # two prompts, attended to in one packed call
    append(2, 150)
    append(5, 333)
    q = randn(483, w.h, w.d_h + w.d_r).bfloat16()
    out = torch.empty(483, w.h, w.d_h, device="cuda")
    ws = M.mlra_prefill(hdl, q, i32([0, 150, 483]), pool, table[[2, 5]].contiguous(), lens[[2, 5]].contiguous(), out)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    for t in (0, 1, 63, 64, 149):
        G.assert_parity(out[t].cpu().numpy(), oracle(w, q[t], w_uk, w_uv, kept[2][:t + 1]), f"prompt token {t}")
    for t in (0, 130, 332):
        G.assert_parity(out[150 + t].cpu().numpy(), oracle(w, q[150 + t], w_uk, w_uv, kept[5][:t + 1]), f"token {t}")

    # three samples of the second prompt, which then go their own ways
    ws = M.mlra_fork_pages(hdl, pool, *state, i32([5, 5, 5]), i32([0, 1, 7]))
    for r in (0, 1, 7):
        kept[r] = kept[5]
    for r, n in ((0, 3), (1, 70), (7, 1), (5, 20)):
        append(r, n)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    decode([0, 1, 2, 5, 7])

    # free some, compact, and read the rest again
    M.mlra_free_pages(hdl, *state, i32([2, 0]))
    used = i32([0])
    M.mlra_compact_pages(hdl, pool, *state, used)
    torch.cuda.synchronize()
    assert int(used) == int((refs > 0).sum()) and int((refs[int(used):] != 0).sum()) == 0
    decode([1, 5, 7])

    if fp8:
        return
    # the same samples as one shared prefix (row 5's first 320 tokens: whole pages) and their own rows
    pre = table[5:6, :5].contiguous()
    own = table[[1, 5, 7], 5:].contiguous()
    own_lens = lens[[1, 5, 7]] - 320
    q = randn(3, w.h, w.d_h + w.d_r).bfloat16()
    out = torch.empty(3, w.h, w.d_h, device="cuda")
    ws = M.mlra_decode_prefix(hdl, q, pool, pre, i32([320]), i32([0, 3]), own, own_lens.contiguous(), out)
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == 0
    for i, r in enumerate((1, 5, 7)):
        G.assert_parity(out[i].cpu().numpy(), oracle(w, q[i], w_uk, w_uv, kept[r]), f"shared prefix row {r}")
