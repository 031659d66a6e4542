"""Host-side checks of the prompt, shared-prefix and page operators (no GPU: they return before any
CUDA call), and the page model the GPU tests compare with."""
import ctypes
import random

import numpy as np
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
from rank_latent_kv_mlra_b200 import build
from tests.pages_model import PagesModel, pages_of


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load_library()


def test_null_handles_are_refused(lib):
    n = ctypes.c_size_t()
    assert lib.mlra_prefill_workspace_size(None, 4, 1, 1, ctypes.byref(n)) == -1
    assert lib.mlra_decode_prefix_workspace_size(None, 4, 1, ctypes.byref(n)) == -1
    assert lib.mlra_pages_workspace_size(None, 4, 1, ctypes.byref(n)) == -1
    P = ctypes.c_void_p
    assert lib.mlra_prefill(None, P(16), 1, P(16), 1, P(16), 1, P(16), 1, P(16), 1, P(16), 1, None, P(256), 1, None) == -1
    assert lib.mlra_decode_prefix(None, P(16), 1, P(16), 1, P(16), 1, P(16), P(16), 1, P(16), 1, P(16), 1, P(16), 1,
                                  None, P(256), 1, None) == -1
    assert lib.mlra_reserve_pages(None, P(16), 1, P(16), 1, 1, P(16), P(16), P(16), 1, P(256), 1, None) == -1
    assert lib.mlra_fork_pages(None, P(16), P(16), 1, P(16), 1, 1, P(16), P(16), P(16), 1, P(256), 1, None) == -1
    assert lib.mlra_free_pages(None, P(16), 1, P(16), 1, 1, P(16), P(16), 1, P(256), 1, None) == -1
    assert lib.mlra_compact_pages(None, P(16), P(16), 1, P(16), 1, 1, P(16), None, P(256), 1, None) == -1


def test_new_status_code_has_a_name(lib):
    assert M.STATUS[-10] == "MLRA_ERR_NO_PAGES"
    assert "free pages" in M.mlra_status_string(-10)


class _Handle:
    ptr = None
    cfg = M.mlra_config(128, 128, 512, 64, 4, 64)


def test_host_tensors_are_refused(lib):
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
    q, out = z(3, 128, 192, dt=torch.bfloat16), z(3, 128, 128, dt=torch.bfloat16)
    pool = z(4, 64, 576, dt=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.mlra_prefill(_Handle, q, z(2), pool, z(1, 4), z(1), out)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.mlra_decode_prefix(_Handle, q, pool, z(1, 4), z(1), z(2), z(3, 4), z(3), out)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.mlra_free_pages(_Handle, z(4), z(1, 4), z(1), z(1))


def test_the_model_keeps_its_counts():
    rng = random.Random(0)
    m = PagesModel(np.zeros(50, dtype=np.int32), np.full((10, 7), -1, dtype=np.int32), np.zeros(10, dtype=np.int32),
                   np.arange(50 * 64).reshape(50, 64, 1).astype(np.int32))
    for _ in range(300):
        live, empty = [r for r in range(10) if m.lens[r]], [r for r in range(10) if not m.lens[r]]
        op = rng.randrange(4)
        before = {r: m.pool[m.table[r, :pages_of(m.lens[r])]].reshape(-1, 1)[:m.lens[r]].copy() for r in live}
        if op == 0:
            ids = rng.sample(range(10), 3)
            m.reserve(ids, [min(448, m.lens[i] + rng.randint(0, 200)) for i in ids])
        elif op == 1 and live and empty:
            src = rng.choice(live)
            if m.fork([src], [empty[0]]) == 0:
                assert np.array_equal(m.pool[m.table[empty[0], :pages_of(m.lens[src])]].reshape(-1, 1)[:m.lens[src]],
                                      before[src])
        elif op == 2:
            m.free(rng.sample(range(10), 2))
        else:
            used = m.compact()
            assert not m.refs[used:].any() and (m.refs[:used] > 0).all()
            for r in live:                                  # every sequence reads what it read before
                assert np.array_equal(m.pool[m.table[r, :pages_of(m.lens[r])]].reshape(-1, 1)[:m.lens[r]], before[r])
        assert m.consistent()
