"""Page operators on the GPU against the host model, value for value (they move whole numbers and
bytes: nothing is rounded)."""
import random

import numpy as np
import pytest
import torch

import rank_latent_kv_mlra_b200 as M
import workloads as W
from tests.pages_model import PagesModel, pages_of

pytestmark = pytest.mark.gpu

TINY = W.WORKLOADS["mlra4_h8_b1_n256_f32"]      # 288-byte rows
MLRA4 = W.WORKLOADS["mlra4_h128_b32_n8192"]     # 1152-byte rows
E4M3 = W.WORKLOADS["mlra4fp8_h128_b32_n8192"]   # 576-byte rows


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    M.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """The device state and the model's, moved together and compared after every operator."""

    def __init__(self, w, num_pages, rows, stride, seed=0):
        shape = (w.h, w.d_b, w.d_h)
        wt = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        fp8 = dict(cache_fp8=True) if w.cache == "e4m3" else {}
        self.handle = M.mlra_create(w.h, w.d_h, w.d_c, w.d_r, w.k, wt, wt, **fp8)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        width = w.d_c + w.d_r
        raw = torch.randint(0, 256, (num_pages, 64, width * (1 if fp8 else 2)), generator=g, device="cuda",
                            dtype=torch.uint8)
        self.pool = raw if fp8 else raw.view(torch.bfloat16)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, stride), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.model = PagesModel(self.refs.cpu().numpy(), self.table.cpu().numpy(), self.lens.cpu().numpy(),
                                self.pool.view(torch.uint8).cpu().numpy())
        self.state = (self.refs, self.table, self.lens)

    def compare(self, ws, want):
        torch.cuda.synchronize()
        assert M.mlra_get_status(ws) == want
        assert np.array_equal(self.refs.cpu().numpy(), self.model.refs)
        assert np.array_equal(self.table.cpu().numpy(), self.model.table)
        assert np.array_equal(self.lens.cpu().numpy(), self.model.lens)
        assert np.array_equal(self.pool.view(torch.uint8).cpu().numpy(), self.model.pool)
        assert self.model.consistent()

    def reserve(self, ids, lens):
        ws = M.mlra_reserve_pages(self.handle, *self.state, i32(ids), i32(lens))
        want = self.model.reserve(ids, lens)
        self.compare(ws, want)
        return want

    def fork(self, src, dst):
        ws = M.mlra_fork_pages(self.handle, self.pool, *self.state, i32(src), i32(dst))
        want = self.model.fork(src, dst)
        self.compare(ws, want)
        return want

    def free(self, ids):
        ws = M.mlra_free_pages(self.handle, *self.state, i32(ids))
        want = self.model.free(ids)
        self.compare(ws, want)
        return want

    def compact(self):
        used = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        ws = M.mlra_compact_pages(self.handle, self.pool, *self.state, used)
        want = self.model.compact()
        self.compare(ws, 0)
        assert int(used) == want


@pytest.mark.parametrize("w,num_pages,rows,stride", [
    (TINY, 1, 1, 1), (TINY, 31, 5, 9), (TINY, 1000, 40, 33), (MLRA4, 300, 16, 40), (E4M3, 257, 12, 30),
    (TINY, 8192, 12, 1500), (TINY, 8193, 12, 1500), (TINY, 20000, 30, 900),
], ids=["one_page", "31", "1000", "mlra4", "e4m3", "one_stretch", "stretch_and_one", "three_stretches"])
def test_a_random_run_of_operators(w, num_pages, rows, stride):
    rng = random.Random(num_pages)
    both = Both(w, num_pages, rows, stride, seed=num_pages)
    seen = set()
    for step in range(60 if num_pages < 5000 else 25):
        live = [r for r in range(rows) if both.model.lens[r]]
        empty = [r for r in range(rows) if not both.model.lens[r]]
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        if op == "reserve":
            ids = rng.sample(range(rows), rng.randint(1, rows))
            cap = stride * 64
            lens = [min(cap, int(both.model.lens[i]) + rng.choice([0, 1, 63, 64, 65, rng.randint(0, cap)])) for i in ids]
            seen.add(("reserve", both.reserve(ids, lens)))
        elif op == "fork" and live and empty:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            seen.add(("fork", both.fork([rng.choice(live) for _ in dst], dst)))
        elif op == "free":
            both.free(rng.sample(range(rows), rng.randint(1, max(1, rows // 2))))
        elif op == "compact":
            both.compact()
    if num_pages >= 31:
        assert ("reserve", 0) in seen and ("fork", 0) in seen


def test_refused_requests_change_nothing():
    both = Both(TINY, 40, 6, 8, seed=1)
    assert both.reserve([0, 1, 2], [100, 64, 512]) == 0
    assert both.reserve([0, 0], [101, 102]) == -7          # the same row twice
    assert both.reserve([3, 6], [1, 1]) == -7              # a row outside the table
    assert both.reserve([3, -1], [1, 1]) == -7
    assert both.reserve([0], [99]) == -7                   # shorter than it is
    assert both.reserve([3], [8 * 64 + 1]) == -7           # longer than its row
    assert both.fork([0, 1], [3, 3]) == -7
    assert both.fork([0], [1]) == -7                       # onto a row in use
    assert both.fork([4], [4]) == -7                       # onto itself
    assert both.fork([0, 3], [3, 4]) == -7                 # a destination that is a source
    assert both.fork([9], [3]) == -7
    assert both.free([1, 1]) == -7
    assert both.free([6]) == -7
    assert both.free([3, 1]) == 0                          # an empty row may be freed
    assert both.reserve([1, 3, 4, 5], [512, 512, 512, 512]) == -10
    assert both.reserve([1, 3, 4], [512, 512, 512]) == 0
    assert both.reserve([5], [512]) == -10


def test_forks_of_one_source_and_of_an_empty_one():
    both = Both(MLRA4, 100, 20, 8, seed=2)
    both.reserve([7], [200])
    assert both.fork([7] * 10, list(range(8, 18))) == 0
    assert both.fork([0], [1]) == 0                        # nothing to share
    both.free([7])
    both.compact()
    both.free(list(range(8, 18)))
    assert not both.refs.any()


def test_no_requests():
    both = Both(TINY, 40, 6, 8, seed=3)
    assert both.reserve([], []) == 0 and both.fork([], []) == 0 and both.free([]) == 0
    both.compact()


def test_full_pool_and_many_rows():
    both = Both(TINY, 700, 700, 2, seed=4)
    assert both.reserve(list(range(700)), [64] * 700) == 0
    both.compact()
    assert both.reserve([3], [65]) == -10
    both.free(list(range(0, 700, 3)))
    both.compact()
    assert both.fork([1] * 200, list(range(0, 600, 3))) == 0


def test_large_pool_without_its_contents():
    """300,000 pages (37 stretches of the bitmap), counts and tables only."""
    P, R, S = 300000, 200, 1500
    both = Both(TINY, 1, 1, 1)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((R, S), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    model = PagesModel(refs.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy())
    rng = random.Random(7)
    for step in range(6):
        ids = rng.sample(range(R), 120)
        new = [rng.randint(int(model.lens[i]), S * 64) for i in ids]
        ws = M.mlra_reserve_pages(both.handle, refs, table, lens, i32(ids), i32(new))
        assert M.mlra_get_status(ws) == model.reserve(ids, new)
        gone = rng.sample(range(R), 60)
        ws = M.mlra_free_pages(both.handle, refs, table, lens, i32(gone))
        assert M.mlra_get_status(ws) == model.free(gone)
        assert np.array_equal(refs.cpu().numpy(), model.refs) and np.array_equal(table.cpu().numpy(), model.table)
        assert np.array_equal(lens.cpu().numpy(), model.lens)


def test_refused_arguments():
    both = Both(TINY, 40, 6, 8, seed=8)
    with pytest.raises(ValueError, match="one length"):
        M.mlra_reserve_pages(both.handle, *both.state, i32([1, 2]), i32([5]))
    with pytest.raises(M.MlraError, match="INVALID_ARG"):   # more requests than rows
        M.mlra_free_pages(both.handle, *both.state, i32([0] * 7))
    with pytest.raises(ValueError, match="pool must be"):
        M.mlra_compact_pages(both.handle, both.pool[:39], *both.state)
    with pytest.raises(TypeError, match="refs"):
        M.mlra_free_pages(both.handle, both.refs.long(), both.table, both.lens, i32([0]))
    ws = torch.empty(M.mlra_pages_workspace_size(both.handle, 40, 6) - 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(M.MlraError, match="WORKSPACE"):
        M.mlra_free_pages(both.handle, *both.state, i32([0]), workspace=ws)


def test_bad_table_entries_are_passed_over():
    both = Both(TINY, 40, 6, 8, seed=5)
    both.reserve([0, 1], [200, 200])
    refs = both.refs.clone()
    both.table[0, 1] = 40
    ws = M.mlra_free_pages(both.handle, *both.state, i32([0]))
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == -4
    assert both.refs.tolist() == [0, 1, 0, 0] + refs.tolist()[4:]  # page 1's entry was overwritten
    both.table[1, 3] = -5                                           # the partly filled last page
    ws = M.mlra_fork_pages(both.handle, both.pool, *both.state, i32([1]), i32([2]))
    torch.cuda.synchronize()
    assert M.mlra_get_status(ws) == -4


def test_captured_turn_replays():
    both = Both(MLRA4, 200, 12, 8, seed=6)
    both.reserve([0, 1, 2, 3], [100, 200, 300, 64])
    ids, lens, src, dst = i32([0, 1]), i32([100, 200]), i32([2, 3]), i32([5, 6])
    gone = i32([5, 6])
    ws = torch.empty(M.mlra_pages_workspace_size(both.handle, 200, 12), dtype=torch.uint8, device="cuda")

    def turn():
        M.mlra_free_pages(both.handle, *both.state, gone, workspace=ws)
        M.mlra_reserve_pages(both.handle, *both.state, ids, lens, workspace=ws)
        M.mlra_fork_pages(both.handle, both.pool, *both.state, src, dst, workspace=ws)

    def model(l):
        both.model.free([5, 6])
        both.model.reserve([0, 1], l)
        both.model.fork([2, 3], [5, 6])

    turn()
    model([100, 200])
    both.compare(ws, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for step in range(1, 4):
        lens.copy_(i32([100 + 40 * step, 200 + step]))
        graph.replay()
        model([100 + 40 * step, 200 + step])
        both.compare(ws, 0)
