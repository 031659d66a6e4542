"""Device memory that a call takes for itself comes from the pool of the stream it runs on (no GPU: the
library and torch's stream context are stood in for, and the calls' own allocations recorded). A block
of the current stream's pool may still be in use by work queued there, which the other stream does not
wait for."""
import contextlib

import pytest
import torch

import rank_latent_kv_mlra_b200 as M


class _Lib:
    def __getattr__(self, name):
        return lambda *a: 0


class _Handle:
    ptr = None
    cfg = M.mlra_config(128, 128, 512, 64, 4, 64)


class _Stream:
    cuda_stream = 0


class _Event:
    cuda_event = 1


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


Q, POOL, OUT = bf16(3, 128, 192), bf16(4, 64, 576), bf16(3, 128, 128)
LENS = i32(3)
CALLS = {
    "mlra_prefill": (Q, i32(2), POOL, i32(1, 4), i32(1), OUT),
    "mlra_decode_prefix": (Q, POOL, i32(1, 4), i32(1), i32(2), i32(3, 4), i32(3), OUT),
    "mlra_decode": (Q, POOL, i32(3, 4), i32(3), OUT),
    "mlra_decode_latent": (Q, POOL, i32(3, 4), i32(3), torch.zeros(3, 128, 128)),
    "mlra_decode_profiled": (Q, POOL, i32(3, 4), i32(3), OUT, [_Event()] * 4),
    "mlra_project_append": (bf16(3, 128), bf16(576, 128), i32(3), POOL, i32(3, 4)),
}


@pytest.fixture
def taken(monkeypatch):
    """The stream (None: the current one) in whose context each allocation was made."""
    current, where = [None], []

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    def record(fn):
        def call(*a, **kw):
            where.append(current[-1])
            kw.pop("device", None)
            return fn(*a, **kw)
        return call

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", record(torch.empty))
    monkeypatch.setattr(torch, "zeros", record(torch.zeros))
    monkeypatch.setattr(M, "load_library", lambda: _Lib())
    monkeypatch.setattr(M, "_require", lambda *a: None)
    monkeypatch.setattr(M, "_call", lambda *a: None)
    monkeypatch.setattr(M, "_stream", lambda stream: None)
    return where


@pytest.mark.parametrize("name", list(CALLS))
def test_workspaces_belong_to_the_call_s_stream(taken, name):
    getattr(M, name)(_Handle, *CALLS[name], stream=None)
    assert taken == [None]
    stream = _Stream()
    getattr(M, name)(_Handle, *CALLS[name], stream=stream)
    assert taken == [None, stream]


def test_page_workspaces_belong_to_the_call_s_stream(taken):
    """(The page operators' own checks refuse host tensors: the function they take the workspace from.)"""
    stream = _Stream()
    M._new_workspace(16, torch.device("cpu"), stream)
    M._new_workspace(16, torch.device("cpu"), None)
    assert taken == [stream, None]


def test_the_plan_is_cleared_and_read_on_the_call_s_stream(taken):
    stream, lens = _Stream(), LENS
    M.mlra_plan(_Handle, lens, 4, stream=stream)
    M.mlra_plan(_Handle, lens, 4)
    assert taken == [stream, stream, None, None]
