"""The attention block's tensor helpers on the host: fake CUDA tensors and a stub in place of the library, so that
what a call passes, and what is still alive while it runs, can be looked at without a GPU."""
import weakref

import pytest
import torch

import blockwise_fp8_gemm_act_amd as puro
from blockwise_fp8_gemm_act_amd import _attention

NEED = 4096           # bytes of workspace that every stub call asks for


class Cuda(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = property(lambda self: True)


def fake(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Cuda)


class Library:
    """Records each call's arguments and hands them to `during` while the call runs."""

    def __init__(self, during):
        self.calls, self.during = [], during

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_bytes"):
                return NEED
            self.calls.append((name, args))
            self.during(name, args)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    made = []

    def empty(shape, dtype, device):
        t = fake(tuple(shape), dtype)
        made.append((t.data_ptr(), t.numel() * t.element_size(), weakref.ref(t)))
        return t

    def during(name, args):
        lib.alive = [(at, size) for at, size, ref in made if ref() is not None]

    lib = Library(during)
    monkeypatch.setattr(puro, "empty", empty)
    monkeypatch.setattr(_attention, "_lib", lib)
    monkeypatch.setattr(_attention, "_current", lambda index: 0)
    return lib


def attention(**k):
    return puro.attention(fake((5, 4, 64)), fake((9, 2, 64)), fake((9, 2, 64)), **k)


def attention_backward(**k):
    q, kv, lse = fake((5, 4, 64)), fake((9, 2, 64)), fake((4, 5), torch.float32)
    return puro.attention_backward(q, q, kv, kv, q, lse, **k)


def norm_backward(**k):
    w, table = fake((64,)), fake((8, 2, 32), torch.float32)
    return puro.qk_norm_rope_backward(fake((5, 4, 64)), fake((5, 2, 64)), fake((5, 512)), w, w, table, **k)


@pytest.mark.parametrize("call", [attention, attention_backward, norm_backward])
def test_a_new_workspace_lives_until_the_kernels_are_enqueued(library, call):
    """Released earlier, its memory could go to another thread's work on the same stream between a call's kernels, or
    be unmapped before they run."""
    call()
    name, args = library.calls[-1]
    at, size = args[-3:-1]
    assert size == NEED and (at, size) in library.alive, name


@pytest.mark.parametrize("call", [attention, attention_backward, norm_backward])
def test_the_callers_workspace_is_passed(library, call):
    ws = fake((3 * NEED,), torch.uint8)
    call(workspace=ws)
    assert library.calls[-1][1][-3:-1] == (ws.data_ptr(), 3 * NEED)
    with pytest.raises(ValueError):
        call(workspace=torch.zeros(NEED, dtype=torch.uint8))
