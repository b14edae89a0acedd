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


@pytest.mark.parametrize("tokens", [0, 1])
def test_one_tokens_strides_mean_nothing(library, tokens):
    """Slices of rows of any length, also past the longest distance between tokens, where there is no second token."""
    def part(heads, at, width):
        return torch.zeros(at + heads * 64, dtype=torch.bfloat16)[at:].as_strided((tokens, heads, 64), (width, 64, 1)).as_subclass(Cuda)

    q, k, v, o, do = part(4, 8, 512), part(2, 16, 1 << 24), part(2, 24, 7), part(4, 0, 256), part(4, 32, 1 << 30)
    lse = fake((4, tokens), torch.float32)
    puro.attention(q, k, v, out=o)
    puro.attention_backward(do, q, k, v, o, lse)
    assert [n for n, _ in library.calls] == ["puro_attention", "puro_attention_backward"]
    for _, args in library.calls:
        a = args[0]
        assert (a.q_stride, a.k_stride, a.v_stride, a.o_stride) == (256, 128, 128, 256)
    x = torch.zeros(512, dtype=torch.bfloat16).as_strided((tokens, 512), (1 << 25, 1)).as_subclass(Cuda)
    w, table = fake((64,)), fake((8, 2, 32), torch.float32)
    puro.qk_norm_rope(x, w, w, table, q_heads=4, k_heads=2)
    assert library.calls[-1][1][2] == 384


def test_several_tokens_keep_their_strides(library):
    q, kv, lse = fake((5, 6, 64))[:, 1:5], fake((9, 2, 64)), fake((4, 5), torch.float32)
    puro.attention_backward(q, q, kv, kv, q, lse)
    a = library.calls[-1][1][0]
    assert (a.q_stride, a.k_stride, a.o_stride, a.dq_stride) == (384, 128, 384, 256)
    with pytest.raises(ValueError):
        puro.attention_backward(fake((5, 4, 64)), q, kv, kv, q, lse)
