"""The kernel for many queries on the GPU: each number of heads a workgroup takes, long walks, windows, caches; offsets past 32
bits and starts out of range through every kernel.  tests/test_attention_plan.py holds the shapes to their kernel."""
import math

import pytest
import torch

import attention_plan as ap
import attention_reference as ref
from attention_reference import U, f64

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lengths):
    return ints([sum(lengths[:i]) for i in range(len(lengths) + 1)])


def check_heads(q, k, v, got, seqs, window, sinks, scale=None):
    """Some query heads against the 64-bit form: the first and last of a workgroup and of all."""
    qh, kh = q.shape[1], k.shape[1]
    for h in sorted({0, 1, qh // 2, qh - 1}):
        g = h * kh // qh
        want = ref.attention(q[:, h:h + 1], k[:, g:g + 1], v[:, g:g + 1], seqs, window, sinks, scale, bounds=True)
        ref.check(got[0][:, h:h + 1], want["o"], want["b_o"], "o of head %d" % h)
        ref.check(got[1][h:h + 1], want["lse"], want["b_lse"], "lse of head %d" % h)


@pytest.mark.parametrize("case", ap.MANY, ids=str)
def test_long_walks(case):
    qh, kh, hd, _, ql, kl, window, sinks = case
    q, k, v = normal((sum(ql), qh, hd), 1), normal((sum(kl), kh, hd), 2), normal((sum(kl), kh, hd), 3)
    got = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    check_heads(q, k, v, got, [(sum(ql[:i]), ql[i], sum(kl[:i]), kl[i]) for i in range(len(ql))], window, sinks)


@pytest.mark.parametrize("case", [c for c in ap.MANY if sum(c[4]) > sum(c[5])], ids=str)
def test_rows_that_see_nothing(case):
    qh, kh, hd, _, ql, kl, window, sinks = case
    q, k, v = normal((sum(ql), qh, hd), 1), normal((sum(kl), kh, hd), 2), normal((sum(kl), kh, hd), 3)
    for i, (n, m) in enumerate(zip(ql, kl)):
        q[sum(ql[:i]):sum(ql[:i]) + n - m] = float("nan")
    o, lse = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    for i, (n, m) in enumerate(zip(ql, kl)):
        gone = slice(sum(ql[:i]), sum(ql[:i]) + n - m)
        assert not bool(o[gone].any()) and bool((lse[:, gone] == -math.inf).all())
        assert bool(o[gone.stop:sum(ql[:i + 1])].isfinite().all())


@pytest.mark.parametrize("at,by", [(0, 40.0), (63, 400.0), (64, 4000.0), (1000, 400.0), (2099, 4000.0)])
@pytest.mark.parametrize("case", [c for c in ap.MANY if c[4] == [2100] and not c[6]], ids=str)
def test_a_score_that_outgrows_the_others(case, at, by):
    """One key far above all before and after it, up to where exp(s - running maximum) leaves fp32."""
    qh, kh, hd, _, ql, kl, _, _ = case
    q, k, v = normal((ql[0], qh, hd), 16, 0.1), normal((kl[0], kh, hd), 17, 0.1), normal((kl[0], kh, hd), 18)
    q[:, :, 0] = 1.0
    k[at, :, 0] = by
    got = puro.attention(q, k, v, scale=1.0)
    check_heads(q, k, v, got, [(0, ql[0], 0, kl[0])], 0, 0, scale=1.0)


@pytest.mark.parametrize("case", ap.MANY_CACHED, ids=str)
def test_prompts_over_a_cache(case):
    """Rows past the keys in use and keys that left every query's window hold NaN."""
    qh, kh, hd, _, ql, kl, room, window, sinks = case
    n = len(ql)
    q, k, v = normal((sum(ql), qh, hd), 4), normal((room * n, kh, hd), 5), normal((room * n, kh, hd), 6)
    for s in range(n):
        k[s * room + kl[s]:(s + 1) * room] = v[s * room + kl[s]:(s + 1) * room] = float("nan")
        if window:
            gone = slice(s * room + sinks, s * room + max(sinks, kl[s] - ql[s] - window + 1))
            k[gone] = v[gone] = float("nan")
    got = puro.attention(q, k, v, starts(ql), starts([room] * n), ints(kl), window=window, sinks=sinks, max_k=max(kl))
    check_heads(q, k, v, got, [(sum(ql[:s]), ql[s], s * room, kl[s]) for s in range(n)], window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_offsets_past_32_bits(window, sinks):
    """A sequence past the 2^32nd element of queries, keys, values and their gradients, forward and backward."""
    stride, qh, kh, hd, n = 4096, 16, 8, 128, 700
    room = (1 << 32) // stride + 1000
    at = room - n - 5
    big, big_do = (torch.empty(room, stride, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big[at:at + n] = normal((n, stride), 7)
    big_do[at:at + n] = normal((n, stride), 8, 1e-3)
    heads = big.view(room, -1, hd)
    q, k, v = heads[:, :qh], heads[:, qh:qh + kh], heads[:, qh + kh:]
    do = big_do.view(room, -1, hd)[:, :qh]
    place = ints([at, at + n])
    kw = dict(window=window, sinks=sinks)
    out = torch.empty(room, stride, dtype=torch.bfloat16, device="cuda").view(room, -1, hd)[:, :qh]
    o, lse = puro.attention(q, k, v, place, place, out=out, **kw)
    rows = slice(at, at + n)
    check_heads(q[rows], k[rows], v[rows], (o[rows], lse[:, rows]), [(0, n, 0, n)], window, sinks)
    grads = torch.empty(room, stride, dtype=torch.bfloat16, device="cuda").view(room, -1, hd)
    dq, dk, dv = grads[:, :qh], grads[:, qh:qh + kh], grads[:, qh + kh:]
    puro.attention_backward(do, q, k, v, o, lse, place, place, dq=dq, dk=dk, dv=dv, **kw)
    for g in (0, kh - 1):
        hs = slice(g * qh // kh, (g + 1) * qh // kh)
        want = ref.attention(q[rows, hs], k[rows, g:g + 1], v[rows, g:g + 1], [(0, n, 0, n)], window, sinks, do=do[rows, hs], bounds=True)
        for name, x in (("dq", dq[rows, hs]), ("dk", dk[rows, g:g + 1]), ("dv", dv[rows, g:g + 1])):
            ref.check(x, want[name], want["b_" + name], name)


@pytest.mark.parametrize("qh,kh,hd,tokens", [(4, 2, 64, 100), (16, 8, 128, 2100)])
def test_starts_and_lengths_out_of_range(qh, kh, hd, tokens):
    """Clamped into the tensors' rows."""
    q, k, v, do = (normal((tokens, h, hd), 9 + i) for i, h in enumerate((qh, kh, kh, qh)))
    mid = tokens // 3
    wild, tame = ints([-70, mid, tokens + 900]), ints([0, mid, tokens])
    for lens, clamped in ((None, None), (ints([1 << 30, -5]), ints([mid, 0])), (ints([7, tokens]), ints([7, tokens - mid]))):
        got, want = puro.attention(q, k, v, wild, wild, lens), puro.attention(q, k, v, tame, tame, clamped)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    o, lse = puro.attention(q, k, v, tame, tame)
    got, want = (puro.attention_backward(do, q, k, v, o, lse, s, s) for s in (wild, tame))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("case", ap.FEW, ids=str)
def test_few_queries_are_as_exact_as_their_output(case):
    """P held in two bf16 adds nothing to the output's own rounding, whose relative error is 2^-7 / sqrt(12) times the root of
    the mean of 1/m^2 over mantissas m (0.736): 0.00166 in the norm.  One bf16 would make it 0.00235."""
    qh, kh, hd, queries, n, kl = case
    q, k, v = normal((queries * n, qh, hd), 13), normal((n * kl, kh, hd), 14), normal((n * kl, kh, hd), 15)
    o, _ = puro.attention(q, k, v, starts([queries] * n), starts([kl] * n))
    want = ref.attention(q, k, v, [(queries * s, queries, kl * s, kl) for s in range(n)])["o"]
    assert float((f64(o) - want).norm() / want.norm()) < 1.1 * U * 2 * 0.736 / 12 ** 0.5
