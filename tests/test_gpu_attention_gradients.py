"""Attention's gradients on the GPU, norm by norm, where D (the row sums of do o) cancels nearly all of do v: rows with a
dominating key, keys and values with a mean, large queries."""
import pytest
import torch

import attention_gradients as ag
from attention_reference import f64

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")


def gradients(q, k, v, do, lengths, window=0, sinks=0):
    s = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    o, lse = puro.attention(q, k, v, s, s, window=window, sinks=sinks)
    return puro.attention_backward(do, q, k, v, o, lse, s, s, window=window, sinks=sinks)


@pytest.mark.parametrize("lengths,window,sinks", [([1100], 0, 0), ([701, 400], 0, 0), ([900], 300, 4), ([300], 90, 5)])
@pytest.mark.parametrize("qh,kh,hd", [(2, 1, 128), (3, 3, 128), (4, 1, 64)])
@pytest.mark.parametrize("kind", ag.KINDS)
def test_rows_of_gradients(kind, qh, kh, hd, lengths, window, sinks):
    x = ag.inputs(kind, sum(lengths), qh, kh, hd, 7)
    ag.Exact(*x, lengths, window, sinks).check(*gradients(*x, lengths, window, sinks))


def test_a_block_with_one_such_row():
    """Among independent rows one that a single key takes: its block's other rows, and other blocks, keep their bounds."""
    q, k, v, do = ag.inputs("independent", 1000, 2, 1, 64, 8)
    q[777] = (60.0 * k[500, 0] / k[500, 0].float().norm()).to(torch.bfloat16)
    ag.Exact(q, k, v, do, [1000]).check(*gradients(q, k, v, do, [1000]))


@pytest.mark.parametrize("kind", ["independent", "means"])
def test_against_differences_along_the_gradient(kind):
    """Each gradient's product with a direction against the central difference of sum(o do) along it.  The direction is
    the gradient itself, so that the product is its norm, far above the roundings: zero, reversed or scaled gradients
    of any one tensor fail."""
    lengths, window, sinks = [150, 61], 40, 3
    x = ag.inputs(kind, sum(lengths), 4, 2, 64, 9)
    got = gradients(*x, lengths, window, sinks)
    x = [f64(t) for t in x]
    e = ag.Exact(*x, lengths, window, sinks)
    for i, name in enumerate(("dq", "dk", "dv")):
        want = getattr(e, name)
        d = want / want.norm()

        def loss(h):
            y = list(x)
            y[i] = y[i] + h * d
            return float((ag.Exact(*y, lengths, window, sinks).o * x[3]).sum())

        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        tol = float(getattr(e, "bound_" + name).norm())       # of the whole error's norm; the difference is off by 1e-5 of itself
        assert tol < 0.1 * diff
        assert abs(float((f64(got[i]) * d).sum()) - diff) <= tol + 1e-5 * diff, name


@pytest.mark.parametrize("heads", [(2, 1), (4, 4)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("ql,kl,window,sinks", [([90], [40], 0, 0), ([300, 20], [200, 20], 0, 0), ([70, 5], [30, 0], 16, 2)])
def test_rows_that_see_nothing_whatever_they_hold(ql, kl, window, sinks, hd, heads):
    """Queries and gradients of rows that see no key hold NaN or infinities: zero gradients, and no other one changes."""
    starts = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(11)
    new = lambda n, h: torch.randn(n, h, hd, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v, do = new(sum(ql), heads[0]), new(sum(kl), heads[1]), new(sum(kl), heads[1]), new(sum(ql), heads[0])
    gone = torch.zeros(sum(ql), dtype=torch.bool, device="cuda")
    for i, (n, m) in enumerate(zip(ql, kl)):
        gone[sum(ql[:i]):sum(ql[:i]) + max(0, n - m)] = True
    seqs, mask = (starts(ql), starts(kl)), dict(window=window, sinks=sinks)

    def path(fill):
        q[gone], do[gone] = fill, -fill
        o, lse = puro.attention(q, k, v, *seqs, **mask)
        return (o, lse) + puro.attention_backward(do, q, k, v, o, lse, *seqs, **mask)

    want = path(0.0)
    assert not bool(want[0][gone].any()) and not bool(want[2][gone].any()) and all(bool(t.isfinite().all()) for t in want[2:])
    for fill in (float("nan"), float("inf")):
        assert all(torch.equal(a, b) for a, b in zip(path(fill), want))
