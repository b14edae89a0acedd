"""The bounds of tests/attention_gradients.py on the CPU: they hold for gradients with the kernels' roundings, and not where D
carries the rounding of o."""
import pytest
import torch

import attention_gradients as ag


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kind", ag.KINDS)
def test_bounds(kind, hd):
    x = ag.inputs(kind, 500, 2, 1, hd, 1)
    want = ag.Exact(*x, [500])
    good = ag.Exact(*x, [500], rounded=True)
    b = lambda t: t.to(torch.bfloat16)  # noqa: E731
    want.check(b(good.dq), b(good.dk), b(good.dv))
    bad = ag.Exact(*x, [500], rounded=True, d_from=b(want.o))
    if kind != "independent":
        assert want.worst("dq", b(bad.dq)) > 2.0
    assert want.worst("dq", 0 * good.dq) > 10 and want.worst("dk", 0 * good.dk) > 10 and want.worst("dv", 0 * good.dv) > 10


def test_formula_against_differences():
    """Each gradient against a central difference of sum(o do) along itself, where nothing cancels."""
    x = [t.double() for t in ag.inputs("means", 40, 2, 1, 64, 2)]
    kw = dict(lengths=[23, 17], window=9, sinks=2)
    e = ag.Exact(*x, **kw)
    for i, d in enumerate((e.dq, e.dk, e.dv)):
        d = d / d.norm()

        def loss(h):
            y = list(x)
            y[i] = y[i] + h * d
            return float((ag.Exact(*y, **kw).o * x[3]).sum())

        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs(diff / float(((e.dq, e.dk, e.dv)[i] * d).sum()) - 1) < 1e-5
