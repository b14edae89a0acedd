"""Which kernel the attention calls launch, on the host."""
import shutil

import pytest

import attention_plan as ap


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    return ap.Plans(tmp_path_factory.mktemp("plan"))


@pytest.mark.parametrize("case", ap.MANY, ids=str)
def test_shapes_of_the_kernel_for_many_queries(plans, case):
    qh, kh, hd, pack, ql, kl, window, sinks = case
    p = plans.forward(ap.shape(qh, kh, hd, sum(ql), sum(kl), len(ql), window, sinks))
    assert (p.few, p.pack, p.splits) == (0, pack, 1)


@pytest.mark.parametrize("case", ap.MANY_CACHED, ids=str)
def test_shapes_of_the_kernel_for_many_queries_over_a_cache(plans, case):
    qh, kh, hd, pack, ql, kl, room, window, sinks = case
    p = plans.forward(ap.shape(qh, kh, hd, sum(ql), room * len(ql), len(ql), window, sinks, max(kl)))
    assert (p.few, p.pack, p.splits) == (0, pack, 1)


@pytest.mark.parametrize("case", ap.FEW, ids=str)
def test_shapes_of_the_kernel_for_few_queries(plans, case):
    qh, kh, hd, queries, n, kl = case
    p = plans.forward(ap.shape(qh, kh, hd, queries * n, kl * n, n))
    assert p.few == 1 and p.splits == (7 if n == 1 else 1)
