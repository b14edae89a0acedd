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


THREADS = 1 << 32          # a launch of this many is refused by the runtime


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (16, 8), (65536, 1), (65536, 65536)])
@pytest.mark.parametrize("sequences", [1, 2, 1000, 1 << 16, 1 << 22])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 256), (1000, 4)])
@pytest.mark.parametrize("backward", [False, True])
def test_largest_launches(plans, backward, hd, heads, sequences, window, sinks):
    """Grids at the largest token counts that a call accepts."""
    import blockwise_fp8_gemm_act_amd as puro
    import torch
    qh, kh = heads
    limit = (1 << 31) // 4 * 3 if backward else 1 << 31
    q_most, k_most = (min(1 << 30, (1 << 40) // (h * hd), (limit - 4) // h - 512 * sequences) for h in heads)
    if q_most < 1 or k_most < 1:
        return
    at = [1 << 56 | i << 52 for i in range(12)]
    for qt, kt in ((q_most, k_most), (q_most, 300), (600, k_most), (600, 300)):
        s = ap.shape(qh, kh, hd, min(qt, q_most), min(kt, k_most), sequences, window, sinks)
        if backward:
            p = plans.backward(s)
            threads = [256 * n for n in (p.dq_blocks, p.dk_blocks, p.join_blocks)]
            accepted = lambda s: puro.puro_attention_backward(s, *at, 1 << 62, None)  # noqa: E731
        else:
            p = plans.forward(s)
            threads = [p.threads * p.blocks, 256 * p.join_blocks]
            accepted = lambda s: puro.puro_attention(s, *at[:9], 1 << 62, None)  # noqa: E731
        assert max(threads) < THREADS, vars(p)
        if not torch.cuda.is_available() and qh * hd < 1 << 23:          # stopped only by the missing device; one more is refused
            assert accepted(s) == 7
            if s.q_tokens < 1 << 30 and s.q_tokens * qh * hd < (1 << 40) - qh * hd and s.q_tokens == q_most:
                s.q_tokens += 4
                assert accepted(s) == 2


@pytest.mark.parametrize("tokens", [1, 511, 4096, 1 << 25, 1 << 26, (1 << 31) - 1])
@pytest.mark.parametrize("heads,hd", [(1, 64), (24, 128), (65536, 64)])
def test_largest_launches_of_the_rotation(plans, tokens, heads, hd):
    parts, launches, blocks = plans.rope(tokens, heads, hd)
    assert blocks * 256 < THREADS and launches == max(1, tokens >> 25) + (tokens > 1 << 25 and tokens % (1 << 25) > 0)
    assert 1 <= parts <= -(-heads // (512 // hd))


# (sequences, queries, earlier keys, query heads, key heads, head_dim, us of the kernel for many queries and of the one for few)
TIMED = [(1, 256, 0, 16, 8, 128, 14.6, 8.3), (1, 1500, 0, 16, 8, 128, 37.2, 49.3), (16, 64, 2048, 16, 8, 128, 48.6, 63.0),
         (1, 1024, 8192, 16, 8, 128, 171.2, 225.5), (4, 512, 0, 16, 8, 128, 20.4, 36.7), (1, 4096, 0, 16, 8, 128, 91.7, 251.6),
         (64, 8, 2048, 16, 8, 128, 145.3, 126.8), (1, 512, 16384, 16, 8, 128, 308.6, 209.8), (1, 64, 16384, 16, 8, 128, 291.6, 46.7)]


@pytest.mark.parametrize("case", TIMED, ids=str)
def test_the_faster_kernel_is_chosen(plans, case):
    n, ql, earlier, qh, kh, hd, many, few = case
    p = plans.forward(ap.shape(qh, kh, hd, n * ql, n * (ql + earlier), n, max_k=ql + earlier))
    assert p.few == (few < many)
