"""Attention on the GPU against the plain 64-bit form of tests/attention_reference.py."""
import math
import threading

import pytest
import torch

import attention_reference as ref
from attention_reference import f64

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lengths):
    return ints([sum(lengths[:i]) for i in range(len(lengths) + 1)])


def packed(ql, kl, qh, kh, hd, seed, std=1.0):
    q, k, v = normal((sum(ql), qh, hd), seed, std), normal((sum(kl), kh, hd), seed + 1, std), normal((sum(kl), kh, hd), seed + 2)
    seqs = [(sum(ql[:i]), ql[i], sum(kl[:i]), kl[i]) for i in range(len(ql))]
    return q, k, v, seqs


def check_forward(q, k, v, seqs, got, window=0, sinks=0, scale=None):
    want = ref.attention(q, k, v, seqs, window, sinks, scale, bounds=True)
    ref.check(got[0], want["o"], want["b_o"], "o")
    ref.check(got[1], want["lse"], want["b_lse"], "lse")


MASKS = [(0, 0), (1, 0), (17, 0), (64, 4), (65, 1), (100, 70), (33, 200)]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("ql,kl", [([1], [1]), ([31, 1, 65], [31, 1, 65]), ([129], [129]), ([7, 0, 40], [90, 30, 40])])
@pytest.mark.parametrize("qh,kh,hd", [(2, 1, 128), (4, 4, 64)])
def test_forward_few_queries(ql, kl, qh, kh, hd, window, sinks):
    q, k, v, seqs = packed(ql, kl, qh, kh, hd, 1)
    got = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    check_forward(q, k, v, seqs, got, window, sinks)


# enough heads or tokens for the kernel for many queries: (tiles of 256 queries + sequences) x heads >= 256
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 4), (100, 70), (200, 300)])
@pytest.mark.parametrize("qh,kh,hd", [(128, 64, 64), (128, 8, 128)])
def test_forward_many_queries(qh, kh, hd, window, sinks):
    ql, kl = [257, 5, 0, 64], [257, 70, 9, 60]               # the last has more queries than keys
    q, k, v, seqs = packed(ql, kl, qh, kh, hd, 5)
    got = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    few = [0, 1, qh // 2, qh - 1]                            # the reference is slow: some query heads
    for h in few:
        g = h * kh // qh
        part = q[:, h:h + 1], k[:, g:g + 1], v[:, g:g + 1]
        check_forward(*part, seqs, (got[0][:, h:h + 1], got[1][h:h + 1]), window, sinks)


def test_one_long_sequence_many_queries():
    q, k, v, seqs = packed([2100], [2100], 64, 1, 64, 9)
    got = puro.attention(q, k, v, window=300, sinks=3)
    check_forward(q[:, :1], k, v, seqs, (got[0][:, :1], got[1][:1]), 300, 3)


@pytest.mark.parametrize("ql,kl", [([5], [3]), ([40, 3], [7, 0]), ([1], [0]), ([300], [1])])
@pytest.mark.parametrize("heads", [2, 256])
def test_rows_that_see_nothing(ql, kl, heads):
    q, k, v, seqs = packed(ql, kl, heads, heads, 64, 12)
    o, lse = puro.attention(q, k, v, starts(ql), starts(kl))
    check_forward(q[:, :2], k[:, :2], v[:, :2], seqs, (o[:, :2], lse[:2]))
    for q0, n, _, m in seqs:
        gone = max(0, n - m)
        assert not bool(o[q0:q0 + gone].any()) and bool((lse[:, q0:q0 + gone] == -math.inf).all())


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3), (300, 40)])
@pytest.mark.parametrize("queries", [1, 3])
@pytest.mark.parametrize("qh,kh,hd", [(16, 8, 128), (8, 1, 64), (3, 3, 128), (40, 1, 128)])
def test_single_tokens_over_a_cache(qh, kh, hd, queries, window, sinks):
    """Rows past k_len and keys that left the window hold NaN: nothing sees them."""
    lens, room = [1000, 3, 129, 0, 64], 1024
    n = len(lens)
    q = normal((queries * n, qh, hd), 20)
    k, v = normal((room * n, kh, hd), 21), normal((room * n, kh, hd), 22)
    for s, kl in enumerate(lens):
        k[s * room + kl:(s + 1) * room] = v[s * room + kl:(s + 1) * room] = float("nan")
        if window:
            lo = max(0, kl - queries - window + 1)
            if lo > sinks:
                k[s * room + sinks:s * room + lo] = v[s * room + sinks:s * room + lo] = float("nan")
    seqs = [(queries * s, queries, room * s, kl) for s, kl in enumerate(lens)]
    got = puro.attention(q, k, v, starts([queries] * n), starts([room] * n), ints(lens), window=window, sinks=sinks, max_k=max(lens))
    check_forward(q, k, v, seqs, got, window, sinks)


@pytest.mark.parametrize("max_k", [0, 1, 5000, 1 << 20])
@pytest.mark.parametrize("hd", [64, 128])
def test_split_over_a_long_cache(max_k, hd):
    q, k, v, seqs = packed([2], [5000], 4, 2, hd, 30, std=2.0)
    got = puro.attention(q, k, v, starts([2]), starts([5000]), max_k=max_k)
    check_forward(q, k, v, seqs, got)


@pytest.mark.parametrize("heads", [2, 256])
def test_scores_far_apart(heads):
    """Maxima that rise late and by much, and a scale other than the default."""
    q, k, v, seqs = packed([70], [400], heads, heads, 64, 35, std=1.0)
    k *= torch.linspace(0.1, 30.0, 400)[:, None, None].to(torch.bfloat16).cuda()
    got = puro.attention(q, k, v, scale=0.5)
    check_forward(q[:, :2], k[:, :2], v[:, :2], seqs, (got[0][:, :2], got[1][:2]), scale=0.5)


def test_strided_slices_and_outputs():
    T, qh, kh, hd = 150, 4, 2, 128
    wide = normal((T, qh + 2 * kh, hd), 40)
    q, k, v = wide[:, :qh], wide[:, qh:qh + kh], wide[:, qh + kh:]
    out = torch.full((T, qh + 2, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = puro.attention(q, k, v, out=out[:, 1:-1])
    want = puro.attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out[:, 1:-1], want[0]) and torch.equal(lse, want[1])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, -1] == 7).all())
    do = normal((T, qh + 2, hd), 41)[:, 1:-1]
    grad = torch.full((T, qh + 2 * kh, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    puro.attention_backward(do, q, k, v, o, lse, dq=grad[:, :qh], dk=grad[:, qh:qh + kh], dv=grad[:, qh + kh:])
    want = puro.attention_backward(do.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), o.contiguous(), lse)
    for a, b in zip((grad[:, :qh], grad[:, qh:qh + kh], grad[:, qh + kh:]), want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    stride, hd, n = 4096, 128, 200
    room = (1 << 32) // stride + 1000
    big = torch.empty(room, stride, dtype=torch.bfloat16, device="cuda")
    k, v = big[:, :hd].unflatten(1, (1, hd)), big[:, hd:2 * hd].unflatten(1, (1, hd))
    k0 = room - n - 17
    big[k0:k0 + n, :2 * hd] = normal((n, 2 * hd), 45)
    q = normal((n, 2, hd), 46)
    got = puro.attention(q, k, v, ints([0, 0, n]), ints([0, k0, k0 + n]))
    check_forward(q, k[k0:k0 + n], v[k0:k0 + n], [(0, n, 0, n)], got)   # a long cache is split: other sums than a short one's


BACK = [([1], [1], 0, 0), ([130], [130], 0, 0), ([33, 0, 64, 200], [33, 5, 64, 200], 0, 0), ([300], [300], 40, 0),
        ([500], [500], 30, 4), ([500, 20], [500, 20], 64, 130), ([20], [150], 0, 0), ([90], [40], 0, 0), ([90, 10], [40, 0], 16, 2),
        ([900], [900], 20, 3)]


@pytest.mark.parametrize("ql,kl,window,sinks", BACK)
@pytest.mark.parametrize("qh,kh,hd", [(2, 1, 128), (2, 2, 64), (8, 1, 64)])
def test_backward(ql, kl, window, sinks, qh, kh, hd):
    q, k, v, seqs = packed(ql, kl, qh, kh, hd, 50)
    do = normal(q.shape, 53, 1e-3)
    o, lse = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    got = puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(kl), window=window, sinks=sinks)
    want = ref.attention(q, k, v, seqs, window, sinks, do=do, bounds=True)
    for name, g in zip(("dq", "dk", "dv"), got):
        ref.check(g, want[name], want["b_" + name], name)


def test_backward_against_differences():
    ql, window, sinks = [50, 23], 20, 2
    q, k, v, seqs = packed(ql, ql, 4, 2, 64, 60)
    do = normal(q.shape, 63)
    o, lse = puro.attention(q, k, v, starts(ql), starts(ql), window=window, sinks=sinks)
    grads = puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(ql), window=window, sinks=sinks)
    want = ref.attention(q, k, v, seqs, window, sinks, do=do, bounds=True)
    x = [f64(t) for t in (q, k, v)]
    g = torch.Generator().manual_seed(64)
    h = 1e-5

    def loss(x):
        return float((ref.attention(*x, seqs, window, sinks)["o"] * f64(do)).sum())

    for _ in range(2):
        d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in x]
        diff = (loss([a + h * b for a, b in zip(x, d)]) - loss([a - h * b for a, b in zip(x, d)])) / (2 * h)
        got = sum(float((f64(a) * b).sum()) for a, b in zip(grads, d))
        tol = sum(float((want["b_" + n] * b.abs()).sum()) for n, b in zip(("dq", "dk", "dv"), d))
        assert abs(got - diff) <= tol + 1e-6 * abs(diff)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_the_same_bits_every_time(window, sinks):
    ql = [700, 33]
    q, k, v, _ = packed(ql, ql, 8, 2, 64, 70)
    do = normal(q.shape, 73)

    def once():
        o, lse = puro.attention(q, k, v, starts(ql), starts(ql), window=window, sinks=sinks)
        return (o, lse) + puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(ql), window=window, sinks=sinks)

    a = once()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, once()))


def test_captured_in_a_graph():
    """The block captured and replayed with eager work between, each replay against the eager result."""
    T, qh, kh, hd = 300, 4, 2, 128
    qs = starts([T])
    x = normal((T, (qh + 2 * kh) * hd), 80)
    w = normal((hd,), 81, 0.1) + 1
    tab = puro.rope_table(T, hd)
    do = normal((T, qh, hd), 82)
    cache = [normal((3000, kh, hd), 83 + i) for i in range(2)]
    cq, cs, cl = normal((1, qh, hd), 85), starts([3000]), ints([2900])

    def block():
        q, k = puro.qk_norm_rope(x, w, w, tab, q_heads=qh, k_heads=kh)
        v = x.view(T, -1, hd)[:, qh + kh:]
        o, lse = puro.attention(q, k, v, qs, qs, window=64, sinks=4)
        dq, dk, dv = puro.attention_backward(do, q, k, v, o, lse, qs, qs, window=64, sinks=4)
        dx, dwq, dwk = puro.qk_norm_rope_backward(dq, dk, x, w, w, tab)
        d, dl = puro.attention(cq, cache[0], cache[1], starts_1, cs, cl, max_k=3000)
        return [q, k, o, lse, dq, dk, dv, dx, dwq, dwk, d, dl]

    starts_1 = starts([1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            block()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for i in range(3):
        x.copy_(normal(x.shape, 90 + i))
        want = [t.clone() for t in block()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), "replay %d, output %d" % (i, n)


def test_other_streams_and_threads():
    data = []
    for t in range(3):
        q, k, v, _ = packed([400], [400], 4, 2, 64, 100 + 10 * t)
        data.append((q, k, v, normal(q.shape, 103 + 10 * t)))

    def path(q, k, v, do, stream=None):
        o, lse = puro.attention(q, k, v, window=100, sinks=2, stream=stream)
        return (o, lse) + puro.attention_backward(do, q, k, v, o, lse, window=100, sinks=2, stream=stream)

    want = [path(*d) for d in data]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = path(*data[0], stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    errors = []

    def worker(t):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got = path(*data[t])
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[t])):
                errors.append(t)
        except Exception as e:                               # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(t,)) for t in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=60)
    assert not any(th.is_alive() for th in threads) and not errors, errors


def test_empty_calls():
    q, k, v, _ = packed([0], [7], 2, 1, 64, 110)
    o, lse = puro.attention(q, k, v)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    dq, dk, dv = puro.attention_backward(q, q, k, v, o, lse)
    assert dq.shape == (0, 2, 64) and not bool(dk.any()) and not bool(dv.any())
    q, k, v, _ = packed([3], [0], 2, 1, 64, 111)
    o, lse = puro.attention(q, k, v)
    assert not bool(o.any()) and bool((lse == -math.inf).all())
    dq, dk, dv = puro.attention_backward(q, q, k, v, o, lse)
    assert not bool(dq.any()) and dk.shape == (0, 1, 64)


def test_refusals():
    q, k, v, _ = packed([9], [9], 4, 2, 64, 120)
    s = starts([9])
    with pytest.raises(TypeError):
        puro.attention(q.float(), k, v)
    with pytest.raises(ValueError):
        puro.attention(q, k, v[:, :1])
    with pytest.raises(ValueError):
        puro.attention(q, k, v, s)
    with pytest.raises(TypeError):
        puro.attention(q, k, v, s.long(), s.long())
    with pytest.raises(ValueError):
        puro.attention(q, k, v, s, s, ints([9, 9]))
    with pytest.raises(ValueError):
        puro.attention(q.transpose(0, 1), k, v)
    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")), dict(max_k=-1), dict(out=q)):
        with pytest.raises(puro.PuroError):
            puro.attention(q, k, v, **bad)
    with pytest.raises(puro.PuroError):
        puro.attention(q[:, :3], k, v)                       # 2 key heads do not divide 3 query heads
    with pytest.raises(puro.PuroError):
        puro.attention(q.reshape(9, 8, 32), k.reshape(9, 4, 32), v.reshape(9, 4, 32))
    o, lse = puro.attention(q, k, v)
    with pytest.raises(ValueError):
        puro.attention_backward(q, q, k, v, o, lse[:2])
    with pytest.raises(ValueError):
        puro.attention_backward(normal((9, 8, 64), 1)[:, ::2][:, :4], q, k, v, o, lse)
    with pytest.raises(puro.PuroError):
        puro.attention_backward(o, q, k, v, o, lse, dk=k)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(puro.PuroError):
        puro.attention_backward(q, q, k, v, o, lse, workspace=small)


@pytest.mark.parametrize("ql,window,sinks,qh,kh", [([1500, 700], 60, 5, 4, 1), ([2600], 100, 200, 2, 1), ([40] * 30 + [1300], 50, 4, 4, 2)])
def test_backward_of_first_keys_under_long_sequences(ql, window, sinks, qh, kh):
    """Walks of first keys cut into several parts, beside sequences that need none."""
    q, k, v, seqs = packed(ql, ql, qh, kh, 64, 130)
    do = normal(q.shape, 133, 1e-3)
    o, lse = puro.attention(q, k, v, starts(ql), starts(ql), window=window, sinks=sinks)
    got = puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(ql), window=window, sinks=sinks)
    want = ref.attention(q, k, v, seqs, window, sinks, do=do, bounds=True)
    for name, g in zip(("dq", "dk", "dv"), got):
        ref.check(g, want[name], want["b_" + name], name)


@pytest.mark.parametrize("ql,kl,window,sinks", [([40], [400], 50, 0), ([40, 3], [400, 300], 50, 3), ([1000], [1900], 100, 4)])
@pytest.mark.parametrize("qh,kh,hd", [(2, 1, 128), (4, 1, 64)])
def test_backward_of_keys_that_nothing_sees(ql, kl, window, sinks, qh, kh, hd):
    """Keys that left every query's window hold NaN: their gradients are 0, and no other one changes."""
    q, k, v, seqs = packed(ql, kl, qh, kh, hd, 140)
    do = normal(q.shape, 143, 1e-3)
    gone = [slice(k0 + sinks, k0 + n - m - window + 1) for _, m, k0, n in seqs]
    for g in gone:
        k[g] = v[g] = 0.0
    want = ref.attention(q, k, v, seqs, window, sinks, do=do, bounds=True)
    for g in gone:
        k[g] = v[g] = float("nan")
    o, lse = puro.attention(q, k, v, starts(ql), starts(kl), window=window, sinks=sinks)
    got = puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(kl), window=window, sinks=sinks)
    for name, x in zip(("dq", "dk", "dv"), got):
        ref.check(x, want[name], want["b_" + name], name)
    for g in gone:
        assert not bool(got[1][g].any()) and not bool(got[2][g].any())


@pytest.mark.parametrize("heads", [2, 256])
def test_a_query_that_is_nan(heads):
    """Its row and its log-sum are NaN, in either kernel; the other rows keep their values."""
    q, k, v, seqs = packed([70], [200], heads, heads, 64, 150)
    want = ref.attention(q[:, :2], k[:, :2], v[:, :2], seqs, bounds=True)
    q[13] = float("nan")
    o, lse = puro.attention(q, k, v)
    keep = [i for i in range(70) if i != 13]
    assert bool(o[13].isnan().all()) and bool(lse[:, 13].isnan().all())
    ref.check(o[keep, :2], want["o"][keep], want["b_o"][keep], "o")
    ref.check(lse[:2, keep], want["lse"][:, keep], want["b_lse"][:, keep], "lse")


@pytest.mark.parametrize("n", [62, 63, 64, 127, 200])
def test_many_sequences(n):
    """Short and empty sequences in numbers around what one lookup step covers."""
    g = torch.Generator().manual_seed(160 + n)
    ql = torch.randint(0, 5, (n,), generator=g).tolist()
    ql[-1] = 3
    kl = [m + e for m, e in zip(ql, torch.randint(0, 40, (n,), generator=g).tolist())]
    q, k, v, seqs = packed(ql, kl, 2, 1, 64, 161)
    do = normal(q.shape, 164, 1e-3)
    o, lse = puro.attention(q, k, v, starts(ql), starts(kl))
    check_forward(q, k, v, seqs, (o, lse))
    got = puro.attention_backward(do, q, k, v, o, lse, starts(ql), starts(kl))
    want = ref.attention(q, k, v, seqs, do=do, bounds=True)
    for name, x in zip(("dq", "dk", "dv"), got):
        ref.check(x, want[name], want["b_" + name], name)


@pytest.mark.parametrize("at,by", [(0, 40.0), (64, 40.0), (70, 400.0), (127, 4000.0), (320, 400.0)])
@pytest.mark.parametrize("heads", [2, 256])
def test_a_score_that_outgrows_the_others(heads, at, by):
    """One key far above all before and after it, up to where exp(s - running maximum) leaves fp32."""
    q, k, v, seqs = packed([100], [400], heads, heads, 64, 170, std=0.1)
    q[:, :, 0] = 1.0
    k[at, :, 0] = by
    got = puro.attention(q, k, v, scale=1.0)
    check_forward(q[:, :2], k[:, :2], v[:, :2], seqs, (got[0][:, :2], got[1][:2]), scale=1.0)
