"""Rotary positions, query/key norms with the rotation, and their gradients on the
GPU against the plain 64-bit forms of tests/attention_reference.py."""
import pytest
import torch

import attention_reference as ref
from attention_reference import E, U, f64

pytestmark = pytest.mark.gpu

puro = pytest.importorskip("blockwise_fp8_gemm_act_amd")

EPS = 1e-6


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def positions(n, most, seed):
    return torch.randint(0, most, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("scaling,factor,trained", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0), ("yarn", 8.0, 512)])
@pytest.mark.parametrize("rot,n", [(128, 1), (64, 700), (16, 33)])
def test_table(scaling, factor, trained, rot, n):
    got = puro.rope_table(n, rot, base=1e6, scaling=scaling, factor=factor, trained=trained)
    want = ref.table(n, rot, 1e6, scaling, factor, trained)
    # fp64 angles (relative error of the frequency below 2^-48) and one rounding to fp32
    assert (f64(got) - want).abs().max() <= 2 * E * 1.3 + n * 2.0 ** -46


def test_table_far_positions():
    n = 300000
    got = puro.rope_table(n, 16, base=1e4)
    want = ref.table(n, 16, 1e4)
    assert (f64(got)[-100:] - want[-100:]).abs().max() <= E + n * 2.0 ** -46


@pytest.mark.parametrize("hd,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32), (64, 48)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (3, 5), (130, 24), (1031, 3)])
def test_rope(hd, rot, layout, tokens, heads):
    tab = puro.rope_table(200, rot)
    x, pos = normal((tokens, heads, hd), 1), positions(tokens, 200, 2)
    for inverse in (False, True):
        got = puro.rope(x, tab, pos, layout=layout, inverse=inverse)
        want = ref.rotate(f64(x), f64(tab), pos.cpu(), layout, inverse)
        ref.check(got, want, U * want.abs() + 4 * E * ref.partner_sum(f64(x), rot, layout), "rope")


def test_rope_passes_the_other_dimensions_bit_for_bit():
    x = normal((9, 2, 128), 3)
    x[0, 0, 100] = float("inf")
    got = puro.rope(x, puro.rope_table(16, 64))
    assert torch.equal(got[..., 64:], x[..., 64:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_default_positions_and_output(layout):
    wide = normal((50, 9, 128), 4)
    tab = puro.rope_table(64, 128)
    out = torch.full((50, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    puro.rope(wide[:, 2:6], tab, layout=layout, out=out[:, 1:5])
    want = puro.rope(wide[:, 2:6].contiguous(), tab, torch.arange(50, dtype=torch.int32, device="cuda"), layout=layout)
    assert torch.equal(out[:, 1:5], want)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 5] == 7).all())


def test_rope_inverse_undoes():
    x = normal((40, 4, 64), 5)
    tab = puro.rope_table(64, 64)
    back = puro.rope(puro.rope(x, tab), tab, inverse=True)
    # two roundings of values no larger than the pair's
    assert ((f64(back) - f64(x)).abs() <= 2.1 * U * ref.partner_sum(f64(x), 64, "half")).all()


@pytest.mark.parametrize("rot", [128, 64])
def test_position_outside_the_table_is_nan(rot):
    pos = torch.tensor([0, 8, -1, 7], dtype=torch.int32, device="cuda")
    y = puro.rope(normal((4, 2, 128), 6), puro.rope_table(8, rot), pos)
    for t, gone in enumerate([False, True, True, False]):
        assert bool(torch.isnan(y[t, :, :rot]).all()) == gone
        assert not bool(torch.isnan(y[t, :, rot:]).any())


def test_empty_calls():
    tab = puro.rope_table(8, 128)
    w = normal((128,), 0)
    assert puro.rope(normal((0, 3, 128), 0), tab).shape == (0, 3, 128)
    q, k = puro.qk_norm_rope(normal((0, 512), 0), w, w, tab, q_heads=2, k_heads=1)
    assert q.shape == (0, 2, 128) and k.shape == (0, 1, 128)
    dx, dwq, dwk = puro.qk_norm_rope_backward(normal((0, 2, 128), 0), normal((0, 1, 128), 0), normal((0, 512), 0), w, w, tab)
    assert dx.shape == (0, 3, 128) and not bool(dwq.any()) and not bool(dwk.any())


def norm_case(tokens, qh, kh, hd, seed, extra=0):
    x = normal((tokens, (qh + kh + extra) * hd), seed)
    x *= torch.exp(torch.randn(1, x.shape[1], generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()
    wq, wk = (normal((hd,), seed + i, 0.2) + 1 for i in (1, 2))
    return x, wq, wk


SHAPES = [(1, 16, 8, 128, 128, "half"), (5, 1, 1, 64, 64, "interleaved"), (77, 4, 2, 128, 64, "half"),
          (300, 6, 3, 64, 32, "half"), (1100, 16, 8, 128, 128, "interleaved"), (1500, 5, 0, 128, 128, "half"),
          (9, 0, 3, 64, 64, "half")]


@pytest.mark.parametrize("tokens,qh,kh,hd,rot,layout", SHAPES)
def test_qk_norm_rope(tokens, qh, kh, hd, rot, layout):
    x, wq, wk = norm_case(tokens, qh, kh, hd, 10, extra=kh)
    tab, pos = puro.rope_table(128, rot), positions(tokens, 128, 11)
    got = puro.qk_norm_rope(x, wq, wk, tab, pos, q_heads=qh, k_heads=kh, eps=EPS, layout=layout)
    xs = f64(x).view(tokens, -1, hd)
    for y, part, w in ((got[0], xs[:, :qh], wq), (got[1], xs[:, qh:qh + kh], wk)):
        n = ref.norm(part, f64(w), EPS)
        want = ref.rotate(n, f64(tab), pos.cpu(), layout)
        # the norm: a sum of hd squares (relative error hd E), a root, a division, two products
        ref.check(y, want, U * want.abs() * (1 + U) + (hd + 16) * E * ref.partner_sum(n, rot, layout), "norm and rotation")


def test_zero_rows_and_large_values():
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** 50
    x[2, 5] = 2.0 ** -50
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    q, k = puro.qk_norm_rope(x, w, w, puro.rope_table(1, 128), torch.zeros(3, dtype=torch.int32, device="cuda"), q_heads=1, k_heads=0)
    assert not bool(q[0].any()) and k.shape[1] == 0
    assert bool((q[1] == 1).all())
    assert abs(float(q[2, 0, 5]) / (2.0 ** -50 * 1000.0) - 1) < 2 * U


@pytest.mark.parametrize("tokens,qh,kh,hd,rot,layout", [s for s in SHAPES if s[2] > 0])
def test_append(tokens, qh, kh, hd, rot, layout):
    x, wq, wk = norm_case(tokens, qh, kh, hd, 20, extra=kh)
    tab, pos = puro.rope_table(128, rot), positions(tokens, 128, 21)
    room = 2 * tokens + 3
    rows = torch.randperm(room, generator=torch.Generator().manual_seed(22))[:tokens].to(torch.int32)
    rows[0] = room if tokens > 1 else rows[0]              # outside: left alone
    if tokens > 2:
        rows[2] = -1
    wide = normal((room, kh + 1, hd), 23)
    ck, cv = normal((room, kh, hd), 24), wide[:, 1:]
    want_k, want_v, first = ck.clone(), cv.clone(), wide[:, 0].clone()
    q = puro.qk_norm_rope_append(x, wq, wk, tab, pos, ck, cv, rows.cuda(), q_heads=qh, eps=EPS, layout=layout)
    plain_q, plain_k = puro.qk_norm_rope(x, wq, wk, tab, pos, q_heads=qh, k_heads=kh, eps=EPS, layout=layout)
    xs = x.view(tokens, -1, hd)
    for t, row in enumerate(rows.tolist()):
        if 0 <= row < room:
            want_k[row], want_v[row] = plain_k[t], xs[t, qh + kh:]
    assert torch.equal(q, plain_q) and torch.equal(ck, want_k) and torch.equal(cv, want_v) and torch.equal(wide[:, 0], first)


def test_append_far_cache_rows():
    """Cache rows whose element offset passes 2^32."""
    stride, hd = 4096, 128
    room = (1 << 32) // stride + 100
    big = torch.empty(room, stride, dtype=torch.bfloat16, device="cuda")
    ck, cv = big[:, :hd].unflatten(1, (1, hd)), big[:, hd:2 * hd].unflatten(1, (1, hd))
    x, wq, wk = norm_case(2, 1, 1, hd, 30, extra=1)
    tab = puro.rope_table(8, hd)
    rows = torch.tensor([room - 1, 5], dtype=torch.int32, device="cuda")
    puro.qk_norm_rope_append(x, wq, wk, tab, None, ck, cv, rows, q_heads=1)
    _, k = puro.qk_norm_rope(x, wq, wk, tab, None, q_heads=1, k_heads=1)
    assert torch.equal(ck[rows.long()], k) and torch.equal(cv[rows.long(), 0], x[:, 2 * hd:])


@pytest.mark.parametrize("tokens,qh,kh,hd,rot,layout", SHAPES + [(4500, 2, 1, 128, 128, "half")])
def test_backward(tokens, qh, kh, hd, rot, layout):
    x, wq, wk = norm_case(tokens, qh, kh, hd, 40, extra=kh)
    tab, pos = puro.rope_table(128, rot), positions(tokens, 128, 41)
    dq, dk = normal((tokens, qh, hd), 42, 1e-3), normal((tokens, kh, hd), 43, 1e-3)
    wide = torch.full((tokens, (qh + 2 * kh) * hd), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :(qh + kh) * hd].unflatten(1, (qh + kh, hd))
    dx, dwq, dwk = puro.qk_norm_rope_backward(dq, dk, x, wq, wk, tab, pos, eps=EPS, layout=layout, dx=out)
    assert bool((wide[:, (qh + kh) * hd:] == 7).all())
    xs = f64(x).view(tokens, -1, hd)
    for lo, hi, d, w, dw in ((0, qh, dq, wq, dwq), (qh, qh + kh, dk, wk, dwk)):
        part, g = xs[:, lo:hi], ref.rotate(f64(d), f64(tab), pos.cpu(), layout, inverse=True)
        want, want_w, mag = ref.norm_backward(g, part, f64(w), EPS)
        r = 1 / (part.square().mean(-1, keepdim=True) + EPS).sqrt()
        size = r * (f64(w) * ref.partner_sum(f64(d), rot, layout)).abs()
        size = size + (part * r).abs() * r * (f64(w) * g * part * r).abs().mean(-1, keepdim=True)
        ref.check(dx[:, lo:hi], want, U * want.abs() * (1 + U) + 4 * (hd + 16) * E * size, "dx")
        # at most 16 tokens x heads a lane in a row, then 16 teams and runs of 64 workgroups: far under 2^10 additions
        # one after the other; each term carries the norm's error
        ref.check(dw, want_w, (1024 + hd + 32) * E * mag, "dw")


def test_backward_against_differences():
    """Directional derivatives of the 64-bit forward form."""
    tokens, qh, kh, hd = 12, 2, 1, 64
    x, wq, wk = norm_case(tokens, qh, kh, hd, 50)
    tab = puro.rope_table(32, hd)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    dq, dk = normal((tokens, qh, hd), 51), normal((tokens, kh, hd), 52)
    dx, dwq, dwk = puro.qk_norm_rope_backward(dq, dk, x, wq, wk, tab, pos, eps=EPS)
    X, T, P = f64(x).view(tokens, -1, hd), f64(tab), pos.cpu()

    def loss(X, a, b):
        q = ref.rotate(ref.norm(X[:, :qh], a, EPS), T, P, "half")
        k = ref.rotate(ref.norm(X[:, qh:], b, EPS), T, P, "half")
        return float((q * f64(dq)).sum() + (k * f64(dk)).sum())

    g = torch.Generator().manual_seed(53)
    rnd = lambda t: torch.randn(t.shape, generator=g, dtype=torch.float64)  # noqa: E731
    h = 1e-5
    for _ in range(3):
        vx, va, vb = rnd(X), rnd(f64(wq)), rnd(f64(wk))
        diff = (loss(X + h * vx, f64(wq) + h * va, f64(wk) + h * vb) - loss(X - h * vx, f64(wq) - h * va, f64(wk) - h * vb)) / (2 * h)
        parts = [(f64(dx) * vx), (f64(dwq) * va), (f64(dwk) * vb)]
        # each product is off by at most U of itself; the difference quotient by O(h^2)
        tol = (U * 1.1) * sum(float(p.abs().sum()) for p in parts[:1]) + 1e-4 * sum(float(p.abs().sum()) for p in parts)
        assert abs(sum(float(p.sum()) for p in parts) - diff) <= tol


def test_backward_is_deterministic():
    x, wq, wk = norm_case(3000, 4, 2, 128, 60)
    tab = puro.rope_table(4096, 128)
    dq, dk = normal((3000, 4, 128), 61), normal((3000, 2, 128), 62)
    a = puro.qk_norm_rope_backward(dq, dk, x, wq, wk, tab)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, puro.qk_norm_rope_backward(dq, dk, x, wq, wk, tab)))


def test_refusals():
    tab = puro.rope_table(8, 128)
    x, w = normal((4, 3 * 128), 0), normal((128,), 1)
    with pytest.raises(TypeError):
        puro.rope(x.view(4, 3, 128).float(), tab)
    with pytest.raises(ValueError):
        puro.rope(x.view(4, 3, 128), tab, layout="quarter")
    with pytest.raises(TypeError):
        puro.rope(x.view(4, 3, 128), tab, torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        puro.rope(x.view(4, 3, 128), tab, torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        puro.rope(x.view(4, 3, 128).transpose(0, 1), tab)
    with pytest.raises(puro.PuroError):
        puro.rope(x.view(4, 6, 64), tab)                    # more rotated dimensions than the head has
    y = x.view(4, 3, 128)
    with pytest.raises(puro.PuroError):
        puro.rope(y, tab, out=y)                            # in place
    with pytest.raises(ValueError):
        puro.qk_norm_rope(x, w, w, tab, q_heads=3, k_heads=1)
    with pytest.raises(puro.PuroError):
        puro.qk_norm_rope(x, w, w, tab, q_heads=2, k_heads=1, eps=0.0)
    with pytest.raises(TypeError):
        puro.qk_norm_rope(x, w.float(), w, tab, q_heads=2, k_heads=1)
    with pytest.raises(puro.PuroError):
        puro.rope_table(8, 128, base=0.5)
    with pytest.raises(ValueError):
        puro.rope_table(8, 128, scaling="cubic")
