"""C-ABI checks of include/puro_attention.h that need no GPU: every declared function
is exported, and invalid arguments are rejected on the host before a device is
touched (fake, never dereferenced pointers)."""
import os
import re
import subprocess

import pytest

import blockwise_fp8_gemm_act_amd as puro

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "puro_attention.h")
OK, NULL, SHAPE, ALIGN, MODE, DTYPE, WS, DEVICE, LAUNCH, ALIAS, SCRATCH, VALUE = range(12)
A = [0x7F0000000000 + i * (1 << 36) for i in range(16)]
EPS = 1e-6


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def valid(status):
    """A call that passes every check stops at the missing device here."""
    if no_gpu():
        assert status() == DEVICE


def test_library_exports_every_declared_function():
    names = sorted(set(re.findall(r"^\s*[\w\s\*]*?\b(puro_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert len(names) == 10
    out = subprocess.run(["nm", "-D", "--defined-only", puro.LIB_PATH], check=True, capture_output=True, text=True).stdout
    exported = set(re.findall(r"\bT (puro_\w+)", out))
    for name in names:
        assert name in exported and callable(getattr(puro, name)), name


def test_the_new_status_has_a_name():
    assert puro.puro_status_str(VALUE) != "unknown status"
    assert puro.STATUS_NAMES[VALUE] == "PURO_ERR_VALUE"


def test_rope_table():
    f = puro.puro_rope_table
    for scaling in range(4):
        valid(lambda: f(16, 128, 1e4, scaling, 8.0, 4096, A[0], None))
    assert f(16, 128, 1e4, 4, 8.0, 4096, A[0], None) == MODE
    for positions, rot in ((-1, 128), (1 << 24, 128), (16, 0), (16, 24), (16, 144)):
        assert f(positions, rot, 1e4, 0, 1.0, 0, A[0], None) == SHAPE
    for base in (1.0, -3.0, float("inf"), float("nan")):
        assert f(16, 128, base, 0, 1.0, 0, A[0], None) == VALUE
    assert f(16, 128, 1e4, 1, 0.5, 0, A[0], None) == VALUE
    assert f(16, 128, 1e4, 2, float("nan"), 0, A[0], None) == VALUE
    assert f(16, 128, 1e4, 3, 2.0, 0, A[0], None) == VALUE
    assert f(0, 128, 1e4, 0, 1.0, 0, None, None) == OK
    assert f(16, 128, 1e4, 0, 1.0, 0, None, None) == NULL
    assert f(16, 128, 1e4, 0, 1.0, 0, A[0] + 4, None) == ALIGN


def rotation(**k):
    return puro.Rotation(*[{**dict(table=A[0], positions=64, rot=128, layout=0, pos=A[1]), **k}[n]
                           for n in ("table", "positions", "rot", "layout", "pos")])


BAD_ROTATIONS = [(dict(layout=2), MODE), (dict(layout=-1), MODE), (dict(rot=0), SHAPE), (dict(rot=40), SHAPE),
                 (dict(rot=256), SHAPE), (dict(positions=0), SHAPE), (dict(positions=1 << 24), SHAPE),
                 (dict(table=None), NULL), (dict(table=A[0] + 8), ALIGN), (dict(pos=A[1] + 2), ALIGN)]


def test_rope():
    def f(r=None, x=A[2], xs=512, tokens=4, heads=3, hd=128, y=A[3], ys=384):
        return puro.puro_rope(r or rotation(), 0, x, xs, tokens, heads, hd, y, ys, None)
    valid(f)
    valid(lambda: f(rotation(pos=None)))
    assert puro.puro_rope(None, 0, A[2], 512, 4, 3, 128, A[3], 384, None) == NULL
    for change, status in BAD_ROTATIONS:
        assert f(rotation(**change)) == status, change
    for change in (dict(tokens=-1), dict(heads=-1), dict(hd=96), dict(hd=256), dict(xs=376), dict(ys=376), dict(xs=513), dict(ys=385),
                   dict(tokens=1 << 31), dict(tokens=1 << 30, xs=1 << 20)):
        assert f(**change) == SHAPE, change
    assert f(tokens=0, x=None, y=None) == OK and f(heads=0, x=None, y=None) == OK
    assert f(x=None) == NULL and f(y=None) == NULL
    assert f(x=A[2] + 8) == ALIGN and f(y=A[3] + 2) == ALIGN
    for y in (A[2], A[2] + 16, A[2] + 512 * 2 * 3, A[0] + 1024, A[1]):
        assert f(y=y) == ALIAS, hex(y)
    # two slices of the same rows: apart when their columns are
    valid(lambda: f(xs=1024, ys=1024, y=A[2] + 384 * 2))
    valid(lambda: f(xs=1024, ys=1024, y=A[2] - (1024 - 640) * 2))
    assert f(xs=1024, ys=1024, y=A[2] + 376 * 2) == ALIAS
    assert f(xs=1024, ys=1024, y=A[2] + 648 * 2) == ALIAS          # wraps into the next row's columns


def norm(append=False, r=None, x=A[2], xs=8192, tokens=4, qh=16, kh=8, hd=128, wq=A[4], wk=A[5], eps=EPS, q=A[6], qs=2048,
         k=A[7], ks=1024, v=A[8], vs=1024, rows=A[9], room=100):
    r = r or rotation()
    if append:
        return puro.puro_qk_norm_rope_append(r, x, xs, tokens, qh, kh, hd, wq, wk, eps, q, qs, k, ks, v, vs, rows, room, None)
    return puro.puro_qk_norm_rope(r, x, xs, tokens, qh, kh, hd, wq, wk, eps, q, qs, k, ks, None)


@pytest.mark.parametrize("append", [False, True])
def test_qk_norm_rope(append):
    f = lambda **k: norm(append, **k)  # noqa: E731
    valid(f)
    valid(lambda: f(qh=0, q=None, wq=None))
    valid(lambda: f(kh=0, k=None, v=None, wk=None))
    for change, status in BAD_ROTATIONS:
        assert f(r=rotation(**change)) == status, change
    for change in (dict(tokens=-1), dict(qh=-1), dict(kh=-1), dict(hd=32), dict(xs=2040), dict(qs=2040), dict(ks=1016), dict(ks=1025)):
        assert f(**change) == SHAPE, change
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(eps=eps) == VALUE
    assert f(tokens=0, x=None) == OK
    for change in (dict(x=None), dict(q=None), dict(k=None), dict(wq=None), dict(wk=None)):
        assert f(**change) == NULL, change
    for name, at in (("x", A[2]), ("q", A[6]), ("k", A[7]), ("wq", A[4]), ("wk", A[5])):
        assert f(**{name: at + 8}) == ALIGN, name
    for change in (dict(q=A[2]), dict(k=A[6]), dict(q=A[4]), dict(k=A[5]), dict(q=A[0])):
        assert f(**change) == ALIAS, change
    if append:
        assert f(xs=4088) == SHAPE and f(vs=1016) == SHAPE and f(room=-1) == SHAPE
        assert f(rows=None) == NULL and f(v=None) == NULL
        assert f(rows=A[9] + 2) == ALIGN and f(v=A[8] + 4) == ALIGN
        assert f(v=A[7]) == ALIAS and f(k=A[9]) == ALIAS
        valid(lambda: f(room=0, k=None, v=None))


def test_qk_norm_rope_backward():
    def f(r=None, dq=A[2], dqs=2048, dk=A[3], dks=1024, x=A[4], xs=4096, tokens=4, qh=16, kh=8, hd=128, wq=A[5], wk=A[6], eps=EPS,
          dx=A[7], dxs=4096, dwq=A[8], dwk=A[9], ws=A[10], size=1 << 20):
        return puro.puro_qk_norm_rope_backward(r or rotation(), dq, dqs, dk, dks, x, xs, tokens, qh, kh, hd, wq, wk, eps, dx, dxs,
                                               dwq, dwk, ws, size, None)
    need = puro.puro_qk_norm_rope_backward_workspace_bytes
    assert need(0, 128) == 0 and need(-1, 128) == 0 and need(4, 100) == 0
    assert need(4, 128) == 1024 and need(1 << 20, 64) == 1024 * 512
    valid(f)
    valid(lambda: f(tokens=0, x=None, dx=None, dq=None, dk=None, ws=None, size=0))       # zero weight gradients are written
    for change, status in BAD_ROTATIONS:
        assert f(r=rotation(**change)) == status, change
    for change in (dict(tokens=-1), dict(hd=80), dict(dqs=2040), dict(dks=1000), dict(xs=2040), dict(dxs=2040)):
        assert f(**change) == SHAPE, change
    assert f(eps=0.0) == VALUE
    for name in ("dq", "dk", "x", "wq", "wk", "dx", "dwq", "dwk"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: A[14] + 4}) == ALIGN, name
    for change in (dict(dx=A[4]), dict(dx=A[2]), dict(dwq=A[9]), dict(ws=A[4]), dict(ws=A[8])):
        assert f(**change) == ALIAS, change
    assert f(ws=None) == WS and f(size=1023) == WS


def shape(**k):
    d = dict(q_tokens=100, k_tokens=300, sequences=2, q_heads=16, k_heads=8, head_dim=128, q_stride=2048, k_stride=1024,
             v_stride=1024, o_stride=2048, dq_stride=2048, dk_stride=1024, dv_stride=1024, max_k=0, window=0, sinks=0, scale=0.1)
    return puro.AttentionShape(**{**d, **k})


BAD_SHAPES = [dict(q_tokens=-1), dict(k_tokens=-1), dict(q_tokens=(1 << 30) + 1), dict(k_tokens=(1 << 30) + 1), dict(sequences=0),
              dict(q_heads=0), dict(k_heads=0), dict(k_heads=3), dict(head_dim=96), dict(q_stride=2040), dict(k_stride=1016),
              dict(v_stride=1020), dict(o_stride=2047), dict(max_k=-1), dict(window=-1), dict(sinks=-1), dict(q_tokens=1 << 28),
              dict(sequences=1 << 23)]


def test_attention():
    def f(s=None, q=A[0], k=A[1], v=A[2], qst=A[3], kst=A[4], kl=A[5], o=A[6], lse=A[7], ws=A[8], size=1 << 33):
        return puro.puro_attention(s or shape(), q, k, v, qst, kst, kl, o, lse, ws, size, None)
    valid(f)
    valid(lambda: f(kl=None, lse=None))
    valid(lambda: f(shape(sequences=1), qst=None, kst=None))
    valid(lambda: f(shape(k_tokens=0), k=None, v=None))
    assert puro.puro_attention(None, *A[:9], 0, None) == NULL
    for change in BAD_SHAPES:
        assert f(shape(**change)) == SHAPE, change
        assert puro.puro_attention_workspace_bytes(shape(**change)) == 0
    for scale in (0.0, -1.0, 1e-31, float("inf"), float("nan")):
        assert f(shape(scale=scale)) == VALUE
    assert f(shape(q_tokens=0), q=None, o=None) == OK
    for change in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(qst=None), dict(kst=None), dict(qst=None, kst=None)):
        assert f(**change) == NULL, change
    for name in ("q", "k", "v", "o", "lse", "ws"):
        assert f(**{name: A[14] + 4}) == ALIGN, name
    for name in ("qst", "kst", "kl"):
        assert f(**{name: A[14] + 2}) == ALIGN, name
    for change in (dict(o=A[0]), dict(o=A[1]), dict(o=A[2] + 64), dict(lse=A[6]), dict(lse=A[0]), dict(o=A[3]), dict(lse=A[5])):
        assert f(**change) == ALIAS, change


def test_attention_workspace():
    need = puro.puro_attention_workspace_bytes
    long = dict(q_tokens=1, k_tokens=100000, sequences=1)
    n = need(shape(**long))
    assert n > 0 and n == need(shape(**long))
    assert need(shape(q_tokens=1 << 16, k_tokens=1 << 16)) == 0                  # many queries: no split
    assert need(shape(max_k=10, **long)) == 0                                    # nothing to split
    s = shape(**long)
    f = lambda ws, size: puro.puro_attention(s, A[0], A[1], A[2], A[3], A[4], None, A[6], None, ws, size, None)  # noqa: E731
    assert f(None, 0) == WS and f(A[8], n - 1) == WS
    assert f(A[0], n) == ALIAS
    valid(lambda: f(A[8], n))


def test_attention_backward():
    def f(s=None, do=A[0], q=A[1], k=A[2], v=A[3], o=A[4], lse=A[5], qst=A[6], kst=A[7], dq=A[8], dk=A[9], dv=A[10], ws=A[11], size=1 << 33):
        return puro.puro_attention_backward(s or shape(), do, q, k, v, o, lse, qst, kst, dq, dk, dv, ws, size, None)
    valid(f)
    valid(lambda: f(shape(sequences=1), qst=None, kst=None))
    for change in BAD_SHAPES + [dict(dq_stride=2040), dict(dk_stride=8), dict(dv_stride=1025)]:
        assert f(shape(**change)) == SHAPE, change
        assert puro.puro_attention_backward_workspace_bytes(shape(**change)) == 0
    assert f(shape(scale=0.0)) == VALUE
    assert f(shape(q_tokens=0, k_tokens=0)) == OK
    for name in ("do", "q", "k", "v", "o", "lse", "qst", "kst", "dq", "dk", "dv"):
        assert f(**{name: None}) == NULL, name
    for name in ("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"):
        assert f(**{name: A[14] + 4}) == ALIGN, name
    for change in (dict(dq=A[1]), dict(dk=A[2]), dict(dv=A[10], dk=A[10]), dict(dq=A[5]), dict(ws=A[8]), dict(ws=A[0])):
        assert f(**change) == ALIAS, change
    n = puro.puro_attention_backward_workspace_bytes(shape())
    assert n >= 2 * 4 * 16 * 100
    assert f(ws=None) == WS and f(size=n - 1) == WS
    valid(lambda: f(size=n))
    # the three gradients as columns of one tensor
    s = shape(k_tokens=100, k_heads=4, dq_stride=4096, dk_stride=4096, dv_stride=4096)
    valid(lambda: f(s, dk=A[8] + 2048 * 2, dv=A[8] + 2560 * 2))
    assert f(s, dk=A[8] + 2040 * 2, dv=A[8] + 2560 * 2) == ALIAS


@pytest.mark.parametrize("seed", range(20))
def test_tile_numbers_cover_every_sequence(seed):
    """Replays the kernels' numbering of tiles over sequences: start(s) mul / unit + s numbers are enough for every
    sequence's tiles, each number belongs to one sequence, and the launch has them all."""
    import random
    rng = random.Random(seed)
    unit, mul = rng.choice([(32, 1), (32, 2), (32, 7), (64, 1), (128, 1), (256, 1)])
    lengths = [rng.choice([0, 0, 1, 5, unit - 1, unit, unit + 1, rng.randint(0, 1000)]) for _ in range(rng.randint(1, 200))]
    start = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    base = [start[s] * mul // unit + s for s in range(len(lengths))]
    slots = start[-1] * mul // unit + len(lengths)
    seen = {}
    for slot in range(slots):
        s = max(i for i, b in enumerate(base) if b <= slot)
        tile = slot - base[s]
        if tile * unit < lengths[s] * mul:
            assert (s, tile) not in seen
            seen[s, tile] = slot
    assert len(seen) == sum(-(-n * mul // unit) for n in lengths)


@pytest.mark.parametrize("hd", [64, 128])
def test_lds_tiles(hd):
    """Host model of the attention kernels' LDS tiles: the elements that each lane copies, and that the lanes of row
    fragments and of transposing reads address the elements that they stand for."""
    group_rows, group_bytes = 512 // hd, 1040
    lds = {}
    for g in range(64 // group_rows):
        for lane in range(64):
            if hd == 128:
                r, c = (lane >> 2) & 3, 4 * (lane >> 4) + (lane & 3)
            else:
                r, c = ((lane >> 2) & 3) + 4 * (lane >> 5), 4 * ((lane >> 4) & 1) + (lane & 3)
            for i in range(8):
                at = g * group_bytes + 16 * lane + 2 * i
                assert at not in lds
                lds[at] = (g * group_rows + r, 8 * c + i)
    assert sorted(lds.values()) == [(r, c) for r in range(64) for c in range(hd)]

    def tile_bytes(rows):
        return rows // group_rows * group_bytes

    for lane in range(64):
        half, i = lane >> 5, lane & 15
        for r0 in (0, 32):
            for kk in range(hd // 16):
                r = lane & 31
                at = r // group_rows * group_bytes + (r & 3) * 64 + half * 16 + (0 if hd == 128 else ((r >> 2) & 1) * 512)
                at += (kk >> 1) * 256 + (kk & 1) * 32 + tile_bytes(r0)
                assert [lds[at + 2 * e] for e in range(8)] == [(r0 + r, 16 * kk + 8 * half + e) for e in range(8)]
        for r0 in (0, 16, 32, 48):
            for db in range(hd // 32):
                for w in range(2):
                    at = (i >> 2) * 64 + (i & 3) * 8 + (lane & 16) * 2 + half * (1040 if hd == 128 else 512)
                    at += db * 256 + tile_bytes(r0 + 8 * w)
                    row, col = r0 + 8 * w + 4 * half + (i >> 2), 32 * db + (lane & 16) + 4 * (i & 3)
                    assert [lds[at + 2 * e] for e in range(4)] == [(row, col + e) for e in range(4)]
