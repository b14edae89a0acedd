"""Measured cases of the attention block's operators: rotary positions, the per-head norms of queries and keys
with the rotation in the same pass, and attention with a sliding window and first tokens that stay visible.

``own`` false: the plain form in elementary torch operations, in 32 bits, rounded once at the end.
``own`` true: the calls a user makes of ``blockwise_fp8_gemm_act_amd``.

The shapes are the repository's layer (16 query and 8 key/value heads of 128, a 4096-token context, 16384 tokens a
step) and generic ones around it."""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 1e6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the rotation of one new token of one sequence: launch latency
        dict(name="rope 1 token", op="rope", tokens=1, heads=24, head_dim=128, rot=128, layout="half", inverse=False,
             positions=4096, scaling="none", strided=True),
        # gradient of a rotation of half of each head, interleaved pairs, a context stretched eightfold
        dict(name="rope 16381 tokens inverse", op="rope", tokens=16381, heads=16, head_dim=128, rot=64,
             layout="interleaved", inverse=True, positions=32768, scaling="yarn", strided=False),
        # one decoding step of 32 sequences: norms, rotation, and the new keys and values put into the cache
        dict(name="qk_norm_rope append 32", op="norm_append", tokens=32, q_heads=16, k_heads=8, head_dim=128, rot=128,
             layout="half", positions=4096, cache=512),
        # the layer's forward step at 16384 tokens, read out of the QKV projection's output
        dict(name="qk_norm_rope 16384", op="norm", tokens=16384, q_heads=16, k_heads=8, head_dim=128, rot=128,
             layout="half", positions=4096, sequences=4),
        # and its backward step
        dict(name="qk_norm_rope backward 16384", op="norm_bwd", tokens=16384, q_heads=16, k_heads=8, head_dim=128,
             rot=128, layout="half", positions=4096, sequences=4),
        # a short prompt: latency of the forward pass
        dict(name="attention 200 tokens", op="attn", q_tokens=200, sequences=1, context=0, ragged=False, q_heads=16,
             k_heads=8, head_dim=128, window=0, sinks=0),
        # the layer's forward step: four full contexts of 4096 tokens
        dict(name="attention 4 x 4096", op="attn", q_tokens=16384, sequences=4, context=0, ragged=False, q_heads=16,
             k_heads=8, head_dim=128, window=0, sinks=0),
        # a long prompt of odd length in a window of 1024 with 4 visible first tokens
        dict(name="attention 16381 window", op="attn", q_tokens=16381, sequences=1, context=0, ragged=False,
             q_heads=16, k_heads=8, head_dim=128, window=1024, sinks=4),
        # the layer's backward step
        dict(name="attention backward 4 x 4096", op="attn_bwd", q_tokens=16384, sequences=4, context=0, ragged=False,
             q_heads=16, k_heads=8, head_dim=128, window=0, sinks=0),
        # backward over packed documents of uneven lengths, windowed, heads of 64 in groups of four
        dict(name="attention backward ragged", op="attn_bwd", q_tokens=8191, sequences=6, context=0, ragged=True,
             q_heads=16, k_heads=4, head_dim=64, window=512, sinks=4),
        # a single token over one long cache: the keys are split over the card
        dict(name="decode 1 x 131071", op="attn", q_tokens=1, sequences=1, context=131070, ragged=False, q_heads=16,
             k_heads=8, head_dim=128, window=0, sinks=0),
        # single tokens of 64 sequences of uneven lengths, a window of 4096 with 4 visible first tokens
        dict(name="decode 64 ragged window", op="attn", q_tokens=64, sequences=64, context=8192, ragged=True,
             q_heads=16, k_heads=8, head_dim=128, window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm", "norm_append", "norm_bwd", "attn", "attn", "attn_bwd", "attn_bwd", "decode", "decode"])
    hd = rng.choice([64, 128, 128])
    kh = rng.choice([1, 2, 4, 8])
    c = dict(head_dim=hd)
    if op in ("rope", "norm", "norm_append", "norm_bwd"):
        c.update(op=op, rot=rng.choice([hd, hd, hd // 2]), layout=rng.choice(["half", "interleaved"]))
        if op == "rope":
            c.update(tokens=_log(rng, 1, 16384), heads=rng.choice([1, 5, 8, 16, 24]), inverse=rng.random() < 0.5,
                     positions=_log(rng, 2048, 65536), scaling=rng.choice(["none", "linear", "yarn"]),
                     strided=rng.random() < 0.5)
        else:
            c.update(q_heads=kh * rng.choice([1, 2, 4]) if kh < 8 else 16, k_heads=kh, positions=_log(rng, 2048, 16384))
            if op == "norm_append":
                c.update(tokens=_log(rng, 1, 128), cache=rng.randint(64, 512))
            else:
                c.update(tokens=_log(rng, 64, 16384), sequences=rng.randint(1, 8))
        return c
    c.update(q_heads=kh * rng.choice([1, 2, 4]) if kh < 8 else 16, k_heads=kh)
    window = rng.choice([0, _log(rng, 64, 4096)])
    c.update(window=window, sinks=rng.choice([0, 1, 4, 16]) if window else 0)
    if op == "decode":
        n = _log(rng, 1, 64)
        c.update(op="attn", q_tokens=n * rng.choice([1, 1, 1, 3]), sequences=n, ragged=n > 1,
                 context=_log(rng, 16, min(131072, 262144 // n)))
    else:
        n = rng.randint(1, 6)
        c.update(op=op, q_tokens=_log(rng, 32, 8192), sequences=n, ragged=n > 1,
                 context=0 if op == "attn_bwd" else rng.choice([0, 0, rng.randint(1, 2048)]))
    return c


def _lengths(c):
    """(queries, keys) of each sequence: the same for every seed. Where the case says so they are uneven."""
    n, t = c["sequences"], c["q_tokens"]
    rng = random.Random("%d/%d/%d" % (n, t, c["context"]))
    if t == n or t == 3 * n or not c["ragged"]:
        q = [t // n + (i < t % n) for i in range(n)]
    else:
        cuts = sorted(rng.randint(0, t) for _ in range(n - 1))
        q = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    k = [a + (rng.randint(c["context"] // 4, c["context"]) if c["ragged"] else c["context"]) for a in q]
    return q, k


def _visible(ql, kl, window, sinks):
    """Visible (query, key) pairs of one sequence, and the keys that any of its queries sees."""
    pairs = 0
    for i in range(ql) if ql <= 64 else ():
        p = kl - ql + i
        seen = p + 1 if not window else min(window, p + 1) + max(0, min(sinks, p + 1 - window))
        pairs += max(0, seen)
    if ql > 64:
        p = torch.arange(kl - ql, kl, dtype=torch.int64)
        seen = (p + 1).clamp(min=0)
        if window:
            seen = seen.clamp(max=window) + (p + 1 - window).clamp(min=0, max=sinks)
        pairs = int(seen.sum())
    first = 0 if not window else max(0, kl - ql - window + 1)
    keys = kl - first + min(sinks if window else 0, first) if ql else 0
    return pairs, keys


def work(c):
    hd = c["head_dim"]
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * hd
        return {"bytes": 4 * n + 4 * c["rot"] * min(c["tokens"], c["positions"]), "flops": 3 * n}
    if c["op"] in ("norm", "norm_append", "norm_bwd"):
        n = c["tokens"] * (c["q_heads"] + c["k_heads"]) * hd
        more = 4 * c["rot"] * min(c["tokens"], c["positions"]) + 4 * hd
        if c["op"] == "norm_append":
            more += 4 * c["tokens"] * c["k_heads"] * hd
        return {"bytes": (6 if c["op"] == "norm_bwd" else 4) * n + more, "flops": (14 if c["op"] == "norm_bwd" else 7) * n}
    each = [_visible(a, b, c["window"], c["sinks"]) for a, b in zip(*_lengths(c))]
    pairs, keys = sum(p for p, _ in each), sum(k for _, k in each)
    q = c["q_tokens"] * c["q_heads"] * hd
    kv = keys * c["k_heads"] * hd
    if c["op"] == "attn":
        return {"bytes": 4 * q + 4 * kv + 4 * c["q_tokens"] * c["q_heads"], "flops": 4 * hd * pairs * c["q_heads"]}
    return {"bytes": 8 * q + 8 * kv + 4 * c["q_tokens"] * c["q_heads"], "flops": 10 * hd * pairs * c["q_heads"]}


# ---------------------------------------------------------------- what a program has in hand
def _table(rot, positions, scaling="none", factor=8.0, trained=4096):
    """[positions][2][rot/2] fp32: cosines, then sines."""
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        g = ((trained * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f = f * ((1 - g) / factor + g)
        m = 0.1 * math.log(factor) + 1
    phi = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((m * phi.cos(), m * phi.sin()), dim=1).float().contiguous()


def _normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _weight(g, hd):
    return (1 + 0.1 * torch.randn(hd, generator=g, device="cuda")).to(torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hd = c["head_dim"]
    if c["op"] == "rope":
        t, h = c["tokens"], c["heads"]
        # a slice of a wider row, as a fused projection gives it, or a dense tensor
        wide = _normal(g, t, h + 8 if c["strided"] else h, hd)
        pos = torch.randint(0, c["positions"], (t,), generator=g, device="cuda", dtype=torch.int32)
        return dict(c=c, x=wide[:, :h], table=_table(c["rot"], c["positions"], c["scaling"]), pos=pos)
    if c["op"] in ("norm", "norm_append", "norm_bwd"):
        t, qh, kh = c["tokens"], c["q_heads"], c["k_heads"]
        x = _normal(g, t, qh + 2 * kh, hd)
        x *= torch.exp(0.5 * torch.randn(1, qh + 2 * kh, 1, generator=g, device="cuda")).to(torch.bfloat16)
        s = dict(c=c, x=x.view(t, -1), wq=_weight(g, hd), wk=_weight(g, hd), table=_table(c["rot"], c["positions"]))
        if c["op"] == "norm_append":
            s["pos"] = torch.randint(0, c["cache"], (t,), generator=g, device="cuda", dtype=torch.int32)
            s["rows"] = s["pos"] + c["cache"] * torch.arange(t, device="cuda", dtype=torch.int32)
            s["cache_k"] = _normal(g, t * c["cache"], kh, hd)
            s["cache_v"] = _normal(g, t * c["cache"], kh, hd)
        else:
            per = -(-t // c["sequences"])
            s["pos"] = (torch.arange(t, device="cuda", dtype=torch.int32) % per) % c["positions"]
        if c["op"] == "norm_bwd":
            s["dq"], s["dk"] = _normal(g, t, qh, hd, std=1e-3), _normal(g, t, kh, hd, std=1e-3)
        return s
    t, qh, kh, n = c["q_tokens"], c["q_heads"], c["k_heads"], c["sequences"]
    ql, kl = _lengths(c)
    cache = c["op"] == "attn" and c["context"] > 0
    room = [max(kl)] * n if cache else kl           # a cache keeps room for the longest sequence
    gain = torch.exp(0.3 * torch.randn(1, qh, 1, generator=g, device="cuda")).to(torch.bfloat16)
    s = dict(c=c, q=_normal(g, t, qh, hd) * gain, max_q=max(ql), max_k=max(kl), scale=hd ** -0.5)
    wide = _normal(g, sum(room), kh if cache else 2 * kh, hd)
    s["k"] = _normal(g, sum(room), kh, hd)
    s["v"] = wide if cache else wide[:, kh:]        # in training the values stay in the projection's output
    starts = lambda v: torch.tensor([sum(v[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    s["q_start"], s["k_start"] = starts(ql), starts(room)
    s["k_len"] = torch.tensor(kl, dtype=torch.int32, device="cuda") if cache else None
    if c["op"] == "attn_bwd":
        s["do"] = _normal(g, t, qh, hd, std=1e-3)
        s["o"], s["lse"] = _plain_attention(s)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import blockwise_fp8_gemm_act_amd as puro

    c = s["c"]
    if c["op"] == "rope":
        return puro.rope(s["x"], s["table"], s["pos"], layout=c["layout"], inverse=c["inverse"])
    if c["op"] == "norm":
        return puro.qk_norm_rope(s["x"], s["wq"], s["wk"], s["table"], s["pos"], q_heads=c["q_heads"],
                                 k_heads=c["k_heads"], eps=EPS, layout=c["layout"])
    if c["op"] == "norm_append":
        q = puro.qk_norm_rope_append(s["x"], s["wq"], s["wk"], s["table"], s["pos"], s["cache_k"], s["cache_v"],
                                     s["rows"], q_heads=c["q_heads"], eps=EPS, layout=c["layout"])
        return q, s["cache_k"], s["cache_v"]
    if c["op"] == "norm_bwd":
        return puro.qk_norm_rope_backward(s["dq"], s["dk"], s["x"], s["wq"], s["wk"], s["table"], s["pos"], eps=EPS,
                                          layout=c["layout"])
    more = dict(q_start=s["q_start"], k_start=s["k_start"], window=c["window"], sinks=c["sinks"], scale=s["scale"])
    if c["op"] == "attn":
        return puro.attention(s["q"], s["k"], s["v"], k_len=s["k_len"], max_k=s["max_k"], **more)
    return puro.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **more)


def _plain(s):
    op = s["c"]["op"]
    if op == "rope":
        c = s["c"]
        cos, sin = _cos_sin(s, c["inverse"])
        return _rotate(s["x"].float(), cos, sin, c["layout"]).to(torch.bfloat16)
    if op == "norm":
        return _plain_norm(s)[:2]
    if op == "norm_append":
        q, k, v = _plain_norm(s)
        s["cache_k"].index_copy_(0, s["rows"].long(), k)
        s["cache_v"].index_copy_(0, s["rows"].long(), v)
        return q, s["cache_k"], s["cache_v"]
    if op == "norm_bwd":
        return _plain_norm_backward(s)
    return _plain_attention(s) if op == "attn" else _plain_attention_backward(s)


def _cos_sin(s, inverse=False):
    cs = s["table"][s["pos"]]                       # [T][2][rot/2]
    cos, sin = cs[:, None, 0], cs[:, None, 1]
    return cos, -sin if inverse else sin


def _rotate(x, cos, sin, layout):
    half = cos.shape[-1]
    rot = 2 * half
    if layout == "half":
        a, b = x[..., :half], x[..., half:rot]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), dim=-1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _heads(s):
    c = s["c"]
    x = s["x"].view(s["x"].shape[0], -1, c["head_dim"])
    return x[:, :c["q_heads"]], x[:, c["q_heads"]:c["q_heads"] + c["k_heads"]], x[:, c["q_heads"] + c["k_heads"]:]


def _plain_norm(s):
    xq, xk, xv = _heads(s)
    cos, sin = _cos_sin(s)
    x = torch.cat((xq, xk), dim=1).float()
    w = torch.cat((s["wq"].expand(xq.shape[1], -1), s["wk"].expand(xk.shape[1], -1))).float()
    y = _rotate(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w, cos, sin, s["c"]["layout"]).to(torch.bfloat16)
    return y[:, :xq.shape[1]], y[:, xq.shape[1]:], xv


def _plain_norm_backward(s):
    xq, xk, _ = _heads(s)
    qh = xq.shape[1]
    cos, sin = _cos_sin(s, inverse=True)
    x = torch.cat((xq, xk), dim=1).float()
    w = torch.cat((s["wq"].expand(qh, -1), s["wk"].expand(xk.shape[1], -1))).float()
    g = _rotate(torch.cat((s["dq"], s["dk"]), dim=1).float(), cos, sin, s["c"]["layout"])
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    gx = g * xh
    dx = r * (w * g - xh * (w * gx).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), gx[:, :qh].sum((0, 1)), gx[:, qh:].sum((0, 1))


def _padded(s):
    """Sequences side by side: q [B][Hk][G Lq][hd], k and v [B][Hk][Lk][hd] in 32 bits, the mask [B][1][1][Lq][Lk], and the
    place of each token among them."""
    c = s["c"]
    n, kh, hd = c["sequences"], c["k_heads"], c["head_dim"]
    grp = c["q_heads"] // kh
    q0, k0 = s["q_start"][:-1].long(), s["k_start"][:-1].long()
    ql = s["q_start"][1:].long() - q0
    kl = s["k_len"].long() if s["k_len"] is not None else s["k_start"][1:].long() - k0
    i = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_k"], device="cuda")
    qi = (q0[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    kj = (k0[:, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][qi].float().view(n, -1, kh, grp, hd).permute(0, 2, 3, 1, 4).reshape(n, kh, -1, hd)
    k = s["k"][kj].float().transpose(1, 2).contiguous()
    v = s["v"][kj].float().transpose(1, 2).contiguous()
    p = ((kl - ql)[:, None] + i)[:, :, None]
    mask = (i < ql[:, None])[:, :, None] & (j <= p) & (j < kl[:, None, None])
    if c["window"]:
        mask = mask & ((j > p - c["window"]) | (j < c["sinks"]))
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.bucketize(t, s["q_start"][1:].long(), right=True)
    return q, k, v, mask[:, None, None], (seq, t - q0[seq]), (qi, ql, kj, kl)


def _probabilities(q, k, mask, scale):
    """exp(S - m), its row sums and the row maxima m (0 where a row sees nothing)."""
    n, _, _, lq, lk = mask.shape
    e = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale).view(n, k.shape[1], -1, lq, lk)
    e.masked_fill_(~mask, -math.inf)
    m = e.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e.sub_(m).exp_()
    return e, e.sum(-1, keepdim=True), m


def _plain_attention(s):
    c = s["c"]
    q, k, v, mask, (seq, at), _ = _padded(s)
    e, z, m = _probabilities(q, k, mask, s["scale"])
    o = torch.matmul(e.view(*q.shape[:3], -1), v).view(*e.shape[:4], -1) / torch.where(z == 0, 1.0, z)
    lse = (m + z.log())[..., 0]                     # [B][Hk][G][Lq]
    o = o[seq, :, :, at].reshape(-1, c["q_heads"], c["head_dim"]).to(torch.bfloat16)
    return o, lse[seq, :, :, at].reshape(-1, c["q_heads"]).t().contiguous()


def _plain_attention_backward(s):
    c = s["c"]
    q, k, v, mask, (seq, at), (qi, ql, kj, kl) = _padded(s)
    n, kh, _, hd = k.shape
    e, z, _ = _probabilities(q, k, mask, s["scale"])
    e.div_(torch.where(z == 0, 1.0, z))
    do = s["do"][qi].float().view(n, -1, kh, c["q_heads"] // kh, hd).permute(0, 2, 3, 1, 4).reshape(q.shape)
    p = e.view(*q.shape[:3], -1)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k).view(n, kh, -1, mask.shape[3], hd)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    t = torch.arange(s["k"].shape[0], device="cuda")
    sk = torch.bucketize(t, s["k_start"][1:].long(), right=True)
    ak = t - s["k_start"][:-1].long()[sk]
    dq = dq[seq, :, :, at].reshape(-1, c["q_heads"], hd)
    return dq.to(torch.bfloat16), dk[sk, :, ak].to(torch.bfloat16), dv[sk, :, ak].to(torch.bfloat16)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rope":
        return _turn(s["x"].double(), s, c["inverse"])
    if c["op"] in ("norm", "norm_append", "norm_bwd"):
        return _exact_norm(s)
    return _exact_attention(s)


def _turn(x, s, inverse):
    """The rotation as products of complex numbers."""
    cs = s["table"].double()[s["pos"].long()]
    z = torch.complex(cs[:, 0], cs[:, 1])[:, None]
    z = z.conj() if inverse else z
    half = z.shape[-1]
    y = x.clone()
    if s["c"]["layout"] == "half":
        w = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * z
        y[..., :half], y[..., half:2 * half] = w.real, w.imag
    else:
        w = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * z
        y[..., :2 * half] = torch.view_as_real(w).flatten(-2)
    return y


def _exact_norm(s):
    c = s["c"]
    qh, kh, hd = c["q_heads"], c["k_heads"], c["head_dim"]
    x = s["x"].double().view(-1, qh + 2 * kh, hd)
    out = []
    for part, w, d in ((x[:, :qh], s["wq"], "dq"), (x[:, qh:qh + kh], s["wk"], "dk")):
        w = w.double()
        norm = (part.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt()
        if c["op"] != "norm_bwd":
            out.append(_turn(part / norm * w, s, False))
            continue
        g = _turn(s[d].double(), s, True)
        dot = (g * w * part).sum(-1, keepdim=True)
        out.append((g * w / norm - part * dot / (hd * norm.pow(3)), (g * part / norm).flatten(0, 1).sum(0)))
    if c["op"] == "norm_bwd":
        return torch.cat((out[0][0], out[1][0]), dim=1), out[0][1], out[1][1]
    if c["op"] == "norm":
        return out[0], out[1]
    ck, cv = s["cache_k"].double(), s["cache_v"].double()
    for t, row in enumerate(s["rows"].tolist()):
        ck[row], cv[row] = out[1][t], x[t, qh + kh:]
    return out[0], ck, cv


def _exact_attention(s):
    c = s["c"]
    back = c["op"] == "attn_bwd"
    t, qh, kh, hd = c["q_tokens"], c["q_heads"], c["k_heads"], c["head_dim"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(t, qh, hd), torch.full((qh, t), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = new(t, qh, hd), new(s["k"].shape[0], kh, hd), new(s["k"].shape[0], kh, hd)
    ql, kl = _lengths(c)
    for b in range(c["sequences"]):
        q0, k0 = int(s["q_start"][b]), int(s["k_start"][b])
        for h in range(qh):
            hk = h * kh // qh
            k, v = s["k"][k0:k0 + kl[b], hk].double(), s["v"][k0:k0 + kl[b], hk].double()
            for lo in range(0, ql[b], 4096):
                hi = min(lo + 4096, ql[b])
                rows = slice(q0 + lo, q0 + hi)
                q = s["q"][rows, h].double()
                place = torch.arange(kl[b] - ql[b] + lo, kl[b] - ql[b] + hi, device="cuda")[:, None]
                key = torch.arange(kl[b], device="cuda")[None]
                gone = key > place
                if c["window"]:
                    gone = gone | ((place - key >= c["window"]) & (key >= c["sinks"]))
                x = (q @ k.T * s["scale"]).masked_fill(gone, -math.inf)
                if kl[b]:
                    lse[h, rows] = torch.logsumexp(x, dim=-1)
                p = torch.exp(x - lse[h, rows][:, None])
                p = torch.where(gone, 0.0, p)
                o[rows, h] = p @ v
                if back:
                    do = s["do"][rows, h].double()
                    dp = do @ v.T
                    ds = p * (dp - (do * o[rows, h]).sum(-1, keepdim=True)) * s["scale"]
                    dq[rows, h] = ds @ k
                    dk[k0:k0 + kl[b], hk] += ds.T @ q
                    dv[k0:k0 + kl[b], hk] += p.T @ do
    return (dq, dk, dv) if back else (o, lse)
