"""Plain 64-bit implementations of the attention block's operators, on the CPU, and
the error bounds that the GPU's outputs are held to.  Tests only: no code shared with
the library.

The bounds follow from the operators' roundings.  U = 2^-8 is bf16's largest relative
rounding error and E = 2^-24 fp32's.  A result held in fp32 and rounded once to bf16
differs from the exact one by at most U |y| (1 + U) plus the fp32 part, which each
bound states in terms of the magnitudes that were added up."""
import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64)


# ---------------------------------------------------------------- rotation, norms
def table(positions, rot, base=10000.0, scaling="none", factor=1.0, trained=0):
    """Cosines and sines in 64 bits, [positions][2][rot/2], one frequency at a time."""
    out = torch.zeros(positions, 2, rot // 2, dtype=torch.float64)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    b = base * factor ** (rot / (rot - 2.0)) if scaling == "ntk" else base
    p = torch.arange(positions, dtype=torch.float64)
    for i in range(rot // 2):
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "yarn":
            turns = trained * f / (2.0 * math.pi)
            keep = min(max((turns - 1.0) / 31.0, 0.0), 1.0)
            f = f / factor * (1.0 - keep) + f * keep
        out[:, 0, i], out[:, 1, i] = m * torch.cos(p * f), m * torch.sin(p * f)
    return out


def pairs(rot, layout):
    half = rot // 2
    return [(i, i + half) for i in range(half)] if layout == "half" else [(2 * i, 2 * i + 1) for i in range(half)]


def rotate(x, tab, pos, layout, inverse=False):
    """x [T][H][hd] (64 bits), tab [P][2][rot/2] -> rotated, pair by pair."""
    y = x.clone()
    rot = 2 * tab.shape[2]
    for i, (a, b) in enumerate(pairs(rot, layout)):
        c, s = tab[pos.long(), 0, i][:, None], tab[pos.long(), 1, i][:, None]
        s = -s if inverse else s
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def partner_sum(x, rot, layout):
    """|a| + |b| of each element's pair: the magnitudes a rotated value is made of."""
    y = x.abs().clone()
    for a, b in pairs(rot, layout):
        y[:, :, a] = y[:, :, b] = x[:, :, a].abs() + x[:, :, b].abs()
    return y


def norm(x, w, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w


def norm_backward(g, x, w, eps):
    """g: the gradient of norm's result -> (dx, dw, |terms| of dw)."""
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    h = x * r
    dx = r * (w * g - h * (w * g * h).mean(-1, keepdim=True))
    return dx, (g * h).sum((0, 1)), (g * h).abs().sum((0, 1))


# ---------------------------------------------------------------- attention
def mask(ql, kl, window, sinks):
    p = torch.arange(ql)[:, None] + (kl - ql)
    j = torch.arange(kl)[None]
    return (j <= p) & ((j > p - window) | (j < sinks) if window else torch.ones(1, 1, dtype=torch.bool))


def attention(q, k, v, seqs, window=0, sinks=0, scale=None, do=None, bounds=False):
    """q [T][Hq][hd], k, v [S][Hk][hd]; seqs: (first query, queries, first key, keys) of each sequence.

    Returns a dict of 64-bit tensors: o, lse [Hq][T] and, with do, dq, dk, dv; with bounds also the error bounds
    (``b_o``, ``b_lse``, ...) of outputs computed as the kernels do: bf16 operands, fp32 sums, the probabilities and
    dS rounded to bf16 for their products, o rounded to bf16 before D.  Rows and keys of no sequence hold NaN."""
    q, k, v = f64(q), f64(k), f64(v)
    do = None if do is None else f64(do)
    T, hq, hd = q.shape
    S, hk, _ = k.shape
    scale = hd ** -0.5 if scale is None else scale
    nan = float("nan")
    full = lambda *s: torch.full(s, nan, dtype=torch.float64)  # noqa: E731
    r = {"o": full(T, hq, hd), "lse": full(hq, T)}
    if do is not None:
        r.update(dq=full(T, hq, hd), dk=full(S, hk, hd), dv=full(S, hk, hd))
    if bounds:
        r.update({"b_" + n: torch.zeros_like(t) for n, t in list(r.items())})
    for q0, ql, k0, kl in seqs:
        m = mask(ql, kl, window, sinks)
        if do is not None:
            r["dk"][k0:k0 + kl] = r["dv"][k0:k0 + kl] = 0.0
        for h in range(hq):
            g = h * hk // hq
            Q, K, V = q[q0:q0 + ql, h], k[k0:k0 + kl, g].clone(), v[k0:k0 + kl, g].clone()
            seen = m.any(0)
            K[~seen], V[~seen] = 0.0, 0.0                    # rows that nothing sees have no part
            s = (scale * (Q @ K.T)).masked_fill(~m, -math.inf)
            lse = torch.logsumexp(s, -1) if kl else torch.full((ql,), -math.inf, dtype=torch.float64)
            P = torch.where(m, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
            o = P @ V
            r["o"][q0:q0 + ql, h], r["lse"][h, q0:q0 + ql] = o, lse
            if bounds:
                # fp32 sums of hd products, then the scaling, the difference to the maximum and exp2.
                es = (hd + 8) * E * (scale * (Q.abs() @ K.abs().T)).amax(-1, keepdim=True).clamp(min=1.0) * 2.0 if kl else 0.0
                eP = es + (kl + 8) * E
                mag = P @ V.abs()
                b = (U + 2 * eP) * mag * (1 + U) + U * o.abs() * (1 + 4 * U)
                r["b_o"][q0:q0 + ql, h] = b
                r["b_lse"][h, q0:q0 + ql] = torch.where(lse == -math.inf, 0.0, ((es + (kl + 8) * E) if kl else torch.zeros(ql, 1, dtype=torch.float64))[:, 0]
                                                        + 4 * E * lse.abs().clamp(max=1e30))
            if do is None:
                continue
            dO = do[q0:q0 + ql, h]
            dP = dO @ V.T
            D = (dO * o).sum(-1, keepdim=True)
            dS = P * (dP - D)
            r["dq"][q0:q0 + ql, h] = scale * (dS @ K)
            r["dk"][k0:k0 + kl, g] += scale * (dS.T @ Q)
            r["dv"][k0:k0 + kl, g] += P.T @ dO
            if bounds:
                eD = (dO.abs() * b).sum(-1, keepdim=True) \
                    + 2 * hd * E * (dO.abs() * o.abs()).sum(-1, keepdim=True)
                # lse in fp32 as the forward call wrote it, S, dP and D in fp32; dS rounded to bf16.
                elP = 2 * eP + 8 * E * torch.where(lse == -math.inf, 0.0, lse).abs()[:, None]
                edP = 2 * hd * E * (dO.abs() @ V.abs().T)
                eS = dS.abs() * (U + elP) * (1 + U) + P * (eD + edP) * (1 + U)
                r["b_dq"][q0:q0 + ql, h] = scale * (eS @ K.abs()) * (1 + U)
                r["b_dk"][k0:k0 + kl, g] += scale * (eS.T @ Q.abs()) * (1 + U)
                r["b_dv"][k0:k0 + kl, g] += (P.T * (U + elP.T)) @ dO.abs() * (1 + U)
                # the fp32 sums themselves
                r["b_dq"][q0:q0 + ql, h] += 2 * (kl + 8) * E * scale * (dS.abs() @ K.abs())
                r["b_dk"][k0:k0 + kl, g] += 2 * (ql * hq + 8) * E * scale * (dS.abs().T @ Q.abs())
                r["b_dv"][k0:k0 + kl, g] += 2 * (ql * hq + 8) * E * (P.T @ dO.abs())
    if bounds and do is not None:
        for n in ("dq", "dk", "dv"):
            r["b_" + n] += U * r[n].abs() * (1 + 4 * U)       # the output's rounding
    return r


def check(got, want, bound, what, floor=1e-37):
    """Every element within its bound; infinities where the reference has them; rows of no sequence (NaN) skipped."""
    got = f64(got)
    known = ~torch.isnan(want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities differ"
    use = known & ~inf
    bad = ~((got[use] - want[use]).abs() <= bound[use] + floor)
    if bad.any():
        i = int(bad.nonzero()[0])
        raise AssertionError("%s: %d of %d elements outside their bound, first: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), float(got[use][i]), float(want[use][i]), float(bound[use][i])))
