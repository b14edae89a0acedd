"""Gradients of attention in 64 bits, row by row, with bounds on the norm of each row's error.  Tests only.

A kernel that rounds dS and P to bf16 for their products is off by the sum of the roundings' products: errors of at most
U of each term, independent of each other, so that their norms add in quadrature.  (U = 2^-8 is the largest relative
rounding error and 2^-9.2 the one to be expected: twice the quadrature of U is over four deviations, which holds for
one direction as well as for a whole row.)  To that come the output's own rounding, at most U of it, the fp32 part, and
what D may be off in dq: at most 2^-6 of the root of the row's squared dS, times the row's mean key."""
import math

import torch

from attention_reference import E, U, f64, mask

D_SHARE = 2.0 ** -6


def inputs(kind, tokens, qh, kh, hd, seed):
    """q, k, v, do in bf16 on the CPU."""
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v, do = new(tokens, qh, hd), new(tokens, kh, hd), new(tokens, kh, hd), new(tokens, qh, hd) * 1e-3
    if kind == "means":                        # keys and values that share a direction
        k, v = k + 3 * new(1, kh, hd), v + 3 * new(1, kh, hd)
    elif kind == "dominating key":             # one key that takes most of every row, more or less of it
        u = new(1, 1, hd)
        u = 8 * u / u.norm()
        q = q + u
        k[3] = u[0] * (13 / 8) * (hd / 64) ** 0.5
    elif kind == "large queries":
        q = 8 * q
    elif kind == "tiny":                       # gradients whose squares leave fp32
        k, v, do = k + 3 * new(1, kh, hd), v + 3 * new(1, kh, hd), do * 1e-21
    return [t.to(torch.bfloat16) for t in (q, k, v, do)]


KINDS = ["independent", "means", "dominating key", "large queries", "tiny"]


def rows(x):
    return x.norm(dim=-1)


class Exact:
    """Gradients of packed sequences of equal queries and keys: dq [T][Hq][hd], dk, dv, and bounds [T][H] of each row's error."""

    def __init__(self, q, k, v, do, lengths, window=0, sinks=0, d_from=None, rounded=False):
        """rounded: P and dS are rounded to bf16, as a kernel does; d_from: o that D is taken from (None: the exact one)."""
        q, k, v, do = (f64(t) for t in (q, k, v, do))
        T, qh, hd = q.shape
        kh = k.shape[1]
        scale = hd ** -0.5
        z = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
        self.dq, self.dk, self.dv, self.o = z(T, qh, hd), z(T, kh, hd), z(T, kh, hd), z(T, qh, hd)
        bq, bk, bv = z(T, qh), z(T, kh), z(T, kh)           # squares of what adds up in quadrature
        eq = z(T, qh)
        r = (lambda t: t.to(torch.bfloat16).double()) if rounded else (lambda t: t)
        q0 = 0
        for n in lengths:
            s, q0 = slice(q0, q0 + n), q0 + n
            m = mask(n, n, window, sinks)
            for h in range(qh):
                g = h * kh // qh
                Q, K, V, O = q[s, h], k[s, g], v[s, g], do[s, h]
                S = (scale * (Q @ K.T)).masked_fill(~m, -math.inf)
                lse = torch.logsumexp(S, -1, keepdim=True)
                P = torch.exp(S - lse)
                self.o[s, h] = P @ V
                dP = O @ V.T
                D = (O * (self.o[s, h] if d_from is None else f64(d_from[s, h]))).sum(-1, keepdim=True)
                dS = P * (dP - D)
                self.dq[s, h] = scale * (r(dS) @ K)
                self.dk[s, g] += scale * (r(dS).T @ Q)
                self.dv[s, g] += r(P).T @ O
                # fp32: S and lse to a few units of their magnitude, in P; dP and D by sums of hd products
                eP = 8 * E * (1 + lse.abs() + S.masked_fill(~m, 0.0).abs().amax(-1, keepdim=True))
                eS = P * (4 * hd ** 0.5 * E) * (rows(O)[:, None] * rows(V) + D.abs()) + eP * dS.abs()
                t = (2 * U * dS.abs() + eS).square()
                bq[s, h] = scale ** 2 * (t @ rows(K).square())
                bk[s, g] += scale ** 2 * (t.T @ rows(Q).square())
                bv[s, g] += ((2 * U + eP) * P).square().T @ rows(O).square()
                eq[s, h] = scale * D_SHARE * rows(dS) * rows(P @ K)
        self.bound_dq = bq.sqrt() + eq + 2 * U * rows(self.dq)
        self.bound_dk = bk.sqrt() + 2 * U * rows(self.dk)
        self.bound_dv = bv.sqrt() + 2 * U * rows(self.dv)

    def worst(self, name, got):
        """The largest error of a row over its bound."""
        err = rows(f64(got) - getattr(self, name))
        return float((err / (getattr(self, "bound_" + name) + 1e-40)).max())

    def check(self, dq, dk, dv):
        for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            assert self.worst(name, got) <= 1.0, "%s: error of a row %.2f of its bound" % (name, self.worst(name, got))
