"""Fused attention and its gradients in 64 bits from their definitions, with
the distance that the kernels' roundings may put between the two.

The kernels round twice to bf16 besides their result: the weights P (forward,
grad_values) and dS (grad_query, grad_keys), each by at most half a step,
2^-8 of the value.  A sum of n such products errs by the sum of independent
roundings c_j, |c_j| <= 2^-8 |P_j v_j|: beyond 7 sqrt(sum c_j^2) with a
probability below 2 e^(-49/2) < 1e-10 per element (Hoeffding).  fp32 parts:
a dot product of D terms errs by at most (D + 8) 2^-23 of the sum of its
terms' magnitudes (accumulation in any order, one bit spare for a truncating
accumulator), 2^x by 2^-21, and the running sums are bounded below by
2^-18 of the sum of magnitudes (n <= 4096 terms of half a step, mostly
cancelling; 64 n would be needed to exceed it).  Numbers below 2^-126 are
flushed to zero, by 2^x and as operands: a P or dS errs by up to 2^-126
whatever its size, which shows only where nothing larger is summed."""
import math

import torch

HALF = 2.0 ** -8     # half a step of bf16
F32 = 2.0 ** -23
SUMS = 2.0 ** -18
FLUSH = 2.0 ** -126


def kept_pairs(mask, causal, B, Sq, Sk):
    kept = torch.ones(B, 1, Sq, Sk, dtype=torch.bool)
    if causal:
        i = torch.arange(Sq)[:, None]
        kept &= torch.arange(Sk)[None, :] <= i + (Sk - Sq)
    if mask is not None:
        kept &= mask.cpu()[:, None, None, :]
    return kept


def _wide(x, group=1):
    return x.detach().cpu().double().repeat_interleave(group, 1)


class Forward:
    """out, lse of the definition and the kernels' allowances."""

    def __init__(self, q, k, v, mask, causal, scale):
        B, H, Sq, D = q.shape
        self.group = H // k.shape[1]
        self.q, self.D, self.scale = _wide(q), D, scale
        self.k, self.v = _wide(k, self.group), _wide(v, self.group)
        self.kept = kept_pairs(mask, causal, B, Sq, k.shape[2])
        if mask is not None:   # what removed keys hold has no effect
            gone = ~mask.cpu()[:, None, :, None]
            self.k = self.k.masked_fill(gone, 0.0)
            self.v = self.v.masked_fill(gone, 0.0)
        s = self.q @ self.k.mT * scale
        s = s.masked_fill(~self.kept, -math.inf)
        self.lse = torch.logsumexp(s, -1)
        self.P = torch.exp(s - self.lse[..., None].nan_to_num(neginf=0.0))
        self.out = self.P @ self.v
        # Largest error of a score of the row, and of its exponent.
        self.ds = ((D + 8) * F32 * scale
                   * (self.q.abs() @ self.k.abs().mT).amax(-1)
                   if k.shape[2] else torch.zeros(B, H, Sq).double())
        m = s.amax(-1).abs() if k.shape[2] else torch.zeros(B, H, Sq)
        m = torch.where(m == math.inf, 0.0, m)
        # e^(s - m) from fp32 s c - m c: one rounding of each product.
        self.es = 2 * self.ds + 4 * F32 * m + 2.0 ** -21 + SUMS

    def out_tol(self):
        c = torch.sqrt((self.P ** 2) @ (self.v ** 2))
        return (HALF * self.out.abs() + 7 * HALF * c
                + self.es[..., None] * 2 * (self.P @ self.v.abs()) + 1e-37)

    def lse_tol(self):
        lse = self.lse.abs()
        return self.es + 4 * F32 * torch.where(lse == math.inf, 0.0, lse)


def gradients(f, out, g):
    """(dq, dk, dv) of the definition at the given (rounded) out, and their
    allowances."""
    o, g = _wide(out), _wide(g)
    B, Hk = f.k.shape[0], f.k.shape[1] // f.group
    dP = g @ f.v.mT
    delta = (g * o).sum(-1, keepdim=True)
    dS = f.P * (dP - delta)
    # fp32 errors of dS: P's relative one, and those of the two dot products.
    dot = (f.D + 8) * F32 * (g.abs() @ f.v.abs().mT
                             + (g * o).abs().sum(-1, keepdim=True))
    # P flushed shows as much as G V^T - delta is large, dS flushed once more.
    eS = (dS.abs() * f.es[..., None] + f.P * dot
          + FLUSH * ((dP - delta).abs() + 1))

    def fold(x):
        return x.reshape(B, Hk, f.group, *x.shape[2:]).sum(2)

    def tol(value, weights, err, other):
        c = torch.sqrt(fold_or((weights ** 2) @ (other ** 2)))
        return (HALF * value.abs() + 7 * HALF * c
                + fold_or(err @ other.abs()) + SUMS * fold_or(
                    weights.abs() @ other.abs()) + 1e-37)

    fold_or = lambda x: x                                     # noqa: E731
    dq = dS @ f.k
    tq = tol(dq, dS, eS, f.k) * f.scale
    fold_or = fold
    dk, dv = fold(dS.mT @ f.q), fold(f.P.mT @ g)
    tk = tol(dk, dS.mT, eS.mT, f.q) * f.scale
    tv = tol(dv, f.P.mT, (f.P * f.es[..., None] + 2 * FLUSH).mT, g)
    return (dq * f.scale, dk * f.scale, dv), (tq, tk, tv)


def excess(x, ref, tol):
    """The largest |x - ref| / tol (NaN counts as infinite)."""
    if not ref.numel():
        return 0.0
    r = (x.detach().cpu().double() - ref).abs() / tol
    return float(r.nan_to_num(nan=math.inf).max())
