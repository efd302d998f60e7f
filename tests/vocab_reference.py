"""The vocabulary losses and their gradients from the formulas, in 64 bits on the
CPU, with bounds on how far a computation in the library's number formats can be.

Bounds (first order, u32 = 2^-24):
  products  FP32 accumulation of K products in any order, each step rounded or
            truncated (2 u32 of the magnitude so far), and operands that enter as
            bfloat16 parts: |err| <= (K + 16) 2 u32 sum |a||b|. Two parts only
            (SGEMM_MATH_TF32): 2^-15 sum |a||b| more.
  logits    ez = the largest such bound over a token's row, times the scale.
  lse       ez + 2^-21 (1 + |lse|): the exponentials and their sum are relative
            errors of a few units, the logarithm and the last sum one each.
  loss      factor * (the target's ez + that of lse + 2^-21 |log p| + 2^-21 |log q|).
  p         relative: ep = ez + (error of lse) + 2^-21 (1 + |log p|).
  dZ        |g| (p ep + 2^-21 q) + ud |dZ|, where ud = 2^-8 for bfloat16 (rounded to 8
            bits), 2^-22 for three parts, 2^-15 for two.
  dH, dW    sum of those times the other operand, the product bound with K = V or T
            and |dZ|, and the rounding of the result (2^-8 or u32 of it).
"""

import math

import torch

U = 2.0 ** -24
FEW = 2.0 ** -21


def reference(H, W, scale, factor, ids, q, logq, dloss=None, two_parts=False, bf16=False):
    """ids / q / logq: (T, n) targets, id -1 where there is none (q = 0). Returns {name: (value, bound)}."""
    H, W = H.detach().cpu().double(), W.detach().cpu().double()
    T, D = H.shape
    V = W.shape[0]
    ids, q, logq = ids.cpu(), q.cpu().double(), logq.cpu().double()
    extra = 2.0 ** -15 if two_parts else 0.0

    def product_bound(a, b, k):
        return ((k + 16) * 2 * U + extra) * (a.abs() @ b.abs())

    z = scale * (H @ W.T)
    ez = abs(scale) * product_bound(H, W.T, D).amax(1)
    lse = torch.logsumexp(z, 1)
    elo = ez + FEW * (1 + lse.abs())
    real = ids >= 0
    at = ids.clamp_min(0)
    logp = z - lse[:, None]
    logpt = logp.gather(1, at)
    term = torch.where(q > 0, q * (logq - logpt), 0.0)
    eterm = torch.where(q > 0, q * ((ez + elo)[:, None] + FEW * (logpt.abs() + logq.abs() + 1)), 0.0)
    out = {"lse": (lse, elo), "loss": (factor * term.sum(1), factor * eterm.sum(1) + U * (factor * term.sum(1)).abs())}
    if dloss is None:
        return out
    used = real.any(1)
    g = torch.where(used, factor * scale * dloss.cpu().double(), 0.0)[:, None]
    p = logp.exp()
    qs = torch.zeros_like(p).scatter_add_(1, at, torch.where(real, q, 0.0))
    dz = g * (p - qs)
    ud = 2.0 ** -8 if bf16 else 2.0 ** -15 if two_parts else 2.0 ** -22
    ep = (ez + elo)[:, None] + FEW * (1 + logp.abs())
    edz = g.abs() * (p * ep + FEW * qs) + ud * dz.abs()
    uo = 2.0 ** -8 if bf16 else U
    dH, dW = dz @ W, dz.T @ H
    out["dH"] = (dH, edz @ W.abs() + product_bound(dz, W, V) + uo * dH.abs())
    out["dW"] = (dW, edz.T @ H.abs() + product_bound(dz.T, H, T) + uo * dW.abs())
    return out


def xent_targets(labels, V):
    """Targets of the cross entropy: one of weight 1 where the label is in the vocabulary."""
    labels = labels.cpu()
    ok = (labels >= 0) & (labels < V)
    return torch.where(ok, labels, -1)[:, None], ok.double()[:, None], torch.zeros(len(labels), 1, dtype=torch.float64)


def teacher_targets(ids, logits, temperature, V):
    """Targets of the distillation: the softmax over the entries that count."""
    ids, logits = ids.cpu(), logits.cpu().double()
    ok = (ids >= 0) & (ids < V) & (torch.where(ids >= 0, logits, 0.0) > -math.inf)
    t = torch.where(ok, logits, 0.0) / temperature
    t = torch.where(ok, t, -math.inf)
    some = ok.any(1, keepdim=True)
    t = t - torch.where(some, t.amax(1, keepdim=True), 0.0)  # first: next to 1e38 the log of the sum would vanish
    logq = torch.where(ok, t - torch.logsumexp(torch.where(some, t, 0.0), 1, keepdim=True), 0.0)
    q = torch.where(ok, logq.exp(), 0.0)
    return torch.where(ok, ids, -1), q, logq


def check(name, got, ref):
    """Assert one output against its value and bound (NaN where the value is)."""
    value, bound = ref
    got = got.detach().cpu().double()
    assert got.shape == value.shape, name
    off = (got - value).abs()
    bad = ~(off <= bound) & ~(torch.isnan(got) & torch.isnan(value))
    worst = (off / bound.clamp_min(1e-300))[bad]
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {worst.max().item():.3g} x"
