"""Error bounds for the attention with modified scores where a cap saturates and where a row's
differences dP - D are small beside |do| |o|: narrower than those of tests/attention_mod_ref.py, whose
allowance for D and dP leaves out the factor 1 - t^2 that every kernel multiplies them by, and which
allows o's rounding in D although the backward corrects it.

Counted to first order (h = finfo(type).eps / 2, u = 2^-24, z half a subnormal step of the type, t = tanh(x / cap),
w = 1 - t^2; 1 and 0 in their place without a cap):

  raw score  e_x = u (D + 8) scale |q|.|k|: D exact products summed in 32 bits, the scale
  edge       w at |x / cap| - e_x / cap, the largest derivative within the raw score's error
  score      e_s = e_x edge + u (16 cap + 4 slope |pos - j| + 8 |s| + 4)
  P          relative p_i = 2 max_j e_s + u (n + 16)
  w          absolute e_w = 2 edge e_x / cap + 12 u: the raw score's error; t is off by 4 u at most (tanh as
             1 - 2 / (1 + e^2x) within 2^-22), t^2 by 8 u, and four roundings behind that
  lse        max_j e_s + u (n + 8 + 2 |lse|)
  o          (h + p_i + u n) sum_j P |v| + z sum_j |v| + h |o| + z
  dv         sum_i (h + p_i + u n) P |do| + z sum |do| + h |dv| + z
  D          o as it was rounded is off by e_o = |do| . (bound of o) + u (D + 2) |do|.|o|; corrected by
             r = sum_j P (dP - D), which leaves
             e_d = p_i sum_j P |dP - D| + sum_j P (u (D + 2) |do|.|v| + u (n + 16) (|dP| + |D|))
                   + 2^-11 sum_j P t^2 |dP - D| + 2^-39 sum_j (|dP| + |D|)
             (with a cap r takes P t^2 2^14 as fp16, which steps by 2^-10, half of it is the rounding, and by 2^-24 where
             it is subnormal)
  dS         (h + p_i) |dS| + z + 2^-126 w (|dP| + |D|) + P w (u (D + 2) |do|.|v| + e_d + 2 h e_o + 16 u (|dP| + |D|))
             + P e_w (|dP| + |D|)
             (2 h e_o: dS is rounded to the type before the correction, and so is the P w that carries it)
  dq         scale (sum_j e_dS |k| + u n sum_j |dS| |k|) + h |dq| + z;  dk likewise over i
"""
import math

import torch

U = 2.0 ** -24


def reference(q, k, v, scale, seen, pos, softcap=0.0, slopes=None, d_o=None):
    """As tests.attention_mod_ref.reference: {name: (value, bound)} in 64 bits.  An infinite element of k, which
    only a cap makes a finite score of, is taken as 2^500 (times the sign)."""
    dt = q.dtype
    h = torch.finfo(dt).eps / 2
    z = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -126
    B, H, n, D = q.shape
    heads = k.shape[1]
    m = k.shape[2]
    g = H // heads
    kd = torch.where(seen.any(1)[:, None, :, None], k.double().clamp(-2.0 ** 500, 2.0 ** 500), 0.0)
    vd = torch.where(seen.any(1)[:, None, :, None], v.double(), 0.0)
    kd, vd = kd.repeat_interleave(g, 1), vd.repeat_interleave(g, 1)
    rows = seen.any(2)[:, None, :, None]
    qd = torch.where(rows, q.double(), 0.0)
    sn = seen[:, None]
    x = scale * (qd @ kd.transpose(-1, -2))
    ex = U * (D + 8) * scale * (qd.abs() @ kd.abs().transpose(-1, -2))
    w, edge, ew = 1.0, 1.0, torch.zeros_like(x)
    if softcap > 0:
        t = torch.tanh(x / softcap)
        w = 1 - t * t
        edge = 1 - torch.tanh(((x.abs() - ex) / softcap).clamp_min(0.0)) ** 2
        ew = 2 * edge * ex / softcap + 12 * U
        x = softcap * t
    far = (pos[:, :, None] - torch.arange(m, device=q.device)).abs().double()[:, None]
    bias = 0.0 if slopes is None else slopes.double()[None, :, None, None] * far
    s = (x - bias).masked_fill(~sn, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isneginf(top), 0.0, top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    o = p @ vd
    es = torch.where(sn, ex * edge + U * (16 * softcap + 4 * abs(bias) + 8 * torch.where(sn, s.abs(), 0.0) + 4), 0.0)
    worst = es.amax(-1, keepdim=True)
    pi = 2 * worst + U * (m + 16)
    lse_b = worst[..., 0] + U * (m + 8 + 2 * torch.where(torch.isinf(lse), 0.0, lse.abs()))
    ob = (h + pi + U * m) * (p @ vd.abs()) + z * (sn.double() @ vd.abs()) + h * o.abs() + z
    out = {"o": (o, ob), "lse": (lse, lse_b)}
    if d_o is None:
        return out
    gd = torch.where(rows, d_o.double(), 0.0)

    def group(a):
        return a.reshape(B, heads, g, *a.shape[2:]).sum(2)

    dv = group(p.transpose(-1, -2) @ gd)
    dvb = group((p * (h + pi + U * n)).transpose(-1, -2) @ gd.abs() + z * (sn.double().transpose(-1, -2) @ gd.abs()))
    dP = gd @ vd.transpose(-1, -2)
    delta = (gd * o).sum(-1, keepdim=True)
    dS = p * (dP - delta) * w
    size = torch.where(sn, dP.abs() + delta.abs(), 0.0)
    prod = U * (D + 2) * (gd.abs() @ vd.abs().transpose(-1, -2))
    eo = (gd.abs() * ob).sum(-1, keepdim=True) + U * (D + 2) * (gd.abs() * o.abs()).sum(-1, keepdim=True)
    ed = pi * (p * (dP - delta).abs()).sum(-1, keepdim=True) + (p * (prod + U * (m + 16) * size)).sum(-1, keepdim=True)
    if softcap > 0:
        ed = ed + (2.0 ** -11 * p * (1 - w) * (dP - delta).abs() + 2.0 ** -39 * size).sum(-1, keepdim=True)
    dsb = (h + pi) * dS.abs() + torch.where(sn, z, 0.0) + 2.0 ** -126 * w * size \
        + p * w * (prod + ed + 2 * h * eo + 16 * U * size) + p * ew * size
    dq = scale * (dS @ kd)
    dqb = scale * ((dsb + U * m * dS.abs()) @ kd.abs()) + h * dq.abs() + z
    dk = scale * group(dS.transpose(-1, -2) @ qd)
    dkb = scale * group((dsb + U * n * dS.abs()).transpose(-1, -2) @ qd.abs()) + h * dk.abs() + z
    out.update(dq=(dq, dqb), dk=(dk, dkb), dv=(dv, dvb + h * dv.abs() + z))
    return out
