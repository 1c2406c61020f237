"""Plain 64-bit attention and the error bounds that the kernels are held to.

Bounds (u = unit roundoff, half a step: bf16 2^-8, fp32 2^-24), per output
element, with a = sum_j p_j |v_j| / l >= |o|:
  logits      an fp32 dot product of 128 terms, scaled, less the maximum: off by
              at most e0 = (128 + 8) 2^-24 (scale sum_d |q_d k_d| + |scale q.k|)
  p           relative error of e0 from its logit, 2^-21 from the fp32 exponential
  sums        n fp32 additions in any order: n 2^-24 relative to the sum of moduli
  bf16        p rounded to bf16 for the product (2^-8 of p), o rounded (2^-8 of |o|)
so |out - o| <= (2 (e0 + 2^-21 + n 2^-24) + u_p) a + u_o |o|, and
|lse - exact| <= e0 + 2^-21 + n 2^-24 + 2^-22 |lse|."""
import math

import torch

U = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


def attend(q, k, v, seen, scale):
    """q [r, 128], k, v [c, 128] (any type), seen bool [r, c]: 64-bit out, lse, the
    bound of out for bf16 / fp32 outputs (by q's dtype) and of lse."""
    dt = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    # masked values do not take part, whatever they are
    some = seen.any(0)
    k, v = torch.where(some[:, None], k, 0.0), torch.where(some[:, None], v, 0.0)
    s = scale * (q @ k.T)
    s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, 1) if s.shape[1] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    o, a = p @ v, p @ v.abs()
    n = max(1, s.shape[1])
    mod = scale * (q.abs() @ k.abs().T)
    e0 = 136 * 2.0**-24 * 2 * (torch.where(seen, mod, 0.0).amax(1) if s.shape[1] else torch.zeros_like(lse))
    e = e0 + 2.0**-21 + n * 2.0**-24
    u = U[dt]
    up = u if dt == torch.bfloat16 else 0.0
    tol = (2 * e[:, None] + up) * a + u * o.abs()
    return o, lse, tol, e + 2.0**-22 * torch.where(lse == -math.inf, 0.0, lse).abs()


def check(out, lse, ref):
    o, x, tol, tol_lse = ref
    assert torch.isfinite(out).all()
    d = (out.double() - o).abs() - tol
    assert (d <= 0).all(), ("out", float(d.max()), float(tol.max()))
    empty = x == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (out[empty] == 0).all()
    d = torch.where(empty, 0.0, (lse.double() - x).abs() - tol_lse)
    assert (d <= 0).all(), ("lse", float(d.max()))
