"""Float64 definitions and error bounds of the packed and paged attention tests.

Bounds, derived from the roundings of the method (h = 2^-8, half a bf16 step
relative to the value; e = 2^-14 for the float32 steps together: scores of up to
a few hundred units in the exponent at 2^-24 each, exp2 within 2^-22, sums):
  P is rounded to bf16         |dO|   <= (h + e) sum_j p_j |v_j| + h |o|
  lse is float32               |dlse| <= 2^-20 (1 + |lse|) + 2^-18
  delta = dout . o, o rounded  |dD|   <= sum_d |dout_d| (bound of o_d)
  dS = P (dP - D), rounded     |ddS|  <= (h + e) |dS| + P |dD| + e P (|dout| . |v| + |D|)
  dQ, dK from dS, dV from P, each rounded once more at the end."""
import math

import torch

H, E = 2.0 ** -8, 2.0 ** -14


def attention(q, k, v, scale, keep, dout=None):
    """q [Lq, D], k, v [Lk, D] float64, keep [Lq, Lk] bool.  Returns a dict of
    values and bounds (o, lse, and with dout the gradients)."""
    x = (q @ k.T) * scale
    x = x.masked_fill(~keep, -math.inf)
    m = x.amax(1, keepdim=True) if x.shape[1] else torch.full_like(x[:, :1], -math.inf)
    if x.shape[1] == 0:
        m = torch.full((q.shape[0], 1), -math.inf, dtype=q.dtype, device=q.device)
    mm = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - mm).exp()
    t = p.sum(1, keepdim=True)
    p = p / torch.where(t == 0, torch.ones_like(t), t)
    o = p @ v
    out = {"o": o, "lse": (mm + t.log())[:, 0], "o_tol": (H + E) * (p @ v.abs()) + H * o.abs()}
    if dout is not None:
        dp = dout @ v.T
        delta = (dout * o).sum(1, keepdim=True)
        ds = p * (dp - delta)
        ddelta = (dout.abs() * out["o_tol"]).sum(1, keepdim=True)
        dds = (H + E) * ds.abs() + p * ddelta + E * p * (dout.abs() @ v.abs().T + delta.abs())
        out["dq"], out["dk"], out["dv"] = ds @ k * scale, ds.T @ q * scale, p.T @ dout
        out["dq_tol"] = dds @ k.abs() * scale
        out["dk_tol"] = dds.T @ q.abs() * scale
        out["dv_tol"] = (H + E) * (p.T @ dout.abs())
    return out


def keep_mask(Lq, Lk, causal, device):
    i = torch.arange(Lq, device=device)[:, None]
    j = torch.arange(Lk, device=device)[None]
    return (j <= i + Lk - Lq) if causal else torch.ones(Lq, Lk, dtype=torch.bool, device=device)


def packed(q, k, v, cu_q, cu_k, causal, scale=None, dout=None):
    """Values and bounds over packed tensors; rows of no sequence stay NaN."""
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    G = q.shape[1] // k.shape[1]
    d = torch.float64
    nan = lambda t: torch.full(t.shape, math.nan, dtype=d, device=q.device)
    r = {"o": nan(q), "o_tol": nan(q),
         "lse": torch.full((q.shape[1], q.shape[0]), math.nan, dtype=d, device=q.device)}
    if dout is not None:
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_tol"] = nan(t), nan(t)
    for a, b, c, e in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        if dout is not None:
            for n in ("dk", "dk_tol", "dv", "dv_tol"):
                r[n][c:e] = 0
        for h in range(q.shape[1]):
            x = attention(q[a:b, h].to(d), k[c:e, h // G].to(d), v[c:e, h // G].to(d), scale,
                          keep_mask(b - a, e - c, causal, q.device),
                          None if dout is None else dout[a:b, h].to(d))
            r["o"][a:b, h], r["o_tol"][a:b, h], r["lse"][h, a:b] = x["o"], x["o_tol"], x["lse"]
            if dout is not None:
                r["dq"][a:b, h], r["dq_tol"][a:b, h] = x["dq"], x["dq_tol"]
                for n in ("dk", "dv"):
                    r[n][c:e, h // G] += x[n]
                    r[n + "_tol"][c:e, h // G] += x[n + "_tol"]
    if dout is not None:
        for n in ("dq", "dk", "dv"):
            r[n + "_tol"] += H * r[n].abs()
    return r


def check(got, want, tol, name):
    """Within tol where `want` is a number; rows of no sequence are not looked at."""
    live = ~torch.isnan(want)
    g, w = got.double()[live], want[live]
    same = g == w  # -inf among them
    t = tol[live] if torch.is_tensor(tol) else tol
    over = torch.where(same, torch.zeros_like(w), (g - w).abs() - t)
    over = torch.where(torch.isnan(over), torch.full_like(over, math.inf), over)
    assert over.numel() == 0 or float(over.max()) <= 1e-30, "%s exceeds its bound by %.3g" % (
        name, float(over.max()))


def check_lse(got, want):
    check(got, want, 2.0 ** -20 * (1 + want.abs()) + 2.0 ** -18, "lse")
