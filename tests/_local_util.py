"""Plain 64-bit references (CPU, torch) of the norm-and-rotation, window
attention and decoding operators, with the error bounds of their kernels.

Bounds count roundings: bf16 storage of an output is off by at most 2^-8 of
the value; P and dS are rounded to bf16 as tensor-core operands, so a sum
over them is off by at most 2^-8 (dS: twice, through P and itself) of the
same sum of absolute values.  What remains is fp32 arithmetic."""
import math

import numpy as np
import torch

import oracle

BF = 2.0 ** -8   # half a step of bf16, relative
F32 = 2.0 ** -24


def positions(S, N, layout):
    return torch.as_tensor(np.asarray(oracle.layout_positions(S, N, layout)).astype(np.int64))


def keep_mask(qpos, kpos, window, sinks):
    """[.., queries, keys]; window 0: plain causal."""
    q, k = qpos[..., :, None], kpos[..., None, :]
    keep = k <= q
    if window:
        keep = keep & ((q - k < window) | (k < sinks))
    return keep


def attention(q, k, v, keep, scale):
    """One head in fp64: (o, lse, p); rows without a kept key give 0 and -inf."""
    s = (q @ k.T * scale).masked_fill(~keep, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    p = torch.where(z > 0, e / z, torch.zeros_like(e))
    return p @ v, (m + z.log())[:, 0], p


def window_reference(q, k, v, pos, window, sinks, scale, dO=None, o_given=None):
    """[B,H,S,D] tensors in placed rows -> dict of fp64 results and bounds."""
    B, H, S, D = q.shape
    G = H // k.shape[1]
    keep = keep_mask(pos, pos, window, sinks)
    q, k, v = q.double(), k.double(), v.double()
    r = {n: torch.zeros(B, H, S, D, dtype=torch.float64) for n in ("o", "o_tol", "dq", "dq_tol")}
    r["lse"] = torch.zeros(B, H, S, dtype=torch.float64)
    for n in ("dk", "dk_tol", "dv", "dv_tol"):
        r[n] = torch.zeros_like(k)
    for b in range(B):
        for h in range(H):
            g = h // G
            o, lse, p = attention(q[b, h], k[b, g], v[b, g], keep, scale)
            r["o"][b, h], r["lse"][b, h] = o, lse
            r["o_tol"][b, h] = BF * (o.abs() + 1.02 * p @ v[b, g].abs()) + 1e-5
            if dO is None:
                continue
            do = dO[b, h].double()
            dp = do @ v[b, g].T
            delta = (do * (o if o_given is None else o_given[b, h].double())).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            # fp32 error of dP - Delta: sums of up to 128 products, twice
            soft = p * (2.0 ** -16 * (do.abs() @ v[b, g].abs().T + delta.abs()))
            mag = 1.02 * BF * ds.abs() + soft
            r["dq"][b, h] = scale * ds @ k[b, g]
            r["dq_tol"][b, h] = scale * mag @ k[b, g].abs()
            r["dk"][b, g] += scale * ds.T @ q[b, h]
            r["dk_tol"][b, g] += scale * mag.T @ q[b, h].abs()
            r["dv"][b, g] += p.T @ do
            r["dv_tol"][b, g] += 1.02 * BF * p.T @ do.abs()
    for n in ("dq", "dk", "dv"):
        r[n + "_tol"] = r[n + "_tol"] + BF * r[n].abs() + 1e-5
    return r


def within(got, ref, tol, name=""):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), f"{name}: non-finite values differ"
    assert torch.equal(got[~fin], ref[~fin]), f"{name}: infinities differ"
    tol = torch.as_tensor(tol, dtype=torch.float64).expand_as(ref)
    over = ((got - ref).abs() / tol)[fin]
    assert over.numel() == 0 or float(over.max()) <= 1.0, f"{name}: {float(over.max()):.3g} times the bound"


# ------------------------------------------------------------------ norm and rotation
def _split(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _merge(x, a, b, rot, interleaved):
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


def turned(x, pos, inv_freq, interleaved, sign=1.0):
    """x [B,H,S,D] rotated by the angle of pos [B or 1, S]."""
    rot = 2 * inv_freq.numel()
    ang = pos.double()[:, None, :, None] * inv_freq
    a, b = _split(x, rot, interleaved)
    c, s = ang.cos(), sign * ang.sin()
    return _merge(x, a * c - b * s, b * c + a * s, rot, interleaved)


def spread(x, inv_freq, interleaved):
    """|a| + |b| of every pair at both of its places: the scale of a rotation's rounding error."""
    rot = 2 * inv_freq.numel()
    a, b = _split(x.abs(), rot, interleaved)
    return _merge(x.abs(), a + b, a + b, rot, interleaved)


def norm_rope_reference(x, w, pos, inv_freq, eps, interleaved, dy=None):
    x, w = x.double(), w.double()
    r = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    y = x * r * w
    out = {"y": turned(y, pos, inv_freq, interleaved), "y_mag": spread(y, inv_freq, interleaved)}
    if dy is None:
        return out
    g = turned(dy.double(), pos, inv_freq, interleaved, -1.0)
    gm = spread(dy.double(), inv_freq, interleaved)
    h, hm = g * w, gm * w.abs()
    out["dx"] = r * h - x * r ** 3 * (h * x).mean(-1, keepdim=True)
    out["dx_mag"] = r * hm + x.abs() * r ** 3 * (hm * x.abs()).mean(-1, keepdim=True)
    out["dw"] = (g * x * r).sum((0, 1, 2))
    out["dw_mag"] = (gm * (x * r).abs()).sum((0, 1, 2))
    return out
