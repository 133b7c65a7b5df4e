"""Plain 64-bit references (CPU, torch) of the operators of a kept prompt: rows in 4 bits, the weights of the keys, the
rows that stay."""
import math

import torch

GROUP = 32


def kv4_reference(x):
    """(codes -7 .. 7, scales, values) of x [..., D]: the definition, every step exact or rounded once in 64 bits."""
    g = x.double().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / 7)
    scale = torch.where(top < 2.0 ** -100, 0.0, torch.ldexp((m * 32).round() / 32, e))
    codes = torch.where(scale > 0, (g / torch.where(scale > 0, scale, 1.0)).round().clamp(-7, 7), 0.0)
    return codes.flatten(-2), scale[..., 0], (codes * scale).flatten(-2)


def kv4_codes(packed):
    """uint8 [..., D/2] -> codes [..., D], a channel at a time."""
    D = 2 * packed.shape[-1]
    out = torch.empty(*packed.shape[:-1], D, dtype=torch.float64)
    for c in range(D):
        bit = 16 * (c % 2) + 4 * (c % 8 // 2)  # of the 32-bit word of channel c
        out[..., c] = ((packed[..., c // 8 * 4 + bit // 8] >> (bit % 8)) & 15).double() - 8
    return out


def kv4_values(packed, scales):
    return kv4_codes(packed) * scales.double().repeat_interleave(GROUP, -1)


def weight_reference(q, k, lse, pos, first, scale):
    """(weight, bound) [B,Hkv,S] in placed rows.  A score is an fp32 sum of up to 128 products (2^-16 of the sum of
    their sizes); its exponent, the exponential and the sums are a few fp32 roundings each."""
    B, H, S, D = q.shape
    Hkv = k.shape[1]
    w, tol = torch.zeros(B, Hkv, S, dtype=torch.float64), torch.zeros(B, Hkv, S, dtype=torch.float64)
    keep = (pos[:, None] >= pos[None, :]) & (pos[:, None] >= first)
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            counts = torch.isfinite(lse[b, h])
            qd, kd, l = q[b, h].double(), k[b, g].double(), torch.where(counts, lse[b, h].double(), 0.0)[:, None]
            s = qd @ kd.T * scale
            p = torch.where(keep & counts[:, None], torch.exp(s - l), 0.0)
            w[b, g] += p.sum(0)
            size = qd.abs() @ kd.abs().T * scale
            tol[b, g] += (p * (2.0 ** -16 * size + 2.0 ** -20 * (1 + s.abs() + l.abs()))).sum(0)
    return w, tol + 2.0 ** -18 * w + 1e-30


def evict_reference(weight, pos, keep, sinks, recent):
    """Kept positions [B,Hkv,keep], one comparison at a time."""
    B, Hkv, S = weight.shape
    row = torch.argsort(pos).tolist()
    out = torch.empty(B, Hkv, keep, dtype=torch.int32)
    for b in range(B):
        for h in range(Hkv):
            w = weight[b, h].tolist()

            def rank(p):
                x = w[row[p]]
                if p < sinks or p >= S - recent:
                    return (0, 0.0, p)
                return (2, 0.0, p) if math.isnan(x) else (1, -x if x != 0 else 0.0, p)

            out[b, h] = torch.tensor(sorted(sorted(range(S), key=rank)[:keep]), dtype=torch.int32)
    return out, torch.tensor(row)
