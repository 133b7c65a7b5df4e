"""Cases, plain forms and exact values of the operators of a prompt that is kept for decoding:

* ``kv4``: the keys and values of a prompt stored in 4 bits with a scale for every 32 channels, and read back;
* ``decode_kv4``: a few new tokens of every request against a prompt held in 4 bits, shared by several requests or
  their own, and each request's own tail in bf16;
* ``key_weight``: the attention weight that every key of a prompt got from its queries, summed over them and over the
  query heads of a key/value head;
* ``evict``: the rows of a prompt that are kept by that weight, beside its first and its last ones, moved together.

``run`` computes a case in elementary torch operations, or with the library's calls where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

LAYOUTS = ("striped", "contiguous", "zigzag")
GROUP = 32  # channels that share a scale
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new row of 64 requests goes into their caches: the latency of a launch
        {"name": "kv4 64 single rows", "op": "kv4", "B": 64, "Hkv": 8, "S": 1, "D": 128},
        # ragged prompts of a small model
        {"name": "kv4 S5003 d64", "op": "kv4", "B": 2, "Hkv": 3, "S": 5003, "D": 64},
        # a long prompt is stored after its prefill
        {"name": "kv4 S131072", "op": "kv4", "B": 1, "Hkv": 8, "S": 131072, "D": 128},
        # one request, short prompt: the latency of a decoding step
        {"name": "decode4 1 request", "op": "decode_kv4", "B": 1, "Bp": 1, "H": 32, "Hkv": 8, "T": 1, "P": 4096,
         "C": 128, "D": 128, "N": 8, "layout": "striped"},
        # five requests that verify three drafted tokens each, ragged prompts
        {"name": "decode4 5 drafts d64", "op": "decode_kv4", "B": 5, "Bp": 5, "H": 12, "Hkv": 3, "T": 3, "P": 9999,
         "C": 333, "D": 64, "N": 3, "layout": "striped"},
        # 16 requests with long prompts of their own: the bandwidth of the cache
        {"name": "decode4 16 on P32768", "op": "decode_kv4", "B": 16, "Bp": 16, "H": 32, "Hkv": 8, "T": 1, "P": 32768,
         "C": 256, "D": 128, "N": 8, "layout": "striped"},
        # 32 requests that continue one long prompt
        {"name": "decode4 32 on P131072", "op": "decode_kv4", "B": 32, "Bp": 1, "H": 32, "Hkv": 8, "T": 1,
         "P": 131072, "C": 1000, "D": 128, "N": 8, "layout": "striped"},
        # the last 64 tokens of a long prompt judge its keys
        {"name": "weight last 64 of S65536", "op": "key_weight", "B": 1, "H": 32, "Hkv": 8, "S": 65536, "D": 128,
         "N": 8, "layout": "striped", "first": 65536 - 64},
        # ragged stripes, a small head dimension, the last fifth of the queries
        {"name": "weight S5000 d64", "op": "key_weight", "B": 2, "H": 6, "Hkv": 2, "S": 5000, "D": 64, "N": 8,
         "layout": "striped", "first": 4001},
        # every query of a prompt, grouped-query layer
        {"name": "weight S16384 gqa", "op": "key_weight", "B": 1, "H": 32, "Hkv": 8, "S": 16384, "D": 128, "N": 8,
         "layout": "striped", "first": 0},
        # short prompts of four requests
        {"name": "evict S1500 d64", "op": "evict", "B": 4, "Hkv": 2, "S": 1500, "D": 64, "N": 4, "layout": "striped",
         "keep": 201, "sinks": 4, "recent": 32},
        # an eighth of a long prompt stays
        {"name": "evict S131072", "op": "evict", "B": 1, "Hkv": 8, "S": 131072, "D": 128, "N": 8, "layout": "striped",
         "keep": 16384, "sinks": 4, "recent": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _placed(rng, S, layout, N):
    """A length near S that the placement takes: whole stripes; zig-zag chunks of whole 128-row tiles."""
    unit = 256 * N if layout == "zigzag" else N
    return max(1, S // unit) * unit


def draw(rng):
    op = rng.choice(("kv4", "decode_kv4", "key_weight", "evict"))
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    H = Hkv * rng.choice((1, 2, 3, 4))
    layout = rng.choice(LAYOUTS)
    N = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
    if op == "kv4":
        S = _log(rng, 1, 131072)
        B = rng.choice((1, 2, 3)) if S > 512 else _log(rng, 1, 64)
        return {"op": op, "B": B, "Hkv": Hkv, "S": min(S, 131072 // B), "D": D}
    if op == "decode_kv4":
        B = _log(rng, 1, 48)
        Bp = rng.choice((1, B, max(d for d in range(1, B + 1) if B % d == 0 and d * d <= B)))
        P = _placed(rng, _log(rng, 1, 131072 if Bp == 1 else max(16, 131072 // Bp)), layout, N)
        T = rng.choice((1, 1, 1, 2, 5))
        return {"op": op, "B": B, "Bp": Bp, "H": H, "Hkv": Hkv, "T": T, "P": P, "C": _log(rng, T, 1000), "D": D,
                "N": N, "layout": layout}
    if op == "key_weight":
        S = _log(rng, 16, 16384)
        B = 1 if S > 4096 else rng.choice((1, 2, 3))
        S = min(_placed(rng, S, layout, N), 16384 // (256 * N) * 256 * N)
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "S": S, "D": D, "N": N, "layout": layout,
                "first": rng.choice((0, S - _log(rng, 1, S)))}
    S = _placed(rng, _log(rng, 16, 131072), layout, N)
    S = min(S, 131072 // (256 * N) * 256 * N)
    keep = _log(rng, 1, min(S, 16384))
    sinks = min(rng.choice((0, 1, 4, 100)), keep)
    return {"op": op, "B": 1 if S > 2048 else rng.choice((1, 2, 5)), "Hkv": Hkv, "S": S, "D": D, "N": N,
            "layout": layout, "keep": keep, "sinks": sinks, "recent": min(rng.choice((0, 1, 32, 200)), keep - sinks)}


# ------------------------------------------------------------------ inputs
def _positions(S, N, layout, device):
    """Position held by every row of a placed sequence."""
    p = torch.arange(S, device=device)
    if layout == "striped":
        return p.view(S // N, N).t().reshape(-1)
    if layout == "zigzag":
        chunk = p.view(2 * N, S // (2 * N))
        order = [c for d in range(N) for c in (d, 2 * N - 1 - d)]
        return chunk[order].reshape(-1)
    return p


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(BF16)

    def keys(*shape):
        # a few channels of a key are several times as large as the others
        size = torch.exp(0.7 * torch.randn(shape[1], 1, shape[3], generator=gen, device=dev))
        return (torch.randn(*shape, generator=gen, device=dev) * size).to(BF16)

    s = dict(case)
    Hkv, D = case["Hkv"], case["D"]
    s["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "kv4":
        B, S = case["B"], case["S"]
        s["k"], s["v"] = keys(B, Hkv, S, D), normal(B, Hkv, S, D)
        return s
    if case["op"] == "decode_kv4":
        B, Bp, H, T, P, C = (case[n] for n in ("B", "Bp", "H", "T", "P", "C"))
        s["q"] = normal(B, H, T, D)
        for n, x in (("k", keys(Bp, Hkv, P, D)), ("v", normal(Bp, Hkv, P, D))):
            codes, scales = zip(*(_stored(one) for one in x))  # a prompt at a time
            s[n + "c"], s[n + "s"] = torch.stack([_packed(c) for c in codes]), torch.stack(scales)
        s["kt"], s["vt"] = keys(B, Hkv, C, D), normal(B, Hkv, C, D)
        lens = torch.randint(max(T, C // 2), C + 1, (B,), generator=gen, device=dev)
        s["lens"] = lens.to(torch.int32)
        behind = (torch.arange(C, device=dev) >= lens[:, None])[:, None, :, None]
        s["kt"].masked_fill_(behind, float("nan"))  # rows behind a tail's end were never written
        s["vt"].masked_fill_(behind, float("nan"))
        return s
    B, S = case["B"], case["S"]
    s["pos"] = _positions(S, case["N"], case["layout"], dev)
    if case["op"] == "key_weight":
        s["q"], s["k"] = normal(B, case["H"], S, D), normal(B, Hkv, S, D)
        s["lse"] = _lse(s)
        return s
    s["k"], s["v"] = normal(B, Hkv, S, D), normal(B, Hkv, S, D)
    # a few keys have most of the weight, some have none at all
    w = torch.exp(2.0 * torch.randn(B, Hkv, S, generator=gen, device=dev))
    s["weight"] = w * (torch.rand(B, Hkv, S, generator=gen, device=dev) < 0.95)
    return s


# ------------------------------------------------------------------ 4 bits
def _stored(x):
    """Codes -7 .. 7 and the scales of groups of channels: amax / 7 to 5 significant bits, so that a code times its
    scale is a bf16 number."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / 7)
    scale = torch.ldexp((m * 32).round() / 32, e)
    scale = torch.where(top < 2.0 ** -100, 0.0, scale)
    codes = torch.where(scale > 0, (g / scale).round().clamp(-7, 7), 0.0)
    return codes.flatten(-2), scale[..., 0].to(BF16)


def _values(codes, scales):
    return codes * scales.float().repeat_interleave(GROUP, -1)


_NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)  # the channel of every nibble of a 32-bit word, from the lowest on


def _packed(codes):
    n = (codes + 8).to(torch.uint8).unflatten(-1, (-1, 8))[..., list(_NIBBLE)].unflatten(-1, (4, 2))
    return (n[..., 0] | (n[..., 1] << 4)).flatten(-2)


def _unpacked(b):
    n = torch.stack([b & 15, b >> 4], -1).unflatten(-2, (-1, 4)).flatten(-2)
    out = torch.empty_like(n)
    out[..., list(_NIBBLE)] = n
    return out.flatten(-2).float() - 8


# ------------------------------------------------------------------ plain forms
def _kv4(s):
    return [_values(*_stored(s[n])).to(BF16) for n in ("k", "v")]


def _decode(s):
    B, Bp, H, Hkv, T, P, C, D = (s[n] for n in ("B", "Bp", "H", "Hkv", "T", "P", "C", "D"))
    R, G = B // Bp, H // Hkv
    dev = s["q"].device
    lens = s["lens"].long()
    qpos = P + lens[:, None] - T + torch.arange(T, device=dev)  # [B, T]
    keep_p = _positions(P, s["N"], s["layout"], dev) <= qpos[..., None]
    keep_t = P + torch.arange(C, device=dev) <= qpos[..., None]
    q = s["q"].float().view(B, Hkv, G, T, D)
    # the prompt: all rows of the requests that share it in one product
    qp = q.view(Bp, R, Hkv, G * T, D).transpose(1, 2).reshape(Bp, Hkv, R * G * T, D)
    sp = (qp @ _values(_unpacked(s["kc"]), s["ks"]).transpose(-1, -2)).mul_(s["scale"])
    sp = sp.view(Bp, Hkv, R, G, T, P).masked_fill_(~keep_p.view(Bp, 1, R, 1, T, P), -math.inf)
    st = (q.view(B, Hkv, G * T, D) @ s["kt"].float().transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, T, C)
    st = torch.where(keep_t.view(B, 1, 1, T, C), st, -math.inf).view(Bp, R, Hkv, G, T, C).transpose(1, 2)
    top = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
    top = top.masked_fill(top == -math.inf, 0.0)
    sp, st = sp.sub_(top).exp_(), st.sub(top).exp_()
    total = sp.sum(-1, keepdim=True) + st.sum(-1, keepdim=True)
    written = (torch.arange(C, device=dev) < lens[:, None])[:, None, :, None]
    vt = torch.where(written, s["vt"].float(), 0.0)
    o = sp.reshape(Bp, Hkv, R * G * T, P) @ _values(_unpacked(s["vc"]), s["vs"])
    o = o.view(Bp, Hkv, R, G * T, D).transpose(1, 2).reshape(B, Hkv, G * T, D)
    o = o + st.transpose(1, 2).reshape(B, Hkv, G * T, C) @ vt
    total, top = (x.transpose(1, 2).reshape(B, Hkv, G * T, 1) for x in (total, top))
    o = torch.where(total > 0, o / total, 0.0).reshape(B, H, T, D)
    return o.to(BF16), (top + total.log()).reshape(B, H, T)


def _query_blocks(s, first):
    """Blocks of queries from `first` on, in position order, and the scores of the keys up to their last one."""
    B, H, Hkv, S, D = (s[n] for n in ("B", "H", "Hkv", "S", "D"))
    row = torch.argsort(s["pos"])
    k = s["k"][:, :, row].float()
    at = torch.arange(S, device=row.device)
    for p0 in range(first, S, 1024):
        p = at[p0 : p0 + 1024]
        end = p0 + p.numel()
        q = s["q"][:, :, row[p]].float().view(B, Hkv, H // Hkv, p.numel(), D)
        x = (q.flatten(2, 3) @ k[:, :, :end].transpose(-1, -2)).mul_(s["scale"]).view(*q.shape[:4], end)
        yield row, p, x.masked_fill_(at[:end] > p[:, None], -math.inf)


def _lse(s):
    out = torch.zeros(s["B"], s["H"], s["S"], device=s["q"].device)
    for row, p, x in _query_blocks(s, s["first"]):
        top = x.amax(-1, keepdim=True)
        out[:, :, row[p]] = (top + x.sub_(top).exp_().sum(-1, keepdim=True).log()).view(s["B"], s["H"], -1)
    return out


def _key_weight(s):
    total = torch.zeros(s["B"], s["Hkv"], s["S"], device=s["q"].device)
    for row, p, x in _query_blocks(s, s["first"]):
        lse = s["lse"][:, :, row[p]].view(*x.shape[:4], 1)
        total[:, :, : x.shape[-1]] += x.sub_(lse).exp_().sum((2, 3))
    out = torch.empty_like(total)
    out[:, :, row] = total
    return out


def _evict(s):
    S, D, keep = s["S"], s["D"], s["keep"]
    row = torch.argsort(s["pos"])
    w = s["weight"][:, :, row]
    rank = w.clone()
    rank[..., : s["sinks"]] = math.inf
    rank[..., S - s["recent"] :] = math.inf
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    index = order.sort(-1).values
    rows = row[index][..., None].expand(-1, -1, -1, D)
    return s["k"].gather(2, rows), s["v"].gather(2, rows), index.to(torch.int32), w.gather(2, index)


# ------------------------------------------------------------------ one pass
def _run_own(s):
    import sequence_parallelism_striped_gb300 as sp

    if s["op"] == "kv4":
        return sp.striped_kv4_load(*sp.striped_kv4_store(s["k"], s["v"]))
    layout = {"striped": sp.STRIPED, "contiguous": sp.CONTIGUOUS, "zigzag": sp.ZIGZAG}[s["layout"]]
    if s["op"] == "decode_kv4":
        return sp.striped_attn_decode_kv4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["kt"], s["vt"], s["lens"],
                                          s["N"], layout, s["scale"])
    if s["op"] == "key_weight":
        return sp.striped_attn_key_weight(s["q"], s["k"], s["lse"], s["N"], layout, s["first"], s["scale"])
    return sp.striped_kv_evict(s["k"], s["v"], s["weight"], s["keep"], s["sinks"], s["recent"], s["N"], layout)


def run(s):
    if own:
        return _run_own(s)
    return {"kv4": _kv4, "decode_kv4": _decode, "key_weight": _key_weight, "evict": _evict}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hkv, D = case["Hkv"], case["D"]
    packed = D // 2 + D // GROUP * 2  # bytes of a stored row
    if case["op"] == "kv4":
        n = 2 * case["B"] * Hkv * case["S"]
        return {"bytes": n * (4 * D + 2 * packed), "flops": 6 * n * D}
    if case["op"] == "decode_kv4":
        B, H, T, P, C = (case[n] for n in ("B", "H", "T", "P", "C"))
        tail = (max(T, C // 2) + C) / 2  # lengths are drawn evenly from the upper half
        kv = 2 * Hkv * (case["Bp"] * P * packed + B * tail * 2 * D)
        return {"bytes": kv + B * H * T * (4 * D + 4), "flops": 4.0 * D * B * H * T * (P + tail)}
    B, S = case["B"], case["S"]
    if case["op"] == "key_weight":
        H, n = case["H"], S - case["first"]
        pairs = n * (n + 1) // 2 + case["first"] * n
        return {"bytes": B * (H * n * (2 * D + 4) + Hkv * S * (2 * D + 4)), "flops": 2.0 * D * B * H * pairs}
    keep = case["keep"]
    return {"bytes": B * Hkv * (4 * S + keep * (8 * D + 8)), "flops": 2.0 * B * Hkv * S}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_kv4(s):
    out = []
    for n in ("k", "v"):
        x = s[n].double()
        x = x.view(*x.shape[:-1], -1, GROUP)
        top = x.abs().max(-1, keepdim=True).values
        step = top / 7
        unit = torch.exp2(torch.floor(torch.log2(step.clamp(min=1e-300))) - 4)  # of the fifth significant bit
        unit = torch.where(step / unit >= 32, 2 * unit, torch.where(step / unit < 16, unit / 2, unit))
        step = torch.round(step / unit) * unit
        y = torch.round(x / step).clamp(-7, 7) * step
        out.append(torch.where(top < 2.0 ** -100, 0.0, y).view(s[n].shape))
    return out


def _exact_decode(s):
    """Request by request: the keys in order of position, prompt then tail."""
    B, H, T, P, D = s["B"], s["H"], s["T"], s["P"], s["D"]
    R, G = B // s["Bp"], H // s["Hkv"]
    row = torch.argsort(_positions(P, s["N"], s["layout"], "cuda"))
    channel = torch.arange(D, device="cuda")
    byte = channel // 8 * 4 + channel % 2 * 2 + channel % 8 // 4
    shift = (channel % 4 // 2 * 4).to(torch.uint8)

    def prompt(codes, scales, at):
        c = (codes[at][..., byte] >> shift) & 15
        return ((c.double() - 8) * scales[at].double()[..., channel // GROUP])[:, row]

    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        if b % R == 0:
            kp, vp = prompt(s["kc"], s["ks"], b // R), prompt(s["vc"], s["vs"], b // R)
        k = torch.cat([kp, s["kt"][b][:, :n].double()], 1)
        v = torch.cat([vp, s["vt"][b][:, :n].double()], 1)
        for i in range(T):
            seen = P + n - T + i + 1
            if seen <= 0:
                continue
            q = s["q"][b, :, i].double().view(-1, G, D)
            x = (q @ k[:, :seen].transpose(1, 2)) * s["scale"]
            lse[b, :, i] = torch.logsumexp(x, -1).reshape(-1)
            o[b, :, i] = (torch.softmax(x, -1) @ v[:, :seen]).reshape(H, -1)
    return [o, lse]


def _exact_weight(s):
    """Query head by query head, a stretch of keys at a time, against every query at or after its first one."""
    B, H, Hkv, S, first = (s[n] for n in ("B", "H", "Hkv", "S", "first"))
    row = torch.argsort(s["pos"])
    at = torch.arange(S, device="cuda")
    w = torch.zeros(B, Hkv, S, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            q, lse = s["q"][b, h, row].double(), s["lse"][b, h, row].double()
            for t0 in range(0, S, 4096):
                t, p = at[t0 : t0 + 4096], at[max(t0, first) :]
                x = s["k"][b, g, row[t]].double() @ q[p].T * s["scale"] - lse[p]
                w[b, g, row[t]] += torch.where(t[:, None] <= p, torch.exp(x), 0.0).sum(-1)
    return w


def _exact_evict(s):
    B, Hkv, S, keep = s["B"], s["Hkv"], s["S"], s["keep"]
    row = np.argsort(s["pos"].cpu().numpy())
    weight = s["weight"].cpu().numpy()
    middle = np.arange(s["sinks"], S - s["recent"])
    ends = np.concatenate([np.arange(s["sinks"]), np.arange(S - s["recent"], S)])
    index = np.empty((B, Hkv, keep), dtype=np.int32)
    for b in range(B):
        for h in range(Hkv):
            w = weight[b, h, row[middle]]
            best = np.lexsort((middle, -w))[: keep - ends.size]
            index[b, h] = np.sort(np.concatenate([ends, middle[best]]))
    kept = torch.as_tensor(row[index], device="cuda")
    b, h = torch.meshgrid(torch.arange(B, device="cuda"), torch.arange(Hkv, device="cuda"), indexing="ij")
    b, h = b[..., None], h[..., None]
    return [s["k"][b, h, kept].double(), s["v"][b, h, kept].double(), torch.as_tensor(index, device="cuda"),
            s["weight"][b, h, kept].double()]


def exact(case, seed):
    s = prepare(case, seed)
    return {"kv4": _exact_kv4, "decode_kv4": _exact_decode, "key_weight": _exact_weight,
            "evict": _exact_evict}[s["op"]](s)
