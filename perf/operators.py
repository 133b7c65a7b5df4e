"""Cases, plain forms and exact values of the operators around the striped attention:

* ``norm_rope`` / ``norm_rope_bwd``: RMS norm of every query and key head followed by the rotary position rotation,
  rows in the order of a stripe placement (or at given positions), and its gradient;
* ``window_fwd`` / ``window_bwd``: causal attention that sees a sliding window and a few first tokens (sinks), rows in
  the order of a stripe placement, and its gradient;
* ``decode``: a few new tokens of every request against a placed prompt, shared by several requests or their own, and
  each request's own tail.

``run`` computes a case in elementary torch operations, or with the library's calls where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
LAYOUTS = ("striped", "contiguous", "zigzag")
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    rope = {"base": 500000.0, "interleaved": False}
    return [
        # one decoding step of 64 requests, each at its own position: the latency of a launch
        {"name": "rope step 64 requests", "op": "norm_rope", "B": 64, "H": 32, "Hkv": 8, "S": 1, "D": 128, "rot": 128,
         "N": 1, "layout": "contiguous", "at": True, "dtype": "bf16", **rope},
        # grouped-query layer of a long training sequence in its striped rows
        {"name": "rope S65536 gqa", "op": "norm_rope", "B": 1, "H": 32, "Hkv": 8, "S": 65536, "D": 128, "rot": 128,
         "N": 8, "layout": "striped", "at": False, "dtype": "bf16", **rope},
        # fp32 check run with half of each head rotated, adjacent pairs, odd stripe count
        {"name": "rope bwd fp32 S6003", "op": "norm_rope_bwd", "B": 2, "H": 5, "Hkv": 5, "S": 6003, "D": 64, "rot": 32,
         "N": 3, "layout": "striped", "at": False, "dtype": "fp32", "base": 10000.0, "interleaved": True},
        # gradient of the long training sequence
        {"name": "rope bwd S65536 gqa", "op": "norm_rope_bwd", "B": 1, "H": 32, "Hkv": 8, "S": 65536, "D": 128,
         "rot": 128, "N": 8, "layout": "striped", "at": False, "dtype": "bf16", **rope},
        # the short-sequence workload of the benchmark, as a local layer
        {"name": "window S8192", "op": "window_fwd", "B": 1, "H": 8, "Hkv": 8, "S": 8192, "D": 128, "N": 8,
         "layout": "striped", "window": 1024, "sinks": 4, "dtype": "bf16"},
        # ragged stripes, a small head dimension, a window that is no whole tile
        {"name": "window S5000 d64", "op": "window_fwd", "B": 2, "H": 6, "Hkv": 2, "S": 5000, "D": 64, "N": 8,
         "layout": "striped", "window": 300, "sinks": 1, "dtype": "bf16"},
        # long prefill of a grouped-query local layer
        {"name": "window S65536 gqa", "op": "window_fwd", "B": 1, "H": 32, "Hkv": 8, "S": 65536, "D": 128, "N": 8,
         "layout": "striped", "window": 1024, "sinks": 4, "dtype": "bf16"},
        # training step of the short workload
        {"name": "window bwd S8192", "op": "window_bwd", "B": 1, "H": 8, "Hkv": 8, "S": 8192, "D": 128, "N": 8,
         "layout": "striped", "window": 1024, "sinks": 4, "dtype": "bf16"},
        # training step of a long grouped-query layer in the zig-zag placement, wider window
        {"name": "window bwd S32768 gqa", "op": "window_bwd", "B": 1, "H": 32, "Hkv": 8, "S": 32768, "D": 128, "N": 8,
         "layout": "zigzag", "window": 2048, "sinks": 16, "dtype": "bf16"},
        # one request, short prompt: the latency of a decoding step
        {"name": "decode 1 request", "op": "decode", "B": 1, "Bp": 1, "H": 32, "Hkv": 8, "T": 1, "P": 4096, "C": 128,
         "D": 128, "N": 8, "layout": "striped", "window": 0, "sinks": 0, "dtype": "bf16"},
        # 32 requests that continue one long prompt
        {"name": "decode 32 on P131072", "op": "decode", "B": 32, "Bp": 1, "H": 32, "Hkv": 8, "T": 1, "P": 131072,
         "C": 1000, "D": 128, "N": 8, "layout": "striped", "window": 0, "sinks": 0, "dtype": "bf16"},
        # a local layer of 24 requests with prompts of their own, three drafted tokens each
        {"name": "decode 24 window 4096", "op": "decode", "B": 24, "Bp": 24, "H": 16, "Hkv": 4, "T": 3, "P": 8192,
         "C": 700, "D": 64, "N": 4, "layout": "zigzag", "window": 4096, "sinks": 4, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _placed(rng, S, layout, N):
    """A length near S that the placement takes: whole stripes; zig-zag chunks of whole 128-row tiles."""
    unit = 256 * N if layout == "zigzag" else N
    return max(1, S // unit) * unit


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope_bwd", "window_fwd", "window_bwd", "decode"))
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    H = Hkv * rng.choice((1, 2, 3, 4))
    layout = rng.choice(LAYOUTS)
    N = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
    if op in ("norm_rope", "norm_rope_bwd"):
        at = rng.random() < 0.3
        S = _log(rng, 1, 65536)
        B = rng.choice((1, 2, 3)) if S > 512 else _log(rng, 1, 64)
        S = min(S, 65536 // B)
        if at:
            layout, N = "contiguous", 1
        elif layout == "zigzag":
            S = max(1, S // (2 * N)) * 2 * N
        else:
            S = max(1, S // N) * N
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "S": S, "D": D, "rot": rng.choice((D, D, D // 2)), "N": N,
                "layout": layout, "at": at, "dtype": rng.choice(("bf16", "bf16", "fp32")),
                "base": rng.choice((10000.0, 500000.0)), "interleaved": rng.random() < 0.3}
    window = _log(rng, 2, 2048)  # at 1 without sinks a query sees itself alone and its gradients are 0
    sinks = rng.choice((0, 1, 4, 16, 100, 200))
    if op in ("window_fwd", "window_bwd"):
        S = _log(rng, 16, 32768)
        B = 1 if S > 4096 else rng.choice((1, 2, 3))
        S = _placed(rng, S, layout, N)
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "S": S, "D": D, "N": N, "layout": layout, "window": window,
                "sinks": sinks, "dtype": "bf16"}
    B = _log(rng, 1, 48)
    Bp = rng.choice((1, B, max(d for d in range(1, B + 1) if B % d == 0 and d * d <= B)))
    T = rng.choice((1, 1, 1, 2, 5))
    P = _log(rng, 1, 131072 if Bp == 1 else max(16, 131072 // Bp))
    P = _placed(rng, P, layout, N)
    full = rng.random() < 0.5
    return {"op": op, "B": B, "Bp": Bp, "H": H, "Hkv": Hkv, "T": T, "P": P, "C": _log(rng, T, 2000), "D": D, "N": N,
            "layout": layout, "window": 0 if full else 2 * window, "sinks": 0 if full else sinks, "dtype": "bf16"}


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
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(dt)

    s = dict(case)
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    s["scale"] = 1.0 / math.sqrt(D)
    if case["op"].startswith("norm_rope"):
        S, rot = case["S"], case["rot"]
        # projections: every row has a size of its own
        size = torch.randn(B, 1, S, 1, generator=gen, device=dev).mul_(0.5).exp_()
        s["q"] = (torch.randn(B, H, S, D, generator=gen, device=dev) * size).to(dt)
        s["k"] = (torch.randn(B, Hkv, S, D, generator=gen, device=dev) * size).to(dt)
        s["qw"] = 1 + 0.2 * torch.randn(D, generator=gen, device=dev)
        s["kw"] = 1 + 0.2 * torch.randn(D, generator=gen, device=dev)
        j = torch.arange(rot // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = case["base"] ** (-2.0 * j / rot)
        s["positions"] = None
        if case["at"]:
            first = torch.randint(0, 786432, (B, 1), generator=gen, device=dev)
            s["positions"] = first + torch.arange(S, device=dev)
        s["pos"] = s["positions"] if case["at"] else _positions(S, case["N"], case["layout"], dev)[None]
        if case["op"] == "norm_rope_bwd":
            s["dqo"], s["dko"] = normal(B, H, S, D), normal(B, Hkv, S, D)
        return s
    if case["op"] == "decode":
        Bp, T, P, C = case["Bp"], case["T"], case["P"], case["C"]
        s["q"] = normal(B, H, T, D)
        s["kp"], s["vp"] = normal(Bp, Hkv, P, D), normal(Bp, Hkv, P, D)
        s["kt"], s["vt"] = normal(B, Hkv, C, D), normal(B, Hkv, C, D)
        lens = torch.randint(max(T, C // 2), C + 1, (B,), generator=gen, device=dev)
        s["lens"] = lens.to(torch.int32)
        behind = (torch.arange(C, device=dev) >= lens[:, None])[:, None, :, None]
        s["kt"].masked_fill_(behind, float("nan"))  # rows behind a tail's end were never written
        s["vt"].masked_fill_(behind, float("nan"))
        s["pos"] = _positions(P, case["N"], case["layout"], dev)
        return s
    S = case["S"]
    s["q"], s["k"], s["v"] = normal(B, H, S, D), normal(B, Hkv, S, D), normal(B, Hkv, S, D)
    s["pos"] = _positions(S, case["N"], case["layout"], dev)
    if case["op"] == "window_bwd":
        s["dO"] = normal(B, H, S, D)
        s["o"], s["lse"] = _window_fwd(s)
    return s


# ------------------------------------------------------------------ plain forms
def _rotation(s):
    angle = s["pos"].double()[..., None] * s["inv_freq"]
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2 : rot]


def _joined(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _normed(x, w):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_rope(s):
    c, si = _rotation(s)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = _normed(x, w)[0] * w
        a, b = _pairs(y, s["rot"], s["interleaved"])
        out.append(_joined(a * c - b * si, b * c + a * si, y[..., s["rot"]:], s["interleaved"]).to(x.dtype))
    return out


def _norm_rope_bwd(s):
    c, si = _rotation(s)
    dx, dw = [], []
    for x, w, g in ((s["q"], s["qw"], s["dqo"]), (s["k"], s["kw"], s["dko"])):
        n, r = _normed(x, w)
        g = g.float()
        a, b = _pairs(g, s["rot"], s["interleaved"])
        g = _joined(a * c + b * si, b * c - a * si, g[..., s["rot"]:], s["interleaved"])
        dw.append((g * n).sum((0, 1, 2)))
        g = g * w
        dx.append((r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype))
    return dx + dw


BLOCK = 256


def _blocks(s):
    """Position order, cut into blocks of queries and the stretch of keys that each can see; and the masks."""
    B, H, Hkv, S, D, W, ns = (s[n] for n in ("B", "H", "Hkv", "S", "D", "window", "sinks"))
    W, ns = min(W, S), min(ns, S)
    row = torch.argsort(s["pos"])
    nb = -(-S // BLOCK)
    back = -(-(W - 1) // BLOCK) * BLOCK
    dev = row.device
    qpos = torch.arange(nb * BLOCK, device=dev).view(nb, BLOCK, 1)
    kpos = (torch.arange(nb, device=dev)[:, None] * BLOCK - back + torch.arange(back + BLOCK, device=dev))[:, None]
    near = (kpos >= 0) & (kpos <= qpos) & (qpos - kpos < W) & (kpos < S)
    far = qpos - torch.arange(ns, device=dev) >= W

    def queries(x):
        x = torch.nn.functional.pad(x[:, :, row].float(), (0, 0, 0, nb * BLOCK - S))
        return x.view(B, Hkv, H // Hkv, nb, BLOCK, -1).transpose(2, 3).reshape(B, Hkv, nb, H // Hkv * BLOCK, -1)

    def keys(x):
        x = x[:, :, row].float()
        x = torch.nn.functional.pad(x, (0, 0, back, nb * BLOCK - S))
        return x.unfold(2, back + BLOCK, BLOCK).transpose(-1, -2), x[:, :, None, back : back + ns]

    G = H // Hkv
    return row, nb, back, ns, queries, keys, near.repeat(1, G, 1), far.repeat(1, G, 1)


def _rows(x, s, row, nb):
    """Blocks of queries back to the placed rows of [B, H, S, .]."""
    B, H, Hkv, S = s["B"], s["H"], s["Hkv"], s["S"]
    x = x.view(B, Hkv, nb, H // Hkv, BLOCK, -1).transpose(2, 3).reshape(B, H, nb * BLOCK, -1)[:, :, :S]
    out = torch.empty_like(x)
    out[:, :, row] = x
    return out


def _scores(s, q, kn, ks, near, far):
    a = (q @ kn.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~near, -math.inf)
    b = (q @ ks.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~far, -math.inf)
    return a, b


def _window_fwd(s):
    row, nb, back, ns, queries, keys, near, far = _blocks(s)
    q, (kn, ks), (vn, vs) = queries(s["q"]), keys(s["k"]), keys(s["v"])
    a, b = _scores(s, q, kn, ks, near, far)
    top = torch.cat([a.amax(-1, keepdim=True), b], -1).amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)  # rows that only fill the last block
    a, b = a.sub_(top).exp_(), b.sub_(top).exp_()
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = (a @ vn + b @ vs) / total
    return _rows(o, s, row, nb).to(s["q"].dtype), _rows(top + total.log(), s, row, nb)[..., 0]


def _window_bwd(s):
    B, Hkv, S, D = s["B"], s["Hkv"], s["S"], s["D"]
    row, nb, back, ns, queries, keys, near, far = _blocks(s)
    q, do = queries(s["q"]), queries(s["dO"])
    delta = (do * queries(s["o"])).sum(-1, keepdim=True)
    (kn, ks), (vn, vs) = keys(s["k"]), keys(s["v"])
    lse = queries(s["lse"][..., None])
    a, b = _scores(s, q, kn, ks, near, far)
    a, b = a.sub_(lse).exp_(), b.sub_(lse).exp_()
    at = torch.arange(nb, device=q.device)[:, None] * BLOCK + torch.arange(back + BLOCK, device=q.device)

    def gathered(pa, pb, x):
        y = torch.zeros(B, Hkv, back + nb * BLOCK, D, device=x.device)
        y.index_add_(2, at.reshape(-1), (pa.transpose(-1, -2) @ x).reshape(B, Hkv, -1, D))
        y = y[:, :, back : back + S]
        y[:, :, :ns] += (pb.transpose(-1, -2) @ x).sum(2)
        out = torch.empty_like(y)
        out[:, :, row] = y
        return out

    dv = gathered(a, b, do)
    a.mul_((do @ vn.transpose(-1, -2)).sub_(delta))
    b.mul_((do @ vs.transpose(-1, -2)).sub_(delta))
    dk = gathered(a, b, q).mul_(s["scale"])
    dq = _rows((a @ kn + b @ ks).mul_(s["scale"]), s, row, nb)
    dt = s["q"].dtype
    return dq.to(dt), dk.to(dt), dv.to(dt)


def _decode(s):
    B, Bp, H, Hkv, T, P, C, D, W, ns = (s[n] for n in ("B", "Bp", "H", "Hkv", "T", "P", "C", "D", "window", "sinks"))
    R, G = B // Bp, H // Hkv
    dev = s["q"].device
    lens = s["lens"].long()
    qpos = P + lens[:, None] - T + torch.arange(T, device=dev)  # [B, T]

    def kept(kpos):
        keep = kpos <= qpos[..., None]
        return keep if W == 0 else keep & ((qpos[..., None] - kpos < W) | (kpos < ns))

    keep_p, keep_t = kept(s["pos"]), kept(P + torch.arange(C, device=dev))  # [B, T, .]
    q = s["q"].float().view(B, Hkv, G, T, D)
    # the prompt: all rows of the requests that share it in one product
    qp = q.view(Bp, R, Hkv, G * T, D).transpose(1, 2).reshape(Bp, Hkv, R * G * T, D)
    sp = (qp @ s["kp"].float().transpose(-1, -2)).mul_(s["scale"])
    sp = sp.view(Bp, Hkv, R, G, T, P).masked_fill_(~keep_p.view(Bp, 1, R, 1, T, P), -math.inf)
    st = (q.view(B, Hkv, G * T, D) @ s["kt"].float().transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, T, C)
    st = torch.where(keep_t.view(B, 1, 1, T, C), st, -math.inf).view(Bp, R, Hkv, G, T, C).transpose(1, 2)
    top = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
    safe = top.masked_fill(top == -math.inf, 0.0)
    sp, st = sp.sub_(safe).exp_(), st.sub(safe).exp_()
    total = sp.sum(-1, keepdim=True) + st.sum(-1, keepdim=True)
    written = (torch.arange(C, device=dev) < lens[:, None])[:, None, :, None]
    vt = torch.where(written, s["vt"].float(), 0.0)
    o = (sp.reshape(Bp, Hkv, R * G * T, P) @ s["vp"].float()).reshape(Bp, Hkv, R, G * T, D)
    o = o.transpose(1, 2).reshape(B, Hkv, G * T, D) + st.transpose(1, 2).reshape(B, Hkv, G * T, C) @ vt
    total, safe = (x.transpose(1, 2).reshape(B, Hkv, G * T, 1) for x in (total, safe))
    o = torch.where(total > 0, o / total, 0.0).reshape(B, H, T, D)
    return o.to(s["q"].dtype), (safe + total.log()).reshape(B, H, T)


# ------------------------------------------------------------------ one pass
def _run_own(s):
    import sequence_parallelism_striped_gb300 as sp

    layout = {"striped": sp.STRIPED, "contiguous": sp.CONTIGUOUS, "zigzag": sp.ZIGZAG}[s["layout"]]
    op, N = s["op"], s["N"]
    if op == "norm_rope":
        return sp.striped_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], N, layout, eps=EPS,
                                       interleaved=s["interleaved"], positions=s["positions"])
    if op == "norm_rope_bwd":
        return sp.striped_qk_norm_rope_bwd(s["q"], s["k"], s["dqo"], s["dko"], s["qw"], s["kw"], s["inv_freq"], N,
                                           layout, eps=EPS, interleaved=s["interleaved"], positions=s["positions"])
    if op == "window_fwd":
        return sp.striped_attn_window_fwd(s["q"], s["k"], s["v"], N, s["window"], s["sinks"], layout, s["scale"])
    if op == "window_bwd":
        return sp.striped_attn_window_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], N, s["window"],
                                          s["sinks"], layout, s["scale"])
    return sp.striped_attn_decode(s["q"], s["kp"], s["vp"], s["kt"], s["vt"], s["lens"], N, layout, s["window"],
                                  s["sinks"], s["scale"])


def run(s):
    if own:
        return _run_own(s)
    return {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "window_fwd": _window_fwd,
            "window_bwd": _window_bwd, "decode": _decode}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(S, W, sinks):
    """Kept (query, key) pairs of one head."""
    W = min(W, S)
    pairs = W * (W + 1) // 2 + (S - W) * W
    far = min(sinks, S - W)  # a query p >= W sees min(sinks, p + 1 - W) keys before its window
    return pairs + far * (far + 1) // 2 + (S - W - far) * far


def work(case):
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm_rope"):
        n = B * (H + Hkv) * case["S"] * D
        if case["op"] == "norm_rope":
            return {"bytes": 2 * n * es, "flops": 8 * n}
        return {"bytes": 3 * n * es, "flops": 16 * n}
    if case["op"] == "decode":
        P, C, T = case["P"], case["C"], case["T"]
        tail = (max(T, C // 2) + C) / 2  # lengths are drawn evenly from the upper half
        if case["window"]:
            seen = min(P + tail, case["window"] + T - 1 + case["sinks"])
            in_tail = min(tail, case["window"] + T - 1)
            prompt = min(P, max(0.0, seen - in_tail))
        else:
            prompt, in_tail = P, tail
        kv = 2 * Hkv * D * es * (case["Bp"] * prompt + B * in_tail)
        return {"bytes": kv + B * H * T * (2 * D * es + 4), "flops": 4.0 * D * B * H * T * (prompt + in_tail)}
    S = case["S"]
    pairs = B * H * _seen(S, case["window"], case["sinks"])
    q, k = B * H * S * D * es, B * Hkv * S * D * es
    if case["op"] == "window_fwd":
        return {"bytes": 2 * q + 2 * k + 4 * B * H * S, "flops": 4.0 * D * pairs}
    return {"bytes": 4 * q + 4 * k + 4 * B * H * S, "flops": 10.0 * D * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rope(s):
    """Each pair is one complex number: the rotation multiplies it by e^(i angle), the gradient by e^(-i angle)."""
    rot, il = s["rot"], s["interleaved"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None, :, None] * s["inv_freq"])
    first = torch.arange(0, rot, 2) if il else torch.arange(rot // 2)
    second = first + (1 if il else rot // 2)

    def rotated(y, by):
        z = torch.complex(y[..., first], y[..., second]) * by
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    outs, sums = [], []
    for name, w, d in (("q", "qw", "dqo"), ("k", "kw", "dko")):
        x, w = s[name].double(), s[w].double()
        ms = (x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS
        if s["op"] == "norm_rope":
            outs.append(rotated(x / ms.sqrt() * w, turn))
        else:
            g = rotated(s[d].double(), turn.conj())
            sums.append((g * x / ms.sqrt()).sum((0, 1, 2)))
            g = g * w
            outs.append(g / ms.sqrt() - x * (g * x).sum(-1, keepdim=True) / (x.shape[-1] * ms ** 1.5))
    return outs + sums


def _exact_window(s):
    """Head by head, a stretch of positions at a time, against every key up to its last position that any of them sees."""
    B, H, Hkv, S, D, W, ns = (s[n] for n in ("B", "H", "Hkv", "S", "D", "window", "sinks"))
    back = s["op"] == "window_bwd"
    row = torch.argsort(s["pos"])
    at = torch.arange(S, device="cuda")
    grad = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")}
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, S, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            q, k, v = s["q"][b, h, row].double(), s["k"][b, g, row].double(), s["v"][b, g, row].double()
            step = max(512, min(4096, W))
            for p0 in range(0, S, step):
                p = at[p0 : p0 + step]
                t = torch.cat([at[: min(ns, max(0, p0 - W + 1))], at[max(0, p0 - W + 1) : p0 + step]])
                keep = (t <= p[:, None]) & ((p[:, None] - t < W) | (t < ns))
                x = (q[p] @ k[t].T * s["scale"]).masked_fill(~keep, -math.inf)
                z = torch.logsumexp(x, -1)
                pr = torch.exp(x - z[:, None])
                if not back:
                    o[b, h, row[p]], lse[b, h, row[p]] = pr @ v[t], z
                    continue
                do = s["dO"][b, h, row[p]].double()
                dp = do @ v[t].T
                ds = pr * (dp - (pr * dp).sum(-1, keepdim=True)) * s["scale"]
                grad["q"][b, h, row[p]] = ds @ k[t]
                grad["k"][b, g, row[t]] += ds.T @ q[p]
                grad["v"][b, g, row[t]] += pr.T @ do
    return [grad["q"], grad["k"], grad["v"]] if back else [o, lse]


def _exact_decode(s):
    """Request by request: the keys in order of position, prompt then tail."""
    B, H, T, P = s["B"], s["H"], s["T"], s["P"]
    R, G = B // s["Bp"], H // s["Hkv"]
    row = torch.argsort(s["pos"])
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        k = torch.cat([s["kp"][b // R][:, row], s["kt"][b][:, :n]], 1).double()
        v = torch.cat([s["vp"][b // R][:, row], s["vt"][b][:, :n]], 1).double()
        t = torch.arange(P + n, device="cuda")
        for i in range(T):
            p = P + n - T + i
            keep = t <= p
            if s["window"]:
                keep &= (p - t < s["window"]) | (t < s["sinks"])
            if not bool(keep.any()):
                continue
            q = s["q"][b, :, i].double().view(-1, G, s["D"])
            x = (q @ k[:, keep].transpose(1, 2)) * s["scale"]
            lse[b, :, i] = torch.logsumexp(x, -1).reshape(-1)
            o[b, :, i] = (torch.softmax(x, -1) @ v[:, keep]).reshape(H, -1)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm_rope"):
        return _exact_rope(s)
    return _exact_decode(s) if case["op"] == "decode" else _exact_window(s)
