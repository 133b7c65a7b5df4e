"""striped_attn_decode against the 64-bit masked formula."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import BF, attention, keep_mask, positions, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
LSE_TOL = 1e-4  # as for the window attention

CASES = [
    # layout, B, Bp, H, Hkv, T, P, C, D, N, window, sinks, lens
    (sp.STRIPED, 1, 1, 4, 2, 1, 256, 16, 128, 4, 0, 0, [7]),
    (sp.STRIPED, 1, 1, 1, 1, 1, 0, 1, 64, 1, 0, 0, [1]),
    (sp.STRIPED, 3, 1, 4, 1, 1, 1000, 300, 64, 8, 0, 0, [300, 1, 129]),
    (sp.STRIPED, 3, 3, 4, 2, 2, 904, 40, 128, 8, 0, 0, [40, 2, 3]),
    (sp.STRIPED, 4, 2, 6, 2, 5, 903, 200, 128, 3, 0, 0, [200, 128, 5, 77]),
    (sp.STRIPED, 40, 1, 8, 1, 1, 2048, 20, 128, 8, 0, 0, None),         # 320 rows on one prompt: three row tiles
    (sp.STRIPED, 2, 1, 16, 1, 20, 700, 64, 64, 7, 0, 0, [64, 20]),      # 320 rows a request
    (sp.STRIPED, 200, 200, 2, 1, 1, 24, 9, 64, 4, 0, 0, None),          # many small prompts
    (sp.STRIPED, 5, 1, 4, 4, 1, 1300, 150, 128, 13, 0, 0, [0, 1, 150, 128, 127]),   # length 0: the prompt's last token
    (sp.CONTIGUOUS, 2, 1, 4, 2, 3, 777, 130, 64, 7, 0, 0, [1, 2]),      # queries that stand inside the prompt
    (sp.CONTIGUOUS, 2, 2, 2, 2, 4, 2, 8, 128, 1, 0, 0, [0, 1]),         # tokens before position 0
    (sp.STRIPED, 3, 1, 2, 2, 1, 0, 400, 128, 1, 0, 0, [0, 400, 129]),   # no prompt, an empty tail
    (sp.ZIGZAG, 2, 1, 4, 1, 2, 2048, 60, 128, 4, 0, 0, [60, 2]),
    (sp.STRIPED, 3, 1, 4, 2, 1, 1000, 300, 128, 8, 100, 4, [300, 1, 129]),
    (sp.STRIPED, 3, 3, 4, 2, 3, 1000, 300, 64, 8, 280, 1, [300, 3, 129]),
    (sp.STRIPED, 2, 2, 4, 2, 1, 1040, 900, 64, 65, 1, 0, [900, 3]),
    (sp.ZIGZAG, 4, 2, 2, 1, 2, 1536, 500, 64, 3, 300, 200, [500, 400, 2, 130]),
    (sp.STRIPED, 2, 1, 2, 1, 1, 16, 700, 128, 4, 64, 300, [700, 299]),  # sinks that reach into the tails
    (sp.STRIPED, 2, 1, 2, 1, 6, 0, 700, 64, 1, 5, 2, [700, 4]),
    (sp.STRIPED, 2, 1, 2, 1, 1, 512, 700, 64, 4, 5000, 2, [700, 4]),    # a window that none leaves
]


def _make(B, Bp, H, Hkv, T, P, C, D, lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    q, kt, vt = mk(B, H, T, D), mk(B, Hkv, C, D), mk(B, Hkv, C, D)
    kp, vp = (mk(Bp, Hkv, P, D), mk(Bp, Hkv, P, D)) if P else (None, None)
    lens = torch.randint(0, C + 1, (B,), generator=g) if lens is None else torch.tensor(lens)
    return q, kp, vp, kt, vt, lens.to(torch.int32)


def _reference(q, kp, vp, kt, vt, lens, pos, W, ns, scale):
    B, H, T, D = q.shape
    Hkv = kt.shape[1]
    P = 0 if kp is None else kp.shape[2]
    o = torch.zeros(B, H, T, D, dtype=torch.float64)
    tol, lse = torch.zeros_like(o), torch.zeros(B, H, T, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            g = h // (H // Hkv)
            k, v, at = kt[b, g, :n].double(), vt[b, g, :n].double(), P + torch.arange(n)
            if P:
                bp = b // (B // kp.shape[0])
                k, v = torch.cat([kp[bp, g].double(), k]), torch.cat([vp[bp, g].double(), v])
                at = torch.cat([pos, at])
            keep = keep_mask(P + n - T + torch.arange(T), at, W, ns)
            if k.shape[0] == 0:
                lse[b, h] = -float("inf")
                continue
            o[b, h], lse[b, h], p = attention(q[b, h].double(), k, v, keep, scale)
            tol[b, h] = BF * (o[b, h].abs() + 1.02 * p @ v.abs())
    return o, lse, tol + 1e-5


def _gpu(*t):
    return [None if x is None else x.to(DEV) for x in t]


@pytest.mark.parametrize("layout,B,Bp,H,Hkv,T,P,C,D,N,W,ns,lens", CASES)
def test_decode(layout, B, Bp, H, Hkv, T, P, C, D, N, W, ns, lens):
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, lens)
    pos = positions(P, N, layout) if P else None
    o, lse, tol = _reference(q, kp, vp, kt, vt, lens, pos, W, ns, D ** -0.5)
    # what lies behind a tail's end was never written
    behind = (torch.arange(C) >= lens[:, None])[:, None, :, None].expand_as(kt)
    for bad in (float("nan"), float("inf"), -torch.finfo(torch.bfloat16).max):
        kt[behind], vt[behind] = bad, bad
        go, gl = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, lens), N, layout, W, ns)
        assert sp.check_error() == 0
        within(gl, lse, LSE_TOL, "lse")
        within(go, o, tol, "o")


@pytest.mark.parametrize("D,B,H", [(128, 2, 8), (64, 20, 32)])
def test_long_segments_with_a_growing_maximum(D, B, H):
    """Many tiles per multiprocessor, and scores that keep growing with the
    position, so that the running maximum moves again and again; all four
    warps of the row tile at work, or one of them."""
    Hkv, P, C, N = 4, 40000, 200, 8
    q, kp, vp, kt, vt, lens = _make(B, 1, H, Hkv, 1, P, C, D, None, 7)
    pos = positions(P, N, sp.STRIPED)
    grow = (0.2 + 6.0 * pos.double() / P)[None, None, :, None]
    kp = (kp.double().abs() * q[:1, :Hkv].double().sign() * grow).to(torch.bfloat16)
    o, lse, tol = _reference(q, kp, vp, kt, vt, lens, pos, 0, 0, D ** -0.5)
    go, gl = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, lens), N)
    assert sp.check_error() == 0
    within(gl, lse, 4 * LSE_TOL, "lse")  # scores up to a few hundred
    # a score s is off by up to 2^-20 |s| in fp32 sums: its weight by that
    within(go, o, tol + 2.0 ** -11 * vp.double().abs().max(), "o")


def test_lengths_outside_the_tail_are_clamped():
    q, kp, vp, kt, vt, _ = _make(2, 1, 2, 1, 1, 64, 20, 64, [0, 0], 1)
    a = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, torch.tensor([-5, 1 << 30], dtype=torch.int32)), 4)
    b = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, torch.tensor([0, 20], dtype=torch.int32)), 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_then_decode():
    """The run of a request: norm and rotation of the prompt in striped rows,
    the prefill's attention, then tokens one by one with their own positions:
    each gives what the whole sequence's attention gives at its place."""
    B, H, Hkv, P, D, N, steps = 2, 4, 2, 512, 64, 8, 6
    S = P + 8
    g = torch.Generator().manual_seed(2)
    mk = lambda h: torch.randn(B, h, S, D, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, y, v = mk(H), mk(Hkv), mk(Hkv)
    w, f = torch.ones(D, device=DEV), sp.rope_frequencies(D, 1e4, DEV)
    # the whole sequence at once, rows in order
    q_all, k_all = sp.striped_qk_norm_rope(x, y, w, w, f)
    for W, ns in ((0, 0), (100, 4)):
        o_all, lse_all = sp.striped_attn_window_fwd(q_all, k_all, v, 1, W or S, ns)
        first = [sp.striped_permute(t[:, :, :P].contiguous(), N) for t in (x, y, v)]
        qp, kp = sp.striped_qk_norm_rope(first[0], first[1], w, w, f, N)
        o, lse = sp.striped_attn_window_fwd(qp, kp, first[2], N, W or P, ns)
        assert float((sp.striped_unpermute(o, N).float() - o_all[:, :, :P].float()).abs().max()) <= 2e-2
        kt, vt = (torch.full((B, Hkv, 32, D), float("nan"), device=DEV, dtype=torch.bfloat16) for _ in range(2))
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        for i in range(steps):
            at = torch.full((B, 1), P + i, device=DEV)
            qi, ki = sp.striped_qk_norm_rope(x[:, :, P + i:P + i + 1].contiguous(),
                                             y[:, :, P + i:P + i + 1].contiguous(), w, w, f, positions=at)
            kt[:, :, i], vt[:, :, i] = ki[:, :, 0], v[:, :, P + i]
            lens += 1
            oi, li = sp.striped_attn_decode(qi, kp, first[2], kt, vt, lens, N, sp.STRIPED, W, ns)
            assert float((li[:, :, 0] - lse_all[:, :, P + i]).abs().max()) <= 2 * LSE_TOL
            assert float((oi[:, :, 0].float() - o_all[:, :, P + i].float()).abs().max()) <= 2e-2
        # the last tokens again, several at a time
        qi = q_all[:, :, P + 2:P + steps].contiguous()
        oi, li = sp.striped_attn_decode(qi, kp, first[2], kt, vt, lens, N, sp.STRIPED, W, ns)
        assert float((li - lse_all[:, :, P + 2:P + steps]).abs().max()) <= 2 * LSE_TOL


def test_shared_prompt_is_each_requests_own():
    B, H, Hkv, P, C, D, N = 6, 4, 2, 1024, 40, 128, 8
    q, kp, vp, kt, vt, lens = _gpu(*_make(B, 1, H, Hkv, 1, P, C, D, None, 3))
    o, lse = sp.striped_attn_decode(q, kp, vp, kt, vt, lens, N)
    own = [t.expand(B, -1, -1, -1).contiguous() for t in (kp, vp)]
    o2, lse2 = sp.striped_attn_decode(q, *own, kt, vt, lens, N)
    assert float((lse - lse2).abs().max()) <= LSE_TOL
    assert float((o.float() - o2.float()).abs().max()) <= 2e-2


def test_run_to_run_stream_and_graph():
    B, H, Hkv, P, C, D, N = 5, 8, 2, 4096, 300, 128, 8
    args = _gpu(*_make(B, 1, H, Hkv, 1, P, C, D, None, 4))
    want = sp.striped_attn_decode(*args, N)
    again = sp.striped_attn_decode(*args, N)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sp.striped_attn_decode(*args, N, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # a captured step replayed for growing tails: the lengths are read on the device
    bufs = [torch.zeros_like(t) for t in args]
    ws = sp.new_decode_workspace(bufs[0], bufs[1], bufs[3], N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = sp.striped_attn_decode(*bufs, N, workspace=ws)
    for t, s in zip(bufs, args):
        t.copy_(s)
    for n in (1, 128, 129, 300):
        bufs[5].fill_(n)
        graph.replay()
        o, lse = sp.striped_attn_decode(*args[:5], torch.full_like(args[5], n), N)
        torch.cuda.synchronize()
        assert torch.equal(go, o) and torch.equal(gl, lse)
    assert sp.check_error() == 0


def test_a_missing_tile_times_out():
    args = _gpu(*_make(2, 1, 2, 1, 1, 1024, 40, 128, [3, 40], 5))
    want = sp.striped_attn_decode(*args, 8)
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 20_000_000)
        sp.striped_attn_decode(*args, 8)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    got = sp.striped_attn_decode(*args, 8)
    assert torch.equal(want[0], got[0]) and sp.check_error() == 0


def test_wrapper_refusals():
    q, kp, vp, kt, vt, lens = _gpu(*_make(4, 2, 4, 2, 1, 256, 16, 64, None, 6))
    with pytest.raises(TypeError):
        sp.striped_attn_decode(q, kp, vp, kt, vt, lens.long(), 4)
    with pytest.raises(TypeError):
        sp.striped_attn_decode(q, kp, vp, kt, vt, lens.cpu(), 4)
    with pytest.raises(ValueError):
        sp.striped_attn_decode(q, kp, vp[:, :, :128].contiguous(), kt, vt, lens, 4)
    with pytest.raises(ValueError):
        sp.striped_attn_decode(q, kp, vp, kt, vt, lens[:3].contiguous(), 4)
    with pytest.raises(TypeError):
        sp.striped_attn_decode(q, kp, vp, kt.float(), vt, lens, 4)
    with pytest.raises(sp.StripedError):
        sp.striped_attn_decode(q, kp, vp, kt, vt, lens, 3)
    with pytest.raises(sp.StripedError):
        sp.striped_attn_decode(q[:3].contiguous(), kp, vp, kt[:3].contiguous(), vt[:3].contiguous(),
                               lens[:3].contiguous(), 4)
    with pytest.raises(sp.StripedError):
        sp.striped_attn_decode(q, kp, vp, kt, vt, lens, 4,
                               workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.fixture
def emptied_cache():
    """The memory of a large test goes back to the device."""
    yield
    torch.cuda.empty_cache()


def test_offsets_past_32_bits(emptied_cache):
    """More than 2^31 elements of prompt and of tails: the last key/value head
    of the last request is what it is alone."""
    B, H, Hkv, P, C, D, N = 2, 64, 32, 1 << 20, 1 << 19, 128, 8
    g = torch.Generator(device=DEV).manual_seed(6)
    mk = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV).normal_(generator=g)  # noqa: E731
    q, kp, vp, kt, vt = mk(B, H, 1, D), mk(1, Hkv, P, D), mk(1, Hkv, P, D), mk(B, Hkv, C, D), mk(B, Hkv, C, D)
    lens = torch.tensor([5, C], dtype=torch.int32, device=DEV)
    last = [q[1:, -2:], kp[:, -1:], vp[:, -1:], kt[1:, -1:], vt[1:, -1:], lens[1:]]
    last = [t.contiguous() for t in last]
    for W, ns in ((0, 0), (C + 1000, 9)):
        o, lse = sp.striped_attn_decode(q, kp, vp, kt, vt, lens, N, sp.STRIPED, W, ns)
        o1, lse1 = sp.striped_attn_decode(*last, N, sp.STRIPED, W, ns)
        # cut into other segments: their sums are rounded in another order
        assert float((lse[1:, -2:] - lse1).abs().max()) <= LSE_TOL
        assert float((o[1:, -2:].float() - o1.float()).abs().max()) <= 2.0 ** -7 * float(o1.float().abs().max())
    assert sp.check_error() == 0


ROW_TILES = [
    # more than 128 rows on a prompt: layout, B, Bp, H, Hkv, T, P, C, D, N, window, sinks
    (sp.STRIPED, 40, 1, 8, 1, 1, 8192, 20, 64, 8, 0, 0),      # 320 rows
    (sp.STRIPED, 20, 2, 8, 1, 5, 2048, 20, 128, 4, 0, 0),     # 400 rows on each of two prompts
    (sp.STRIPED, 33, 1, 16, 2, 1, 6000, 1, 128, 3, 0, 0),     # 264 rows, tails of one row
    (sp.ZIGZAG, 64, 1, 8, 2, 1, 12288, 30, 128, 4, 6000, 5),  # 256 rows, a window
    (sp.STRIPED, 10, 1, 8, 1, 13, 4096, 100, 64, 8, 0, 0),    # 1040 rows: nine row tiles
]


@pytest.mark.parametrize("layout,B,Bp,H,Hkv,T,P,C,D,N,W,ns", ROW_TILES)
def test_several_row_tiles(layout, B, Bp, H, Hkv, T, P, C, D, N, W, ns):
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, None, 8)
    o, lse, tol = _reference(q, kp, vp, kt, vt, lens, positions(P, N, layout), W, ns, D ** -0.5)
    go, gl = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, lens), N, layout, W, ns)
    assert sp.check_error() == 0
    within(gl, lse, LSE_TOL, "lse")
    within(go, o, tol, "o")


@pytest.mark.parametrize("B,Bp,H,Hkv,T,P,C,D,N,W,ns", [(40, 1, 8, 1, 1, 2048, 20, 64, 8, 0, 0),
                                                       (3, 3, 4, 2, 3, 1000, 300, 128, 8, 280, 1),
                                                       (5, 1, 4, 4, 1, 0, 700, 64, 1, 0, 0)])
def test_missing_tiles_end_and_leave_the_device_usable(B, Bp, H, Hkv, T, P, C, D, N, W, ns):
    """Row tiles with one and with four warps at work, tails with unwritten rows."""
    args = _gpu(*_make(B, Bp, H, Hkv, T, P, C, D, None, 9))
    want = sp.striped_attn_decode(*args, N, sp.STRIPED, W, ns)
    assert sp.check_error() == 0
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 5_000_000)
        sp.striped_attn_decode(*args, N, sp.STRIPED, W, ns)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    got = sp.striped_attn_decode(*args, N, sp.STRIPED, W, ns)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and sp.check_error() == 0


@pytest.mark.parametrize("layout,B,Bp,H,Hkv,T,P,C,D,N,W,ns", [
    (sp.STRIPED, 1024, 1024, 2, 1, 1, 24, 9, 64, 4, 0, 0),    # 1024 prompts and 1024 tails: the most that a call takes
    (sp.STRIPED, 2048, 1, 1, 1, 1, 0, 140, 128, 1, 100, 3),   # 2048 tails
    (sp.CONTIGUOUS, 1000, 2, 1, 1, 2, 300, 3, 64, 1, 64, 0)])
def test_the_most_requests_of_a_call(layout, B, Bp, H, Hkv, T, P, C, D, N, W, ns):
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, None, 15)
    o, lse, tol = _reference(q, kp, vp, kt, vt, lens, positions(P, N, layout) if P else None, W, ns, D ** -0.5)
    behind = (torch.arange(C) >= lens[:, None])[:, None, :, None].expand_as(kt)
    kt[behind], vt[behind] = float("nan"), float("nan")
    go, gl = sp.striped_attn_decode(*_gpu(q, kp, vp, kt, vt, lens), N, layout, W, ns)
    assert sp.check_error() == 0
    within(gl, lse, LSE_TOL, "lse")
    within(go, o, tol, "o")


def test_half_a_prompt_is_refused():
    q, kp, vp, kt, vt, lens = _gpu(*_make(4, 2, 4, 2, 1, 256, 16, 64, None, 16))
    with pytest.raises(ValueError):
        sp.striped_attn_decode(q, None, vp, kt, vt, lens, 4)
    with pytest.raises(TypeError):
        sp.striped_attn_decode(q, kp, None, kt, vt, lens, 4)
    sp.striped_attn_decode(q, None, None, kt, vt, lens)
    assert sp.check_error() == 0
