"""striped_attn_window_fwd / _bwd against the 64-bit masked formula."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions, window_reference, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
# LSE: the scores' fp32 sums (128 products) and the row sum's at most 2^-22 of
# the row each, ex2 2^-22; under 1e-4 at scores below 100
LSE_TOL = 1e-4

CASES = [
    # layout, B, H, Hkv, S, D, N, window, sinks
    (sp.STRIPED, 1, 2, 2, 256, 128, 4, 64, 0),
    (sp.STRIPED, 1, 1, 1, 1, 64, 1, 1, 0),
    (sp.STRIPED, 1, 1, 1, 1, 128, 1, 7, 3),
    (sp.STRIPED, 2, 2, 2, 40, 128, 8, 1, 0),
    (sp.STRIPED, 1, 4, 1, 1000, 64, 8, 100, 4),
    (sp.STRIPED, 1, 2, 1, 1000, 128, 8, 128, 128),
    (sp.STRIPED, 1, 2, 2, 1024, 128, 8, 129, 1),
    (sp.STRIPED, 1, 4, 2, 903, 128, 3, 200, 5),
    (sp.STRIPED, 1, 1, 1, 1300, 64, 13, 37, 130),
    (sp.STRIPED, 1, 2, 1, 1040, 64, 65, 300, 3),
    (sp.STRIPED, 1, 1, 1, 1280, 128, 128, 5, 1024),
    (sp.STRIPED, 1, 2, 2, 1920, 128, 96, 500, 2),
    (sp.STRIPED, 1, 2, 2, 640, 128, 5, 10000, 0),
    (sp.STRIPED, 1, 2, 2, 640, 64, 16, 640, 640),
    (sp.CONTIGUOUS, 1, 2, 2, 777, 128, 7, 100, 9),
    (sp.CONTIGUOUS, 3, 3, 1, 130, 64, 1, 2, 1),
    (sp.ZIGZAG, 1, 2, 1, 2048, 128, 4, 300, 16),
    (sp.ZIGZAG, 1, 2, 2, 1024, 64, 1, 257, 0),
    (sp.ZIGZAG, 1, 3, 3, 1536, 64, 3, 1, 4),
]


def _make(B, H, Hkv, S, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h: torch.randn(B, h, S, D, generator=g).to(torch.bfloat16)  # noqa: E731
    return mk(H), mk(Hkv), mk(Hkv), mk(H)


@pytest.mark.parametrize("layout,B,H,Hkv,S,D,N,W,ns", CASES)
def test_forward(layout, B, H, Hkv, S, D, N, W, ns):
    q, k, v, _ = _make(B, H, Hkv, S, D)
    scale = D ** -0.5
    r = window_reference(q, k, v, positions(S, N, layout), W, ns, scale)
    o, lse = sp.striped_attn_window_fwd(q.to(DEV), k.to(DEV), v.to(DEV), N, W, ns, layout)
    assert sp.check_error() == 0
    within(lse, r["lse"], LSE_TOL, "lse")
    within(o, r["o"], r["o_tol"], "o")


@pytest.mark.parametrize("layout,B,H,Hkv,S,D,N,W,ns", CASES)
def test_backward(layout, B, H, Hkv, S, D, N, W, ns):
    q, k, v, do = _make(B, H, Hkv, S, D, 1)
    scale = 0.11
    pos = positions(S, N, layout)
    r = window_reference(q, k, v, pos, W, ns, scale)
    o, lse = r["o"].to(torch.bfloat16), r["lse"].float()
    r = window_reference(q, k, v, pos, W, ns, scale, do, o)
    dq, dk, dv = sp.striped_attn_window_bwd(*[t.to(DEV) for t in (q, k, v, o, lse, do)], N, W, ns, layout, scale)
    assert sp.check_error() == 0
    within(dv, r["dv"], r["dv_tol"], "dv")
    within(dk, r["dk"], r["dk_tol"], "dk")
    within(dq, r["dq"], r["dq_tol"], "dq")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout,N", [(sp.STRIPED, 8), (sp.ZIGZAG, 4), (sp.CONTIGUOUS, 2)])
def test_whole_window_is_the_full_attention(layout, N, D):
    """window >= S: the same function as striped_attn_fwd / _bwd."""
    B, H, Hkv, S = 1, 4, 2, 1024
    q, k, v, do = (t.to(DEV) for t in _make(B, H, Hkv, S, D, 2))
    o1, l1 = sp.striped_attn_fwd(q, k, v, N, layout)
    o2, l2 = sp.striped_attn_window_fwd(q, k, v, N, S, 0, layout)
    assert float((l1 - l2).abs().max()) <= LSE_TOL
    assert float((o1.float() - o2.float()).abs().max()) <= 2e-2
    for a, b in zip(sp.striped_attn_bwd(q, k, v, o1, l1, do, N, layout),
                    sp.striped_attn_window_bwd(q, k, v, o1, l1, do, N, S, 0, layout)):
        # both sides of two query heads' bf16 gradients
        assert float((a.float() - b.float()).abs().max()) <= 2 * 2e-2 * 2 ** 0.5


def test_rotation_then_window_then_gradient():
    """The run of a local layer's step: norm and rotation in striped rows,
    window attention, and both gradients back to the projections."""
    from tests._local_util import norm_rope_reference

    B, H, Hkv, S, D, N, W, ns = 1, 4, 2, 480, 64, 8, 70, 3
    g = torch.Generator().manual_seed(9)
    mk = lambda h: torch.randn(B, h, S, D, generator=g).to(torch.bfloat16)  # noqa: E731
    x, y, v, do = mk(H), mk(Hkv), mk(Hkv), mk(H)
    w = 1 + 0.1 * torch.randn(D, generator=g)
    f = sp.rope_frequencies(D, 1e4, "cpu")
    pos = positions(S, N, sp.STRIPED)
    d = [t.to(DEV) for t in (x, y, w, w, f)]
    q, k = sp.striped_qk_norm_rope(*d, N)
    o, lse = sp.striped_attn_window_fwd(q, k, v.to(DEV), N, W, ns)
    dq, dk, dv = sp.striped_attn_window_bwd(q, k, v.to(DEV), o, lse, do.to(DEV), N, W, ns)
    dx, dy, dwq, dwk = sp.striped_qk_norm_rope_bwd(d[0], d[1], dq, dk, d[2], d[3], d[4], N)
    # the attention against its formula on the rotated tensors that it got
    r = window_reference(q.cpu(), k.cpu(), v, pos, W, ns, D ** -0.5, do, o.cpu())
    within(o, r["o"], r["o_tol"], "o")
    for n, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, r[n], r[n + "_tol"] + 1e-3 * r[n].abs(), n)  # lse is the kernel's own (1e-4 off)
    # the whole chain in 64 bits, by automatic differentiation of the formula
    x6, y6, w6 = x.double().requires_grad_(), y.double().requires_grad_(), w.double().requires_grad_()
    q6 = norm_rope_reference(x6, w6, pos[None], f, 1e-6, False)["y"]
    k6 = norm_rope_reference(y6, w6, pos[None], f, 1e-6, False)["y"]
    keep = (pos[None] <= pos[:, None]) & ((pos[:, None] - pos[None] < W) | (pos[None] < ns))
    kk, vv = (t.repeat_interleave(H // Hkv, 1) for t in (k6, v.double()))
    p = torch.softmax((q6 @ kk.transpose(-1, -2) * D ** -0.5).masked_fill(~keep, float("-inf")), -1)
    ((p @ vv) * do.double()).sum().backward()
    for got, ref in ((dx, x6.grad), (dy, y6.grad), (dwq + dwk, w6.grad)):
        # q, k, o, dq and dk are rounded to bf16 between the calls: five roundings of 2^-8
        assert float((got.double().cpu() - ref).norm() / ref.norm()) <= 5 * 2.0 ** -8


def test_run_to_run_stream_and_graph():
    B, H, Hkv, S, D, N, W, ns = 1, 4, 2, 2048, 128, 8, 300, 4
    q, k, v, do = (t.to(DEV) for t in _make(B, H, Hkv, S, D, 3))
    o, lse = sp.striped_attn_window_fwd(q, k, v, N, W, ns)
    grads = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = sp.striped_attn_window_fwd(q, k, v, N, W, ns, stream=side)
    g2 = None
    with torch.cuda.stream(side):
        g2 = sp.striped_attn_window_bwd(q, k, v, o2, lse2, do, N, W, ns)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(grads[1], g2[1]) and torch.equal(grads[2], g2[2])  # dK and dV: fixed order
    bufs = [torch.zeros_like(t) for t in (q, k, v, do)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = sp.striped_attn_window_fwd(*bufs[:3], N, W, ns)
        gg = sp.striped_attn_window_bwd(*bufs[:3], go, gl, bufs[3], N, W, ns)
    for t, s in zip(bufs, (q, k, v, do)):
        t.copy_(s)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(go, o) and torch.equal(gl, lse)
    assert torch.equal(gg[1], grads[1]) and torch.equal(gg[2], grads[2])
    assert sp.check_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_results_at_16_byte_addresses(D):
    """Results that start 16 bytes past a 32-byte boundary: the same values."""
    B, H, Hkv, S, N, W, ns = 1, 2, 1, 600, 4, 100, 3
    q, k, v, do = (t.to(DEV) for t in _make(B, H, Hkv, S, D, 8))

    def off(t):  # an uninitialised tensor like t, 16 bytes into its storage
        return torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8:].view(t.shape)

    o, lse = sp.striped_attn_window_fwd(q, k, v, N, W, ns)
    o2, lse2 = sp.striped_attn_window_fwd(q, k, v, N, W, ns, out=off(o))
    assert o2.data_ptr() % 32 == 16 and torch.equal(o, o2) and torch.equal(lse, lse2)
    want = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns)
    got = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, dq=off(q), dk=off(k), dv=off(v))
    assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])
    # dQ is summed by atomics: a bf16 rounding apart at most
    assert float((want[0].float() - got[0].float()).abs().max()) <= 2.0 ** -7 * float(want[0].float().abs().max())


def test_a_missing_tile_times_out():
    """The bounded waits end, report and leave the device usable."""
    q, k, v, do = (t.to(DEV) for t in _make(1, 2, 2, 512, 128, 4))
    o, lse = sp.striped_attn_window_fwd(q, k, v, 4, 100, 1)
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 20_000_000)
        sp.striped_attn_window_fwd(q, k, v, 4, 100, 1)
        assert sp.check_error() == -5
        sp.test_inject(sp.FAULT_BWD_SKIP_Q, 20_000_000)
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, 4, 100, 1)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    o2, _ = sp.striped_attn_window_fwd(q, k, v, 4, 100, 1)
    assert torch.equal(o, o2) and sp.check_error() == 0


def test_wrapper_refusals():
    q = torch.zeros(1, 4, 256, 64, dtype=torch.bfloat16, device=DEV)
    k = q[:, :2].contiguous()
    with pytest.raises(ValueError):
        sp.striped_attn_window_fwd(q, k, q, 4, 10)
    with pytest.raises(TypeError):
        sp.striped_attn_window_fwd(q, k, k.float(), 4, 10)
    with pytest.raises(ValueError):
        sp.striped_attn_window_fwd(q, k.transpose(1, 2), k, 4, 10)
    with pytest.raises(TypeError):
        sp.striped_attn_window_fwd(q, k, k, 4, 10, lse_out=torch.zeros(1, 4, 256, device=DEV, dtype=torch.float64))
    with pytest.raises(sp.StripedError):
        sp.striped_attn_window_fwd(q.float(), k.float(), k.float(), 4, 10)
    with pytest.raises(sp.StripedError):
        sp.striped_attn_window_fwd(q, k, k, 4, 0)
    with pytest.raises(sp.StripedError):
        sp.striped_attn_window_fwd(q, k, k, 4, 10, 1025)


@pytest.mark.parametrize("layout,N,D", [(sp.STRIPED, 4, 128), (sp.CONTIGUOUS, 1, 64)])
def test_padded_rows_do_not_reach_the_real_ones(layout, N, D):
    """Rows behind the last token of a padded sequence may hold anything
    finite: the real rows are those of the short sequence, and with dO = 0
    there the padding's dK and dV are 0."""
    B, H, Hkv, S, real, W, ns = 1, 2, 1, 512, 300, 70, 2
    q, k, v, do = _make(B, H, Hkv, real, D, 11)
    scale = D ** -0.5

    def padded(t, fill):
        return torch.cat([t, torch.full((B, t.shape[1], S - real, D), fill, dtype=t.dtype)], 2)

    def place(t):
        t = t.to(DEV)
        return sp.striped_permute(t, N) if layout == sp.STRIPED else t

    def back(t):
        return sp.striped_unpermute(t, N) if layout == sp.STRIPED else t

    args = [place(padded(t, fill)) for t, fill in ((q, 300.0), (k, -200.0), (v, 1e30))]
    o, lse = sp.striped_attn_window_fwd(*args, N, W, ns, layout)
    r = window_reference(q, k, v, torch.arange(real), W, ns, scale, do, back(o)[:, :, :real].cpu())
    within(back(o)[:, :, :real], r["o"], r["o_tol"], "o")
    dq, dk, dv = sp.striped_attn_window_bwd(*args, o, lse, place(padded(do, 0.0)), N, W, ns, layout)
    for name, t in (("dk", dk), ("dv", dv)):
        within(back(t)[:, :, :real], r[name], r[name + "_tol"], name)
        assert not back(t)[:, :, real:].any()
    within(back(dq)[:, :, :real], r["dq"], r["dq_tol"], "dq")
    assert sp.check_error() == 0


def test_calls_side_by_side():
    """Two threads on streams of their own: every call has its own workspace,
    and kernels that share a multiprocessor wait for its tensor memory."""
    import threading

    jobs = []
    for D, seed in ((128, 21), (64, 22)):
        q, k, v, do = (t.to(DEV) for t in _make(1, 4, 2, 1500, D, seed))
        w, f = torch.ones(D, device=DEV), sp.rope_frequencies(D, 1e4, DEV)
        kt, vt = (t[:, :, :200].expand(3, -1, -1, -1).contiguous() for t in (k, v))
        lens = torch.tensor([1, 77, 200], dtype=torch.int32, device=DEV)
        new = q[:, :, :1].expand(3, -1, -1, -1).contiguous()

        def run(q=q, k=k, v=v, do=do, w=w, f=f, kt=kt, vt=vt, lens=lens, new=new):
            a, b = sp.striped_qk_norm_rope(q, k, w, w, f, 4)
            o, lse = sp.striped_attn_window_fwd(a, b, v, 4, 200, 2)
            _, dk, dv = sp.striped_attn_window_bwd(a, b, v, o, lse, do, 4, 200, 2)
            g = sp.striped_qk_norm_rope_bwd(q, k, o, dk, w, w, f, 4)
            return (a, b, o, lse, dk, dv) + g + sp.striped_attn_decode(new, b, v, kt, vt, lens, 4)

        jobs.append((run, run()))
    torch.cuda.synchronize()
    bad = []

    def work(run, want):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = [run() for _ in range(10)]
        side.synchronize()
        bad.extend(i for g in got for i, (x, y) in enumerate(zip(g, want)) if not torch.equal(x, y))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and sp.check_error() == 0


@pytest.fixture
def emptied_cache():
    """The memory of a large test goes back to the device."""
    yield
    torch.cuda.empty_cache()


def test_offsets_past_32_bits(emptied_cache):
    """More than 2^31 elements a tensor: the last head is what it is alone."""
    S, D, N, W, ns = 1 << 19, 128, 8, 100, 3
    H = (1 << 31) // (S * D) + 1
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v, do = (torch.empty(1, H, S, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(4))
    w, f = torch.ones(D, device=DEV), sp.rope_frequencies(D, 1e4, DEV)
    one = [t[:, -1:].contiguous() for t in (q, k, v, do)]
    a, b = sp.striped_qk_norm_rope(q, k, w, w, f, N)
    a1, b1 = sp.striped_qk_norm_rope(one[0], one[1], w, w, f, N)
    assert torch.equal(a[:, -1:], a1) and torch.equal(b[:, -1:], b1)
    o, lse = sp.striped_attn_window_fwd(a, b, v, N, W, ns)
    o1, lse1 = sp.striped_attn_window_fwd(a1, b1, one[2], N, W, ns)
    assert torch.equal(o[:, -1:], o1) and torch.equal(lse[:, -1:], lse1)
    grads = sp.striped_attn_window_bwd(a, b, v, o, lse, do, N, W, ns)
    grads1 = sp.striped_attn_window_bwd(a1, b1, one[2], o1, lse1, one[3], N, W, ns)
    assert torch.equal(grads[1][:, -1:], grads1[1]) and torch.equal(grads[2][:, -1:], grads1[2])
    # dQ is summed by atomics: a bf16 rounding apart at most
    off = (grads[0][:, -1:].float() - grads1[0].float()).abs().max()
    assert float(off) <= 2.0 ** -7 * float(grads1[0].float().abs().max())
    dx = sp.striped_qk_norm_rope_bwd(q, k, grads[1], grads[2], w, w, f, N)
    dx1 = sp.striped_qk_norm_rope_bwd(one[0], one[1], grads1[1], grads1[2], w, w, f, N)
    assert torch.equal(dx[0][:, -1:], dx1[0]) and torch.equal(dx[1][:, -1:], dx1[1])
    assert sp.check_error() == 0


@pytest.mark.parametrize("layout,N,D,W,ns", [(sp.STRIPED, 8, 64, 200, 4), (sp.STRIPED, 3, 128, 1500, 0),
                                             (sp.CONTIGUOUS, 1, 64, 1, 0), (sp.ZIGZAG, 2, 128, 300, 200)])
def test_missing_tiles_end_and_leave_the_device_usable(layout, N, D, W, ns):
    """Every role's waits run out: the calls return, report, and the next ones
    give what they gave before."""
    S = 1536 if layout != sp.STRIPED else 1503 // N * N
    q, k, v, do = (t.to(DEV) for t in _make(2, 4, 2, S, D, 12))
    o, lse = sp.striped_attn_window_fwd(q, k, v, N, W, ns, layout)
    grads = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, layout)
    assert sp.check_error() == 0
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 5_000_000)
        sp.striped_attn_window_fwd(q, k, v, N, W, ns, layout)
        assert sp.check_error() == -5
        sp.test_inject(sp.FAULT_BWD_SKIP_Q, 5_000_000)
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, layout)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    o2, lse2 = sp.striped_attn_window_fwd(q, k, v, N, W, ns, layout)
    again = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, layout)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and sp.check_error() == 0
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])


def test_many_heads_with_sinks(emptied_cache):
    """More than 65535 sink tiles: the last heads are what they are alone."""
    B, H, S, D, N, W, ns = 16500, 4, 300, 64, 4, 5, 3
    g = torch.Generator(device=DEV).manual_seed(13)
    q, k, v, do = (torch.empty(B, H, S, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(4))
    o, lse = sp.striped_attn_window_fwd(q, k, v, N, W, ns)
    dq, dk, dv = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns)
    last = [t[-2:].contiguous() for t in (q, k, v, o, lse, do)]
    o1, lse1 = sp.striped_attn_window_fwd(*last[:3], N, W, ns)
    dq1, dk1, dv1 = sp.striped_attn_window_bwd(*last, N, W, ns)
    assert torch.equal(o[-2:], o1) and torch.equal(lse[-2:], lse1)
    assert torch.equal(dk[-2:], dk1) and torch.equal(dv[-2:], dv1) and sp.check_error() == 0
    # dQ is summed by atomics: a bf16 rounding apart at most
    assert float((dq[-2:].float() - dq1.float()).abs().max()) <= 2.0 ** -7 * float(dq1.float().abs().max())


def test_workspace_of_the_caller():
    q, k, v, do = (t.to(DEV) for t in _make(1, 4, 2, 1500, 64, 14))
    N, W, ns = 4, 200, 130
    o, lse = sp.striped_attn_window_fwd(q, k, v, N, W, ns)
    want = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns)
    ws = sp.new_window_workspace(q, k, N, W, ns)
    for i in (255, 0):  # contents on entry are ignored
        ws.fill_(i)
        got = sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, workspace=ws)
        assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])
        off = (want[0].float() - got[0].float()).abs().max()
        assert float(off) <= 2.0 ** -7 * float(want[0].float().abs().max())
    with pytest.raises(sp.StripedError):
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, workspace=ws[:-256])
    with pytest.raises(sp.StripedError):
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, workspace=ws[16:])
    with pytest.raises(ValueError):
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, workspace=ws.view(2, -1))
    with pytest.raises(TypeError):
        sp.striped_attn_window_bwd(q, k, v, o, lse, do, N, W, ns, workspace=ws.cpu())
    assert sp.check_error() == 0
