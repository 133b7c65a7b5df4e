"""striped_qk_norm_rope and its gradient against the 64-bit formula."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import BF, F32, norm_rope_reference, positions, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
# Angles, the norm and the products: under 24 fp32 half-steps of a pair's
# magnitude (the mean of up to 256 squares adds at most 8, sincospi and the
# rounded phase 4, products and sums the rest).
STEPS = 24 * F32


def _make(B, H, Hkv, S, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    size = torch.randn(B, 1, S, 1, generator=g).exp()
    q = (torch.randn(B, H, S, D, generator=g) * size).to(dtype)
    k = (torch.randn(B, Hkv, S, D, generator=g) * size).to(dtype)
    qw, kw = 1 + 0.3 * torch.randn(D, generator=g), 1 + 0.3 * torch.randn(D, generator=g)
    dq, dk = torch.randn(B, H, S, D, generator=g).to(dtype), torch.randn(B, Hkv, S, D, generator=g).to(dtype)
    return q, k, qw, kw, dq, dk


def _rel(dtype):
    return BF if dtype == torch.bfloat16 else F32


CASES = [
    # layout, B, H, Hkv, S, D, rot, N, interleaved
    (sp.STRIPED, 1, 4, 2, 96, 128, 128, 8, False),
    (sp.STRIPED, 2, 3, 1, 303, 64, 64, 3, True),
    (sp.STRIPED, 1, 1, 1, 1, 128, 128, 1, False),
    (sp.CONTIGUOUS, 3, 9, 3, 37, 64, 32, 1, False),
    (sp.ZIGZAG, 1, 2, 2, 120, 128, 64, 5, True),
    (sp.STRIPED, 1, 17, 1, 40, 96, 32, 4, False),
    (sp.STRIPED, 2, 1, 2, 14, 256, 256, 7, False),
    (sp.STRIPED, 1, 2, 2, 33, 16, 16, 1, True),
    (sp.CONTIGUOUS, 1, 2, 1, 5000, 64, 0, 1, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,B,H,Hkv,S,D,rot,N,il", CASES)
def test_forward_and_gradient(layout, B, H, Hkv, S, D, rot, N, il, dtype):
    q, k, qw, kw, dq, dk = _make(B, H, Hkv, S, D, dtype)
    f = sp.rope_frequencies(rot, 10000.0, "cpu")
    pos = positions(S, N, layout)[None]
    d = [t.to(DEV) for t in (q, k, qw, kw, f)]
    yq, yk = sp.striped_qk_norm_rope(*d, N, layout, eps=EPS, interleaved=il)
    gq, gk, gqw, gkw = sp.striped_qk_norm_rope_bwd(d[0], d[1], dq.to(DEV), dk.to(DEV), d[2], d[3], d[4], N, layout,
                                                   eps=EPS, interleaved=il)
    for x, w, g, y, dx, dw in ((q, qw, dq, yq, gq, gqw), (k, kw, dk, yk, gk, gkw)):
        r = norm_rope_reference(x, w, pos, f, EPS, il, g)
        assert y.dtype == dtype and dx.dtype == dtype and dw.dtype == torch.float32
        within(y, r["y"], _rel(dtype) * r["y"].abs() + STEPS * r["y_mag"] + 1e-30, "y")
        within(dx, r["dx"], _rel(dtype) * r["dx"].abs() + STEPS * r["dx_mag"] + 1e-30, "dx")
        # a thread adds at most 64 rows here, the block and the last kernel 64 shares
        within(dw, r["dw"], (128 * F32 + STEPS) * r["dw_mag"] + 1e-30, "dw")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_given_positions_far_out(dtype):
    """Positions of their own, beyond 2^31 and negative: the phase is exact."""
    B, H, Hkv, S, D = 3, 4, 2, 5, 128
    q, k, qw, kw, dq, dk = _make(B, H, Hkv, S, D, dtype, 3)
    f = sp.rope_frequencies(D, 500000.0, "cpu")
    pos = torch.tensor([[0, 1, 786431, 2 ** 20 + 1, 5], [2 ** 31 - 1, 2 ** 31 + 7, 3, 4, 2 ** 33], [-1, -4097, 0, 9, 1]])
    yq, yk = sp.striped_qk_norm_rope(*[t.to(DEV) for t in (q, k, qw, kw, f)], positions=pos.to(DEV), eps=EPS)
    # 2 pi p f in 64 bits is itself off by 2^-53 of the angle, under 1e-6 at 2^33
    for x, w, y in ((q, qw, yq), (k, kw, yk)):
        r = norm_rope_reference(x, w, pos, f, EPS, False)
        within(y, r["y"], _rel(dtype) * r["y"].abs() + (STEPS + 1e-6) * r["y_mag"], "y")


@pytest.mark.parametrize("layout", [sp.STRIPED, sp.CONTIGUOUS, sp.ZIGZAG])
def test_one_stripe_is_its_slice(layout):
    """Rank d of a ring gets, for its own rows, the rows of the whole call."""
    B, H, Hkv, N, L, D = 2, 3, 1, 4, 22, 64
    q, k, qw, kw, dq, dk = _make(B, H, Hkv, N * L, D, torch.bfloat16, 4)
    f = sp.rope_frequencies(D, 10000.0, DEV)
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in (q, k, qw, kw, dq, dk))
    yq, yk = sp.striped_qk_norm_rope(q, k, qw, kw, f, N, layout)
    gq, gk, _, _ = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, N, layout)
    for d in range(N):
        c = [t[:, :, d * L:(d + 1) * L].contiguous() for t in (q, k, dq, dk)]
        zq, zk = sp.striped_qk_norm_rope(c[0], c[1], qw, kw, f, N, layout, stripe=d)
        hq, hk, _, _ = sp.striped_qk_norm_rope_bwd(*c, qw, kw, f, N, layout, stripe=d)
        for whole, part in ((yq, zq), (yk, zk), (gq, hq), (gk, hk)):
            assert torch.equal(whole[:, :, d * L:(d + 1) * L], part)


def test_in_place_and_run_to_run():
    B, H, Hkv, S, D = 1, 8, 2, 777, 128
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in _make(B, H, Hkv, S, D, torch.bfloat16, 5))
    f = sp.rope_frequencies(D, 10000.0, DEV)
    yq, yk = sp.striped_qk_norm_rope(q, k, qw, kw, f)
    a, b = q.clone(), k.clone()
    sp.striped_qk_norm_rope(a, b, qw, kw, f, q_out=a, k_out=b)
    assert torch.equal(a, yq) and torch.equal(b, yk)
    first = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f)
    again = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    a, b = dq.clone(), dk.clone()
    over = sp.striped_qk_norm_rope_bwd(q, k, a, b, qw, kw, f, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(first, over))


def test_gradient_against_differences():
    """Central differences of the fp32 kernel's own forward.  The loss
    sum(c * y) is linear in w, quadratic at most over the small step in x: a
    step h leaves an error of about h^2 of the third derivative plus the fp32
    rounding of the loss over 2h, below 2e-3 of the sums' size here."""
    B, H, S, D, N = 1, 2, 12, 32, 4
    q, k, qw, kw, cq, ck = (t.to(DEV) for t in _make(B, H, H, S, D, torch.float32, 6))
    q, k = q.clamp(-2, 2) + 0.1, k.clamp(-2, 2) - 0.1
    f = sp.rope_frequencies(D, 100.0, DEV)

    def loss(q, k, qw, kw):
        y, z = sp.striped_qk_norm_rope(q, k, qw, kw, f, N)
        return float((y.double() * cq.double()).sum() + (z.double() * ck.double()).sum())

    got = sp.striped_qk_norm_rope_bwd(q, k, cq, ck, qw, kw, f, N)
    g = torch.Generator().manual_seed(1)
    args = [q, k, qw, kw]
    for i in range(4):
        for _ in range(3):
            u = torch.randn(args[i].shape, generator=g).to(DEV)
            u /= u.norm()
            h = 2e-2
            up = loss(*[a + h * u if j == i else a for j, a in enumerate(args)])
            dn = loss(*[a - h * u if j == i else a for j, a in enumerate(args)])
            want = float((got[i].double() * u.double()).sum())
            assert abs((up - dn) / (2 * h) - want) <= 2e-3 * float(got[i].norm()), (i, (up - dn) / (2 * h), want)


def test_side_stream_and_captured_graph():
    B, H, Hkv, S, D, N = 1, 4, 2, 512, 128, 8
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in _make(B, H, Hkv, S, D, torch.bfloat16, 7))
    f = sp.rope_frequencies(D, 10000.0, DEV)
    want = sp.striped_qk_norm_rope(q, k, qw, kw, f, N)
    grads = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, N)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sp.striped_qk_norm_rope(q, k, qw, kw, f, N, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    a, b, ga, gb = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(dq), torch.zeros_like(dk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sp.striped_qk_norm_rope(a, b, qw, kw, f, N)
        z = sp.striped_qk_norm_rope_bwd(a, b, ga, gb, qw, kw, f, N)
    for t, s in ((a, q), (b, k), (ga, dq), (gb, dk)):
        t.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want + grads, tuple(y) + tuple(z)))


def test_wrapper_refusals():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    w, f = torch.ones(64, device=DEV), sp.rope_frequencies(64, 1e4, DEV)
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope(q, q.clone(), w.double(), w, f)
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope(q, q.float(), w, w, f)
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope(q, q.clone(), w, w, f.float())
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope(q, q.clone(), w, w, f, positions=torch.zeros(1, 8, device=DEV, dtype=torch.int32))
    with pytest.raises(ValueError):
        sp.striped_qk_norm_rope(q, q.clone(), w[:32].clone(), w, f)
    with pytest.raises(ValueError):
        sp.striped_qk_norm_rope(q, q.transpose(1, 2), w, w, f)
    with pytest.raises(ValueError):
        sp.striped_qk_norm_rope(q, q.clone(), w, w, f, positions=torch.zeros(2, 8, device=DEV, dtype=torch.int64))
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope(q.cpu(), q.clone(), w, w, f)
    with pytest.raises(sp.StripedError):
        sp.striped_qk_norm_rope(q, q.clone(), w, w, f, N=3)
    with pytest.raises(sp.StripedError):
        sp.striped_qk_norm_rope(q, q.clone(), w, w, f, k_out=q)


def test_given_positions_ignore_the_placement():
    B, H, Hkv, S, D = 1, 2, 1, 6, 64
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in _make(B, H, Hkv, S, D, torch.bfloat16, 9))
    f = sp.rope_frequencies(D, 1e4, DEV)
    pos = torch.arange(S, device=DEV)[None]
    want = sp.striped_qk_norm_rope(q, k, qw, kw, f) + sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f)
    odd = dict(N=0, layout=9, stripe=77, positions=pos)
    got = sp.striped_qk_norm_rope(q, k, qw, kw, f, **odd) + sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, **odd)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e17, EPS), (1e14, EPS), (1e7, EPS), (1e-14, 0.0), (1e-17, 0.0)])
def test_rows_far_from_one(size, eps, dtype):
    """Rows whose squares fit fp32 and the cube of whose 1 / RMS does not."""
    B, H, Hkv, S, D, N = 1, 3, 1, 40, 128, 4
    q, k, qw, kw, dq, dk = _make(B, H, Hkv, S, D, torch.float32, 10)
    rms = lambda x: x.square().mean(-1, keepdim=True).sqrt()  # noqa: E731
    q, k = ((x / rms(x) * size).to(dtype) for x in (q, k))  # |x| <= sqrt(128) * size at most, 5 * size here
    dq, dk = dq.to(dtype), dk.to(dtype)
    f = sp.rope_frequencies(D, 10000.0, "cpu")
    pos = positions(S, N, sp.STRIPED)[None]
    d = [t.to(DEV) for t in (q, k, qw, kw, f)]
    yq, yk = sp.striped_qk_norm_rope(*d, N, eps=eps)
    gq, gk, gqw, gkw = sp.striped_qk_norm_rope_bwd(d[0], d[1], dq.to(DEV), dk.to(DEV), *d[2:], N, eps=eps)
    for x, w, g, y, dx, dw in ((q, qw, dq, yq, gq, gqw), (k, kw, dk, yk, gk, gkw)):
        r = norm_rope_reference(x, w, pos, f, eps, False, g)
        within(y, r["y"], _rel(dtype) * r["y"].abs() + STEPS * r["y_mag"], "y")
        within(dx, r["dx"], _rel(dtype) * r["dx"].abs() + STEPS * r["dx_mag"], "dx")
        within(dw, r["dw"], (128 * F32 + STEPS) * r["dw_mag"], "dw")


MANY_BLOCKS = [
    # layout, B, H, Hkv, S, D, N, dtype, positions given
    (sp.STRIPED, 1, 20, 3, 2100, 128, 4, torch.bfloat16, False),   # chunks of eight heads and one of four
    (sp.STRIPED, 1, 9, 3, 66000, 64, 8, torch.bfloat16, False),    # chunks of eight heads and one of one
    (sp.ZIGZAG, 1, 20, 3, 65536, 128, 8, torch.bfloat16, False),   # four rounds of blocks
    (sp.STRIPED, 1, 20, 3, 60000, 64, 5, torch.float32, False),    # the same
    (sp.CONTIGUOUS, 2, 17, 16, 2000, 96, 1, torch.float32, False),
    (sp.STRIPED, 700, 17, 3, 4, 128, 1, torch.bfloat16, True),     # rows read one by one
    (sp.STRIPED, 900, 12, 9, 3, 64, 1, torch.float32, True),
]


@pytest.mark.parametrize("layout,B,H,Hkv,S,D,N,dtype,at", MANY_BLOCKS)
def test_gradients_of_many_blocks(layout, B, H, Hkv, S, D, N, dtype, at):
    """Blocks with several heads, a last chunk with fewer, several rounds."""
    g = torch.Generator(device=DEV).manual_seed(11)
    mk = lambda h: torch.randn(B, h, S, D, generator=g, device=DEV).to(dtype)  # noqa: E731
    q, k, dq, dk = mk(H), mk(Hkv), mk(H), mk(Hkv)
    qw, kw = (1 + 0.3 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    f = sp.rope_frequencies(D, 10000.0, DEV)
    pos = torch.randint(0, 100000, (B, S), generator=g, device=DEV) if at else positions(S, N, layout)[None].to(DEV)
    ws = sp.qk_norm_rope_workspace(q, k)
    ws.fill_(255)  # NaN in every share that is not written
    got = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, N, layout, eps=EPS, positions=pos if at else None,
                                      workspace=ws)
    assert sp.check_error() == 0
    for x, w, c, dx, dw in ((q, qw, dq, got[0], got[2]), (k, kw, dk, got[1], got[3])):
        want, mag = torch.zeros(2, D, dtype=torch.float64, device=DEV)
        for h in range(x.shape[1]):
            r = norm_rope_reference(x[:, h:h + 1], w, pos, f, EPS, False, c[:, h:h + 1])
            tol = _rel(dtype) * r["dx"].abs() + STEPS * r["dx_mag"] + 1e-30
            assert float(((dx[:, h:h + 1].double() - r["dx"]).abs() / tol).max()) <= 1.0, h
            want += r["dw"]
            mag += r["dw_mag"]
        # a thread adds at most 112 rows one after another, its block 9 such sums, and the last kernel 43 and 32
        within(dw, want.cpu(), ((196 * F32 + STEPS) * mag + 1e-30).cpu(), "dw")


def test_workspace_of_the_caller():
    B, H, Hkv, S, D = 1, 4, 2, 300, 64
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in _make(B, H, Hkv, S, D, torch.bfloat16, 12))
    f = sp.rope_frequencies(D, 1e4, DEV)
    want = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f)
    ws = sp.qk_norm_rope_workspace(q, k)
    for i in (255, 0):  # contents on entry are ignored
        ws.fill_(i)
        got = sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(sp.StripedError):
        sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, workspace=ws[:-256])
    with pytest.raises(sp.StripedError):
        sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, workspace=ws[1:])
    with pytest.raises(ValueError):
        sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, workspace=ws[::2])
    with pytest.raises(TypeError):
        sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, workspace=ws.cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [sp.STRIPED, sp.CONTIGUOUS, sp.ZIGZAG])
def test_one_stripe_of_a_long_sequence(layout, dtype):
    """The same for stripes long enough to be streamed."""
    B, H, Hkv, N, L, D = 2, 9, 3, 3, 250, 128
    q, k, qw, kw, dq, dk = (t.to(DEV) for t in _make(B, H, Hkv, N * L, D, dtype, 13))
    f = sp.rope_frequencies(64, 10000.0, DEV)
    whole = sp.striped_qk_norm_rope(q, k, qw, kw, f, N, layout)
    whole += sp.striped_qk_norm_rope_bwd(q, k, dq, dk, qw, kw, f, N, layout)[:2]
    for d in range(N):
        c = [t[:, :, d * L:(d + 1) * L].contiguous() for t in (q, k, dq, dk)]
        part = sp.striped_qk_norm_rope(c[0], c[1], qw, kw, f, N, layout, stripe=d)
        part += sp.striped_qk_norm_rope_bwd(*c, qw, kw, f, N, layout, stripe=d)[:2]
        for a, b in zip(whole, part):
            assert torch.equal(a[:, :, d * L:(d + 1) * L], b)
