"""striped_kv4_store, striped_kv4_load and striped_attn_decode_kv4 against the 64-bit definition."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions, within
from tests._prompt_util import kv4_codes, kv4_reference, kv4_values
from tests.test_gpu_decode import CASES as DECODE_CASES
from tests.test_gpu_decode import LSE_TOL, ROW_TILES, _gpu, _make, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _stored(x):
    """codes and scales of striped_kv4_store on the GPU (x as keys and as values)."""
    x = x.to(DEV)
    out = sp.striped_kv4_store(x, x.flip(2).contiguous())
    assert torch.equal(out[0].flip(2), out[2]) and torch.equal(out[1].flip(2), out[3])
    return out[0].cpu(), out[1].cpu()


def _check(x):
    codes, scales = _stored(x)
    c, s, v = kv4_reference(x)
    assert torch.equal(scales.double(), s)
    assert torch.equal(kv4_codes(codes), c)
    assert torch.equal(v.to(BF).double(), v)  # a value is a bf16 number
    k, w = sp.striped_kv4_load(codes.to(DEV), scales.to(DEV), codes.to(DEV), scales.to(DEV))
    assert torch.equal(k.cpu().double(), v) and torch.equal(w, k)


@pytest.mark.parametrize("B,Hkv,S,D", [(1, 1, 1, 32), (2, 3, 5, 64), (64, 8, 1, 128), (1, 2, 1003, 128), (3, 1, 257, 96),
                                       (1, 1, 33, 256), (1, 4, 4097, 64)])
def test_store_and_load(B, Hkv, S, D):
    g = torch.Generator().manual_seed(S)
    x = torch.randn(B, Hkv, S, D, generator=g) * torch.exp(2 * torch.randn(B, Hkv, S, 1, generator=g))
    _check(x.to(BF))


def test_every_quotient():
    """Every significand of the largest value with every significand of another, at every distance where a code
    is not 0: all ties among them."""
    top = torch.arange(128, 256, dtype=torch.float64)
    other = (torch.arange(128, 256, dtype=torch.float64)[None, :] * 2.0 ** -torch.arange(5.0)[:, None]).flatten()
    rows = []
    for t in top:
        o = other[other <= t]
        o = torch.cat([o, o.new_zeros(-o.numel() % 31)]).view(-1, 31)
        sign = torch.where(torch.arange(31) % 2 == 0, 1.0, -1.0)
        rows.append(torch.cat([o.new_full((o.shape[0], 1), float(t)), o * sign], 1))
    x = torch.cat(rows)
    s = kv4_reference(x.view(1, 1, -1, 32))[1]
    q = x / s[0, 0]
    assert int(((q - q.floor()) == 0.5).sum()) > 100  # ties
    for e in (-90, 0, 100):
        _check((x * 2.0 ** e).to(BF).view(1, 1, -1, 32))


def test_wide_and_empty_groups():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 2, 300, 128, generator=g) * 2.0 ** torch.randint(-120, 100, (1, 2, 300, 128), generator=g)
    x[:, :, 5] = 0.0
    x[:, :, 6, 32:64] = 2.0 ** -100
    x[:, :, 7, 32:64] = -(2.0 ** -101)
    x[:, :, 8] = -3e38
    x[:, :, 9, 1:] = 0.0
    _check(x.to(BF))


def test_store_streams_graphs_and_outputs():
    x, y = (torch.randn(2, 2, 700, 128, device=DEV).to(BF) for _ in range(2))
    want = sp.striped_kv4_store(x, y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = sp.striped_kv4_store(x, y, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    bufs = [torch.zeros_like(t) for t in (x, y, *want)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.striped_kv4_store(bufs[0], bufs[1], *bufs[2:])
        back = sp.striped_kv4_load(*bufs[2:])
    bufs[0].copy_(y), bufs[1].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bufs[2:], (*want[2:], *want[:2])))
    assert torch.equal(back[1], sp.striped_kv4_load(*want)[0])


def test_store_refusals():
    x = torch.zeros(1, 2, 8, 64, device=DEV, dtype=BF)
    out = sp.striped_kv4_store(x, x)
    with pytest.raises(TypeError):
        sp.striped_kv4_store(x, x.float())
    with pytest.raises(TypeError):
        sp.striped_kv4_store(x.cpu(), x)
    with pytest.raises(sp.StripedError):
        sp.striped_kv4_store(x.float(), x.float())
    with pytest.raises(ValueError):
        sp.striped_kv4_store(x, x[:, :, :4].contiguous())
    with pytest.raises(ValueError):
        sp.striped_kv4_store(x.transpose(1, 2), x.transpose(1, 2))
    with pytest.raises(ValueError):
        sp.striped_kv4_store(x, x, k_scales=torch.zeros(1, 2, 8, 1, device=DEV, dtype=BF))
    with pytest.raises(sp.StripedError):
        sp.striped_kv4_store(x[..., :40].contiguous(), x[..., :40].contiguous())
    with pytest.raises(TypeError):
        sp.striped_kv4_load(out[0], out[1].float(), out[2], out[3])
    with pytest.raises(sp.StripedError):
        sp.striped_kv4_load(*out, k=x, v=x)


# ------------------------------------------------------------------ decoding
# layout, B, Bp, H, Hkv, T, P, C, D, N, lens: those of striped_attn_decode with a prompt, and further ones
CASES = [c[:10] + (c[12],) for c in DECODE_CASES if c[6] > 0 and c[10] == 0]
CASES += [c[:10] + (None,) for c in ROW_TILES if c[10] == 0]
CASES += [
    (sp.STRIPED, 1, 1, 4, 1, 1, 1, 1, 128, 1, [0]),            # one stored key, nothing behind it
    (sp.STRIPED, 1, 1, 4, 1, 1, 1, 1, 64, 1, [1]),
    (sp.CONTIGUOUS, 2, 2, 8, 8, 1, 129, 5, 128, 3, [5, 0]),
    (sp.STRIPED, 3, 3, 12, 3, 3, 999, 37, 64, 3, [37, 3, 1]),  # a length below T: queries inside the prompt
    (sp.STRIPED, 3, 3, 8, 1, 2, 640, 300, 128, 5, [0, 1, 300]),  # 16 rows, inside the prompt
    (sp.ZIGZAG, 2, 1, 4, 2, 2, 2048, 60, 64, 4, [1, 0]),       # zig-zag rows, inside the prompt
    (sp.CONTIGUOUS, 2, 2, 2, 1, 4, 2, 8, 128, 1, [0, 1]),      # tokens before position 0
    (sp.STRIPED, 2, 2, 17, 1, 1, 700, 260, 128, 7, [260, 31]),  # 17 rows
    (sp.STRIPED, 2, 2, 9, 1, 1, 700, 260, 64, 7, [129, 31]),   # 9 rows
    (sp.STRIPED, 2, 2, 24, 1, 1, 700, 70, 64, 7, [70, 1]),
    (sp.STRIPED, 2, 2, 5, 1, 5, 700, 70, 128, 7, [70, 3]),     # 25 rows, some inside the prompt
    (sp.STRIPED, 2, 2, 32, 1, 1, 700, 300, 128, 7, [290, 31]),
    (sp.STRIPED, 2, 2, 32, 1, 1, 700, 300, 64, 7, [290, 0]),
    (sp.STRIPED, 8, 2, 8, 1, 1, 1400, 40, 64, 7, None),        # 32 rows of four requests
    (sp.STRIPED, 2, 2, 33, 1, 1, 700, 300, 128, 7, [290, 31]),
    (sp.ZIGZAG, 3, 3, 11, 1, 3, 1024, 50, 64, 4, [50, 2, 0]),  # 33 rows, some inside the prompt
    (sp.STRIPED, 2, 1, 9, 1, 4, 1000, 50, 128, 4, [1, 3]),     # 72 rows, all inside the prompt
    (sp.STRIPED, 5, 1, 4, 4, 1, 1300, 150, 128, 13, [0, 1, 150, 128, 127]),
    (sp.STRIPED, 1, 1, 8, 8, 1, 5000, 9, 128, 8, [4]),         # a row a head
    (sp.STRIPED, 1, 1, 8, 2, 1, 70000, 9, 64, 8, [9]),
]


def _prompt(kp, vp):
    """The stored prompt on the GPU, and the values it stands for."""
    st = sp.striped_kv4_store(kp.to(DEV), vp.to(DEV))
    return st, [kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())]


@pytest.mark.parametrize("layout,B,Bp,H,Hkv,T,P,C,D,N,lens", CASES)
def test_decode(layout, B, Bp, H, Hkv, T, P, C, D, N, lens):
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, lens)
    st, (kd, vd) = _prompt(kp, vp)
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, positions(P, N, layout), 0, 0, D ** -0.5)
    behind = (torch.arange(C) >= lens[:, None])[:, None, :, None].expand_as(kt)
    for bad in (float("nan"), float("inf"), -torch.finfo(BF).max):
        kt[behind], vt[behind] = bad, bad
        qg, ktg, vtg, lg = _gpu(q, kt, vt, lens)
        go, gl = sp.striped_attn_decode_kv4(qg, *st, ktg, vtg, lg, N, layout)
        assert sp.check_error() == 0
        within(gl, lse, LSE_TOL, "lse")
        within(go, o, tol, "o")


@pytest.mark.parametrize("D,B,H", [(128, 2, 8), (64, 20, 32), (128, 1, 4), (64, 3, 12), (128, 12, 8), (128, 40, 8)])
def test_long_segments_with_a_growing_maximum(D, B, H):
    Hkv, P, C, N = 4, 40000, 200, 8
    q, kp, vp, kt, vt, lens = _make(B, 1, H, Hkv, 1, P, C, D, None, 7)
    pos = positions(P, N, sp.STRIPED)
    grow = (0.2 + 6.0 * pos.double() / P)[None, None, :, None]
    kp = (kp.double().abs() * q[:1, :Hkv].double().sign() * grow).to(BF)
    st, (kd, vd) = _prompt(kp, vp)
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, pos, 0, 0, D ** -0.5)
    go, gl = sp.striped_attn_decode_kv4(q.to(DEV), *st, *_gpu(kt, vt, lens), N)
    assert sp.check_error() == 0
    within(gl, lse, 4 * LSE_TOL, "lse")  # scores up to a few hundred
    # a score s is off by up to 2^-20 |s| in fp32 sums: its weight by that
    within(go, o, tol + 2.0 ** -11 * vd.abs().max(), "o")


@pytest.mark.parametrize("B,Bp,H,Hkv", [(3, 3, 8, 2), (24, 1, 8, 2)])
def test_scores_far_apart(B, Bp, H, Hkv):
    """Scores of size 1e4: one key has all the weight, and it may stand anywhere."""
    T, P, C, D, N = 1, 1111, 50, 128, 11
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, None, 8)
    q = (q.float() * 100).to(BF)
    kp, kt = (kp.float() * 30).to(BF), (kt.float() * 30).to(BF)
    st, (kd, vd) = _prompt(kp, vp)
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, positions(P, N, sp.STRIPED), 0, 0, D ** -0.5)
    go, gl = sp.striped_attn_decode_kv4(q.to(DEV), *st, *_gpu(kt, vt, lens), N)
    assert sp.check_error() == 0
    # a score is a sum of 128 products of sizes up to 100 * 30 * 16: off by up to 2^-16 of the sum of sizes
    size = float((q.double().abs().sum(-1).max() * kp.double().abs().max()) * D ** -0.5)
    err = 2.0 ** -17 * size
    within(gl, lse, err, "lse")
    assert err < 3  # weights are off by at most this factor
    clear = torch.isfinite(go.cpu().double()).all()
    assert bool(clear)


@pytest.mark.parametrize("B,H", [(5, 8), (40, 8)])
def test_run_to_run_stream_and_graph(B, H):
    Hkv, P, C, D, N = 2, 4096, 300, 128, 8
    q, kp, vp, kt, vt, lens = _make(B, 1, H, Hkv, 1, P, C, D, None, 4)
    st, _ = _prompt(kp, vp)
    args = [q.to(DEV), *st, *_gpu(kt, vt, lens)]
    want = sp.striped_attn_decode_kv4(*args, N)
    again = sp.striped_attn_decode_kv4(*args, N)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sp.striped_attn_decode_kv4(*args, N, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    bufs = [torch.zeros_like(t) for t in args]
    ws = sp.new_decode_kv4_workspace(bufs[0], bufs[1], bufs[5], N)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = sp.striped_attn_decode_kv4(*bufs, N, workspace=ws)
    for t, s in zip(bufs, args):
        t.copy_(s)
    for n in (0, 1, 128, 129, 300):
        bufs[7].fill_(n)
        ws.fill_(0xff)  # whatever it held
        graph.replay()
        o, lse = sp.striped_attn_decode_kv4(*args[:7], torch.full_like(args[7], n), N)
        torch.cuda.synchronize()
        assert torch.equal(go, o) and torch.equal(gl, lse)
    assert sp.check_error() == 0


@pytest.mark.parametrize("B,H,P", [(2, 4, 1024), (40, 8, 1024), (1, 4, 100)])
def test_same_as_decoding_on_the_stored_values(B, H, P):
    Hkv, C, D, N = 2, 40, 64, 4
    q, kp, vp, kt, vt, lens = _make(B, 1, H, Hkv, 1, P, C, D, None, 5)
    st, _ = _prompt(kp, vp)
    k, v = sp.striped_kv4_load(*st)
    rest = _gpu(kt, vt, lens)
    o, lse = sp.striped_attn_decode_kv4(q.to(DEV), *st, *rest, N)
    o2, lse2 = sp.striped_attn_decode(q.to(DEV), k, v, *rest, N)
    assert float((lse - lse2).abs().max()) <= LSE_TOL
    assert float((o.float() - o2.float()).abs().max()) <= 2e-2


def test_lengths_outside_the_tail_are_clamped():
    q, kp, vp, kt, vt, _ = _make(2, 1, 2, 1, 1, 64, 20, 64, [0, 0], 1)
    st, _ = _prompt(kp, vp)
    a = [sp.striped_attn_decode_kv4(q.to(DEV), *st, *_gpu(kt, vt, torch.tensor(n, dtype=torch.int32)), 4)
         for n in ([-5, 1 << 30], [0, 20])]
    assert torch.equal(a[0][0], a[1][0]) and torch.equal(a[0][1], a[1][1])


@pytest.mark.parametrize("B,Bp,H,Hkv,T,P,C,D,N", [(40, 1, 8, 1, 1, 2048, 20, 64, 8), (3, 3, 40, 1, 1, 1000, 300, 128, 8)])
def test_missing_tiles_end_and_leave_the_device_usable(B, Bp, H, Hkv, T, P, C, D, N):
    """Tiles of the tails are never loaded."""
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, [C] * B, 9)
    st, _ = _prompt(kp, vp)
    args = [q.to(DEV), *st, *_gpu(kt, vt, lens), N]
    want = sp.striped_attn_decode_kv4(*args)
    assert sp.check_error() == 0
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 5_000_000)
        sp.striped_attn_decode_kv4(*args)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    got = sp.striped_attn_decode_kv4(*args)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and sp.check_error() == 0


@pytest.mark.parametrize("layout,B,Bp,H,Hkv,T,P,C,D,N", [
    (sp.STRIPED, 1024, 1024, 2, 1, 1, 24, 9, 64, 4), (sp.CONTIGUOUS, 1000, 2, 1, 1, 2, 300, 3, 64, 1)])
def test_the_most_requests_of_a_call(layout, B, Bp, H, Hkv, T, P, C, D, N):
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, None, 15)
    st, (kd, vd) = _prompt(kp, vp)
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, positions(P, N, layout), 0, 0, D ** -0.5)
    behind = (torch.arange(C) >= lens[:, None])[:, None, :, None].expand_as(kt)
    kt[behind], vt[behind] = float("nan"), float("nan")
    go, gl = sp.striped_attn_decode_kv4(q.to(DEV), *st, *_gpu(kt, vt, lens), N, layout)
    assert sp.check_error() == 0
    within(gl, lse, LSE_TOL, "lse")
    within(go, o, tol, "o")


@pytest.fixture
def emptied_cache():
    """The memory of a large test goes back to the device."""
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [32, 2048])
def test_offsets_past_32_bits(emptied_cache, H):
    """More than 2^31 bytes of codes and elements of tails: the last key/value head of the last request is what it is
    alone, and so are its stored rows."""
    B, Hkv, P, C, D, N = 2, 32, 1 << 20, 1 << 19, 128, 8
    g = torch.Generator(device=DEV).manual_seed(6)
    mk = lambda *s: torch.empty(*s, dtype=BF, device=DEV).normal_(generator=g)  # noqa: E731
    kp, vp = mk(2, Hkv, P, D), mk(2, Hkv, P, D)
    st = sp.striped_kv4_store(kp, vp)
    one = sp.striped_kv4_store(kp[1:, -1:].contiguous(), vp[1:, -1:].contiguous())
    assert all(torch.equal(a[1:, -1:], b) for a, b in zip(st, one))
    k, v = sp.striped_kv4_load(*st)
    assert torch.equal(k[1:, -1:], sp.striped_kv4_load(*one)[0])
    del k, v, kp, vp
    q, kt, vt = mk(B, H, 1, D), mk(B, Hkv, C, D), mk(B, Hkv, C, D)
    lens = torch.tensor([5, C], dtype=torch.int32, device=DEV)
    o, lse = sp.striped_attn_decode_kv4(q, *st, kt, vt, lens, N)
    n = H // Hkv
    last = [q[1:, -n:], *one, kt[1:, -1:], vt[1:, -1:], lens[1:]]
    o1, lse1 = sp.striped_attn_decode_kv4(*[t.contiguous() for t in last], N)
    assert float((lse[1:, -n:] - lse1).abs().max()) <= LSE_TOL
    assert float((o[1:, -n:].float() - o1.float()).abs().max()) <= 2.0 ** -7 * float(o1.float().abs().max())
    assert sp.check_error() == 0


def test_wrapper_refusals():
    q, kp, vp, kt, vt, lens = _make(4, 2, 4, 2, 1, 256, 16, 64, None, 6)
    st, _ = _prompt(kp, vp)
    q, kt, vt, lens = _gpu(q, kt, vt, lens)
    f = sp.striped_attn_decode_kv4
    with pytest.raises(TypeError):
        f(q, *st, kt, vt, lens.long(), 4)
    with pytest.raises(TypeError):
        f(q, st[0].to(BF), *st[1:], kt, vt, lens, 4)
    with pytest.raises(TypeError):
        f(q, None, *st[1:], kt, vt, lens, 4)
    with pytest.raises(TypeError):
        f(q, st[0], st[1].half(), *st[2:], kt, vt, lens, 4)
    with pytest.raises(ValueError):
        f(q, st[0], st[1][..., :1].contiguous(), *st[2:], kt, vt, lens, 4)
    with pytest.raises(ValueError):
        f(q, *st[:2], st[2][:, :, :128].contiguous(), st[3], kt, vt, lens, 4)
    with pytest.raises(sp.StripedError):
        f(q, *st, kt, vt, lens, 3)
    with pytest.raises(sp.StripedError):
        f(q, *st, kt, vt, lens, 4, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(sp.StripedError):
        f(q, *st, kt, vt, lens, 4, out=q)
    with pytest.raises(ValueError):
        f(q[..., :32].contiguous(), *st, kt, vt, lens, 4)
