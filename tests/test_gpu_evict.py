"""striped_kv_evict and striped_kv4_evict against a sort on the CPU, and the whole life of a kept prompt."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions, within
from tests._prompt_util import evict_reference, kv4_reference, kv4_values, weight_reference
from tests.test_gpu_decode import LSE_TOL, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
INF, NAN = float("inf"), float("nan")


def _rows(B, Hkv, S, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, Hkv, S, D, generator=g).to(BF) for _ in range(2)]


def _check(k, v, weight, keep, sinks, recent, N, layout):
    pos = positions(weight.shape[2], N, layout)
    index, row = evict_reference(weight, pos, keep, sinks, recent)
    ko, vo, io, wo = sp.striped_kv_evict(k.to(DEV), v.to(DEV), weight.to(DEV), keep, sinks, recent, N, layout)
    assert torch.equal(io.cpu(), index)
    at = row[index.long()]
    take = at[..., None].expand(-1, -1, -1, k.shape[-1])
    assert torch.equal(ko.cpu(), k.gather(2, take)) and torch.equal(vo.cpu(), v.gather(2, take))
    same = weight.gather(2, at)
    assert torch.equal(wo.cpu().view(torch.int32), same.view(torch.int32))


@pytest.mark.parametrize("layout,B,Hkv,S,D,N,keep,sinks,recent", [
    (sp.STRIPED, 1, 1, 1, 64, 1, 1, 0, 0),
    (sp.STRIPED, 1, 1, 1, 64, 1, 1, 1, 0),
    (sp.STRIPED, 2, 3, 40, 64, 8, 1, 0, 0),
    (sp.STRIPED, 2, 3, 40, 64, 8, 40, 0, 0),      # all stay
    (sp.STRIPED, 2, 3, 40, 64, 8, 20, 10, 10),    # nothing left to choose
    (sp.STRIPED, 4, 2, 1500, 64, 4, 201, 4, 32),
    (sp.STRIPED, 1, 2, 8193, 128, 3, 1000, 0, 1),
    (sp.STRIPED, 1, 1, 8192, 128, 8192, 100, 3, 0),  # a stripe a row
    (sp.STRIPED, 1, 1, 6000, 128, 2000, 777, 3, 5),
    (sp.CONTIGUOUS, 3, 1, 5000, 128, 5, 4999, 1, 1),
    (sp.ZIGZAG, 1, 2, 600, 64, 3, 77, 0, 9),         # chunks that are no tiles
    (sp.ZIGZAG, 1, 2, 32768, 64, 4, 1200, 5, 60),
    (sp.STRIPED, 1, 2, 65536, 64, 16, 8192, 4, 64),
    (sp.CONTIGUOUS, 1, 2, 66000, 64, 1, 5, 0, 0),
])
def test_rows_that_stay(layout, B, Hkv, S, D, N, keep, sinks, recent):
    k, v = _rows(B, Hkv, S, D)
    g = torch.Generator().manual_seed(1)
    w = torch.exp(2 * torch.randn(B, Hkv, S, generator=g))
    _check(k, v, w, keep, sinks, recent, N, layout)
    _check(k, v, (w * 2).round(), keep, sinks, recent, N, layout)  # many equal ones
    _check(k, v, torch.zeros_like(w), keep, sinks, recent, N, layout)


def test_weights_of_every_kind():
    B, Hkv, S, D, N = 1, 3, 4000, 64, 8
    k, v = _rows(B, Hkv, S, D, 2)
    g = torch.Generator().manual_seed(3)
    w = torch.randn(B, Hkv, S, generator=g) * 10.0 ** torch.randint(-44, 38, (B, Hkv, S), generator=g)
    kind = torch.randint(0, 12, (B, Hkv, S), generator=g)
    for i, x in enumerate((NAN, -NAN, INF, -INF, 0.0, -0.0, 1e-45, -1e-45, torch.finfo(torch.float32).max)):
        w[kind == i] = x
    for keep in (1, 300, 333, 1000, 2000, 3300, 3700, 3999):
        _check(k, v, w, keep, min(2, keep), min(keep - 1, 30) // 2, N, sp.STRIPED)
    _check(k, v, torch.full_like(w, NAN), 17, 2, 3, N, sp.STRIPED)
    _check(k, v, torch.full_like(w, -INF), 17, 2, 3, N, sp.STRIPED)


@pytest.mark.parametrize("S,N", [(600000, 8), (393217 + 7, 1)])
def test_parts_beyond_shared_memory(S, N):
    Hkv, keep = 2, 3001
    g = torch.Generator().manual_seed(4)
    w = torch.exp(torch.randn(1, Hkv, S, generator=g)).to(BF).float()  # ties
    x = torch.arange(2 * S, dtype=torch.int32).view(1, Hkv, S, 1)
    pos = positions(S, N, sp.STRIPED)
    byp = w[:, :, torch.argsort(pos)]
    want = torch.sort(byp, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    o = sp.striped_kv_evict(*[t.to(DEV) for t in (x, x, w)], keep, 0, 0, N)
    assert torch.equal(o[2].cpu().long(), want)
    assert torch.equal(o[0].cpu()[..., 0], torch.gather(x[..., 0], 2, torch.argsort(pos)[want]))


@pytest.mark.parametrize("row", [4, 8, 12, 16, 20, 48, 512, 1008, 1024])
def test_row_sizes(row):
    """Rows of any number of words."""
    B, Hkv, S, keep = 2, 2, 300, 77
    g = torch.Generator().manual_seed(row)
    x = torch.randint(0, 256, (B, Hkv, S, row), generator=g, dtype=torch.uint8)
    y = torch.randint(0, 256, (B, Hkv, S, 4), generator=g, dtype=torch.uint8)
    w = torch.rand(B, Hkv, S, generator=g)
    index, _ = evict_reference(w, torch.arange(S), keep, 0, 0)
    o = sp.striped_kv_evict(*[t.to(DEV) for t in (x, y, w)], keep)
    for t, got in zip((x, y), o):
        assert torch.equal(got.cpu(), t.gather(2, index.long()[..., None].expand(-1, -1, -1, t.shape[-1])))


@pytest.mark.parametrize("D", [64, 128])
def test_stored_rows_stay_as_they_are(D):
    """Eviction of stored rows is the storage of the evicted ones."""
    k, v = (t.to(DEV) for t in _rows(2, 3, 1100, D, 5))
    w = torch.rand(2, 3, 1100, device=DEV)
    k1, v1, i1, w1 = sp.striped_kv_evict(k, v, w, 333, 4, 20, 4)
    st = sp.striped_kv4_store(k, v)
    *rows, i2, w2 = sp.striped_kv4_evict(*st, w, 333, 4, 20, 4)
    assert torch.equal(i1, i2) and torch.equal(w1, w2)
    assert all(torch.equal(a, b) for a, b in zip(rows, sp.striped_kv4_store(k1, v1)))


def test_stream_graph_and_outputs():
    k, v = (t.to(DEV) for t in _rows(1, 4, 20000, 128, 6))
    ws = [torch.rand(1, 4, 20000, device=DEV) for _ in range(2)]
    want = [sp.striped_kv_evict(k, v, w, 2500, 4, 60, 8) for w in ws]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sp.striped_kv_evict(k, v, ws[0], 2500, 4, 60, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    buf, outs = ws[0].clone(), [torch.zeros_like(t) for t in want[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.striped_kv_evict(k, v, buf, 2500, 4, 60, 8, sp.STRIPED, *outs)
    for w, x in zip(ws, want):
        buf.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, x))


@pytest.fixture
def emptied_cache():
    yield
    torch.cuda.empty_cache()


def test_offsets_past_32_bits(emptied_cache):
    Hkv, S, D, keep = 32, 1 << 20, 128, 5000
    g = torch.Generator(device=DEV).manual_seed(6)
    k = torch.empty(1, Hkv, S, D, dtype=BF, device=DEV).normal_(generator=g)
    w = torch.rand(1, Hkv, S, generator=g, device=DEV)
    o = sp.striped_kv_evict(k, k, w, keep, 4, 100, 8)
    one = sp.striped_kv_evict(*[t[:, -1:].contiguous() for t in (k, k, w)], keep, 4, 100, 8)
    assert all(torch.equal(a[:, -1:], b) for a, b in zip(o, one))


def test_wrapper_refusals():
    k, v = (t.to(DEV) for t in _rows(1, 2, 64, 64))
    w = torch.rand(1, 2, 64, device=DEV)
    f = sp.striped_kv_evict
    for keep, sinks, recent in ((0, 0, 0), (65, 0, 0), (10, 6, 5), (10, -1, 0), (10, 0, -1), (-3, 0, 0)):
        with pytest.raises(sp.StripedError):
            f(k, v, w, keep, sinks, recent)
    with pytest.raises(sp.StripedError):
        f(k, v, w, 8, N=5)
    with pytest.raises(sp.StripedError):
        f(k, v, w, 8, layout=9)
    with pytest.raises(sp.StripedError):
        f(k, v, w, 64, k_out=k)
    with pytest.raises(TypeError):
        f(k, v, w.double(), 8)
    with pytest.raises(TypeError):
        f(k, v, w.cpu(), 8)
    with pytest.raises(ValueError):
        f(k, v[:, :1].contiguous(), w, 8)
    with pytest.raises(ValueError):
        f(k, v, w, 8, index=torch.zeros(1, 2, 9, device=DEV, dtype=torch.int32))
    with pytest.raises(ValueError):
        f(k.transpose(1, 2).contiguous().transpose(1, 2), v, w, 8)


@pytest.mark.parametrize("stored", [False, True])
def test_a_kept_prompt(stored):
    """Prefill, the weights of the last queries, eviction, storage, decoding: each step against its formula on what
    the step before gave."""
    B, H, Hkv, P, C, D, N, keep, T = 2, 8, 2, 1024, 20, 64, 4, 200, 2
    g = torch.Generator().manual_seed(9)
    mk = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)  # noqa: E731
    q, k, v = mk(B, H, P, D), mk(B, Hkv, P, D), mk(B, Hkv, P, D)
    q, k, v = (sp.striped_permute(t, N) for t in (q, k, v))
    pos = positions(P, N, sp.STRIPED)
    o, lse = sp.striped_attn_fwd(q, k, v, N)
    w = sp.striped_attn_key_weight(q, k, lse, N, first=P - 32)
    ref, tol = weight_reference(q.cpu(), k.cpu(), lse.cpu(), pos, P - 32, D ** -0.5)
    within(w, ref, tol, "weight")
    index, row = evict_reference(w.cpu(), pos, keep, 4, 16)
    qn, kt, vt = mk(B, H, T, D), mk(B, Hkv, C, D), mk(B, Hkv, C, D)
    lens = torch.tensor([C, 7], dtype=torch.int32, device=DEV)
    if stored:
        *st, io, _ = sp.striped_kv4_evict(*sp.striped_kv4_store(k, v), w, keep, 4, 16, N)
        kd, vd = kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())
        want = [kv4_reference(t.cpu())[2] for t in (k, v)]
    else:
        kk, vk, io, _ = sp.striped_kv_evict(k, v, w, keep, 4, 16, N)
        st = sp.striped_kv4_store(kk, vk)
        kd, vd = kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())
        want = [kv4_reference(t.cpu())[2] for t in (k, v)]
    assert torch.equal(io.cpu(), index)
    take = row[index.long()][..., None].expand(-1, -1, -1, D)
    assert torch.equal(kd, want[0].gather(2, take)) and torch.equal(vd, want[1].gather(2, take))
    go, gl = sp.striped_attn_decode_kv4(qn, *st, kt, vt, lens)
    ro, rl, rt = _reference(qn.cpu(), kd, vd, kt.cpu(), vt.cpu(), lens.cpu(), torch.arange(keep), 0, 0, D ** -0.5)
    within(gl, rl, LSE_TOL, "lse")
    within(go, ro, rt, "o")
    assert sp.check_error() == 0
