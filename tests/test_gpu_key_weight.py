"""striped_attn_key_weight against the 64-bit formula."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import attention, keep_mask, positions, within
from tests._prompt_util import weight_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _make(layout, B, H, Hkv, S, D, N, seed=0):
    """q, k, the lse of causal attention (64 bits, rounded once) and the rows' positions."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(B, h, S, D, generator=g).to(BF) for h in (H, Hkv))
    pos = positions(S, N, layout)
    keep = keep_mask(pos, pos, 0, 0)
    lse = torch.zeros(B, H, S)
    for b in range(B):
        for h in range(H):
            kd = k[b, h // (H // Hkv)].double()
            lse[b, h] = attention(q[b, h].double(), kd, kd, keep, D ** -0.5)[1].float()
    return q, k, lse, pos


CASES = [
    # layout, B, H, Hkv, S, D, N, first
    (sp.STRIPED, 1, 1, 1, 1, 64, 1, 0),
    (sp.STRIPED, 1, 2, 1, 2, 128, 2, 1),
    (sp.STRIPED, 1, 4, 2, 256, 128, 4, 0),
    (sp.STRIPED, 2, 6, 2, 1000, 64, 8, 0),
    (sp.STRIPED, 2, 6, 2, 1000, 64, 8, 801),
    (sp.STRIPED, 1, 2, 2, 903, 128, 3, 0),        # 126 positions a tile
    (sp.STRIPED, 1, 3, 1, 903, 64, 7, 500),
    (sp.STRIPED, 1, 2, 1, 1040, 128, 65, 300),    # 65 positions a tile
    (sp.STRIPED, 1, 2, 2, 1280, 64, 128, 1279),   # one query
    (sp.STRIPED, 1, 8, 1, 2048, 128, 8, 2048 - 64),
    (sp.STRIPED, 3, 5, 5, 385, 128, 1, 129),
    (sp.CONTIGUOUS, 1, 4, 1, 777, 128, 7, 0),
    (sp.CONTIGUOUS, 1, 4, 4, 640, 64, 5, 130),
    (sp.ZIGZAG, 1, 4, 2, 2048, 128, 4, 0),
    (sp.ZIGZAG, 1, 3, 1, 1536, 64, 3, 1000),
    (sp.STRIPED, 200, 2, 1, 24, 64, 4, 3),        # many short prompts
    (sp.STRIPED, 1, 2, 1, 128, 128, 8, 32),       # whole columns left out of the keys' own tile
    (sp.STRIPED, 1, 2, 1, 4096, 64, 8, 0),
]


@pytest.mark.parametrize("layout,B,H,Hkv,S,D,N,first", CASES)
def test_weight(layout, B, H, Hkv, S, D, N, first):
    q, k, lse, pos = _make(layout, B, H, Hkv, S, D, N)
    w, tol = weight_reference(q, k, lse, pos, first, D ** -0.5)
    lse[:, :, pos < first] = float("nan")  # never read
    args = [t.to(DEV) for t in (q, k, lse)]
    got = sp.striped_attn_key_weight(*args, N, layout, first)
    assert sp.check_error() == 0
    within(got, w, tol, "weight")
    # every counted query hands out a weight of 1 a head
    assert abs(float(got.double().sum()) - B * H * (S - first)) <= 1e-4 * B * H * (S - first)
    # added to what is there
    again = sp.striped_attn_key_weight(*args, N, layout, first, accumulate=True, weight=got.clone())
    within(again, w + got.cpu().double(), tol + 2.0 ** -24 * 2 * w.abs(), "accumulated")
    assert torch.equal(got, sp.striped_attn_key_weight(*args, N, layout, first))  # the same from run to run


def test_two_halves_are_the_whole():
    layout, B, H, Hkv, S, D, N = sp.STRIPED, 1, 4, 2, 1600, 128, 8
    q, k, lse, pos = _make(layout, B, H, Hkv, S, D, N, 1)
    w, tol = weight_reference(q, k, lse, pos, 0, D ** -0.5)
    q, k, lse = (t.to(DEV) for t in (q, k, lse))
    got = sp.striped_attn_key_weight(q, k, lse, N, layout, 700)
    # the queries before 700 alone: the others' lse says that they do not count
    head = lse.clone()
    head[:, :, (pos >= 700).to(DEV)] = float("inf")
    sp.striped_attn_key_weight(q, k, head, N, layout, 0, accumulate=True, weight=got)
    within(got, w, tol + 2.0 ** -22 * w, "sum")


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_queries_that_do_not_count(bad):
    layout, B, H, Hkv, S, D, N = sp.STRIPED, 2, 4, 2, 600, 64, 4
    q, k, lse, pos = _make(layout, B, H, Hkv, S, D, N, 2)
    lse[0, 1, ::3] = bad
    lse[1, :, 200:] = bad
    w, tol = weight_reference(q, k, lse, pos, 0, D ** -0.5)
    got = sp.striped_attn_key_weight(*[t.to(DEV) for t in (q, k, lse)], N, layout)
    within(got, w, tol, "weight")


def test_a_broken_key_spoils_its_own_weight_alone():
    layout, B, H, Hkv, S, D, N = sp.STRIPED, 1, 2, 1, 520, 128, 8
    q, k, lse, pos = _make(layout, B, H, Hkv, S, D, N, 3)
    q, k, lse = (t.to(DEV) for t in (q, k, lse))
    want = sp.striped_attn_key_weight(q, k, lse, N, layout)
    k[0, 0, 77] = float("nan")
    got = sp.striped_attn_key_weight(q, k, lse, N, layout)
    assert bool(torch.isnan(got[0, 0, 77]))
    rest = torch.arange(S, device=DEV) != 77
    assert torch.equal(got[..., rest], want[..., rest])


def test_stream_graph_and_wide_scores():
    layout, B, H, Hkv, S, D, N = sp.STRIPED, 1, 8, 2, 1024, 128, 8
    sets = []
    for seed, size in ((4, 1.0), (5, 6.0)):
        q, k, lse, pos = _make(layout, B, H, Hkv, S, D, N, seed)
        q = (q.float() * size).to(BF)
        kd, keep = k.double(), keep_mask(pos, pos, 0, 0)
        for h in range(H):
            lse[0, h] = attention(q[0, h].double(), kd[0, h // 4], kd[0, h // 4], keep, D ** -0.5)[1].float()
        w, tol = weight_reference(q, k, lse, pos, 0, D ** -0.5)
        sets.append(([t.to(DEV) for t in (q, k, lse)], w, tol))
    bufs = [t.clone() for t in sets[0][0]]
    ws = sp.new_key_weight_workspace(bufs[0], bufs[1], N, layout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sp.striped_attn_key_weight(*bufs, N, layout, workspace=ws)
    for args, w, tol in sets:
        for b, a in zip(bufs, args):
            b.copy_(a)
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        within(got, w, tol, "replayed")
        side = torch.cuda.Stream()
        other = sp.striped_attn_key_weight(*args, N, layout, stream=side)
        side.synchronize()
        assert torch.equal(other, got)
    assert sp.check_error() == 0


def test_a_missing_tile_times_out():
    q, k, lse, _ = _make(sp.STRIPED, 1, 4, 2, 1024, 128, 8, 6)
    args = [t.to(DEV) for t in (q, k, lse)]
    want = sp.striped_attn_key_weight(*args, 8)
    try:
        sp.test_inject(sp.FAULT_FWD_SKIP_KV, 5_000_000)
        sp.striped_attn_key_weight(*args, 8)
        assert sp.check_error() == -5
    finally:
        sp.test_inject(sp.FAULT_NONE, 0)
    assert torch.equal(want, sp.striped_attn_key_weight(*args, 8)) and sp.check_error() == 0


@pytest.fixture
def emptied_cache():
    yield
    torch.cuda.empty_cache()


def test_offsets_past_32_bits(emptied_cache):
    """More than 2^31 elements of queries and keys: the last head's weights are what they are alone."""
    H, Hkv, S, D, N = 64, 32, 1 << 19, 128, 8
    g = torch.Generator(device=DEV).manual_seed(6)
    mk = lambda h: torch.empty(1, h, S, D, dtype=BF, device=DEV).normal_(generator=g)  # noqa: E731
    q, k = mk(H), mk(Hkv)
    lse = torch.full((1, H, S), 13.0, device=DEV)
    first = S - 100
    got = sp.striped_attn_key_weight(q, k, lse, N, sp.STRIPED, first)
    one = sp.striped_attn_key_weight(q[:, -2:].contiguous(), k[:, -1:].contiguous(), lse[:, -2:].contiguous(), N,
                                     sp.STRIPED, first)
    # cut into other shares: added in another order
    assert float(((got[:, -1:] - one).abs() / one).max()) <= 1e-5
    assert sp.check_error() == 0


def test_wrapper_refusals():
    q, k, lse, _ = _make(sp.STRIPED, 1, 4, 2, 64, 64, 4)
    q, k, lse = (t.to(DEV) for t in (q, k, lse))
    f = sp.striped_attn_key_weight
    with pytest.raises(TypeError):
        f(q, k, lse.double(), 4)
    with pytest.raises(TypeError):
        f(q, k.float(), lse, 4)
    with pytest.raises(TypeError):
        f(q.cpu(), k, lse, 4)
    with pytest.raises(ValueError):
        f(q, k, lse[:, :2].contiguous(), 4)
    with pytest.raises(ValueError):
        f(q, k, lse, 4, accumulate=True)
    with pytest.raises(ValueError):
        f(q, k, lse, 4, weight=torch.zeros(1, 4, 64, device=DEV))
    for kw in (dict(first=64), dict(first=-1), dict(layout=7), dict(scale=0.0)):
        with pytest.raises(sp.StripedError):
            f(q, k, lse, 4, **kw)
    with pytest.raises(sp.StripedError):
        f(q, k, lse, 3)
    with pytest.raises(sp.StripedError):
        f(q.float(), k.float(), lse, 4)
