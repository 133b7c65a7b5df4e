"""The operators of a kept prompt side by side: several streams at once, captured graphs replayed together, outputs and
streams given by the caller."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _set(seed, B, H, Hkv, P, D, N):
    """Everything that a kept prompt's calls take, and what they give one after another."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    q, k, v = mk(1, H, P, D), mk(1, Hkv, P, D), mk(1, Hkv, P, D)
    _, lse = sp.striped_attn_fwd(q, k, v, N)
    qn, kt, vt = mk(B, H, 1, D), mk(B, Hkv, 60, D), mk(B, Hkv, 60, D)
    lens = torch.randint(1, 61, (B,), generator=g, device=DEV).to(torch.int32)
    return dict(q=q, k=k, v=v, lse=lse, qn=qn, kt=kt, vt=vt, lens=lens, N=N, keep=P // 3)


def _run(s, stream=None):
    N = s["N"]
    w = sp.striped_attn_key_weight(s["q"], s["k"], s["lse"], N, first=100, stream=stream)
    st = sp.striped_kv4_store(s["k"], s["v"], stream=stream)
    *kept, index, weight = sp.striped_kv4_evict(*st, w, s["keep"], 4, 20, N, stream=stream)
    back = sp.striped_kv4_load(*kept, stream=stream)
    o, lse = sp.striped_attn_decode_kv4(s["qn"], *kept, s["kt"], s["vt"], s["lens"], stream=stream)
    out = [w, *st, *kept, index, weight, *back, o, lse]
    for t in out:
        if stream is not None:
            t.record_stream(stream)
    return out


SETS = [(1, 3, 8, 2, 2048, 128, 4), (2, 40, 8, 2, 1024, 64, 8), (3, 5, 4, 4, 4096, 128, 1), (4, 20, 16, 2, 1024, 128, 2)]


def test_streams_at_once():
    sets = [_set(*a) for a in SETS]
    want = [_run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [_run(s, t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert sp.check_error() == 0


def test_graphs_replayed_side_by_side():
    sets = [_set(*a) for a in SETS]
    want = [_run(s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_run(s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert sp.check_error() == 0


def test_neighbours_of_the_results_stay():
    """Results in the middle of larger buffers: nothing around them is written."""
    s = _set(5, 3, 8, 2, 1001 * 4, 64, 4)
    want = _run(s)
    pads = []

    def inner(t):
        n = t.numel() * t.element_size()
        buf = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device=DEV)
        pads.append((buf, n))
        return buf[256:256 + n].view(t.dtype).view(t.shape)

    w = sp.striped_attn_key_weight(s["q"], s["k"], s["lse"], 4, first=100, weight=inner(want[0]))
    st = sp.striped_kv4_store(s["k"], s["v"], *[inner(t) for t in want[1:5]])
    kept = sp.striped_kv4_evict(*st, w, s["keep"], 4, 20, 4, sp.STRIPED, *[inner(t) for t in want[5:11]])
    back = sp.striped_kv4_load(*kept[:4], *[inner(t) for t in want[11:13]])
    o = sp.striped_attn_decode_kv4(s["qn"], *kept[:4], s["kt"], s["vt"], s["lens"], out=inner(want[13]),
                                   lse_out=inner(want[14]))
    got = [w, *st, *kept, *back, *o]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for buf, n in pads:
        assert bool((buf[:256] == 0x5a).all()) and bool((buf[256 + n:] == 0x5a).all())


def test_a_stream_of_another_kind_is_refused():
    k = torch.zeros(1, 1, 8, 64, device=DEV, dtype=BF)
    with pytest.raises((TypeError, ValueError, AttributeError)):
        sp.striped_kv4_store(k, k, stream="side")
