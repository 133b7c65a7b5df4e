"""The calls that csrc/binding.cpp takes in one step: the same results as the wrappers' own way, the same refusals, and
nothing that it should leave to them."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def binding():
    sp.load()
    if sp._fast is None:
        pytest.skip("the binding was not built for this torch")
    yield
    assert sp._fast is not None


def _slow(f, *a, **kw):
    fast, sp._fast = sp._fast, None
    try:
        return f(*a, **kw)
    finally:
        sp._fast = fast


def _calls(D=64, H=4, Hkv=2, P=512, N=4, B=3):
    g = torch.Generator(device=DEV).manual_seed(D)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    q, k, v = mk(1, H, P, D), mk(1, Hkv, P, D), mk(1, Hkv, P, D)
    _, lse = sp.striped_attn_fwd(q, k, v, N)
    st = _slow(sp.striped_kv4_store, k, v)
    w = torch.rand(1, Hkv, P, generator=g, device=DEV)
    tail = mk(B, Hkv, 30, D), mk(B, Hkv, 30, D), torch.tensor([30, 0, 7][:B], dtype=torch.int32, device=DEV)
    return [
        (sp.striped_kv4_store, (k, v), {}),
        (sp.striped_kv4_load, st, {}),
        (sp.striped_attn_decode_kv4, (mk(B, H, 2, D), *st, *tail, N), {}),
        (sp.striped_attn_decode_kv4, (mk(B, H, 1, D), *st, *tail), dict(N=N, layout=sp.STRIPED, scale=0.3)),
        (sp.striped_attn_key_weight, (q, k, lse, N), {}),
        (sp.striped_attn_key_weight, (q, k, lse, N, sp.STRIPED, 100, 0.2), {}),
        (sp.striped_kv_evict, (k, v, w, 100), {}),
        (sp.striped_kv_evict, (k, v, w, 100, 4, 20, N), {}),
        (sp.striped_kv4_evict, (*st, w, 100, 4, 20, N), {}),
    ]


def _equal(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    return len(a) == len(b) and all(x.dtype == y.dtype and x.shape == y.shape and x.device == y.device
                                    and torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("D", [64, 128])
def test_the_same_results(D, monkeypatch):
    calls = _calls(D)
    want = [_slow(f, *a, **kw) for f, a, kw in calls]
    # from here on the wrappers' own way would fail
    monkeypatch.setattr(sp, "_need", None)
    got = [f(*a, **kw) for f, a, kw in calls]
    assert all(_equal(a, b) for a, b in zip(want, got))
    assert all(not t.requires_grad for r in got for t in (r if isinstance(r, tuple) else (r,)))


def test_what_it_leaves_to_the_wrappers():
    """Other types, shapes, strides, devices and numbers: None, and the wrapper's answer."""
    f = sp._fast
    k = torch.zeros(1, 2, 16, 64, device=DEV, dtype=BF)
    for a, b in ((k, k.float()), (k.cpu(), k), (k, k[:, :, :8].contiguous()), (k.transpose(1, 2), k.transpose(1, 2)),
                 (k[0], k[0]), (k, None), (k.half(), k.half()), (k[..., :40].contiguous(), k[..., :40].contiguous())):
        assert f.kv4_store(a, b) is None
    assert f.kv4_store(k) is None and f.kv4_store(k, k, k) is None
    assert f.kv_evict(torch.zeros(1, 2, 16, device=DEV), 0, 0, 0, 1, 0, k, k) is None
    assert f.kv_evict(torch.zeros(1, 2, 16, device=DEV), 17, 0, 0, 1, 0, k, k) is None
    assert f.kv_evict(torch.zeros(1, 2, 16, device=DEV), 4.0, 0, 0, 1, 0, k, k) is None
    assert f.kv_evict(torch.zeros(1, 2, 16, device=DEV), 4, 1 << 70, 0, 1, 0, k, k) is None
    lse = torch.zeros(1, 2, 16, device=DEV)
    assert f.key_weight(k, k, lse, 3, 0, 0, None) is None      # 16 rows on 3 stripes
    assert f.key_weight(k, k, lse, 4, 0, 16, None) is None
    assert f.key_weight(k, k, lse, 4, 0, 0, 0.0) is None
    assert f.key_weight(k, k, lse, 1 << 40, 0, 0, None) is None
    with pytest.raises(sp.StripedError):
        sp.striped_attn_key_weight(k, k, lse, 3)
    with pytest.raises(TypeError):
        sp.striped_kv4_store(k, k.float())


def test_streams_and_graphs():
    calls = _calls(128)
    want = [_slow(f, *a, **kw) for f, a, kw in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # the current stream is the call's
        got = [f(*a, **kw) for f, a, kw in calls]
    side.synchronize()
    assert all(_equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [f(*a, **kw) for f, a, kw in calls]
    for r in got:
        for t in r if isinstance(r, tuple) else (r,):
            t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(_equal(a, b) for a, b in zip(want, got))
    assert sp.check_error() == 0


def test_parameters_are_taken_as_tensors():
    k = torch.nn.Parameter(torch.randn(1, 2, 16, 64, device=DEV).to(BF))
    a, b = sp.striped_kv4_store(k, k), _slow(sp.striped_kv4_store, k.detach(), k.detach())
    assert _equal(a, b)
