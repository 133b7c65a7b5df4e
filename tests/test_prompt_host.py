"""CPU checks of the operators of a kept prompt: the references against one another and the C entry points' refusals."""
import ctypes

import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions
from tests._prompt_util import evict_reference, kv4_reference, weight_reference

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -6
P = 1 << 20  # 16-byte aligned addresses that no rejected call touches
A = [P * (i + 1) * 16 for i in range(16)]
F = ctypes.c_float


# ------------------------------------------------------------------ the references
def test_stored_values_are_near_and_bf16():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, 64, generator=g).to(torch.bfloat16)
    codes, scale, y = kv4_reference(x)
    s = scale.repeat_interleave(32, -1)
    assert float(codes.abs().max()) == 7 and torch.equal(y, codes * s) and torch.equal(y.to(torch.bfloat16).double(), y)
    # half a step, and 1/32 of 7 steps where the scale was rounded down below the largest value
    assert bool(((x.double() - y).abs() <= s * 0.5 * (1 + 2.0 ** -40)).all())
    assert bool(((scale * 7 / x.double().unflatten(-1, (-1, 32)).abs().amax(-1) - 1).abs() <= 2.0 ** -5).all())


def test_weights_add_up_to_the_queries():
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(1, 4, 30, 8, generator=g), torch.randn(1, 2, 30, 8, generator=g)
    pos = positions(30, 3, sp.STRIPED)
    s = torch.einsum("bhqd,bhkd->bhqk", q.double(), k.double().repeat_interleave(2, 1)) * 0.3
    lse = torch.logsumexp(s.masked_fill(pos[:, None] < pos[None, :], -float("inf")), -1)
    w, _ = weight_reference(q, k, lse, pos, 11, 0.3)
    assert abs(float(w.sum()) - 4 * 19) < 1e-9
    assert float(w[..., pos == 29].max()) <= 2 * 1.0  # the last key is seen by the last query alone


def test_eviction_reference():
    w = torch.tensor([[[3.0, 1.0, 2.0, 2.0, float("nan"), 0.5]]])
    idx, _ = evict_reference(w, torch.arange(6), 3, 0, 0)
    assert idx.tolist() == [[[0, 2, 3]]]
    idx, _ = evict_reference(w, torch.arange(6), 3, 0, 1)
    assert idx.tolist() == [[[0, 2, 5]]]  # of equal ones the lower position
    idx, _ = evict_reference(w, torch.arange(6), 6, 0, 0)
    assert idx.tolist() == [[[0, 1, 2, 3, 4, 5]]]


# ------------------------------------------------------------------ refusals
def _store(lib, k=A[0], v=A[1], kc=A[2], ks=A[3], vc=A[4], vs=A[5], B=2, Hkv=2, S=64, D=64, dtype=0):
    return lib.striped_kv4_store(k, v, kc, ks, vc, vs, B, Hkv, S, D, dtype, None)


N_X = 2 * 2 * 64 * 64 * 2
SIZES = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(S=0), INVALID), (dict(D=0), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(D=48), UNSUPPORTED), (dict(D=288), UNSUPPORTED),
    (dict(B=2 ** 33, Hkv=2 ** 31), UNSUPPORTED), (dict(B=2 ** 20, Hkv=2 ** 10, S=2 ** 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(k=None), INVALID), (dict(vs=None), INVALID), (dict(kc=A[0]), INVALID), (dict(ks=A[1] + N_X - 16), INVALID),
    (dict(vc=A[2]), INVALID), (dict(k=A[0] + 8), ALIGN), (dict(ks=A[3] + 2), ALIGN), (dict(vc=A[4] + 4), ALIGN)])
def test_store_refusals(kw, want):
    assert _store(sp.load(), **kw) == want


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(k=A[2]), INVALID), (dict(k=A[1]), INVALID),
    (dict(v=A[3] - N_X + 16), INVALID), (dict(v=A[1] + 2), ALIGN), (dict(vs=A[5] + 8), ALIGN)])
def test_load_refusals(kw, want):
    a = dict(k=A[0], v=A[1], kc=A[2], ks=A[3], vc=A[4], vs=A[5], B=2, Hkv=2, S=64, D=64, dtype=0) | kw
    assert sp.load().striped_kv4_load(a["kc"], a["ks"], a["vc"], a["vs"], a["k"], a["v"], a["B"], a["Hkv"], a["S"],
                                      a["D"], a["dtype"], None) == want


def _decode(lib, q=A[0], kc=A[1], ks=A[2], vc=A[3], vs=A[4], kt=A[5], vt=A[6], lens=A[7], o=A[8], lse=A[9], ws=A[10],
            n=1 << 40, B=4, Bp=2, H=4, Hkv=2, T=1, P=256, C=16, D=64, N=4, layout=0, dtype=0, scale=0.1):
    return lib.striped_attn_decode_kv4(q, kc, ks, vc, vs, kt, vt, lens, o, lse, ws, n, B, Bp, H, Hkv, T, P, C, D, N,
                                       layout, dtype, F(scale), None)


DECODE_SIZES = [
    (dict(B=0), INVALID), (dict(Bp=3), INVALID), (dict(Bp=0), INVALID), (dict(Hkv=3), INVALID), (dict(T=0), INVALID),
    (dict(P=0), INVALID), (dict(P=-4), INVALID), (dict(C=0), INVALID), (dict(P=255), INVALID), (dict(N=0), INVALID),
    (dict(layout=4), INVALID), (dict(dtype=5), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(D=32), UNSUPPORTED), (dict(N=129, P=1290), UNSUPPORTED), (dict(layout=2, P=264), UNSUPPORTED),
    (dict(C=2 ** 31), UNSUPPORTED), (dict(B=4096, Bp=1), UNSUPPORTED), (dict(B=2048, Bp=2048), UNSUPPORTED),
    (dict(T=2 ** 31), UNSUPPORTED), (dict(B=2 ** 33, Bp=2 ** 33, H=2 ** 31, Hkv=2 ** 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", DECODE_SIZES + [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID),
    (dict(vs=None), INVALID), (dict(kt=None), INVALID), (dict(lens=None), INVALID), (dict(lse=None), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE),
    (dict(ws=A[10] + 16), ALIGN), (dict(q=A[0] + 2), ALIGN), (dict(kc=A[1] + 8), ALIGN), (dict(ks=A[2] + 4), ALIGN),
    (dict(vs=A[4] + 2), ALIGN), (dict(lens=A[7] + 2), ALIGN), (dict(lse=A[9] + 4), ALIGN), (dict(o=A[0]), INVALID),
    (dict(o=A[1]), INVALID), (dict(lse=A[2] + 16), INVALID), (dict(ws=A[4]), INVALID), (dict(ws=A[8]), INVALID),
    (dict(o=A[7] - 16), INVALID), (dict(vt=A[10]), INVALID)])
def test_decode_refusals(kw, want):
    assert _decode(sp.load(), **kw) == want


def test_decode_workspace_size():
    size = sp.load().striped_attn_decode_kv4_workspace_size
    base = dict(B=4, Bp=2, H=4, Hkv=2, T=1, P=256, C=16, D=64, N=4, layout=0, dtype=0)
    assert size(*base.values()) > 0
    for kw, _ in DECODE_SIZES:
        assert size(*(base | kw).values()) == 0


def _weight(lib, q=A[0], k=A[1], lse=A[2], w=A[3], ws=A[4], n=1 << 40, B=1, H=4, Hkv=2, S=256, D=64, N=4, layout=0,
            dtype=0, first=0, scale=0.1):
    return lib.striped_attn_key_weight(q, k, lse, w, ws, n, B, H, Hkv, S, D, N, layout, dtype, first, 0, F(scale), None)


WEIGHT_SIZES = [
    (dict(B=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(S=255), INVALID), (dict(S=0), INVALID),
    (dict(N=0), INVALID), (dict(layout=7), INVALID), (dict(dtype=9), INVALID), (dict(first=256), INVALID),
    (dict(first=-1), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(N=129, S=1290), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED),
    (dict(S=2 ** 30, H=64, Hkv=64), UNSUPPORTED), (dict(B=2 ** 33, H=2 ** 31, Hkv=2 ** 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", WEIGHT_SIZES + [
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID), (dict(scale=-1.0), INVALID),
    (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=A[4] + 64), ALIGN), (dict(k=A[1] + 8), ALIGN),
    (dict(w=A[3] + 4), ALIGN), (dict(lse=A[2] + 4), ALIGN), (dict(w=A[0]), INVALID), (dict(w=A[2]), INVALID),
    (dict(ws=A[1]), INVALID), (dict(ws=A[3]), INVALID)])
def test_key_weight_refusals(kw, want):
    assert _weight(sp.load(), **kw) == want


def test_key_weight_workspace_size():
    size = sp.load().striped_attn_key_weight_workspace_size
    base = dict(B=1, H=4, Hkv=2, S=256, D=64, N=4, layout=0, dtype=0, first=0)
    assert size(*base.values()) > 0
    for kw, _ in WEIGHT_SIZES:
        assert size(*(base | kw).values()) == 0


def _evict(lib, x=(A[0], A[1]), y=(A[2], A[3]), row=(128, 128), weight=A[4], index=A[5], wo=A[6], B=1, Hkv=2, S=64, keep=8,
           sinks=1, recent=1, N=4, layout=0):
    n = len(x)
    return lib.striped_kv_evict((ctypes.c_void_p * n)(*x), (ctypes.c_void_p * n)(*y), (ctypes.c_int64 * n)(*row), n,
                                weight, index, wo, B, Hkv, S, keep, sinks, recent, N, layout, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=(None, A[1])), INVALID), (dict(y=(A[2], None)), INVALID), (dict(weight=None), INVALID),
    (dict(index=None), INVALID), (dict(B=0), INVALID), (dict(S=63), INVALID), (dict(keep=0), INVALID),
    (dict(keep=65), INVALID), (dict(keep=-1), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=5, recent=4), INVALID), (dict(sinks=2 ** 62, recent=2 ** 62), INVALID), (dict(N=0), INVALID),
    (dict(layout=3), INVALID), (dict(layout=2, S=60, N=4, keep=4), INVALID), (dict(row=(0, 128)), INVALID),
    (dict(row=(6, 128)), UNSUPPORTED), (dict(row=(128, 1028)), UNSUPPORTED),
    (dict(x=A[:5], y=A[8:13], row=(4,) * 5), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED),
    (dict(B=2 ** 33, Hkv=2 ** 31), UNSUPPORTED), (dict(B=2 ** 20, Hkv=2 ** 11, S=2 ** 30), UNSUPPORTED),
    (dict(x=(A[0] + 8, A[1])), ALIGN), (dict(y=(A[2], A[3] + 4)), ALIGN), (dict(weight=A[4] + 2), ALIGN),
    (dict(index=A[5] + 2), ALIGN), (dict(wo=A[6] + 1), ALIGN), (dict(y=(A[0], A[3])), INVALID),
    (dict(y=(A[2], A[2])), INVALID), (dict(y=(A[2], A[4])), INVALID), (dict(index=A[4] + 16), INVALID),
    (dict(wo=A[5]), INVALID), (dict(wo=A[3] + 16), INVALID)])
def test_evict_refusals(kw, want):
    assert _evict(sp.load(), **kw) == want
