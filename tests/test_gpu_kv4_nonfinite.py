"""Rows with a NaN or an infinity in 4 bits: nothing of it is lost by storing."""
import math

import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._prompt_util import kv4_reference
from tests.test_gpu_decode import _make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("bad", [(NAN,), (-NAN,), (INF,), (-INF,), (INF, NAN), (NAN, -INF)])
def test_storing_keeps_what_is_no_number(bad, D):
    """A group with a NaN or an infinity reads back without a finite value; the others are what they are without it."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(1, 2, 70, D, generator=g).to(BF)
    hit = torch.zeros(1, 2, 70, D // 32, dtype=torch.bool)
    for r in range(70):  # every channel of a group, several groups
        c = (7 * r + 3) % D
        for i, b in enumerate(bad):
            x[0, r % 2, r, c // 32 * 32 + (c + 9 * i) % 32] = b
        hit[0, r % 2, r, c // 32] = True
    x = x.to(DEV)
    kc, ks, vc, vs = sp.striped_kv4_store(x, x)
    assert torch.equal(kc, vc) and torch.equal(ks.view(torch.int16), vs.view(torch.int16))
    k, v = (t.cpu().unflatten(-1, (-1, 32)) for t in sp.striped_kv4_load(kc, ks, vc, vs))
    assert not bool(torch.isfinite(k[hit]).any()) and not bool(torch.isfinite(v[hit]).any())
    has_nan = any(math.isnan(b) for b in bad)
    assert bool(torch.isnan(ks.cpu()[hit]).all() if has_nan else torch.isinf(ks.cpu()[hit]).all())
    _, s, y = kv4_reference(torch.where(hit[..., None].expand_as(k).flatten(-2), 0.0, x.cpu().double()).to(BF))
    assert torch.equal(ks.cpu()[~hit].double(), s[~hit])
    assert torch.equal(k[~hit].double(), y.unflatten(-1, (-1, 32))[~hit])


def test_a_broken_row_shows_in_what_is_decoded_on_it():
    """Storage to decoding: a NaN in a key or a value of one head reaches that head's queries and no others."""
    B, H, Hkv, P, C, D, N = 3, 8, 2, 640, 30, 64, 5
    q, kp, vp, kt, vt, lens = _make(B, 1, H, Hkv, 1, P, C, D, None, 13)
    for which in (kp, vp):
        x = [t.clone() for t in (kp, vp)]
        x[0 if which is kp else 1][0, 1, 333, 40] = NAN
        st = sp.striped_kv4_store(x[0].to(DEV), x[1].to(DEV))
        o, lse = sp.striped_attn_decode_kv4(q.to(DEV), *st, kt.to(DEV), vt.to(DEV), lens.to(DEV), N)
        assert bool(torch.isfinite(o[:, :4]).all()) and bool(torch.isfinite(lse[:, :4]).all())
        if which is kp:
            assert bool(torch.isnan(o[:, 4:]).all())
        else:
            assert bool(torch.isnan(o[:, 4:, :, 32:]).all()) and bool(torch.isfinite(o[:, 4:, :, :32]).all())
    assert sp.check_error() == 0
