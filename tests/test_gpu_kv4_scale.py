"""Decoding on 4-bit rows with the largest scales that a call takes."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions, within
from tests._prompt_util import kv4_values
from tests.test_gpu_decode import LSE_TOL, _make, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _prompt(kp, vp):
    """The stored prompt on the GPU, and the values it stands for."""
    st = sp.striped_kv4_store(kp.to(DEV), vp.to(DEV))
    return st, kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Bp,H,Hkv", [(2, 2, 4, 2), (2, 2, 24, 1), (20, 1, 8, 2)])  # 2, 24 and 80 rows
@pytest.mark.parametrize("scale", [1e38, 3e36])
def test_the_largest_scales(scale, B, Bp, H, Hkv, D):
    """Whole keys times 2^-66 and queries of one channel 2^-60: a score is a whole number times 2^-126, without a rounding
    until it is scaled."""
    P, C, N = 700, 40, 7
    g = torch.Generator().manual_seed(D + B)
    _, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, 1, P, C, D, None, 3)
    for k in (kp, kt):
        k.copy_(torch.randint(-7, 8, k.shape, generator=g) * 2.0 ** -66)
        k[..., ::32] = 7 * 2.0 ** -66
    q = torch.zeros(B, H, 1, D, dtype=BF)
    q.scatter_(-1, torch.randint(0, D, (B, H, 1, 1), generator=g), 2.0 ** -60)
    q[:, 1] = 0.0
    st, kd, vd = _prompt(kp, vp)
    assert torch.equal(kd, kp.double())
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, positions(P, N, sp.STRIPED), 0, 0, scale)
    go, gl = sp.striped_attn_decode_kv4(q.to(DEV), *st, kt.to(DEV), vt.to(DEV), lens.to(DEV), N, sp.STRIPED, scale)
    assert sp.check_error() == 0
    within(gl, lse, LSE_TOL, "lse")
    within(go, o, tol, "o")
