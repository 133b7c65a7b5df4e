"""Queries that are no numbers, in both kinds of decoding."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions
from tests._prompt_util import kv4_values
from tests.test_gpu_decode import LSE_TOL, _make, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
NAN = float("nan")


def _prompt(kp, vp):
    """The stored prompt on the GPU, and the values it stands for."""
    st = sp.striped_kv4_store(kp.to(DEV), vp.to(DEV))
    return st, kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())


ROWS = [(3, 3, 8, 2, 1), (2, 2, 24, 1, 1), (40, 1, 8, 2, 1), (3, 3, 20, 1, 3)]  # 4, 24, 160 and 60 rows


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Bp,H,Hkv,T", ROWS)
@pytest.mark.parametrize("stored", [False, True])
def test_a_broken_query_shows(stored, B, Bp, H, Hkv, T, D):
    """A query with a NaN gives NaN, not the answer of a query that keeps nothing; the other rows are right."""
    P, C, N = 777, 200, 7
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, T, P, C, D, None, 12)
    lens[-1] = 0
    kd, vd = kp, vp
    if stored:
        st, kd, vd = _prompt(kp, vp)
    o, lse, tol = _reference(q, kd, vd, kt, vt, lens, positions(P, N, sp.STRIPED), 0, 0, D ** -0.5)
    bad = torch.zeros(B, H, T, dtype=torch.bool)
    for i in range(B * H * T):
        bad.view(-1)[i] = i % 5 == 2
    # one channel, or all of them
    q[bad] = torch.where(torch.arange(D) == 5, NAN, q[bad].float()).to(BF)
    q[0, 1, 0], bad[0, 1, 0] = NAN, True
    rest = [t.to(DEV) for t in (kt, vt, lens)]
    if stored:
        go, gl = sp.striped_attn_decode_kv4(q.to(DEV), *st, *rest, N)
    else:
        go, gl = sp.striped_attn_decode(q.to(DEV), kp.to(DEV), vp.to(DEV), *rest, N)
    assert sp.check_error() == 0
    go, gl = go.cpu(), gl.cpu()
    assert bool(torch.isnan(go[bad]).all()) and bool(torch.isnan(gl[bad]).all())
    assert bool(((go[~bad].double() - o[~bad]).abs() <= tol[~bad]).all())
    assert bool(((gl[~bad].double() - lse[~bad]).abs() <= LSE_TOL).all())
