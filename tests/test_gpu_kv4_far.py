"""Decoding on 4-bit rows whose scores are far apart: which values the result is made of."""
import math

import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import BF as HALF_STEP
from tests._prompt_util import kv4_values
from tests.test_gpu_decode import _make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _prompt(kp, vp):
    """The stored prompt on the GPU, and the values it stands for."""
    st = sp.striped_kv4_store(kp.to(DEV), vp.to(DEV))
    return st, kv4_values(st[0].cpu(), st[1].cpu()), kv4_values(st[2].cpu(), st[3].cpu())


@pytest.mark.parametrize("B,Bp,H,Hkv,D", [(3, 3, 8, 2, 128), (2, 2, 24, 1, 64), (24, 1, 8, 2, 128), (24, 1, 8, 2, 64)])
def test_far_apart_scores_take_the_right_rows(B, Bp, H, Hkv, D):
    """Scores of size 1e4: where one key is ahead by more than scores can be off, o is its value; elsewhere o lies
    among the values of the keys that may be ahead."""
    P, C, N = 1111, 50, 11
    q, kp, vp, kt, vt, lens = _make(B, Bp, H, Hkv, 1, P, C, D, None, 8)
    q = (q.float() * 100).to(BF)
    kp, kt = (kp.float() * 30).to(BF), (kt.float() * 30).to(BF)
    st, kd, vd = _prompt(kp, vp)
    go, _ = sp.striped_attn_decode_kv4(q.to(DEV), *st, kt.to(DEV), vt.to(DEV), lens.to(DEV), N)
    assert sp.check_error() == 0
    go, clear = go.cpu().double(), 0
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            hkv = h // (H // Hkv)
            k = torch.cat([kd[b // (B // Bp), hkv], kt[b, hkv, :n].double()])
            v = torch.cat([vd[b // (B // Bp), hkv], vt[b, hkv, :n].double()])
            x = q[b, h, 0].double()
            s = k @ x * D ** -0.5
            # an fp32 sum of D products is off by up to D 2^-24 of the sum of their sizes
            err = float((k.abs() @ x.abs()).max()) * D ** -0.5 * D * 2.0 ** -24
            # all keys further behind than this have less than e^-20 of the weight together
            near = s >= s.max() - (2 * err + math.log(s.numel()) + 20)
            lo, hi = v[near].min(0).values, v[near].max(0).values
            # o and P are rounded to bf16; e^-20 of the other values
            tol = HALF_STEP * 2.02 * v[near].abs().max(0).values + 2 * math.exp(-20) * v.abs().max()
            assert bool(((go[b, h, 0] >= lo - tol) & (go[b, h, 0] <= hi + tol)).all()), (b, h)
            clear += int(near.sum()) == 1
    assert 4 * clear >= 3 * B * H
