"""Eviction at the ends of its range: more lines than a grid has rows, parts that shared memory does not hold."""
import pytest
import torch

import sequence_parallelism_striped_gb300 as sp
from tests._local_util import positions

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _want(weight, pos, keep, sinks, recent):
    """(kept positions, kept rows): ends first, then by weight, the lower position of equal ones."""
    S = weight.shape[-1]
    row = torch.argsort(pos)
    rank = weight[..., row].double()
    rank[..., :sinks] = float("inf")
    rank[..., S - recent:] = float("inf")
    index = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    return index, row[index]


@pytest.mark.parametrize("layout,N,S,keep", [(sp.STRIPED, 1, 3, 2), (sp.STRIPED, 3, 3, 2), (sp.ZIGZAG, 2, 4, 3)])
def test_more_lines_than_a_grid_has_rows(layout, N, S, keep):
    B, Hkv = 35001, 2
    g = torch.Generator().manual_seed(0)
    w = torch.randint(0, 4, (B, Hkv, S), generator=g).float()
    x = torch.randint(0, 1 << 30, (B, Hkv, S, 4), generator=g, dtype=torch.int32)  # rows of 16 bytes
    y = torch.randint(0, 1 << 30, (B, Hkv, S, 1), generator=g, dtype=torch.int32)  # of 4
    index, row = _want(w, positions(S, N, layout), keep, 1, 0)
    xo, yo, io, wo = sp.striped_kv_evict(*[t.to(DEV) for t in (x, y, w)], keep, 1, 0, N, layout)
    assert torch.equal(io.cpu().long(), index)
    assert torch.equal(wo.cpu(), w.gather(2, row))
    assert torch.equal(xo.cpu(), x.gather(2, row[..., None].expand(-1, -1, -1, 4)))
    assert torch.equal(yo.cpu(), y.gather(2, row[..., None]))


@pytest.mark.parametrize("layout,N,S", [(sp.ZIGZAG, 3, 600000), (sp.STRIPED, 8, 600000), (sp.CONTIGUOUS, 4, 400000)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (5, 70), (70000, 3000)])
def test_parts_beyond_shared_memory_with_ends(layout, N, S, sinks, recent):
    Hkv, keep = 2, 80001
    g = torch.Generator().manual_seed(4)
    w = torch.exp(torch.randn(1, Hkv, S, generator=g)).to(torch.bfloat16).float()  # ties
    x = torch.arange(Hkv * S, dtype=torch.int32).view(1, Hkv, S, 1)
    index, row = _want(w, positions(S, N, layout), keep, sinks, recent)
    o = sp.striped_kv_evict(*[t.to(DEV) for t in (x, x, w)], keep, sinks, recent, N, layout)
    assert torch.equal(o[2].cpu().long(), index)
    assert torch.equal(o[0].cpu()[..., 0], x[..., 0].gather(2, row)) and torch.equal(o[3].cpu(), w.gather(2, row))
