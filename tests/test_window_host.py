"""CPU checks of the window and norm-and-rotation operators: the position
tiles against the oracle's placement, the references' gradients against
differences, and the C entry points' refusals."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
import sequence_parallelism_striped_gb300 as sp
from tests._local_util import norm_rope_reference, positions, window_reference

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -6


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("window") / "window_harness")
    cmd = [nvcc, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "sequence_parallelism_striped_gb300", "csrc"),
           "-gencode", "arch=compute_103a,code=sm_103a",
           os.path.join(ROOT, "tests", "window_harness.cu"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


@pytest.mark.parametrize("layout,S,N,W", [
    (sp.STRIPED, 256, 4, 64), (sp.STRIPED, 1000, 8, 100), (sp.STRIPED, 903, 3, 200), (sp.STRIPED, 1300, 13, 1),
    (sp.STRIPED, 1040, 65, 300), (sp.STRIPED, 1280, 128, 5), (sp.STRIPED, 1, 1, 1), (sp.STRIPED, 640, 5, 640),
    (sp.CONTIGUOUS, 777, 7, 128), (sp.CONTIGUOUS, 130, 1, 129), (sp.ZIGZAG, 2048, 4, 300), (sp.ZIGZAG, 1536, 3, 257),
    (sp.ZIGZAG, 512, 1, 2)])
def test_position_tiles(harness, layout, S, N, W):
    out = subprocess.run([harness, str(layout), str(S), str(N), str(W)], capture_output=True, text=True, check=True)
    lines = [[x[0]] + [int(v) for v in x.split()[1:]] for x in out.stdout.splitlines()]
    pos_of_row = np.asarray(oracle.layout_positions(S, N, layout))
    rows = [x[1:] for x in lines if x[0] == "T"]
    real = [(t, r, row, pos) for t, r, has, row, pos in rows if has]
    # every row once, holding the position that the placement puts there
    assert sorted(x[2] for x in real) == list(range(S))
    assert all(pos_of_row[row] == pos for _, _, row, pos in real)
    tiles = {}
    for t, r, row, pos in real:
        tiles.setdefault(t, []).append((r, row, pos))
    P = max(len(v) for v in tiles.values())
    for t, v in tiles.items():  # consecutive positions, tile after tile
        assert sorted(x[2] for x in v) == list(range(t * P, min(S, t * P + P)))
    # the copy box brings row r of the tile to place r: stripes inside rows
    for _, t, row0, stripe0, R, ns, L in [x for x in lines if x[0] == "B"]:
        assert R * ns <= 128 and R <= 256 and ns <= 256
        got = {i * ns + s: (stripe0 + s) * L + row0 + i for s in range(ns) for i in range(R) if row0 + i < L}
        for r, row, _ in tiles.get(t, []):
            assert got[r] == row
    # window spans: exactly the tiles that hold a kept pair
    for _, t, lo, hi in [x for x in lines if x[0] == "W"]:
        q = [x[2] for x in tiles[t]]
        first = max(0, t * P - W + 1)  # of the tile's first position
        assert lo == first // P
        last_q = min(S - 1, t * P + P - 1 + W - 1)
        assert hi == min(max(tiles), last_q // P if t * P + P <= S else max(tiles)) and min(q) == t * P


def test_kept_bits(harness):
    out = subprocess.run([harness, "1", "128", "1", "1"], capture_output=True, text=True, check=True).stdout
    rows = [[int(v) for v in x.split()[1:]] for x in out.splitlines() if x[0] == "K"]
    assert len(rows) > 1000
    for base, hi, lo, sk, bits in rows:
        want = sum(1 << c for c in range(32) if base + c <= hi and (base + c >= lo or base + c < sk))
        assert bits == want


def test_more_stripes_than_a_tile(harness):
    assert subprocess.run([harness, str(sp.STRIPED), "1290", "129", "4"]).returncode == 3


@pytest.mark.parametrize("W,ns", [(5, 2), (1, 0), (3, 9)])
def test_window_reference_gradient_against_differences(W, ns):
    """The formula of the gradient against central differences in 64 bits."""
    B, H, Hkv, S, D, N = 1, 2, 1, 24, 8, 4
    g = torch.Generator().manual_seed(0)
    mk = lambda h: torch.randn(B, h, S, D, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = mk(H), mk(Hkv), mk(Hkv), mk(H)
    pos = positions(S, N, sp.STRIPED)
    r = window_reference(q, k, v, pos, W, ns, 0.4, do)
    f = lambda *a: float((window_reference(*a, pos, W, ns, 0.4)["o"] * do).sum())  # noqa: E731
    for i, n in enumerate(("dq", "dk", "dv")):
        u = torch.randn(r[n].shape, generator=g, dtype=torch.float64)
        args = [q, k, v]
        up = f(*[a + 1e-5 * u if j == i else a for j, a in enumerate(args)])
        dn = f(*[a - 1e-5 * u if j == i else a for j, a in enumerate(args)])
        assert abs((up - dn) / 2e-5 - float((r[n] * u).sum())) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_reference_gradient_against_differences(interleaved):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(1, 2, 6, 16, generator=g, dtype=torch.float64)
    dy = torch.randn(1, 2, 6, 16, generator=g, dtype=torch.float64)
    w = torch.randn(16, generator=g, dtype=torch.float64)
    f = sp.rope_frequencies(8, 100.0, "cpu")
    pos = positions(6, 3, sp.STRIPED)[None]
    r = norm_rope_reference(x, w, pos, f, 1e-6, interleaved, dy)
    loss = lambda x, w: float((norm_rope_reference(x, w, pos, f, 1e-6, interleaved)["y"] * dy).sum())  # noqa: E731
    u = torch.randn(x.shape, generator=g, dtype=torch.float64)
    assert abs((loss(x + 1e-5 * u, w) - loss(x - 1e-5 * u, w)) / 2e-5 - float((r["dx"] * u).sum())) < 1e-8
    u = torch.randn(16, generator=g, dtype=torch.float64)
    assert abs((loss(x, w + 1e-5 * u) - loss(x, w - 1e-5 * u)) / 2e-5 - float((r["dw"] * u).sum())) < 1e-8


# ------------------------------------------------------------------ refusals
P = 1 << 20  # 16-byte aligned addresses that no rejected call touches
A = [P * (i + 1) * 16 for i in range(16)]


def _window(lib, q=A[0], B=1, H=4, Hkv=2, S=256, D=64, N=4, layout=0, dtype=0, W=10, ns=0, o=A[3]):
    return lib.striped_attn_window_fwd(q, A[1], A[2], o, A[4], B, H, Hkv, S, D, N, layout, dtype, W, ns,
                                       ctypes.c_float(0.1), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(B=0), INVALID), (dict(Hkv=3), INVALID),
    (dict(Hkv=0), INVALID), (dict(S=255), INVALID), (dict(S=0), INVALID), (dict(N=0), INVALID),
    (dict(layout=7), INVALID), (dict(dtype=9), INVALID), (dict(W=0), INVALID), (dict(W=-5), INVALID),
    (dict(ns=-1), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(ns=1025), UNSUPPORTED),
    (dict(N=129, S=1290), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED),
    (dict(q=A[0] + 8), ALIGN), (dict(o=A[3] + 2), ALIGN)])
def test_window_refusals(kw, want):
    assert _window(sp.load(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dO=None), INVALID), (dict(ws=None), WORKSPACE), (dict(n=-1), WORKSPACE), (dict(ws=A[10] + 64), ALIGN),
    (dict(dv=A[9] + 4), ALIGN), (dict(ns=2000), UNSUPPORTED), (dict(W=0), INVALID)])
def test_window_backward_refusals(kw, want):
    lib = sp.load()
    a = dict(dO=A[5], dv=A[9], ws=A[10], n=0, W=10, ns=4) | kw
    need = lib.striped_attn_window_workspace_size(1, 4, 2, 256, 64, 4, 0, 0, 10, 4)
    assert need > 0
    got = lib.striped_attn_window_bwd(A[0], A[1], A[2], A[3], A[4], a["dO"], A[7], A[8], a["dv"], a["ws"],
                                      need + a["n"], 1, 4, 2, 256, 64, 4, 0, 0, a["W"], a["ns"], ctypes.c_float(0.1),
                                      None)
    assert got == want


def test_window_workspace_size():
    size = sp.load().striped_attn_window_workspace_size
    assert size(1, 4, 2, 256, 64, 4, 0, 0, 0, 4) == 0 and size(1, 4, 2, 256, 64, 4, 0, 1, 8, 4) == 0
    # fp32 dQ and two statistics a row; two tiles, no query lies above both windows
    assert size(1, 4, 2, 256, 64, 4, 0, 0, 256, 4) == 4 * 256 * (64 * 4 + 8)
    assert size(1, 4, 2, 4096, 64, 4, 0, 0, 10, 4) > 4 * 4096 * (64 * 4 + 8)


def _rope(lib, q=A[0], k=A[1], yq=A[2], yk=A[3], w=A[4], f=A[5], pos=None, B=1, H=4, Hkv=2, S=64, D=64, rot=64, N=4,
          layout=0, stripe=-1, eps=1e-6, dtype=0):
    return lib.striped_qk_norm_rope(q, k, yq, yk, w, w, f, pos, B, H, Hkv, S, D, rot, 0, N, layout, stripe,
                                    ctypes.c_float(eps), dtype, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(yk=None), INVALID), (dict(w=None), INVALID), (dict(f=None), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(S=0), INVALID), (dict(S=63), INVALID),
    (dict(N=0), INVALID), (dict(layout=3), INVALID), (dict(dtype=2), INVALID), (dict(rot=-16), INVALID),
    (dict(rot=80), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(stripe=4), INVALID),
    (dict(stripe=-2), INVALID), (dict(layout=2, S=60), INVALID), (dict(layout=2, S=63, stripe=1), INVALID),
    (dict(yq=A[1]), INVALID), (dict(yq=A[0] + 16), INVALID), (dict(yk=A[2] + 32), INVALID), (dict(yk=A[0]), INVALID),
    (dict(D=40, rot=16), UNSUPPORTED), (dict(D=272, rot=16), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(q=A[0] + 2), ALIGN), (dict(yq=A[2] + 8), ALIGN), (dict(w=A[4] + 2), ALIGN), (dict(f=A[5] + 4), ALIGN),
    (dict(pos=A[6] + 4), ALIGN)])
def test_norm_rope_refusals(kw, want):
    assert _rope(sp.load(), **kw) == want


def test_norm_rope_backward_refusals():
    lib = sp.load()
    need = lib.striped_qk_norm_rope_workspace_size(1, 4, 2, 64, 64, 0)
    assert need > 0 and lib.striped_qk_norm_rope_workspace_size(1, 4, 2, 64, 40, 0) == 0

    def call(ws=A[12], n=need, g=A[2], dw=A[8]):
        return lib.striped_qk_norm_rope_bwd(A[0], A[1], g, A[3], A[6], A[7], dw, A[9], A[10], A[11], A[13], None, ws,
                                            n, 1, 4, 2, 64, 64, 64, 0, 4, 0, -1, ctypes.c_float(1e-6), 0, None)

    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(g=None) == INVALID and call(dw=None) == INVALID and call(ws=A[12] + 4) == ALIGN


def _decode(lib, q=A[0], kp=A[1], vp=A[2], kt=A[3], vt=A[4], lens=A[5], o=A[6], lse=A[7], ws=A[8], n=1 << 40, B=4, Bp=2,
            H=4, Hkv=2, T=1, P=256, C=16, D=64, N=4, layout=0, dtype=0, W=0, ns=0):
    return lib.striped_attn_decode(q, kp, vp, kt, vt, lens, o, lse, ws, n, B, Bp, H, Hkv, T, P, C, D, N, layout,
                                   dtype, W, ns, ctypes.c_float(0.1), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(vt=None), INVALID),
    (dict(lens=None), INVALID), (dict(lse=None), INVALID), (dict(B=0), INVALID), (dict(Bp=3), INVALID),
    (dict(Bp=0), INVALID), (dict(Hkv=3), INVALID), (dict(T=0), INVALID), (dict(P=-4), INVALID), (dict(C=0), INVALID),
    (dict(P=255), INVALID), (dict(N=0), INVALID), (dict(layout=4), INVALID), (dict(dtype=5), INVALID),
    (dict(W=-1), INVALID), (dict(ns=-1), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(N=129, P=1290), UNSUPPORTED), (dict(layout=2, P=264), UNSUPPORTED), (dict(C=2 ** 31), UNSUPPORTED),
    (dict(B=4096, Bp=1), UNSUPPORTED), (dict(B=2048, Bp=2048), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE), (dict(ws=A[8] + 16), ALIGN), (dict(q=A[0] + 2), ALIGN),
    (dict(vp=A[2] + 8), ALIGN), (dict(lens=A[5] + 2), ALIGN), (dict(lse=A[7] + 4), ALIGN)])
def test_decode_refusals(kw, want):
    assert _decode(sp.load(), **kw) == want


def test_decode_workspace_size():
    size = sp.load().striped_attn_decode_workspace_size
    assert size(4, 2, 4, 2, 1, 256, 16, 64, 4, 0, 0, 0, 0) > 0
    assert size(4, 3, 4, 2, 1, 256, 16, 64, 4, 0, 0, 0, 0) == 0
    assert size(4, 2, 4, 2, 1, 256, 16, 64, 4, 0, 1, 0, 0) == 0
    assert size(4, 1, 4, 2, 1, 0, 16, 64, 4, 0, 0, 0, 0) > 0  # no prompt: N and layout are not looked at


# ------------------------------------------------------------------ scales, overlapping buffers, ignored arguments
BAD_SCALES = [0.0, -0.1, float("nan"), float("inf"), 1e-40, 2e38]


@pytest.mark.parametrize("scale", BAD_SCALES)
def test_scale_refusals(scale):
    lib, s = sp.load(), ctypes.c_float(scale)
    assert lib.striped_attn_window_fwd(*A[:5], 1, 4, 2, 256, 64, 4, 0, 0, 10, 0, s, None) == INVALID
    assert lib.striped_attn_window_bwd(*A[:10], 1 << 40, 1, 4, 2, 256, 64, 4, 0, 0, 10, 0, s, None) == INVALID
    assert lib.striped_attn_decode(*A[:9], 1 << 40, 4, 2, 4, 2, 1, 256, 16, 64, 4, 0, 0, 0, 0, s, None) == INVALID


# results and the workspace over every other tensor, at the last byte of it or of themselves
Q, KV, LSE = 4 * 256 * 64 * 2, 2 * 256 * 64 * 2, 4 * 256 * 4  # bytes at B 1, H 4, Hkv 2, S 256, D 64


@pytest.mark.parametrize("res,at", [
    (3, A[0]), (3, A[1]), (3, A[2] + KV - 16), (3, A[0] - Q + 16), (3, A[4] - Q + 16), (4, A[0] + 32),
    (4, A[1] + KV - 16), (4, A[2] - LSE + 16)])
def test_window_overlap_refusals(res, at):
    a = A[:5]
    a[res] = at
    assert sp.load().striped_attn_window_fwd(*a, 1, 4, 2, 256, 64, 4, 0, 0, 10, 0, ctypes.c_float(0.1),
                                             None) == INVALID


@pytest.mark.parametrize("res,at", [
    (6, A[0]), (6, A[5]), (6, A[7]), (7, A[1]), (7, A[8] + KV - 16), (8, A[2]), (8, A[4]), (8, A[3] - KV + 16),
    (9, A[0]), (9, A[6]), (9, A[8] + KV - 256)])
def test_window_backward_overlap_refusals(res, at):
    a = A[:10]
    a[res] = at
    assert sp.load().striped_attn_window_bwd(*a, 1 << 40, 1, 4, 2, 256, 64, 4, 0, 0, 10, 4, ctypes.c_float(0.1),
                                             None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(o=A[0]), dict(o=A[1]), dict(o=A[5] - 16), dict(lse=A[3]), dict(lse=A[6] + 16), dict(ws=A[4]), dict(ws=A[7]),
    dict(vt=A[8])])
def test_decode_overlap_refusals(kw):
    assert _decode(sp.load(), **kw) == INVALID


def test_norm_rope_overlap_refusals():
    lib = sp.load()
    assert _rope(lib, yq=A[4]) == INVALID and _rope(lib, yk=A[5]) == INVALID and _rope(lib, pos=A[2]) == INVALID
    need = lib.striped_qk_norm_rope_workspace_size(1, 4, 2, 64, 64, 0)

    def call(dq=A[6], dw=A[8], ws=A[12]):
        return lib.striped_qk_norm_rope_bwd(A[0], A[1], A[2], A[3], dq, A[7], dw, A[9], A[10], A[11], A[13], None, ws,
                                            need, 1, 4, 2, 64, 64, 64, 0, 4, 0, -1, ctypes.c_float(1e-6), 0, None)

    assert call(dq=A[1]) == INVALID and call(dq=A[3]) == INVALID and call(dq=A[9]) == INVALID
    assert call(dw=A[9] + 252) == INVALID and call(dw=A[10]) == INVALID and call(dw=A[0]) == INVALID
    assert call(ws=A[0]) == INVALID and call(ws=A[9]) == INVALID and call(ws=A[13]) == INVALID


def test_sizes_that_no_gpu_holds():
    """Byte counts past 64 bits, and heads past the grid."""
    lib = sp.load()
    assert _window(lib, B=2 ** 20, H=2 ** 11, Hkv=2 ** 11, S=2 ** 30) == UNSUPPORTED
    assert lib.striped_attn_window_workspace_size(2 ** 20, 2 ** 11, 2 ** 11, 2 ** 30, 64, 4, 0, 0, 10, 4) == 0
    assert _decode(lib, B=1, Bp=1, H=2 ** 30, Hkv=2 ** 30, P=2 ** 30) == UNSUPPORTED
    assert _decode(lib, P=2 ** 30, C=2 ** 30 - 256, T=1) == UNSUPPORTED
    assert _rope(lib, H=65537) == UNSUPPORTED and _rope(lib, Hkv=65537) == UNSUPPORTED
    assert lib.striped_qk_norm_rope_workspace_size(1, 65537, 2, 64, 64, 0) == 0
    assert _rope(lib, B=2 ** 15, H=2 ** 16, S=2 ** 31) == UNSUPPORTED


@pytest.mark.parametrize("B,H", [(2 ** 62, 4), (2 ** 61, 8), (4, 2 ** 62), (2 ** 33, 2 ** 31), (2 ** 40, 2 ** 24)])
def test_products_of_sizes_that_wrap(B, H):
    """B * H is 0 (or small) modulo 2^64: refused, not taken for an empty call."""
    lib = sp.load()
    assert (B * H) % 2 ** 64 == 0
    assert _window(lib, B=B, H=H, Hkv=H) == UNSUPPORTED
    assert lib.striped_attn_window_workspace_size(B, H, H, 256, 64, 4, 0, 0, 10, 4) == 0
    assert lib.striped_attn_window_bwd(*A[:10], 1 << 40, B, H, H, 256, 64, 4, 0, 0, 10, 4, ctypes.c_float(0.1),
                                       None) == UNSUPPORTED
    assert _rope(lib, B=B, H=H, Hkv=H) == UNSUPPORTED and _rope(lib, B=B, H=1, Hkv=H) == UNSUPPORTED
    assert lib.striped_qk_norm_rope_workspace_size(B, H, H, 64, 64, 0) == 0
    assert lib.striped_qk_norm_rope_workspace_size(B, 1, H, 64, 64, 0) == 0
    assert _decode(lib, B=B, Bp=B, H=H, Hkv=H) == UNSUPPORTED
    assert lib.striped_attn_fwd(*A[:5], B, H, 64, 128, 4, 0, 0, ctypes.c_float(0.1), None, None) == UNSUPPORTED
    assert lib.striped_permute(A[0], A[1], B, H, 64, 128, 4, 0, None) == UNSUPPORTED


def test_window_backward_takes_what_the_forward_takes():
    """Many heads with sinks: the sink tiles' shares do not bound the batch."""
    size = sp.load().striped_attn_window_workspace_size
    one = size(1, 1, 1, 384, 64, 4, 0, 0, 64, 4)
    # per head: three tiles of fp32 dQ and statistics, and two fp32 shares of one sink tile's dK and dV
    assert one == 384 * (64 * 4 + 8) + 2 * 2 * 128 * 64 * 4
    for B, H in ((8192, 8), (65536, 1), (200000, 4)):
        assert size(B, H, H, 384, 64, 4, 0, 0, 64, 4) == B * H * one
