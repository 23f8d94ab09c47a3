"""Host-side layouts and refusals of the router by scores, the microscaled
formats, their product and the RMSNorm: every call below returns before any
CUDA call."""
import ctypes

import pytest

import bit_expert_gemv_b200 as G
from oracle import mx_oracle as M

P = 0x100000   # an aligned address that is never read


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 127), (2050, 1001), (65536, 4096), (1000, 130)])
def test_layouts_match_oracle(rows, cols):
    for mx4, fn in ((True, G.gale_mx4_layout), (False, G.gale_mx8_layout)):
        L, want = fn(rows, cols), M.layout(rows, cols, mx4)
        assert {k: getattr(L, k) for k in want} == want and L.q_offset == 0
        assert (L.rows, L.cols) == (rows, cols)


def test_layout_refusals():
    lib, out = G.lib(), G.gale_mx_layout_t()
    for fn in (lib.gale_mx4_layout, lib.gale_mx8_layout):
        assert fn(1, 1, None) == G.GALE_ERR_ARG
        for r, c in ((0, 1), (1, 0), (-1, 8), ((1 << 24) + 1, 1), (1, (1 << 20) + 1), (1 << 24, 1 << 20)):
            assert fn(r, c, ctypes.byref(out)) == G.GALE_ERR_ARG
    assert G.gale_mx_gemm_workspace_size(0, 128, 1) == 0
    assert G.gale_mx_gemm_workspace_size(128, 128, 0) == 0
    assert G.gale_mx_gemm_workspace_size(128, 128, 1) >= 256


def test_quantize_refusals():
    lib = G.lib()
    for q in (lib.gale_mx4_quantize, lib.gale_mx8_quantize):
        assert q(None, G.GALE_F32, 128, 4, 128, P, None) == G.GALE_ERR_ARG
        assert q(P, 9, 128, 4, 128, P, None) == G.GALE_ERR_ARG
        assert q(P, G.GALE_F32, 127, 4, 128, P, None) == G.GALE_ERR_ARG         # ld < cols
        assert q(P, G.GALE_F32, 128, 4, 128, P + 16, None) == G.GALE_ERR_ALIGN
        assert q(P + 2, G.GALE_F32, 128, 4, 128, P, None) == G.GALE_ERR_ALIGN
    assert lib.gale_mx8_quantize(None, G.GALE_BF16, 128, 0, 128, None, None) == G.GALE_OK
    assert lib.gale_mx4_unpack(P, 4, 128, None, G.GALE_F32, 128, None) == G.GALE_ERR_ARG
    assert lib.gale_mx4_unpack(P, 4, 128, P, G.GALE_F32, 100, None) == G.GALE_ERR_ARG
    assert lib.gale_mx4_unpack(P, 4, 128, P + 1, G.GALE_BF16, 128, None) == G.GALE_ERR_ALIGN


def test_gemm_refusals():
    g = G.lib().gale_mx_gemm
    n = G.gale_mx_gemm_workspace_size(64, 128, 4)
    assert g(P, 64, 128, P, 0, None, G.GALE_F32, 64, None, 0, None) == G.GALE_OK
    assert g(None, 64, 128, P, 4, P, G.GALE_F32, 64, P, n, None) == G.GALE_ERR_ARG
    assert g(P, 64, 128, P, -1, P, G.GALE_F32, 64, P, n, None) == G.GALE_ERR_ARG
    assert g(P, 64, 128, P, 4, P, 7, 64, P, n, None) == G.GALE_ERR_ARG
    assert g(P, 64, 128, P, 4, P, G.GALE_F32, 63, P, n, None) == G.GALE_ERR_ARG      # ldy < rows
    assert g(P, 64, 128, P, 4, P, G.GALE_F32, 64, P, n - 1, None) == G.GALE_ERR_WORKSPACE
    assert g(P, 64, 128, P, 4, P, G.GALE_F32, 64, None, n, None) == G.GALE_ERR_WORKSPACE
    assert g(P, 64, 128, P, 4, P, G.GALE_F32, 64, P + 16, n, None) == G.GALE_ERR_ALIGN
    assert g(P + 128, 64, 128, P, 4, P, G.GALE_F32, 64, P, n, None) == G.GALE_ERR_ALIGN
    assert g(P, 64, 128, P, 4, P + 2, G.GALE_F32, 64, P, n, None) == G.GALE_ERR_ALIGN
    big = 1 << 22
    assert g(P, big, 128, P, big, P, G.GALE_F32, big, P, n, None) == G.GALE_ERR_UNSUPPORTED


def test_rmsnorm_refusals():
    f = G.lib().gale_rmsnorm

    def call(x=P, r=None, dt=G.GALE_BF16, ldx=64, ldr=64, w=None, wt=0, eps=1e-6, t=2, c=64, h=None, ldh=64, y=P,
             yt=G.GALE_BF16, ldy=64, m=None):
        return f(x, r, dt, ldx, ldr, w, wt, eps, t, c, h, ldh, y, yt, ldy, m, None)

    assert call(t=0) == G.GALE_OK
    assert call(x=None) == G.GALE_ERR_ARG
    assert call(y=None) == G.GALE_ERR_ARG                       # no output
    assert call(dt=5) == G.GALE_ERR_ARG
    assert call(yt=5) == G.GALE_ERR_ARG
    assert call(w=P, wt=5) == G.GALE_ERR_ARG
    assert call(eps=-1.0) == G.GALE_ERR_ARG
    assert call(eps=float("nan")) == G.GALE_ERR_ARG
    assert call(t=-1) == G.GALE_ERR_ARG
    assert call(c=0) == G.GALE_ERR_ARG
    assert call(c=32769, ldx=40000) == G.GALE_ERR_UNSUPPORTED
    assert call(ldx=63) == G.GALE_ERR_ARG
    assert call(r=P, ldr=63) == G.GALE_ERR_ARG
    assert call(h=P, ldh=63) == G.GALE_ERR_ARG
    assert call(ldy=63) == G.GALE_ERR_ARG
    assert call(x=P + 1) == G.GALE_ERR_ALIGN
    assert call(w=P + 2, wt=G.GALE_F32) == G.GALE_ERR_ALIGN
    assert call(m=P + 16) == G.GALE_ERR_ALIGN


def test_route_select_refusals():
    f = G.lib().gale_route_select

    def call(l=P, dt=G.GALE_F32, ld=64, b=None, B=2, E=64, K=4, score=0, n=1, keep=1, top=1, ids=P, gates=P):
        return f(l, dt, ld, b, B, E, K, score, n, keep, top, 1, 1.0, ids, gates, None)

    assert call(B=0) == G.GALE_OK
    for bad in (dict(l=None), dict(ids=None), dict(gates=None), dict(dt=3), dict(ld=63), dict(B=-1), dict(E=0),
                dict(E=1025, ld=1025), dict(K=0), dict(K=17), dict(E=3, K=4), dict(score=2), dict(n=0), dict(n=5),
                dict(n=33, E=66, ld=66), dict(n=4, keep=0), dict(n=4, keep=5), dict(top=0), dict(top=3),
                dict(n=32, keep=1, K=4)):
        assert call(**bad) == G.GALE_ERR_ARG, bad
    assert call(l=P + 2) == G.GALE_ERR_ALIGN
    assert call(b=P + 2) == G.GALE_ERR_ALIGN
    assert call(gates=P + 1) == G.GALE_ERR_ALIGN


def test_binding_refuses_wrong_shapes():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(G.GaleError):
        G.gale_rmsnorm(x, y=torch.zeros(4, 63), stream=0)
    with pytest.raises(G.GaleError):
        G.gale_rmsnorm(x, y=x, residual=x.float(), stream=0)
    with pytest.raises(G.GaleError):
        G.gale_rmsnorm(x.t(), y=x.t(), stream=0)                  # columns not contiguous
    with pytest.raises(G.GaleError):
        G.gale_rmsnorm(x, mx8=torch.zeros(64, dtype=torch.uint8), stream=0)
    with pytest.raises(G.GaleError):
        G.gale_mx4_quantize(x, torch.zeros(64, dtype=torch.uint8), stream=0)
    with pytest.raises(G.GaleError):
        G.gale_route_select(x, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4), stream=0)
    with pytest.raises(G.GaleError):                              # 64-bit ids
        G.gale_route_select(x, torch.zeros(4, 4, dtype=torch.int64), torch.zeros(4, 4), stream=0)
    with pytest.raises(G.GaleError):                              # a bias of another size
        G.gale_route_select(x, torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4), bias=torch.zeros(63), stream=0)
    with pytest.raises(G.GaleError):                              # integers are no weights
        G.gale_mx8_quantize(torch.zeros(4, 64, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8), stream=0)
    with pytest.raises(G.GaleError):                              # a missing tensor
        G.gale_mx_gemm(None, 64, 64, x, x, x, stream=0)
    with pytest.raises(G.GaleError) as e:                         # all right but for the device
        G.gale_rmsnorm(x, y=x, stream=0)
    assert e.value.code == G.GALE_ERR_ARG and "device" in str(e.value)
