"""GPU parity of gale_rmsnorm against fp64.

A thread adds at most 32 squares in order and then 10 warp steps, all terms
positive: the sum is within 42 half units (2^-24) relatively, the norm's factor
within 21 and three more roundings (mean, square root, quotient), h, its
product with the factor and the weight add three: 30 * 2^-24 relative, plus
half a unit of the output type.
"""
import numpy as np
import pytest

from oracle import mx_oracle as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("bit_expert_gemv_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 30 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.lib()


def _rand(shape, seed, dtype, scale=1.0):
    v = np.random.default_rng(seed).normal(size=shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(v).to(DT[dtype]).cuda()


def _close(got, want, dtype):
    t = DT[dtype]
    tol = np.abs(want) * (REL + torch.finfo(t).eps / 2) + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


def _close_mx8(buf, want, tokens, cols):
    """Each value within half a step of its block's e4m3 grid, the scale the
    smallest that does not clip (to the norm's own error)."""
    codes, k = M.unpack8(buf.cpu().numpy(), tokens, cols)
    assert not codes[:, cols:].any() and (k[:, M.up(cols, 32) // 32:] == -127).all()
    k = k[:, :M.up(cols, 32) // 32]
    got = M.values(codes[:, :cols], k, M.GRID8)
    unit = 2.0 ** np.repeat(k, 32, axis=1)[:, :cols]
    tol = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10 * unit) + 2 * REL * np.abs(want)
    assert (np.abs(got - want) <= tol).all()
    pad = np.zeros((tokens, M.up(cols, 32)))
    pad[:, :cols] = np.abs(want)
    amax = pad.reshape(tokens, -1, 32).max(-1)
    some = amax > 0
    assert (amax[some] * (1 - REL) <= 448 * 2.0 ** k[some]).all()
    assert (amax[some] * (1 + REL) > 224 * 2.0 ** k[some])[k[some] > -127].all()


@pytest.mark.parametrize("tokens,cols", [(1, 1), (3, 31), (9, 32), (5, 64), (17, 100), (2, 256), (33, 257), (4, 512),
                                         (7, 1000), (16, 1024), (3, 1032), (2, 2048), (5, 4096), (2, 5001), (3, 8192),
                                         (2, 9000), (1, 16384), (2, 20001), (1, 32768)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f32", "f16")])
def test_norm_parity(tokens, cols, dtype, out):
    x, r = _rand((tokens, cols), cols, dtype, 2.0), _rand((tokens, cols), cols + 1, dtype)
    w = 1 + 0.1 * _rand((cols,), 3, "f32")
    y = torch.full((tokens, cols), 9.0, dtype=DT[out], device="cuda")
    h = torch.empty_like(x)
    m = torch.full((G.gale_mx8_layout(tokens, cols).total,), 0xEE, dtype=torch.uint8, device="cuda")
    G.gale_rmsnorm(x, y=y, residual=r, weight=w, sum_out=h, mx8=m, eps=1e-5)
    hw, yw = M.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), w.double().cpu().numpy(), 1e-5)
    _close(h, hw, dtype)
    _close(y, yw, out)
    _close_mx8(m, yw, tokens, cols)


@pytest.mark.parametrize("wt", ["f32", "bf16", "f16", None])
@pytest.mark.parametrize("cols", [96, 4096, 5001])
def test_norm_weights_and_single_outputs(wt, cols):
    x = _rand((6, cols), 1, "bf16")
    w = None if wt is None else (1 + 0.1 * _rand((cols,), 3, "f32")).to(DT[wt])
    _, yw = M.rmsnorm(x.double().cpu().numpy(), None, None if w is None else w.double().cpu().numpy(), 1e-6)
    y = torch.empty_like(x)
    G.gale_rmsnorm(x, y=y, weight=w)
    _close(y, yw, "bf16")
    m = torch.empty(G.gale_mx8_layout(6, cols).total, dtype=torch.uint8, device="cuda")
    G.gale_rmsnorm(x, mx8=m, weight=w)
    _close_mx8(m, yw, 6, cols)
    h = torch.empty_like(x)
    G.gale_rmsnorm(x, sum_out=h, residual=x)
    assert torch.equal(h, (2 * x.float()).to(x.dtype))


@pytest.mark.parametrize("cols,ld,off", [(200, 216, 0), (200, 216, 1), (4096, 4100, 0), (4096, 4104, 0), (5000, 5008, 3)])
def test_norm_strides_in_place(cols, ld, off):
    tokens = 5
    base = _rand((tokens * ld + 8,), ld, "bf16")
    x = base[off:].as_strided((tokens, cols), (ld, 1))
    r = _rand((tokens, cols), 2, "bf16")
    hw, yw = M.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), None)
    before = base.clone()
    rest = torch.ones(base.shape, dtype=torch.bool, device="cuda")
    rest[off:].as_strided((tokens, cols), (ld, 1)).fill_(False)
    G.gale_rmsnorm(x, y=x, residual=r, sum_out=r)            # y over x, the sum over the residual
    _close(x, yw, "bf16")
    _close(r, hw, "bf16")
    assert torch.equal(base[rest], before[rest])             # between and behind the rows: untouched


@pytest.mark.parametrize("cols", [64, 4096, 5001])
def test_norm_zero_nan_and_inf_rows(cols):
    x = _rand((6, cols), 8, "f32")
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y = torch.empty_like(x)
    m = torch.empty(G.gale_mx8_layout(6, cols).total, dtype=torch.uint8, device="cuda")
    G.gale_rmsnorm(x, y=y, mx8=m, eps=1e-6)
    assert (y[1] == 0).all() and torch.isnan(y[2]).all()
    # an infinity: its factor is 0, so the row is 0 but for inf * 0
    assert torch.isnan(y[3, 7]) and (y[3, :7] == 0).all() and (y[3, 8:] == 0).all()
    codes, k = M.unpack8(m.cpu().numpy(), 6, cols)
    n = M.up(cols, 32) // 32
    assert (k[1, :n] == -127).all() and (k[2, :n] == 128).all() and k[3, 0] == 128 and (k[3, 1:n] == -127).all()
    rows = [0, 4, 5]
    _close(y[rows], M.rmsnorm(x[rows].double().cpu().numpy())[1], "f32")


@pytest.mark.parametrize("tokens,cols", [(520, 9000), (520, 9001), (330, 16384), (330, 16387), (2, 9003), (1, 300), (9, 511)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("res", [False, True])
def test_norm_wide_rows_and_few(tokens, cols, dtype, out, res):
    # rows of the ring's widest form and past it, and single rows that start at any element
    x = _rand((tokens, cols), cols, dtype)
    r = _rand((tokens, cols), cols + 1, dtype) if res else None
    w = 1 + 0.1 * _rand((cols,), 3, dtype).float()
    y = torch.full((tokens * cols + 8,), 7.0, dtype=DT[out], device="cuda")
    yv = y[:tokens * cols].view(tokens, cols)
    G.gale_rmsnorm(x, y=yv, residual=r, weight=w)
    _, yw = M.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy() if res else None, w.double().cpu().numpy())
    _close(yv, yw, out)
    assert (y[tokens * cols:] == 7).all()


@pytest.mark.parametrize("cols", [40, 257, 700, 1001, 2000, 4093, 5001])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("f16", "f16")])
def test_norm_many_rows_of_every_width(cols, dtype, out):
    # more rows than CTAs in flight: every kernel, rows that start at every element modulo 8
    tokens = 3001
    x, r = _rand((tokens, cols), cols, dtype), _rand((tokens, cols), cols + 1, dtype)
    w = 1 + 0.1 * _rand((cols,), 3, "f32")
    y, h = torch.empty(tokens, cols, dtype=DT[out], device="cuda"), torch.empty_like(x)
    G.gale_rmsnorm(x, y=y, residual=r, weight=w, sum_out=h)
    hw, yw = M.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), w.double().cpu().numpy())
    _close(y, yw, out)
    _close(h, hw, dtype)
    # without the residual, in place
    G.gale_rmsnorm(x, y=x, weight=w)
    # (the rows are the inputs' own buffer)
    _, yw = M.rmsnorm(_rand((tokens, cols), cols, dtype).double().cpu().numpy(), None, w.double().cpu().numpy())
    _close(x, yw, dtype)


@pytest.mark.parametrize("cols,ldx,ldr,ldy", [(1000, 1003, 1011, 1019), (1000, 1001, 1001, 1002), (700, 704, 712, 720),
                                              (513, 513, 521, 513)])
def test_norm_many_strided_rows(cols, ldx, ldr, ldy):
    # strides that agree modulo 8 (the ring) and ones that do not
    tokens = 2500
    x, r = _rand((tokens, ldx), 1, "bf16"), _rand((tokens, ldr), 2, "bf16")
    y = torch.full((tokens, ldy), 5.0, device="cuda", dtype=torch.bfloat16)
    G.gale_rmsnorm(x[:, :cols], y=y[:, :cols], residual=r[:, :cols])
    _close(y[:, :cols], M.rmsnorm(x[:, :cols].double().cpu().numpy(), r[:, :cols].double().cpu().numpy())[1], "bf16")
    assert (y[:, cols:] == 5).all()


def test_norm_many_rows_mx8():
    for cols in (300, 1000, 4000):
        x, r = _rand((2000, cols), cols, "bf16"), _rand((2000, cols), 7, "bf16")
        m = torch.empty(G.gale_mx8_layout(2000, cols).total, dtype=torch.uint8, device="cuda")
        G.gale_rmsnorm(x, mx8=m, residual=r, sum_out=r)
        hw = x.double().cpu().numpy() + _rand((2000, cols), 7, "bf16").double().cpu().numpy()
        _close(r, hw, "bf16")
        _close_mx8(m, M.rmsnorm(hw)[1], 2000, cols)


def test_norm_graph_on_another_stream():
    x, r = _rand((64, 4096), 1, "bf16"), _rand((64, 4096), 2, "bf16")
    y, h = torch.empty_like(x), torch.empty_like(x)
    G.gale_rmsnorm(x, y=y, residual=r, sum_out=h)
    want = y.clone()
    y.zero_()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        G.gale_rmsnorm(x, y=y, residual=r, sum_out=h)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("cols,ld", [(32760, 32769), (32761, 32761), (32764, 32771), (32768, 32769), (32768, 32770)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("tokens", [2, 9])
def test_norm_widest_rows_at_any_start(cols, ld, dtype, out, tokens):
    # with the columns before its first aligned ones such a row takes more than 512 threads' share
    x, r = _rand((tokens, ld), cols, dtype)[:, :cols], _rand((tokens, ld), 2, dtype)[:, :cols]
    w = 1 + 0.1 * _rand((cols,), 3, "f32")
    y = torch.full((tokens, ld), 9.0, dtype=DT[out], device="cuda")
    h = torch.full((tokens, ld), 9.0, dtype=DT[dtype], device="cuda")
    G.gale_rmsnorm(x, y=y[:, :cols], residual=r, weight=w, sum_out=h[:, :cols])
    hw, yw = M.rmsnorm(x.double().cpu().numpy(), r.double().cpu().numpy(), w.double().cpu().numpy())
    _close(h[:, :cols], hw, dtype)
    _close(y[:, :cols], yw, out)
    assert (y[:, cols:] == 9).all() and (h[:, cols:] == 9).all()


@pytest.mark.parametrize("cols", [16384, 20480, 32768])
@pytest.mark.parametrize("first", [0, 1, 2, 3])
def test_norm_sum_order_of_wide_rows(cols, first):
    """Squares just below half a unit of a thread's first one: each addition in
    order loses one whole, so a thread that added 64 of them in order would be
    off by 63 half units.  32 in order are what the bound above allows."""
    x = torch.full((2, cols), 2.0 ** -12 * (1 - 2.0 ** -12), device="cuda")
    x[:, first:2048:4] = 1.0                    # every thread's first column, whatever its unit
    x[1] *= 1.25
    w = 1 + _rand((cols,), 5, "f32").abs().clamp(max=0.99)
    y = torch.empty_like(x)
    G.gale_rmsnorm(x, y=y, weight=w, eps=0.0)
    _close(y, M.rmsnorm(x.double().cpu().numpy(), None, w.double().cpu().numpy(), 0.0)[1], "f32")
