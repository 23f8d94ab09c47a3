"""GPU parity of the microscaled formats and their product.

Quantisers and unpacker are exact: every decision is a comparison with a power
of two or a rounding to nearest even of a value that fp32 holds exactly.  The
product is compared with the fp64 product of the same packed values:

  |y - want| <= (cols/32 + 34) 2^-23 sum|w x| + |want| eps_out / 2

(products of two codes and their scales are exact in fp32; a sum of 32 of them
and the cols/32 additions into the accumulator lose at most one unit in the
last place, 2^-23, of the running magnitude each, whether an adder rounds or
truncates; the result is rounded once).
"""
import numpy as np
import pytest

from oracle import mx_oracle as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("bit_expert_gemv_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.lib()


def _matrix(rows, cols, seed, dtype="f32", scale=1.0):
    v = np.random.default_rng(seed).normal(size=(rows, cols)).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(v).to(DT[dtype]).cuda()


def _pack4(w):
    buf = torch.full((G.gale_mx4_layout(*w.shape).total,), 0xEE, dtype=torch.uint8, device="cuda")
    G.gale_mx4_quantize(w, buf)
    return buf


def _pack8(x):
    buf = torch.full((G.gale_mx8_layout(*x.shape).total,), 0xEE, dtype=torch.uint8, device="cuda")
    G.gale_mx8_quantize(x, buf)
    return buf


def _hard(w):
    """Zeros, ties, extremes, infinities and NaN in blocks of their own."""
    w = w.clone()
    r, c = w.shape
    if r > 6 and c >= 32:
        w[1, :32] = 0.0
        w[2, :11] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, -0.0]).to(w.dtype)
        w[2, 11:32] = 0.0
        w[3, 0] = float("inf")
        w[4, 31] = float("nan")
        w[5, :32] = torch.finfo(w.dtype).tiny
        w[6, 5] = torch.finfo(w.dtype).max
    return w


@pytest.mark.parametrize("rows,cols,dtype", [(1, 1, "f32"), (7, 33, "bf16"), (128, 128, "f16"), (130, 200, "f32"),
                                             (257, 1001, "bf16"), (64, 4096, "f32"), (300, 416, "f16")])
def test_mx4_quantize_and_unpack_exact(rows, cols, dtype):
    w = _hard(_matrix(rows, cols, rows + cols, dtype))
    buf = _pack4(w)
    codes, k = M.quantize(w.double().cpu().numpy(), M.GRID4)
    want, L = M.pack4(codes, k), M.layout(rows, cols, True)
    got = buf.cpu().numpy()
    assert np.array_equal(got[:L["q_bytes"]], want[:L["q_bytes"]])
    s = slice(L["s_offset"], L["s_offset"] + L["s_bytes"])
    assert np.array_equal(got[s], want[s])
    vals = M.values(codes, k, M.GRID4)
    for name, t in DT.items():
        out = torch.empty(rows, cols, dtype=t, device="cuda")
        G.gale_mx4_unpack(buf, out)
        # rounded once into the type, from a value that fp32 holds exactly
        assert torch.equal(out.cpu().nan_to_num(nan=12345.0),
                           torch.from_numpy(vals).float().to(t).nan_to_num(nan=12345.0)), name


def test_mx4_strided_and_unaligned():
    # rows of 200 elements 216 apart, from an odd element: no 16-byte reads or writes
    base = _matrix(60, 216, 9, "bf16")
    w = base.view(-1)[1:1 + 59 * 216 + 200].as_strided((59, 200), (216, 1))
    assert torch.equal(_pack4(w), _pack4(w.contiguous()))
    buf = _pack4(w)
    wide = torch.full((59, 231), 7.0, device="cuda")
    G.gale_mx4_unpack(buf, wide[:, 3:203])
    flat = torch.empty(59, 200, device="cuda")
    G.gale_mx4_unpack(buf, flat)
    assert torch.equal(wide[:, 3:203], flat)
    assert (wide[:, :3] == 7).all() and (wide[:, 203:] == 7).all()


@pytest.mark.parametrize("tokens,cols,dtype", [(1, 1, "f32"), (1, 4096, "bf16"), (5, 100, "f16"), (129, 257, "bf16"),
                                               (64, 128, "f32"), (200, 1000, "bf16")])
def test_mx8_quantize_exact(tokens, cols, dtype):
    x = _hard(_matrix(tokens, cols, tokens * 3 + cols, dtype, 5.0))
    L = M.layout(tokens, cols, False)
    got = _pack8(x).cpu().numpy()
    codes, k = M.quantize(x.double().cpu().numpy(), M.GRID8)
    gc, gk = M.unpack8(got, tokens, cols)
    assert np.array_equal(gc[:, :cols], codes) and not gc[:, cols:].any()
    assert np.array_equal(gk[:, :k.shape[1]], k) and (gk[:, k.shape[1]:] == -127).all()
    # nothing behind the layout's used bytes is touched: scales of rows that do not exist
    live = np.zeros(L["s_bytes"], bool)
    live[M.scale_places(tokens, cols).ravel()] = True
    assert (got[L["s_offset"]:L["s_offset"] + L["s_bytes"]][~live] == 0xEE).all()


def _gemm(w4, rows, cols, x8, tokens, out="f32", ldy=None):
    y = torch.full((tokens, ldy or rows), 99.0, dtype=DT[out], device="cuda")
    ws = torch.zeros(G.gale_mx_gemm_workspace_size(rows, cols, tokens), dtype=torch.uint8, device="cuda")
    G.gale_mx_gemm(w4, rows, cols, x8, y[:, :rows], ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    assert (y[:, rows:] == 99).all()
    return y[:, :rows]


def _want(w, x):
    wv = M.values(*M.quantize(w.double().cpu().numpy(), M.GRID4), M.GRID4)
    xv = M.values(*M.quantize(x.double().cpu().numpy(), M.GRID8), M.GRID8)
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def _check(y, want, mag, cols, out):
    got = y.double().cpu().numpy()
    tol = (cols / 32 + 34) * 2.0 ** -23 * mag + np.abs(want) * torch.finfo(DT[out]).eps / 2 * (1 + 1e-6)
    if out == "f16":
        tol += 2.0 ** -25                                    # half a subnormal step
    worst = np.max(np.abs(got - want) - tol)
    assert worst <= 0, f"off by {worst:.3g} more than the bound"


@pytest.mark.parametrize("rows,cols,tokens,out", [
    (1, 1, 1, "f32"), (128, 128, 1, "f32"), (128, 128, 16, "f32"), (16, 32, 3, "bf16"), (130, 100, 2, "f32"),
    (256, 4096, 1, "f32"), (256, 4096, 8, "bf16"), (2048, 4096, 8, "f32"), (300, 1000, 17, "f16"),
    (257, 640, 33, "f32"), (512, 512, 64, "bf16"), (384, 2048, 100, "f32"), (128, 256, 128, "f32"),
    (200, 260, 129, "bf16"), (640, 384, 255, "f32"), (1000, 777, 300, "f16"), (129, 4096, 257, "f32"),
    (4100, 512, 700, "f32"), (64, 16384, 5, "f32"), (2050, 4000, 513, "bf16"),
    # several tiles per CTA, alone and with left-over tiles that clusters share
    (38000, 300, 3, "f32"), (12800, 1024, 16, "bf16"), (20000, 260, 60, "f32"), (19072, 512, 200, "f32"),
    (5000, 200, 2100, "f32"), (3000, 390, 4000, "bf16"), (130, 130, 10000, "f16")])
def test_gemm_parity(rows, cols, tokens, out):
    w, x = _matrix(rows, cols, rows * 7 + cols, scale=0.02), _matrix(tokens, cols, tokens, "bf16", 3.0)
    y = _gemm(_pack4(w), rows, cols, _pack8(x), tokens, out)
    _check(y, *_want(w, x), cols, out)


def test_gemm_every_element_counts():
    # unit vectors as tokens: y[t][r] = W[r][c_t], each column once, at its own scale
    rows, cols = 200, 384
    w = _matrix(rows, cols, 5) * torch.exp2(torch.randint(-20, 20, (rows, cols), device="cuda").float())
    x = torch.eye(cols, device="cuda") * torch.exp2((torch.arange(cols, device="cuda") % 15 - 7).float())
    y = _gemm(_pack4(w), rows, cols, _pack8(x), cols)
    assert np.array_equal(y.double().cpu().numpy(), _want(w, x)[0])


def test_gemm_row_stride_and_repeat():
    rows, cols, tokens = 130, 256, 40
    w4, x8 = _pack4(_matrix(rows, cols, 1)), _pack8(_matrix(tokens, cols, 2))
    a = _gemm(w4, rows, cols, x8, tokens, "bf16")
    for ldy in (131, 136, 160):
        assert torch.equal(_gemm(w4, rows, cols, x8, tokens, "bf16", ldy), a)


def test_gemm_zero_token_and_nan_blocks():
    rows, cols, tokens = 256, 512, 20
    w, x = _matrix(rows, cols, 3), _matrix(tokens, cols, 4)
    x[7] = 0.0
    x[9, 40] = float("inf")
    w[100, 300] = float("nan")
    y = _gemm(_pack4(w), rows, cols, _pack8(x), tokens)
    assert torch.isnan(y[9]).all() and torch.isnan(y[:, 100]).all()
    keep = [i for i in range(rows) if i != 100]
    assert (y[7, keep] == 0).all()
    fine = [t for t in range(tokens) if t != 9]
    want, mag = _want(w, x)
    _check(y[fine][:, keep], want[fine][:, keep], mag[fine][:, keep], cols, "f32")


def test_gemm_other_stream_graph_and_two_workspaces():
    rows, cols, tokens = 512, 1024, 24
    w4, x8 = _pack4(_matrix(rows, cols, 11)), _pack8(_matrix(tokens, cols, 12))
    want = _gemm(w4, rows, cols, x8, tokens)
    n = G.gale_mx_gemm_workspace_size(rows, cols, tokens)
    outs, graphs = [], []
    for _ in range(2):
        y = torch.zeros(tokens, rows, device="cuda")
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            G.gale_mx_gemm(w4, rows, cols, x8, y, ws)
        outs.append((y, ws))
        graphs.append((g, s))
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for y, ws in outs:
        assert torch.equal(y, want) and int(ws[:4].view(torch.int32).item()) == 0


def test_gemm_behind_copies_and_other_kernels():
    """The product's set-up may overlap the kernel before it: behind memory sets,
    copies, library kernels and its own kind, eagerly and captured, it reads what
    they wrote."""
    rows, cols, tokens = 1024, 512, 40
    ws_ = [_matrix(rows, cols, s) for s in (1, 2)]
    xs = [_matrix(tokens, cols, s, "bf16") for s in (3, 4)]
    packs = [_pack4(w) for w in ws_]
    want = [[_gemm(p, rows, cols, _pack8(x), tokens).clone() for x in xs] for p in packs]
    w4, x8 = torch.zeros_like(packs[0]), torch.zeros(G.gale_mx8_layout(tokens, cols).total, dtype=torch.uint8, device="cuda")
    x = torch.zeros_like(xs[0])
    y = [torch.zeros(tokens, rows, device="cuda") for _ in range(6)]
    ws = torch.zeros(G.gale_mx_gemm_workspace_size(rows, cols, tokens), dtype=torch.uint8, device="cuda")

    def run():
        x.copy_(xs[0])
        G.gale_mx8_quantize(x, x8)
        w4.copy_(packs[0])                                     # a copy right before the product
        G.gale_mx_gemm(w4, rows, cols, x8, y[0], ws)
        G.gale_mx_gemm(packs[1], rows, cols, x8, y[1], ws)     # behind its own kind
        x.copy_(xs[1])
        G.gale_mx8_quantize(x, x8)                             # overwrites what the last product read
        G.gale_mx_gemm(w4, rows, cols, x8, y[2], ws)
        G.gale_mx4_quantize(ws_[1], w4)                        # overwrites its weights
        G.gale_mx_gemm(w4, rows, cols, x8, y[3], ws)
        y[4].zero_()                                           # a memory set right before
        G.gale_mx_gemm(w4, rows, cols, x8, y[4], ws)
        torch.add(y[4], 1.0, out=y[5])                         # a library kernel behind

    def check():
        torch.cuda.synchronize()
        for got, w in zip(y, (want[0][0], want[1][0], want[0][1], want[1][1], want[1][1], want[1][1] + 1.0)):
            assert torch.equal(got, w)

    for _ in range(3):
        run()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        run()
    for t in y:
        t.zero_()
    for _ in range(4):
        g.replay()
    check()


@pytest.mark.parametrize("rows,cols,tokens", [(3900, 1600, 1100), (16400, 900, 600), (8192, 2100, 513), (130, 4000, 9000)])
def test_gemm_pairs_repeat_under_load(rows, cols, tokens):
    """Tiles over CTA pairs: odd numbers of row tiles, of column tiles and of
    tokens, several tiles per pair, and the same bits from call to call while
    another stream keeps the memory busy (what one CTA copies or frees, the other
    one's MMAs read or overwrite)."""
    w, x = _matrix(rows, cols, rows, scale=0.02), _matrix(tokens, cols, tokens, "bf16", 3.0)
    w4, x8 = _pack4(w), _pack8(x)
    first = _gemm(w4, rows, cols, x8, tokens, "f32")
    _check(first, *_want(w, x), cols, "f32")
    s, noise = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    ws = torch.zeros(G.gale_mx_gemm_workspace_size(rows, cols, tokens), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(tokens, rows, device="cuda") for _ in range(12)]
    torch.cuda.synchronize()
    for y in ys:
        with torch.cuda.stream(s):
            noise.add_(1.0)
        G.gale_mx_gemm(w4, rows, cols, x8, y, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for y in ys) and int(ws[:4].view(torch.int32).item()) == 0
