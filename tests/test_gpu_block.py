"""The operators around the experts as one block, the way a layer runs them:
norm of the residual sum (16-bit and 8-bit outputs) -> router product -> router
by scores -> routed experts -> next norm.  Every step is compared with the fp64
oracle on the step's own inputs (an expert choice that flips on a rounding
upstream would say nothing), and the block as a captured graph with the eager
calls, bit for bit.
"""
import numpy as np
import pytest

import gale_synth as gs
from oracle import gale_oracle as O
from oracle import mx_oracle as M
from oracle import route_oracle as R

from .helpers import Layer, assert_tokens

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("bit_expert_gemv_b200")

D, FF, E, K = 2048, 1024, 32, 6
GROUPS = (8, 4, 2)


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return Layer(E, D, FF, layer=3)


def _normal(shape, tag, scale=1.0):
    n = int(np.prod(shape))
    v = gs.normal(gs.stream_key(91, tag), n).astype(np.float32).reshape(shape) * np.float32(scale)
    return torch.from_numpy(v).cuda()


class Block:
    def __init__(self, layer, T):
        self.layer, self.T = layer, T
        self.x = _normal((T, D), 1).bfloat16()
        self.res = _normal((T, D), 2, 3.0).bfloat16()
        self.w1, self.w2 = 1 + 0.1 * _normal((D,), 3), (1 + 0.1 * _normal((D,), 4)).bfloat16()
        self.router = _normal((E, D), 5, 0.02)
        self.bias = _normal((E,), 6, 0.05)
        self.w4 = torch.empty(G.gale_mx4_layout(E, D).total, dtype=torch.uint8, device="cuda")
        G.gale_mx4_quantize(self.router, self.w4)
        self.h, self.y, self.out, self.h2, self.y2 = (torch.zeros_like(self.x) for _ in range(5))
        self.x8 = torch.zeros(G.gale_mx8_layout(T, D).total, dtype=torch.uint8, device="cuda")
        self.logits = torch.zeros(T, E, device="cuda")
        self.gemm_ws = torch.zeros(G.gale_mx_gemm_workspace_size(E, D, T), dtype=torch.uint8, device="cuda")
        self.ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
        self.gates = torch.zeros(T, K, device="cuda")
        self.ws = torch.zeros(G.gale_moe_workspace_size(layer.desc, T, K), dtype=torch.uint8, device="cuda")

    def run(self):
        G.gale_rmsnorm(self.x, y=self.y, mx8=self.x8, residual=self.res, weight=self.w1, sum_out=self.h)
        G.gale_mx_gemm(self.w4, E, D, self.x8, self.logits, self.gemm_ws)
        G.gale_route_select(self.logits, self.ids, self.gates, bias=self.bias, score=G.GALE_SCORE_SIGMOID,
                            n_groups=GROUPS[0], keep_groups=GROUPS[1], group_top=GROUPS[2], scale=2.5)
        G.gale_moe_forward(self.layer.desc, self.y, self.ids, self.gates, self.out, self.ws)
        G.gale_rmsnorm(self.out, y=self.y2, residual=self.h, weight=self.w2, sum_out=self.h2)

    def outputs(self):
        return [t.clone() for t in (self.h, self.y, self.logits, self.ids, self.gates, self.out, self.h2, self.y2)]


def _f64(t):
    return t.double().cpu().numpy()


def _bf16_close(got, want):
    # 30 * 2^-24 of the norm and half a unit of bf16
    assert (np.abs(_f64(got) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -19) + 1e-38).all()


@pytest.mark.parametrize("T", [1, 7, 300])
def test_block_step_by_step(layer, T):
    b = Block(layer, T)
    b.run()
    torch.cuda.synchronize()
    assert int(b.gemm_ws[:4].view(torch.int32).item()) == 0 and int(b.ws[:4].view(torch.int32).item()) == 0
    hw, yw = M.rmsnorm(_f64(b.x), _f64(b.res), _f64(b.w1))
    _bf16_close(b.h, hw)
    _bf16_close(b.y, yw)
    codes, k = M.unpack8(b.x8.cpu().numpy(), T, D)
    xv = M.values(codes[:, :D], k[:, :D // 32], M.GRID8)
    wv = M.values(*M.quantize(_f64(b.router), M.GRID4), M.GRID4)
    # products and scales are exact, D / 32 + 34 additions lose a unit in the last place each
    tol = (D / 32 + 34) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)
    assert (np.abs(_f64(b.logits) - xv @ wv.T) <= tol + np.abs(xv @ wv.T) * 2.0 ** -24).all()
    ids, gates = R.route_select(_f64(b.logits), _f64(b.bias), K, True, *GROUPS, True, 2.5)
    assert np.array_equal(b.ids.cpu().numpy(), ids)
    assert (np.abs(_f64(b.gates) - gates) <= 2e-5 * gates).all()
    sel = np.arange(T) if T < 50 else np.arange(0, T, 13)
    want = O.moe_layer(layer.dense, _f64(b.y)[sel], ids[sel], _f64(b.gates)[sel])
    # the layer's own tolerance, and half a unit of its bf16 output
    assert_tokens(_f64(b.out)[sel], want, tol=2e-3 + 2.0 ** -9, what="experts")
    hw, yw = M.rmsnorm(_f64(b.out), _f64(b.h), _f64(b.w2))
    _bf16_close(b.h2, hw)
    _bf16_close(b.y2, yw)


@pytest.mark.parametrize("T", [1, 40])
def test_block_captured_and_replayed(layer, T):
    b = Block(layer, T)
    b.run()
    torch.cuda.synchronize()
    want = b.outputs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        b.run()
    for t in (b.h, b.y, b.out, b.h2, b.y2, b.logits, b.ids, b.gates):
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for got, w in zip(b.outputs(), want):
        assert torch.equal(got, w)
    # other inputs through the same graph
    b.x.copy_(_normal((T, D), 11).bfloat16())
    g.replay()
    torch.cuda.synchronize()
    got = b.outputs()
    b.run()
    torch.cuda.synchronize()
    for a, w in zip(b.outputs(), got):
        assert torch.equal(a, w)


def test_blocks_on_two_streams(layer):
    blocks = [Block(layer, T) for T in (8, 33)]
    want = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        want.append(b.outputs())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for x, y in zip(b.outputs(), w):
            assert torch.equal(x, y)


def test_two_threads_alternate_small_and_large_shapes():
    """Two Python threads in the library at once, each on its own stream: products
    and norms whose shared memory differs from call to call."""
    import threading

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    jobs = []
    for rows, cols, tokens in ((130, 200, 3), (2048, 4096, 300), (512, 512, 64), (300, 7000, 17)):
        w = torch.empty(G.gale_mx4_layout(rows, cols).total, dtype=torch.uint8, device="cuda")
        x = torch.empty(G.gale_mx8_layout(tokens, cols).total, dtype=torch.uint8, device="cuda")
        G.gale_mx4_quantize(torch.randn(rows, cols, device="cuda"), w)
        G.gale_mx8_quantize(torch.randn(tokens, cols, device="cuda"), x)
        n = G.gale_mx_gemm_workspace_size(rows, cols, tokens)
        jobs.append((lambda y, ws, w=w, x=x, rows=rows, cols=cols: G.gale_mx_gemm(w, rows, cols, x, y, ws), (tokens, rows),
                     torch.float32, n))
    for cols in (1024, 4096, 9000):
        x = torch.randn(5000000 // cols, cols, device="cuda").bfloat16()
        jobs.append((lambda y, ws, x=x: G.gale_rmsnorm(x, y=y), tuple(x.shape), torch.bfloat16, 256))

    def run_all(order):
        out = {}
        for i in order:
            call, shape, dtype, n = jobs[i]
            y, ws = torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
            call(y, ws)
            out[i] = y
        return out

    errors, got = [], {}

    def work(name, order):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    got[name] = run_all(order)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    torch.cuda.synchronize()
    n = len(jobs)
    threads = [threading.Thread(target=work, args=a) for a in (("a", range(n)), ("b", range(n - 1, -1, -1)))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    want = run_all(range(n))
    torch.cuda.synchronize()
    for out in got.values():
        assert all(torch.equal(out[i], want[i]) for i in range(n))


def _last_rows_only(make, rows, cols, dtype):
    """A [rows, cols] tensor whose last 3 rows alone hold values."""
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    t[-3:] = make((3, cols)).to(dtype)
    return t


@pytest.mark.parametrize("cols", [700, 4096, 4097, 32768])
def test_norm_offsets_beyond_32_bits(cols):
    if not torch.cuda.is_available() or torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    rows = 2 ** 31 // cols + 9
    x = _last_rows_only(lambda s: _normal(s, 71), rows, cols, torch.bfloat16)
    r = _last_rows_only(lambda s: _normal(s, 72), rows, cols, torch.bfloat16)
    y, h = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    G.gale_rmsnorm(x, y=y, residual=r, sum_out=h)
    tail = [torch.empty(3, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    G.gale_rmsnorm(x[-3:].clone(), y=tail[0], residual=r[-3:].clone(), sum_out=tail[1])
    hw, yw = M.rmsnorm(x[-3:].double().cpu().numpy(), r[-3:].double().cpu().numpy())
    for got, few, want in ((y, tail[0], yw), (h, tail[1], hw)):
        tol = np.abs(want) * (30 * 2.0 ** -24 + 2.0 ** -8) + 1e-30       # as in the norm's own tests
        assert (np.abs(got[-3:].double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(few.double().cpu().numpy() - want) <= tol).all()
        assert not got[:-3].any()


def test_product_offsets_beyond_32_bits():
    if not torch.cuda.is_available() or torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    rows, cols, tokens = 40000, 130, 2 ** 31 // 40000 + 9
    w, x = _normal((rows, cols), 73), _last_rows_only(lambda s: _normal(s, 74), tokens, cols, torch.bfloat16)
    w4 = torch.empty(G.gale_mx4_layout(rows, cols).total, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(G.gale_mx_gemm_workspace_size(rows, cols, tokens), dtype=torch.uint8, device="cuda")
    G.gale_mx4_quantize(w, w4)
    out = []
    for part in (x, x[-3:].clone()):
        x8 = torch.empty(G.gale_mx8_layout(part.shape[0], cols).total, dtype=torch.uint8, device="cuda")
        G.gale_mx8_quantize(part, x8)
        out.append(torch.full((part.shape[0], rows), 5.0, dtype=torch.bfloat16, device="cuda"))
        G.gale_mx_gemm(w4, rows, cols, x8, out[-1], ws)
    wv = torch.empty(rows, cols, device="cuda")
    G.gale_mx4_unpack(w4, wv)                                          # exact in fp32
    xv = torch.from_numpy(M.values(*M.quantize(x[-3:].double().cpu().numpy(), M.GRID8), M.GRID8)).cuda()
    want, mag = xv @ wv.double().t(), xv.abs() @ wv.double().abs().t()
    tol = (cols / 32 + 34) * 2.0 ** -23 * mag + want.abs() * 2.0 ** -8 * (1 + 1e-6)      # as in the product's own tests
    for got in (out[0][-3:], out[1]):
        assert ((got.double() - want).abs() <= tol).all()
    assert not out[0][:-3].any() and int(ws[:4].view(torch.int32).item()) == 0


def test_microscaled_offsets_beyond_32_bits():
    if not torch.cuda.is_available() or torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    for cols in (4096, 4097):
        rows = (2 ** 31 // cols + 9) // 128 * 128 + 131          # 3 rows in the last tile
        w = _last_rows_only(lambda s: _normal(s, 75), rows, cols, torch.bfloat16)
        back, few = torch.full_like(w, 5.0), torch.empty(3, cols, dtype=torch.bfloat16, device="cuda")
        for src, dst in ((w, back), (w[-3:].clone(), few)):
            p = torch.empty(G.gale_mx4_layout(src.shape[0], cols).total, dtype=torch.uint8, device="cuda")
            G.gale_mx4_quantize(src, p)
            G.gale_mx4_unpack(p, dst)
        assert torch.equal(back[-3:], few) and few.any() and not back[:-3].any()
        L, L3 = G.gale_mx8_layout(rows, cols), G.gale_mx8_layout(3, cols)
        p, p3 = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (L.total, L3.total))
        G.gale_mx8_quantize(w, p)
        G.gale_mx8_quantize(w[-3:].clone(), p3)
        assert torch.equal(p[L.q_bytes - 3 * L.cols_padded:L.q_bytes], p3[:L3.q_bytes])
        assert not p[:L.q_bytes - 3 * L.cols_padded].any()
        del w, back, p
