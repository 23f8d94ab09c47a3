"""GPU parity of gale_route_select: ids equal to the fp64 oracle's, gates within
fp32's own error.

A gate is a quotient of exponentials: expf of an argument that is rounded by
half a unit (|l - m| 2^-24 relative in the result) and is itself good to 2
units, at most 16 (or 1024 / 32 + 5) additions of positive terms, a quotient
and the scale: below (|l - m| + 50) 2^-23, with |l - m| < 100 wherever the gate
is not subnormal: 2e-5.
"""
import numpy as np
import pytest

from oracle import route_oracle as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("bit_expert_gemv_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.lib()


def _run(logits, K, bias=None, sigmoid=False, groups=(1, 1, 1), renorm=True, scale=1.0):
    B = logits.shape[0]
    ids = torch.full((B, K), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((B, K), -7.0, device="cuda")
    G.gale_route_select(logits, ids, gates, bias=bias, score=G.GALE_SCORE_SIGMOID if sigmoid else G.GALE_SCORE_SOFTMAX,
                        n_groups=groups[0], keep_groups=groups[1], group_top=groups[2], renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    want_ids, want = R.route_select(logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(),
                                    K, sigmoid, *groups, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids), np.nonzero((ids.cpu().numpy() != want_ids).any(1))[0][:8]
    got = gates.double().cpu().numpy()
    assert (np.abs(got - want) <= 2e-5 * np.abs(want) + 1e-36).all()
    return ids, gates


def _logits(B, E, seed, dtype="f32"):
    rng = np.random.default_rng(seed)
    v = rng.normal(size=(B, E)) + 0.5 * rng.normal(size=E)
    return torch.from_numpy(v.astype(np.float32)).to(DT[dtype]).cuda()


def _bias(E, seed, scale=0.05):
    return torch.from_numpy((np.random.default_rng(seed).normal(size=E) * scale).astype(np.float32)).cuda()


SIZES = [(1, 1, 1), (3, 2, 2), (5, 17, 3), (9, 32, 6), (4, 33, 16), (7, 64, 8), (6, 100, 5), (11, 128, 6),
         (64, 256, 6), (5, 257, 8), (3, 512, 16), (4, 1000, 7), (2, 1024, 16)]


@pytest.mark.parametrize("B,E,K", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sigmoid,biased,renorm", [(False, False, True), (True, True, True), (False, True, False),
                                                   (True, False, False)])
def test_select_parity(B, E, K, dtype, sigmoid, biased, renorm):
    _run(_logits(B, E, E + K, dtype), K, _bias(E, 3) if biased else None, sigmoid, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,K", [(256, (8, 4, 2), 8), (256, (8, 1, 1), 6), (64, (32, 16, 2), 16),
                                        (96, (3, 2, 2), 9), (1000, (8, 3, 2), 16), (1024, (32, 4, 1), 8),
                                        (34, (2, 1, 1), 16), (8, (8, 8, 1), 8), (24, (4, 2, 2), 12), (32, (32, 5, 2), 5)])
@pytest.mark.parametrize("sigmoid,biased,dtype", [(True, True, "f32"), (False, False, "bf16"), (False, True, "f16"),
                                                  (True, False, "f32")])
def test_select_groups(E, groups, K, sigmoid, biased, dtype):
    _run(_logits(150, E, E, dtype), K, _bias(E, 5) if biased else None, sigmoid, groups)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 2)])
@pytest.mark.parametrize("dtype,renorm", [("f32", True), ("f32", False), ("bf16", False), ("bf16", True), ("f16", False)])
def test_select_masks_and_extremes(sigmoid, biased, groups, dtype, renorm):
    l = _logits(16, 64, 1, dtype)
    inf, big = float("inf"), float(torch.finfo(DT[dtype]).max)
    l[0] = -inf                                  # nothing is left
    l[1] = float("nan")
    l[2, 3:] = -inf                              # fewer experts than picks
    l[3, ::2] = -inf
    l[4, :32] = -big                             # the type's lowest value is a logit like any other
    l[5] = -big
    l[6, 9] = inf
    l[7, [9, 11]] = inf
    l[8] = 0.0                                   # all equal
    l[9] = 100.0 * l[9]                          # saturated scores: ties among keys, not among logits
    l[10] = -200.0 + l[10]
    l[11, :8] = -inf                             # a masked group
    l[12, 1:8] = -inf                            # a group with one expert
    l[13, 40] = float("nan")
    l[14] = 1e-20 * l[14]
    l[15] = -0.0
    l[15, 30] = 0.0
    _run(l, 6, _bias(64, 2) if biased else None, sigmoid, groups, renorm=renorm)


@pytest.mark.parametrize("spread", [0.5, 2.0, 30.0, 1e4, 1e20])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_wide_biases(sigmoid, spread):
    # keys far below the largest: picks outside a window of one, down to keys that the bias swallows
    l = _logits(60, 256, 12)
    b = _bias(256, 13, spread)
    _run(l, 8, b, sigmoid)
    _run(l, 8, b, sigmoid, (8, 3, 2))
    b[::2] = -1e9                                # a mask by a large finite value
    _run(l, 16, b, sigmoid)
    _run(l, 16, b, sigmoid, (8, 1, 2))


@pytest.mark.parametrize("offset", [-3e3, 1e3, 3e3, 1e4, 1e5, 1e7, 1e15, 2.5e38])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_large_biases(sigmoid, offset):
    # a bias that all experts share up to a little: the window's own offset rounds, and sums of two leave fp32
    l = _logits(60, 256, 14)
    b = (_bias(256, 15, 0.3).double() + offset).float()
    _run(l, 8, b, sigmoid)
    _run(l, 8, b, sigmoid, (8, 3, 2))
    b = (offset * (1 + 0.2 * _bias(256, 16, 1.0).double().clamp(-1, 1))).float()
    _run(l, 8, b, sigmoid, (8, 3, 2))


def test_select_bias_extremes():
    b = _bias(64, 4)
    b[3], b[9], b[20] = float("inf"), -float("inf"), float("nan")
    l = _logits(8, 64, 2)
    l[1, 3] = -float("inf")
    for groups in ((1, 1, 1), (8, 4, 2)):
        for sigmoid in (False, True):
            _run(l, 6, b, sigmoid, groups)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_near_ties(sigmoid):
    """Keys that differ by less than fp32 can tell: the order is the 64-bit
    values'.  Half of the experts share one value up to a unit in the last
    place, in the logits or in the bias."""
    B, E, K = 64, 256, 8
    rng = np.random.default_rng(6)
    l = np.full((B, E), 1.5, dtype=np.float32)
    step = rng.integers(-2, 3, size=(B, E)).astype(np.int32)
    l = (l.view(np.int32) + step).view(np.float32)
    l[:, ::2] = rng.normal(size=(B, E // 2))
    b = np.full(E, 0.25, dtype=np.float32)
    b = (b.view(np.int32) + rng.integers(-2, 3, size=E).astype(np.int32)).view(np.float32)
    b[::3] = 0.0
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(b).cuda()
    _run(lt, K, bt, sigmoid)
    _run(lt, K, bt, sigmoid, (8, 4, 2))
    _run(lt, K, None, sigmoid)
    _run(lt, K, None, sigmoid, (8, 4, 2))
    _run(lt.bfloat16(), K, bt, sigmoid, (8, 4, 2))


def test_select_strided_rows():
    wide = _logits(40, 300, 3)
    ids, gates = _run(wide[:, 20:276], 6, _bias(256, 1), True, (8, 4, 2))
    ids2, gates2 = _run(wide[:, 20:276].contiguous(), 6, _bias(256, 1), True, (8, 4, 2))
    assert torch.equal(ids, ids2) and torch.equal(gates, gates2)


def test_select_agrees_with_topk():
    # without bias, groups and scale it is the router that picks by logit
    l = _logits(500, 256, 9)
    ids, gates = torch.empty(500, 6, dtype=torch.int32, device="cuda"), torch.empty(500, 6, device="cuda")
    G.gale_route_topk(l, ids, gates)
    ids2, gates2 = _run(l, 6)
    assert torch.equal(ids, ids2)
    assert torch.allclose(gates, gates2, rtol=2e-6, atol=0)


def test_select_many_tokens():
    l = _logits(20000, 256, 10)
    want = {}
    for dtype, bias in (("f32", _bias(256, 7)), ("bf16", None)):
        x = l.to(DT[dtype])
        ids = torch.empty(20000, 8, dtype=torch.int32, device="cuda")
        gates = torch.empty(20000, 8, device="cuda")
        G.gale_route_select(x, ids, gates, bias=bias, score=G.GALE_SCORE_SIGMOID, n_groups=8, keep_groups=4,
                            group_top=2, scale=2.5)
        s = torch.sigmoid(x.double())
        sel = s if bias is None else s + bias.double()
        score = sel.view(-1, 8, 32).topk(2, -1).values.sum(-1)
        stay = torch.zeros(20000, 8, dtype=torch.bool, device="cuda").scatter(1, score.topk(4, -1).indices, True)
        key = torch.where(stay.repeat_interleave(32, 1), sel, -1.0)
        order = key.sort(dim=-1, descending=True, stable=True).indices[:, :8]
        same = (order == ids).all(1)
        # a tie between two groups' scores may fall either way in topk(): every other token is equal
        top = score.sort(-1, descending=True).values
        tied = top[:, 3] == top[:, 4]
        assert bool((same | tied).all())
        g = s.gather(1, ids.long())
        g = 2.5 * g / g.sum(-1, keepdim=True)
        assert torch.allclose(gates.double(), g, rtol=2e-5, atol=0)


# beyond 256 experts a packed key's fraction gives bits to the index
MANY = [(257, (1, 1, 1)), (384, (8, 3, 2)), (512, (16, 5, 1)), (1024, (32, 7, 2))]


@pytest.mark.parametrize("E,groups", MANY)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_many_experts_below_the_window(E, groups, sigmoid):
    # keys more than a window of one below the largest are ordered too
    for shape in {(1, 1, 1), groups}:
        l = _logits(24, E, E)
        l[:, 100] = 20.0                         # one logit leads, no bias to speak of
        _run(l, 6, torch.zeros(E, device="cuda"), sigmoid, shape)
        l, b = _logits(24, E, E + 1), torch.zeros(E, device="cuda")
        b[100] = 2.0                             # one expert is wanted by its bias
        _run(l, 6, b, sigmoid, shape)
        l = 100.0 * l                            # saturated scores
        _run(l, 6, b, sigmoid, shape)


@pytest.mark.parametrize("E,groups", MANY)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("lead", [0.05, 1.03, 3.0])
def test_select_many_experts_behind_masks(E, groups, sigmoid, lead):
    # ten live experts at high indices: none of the masked ones below them is picked first
    l = torch.full((16, E), -float("inf"), device="cuda")
    live = list(range(E - 50, E, 5))
    l[:, live] = -4.0 + 0.1 * _logits(16, 10, 3)
    b = torch.zeros(E, device="cuda")
    b[live[3]] = lead
    for shape in {(1, 1, 1), groups}:
        _run(l, 6, b, sigmoid, shape)
        _run(l, 12, b, sigmoid, shape)           # fewer live ones than picks


@pytest.mark.parametrize("E,groups", MANY)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_many_experts_wide_and_large_biases(E, groups, sigmoid):
    l = _logits(24, E, 12)
    for shape in {(1, 1, 1), groups}:
        for spread in (0.5, 2.0, 30.0, 1e4, 1e20):
            b = _bias(E, 13, spread)
            _run(l, 8, b, sigmoid, shape)
            b[::2] = -1e9
            _run(l, 16, b, sigmoid, shape)
        for offset in (-3e3, 1e3, 1e5, 1e7, 1e15, 2.5e38):
            _run(l, 8, (_bias(E, 15, 0.3).double() + offset).float(), sigmoid, shape)


@pytest.mark.parametrize("E,groups", MANY)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_many_experts_near_ties(E, groups, sigmoid):
    rng = np.random.default_rng(E)
    l = np.full((24, E), 1.5, dtype=np.float32)
    l = (l.view(np.int32) + rng.integers(-2, 3, size=l.shape).astype(np.int32)).view(np.float32)
    l[:, ::2] = rng.normal(size=l[:, ::2].shape)
    b = np.full(E, 0.25, dtype=np.float32)
    b = (b.view(np.int32) + rng.integers(-2, 3, size=E).astype(np.int32)).view(np.float32)
    b[::3] = 0.0
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(b).cuda()
    for shape in {(1, 1, 1), groups}:
        _run(lt, 8, bt, sigmoid, shape)
        _run(lt.bfloat16(), 8, bt, sigmoid, shape)
        bt2 = bt.clone()
        bt2[7] = 3.0                             # the ties lie below the window
        _run(lt, 8, bt2, sigmoid, shape)


@pytest.mark.parametrize("E,groups", MANY)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_many_experts_masks_and_extremes(E, groups, sigmoid, dtype):
    l = _logits(9, E, 1, dtype)
    inf, big = float("inf"), float(torch.finfo(DT[dtype]).max)
    l[0] = -inf
    l[1, 3:] = -inf
    l[2, ::2] = -inf
    l[3, :E // 2] = -big
    l[4, 9] = inf
    l[5] = 0.0
    l[6] = 100.0 * l[6]
    l[7] = -200.0 + l[7]
    l[8, :E - 3] = float("nan")
    b = _bias(E, 2)
    b[E // 2] = -inf
    for shape in {(1, 1, 1), groups}:
        for bias in (None, b):
            _run(l, 6, bias, sigmoid, shape)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_gates_of_far_picks(dtype):
    """Gates to within what their own formula rounds, also of picks far below the
    largest logit and of scores near the smallest fp32.  Sigmoid: the exponential
    2 units, the sum half, a quotient 2: the score of a pick 4.5, the sum of at
    most 16 of them 4.5 and its additions 2, the last quotient 2, together 13.
    Softmax: half a unit of the argument's size |x| as well, in the pick's own
    exponential (|x| / 2 + 2) and, weighed by exp(-|x|) |x| < 1, in the sum (0.5 +
    2 + 2), with the quotient |x| / 2 + 9; the denominator over all experts 8 units
    and 10 for its additions: |x| / 2 + 22.  A subnormal result is off by its own
    rounding too."""
    l = torch.full((64, 64), -300.0, device="cuda")
    pick = -torch.from_numpy(np.random.default_rng(3).uniform(0, 103, size=(64, 8)).astype(np.float32)).cuda()
    pick[:, 0] = 0.0
    l[:, 5:61:7] = pick
    l = l.to(DT[dtype])
    l[:32] -= 60.0                                # the sigmoids of half of the tokens: all tiny
    l64 = l.double().cpu().numpy()
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids = torch.empty(64, 8, dtype=torch.int32, device="cuda")
            gates = torch.empty(64, 8, device="cuda")
            G.gale_route_select(l, ids, gates, score=G.GALE_SCORE_SIGMOID if sigmoid else G.GALE_SCORE_SOFTMAX,
                                renorm=renorm)
            want_ids, want = R.route_select(l64, None, 8, sigmoid, renorm=renorm)
            assert np.array_equal(ids.cpu().numpy(), want_ids)
            x = l64.max(1, keepdims=True) - np.take_along_axis(l64, want_ids, 1)
            units = 13.0 if sigmoid else 0.5 * x + (9.0 if renorm else 22.0)
            off = np.abs(gates.double().cpu().numpy() - want)
            assert (off <= units * 2.0 ** -23 * want + 4 * 2.0 ** -149).all(), (sigmoid, renorm)


@pytest.mark.parametrize("E", [64, 256, 1024])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_group_sums_below_fp32(E, sigmoid):
    # experts pushed out by the lowest finite biases: the sum of two leaves fp32, but their groups come before
    # masked ones, and before each other by the 64-bit sums
    low, size = float(torch.finfo(torch.float32).min), E // 8
    l = _logits(6, E, 4)
    l[:, :size] = -float("inf")                  # group 0 is masked
    b = torch.full((E,), low, device="cuda")
    b[5 * size:6 * size] = 0.0                   # one group as it should be
    _run(l, size + 4 if size < 12 else 12, b, sigmoid, (8, 2, 2))
    b[5 * size:6 * size] = low
    b[3 * size:4 * size] = 0.98 * low
    b[6 * size:7 * size] = 0.97 * low
    for keep in (1, 2, 3, 7):
        _run(l, 8, b, sigmoid, (8, keep, 2))


def test_select_as_many_tokens_as_an_int_counts():
    B = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    l = torch.zeros(B, 1, dtype=torch.float16, device="cuda")
    ids = torch.full((B, 1), 7, dtype=torch.int32, device="cuda")
    gates = torch.full((B, 1), 7.0, device="cuda")
    G.gale_route_select(l, ids, gates)
    step = 1 << 28
    for t in range(0, B, step):
        assert not ids[t:t + step].any() and (gates[t:t + step] == 1.0).all()
