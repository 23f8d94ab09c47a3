"""What the compiled argument marshalling does with arguments of the right kind
but a wrong value: it refuses them, whole, before the library is called."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("bit_expert_gemv_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.lib()


def _router():
    return (torch.randn(4, 64, device="cuda"), torch.full((4, 6), -7, dtype=torch.int32, device="cuda"),
            torch.full((4, 6), -7.0, device="cuda"))


class NoTruth:
    def __bool__(self):
        raise ValueError("no truth")


@pytest.mark.parametrize("renorm", [NoTruth(), torch.zeros(2)])
def test_arguments_without_a_truth_value(renorm):
    l, ids, gates = _router()
    with pytest.raises(G.GaleError):
        G.gale_route_select(l, ids, gates, renorm=renorm)
    torch.cuda.synchronize()
    assert (ids == -7).all() and (gates == -7).all()


def test_streams_that_are_no_handles():
    l, ids, gates = _router()
    for stream in (1 << 70, -1 << 70, object(), type("S", (), {"cuda_stream": "x"})()):
        with pytest.raises(G.GaleError):
            G.gale_route_select(l, ids, gates, stream=stream)
    torch.cuda.synchronize()
    assert (ids == -7).all()


@pytest.mark.parametrize("name", ["score", "n_groups", "keep_groups", "group_top"])
@pytest.mark.parametrize("offset", [1 << 32, -1 << 32, 1 << 62])
def test_integers_beyond_32_bits(name, offset):
    # 2^32 + 1 is not 1
    l, ids, gates = _router()
    with pytest.raises(G.GaleError):
        G.gale_route_select(l, ids, gates, **{name: offset + 1})
    torch.cuda.synchronize()
    assert (ids == -7).all()


TRACED = """
import torch, bit_expert_gemv_b200 as G
x = torch.randn(3, 4, 64, device="cuda")
y = torch.zeros(4, 64, device="cuda")
ids = torch.zeros(4, 6, dtype=torch.int32, device="cuda")
def norm(v):
    G.gale_rmsnorm(v, y=y)
    return v
def router(v):
    G.gale_route_select(v, ids, torch.zeros(4, 6, device="cuda"))
    return v
for f in (norm, router):
    try:
        torch.func.vmap(f)(x)
    except RuntimeError as e:
        print("refused")
torch.cuda.synchronize()
assert not y.any()
"""


def test_tensors_without_memory_of_their_own():
    # (in a process of its own: an exception while other threads may run would end it)
    r = subprocess.run([sys.executable, "-c", TRACED], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused", "refused"], r.stderr[-2000:]


def test_lazily_negated_tensors():
    # the sign is a flag of the view, not in memory
    x = torch.randn(4, 64, device="cuda")
    y, (l, ids, gates) = torch.empty_like(x), _router()
    for call in (lambda: G.gale_rmsnorm(torch._neg_view(x), y=y), lambda: G.gale_rmsnorm(x, y=torch._neg_view(y)),
                 lambda: G.gale_route_select(torch._neg_view(l), ids, gates)):
        with pytest.raises(G.GaleError):
            call()
