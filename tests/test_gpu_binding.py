"""What the compiled argument marshalling does with arguments of the right kind
but a wrong value: it refuses them, whole, before the library is called."""
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
