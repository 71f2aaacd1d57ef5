"""How near the router's probabilities, their sums, gates and losses come to their
definitions.

U = 2^-24.  A probability exp2((l - top) * log2(e)) / sum has the roundings of the
difference, of the product and of the constant (3.5 U of far = top - l together), the
exponential's, the reciprocal's and the sum's (some 8 U): 4 far + 12.  A sum of them over
many tokens has what these have in common, a U or two, and its own roundings, U r / (3
sqrt(n)) for chains of r of n tokens: 16 U."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_router import U, logits, oracle  # noqa: E402


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k,W", [(4096, 8, 2, 1), (2048, 64, 6, 2), (65536, 64, 6, 16), (20000, 100, 3, 5), (131072, 256, 8, 8),
                                     (8192, 512, 8, 1), (16384, 1024, 32, 4)])
def test_routing_and_load(ga, T, E, k, W, x):
    l = logits(T, E, x)
    for norm in (False, True):
        router = ga.Router(E, k, l.dtype, workers=W, normalize=norm)
        r, load = router.empty_routing(T), router.empty_load()
        router.forward(l, r, load)
        o = oracle(l, None, None, k, W, norm, "all")
        assert torch.equal(r.experts.long(), o["experts"]) and torch.equal(load.counts.long(), o["counts"])
        far = l.double().amax(1, keepdim=True) - l.double().gather(1, o["experts"])
        assert bool(((r.gates.double() / o["gates"] - 1).abs() <= (4 * far + 12) * U).all())
        assert bool(((r.lse.double() - o["lse"]).abs() <= (2 * o["lse"].abs() + 12) * U).all())
        assert bool(((load.probs.double() / o["probs"] - 1).abs() <= 16 * U).all())
        assert bool(((load.loss.double() / o["loss"] - 1).abs() <= 16 * U).all())
