"""Selection among many equal logits: the lowest indexes, and in a time that does not grow
with the square of their number (a router whose weights start at zero gives nothing else)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_router import DT, check_forward, logits  # noqa: E402


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("E,k", [(3, 2), (8, 1), (8, 2), (16, 2), (32, 5), (60, 6), (64, 1), (100, 10), (128, 8), (250, 1), (256, 8), (257, 3), (512, 12),
                                 (700, 32), (1024, 1), (1024, 8), (1024, 32)])
def test_any_number_of_equal_logits(ga, E, k, x):
    """Tokens with 1, 2, 3, ... of the largest logit, above distinct ones, few others and none; some with
    experts at -infinity, so that fewer than k are left."""
    T = 96
    gen = torch.Generator(device="cuda").manual_seed(E + k)
    l = logits(T, E, x)
    for t in range(T):
        many = 1 + (t * t) % E
        at = torch.rand(E, generator=gen, device="cuda").argsort()
        kind = t % 4
        if kind == 1:
            l[t] = torch.randint(-1, 2, (E,), generator=gen, device="cuda").to(DT[x])
        elif kind == 2:
            l[t] = -1.5
        elif kind == 3:
            l[t] = -math.inf
        l[t, at[:many]] = 20.0 if kind else 0.25
    check_forward(ga, l, k, 3, True, "worker")
    check_forward(ga, l, k, 1, False)


def passes(f):
    """Microseconds of a pass, the least of some."""
    for _ in range(3):
        f()
    best = math.inf
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        for _ in range(5):
            f()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) / 5 * 1e3)
    return best


@pytest.mark.parametrize("T,E,k", [(131072, 256, 8), (131072, 256, 2), (32768, 512, 8), (16384, 1024, 32)])
def test_equal_logits_take_no_many_times_longer(ga, T, E, k):
    """2 to 5 times as long as distinct ones (k largest of E candidates, one after the other), where ranking E
    candidates against each other takes 20 to 40 times."""
    router = ga.Router(E, k, torch.bfloat16)
    r, load = router.empty_routing(T), router.empty_load()
    some = logits(T, E, "bf16")
    plain, loaded = passes(lambda: router.forward(some, r)), passes(lambda: router.forward(some, r, load))
    for l in (torch.zeros_like(some), (some > 1).to(some.dtype), some.clamp(-0.5, 0.5).round()):
        assert passes(lambda: router.forward(l, r)) <= 10 * plain
        assert passes(lambda: router.forward(l, r, load)) <= 10 * loaded
