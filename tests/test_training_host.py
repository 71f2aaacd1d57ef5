"""The training-step operators on the host: what they refuse, before any
launch.  No kernel runs here; argument checks that need a handle get an
all-zero block in its place, of which only sizes and types are read."""
import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gradagg.h")


@pytest.fixture(scope="module")
def ga():
    import gradient_aggregation_amd as ga
    if not os.path.exists(ga.LIB_PATH):
        from gradient_aggregation_amd import build
        build.build()
    return ga


@pytest.fixture
def handle():
    block = ctypes.create_string_buffer(1024)
    yield ctypes.addressof(block)


def numels(*n):
    return (ctypes.c_int64 * len(n))(*n)


def test_structs_match_the_header(ga):
    assert ctypes.sizeof(ga.AdamWParams) == 32 and ga.AdamWParams.t.offset == 24
    assert ctypes.sizeof(ga.AdamWStatePtrs) == 32 and ctypes.sizeof(ga.Rows) == 16
    from gradient_aggregation_amd import training
    src = open(HEADER).read()
    assert int(re.search(r"#define GA_STATE_BLOCK (\d+)", src).group(1)) == training.STATE_BLOCK
    assert int(re.search(r"#define GA_MAX_WORKERS (\d+)", src).group(1)) == training.MAX_GROUPS


@pytest.mark.parametrize("W,layers,dtype,bits,status", [
    (0, [8], 0, 32, 1), (1025, [8], 0, 32, 1), (1, [8, 0], 0, 32, 1), (1, [8], 3, 32, 1), (1, [8], -1, 32, 1),
    (1, [8], 0, 16, 1), (1, [8], 0, 0, 1), (1, [(1 << 33) + 1], 0, 8, 4),
])
def test_adamw_create_refusals(ga, W, layers, dtype, bits, status):
    h = ctypes.c_void_p(1)
    assert ga.lib().ga_adamw_create(W, len(layers), numels(*layers), dtype, bits, None, ctypes.byref(h)) == status
    assert h.value is None and ga.lib().ga_last_error()


def test_adamw_create_needs_layers_and_out(ga):
    h = ctypes.c_void_p()
    assert ga.lib().ga_adamw_create(1, 0, numels(1), 0, 32, None, ctypes.byref(h)) == ga.GA_ERR_INVALID
    assert ga.lib().ga_adamw_create(1, 1, None, 0, 32, None, ctypes.byref(h)) == ga.GA_ERR_INVALID
    assert ga.lib().ga_adamw_create(1, 1, numels(1), 0, 32, None, None) == ga.GA_ERR_INVALID
    ga.lib().ga_adamw_destroy(None)
    ga.lib().ga_layernorm_destroy(None)


def params(ga, **kw):
    p = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, t=1)
    p.update(kw)
    return ga.AdamWParams(**p)


@pytest.mark.parametrize("kw", [
    dict(t=0), dict(t=-3), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
    dict(lr=-1e-3), dict(lr=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(weight_decay=-0.1),
    dict(weight_decay=math.inf),
])
def test_adamw_step_refuses_parameters(ga, handle, kw):
    state = ga.AdamWStatePtrs(16, 16, None, None)
    assert ga.lib().ga_adamw_step(handle, 16, params(ga, **kw), 16, state, None, None, 0, None) == ga.GA_ERR_INVALID


def test_adamw_step_refuses_pointers(ga, handle):
    step, ok = ga.lib().ga_adamw_step, ga.AdamWStatePtrs(16, 16, None, None)
    p = params(ga)
    for args in ((None, 16, p, 16, ok), (handle, None, p, 16, ok), (handle, 16, None, 16, ok), (handle, 16, p, None, ok),
                 (handle, 16, p, 16, None), (handle, 16, p, 16, ga.AdamWStatePtrs(None, 16)),
                 (handle, 16, p, 16, ga.AdamWStatePtrs(16, None))):
        assert step(*args, None, None, 0, None) == ga.GA_ERR_INVALID
    # a binary32 copy is no copy
    assert step(handle, 16, p, 16, ok, None, 16, ga.GA_FP32, None) == ga.GA_ERR_INVALID
    assert step(handle, 16, p, 16, ok, None, 16, 7, None) == ga.GA_ERR_INVALID
    for args in ((4, p, 16, ok, None, None, 0), (16, p, 8, ok, None, None, 0), (16, p, 16, ok, 8, None, 0),
                 (16, p, 16, ok, None, 8, ga.GA_BF16), (16, p, 16, ga.AdamWStatePtrs(8, 16), None, None, 0),
                 (16, p, 16, ga.AdamWStatePtrs(16, 4), None, None, 0)):
        assert step(handle, *args, None) == ga.GA_ERR_ALIGN


def test_grad_norm_refusals(ga, handle):
    f = ga.lib().ga_grad_norm
    assert f(None, 16, 1.0, None, 16, None) == ga.GA_ERR_INVALID
    assert f(handle, None, 1.0, None, 16, None) == ga.GA_ERR_INVALID
    assert f(handle, 16, 1.0, None, None, None) == ga.GA_ERR_INVALID
    for bad in (0.0, -1.0, math.nan):
        assert f(handle, 16, bad, None, 16, None) == ga.GA_ERR_INVALID
    assert f(handle, 4, 1.0, None, 16, None) == ga.GA_ERR_ALIGN
    assert f(handle, 16, 1.0, 8, 16, None) == ga.GA_ERR_ALIGN
    assert f(handle, 16, 1.0, None, 8, None) == ga.GA_ERR_ALIGN


@pytest.mark.parametrize("dim,x,p,status", [(0, 0, 0, 1), (-1, 0, 0, 1), (8, 3, 0, 1), (8, 1, 2, 1), (8, 0, 1, 1),
                                            ((1 << 20) + 1, 0, 0, 4)])
def test_layernorm_create_refusals(ga, dim, x, p, status):
    h = ctypes.c_void_p(1)
    assert ga.lib().ga_layernorm_create(dim, x, p, 1, ctypes.byref(h)) == status and h.value is None
    assert ga.lib().ga_layernorm_create(8, 0, 0, 1, None) == ga.GA_ERR_INVALID


def test_layernorm_forward_refusals(ga, handle):
    f, R = ga.lib().ga_layernorm_forward, ga.Rows
    r, odd = R(64, 8), R(65, 8)
    good = [handle, 4, r, None, None, None, 1e-5, R(128, 8), None, None, None, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_0=None) == call(_2=None) == call(_7=None) == ga.GA_ERR_INVALID
    assert call(_2=R(None, 8)) == call(_7=R(None, 8)) == ga.GA_ERR_INVALID
    assert call(_1=-1) == ga.GA_ERR_INVALID
    assert call(_1=0) == ga.GA_OK                       # no rows: nothing to do
    for eps in (0.0, -1e-5, math.inf, math.nan):
        assert call(_6=eps) == ga.GA_ERR_INVALID
    assert call(_2=R(64, -1)) == ga.GA_ERR_INVALID      # a stride shorter than a row
    assert call(_8=R(256, 8)) == ga.GA_ERR_INVALID      # a sum without a residual
    assert call(_3=r, _8=R(128, 8)) == ga.GA_ERR_INVALID  # y and sum are one tensor
    assert call(_2=odd) == call(_3=odd) == call(_7=odd) == ga.GA_ERR_ALIGN
    assert call(_4=2) == call(_5=1) == call(_9=2) == call(_10=2) == ga.GA_ERR_ALIGN


def test_layernorm_backward_refusals(ga, handle):
    f, R = ga.lib().ga_layernorm_backward, ga.Rows
    # a zero handle has no workspace: refused before anything is read through it
    r = R(64, 8)
    good = [handle, 4, r, r, None, 64, 64, None, r, 2, 64, 64, 0, None]

    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call() == ga.GA_ERR_INVALID and b"without a backward pass" in ga.lib().ga_last_error()
    assert call(_0=None) == call(_2=None) == call(_3=None) == call(_8=None) == ga.GA_ERR_INVALID
    assert call(_1=-4) == call(_9=0) == call(_9=3) == ga.GA_ERR_INVALID
    assert call(_10=None) == call(_11=None) == call(_12=5) == ga.GA_ERR_INVALID
    assert call(_1=2048, _9=1025) == ga.GA_ERR_UNSUPPORTED


def test_no_cpu_fallback(ga):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    with pytest.raises(RuntimeError):
        ga.AdamW([100])
    with pytest.raises(RuntimeError):
        ga.LayerNorm(64)


def test_binding_refuses_types(ga):
    import torch
    with pytest.raises(ValueError):
        ga.AdamW([100], grad_dtype=torch.float64)
    with pytest.raises(ValueError):
        ga.AdamW([100, 5], decay=[True])
    with pytest.raises(ValueError):
        ga.LayerNorm(64, x_dtype=torch.int8)


def test_package_imports_without_torch(ga):
    """Plan arithmetic needs no torch; the training-step names load it when asked for."""
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None\n"
            "import gradient_aggregation_amd as ga\n"
            "print(ga.compute_info(4, [100], False).P)\n"
            "try:\n    ga.AdamW\nexcept ImportError:\n    print('needs torch')\n")
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert p.stdout.split("\n")[:2] == ["100", "needs torch"], p.stderr
