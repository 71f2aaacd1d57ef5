"""The layer operators on the host: what they refuse, before any launch.  No
kernel runs here; argument checks that need a handle get a block in its place,
of which only sizes and types are read."""
import ctypes
import math
import os
import re
import subprocess

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


def block(*ints):
    """A handle whose first fields are these 32-bit numbers, the rest zero."""
    b = ctypes.create_string_buffer(1024)
    for i, v in enumerate(ints):
        ctypes.c_int32.from_buffer(b, 4 * i).value = v
    return b


@pytest.fixture
def gn():
    b = block(8, 2)           # channels, groups; binary32, no backward pass
    yield ctypes.addressof(b)


@pytest.fixture
def router():
    b = block(8, 2, 2)        # experts, k, workers; binary32
    yield ctypes.addressof(b)


def caller(f, good):
    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    return call


def test_constants_match_the_header(ga):
    from gradient_aggregation_amd import layers
    src = open(HEADER).read()
    for name, value in (("CHANNELS", layers.MAX_CHANNELS), ("EXPERTS", layers.MAX_EXPERTS), ("TOPK", layers.MAX_TOPK)):
        assert int(re.search(r"#define GA_MAX_%s (\d+)" % name, src).group(1)) == value
    assert int(re.search(r"#define GA_LAYERS_VERSION (\d+)", src).group(1)) == ga.lib().ga_layers_version() == 1


def test_c_layout(ga, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text("""
#include "gradagg.h"
_Static_assert(sizeof(ga_images) == %d && sizeof(ga_routing) == %d && sizeof(ga_load) == %d, "sizes");
_Static_assert(GA_ACT_NONE == 0 && GA_ACT_RELU == 1 && GA_ACT_SILU == 2, "activations");
_Static_assert(GA_BALANCE_ALL == 0 && GA_BALANCE_WORKER == 1, "scopes");
""" % (ctypes.sizeof(ga.Images), ctypes.sizeof(ga.RoutingPtrs), ctypes.sizeof(ga.LoadPtrs)))
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-fsyntax-only", str(src)], check=True)


@pytest.mark.parametrize("args,status", [
    ((0, 1, 0, 0, 0), 1), ((-4, 2, 0, 0, 0), 1), ((8, 0, 0, 0, 0), 1), ((8, 3, 0, 0, 0), 1), ((8, 16, 0, 0, 0), 1),
    ((8, -2, 0, 0, 0), 1), ((8, 2, 3, 0, 0), 1), ((8, 2, 0, 1, 0), 1), ((8, 2, 1, 2, 0), 1), ((8, 2, 0, 0, 3), 1),
    ((8, 2, 0, 0, -1), 1), ((65537, 1, 0, 0, 0), 4),
])
def test_groupnorm_create_refusals(ga, args, status):
    h = ctypes.c_void_p(1)
    assert ga.lib().ga_groupnorm_create(*args, 1, ctypes.byref(h)) == status
    assert h.value is None and ga.lib().ga_last_error()


@pytest.mark.parametrize("args,status", [
    ((0, 1, 0, 1, 0, 0), 1), ((8, 0, 0, 1, 0, 0), 1), ((8, 9, 0, 1, 0, 0), 1), ((8, 2, 3, 1, 0, 0), 1),
    ((8, 2, 0, 0, 0, 0), 1), ((8, 2, 0, 1, 0, 2), 1), ((1025, 2, 0, 1, 0, 0), 4), ((64, 33, 0, 1, 0, 0), 4),
    ((8, 2, 0, 1025, 0, 0), 4),
])
def test_router_create_refusals(ga, args, status):
    h = ctypes.c_void_p(1)
    assert ga.lib().ga_router_create(*args, ctypes.byref(h)) == status
    assert h.value is None and ga.lib().ga_last_error()


def test_create_needs_out(ga):
    assert ga.lib().ga_groupnorm_create(8, 2, 0, 0, 0, 1, None) == ga.GA_ERR_INVALID
    assert ga.lib().ga_router_create(8, 2, 0, 1, 0, 0, None) == ga.GA_ERR_INVALID
    ga.lib().ga_groupnorm_destroy(None)
    ga.lib().ga_router_destroy(None)


def test_groupnorm_forward_refusals(ga, gn):
    M = ga.Images
    x, y = M(64, 8, 32), M(4096, 8, 32)
    call = caller(ga.lib().ga_groupnorm_forward, [gn, 4, 4, x, None, None, 1e-5, y, None, None, None])
    bad = ga.GA_ERR_INVALID
    assert call(_0=None) == call(_3=None) == call(_7=None) == bad
    assert call(_3=M(None, 8, 32)) == call(_7=M(None, 8, 32)) == bad
    assert call(_1=-1) == call(_2=-1) == bad
    assert call(_1=0) == call(_2=0) == ga.GA_OK                    # nothing to do
    for eps in (0.0, -1e-5, math.inf, math.nan):
        assert call(_6=eps) == bad
    # positions, then samples, that overlap; strides without a meaning
    for m in (M(64, 7, 32), M(64, 8, 7), M(64, 8, 31), M(64, 31, 8), M(64, 0, 32), M(64, 8, 0), M(64, -8, 32),
              M(64, 8, -32), M(64, 1 << 60, 32), M(64, 8, 1 << 60)):
        assert call(_3=m) == call(_7=m) == bad
    assert call(_3=M(66, 8, 32)) == call(_7=M(65, 8, 32)) == ga.GA_ERR_ALIGN
    assert call(_4=2) == call(_5=1) == call(_8=2) == call(_9=2) == ga.GA_ERR_ALIGN
    assert call(_2=1 << 31) == call(_1=1 << 31) == call(_1=1 << 30) == ga.GA_ERR_UNSUPPORTED


def test_groupnorm_backward_refusals(ga):
    M = ga.Images
    m = M(64, 8, 32)
    h = block(8, 2)
    call = caller(ga.lib().ga_groupnorm_backward,
                  [ctypes.addressof(h), 4, 4, m, m, None, None, 64, 64, m, 2, 64, 64, 0, None])
    bad = ga.GA_ERR_INVALID
    assert call() == bad and b"without a backward pass" in ga.lib().ga_last_error()
    assert call(_0=None) == call(_3=None) == call(_4=None) == call(_9=None) == bad
    assert call(_1=-4) == call(_2=-4) == call(_10=0) == call(_10=3) == bad
    assert call(_11=None) == call(_12=None) == call(_13=5) == bad
    assert call(_1=2048, _10=1025) == ga.GA_ERR_UNSUPPORTED


def test_router_forward_refusals(ga, router):
    R, P, L = ga.Rows, ga.RoutingPtrs, ga.LoadPtrs
    load = L(64, 64, 64, 64, 64)
    call = caller(ga.lib().ga_router_forward, [router, 4, R(64, 8), None, 1, P(64, 64, 64), load, None])
    bad = ga.GA_ERR_INVALID
    assert call(_0=None) == call(_2=None) == call(_5=None) == bad
    assert call(_2=R(None, 8)) == call(_5=P(None, 64, 64)) == bad
    assert call(_1=-2) == call(_1=3) == bad                        # workers does not divide tokens
    for i in range(5):
        assert call(_6=L(*[None if j == i else 64 for j in range(5)])) == bad
        assert call(_6=L(*[66 if j == i else 64 for j in range(5)])) == ga.GA_ERR_ALIGN
    assert call(_2=R(64, 7)) == call(_2=R(64, -8)) == call(_2=R(64, 1 << 60)) == bad
    assert call(_2=R(66, 8)) == ga.GA_ERR_ALIGN
    for i in range(3):
        assert call(_5=P(*[66 if j == i else 64 for j in range(3)])) == ga.GA_ERR_ALIGN
    assert call(_1=1 << 30) == ga.GA_ERR_UNSUPPORTED
    assert call(_1=0, _6=None) == ga.GA_OK                         # nothing to do


def test_router_backward_refusals(ga):
    R, P = ga.Rows, ga.RoutingPtrs
    h = block(8, 2, 2, 0, 1)                                       # normalized gates
    call = caller(ga.lib().ga_router_backward,
                  [ctypes.addressof(h), 4, R(64, 8), None, P(64, 64, 64), 64, 64, 0.1, 0.1, R(128, 8), None])
    bad = ga.GA_ERR_INVALID
    assert call(_0=None) == call(_2=None) == call(_4=None) == call(_9=None) == bad
    assert call(_1=-2) == call(_1=3) == bad
    assert call(_7=math.inf) == call(_7=math.nan) == call(_8=-math.inf) == bad
    assert call(_5=None) == call(_5=None, _8=0.0) == call(_5=None, _7=0.0) == bad
    assert call(_4=P(None, 64, 64)) == call(_4=P(64, None, 64)) == call(_4=P(64, 64, None)) == bad
    assert call(_2=R(64, 7)) == call(_9=R(64, 7)) == call(_2=R(None, 8)) == call(_9=R(None, 8)) == bad
    assert call(_2=R(65, 8)) == call(_9=R(66, 8)) == call(_5=66) == call(_6=66) == ga.GA_ERR_ALIGN
    assert call(_4=P(64, 64, 66)) == call(_4=P(66, 64, 64)) == call(_4=P(64, 66, 64)) == ga.GA_ERR_ALIGN
    assert call(_1=1 << 30) == ga.GA_ERR_UNSUPPORTED
    assert call(_1=0) == ga.GA_OK


def test_no_cpu_fallback(ga):
    import torch
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    with pytest.raises(RuntimeError):
        ga.GroupNorm(64, 8)
    with pytest.raises(RuntimeError):
        ga.Router(8, 2)


def test_binding_refuses_types(ga):
    import torch
    for kw in (dict(x_dtype=torch.float64), dict(p_dtype=torch.int8), dict(activation="tanh")):
        with pytest.raises(ValueError):
            ga.GroupNorm(64, 8, **kw)
    for kw in (dict(dtype=torch.float64), dict(scope="token")):
        with pytest.raises(ValueError):
            ga.Router(8, 2, **kw)


def test_images_of_tensors(ga):
    """Which layouts the binding takes; the addresses are not read."""
    import torch
    from gradient_aggregation_amd import layers

    class Gpu(torch.Tensor):
        is_cuda = property(lambda self: True)

    def strides(t):
        t = t.as_subclass(Gpu)
        m = layers._images(t, t, "x")
        return m.ld, m.sample

    x = torch.zeros(3, 5, 7, 16)
    assert strides(x) == (16, 560)
    assert strides(x[..., :10]) == (16, 560)
    assert strides(torch.zeros(3, 16, 5, 7).to(memory_format=torch.channels_last).permute(0, 2, 3, 1)) == (16, 560)
    assert strides(x.permute(1, 0, 2, 3)[:, 1]) == (16, 560 // 5)  # rows of one sample as samples
    assert strides(torch.zeros(5, 3, 16).transpose(0, 1)) == (48, 16)
    assert strides(x[:, ::2, :1]) == (224, 560)
    assert strides(torch.zeros(4, 16)) == (16, 16)
    with pytest.raises(ValueError):
        strides(x[:, :, :6])                                       # positions that are not evenly spaced
    with pytest.raises(ValueError):
        strides(torch.zeros(3, 16, 5, 7).permute(0, 2, 3, 1))      # channels apart
