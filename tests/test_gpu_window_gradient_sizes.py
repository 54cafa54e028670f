"""Gradients of the sliding-window attention at cotangents of any size, against
the 64-bit form in the relative norm.

Three roundings to the 16-bit format stand behind a value of a gradient: its
own (measured: the exact gradient rounded once), that of dS or P in the product
(a weighted sum of as many independent roundings, so no more than one in the
norm), and that of out inside delta (|out| <= max |v|, so no more than one).
The last two do not depend on the cotangent's size, so they are measured as the
rounding of the exact gradient scaled into the format's normal range.  Their
root of squares, and a tenth for the sample, is the bound; fp32 arithmetic in
between (1e-6) does not show."""
import math

import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import window_reference

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
# B, N, H, Hkv, D, window, sinks: on both sides of the 512 visible keys up to which delta is summed from P
SHAPES = [
    (1, 700, 4, 2, 64, 300, 4),
    (1, 1500, 4, 2, 64, 900, 4),
    (1, 700, 4, 2, 128, 300, 4),
    (1, 1500, 4, 2, 128, 900, 4),
    (2, 300, 3, 1, 32, 100, 0),
    (1, 1300, 3, 3, 16, 800, 70),
]


def inputs(shape, dtype, size, seed=3):
    B, N, H, Hkv, D = shape[:5]
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h, s=1.0: (s * torch.randn((B, N, h, D), generator=g, device="cuda")).to(dtype)  # noqa: E731
    return mk(H), mk(Hkv), mk(Hkv), mk(H, size)


def gradients(q, k, v, dout, window, sinks, impl=bd.LONGNET_IMPL_AUTO):
    out, lse = bd.window_attn(q, k, v, window, sinks, impl)
    grads = bd.window_attn_bwd(q, k, v, out, lse, dout, window, sinks, impl)
    assert bd.longnet_last_device_status() == 0
    return grads


def off(x, ref):
    return float((x.double() - ref).norm() / ref.norm())


def close(name, got, ref, dtype):
    once = off(ref.to(dtype), ref)
    unit = ref / ref.abs().max()  # values below 2^-14 of the largest hardly count in the norm
    step = off(unit.to(dtype), unit)
    bound = 1.1 * math.sqrt(once ** 2 + 2 * step ** 2)
    assert off(got, ref) <= bound, f"{name}: {off(got, ref):.2e} against {bound:.2e} (rounded once {once:.2e})"


@pytest.mark.parametrize("size", [1e3, 1.0, 1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_relative_error(shape, dtype, size):
    x = inputs(shape, dtype, size)
    ref, _ = window_reference(*x, *shape[5:])
    for name, got, want in zip(("dq", "dk", "dv"), gradients(*x, *shape[5:]), ref[2:]):
        close(name, got, want, dtype)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=str)
def test_one_token_with_a_large_cotangent(shape):
    """The others' gradients keep their accuracy beside it."""
    N, window, sinks = shape[1], shape[5], shape[6]
    q, k, v, dout = inputs(shape, F16, 1e-3)
    at = N // 3
    dout[:, at] *= 1e3
    ref, _ = window_reference(q, k, v, dout, window, sinks)
    dq, dk, dv = gradients(q, k, v, dout, window, sinks)
    rest = [i for i in range(N) if i != at]
    close("dq", dq[:, rest], ref[2][:, rest], F16)
    close("dk", dk[:, at + 1:], ref[3][:, at + 1:], F16)  # keys it does not see
    close("dv", dv[:, at + 1:], ref[4][:, at + 1:], F16)
    v[:, at] *= 100  # and a large value row
    ref, _ = window_reference(q, k, v, dout, window, sinks)
    dq, dk, dv = gradients(q, k, v, dout, window, sinks)
    unseen = list(range(at)) + list(range(at + window, N))
    close("dq", dq[:, unseen], ref[2][:, unseen], F16)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=str)
def test_zero_and_infinite_cotangents(shape):
    N, window, sinks = shape[1], shape[5], shape[6]
    q, k, v, dout = inputs(shape, F16, 1e-4)
    for g in gradients(q, k, v, torch.zeros_like(dout), window, sinks):
        assert bool((g == 0).all())
    for g in gradients(q, k, torch.zeros_like(v), dout, window, sinks)[:2]:
        assert bool((g == 0).all())
    ref, _ = window_reference(q, k, v, dout, window, sinks)
    at = N // 2
    dout[:, at, 0, 3] = float("inf")
    dq = gradients(q, k, v, dout, window, sinks)[0]
    rest = [i for i in range(N) if i != at]
    close("dq", dq[:, rest], ref[2][:, rest], F16)


@pytest.mark.parametrize("shape", SHAPES[:2], ids=str)
def test_a_captured_step_takes_cotangents_of_other_sizes(shape):
    q, k, v, dout = inputs(shape, F16, 1.0)
    graph = torch.cuda.CUDAGraph()
    gradients(q, k, v, dout, *shape[5:])
    out, lse = bd.window_attn(q, k, v, *shape[5:])
    with torch.cuda.graph(graph):
        captured = bd.window_attn_bwd(q, k, v, out, lse, dout, *shape[5:])
    for size in (1.0, 1e-4, 100.0, 1e-4):
        dout.copy_(inputs(shape, F16, size, seed=8)[3])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, bd.window_attn_bwd(q, k, v, out, lse, dout, *shape[5:])):
            assert torch.equal(a, b)
    assert bd.longnet_last_device_status() == 0
