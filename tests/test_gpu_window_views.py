"""window_attention of views that start off a 16-byte boundary, and with a
cotangent that does: a program chooses neither where its parameters lie in a
flat buffer nor where autograd cuts a gradient."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd

pytestmark = pytest.mark.gpu

N, H, Hkv, D, WINDOW, SINKS = 130, 4, 2, 32, 50, 3


def leaves(dtype):
    g = torch.Generator(device="cuda").manual_seed(6)
    return [torch.randn((1, N, h, D), generator=g, device="cuda").to(dtype) for h in (H, Hkv, Hkv)]


def step(q, k, v, head):
    """Gradients of a weighted sum over `head` (one number each) and the output, joined in one vector."""
    out = bd.window_attention(q, k, v, WINDOW, SINKS)
    joined = torch.cat([head, out.flatten()])
    w = torch.linspace(-1, 1, N * H * D, device="cuda").to(out.dtype)
    (joined * torch.cat([torch.ones_like(head), w])).sum().backward()
    return out.detach()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shift", [1, 3])
def test_views_off_the_boundary(dtype, shift):
    x = leaves(dtype)
    plain = [t.clone().requires_grad_() for t in x]
    want = step(*plain, torch.ones(8, device="cuda", dtype=dtype))  # 8 numbers: the cotangent starts at 16 bytes
    flat = torch.cat([torch.zeros(shift, device="cuda", dtype=dtype)] + [t.flatten() for t in x]).requires_grad_()
    at, views = shift, []
    for t in x:
        views.append(flat[at:at + t.numel()].view(t.shape))
        at += t.numel()
    assert views[0].data_ptr() % 16 != 0
    got = step(*views, torch.ones(shift, device="cuda", dtype=dtype))
    assert torch.equal(got, want)
    assert torch.equal(flat.grad[shift:], torch.cat([t.grad.flatten() for t in plain]))
    assert bd.longnet_last_device_status() == 0
