"""Sliding-window attention with sinks against its 64-bit form: forward and
backward, every dtype and kernel family, at the lengths, windows, sinks and
head layouts where tiles, blocks and groups end."""
import pytest
import torch

from sparse_long_sequence_attn_b200 import binding as bd
from tests.window_reference import window_reference, within

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
AUTO, SIMT = bd.LONGNET_IMPL_AUTO, bd.LONGNET_IMPL_SIMT

# B, N, H, Hkv, D, window, sinks
SHAPES = [
    (1, 1, 1, 1, 16, 1, 0),
    (2, 2, 2, 1, 32, 1, 5),
    (1, 63, 3, 3, 64, 7, 2),
    (1, 64, 4, 2, 128, 64, 0),
    (2, 65, 2, 2, 16, 64, 1),
    (1, 129, 6, 2, 64, 1, 129),
    (3, 128, 2, 1, 128, 300, 4),
    (1, 257, 5, 1, 64, 100, 65),
    (1, 333, 3, 1, 32, 33, 4),
    (1, 700, 7, 1, 64, 128, 3),
    (1, 900, 2, 1, 128, 129, 130),
    (1, 1500, 2, 2, 64, 90, 16),
    (1, 1200, 2, 1, 16, 2, 1),
    (1, 520, 24, 1, 32, 250, 0),
    (1, 1000, 1, 1, 128, 1000, 0),
    (1, 2600, 1, 1, 64, 40, 2600),
    (2, 70, 80, 1, 16, 30, 3),    # more shared heads than a streamed block has rows
    (1, 40, 130, 1, 32, 17, 0),   # and than a tile has
    (2, 1030, 8, 4, 64, 515, 1),
    (1, 5000, 2, 1, 32, 70, 300),
]


def inputs(B, N, H, Hkv, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda h: torch.randn((B, N, h, D), generator=g, device="cuda").to(dtype)  # noqa: E731
    return mk(H), mk(Hkv), mk(Hkv), mk(H)


def guarded(t):
    """A NaN-filled tensor like t inside a larger NaN-filled one."""
    pad = 256
    buf = torch.full((t.numel() + 2 * pad,), float("nan"), dtype=t.dtype, device=t.device)
    return buf, buf[pad:pad + t.numel()].view(t.shape)


def run(q, k, v, dout, window, sinks, impl):
    bufs, views = zip(*(guarded(z) for z in (q, torch.empty(q.shape[0], q.shape[2], q.shape[1], device="cuda"),
                                             q, k, k)))
    out, lse, dq, dk, dv = views
    bd.longnet_window_attn_fwd(q, k, v, out, lse, window, sinks, impl)
    B, N, H, D = q.shape
    n = bd.longnet_window_bwd_workspace_bytes(B, N, H, k.shape[2], D, window, sinks, q.dtype)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    bd.longnet_window_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, window, sinks, ws[:n], impl)
    assert bd.longnet_last_device_status() == 0
    assert bool((ws[n:] == 255).all()), "write past the workspace"
    for b, t in zip(bufs, views):
        assert bool(b[:256].isnan().all()) and bool(b[-256:].isnan().all()), "write outside an output"
    return out, lse, dq, dk, dv


@pytest.mark.parametrize("impl", [AUTO, SIMT])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, dtype, impl):
    if impl == SIMT and dtype != F32 and shape[1] > 800:
        pytest.skip("the 16-bit loads of this family are covered by the shorter shapes")
    B, N, H, Hkv, D, window, sinks = shape
    x = inputs(B, N, H, Hkv, D, dtype, 1 + N)
    ref, bound = window_reference(*x, window, sinks)
    got = run(*x, window, sinks, impl)
    for name, a, r, b in zip(("out", "lse", "dq", "dk", "dv"), got, ref, bound):
        within(name, a, r, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_again(dtype):
    x = inputs(2, 1500, 6, 2, 64, dtype, 5)
    a, b = (run(*x, 100, 70, AUTO) for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_gradients_against_differences():
    q, k, v, dout = (z.double() for z in inputs(1, 150, 4, 2, 32, F32, 9))
    args = [z.float().requires_grad_() for z in (q, k, v)]
    out = bd.window_attention(*args, 40, 3)
    grads = torch.autograd.grad(out, args, dout.float())
    g = torch.Generator(device="cuda").manual_seed(3)
    from tests.window_reference import attend

    def f(q, k, v):
        return sum((attend(q[0, :, h], k[0, :, h // 2], v[0, :, h // 2], 0, 40, 3)[0] * dout[0, :, h]).sum()
                   for h in range(4))

    for i, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = [q, k, v], [q, k, v]
        plus[i], minus[i] = plus[i] + 1e-5 * d, minus[i] - 1e-5 * d
        want = float((f(*plus) - f(*minus)) / 2e-5)
        have = float((grad.double() * d).sum())
        # |grad| |d| times the fp32 error of a gradient
        assert abs(have - want) <= 1e-4 * float(grad.double().norm() * d.norm()), (i, have, want)


def test_autograd_op_takes_strided_inputs_and_shared_leaves():
    x = torch.randn((2, 90, 3, 4, 64), device="cuda", dtype=BF16, requires_grad=True)  # fused qkv
    q, k, v = x.unbind(2)
    out = bd.window_attention(q, k, v, 30, 2)
    out.float().square().sum().backward()
    dout = (2 * out.detach().float()).to(BF16)
    ref, bound = window_reference(*(z.detach().contiguous() for z in (q, k, v)), dout, 30, 2)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(name, x.grad[:, :, i], ref[2 + i], bound[2 + i])


def test_expanded_cotangent_and_frozen_keys():
    q, k, v, _ = inputs(1, 70, 2, 2, 32, F16, 4)
    q.requires_grad_()
    out = bd.window_attention(q, k, v, 20, 0)
    out.sum().backward()  # the cotangent is one value, expanded
    ref, bound = window_reference(q.detach(), k, v, torch.ones_like(q), 20, 0)
    within("dq", q.grad, ref[2], bound[2])
    assert k.grad is None


def test_another_stream_and_a_captured_graph():
    q, k, v, dout = inputs(1, 600, 4, 2, 64, BF16, 8)
    want = run(q, k, v, dout, 100, 4, AUTO)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = bd.window_attn(q, k, v, 100, 4)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graphs = []
    for _ in range(2):  # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, lse = bd.window_attn(q, k, v, 100, 4)
            grads = bd.window_attn_bwd(q, k, v, out, lse, dout, 100, 4)
        graphs.append((g, (out, lse, *grads)))
    q2, k2, v2, dout2 = inputs(1, 600, 4, 2, 64, BF16, 18)
    want2 = run(q2, k2, v2, dout2, 100, 4, AUTO)
    for t, n in zip((q, k, v, dout), (q2, k2, v2, dout2)):
        t.copy_(n)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want2))


def test_later_rows_do_not_reach_earlier_ones():
    q, k, v, dout = inputs(1, 300, 2, 1, 64, BF16, 2)
    a, _ = bd.window_attn(q, k, v, 50, 4)
    k[:, 200:], v[:, 200:], q[:, 200:] = 300.0, -300.0, 300.0
    b, _ = bd.window_attn(q, k, v, 50, 4)
    assert torch.equal(a[:, :200], b[:, :200])


@pytest.mark.parametrize("scale", [30.0, 200.0])
def test_scores_far_apart(scale):
    """One key takes the whole softmax, far keys underflow: out is that key's value row."""
    q, k, v, dout = inputs(1, 260, 2, 2, 64, BF16, 6)
    q = (q.float() * scale).to(BF16)
    ref, bound = window_reference(q, k, v, dout, 120, 8)
    out, lse = bd.window_attn(q, k, v, 120, 8)
    # a score's fp32 error grows with the score: |s| FP32 / 4 beside the bound of its unit size
    within("out", out, ref[0], bound[0] + 1e-5 * scale * 4)
    within("lse", lse, ref[1], bound[1] + 1e-6 * ref[1].abs())


def test_given_stream():
    """Outputs and workspaces belong to the stream that the call is given."""
    q, k, v, dout = inputs(1, 400, 4, 2, 64, BF16, 3)
    want = run(q, k, v, dout, 60, 2, AUTO)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, lse = bd.window_attn(q, k, v, 60, 2, stream=side)
        grads = bd.window_attn_bwd(q, k, v, out, lse, dout, 60, 2, stream=side)
        junk = [torch.full_like(q, 9.0) for _ in range(4)]  # what the freed workspace must not be given to meanwhile
    side.synchronize()
    del junk
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_backward_of_scores_far_apart(dtype, D):
    """Scores of some hundreds: lse is far from 0, and one or two keys take a row."""
    scale = 20.0
    q, k, v, dout = inputs(1, 300, 4, 2, D, dtype, 7)
    q = (q.float() * scale).to(dtype)
    ref, bound = window_reference(q, k, v, dout, 120, 8)
    got = run(q, k, v, dout, 120, 8, AUTO)
    # a score of |s| <= 6 sqrt(D) scale / 4 carries its fp32 error, 2^-22 of it at most, into P, which
    # the products with terms of up to 5 (v, dout) or 5 scale (q) then spread over a row's or key's terms
    slack = 2.0 ** -22 * 6 * D ** 0.5 * scale / 4 * 5 * 5 * D ** 0.5
    for name, a, r, b in zip(("out", "lse", "dq", "dk", "dv"), got, ref, bound):
        within(name, a, r, b + (1e-6 * r.abs() if name == "lse" else slack * (scale if name == "dk" else 1)))


@pytest.mark.parametrize("shape", [
    (1, 1578, 3, 1, 64, 90, 16),    # the largest grid of 16-row tiles with a group of 3
    (1, 1579, 3, 1, 64, 90, 16),    # and one row past it: tiles of 64
    (1, 2500, 2, 1, 128, 300, 70),
    (3, 800, 4, 2, 16, 65, 700),
    (1, 2400, 1, 1, 128, 17, 1200),  # sinks over many tiles of 16 keys
    (1, 330, 1, 1, 64, 400, 270),
], ids=str)
def test_fp32_tiles_of_both_sizes(shape):
    B, N, H, Hkv, D, window, sinks = shape
    x = inputs(B, N, H, Hkv, D, F32, 2 + N)
    ref, bound = window_reference(*x, window, sinks)
    for name, a, r, b in zip(("out", "lse", "dq", "dk", "dv"), run(*x, window, sinks, AUTO), ref, bound):
        within(name, a, r, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_training_step(dtype):
    """Forward and backward through autograd in one graph; the eager warm-up is dropped before the capture."""
    q, k, v, dout = inputs(2, 300, 4, 2, 64, dtype, 12)
    leaves = [z.clone().requires_grad_() for z in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.window_attention(*leaves, 70, 4).backward(dout)
    torch.cuda.current_stream().wait_stream(side)
    for z in leaves:
        z.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bd.window_attention(*leaves, 70, 4)
        out.backward(dout)
    new = inputs(2, 300, 4, 2, 64, dtype, 13)
    with torch.no_grad():
        for z, n in zip((*leaves, dout), new):
            z.copy_(n)
    for _ in range(2):  # the second replay writes the same gradients again, it does not add to them
        graph.replay()
    torch.cuda.synchronize()
    want = run(*new, 70, 4, AUTO)
    assert torch.equal(out, want[0])
    for z, w in zip(leaves, want[2:]):
        assert torch.equal(z.grad, w)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", [
    (1, 1100, 4, 1, 64, 1, 0),       # one block a row tile, then one more where it ends
    (1, 900, 3, 1, 128, 700, 0),     # tiles of 42 tokens: runs that begin blocks apart
    (2, 640, 2, 2, 64, 513, 64),     # past the lengths whose delta has a pass of its own
    (1, 1300, 1, 1, 32, 600, 129),
    (1, 85, 3, 3, 16, 85, 0),        # the second tile has no keys of its own
], ids=str)
def test_backward_runs_of_blocks(shape, dtype):
    """The two tiles of a block share a ring of streamed blocks, each over a run of its own."""
    B, N, H, Hkv, D, window, sinks = shape
    x = inputs(B, N, H, Hkv, D, dtype, 3 + N)
    ref, bound = window_reference(*x, window, sinks)
    for name, a, r, b in zip(("out", "lse", "dq", "dk", "dv"), run(*x, window, sinks, AUTO), ref, bound):
        within(name, a, r, b)
