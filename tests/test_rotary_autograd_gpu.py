"""GPU tests of rotary under autograd: gradients against the formula's and against differences of it, whatever part of the
results is used.  Bounds as in tests/test_paged_gpu.py.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import paged
from test_paged_gpu import DTYPES, built, freqs_of, i32, near, np64, randn  # noqa: F401

pytestmark = pytest.mark.gpu

T, D, R, BASE = 9, 64, 32, 1e3


def leaf(heads, dtype, seed):
    return randn((T, heads, D), dtype, seed).requires_grad_()


def back(g, pos, neighbours, inverse):
    return paged.rotary(np64(g), np64(pos)[None], freqs_of(R, BASE), [0] * (R // 2), neighbours, not inverse)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradients_of_queries_and_keys(dtype, neighbours, inverse):
    q, k, pos = leaf(4, dtype, 1), leaf(2, dtype, 2), torch.arange(T, dtype=torch.int32, device="cuda") * 7 - 3
    plan = gdn.rotary_plan(R, BASE, neighbours=neighbours)
    qo, ko = gdn.rotary(q, k, pos, plan, inverse=inverse)
    with torch.no_grad():
        want = gdn.rotary(q, k, pos, plan, inverse=inverse)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and not want[0].requires_grad
    gq, gk = randn(qo.shape, dtype, 3), randn(ko.shape, dtype, 4)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
    near(dq, back(gq, pos, neighbours, inverse), np64(gq), R, neighbours)
    near(dk, back(gk, pos, neighbours, inverse), np64(gk), R, neighbours)


def test_gradients_against_differences():
    q, pos, plan = leaf(1, "f32", 5), i32(list(range(T))), gdn.rotary_plan(R, BASE)
    y = randn(q.shape, "f32", 6)
    (gdn.rotary(q, None, pos, plan)[0] * y).sum().backward()
    loss = lambda z: (paged.rotary(z, np64(pos)[None], freqs_of(R, BASE), [0] * (R // 2)) * np64(y)).sum()  # noqa: E731
    x, h = np64(q), 1e-4
    for i in range(0, T * D, 37):
        e = np.zeros(T * D)
        e[i] = h
        e = e.reshape(x.shape)
        assert abs((loss(x + e) - loss(x - e)) / (2 * h) - float(q.grad.flatten()[i])) <= 1e-5


def test_parts_that_are_not_used_or_need_none():
    q, k, pos, plan = leaf(4, "f32", 1), leaf(2, "f32", 2), i32(list(range(T))), gdn.rotary_plan(R, BASE)
    one = torch.ones((T, 4, D), device="cuda")
    want = back(one, pos, False, False)
    gdn.rotary(q, k, pos, plan)[0].sum().backward()            # an expanded gradient, and none for the keys
    near(q.grad, want, np64(one), R, False)
    assert k.grad is None
    q.grad = None
    gdn.rotary(q, k, pos, plan)[1].sum().backward()
    near(k.grad, want[:, :2], np64(one)[:, :2], R, False)
    assert q.grad is None
    k.grad = None
    qo, ko = gdn.rotary(q.detach(), k, pos, plan)              # frozen queries
    (qo.sum() + ko.sum()).backward()
    near(k.grad, want[:, :2], np64(one)[:, :2], R, False)
    (gdn.rotary(q, None, pos, plan)[0][:, :, 1:] * 1.0).sum().backward()       # rows cut at odd places
    assert torch.isfinite(q.grad).all()


def test_a_gradient_of_the_gradient():
    """<rotary(x), y> is linear in y: its gradient's gradient is the turn of what it is multiplied by."""
    q, y, pos, plan = leaf(2, "f32", 1), leaf(2, "f32", 2), i32(list(range(T))), gdn.rotary_plan(R, BASE)
    dq, = torch.autograd.grad(gdn.rotary(q, None, pos, plan)[0], q, y, create_graph=True)
    z = randn(dq.shape, "f32", 3)
    dy, = torch.autograd.grad(dq, y, z)
    near(dy, back(z, pos, False, True), np64(z), R, False)


def test_given_outputs_and_other_streams():
    q, k, pos, plan = leaf(4, "bf16", 1), leaf(2, "bf16", 2), i32(list(range(T))), gdn.rotary_plan(R, BASE)
    out = torch.empty_like(q, requires_grad=False)
    assert not gdn.rotary(q, k, pos, plan, q_out=out)[0].requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qo, ko = gdn.rotary(q, k, pos, plan, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = randn(qo.shape, "bf16", 3)
    dq, = torch.autograd.grad(qo, q, g)
    torch.cuda.synchronize()
    assert torch.equal(qo, out)
    near(dq, back(g, pos, False, False), np64(g), R, False)


def test_a_captured_training_step():
    pos, plan = i32(list(range(T))), gdn.rotary_plan(R, BASE)
    q, g = leaf(4, "bf16", 1), randn((T, 4, D), "bf16", 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            q.grad = None
            gdn.rotary(q, None, pos, plan)[0].backward(g)
    torch.cuda.current_stream().wait_stream(s)
    q.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.rotary(q, None, pos, plan)[0].backward(g)
    g.copy_(randn(g.shape, "bf16", 7))
    graph.replay()
    torch.cuda.synchronize()
    near(q.grad, back(g, pos, False, False), np64(g), R, False)
