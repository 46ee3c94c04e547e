"""GPU tests of the common norm and the clipping against fp64.  The norm: squares are summed in fp32 over at most 32
values (a sum's relative error is at most 32 roundings), in fp64 beyond, so its root is off by at most 16 2^-24 and its
own rounding.  A clipped value: the factor's rounding and two products', 4 2^-24, and half a step of its type."""
import math

import numpy as np
import pytest
import torch

from oracle import mix_oracle as O

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def S():
    from sequential_rnn_gb300 import build
    build.build()
    import sequential_rnn_gb300 as S
    return S


def rand(seed, *shape, dtype=torch.float32, scale=1.0):
    x = np.random.default_rng(seed).normal(size=shape) * scale
    return torch.from_numpy(np.asarray(x, np.float32)).to("cuda", dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def check_norm(norm, want):
    if want > torch.finfo(torch.float32).max * (1 + 2.0 ** -25):  # no fp32 number: rounds to infinity
        assert norm.item() == float("inf")
    else:
        assert abs(norm.item() - want) <= 17 * 2.0 ** -24 * want + 2.0 ** -149


def check(S, grads, limit):
    old = [np64(g) for g in grads]
    want, scaled = O.clip(old, limit)
    check_norm(S.grad_norm(grads), want)
    for g, o in zip(grads, old):
        assert np.array_equal(np64(g), o)
    norm = S.clip_grad_norm(grads, limit)
    assert norm.shape == () and norm.dtype == torch.float32
    check_norm(norm, want)
    for g, s in zip(grads, scaled):
        tiny = 2.0 ** -149 if g.dtype == torch.float32 else 2.0 ** -134
        assert (np.abs(np64(g) - s) <= (HALF[g.dtype] + 24 * 2.0 ** -24) * np.abs(s) + tiny).all()


BF, F = torch.bfloat16, torch.float32


# around a vector, a thread's share, a unit (4096 fp32, 8192 bf16 values) and several
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 255, 1024, 4095, 4096, 4097, 8192, 8193, 100003])
def test_sizes(S, n, dtype):
    check(S, [rand(n, n, dtype=dtype)], 0.5)


def test_many_tensors(S):
    """More than one launch's table, types mixed, empty ones among them."""
    g = [rand(i, (i * 37) % 411, 1 + i % 3, dtype=BF if i % 3 else F) for i in range(700)]
    check(S, g, 2.0)
    check(S, g[:256], 0.1)
    check(S, g[:257], 0.01)


def test_layer_gradients(S):
    check(S, [rand(1, 2304, 768, dtype=BF), rand(2, 6, 128, 384), rand(3, 6, 384), rand(4, 768), rand(5, 1)], 1.0)


def test_more_units_than_ctas(S):
    g = [rand(1, 5_000_001, dtype=BF), rand(2, 3_000_001)]
    check(S, g, 1.0)


@pytest.mark.parametrize("off", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [BF, F])
def test_unaligned_views(S, off, dtype):
    whole = rand(1, 20000, dtype=dtype)
    old = whole.clone()
    check(S, [whole[off:9001 + off], whole[10001:10001 + off]], 0.25)
    assert torch.equal(whole[:off], old[:off]) and torch.equal(whole[9001 + off:10001], old[9001 + off:10001])


def test_dense_orders(S):
    check(S, [rand(1, 30, 40).t(), rand(2, 4, 5, 6, dtype=BF).permute(2, 0, 1)], 0.5)


def test_below_the_limit_nothing_changes(S):
    g = [rand(1, 1000), rand(2, 1000, dtype=BF)]
    old = [x.clone() for x in g]
    n = S.grad_norm(g).item()
    for limit in (n * 1.001, 1e30, float("inf")):
        S.clip_grad_norm(g, limit)
        assert all(torch.equal(a, b) for a, b in zip(g, old))
    S.clip_grad_norm(g, 0.0)
    assert all((x == 0).all() for x in g)
    S.clip_grad_norm(g, 0.0)  # a norm of zero


@pytest.mark.parametrize("scale", [1e30, 3e37, 1e-25, 1e-38])
def test_squares_that_leave_fp32(S, scale):
    g = [rand(1, 5000, scale=scale), rand(2, 777), torch.zeros(5000, device="cuda")]
    check(S, g, 1.0 if scale > 1 else 1e-3)
    check(S, [rand(3, 5000, scale=scale), rand(4, 300, dtype=BF, scale=scale)], 0.5 * scale)


def test_factor_below_fp32(S):
    g = [torch.full((64,), 3e38, device="cuda"), rand(1, 64)]
    check(S, g, 1e-6)
    assert g[0].abs().max().item() == pytest.approx(1e-6 / 8, rel=1e-5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_norm_that_is_not_finite_changes_nothing(S, bad, dtype):
    g = [rand(1, 9000, dtype=dtype), rand(2, 100)]
    g[0][8999] = bad
    old = [x.clone() for x in g]
    n = S.clip_grad_norm(g, 1.0).item()
    assert math.isnan(n) if math.isnan(bad) else n == float("inf")
    for a, b in zip(g, old):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_none_empty_and_no_tensors(S):
    x = rand(1, 10)
    check(S, [x], 0.5)
    assert S.grad_norm([None, x, None]).item() == S.grad_norm([x]).item()
    assert S.grad_norm([]).item() == 0.0 and S.clip_grad_norm((torch.empty(0, device="cuda"),), 1.0).item() == 0.0
    assert S.clip_grad_norm([], 1.0).item() == 0.0


def test_captured_on_a_side_stream_and_repeated(S):
    g = [rand(1, 300_000, dtype=BF), rand(2, 70_001)]
    keep = [x.clone() for x in g]
    a = S.clip_grad_norm(g, 1.0)
    first = [x.clone() for x in g]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = S.clip_grad_norm(g, 1.0)
    for _ in range(2):
        for x, k in zip(g, keep):
            x.copy_(k)
        graph.replay()
        assert norm.item() == a.item() and all(torch.equal(x, y) for x, y in zip(g, first))
    for x, k in zip(g, keep):
        x.copy_(k)
    side.wait_stream(torch.cuda.current_stream())
    n = S.clip_grad_norm(g, 1.0, stream=side)
    side.synchronize()
    assert n.item() == a.item() and all(torch.equal(x, y) for x, y in zip(g, first))


def test_refusals(S):
    x = rand(1, 64)
    with pytest.raises(S.RnnError):
        S.clip_grad_norm([x, x], 1.0)
    with pytest.raises(S.RnnError):
        S.clip_grad_norm([x[32:], rand(2, 4), x[:33]], 1.0)
    assert S.grad_norm([x, x]).item() == pytest.approx(2 ** 0.5 * S.grad_norm([x]).item(), rel=1e-6)
    with pytest.raises(S.RnnError):
        S.clip_grad_norm([x], -1.0)
    with pytest.raises(S.RnnError):
        S.clip_grad_norm([x], float("nan"))
    with pytest.raises(ValueError):
        S.clip_grad_norm([x[::2]], 1.0)
    with pytest.raises(ValueError):
        S.clip_grad_norm([x.expand(2, 64)], 1.0)
    with pytest.raises(TypeError):
        S.clip_grad_norm([x.half()], 1.0)
    with pytest.raises(TypeError):
        S.clip_grad_norm([x], None)
