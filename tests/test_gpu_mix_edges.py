"""GPU tests of the gated recurrence, the head norm with rotation and the clipping where a lost term or a value that is not
finite would pass the operators' other tests.  Tolerances as there (the oracle's bounds), or exact."""
import pytest
import torch

from tests.test_gpu_mix_rotary import S, check, ints, rand  # noqa: F401 (S: the fixture)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------ rotation --
# heads that fill no whole batch of lanes; vector forms of both pair layouts, value by value, the ring, heads above 256
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 3, 5])
@pytest.mark.parametrize("T,B,D,rot,inter", [
    (5, 3, 32, 32, False), (5, 3, 64, 64, False), (4, 3, 128, 64, True), (6, 2, 34, 20, False), (5, 3, 100, 98, True),
    (5, 2, 264, 128, False), (613, 2, 64, 64, False), (613, 2, 128, 128, True)])
def test_gradient_without_eps(S, T, B, H, D, rot, inter, dtype):
    q, k = rand(1, T, B, H, D, dtype=dtype, scale=3), rand(2, T, B, 1 + H % 3, D, dtype=dtype)
    w = 1 + rand(3, 2, D, scale=0.2)
    check(S, q, k, w[0], w[1], S.rotary_frequencies(rot), ints(list(range(7, 7 + B))), inter, dtype, eps=0.0)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("D", [264, 1000, 34, 128])
def test_without_norm_the_gradient_does_not_look_at_x(S, D, T):
    f = S.rotary_frequencies(D // 4 * 2)
    q, d = rand(1, T, 2, 3, D, dtype="bf16"), rand(2, T, 2, 3, D, dtype="bf16")
    bad = torch.full_like(q, NAN)
    bad[::2] = INF
    a, b = (S.head_norm_rotary_backward(x, x, None, None, f, None, d, d) for x in (q, bad))
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["dk"], b["dk"]) and torch.isfinite(b["dq"]).all()
