"""The references of the windowed and paged operators, pinned without a GPU: the mask by its
definition pair by pair, the forward and the gradients by the general oracle, the gradients also by
differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import window as ref


@pytest.mark.parametrize("Lq,Lk,window,sinks,qo,ko", [
    (7, 9, 3, 0, 2, 0), (9, 9, 1, 2, 0, 0), (6, 8, 4, 3, 10, 1), (5, 6, 2, 9, 0, 4), (4, 3, 100, 1, 0, 0)])
def test_mask_pair_by_pair(Lq, Lk, window, sinks, qo, ko):
    mask = ref.window_mask(Lq, Lk, window, sinks, qo, ko)
    for i in range(Lq):
        for j in range(Lk):
            t = (i + qo) - (j + ko)
            assert bool(mask[i, j]) == (t >= 0 and (t < window or j + ko < sinks))


def draw(B, H, Hkv, Lq, Lk, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g, dtype=torch.float64)
            for s in ((B, H, Lq, d), (B, Hkv, Lk, d), (B, Hkv, Lk, d), (B, H, Lq, d))]


def test_wide_windows_are_causal_attention():
    q, k, v, do = draw(1, 4, 2, 40, 40, 8)
    mask = ref.window_mask(40, 40, 1000)
    O, L, _ = ref.forward(q, k, v, mask, 0.3)
    O2, L2 = oracle.attention_forward(*(x.numpy() for x in (q, k, v)), 0.3, causal=True)
    assert np.allclose(O, O2, atol=1e-12) and np.allclose(L, L2, atol=1e-12)
    got = ref.backward(q, k, v, do, mask, 0.3)
    want = oracle.attention_backward(*(x.numpy() for x in (q, k, v, do)), 0.3, causal=True)
    for a, b in zip(got, want):
        assert np.allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("Lq,Lk,window,sinks,qo", [(11, 11, 4, 2, 0), (6, 9, 3, 0, 5), (5, 12, 20, 1, 7)])
def test_gradients_by_differences(Lq, Lk, window, sinks, qo):
    q, k, v, do = draw(1, 2, 1, Lq, Lk, 4, Lq)
    mask = ref.window_mask(Lq, Lk, window, sinks, qo)

    def loss(q, k, v):
        return float((ref.forward(q, k, v, mask, 0.5)[0] * do).sum())

    grads = ref.backward(q, k, v, do, mask, 0.5)[:3]
    g = torch.Generator().manual_seed(3)
    for n, grad in enumerate(grads):
        for _ in range(6):
            way = torch.randn(grad.shape, generator=g, dtype=torch.float64)
            args = [q, k, v]
            e = 1e-5
            hi = loss(*[a + e * way if i == n else a for i, a in enumerate(args)])
            lo = loss(*[a - e * way if i == n else a for i, a in enumerate(args)])
            slope = float((grad * way).sum())
            # third derivatives are of order 10 here: e^2 times that, and the
            # subtraction's 1e-15 / e
            assert abs((hi - lo) / (2 * e) - slope) <= 1e-7 * max(1.0, abs(slope))


def test_bounds_cover_a_bf16_computation():
    """The bounds hold for a computation that rounds where the kernels do."""
    q, k, v, do = (x.bfloat16().double() for x in draw(1, 2, 2, 70, 70, 16, 5))
    mask = ref.window_mask(70, 70, 20, 2)
    r = lambda x: x.bfloat16().double()  # noqa: E731
    O, L, P = ref.forward(q, k, v, mask, 0.25)
    bo, _ = ref.forward_bounds(q, k, v, mask, 0.25)
    o = r(r(P) @ v)
    assert ((o - O).abs() <= bo).all()
    D = (do * o).sum(-1, keepdim=True)
    dS = r(0.25 * P * (do @ v.transpose(-1, -2) - D))
    got = r(dS @ k), r(dS.transpose(-1, -2) @ q), r(r(P).transpose(-1, -2) @ do)
    want = ref.backward(q, k, v, do, mask, 0.25)
    bound = ref.backward_bounds(q, k, v, do, mask, 0.25)
    for a, w, b in zip(got, want, bound):
        # rows of few keys: their bound counts on the exact D
        assert ((a - w).abs()[..., 40:, :] <= b[..., 40:, :]).all()
