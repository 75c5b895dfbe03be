"""The bounds of the adapters' float32 sums, on the CPU: the model of a running sum
that loses bits at each step keeps within them, and longer sums, a u of two bf16
parts or its three parts in one sum do not."""
import numpy as np
import pytest
import torch

from test_gpu_adapter_sums import PARTS, SEGMENT, norm_bound

OUTPUTS = 4096


def towards_zero(v):
    """float64 cut to 24 bits."""
    m, e = np.frexp(v)
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def running_sum(terms):
    s = np.zeros(terms.shape[1])
    for t in terms:
        s = towards_zero(s + t)
    return s


def far(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


def steps(n, seed=0):
    return np.random.default_rng(seed).standard_normal((n, OUTPUTS))


@pytest.mark.parametrize("n", [PARTS, SEGMENT, 2 * SEGMENT])
def test_the_model_of_a_sum(n):
    t = steps(n)
    off = far(running_sum(t), t.sum(0))
    assert 0.5 * norm_bound(n) - 2.0 ** -22 <= off <= norm_bound(n)


def test_segments_keep_the_bound_and_one_sum_does_not():
    t = steps(8 * SEGMENT, seed=1)
    joined = np.zeros(OUTPUTS, np.float32)
    for k in range(0, len(t), SEGMENT):
        joined = joined + running_sum(t[k:k + SEGMENT]).astype(np.float32)
    assert far(joined.astype(np.float64), t.sum(0)) <= norm_bound(SEGMENT)
    assert far(running_sum(t), t.sum(0)) > norm_bound(SEGMENT)


def test_the_large_part_in_a_sum_of_three_does_not_keep_the_bound():
    # the small parts' steps cut the same running sum
    t = np.repeat(steps(SEGMENT, seed=2), 3, axis=0)
    t[1::3] *= 2.0 ** -9
    t[2::3] *= 2.0 ** -18
    assert far(running_sum(t), t.sum(0)) > norm_bound(SEGMENT)


def parts(u, k):
    got, left = torch.zeros_like(u), u.clone()
    for _ in range(k):
        p = left.bfloat16().float()
        got, left = got + p, left - p
    return got


def test_two_parts_of_u_do_not_keep_the_bound():
    g = torch.Generator().manual_seed(3)
    u = torch.randn(500, 64, generator=g)
    b = (torch.randn(64, 264, generator=g) / 8).bfloat16().double()
    want = (u.double() @ b).numpy()
    assert far((parts(u, 3).double() @ b).numpy(), want) <= 2.0 ** -24
    assert far((parts(u, 2).double() @ b).numpy(), want) > norm_bound(PARTS)
