"""bf16 verify attention over the block-scaled cache: what its operands' codes may lose.

Two positions share a row's weight, so that no averaging over positions hides what one weight or one query value loses."""
import numpy as np
import pytest
import torch

from bs8_harness import Bs8Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _half_step(x):
    """Half of bf16's step (8 significant bits) at each value."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def _second_of_two(T, keys, rest, q, seed):
    """16 slots of T + 2 positions, whose keys are keys[0], keys[1] and then `rest` and whose
    values are zero but for the second's: every row is w v, w the second position's weight.  Returns the call's rows and the exact ones,
    [16, T, 8, 256] in float64."""
    slots, L = 16, T + 2
    cache = Bs8Cache([L] * slots, kv=1)

    def shape(k, v, b):
        k = np.zeros_like(k)
        k[0, 0], k[1, 0], k[2:, 0] = keys[0], keys[1], rest
        v[0], v[2:] = 0.0, 0.0
        return k, v

    cache.fill([L] * slots, seed=seed, shape=shape)
    got = cache.verify([L] * slots, [T] * slots, q).double().cpu().numpy().reshape(slots, T, 8, 256)
    s = q.double().cpu().numpy().reshape(slots, T, 8, 256) @ cache.values(0, L)[0][0].T / 16.0
    s = np.where(np.arange(L) <= 2 + np.arange(T)[:, None, None], s, -np.inf)
    p = np.exp(s - s.max(axis=3, keepdims=True))
    w = p[..., 1] / p.sum(axis=3)
    v = np.stack([cache.values(b, L)[1][0, 1] for b in range(slots)])
    return got, w[..., None] * v[:, None, None, :]


def _within(got, want, relative):
    tol = relative * np.abs(want)
    assert np.all(np.abs(got - want) <= tol + _half_step(np.abs(want) + tol))


@pytest.mark.parametrize("T", [1, 4, 6, 8])
def test_weights_hold_eleven_bits(T):
    """The weight is rounded to fp16, by 2^-11 of it at most, and its codes hold that number.  The scores (8 at most) are off by
    2^-22 (|s| + max |s|) and the exponentials by 2^-22: 2^-17 in all, for weight and row sum."""
    one = np.eye(256, dtype=np.float32)[0]
    gen = torch.Generator(device="cuda").manual_seed(71)
    q = torch.zeros((16 * T, 8, 256), device="cuda")
    q[:, :, 0] = 16.0 * (0.25 + 0.75 * torch.rand((16 * T, 8), generator=gen, device="cuda"))
    q = q.to(torch.bfloat16)
    _within(*_second_of_two(T, (8.0 * one, 4.0 * one), -64.0 * one, q, 70), 2.0 ** -11 + 2.0 ** -17)


@pytest.mark.parametrize("T", [1, 4, 6, 8])
def test_queries_next_to_a_large_value(T):
    """One value of a query row is 2^10.5 to 2^11.5 times the others, at a dim where the keys are zero: the others count with all of
    their 8 bits (two codes hold them down to 2^-14 of the largest value).

    All small values of a row are alike, so that what one loses all lose.  The scores are off by 2^-22 times the sum of their
    products' magnitudes and by 2^-22 (|s| + max |s|), all of them 10 at most: 2^-16 in all, for weight and row sum.  The weight is
    rounded to fp16 as above."""
    many = np.ones(256, np.float32)
    many[0] = 0.0
    gen = torch.Generator(device="cuda").manual_seed(73)
    q = (2.0 ** -11.5 * (1.0 + torch.rand((16 * T, 8, 1), generator=gen, device="cuda"))).expand(-1, -1, 256).clone()
    q[:, :, 0] = 1.0
    q = q.to(torch.bfloat16)
    _within(*_second_of_two(T, (896.0 * many, 448.0 * many), -896.0 * many, q, 72), 2.0 ** -11 + 2.0 ** -16)
