"""Block-scaled verify attention over shares of many tiles: scores far from zero, maxima that rise, pages out of range in front.

A CTA takes several tiles of one context only where a call has more tiles than the GPU has SMs, so 160 slots share the pages of one
context here; their shares begin and end at different tiles, and outputs of several slots are compared with float64."""
import numpy as np
import pytest
import torch

from bs8_harness import Bs8Cache, check, i32, offsets, queries
from speculative_verify_attention_q3kv_gb300 import _lib, api
from test_gpu_bs8 import KINDS, _late, _quiet, _rising, _scales

pytestmark = pytest.mark.gpu
SLOTS = 160
# Tokens of every row configuration: 16, 32, 48, 64 rows, two chunks of 48 and of 64 (float32: 16, 32, two to four chunks of 32)
TOKENS = [1, 4, 6, 8, 12, 16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _shared(cache, L, T, q, impl):
    """One context and its queries [T, heads, 256], as every slot's; the slots' outputs [SLOTS, T, heads, 256]."""
    out = torch.full((SLOTS * T, *q.shape[1:]), 77.0, dtype=q.dtype, device="cuda")
    api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table.repeat(SLOTS, 1), i32([L] * SLOTS), i32([T] * SLOTS), offsets([T] * SLOTS),
                        L, T, 0, q.repeat(SLOTS, 1, 1), out, cache.workspace([L], [T], SLOTS), impl, cache.status)
    return out.view(SLOTS, T, *q.shape[1:])


def _check_some(out, q, cache, L, T, kind, hidden=None):
    for b in (0, 1, 2, 77, 78, SLOTS - 1):
        check(out[b], q, cache, [L], [T], kind, hidden=hidden)


def _at_score(score, v_scale=1.0, spread=0.02):
    """Keys whose scores with queries around 1 lie around `score` (natural units), a little apart from each other."""
    def shape(k, v, b):
        return (score * 16 / 256 * (1.0 + spread * k)).astype(np.float32), (v_scale * v).astype(np.float32)
    return shape


@pytest.mark.parametrize("score,v_scale", [(-90.0, 1.0), (-300.0, 1.0), (-60.0, 2.0 ** -55), (90.0, 1.0), (300.0, 2.0 ** -55)])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
@pytest.mark.parametrize("L,T", [(1, 1), (40, 4), (300, 6)])
def test_scores_far_from_zero(L, T, kind, dtype, impl, score, v_scale):
    """A softmax does not change with its scores' level: one position alone gives its V, several tiles their weighted mean."""
    cache = Bs8Cache([L], kv=1)
    cache.fill([L], seed=50, shape=_at_score(score, v_scale))
    q = (1.0 + 0.05 * queries(T, 1, 51, torch.float32)).to(dtype)
    check(cache.verify([L], [T], q, impl=impl), q, cache, [L], [T], kind)


@pytest.mark.parametrize("score,v_scale", [(-90.0, 1.0), (-300.0, 1.0), (-60.0, 2.0 ** -55)])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_scores_far_from_zero_in_long_shares(kind, dtype, impl, score, v_scale):
    L, T = 1100, 6
    cache = Bs8Cache([L], kv=1)
    cache.fill([L], seed=52, shape=_at_score(score, v_scale))
    q = (1.0 + 0.05 * queries(T, 1, 53, torch.float32)).to(dtype)
    _check_some(_shared(cache, L, T, q, impl), q, cache, L, T, kind)
    assert int(cache.status) == 0


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_zero_values_in_front_of_the_others(kind, dtype, impl):
    """A first tile of zero V has the smallest scales there are, 2^-64: with scores of -45 its largest weight is below 2^-126."""
    L, T = 700, 4
    cache = Bs8Cache([L], kv=1)

    def shape(k, v, b):
        k, v = _at_score(-45.0)(k, v, b)
        v[:128] = 0.0
        return k, v

    cache.fill([L], seed=54, shape=shape)
    q = (1.0 + 0.05 * queries(T, 1, 55, torch.float32)).to(dtype)
    _check_some(_shared(cache, L, T, q, impl), q, cache, L, T, kind)
    check(cache.verify([L], [T], q, impl=impl), q, cache, [L], [T], kind)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("score,v_scale", [(-14.0, 1.0), (0.0, 1e-5), (-90.0, 1.0), (40.0, 1.0)])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_pages_out_of_range_in_front_of_a_share(kind, dtype, impl, score, v_scale, T):
    """The first page and one further back are hidden; the visible tiles behind them count as if those were not there."""
    L = 1100
    cache = Bs8Cache([L], kv=1)
    cache.fill([L], seed=56, shape=_at_score(score, v_scale, spread=0.5 / max(1.0, abs(score)) if score else 0.0))
    q = (1.0 + 0.05 * queries(T, 1, 57, torch.float32)).to(dtype)
    hidden = np.zeros(L, bool)
    hidden[:256] = hidden[768:1024] = True
    cache.page_table[0, 0], cache.page_table[0, 3] = -1, cache.num_pages
    out = _shared(cache, L, T, q, impl)
    assert int(cache.status) == _lib.Q3KV_STATUS_BAD_PAGE
    _check_some(out, q, cache, L, T, kind, [hidden])


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_only_the_last_page_is_in_range(kind, dtype, impl):
    L, T = 1100, 5
    cache = Bs8Cache([L], kv=1)
    cache.fill([L], seed=58, shape=_at_score(-20.0))
    q = (1.0 + 0.05 * queries(T, 1, 59, torch.float32)).to(dtype)
    cache.page_table[0, :4] = -1
    _check_some(_shared(cache, L, T, q, impl), q, cache, L, T, kind, [np.arange(L) < 1024])


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("shape,scale", [(_rising, 1.5), (_rising, 6.0), (_late, 1.5), (_scales, 1.5), (_quiet, 1.5)])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_uneven_caches_in_long_shares(shape, scale, kind, dtype, impl, T):
    """The running maximum is raised within a share, several times where keys rise (scores to over 100)."""
    L = 1500
    cache = Bs8Cache([L], kv=1)
    cache.fill([L], seed=60, shape=shape)
    q = queries(T, 1, 61, dtype, scale)
    if shape is _quiet:
        q = q.float().abs().to(dtype)
    _check_some(_shared(cache, L, T, q, impl), q, cache, L, T, kind)
    assert int(cache.status) == 0


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
@pytest.mark.parametrize("kind,dtype,impl", KINDS)
def test_infinite_queries_whatever_the_scores_sign(kind, dtype, impl, inf, sign):
    """An infinity against keys of one sign makes every score the same infinity, minus infinity too: the row is NaN."""
    L, T = [300], [2]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=62, shape=lambda k, v, b: (sign * (0.5 + np.abs(k)), v))
    q = queries(2, 1, 63, dtype)
    clean = cache.verify(L, T, q, impl=impl)
    q[1, 4, 30] = inf
    out = cache.verify(L, T, q, impl=impl)
    bad = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    bad[1, 4] = True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("score", [-1e36, 1e36])
@pytest.mark.parametrize("kind,dtype,impl", KINDS)
def test_scores_near_the_ends_of_float32(kind, dtype, impl, score):
    """One position has all of the weight whatever its score: its V, off by the roundings of the weight (2^-11 as fp16), of the quotient
    and of the output."""
    cache = Bs8Cache([1], kv=1)
    cache.fill([1], seed=64, shape=lambda k, v, b: (np.full_like(k, score / 1e18 / 16), v))
    q = torch.full((1, 8, 256), 1e18, device="cuda").to(dtype)
    got = cache.verify([1], [1], q, impl=impl).double().cpu().numpy()
    v = cache.values(0, 1)[1][0, 0]
    assert np.all(np.abs(got - v) <= (2.0 ** -11 + 2.0 ** -8 + 2.0 ** -18) * np.abs(v))
