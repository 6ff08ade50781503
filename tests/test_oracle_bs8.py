"""Pins of the block-scaled cache's and the logits' oracles (no GPU)."""
import math

import numpy as np
import pytest

from oracle import bs8, fp8, logits


@pytest.mark.parametrize("top,e", [(0.0, -64), (448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1.0, -8), (3.5, -7),
                                   (2.0 ** -70, -64), (448 * 2.0 ** 64, 64), (1e38, 64), (math.inf, -64), (math.nan, -64)])
def test_exponent_is_the_smallest_that_holds_the_block(top, e):
    x = np.zeros((3, 256), np.float32)
    x[1, 7] = -top if top == top else top
    got = bs8.exponent(x)
    assert got == e
    if np.isfinite(top) and 0 < top <= 448 * 2.0 ** 64 and e > -64:
        v = float(abs(x[1, 7]))
        assert v <= 448 * 2.0 ** e and v > 448 * 2.0 ** (e - 1)


def test_offsets_are_a_permutation_of_the_unit():
    assert sorted(bs8._OFFSETS.ravel().tolist()) == list(range(bs8.CODE_BYTES))
    assert bs8.code_offset(0, 0) == 0 and bs8.code_offset(1, 0) == 16 and bs8.code_offset(0, 16) == 128 and bs8.code_offset(8, 0) == 2048
    assert bs8.code_offset(255, 255) == bs8.CODE_BYTES - 1


def test_block_by_hand():
    c = bs8.Cache()
    x = np.zeros((2, 256), np.float32)
    x[0, 0], x[1, 1] = 3.5, 1.0                       # e = -7: codes of 448 and 128
    c.append(x)
    assert c.exps == [-7] and c.codes[0, 0] == 0x7E and fp8.decode(c.codes[1, 1:2])[0] == 128.0
    y = np.zeros((1, 256), np.float32)
    y[0, 2] = 7.5                                     # needs e = -5: the earlier codes are divided by 4
    c.append(y)
    assert c.exps == [-5] and fp8.decode(c.codes[0, :1])[0] == 112.0 and fp8.decode(c.codes[1, 1:2])[0] == 32.0
    assert fp8.decode(c.codes[2, 2:3])[0] == 240.0
    assert c.values()[0, 0] == 3.5 and c.values()[1, 1] == 1.0 and c.values()[2, 2] == 7.5


def test_growth_rounds_only_codes_that_become_subnormal():
    rng = np.random.default_rng(0)
    c = bs8.Cache()
    c.append(rng.standard_normal((5, 256)).astype(np.float32))
    before = c.values()
    codes = np.abs(fp8.decode(c.codes))
    c.append((16 * rng.standard_normal((1, 256))).astype(np.float32))
    shift = c.exps[0] - bs8.exponent(before)
    assert shift >= 2
    changed = c.values()[:5] != before
    assert not np.any(changed & (codes * 2.0 ** -shift >= 2.0 ** -6))
    # half a subnormal step, in the new scale
    assert np.max(np.abs(c.values()[:5] - before)) <= 2.0 ** -10 * 2.0 ** c.exps[0]


def test_values_are_within_half_a_step_of_the_block():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 256)) * np.exp2(rng.integers(-3, 4, (40, 1)))).astype(np.float32)
    c = bs8.Cache()
    c.append(x)
    e = np.repeat(c.exps, 16)[:40, None]
    assert np.all(np.abs(c.values() - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * np.exp2(e)))


def test_one_append_equals_several_where_scales_do_not_grow_and_a_rollback_keeps_them():
    rng = np.random.default_rng(2)
    x = rng.uniform(-1, 1, (33, 256)).astype(np.float32)
    x[::16, 0] = 1.5                                  # every block's largest value comes first
    a, b = bs8.Cache(), bs8.Cache()
    a.append(x)
    for part in (x[:1], x[1:18], x[18:]):
        b.append(part)
    assert np.array_equal(a.codes, b.codes) and a.exps == b.exps
    b.append(100 * x[:3])
    grown = b.exps[2]
    b.truncate(33)
    assert b.exps[2] == grown and grown > a.exps[2]


def test_attention_against_library_softmax():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 8, 256)), rng.standard_normal((1, 20, 256)), rng.standard_normal((1, 20, 256))
    mask = torch.tensor(np.arange(20)[None, :] <= 17 + np.arange(3)[:, None])
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).permute(1, 0, 2), torch.tensor(np.repeat(k, 8, 0)), torch.tensor(np.repeat(v, 8, 0)), mask, scale=1 / 16)
    assert np.allclose(bs8.attention(q, k, v, 17), want.permute(1, 0, 2).numpy(), atol=1e-12)
    assert np.allclose(bs8.attention(q[:1], k[:, :1], v[:, :1], 0)[0, 3], v[0, 0])          # one position


def test_counts_by_hand():
    c = np.zeros(4, np.int16)
    logits.count(c, [1, 1, 9, -1, 2], False)
    logits.count(c, [1, 3], True)
    assert [int(np.uint16(x)) for x in c] == [0, 0x8002, 1, 0x8000]
    c[0] = 32766
    logits.count(c, [0, 0, 0], False)
    assert c[0] == 32767


def test_logits_by_hand():
    c = np.array([0, 2, -32768, -32767], np.int16)    # unseen, twice, prompt, prompt and once
    x = np.array([[2.0, 2.0, -2.0, 4.0]] * 2)
    got = logits.process(x, [0, 1], c, 2.0, 0.5, 0.25, [(2, 10.0)], np.array([[1, 1, 1, 1], [1, 0, 1, 1]], bool))
    # row 0: t_0 = 0 counts; row 1: t_1 = 1 too, and masked
    assert np.allclose(got[0], [2 / 2 - 0.5 - 0.25, 2 / 2 - 1.0 - 0.25, -4.0 + 10.0, 4 / 2 - 0.5 - 0.25])
    assert got[1, 1] == -np.inf and np.allclose(got[1, [0, 2, 3]], got[0, [0, 2, 3]])
