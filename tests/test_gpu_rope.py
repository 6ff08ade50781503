"""GPU parity of q3kv_rope against the float64 definition.

Tolerance, per element, with x and y the pair's inputs and u = 2^-24 (half a
float32 step): the angle is off by at most the frequency's double rounding times
the position (|p| f 2^-51 covers this side's and the oracle's), 2^-33 of a turn
from the fixed-point cut and half a step of its float32 value of at most pi
(pi u = 1.9e-7); sincospi is within two steps (4 u); two products and a sum round
three times: (|x| + |y|) (1.9e-7 + 7.4e-10 + 7 u + |p| f 2^-51) < (|x| + |y|)
(6.2e-7 + |p| f 2^-51).  bf16 outputs add half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import rope as ref
from speculative_verify_attention_q3kv_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _check(got, x, positions, **kw):
    x64 = x.detach().double().cpu().numpy()
    pos = positions.cpu().numpy()
    want = ref.rotate(x64, pos, **kw)
    axis, f = ref.pairs(kw["rotary_dim"], kw["theta"], kw["sections"], kw.get("deal_axes", False), kw.get("axis_freqs", False))
    half = kw["rotary_dim"] // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if kw.get("adjacent") else (i, i + half)
    far = np.abs(pos[:, axis].astype(np.float64)) * f * 2.0 ** -51
    size = np.abs(x64[..., a]) + np.abs(x64[..., b])
    tol = np.zeros_like(x64)
    tol[..., a] = tol[..., b] = size * (6.2e-7 + far[:, None, :])
    if x.dtype == torch.bfloat16:
        tol += np.abs(want) * 2.0 ** -8
        tol[..., kw["rotary_dim"]:] = 0.0
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err - tol).max())


CASES = [
    # rows, q heads, kv heads, rotary, sections, deal, axis_freqs, adjacent, dtype, farthest position
    (1, 16, 2, 64, (11, 11, 10), True, False, False, torch.bfloat16, 1),
    (6, 16, 2, 64, (11, 11, 10), True, False, False, torch.bfloat16, 655360),
    (37, 8, 1, 256, (32, 48, 48), False, True, True, torch.float32, 4096),
    (5, 3, 3, 16, (8,), False, False, False, torch.float32, 1 << 20),
    (129, 1, 4, 240, (1, 118, 1), True, True, False, torch.bfloat16, 77),
    (9, 16, 2, 128, (0, 32, 0, 32), True, True, True, torch.float32, 100),
    (3, 16, 0, 256, (128,), False, False, False, torch.bfloat16, (1 << 31) - 1),
    (3, 0, 2, 32, (8, 8), False, False, True, torch.float32, 1 << 24),
    (1000, 16, 2, 96, (16, 16, 16), False, False, False, torch.float32, 131072),
]


@pytest.mark.parametrize("rows,hq,hk,rotary,sections,deal,freqs,adj,dtype,far", CASES)
def test_rotation(rows, hq, hk, rotary, sections, deal, freqs, adj, dtype, far):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    q = torch.randn((rows, hq, 256), generator=gen, device="cuda").to(dtype)
    k = torch.randn((rows, hk, 256), generator=gen, device="cuda").to(dtype)
    pos = torch.randint(-far, far, (rows, len(sections)), generator=gen, device="cuda").to(torch.int32)
    pos[0] = far
    kw = dict(rotary_dim=rotary, theta=1e6, sections=sections, deal_axes=deal, axis_freqs=freqs, adjacent=adj)
    plan = api.make_rope_plan(**kw)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    api.rope(plan, pos, q, qo, k, ko)
    torch.cuda.synchronize()
    if hq:
        _check(qo, q, pos, **kw)
    if hk:
        _check(ko, k, pos, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_in_place_give_the_same_bits(dtype):
    rows, hq, hk = 70, 16, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((rows, (hq + 2 * hk) * 256), generator=gen, device="cuda").to(dtype)
    before = qkv.clone()
    q, k = qkv[:, :hq * 256].unflatten(1, (hq, 256)), qkv[:, hq * 256:(hq + hk) * 256].unflatten(1, (hk, 256))
    pos = torch.arange(3 * rows, device="cuda", dtype=torch.int32).view(rows, 3)
    plan = api.make_rope_plan(128, 1e4, (20, 22, 22), deal_axes=True)
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k, memory_format=torch.contiguous_format)
    api.rope(plan, pos, q, qo, k, ko)
    q2, k2 = torch.empty_like(qo), torch.empty_like(ko)
    api.rope(plan, pos, q.contiguous(), q2, k.contiguous(), k2)
    assert torch.equal(qkv, before)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    api.rope(plan, pos, q, q, k, k)                       # in place in the projection's own output
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, (hq + hk) * 256:], before[:, (hq + hk) * 256:])     # v is left alone
    q_only = torch.empty_like(qo)
    api.rope(plan, pos, before[:, :hq * 256].unflatten(1, (hq, 256)), q_only)
    assert torch.equal(q_only, qo)


def test_scores_depend_on_relative_positions_only():
    """The rotation keeps q . k of equal distances: what makes it usable before an append."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((1, 1, 256), generator=gen, device="cuda").expand(4, 1, 256).contiguous()
    k = torch.randn((1, 1, 256), generator=gen, device="cuda").expand(4, 1, 256).contiguous()
    plan = api.make_rope_plan(256, 1e4, (64, 64))
    pos = torch.tensor([[0, 0], [1000, 7], [300000, 12], [655360, 655360]], device="cuda", dtype=torch.int32)
    shift = torch.tensor([[5, 3]], device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    api.rope(plan, pos + shift, q, qo)
    api.rope(plan, pos, k, ko)
    dots = (qo.double() * ko.double()).sum(dim=2).flatten()
    # 256 products of two elements, each off by 6.2e-7 (|x| + |y|) at most on both sides
    tol = 2 * 6.2e-7 * float((q.double().abs().sum() / 4) * k.double().abs().max() * 4)
    assert float((dots - dots[0]).abs().max()) <= tol


def test_zero_rows_and_another_stream():
    plan = api.make_rope_plan(64, 1e4, (32,))
    e = torch.empty((0, 16, 256), device="cuda")
    api.rope(plan, torch.empty((0, 1), device="cuda", dtype=torch.int32), e, torch.empty_like(e))
    q = torch.randn((300, 16, 256), device="cuda")
    pos = torch.arange(300, device="cuda", dtype=torch.int32)[:, None].contiguous()
    want, got = torch.empty_like(q), torch.empty_like(q)
    api.rope(plan, pos, q, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        api.rope(plan, pos, q, got)
    side.synchronize()
    assert torch.equal(want, got)


def test_captured_and_replayed():
    plan = api.make_rope_plan(64, 1e4, (16, 16))
    q = torch.randn((40, 16, 256), device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros((40, 2), device="cuda", dtype=torch.int32)
    out, want = torch.empty_like(q), torch.empty_like(q)
    api.rope(plan, pos, q, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rope(plan, pos, q, out)
    pos.copy_(torch.arange(80, device="cuda", dtype=torch.int32).view(40, 2))
    g.replay()
    api.rope(plan, pos, q, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_rows_that_interleave_and_outputs_over_other_operands():
    """Input and output rows side by side in one buffer; what would overwrite an operand is refused."""
    rows = 33
    gen = torch.Generator(device="cuda").manual_seed(9)
    buf = torch.randn((rows, (16 + 2 + 16 + 2) * 256), generator=gen, device="cuda")
    at = lambda h, n: buf[:, h * 256:(h + n) * 256].unflatten(1, (n, 256))  # noqa: E731
    q, k, qo, ko = at(0, 16), at(16, 2), at(18, 16), at(34, 2)
    pos = torch.randint(0, 5000, (rows, 2), generator=gen, device="cuda").to(torch.int32)
    plan = api.make_rope_plan(64, 1e4, (16, 16))
    want_q, want_k, before = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous()), buf.clone()
    api.rope(plan, pos, q.contiguous(), want_q, k.contiguous(), want_k)
    api.rope(plan, pos, q, qo, k, ko)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k) and torch.equal(buf[:, :18 * 256], before[:, :18 * 256])
    after = buf.clone()
    for a in ((q, qo, k, at(15, 2)), (q, at(17, 16), k, ko), (q, qo, k, at(33, 2)), (q, at(2, 16), k, ko)):
        with pytest.raises((api.Q3KVError, ValueError)):
            api.rope(plan, pos, *a)
    torch.cuda.synchronize()
    assert torch.equal(buf, after)
