"""The rotary plan, and the refusals of the rotary, draft-acceptance, attention-mass and eviction calls (no GPU).

Refusals are checked at the C entry points (host checks come before any device
work) and in the binding, with the library replaced by a recorder as in the
binding's other tests, so that no call with these host tensors reaches a device.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import rope as ref
from speculative_verify_attention_q3kv_gb300 import _lib, api

INVALID, UNSUPPORTED, SMALL = _lib.Q3KV_ERR_INVALID_ARG, _lib.Q3KV_ERR_UNSUPPORTED, _lib.Q3KV_ERR_WORKSPACE_TOO_SMALL
i32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


# ------------------------------------------------------------------ rotary plan
@pytest.mark.parametrize("rotary,sections,deal,freqs,theta", [
    (64, (11, 11, 10), True, False, 1e7), (256, (32, 48, 48), False, True, 1e4), (16, (8,), False, False, 1e6),
    (128, (0, 32, 0, 32), True, True, 10000.0), (96, (1, 46, 1), True, False, 500000.0), (240, (60, 60), False, False, 1.5)])
def test_plan_holds_the_frequencies_in_turns(rotary, sections, deal, freqs, theta):
    plan = api.make_rope_plan(rotary, theta, sections, deal_axes=deal, axis_freqs=freqs, adjacent=True)
    axis, f = ref.pairs(rotary, theta, sections, deal, freqs)
    half = rotary // 2
    assert list(plan.axis[:half]) == axis.tolist() and plan.num_axes == len(sections) and plan.rotary_dim == rotary
    got = np.array([int(t) / 2.0 ** 64 * 2 * np.pi for t in plan.turns[:half]])
    # pow, the division by 2 pi and the product with 2 pi here: a few double roundings; and the
    # fixed-point cut, at most one unit of 2^-64 turns = 2 pi 2^-64 rad, whatever the frequency
    assert np.all(np.abs(got - f) <= 8 * 2.0 ** -53 * f + 2 * np.pi * 2.0 ** -64)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=272), dict(rotary_dim=-16), dict(theta=1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(num_axes=0), dict(num_axes=5), dict(sections=(16, 15, 0, 0)), dict(sections=(33, -1, 0, 0)),
    dict(flags=8), dict(reserved=1)])
def test_plan_refusals(lib, kw):
    base = dict(theta=1e4, rotary_dim=64, num_axes=2, sections=(16, 16, 0, 0), flags=0, reserved=0)
    base.update(kw)
    c = _lib.RopeConfig(base["theta"], base["rotary_dim"], base["num_axes"], (ctypes.c_int32 * 4)(*base["sections"]), base["flags"],
                        base["reserved"])
    plan = _lib.RopePlan()
    plan.rotary_dim = 77
    assert lib.q3kv_rope_plan_init(ctypes.byref(c), ctypes.byref(plan)) == INVALID
    assert plan.rotary_dim == 77                     # left as it was
    assert lib.q3kv_rope_plan_init(None, ctypes.byref(plan)) == INVALID
    assert lib.q3kv_rope_plan_init(ctypes.byref(c), None) == INVALID


def test_rope_refusals(lib):
    plan = api.make_rope_plan(64, 1e4, (16, 16))
    a = 4096                                         # an aligned address that no check follows

    def call(plan=plan, pos=a, rows=4, qi=a, qs=4096, qo=a, qos=4096, hq=16, ki=a, ks=512, ko=a, kos=512, hk=2, dtype=1):
        return lib.q3kv_rope(None, ctypes.byref(plan) if plan is not None else None, pos, rows, qi, qs, qo, qos, hq, ki, ks, ko, kos,
                             hk, dtype)

    assert call(rows=0) == 0 and call(hq=0, hk=0) == 0          # nothing to do
    for kw in (dict(plan=None), dict(rows=-1), dict(hq=-1), dict(hk=-1), dict(dtype=2), dict(pos=None), dict(qi=None), dict(qo=None),
               dict(ki=None), dict(qi=a + 8), dict(ko=a + 2), dict(qs=4095), dict(qs=4088), dict(qos=4100), dict(ks=0), dict(kos=-512)):
        assert call(**kw) == INVALID, kw
    assert call(hq=5000, qs=5000 * 256, qos=5000 * 256) == UNSUPPORTED
    for field, value in (("rotary_dim", 40), ("num_axes", 0), ("num_axes", 5)):
        bad = api.make_rope_plan(64, 1e4, (16, 16))
        setattr(bad, field, value)
        assert call(plan=bad) == INVALID
    bad = api.make_rope_plan(64, 1e4, (16, 16))
    bad.axis[31] = 2                                 # beyond num_axes: would read past a row's positions
    assert call(plan=bad) == INVALID


# ------------------------------------------------------------------ C entry points
def _desc(**kw):
    d = dict(num_layers=3, num_kv_heads=2, num_q_heads=16, head_dim=256, page_size=256, num_pages=8)
    d.update(kw)
    return _lib.CacheDesc(*[d[k] for k in ("num_layers", "num_kv_heads", "num_q_heads", "head_dim", "page_size", "num_pages")])


@pytest.mark.parametrize("name", ["q3kv_attn_mass", "q3kv_fp8_attn_mass", "q3kv_t5k_attn_mass"])
def test_mass_refusals(lib, name):
    a = 4096

    def call(desc=_desc(), pool=a, table=a, mpps=4, ctx=a, nq=a, off=a, slots=2, max_ctx=1000, max_nq=8, layer=0, q=a, dtype=0, lse=a,
             decay=1.0, mass=a, stride=1000):
        return getattr(lib, name)(None, ctypes.byref(desc) if desc is not None else None, pool, table, mpps, ctx, nq, off, slots,
                                  max_ctx, max_nq, layer, q, dtype, lse, decay, mass, stride, None)

    assert call(slots=0) == 0 and call(max_nq=0) == 0 and call(max_ctx=0) == 0
    for kw in (dict(desc=None), dict(desc=_desc(num_layers=0)), dict(pool=None), dict(pool=a + 8), dict(table=None), dict(mpps=0),
               dict(ctx=None), dict(nq=None), dict(off=None), dict(slots=-1), dict(max_ctx=-1), dict(max_nq=-1), dict(layer=-1),
               dict(layer=3), dict(q=None), dict(q=a + 4), dict(dtype=3), dict(lse=None), dict(decay=-0.1), dict(decay=1.01),
               dict(decay=float("nan")), dict(mass=None), dict(stride=999), dict(max_ctx=1 << 31, stride=1 << 31)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(desc=_desc(head_dim=128)), dict(desc=_desc(num_q_heads=8)), dict(max_nq=17), dict(slots=65536)):
        assert call(**kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("name", ["q3kv_evict", "q3kv_fp8_evict", "q3kv_t5k_evict"])
def test_evict_refusals(lib, name):
    a = 4096

    def call(desc=_desc(), pool=a, table=a, mpps=4, ctx=a, slots=2, max_ctx=1000, budget=a, max_budget=100, sink=1, recent=2, layer=0,
             layers=3, mass=a, stride=1000, dst=a, dst_pages=4, kept=a, out=a, new=a):
        return getattr(lib, name)(None, ctypes.byref(desc) if desc is not None else None, pool, table, mpps, ctx, slots, max_ctx, budget,
                                  max_budget, sink, recent, layer, layers, mass, stride, dst, dst_pages, kept, out, new, None)

    assert call(slots=0) == 0
    for kw in (dict(desc=None), dict(desc=_desc(num_pages=0)), dict(pool=None), dict(pool=a + 4), dict(table=None), dict(mpps=0),
               dict(ctx=None), dict(slots=-1), dict(max_ctx=-1), dict(budget=None), dict(max_budget=-1), dict(sink=-1), dict(recent=-1),
               dict(layer=-1), dict(layer=1), dict(layer=4, layers=0), dict(layers=-1), dict(layers=4), dict(mass=None), dict(stride=999),
               dict(dst=None), dict(dst_pages=0), dict(kept=None), dict(new=None), dict(max_ctx=1 << 31, stride=1 << 31)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(desc=_desc(page_size=128)), dict(slots=65536)):
        assert call(**kw) == UNSUPPORTED, kw


def test_accept_draft_refusals(lib):
    a = 4096

    def call(lg=a, dtype=0, vocab=100, dr=a, ddtype=1, off=a, nq=a, tok=a, slots=2, rows=5, max_nq=8, ctx=a, tau=1.0, uni=a, acc=a, nxt=a,
             com=a, ws=a, nbytes=1 << 20):
        return lib.q3kv_accept_draft(None, lg, dtype, vocab, dr, ddtype, off, nq, tok, slots, rows, max_nq, ctx, tau, uni, 7, acc, nxt,
                                     com, None, ws, nbytes, None)

    for kw in (dict(dtype=2), dict(ddtype=-1), dict(vocab=0), dict(slots=-1), dict(rows=-1), dict(max_nq=-1), dict(tau=0.0),
               dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf"))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(max_nq=17), dict(rows=65536), dict(slots=65536), dict(vocab=(1 << 28) + 1)):
        assert call(**kw) == UNSUPPORTED, kw
    n = ctypes.c_size_t()
    assert lib.q3kv_accept_draft_workspace_bytes(1, 1, 100, None) == INVALID
    assert lib.q3kv_accept_draft_workspace_bytes(-1, 1, 100, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("name", ["q3kv_verify_attn_lse", "q3kv_prefill_attn_lse", "q3kv_fp8_verify_attn_lse", "q3kv_t5k_verify_attn_lse"])
def test_lse_calls_need_the_output(lib, name):
    a = 4096
    call = lambda lse, slots=1: getattr(lib, name)(None, ctypes.byref(_desc()), a, a, 4, a, a, a, slots, 100, 4, 0, a, 0, a, lse, 0, 256, a,  # noqa: E731
                                                   1 << 30, None)
    assert call(None) == INVALID
    assert call(None, slots=0) == 0                  # nothing to do


def test_accept_draft_refuses_probabilities_over_the_uniforms(lib):
    # other CTAs read the uniforms while accept_prob is written: 8 rows of 4 bytes from either side
    def call(prob):                                  # no slots: nothing is launched where there is a device
        a = 1 << 20
        return lib.q3kv_accept_draft(None, a, 0, 100, a, 0, a, a, a, 0, 8, 3, a, 1.0, 4096, 7, a, a, a, prob, a, 1 << 30, None)

    for prob in (4096, 4096 + 28, 4096 - 28):
        assert call(prob) == INVALID
    for prob in (4096 + 32, 4096 - 32, None):
        assert call(prob) != INVALID


# ------------------------------------------------------------------ binding
class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    rec = _Recorder()
    plan = api.make_rope_plan(64, 1e4, (16, 16))
    monkeypatch.setattr(_lib, "load", lambda: rec)
    monkeypatch.setattr(api, "_device_index", lambda t: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(api, "_stream", lambda s: 0)
    rec.plan = plan
    return rec


def _names(rec):
    return [n for n, _ in rec.calls if not n.endswith("_bytes")]


def test_host_tensors_are_refused():
    plan = api.make_rope_plan(64, 1e4, (32,))
    q, pos = torch.zeros((2, 16, 256)), torch.zeros((2, 1), dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.rope(plan, pos, q, q)
    z, lg = torch.zeros(2, dtype=i32), torch.zeros((5, 9))
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.accept_draft(lg, lg, z, z, torch.zeros(5, dtype=i32), 3, z, 1.0, torch.zeros(5), 1, z, z, z, torch.zeros(64, dtype=torch.uint8))
    d = api.make_desc(1, 2, 4)
    pool, table = torch.zeros(64, dtype=torch.uint8), torch.zeros((2, 4), dtype=i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.attn_mass(d, pool, table, z, z, z, 4, 1, 0, q, torch.zeros((2, 16)), 1.0, torch.zeros((2, 2, 4)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.evict(d, pool, table, z, 4, z, 4, 0, 0, 0, torch.zeros((1, 2, 2, 4)), table, torch.zeros((1, 2, 2, 4), dtype=i32), None, z)


def test_rope_binding_rules(fake):
    pos = torch.zeros((3, 2), dtype=i32)
    qkv = torch.zeros((3, 20 * 256), dtype=torch.bfloat16)
    q, k = qkv[:, :16 * 256].unflatten(1, (16, 256)), qkv[:, 16 * 256:18 * 256].unflatten(1, (2, 256))
    qo, ko = torch.zeros((3, 16, 256), dtype=torch.bfloat16), torch.zeros((3, 2, 256), dtype=torch.bfloat16)
    api.rope(fake.plan, pos, q, qo, k, ko)
    api.rope(fake.plan, pos, q, q)                   # in place, queries only
    args = fake.calls[0][1]
    assert args[5] == 20 * 256 and args[7] == 16 * 256 and args[8] == 16 and args[13] == 2 and args[14] == _lib.Q3KV_BF16
    assert fake.calls[1][1][9] is None and fake.calls[1][1][13] == 0
    n = len(fake.calls)
    for bad in (dict(positions=pos.long()), dict(q_out=qo.float()), dict(q_out=ko), dict(k=k.float(), k_out=ko.float()),
                dict(q=q.half(), q_out=qo.half(), k=None, k_out=None)):
        a = dict(positions=pos, q=q, q_out=qo, k=k, k_out=ko)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            api.rope(fake.plan, **a)
    for bad, what in ((dict(positions=pos[:, :1]), "contiguous"), (dict(positions=pos[:, :1].contiguous()), "positions must be"), (dict(positions=None), "positions must be"),
                      (dict(q=q[:2]), r"\[3, heads, 256\]"), (dict(q=q.transpose(0, 1)), r"\[3, heads, 256\]"),
                      (dict(q=torch.zeros((3, 16, 512), dtype=torch.bfloat16)[:, :, ::2]), "contiguous"), (dict(k_out=None), "together"),
                      (dict(q=qo.view(-1)[:-4096].view(2, 16, 256), q_out=qo.view(-1)[4096:].view(2, 16, 256), positions=pos[:2].contiguous(),
                            k=k[:2], k_out=ko[:2]), "overlaps")):
        a = dict(positions=pos, q=q, q_out=qo, k=k, k_out=ko)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            api.rope(fake.plan, **a)
    assert len(fake.calls) == n
    with pytest.raises(ValueError, match="at most 4 axes"):
        api.make_rope_plan(64, 1e4, (8, 8, 8, 4, 4))


def _mass_args():
    return dict(desc=api.make_desc(1, 2, 8), pool=torch.zeros(64, dtype=torch.uint8), page_table=torch.zeros((2, 4), dtype=i32),
                ctx_len=torch.zeros(2, dtype=i32), n_q=torch.zeros(2, dtype=i32), q_offsets=torch.zeros(3, dtype=i32), max_ctx_len=100,
                max_n_q=3, layer=0, q=torch.zeros((5, 16, 256)), lse=torch.zeros((5, 16)), decay=1.0, mass=torch.zeros((2, 2, 120)))


def test_mass_binding_rules(fake, monkeypatch):
    api.attn_mass(**_mass_args())
    api.fp8_attn_mass(**_mass_args())
    api.t5k_attn_mass(**_mass_args())
    assert _names(fake) == ["q3kv_attn_mass", "q3kv_fp8_attn_mass", "q3kv_t5k_attn_mass"]
    assert fake.calls[-1][1][-2] == 120 and fake.calls[-1][1][8] == 2
    n = len(_names(fake))
    for bad in (dict(lse=torch.zeros((5, 16), dtype=torch.float64)), dict(mass=torch.zeros((2, 2, 120), dtype=torch.bfloat16)),
                dict(ctx_len=torch.zeros(2)), dict(pool=None), dict(lse=None), dict(mass=None), dict(q=None),
                dict(q=torch.zeros((5, 16, 256), dtype=torch.float16)), dict(page_table=torch.zeros(8, dtype=i32)),
                dict(n_q=torch.zeros(1, dtype=i32)), dict(status=torch.zeros(0, dtype=i32))):
        with pytest.raises((TypeError, ValueError)):
            api.attn_mass(**{**_mass_args(), **bad})
    for bad, what in ((dict(lse=torch.zeros((4, 16))), "lse must be"), (dict(lse=torch.zeros((5, 8))), "lse must be"),
                      (dict(mass=torch.zeros((2, 2, 99))), "mass must be"), (dict(mass=torch.zeros((1, 2, 120))), "mass must be"),
                      (dict(mass=torch.zeros((2, 120))), "mass must be"), (dict(q=torch.zeros((5, 8, 256))), "q must be"),
                      (dict(mass=torch.zeros((2, 2, 240))[:, :, ::2]), "contiguous"),
                      (dict(ctx_len=torch.zeros((2, 1), dtype=i32)), "one-dimensional")):
        with pytest.raises(ValueError, match=what):
            api.attn_mass(**{**_mass_args(), **bad})
    monkeypatch.setattr(api, "pool_bytes", lambda d: 65)
    with pytest.raises(ValueError, match="pool holds 64 bytes"):
        api.attn_mass(**_mass_args())
    assert len(_names(fake)) == n


def _evict_args():
    return dict(desc=api.make_desc(3, 2, 8), pool=torch.zeros(64, dtype=torch.uint8), page_table=torch.zeros((2, 4), dtype=i32),
                ctx_len=torch.zeros(2, dtype=i32), max_ctx_len=100, budget=torch.zeros(2, dtype=i32), max_budget=50, n_sink=1, n_recent=2,
                layer=1, mass=torch.zeros((2, 2, 2, 110)), dst_page_table=torch.zeros((2, 3), dtype=i32),
                kept=torch.zeros((2, 2, 2, 50), dtype=i32), mass_out=torch.zeros((2, 2, 2, 50)), new_len=torch.zeros(2, dtype=i32))


def test_evict_binding_rules(fake):
    api.evict(**_evict_args())
    api.fp8_evict(**{**_evict_args(), "mass_out": None})
    api.t5k_evict(**_evict_args())
    assert _names(fake) == ["q3kv_evict", "q3kv_fp8_evict", "q3kv_t5k_evict"]
    args = [a for n, a in fake.calls if n == "q3kv_evict"][0]
    assert args[13] == 2 and args[15] == 110 and args[17] == 3
    n = len(_names(fake))
    for bad in (dict(budget=torch.zeros(1, dtype=i32)), dict(new_len=torch.zeros(2)), dict(kept=torch.zeros((2, 2, 2, 50))),
                dict(mass_out=torch.zeros((2, 2, 2, 50), dtype=torch.float64)), dict(budget=None), dict(kept=None), dict(mass=None),
                dict(dst_page_table=None), dict(new_len=None)):
        with pytest.raises((TypeError, ValueError)):
            api.evict(**{**_evict_args(), **bad})
    for bad, what in ((dict(mass=torch.zeros((2, 2, 110))), "mass must be"), (dict(mass=torch.zeros((2, 3, 2, 110))), "mass must be"),
                      (dict(mass=torch.zeros((2, 2, 2, 99))), "mass must be"), (dict(kept=torch.zeros((2, 2, 2, 49), dtype=i32)), "kept must be"),
                      (dict(mass_out=torch.zeros((1, 2, 2, 50))), "mass_out must be"),
                      (dict(dst_page_table=torch.zeros(6, dtype=i32)), "dst_page_table"),
                      (dict(dst_page_table=torch.zeros((1, 6), dtype=i32)), "dst_page_table")):
        with pytest.raises(ValueError, match=what):
            api.evict(**{**_evict_args(), **bad})
    assert len(_names(fake)) == n


def test_accept_draft_and_lse_binding_rules(fake):
    z = lambda n=2: torch.zeros(n, dtype=i32)  # noqa: E731
    base = dict(logits=torch.zeros((5, 9)), draft_probs=torch.zeros((5, 9), dtype=torch.bfloat16), q_offsets=z(), n_q=z(), tokens=z(5),
                max_n_q=3, ctx_len=z(), temperature=0.5, uniforms=torch.zeros(5), seed=-1, n_accepted=z(), next_token=z(),
                committed_len=z(), workspace=torch.zeros(640, dtype=torch.uint8))
    api.accept_draft(**base)
    args = fake.calls[-1][1]
    assert args[2] == _lib.Q3KV_F32 and args[5] == _lib.Q3KV_BF16 and args[15] == (1 << 64) - 1 and args[21] == 640
    n = len(fake.calls)
    for bad in (dict(draft_probs=torch.zeros((5, 8))), dict(draft_probs=torch.zeros((5, 9), dtype=torch.float16)), dict(tokens=z(4)),
                dict(uniforms=torch.zeros(4)), dict(uniforms=torch.zeros(5, dtype=torch.float64)), dict(logits=torch.zeros(9)),
                dict(accept_prob=torch.zeros(4)), dict(n_q=z().view(2, 1)), dict(q_offsets=z(1)), dict(next_token=None),
                dict(logits=torch.zeros((5, 18))[:, ::2])):
        with pytest.raises((TypeError, ValueError)):
            api.accept_draft(**{**base, **bad})
    assert len(fake.calls) == n
    d = api.make_desc(1, 2, 8)
    q, out = torch.zeros((5, 16, 256)), torch.zeros((5, 16, 256))
    call = lambda lse, fn=api.verify_attn_lse: fn(d, torch.zeros(64, dtype=torch.uint8), torch.zeros((2, 4), dtype=i32), z(), z(), z(3), 100, 3,  # noqa: E731
                                                  0, q, out, lse, torch.zeros(16, dtype=torch.uint8))
    for fn in (api.verify_attn_lse, api.prefill_attn_lse, api.fp8_verify_attn_lse, api.t5k_verify_attn_lse):
        call(torch.zeros((5, 16)), fn)
    assert _names(fake)[-4:] == ["q3kv_verify_attn_lse", "q3kv_prefill_attn_lse", "q3kv_fp8_verify_attn_lse", "q3kv_t5k_verify_attn_lse"]
    for bad in (torch.zeros((4, 16)), torch.zeros((5, 8)), torch.zeros((5, 16), dtype=torch.float64), None):
        with pytest.raises((TypeError, ValueError)):
            call(bad)


def test_accept_draft_refuses_temperatures_without_a_float32_inverse(lib):
    def call(tau):                                   # no slots: nothing is launched where there is a device
        a = 1 << 20
        return lib.q3kv_accept_draft(None, a, 0, 100, a, 0, a, a, a, 0, 8, 3, a, tau, a, 7, a, a, a, None, a, 1 << 30, None)

    for tau in (1e-45, 1e-40, 4.2e-39):              # log2(e) / tau is above the largest float32, 3.4028e38
        assert call(tau) == INVALID
    for tau in (4.3e-39, 1.2e-38, 1e-30, 2.9e38):
        assert call(tau) != INVALID


@pytest.mark.parametrize("name", ["q3kv_evict", "q3kv_fp8_evict", "q3kv_t5k_evict"])
def test_evict_refuses_outputs_over_what_it_reads(lib, name):
    # 3 layers x 2 slots x 2 kv heads: masses of 12 x 1,000 floats, kept positions and masses of 12 x 100
    mass, kept, out, read, written = 1 << 24, 1 << 26, 1 << 28, 48000, 4800

    def call(mass=mass, kept=kept, out=out, ctx=4096, budget=8192, new=12288):
        return getattr(lib, name)(None, ctypes.byref(_desc()), 1 << 20, 4096, 4, ctx, 2, 1000, budget, 100, 1, 2, 0, 3, mass, 1000,
                                  4096, 4, kept, out, new, None)

    over = [dict(out=mass), dict(out=mass + read - 4), dict(out=mass - written + 4), dict(kept=mass), dict(kept=mass + read - 4),
            dict(kept=mass - written + 4), dict(out=kept), dict(out=kept + written - 4), dict(new=4100), dict(new=4092), dict(new=8196),
            dict(new=8188)]
    for kw in over:
        assert call(**kw) == INVALID, kw
    if torch.cuda.is_available():
        return                                       # these addresses go no further than a machine without a device
    for kw in (dict(), dict(out=None), dict(out=mass + read), dict(kept=mass - written), dict(out=kept + written), dict(new=4096),
               dict(new=8192), dict(new=4104), dict(new=4088)):
        assert call(**kw) != INVALID, kw


def _brute_meet(a, a_step, a_width, a_rows, b, b_step, b_width, b_rows):
    first = {a + i * a_step + x for i in range(a_rows) for x in range(a_width)}
    return any(b + j * b_step + x in first for j in range(b_rows) for x in range(b_width))


def test_rows_meet_against_every_byte():
    rng = np.random.default_rng(3)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        rows, width = int(rng.integers(1, 6)), int(rng.integers(1, 6))
        sa, sb = width + int(rng.integers(0, 8)), width + int(rng.integers(0, 8))
        if rng.random() < 0.5:
            sb = sa
        a, b = 1000, 1000 + int(rng.integers(-60, 60))
        want = _brute_meet(a, sa, width, rows, b, sb, width, rows)
        assert api._rows_meet(a, sa, b, sb, width, rows) == want, (a, sa, b, sb, width, rows)
        seen[want] += 1
    assert min(seen.values()) > 300


def test_rope_binding_takes_rows_that_interleave(fake):
    """Query rows and output rows side by side in one buffer share nothing; a shifted copy of the rows does."""
    buf = torch.zeros((5, 3 * 4096))
    pos = torch.zeros((5, 2), dtype=i32)
    at = lambda x, n=4096: buf[:, x:x + n].unflatten(1, (n // 256, 256))  # noqa: E731
    api.rope(fake.plan, pos, at(0), at(4096))
    api.rope(fake.plan, pos, at(8192), at(0))
    assert _names(fake) == ["q3kv_rope"] * 2
    flat = torch.zeros(5 * 12288 + 8192)
    wide, narrow = flat[:5 * 12288].view(5, 12288)[:, :4096].unflatten(1, (16, 256)), flat[4096:4096 + 5 * 8192].view(5, 8192)[:, :4096].unflatten(1, (16, 256))
    for bad in ((at(0), at(256)), (at(4096), at(3840)), (wide, narrow)):
        with pytest.raises(ValueError, match="overlaps"):
            api.rope(fake.plan, pos, *bad)
    assert _names(fake) == ["q3kv_rope"] * 2


def test_rope_refuses_outputs_over_other_operands(lib):
    """f32 rows of 4 q heads and 2 kv heads (4,096 and 2,048 bytes) in slices of one buffer, 8 rows."""
    plan, base, pos = api.make_rope_plan(64, 1e4, (16, 16)), 1 << 24, 1 << 20

    def call(q=(0, 4096), qo=(1 << 20, 4096), k=(4096, 4096), ko=(1 << 22, 2048), pos=pos):      # (byte offset, stride in floats)
        return lib.q3kv_rope(None, ctypes.byref(plan), pos, 8, base + q[0], q[1], base + qo[0], qo[1], 4, base + k[0], k[1], base + ko[0],
                             ko[1], 2, _lib.Q3KV_F32)

    same = dict(q=(0, 4096), qo=(0, 4096), k=(4096, 4096), ko=(4096, 4096))       # in place in the projection's output
    for kw in (dict(qo=(4096, 4096)), dict(qo=(2048, 4096)), dict(qo=(5120, 4096)), dict(ko=(0, 4096)), dict(ko=(3088, 4096)), dict(ko=(1 << 20, 2048)),
               dict(qo=(16, 4096)), dict(qo=(16384, 4096)), dict(qo=(0, 1024)), dict(ko=(4112, 4096)), dict(pos=base + (1 << 20)),
               dict(pos=base + (1 << 20) - 60), dict(pos=base + (1 << 22) + 2044), {**same, "pos": base + 4096 + 16384},
               {**same, "ko": (6144, 4096), "k": (6128, 4096)}, dict(qo=(6128, 4096), ko=(6144, 4096), k=(1 << 23, 512))):
        assert call(**kw) == INVALID, kw
    if torch.cuda.is_available():
        return                                       # these addresses go no further than a machine without a device
    for kw in (dict(), same, dict(pos=base + (1 << 22) + 2048), dict(qo=(6144, 4096)), dict(ko=(6144, 4096)), dict(qo=(8192, 4096), ko=(6144, 4096)),
               dict(pos=base + (1 << 20) - 64), {**same, "pos": base + 6144 + 7 * 16384}, dict(qo=(12288, 8192), q=(0, 8192), k=(4096, 8192))):
        assert call(**kw) != INVALID, kw


def test_mass_binding_refuses_masses_over_what_the_call_reads(fake):
    """Other CTAs read the queries, the statistic and the records while masses are stored."""
    buf = torch.zeros(5 * 16 * 256 + 480 + 80)
    q, lse, mass = buf[:20480].view(5, 16, 256), buf[20480:20560].view(5, 16), buf[20560:21040].view(2, 2, 120)
    api.attn_mass(**{**_mass_args(), "q": q, "lse": lse, "mass": mass})       # side by side
    n = len(_names(fake))
    pool = torch.zeros(4096, dtype=torch.uint8)
    for bad in (dict(q=q, mass=buf[20000:20480].view(2, 2, 120)), dict(q=q, mass=buf[20479:20959].view(2, 2, 120)),
                dict(lse=lse, mass=buf[20559:21039].view(2, 2, 120)), dict(lse=lse, mass=buf[20001:20481].view(2, 2, 120)),
                dict(pool=pool, mass=pool[16:1936].view(torch.float32).view(2, 2, 120))):
        with pytest.raises(ValueError, match="mass overlaps"):
            api.fp8_attn_mass(**{**_mass_args(), **bad})
    assert len(_names(fake)) == n
