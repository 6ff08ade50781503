"""GPU parity of the attention mass, its softmax statistic and the eviction.

Tolerances.  A score is a sum of 256 products; with A = sum |q_d k_d| / 16 over the
rotated values, every float32 evaluation of at most 512 terms is within
512 2^-24 A = 2^-15 A of the exact one (any order), and an fp16 hi / lo split of an
operand adds 2^-22 A.  A weight e^(s - lse) then carries that absolute error of s as
a relative one, plus 2^-22 (1 + |s| + |lse|) for the exponent's own roundings: the
bound of a position is the sum of its rows' bounds and 2^-23 of the result per
addition (at most 129).  The statistic's bound is the largest score bound of the row.
"""
import numpy as np
import pytest
import torch

from operator_harness import APPEND, EVICT, MASS, POOL_BYTES, VERIFY, VERIFY_LSE, Cache, i32, offsets, queries
from oracle import eviction as ev
from speculative_verify_attention_q3kv_gb300 import _lib, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _reference(c, lengths, widths, q, layer, b, g):
    """(scores, bound of each score) of one slot and kv head."""
    r0 = sum(widths[:b])
    n, t = lengths[b], widths[b]
    qb = c.q_basis(q[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy())
    kh = c.k_hat(b, layer, g, n)
    s = ev.scores(qb, kh, n - t, 8)
    size = np.abs(qb.reshape(8 * t, 256)) @ np.abs(kh).T / 16.0
    return s, size * (2.0 ** -15 + 2.0 ** -22)


def _lse_of(c, lengths, widths, q, layer):
    lse = torch.full((q.shape[0], q.shape[1]), float("nan"), device="cuda")
    for b, t in enumerate(widths):
        r0 = sum(widths[:b])
        for g in range(c.kv):
            if t:
                s, _ = _reference(c, lengths, widths, q, layer, b, g)
                lse[r0:r0 + t, 8 * g:8 * g + 8] = torch.from_numpy(ev.log_sum_exp(s).reshape(t, 8)).float().cuda()
    return lse


def _mass_call(c, lengths, widths, q, lse, decay, mass, layer=0, status=None, **kw):
    MASS[c.fmt](c.desc, c.pool, c.page_table, i32(lengths), i32(widths), offsets(widths), kw.pop("max_ctx", max(lengths)),
                kw.pop("max_n_q", max(max(widths), 1)), layer, q, lse, decay, mass, status, **kw)


def _check_mass(c, got, old, lengths, widths, q, lse, decay, layer=0):
    for b, (n, t) in enumerate(zip(lengths, widths)):
        for g in range(c.kv):
            row = got[b, g].double().cpu().numpy()
            was = old[b, g].double().cpu().numpy()
            assert np.array_equal(row[n if t else 0:], was[n if t else 0:], equal_nan=True)      # not this step's: left as it was
            if not t:
                continue
            s, bound = _reference(c, lengths, widths, q, layer, b, g)
            r0 = sum(widths[:b])
            l = lse[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
            want = ev.mass(was[:n], s, l, float(np.float32(decay)), n - t)
            w = np.exp(s - l[:, None])
            seen = np.isfinite(s)
            rel = np.where(seen, bound + 2.0 ** -22 * (1 + np.abs(np.where(seen, s, 0)) + np.abs(l[:, None])), 0)
            tol = (w * rel).sum(axis=0) + 130 * 2.0 ** -23 * np.abs(want) + 1e-37
            err = np.abs(row[:n] - want)
            assert np.all(err <= tol), (b, g, float((err / np.maximum(tol, 1e-300)).max()))


MASS_CASES = [
    # fmt, lengths, widths, kv heads, dtype, decay, layers
    ("q3", [1], [1], 1, torch.float32, 1.0, 1),
    ("q3", [300], [4], 2, torch.bfloat16, 1.0, 1),
    ("q3", [256, 257, 1023], [1, 16, 7], 2, torch.float32, 0.5, 2),
    ("q3", [5, 900, 700, 640], [5, 0, 8, 9], 3, torch.bfloat16, 0.0, 1),
    ("q3", [4097], [2], 1, torch.bfloat16, 0.9, 1),
    ("fp8", [700, 130], [3, 16], 2, torch.float32, 1.0, 2),
    ("fp8", [513], [1], 4, torch.bfloat16, 0.25, 1),
    ("t5k", [700, 130], [3, 16], 2, torch.float32, 1.0, 2),
    ("t5k", [2000], [8], 1, torch.bfloat16, 0.0, 1),
    # every pass shape (16, 32, 48, 64 and 2 x 64 rows) in one call, and several tiles of each for a CTA
    ("q3", [3001, 2600, 2801, 3100, 2222, 1999], [6, 1, 16, 3, 8, 5], 2, torch.bfloat16, 1.0, 1),
    ("fp8", [600, 520, 811, 300, 222], [5, 16, 3, 6, 1], 2, torch.bfloat16, 1.0, 1),
    ("t5k", [600, 520, 811, 300, 222], [6, 9, 4, 5, 2], 1, torch.float32, 0.5, 1),
    ("q3", [20000], [6], 2, torch.float32, 1.0, 1),
    ("q3", [19000], [13], 2, torch.bfloat16, 1.0, 1),
]


@pytest.mark.parametrize("fmt,lengths,widths,kv,dtype,decay,layers", MASS_CASES)
def test_mass(fmt, lengths, widths, kv, dtype, decay, layers):
    c = Cache(fmt, lengths, kv, layers, seed=len(lengths) + lengths[0])
    q = queries(sum(widths), 8 * kv, 4, dtype)
    layer = layers - 1
    lse = _lse_of(c, lengths, widths, q, layer)
    mass = torch.rand((len(lengths), kv, max(lengths) + 9), device="cuda")
    if decay == 0.0:
        mass.fill_(float("nan"))                     # never read
    else:
        for b, (n, t) in enumerate(zip(lengths, widths)):
            if t:
                mass[b, :, n - t:] = float("nan")    # the step's own positions have no history; later ones are not this call's
    old = mass.clone()
    _mass_call(c, lengths, widths, q, lse, decay, mass, layer, c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    _check_mass(c, mass, old, lengths, widths, q, lse, decay, layer)
    # without a history, a row's weights add up to one
    if decay == 0.0:
        for b, (n, t) in enumerate(zip(lengths, widths)):
            if t:
                assert torch.allclose(mass[b, :, :n].double().sum(dim=1), torch.full((kv,), 8.0 * t, device="cuda", dtype=torch.float64),
                                      rtol=1e-3)


@pytest.mark.parametrize("fmt", ["q3", "fp8", "t5k"])
def test_mass_with_extreme_scores(fmt):
    """One position takes a row's whole weight, others underflow to nothing."""
    lengths, widths = [600], [2]
    c = Cache(fmt, lengths, 1, seed=2, scale=6.0)
    q = queries(2, 8, 9, scale=12.0)
    lse = _lse_of(c, lengths, widths, q, 0)
    mass = torch.zeros((1, 1, 600), device="cuda")
    old = mass.clone()
    _mass_call(c, lengths, widths, q, lse, 1.0, mass)
    torch.cuda.synchronize()
    _check_mass(c, mass, old, lengths, widths, q, lse, 1.0)


def test_mass_batch_equals_solo_and_repeats_bitwise():
    lengths, widths = [900, 130, 2048], [6, 16, 1]
    c = Cache("q3", lengths, 2, seed=5)
    q = queries(sum(widths), 16, 6, torch.bfloat16)
    lse = _lse_of(c, lengths, widths, q, 0)
    both = torch.zeros((3, 2, 2048), device="cuda")
    _mass_call(c, lengths, widths, q, lse, 1.0, both)
    again = torch.zeros_like(both)
    _mass_call(c, lengths, widths, q, lse, 1.0, again)
    torch.cuda.synchronize()
    assert torch.equal(both, again)
    for b in range(3):
        w = [widths[b] if i == b else 0 for i in range(3)]
        one = torch.zeros_like(both)
        MASS["q3"](c.desc, c.pool, c.page_table, i32(lengths), i32(w), offsets(widths), 2048, 16, 0, q, lse, 1.0, one)
        torch.cuda.synchronize()
        assert torch.equal(one[b], both[b])


def test_mass_after_a_rollback():
    """With the committed lengths, only the kept tokens' rows count and rolled-back positions have no history."""
    L, T, acc = 700, 6, 3
    c = Cache("q3", [L], 2, seed=8)
    q = queries(T, 16, 7)
    lse = _lse_of(c, [L], [T], q, 0)
    mass = torch.rand((1, 2, L), device="cuda")
    old = mass.clone()
    kept = acc + 1
    MASS["q3"](c.desc, c.pool, c.page_table, i32([L - (T - kept)]), i32([kept]), i32([0, kept]), L, T, 0, q, lse, 1.0, mass)
    torch.cuda.synchronize()
    _check_mass(c, mass, old, [L - (T - kept)], [kept], q, lse, 1.0)


def test_mass_status_bits():
    lengths, widths = [600, 520], [2, 3]
    c = Cache("q3", lengths, 2, seed=3)
    q = queries(5, 16, 1)
    lse = _lse_of(c, lengths, widths, q, 0)
    start = torch.rand((2, 2, 600), device="cuda")

    def run(**kw):
        mass, st = start.clone(), i32([0])
        a = dict(lengths=lengths, widths=widths, lse=lse, table=c.page_table, max_ctx=600, max_n_q=16)
        a.update(kw)
        MASS["q3"](c.desc, c.pool, a["table"], i32(a["lengths"]), i32(a["widths"]), offsets(widths), a["max_ctx"], a["max_n_q"], 0, q,
                   a["lse"], 1.0, mass, st)
        torch.cuda.synchronize()
        return mass, int(st.item())

    good, st = run()
    assert st == 0
    # too many tokens for the host bound, for the length; a length beyond the host bound, beyond the page table
    for kw in (dict(max_n_q=2), dict(lengths=[600, 2]), dict(max_ctx=599, lengths=[599, 600]), dict(lengths=[600, 800], max_ctx=600)):
        mass, st = run(**kw)
        assert st == _lib.Q3KV_STATUS_BAD_LENGTH
        assert torch.equal(mass[1], start[1])
    # a page id out of range: its positions keep their history
    for bad in (-1, c.num_pages, 1 << 30):
        table = c.page_table.clone()
        table[0, 1] = bad
        mass, st = run(table=table)
        assert st == _lib.Q3KV_STATUS_BAD_PAGE
        assert torch.equal(mass[0, :, 256:512], start[0, :, 256:512])
        assert torch.equal(mass[0, :, :256], good[0, :, :256]) and torch.equal(mass[1], good[1])
    # statistics that are not finite: the row is left out
    for bad in (float("nan"), float("inf"), -float("inf")):
        l2 = lse.clone()
        l2[0, 3] = bad
        mass, st = run(lse=l2)
        assert st == _lib.Q3KV_STATUS_NONFINITE_INPUT
        l3 = lse.clone()
        l3[0, 3] = 3.0e38                            # e^(s - 3e38) = 0
        assert torch.equal(mass, run(lse=l3)[0])


@pytest.mark.parametrize("fmt", ["q3", "fp8", "t5k"])
@pytest.mark.parametrize("impl,split", [(0, 0), (2, 256), (1, 256), (1, 2048)])
def test_verify_lse(fmt, impl, split):
    """The statistic against float64, and the outputs bit for bit those of the call without it."""
    if fmt == "fp8" and impl == 1:
        pytest.skip("the fp8 cache has the tensor-core leg only")
    lengths, widths = [1300, 700, 9], [5, 0, 9]
    c = Cache(fmt, lengths, 2, 2, seed=12)
    q = queries(sum(widths), 16, 2, torch.bfloat16, scale=1.0)
    ws = torch.zeros(max(16, api.workspace_bytes(c.desc, 3, 1300, 9, impl, split)), dtype=torch.uint8, device="cuda")
    args = (c.desc, c.pool, c.page_table, i32(lengths), i32(widths), offsets(widths), 1300, 9, 1, q)
    plain = torch.full((q.shape[0], 16, 256), float("nan"), device="cuda")
    out, lse = plain.clone(), torch.full((q.shape[0] + 2, 16), -5.0, device="cuda")
    VERIFY[fmt](*args, plain, ws, impl, split, c.status)
    VERIFY_LSE[fmt](*args, out, lse, ws, impl, split, c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert torch.equal(out, plain)
    assert torch.all(lse[q.shape[0]:] == -5.0)
    for b in (0, 2):
        for g in range(2):
            s, bound = _reference(c, lengths, widths, q, 1, b, g)
            r0 = sum(widths[:b])
            got = lse[r0:r0 + widths[b], 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
            want = ev.log_sum_exp(s)
            # the legs drop the product of two low halves, 2^-20 of A
            tol = bound.max(axis=1) * 1.04 + 2.0 ** -20 * (1 + np.abs(want))
            assert np.all(np.abs(got - want) <= tol)


def test_prefill_lse():
    L, T = 900, 200
    c = Cache("q3", [L], 2, seed=13)
    q = queries(T, 16, 3, torch.bfloat16, scale=1.0)
    args = (c.desc, c.pool, c.page_table, i32([L]), i32([T]), i32([0, T]), L, T, 0, q)
    for impl, split in ((0, 0), (1, 256)):
        ws = torch.zeros(max(16, api.prefill_workspace_bytes(c.desc, 1, L, T, impl, split)), dtype=torch.uint8, device="cuda")
        plain = torch.empty((T, 16, 256), device="cuda")
        out, lse = plain.clone(), torch.empty((T, 16), device="cuda")
        api.prefill_attn(*args, plain, ws, impl, split, c.status)
        api.prefill_attn_lse(*args, out, lse, ws, impl, split, c.status)
        torch.cuda.synchronize()
        assert torch.equal(out, plain)
        for g in range(2):
            s, bound = _reference(c, [L], [T], q, 0, 0, g)
            want = ev.log_sum_exp(s)
            got = lse[:, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
            assert np.all(np.abs(got - want) <= bound.max(axis=1) * 1.04 + 2.0 ** -20 * (1 + np.abs(want)))


# ------------------------------------------------------------------ eviction
def _evict_call(c, lengths, budgets, sink, recent, mass, layer=0, status=None, max_budget=None, with_mass=True, table=None, dst=None,
                max_ctx=None, in_place=False):
    S = len(lengths)
    most = max(max(budgets), 1) if max_budget is None else max_budget
    room = [(max(0, min(n, k)) + 255) // 256 for n, k in zip(lengths, budgets)]
    if dst is None:
        d = np.full((S, max(max(room), 1)), -1, np.int32)
        at = 0
        for b, r in enumerate(room):
            d[b, :r] = c.free[at:at + r]
            at += r
        dst = torch.from_numpy(d).cuda()
    layers = mass.shape[0]
    kept = torch.full((layers, S, c.kv, most), -9, dtype=torch.int32, device="cuda")
    out = torch.full((layers, S, c.kv, most), -9.0, device="cuda") if with_mass else None
    ctx = i32(lengths)
    new_len = ctx if in_place else i32([-9] * S)
    EVICT[c.fmt](c.desc, c.pool, c.page_table if table is None else table, ctx, mass.shape[3] if max_ctx is None else max_ctx,
                 i32(budgets), most, sink, recent, layer, mass, dst, kept, out, new_len, status)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), None if out is None else out.cpu().numpy(), new_len.cpu().numpy(), dst.cpu().numpy()


def _check_evict(c, before, lengths, budgets, sink, recent, mass, layer, got):
    """Kept positions, masses, lengths and records; every other byte of the pool is as it was."""
    kept, out, new_len, dst = got
    m = mass.cpu().numpy()
    pool_now = c.pool.clone()
    for b, (n, k) in enumerate(zip(lengths, budgets)):
        if k <= 0:
            assert new_len[b] == n and np.all(kept[:, b] == -9)
            continue
        assert new_len[b] == min(n, k)
        for la in range(m.shape[0]):
            for g in range(c.kv):
                want = ev.keep(m[la, b, g, :n], k, sink, recent)
                assert np.array_equal(kept[la, b, g, :len(want)], want)
                assert np.all(kept[la, b, g, len(want):] == -9)
                if out is not None:
                    assert np.array_equal(out[la, b, g, :len(want)], m[la, b, g, want], equal_nan=True)
                    assert np.all(out[la, b, g, len(want):] == -9.0)
                for kv in range(2):
                    c.pool = before
                    src = c.records(c.pt[b], layer + la, g, kv, want)
                    c.pool = pool_now
                    assert np.array_equal(c.records(dst[b], layer + la, g, kv, np.arange(len(want))), src)
    c.pool = pool_now


EVICT_CASES = [
    # fmt, lengths, budgets, sink, recent, kv heads, layers of the pool, first layer, layers of the call
    ("q3", [1], [1], 0, 0, 1, 1, 0, 1),
    ("q3", [600], [300], 4, 32, 2, 1, 0, 1),
    ("q3", [700, 90, 513], [256, 200, 257], 4, 16, 2, 3, 1, 2),
    ("q3", [700, 90, 513], [0, 1, 512], 0, 0, 1, 2, 0, 2),
    ("q3", [400], [50], 40, 30, 1, 1, 0, 1),                 # protected positions alone exceed the budget
    ("q3", [400], [70], 40, 30, 1, 1, 0, 1),                 # and fill it exactly
    ("q3", [20000, 9000], [3000, 8999], 16, 100, 2, 1, 0, 1),
    ("fp8", [600, 300], [100, 299], 1, 1, 2, 2, 1, 1),
    ("t5k", [600, 300], [100, 299], 1, 1, 2, 2, 0, 2),
]


@pytest.mark.parametrize("fmt,lengths,budgets,sink,recent,kv,layers,first,count", EVICT_CASES)
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict(fmt, lengths, budgets, sink, recent, kv, layers, first, count, kind):
    room = sum((max(0, min(n, k)) + 255) // 256 for n, k in zip(lengths, budgets))
    c = Cache(fmt, lengths, kv, layers, seed=21, extra_pages=room + 1)
    gen = torch.Generator(device="cuda").manual_seed(31)
    mass = torch.rand((count, len(lengths), kv, max(lengths) + 5), generator=gen, device="cuda")
    want_status = 0
    if kind == "ties":
        mass = (mass * 3).floor() / 3                        # three values
    elif kind == "special":
        mass = mass - 0.5
        mass[..., ::7] = 0.0
        mass[..., 1::7] = -0.0
        mass[..., 2::11] = float("inf")
        mass[..., 3::13] = -float("inf")
        mass[..., 5::17] = 1e-40                             # subnormal
        if kind == "special" and fmt == "q3" and lengths[0] == 600:
            mass[..., 6::19] = float("nan")
            want_status = _lib.Q3KV_STATUS_NONFINITE_INPUT
    before = c.pool.clone()
    got = _evict_call(c, lengths, budgets, sink, recent, mass, first, c.status)
    assert int(c.status.item()) == want_status
    _check_evict(c, before, lengths, budgets, sink, recent, mass, first, got)
    # outside the destination pages' first records nothing changes
    changed = (c.pool != before).nonzero().flatten()
    per_page = c.pool.numel() // c.num_pages
    pages = set((changed // per_page).unique().tolist())
    assert pages <= set(got[3][got[3] >= 0].tolist())


def test_evict_all_equal_and_all_nan():
    c = Cache("q3", [900], 1, seed=1, extra_pages=2)
    for value, status in ((0.25, 0), (float("nan"), _lib.Q3KV_STATUS_NONFINITE_INPUT)):
        mass = torch.full((1, 1, 1, 900), value, device="cuda")
        st = i32([0])
        kept, _, n, _ = _evict_call(c, [900], [300], 2, 10, mass, 0, st)
        want = np.concatenate([np.arange(290), np.arange(890, 900)])
        assert np.array_equal(kept[0, 0, 0], want) and n[0] == 300 and int(st.item()) == status


def test_evict_without_masses_in_place_length_and_repeats():
    lengths, budgets = [5000, 3000], [1000, 700]
    c = Cache("q3", lengths, 2, seed=4, extra_pages=8)
    mass = torch.rand((1, 2, 2, 5000), device="cuda")
    first = _evict_call(c, lengths, budgets, 4, 64, mass)
    pool = c.pool.clone()
    for _ in range(3):
        again = _evict_call(c, lengths, budgets, 4, 64, mass, with_mass=False, in_place=True)
        assert np.array_equal(first[0], again[0]) and again[1] is None and np.array_equal(first[2], again[2])
        assert torch.equal(c.pool, pool)


def test_evict_status_bits():
    lengths, budgets = [600, 700], [300, 290]
    c = Cache("q3", lengths, 1, seed=6, extra_pages=4)
    mass = torch.rand((1, 2, 1, 700), device="cuda")
    good = c.pool.clone()
    bad_len, bad_page = _lib.Q3KV_STATUS_BAD_LENGTH, _lib.Q3KV_STATUS_BAD_PAGE

    def run(lens=lengths, buds=budgets, **kw):
        c.pool.copy_(good)
        st = i32([0])
        got = _evict_call(c, lens, buds, 1, 2, mass, status=st, **kw)
        return got, int(st.item())

    (kept, _, n, dst), st = run()
    assert st == 0 and n.tolist() == [300, 290]
    for kw in (dict(max_budget=295), dict(max_ctx=650), dict(lens=[600, 800], max_ctx=700), dict(lens=[600, -1])):
        (k2, _, n2, _), st = run(**kw)
        slot = 0 if "max_budget" in kw else 1
        assert st == bad_len and n2[slot] == kw.get("lens", lengths)[slot] and np.all(k2[:, slot] == -9)
        assert np.array_equal(k2[:, 1 - slot, :, :290], kept[:, 1 - slot, :, :290])
    narrow = torch.from_numpy(np.ascontiguousarray(dst[:, :1])).cuda()
    (_, _, n2, _), st = run(dst=narrow)              # 300 and 290 records do not fit one page
    assert st == bad_len and n2.tolist() == lengths and torch.equal(c.pool, good)
    for bad in (-1, c.num_pages):
        d = torch.from_numpy(dst).cuda()
        d[0, 0] = bad
        (k2, _, n2, _), st = run(dst=d)
        assert st == bad_page and np.array_equal(k2, kept) and n2.tolist() == [300, 290]
        table = c.page_table.clone()
        table[1, 1] = bad
        (k2, _, _, _), st = run(table=table)
        assert st == bad_page and np.array_equal(k2, kept)


def test_evict_captured_and_replayed():
    lengths, budgets = [3000, 1000], [500, 400]
    c = Cache("q3", lengths, 2, seed=9, extra_pages=4)
    mass = torch.rand((1, 2, 2, 3000), device="cuda")
    dst = torch.tensor([[int(c.free[0]), int(c.free[1])], [int(c.free[2]), int(c.free[3])]], dtype=torch.int32, device="cuda")
    ctx, bud = i32(lengths), i32(budgets)
    kept = torch.zeros((1, 2, 2, 500), dtype=torch.int32, device="cuda")
    out, n = torch.zeros((1, 2, 2, 500), device="cuda"), i32([0, 0])
    call = lambda: api.evict(c.desc, c.pool, c.page_table, ctx, 3000, bud, 500, 2, 50, 0, mass, dst, kept, out, n)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    mass.copy_(torch.rand_like(mass))
    before = c.pool.clone()
    g.replay()
    torch.cuda.synchronize()
    kept_h = kept.cpu().numpy()
    for b in range(2):
        kept_h[:, b, :, budgets[b]:] = -9
    outs = out.cpu().numpy()
    outs[:, 1, :, 400:] = -9.0
    _check_evict(c, before, lengths, budgets, 2, 50, mass, 0, (kept_h, outs, n.cpu().numpy(), dst.cpu().numpy()))


def test_mass_many_slots_with_invalid_ones_between():
    """More slots than a warp, more segments than CTAs; invalid and idle slots take no part."""
    rng = np.random.default_rng(2)
    lengths = [int(x) for x in rng.integers(1, 700, 75)]
    widths = [int(min(n, t)) for n, t in zip(lengths, rng.integers(0, 17, 75))]
    c = Cache("q3", lengths, 2, seed=33)
    q = queries(sum(widths), 16, 5, torch.bfloat16)
    lse = _lse_of(c, lengths, widths, q, 0)
    told = list(widths)
    told[3] = 17                                        # above the host bound
    told[40] = lengths[40] + 1 if lengths[40] < 16 else 99
    mass = torch.rand((75, 2, 800), device="cuda")
    old = mass.clone()
    st = i32([0])
    MASS["q3"](c.desc, c.pool, c.page_table, i32(lengths), i32(told), offsets(widths), 700, 16, 0, q, lse, 1.0, mass, st)
    torch.cuda.synchronize()
    assert int(st.item()) == _lib.Q3KV_STATUS_BAD_LENGTH
    for b in (3, 40):
        assert torch.equal(mass[b], old[b])
    for b in range(75):
        if b not in (3, 40) and widths[b] and b % 7 < 2:
            _check_one(c, mass, old, lengths, widths, q, lse, b)
        elif not widths[b]:
            assert torch.equal(mass[b], old[b])


def _check_one(c, got, old, lengths, widths, q, lse, b):
    n, t, r0 = lengths[b], widths[b], sum(widths[:b])
    for g in range(c.kv):
        s, bound = _reference(c, lengths, widths, q, 0, b, g)
        l = lse[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
        want = ev.mass(old[b, g].double().cpu().numpy()[:n], s, l, 1.0, n - t)
        w, seen = np.exp(s - l[:, None]), np.isfinite(s)
        rel = np.where(seen, bound + 2.0 ** -22 * (1 + np.abs(np.where(seen, s, 0)) + np.abs(l[:, None])), 0)
        tol = (w * rel).sum(axis=0) + 130 * 2.0 ** -23 * np.abs(want) + 1e-37
        assert np.all(np.abs(got[b, g].double().cpu().numpy()[:n] - want) <= tol)


def test_mass_captured_replayed_and_on_another_stream():
    lengths, widths = [1000, 400], [4, 9]
    c = Cache("fp8", lengths, 2, seed=14)
    q = queries(13, 16, 8)
    lse = _lse_of(c, lengths, widths, q, 0)
    ctx, nq, off = i32(lengths), i32(widths), offsets(widths)
    mass = torch.zeros((2, 2, 1000), device="cuda")
    call = lambda m: api.fp8_attn_mass(c.desc, c.pool, c.page_table, ctx, nq, off, 1000, 9, 0, q, lse, 1.0, m)  # noqa: E731
    call(mass)
    torch.cuda.synchronize()
    want = mass.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(mass)
    mass.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, want)
    side, other = torch.cuda.Stream(), torch.zeros_like(mass)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(other)
    third = torch.zeros_like(mass)
    call(third)                                         # two calls at once, on two streams
    torch.cuda.synchronize()
    assert torch.equal(other, want) and torch.equal(third, want)


def _long_masses(kind, n, gen):
    """[2 rows] of n masses: the threshold in a wide first-level bin, in a narrow one, among NaN, and among equal ones."""
    m = torch.rand((1, 1, 2, n), generator=gen, device="cuda")
    if kind == "decades":
        m = 10.0 ** (-12 * m)
    elif kind == "signed":
        m = m - 0.5
        m[..., ::5] = 0.0
        m[..., 1::5] = -0.0
        m[..., 7::10007] = float("inf")
        m[..., 8::10007] = -float("inf")
    elif kind == "nan":
        m[..., ::2] = float("nan")
        m[..., 1::3] = float("nan")
    elif kind == "equal":
        m = (m * 2).floor() + 1.0                            # 1 or 2
    elif kind == "crowded":
        m = 1.0 + m * 2.0 ** -9                              # one first-level bin holds everything
    return m


@pytest.mark.parametrize("kind", ["decades", "signed", "nan", "equal", "crowded"])
@pytest.mark.parametrize("n,budget", [(70001, 7000), (70001, 69990), (70001, 35001), (150000, 200)])
def test_evict_long_rows(kind, n, budget):
    # more positions per warp than stay in its registers: its masses are read again, or filtered into its list
    gen = torch.Generator(device="cuda").manual_seed(n + budget)
    mass = _long_masses(kind, n, gen)
    c = Cache("q3", [n], 2, seed=13, extra_pages=(budget + 255) // 256)
    before = c.pool.clone()
    got = _evict_call(c, [n], [budget], 3, 11, mass, 0, c.status)
    assert int(c.status.item()) == (_lib.Q3KV_STATUS_NONFINITE_INPUT if kind == "nan" else 0)
    kept, out, new_len, _ = got
    assert new_len[0] == budget
    for g in range(2):
        want = ev.keep(mass[0, 0, g].cpu().numpy(), budget, 3, 11)
        assert np.array_equal(kept[0, 0, g], want)
        assert np.array_equal(out[0, 0, g], mass[0, 0, g].cpu().numpy()[want], equal_nan=True)
    _check_evict(c, before, [n], [budget], 3, 11, mass, 0, got)


def test_evict_length_in_the_budgets_place_and_without_layers():
    c = Cache("q3", [900, 700], 1, seed=1, extra_pages=4)
    mass = torch.rand((1, 2, 1, 900), device="cuda")
    dst = torch.from_numpy(np.asarray(c.free[:4], np.int32).reshape(2, 2)).cuda()
    kept = torch.zeros((1, 2, 1, 400), dtype=torch.int32, device="cuda")
    ctx, bud, st = i32([900, 700]), i32([300, 400]), i32([0])
    api.evict(c.desc, c.pool, c.page_table, ctx, 900, bud, 400, 0, 5, 0, mass, dst, kept, None, bud, st)
    assert bud.tolist() == [300, 400] and ctx.tolist() == [900, 700] and int(st.item()) == 0
    for b, n in enumerate((300, 400)):
        m = mass[0, b, 0, :ctx[b].item()].cpu().numpy()
        assert np.array_equal(kept[0, b, 0, :n].cpu().numpy(), ev.keep(m, n, 0, 5))
    bud, new = i32([600, 0]), i32([-1, -1])                  # a budget above max_budget, in a call of no layers
    none = torch.zeros((0, 2, 1, 900), device="cuda")
    api.evict(c.desc, c.pool, c.page_table, ctx, 900, bud, 500, 0, 5, 0, none, dst,
              torch.zeros((0, 2, 1, 500), dtype=torch.int32, device="cuda"), None, new, st)
    assert new.tolist() == [900, 700] and int(st.item()) == _lib.Q3KV_STATUS_BAD_LENGTH


@pytest.mark.parametrize("fmt", ["q3", "fp8", "t5k"])
def test_records_beyond_32_bit_offsets(fmt):
    # the same cache in the last layer and pages of a pool of more than 4 GB, and in a small pool
    layers, n, T, keep = 64, 600, 4, 300
    per_page = POOL_BYTES[fmt](api.make_desc(layers, 2, 1))
    pages = int(1.1 * 2 ** 32) // per_page
    assert pages * per_page > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.randn((n, 2, 256), generator=gen, device="cuda"), torch.randn((n, 2, 256), generator=gen, device="cuda")
    q = torch.randn((T, 16, 256), generator=gen, device="cuda")
    results = []
    for desc, layer, table, dst in ((api.make_desc(1, 2, 8), 0, [3, 1, 2], [5, 4]),
                                    (api.make_desc(layers, 2, pages), layers - 1, [pages - 1, pages - 3, pages // 2], [pages - 2, 1])):
        pool = torch.zeros(POOL_BYTES[fmt](desc), dtype=torch.uint8, device="cuda")
        table, dst, st = i32([table]), i32([dst]), i32([0])
        ws = torch.zeros(api.workspace_bytes(desc, 1, n, T), dtype=torch.uint8, device="cuda")
        out, lse, mass = torch.zeros((T, 16, 256), device="cuda"), torch.zeros((T, 16), device="cuda"), torch.zeros((1, 1, 2, n), device="cuda")
        APPEND[fmt](desc, pool, table, i32([0]), i32([n]), i32([0, n]), n, layer, k, v)
        VERIFY_LSE[fmt](desc, pool, table, i32([n]), i32([T]), i32([0, T]), n, T, layer, q, out, lse, ws, status=st)
        MASS[fmt](desc, pool, table, i32([n]), i32([T]), i32([0, T]), n, T, layer, q, lse, 0.0, mass[0], st)
        kept, kept_mass, new = torch.zeros((1, 1, 2, keep), dtype=torch.int32, device="cuda"), torch.zeros((1, 1, 2, keep), device="cuda"), i32([0])
        EVICT[fmt](desc, pool, table, i32([n]), n, i32([keep]), keep, 4, 32, layer, mass, dst, kept, kept_mass, new, st)
        after = torch.zeros((T, 16, 256), device="cuda")
        VERIFY[fmt](desc, pool, dst, new, i32([T]), i32([0, T]), keep, T, layer, q, after, ws, status=st)
        assert int(st.item()) == 0 and new.tolist() == [keep]
        results.append([x.cpu() for x in (out, lse, mass, kept, kept_mass, after)])
        del pool
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][5].abs().max() > 0


@pytest.mark.parametrize("fmt,lengths,widths,kv", [
    ("q3", [40000, 33000, 10000, 37001, 21000, 12345, 28000, 39999], [6, 1, 16, 3, 8, 2, 5, 9], 4),
    ("q3", [40000, 33000, 10000, 37001, 21000, 12345, 28000, 39999], [1, 9, 4, 16, 2, 7, 1, 3], 4),
    ("fp8", [30000, 12000, 20001, 9000], [4, 16, 1, 6], 4),
    ("t5k", [30000, 12000, 20001, 9000], [4, 16, 1, 6], 4),
])
def test_mass_long_segments_of_several_pairs(fmt, lengths, widths, kv):
    """Uneven slots in even shares: a CTA runs long segments of several (slot, kv head) pairs, of one operand buffer
    and of two, so that every ring of the pipeline wraps inside a segment and goes on in the next.  A slot alone,
    in shares of its own, gives the same bits; the row sums are what the definition makes them."""
    c = Cache(fmt, lengths, kv, seed=46)
    q = queries(sum(widths), 8 * kv, 47, torch.bfloat16)
    n, T = max(lengths), max(widths)
    lse = torch.zeros((q.shape[0], 8 * kv), device="cuda")
    out = torch.empty((q.shape[0], 8 * kv, 256), device="cuda")
    ws = torch.zeros(api.workspace_bytes(c.desc, len(lengths), n, T), dtype=torch.uint8, device="cuda")
    VERIFY_LSE[fmt](c.desc, c.pool, c.page_table, i32(lengths), i32(widths), offsets(widths), n, T, 0, q, out, lse, ws, status=c.status)
    mass = torch.full((len(lengths), kv, n), float("nan"), device="cuda")
    _mass_call(c, lengths, widths, q, lse, 0.0, mass, status=c.status)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    for b, (L, t) in enumerate(zip(lengths, widths)):
        one = torch.full_like(mass, float("nan"))
        alone = [t if i == b else 0 for i in range(len(widths))]
        MASS[fmt](c.desc, c.pool, c.page_table, i32(lengths), i32(alone), offsets(widths), n, T, 0, q, lse, 0.0, one, c.status)
        torch.cuda.synchronize()
        assert torch.equal(one[b, :, :L], mass[b, :, :L]) and bool(torch.isnan(mass[b, :, L:]).all())
        # every row's weights add up to one, as far as the statistic and the scores are bounded (A < 2^7: 2^-8)
        total = mass[b, :, :L].double().sum(dim=1)
        assert torch.allclose(total, torch.full_like(total, 8.0 * t), rtol=2.0 ** -8)
    b = len(lengths) - 1
    _check_mass_slot(c, mass, lengths, widths, q, lse, b)
    assert int(c.status.item()) == 0


def _check_mass_slot(c, got, lengths, widths, q, lse, b):
    n, t, r0 = lengths[b], widths[b], sum(widths[:b])
    for g in range(c.kv):
        s, bound = _reference(c, lengths, widths, q, 0, b, g)
        l = lse[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
        want = ev.mass(np.zeros(n), s, l, 0.0, n - t)
        w, seen = np.exp(s - l[:, None]), np.isfinite(s)
        rel = np.where(seen, bound + 2.0 ** -22 * (1 + np.abs(np.where(seen, s, 0)) + np.abs(l[:, None])), 0)
        tol = (w * rel).sum(axis=0) + 130 * 2.0 ** -23 * np.abs(want) + 1e-37
        assert np.all(np.abs(got[b, g].double().cpu().numpy()[:n] - want) <= tol)


# Queries of one (slot, kv head) pair share a power of two before they are split into fp16 halves, with which
# a half's finest step is at most 2^-27 of the pair's largest (rotated) value y: beside the bounds above, every
# score may be off by 2^-27 y sum|k_hat| / 16.
@pytest.mark.parametrize("fmt,qscale,kscale", [("q3", 1e-4, 2.8e4), ("q3", 1e-3, 1e3), ("q3", 2e6, 1e-6), ("q3", 1e-20, 1.0), ("t5k", 1e-4, 1e4),
                                               ("t5k", 2e6, 1e-6), ("fp8", 1e-3, 100.0), ("fp8", 2e6, 0.02), ("q3", 1e12, 1e-6),
                                               ("q3", 0.04, 30.0), ("fp8", 0.05, 10.0), ("q3", 400.0, 0.01), ("fp8", 2000.0, 0.02)])
@pytest.mark.parametrize("widths", [[2, 1], [6, 9]])
def test_mass_of_small_and_large_queries(fmt, qscale, kscale, widths):
    lengths = [600, 300]
    c = Cache(fmt, lengths, 2, seed=41, scale=kscale)
    q = queries(sum(widths), 16, 43, scale=qscale)
    q[0, 3] *= 3000.0                                # one row far above the others of its pair
    lse = _lse_of(c, lengths, widths, q, 0)
    mass = torch.rand((2, 2, 600), device="cuda")
    old, st = mass.clone(), i32([0])
    _mass_call(c, lengths, widths, q, lse, 1.0, mass, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool(torch.isfinite(mass).all())
    for b, (n, t) in enumerate(zip(lengths, widths)):
        r0 = sum(widths[:b])
        for g in range(2):
            s, bound = _reference(c, lengths, widths, q, 0, b, g)
            most = np.abs(c.q_basis(q[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy())).max()
            bound = bound + 2.0 ** -27 * most * np.abs(c.k_hat(b, 0, g, n)).sum(axis=1)[None, :] / 16.0
            l = lse[r0:r0 + t, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
            want = ev.mass(old[b, g].double().cpu().numpy()[:n], s, l, 1.0, n - t)
            w, seen = np.exp(s - l[:, None]), np.isfinite(s)
            rel = np.where(seen, bound + 2.0 ** -22 * (1 + np.abs(np.where(seen, s, 0)) + np.abs(l[:, None])), 0)
            # e^x of an error x that is not small: the factor is e^x - 1
            tol = (w * np.expm1(np.minimum(rel, 50.0))).sum(axis=0) + 130 * 2.0 ** -23 * np.abs(want) + 1e-37
            err = np.abs(mass[b, g].double().cpu().numpy()[:n] - want)
            assert np.all(err <= tol), (b, g, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("fmt", ["q3", "fp8", "t5k"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [1, 3, 7, 16])
def test_mass_leaves_rows_out_that_are_not_finite(fmt, dtype, width):
    """A row with a NaN, an infinity or a value of 2^100 in its queries, with the statistic that comes of it or a finite
    one: the bits of a call in which the row is zeros and weighs nothing."""
    lengths, widths = [600, 300], [width, 2]
    c = Cache(fmt, lengths, 2, seed=44)
    q = queries(sum(widths), 16, 45, dtype)
    lse = _lse_of(c, lengths, widths, q, 0)
    start = torch.rand((2, 2, 600), device="cuda")
    rows = [(0, 3), (width - 1, 8)]
    q0, l0 = q.clone(), lse.clone()
    for t, h in rows:
        q0[t, h], l0[t, h] = 0.0, 3.0e38             # e^(0 - 3e38) = 0
    want, st = start.clone(), i32([0])
    _mass_call(c, lengths, widths, q0, l0, 1.0, want, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    nan, inf = float("nan"), float("inf")
    for value, stat in ((nan, nan), (inf, inf), (-inf, nan), (nan, 1.5), (inf, 1.5), (2.0 ** 100, 1.5), (-2.0 ** 127, nan)):
        q1, l1 = q.clone(), lse.clone()
        for t, h in rows:
            q1[t, h, 77], l1[t, h] = value, stat
        got, st = start.clone(), i32([0])
        _mass_call(c, lengths, widths, q1, l1, 1.0, got, status=st)
        torch.cuda.synchronize()
        assert torch.equal(got, want), (value, stat)
        assert int(st.item()) == _lib.Q3KV_STATUS_NONFINITE_INPUT


@pytest.mark.parametrize("n", [600, 20000])
@pytest.mark.parametrize("where", ["sink", "recent", "between, none of them kept", "between, all of them kept"])
@pytest.mark.parametrize("with_mass", [True, False])
def test_evict_status_of_a_nan_anywhere(n, where, with_mass):
    """A NaN sets the status wherever it lies in the row, also where the selection has nothing to choose."""
    sink, recent, budget, at = {"sink": (5, 20, 100, 3), "recent": (5, 20, 100, n - 1), "between, none of them kept": (30, 20, 50, n // 2),
                                "between, all of them kept": (5, 20, n, n // 2)}[where]
    c = Cache("q3", [n], 1, seed=48, extra_pages=(budget + 255) // 256)
    mass = torch.rand((1, 1, 1, n), device="cuda")
    for value, status in ((0.5, 0), (float("nan"), _lib.Q3KV_STATUS_NONFINITE_INPUT)):
        mass[..., at] = value
        before, st = c.pool.clone(), i32([0])
        got = _evict_call(c, [n], [budget], sink, recent, mass, 0, st, with_mass=with_mass)
        assert int(st.item()) == status
        _check_evict(c, before, [n], [budget], sink, recent, mass, 0, got)


def test_evict_into_buffers_that_touch():
    """Masses, kept positions and kept masses end to end in one allocation: neighbours are no overlap."""
    n, k = 900, 300
    c = Cache("q3", [n], 1, seed=49, extra_pages=2)
    buf = torch.zeros(n + 2 * k, device="cuda")
    kept = buf[:k].view(torch.int32).view(1, 1, 1, k)
    mass, out = buf[k:k + n].view(1, 1, 1, n), buf[k + n:].view(1, 1, 1, k)
    mass.copy_(torch.rand_like(mass))
    lens, was = i32([k, n, n]), mass.clone()          # budget, lengths and new lengths side by side
    dst = torch.from_numpy(np.asarray(c.free[:2], np.int32).reshape(1, 2)).cuda()
    api.evict(c.desc, c.pool, c.page_table, lens[1:2], n, lens[0:1], k, 3, 9, 0, mass, dst, kept, out, lens[2:3], c.status)
    want = ev.keep(was[0, 0, 0].cpu().numpy(), k, 3, 9)
    assert np.array_equal(kept[0, 0, 0].cpu().numpy(), want) and np.array_equal(out[0, 0, 0].cpu().numpy(), was[0, 0, 0].cpu().numpy()[want])
    assert lens.tolist() == [k, n, k] and torch.equal(mass, was) and int(c.status.item()) == 0
    for over in (mass[..., :k], mass[..., n - k:]):
        with pytest.raises(api.Q3KVError):
            api.evict(c.desc, c.pool, c.page_table, lens[1:2], n, lens[0:1], k, 3, 9, 0, mass, dst, kept, over, lens[2:3], c.status)


def test_mass_goes_on_in_the_evicted_masses():
    """With max_budget as large as the lengths to come, mass_out is the next attn_mass call's buffer: no copy."""
    n, k, T, room = 900, 300, 4, 700
    c = Cache("q3", [n], 2, seed=51, extra_pages=3)
    mass = torch.rand((1, 1, 2, n), device="cuda")
    dst = torch.from_numpy(np.asarray(c.free[:3], np.int32).reshape(1, 3)).cuda()
    kept = torch.zeros((1, 1, 2, room), dtype=torch.int32, device="cuda")
    out, new = torch.full((1, 1, 2, room), float("nan"), device="cuda"), i32([0])
    api.evict(c.desc, c.pool, c.page_table, i32([n]), n, i32([k]), room, 4, 32, 0, mass, dst, kept, out, new, c.status)
    L = k + T
    gen = torch.Generator(device="cuda").manual_seed(52)
    kv = torch.randn((2, T, 2, 256), generator=gen, device="cuda")
    api.append(c.desc, c.pool, dst, new, i32([T]), i32([0, T]), T, 0, kv[0], kv[1], c.status)
    q = queries(T, 16, 53)
    lse = torch.zeros((T, 16), device="cuda")
    o, ws = torch.empty((T, 16, 256), device="cuda"), torch.zeros(api.workspace_bytes(c.desc, 1, L, T), dtype=torch.uint8, device="cuda")
    api.verify_attn_lse(c.desc, c.pool, dst, i32([L]), i32([T]), i32([0, T]), L, T, 0, q, o, lse, ws, status=c.status)
    copy = torch.zeros((1, 2, L), device="cuda")
    copy[..., :k] = out[0, ..., :k]
    api.attn_mass(c.desc, c.pool, dst, i32([L]), i32([T]), i32([0, T]), L, T, 0, q, lse, 0.9, copy, c.status)
    api.attn_mass(c.desc, c.pool, dst, i32([L]), i32([T]), i32([0, T]), room, T, 0, q, lse, 0.9, out[0], c.status)
    assert torch.equal(out[0, ..., :L], copy) and bool(torch.isnan(out[0, ..., L:]).all()) and int(c.status.item()) == 0


@pytest.mark.parametrize("fmt", ["q3", "fp8", "t5k"])
@pytest.mark.parametrize("slots", [75, 9])
def test_mass_pairs_prepared_twice_between_others(fmt, slots):
    """Slots with small, usual and large queries and with rows that are not finite, next to one another in a CTA's
    segments: every slot's bits are those of the slot alone."""
    rng = np.random.default_rng(slots)
    top = 700 if slots > 32 else 9000
    lengths = [int(x) for x in rng.integers(1, top, slots)]
    widths = [int(min(n, t)) for n, t in zip(lengths, rng.integers(0, 17, slots))]
    widths[0] = min(lengths[0], 3)
    c = Cache(fmt, lengths, 2, seed=61)
    q = queries(sum(widths), 16, 62, torch.bfloat16)
    n = max(lengths)
    lse = torch.zeros((q.shape[0], 16), device="cuda")
    out = torch.empty((q.shape[0], 16, 256), device="cuda")
    ws = torch.zeros(api.workspace_bytes(c.desc, slots, n, 16), dtype=torch.uint8, device="cuda")
    VERIFY_LSE[fmt](c.desc, c.pool, c.page_table, i32(lengths), i32(widths), offsets(widths), n, 16, 0, q, out, lse, ws)
    r0 = 0
    for b, t in enumerate(widths):
        kind = rng.integers(0, 5)
        if kind < 3:
            q[r0:r0 + t] *= 10.0 ** [-5, 0, 5][kind]
        if kind == 2:
            # above every score of queries 1e5 times larger, |q| |k| / 16 <= 1e5 * 2 * 20 * 20 / 16 = 5e6: masses stay finite
            lse[r0:r0 + t] = 1.0e7
        if t and kind == 3:
            q[r0 + t - 1, 5, 9] = float("nan")
        if t and kind == 4:
            lse[r0, 11] = float("inf")
        r0 += t
    start = torch.rand((slots, 2, n), device="cuda")
    mass = start.clone()
    _mass_call(c, lengths, widths, q, lse, 1.0, mass)
    again = start.clone()
    _mass_call(c, lengths, widths, q, lse, 1.0, again)
    torch.cuda.synchronize()
    assert torch.equal(mass, again) and bool(torch.isfinite(mass).all())
    for b in range(slots):
        alone = [t if i == b else 0 for i, t in enumerate(widths)]
        one = start.clone()
        MASS[fmt](c.desc, c.pool, c.page_table, i32(lengths), i32(alone), offsets(widths), n, 16, 0, q, lse, 1.0, one)
        torch.cuda.synchronize()
        assert torch.equal(one[b], mass[b]), b
