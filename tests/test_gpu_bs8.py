"""GPU parity of the block-scaled 8-bit cache: records bit-exact, outputs of both legs within derived tolerances of float64."""
import numpy as np
import pytest
import torch

from bs8_harness import FMA, MMA, Bs8Cache, check, i32, offsets, queries
from oracle import bs8
from speculative_verify_attention_q3kv_gb300 import _lib, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# ------------------------------------------------------------------ append
def _same(cache, want, slot, layer=0):
    """The slot's codes and scales against the oracle's caches want[g][kv]."""
    for g in range(cache.kv):
        for kv in range(2):
            n = len(want[g][kv].codes)
            codes, scales = cache.raw(slot, n, layer, g, kv)
            nan = (codes & 0x7F) == 0x7F                 # a NaN's sign is nobody's
            assert np.array_equal(nan, (want[g][kv].codes & 0x7F) == 0x7F)
            assert np.array_equal(codes[~nan], want[g][kv].codes[~nan]), (slot, g, kv)
            assert np.array_equal(np.log2(scales.astype(np.float64)), np.array(want[g][kv].exps, np.float64)), (slot, g, kv)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("steps", [[(1,)], [(16,), (16,)], [(5,), (6,), (6,), (300,)], [(700,)], [(255,), (2,), (15,), (1,)]])
def test_appends_of_one_slot(steps, dtype):
    rng = np.random.default_rng(len(steps))
    cache = Bs8Cache([1024], kv=2, layers=2)
    want = [[bs8.Cache() for _ in range(2)] for _ in range(2)]
    at = 0
    for i, (n,) in enumerate(steps):
        # each step is louder or quieter than the last: scales grow within blocks, or stay
        x = (rng.standard_normal((2, n, 2, 256)) * 4.0 ** rng.integers(-3, 4)).astype(np.float32)
        x = torch.from_numpy(x).to(dtype).float().numpy()
        cache.append([at], [x[0]], [x[1]], layer=1, dtype=dtype)
        for g in range(2):
            for kv in range(2):
                want[g][kv].append(x[kv, :, g])
        at += n
    _same(cache, want, 0, layer=1)
    assert int(cache.status) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_on_16_bytes_only(dtype):
    # rows are read in pieces of 32 bytes where both tensors begin on 32, of 16 elsewhere
    n, step = 300, 16 // dtype.itemsize
    rng = np.random.default_rng(16)
    x = [torch.from_numpy(rng.standard_normal((n, 2, 256)).astype(np.float32)).cuda().to(dtype) for _ in range(2)]
    pools = []
    for shift_k, shift_v in ((0, 0), (1, 0), (0, 1), (1, 1)):
        cache = Bs8Cache([n])
        rows = []
        for t, shift in zip(x, (shift_k, shift_v)):
            room = torch.zeros(t.numel() + step, dtype=dtype, device="cuda")
            at = room[shift * step:shift * step + t.numel()].view(n, 2, 256)
            at.copy_(t)
            assert at.data_ptr() % 32 == 16 * shift
            rows.append(at)
        api.bs8_append(cache.desc, cache.pool, cache.page_table, i32([0]), i32([n]), i32([0]), n, 0, *rows, cache.status)
        assert int(cache.status) == 0
        pools.append(cache.pool)
    assert all(torch.equal(p, pools[0]) for p in pools)


def test_ragged_appends_leave_everything_else():
    rng = np.random.default_rng(5)
    starts, n = [0, 250, 16, 511, 7], [40, 20, 0, 2, 300]
    cache = Bs8Cache([s + m for s, m in zip(starts, n)], kv=3, layers=3, extra_pages=2)
    want = [[[bs8.Cache() for _ in range(2)] for _ in range(3)] for _ in starts]
    for part, at in ((starts, [0] * 5), (n, starts)):
        rows = [rng.standard_normal((2, m, 3, 256)).astype(np.float32) for m in part]
        before = cache.pool.clone()
        cache.append(at, [r[0] for r in rows], [r[1] for r in rows], layer=1)
        for b, r in enumerate(rows):
            for g in range(3):
                for kv in range(2):
                    want[b][g][kv].append(r[kv, :, g])
        # bytes outside the touched units of layer 1 are as before; so are codes of rows outside the appended ones
        now = cache.pool.cpu().numpy().reshape(cache.num_pages, 3, 3, 2, bs8.UNIT_BYTES)
        old = before.cpu().numpy().reshape(now.shape)
        assert np.array_equal(now[:, [0, 2]], old[:, [0, 2]])
        for b, (a, m) in enumerate(zip(at, part)):
            for p in range(256 * cache.pt.shape[1]):
                if cache.pt[b, p // 256] >= 0 and not (a - a % 16 <= p < a + m) and p % 37 == 0:
                    rows_at = bs8._OFFSETS[p % 256]
                    assert np.array_equal(now[cache.pt[b, p // 256], 1][..., rows_at], old[cache.pt[b, p // 256], 1][..., rows_at])
        assert np.array_equal(now[cache.free], old[cache.free])
    for b in range(5):
        _same(cache, want[b], b, layer=1)


def test_rollback_and_blocks_that_start_afresh():
    rng = np.random.default_rng(6)
    cache, want = Bs8Cache([256], kv=1), [[bs8.Cache(), bs8.Cache()]]
    for at, n, loud in ((0, 10, 1.0), (10, 6, 50.0), (12, 3, 0.01), (15, 1, 1.0), (16, 5, 80.0), (16, 4, 0.1), (18, 2, 0.1)):
        x = (loud * rng.standard_normal((2, n, 1, 256))).astype(np.float32)
        cache.append([at], [x[0]], [x[1]])
        for kv in range(2):
            want[0][kv].truncate(at)
            want[0][kv].append(x[kv, :, 0])
        _same(cache, want, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_at_the_borders(dtype):
    """Largest values at a power of two times 448 and next to it, ties of the codes, zeros, subnormals, and values beyond the scales."""
    eps = torch.finfo(dtype).eps
    rows = []
    for top in (448.0, 448.0 * (1 + eps), 448.0 * (1 - eps / 2), 1.75, 1.75 * (1 + eps), 2.0 ** -66, 448 * 2.0 ** 64, 2.0 ** -120, 0.0):
        x = np.zeros((16, 256), np.float64)
        x[3, 5] = top
        x[4] = top * (2 * np.arange(256) + 1) / 512          # every tie between codes, and the values between
        x[5, :16] = -top * 2.0 ** -np.arange(2, 18)
        rows.append(x)
    x = torch.from_numpy(np.concatenate(rows)).to(dtype).float().numpy()
    cache, want = Bs8Cache([len(x)], kv=1), [[bs8.Cache(), bs8.Cache()]]
    cache.append([0], [x[:, None]], [-x[:, None]], dtype=dtype)
    want[0][0].append(x)
    want[0][1].append(-x)
    _same(cache, want, 0)
    assert int(cache.status) == 0


def test_values_that_are_not_finite_and_scales_that_overflow():
    rng = np.random.default_rng(7)
    for bad, bits in ((np.inf, 1), (-np.inf, 1), (np.nan, 1), (3e38, 2), (449 * 2.0 ** 64, 2)):
        cache, want = Bs8Cache([40], kv=1), [[bs8.Cache(), bs8.Cache()]]
        x = rng.standard_normal((2, 40, 1, 256)).astype(np.float32)
        x[0, 20, 0, 9] = bad
        cache.append([0], [x[0]], [x[1]])
        for kv in range(2):
            want[0][kv].append(x[kv, :, 0])
        _same(cache, want, 0)
        assert int(cache.status) == bits, bad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_nan_in_v_reaches_those_who_see_it_and_no_others(dtype):
    L, T = [300], [6]
    cache = Bs8Cache(L, kv=1)
    rng = np.random.default_rng(40)
    k, v = (rng.standard_normal((300, 1, 256)).astype(np.float32) for _ in range(2))
    q = queries(6, 1, 41, dtype)
    cache.append([0], [k], [v], dtype=dtype)
    clean = {impl: cache.verify(L, T, q, impl=impl) for impl in (FMA, MMA)}
    for d, bad in ((7, np.nan), (8, np.nan), (200, -np.nan)):
        v2 = v.copy()
        v2[297, 0, d], v2[298, 0, 0] = bad, np.inf       # the fourth draft's; an infinity saturates
        cache.append([0], [k], [v2], dtype=dtype)
        codes_k, _ = cache.raw(0, 300, 0, 0, 0)
        codes_v, _ = cache.raw(0, 300, 0, 0, 1)
        assert np.array_equal(np.argwhere((codes_k & 0x7F) == 0x7F), [[297, d]]) and codes_v[297, d] & 0x7F == 0 and codes_v[298, 0] == 0x7E
        assert not np.any((codes_v & 0x7F) == 0x7F)
        for impl in (FMA, MMA):
            out = cache.verify(L, T, q, impl=impl)
            assert torch.equal(out[:3], clean[impl][:3]) and bool(torch.isnan(out[3:]).all())
    assert int(cache.status) == 1


def test_append_status_words():
    x = np.zeros((1, 5, 1, 256), np.float32)

    def run(start, n, page=None, most=None, room=256):
        cache = Bs8Cache([room], kv=1)
        if page is not None:
            cache.page_table[0, 0] = page
        before = cache.pool.clone()
        k = torch.ones((max(n, 1), 1, 256), device="cuda")
        api.bs8_append(cache.desc, cache.pool, cache.page_table, i32([start]), i32([n]), i32([0, n]), n if most is None else most, 0, k, k,
                       cache.status)
        return int(cache.status), bool((cache.pool != before).any())

    assert run(0, 5) == (0, True) and x.size
    assert run(0, 5, page=1) == (4, False) and run(0, 5, page=-1) == (4, False)
    assert run(-1, 5) == (8, False) and run(0, 5, most=4) == (8, False)
    assert run(250, 10) == (8, True)                  # what fits the table is stored
    assert run(256, 3) == (8, False) and run(2 ** 31 - 2, 5) == (8, False)
    cache = Bs8Cache([256], kv=1)
    rows = torch.ones((4, 1, 256), device="cuda")
    api.bs8_append(cache.desc, cache.pool, cache.page_table, i32([0]), i32([2]), i32([-1, 1]), 2, 0, rows, rows, cache.status)
    assert int(cache.status) == 8 and bool((cache.pool == 0xFF).all())


# ------------------------------------------------------------------ verify
KINDS = [("bf16", torch.bfloat16, 0), ("f32", torch.float32, MMA), ("fma", torch.float32, FMA), ("fma", torch.bfloat16, FMA)]
SHAPES = [([1], [1]), ([16], [16]), ([17, 128, 129, 255, 256, 257], [3, 1, 5, 16, 2, 8]), ([900, 40, 1300], [1, 2, 1]),
          ([600, 300, 70], [4, 3, 4]), ([2600, 9, 700], [8, 0, 6]), ([5, 1000], [5, 12])]


@pytest.mark.parametrize("kind,dtype,impl", KINDS)
@pytest.mark.parametrize("L,T", SHAPES)
def test_verify(L, T, kind, dtype, impl):
    cache = Bs8Cache(L, kv=2, layers=2, seed=len(L))
    cache.fill(L, seed=sum(L), layer=1)
    q = queries(sum(T) + 5, 2, 3 + sum(T), dtype, 2.0)
    out = cache.verify(L, T, q, layer=1, impl=impl, gap=2)
    check(out, q, cache, L, T, kind, layer=1, gap=2)
    assert int(cache.status) == 0


@pytest.mark.parametrize("kv", [1, 3, 4])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_verify_of_other_head_counts(kv, kind, dtype, impl):
    L, T = [333, 1025], [7, 2]
    cache = Bs8Cache(L, kv=kv)
    cache.fill(L, seed=kv)
    q = queries(sum(T), kv, kv, dtype, 1.5)
    check(cache.verify(L, T, q, impl=impl), q, cache, L, T, kind)


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_many_slots(kind, dtype, impl):
    rng = np.random.default_rng(8)
    L = rng.integers(1, 200, 70).tolist()
    T = [int(min(n, t)) for n, t in zip(L, rng.integers(0, 5, 70))]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=9)
    q = queries(sum(T), 1, 10, dtype)
    check(cache.verify(L, T, q, impl=impl), q, cache, L, T, kind)


def _rising(k, v, b):
    """Keys that grow along the context, so that every tile has larger scores than the one before."""
    return k * np.linspace(0.05, 6.0, len(k))[:, None, None].astype(np.float32), v


def _late(k, v, b):
    """One late key that takes nearly all of the weight."""
    k = k.copy()
    k[-5] *= 20
    return k, v


def _scales(k, v, b):
    """V blocks whose scales differ by up to 2^30, blocks of zeros among them; K blocks by up to 2^4."""
    n = len(k)
    e = np.random.default_rng(3).integers(-15, 16, n // 16 + 1)
    f = np.random.default_rng(4).integers(-2, 3, n // 16 + 1)
    v = v * np.exp2(np.repeat(e, 16)[:n])[:, None, None]
    v[32:48] = 0.0
    return (k * np.exp2(np.repeat(f, 16)[:n])[:, None, None]).astype(np.float32), v.astype(np.float32)


def _quiet(k, v, b):
    """Many small weights next to one key that all queries agree with."""
    k = 0.02 * k
    k[0] = 3.0
    return k, v + 1.0


@pytest.mark.parametrize("shape", [_rising, _late, _scales, _quiet])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_verify_of_uneven_caches(shape, kind, dtype, impl):
    L, T = [1500, 400], [6, 3]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=12, shape=shape)
    q = queries(sum(T), 1, 13, dtype, 1.5)
    if shape is _quiet:
        q = (q.float().abs()).to(dtype)
    check(cache.verify(L, T, q, impl=impl), q, cache, L, T, kind)


@pytest.mark.parametrize("T", [2, 4])
@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_one_large_weight_and_many_equal_small_ones(kind, dtype, impl, T):
    """Half of the weight on one early key, the rest shared out evenly: what one weight's codes lose is lost by all.  More
    slots than CTAs, which share their pages, so that a CTA goes through a whole context."""
    L, slots = 20000, 160
    one = Bs8Cache([L], kv=1)
    one.fill([L], seed=21, shape=lambda k, v, b: (np.where(np.arange(L)[:, None, None] == 3, np.log(L) / 16, 0.0 * k).astype(np.float32), v + 1.0))
    q = (1.0 + 0.05 * queries(T, 1, 22, torch.float32)).to(dtype)
    out = torch.full((slots * T, 8, 256), 77.0, dtype=dtype, device="cuda")
    api.bs8_verify_attn(one.desc, one.pool, one.page_table.repeat(slots, 1), i32([L] * slots), i32([T] * slots), offsets([T] * slots), L, T,
                        0, q.repeat(slots, 1, 1), out, one.workspace([L], [T], slots), impl, one.status)
    assert int(one.status) == 0
    for b in (0, 1, 77, slots - 1):
        check(out[b * T:b * T + T], q, one, [L], [T], kind)


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_rows_of_very_different_sizes(kind, dtype, impl):
    """Each row has a scale of its own: 2^-40 .. 2^3, and a row of zeros."""
    L, T = [300], [8]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=14)
    q = queries(8, 1, 15, torch.float32)
    q = (q * torch.exp2(torch.arange(-40, 4, device="cuda").float().repeat(2)[:64].reshape(8, 8, 1))).to(dtype)
    q[3, 2] = 0
    check(cache.verify(L, T, q, impl=impl), q, cache, L, T, kind)


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_query_rows_that_are_not_finite(kind, dtype, impl):
    L, T = [700], [4]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=16)
    q = queries(4, 1, 17, dtype)
    clean = cache.verify(L, T, q, impl=impl)
    q[1, 3, 100], q[2, 0, 0], q[3, 7, 255] = float("nan"), float("inf"), float("-inf")
    out = cache.verify(L, T, q, impl=impl)
    bad = torch.zeros((4, 8), dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[2, 0] = bad[3, 7] = True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("kind,dtype,impl", KINDS[:3])
def test_pages_out_of_range_are_hidden(kind, dtype, impl):
    L, T = [1100, 300], [5, 2]
    cache = Bs8Cache(L, kv=2)
    cache.fill(L, seed=18)
    keep = cache.pt.copy()
    cache.page_table[0, 1], cache.page_table[0, 4] = cache.num_pages, -1
    q = queries(7, 2, 19, dtype)
    out = cache.verify(L, T, q, impl=impl)
    assert int(cache.status) == _lib.Q3KV_STATUS_BAD_PAGE
    cache.pt = keep
    hidden = [np.zeros(n, bool) for n in L]
    hidden[0][256:512] = hidden[0][1024:] = True
    check(out, q, cache, L, T, kind, hidden=hidden)
    cache.page_table[1] = -1                             # a slot that sees nothing gives zeros
    out = cache.verify(L, T, q, impl=impl)
    assert bool((out[5:] == 0).all())


@pytest.mark.parametrize("dtype,impl", [(torch.bfloat16, 0), (torch.float32, 0), (torch.float32, FMA)])
def test_lengths_that_the_call_does_not_allow(dtype, impl):
    L, T = [300, 40, 500, 90], [2, 3, 1, 4]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=20)
    q = queries(10, 1, 21, dtype)
    good = cache.verify(L, T, q, impl=impl)
    for bad_L, bad_T in (([300, 2, 500, 90], T), ([300, 800, 500, 90], T), ([300, -1, 500, 90], T)):
        cache.status.zero_()
        out = torch.full_like(q, 77.0)
        api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table, i32(bad_L), i32(bad_T), offsets(T), 700, 4, 0, q, out,
                            cache.workspace(L, T), impl, cache.status)
        assert int(cache.status) == 8 and bool((out[2:5] == 77.0).all())
        # the others' rows: the work is shared out anew, so not bitwise
        for rows in (slice(0, 2), slice(5, 10)):
            assert float((out[rows].float() - good[rows].float()).abs().max()) < 0.05
    cache.status.zero_()
    out = torch.full_like(q, 77.0)
    api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table, i32(L), i32([2, 17, 1, -3]), i32([0, 2, -1, 6, 6]), 700, 4, 0, q, out,
                        cache.workspace(L, T), impl, cache.status)
    assert int(cache.status) == 8 and bool((out[2:] == 77.0).all())


def test_one_capture_many_lengths():
    """A captured call reads its lengths anew, shares its work out anew and leaves nothing behind in the workspace."""
    room = [2000, 600, 1200]
    cache = Bs8Cache(room, kv=2)
    cache.fill(room, seed=22)
    T = [3, 8, 1]
    q = queries(sum(T), 2, 23, torch.bfloat16)
    ctx, n_q, offs, out, ws = i32(room), i32(T), offsets(T), torch.full_like(q, 77.0), cache.workspace(room, [8])
    call = lambda: api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table, ctx, n_q, offs, 2000, 8, 0, q, out, ws, status=cache.status)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for L in (room, [3, 9, 1], [2000, 8, 1200], [129, 257, 128]):
        ctx.copy_(i32(L))
        out.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        check(out, q, cache, L, T, "bf16")
    assert int(cache.status) == 0


def test_a_step_captured_with_its_append():
    """Append and verify in one graph; each replay appends behind the last one's tokens."""
    cache = Bs8Cache([1000], kv=1)
    cache.fill([500], seed=24)
    n = 6
    k, v, q = (torch.zeros((n, h, 256), device="cuda", dtype=torch.bfloat16) for h in (1, 1, 8))
    at, L, T, offs, out, ws = i32([500]), i32([506]), i32([n]), offsets([n]), torch.zeros_like(q), cache.workspace([1000], [n])

    def step():
        api.bs8_append(cache.desc, cache.pool, cache.page_table, at, T, offs, n, 0, k, v, cache.status)
        api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table, L, T, offs, 1000, n, 0, q, out, ws, status=cache.status)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    gen = torch.Generator(device="cuda").manual_seed(25)
    for i in range(5):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda") * (1 + i))
        at.fill_(500 + n * i)
        L.fill_(500 + n * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        check(out, q, cache, [500 + n * (i + 1)], [n], "bf16")


def test_calls_on_two_streams_with_workspaces_of_their_own():
    L, T = [1800, 700], [8, 5]
    cache = Bs8Cache(L, kv=2)
    cache.fill(L, seed=26)
    qs = [queries(13, 2, 27 + i, torch.bfloat16 if i % 2 else torch.float32) for i in range(4)]
    want = [cache.verify(L, T, q).clone() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    spaces, outs = [cache.workspace(L, T) for _ in qs], [torch.zeros_like(q) for q in qs]
    args = (i32(L), i32(T), offsets(T))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, s, ws, out in zip(qs, streams, spaces, outs):
            api.bs8_verify_attn(cache.desc, cache.pool, cache.page_table, *args, 1800, 8, 0, q, out, ws, status=cache.status, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)                      # no atomics: the same bits


def test_units_beyond_32_bit_offsets():
    """A pool of 5.4 GB whose used pages lie behind the first 4 GiB."""
    desc = api.make_desc(16, 4, 640)
    pool = torch.empty(api.bs8_pool_bytes(desc), dtype=torch.uint8, device="cuda")
    cache = Bs8Cache([600], kv=1)                     # for its helpers only
    cache.desc, cache.pool, cache.kv, cache.layers, cache.num_pages = desc, pool, 4, 16, 640
    cache.pt = np.array([[639, 520, 630]], np.int32)
    cache.page_table = torch.from_numpy(cache.pt).cuda()
    pool[520 * (pool.numel() // 640):].fill_(0xFF)
    cache.fill([600], seed=30, layer=15)
    for dtype, kind in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        q = queries(5, 4, 31, dtype)
        check(cache.verify([600], [5], q, layer=15), q, cache, [600], [5], kind, layer=15)


@pytest.mark.parametrize("dtype,impl", [(torch.bfloat16, 0), (torch.float32, 0), (torch.float32, FMA)])
def test_bounds_beyond_32_bit_tile_counts(dtype, impl):
    """The largest max_ctx_len: tiles x CTAs no longer fit 32 bits by the host's bound, the results are the same bits."""
    rng = np.random.default_rng(42)
    L = rng.integers(10, 900, 40).tolist()
    T = rng.integers(0, 10, 40).tolist()
    cache = Bs8Cache(L, kv=2)
    cache.fill(L, seed=43)
    q = queries(sum(T), 2, 44, dtype)
    a = cache.verify(L, T, q, impl=impl)
    b = cache.verify(L, T, q, impl=impl, max_ctx=2 ** 31 - 300)
    assert torch.equal(a, b) and int(cache.status) == 0


def test_the_longest_share():
    """One head, one token: every CTA works through many tiles of one pair (bits of both float32 legs against each other)."""
    n = 60000
    cache = Bs8Cache([n], kv=1)
    gen = torch.Generator(device="cuda").manual_seed(32)
    k, v = (torch.randn((n, 1, 256), generator=gen, device="cuda") for _ in range(2))
    api.bs8_append(cache.desc, cache.pool, cache.page_table, i32([0]), i32([n]), i32([0, n]), n, 0, k, v, cache.status)
    q = queries(1, 1, 33, torch.float32, 3.0)
    a, b = cache.verify([n], [1], q, impl=MMA), cache.verify([n], [1], q, impl=FMA)
    # two legs: twice the float32 leg's bounds at G <= 30, and float32 sums of 60,000 positions over 152 CTAs
    assert float((a - b).abs().max()) <= 3e-4 * float(b.abs().max())
    c = cache.verify([n], [1], q.bfloat16())
    d = cache.verify([n], [1], q.bfloat16().float(), impl=FMA)
    assert float((c.float() - d).abs().max()) <= 2.0 ** -7 * float(d.abs().max())


def test_workspaces_over_other_operands_are_refused():
    """What the call uses of its workspace is nobody else's; what lies behind that in the same buffer may be."""
    L, T = [300, 40], [2, 1]
    cache = Bs8Cache(L, kv=1)
    cache.fill(L, seed=45)
    q = queries(3, 1, 46, torch.bfloat16)
    want = cache.verify(L, T, q)
    need = api.bs8_workspace_bytes(cache.desc, 2, 300, 2)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    base, lib = room.data_ptr(), _lib.load()
    lists = dict(table=cache.page_table, ctx=i32(L), nq=i32(T), off=offsets(T), status=cache.status, pool=cache.pool, q=q, out=torch.zeros_like(q))

    def call(**at):
        p = {k: at.get(k, t.data_ptr()) for k, t in lists.items()}
        return lib.q3kv_bs8_verify_attn(None, cache.desc, p["pool"], p["table"], cache.pt.shape[1], p["ctx"], p["nq"], p["off"], 2, 300, 2, 0, p["q"], 1,
                                        p["out"], 0, base, room.numel(), p["status"])

    for name in lists:
        for at in (base, base + need - 16):
            assert call(**{name: at}) == _lib.Q3KV_ERR_INVALID_ARG, name
    torch.cuda.synchronize()
    assert bool((lists["out"] == 0).all()) and not bool(room.any())
    room[need:need + 8].copy_(lists["ctx"].view(torch.uint8))      # the lengths behind it
    torch.cuda.synchronize()
    assert call(ctx=base + need) == 0
    torch.cuda.synchronize()
    assert torch.equal(lists["out"], want) and int(cache.status) == 0
