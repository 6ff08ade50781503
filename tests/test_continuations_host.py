"""Shared pages of the allocator, and the refusals of the block-scaled cache's, the page copies', the counts' and the logits' calls
(no GPU: host checks come before any device work, and the binding is tested over a recorder in the library's place)."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_verify_attention_q3kv_gb300 import _lib, api

INVALID, UNSUPPORTED, SMALL = _lib.Q3KV_ERR_INVALID_ARG, _lib.Q3KV_ERR_UNSUPPORTED, _lib.Q3KV_ERR_WORKSPACE_TOO_SMALL
OUT_OF_PAGES, SLOT = _lib.Q3KV_ERR_OUT_OF_PAGES, _lib.Q3KV_ERR_SLOT_RANGE
i32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def code_of(f, *args):
    with pytest.raises(_lib.Q3KVError) as e:
        f(*args)
    return e.value.code


# ------------------------------------------------------------------ allocator
def test_fork_and_copy_on_write():
    a = api.Allocator(10, 4, 5)
    assert a.alloc_pages(0, 600).tolist() == [0, 1, 2, -1, -1]
    assert a.fork(0, 1, 600).tolist() == [0, 1, 2, -1, -1] and a.free_pages() == 7
    row, copy = a.write(1, 600, 10)                   # positions 512 .. 599 of page 2 have to move
    assert row.tolist() == [0, 1, 3, -1, -1] and copy == (2, 3, 88) and a.free_pages() == 6
    row, copy = a.write(0, 600, 10)                   # page 2 is slot 0's alone now
    assert row.tolist() == [0, 1, 2, -1, -1] and copy is None
    assert a.fork(0, 2, 512).tolist() == [0, 1, -1, -1, -1]
    row, copy = a.write(2, 512, 300)                  # the range begins with a page: nothing moves
    assert row.tolist() == [0, 1, 4, 5, -1] and copy is None
    row, copy = a.write(2, 256, 1)                    # a shared page overwritten from its first position on
    assert row.tolist() == [0, 6, 4, 5, -1] and copy is None
    row, copy = a.write(1, 100, 500)                  # a range over two shared pages and one of its own
    assert copy == (0, row[0], 100) and row[2] == 3 and len({int(x) for x in row[:3]}) == 3
    assert a.write(3, 0, 0)[0].tolist() == [-1] * 5
    a.free_slot(0)
    a.free_slot(1)
    assert a.free_pages() == 10 - 4                   # slot 2's pages stay, one of them slot 0's before
    assert a.pages(2).tolist() == [0, 6, 4, 5, -1]
    assert a.trim(2, 257).tolist() == [0, 6, -1, -1, -1] and a.trim(2, 0).tolist() == [-1] * 5 and a.free_pages() == 10


def test_allocator_refusals_change_nothing():
    a = api.Allocator(4, 3, 3)
    a.alloc_pages(0, 700)
    assert code_of(a.fork, 0, 0, 10) == INVALID and code_of(a.fork, 0, 1, 769) == INVALID and code_of(a.fork, 0, 1, -1) == INVALID
    assert code_of(a.fork, 0, 3, 10) == SLOT and code_of(a.fork, -1, 1, 10) == SLOT
    a.fork(0, 1, 700)
    assert code_of(a.fork, 0, 1, 10) == INVALID        # holds pages already
    assert code_of(a.write, 1, 0, 700) == OUT_OF_PAGES  # three fresh pages, one is left
    assert a.pages(1).tolist() == [0, 1, 2] and a.free_pages() == 1
    assert code_of(a.write, 1, 700, 69) == OUT_OF_PAGES and code_of(a.write, 1, -1, 2) == INVALID and code_of(a.write, 5, 0, 1) == SLOT
    assert code_of(a.write, 1, 1 << 62, 1 << 62) == OUT_OF_PAGES and code_of(a.write, 1, 0, 1 << 62) == OUT_OF_PAGES
    assert code_of(a.trim, 1, -1) == INVALID and code_of(a.trim, 9, 0) == SLOT and code_of(a.pages, 3) == SLOT
    assert code_of(a.compact, -1) == INVALID
    lib = _lib.load()
    n = ctypes.c_int32()
    row = (ctypes.c_int32 * 3)()
    assert lib.q3kv_slot_pages(None, 0, row, ctypes.byref(n)) == INVALID and lib.q3kv_slot_pages(a._h, 0, None, None) == INVALID
    assert lib.q3kv_fork_slot(None, 0, 1, 1, row, None) == INVALID and lib.q3kv_write_pages(a._h, 0, 0, 1, row, None, None) == INVALID
    assert lib.q3kv_trim_slot(a._h, 0, 0, None, None) == INVALID and lib.q3kv_compact_pages(a._h, 1, None, row, ctypes.byref(n)) == INVALID
    assert lib.q3kv_compact_pages(a._h, 0, None, None, None) == INVALID
    assert a.pages(0).tolist() == [0, 1, 2]


@pytest.mark.parametrize("seed", range(6))
def test_allocator_against_a_model(seed):
    """Random calls; every position's content is followed through copies and moves of pages."""
    rng = np.random.default_rng(seed)
    pages, slots, per_slot = 24, 5, 8
    a = api.Allocator(pages, slots, per_slot)
    pool = np.zeros((pages, 256), np.int64)           # what each page's positions hold
    want = [[] for _ in range(slots)]                 # what each slot's positions should hold
    mark = 1
    for _ in range(300):
        op, s = rng.choice(["write", "fork", "free", "trim", "compact"], p=[0.5, 0.2, 0.1, 0.1, 0.1]), int(rng.integers(slots))
        if op == "write":
            at = int(rng.integers(0, len(want[s]) + 1)) if rng.random() < 0.3 else len(want[s])
            n = int(rng.integers(0, 400))
            try:
                row, copy = a.write(s, at, n)
            except _lib.Q3KVError as e:
                assert e.code == OUT_OF_PAGES
                continue
            if copy:
                src, dst, rows = copy
                assert 0 < rows < 256
                pool[dst, :rows] = pool[src, :rows]
            if n:
                want[s] = want[s][:at]
            for _ in range(n):
                p = len(want[s])
                pool[row[p // 256], p % 256] = mark
                want[s].append(mark)
                mark += 1
        elif op == "fork":
            src = int(rng.integers(slots))
            n = int(rng.integers(0, len(want[src]) + 1))
            if src == s or want[s] or (a.pages(s) >= 0).any():
                continue
            a.fork(src, s, n)
            want[s] = want[src][:n]
        elif op == "free":
            a.free_slot(s)
            want[s] = []
        elif op == "trim":
            n = int(rng.integers(0, len(want[s]) + 1))
            a.trim(s, n)
            want[s] = want[s][:n]
        else:
            held = {int(x) for b in range(slots) for x in a.pages(b) if x >= 0}
            src, dst = a.compact(int(rng.integers(0, 30)))
            assert set(src.tolist()) <= held and not set(dst.tolist()) & (held | set(src.tolist())) and len(set(dst.tolist())) == len(dst)
            assert np.all(src > dst)
            pool[dst] = pool[src].copy()
        rows = [a.pages(b) for b in range(slots)]
        held = {int(x) for r in rows for x in r if x >= 0}
        assert a.free_pages() == pages - len(held) and all(0 <= x < pages for x in held)
        for b in range(slots):
            assert [int(pool[rows[b][p // 256], p % 256]) for p in range(len(want[b]))] == want[b]
    src, _ = a.compact(pages)
    held = {int(x) for b in range(slots) for x in a.pages(b) if x >= 0}
    assert held == set(range(len(held)))              # packed


# ------------------------------------------------------------------ C entry points
def _desc(**kw):
    d = api.make_desc(3, 2, 10)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _ref(desc):
    return ctypes.byref(desc) if desc is not None else None


def test_bs8_pool_bytes(lib):
    assert api.bs8_pool_bytes(_desc()) == 10 * 3 * 2 * 2 * 65600
    n = ctypes.c_size_t()
    assert lib.q3kv_bs8_pool_bytes(_ref(_desc(head_dim=64)), ctypes.byref(n)) == UNSUPPORTED
    assert lib.q3kv_bs8_pool_bytes(_ref(_desc()), None) == INVALID


def test_bs8_append_refusals(lib):
    a = 4096

    def call(desc=_desc(), pool=a, table=a, mpps=4, ln=a, new=a, off=a, slots=2, most=3, layer=0, k=a, v=a, dtype=1):
        return lib.q3kv_bs8_append(None, _ref(desc), pool, table, mpps, ln, new, off, slots, most, layer, k, v, dtype, None)

    assert call(slots=0) == 0 and call(most=0) == 0
    for kw in (dict(desc=None), dict(desc=_desc(num_layers=0)), dict(pool=None), dict(pool=a + 8), dict(table=None), dict(mpps=0), dict(ln=None),
               dict(new=None), dict(off=None), dict(slots=-1), dict(most=-1), dict(layer=-1), dict(layer=3), dict(k=None), dict(v=a + 4),
               dict(dtype=2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(desc=_desc(page_size=128)), dict(slots=65536)):
        assert call(**kw) == UNSUPPORTED, kw


def test_bs8_verify_refusals(lib):
    a = 4096

    def call(desc=_desc(), pool=a, table=a, mpps=4, ctx=a, nq=a, off=a, slots=2, max_ctx=1000, max_nq=4, layer=0, q=a, dtype=1, out=a, impl=0,
             ws=a, nbytes=1 << 30):
        return lib.q3kv_bs8_verify_attn(None, _ref(desc), pool, table, mpps, ctx, nq, off, slots, max_ctx, max_nq, layer, q, dtype, out, impl,
                                        ws, nbytes, None)

    assert call(slots=0) == 0 and call(max_nq=0) == 0 and call(max_ctx=0) == 0
    for kw in (dict(desc=None), dict(desc=_desc(num_pages=0)), dict(pool=None), dict(pool=a + 4), dict(table=None), dict(mpps=0), dict(ctx=None),
               dict(nq=None), dict(off=None), dict(slots=-1), dict(max_ctx=-1), dict(max_nq=-1), dict(layer=-1), dict(layer=3), dict(q=None),
               dict(q=a + 2), dict(dtype=2), dict(out=None), dict(out=a + 8), dict(impl=3), dict(impl=-1), dict(ws=a + 8),
               dict(max_ctx=1 << 31)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(desc=_desc(head_dim=128)), dict(max_nq=17), dict(slots=65536)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws=None) == SMALL
    n = ctypes.c_size_t()
    assert lib.q3kv_bs8_workspace_bytes(_ref(_desc()), 1, 10, 1, 0, None) == INVALID
    assert lib.q3kv_bs8_workspace_bytes(_ref(_desc()), -1, 10, 1, 0, ctypes.byref(n)) == INVALID
    assert lib.q3kv_bs8_workspace_bytes(_ref(_desc()), 1, 10, 17, 0, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("name,page", [("q3kv_copy_pages", 3 * 2 * 2 * 256 * 112), ("q3kv_fp8_copy_pages", 3 * 2 * 2 * 65536),
                                       ("q3kv_t5k_copy_pages", 3 * 2 * 256 * 276), ("q3kv_bs8_copy_pages", 3 * 2 * 2 * 65600)])
def test_copy_pages_refusals(lib, name, page):
    a = 1 << 30

    def call(desc=_desc(), src_pool=a, dst_pool=a, pages=10, src=4096, dst=8192, rows=None, n=3, status=None):
        return getattr(lib, name)(None, _ref(desc), src_pool, dst_pool, pages, src, dst, rows, n, status)

    assert call(n=0) == 0
    for kw in (dict(desc=None), dict(desc=_desc(num_layers=-1)), dict(src_pool=None), dict(dst_pool=None), dict(src_pool=a + 8, dst_pool=a + 8),
               dict(pages=0), dict(src=None), dict(dst=None), dict(n=-1), dict(pages=11), dict(dst_pool=a + 9 * page),
               dict(dst_pool=a - 9 * page), dict(src=a + 16), dict(dst=a + 10 * page - 4), dict(rows=a - 8), dict(status=a)):
        assert call(**kw) == INVALID, kw
    assert call(n=4097) == UNSUPPORTED and call(desc=_desc(num_layers=20000)) == UNSUPPORTED


def test_count_tokens_refusals(lib):
    a = 4096

    def call(counts=1 << 30, stride=104, vocab=100, tokens=a, n_tok=50, off=a, n=a, slots=2, most=30, prompt=0, status=None):
        return lib.q3kv_count_tokens(None, counts, stride, vocab, tokens, n_tok, off, n, slots, most, prompt, status)

    assert call(slots=0) == 0 and call(most=0) == 0 and call(n_tok=0) == 0
    for kw in (dict(counts=None), dict(counts=(1 << 30) + 2), dict(stride=96), dict(stride=101), dict(vocab=0), dict(vocab=-1), dict(tokens=None),
               dict(n_tok=-1), dict(off=None), dict(n=None), dict(slots=-1), dict(most=-1), dict(prompt=2), dict(prompt=-1),
               dict(tokens=(1 << 30) + 400), dict(tokens=(1 << 30) - 196), dict(off=1 << 30), dict(n=(1 << 30) + 412), dict(status=1 << 30)):
        assert call(**kw) == INVALID, kw
    assert call(slots=65536) == UNSUPPORTED and call(vocab=(1 << 28) + 1, stride=(1 << 28) + 8) == UNSUPPORTED


def test_process_logits_refusals(lib):
    a, big = 4096, 1 << 30

    def call(lg=big, out=2 * big, dtype=0, vocab=104, off=a, nq=a, tok=a, slots=2, rows=5, max_nq=8, counts=a, stride=104, rep=a, fre=a, pre=a,
             boff=a, btok=a, bval=a, biases=7, mask=a, status=None):
        return lib.q3kv_process_logits(None, lg, out, dtype, vocab, off, nq, tok, slots, rows, max_nq, counts, stride, rep, fre, pre, boff, btok,
                                       bval, biases, mask, status)

    assert call(slots=0) == 0 and call(rows=0) == 0 and call(max_nq=0) == 0
    size = 5 * 104 * 4
    inside = 2 * big + 16
    for kw in (dict(lg=None), dict(lg=big + 4), dict(out=None), dict(out=2 * big + 8), dict(dtype=2), dict(vocab=0), dict(off=None), dict(nq=None),
               dict(tok=None), dict(slots=-1), dict(rows=-1), dict(max_nq=-1), dict(counts=a + 2), dict(stride=96), dict(stride=105),
               dict(biases=-1), dict(btok=None), dict(bval=None), dict(out=big + 16), dict(out=big + size - 16), dict(off=inside), dict(nq=inside),
               dict(tok=inside), dict(counts=inside), dict(rep=inside), dict(fre=inside), dict(pre=inside), dict(boff=inside), dict(btok=inside),
               dict(bval=inside), dict(mask=inside), dict(status=inside)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(max_nq=17), dict(slots=65536), dict(vocab=(1 << 28) + 1, counts=None)):
        assert call(**kw) == UNSUPPORTED, kw


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
    monkeypatch.setattr(_lib, "load", lambda: rec)
    monkeypatch.setattr(api, "_device_index", lambda t: 0)
    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(api, "_stream", lambda s: 0)
    return rec


def _verify_args(**kw):
    t = dict(desc=api.make_desc(1, 2, 4), pool=torch.zeros(64, dtype=torch.uint8), table=torch.zeros((2, 3), dtype=i32),
             ctx=torch.zeros(2, dtype=i32), nq=torch.zeros(2, dtype=i32), off=torch.zeros(3, dtype=i32), q=torch.zeros((4, 16, 256)),
             out=torch.zeros((4, 16, 256)), ws=torch.zeros(64, dtype=torch.uint8))
    t.update(kw)
    return t


def test_bs8_verify_binding(fake):
    call = lambda t: api.bs8_verify_attn(t["desc"], t["pool"], t["table"], t["ctx"], t["nq"], t["off"], 100, 4, 0, t["q"], t["out"],  # noqa: E731
                                         t["ws"])
    call(_verify_args())
    assert fake.calls[-1][0] == "q3kv_bs8_verify_attn"
    n = len(fake.calls)
    q = torch.zeros((4, 16, 256))
    for kw in (dict(q=None), dict(out=None), dict(ws=None), dict(pool=None), dict(table=None), dict(q=torch.zeros((4, 8, 256))),
               dict(q=torch.zeros((4, 16, 128))), dict(out=torch.zeros((3, 16, 256))), dict(out=torch.zeros((4, 16, 256), dtype=torch.bfloat16)),
               dict(q=torch.zeros((4, 16, 256), dtype=torch.float16), out=torch.zeros((4, 16, 256), dtype=torch.float16)),
               dict(off=torch.zeros(1, dtype=i32)), dict(nq=torch.zeros(2)), dict(table=torch.zeros((1, 3), dtype=i32)),
               dict(q=torch.zeros((4, 256, 16)).transpose(1, 2)), dict(q=q, out=q)):
        with pytest.raises((ValueError, TypeError)):
            call(_verify_args(**kw))
    both = torch.zeros(8, 16, 256)
    with pytest.raises(ValueError, match="overlaps"):
        call(_verify_args(q=both[:4], out=both[2:6]))
    with pytest.raises(ValueError, match="overlaps"):
        call(_verify_args(q=both[:4], ws=both[3:]))
    assert all(c[0] == "q3kv_bs8_pool_bytes" for c in fake.calls[n:])      # nothing reached the library


def test_bs8_append_binding(fake):
    def call(k, v, pool=None):
        api.bs8_append(api.make_desc(1, 2, 4), torch.zeros(64, dtype=torch.uint8) if pool is None else pool, torch.zeros((1, 3), dtype=i32),
                       torch.zeros(1, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32), 5, 0, k, v)

    good = torch.zeros(5, 2, 256)
    call(good, good.clone())
    for k, v in ((good, good[:4]), (good, good.bfloat16()), (good[:, :1], good[:, :1]), (None, good), (good, None), (good.half(), good.half())):
        with pytest.raises((ValueError, TypeError)):
            call(k, v)
    with pytest.raises(ValueError, match="overlaps"):
        call(good, good.clone(), pool=good.view(torch.uint8).flatten())


def test_copy_pages_binding(fake, monkeypatch):
    monkeypatch.setattr(api, "_pool_need", lambda *a: 64)
    desc, pool = api.make_desc(1, 2, 4), torch.zeros(64, dtype=torch.uint8)
    two = torch.zeros(2, dtype=i32)
    for f in (api.copy_pages, api.fp8_copy_pages, api.t5k_copy_pages, api.bs8_copy_pages):
        f(desc, pool, two, two.clone())
        f(desc, pool, two, two.clone(), rows=two.clone(), dst_pool=torch.zeros(128, dtype=torch.uint8), dst_num_pages=8)
        assert fake.calls[-1][1][4] == 8
        for kw in (dict(dst=torch.zeros(3, dtype=i32)), dict(dst=torch.zeros(1, dtype=i32)), dict(rows=torch.zeros(3, dtype=i32)),
                   dict(src=two.float()), dict(src=None), dict(dst_pool=pool.clone()), dict(dst_num_pages=4),
                   dict(dst_pool=torch.zeros(127, dtype=torch.uint8), dst_num_pages=8), dict(pool=pool[:63])):
            a = dict(pool=pool, src=two, dst=two.clone())
            a.update(kw)
            with pytest.raises((ValueError, TypeError)):
                f(desc, a.pop("pool"), a.pop("src"), a.pop("dst"), **a)


def test_count_and_logits_binding(fake):
    counts, tok, off, n = torch.zeros((2, 104), dtype=torch.int16), torch.zeros(9, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    api.count_tokens(counts, 100, tok, off, n, 9)
    for args in ((counts.int(), 100, tok, off, n), (counts, 105, tok, off, n), (counts[:1], 100, tok, off, n), (counts, 100, tok.long(), off, n),
                 (counts, 100, tok, off[:1], n), (counts, 100, tok, off, n.view(2, 1)), (None, 100, tok, off, n), (counts, 100, None, off, n)):
        with pytest.raises((ValueError, TypeError)):
            api.count_tokens(*args, 9)
    lg = torch.zeros((9, 100))
    f = torch.zeros(2)
    base = dict(counts=counts, repetition=f, frequency=f, presence=f, bias_offsets=torch.zeros(3, dtype=i32), bias_tokens=torch.zeros(5, dtype=i32),
                bias_values=torch.zeros(5), mask=torch.zeros((9, 4), dtype=i32))
    api.process_logits(lg, lg, off, n, tok, 5, **base)
    api.process_logits(lg, torch.zeros_like(lg), off, n, tok, 5)
    for kw in (dict(counts=counts[:, :96]), dict(counts=counts[:1]), dict(repetition=f[:1]), dict(frequency=f.double()), dict(presence=f.int()),
               dict(bias_offsets=torch.zeros(2, dtype=i32)), dict(bias_tokens=torch.zeros(4, dtype=i32)), dict(bias_values=None),
               dict(mask=torch.zeros((9, 3), dtype=i32)), dict(mask=torch.zeros((8, 4), dtype=i32)), dict(mask=torch.zeros((9, 4)))):
        with pytest.raises((ValueError, TypeError)):
            api.process_logits(lg, lg, off, n, tok, 5, **{**base, **kw})
    for args in ((lg.half(), lg.half(), off, n, tok), (lg, lg.bfloat16(), off, n, tok), (lg, lg[:8], off, n, tok), (lg, lg, off, n, tok[:8]),
                 (lg.view(-1), lg.view(-1), off, n, tok), (lg, None, off, n, tok), (lg.t(), lg.t(), off, n, tok)):
        with pytest.raises((ValueError, TypeError)):
            api.process_logits(*args, 5)


def test_bs8_outputs_over_lists_are_refused(lib):
    """What a call writes may not be what it, or its merge, still reads: lengths that change under it would send rows anywhere."""
    pool, out, lists = 1 << 30, 3 << 30, [1 << 20, 2 << 20, 3 << 20, 4 << 20]
    size = 10 * 3 * 2 * 2 * 65600
    append = dict(table=lists[0], ln=lists[1], new=lists[2], off=lists[3], k=5 << 20, v=6 << 20, status=7 << 20)
    inside = (pool, pool + size - 4, pool - 4)
    for name in append:
        for at in (pool, pool + size - 16) if name in "kv" else inside if name in ("table", "ln", "new", "off") else inside[:2]:
            a = dict(append, **{name: at})
            assert lib.q3kv_bs8_append(None, _ref(_desc()), pool, a["table"], 4, a["ln"], a["new"], a["off"], 2, 3, 0, a["k"], a["v"], 1,
                                       a["status"]) == INVALID, (name, at)
    verify = dict(pool=pool, table=lists[0], ctx=lists[1], nq=lists[2], off=lists[3], q=5 << 20, out=out, status=7 << 20)

    def call(**kw):
        a = dict(verify, **kw)
        return lib.q3kv_bs8_verify_attn(None, _ref(_desc()), a["pool"], a["table"], 4, a["ctx"], a["nq"], a["off"], 2, 1000, 4, 0, a["q"], 1,
                                        a["out"], 0, 2 << 30, 1 << 20, a["status"])

    for name in ("table", "ctx", "nq", "off", "status"):
        for at in (out, out + 12):
            assert call(**{name: at}) == INVALID, (name, at)
    for at in (pool, pool + size - 16):
        assert call(out=at) == INVALID


def test_bs8_binding_refuses_outputs_over_lists(fake):
    words = torch.zeros(40000, dtype=i32)
    out = words[:4 * 16 * 256].view(torch.float32).view(4, 16, 256)
    t = _verify_args(out=out)
    call = lambda t, status=None: api.bs8_verify_attn(t["desc"], t["pool"], t["table"], t["ctx"], t["nq"], t["off"], 100, 4, 0, t["q"], t["out"],  # noqa: E731
                                                      t["ws"], status=status)
    call(t, status=torch.zeros(1, dtype=i32))
    for kw in (dict(table=words[100:106].view(2, 3)), dict(ctx=words[:2]), dict(nq=words[16380:16382]), dict(off=words[16383:16386])):
        with pytest.raises(ValueError, match="out overlaps"):
            call(dict(t, **kw))
    with pytest.raises(ValueError, match="out overlaps the status"):
        call(t, status=words[7:8])
    call(dict(t, off=words[16384:16387]))
