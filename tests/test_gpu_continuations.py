"""The operators of many continuations of one context, run together as a serving loop would."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from bs8_harness import Bs8Cache, check, i32, offsets
from oracle import logits as ref
from speculative_verify_attention_q3kv_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, "bf16"), (torch.float32, "f32")])
def test_forked_continuations(dtype, kind):
    """One prompt, three forks: each appends drafts of its own into copies on write, attends, processes its logits, accepts
    greedily, counts what it committed and rolls back; in between the pool is compacted."""
    kv, vocab, slots, widths = 2, 1003, 3, [5, 3, 1]
    rng = np.random.default_rng(0)
    cache = Bs8Cache([256 * 24], kv=kv)                  # a pool of 24 pages; its own table is not used
    alloc = api.Allocator(24, slots + 1, 8)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731

    def table(rows):
        cache.pt = np.stack(rows)
        cache.page_table = torch.from_numpy(cache.pt).cuda()

    # something else holds the first pages, so that forks lie high in the pool and have to move later
    alloc.alloc_pages(slots, 700)
    prompt = rng.integers(0, 200, 300).astype(np.int32)
    table([alloc.alloc_pages(0, 300)])
    k, v = rand(300, kv, 256), rand(300, kv, 256)
    api.bs8_append(cache.desc, cache.pool, cache.page_table, i32([0]), i32([300]), i32([0, 300]), 300, 0, k, v, cache.status)
    for b in (1, 2):
        alloc.fork(0, b, 300)
    keys, values = [[k.clone()] for _ in range(slots)], [[v.clone()] for _ in range(slots)]
    counts, want_counts = torch.zeros((slots, 1008), dtype=torch.int16, device="cuda"), np.zeros((slots, 1008), np.int16)
    api.count_tokens(counts, vocab, i32(np.tile(prompt, slots)), i32([0, 300, 600]), i32([300] * slots), 300, prompt=True)
    for b in range(slots):
        ref.count(want_counts[b, :vocab], prompt, True)
    theta, alpha = torch.full((slots,), 1.3, device="cuda"), torch.full((slots,), 0.2, device="cuda")
    length, rows = [300] * slots, sum(widths)
    offs, n_q = offsets(widths), i32(widths)
    for step in range(60):
        # pages for the step; the first write of a fork copies the shared page's filled part
        copies, tabs = [], []
        for b in range(slots):
            row, copy = alloc.write(b, length[b], widths[b])
            tabs.append(row)
            copies += [copy] if copy else []
        if copies:
            src, dst, part = zip(*copies)
            api.bs8_copy_pages(cache.desc, cache.pool, i32(src), i32(dst), rows=i32(part), status=cache.status)
            assert step == 0 and len(copies) == 2 and part == (44, 44)
        table(tabs)
        k, v, q = rand(rows, kv, 256), rand(rows, kv, 256), rand(rows, 8 * kv, 256)
        ctx = i32(length)
        api.bs8_append(cache.desc, cache.pool, cache.page_table, ctx, n_q, offs, max(widths), 0, k, v, cache.status)
        L = [n + t for n, t in zip(length, widths)]
        out = cache.verify(L, widths, q)
        if step in (0, 1, 33, 59):
            check(out, q, cache, L, widths, kind)
            at = 0
            for b, w in enumerate(widths):               # the records are still near the rows that went in
                kk = torch.cat(keys[b] + [k[at:at + w]]).double().cpu().numpy()
                got = cache.values(b, L[b])[0]
                # half a step of a value is 2^-4 of it; half of the smallest step, 2^-10 2^e, with 2^e <= 2 max / 448, once per
                # rounding: the append's and one growth's at most where it matters
                kk = kk.transpose(1, 0, 2)
                assert np.all(np.abs(got - kk) <= np.abs(kk) * 2.0 ** -3 + 2 * np.abs(kk).max() / 448 * 2.0 ** -9)
                at += w
        # logits that favour the drafts about half of the time
        tokens = rng.integers(0, vocab, rows).astype(np.int32)
        lg = rand(rows, vocab)
        for r in range(rows - 1):
            if rng.random() < 0.6:
                lg[r, tokens[r + 1]] = 30.0
        done = torch.empty_like(lg)
        api.process_logits(lg, done, offs, n_q, i32(tokens), max(widths), counts=counts, repetition=theta, frequency=alpha)
        acc, nxt, com = i32([0] * slots), i32([0] * slots), i32(L)
        ws = torch.empty(api.accept_workspace_bytes(rows, vocab), dtype=torch.uint8, device="cuda")
        api.accept_greedy(done, offs, n_q, i32(tokens), max(widths), com, acc, nxt, com, ws, cache.status)
        api.count_tokens(counts, vocab, i32(tokens), offs, acc + 1, max(widths))
        taken, com = acc.cpu().tolist(), com.cpu().tolist()
        at = 0
        for b, w in enumerate(widths):
            want = ref.process(lg[at:at + w].double().cpu().numpy(), tokens[at:at + w].tolist(), want_counts[b], 1.3000000, 0.2, 0.0)
            best = want.argmax(axis=1)
            a = 0
            while a < w - 1 and tokens[at + a + 1] == best[a]:
                a += 1
            second = np.sort(want, axis=1)[:, -2:]
            if np.all(second[:, 1] - second[:, 0] > 0.3):  # otherwise rounding may decide
                assert taken[b] == a
            ref.count(want_counts[b, :vocab], tokens[at:at + taken[b] + 1], False)
            assert com[b] == length[b] + taken[b] + 1
            keys[b].append(k[at:at + taken[b] + 1])
            values[b].append(v[at:at + taken[b] + 1])
            length[b] = com[b]
            alloc.trim(b, length[b])
            at += w
        if step == 30:                                   # the other holder leaves, the pool is packed
            alloc.free_slot(slots)
            src, dst = alloc.compact(24)
            assert len(src) > 0
            api.bs8_copy_pages(cache.desc, cache.pool, i32(src), i32(dst), status=cache.status)
            held = {int(x) for b in range(slots) for x in alloc.pages(b) if x >= 0}
            assert held == set(range(len(held)))
    assert np.array_equal(counts.cpu().numpy(), want_counts) and int(cache.status) == 0
    for b in range(slots):
        alloc.free_slot(b)
    assert alloc.free_pages() == 24


_FIRST_CALLS = """
import torch
from speculative_verify_attention_q3kv_gb300 import api
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
desc = api.make_desc(1, 2, 8)
pool = torch.zeros(api.bs8_pool_bytes(desc), dtype=torch.uint8, device="cuda")
table, ctx, n, off, at = i32(0, 1, 2, 3)[None], i32(900), i32(3), i32(0, 3), i32(897)
gen = torch.Generator(device="cuda").manual_seed(0)
k0, v0 = (torch.randn(897, 2, 256, generator=gen, device="cuda") for _ in range(2))
k, v = (torch.randn(3, 2, 256, generator=gen, device="cuda") for _ in range(2))
q = torch.randn(3, 16, 256, generator=gen, device="cuda")
outs = [torch.zeros(3, 16, 256, device="cuda", dtype=d) for d in (torch.float32, torch.float32, torch.bfloat16)]
ws = torch.zeros(api.bs8_workspace_bytes(desc, 1, 900, 3), dtype=torch.uint8, device="cuda")
logits, done = torch.randn(3, 5001, generator=gen, device="cuda"), torch.zeros(3, 5001, device="cuda")
counts, tok, st = torch.zeros(1, 5008, dtype=torch.int16, device="cuda"), i32(5, 6, 7), i32(0)
history, zero, many, theta = torch.randint(0, 5001, (2000,), generator=gen, dtype=torch.int32, device="cuda"), i32(0), i32(2000), torch.full((1,), 1.5, device="cuda")
qb = q.bfloat16()
def step():
    counts.zero_()
    api.bs8_append(desc, pool, table, i32_zero, len0, off0, 897, 0, k0, v0, st)
    api.bs8_append(desc, pool, table, at, n, off, 3, 0, k, v, st)
    api.bs8_verify_attn(desc, pool, table, ctx, n, off, 900, 3, 0, q, outs[0], ws, status=st)
    api.bs8_verify_attn(desc, pool, table, ctx, n, off, 900, 3, 0, q, outs[1], ws, impl=1, status=st)
    api.bs8_verify_attn(desc, pool, table, ctx, n, off, 900, 3, 0, qb, outs[2], ws, status=st)
    api.bs8_copy_pages(desc, pool, src, dst, status=st)
    api.count_tokens(counts, 5001, history, zero, many, 2000, status=st)
    api.count_tokens(counts, 5001, tok, off, n, 3, status=st)
    api.process_logits(logits, done, off, n, tok, 3, counts=counts, repetition=theta, status=st)
i32_zero, len0, off0, src, dst = i32(0), i32(897), i32(0, 897), i32(0, 1), i32(6, 7)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (*outs, pool, counts, done, st)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (*outs, pool, counts, done, st)))
assert st.item() == 0 and int((counts & 0x7fff).sum()) == 2003 and float((outs[0] - outs[1]).abs().max()) < 1e-3
print("captured")
"""


def test_the_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], capture_output=True, text=True, timeout=240, cwd=root)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
