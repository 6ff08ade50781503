"""The operators in the order a serving loop runs them, against one float64 model of the whole.

prompt (rotate, append) -> step (rotate, append, verify with the statistic, accept
sampled drafts, accumulate the mass over the committed tokens) -> eviction into
fresh pages -> another step on the evicted cache.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from operator_harness import i32, offsets
from oracle import eviction as ev
from oracle import rope as ref
from oracle.attention import verify_attention
from oracle.cache import encode_dequantized
from oracle.wht import rotate_f64
from speculative_verify_attention_q3kv_gb300 import api

pytestmark = pytest.mark.gpu

KW = dict(rotary_dim=64, theta=1e6, sections=(11, 11, 10), deal_axes=True)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_prompt_step_evict_step():
    S, KV, N, T, V = 2, 2, [700, 300], 5, 4000
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    alloc = api.Allocator(16, 2 * S, 4)                # a second slot id per slot holds its evicted pages
    rows = [alloc.alloc_pages(b, N[b] + T) for b in range(S)]
    table = torch.from_numpy(np.stack(rows)).cuda()
    desc = api.make_desc(1, KV, 16)
    pool = torch.zeros(api.pool_bytes(desc), dtype=torch.uint8, device="cuda")
    plan = api.make_rope_plan(**KW)
    status = i32([0])
    keys = [np.zeros((0, KV, 256)) for _ in range(S)]  # what the cache holds, as float64 rotated inputs
    vals = [np.zeros((0, KV, 256)) for _ in range(S)]

    def run(lens, new, positions, q_wanted):
        """Rotates and appends `new` tokens per slot at `lens`; returns the rotated queries."""
        total = sum(new)
        qkv = rn(total, (16 + 2 * KV) * 256)
        q, k = qkv[:, :4096].unflatten(1, (16, 256)), qkv[:, 4096:4096 + KV * 256].unflatten(1, (KV, 256))
        v = qkv[:, 4096 + KV * 256:].unflatten(1, (KV, 256)).contiguous()
        qr, kr = torch.empty((total, 16, 256), device="cuda"), torch.empty((total, KV, 256), device="cuda")
        raw = k.double().cpu().numpy()
        api.rope(plan, positions, q, qr, k, kr)
        # the rotation itself, with the tolerance of its own tests
        want = ref.rotate(raw, positions.cpu().numpy(), **KW)
        assert np.abs(kr.double().cpu().numpy() - want).max() <= 1e-6 * 2 * np.abs(raw).max()
        api.append(desc, pool, table, i32(lens), i32(new), offsets(new), max(new), 0, kr, v, status)
        at = 0
        for b, n in enumerate(new):
            keys[b] = np.concatenate([keys[b][:lens[b]], kr[at:at + n].cpu().numpy()])
            vals[b] = np.concatenate([vals[b][:lens[b]], v[at:at + n].cpu().numpy()])
            at += n
        return qr

    def check_attention(out, lse, qr, lens, T):
        for b in range(S):
            kh = np.stack([encode_dequantized(keys[b][:, g].astype(np.float32)) for g in range(KV)])
            vh = np.stack([encode_dequantized(vals[b][:, g].astype(np.float32)) for g in range(KV)])
            q = qr[b * T:(b + 1) * T].double().cpu().numpy()
            want = verify_attention(q, kh, vh, lens[b] - T, 8)
            got = out[b * T:(b + 1) * T].double().cpu().numpy()
            assert np.abs(got - want).max() <= 2e-3          # the library's bound for verify outputs
            for g in range(KV):
                s = ev.scores(rotate_f64(q[:, 8 * g:8 * g + 8]), kh[g], lens[b] - T, 8)
                l64 = ev.log_sum_exp(s)
                l32 = lse[b * T:(b + 1) * T, 8 * g:8 * g + 8].double().cpu().numpy().reshape(-1)
                assert np.abs(l32 - l64).max() <= 1e-4
        return None

    def verify(qr, lens, T):
        out, lse = torch.empty((S * T, 16, 256), device="cuda"), torch.empty((S * T, 16), device="cuda")
        ws = torch.zeros(api.workspace_bytes(desc, S, max(lens), T), dtype=torch.uint8, device="cuda")
        api.verify_attn_lse(desc, pool, table, i32(lens), i32([T] * S), offsets([T] * S), max(lens), T, 0, qr, out, lse, ws, status=status)
        return out, lse

    # ---- prompt
    pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in N])[:, None].expand(-1, 3).contiguous()
    run([0] * S, N, pos, False)

    # ---- step 1
    pos = torch.cat([n + torch.arange(T, device="cuda", dtype=torch.int32) for n in N])[:, None].expand(-1, 3).contiguous()
    qr = run(N, [T] * S, pos, True)
    lens = [n + T for n in N]
    out, lse = verify(qr, lens, T)
    check_attention(out, lse, qr, lens, T)
    logits = 3.0 * rn(S * T, V)
    draft = torch.softmax(logits + rn(S * T, V), dim=1)
    tokens = torch.roll(torch.multinomial(draft, 1, generator=gen).flatten().to(torch.int32), 1).contiguous()
    uni = torch.rand(S * T, generator=gen, device="cuda")
    acc, nxt, committed = i32([0] * S), i32([0] * S), i32([0] * S)
    ws = torch.zeros(api.accept_draft_workspace_bytes(S, S * T, V), dtype=torch.uint8, device="cuda")
    api.accept_draft(logits, draft, offsets([T] * S), i32([T] * S), tokens, T, i32(lens), 1.0, uni, 7, acc, nxt, committed, ws, status=status)
    mass = torch.zeros((1, S, KV, max(lens)), device="cuda")
    kept_q = acc + 1                                    # t_0 and the accepted drafts
    api.attn_mass(desc, pool, table, committed, kept_q, offsets([T] * S), max(lens), T, 0, qr, lse, 1.0, mass[0], status=status)
    a, c = acc.tolist(), committed.tolist()
    assert c == [lens[b] - (T - 1 - a[b]) for b in range(S)]
    for b in range(S):
        # the committed rows' weights add up to one each
        got = mass[0, b, :, :c[b]].double().sum(dim=1).cpu().numpy()
        assert np.allclose(got, 8.0 * (a[b] + 1), rtol=1e-3) and float(mass[0, b, :, c[b]:].abs().max() if c[b] < max(lens) else 0) == 0.0

    # ---- eviction into fresh pages, then the old ones go back
    budget = [256, 200]
    dst = torch.from_numpy(np.stack([alloc.alloc_pages(S + b, budget[b] + T) for b in range(S)])).cuda()
    kept = torch.zeros((1, S, KV, 256), dtype=torch.int32, device="cuda")
    mass_out = torch.zeros((1, S, KV, 256), device="cuda")
    new_len = i32([0] * S)
    api.evict(desc, pool, table, committed, max(lens), i32(budget), 256, 4, 64, 0, mass, dst, kept, mass_out, new_len, status=status)
    torch.cuda.synchronize()
    assert new_len.tolist() == budget
    for b in range(S):
        k2, v2 = np.zeros((budget[b], KV, 256)), np.zeros((budget[b], KV, 256))
        for g in range(KV):
            want = ev.keep(mass[0, b, g, :c[b]].cpu().numpy(), budget[b], 4, 64)
            assert np.array_equal(kept[0, b, g, :budget[b]].cpu().numpy(), want)
            k2[:, g], v2[:, g] = keys[b][want, g], vals[b][want, g]
        keys[b], vals[b] = k2, v2
        alloc.free_slot(b)
    table = dst

    # ---- step 2 on the evicted cache: positions go on from the committed lengths, rows from the new ones
    pos = torch.cat([c[b] + torch.arange(T, device="cuda", dtype=torch.int32) for b in range(S)])[:, None].expand(-1, 3).contiguous()
    qr = run(budget, [T] * S, pos, True)
    lens = [n + T for n in budget]
    out, lse = verify(qr, lens, T)
    check_attention(out, lse, qr, lens, T)
    stride = max(lens)
    m2 = torch.zeros((S, KV, stride), device="cuda")
    m2[:, :, :256] = mass_out[0]
    before = m2.clone()
    api.attn_mass(desc, pool, table, i32(lens), i32([T] * S), offsets([T] * S), max(lens), T, 0, qr, lse, 0.5, m2, status=status)
    for b in range(S):
        n = budget[b]
        grown = m2[b, :, :lens[b]].double().sum(dim=1) - 0.5 * before[b, :, :n].double().sum(dim=1)
        assert torch.allclose(grown, torch.full_like(grown, 8.0 * T), rtol=1e-3)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


_FIRST_CALLS = """
import torch
from speculative_verify_attention_q3kv_gb300 import api
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
desc = api.make_desc(1, 2, 8)
pool = torch.zeros(api.pool_bytes(desc), dtype=torch.uint8, device="cuda")
table, dst = i32(0, 1, 2, 3)[None], i32(4, 5)[None]
q, k = torch.randn(3, 16, 256, device="cuda"), torch.randn(3, 2, 256, device="cuda")
q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
pos, ctx, n, off = i32(1, 2, 3)[:, None], i32(900), i32(3), i32(0, 3)
lse, mass = torch.zeros(3, 16, device="cuda"), torch.zeros(1, 1, 2, 1024, device="cuda")
out, ws = torch.zeros(3, 16, 256, device="cuda"), torch.zeros(api.workspace_bytes(desc, 1, 900, 3), dtype=torch.uint8, device="cuda")
kept, new, budget = torch.zeros(1, 1, 2, 300, dtype=torch.int32, device="cuda"), i32(0), i32(300)
logits, draft = torch.randn(3, 5000, device="cuda"), torch.full((3, 5000), 1 / 5000, device="cuda")
ws2 = torch.zeros(api.accept_draft_workspace_bytes(1, 3, 5000), dtype=torch.uint8, device="cuda")
uni, tok, acc, nxt, com, st = torch.rand(3, device="cuda"), i32(5, 6, 7), i32(0), i32(0), i32(0), i32(0)
plan = api.make_rope_plan(64, 1e4, (32,))
def step():
    api.rope(plan, pos, q, q2, k, k2)
    api.verify_attn_lse(desc, pool, table, ctx, n, off, 900, 3, 0, q2, out, lse, ws, status=st)
    api.attn_mass(desc, pool, table, ctx, n, off, 900, 3, 0, q2, lse, 0.0, mass[0], status=st)
    api.evict(desc, pool, table, ctx, 900, budget, 300, 2, 9, 0, mass, dst, kept, None, new, status=st)
    api.accept_draft(logits, draft, off, n, tok, 3, ctx, 1.0, uni, 5, acc, nxt, com, ws2, status=st)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (q2, k2, lse, mass, kept, new, acc, nxt, com, st)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (q2, k2, lse, mass, kept, new, acc, nxt, com, st)))
assert new.item() == 300 and st.item() == 0 and abs(mass.sum().item() - 48) < 1e-2
print("captured")
"""


def test_the_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], capture_output=True, text=True, timeout=240, cwd=root)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
