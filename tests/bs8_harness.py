"""A block-scaled 8-bit device cache and the float64 definition of its attention, for the GPU tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import bs8, fp8
from speculative_verify_attention_q3kv_gb300 import _lib, api

FMA, MMA = _lib.Q3KV_IMPL_FMA, _lib.Q3KV_IMPL_MMA


def i32(values):
    return torch.tensor(np.asarray(values, np.int32)).cuda()


def offsets(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


class Bs8Cache:
    """Slots over a pool whose unused bytes are NaN codes and NaN scales, pages in random order."""

    def __init__(self, room, kv=2, layers=1, seed=0, extra_pages=0):
        self.kv, self.layers = kv, layers
        pages = [max(1, (n + 255) // 256) for n in room]
        self.num_pages = sum(pages) + extra_pages
        self.desc = api.make_desc(layers, kv, self.num_pages)
        self.pool = torch.full((api.bs8_pool_bytes(self.desc),), 0xFF, dtype=torch.uint8, device="cuda")
        order = np.random.default_rng(seed).permutation(self.num_pages).astype(np.int32)
        self.pt = np.full((len(pages), max(pages)), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.pt[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.page_table = torch.from_numpy(self.pt).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, starts, k_rows, v_rows, layer=0, dtype=torch.float32, stream=None):
        """k_rows, v_rows: per slot float arrays [n, kv, 256]."""
        n = [len(x) for x in k_rows]
        cat = lambda rows: torch.from_numpy(np.concatenate([np.asarray(x, np.float32).reshape(-1, self.kv, 256) for x in rows])).cuda().to(dtype)  # noqa: E731
        api.bs8_append(self.desc, self.pool, self.page_table, i32(starts), i32(n), offsets(n), max(n), layer, cat(k_rows), cat(v_rows),
                       self.status, stream)

    def fill(self, lengths, seed=0, layer=0, dtype=torch.float32, k_scale=1.0, v_scale=1.0, shape=None):
        """Random rows for every slot; shape(x, slot) may change them (float32 [n, kv, 256] K then V)."""
        rng = np.random.default_rng(seed)
        ks = [(k_scale * rng.standard_normal((n, self.kv, 256))).astype(np.float32) for n in lengths]
        vs = [(v_scale * rng.standard_normal((n, self.kv, 256))).astype(np.float32) for n in lengths]
        if shape:
            ks, vs = zip(*[shape(k, v, b) for b, (k, v) in enumerate(zip(ks, vs))])
        self.append([0] * len(lengths), ks, vs, layer, dtype)

    def unit(self, page, layer, g, kv):
        at = bs8.unit_offset(self.layers, self.kv, int(page), layer, g, kv)
        return self.pool[at:at + bs8.UNIT_BYTES].cpu().numpy()

    def raw(self, slot, n, layer, g, kv):
        """(codes [n, 256], scales per block) of a slot's first n positions."""
        codes, scales = [], []
        for p in range((n + 255) // 256):
            u = self.unit(self.pt[slot, p], layer, g, kv)
            rows = np.arange(min(256, n - 256 * p))
            codes.append(bs8.read_codes(u, rows))
            scales.append(bs8.read_scales(u)[:(len(rows) + 15) // 16])
        return np.concatenate(codes), np.concatenate(scales)

    def values(self, slot, n, layer=0):
        """float64 K, V [kv, n, 256]."""
        out = []
        for kv in range(2):
            per = []
            for g in range(self.kv):
                c, s = self.raw(slot, n, layer, g, kv)
                per.append(fp8.decode(c) * np.repeat(s.astype(np.float64), 16)[:n, None])
            out.append(np.stack(per))
        return out

    def workspace(self, L, T, slots=None):
        n = api.bs8_workspace_bytes(self.desc, len(L) if slots is None else slots, max(L), max(T))
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def verify(self, L, T, q, layer=0, impl=0, gap=0, stream=None, ws=None, out=None, max_ctx=None, max_nq=None):
        """Output rows; `gap` rows in front belong to no slot."""
        offs = i32(gap + np.concatenate([[0], np.cumsum(np.maximum(T, 0))]))
        if out is None:
            out = torch.full_like(q, 77.0)
        ws = self.workspace([max(L)], [max(T)], len(L)) if ws is None else ws
        api.bs8_verify_attn(self.desc, self.pool, self.page_table, i32(L), i32(T), offs, max_ctx or max(L), max_nq or max(max(T), 1), layer,
                            q, out, ws, impl, self.status, stream)
        return out


def queries(rows, kv, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((rows, 8 * kv, 256), generator=g, device="cuda")).to(dtype)


def reference(q, k, v, n_ctx, kind, hidden=None):
    """float64 output of one slot and its tolerance.  q [T, Hq, 256] float64 as the call sees it; k, v decoded.

    Errors, relative to A = sum w |v| (the weighted mean magnitude, which bounds what relative errors of the weights do):
    - the score s in float32: the products' sum is off by at most 2^-22 G, G = sum |q_d k_d| / 16 (a few additions of
      exact products per 32 dims; the CUDA-core leg adds 256 terms one after the other, 2^-16 G), the steps to the
      exponent by 2^-22 (|s| + max |s|) in all, and 2^x by 2^-22: twice their sum, for weight and row sum;
    - bf16 queries: codes below 2^-17 of the row's largest value are rounded away, 2^-18 max|q| sum |k_d| / 16 at most;
    - bf16's weights in three codes: 2^-9 and the rounding to fp16 before them, 2^-11 (half of fp16's step);
      float32's in six: 2^-23;
    - a code's smallest step against largest weights of 2^8 or more: half of 2^-21 (bf16; half of fp16's 2^-24 before) or of
      2^-27 (float32), 2^-29 in all or 2^-36 per position;
    - sums in float32 over the tiles of one CTA and the partials, and the row sum: 2^-16;
    and the output's own rounding, half a step: 2^-8 (bf16) or 2^-24 of the value.
    """
    T, Hq, _ = q.shape
    L = k.shape[1]
    group = Hq // k.shape[0]
    out, tol = np.zeros((T, Hq, 256)), np.zeros((T, Hq, 256))
    mask = np.arange(L)[None, :] > n_ctx + np.arange(T)[:, None]
    if hidden is not None:
        mask = mask | hidden[None, :]
    for h in range(Hq):
        K, V = k[h // group], v[h // group]
        s = q[:, h] @ K.T / 16.0
        G = np.abs(q[:, h]) @ np.abs(K).T / 16.0
        s[mask], G[mask] = -np.inf, 0.0
        m = s.max(axis=1, keepdims=True)
        empty = ~np.isfinite(m[:, 0])
        p = np.where(mask, 0.0, np.exp(s - np.where(np.isfinite(m), m, 0.0)))
        w = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        out[:, h] = w @ V
        A = w @ np.abs(V)
        big = np.abs(np.where(mask, 0.0, s)).max(axis=1, keepdims=True)
        e = 2.0 ** (-16 if kind == "fma" else -22) * G.max(axis=1, keepdims=True) + 2.0 ** -21 * big + 2.0 ** -22
        if kind == "bf16":
            visible = np.where(mask, 0.0, np.abs(K).sum(axis=1)[None, :]).max(axis=1, keepdims=True)
            e = e + 2.0 ** -18 * np.abs(q[:, h]).max(axis=1, keepdims=True) * visible / 16.0
        c = {"bf16": 2.0 ** -9 + 2.0 ** -11, "f32": 2.0 ** -23, "fma": 0.0}[kind] + 2.0 * e + 2.0 ** -16
        floor = L * {"bf16": 2.0 ** -29, "f32": 2.0 ** -36, "fma": 0.0}[kind] * np.abs(V).max()
        tol[:, h] = c * A + floor + 2.0 ** -24 * np.abs(out[:, h])
        out[empty, h] = 0.0
    return out, tol


def check(got, q, cache, L, T, kind, layer=0, gap=0, hidden=None):
    """Every slot's rows of an output against the definition."""
    at = gap
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got, qf = got.double().cpu().numpy(), q.double().cpu().numpy()
    assert np.all(got[:gap] == 77.0)
    for b, (n, t) in enumerate(zip(L, T)):
        if t > 0:
            k, v = cache.values(b, n, layer)
            want, tol = reference(qf[at:at + t], k, v, n - t, kind, None if hidden is None else hidden[b])
            err = np.abs(got[at:at + t] - want)
            tol = tol + rounding * (np.abs(want) + tol)
            assert np.all(err <= tol), (b, n, t, float((err / tol).max()), float(err.max()))
            at += t
    assert np.all(got[at:] == 77.0)
