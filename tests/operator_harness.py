"""A device cache of any format with its decoded keys, for the tests of the operators around the cache."""
from __future__ import annotations

import numpy as np
import torch

import q3kv_inputs as qi
from oracle import codec, fp8, packing, turbo5k
from oracle.wht import rotate_f64
from speculative_verify_attention_q3kv_gb300 import api

POOL_BYTES = {"q3": api.pool_bytes, "fp8": api.fp8_pool_bytes, "t5k": api.t5k_pool_bytes}
APPEND = {"q3": api.append, "fp8": api.fp8_append, "t5k": api.t5k_append}
MASS = {"q3": api.attn_mass, "fp8": api.fp8_attn_mass, "t5k": api.t5k_attn_mass}
VERIFY = {"q3": api.verify_attn, "fp8": api.fp8_verify_attn, "t5k": api.t5k_verify_attn}
VERIFY_LSE = {"q3": api.verify_attn_lse, "fp8": api.fp8_verify_attn_lse, "t5k": api.t5k_verify_attn_lse}
EVICT = {"q3": api.evict, "fp8": api.fp8_evict, "t5k": api.t5k_evict}


def i32(values):
    return torch.tensor(np.asarray(values, np.int32)).cuda()


def offsets(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


class Cache:
    """Slots of the given lengths filled with random rows; extra_pages stay free for evictions."""

    def __init__(self, fmt, lengths, kv_heads=2, layers=1, seed=0, extra_pages=0, scale=1.0, dtype=torch.float32):
        self.fmt, self.lengths, self.kv, self.layers = fmt, list(lengths), kv_heads, layers
        pages = [max(1, (n + 255) // 256) for n in lengths]
        self.num_pages = sum(pages) + extra_pages
        self.desc = api.make_desc(layers, kv_heads, self.num_pages)
        self.pool = torch.zeros(POOL_BYTES[fmt](self.desc), dtype=torch.uint8, device="cuda")
        rng = np.random.default_rng(seed)
        order = rng.permutation(self.num_pages).astype(np.int32)
        self.pt = np.full((len(pages), max(pages)), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.pt[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.page_table = torch.from_numpy(self.pt).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        total = sum(lengths)
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        for layer in range(layers):
            k = (scale * torch.randn((total, kv_heads, 256), generator=gen, device="cuda")).to(dtype)
            v = torch.randn((total, kv_heads, 256), generator=gen, device="cuda").to(dtype)
            APPEND[fmt](self.desc, self.pool, self.page_table, i32([0] * len(lengths)), i32(lengths), offsets(lengths),
                        max(lengths), layer, k, v, self.status)

    def records(self, page_row, layer, g, kv, positions):
        """Bytes of the records at the given positions of a page-table row."""
        pos = np.asarray(positions, np.int64)
        pages = np.asarray(page_row, np.int64)[pos // 256]
        if self.fmt == "t5k":
            fn, size = (turbo5k.k_offset, 164) if kv == 0 else (turbo5k.v_offset, 112)
            offs = fn(self.layers, self.kv, pages, layer, g, pos % 256)
        else:
            size = 112 if self.fmt == "q3" else 256
            offs = ((((pages * self.layers + layer) * self.kv + g) * 2 + kv) * 256 + pos % 256) * size
        idx = torch.from_numpy(offs[:, None] + np.arange(size)[None, :]).cuda()
        return self.pool[idx].cpu().numpy()

    def k_hat(self, slot, layer, g, n=None):
        """float64 keys [n, 256] in the cache's basis."""
        rec = self.records(self.pt[slot], layer, g, 0, np.arange(self.lengths[slot] if n is None else n))
        if self.fmt == "q3":
            return codec.dequantize(*packing.unpack_records(rec))
        if self.fmt == "fp8":
            return fp8.decode(rec).astype(np.float64)
        return turbo5k.decode_k(*turbo5k.unpack_k(rec)).astype(np.float64)

    def q_basis(self, q):
        """float64 queries in the cache's basis."""
        q = np.asarray(q, np.float64)
        return q if self.fmt == "fp8" else rotate_f64(q)


def queries(rows, heads, seed, dtype=torch.float32, scale=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((rows, heads, 256), generator=gen, device="cuda")).to(dtype)
