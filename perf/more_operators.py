"""Cases of the operators that serve many continuations of one context, with their plain forms.

Five operators, each in its plain form (elementary torch operations) and as the library's call:

  append   quantise-append into the cache of 8-bit codes with a power-of-two scale per block of 16 positions and head
  attn     verify attention over that cache
  copy     pages copied within a pool: what a fork's first write and a compaction ask for
  count    committed or prompt tokens counted into the slots' token counts
  logits   penalties for repeated tokens, biases and grammar masks on the logits of a verify step

Sizes follow the repository's own workloads: 2 kv heads and 16 q heads of 256 dims, 256-position pages, contexts up to
655,360 positions, up to 16 query tokens per slot, a vocabulary of 248,320.
"""
import math

import torch

own = False

D = 256                       # head dim
PAGE = 256                    # positions per page
GROUP = 8                     # q heads per kv head
BLOCK = 16                    # positions that share a scale
UNIT = PAGE * D + 4 * PAGE // BLOCK     # bytes of one (page, layer, head, K or V): codes, then scales
RECORD = {"q3": 112, "fp8": 256}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the K and V of one slot's verify step, in the middle of a block whose scale may have to grow
        dict(name="append step of 6 tokens", op="append", slots=1, tokens=6, ragged=False, before=32761, kv=2, dtype="bf16"),
        # a batch of ragged prompts behind prefixes that are already there
        dict(name="append 8 prompts of 4096", op="append", slots=8, tokens=4096, ragged=True, before=1000, kv=2, dtype="bf16"),
        # plain decoding of a ragged batch
        dict(name="attn 8 slots x 1 token", op="attn", slots=8, ctx=16384, ragged=True, tokens=1, kv=2, dtype="bf16"),
        # one slot's verify step at 32K
        dict(name="attn 32768 x 6", op="attn", slots=1, ctx=32768, ragged=False, tokens=6, kv=2, dtype="bf16"),
        # the longest context
        dict(name="attn 655360 x 8", op="attn", slots=1, ctx=655360, ragged=False, tokens=8, kv=2, dtype="bf16"),
        # float32 queries, the widest step, short ragged contexts
        dict(name="attn 5 slots x 16 tokens f32", op="attn", slots=5, ctx=4001, ragged=True, tokens=16, kv=2, dtype="f32"),
        # eight forks write for the first time: the filled part of each one's last page, all layers
        dict(name="copy 8 last pages, 16 layers", op="copy", fmt="q3", layers=16, kv=2, pages=8, partial=True),
        # a pool is compacted: 400 pages of 16 layers move
        dict(name="copy 400 pages, 16 layers", op="copy", fmt="q3", layers=16, kv=2, pages=400, partial=False),
        # a step's committed tokens of a batch
        dict(name="count 64 slots x 5 tokens", op="count", slots=64, tokens=5, ragged=True, vocab=248320, prompt=False),
        # the tokens of long histories are counted when their slots come back
        dict(name="count 8 histories of 65536", op="count", slots=8, tokens=65536, ragged=True, vocab=248320, prompt=False),
        # one slot's verify step under a grammar, with penalties
        dict(name="logits 1 slot x 6", op="logits", slots=1, tokens=6, ragged=False, vocab=248320, dtype="bf16", penalties=True, biases=0,
             mask=True),
        # a batch in float32 of an odd vocabulary, penalties, a few hundred biases and masks
        dict(name="logits 8 slots x 16 f32", op="logits", slots=8, tokens=16, ragged=True, vocab=100003, dtype="f32", penalties=True,
             biases=300, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "copy", "count", "logits"])
    if op == "append":
        kv, slots = rng.choice([1, 2, 4]), _log(rng, 1, 16)
        return dict(op=op, slots=slots, tokens=_log(rng, 1, 8 * 4096 * 2 // (kv * slots)), ragged=rng.random() < 0.7,
                    before=rng.choice([0, rng.randint(1, 300), _log(rng, 300, 20000)]), kv=kv, dtype=rng.choice(["bf16", "f32"]))
    if op == "attn":
        kv, tokens, slots, dtype = rng.choice([1, 2, 4]), rng.randint(1, 16), _log(rng, 1, 16), rng.choice(["bf16", "bf16", "f32"])
        most = 655360 * 2 * 8 // (kv * max(tokens, 8) * slots * (8 if dtype == "f32" else 1))
        return dict(op=op, slots=slots, ctx=_log(rng, min(20, most), most), ragged=rng.random() < 0.7, tokens=tokens, kv=kv, dtype=dtype)
    if op == "copy":
        fmt, layers, kv = rng.choice(["q3", "q3", "fp8", "bs8"]), rng.choice([1, 2, 4, 16]), rng.choice([1, 2, 4])
        most = 400 * 16 * 2 // (layers * kv * (1 if fmt == "q3" else 3))
        return dict(op=op, fmt=fmt, layers=layers, kv=kv, pages=_log(rng, 1, min(most, 3000)), partial=rng.random() < 0.5)
    if op == "count":
        slots = _log(rng, 1, 64)
        return dict(op=op, slots=slots, tokens=_log(rng, 1, 65536 * 8 // slots), ragged=rng.random() < 0.7, vocab=_log(rng, 1000, 248320),
                    prompt=rng.random() < 0.5)
    slots, tokens, dtype = _log(rng, 1, 32), rng.randint(1, 16), rng.choice(["bf16", "f32"])
    most = 8 * 16 * 100003 // (slots * tokens)
    return dict(op=op, slots=slots, tokens=tokens, ragged=rng.random() < 0.7, vocab=_log(rng, 1000, min(most, 248320)), dtype=dtype,
                penalties=rng.random() < 0.8, biases=rng.choice([0, 0, 1, 300]), mask=rng.random() < 0.6)


def _lengths(case):
    """Per-slot lengths of an attention case: the first slot has the longest, the others spread down to a quarter of it."""
    n, c = case["slots"], case["ctx"]
    lengths = [max(1, c - (c * 3 // 4) * b // max(1, n - 1) - b) if case["ragged"] and b else c for b in range(n)]
    return [max(x, w) for x, w in zip(lengths, _widths(case))]


def _widths(case):
    """Tokens per slot: ragged slots cycle from the widest down to one."""
    t = case["tokens"]
    return [1 + (t - 1 - 3 * b) % t if case["ragged"] else t for b in range(case["slots"])]


def _counted(case):
    """Tokens per slot of an append or a count: ragged slots spread down to a quarter."""
    t, n = case["tokens"], case["slots"]
    return [max(1, t - (t * 3 // 4) * b // max(1, n - 1)) if case["ragged"] else t for b in range(n)]


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    return {"append": _prepare_append, "attn": _prepare_attn, "copy": _prepare_copy, "count": _prepare_count,
            "logits": _prepare_logits}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _randint(gen, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sums(n):
    return [sum(n[:b]) for b in range(len(n) + 1)]


def _pages(lengths, gen):
    """A page table over a pool in random order: (table, total pages)."""
    counts = [-(-n // PAGE) for n in lengths]
    order = torch.randperm(sum(counts), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, at


E4M3 = torch.float8_e4m3fn


def _codes(pool, pages, kv):
    """[pages, kv heads, K|V, row / 8, dim / 16, row % 8, dim % 16] view of the bytes of a one-layer pool's codes."""
    return pool.view(pages, kv, 2, UNIT)[..., :PAGE * D].unflatten(3, (PAGE // 8, D // 16, 8, 16))


def _scales(pool, pages, kv):
    """[pages, kv heads, K|V, row / 16] view of its scales."""
    return pool.view(torch.float32).view(pages, kv, 2, UNIT // 4)[..., PAGE * D // 4:]


def _fill(pool, pages, kv, gen):
    """Normal K and V: codes that use their range, scales that differ from block to block."""
    codes, scales = _codes(pool, pages, kv), _scales(pool, pages, kv)
    for p in range(0, pages, 256):
        n = min(256, pages - p)
        codes[p:p + n] = _randn(gen, n, kv, 2, PAGE // 8, D // 16, 8, 16).mul_(64.0).to(E4M3).view(torch.uint8)
    scales.copy_(torch.exp2(_randint(gen, -7, -4, pages, kv, 2, PAGE // BLOCK).float()))


def _prepare_append(case, gen):
    slots, kv, n = case["slots"], case["kv"], _counted(case)
    before = [case["before"] + 5 * b if case["ragged"] else case["before"] for b in range(slots)]
    table, pages = _pages([a + t for a, t in zip(before, n)], gen)
    pool = torch.zeros(pages * kv * 2 * UNIT, dtype=torch.uint8, device="cuda")
    _fill(pool, pages, kv, gen)
    rows, dt = sum(n), _dt(case["dtype"])
    # a few channels of K carry most of its weight
    loud = 1.0 + 7.0 * (torch.rand((kv, D), generator=gen, device="cuda") < 4.0 / D)
    state = dict(case=case, pool=pool, table=table, pages=pages, rows=rows, n=n, before=before, len=_i32(before), n_new=_i32(n),
                 offsets=_i32(_sums(n)), k=(_randn(gen, rows, kv, D) * loud).to(dt), v=_randn(gen, rows, kv, D).to(dt))
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["desc"] = api.make_desc(1, kv, pages)
    return state


def _prepare_attn(case, gen):
    slots, kv, widths, lengths = case["slots"], case["kv"], _widths(case), _lengths(case)
    table, pages = _pages(lengths, gen)
    pool = torch.zeros(pages * kv * 2 * UNIT, dtype=torch.uint8, device="cuda")
    _fill(pool, pages, kv, gen)
    rows, dt = sum(widths), _dt(case["dtype"])
    q = _randn(gen, rows, GROUP * kv, D).to(dt)
    state = dict(case=case, pool=pool, table=table, pages=pages, lengths=lengths, widths=widths, ctx=_i32(lengths), n_q=_i32(widths),
                 offsets=_i32(_sums(widths)), q=q, out=torch.zeros((rows, GROUP * kv, D), dtype=dt, device="cuda"))
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["desc"] = api.make_desc(1, kv, pages)
        state["ws"] = torch.zeros(api.bs8_workspace_bytes(state["desc"], slots, max(lengths), max(widths)), dtype=torch.uint8, device="cuda")
    return state


def _page_bytes(case):
    return case["layers"] * case["kv"] * 2 * (UNIT if case["fmt"] == "bs8" else PAGE * RECORD[case["fmt"]])


def _prepare_copy(case, gen):
    pages = case["pages"]
    total = 2 * pages + 3
    pool = _randint(gen, -(1 << 31), (1 << 31) - 1, total * _page_bytes(case) // 4)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    src, dst = order[:pages].contiguous(), order[pages:2 * pages].contiguous()
    rows = _randint(gen, 1, PAGE + 1, pages) if case["partial"] else None
    state = dict(case=case, pool=pool, src=src, dst=dst, rows=rows, total=total)
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["desc"], state["bytes"] = api.make_desc(case["layers"], case["kv"], total), pool.view(torch.uint8)
    return state


def _tokens(gen, rows, vocab):
    """Token ids of text: a few are frequent, most are rare."""
    u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab)) - 1).to(torch.int32).clamp_(0, vocab - 1)


def _prepare_count(case, gen):
    slots, n, vocab = case["slots"], _counted(case), case["vocab"]
    stride = -(-vocab // 8) * 8
    counts = torch.where(torch.rand((slots, stride), generator=gen, device="cuda") < 0.01, _randint(gen, -3, 9, slots, stride), 0)
    counts = torch.where(counts < 0, counts + 3 - 32768, counts).to(torch.int16)
    counts[:, vocab:] = 0
    return dict(case=case, counts=counts, tokens=_tokens(gen, sum(n), vocab), offsets=_i32(_sums(n)), n_list=n, n=_i32(n), most=max(n))


def _prepare_logits(case, gen):
    slots, widths, vocab, dt = case["slots"], _widths(case), case["vocab"], _dt(case["dtype"])
    rows, stride = sum(widths), -(-vocab // 8) * 8
    state = dict(case=case, rows=rows, widths=widths, logits=(3.0 * _randn(gen, rows, vocab)).to(dt),
                 out=torch.zeros((rows, vocab), dtype=dt, device="cuda"), n_q=_i32(widths), offsets=_i32(_sums(widths)),
                 tokens=_tokens(gen, rows, vocab), counts=None, repetition=None, frequency=None, presence=None, bias_offsets=None,
                 bias_tokens=None, bias_values=None, mask=None)
    if case["penalties"]:
        counts = torch.zeros((slots, stride), dtype=torch.int16, device="cuda")
        history = _tokens(gen, slots * 2000, vocab).view(slots, 2000).long()
        counts.scatter_add_(1, history[:, 1000:], torch.ones_like(history[:, 1000:], dtype=torch.int16))
        prompt = torch.zeros_like(counts).scatter_(1, history[:, :1000], -32768)
        state["counts"] = counts | prompt
        state["repetition"] = 1.0 + 0.3 * torch.rand(slots, generator=gen, device="cuda")
        state["frequency"] = 0.2 * torch.rand(slots, generator=gen, device="cuda")
        state["presence"] = 0.5 * torch.rand(slots, generator=gen, device="cuda")
    if case["biases"]:
        each = [min(case["biases"] - b % 2, vocab) for b in range(slots)]
        picked = [torch.randperm(vocab, generator=gen, device="cuda")[:n].sort().values for n in each]
        state["bias_offsets"], state["bias_tokens"] = _i32(_sums(each)), torch.cat(picked).to(torch.int32)
        state["bias_values"] = 4.0 * _randn(gen, sum(each))
    if case["mask"]:
        # a third of the vocabulary is allowed; one row of a batch may end with nothing allowed
        a = _randint(gen, -(1 << 31), (1 << 31) - 1, rows, -(-vocab // 32))
        b = _randint(gen, -(1 << 31), (1 << 31) - 1, rows, -(-vocab // 32))
        state["mask"] = a & b
        if rows > 20:
            state["mask"][rows // 2] = 0
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    return {"append": _append, "attn": _attn, "copy": _copy, "count": _count, "logits": _logits}[state["case"]["op"]](state)


def _append(st):
    case, kv, pages = st["case"], st["case"]["kv"], st["pages"]
    codes, scales = _codes(st["pool"], pages, kv), _scales(st["pool"], pages, kv)
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.bs8_append(st["desc"], st["pool"], st["table"], st["len"], st["n_new"], st["offsets"], max(st["n"]), 0, st["k"], st["v"])
        return {"codes": codes.view(E4M3), "scales": scales}
    slots, rows, most = case["slots"], st["rows"], max(st["n"])
    x = torch.stack([st["k"], st["v"]], dim=2).float()                                  # [rows, kv, 2, D]
    before = st["len"].long()
    slot = torch.repeat_interleave(torch.arange(slots, device="cuda"), st["n_new"].long(), output_size=rows)
    pos = before[slot] + torch.arange(rows, device="cuda") - st["offsets"].long()[slot]
    most_blocks = (most + 2 * BLOCK - 2) // BLOCK
    block = slot * most_blocks + pos // BLOCK - (before // BLOCK)[slot]                 # among the blocks that the call may touch
    top = torch.zeros((slots * most_blocks, kv, 2), device="cuda")
    top.scatter_reduce_(0, block[:, None, None].expand(rows, kv, 2), x.abs().amax(dim=3), "amax")
    mantissa, exponent = torch.frexp(top)
    need = torch.where(top > 0, exponent - 9 + (mantissa > 0.875), -64).clamp(-64, 64)    # the smallest e with top <= 448 * 2^e
    # a first block that holds earlier positions keeps at least its scale, and those positions go to the new one
    kept = before % BLOCK
    first = torch.arange(slots, device="cuda") * most_blocks
    page, at = st["table"].long()[torch.arange(slots, device="cuda"), before // PAGE], before % PAGE // BLOCK
    old = torch.where((kept > 0)[:, None, None], torch.log2(scales[page, :, :, at].clamp_min(2.0 ** -64)).to(need.dtype), -64)
    need[first] = torch.maximum(need[first], old)
    for half in range(2):
        group = at * 2 + half
        was = codes[page, :, :, group].view(E4M3).float()                                          # [slots, kv, 2, D / 16, 8, 16]
        put = (was * torch.exp2((old - need[first]).float())[..., None, None, None]).to(E4M3)
        mine = (torch.arange(8, device="cuda") + 8 * half) < kept[:, None]
        codes[page, :, :, group] = torch.where(mine[:, None, None, None, :, None], put.view(torch.uint8), codes[page, :, :, group])
    y = (x * torch.exp2(-need[block].float())[..., None]).to(E4M3).view(rows, kv, 2, D // 16, 16)
    page = st["table"].long()[slot, pos // PAGE]
    codes[page, :, :, pos % PAGE // 8, :, pos % 8] = y.view(torch.uint8)
    scales[page, :, :, pos % PAGE // BLOCK] = torch.exp2(need[block].float())
    return {"codes": codes.view(E4M3), "scales": scales}


def _decoded(st, b, g, dtype):
    """K and V [length, D] of slot b and kv head g."""
    kv, n = st["case"]["kv"], st["lengths"][b]
    pages = st["table"][b, :-(-n // PAGE)].long()
    c = _codes(st["pool"], st["pages"], kv)[pages, g].view(E4M3).permute(1, 0, 2, 4, 3, 5).reshape(2, -1, BLOCK, D)
    s = _scales(st["pool"], st["pages"], kv)[pages, g].permute(1, 0, 2).reshape(2, -1, 1, 1)
    return (c.to(dtype) * s.to(dtype)).view(2, -1, D)[:, :n]


def _attn(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.bs8_verify_attn(st["desc"], st["pool"], st["table"], st["ctx"], st["n_q"], st["offsets"], max(st["lengths"]),
                            max(st["widths"]), 0, st["q"], st["out"], st["ws"])
        return st["out"]
    r0 = 0
    for b, (n, t) in enumerate(zip(st["lengths"], st["widths"])):      # ragged slots: each one's scores are one product
        token = torch.arange(t * GROUP, device="cuda") // GROUP
        hidden = torch.arange(n, device="cuda") > (n - t + token)[:, None]
        for g in range(case["kv"]):
            k, v = _decoded(st, b, g, torch.float32)
            q = st["q"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].float().reshape(t * GROUP, D)
            s = ((q @ k.t()) / 16).masked_fill_(hidden, -math.inf)
            p = torch.exp(s - s.amax(dim=1, keepdim=True))
            o = (p @ v) / p.sum(dim=1, keepdim=True)
            st["out"][r0:r0 + t, g * GROUP:(g + 1) * GROUP] = o.view(t, GROUP, D).to(st["out"].dtype)
        r0 += t
    return st["out"]


def _copy(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        call = {"q3": api.copy_pages, "fp8": api.fp8_copy_pages, "bs8": api.bs8_copy_pages}[case["fmt"]]
        call(st["desc"], st["bytes"], st["src"], st["dst"], rows=st["rows"])
        return st["pool"]
    src, dst, units = st["src"].long(), st["dst"].long(), case["layers"] * case["kv"] * 2
    if st["rows"] is None:
        whole = st["pool"].view(st["total"], -1)
        whole[dst] = whole[src]
        return st["pool"]
    first = st["rows"].view(-1, 1, 1, 1)                                   # positions of each page that are copied
    if case["fmt"] != "bs8":
        records = st["pool"].view(st["total"], units, PAGE, -1)
        row = torch.arange(PAGE, device="cuda").view(1, 1, -1, 1)
        records[dst] = torch.where(row < first, records[src], records[dst])
        return st["pool"]
    unit = st["pool"].view(st["total"], units, -1)
    word = torch.arange(UNIT // 4, device="cuda")
    # a word of codes belongs to row (word / 512) * 8 + (word % 32) / 4, a scale to the block that begins at its 16th row
    row = torch.where(word < PAGE * D // 4, word // 512 * 8 + word % 32 // 4, (word - PAGE * D // 4) * BLOCK)
    unit[dst] = torch.where(row < st["rows"].view(-1, 1, 1), unit[src], unit[dst])
    return st["pool"]


def _count(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.count_tokens(st["counts"], case["vocab"], st["tokens"], st["offsets"], st["n"], st["most"], prompt=case["prompt"])
        return st["counts"]
    slots, stride = st["counts"].shape
    slot = torch.repeat_interleave(torch.arange(slots, device="cuda"), st["n"].long(), output_size=st["tokens"].numel())
    at = slot * stride + st["tokens"]
    flat = st["counts"].view(-1)
    if case["prompt"]:
        flat[at] = flat[at] | -32768
        return st["counts"]
    seen = torch.zeros(slots * stride, dtype=torch.int32, device="cuda").scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    flat.copy_((flat & -32768) | ((flat & 32767).int() + seen).clamp_max(32767).to(torch.int16))
    return st["counts"]


def _logits(st):
    case, vocab, rows = st["case"], st["case"]["vocab"], st["rows"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.process_logits(st["logits"], st["out"], st["offsets"], st["n_q"], st["tokens"], max(st["widths"]), counts=st["counts"],
                           repetition=st["repetition"], frequency=st["frequency"], presence=st["presence"],
                           bias_offsets=st["bias_offsets"], bias_tokens=st["bias_tokens"], bias_values=st["bias_values"], mask=st["mask"])
        return st["out"]
    slots = case["slots"]
    slot = torch.repeat_interleave(torch.arange(slots, device="cuda"), st["n_q"].long(), output_size=rows)
    first = st["offsets"].long()[slot]
    x = st["logits"].float()
    if case["penalties"]:
        word = st["counts"][:, :vocab][slot].int()
        count, prompt = word & 32767, word < 0
        # row j of a slot comes after the step's tokens t_0 .. t_j
        i = torch.arange(max(st["widths"]), device="cuda")
        before = i <= (torch.arange(rows, device="cuda") - first)[:, None]
        token = st["tokens"].long()[(first[:, None] + i).clamp_max(rows - 1)]
        count.scatter_add_(1, token, before.int())
        theta = st["repetition"][slot][:, None]
        x = torch.where(prompt | (count > 0), torch.where(x > 0, x / theta, x * theta), x)
        x = x - st["frequency"][slot][:, None] * count - st["presence"][slot][:, None] * (count > 0)
    if case["biases"]:
        n = st["bias_offsets"].long()
        owner = torch.repeat_interleave(torch.arange(slots, device="cuda"), n[1:] - n[:-1], output_size=st["bias_tokens"].numel())
        bias = torch.zeros((slots, vocab), device="cuda")
        bias[owner, st["bias_tokens"].long()] = st["bias_values"]
        x = x + bias[slot]
    if case["mask"]:
        token = torch.arange(vocab, device="cuda")
        x = torch.where((st["mask"][:, token // 32] >> (token % 32)) & 1 == 1, x, -math.inf)
    st["out"].copy_(x.to(st["out"].dtype))
    return st["out"]


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "append":
        rows, size = sum(_counted(case)), 2 if case["dtype"] == "bf16" else 4
        elems = rows * case["kv"] * 2 * D
        return {"bytes": elems * (size + 1) + elems // (BLOCK * D) * 4, "flops": 3 * elems}
    if op == "attn":
        size, kv = 2 if case["dtype"] == "bf16" else 4, case["kv"]
        lengths, widths = _lengths(case), _widths(case)
        b = sum(n * kv * (2 * D + 8 / BLOCK) for n in lengths) + sum(widths) * GROUP * kv * D * 2 * size
        return {"bytes": b, "flops": sum(4 * kv * GROUP * w * D * n for n, w in zip(lengths, widths))}
    if op == "copy":
        share = 0.5 if case["partial"] else 1.0
        return {"bytes": 2 * share * case["pages"] * _page_bytes(case), "flops": 0}
    if op == "count":
        return {"bytes": 8 * sum(_counted(case)), "flops": sum(_counted(case))}
    rows, vocab, size = sum(_widths(case)), case["vocab"], 2 if case["dtype"] == "bf16" else 4
    b = rows * vocab * (2 * size + (0.125 if case["mask"] else 0)) + (2 * case["slots"] * vocab if case["penalties"] else 0)
    return {"bytes": b + 8 * case["slots"] * case["biases"], "flops": 6 * rows * vocab}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    return {"append": _exact_append, "attn": _exact_attn, "copy": lambda *_: None, "count": lambda *_: None,
            "logits": _exact_logits}[case["op"]](case, prepare(case, seed))


def _exact_append(case, st):
    """Scales by counting powers of two; codes as the values that they round, block by block of each slot."""
    if max(st["n"]) * case["slots"] > 16384:
        return None                                     # block by block takes too long
    kv, pages = case["kv"], st["pages"]
    codes, scales = _codes(st["pool"], pages, kv).view(E4M3).double(), _scales(st["pool"], pages, kv).double()
    powers = 448.0 * torch.exp2(torch.arange(-64, 65, dtype=torch.float64, device="cuda"))
    x = torch.stack([st["k"], st["v"]], dim=2).double()
    table, r0 = st["table"].tolist(), 0
    for b, (a, n) in enumerate(zip(st["before"], st["n"])):
        for lo in range(a - a % BLOCK, a + n, BLOCK):
            new = range(max(lo, a), min(lo + BLOCK, a + n))
            y = x[r0 + new[0] - a:r0 + new[-1] - a + 1]                                   # [rows, kv, 2, D]
            s = torch.exp2((y.abs().amax(dim=(0, 3))[..., None] > powers).sum(dim=-1).double() - 64.0)
            page, k = table[b][lo // PAGE], lo % PAGE // BLOCK
            if lo < a:
                was = scales[page, :, :, k]
                s = torch.maximum(s, was)
                for p in range(lo, a):
                    codes[page, :, :, p % PAGE // 8, :, p % 8] *= (was / s)[..., None, None]
            for p in new:
                codes[page, :, :, p % PAGE // 8, :, p % 8] = (y[p - new[0]] / s[..., None]).unflatten(2, (D // 16, 16))
            scales[page, :, :, k] = s
        r0 += n
    return {"codes": codes, "scales": scales}


def _exact_attn(case, st):
    """Weights relative to the row's log-sum, positions in pieces."""
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b, (n, t) in enumerate(zip(st["lengths"], st["widths"])):
        r0 = int(st["offsets"][b])
        for g in range(case["kv"]):
            pages = st["table"][b, :-(-n // PAGE)].long()
            c, f = _codes(st["pool"], st["pages"], case["kv"])[pages, g], _scales(st["pool"], st["pages"], case["kv"])[pages, g]
            q = st["q"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].double()

            def rows(kind, lo, hi):
                p = torch.arange(lo, hi, device="cuda")
                return c[p // PAGE, kind, p % PAGE // 8, :, p % 8].view(E4M3).double().flatten(1) * f[p // PAGE, kind, p % PAGE // BLOCK].double()[:, None]

            def scores(lo, hi):
                s = torch.einsum("thd,pd->thp", q, rows(0, lo, hi)) * 0.0625
                p = torch.arange(lo, hi, device="cuda")
                return s.masked_fill(p > (n - t + torch.arange(t, device="cuda"))[:, None, None], -math.inf)

            cuts = [(lo, min(n, lo + 32768)) for lo in range(0, n, 32768)]
            total = torch.logsumexp(torch.stack([torch.logsumexp(scores(lo, hi), dim=2) for lo, hi in cuts]), dim=0)
            for lo, hi in cuts:
                w = torch.exp(scores(lo, hi) - total[..., None])
                out[r0:r0 + t, g * GROUP:(g + 1) * GROUP] += torch.einsum("thp,pd->thd", w, rows(1, lo, hi))
    return out


def _exact_logits(case, st):
    """One row at a time, its tokens counted one by one."""
    vocab = case["vocab"]
    out = st["logits"].double()
    for b, w in enumerate(st["widths"]):
        r0 = int(st["offsets"][b])
        if case["penalties"]:
            word = st["counts"][b, :vocab].long()
            count, prompt = word % 32768, word < 0
            theta, alpha, beta = (float(st[name][b]) for name in ("repetition", "frequency", "presence"))
        for j in range(w):
            x = out[r0 + j]
            if case["penalties"]:
                count[int(st["tokens"][r0 + j])] += 1
                used = count >= 1
                x = torch.where(used | prompt, torch.where(x >= 0, x / theta, x * theta), x) - alpha * count - beta * used
            if case["biases"]:
                lo, hi = int(st["bias_offsets"][b]), int(st["bias_offsets"][b + 1])
                x = x.index_add(0, st["bias_tokens"][lo:hi].long(), st["bias_values"][lo:hi].double())
            if case["mask"]:
                bits = torch.stack([(st["mask"][r0 + j].long() >> i) & 1 for i in range(32)], dim=1).flatten()[:vocab]
                x = torch.where(bits > 0, x, -math.inf)
            out[r0 + j] = x
    return out
