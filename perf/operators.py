"""Cases of the serving step's operators around the quantised cache, with their plain forms.

Four operators, each in its plain form (elementary torch operations) and as the library's call:

  rope     rotary positions with several axes for q and k rows, before the append and the verify
  accept   acceptance of drafted tokens that were sampled from given draft probabilities
  mass     attention weight each cached position received, accumulated over steps
  evict    selection of the positions to keep by that weight, and compaction of their records

Sizes follow the repository's own workloads: 2 kv heads and 16 q heads of 256 dims, 256-position pages, contexts up to
655,360 positions, up to 16 query tokens per slot, a vocabulary of 248,320.
"""
import math

import torch

own = False

D = 256          # head dim
PAGE = 256       # positions per page
GROUP = 8        # q heads per kv head
RECORD = {"q3": 112, "fp8": 256}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the query and key rows of one slot's verify step (text: all axes at one position), deep in a long context
        dict(name="rope step of 6 tokens", op="rope", rows=6, kv=2, q=16, rotary=64, axes=3, sections="11,11,10", deal=True,
             adjacent=False, per_axis=False, theta=1e7, dtype="bf16", strided=False, far=655360),
        # a prompt of mixed text and image tokens: q and k are slices of one projection's output
        dict(name="rope prompt of 4096 tokens", op="rope", rows=4096, kv=2, q=16, rotary=64, axes=3, sections="11,11,10", deal=True,
             adjacent=False, per_axis=False, theta=1e7, dtype="bf16", strided=True, far=8192),
        # float32 rows of an image or video stack, whole head rotated, each axis with its own frequencies, odd row count
        dict(name="rope video of 8191 patches f32", op="rope", rows=8191, kv=2, q=16, rotary=256, axes=3, sections="32,48,48",
             deal=False, adjacent=True, per_axis=True, theta=1e4, dtype="f32", strided=False, far=1024),
        # one slot, five sampled drafts
        dict(name="accept 1 slot x 6", op="accept", slots=1, tokens=6, ragged=False, vocab=248320, dtype="bf16", draft="f32",
             temperature=1.0, masked=False),
        # continuous batching: eight slots of different widths, draft probabilities kept in 16 bits
        dict(name="accept 8 slots ragged", op="accept", slots=8, tokens=8, ragged=True, vocab=248320, dtype="bf16", draft="bf16",
             temperature=0.7, masked=False),
        # float32 logits of an odd vocabulary, most of it masked with -inf (a grammar or a filter ran first)
        dict(name="accept 8 slots masked f32", op="accept", slots=8, tokens=8, ragged=True, vocab=100003, dtype="f32", draft="f32",
             temperature=0.8, masked=True),
        # one token per slot over a batch of short ragged contexts
        dict(name="mass 8 slots x 1 token", op="mass", fmt="q3", slots=8, ctx=16384, ragged=True, tokens=1, kv=2, dtype="bf16", decay=1.0),
        # one slot's verify step at 32K, without a history: the last tokens of a prompt are the observation window
        dict(name="mass 32768 x 6", op="mass", fmt="q3", slots=1, ctx=32768, ragged=False, tokens=6, kv=2, dtype="bf16", decay=0.0),
        # the longest context
        dict(name="mass 655360 x 8", op="mass", fmt="q3", slots=1, ctx=655360, ragged=False, tokens=8, kv=2, dtype="bf16", decay=0.9),
        # one layer of one slot is brought back to a small budget
        dict(name="evict 5000 to 1024", op="evict", fmt="q3", layers=1, slots=1, ctx=5000, ragged=False, budget=1024, sink=4, recent=128, kv=2),
        # all layers of a 32K slot to a quarter
        dict(name="evict 16 layers 32768 to 8192", op="evict", fmt="q3", layers=16, slots=1, ctx=32768, ragged=False, budget=8192,
             sink=16, recent=512, kv=2),
        # all layers of the longest context to a tenth
        dict(name="evict 16 layers 655360 to 65536", op="evict", fmt="q3", layers=16, slots=1, ctx=655360, ragged=False, budget=65536,
             sink=64, recent=4096, kv=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "accept", "mass", "evict"])
    if op == "rope":
        axes = rng.choice([1, 2, 3, 3, 4])
        rotary = rng.choice([32, 64, 96, 128, 192, 256])
        cuts = sorted(rng.sample(range(1, rotary // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rotary // 2])]
        kv = rng.choice([1, 2, 4])
        q = kv * rng.choice([1, 4, 8])
        most = 8191 * 18 // (kv + q)
        return dict(op=op, rows=_log(rng, 1, most), kv=kv, q=q, rotary=rotary, axes=axes, sections=",".join(map(str, sections)),
                    deal=rng.random() < 0.5, adjacent=rng.random() < 0.5, per_axis=rng.random() < 0.5, theta=rng.choice([1e4, 1e6, 1e7]),
                    dtype=rng.choice(["bf16", "f32"]), strided=rng.random() < 0.5, far=_log(rng, 64, 1 << 20))
    if op == "accept":
        vocab = _log(rng, 1000, 248320)
        slots = _log(rng, 1, 8)
        return dict(op=op, slots=slots, tokens=rng.randint(1, 8), ragged=rng.random() < 0.7, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                    draft=rng.choice(["bf16", "f32"]), temperature=round(rng.uniform(0.5, 1.5), 3),
                    masked=rng.random() < 0.3)
    if op == "mass":
        kv, tokens, slots = rng.choice([1, 2, 4]), rng.randint(1, 16), _log(rng, 1, 8)
        fmt = rng.choice(["q3", "q3", "fp8"])
        most = 655360 * 2 * 8 // (kv * max(tokens, 8) * slots)
        return dict(op=op, fmt=fmt, slots=slots, ctx=_log(rng, 300, min(most // (2 if fmt == "fp8" else 1), 655360)), ragged=rng.random() < 0.7,
                    tokens=tokens, kv=kv, dtype=rng.choice(["bf16", "f32"]), decay=rng.choice([0.0, 0.9, 1.0]))
    kv, layers, slots = rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 16]), _log(rng, 1, 8)
    fmt = rng.choice(["q3", "q3", "fp8"])
    most = 655360 * 2 * 16 // (kv * layers * slots * (3 if fmt == "fp8" else 1))
    ctx = _log(rng, 600, min(655360, most))
    budget = max(200, int(ctx * rng.uniform(0.02, 0.1)))
    return dict(op=op, fmt=fmt, layers=layers, slots=slots, ctx=ctx, ragged=rng.random() < 0.7, budget=budget, sink=rng.choice([0, 4, 16]),
                recent=rng.choice([32, 100, 128]), kv=kv)


def _lengths(case, least):
    """Per-slot lengths: the first slot has the longest, the others spread down to a quarter of it."""
    n, c = case["slots"], case["ctx"]
    return [max(least, c - (c * 3 // 4) * b // max(1, n - 1) - b) if case["ragged"] and b else c for b in range(n)]


def _widths(case):
    """Query tokens per slot: ragged slots cycle from the widest down to one."""
    t = case["tokens"]
    return [1 + (t - 1 - 3 * b) % t if case["ragged"] else t for b in range(case["slots"])]


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    return {"rope": _prepare_rope, "accept": _prepare_accept, "mass": _prepare_mass, "evict": _prepare_evict}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(case):
    """(angle per position, axis) of each of the rotary/2 pairs, in double precision on the host."""
    half, sections = case["rotary"] // 2, [int(s) for s in case["sections"].split(",")]
    if case["deal"]:                       # the pairs are dealt to the axes in turn; an axis with its share is passed over
        left, axis = list(sections), []
        a = 0
        while len(axis) < half:
            if left[a % len(left)]:
                left[a % len(left)] -= 1
                axis.append(a % len(left))
            a += 1
    else:
        axis = [a for a, s in enumerate(sections) for _ in range(s)]
    seen, freq = [0] * len(sections), []
    for i, a in enumerate(axis):
        freq.append(case["theta"] ** (-(seen[a] / sections[a])) if case["per_axis"] else case["theta"] ** (-i / half))
        seen[a] += 1
    return freq, axis


def _prepare_rope(case, gen):
    rows, kv, q, dt = case["rows"], case["kv"], case["q"], _dt(case["dtype"])
    if case["strided"]:                    # q | k | v of one projection
        qkv = _randn(gen, rows, (q + 2 * kv) * D).to(dt)
        qi, ki = qkv[:, :q * D].unflatten(1, (q, D)), qkv[:, q * D:(q + kv) * D].unflatten(1, (kv, D))
    else:
        qi, ki = _randn(gen, rows, q, D).to(dt), _randn(gen, rows, kv, D).to(dt)
    first = case["far"] - rows if case["far"] > rows else 0
    pos = torch.randint(0, case["far"], (rows, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
    text = torch.rand(rows, generator=gen, device="cuda") < 0.5      # text tokens: every axis at the token's own position
    own_pos = first + torch.arange(rows, device="cuda", dtype=torch.int32)
    pos = torch.where(text[:, None], own_pos[:, None], pos).contiguous()
    state = dict(case=case, q=qi, k=ki, pos=pos, q_out=torch.zeros((rows, q, D), dtype=dt, device="cuda"),
                 k_out=torch.zeros((rows, kv, D), dtype=dt, device="cuda"))
    freq, axis = _frequencies(case)
    state["freq"], state["axis"] = torch.tensor(freq, dtype=torch.float64, device="cuda"), torch.tensor(axis, device="cuda")
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["plan"] = api.make_rope_plan(case["rotary"], case["theta"], [int(s) for s in case["sections"].split(",")],
                                           deal_axes=case["deal"], axis_freqs=case["per_axis"], adjacent=case["adjacent"])
    return state


def _prepare_accept(case, gen):
    slots, vocab, tau = case["slots"], case["vocab"], case["temperature"]
    widths = _widths(case)
    rows = sum(widths)
    offsets = [sum(widths[:b]) for b in range(slots + 1)]
    # a few likely tokens over a broad tail; the drafter sees the same scores with its own noise
    base = 2.0 * _randn(gen, rows, vocab) + 7.0 * (torch.rand((rows, vocab), generator=gen, device="cuda") < 20.0 / vocab)
    logits = base.to(_dt(case["dtype"]))
    if case["masked"]:                     # the drafter knows nothing of the mask
        logits.masked_fill_((torch.rand((rows, vocab), generator=gen, device="cuda") < 0.8) & (base < 6.0), -math.inf)
    noisy = (base + 0.7 * _randn(gen, rows, vocab)) / tau
    draft = torch.softmax(noisy, dim=1).to(_dt(case["draft"]))
    race = -torch.log(torch.rand((rows, vocab), generator=gen, device="cuda").clamp_min(1e-30))
    drawn = torch.argmax(draft.float() / race, dim=1).to(torch.int32)
    tokens = torch.cat([drawn.new_zeros(1), drawn[:-1]]).contiguous()      # row r + 1's token was drawn from row r
    lengths = [5000 + 17 * b for b in range(slots)]
    state = dict(case=case, logits=logits, draft=draft, tokens=tokens, offsets=_i32(offsets), n_q=_i32(widths), ctx=_i32(lengths),
                 uniforms=torch.rand(rows, generator=gen, device="cuda"),
                 seed=int(torch.randint(0, 1 << 62, (1,), generator=gen, device="cuda").item()), rows=rows, widest=max(widths),
                 accepted=torch.zeros(slots, dtype=torch.int32, device="cuda"), next=torch.zeros(slots, dtype=torch.int32, device="cuda"),
                 committed=torch.zeros(slots, dtype=torch.int32, device="cuda"), prob=torch.full((rows,), -1.0, device="cuda"))
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["ws"] = torch.zeros(api.accept_draft_workspace_bytes(slots, rows, vocab), dtype=torch.uint8, device="cuda")
    return state


def _pages(lengths, gen, extra=0):
    """A page table over a pool in random order: (table, total pages, page ids of each slot)."""
    counts = [-(-n // PAGE) for n in lengths]
    order = torch.randperm(sum(counts) + extra, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(counts)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, order, at


def _encode_q3(y):
    """Records [n, 112] of already rotated vectors y [n, 256]."""
    n = y.shape[0]
    y = y.view(n, 8, 32)
    s = (y.abs().amax(dim=2) / 3.5).to(torch.float16)
    c = (y / s.float()[..., None] + 3.5).round().clamp_(0, 7).to(torch.int32)
    pairs = c[..., :30].view(n, 8, 3, 5, 2)
    shift = torch.arange(0, 15, 3, device=y.device, dtype=torch.int32)
    word = ((pairs[..., 0] << shift) | (pairs[..., 1] << (shift + 16))).sum(dim=3, dtype=torch.int32)
    bit = torch.arange(3, device=y.device, dtype=torch.int32)
    word |= ((c[..., 30:31] >> bit) & 1) << 15
    word |= ((c[..., 31:32] >> bit) & 1) << 31
    return torch.cat([word.view(n, 24).view(torch.uint8), s.view(torch.uint8).view(n, 16)], dim=1)


def _prepare_mass(case, gen):
    slots, kv, fmt = case["slots"], case["kv"], case["fmt"]
    widths = _widths(case)
    lengths = [max(n, w) for n, w in zip(_lengths(case, 300), widths)]
    rec = RECORD[fmt]
    table, order, pages = _pages(lengths, gen)
    pool = torch.randint(0, 1 << 30, (pages * kv * 2 * PAGE * rec // 4,), generator=gen, device="cuda", dtype=torch.int32)
    view = pool.view(torch.uint8).view(pages, 1, kv, 2, PAGE, rec)
    for g in range(kv):
        for p in range(0, pages, 512):
            n = min(512, pages - p)
            y = 1.4 * _randn(gen, n * PAGE, D)
            view[p:p + n, 0, g, 0] = (_encode_q3(y) if fmt == "q3" else y.to(torch.float8_e4m3fn).view(torch.uint8)).view(n, PAGE, rec)
    rows = sum(widths)
    q = (2.0 * _randn(gen, rows, GROUP * kv, D)).to(_dt(case["dtype"]))
    stride = max(lengths) + 100
    # weight from a few dozen earlier steps
    mass = torch.rand((slots, kv, stride), generator=gen, device="cuda") * (40.0 * GROUP * case["tokens"] / case["ctx"])
    state = dict(case=case, pool=pool.view(torch.uint8), view=view, table=table, lengths=lengths, widths=widths, q=q, mass=mass,
                 ctx=_i32(lengths), n_q=_i32(widths), offsets=_i32([sum(widths[:b]) for b in range(slots + 1)]), pages=pages)
    lse = torch.zeros((rows, GROUP * kv), device="cuda")
    r0 = 0
    for b in range(slots):
        for g in range(kv):
            s = _scores(state, b, g)
            lse[r0:r0 + widths[b], g * GROUP:(g + 1) * GROUP] = torch.logsumexp(s, dim=1).view(widths[b], GROUP)
        r0 += widths[b]
    state["lse"] = lse
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["desc"] = api.make_desc(1, kv, pages)
    return state


def _prepare_evict(case, gen):
    slots, kv, layers, rec = case["slots"], case["kv"], case["layers"], RECORD[case["fmt"]]
    lengths = _lengths(case, 300)
    budgets = [max(case["sink"] + case["recent"], case["budget"] - 3 * b) for b in range(slots)] if case["ragged"] else [case["budget"]] * slots
    keep = [min(n, k) for n, k in zip(lengths, budgets)]
    room = [-(-k // PAGE) for k in keep]
    table, order, used = _pages(lengths, gen, extra=sum(room))
    dst = torch.full((slots, max(room)), -1, dtype=torch.int32, device="cuda")
    for b in range(slots):
        dst[b, :room[b]] = order[used:used + room[b]]
        used += room[b]
    pool = torch.randint(-(1 << 31), (1 << 31) - 1, (used * layers * kv * 2 * PAGE * rec // 4,), generator=gen, device="cuda", dtype=torch.int32)
    # accumulated weight has a heavy tail; half of the positions share few values, as after short histories
    stride = max(lengths) + 12
    u = torch.rand((layers, slots, kv, stride), generator=gen, device="cuda")
    mass = torch.where(u < 0.5, (u * 8).floor() / 1024, 1e-3 / (1.0001 - u))
    most = max(budgets)
    state = dict(case=case, pool=pool, table=table, dst=dst, lengths=lengths, budgets=budgets, keep=keep, mass=mass, ctx=_i32(lengths),
                 budget=_i32(budgets), most=most, pages=used,
                 kept=torch.full((layers, slots, kv, most), -1, dtype=torch.int32, device="cuda"),
                 mass_out=torch.zeros((layers, slots, kv, most), device="cuda"), new_len=torch.zeros(slots, dtype=torch.int32, device="cuda"))
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        state["desc"], state["bytes"] = api.make_desc(layers, kv, used), pool.view(torch.uint8)
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    return {"rope": _rope, "accept": _accept, "mass": _mass, "evict": _evict}[state["case"]["op"]](state)


def _rope(st):
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.rope(st["plan"], st["pos"], st["q"], st["q_out"], st["k"], st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    # angles in 64 bits: a far position times a frequency of one radian loses whole digits in 32
    angle = st["pos"].double()[:, st["axis"]] * st["freq"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    return {"q": _turn(st["case"], st["q"], cos, sin), "k": _turn(st["case"], st["k"], cos, sin)}


def _turn(case, x, cos, sin):
    r = case["rotary"]
    y = x.float()
    if case["adjacent"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        head = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        head = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([head, y[..., r:]], dim=-1).to(x.dtype)


def _noise(seed, rows, vocab):
    """E = -log U of the counter-based SplitMix64 stream, [len(rows), vocab] in double precision."""
    def mul(v):
        return v - (1 << 64) if v >= 1 << 63 else v

    k = (rows.long()[:, None] << 32) + torch.arange(vocab, device=rows.device)
    z = (k + 1) * mul(0x9E3779B97F4A7C15) + mul(seed & ((1 << 64) - 1))
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * mul(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * mul(0x94D049BB133111EB)
    z = z ^ ((z >> 31) & ((1 << 33) - 1))
    return -torch.log((((z >> 41) & ((1 << 23) - 1)).double() + 0.5) / (1 << 23))


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _target(logits, tau):
    """Target probabilities in 64 bits: a uniform or a key next to a border decides a token."""
    x = logits.double()
    e = torch.exp((x - x.amax(dim=1, keepdim=True)) / _f32(tau))
    return e / e.sum(dim=1, keepdim=True)


def _accept(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        api.accept_draft(st["logits"], st["draft"], st["offsets"], st["n_q"], st["tokens"], st["widest"], st["ctx"], case["temperature"],
                         st["uniforms"], st["seed"], st["accepted"], st["next"], st["committed"], st["ws"],
                         accept_prob=st["prob"])
        return {"accepted": st["accepted"], "next": st["next"], "committed": st["committed"], "prob": st["prob"]}
    p = _target(st["logits"], case["temperature"])
    slots, widest = case["slots"], st["widest"]
    n_q, first = st["n_q"].long(), st["offsets"][:-1].long()
    j = torch.arange(widest, device=p.device)
    row = (first[:, None] + j).clamp_max(st["rows"] - 1)                       # [slots, widest]
    drafted = j < (n_q - 1)[:, None]                                           # rows whose successor is a draft
    token = st["tokens"].long()[(row + 1).clamp_max(st["rows"] - 1)]
    pd, qd = p[row, token], st["draft"][row, token].double()
    passed = (st["uniforms"].double()[row] * qd < pd) & drafted
    a = torch.cumprod(passed.long(), dim=1).sum(dim=1)                         # accepted drafts per slot
    prob = torch.where(qd > 0, (pd / qd).clamp_max(1.0), (pd > 0).double())
    out = st["prob"].clone()
    out[row[drafted]] = prob[drafted].float()
    at = first + a
    pa = p[at]
    rest = torch.where((a < n_q - 1)[:, None], (pa - st["draft"][at].double()).clamp_min(0.0), pa)
    rest = torch.where(rest.amax(dim=1, keepdim=True) > 0, rest, pa)
    key = rest / _noise(st["seed"], at, case["vocab"])
    index = torch.arange(case["vocab"], device=p.device)
    best = torch.where(key == key.amax(dim=1, keepdim=True), index, case["vocab"]).amin(dim=1)
    return {"accepted": a.to(torch.int32), "next": best.to(torch.int32), "committed": (st["ctx"].long() - (n_q - 1 - a)).to(torch.int32),
            "prob": out}


def _decode(records, fmt):
    """float32 values [n, 256] of records [n, bytes]."""
    n = records.shape[0]
    if fmt == "fp8":
        return records.view(torch.float8_e4m3fn).float()
    w = records[:, :96].contiguous().view(torch.int32).view(n, 8, 3)
    s = records[:, 96:].contiguous().view(torch.float16).float()
    shift = torch.arange(0, 15, 3, device=w.device, dtype=torch.int32)
    c = torch.stack([(w[..., None] >> shift) & 7, (w[..., None] >> (shift + 16)) & 7], dim=-1).view(n, 8, 30)
    bit = torch.tensor([1, 2, 4], device=w.device, dtype=torch.int32)
    last = torch.stack([(((w >> 15) & 1) * bit).sum(dim=2), (((w >> 31) & 1) * bit).sum(dim=2)], dim=-1)
    return ((torch.cat([c, last.to(torch.int32)], dim=-1).float() - 3.5) * s[..., None]).view(n, D)


def _hadamard(dtype):
    i = torch.arange(D, device="cuda")
    x = i[:, None] & i[None, :]
    for s in (4, 2, 1):
        x = x ^ (x >> s)
    return (1 - 2 * (x & 1)).to(dtype) / 16


def _scores(st, b, g):
    """Masked float32 scores [8 T, L] of slot b and kv head g."""
    case, n, t = st["case"], st["lengths"][b], st["widths"][b]
    r0 = sum(st["widths"][:b])
    pages = st["table"][b, :-(-n // PAGE)].long()
    k = _decode(st["view"][pages, 0, g, 0].reshape(-1, RECORD[case["fmt"]])[:n], case["fmt"])
    q = st["q"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].float().reshape(t * GROUP, D)
    if case["fmt"] == "q3":
        q = q @ _hadamard(torch.float32)
    s = (q @ k.t()) / 16
    token = torch.arange(t * GROUP, device=s.device) // GROUP
    return s.masked_fill(torch.arange(n, device=s.device) > (n - t + token)[:, None], -math.inf)


def _mass(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        call = api.attn_mass if case["fmt"] == "q3" else api.fp8_attn_mass
        call(st["desc"], st["pool"], st["table"], st["ctx"], st["n_q"], st["offsets"], max(st["lengths"]), max(st["widths"]), 0, st["q"],
             st["lse"], case["decay"], st["mass"])
        return st["mass"]
    r0 = 0
    for b in range(case["slots"]):       # ragged slots: each one's scores are one product
        n, t = st["lengths"][b], st["widths"][b]
        for g in range(case["kv"]):
            lse = st["lse"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].reshape(-1, 1)
            got = torch.exp(_scores(st, b, g) - lse).sum(dim=0)
            if case["decay"] > 0:
                got[:n - t] += _f32(case["decay"]) * st["mass"][b, g, :n - t]
            st["mass"][b, g, :n] = got
        r0 += t
    return st["mass"]


def _evict(st):
    case = st["case"]
    if own:
        from speculative_verify_attention_q3kv_gb300 import api
        call = api.evict if case["fmt"] == "q3" else api.fp8_evict
        call(st["desc"], st["bytes"], st["table"], st["ctx"], max(st["lengths"]), st["budget"], st["most"], case["sink"], case["recent"], 0,
             st["mass"], st["dst"], st["kept"], st["mass_out"], st["new_len"])
        return {"kept": st["kept"], "mass": st["mass_out"], "len": st["new_len"], "pool": st["pool"]}
    layers, slots, kv, rec = case["layers"], case["slots"], case["kv"], RECORD[case["fmt"]] // 4
    n, keep = st["ctx"].long().view(1, slots, 1, 1), torch.minimum(st["ctx"], st["budget"]).long().view(1, slots, 1, 1)
    at = torch.arange(st["mass"].shape[3], device="cuda")
    # protected positions first, then by weight; a stable sort leaves ties to the lowest index
    key = torch.where((at < case["sink"]) | (at >= n - case["recent"]), math.inf, st["mass"])
    key = torch.where(at < n, key, -math.inf)
    order = torch.sort(key, dim=3, descending=True, stable=True).indices
    chosen = torch.zeros_like(key, dtype=torch.bool).scatter_(3, order, at.expand_as(order) < keep)
    la, sl, he, position = torch.nonzero(chosen, as_tuple=True)                # ascending positions of each row
    rank = (torch.cumsum(chosen, dim=3) - 1)[la, sl, he, position]
    st["kept"][la, sl, he, rank] = position.to(torch.int32)
    st["mass_out"][la, sl, he, rank] = st["mass"][la, sl, he, position]
    records = st["pool"].view(-1, PAGE, rec)                                   # one row per (page, layer, head, K or V)
    src = ((st["table"][sl, position // PAGE].long() * layers + la) * kv + he) * 2
    dst = ((st["dst"][sl, rank // PAGE].long() * layers + la) * kv + he) * 2
    records[dst, rank % PAGE] = records[src, position % PAGE]
    records[dst + 1, rank % PAGE] = records[src + 1, position % PAGE]
    st["new_len"].copy_(torch.minimum(st["ctx"], st["budget"]))
    return {"kept": st["kept"], "mass": st["mass_out"], "len": st["new_len"], "pool": st["pool"]}


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        size, heads = (2 if case["dtype"] == "bf16" else 4), case["q"] + case["kv"]
        return {"bytes": case["rows"] * (2 * heads * D * size + 4 * case["axes"]), "flops": case["rows"] * heads * case["rotary"] * 3}
    if op == "accept":
        rows = sum(_widths(case))
        size, ds = (2 if case["dtype"] == "bf16" else 4), (2 if case["draft"] == "bf16" else 4)
        return {"bytes": case["vocab"] * (rows * size + case["slots"] * ds), "flops": 4 * case["vocab"] * rows}
    if op == "mass":
        widths = _widths(case)
        lengths = [max(n, w) for n, w in zip(_lengths(case, 300), widths)]
        size = 2 if case["dtype"] == "bf16" else 4
        kv = case["kv"]
        b = sum(kv * n * (RECORD[case["fmt"]] + (8 if case["decay"] > 0 else 4)) for n in lengths) + sum(widths) * GROUP * kv * (D * size + 4)
        return {"bytes": b, "flops": sum(2 * kv * GROUP * w * D * n for n, w in zip(lengths, widths))}
    lengths = _lengths(case, 300)
    budgets = [max(case["sink"] + case["recent"], case["budget"] - 3 * b) for b in range(case["slots"])] if case["ragged"] else \
        [case["budget"]] * case["slots"]
    rows = case["layers"] * case["kv"]
    moved = sum(min(n, k) for n, k in zip(lengths, budgets))
    return {"bytes": rows * (4 * sum(lengths) + moved * (4 * RECORD[case["fmt"]] + 8)), "flops": rows * sum(lengths)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "accept": _exact_accept, "mass": _exact_mass, "evict": _exact_evict}[case["op"]](case, st)


def _exact_rope(case, st):
    """Each pair as a complex number times exp(i angle)."""
    angle = torch.stack([st["pos"][:, a].double() for a in st["axis"].tolist()], dim=1) * st["freq"]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    r = case["rotary"]
    pairs = torch.arange(r, device="cuda").view(-1, 2) if case["adjacent"] else torch.arange(r, device="cuda").view(2, -1).t()
    out = {}
    for name in ("q", "k"):
        x = st[name].double().clone()
        z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * turn
        x[..., pairs[:, 0]], x[..., pairs[:, 1]] = z.real, z.imag
        out[name] = x
    return out


def _exact_accept(case, st):
    """Only the probabilities are computed numbers: one slot and one row at a time."""
    prob = torch.full((st["rows"],), -1.0, dtype=torch.float64, device="cuda")
    tau = _f32(case["temperature"])
    for b, w in enumerate(st["n_q"].tolist()):
        for r in range(int(st["offsets"][b]), int(st["offsets"][b]) + w - 1):
            x = st["logits"][r].double() / tau
            p = torch.exp(x - torch.logsumexp(x, dim=0))
            d = int(st["tokens"][r + 1])
            pd, qd = float(p[d]), float(st["draft"][r, d].double())
            prob[r] = min(1.0, pd / qd) if qd > 0 else float(pd > 0)
    return {"accepted": None, "next": None, "committed": None, "prob": prob}


def _exact_mass(case, st):
    mass = st["mass"].double().clone()
    h = _hadamard(torch.float64)
    for b, (n, t) in enumerate(zip(st["lengths"], st["widths"])):
        r0 = int(st["offsets"][b])
        for g in range(case["kv"]):
            q = st["q"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].double().reshape(-1, D)
            q = q @ h if case["fmt"] == "q3" else q
            lse = st["lse"][r0:r0 + t, g * GROUP:(g + 1) * GROUP].double().reshape(-1, 1)
            for p in range(0, n, 65536):
                e = min(n, p + 65536)
                pos = torch.arange(p, e, device="cuda")
                rec = st["view"][st["table"][b].long()[pos // PAGE], 0, g, 0, pos % PAGE]
                s = torch.einsum("rd,pd->rp", q, _decode(rec, case["fmt"]).double()) / 16
                seen = torch.stack([pos <= n - t + r // GROUP for r in range(t * GROUP)])
                w = (torch.exp(s - lse) * seen).sum(dim=0)
                old = torch.where(pos < n - t, mass[b, g, p:e], 0.0)
                mass[b, g, p:e] = w + (_f32(case["decay"]) * old if case["decay"] > 0 else 0.0)
    return mass


def _exact_evict(case, st):
    """The compacted weights, one row at a time; the rest are whole numbers."""
    out = torch.zeros_like(st["mass_out"], dtype=torch.float64)
    for la in range(case["layers"]):
        for b, (n, k) in enumerate(zip(st["lengths"], st["keep"])):
            for g in range(case["kv"]):
                m = st["mass"][la, b, g, :n].double()
                lo, hi = min(case["sink"], n), max(0, n - case["recent"])
                free = m[lo:hi]
                want = k - (n - len(free))
                cut = torch.topk(free, want).values[-1] if want > 0 else math.inf
                above, level = free > cut, free == cut
                level &= torch.cumsum(level, 0) <= want - int(above.sum())
                take = torch.ones(n, dtype=torch.bool, device="cuda")
                take[lo:hi] = above | level
                out[la, b, g, :k] = m[take]
    return {"kept": None, "mass": out, "len": None, "pool": None}
