"""GPU parity of the token counts (equal) and of the logits processing against float64.

Tolerance of the logits: the product with 1 / repetition rounds twice (2^-23 in all) where the definition divides, the
sum frequency c + presence - bias and its subtraction round four times, each by half a step of a value that is at most
M = |y| + frequency c + presence + |bias|: 2^-23 |y| + 2^-22 M <= 2^-21 M.  Then half a step of the logits' type.
"""
import numpy as np
import pytest
import torch

from oracle import logits as ref
from speculative_verify_attention_q3kv_gb300 import _lib, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(np.asarray(v, np.int32)).cuda()


def _stride(vocab):
    return -(-vocab // 8) * 8


# ------------------------------------------------------------------ counts
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("n,vocab", [([0, 1, 5, 16], 1000), ([64, 63, 0, 7], 40), ([65, 3, 0, 1, 300], 2000), ([5000, 1, 70], 50021),
                                     ([20000], 16385), ([1], 1), ([100], 1), ([200000], 3001), ([70001, 30000], 20011)])
def test_counts(n, vocab, prompt):
    rng = np.random.default_rng(len(n))
    slots = len(n)
    counts = rng.integers(-32768, 32767, (slots, _stride(vocab))).astype(np.int16)
    tokens = rng.integers(0, max(1, vocab // 3), sum(n) + 9).astype(np.int32)
    offs = 4 + np.concatenate([[0], np.cumsum(n)])
    want = counts.copy()
    for b in range(slots):
        ref.count(want[b, :vocab], tokens[offs[b]:offs[b] + n[b]], prompt)
    got, status = torch.from_numpy(counts).cuda(), i32([0])
    api.count_tokens(got, vocab, i32(tokens), i32(offs), i32(n), max(max(n), 1), prompt=prompt, status=status)
    assert np.array_equal(got.cpu().numpy(), want) and int(status) == 0


@pytest.mark.parametrize("slots", [6, 200])
def test_counts_at_the_ends_of_rounds(slots):
    # a CTA loads rounds of 8 or 16 times 1,024 tokens, by how many CTAs there are, then single ones; parts of 1, 2 and 4 CTAs
    rng = np.random.default_rng(slots)
    vocab = 16390
    for most in (8193, 16385, 32769, 65537, 65540):
        n = [most - rng.integers(0, 3) if b % 6 < 3 else [0, 1, most // 2][b % 3] for b in range(min(slots, 6))] + [most % 8192 + 1] * (slots - 6)
        tokens = rng.integers(0, vocab, most).astype(np.int32)
        counts = np.zeros((slots, _stride(vocab)), np.int16)
        for b in range(slots):
            counts[b, :vocab] = np.bincount(tokens[:n[b]], minlength=vocab)
        got, status = torch.zeros(counts.shape, dtype=torch.int16, device="cuda"), i32([0])
        api.count_tokens(got, vocab, i32(tokens), i32([0] * slots), i32(n), most, status=status)
        assert np.array_equal(got.cpu().numpy(), counts) and int(status) == 0


@pytest.mark.parametrize("n", [30, 3000])
def test_counts_saturate_and_leave_their_neighbours(n):
    for start in (32767, 32766, 32767 - n + 1, 0):
        counts = torch.zeros((2, 16), dtype=torch.int16, device="cuda")
        counts[:, 5] = start
        counts[:, 4] = -32768
        counts[:, 6] = -1
        api.count_tokens(counts, 16, i32([5] * (2 * n)), i32([0, n]), i32([n, n]), n)
        want = torch.zeros(16, dtype=torch.int16)
        want[4], want[5], want[6] = -32768, min(32767, start + n), -1
        assert torch.equal(counts.cpu(), want.repeat(2, 1))


@pytest.mark.parametrize("n", [20, 2000])
@pytest.mark.parametrize("prompt", [False, True])
def test_count_status_words(n, prompt):
    counts = torch.zeros((4, 104), dtype=torch.int16, device="cuda")
    status = i32([0])
    tokens = torch.full((4 * n,), 3, dtype=torch.int32, device="cuda")
    tokens[1], tokens[2], tokens[5] = -1, 101, 2 ** 31 - 1
    api.count_tokens(counts, 101, tokens, i32([0, n, 2 * n, 3 * n]), i32([n, n, n, n]), n, prompt=prompt, status=status)
    assert int(status) == _lib.Q3KV_STATUS_BAD_TOKEN
    want = np.zeros((4, 104), np.int16)
    for b in range(4):
        ref.count(want[b, :101], tokens[b * n:(b + 1) * n].cpu().tolist(), prompt)
    assert np.array_equal(counts.cpu().numpy(), want)
    for offs, cnt in (([-1, n, 0, 0], [n, 1, 0, 0]), ([0, n, 0, 0], [-1, 1, 0, 0]), ([0, n, 0, 0], [n + 1, 1, 0, 0]),
                      ([3 * n + 1, n, 0, 0], [n, 1, 0, 0])):
        counts.zero_()
        status.zero_()
        api.count_tokens(counts, 101, tokens, i32(offs), i32(cnt), n, prompt=prompt, status=status)
        assert int(status) == _lib.Q3KV_STATUS_BAD_LENGTH and not counts[0].any() and int((counts[1] != 0).sum()) == 1


def test_steps_of_counts_in_a_graph():
    rng = np.random.default_rng(3)
    counts = torch.zeros((3, 504), dtype=torch.int16, device="cuda")
    want = np.zeros((3, 504), np.int16)
    tokens, offs, n = i32(np.zeros(12)), i32([0, 4, 8]), i32([0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.count_tokens(counts, 500, tokens, offs, n, 4)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.count_tokens(counts, 500, tokens, offs, n, 4)
    for _ in range(20):
        t, m = rng.integers(0, 30, 12), rng.integers(0, 5, 3)
        tokens.copy_(i32(t))
        n.copy_(i32(m))
        g.replay()
        for b in range(3):
            ref.count(want[b, :500], t[4 * b:4 * b + m[b]], False)
    assert np.array_equal(counts.cpu().numpy(), want)


# ------------------------------------------------------------------ logits
class Case:
    """Random inputs of a step; every part can be left out."""

    def __init__(self, widths, vocab, dtype, seed=0, counts=True, penalties=True, biases=0, mask=0.0, gap=0, hot=None):
        rng = np.random.default_rng(seed)
        self.widths, self.vocab, self.gap = widths, vocab, gap
        slots, rows = len(widths), sum(widths) + gap
        self.rows = rows
        self.logits = torch.from_numpy((3 * rng.standard_normal((rows, vocab))).astype(np.float32)).to(dtype)
        self.offs = gap + np.concatenate([[0], np.cumsum(widths)])[:-1]
        hot = hot or vocab
        self.tokens = rng.integers(0, hot, rows).astype(np.int32)
        self.counts = None
        if counts:
            c = np.where(rng.random((slots, _stride(vocab))) < 0.2, rng.integers(0, 9, (slots, _stride(vocab))), 0)
            self.counts = np.where(rng.random(c.shape) < 0.1, c - 32768, c).astype(np.int16)
        self.pen = [None] * 3
        if penalties:
            self.pen = [rng.uniform(0.5, 2, slots).astype(np.float32), rng.uniform(-0.5, 1, slots).astype(np.float32),
                        rng.uniform(-1, 1, slots).astype(np.float32)]
        self.bias = None
        if biases:
            each = [min(vocab, biases + b % 3) if b % 4 != 1 else 0 for b in range(slots)]
            toks = [np.sort(rng.choice(vocab, n, replace=False)) for n in each]
            self.bias = (np.concatenate([[0], np.cumsum(each)]), np.concatenate(toks).astype(np.int32),
                         (4 * rng.standard_normal(sum(each))).astype(np.float32))
        self.mask = None
        if mask:
            self.mask = rng.random((rows, vocab)) < mask
            if rows > 3:
                self.mask[rows // 2] = False              # a row that allows nothing

    def call(self, in_place=False, status=None, logits=None, stream=None, out=None):
        x = self.logits.cuda() if logits is None else logits
        if out is None:
            out = x if in_place else torch.full_like(x, 77.0)
        words = None
        if self.mask is not None:
            bits = np.zeros((self.rows, (self.vocab + 31) // 32 * 32), np.uint8)
            bits[:, :self.vocab] = self.mask
            words = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32)).cuda()
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        b = self.bias or (None,) * 3
        api.process_logits(x, out, i32(self.offs), i32(self.widths), i32(self.tokens), max(max(self.widths), 1), counts=dev(self.counts),
                           repetition=dev(self.pen[0]), frequency=dev(self.pen[1]), presence=dev(self.pen[2]),
                           bias_offsets=None if self.bias is None else i32(b[0]), bias_tokens=dev(b[1]), bias_values=dev(b[2]), mask=words,
                           status=status, stream=stream)
        return out

    def check(self, got, in_place=False):
        got = got.double().cpu().numpy()
        x = self.logits.double().numpy()
        if self.gap:
            assert np.array_equal(got[:self.gap], x[:self.gap] if in_place else np.full_like(x[:self.gap], 77.0))
        half = 2.0 ** -8 if self.logits.dtype == torch.bfloat16 else 2.0 ** -24
        for s, (r, w) in enumerate(zip(self.offs, self.widths)):
            if not w:
                continue
            theta, alpha, beta = (float(p[s]) if p is not None else d for p, d in zip(self.pen, (1.0, 0.0, 0.0)))
            pairs = []
            if self.bias is not None:
                lo, hi = self.bias[0][s], self.bias[0][s + 1]
                pairs = list(zip(self.bias[1][lo:hi].tolist(), self.bias[2][lo:hi].astype(np.float64).tolist()))
            c = None if self.counts is None else self.counts[s]
            args = (x[r:r + w], self.tokens[r:r + w].tolist(), c, theta, alpha, beta)
            want = ref.process(*args, pairs, None if self.mask is None else self.mask[r:r + w])
            plain = ref.process(*args[:4], 0.0, 0.0)                                   # after the repetition alone
            with np.errstate(invalid="ignore"):
                terms = np.abs(want - plain)
            M = np.abs(plain) + np.where(np.isfinite(terms), terms, 0.0) + 2 * abs(beta)
            if c is not None:
                M = M + 2 * abs(alpha) * ((c[:self.vocab].astype(np.int64) & 32767) + w)
            else:
                M = M + 2 * abs(alpha) * w
            for t, b in pairs:
                M[:, t] += 2 * abs(b)
            tol = 2.0 ** -21 * M
            tol = tol + half * (np.abs(want) + tol)
            inf = ~np.isfinite(want)
            assert np.array_equal(got[r:r + w][inf], want[inf])
            assert np.all(np.abs(got[r:r + w][~inf] - want[~inf]) <= tol[~inf]), s
        return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("vocab", [1, 7, 31, 33, 64, 2047, 2048, 2056, 5001, 100003])
def test_everything_at_once(vocab, in_place, dtype):
    c = Case([3, 0, 5, 16, 1], vocab, dtype, seed=vocab, biases=20, mask=0.7, gap=2, hot=min(vocab, 40))
    status = i32([0])
    c.check(c.call(in_place, status), in_place)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [4096, 4099])
@pytest.mark.parametrize("kw", [dict(counts=False), dict(penalties=False, mask=0.5), dict(counts=False, penalties=False, biases=300),
                                dict(counts=False, penalties=False, mask=0.1), dict(counts=False, penalties=False), dict()])
def test_parts_left_out(kw, vocab, dtype):
    for in_place in (False, True):
        c = Case([4, 6, 1], vocab, dtype, seed=5, **kw)
        c.check(c.call(in_place), in_place)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [2048, 2049])
def test_repeated_step_tokens_and_the_largest_counts(vocab, dtype):
    c = Case([16, 9], vocab, dtype, seed=6, hot=3)        # three tokens over and over: row j counts them j + 1 times in all
    c.counts[:, 0], c.counts[:, 1], c.counts[:, 2] = 32767, -32768, 0
    c.check(c.call())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [64, 65])
def test_infinite_and_missing_values(vocab, dtype):
    """-inf (an earlier filter) stays, +inf stays, NaN stays NaN unless masked; masked entries are -inf whatever they were."""
    c = Case([2], vocab, dtype, seed=7, mask=1.0)
    c.logits[:, 1], c.logits[:, 2], c.logits[:, 3], c.logits[0, 4:8] = -np.inf, np.inf, np.nan, torch.tensor([np.nan, np.inf, -np.inf, 1.0])
    c.mask[0, 4:8] = False
    for in_place in (False, True):
        got = c.call(in_place, logits=c.logits.clone().cuda()).float().cpu().numpy()
        assert np.all(got[:, 1] == -np.inf) and np.all(got[:, 2] == np.inf) and np.all(np.isnan(got[:, 3])) and np.all(got[0, 4:8] == -np.inf)
        assert np.all(np.isfinite(got[1, 4:8]))


def test_untouched_entries_keep_their_bits():
    x = torch.randint(-2 ** 15, 2 ** 15, (4, 2056), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    out = torch.zeros_like(x)
    api.process_logits(x, out, i32([0]), i32([4]), i32([7, 7, 7, 7]), 4)      # no penalties: even the step's token stays
    keep = torch.ones(2056, dtype=torch.bool, device="cuda")
    keep[:256] = False                                                        # its warp computes
    assert torch.equal(out.view(torch.int16)[:, keep], x.view(torch.int16)[:, keep])


def test_logits_status_words():
    def run(c, widths=None, offs=None, **kw):
        status = i32([0])
        c.widths, c.offs = widths or c.widths, c.offs if offs is None else np.array(offs)
        return c.call(status=status, **kw), int(status)

    for widths, offs in (([2, -1], [0, 2]), ([2, 3], [0, 3]), ([2, 3], [0, -1])):
        c = Case([2, 3], 100, torch.float32)
        out, s = run(c, widths, offs)
        assert s == _lib.Q3KV_STATUS_BAD_LENGTH and bool((out[2:] == 77.0).all()) and bool((out[:2] != 77.0).any())
    c = Case([2, 3], 100, torch.float32, hot=50)
    c.tokens[1], c.tokens[4] = -5, 100                    # counted nowhere
    out, s = run(c)
    assert s == _lib.Q3KV_STATUS_BAD_TOKEN
    c.check(out)
    c = Case([2, 3], 100, torch.float32, biases=10)
    good = c.bias
    c.bias = (good[0], good[1].copy(), good[2])
    c.bias[1][3] = c.bias[1][2]                           # the second of two equal tokens is skipped
    c.bias[1][5] = 100
    out, s = run(c)
    assert s == _lib.Q3KV_STATUS_BAD_TOKEN
    keep = [i for i in range(len(good[1])) if i not in (3, 5)]
    # the entry behind a skipped one is compared with its neighbour in the list all the same
    keep = [i for i in keep if i == good[0][1] or i == 0 or c.bias[1][i] > c.bias[1][i - 1]]
    n0 = sum(i < good[0][1] for i in keep)
    c.bias = (np.array([0, n0, len(keep)]), c.bias[1][keep], good[2][keep])
    c.check(out)
    for offs in ([0, 11, 5], [-1, 3, 5], [0, 3, 10 ** 6]):
        c = Case([2, 3], 100, torch.float32, biases=10)
        c.bias = (np.array(offs), c.bias[1], c.bias[2])
        assert run(c)[1] == _lib.Q3KV_STATUS_BAD_LENGTH


def test_many_slots_and_rows_beyond_32_bit_offsets():
    c = Case([1 + b % 3 for b in range(200)], 1000, torch.bfloat16, seed=8, biases=3, mask=0.5)
    c.check(c.call())
    x = torch.empty((9000, 248320), dtype=torch.bfloat16, device="cuda")            # 4.5 GB
    x[8995:] = 1.0
    counts = torch.zeros((1, 248320), dtype=torch.int16, device="cuda")
    counts[0, 248319] = 2
    two = torch.full((1,), 2.0, device="cuda")
    tokens = torch.zeros(9000, dtype=torch.int32, device="cuda")
    api.process_logits(x, x, i32([8996]), i32([4]), tokens, 4, counts=counts, repetition=two)
    want = torch.ones((5, 248320), dtype=torch.bfloat16, device="cuda")
    want[1:, 0] = want[1:, 248319] = 0.5
    assert torch.equal(x[8995:], want)


def test_logits_on_another_stream_and_in_a_graph():
    c = Case([3, 6], 3001, torch.float32, seed=9, biases=5, mask=0.6)
    want = c.call()
    s = torch.cuda.Stream()
    x = c.logits.cuda()
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    c.call(logits=x, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    offs, n_q, tok, words = i32(c.offs), i32(c.widths), i32(c.tokens), torch.from_numpy(c.counts).cuda()
    theta = torch.from_numpy(c.pen[0]).cuda()
    step = lambda: api.process_logits(x, out, offs, n_q, tok, 6, counts=words, repetition=theta)  # noqa: E731
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.bias = c.mask = None
    c.pen[1:] = [None, None]
    for seed in (10, 11):
        d = Case([3, 6], 3001, torch.float32, seed=seed)
        c.logits, c.counts, c.tokens = d.logits, d.counts, d.tokens
        x.copy_(d.logits)
        words.copy_(torch.from_numpy(d.counts))
        tok.copy_(i32(d.tokens))
        g.replay()
        torch.cuda.synchronize()
        c.check(out)


@pytest.mark.parametrize("n", [3, 70, 700])
def test_biases_out_of_order_do_not_depend_on_one(n):
    """5, 3, 5, 3, ...: every 3 is not above the 5 before it and is skipped; of the entries left for one token the last counts."""
    toks = np.array([5, 3] * n)[:2 * n - 1]
    # and tokens of another chunk, ascending but for one that comes again later
    toks = np.concatenate([toks, [2050, 2060, 2055, 2060, 4000]])
    vals = np.arange(1, len(toks) + 1, dtype=np.float32)
    x = torch.zeros((2, 4096), device="cuda")
    want = torch.zeros((2, 4096))
    want[:, 5], want[:, 2050], want[:, 2060], want[:, 4000] = float(vals[2 * n - 2]), float(vals[-5]), float(vals[-2]), float(vals[-1])
    for _ in range(20):
        out, status = torch.full_like(x, 77.0), i32([0])
        api.process_logits(x, out, i32([0]), i32([2]), i32([0, 0]), 2, bias_offsets=i32([0, len(toks)]), bias_tokens=i32(toks),
                           bias_values=torch.from_numpy(vals).cuda(), status=status)
        assert torch.equal(out.cpu(), want) and int(status) == _lib.Q3KV_STATUS_BAD_TOKEN
