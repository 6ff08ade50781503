"""GPU parity of q3kv_accept_draft against the float64 definition.

Tokens, counts and lengths are equal to the oracle's wherever its decisions are
further than 1e-4 (relative) from a tie: the kernel's p carries the float32
rounding of l - max (2^-24 of at most 60, 3.6e-6 absolute in the exponent for
temperatures >= 0.5: 7.2e-6), of the exponent and its exponential (2^-22) and of a
sum of positive terms in a tree of at most 2^13 additions (2^-11 worst case for a
purely serial sum of 2^13; the kernel's per-thread sums have at most 4,096 terms
in 32-term groups, below 160 roundings, 1e-5): 2e-5 in all, so 1e-4 covers a key
or a test on both sides.  accept_prob: 3e-5 relative by the same count.
"""
import numpy as np
import pytest
import torch

from oracle import accept as oa
from speculative_verify_attention_q3kv_gb300 import _lib, api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(np.asarray(v, np.int32)).cuda()


def _inputs(widths, vocab, dtype, draft_dtype, seed, noise=0.7, tau=1.0, gap=0):
    """Rows of all slots (gap unused rows in front), drafts sampled from the draft rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = sum(widths) + gap
    base = 2.0 * torch.randn((rows, vocab), generator=gen, device="cuda")
    logits = base.to(dtype)
    draft = torch.softmax((base + noise * torch.randn((rows, vocab), generator=gen, device="cuda")) / tau, dim=1).to(draft_dtype)
    drawn = torch.multinomial(draft.float(), 1, generator=gen).flatten().to(torch.int32)
    tokens = torch.cat([drawn.new_zeros(1), drawn[:-1]]).contiguous()
    offs = gap + np.concatenate([[0], np.cumsum(widths)])[:-1]
    uni = torch.rand(rows, generator=gen, device="cuda")
    return logits, draft, tokens, offs, uni


def _run(logits, draft, tokens, offs, widths, uni, tau, seed, ctx=None, max_n_q=16, status=None, prob=True, ws=None, stream=None,
         commit_in_place=False):
    S = len(widths)
    ctx_len = i32([1000 + b for b in range(S)] if ctx is None else ctx)
    acc, nxt = i32([-7] * S), i32([-7] * S)
    com = ctx_len if commit_in_place else i32([-7] * S)
    p = torch.full((logits.shape[0],), -1.0, device="cuda") if prob else None
    if ws is None:
        ws = torch.full((api.accept_draft_workspace_bytes(S, *logits.shape),), 0xA5, dtype=torch.uint8, device="cuda")
    api.accept_draft(logits, draft, i32(offs), i32(widths), tokens, max_n_q, ctx_len, tau, uni, seed, acc, nxt, com, ws,
                     accept_prob=p, status=status, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() if x is not None else None for x in (acc, nxt, com, p)]


def _compare(got, logits, draft, tokens, offs, widths, uni, tau, seed, ctx=None):
    ctx = [1000 + b for b in range(len(widths))] if ctx is None else ctx
    want = oa.draft_accept(logits.double().cpu().numpy(), draft.double().cpu().numpy(), offs, widths, tokens.cpu().numpy(), ctx,
                           float(np.float32(tau)), uni.cpu().numpy().astype(np.float64), seed)
    clear = want[4] > 1e-4
    for g, w in zip(got[:3], want[:3]):
        assert np.array_equal(g[clear], w[clear]), (g, w, want[4])
    if got[3] is not None:
        tested = ~np.isnan(want[3])
        assert np.all(np.abs(got[3][tested] - want[3][tested]) <= 3e-5 * want[3][tested] + 1e-30)
        assert np.all(got[3][~tested] == -1.0)
    return want, clear


CASES = [
    # widths, vocab, logits, draft, tau, noise
    ([6], 248320, torch.bfloat16, torch.float32, 1.0, 0.7),
    ([1], 5, torch.float32, torch.float32, 1.0, 0.5),
    ([2, 1, 16], 1, torch.float32, torch.bfloat16, 0.5, 0.5),
    ([8, 3, 0, 1, 16], 10007, torch.float32, torch.bfloat16, 0.7, 0.3),
    ([4, 4, 4], 2049, torch.bfloat16, torch.bfloat16, 1.3, 0.0),
    ([16] * 9, 4096, torch.bfloat16, torch.float32, 0.9, 1.0),
    ([5], 100003, torch.float32, torch.float32, 2.0, 3.0),
    ([3, 2], 17, torch.bfloat16, torch.float32, 1.0, 5.0),
]


@pytest.mark.parametrize("widths,vocab,dtype,draft_dtype,tau,noise", CASES)
def test_against_the_definition(widths, vocab, dtype, draft_dtype, tau, noise):
    clear = 0
    for seed in (11, 0xFEDCBA9876543210):
        args = _inputs(widths, vocab, dtype, draft_dtype, seed & 0xFFFF, noise, tau, gap=3 if seed == 11 else 0)
        logits, draft, tokens, offs, uni = args
        st = i32([0])
        got = _run(logits, draft, tokens, offs, widths, uni, tau, seed, status=st)
        _, ok = _compare(got, logits, draft, tokens, offs, widths, uni, tau, seed)
        clear += int(ok.sum())
        assert int(st.item()) == 0
    assert clear > len(widths)                       # most decisions are compared


def test_equal_distributions_accept_everything():
    """q = p as the kernel rounds it cannot be told apart from p: with u < 1 - 1e-4 every draft passes."""
    widths, vocab = [16, 7], 3001
    logits, _, tokens, offs, uni = _inputs(widths, vocab, torch.float32, torch.float32, 5)
    draft = torch.softmax(logits.double(), dim=1).float()
    got = _run(logits, draft, tokens, offs, widths, uni.clamp_max(0.999), 1.0, 9)
    assert got[0].tolist() == [15, 6] and got[2].tolist() == [1000, 1001]
    _compare(got, logits, draft, tokens, offs, widths, uni.clamp_max(0.999), 1.0, 9)


def test_masked_logits_and_rows_that_leave_nothing():
    widths, vocab = [4, 3, 2], 1000
    logits, draft, tokens, offs, uni = _inputs(widths, vocab, torch.float32, torch.float32, 6)
    logits[:, ::2] = -float("inf")                   # half of the vocabulary
    logits[2] = -float("inf")
    logits[2, 77] = -3.0e38                          # one token left, at the type's lowest values
    logits[4] = -float("inf")                        # slot 1's first row: nothing left
    tokens[1:] |= 1                                  # odd drafts: not masked
    tokens[3] = 77
    tokens[8] = vocab + 5                            # outside the vocabulary: rejected
    st = i32([0])
    got = _run(logits, draft, tokens, offs, widths, uni, 1.0, 12, status=st)
    _compare(got, logits, draft, tokens, offs, widths, uni, 1.0, 12)
    assert got[0][1] == 0 and got[1][1] == -1        # no token can follow
    assert int(st.item()) == 0


def test_draft_rows_without_mass():
    """A draft distribution of zeros: the token is taken whenever the target allows it, the residual is p."""
    widths, vocab = [3], 500
    logits, draft, tokens, offs, uni = _inputs(widths, vocab, torch.bfloat16, torch.float32, 8)
    draft.zero_()
    got = _run(logits, draft, tokens, offs, widths, uni, 1.0, 3)
    assert got[0][0] == 2 and np.all(got[3][:2] == 1.0)
    _compare(got, logits, draft, tokens, offs, widths, uni, 1.0, 3)


def test_status_bits():
    widths, vocab = [4, 2], 3000
    base = _inputs(widths, vocab, torch.float32, torch.float32, 4)
    bad = _lib.Q3KV_STATUS_NONFINITE_INPUT
    for what in ("nan", "inf", "draft"):
        logits, draft, tokens, offs, uni = [t.clone() if torch.is_tensor(t) else t for t in base]
        if what == "draft":
            draft[0, int(tokens[1])] = float("nan")
        else:
            logits[1, 2999] = float(what)
        st = i32([0])
        acc, nxt, com, _ = _run(logits, draft, tokens, offs, widths, uni, 1.0, 3, status=st)
        assert int(st.item()) == bad
        assert np.all((acc >= 0) & (acc < widths)) and np.all((nxt >= -1) & (nxt < vocab))
    # lengths: more tokens than positions, than the host bound, rows past the logits
    logits, draft, tokens, offs, uni = base
    for kw in (dict(ctx=[3, 1]), dict(max_n_q=1), dict()):
        st = i32([0])
        o = offs if kw else [0, 5]
        acc, nxt, com, p = _run(logits, draft, tokens, o, widths, uni, 1.0, 3, status=st, **kw)
        assert int(st.item()) == _lib.Q3KV_STATUS_BAD_LENGTH
        assert acc[1] == 0 and nxt[1] == -1 and com[1] == (kw.get("ctx", [0, 1001])[1])


def test_commit_in_place_no_prob_and_repeats_give_the_same_bits():
    widths, vocab = [8, 5, 1], 50000
    logits, draft, tokens, offs, uni = _inputs(widths, vocab, torch.bfloat16, torch.bfloat16, 14)
    want = _run(logits, draft, tokens, offs, widths, uni, 0.8, 21)
    for _ in range(5):
        got = _run(logits, draft, tokens, offs, widths, uni, 0.8, 21, commit_in_place=True, prob=False)
        assert all(np.array_equal(g, w) for g, w in zip(got[:3], want[:3]))
    ws = torch.full((api.accept_draft_workspace_bytes(3, *logits.shape),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):                               # a workspace that keeps what the last call left
        got = _run(logits, draft, tokens, offs, widths, uni, 0.8, 21, ws=ws)
        assert all(np.array_equal(g, w) for g, w in zip(got, want))
    # a slot alone decides as it does in the batch (its rows keep their numbers)
    solo = _run(logits, draft, tokens, offs[1:2], widths[1:2], uni, 0.8, 21, ctx=[1001])
    assert [int(x[0]) for x in solo[:3]] == [int(x[1]) for x in want[:3]]


def test_captured_and_replayed_on_another_stream():
    widths, vocab = [6, 6], 30000
    logits, draft, tokens, offs, uni = _inputs(widths, vocab, torch.bfloat16, torch.float32, 15)
    S = 2
    ctx_len, o, w = i32([100, 200]), i32(offs), i32(widths)
    acc, nxt, com = i32([0] * S), i32([0] * S), i32([0] * S)
    ws = torch.zeros(api.accept_draft_workspace_bytes(S, *logits.shape), dtype=torch.uint8, device="cuda")
    call = lambda: api.accept_draft(logits, draft, o, w, tokens, 6, ctx_len, 1.0, uni, 5, acc, nxt, com, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2, 3):
        l2, d2, t2, _, u2 = _inputs(widths, vocab, torch.bfloat16, torch.float32, 100 + seed)
        logits.copy_(l2), draft.copy_(d2), tokens.copy_(t2), uni.copy_(u2)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            g.replay()
            g.replay()
        side.synchronize()
        got = [x.cpu().numpy() for x in (acc, nxt, com)] + [None]
        _compare(got, logits, draft, tokens, offs, widths, uni, 1.0, 5, ctx=[100, 200])


def test_output_follows_the_target():
    """16,384 steps of one draft over four tokens: the committed token's frequencies are the target's.

    Binomial: five standard deviations of a frequency are 5 sqrt(0.25 / 16384) = 0.0196 at most.
    """
    n, vocab = 16384, 4
    p = torch.tensor([0.5, 0.3, 0.15, 0.05], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.4], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(77)
    rows = 2 * n
    logits = p.log().expand(rows, vocab).contiguous()
    draft = q.expand(rows, vocab).contiguous()
    tokens = torch.multinomial(q, rows, replacement=True, generator=gen).to(torch.int32)
    uni = torch.rand(rows, generator=gen, device="cuda")
    acc, nxt, _, _ = _run(logits, draft, tokens, 2 * np.arange(n), [2] * n, uni, 1.0, 99)
    first = np.where(acc == 1, tokens.cpu().numpy()[1::2], nxt)          # the token that follows t_0
    freq = np.bincount(first, minlength=4) / n
    assert np.all(np.abs(freq - p.cpu().numpy()) < 0.02), freq
    bonus = np.bincount(nxt[acc == 1], minlength=4) / max(1, (acc == 1).sum())
    assert np.all(np.abs(bonus - p.cpu().numpy()) < 0.03), bonus
    # accepted with probability sum min(p, q) = 0.1 + 0.3 + 0.15 + 0.05
    assert abs((acc == 1).mean() - 0.6) < 0.02


def test_no_rows_and_no_slots():
    """Idle slots with no logits rows at all, and a call without slots."""
    lg = torch.zeros((0, 77), device="cuda")
    z = torch.zeros(0, device="cuda")
    ws = torch.full((api.accept_draft_workspace_bytes(3, 0, 77),), 9, dtype=torch.uint8, device="cuda")
    acc, nxt, com = i32([5] * 3), i32([5] * 3), i32([5] * 3)
    api.accept_draft(lg, lg, i32([0] * 3), i32([0] * 3), i32([]), 4, i32([10, 20, 30]), 1.0, z, 1, acc, nxt, com, ws)
    torch.cuda.synchronize()
    assert acc.tolist() == [0] * 3 and nxt.tolist() == [-1] * 3 and com.tolist() == [10, 20, 30]
    e = i32([])
    api.accept_draft(lg, lg, e, e, i32([]), 4, e, 1.0, z, 1, e, e, e, None)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mask", ["-inf", "lowest"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [1e-7, 3e-8, 1e-10, 1e-17, 1e-20, 1e-30, 1e-38, 1e28, 1e30, 1e37])
def test_masked_logits_at_extreme_temperatures(tau, dtype, mask):
    """Masks of -inf and of the type's lowest value, over whole chunks of a row, from a one-hot target to a flat one.

    The bounds of this file hold at any temperature: an entry whose exponent counts lies close enough to the
    maximum for an exact difference, or the temperature divides the difference's rounding too.
    """
    widths, vocab = [4, 3, 1], 5003
    logits, draft, tokens, offs, uni = _inputs(widths, vocab, dtype, torch.float32, 23)
    value = -float("inf") if mask == "-inf" else torch.finfo(dtype).min
    logits[:, :2000] = value
    logits[:, 2000::3] = value
    tokens[1] = 17                                   # a masked draft
    tokens[2] = int(logits[1].argmax())              # the one that a cold target takes
    st = i32([0])
    got = _run(logits, draft, tokens, offs, widths, uni, tau, 31, status=st)
    _, clear = _compare(got, logits, draft, tokens, offs, widths, uni, tau, 31)
    assert clear.any() and int(st.item()) == 0
    if mask == "-inf":
        assert np.all(got[1] >= 2000) and np.all((got[1] - 2000) % 3 != 0)      # a masked token never follows
