"""Token counts and logits processing (oracle; test infrastructure only), one token and one row at a time."""
from __future__ import annotations

import numpy as np

CAP = 32767


def count(counts: np.ndarray, tokens, prompt: bool) -> None:
    """Add tokens to one slot's int16 words: bits 0..14 the count, bit 15 the prompt's mark."""
    vocab = len(counts)
    for t in tokens:
        if not 0 <= t < vocab:
            continue
        word = int(np.uint16(counts[t]))
        word = word | 0x8000 if prompt else (word & 0x8000) | min((word & CAP) + 1, CAP)
        counts[t] = np.uint16(word).astype(np.int16)


def process(logits, step, counts=None, repetition=1.0, frequency=0.0, presence=0.0, biases=(), masks=None) -> np.ndarray:
    """float64 rows of one slot: logits [w, vocab], its step tokens t_0 .. t_{w-1}, counts int16 [vocab], biases (token, value)
    pairs, masks bool [w, vocab]."""
    x = np.asarray(logits, np.float64).copy()
    w, vocab = x.shape
    words = np.zeros(vocab, np.int16) if counts is None else counts[:vocab]
    c = (words.astype(np.int64) & CAP).astype(np.float64)
    prompt = words < 0
    for j in range(w):
        if 0 <= step[j] < vocab:
            c[step[j]] += 1
        row = x[j]
        with np.errstate(all="ignore"):
            y = np.where((c > 0) | prompt, np.where(row > 0, row / repetition, row * repetition), row)
            y = np.where(c > 0, y - frequency * c - presence, y)
            for t, b in biases:
                y[t] += b
        if masks is not None:
            y = np.where(masks[j], y, -np.inf)
        x[j] = y
    return x
