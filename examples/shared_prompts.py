"""Several continuations of a few prompts over one paged KV cache.

A toy model of two attention layers with random weights takes ragged prompts in chunks of
any length, forks each of them into several requests, which share the prompt's full
pages, and decodes them greedily, every one with another first token:

  plan -> (norm, rotate, append; attend) per layer -> LM head      chunk by chunk
  fork -> copy per layer
  plan -> (norm, rotate, append; attend) per layer -> LM head      token by token

Prompts leave as soon as they are forked; half-way some continuations leave too, and the
pages in use are moved to the lowest numbers.  `--check` decodes every continuation by
itself, its whole prompt at once and on pages of its own, and compares the tokens wherever
the two best logits are further apart than roundings can bring them.

  python examples/shared_prompts.py [--check] [--fp8] [--tokens N] [--chunk N]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_draft_02_gb300 as dsp  # noqa: E402

PROMPTS, SAMPLES, V, D = 3, 4, 1024, 256
HEADS_Q, HEADS, DIM, PAGE, LAYERS = 8, 2, 64, 16, 2
LENGTHS = (150, 47, 213)


class Model:
    """Two layers of attention (no feed-forward part) and an LM head, on one page pool."""

    def __init__(self, places, n_rows, fp8):
        g = torch.Generator(device="cuda")
        g.manual_seed(11)
        randn = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.embed, self.W_lm = randn(V, D), randn(V, D)
        self.w_qkv = [0.3 * randn(D, (HEADS_Q + 2 * HEADS) * DIM) for _ in range(LAYERS)]
        self.w_out = [0.05 * randn(HEADS_Q * DIM, D) for _ in range(LAYERS)]
        self.norms = [(1 + 0.1 * randn(DIM), 1 + 0.1 * randn(DIM)) for _ in range(LAYERS)]
        self.rotary = dsp.Rotary(1e4 ** (-np.arange(DIM // 2) * 2.0 / DIM))
        n_pages = 400
        self.pool = dsp.PagePool(places, n_pages, PAGE, 512, n_rows, shared=True)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        shape = (n_pages, PAGE, HEADS, DIM)
        scales = [torch.full((HEADS,), 0.05, device="cuda") for _ in range(2)] if fp8 else []
        self.cache = [dsp.KVCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda").to(dtype)
                                    for _ in range(2)), *scales) for _ in range(LAYERS)]
        self.q = torch.zeros((n_rows, HEADS_Q, DIM), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)

    def logits(self, tokens, most):
        """Logits [n_rows, V] of the planned rows with these tokens [n_rows]; `most` rows a
        request."""
        x = self.embed[tokens.long()]
        for layer in range(LAYERS):
            qkv = (x @ self.w_qkv[layer]).view(-1, HEADS_Q + 2 * HEADS, DIM)
            cache = self.cache[layer]
            self.pool.rope_append(cache, qkv[:, :HEADS_Q], qkv[:, HEADS_Q:HEADS_Q + HEADS],
                                  qkv[:, HEADS_Q + HEADS:], self.rotary, self.q, *self.norms[layer])
            self.pool.attend(cache, self.q, most, self.out)
            x = x + self.out.view(-1, HEADS_Q * DIM) @ self.w_out[layer]
        out = torch.empty((x.shape[0], V), dtype=torch.bfloat16, device="cuda")
        dsp.dspark_lm_head(dsp.dims_of(x.shape[0], 1, V, 64, D), x.contiguous(), self.W_lm, out)
        return out

    def feed(self, rows):
        """New tokens of every place (lists, empty for none) into the cache; the logits after
        each place's last one (None without)."""
        pool, n = self.pool, [len(r) for r in rows]
        pool.plan(torch.tensor(n, dtype=torch.int32, device="cuda"), extra=0)
        flat = [t for r in rows for t in r]
        tokens = torch.zeros((pool.n_rows,), dtype=torch.int32, device="cuda")
        tokens[:len(flat)] = torch.tensor(flat, dtype=torch.int32)
        logits = self.logits(tokens, max(n))
        pool.commit(torch.tensor(n, dtype=torch.int32, device="cuda"))
        ends = np.cumsum(n)
        return [logits[e - 1].float() if k else None for e, k in zip(ends, n)]


def prompts():
    return [[(7 * r + 13 * j * j + 5 * j + 1) % V for j in range(n)] for r, n in enumerate(LENGTHS)]


def first_tokens(prompt, sample):
    return [(31 * prompt + 101 * sample + 3) % V]


def decode_shared(tokens, chunk, fp8):
    places = PROMPTS * (SAMPLES + 1)
    model = Model(places, PROMPTS * max(chunk, SAMPLES), fp8)
    pool = model.pool
    pool.ctx[:PROMPTS] = 0
    rest = prompts()
    while any(rest):
        model.feed([rest[r][:chunk] if r < PROMPTS else [] for r in range(places)])
        rest = [p[chunk:] for p in rest]
    source = [p for p in range(PROMPTS) for _ in range(SAMPLES)]
    target = list(range(PROMPTS, places))
    pool.fork(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (source, target)))
    for cache in model.cache:
        pool.copy(cache)
    pool.ctx[:PROMPTS] = -1                     # the prompts' own places are free again
    got = [first_tokens(p, s) for p in range(PROMPTS) for s in range(SAMPLES)]
    live = set(range(len(got)))
    for i in range(tokens):
        if i == tokens // 2:                    # every third one has said enough
            for k in range(0, len(got), 3):
                live.discard(k)
                pool.ctx[PROMPTS + k] = -1
            pool.squeeze()
            for cache in model.cache:
                pool.move(cache)
        rows = [[]] * PROMPTS + [[got[k][-1]] if k in live else [] for k in range(len(got))]
        for k, logits in enumerate(model.feed(rows)[PROMPTS:]):
            if logits is not None:
                got[k].append(int(logits.argmax()))
    dsp.check_device_status()
    pages = len(pool.free_pages) - int(pool.n_free)
    return got, pages


def check(got, fp8):
    """Every continuation by itself, given its own tokens: the next one is its greedy choice."""
    clear = same = 0
    for k, taken in enumerate(got):
        p = k // SAMPLES
        model = Model(1, LENGTHS[p] + len(taken), fp8)
        model.pool.ctx.zero_()
        model.feed([prompts()[p]])
        for t, then in zip(taken, taken[1:]):
            two = model.feed([[t]])[0].topk(2)
            # logits of size 16 in bf16 lie 1/8 apart, and the attention's own roundings are less
            if float(two.values[0] - two.values[1]) > 0.5:
                clear += 1
                same += int(two.indices[0]) == then
    dsp.check_device_status()
    assert clear and same == clear, (same, clear)
    return clear


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--check", action="store_true")
    ap.add_argument("--fp8", action="store_true")
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--chunk", type=int, default=100)
    a = ap.parse_args(argv)
    got, pages = decode_shared(a.tokens, a.chunk, a.fp8)
    print(f"{sum(map(len, got))} tokens of {len(got)} continuations of {PROMPTS} prompts, "
          f"{pages} pages in use at the end")
    if a.check:
        print(f"{check(got, a.fp8)} clear choices, the same as each continuation by itself")
    return got


if __name__ == "__main__":
    main()
