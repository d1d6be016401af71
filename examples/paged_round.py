"""A few rounds of speculative decoding with the target's paged KV cache.

A toy target model of two attention layers with random weights decodes for a
batch of requests.  Every round drafts with the Markov head, schedules, runs
the target over the admitted rows and verifies:

  draft -> schedule -> plan -> (append, attend) per layer -> LM head -> verify

`--tree` drafts a tree instead (each request's chain and, beside every draft, a
sibling), and takes the path that the target's greedy choices confirm:

  draft -> plan -> (append, attend) per layer -> LM head -> accept -> compact

In both forms the emitted tokens are the target's own greedy ones, whatever the
drafts: `--check` decodes the same requests token by token, one row at a time,
and compares.

  python examples/paged_round.py [--tree] [--check] [--fp8] [--rounds N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_draft_02_gb300 as dsp  # noqa: E402
import workloads  # noqa: E402

R, GAMMA, V, RANK, D = 6, 4, 1024, 64, 256
HEADS_Q, HEADS, DIM, PAGE, LAYERS = 8, 2, 64, 16, 2


class Target:
    """Two layers of attention (no feed-forward part) and an LM head, on one page pool."""

    def __init__(self, W_lm, n_rows, fp8):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        randn = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.embed, self.W_lm = randn(V, D), W_lm
        # sharp enough that greedy choices do not hang on a rounding
        self.w_qkv = [0.3 * randn(D, (HEADS_Q + 2 * HEADS) * DIM) for _ in range(LAYERS)]
        self.w_out = [0.05 * randn(HEADS_Q * DIM, D) for _ in range(LAYERS)]
        self.where = randn(4096, D)  # positions
        n_pages = 256
        self.pool = dsp.PagePool(R, n_pages, PAGE, 1024, n_rows)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        shape = (n_pages, PAGE, HEADS, DIM)
        scales = [torch.full((HEADS,), 0.05, device="cuda") for _ in range(2)] if fp8 else []
        self.cache = [dsp.KVCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda").to(dtype)
                                    for _ in range(2)), *scales) for _ in range(LAYERS)]
        self.out = torch.zeros((n_rows, HEADS_Q, DIM), dtype=torch.bfloat16, device="cuda")

    def logits(self, tokens, max_nodes):
        """Target logits [n_rows, V] of planned rows with these tokens [n_rows]."""
        pool = self.pool
        x = self.embed[tokens.long()] + self.where[pool.position.clamp(min=0).long()]
        for layer in range(LAYERS):
            qkv = (x @ self.w_qkv[layer]).view(-1, HEADS_Q + 2 * HEADS, DIM)
            pool.append(self.cache[layer], qkv[:, HEADS_Q:HEADS_Q + HEADS],
                        qkv[:, HEADS_Q + HEADS:])
            pool.attend(self.cache[layer], qkv[:, :HEADS_Q], max_nodes, self.out)
            x = x + self.out.view(-1, HEADS_Q * DIM) @ self.w_out[layer]
        out = torch.empty((x.shape[0], V), dtype=torch.bfloat16, device="cuda")
        dsp.dspark_lm_head(dsp.dims_of(x.shape[0], 1, V, RANK, D), x.contiguous(), self.W_lm, out)
        return out

    def rows_of(self, per_request):
        """[n_rows] of the ragged batch from [R, nodes] (padding rows take token 0)."""
        row = torch.arange(self.pool.n_rows, device="cuda")
        req = torch.searchsorted(self.pool.row_start[1:].long(), row, right=True).clamp(max=R - 1)
        node = (row - self.pool.row_start.long()[req]).clamp(max=per_request.shape[1] - 1)
        return torch.where(self.pool.position >= 0, per_request[req, node], 0)

    def prefill(self, prompts):
        """Prompts [R, n] token by token of position: rows of one node each."""
        self.pool.ctx.zero_()
        none = torch.zeros(R, dtype=torch.int32, device="cuda")
        for j in range(prompts.shape[1]):
            self.pool.plan(none)
            self.logits(self.rows_of(prompts[:, j:j + 1]), 1)
            self.pool.commit(none + 1)


def prompts():
    return torch.tensor([[(7 * r + 13 * j + 1) % V for j in range(5)] for r in range(R)],
                        dtype=torch.int32, device="cuda")


def head_and_inputs():
    w = workloads.WORKLOADS["tiny"].with_(R=R, gamma=GAMMA, V=V, r=RANK, d=D, anchor_hi=V)
    inp = workloads.make_inputs(w, with_target_noise=False)
    head = dsp.DraftHead.from_weights(R, GAMMA, inp["W_lm"], inp["W1"], inp["W2"], inp["w_conf"],
                                      inp["T"])
    return head, inp


def hidden(i):
    """The backbone's hidden states of round i (synthetic, as everywhere here)."""
    return workloads.random_normal((R * GAMMA, D), 1.0, 900 + i).to("cuda")


def decode_chain(rounds, fp8=False):
    head, inp = head_and_inputs()
    rnd = dsp.Round(head)
    sps = workloads.sps_table("concave", R * (GAMMA + 1)).to("cuda")
    target = Target(head.W_lm, R * (GAMMA + 1), fp8)
    start = prompts()
    target.prefill(start[:, :-1])
    anchor = start[:, -1].contiguous()
    emitted = [[] for _ in range(R)]
    for i in range(rounds):
        rnd.draft(hidden(i), anchor, 0.0, i)
        if i % 2:  # every other round: drafts that the target likes, some of the way
            rnd.tokens.copy_(continue_greedily(target, anchor, i))
        rnd.schedule(sps)
        target.pool.plan(rnd.len)
        nodes = torch.cat([anchor[:, None], rnd.tokens], 1)
        logits = target.logits(target.rows_of(nodes), GAMMA + 1)
        # [R, gamma + 1, V]: row j scores position j; rows past a request's are not read
        row = (target.pool.row_start[:-1, None] + torch.arange(GAMMA + 1, device="cuda"))
        per_request = logits[row.clamp(max=logits.shape[0] - 1).long()].contiguous()
        rnd.verify(anchor, per_request, 0.0, i)
        target.pool.commit(rnd.accepted + 1)
        acc, tok, bonus = rnd.accepted.tolist(), rnd.tokens.tolist(), rnd.bonus.tolist()
        for r in range(R):
            emitted[r] += tok[r][:acc[r]] + [bonus[r]]
        anchor = rnd.bonus.clone()
    dsp.check_device_status()
    return emitted


def continue_greedily(target, anchor, i):
    """Drafts that follow the target for i % gamma + 1 tokens and then leave it (made by
    decoding ahead; the rows written are written again by the round)."""
    ctx = target.pool.ctx.clone()
    none = torch.zeros(R, dtype=torch.int32, device="cuda")
    cur, out = anchor, []
    for j in range(GAMMA):
        target.pool.plan(none)
        cur = target.logits(target.rows_of(cur[:, None]), 1)[:R].argmax(-1).to(torch.int32)
        target.pool.commit(none + 1)
        out.append(cur if j <= i % GAMMA else (cur + 1) % V)
    target.pool.ctx.copy_(ctx)
    return torch.stack(out, 1)


def decode_tree(rounds, fp8=False):
    head, _ = head_and_inputs()
    rnd = dsp.Round(head)
    nodes = 2 * GAMMA  # node 2j - 1: draft j's sibling, node 2j: draft j, below draft j - 1
    target = Target(head.W_lm, R * (nodes + 1), fp8)
    start = prompts()
    target.prefill(start[:, :-1])
    anchor = start[:, -1].contiguous()
    parent = torch.tensor([[2 * (j // 2) for j in range(nodes)]] * R, dtype=torch.int32,
                          device="cuda")
    full = torch.full((R,), nodes, dtype=torch.int32, device="cuda")
    path = torch.empty((R, nodes), dtype=torch.int32, device="cuda")
    emitted = [[] for _ in range(R)]
    for i in range(rounds):
        rnd.draft(hidden(i), anchor, 0.0, i)
        if i % 2:
            rnd.tokens.copy_(continue_greedily(target, anchor, i))
        tokens = torch.stack([(rnd.tokens + 3) % V, rnd.tokens], 2).view(R, nodes).contiguous()
        target.pool.plan(full, parent=parent)
        logits = target.logits(target.rows_of(torch.cat([anchor[:, None], tokens], 1)), nodes + 1)
        choice = logits.argmax(-1).to(torch.int32)
        target.pool.accept(tokens, choice, path, parent=parent)
        for cache in target.cache:
            target.pool.compact(cache, path)
        took, bonus, tok = path.tolist(), target.pool.bonus.tolist(), tokens.tolist()
        for r in range(R):
            emitted[r] += [tok[r][n - 1] for n in took[r] if n > 0] + [bonus[r]]
        anchor = target.pool.bonus.clone()
    dsp.check_device_status()
    return emitted


def decode_plainly(n, fp8=False):
    head, _ = head_and_inputs()
    target = Target(head.W_lm, R, fp8)
    start = prompts()
    target.prefill(start[:, :-1])
    cur, emitted = start[:, -1].contiguous(), []
    none = torch.zeros(R, dtype=torch.int32, device="cuda")
    for _ in range(n):
        target.pool.plan(none)
        cur = target.logits(target.rows_of(cur[:, None]), 1).argmax(-1).to(torch.int32)
        target.pool.commit(none + 1)
        emitted.append(cur)
    return torch.stack(emitted, 1).tolist()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tree", action="store_true")
    ap.add_argument("--check", action="store_true")
    ap.add_argument("--fp8", action="store_true")
    ap.add_argument("--rounds", type=int, default=8)
    a = ap.parse_args(argv)
    emitted = (decode_tree if a.tree else decode_chain)(a.rounds, a.fp8)
    total = sum(map(len, emitted))
    print(f"{total} tokens for {R} requests in {a.rounds} rounds "
          f"({total / R / a.rounds:.2f} a round and request)")
    if a.check:
        plain = decode_plainly(max(map(len, emitted)), a.fp8)
        for r in range(R):
            assert emitted[r] == plain[r][:len(emitted[r])], (r, emitted[r], plain[r])
        print("the same tokens as decoding one at a time")
    return emitted


if __name__ == "__main__":
    main()
