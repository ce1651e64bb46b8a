"""Drafted tokens on a small hybrid stack (Mamba-2 layer, attention mixer, Mamba-2 layer).

Every step a draft proposes a tree of tokens for each sequence, one pass of the stack
runs all nodes, the target's probabilities decide which path holds, and state, conv ring
and cache keep that path.  The pass, the verification and the keeping are one captured
graph; only the tokens change.  Embedding, output projection and draft are random
matrices (plain torch): what is shown is the loop, not a model.

    python examples/drafted_tokens.py            # small shapes
    python examples/drafted_tokens.py --wide     # hidden 4096, 32 query and 8 kv heads of 128
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.hybrid_stack import HybridStack  # noqa: E402
from mamba_ssm_layer_gb300 import abi, synth  # noqa: E402

PARENT = (-1, 0, 0, 1, 1, 2, 3)  # two candidates for the next token, two below the first, one below the second, ..


class DraftedStack(HybridStack):
    def __init__(self, mamba_dims, attention_dims, nseq, max_tokens, max_rows, vocab):
        super().__init__(mamba_dims, attention_dims, nseq, max_tokens, max_rows)
        n, T = len(PARENT), nseq * len(PARENT)
        dev, g = "cuda", torch.Generator(device="cuda").manual_seed(1)
        self.vocab, self.gen = vocab, g
        self.cu = [n * i for i in range(nseq + 1)]
        depth = []
        for p in PARENT:
            depth.append(0 if p < 0 else depth[p] + 1)
        self.parent = torch.tensor(PARENT * nseq, dtype=torch.int32, device=dev)
        self.depth = torch.tensor(depth * nseq, dtype=torch.int32, device=dev)
        self.seq = torch.arange(nseq, device=dev).repeat_interleave(n)
        # the row that a node's token is drawn from
        self.above = torch.tensor([n * i + max(p, 0) for i in range(nseq) for p in PARENT], device=dev)
        self.b = self.mixer.buffers(max_rows, nseq * max_tokens, nseq, trees=True)
        self.tree_ws = [layer.workspace_tree(nseq, T) for layer in (self.first, self.last)]
        self.embed = torch.randn(vocab, self.hidden, device=dev, generator=g).to(torch.bfloat16)
        self.head = (torch.randn(self.hidden, vocab, device=dev, generator=g) * self.hidden ** -0.5).to(torch.bfloat16)
        self.rows = torch.empty(T, self.hidden, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty_like(self.rows)
        self.p = torch.empty(T, vocab, device=dev)
        self.q = torch.empty(T, vocab, device=dev)
        self.u, self.u_next = torch.empty(T, device=dev), torch.empty(nseq, device=dev)
        self.token = torch.zeros(T, dtype=torch.int32, device=dev)
        self.path = torch.empty(T, dtype=torch.int32, device=dev)
        self.count, self.next = (torch.empty(nseq, dtype=torch.int32, device=dev) for _ in range(2))

    def draft(self):
        """Tokens of the nodes, level by level, from a small model's probabilities (here: of the token alone)."""
        self.token[::len(PARENT)].copy_(self.next)
        for r in range(1, len(PARENT)):
            here = torch.arange(self.nseq, device="cuda") * len(PARENT)
            logits = (self.embed[self.token[here + PARENT[r]].long()] @ self.head).float()
            q = torch.softmax(logits, -1)
            self.q[here + PARENT[r]] = q
            self.token[here + r] = torch.multinomial(q, 1, generator=self.gen)[:, 0].int()
        self.u.copy_(torch.rand(self.u.shape, device="cuda", generator=self.gen))
        self.u_next.copy_(torch.rand(self.nseq, device="cuda", generator=self.gen))

    def step(self):
        """One pass over all nodes, the walk, and the keeping.  Can be captured."""
        torch.index_select(self.embed, 0, self.token, out=self.rows)
        bits = self.rows.view(torch.int16)
        self.first.tree(bits, self.cu, self.parent, self.states[0], self.tree_ws[0])
        pos = self.cache.pos[self.seq] + self.depth
        self.mixer.tree(self.norm(self.rows), self.cu, self.parent, pos, self.cache, 0, self.b, self.out)
        self.rows.add_(self.out)
        self.last.tree(bits, self.cu, self.parent, self.states[1], self.tree_ws[1])
        torch.softmax((self.norm(self.rows) @ self.head).float(), -1, out=self.p)
        abi.m2_verify_tree(self.p, self.vocab, self.q, self.vocab, abi.M2_PROB_F32, self.vocab, self.cu, self.parent,
                           self.token, self.u, self.u_next, self.path, self.count, self.next,
                           torch.cuda.current_stream())
        for layer, state, ws in zip((self.first, self.last), self.states, self.tree_ws):
            layer.tree_commit(self.cu, self.path, self.count, state, ws)
        self.cache.keep(self.cu, self.path, self.count)


def main(wide=False, steps=32):
    mamba = synth.NEMOTRON_H_8B if wide else synth.TINY
    attention = synth.ATTENTION_4096 if wide else synth.TINY_ATTENTION
    nseq, n = (16 if wide else 3), len(PARENT)
    lens = [int(k) for k in synth.stack_prompt_lengths()[:nseq]]
    stack = DraftedStack(mamba, attention, nseq, 2048, max(sum(lens), nseq * n), 32000 if wide else 500)
    stack.prefill(stack.embed[torch.randint(0, stack.vocab, (sum(lens),), device="cuda", generator=stack.gen)]
                  .view(torch.int16), lens)
    stack.next.zero_()
    tokens, graph, spent = [0] * nseq, None, 0.0
    for k in range(steps):
        stack.cache.reserve([n] * nseq)  # before the pages' next use; the graph reads the table
        stack.draft()
        if k == 0:
            stack.step()  # the first launches load the kernels
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                stack.step()
            graph.replay()
        else:
            torch.cuda.synchronize()
            t = time.perf_counter()
            graph.replay()
            torch.cuda.synchronize()
            spent += time.perf_counter() - t
        count = stack.count.tolist()
        stack.cache.advance(count, on_device=False)
        tokens = [a + b for a, b in zip(tokens, count)]
    print(f"{nseq} sequences, trees of {n}: {sum(tokens) / steps / nseq:.2f} tokens a sequence and step, "
          f"{spent / max(1, steps - 2) * 1e6:.0f} us a step")
    good = stack.cache.pos.tolist() == stack.cache.tokens == [a + b for a, b in zip(lens, tokens)]
    good &= all(s[2].tolist() == stack.cache.tokens for s in stack.states)
    return good and all(1 <= c <= n for c in count) and bool(torch.isfinite(stack.rows).all())


if __name__ == "__main__":
    sys.exit(0 if main("--wide" in sys.argv) else 1)
