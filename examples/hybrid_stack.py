"""A small hybrid stack: a Mamba-2 layer, an attention mixer, a Mamba-2 layer.

Prompts of different lengths go through the stack in one call per layer, a second
chunk of each follows over the cached tokens, then single tokens, replayed from a
captured graph, and one more chunk over all of them.  The attention mixer runs
between an RMS norm and a residual add (plain torch here); everything else is the
library's kernels.

    python examples/hybrid_stack.py            # small shapes
    python examples/hybrid_stack.py --wide     # hidden 4096, 32 query and 8 kv heads of 128
"""
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mamba_ssm_layer_gb300 import synth  # noqa: E402
from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache  # noqa: E402
from mamba_ssm_layer_gb300.layer import DeviceLayer, to_dev  # noqa: E402


class HybridStack:
    def __init__(self, mamba_dims, attention_dims, nseq, max_tokens, max_rows):
        self.nseq, self.hidden = nseq, mamba_dims["hidden"]
        self.first, self.last = (DeviceLayer(synth.make_layer(mamba_dims, synth.WL_8B_STACK8, i)) for i in (0, 1))
        self.mixer = DeviceAttention(synth.make_attention(attention_dims, synth.WL_8B_STACK8))
        self.states = [layer.new_state(nseq) for layer in (self.first, self.last)]
        self.cache = Kv4Cache(1, nseq, nseq * (-(-max_tokens // 64)), max_tokens, attention_dims["kv_heads"],
                              attention_dims["head_dim"])
        self.b = self.mixer.buffers(max_rows, nseq * max_tokens, nseq)
        self.ws = self.first.workspace_varlen(nseq, max_rows)
        self.mixed = torch.empty(max_rows, self.hidden, dtype=torch.bfloat16, device="cuda")
        self.kv_len = torch.empty_like(self.cache.pos)

    @staticmethod
    def norm(x):
        f = x.view(torch.bfloat16).float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(torch.bfloat16)

    def prefill(self, x, new):
        """x [sum(new)][hidden] bf16 bits, in place: the next new[i] tokens of each sequence."""
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.cache.reserve(new)
        pos = torch.from_numpy(np.concatenate([t + np.arange(n) for t, n in zip(self.cache.tokens, new)])
                               .astype(np.int32)).cuda()
        self.first.prefill_varlen(x, cu, self.states[0], self.ws)
        out = self.mixed[:x.shape[0]]
        self.mixer.prefill(self.norm(x), new, pos, self.cache, 0, self.b, out, first_over_cache=False)
        x.view(torch.bfloat16).add_(out)
        self.last.prefill_varlen(x, cu, self.states[1], self.ws)
        self.cache.advance(new)

    def decode(self, x):
        """x [nseq][hidden] bf16 bits, in place: one token of each sequence (pages reserved before).  Can be
        captured: the device counts it, ``decoded`` tells the host."""
        self.first.decode(x, self.states[0], self.ws)
        torch.add(self.cache.pos, 1, out=self.kv_len)
        out = self.mixed[:self.nseq]
        self.mixer.decode(self.norm(x), self.cache, 0, self.b, self.kv_len, out)
        x.view(torch.bfloat16).add_(out)
        self.last.decode(x, self.states[1], self.ws)
        self.cache.pos.add_(1)

    def decoded(self, steps):
        """The decode steps that have run since the last prompt or call of this."""
        self.cache.advance([steps] * self.nseq, on_device=False)


def main(wide=False, steps=32):
    mamba = synth.NEMOTRON_H_8B if wide else synth.TINY
    attention = synth.ATTENTION_4096 if wide else synth.TINY_ATTENTION
    nseq = 16 if wide else 3
    lens = [int(n) for n in synth.stack_prompt_lengths()[:nseq]]
    stack = HybridStack(mamba, attention, nseq, 2048, sum(lens) + 64 * nseq)
    x = to_dev(synth.make_hidden(sum(lens), stack.hidden, 7, 0))
    stack.prefill(x, lens)
    chunk = to_dev(synth.make_hidden(64 * nseq, stack.hidden, 7, 1))
    stack.prefill(chunk, [64] * nseq)
    rows = to_dev(synth.make_hidden(nseq, stack.hidden, 7, 2))
    fresh = rows.clone()
    stack.cache.reserve([steps + 1] * nseq)
    stack.decode(rows)  # the first launches load the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stack.decode(rows)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        rows.copy_(fresh)
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    stack.decoded(steps + 1)
    chunk = to_dev(synth.make_hidden(64 * nseq, stack.hidden, 7, 3))
    stack.prefill(chunk, [64] * nseq)
    finite = all(bool(torch.isfinite(x.view(torch.bfloat16)).all()) for x in (rows, chunk))
    print(f"{nseq} sequences, prompts {min(lens)}..{max(lens)} + 64, {steps} tokens each, + 64: "
          f"{t / steps * 1e6:.1f} us a step, finite {finite}")
    return finite and stack.cache.pos.tolist() == stack.cache.tokens == [n + 64 + 1 + steps + 64 for n in lens]


if __name__ == "__main__":
    sys.exit(0 if main("--wide" in sys.argv) else 1)
