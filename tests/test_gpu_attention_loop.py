"""The attention mixer in a conversation: a prompt, tokens from a captured loop, the next chunk.

Attention is held to the 64-bit form on the rows that the stages before it left in
their buffers, with the tolerances of test_gpu_attention.py."""
import pytest
import torch

from mamba_ssm_layer_gb300 import abi, synth
from mamba_ssm_layer_gb300.attention import DeviceAttention, Kv4Cache
from mamba_ssm_layer_gb300.layer import to_dev
from tests import attention_ref as ref
from tests.test_gpu_attention import BF16, EVAL, F16, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from __graft_entry__ import build
    build()
    abi.m2_device_status(clear=True)
    yield
    assert abi.m2_device_status() == abi.M2_OK


class Talk:
    """A mixer, its cache, and the keys and values that every sequence's cache holds, in 64 bits."""

    def __init__(self, dims, nseq, max_tokens=512):
        self.m, self.n = DeviceAttention(synth.make_attention(dims, 9)), nseq
        self.cache = Kv4Cache(1, nseq, nseq * 8, max_tokens, self.m.Hkv, self.m.D)
        self.b = self.m.buffers(600, 2000, nseq)
        self.held = [[] for _ in range(nseq)], [[] for _ in range(nseq)]
        self.call = 0

    def hidden(self, T):
        self.call += 1
        return to_dev(synth.make_hidden(T, self.m.hidden, 9, self.call)).view(torch.bfloat16)

    def rows(self, T):
        """Queries, keys and values that the last call of T rows computed."""
        m, b = self.m, self.b
        v = b["qkv"][:T, (m.H + m.Hkv) * m.D:].reshape(T, m.Hkv, m.D)
        return b["q"][:T].reshape(T, m.H, m.D), b["k"][:T].reshape(T, m.Hkv, m.D), v

    def hold(self, new):
        _, k, v = self.rows(sum(new))
        at = 0
        for i, n in enumerate(new):
            self.held[0][i].append(ref.rounded_rows(k[at:at + n]))
            self.held[1][i].append(ref.rounded_rows(v[at:at + n]))
            at += n

    def check(self, new, prec, own=()):
        """The last call's attention; sequences in `own` attend to their own rows, the others to the cache's."""
        q, k, v = self.rows(sum(new))
        at = 0
        for i, n in enumerate(new):
            r = slice(at, at + n)
            at += n
            kk, vv = (k[r], v[r]) if i in own else (torch.cat(h[i]) for h in self.held)
            want, size = ref.attend(q[r], kk, vv, self.m.scale)
            close(self.b["attn"][r].reshape(n, self.m.H, self.m.D), want, BF16 * want.abs() + (prec + EVAL) * size + 1e-30)

    def prefill(self, new, **how):
        x = self.hidden(sum(new))
        pos = torch.cat([torch.arange(t, t + k) for t, k in zip(self.cache.tokens, new)]).to(torch.int32).cuda()
        self.cache.reserve(new)
        out = torch.empty_like(x)
        self.m.prefill(x, new, pos, self.cache, 0, self.b, out, **how)
        self.hold(new)
        self.cache.advance(new)
        return out


@pytest.mark.parametrize("dims", [synth.TINY_ATTENTION, dict(synth.ATTENTION_4096, hidden=512)])
def test_chunk_after_a_captured_loop(dims):
    t = Talk(dims, 2)
    t.prefill([60, 5])
    t.check([60, 5], BF16, own=(0, 1))
    steps = 9  # over the first page's end
    t.cache.reserve([steps + 1] * 2)
    x = torch.zeros(2, t.m.hidden, dtype=torch.bfloat16, device="cuda")
    out, n = torch.empty_like(x), torch.empty_like(t.cache.pos)

    def step():
        torch.add(t.cache.pos, 1, out=n)
        t.m.decode(x, t.cache, 0, t.b, n, out)
        t.cache.pos.add_(1)
    x.copy_(t.hidden(2))
    step()  # the first launches load the kernels
    t.hold([1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        x.copy_(t.hidden(2))
        graph.replay()
        t.hold([1, 1])
        t.check([1, 1], F16)
    t.cache.advance([steps + 1] * 2, on_device=False)
    assert t.cache.pos.tolist() == t.cache.tokens == [70, 15]
    for new in ([70, 40], [1, 90]):
        t.prefill(new)
        t.check(new, BF16)
    assert t.cache.pos.tolist() == t.cache.tokens == [141, 145]


def test_cache_changes_are_ordered_with_the_calls_on_their_stream():
    """Appends and counts queued behind a long kernel on a side stream: each append sees the count that the calls
    before it left, and a slot is released only after its last call."""
    K, D = 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(50, K * D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    c = Kv4Cache(1, 1, 2, 64, K, D)
    out = [torch.zeros(50, K * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    # the first launches load the kernels, which may wait for everything
    c.reserve([1])
    abi.m2_kv4_append(c.struct[0], k, K * D, v, K * D, [0, 1], c.pos)
    c.advance([1])
    abi.m2_kv4_gather(c.struct[0], out[0], K * D, out[1], K * D, [0, 1])
    c.release(0)
    torch.cuda._sleep(1)
    c.reserve([50])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    for rows, n in ((slice(0, 30), 30), (slice(30, 50), 20)):
        abi.m2_kv4_append(c.struct[0], k[rows], K * D, v[rows], K * D, [0, n], c.pos, s)
        c.advance([n], stream=s)
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    abi.m2_kv4_gather(c.struct[0], out[0], K * D, out[1], K * D, [0, 50], s)
    c.release(0, stream=s)
    c.reserve([1], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for got, x in zip(out, (k, v)):
        assert torch.equal(got.to(ref.F).view(50, K, D), ref.rounded_rows(x.view(50, K, D)))
    assert c.pos.tolist() == [0] and int((c.table >= 0).sum()) == 1


@pytest.mark.parametrize("dims", [synth.TINY_ATTENTION, dict(synth.ATTENTION_4096, hidden=512)])
@pytest.mark.parametrize("over", [False, True])
def test_a_first_prompt_is_the_same_alone_and_beside_a_conversation(dims, over):
    t = Talk(dims, 4)
    t.prefill([40, 0, 0, 17], first_over_cache=over)
    t.check([40, 0, 0, 17], BF16, own=() if over else (0, 3))
    new = [5, 90, 64, 3]
    out = t.prefill(new, first_over_cache=over)
    t.check(new, BF16, own=() if over else (1, 2))
    alone = Talk(dims, 2)
    x = synth.make_hidden(sum(new), t.m.hidden, 9, t.call)[5:159]  # the rows of sequences 1 and 2
    alone.hidden = lambda T: to_dev(x).view(torch.bfloat16)
    assert torch.equal(alone.prefill([90, 64], first_over_cache=over), out[5:159])


def test_slots_without_a_sequence_report_nothing():
    t = Talk(synth.TINY_ATTENTION, 3)
    t.prefill([60, 5, 20], first_over_cache=False)
    t.cache.release(1, idle=True)
    t.cache.reserve([6, 0, 6])
    pages = t.cache.pages[0].clone()
    for _ in range(6):
        x = t.hidden(3)
        out = torch.empty_like(x)
        t.m.decode(x, t.cache, 0, t.b, t.cache.pos + 1, out)
        q, k, v = t.rows(3)
        for i in (0, 2):
            t.held[0][i].append(ref.rounded_rows(k[i:i + 1]))
            t.held[1][i].append(ref.rounded_rows(v[i:i + 1]))
            want, size = ref.attend(q[i:i + 1], *(torch.cat(h[i]) for h in t.held), t.m.scale)
            close(t.b["attn"][i].reshape(1, t.m.H, t.m.D), want, BF16 * want.abs() + (F16 + EVAL) * size + 1e-30)
        assert bool((t.b["attn"][1] == 0).all())
        t.cache.pos.add_(1)  # every slot, as a captured loop does
    t.cache.advance([6, 0, 6], on_device=False)
    assert abi.m2_device_status() == abi.M2_OK
    owned = torch.zeros(len(pages), dtype=torch.bool, device="cuda")
    owned[t.cache.table[t.cache.table >= 0].long()] = True
    assert torch.equal(t.cache.pages[0][~owned], pages[~owned])
    t.held[0][1], t.held[1][1] = [], []
    t.prefill([3, 80, 0], first_over_cache=False)  # the slot's next sequence
    t.check([3, 80, 0], BF16, own=(1,))
    assert t.cache.pos.tolist() == t.cache.tokens == [69, 80, 26]
    # a slot that was not marked still reports
    t.cache.release(2)
    x = t.hidden(3)
    t.cache.reserve([1, 1, 0])
    t.m.decode(x, t.cache, 0, t.b, t.cache.pos + 1, torch.empty_like(x))
    assert abi.m2_device_status(clear=True) == abi.M2_ERR_ARG
