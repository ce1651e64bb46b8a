"""The attention mixer as a hybrid stack runs it: prompts, chunks over cached tokens, single tokens.

Each stage is held to the 64-bit form of that stage on the values that the stage
before it left in its buffer, with the tolerances of test_gpu_attention.py."""
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


@pytest.mark.parametrize("dims", [synth.TINY_ATTENTION, dict(synth.ATTENTION_4096, hidden=512, rot_dim=64)])
def test_mixer_stages(dims):
    m = DeviceAttention(synth.make_attention(dims, 9))
    H, K, D, n = m.H, m.Hkv, m.D, 3
    cache = Kv4Cache(2, n, 40, 400, K, D)
    b = m.buffers(300, 1200, n)
    held = [[] for _ in range(n)], [[] for _ in range(n)]  # the cache's keys and values of every sequence
    for call, new in enumerate([[100, 0, 37], [5, 130, 64], None, None, [1, 2, 3], None]):
        single = new is None
        new = [1] * n if single else new
        T = sum(new)
        x = to_dev(synth.make_hidden(T, m.hidden, 9, call)).view(torch.bfloat16)
        pos = torch.cat([torch.arange(t, t + k) for t, k in zip(cache.tokens, new)]).to(torch.int32).cuda()
        out = torch.empty(T, m.hidden, dtype=torch.bfloat16, device="cuda")
        cache.reserve(new)
        if single:
            m.decode(x, cache, 1, b, cache.pos + 1, out)
        else:
            m.prefill(x, new, pos, cache, 1, b, out)
        qkv = b["qkv"][:T]
        q0, k0, v0 = (t.reshape(T, -1, D) for t in (qkv[:, :H * D], qkv[:, H * D:(H + K) * D], qkv[:, (H + K) * D:]))
        for got, x0, w in ((b["q"], q0, m.t["q_w"]), (b["k"], k0, m.t["k_w"])):
            y, size = ref.rope(x0, w.view(torch.bfloat16), pos, dims["theta"], dims["rot_dim"], False, dims["eps"])
            close(got[:T].reshape(T, -1, D), y, BF16 * y.abs() + 2.0 ** -19 * size)
        # what each sequence attends to: the cache's values, or its own fresh rows in a first prompt
        q, k, at = b["q"][:T].reshape(T, H, D), b["k"][:T].reshape(T, K, D), 0
        over_cache = single or sum(cache.tokens) > 0
        for i in range(n):
            rows = slice(at, at + new[i])
            at += new[i]
            held[0][i].append(ref.rounded_rows(k[rows]))
            held[1][i].append(ref.rounded_rows(v0[rows]))
            kk, vv = (torch.cat(h[i]) for h in held) if over_cache else (k[rows], v0[rows])
            want, size = ref.attend(q[rows], kk, vv, m.scale)
            prec = F16 if single else BF16
            close(b["attn"][rows].reshape(-1, H, D), want, BF16 * want.abs() + (prec + EVAL) * size + 1e-30)
        # the output projection is w8a16_gemv, whose own tests hold it; here: it saw these rows
        again = torch.empty_like(out)
        abi.w8a16_gemv(b["attn"], m.t["o_w"], m.t["o_s"], again, T, m.hidden, H * D)
        assert torch.equal(again, out)
        cache.advance(new)
    assert cache.pos.tolist() == cache.tokens == [109, 135, 107]


def test_cache_pages_are_handed_out_and_taken_back():
    c = Kv4Cache(1, 2, 4, 192, 2, 64)
    c.reserve([65, 10])
    assert int((c.table >= 0).sum()) == 3 and len(set(c.table[c.table >= 0].tolist())) == 3
    c.advance([65, 10])
    c.reserve([63, 54])  # fits the pages it has
    assert int((c.table >= 0).sum()) == 3
    with pytest.raises(RuntimeError):
        c.reserve([64, 55])
    assert int((c.table >= 0).sum()) == 3  # nothing handed out by a refused call
    c.release(0)
    assert c.pos.tolist() == [0, 10] and int((c.table[0] >= 0).sum()) == 0
    c.reserve([192, 0])
    with pytest.raises(RuntimeError):
        c.reserve([193, 0])


def test_example_runs():
    from examples import hybrid_stack
    assert hybrid_stack.main(wide=False, steps=5)


def test_kernels_time_out_cleanly():
    """Pipeline waits that give up at once: the kernels record it, wait for their own copies and products, return,
    and compute correctly afterwards.  The decode reads 80 MB that L2 does not hold, so that copies are waited for."""
    g = torch.Generator(device="cuda").manual_seed(1)
    H, K, D, T, n_q = 32, 8, 128, 70000, 2000
    q, k, v = (torch.randn(r, w * D, device="cuda", generator=g).to(torch.bfloat16) for r, w in ((n_q, H), (T, K), (T, K)))
    c = Kv4Cache(1, 1, 1100, T, K, D)
    c.reserve([T])
    abi.m2_kv4_append(c.struct[0], k, K * D, v, K * D, [0, T], c.pos)
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = torch.empty(abi.m2_attn_decode_kv4_workspace_bytes(1, H, K, D), dtype=torch.uint8, device="cuda")

    def run():
        o1 = torch.zeros(n_q, H * D, dtype=torch.bfloat16, device="cuda")
        o2 = torch.zeros(1, H * D, dtype=torch.bfloat16, device="cuda")
        abi.m2_attn_prefill_varlen(q, H * D, k, K * D, v, K * D, o1, H * D, H, K, D, [0, n_q], [0, n_q], 0.1)
        s1 = abi.m2_device_status(clear=True)
        torch.zeros(512 << 20, dtype=torch.uint8, device="cuda")  # through L2
        abi.m2_attn_decode_kv4(c.struct[0], q, H * D, o2, H * D, H, n, 0.1, ws, ws.numel())
        return o1, o2, s1, abi.m2_device_status(clear=True)

    first = run()  # the first launch of a kernel in a process starts its roles late
    assert first[2:] == (abi.M2_OK, abi.M2_OK)
    try:
        abi.m2_set_wait_limit(1)
        assert run()[2:] == (abi.M2_ERR_TIMEOUT, abi.M2_ERR_TIMEOUT)
    finally:
        abi.m2_set_wait_limit(0)
    again = run()
    assert again[2:] == (abi.M2_OK, abi.M2_OK)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
