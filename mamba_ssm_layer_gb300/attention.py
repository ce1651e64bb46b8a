"""Device-side holders for the attention mixers of a hybrid stack and their 4-bit cache.

PyTorch provides the device memory and the stream; every computation is one of
the C entry points in ``abi``: the projections (``w8a16_gemv``), the head norm
and rotation, the cache's writes and reads, and attention over a whole prompt or
over the cache.
"""
from __future__ import annotations

import contextlib

import torch

from . import abi
from .layer import _check_count, _check_nodes, _empty, _zeros, to_dev

PAGE = abi.M2_KV4_PAGE


def _on(stream):
    """Torch's own work under the stream of the layers' calls (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class Kv4Cache:
    """The paged 4-bit K/V cache of ``n_layers`` attention layers for ``nseq`` sequences.

    The layers share one page table and one token count per sequence (page p of
    every layer's pool belongs to the same tokens).  ``reserve`` hands out pages
    on the host; appending, reading and attending are the layers' calls; then
    ``advance`` counts the new tokens.  A captured decode loop reserves ahead and
    advances with ``pos.add_(1)`` inside the capture; the host's count follows after
    the replays, before the next ``reserve`` or prompt, with
    ``advance(steps, on_device=False)``.  These calls write the table and the counts
    that the layers' kernels read: they take the same ``stream`` (None: the current
    one), which orders them.
    """

    def __init__(self, n_layers: int, nseq: int, n_pages: int, max_tokens: int, n_kv_heads: int, head_dim: int,
                 device="cuda"):
        self.nseq, self.n_kv_heads, self.head_dim = nseq, n_kv_heads, head_dim
        self.max_pages = -(-max_tokens // PAGE)
        block = abi.m2_kv4_page_bytes(n_kv_heads, head_dim)
        if not block or self.max_pages <= 0:
            raise abi.M2Error("Kv4Cache", abi.M2_ERR_UNSUPPORTED)
        self.pages = [_empty((n_pages, block), torch.uint8, device) for _ in range(n_layers)]
        self.table = _empty((nseq, self.max_pages), torch.int32, device)
        self.table.fill_(-1)
        self.pos = _zeros((nseq,), torch.int32, device)  # tokens held, for the kernels
        self.tokens = [0] * nseq                         # the same, on the host
        self._owned = [[] for _ in range(nseq)]
        self._idle = set()
        self._free = list(range(n_pages - 1, -1, -1))
        self.struct = [abi.kv4_cache(p, n_pages, n_kv_heads, head_dim, self.table, nseq, self.max_pages)
                       for p in self.pages]

    def _counts(self, fn: str, new) -> None:
        if len(new) != self.nseq or min(new) < 0:
            raise abi.M2Error(fn, abi.M2_ERR_ARG)

    def reserve(self, new, stream=None) -> None:
        """Pages for new[i] more tokens of each sequence; all of them or, with an error, none."""
        self._counts("Kv4Cache.reserve", new)
        need = [-(-(t + n) // PAGE) - len(o) for t, n, o in zip(self.tokens, new, self._owned)]
        if sum(max(0, n) for n in need) > len(self._free):
            raise RuntimeError("Kv4Cache: out of pages")
        for i, (n, o) in enumerate(zip(need, self._owned)):
            if len(o) + n > self.max_pages:
                raise RuntimeError(f"Kv4Cache: sequence {i} would pass max_tokens")
        for i, n in enumerate(need):
            if n <= 0:
                continue
            if i in self._idle:
                self._idle.remove(i)
                with _on(stream):
                    self.pos[i] = 0
            have = len(self._owned[i])
            got = [self._free.pop() for _ in range(n)]
            self._owned[i] += got
            with _on(stream):
                self.table[i, have:have + n].copy_(torch.tensor(got, dtype=torch.int32))

    def advance(self, new, on_device: bool = True, stream=None) -> None:
        """Counts new[i] appended tokens of each sequence.  on_device False: on the host only, where ``pos`` has
        counted them already (a captured loop)."""
        self._counts("Kv4Cache.advance", new)
        if on_device:
            with _on(stream):
                self.pos.add_(torch.tensor(list(new), dtype=torch.int32).to(self.pos.device))
        self.tokens = [t + n for t, n in zip(self.tokens, new)]

    def keep(self, cu_nodes, path: torch.Tensor, count: torch.Tensor, stream=None) -> None:
        """After a tree of drafted tokens (``DeviceAttention.tree`` of every layer): the accepted nodes' rows moved
        behind the context in all layers, and ``pos`` advanced by ``count`` (both device int32, of
        ``abi.m2_verify_tree``).  Can be captured; the host's count follows with
        ``advance(count, on_device=False)``."""
        _check_nodes("Kv4Cache.keep", cu_nodes, self.nseq, path)
        _check_count("Kv4Cache.keep", count, self.nseq)
        s = stream if stream is not None else torch.cuda.current_stream()
        for c in self.struct:
            abi.m2_kv4_keep(c, cu_nodes, path, count, self.pos, s)
        with _on(stream):
            self.pos.add_(count.view(-1))

    def release(self, seq: int, stream=None, idle: bool = False) -> None:
        """Gives a finished sequence's pages back.  idle: the slot may stay in decode steps without a sequence (its
        rows are not stored, its output is zeros) until pages are reserved for it; without it such a step reports
        M2_ERR_ARG."""
        self._free += reversed(self._owned[seq])
        self._owned[seq] = []
        self.tokens[seq] = 0
        (self._idle.add if idle else self._idle.discard)(seq)
        with _on(stream):
            self.pos[seq] = abi.M2_KV4_IDLE if idle else 0
            self.table[seq].fill_(-1)


class DeviceAttention:
    """One attention mixer: rows of hidden -> q, k, v projection -> head norm and rotation ->
    attention -> output projection.  ``p``: ``synth.make_attention`` or the like."""

    def __init__(self, p: dict, device="cuda"):
        d = p["dims"]
        self.hidden, self.H, self.Hkv, self.D = d["hidden"], d["heads"], d["kv_heads"], d["head_dim"]
        self.rot, self.eps = d["rot_dim"], d["eps"]
        self.scale = self.D ** -0.5
        self.n_qkv = (self.H + 2 * self.Hkv) * self.D
        self.t = {k: to_dev(p[k], device) for k in ("qkv_w", "qkv_s", "o_w", "o_s")}
        for k in ("q_w", "k_w"):  # head norms, optional
            self.t[k] = None if p.get(k) is None else to_dev(p[k], device)
        self.steps = None
        if self.rot:
            self.steps = torch.tensor(abi.m2_rope_steps(d["theta"], self.rot), dtype=torch.int64).to(device)
        self.device = device

    def buffers(self, max_rows: int, max_keys: int = 0, nseq: int = 1, trees: bool = False) -> dict:
        """Scratch for calls of up to max_rows token rows (prompts over cached tokens: max_keys cached and new
        tokens of all sequences; trees: for ``tree`` too; calls that need more are refused).  Layers run one after
        the other can share it."""
        bf, dev = torch.bfloat16, self.device
        more = {}
        if trees:
            more["tree_ws"] = _empty((abi.m2_attn_tree_kv4_workspace_bytes(self.H, self.Hkv, self.D),), torch.uint8, dev)
        return dict(more, qkv=_empty((max_rows, self.n_qkv), bf, dev), q=_empty((max_rows, self.H * self.D), bf, dev),
                    k=_empty((max_rows, self.Hkv * self.D), bf, dev),
                    attn=_empty((max_rows, self.H * self.D), bf, dev),
                    keys=_empty((max(max_keys, 1), 2 * self.Hkv * self.D), bf, dev),
                    ws=_empty((abi.m2_attn_decode_kv4_workspace_bytes(nseq, self.H, self.Hkv, self.D),), torch.uint8, dev))

    def _check(self, fn, T, x, out, row_pos, cache, b, keys=0) -> None:
        """T rows of x, out and row_pos, and scratch and cache of this mixer's heads that hold them: the kernels
        see pointers only."""
        def dense(t, rows, width):
            return t.shape == (rows, width) and t.element_size() == 2 and t.is_contiguous()
        if not (dense(x, T, self.hidden) and dense(out, T, self.hidden) and row_pos.dtype == torch.int32
                and row_pos.numel() == T and row_pos.is_contiguous()
                and (cache.n_kv_heads, cache.head_dim) == (self.Hkv, self.D)):
            raise abi.M2Error(fn, abi.M2_ERR_ARG)
        widths = dict(qkv=self.n_qkv, q=self.H * self.D, k=self.Hkv * self.D, attn=self.H * self.D,
                      keys=2 * self.Hkv * self.D)
        if any(b[k].shape[1] != w or b[k].shape[0] < (keys if k == "keys" else T) for k, w in widths.items()):
            raise abi.M2Error(fn, abi.M2_ERR_WORKSPACE)

    def _project(self, x, b, row_pos, stream):
        T, H, Hkv, D, n = x.shape[0], self.H, self.Hkv, self.D, self.n_qkv
        qkv = b["qkv"]
        abi.w8a16_gemv(x, self.t["qkv_w"], self.t["qkv_s"], qkv, T, n, self.hidden, stream)
        abi.m2_qk_norm_rope(qkv, n, qkv[:, H * D:], n, b["q"], H * D, b["k"], Hkv * D, self.t["q_w"], self.t["k_w"],
                            row_pos, self.steps, T, H, Hkv, D, self.rot, False, self.eps, stream)
        return b["q"], b["k"], qkv[:, (H + Hkv) * D:]

    def _output(self, b, out, stream):
        abi.w8a16_gemv(b["attn"], self.t["o_w"], self.t["o_s"], out, out.shape[0], self.hidden, self.H * self.D, stream)

    def prefill(self, x, new, row_pos, cache: Kv4Cache, layer: int, b: dict, out, stream=None,
                first_over_cache: bool | None = None) -> None:
        """x, out [sum(new)][hidden] bf16: new[i] tokens of each sequence, after those that the cache holds.
        row_pos: device int32, each row's position.  Appends to the cache (reserved before); the caller advances.

        A sequence that the cache holds tokens of attends to the cache's rows, as the single tokens after this will.
        first_over_cache says what the others attend to: True, to the cache's 4-bit rows too; False, to their own
        bf16 rows (one call for each run of sequences of a kind).  Either way a sequence's result does not depend on
        the rest of the batch.  None, in one call: their own rows if the cache holds no token of any sequence, else
        the cache's, so that a first prompt's result then differs by the 4-bit rounding of its keys and values."""
        cache._counts("DeviceAttention.prefill", new)
        if first_over_cache is None:
            first_over_cache = any(cache.tokens)
        cu, held, runs = [0], [0], []  # row offsets, those of the rows read back; a run: [over the cache, q, k offsets]
        for n, t in zip(new, cache.tokens):
            over = t > 0 or first_over_cache
            held.append(held[-1] + (n + t if n and over else 0))
            cu.append(cu[-1] + n)
            if n:
                at = held if over else cu
                if not runs or runs[-1][0] != over:
                    runs.append([over, [cu[-2]], [at[-2]]])
                runs[-1][1].append(cu[-1])
                runs[-1][2].append(at[-1])
        self._check("DeviceAttention.prefill", cu[-1], x, out, row_pos, cache, b, held[-1])
        s = stream if stream is not None else torch.cuda.current_stream()
        H, Hkv, D = self.H, self.Hkv, self.D
        q, k, v = self._project(x, b, row_pos, s)
        abi.m2_kv4_append(cache.struct[layer], k, Hkv * D, v, self.n_qkv, cu, cache.pos, s)
        fresh, read = (k, Hkv * D, v, self.n_qkv), (b["keys"], 2 * Hkv * D, b["keys"][:, Hkv * D:], 2 * Hkv * D)
        if held[-1]:
            abi.m2_kv4_gather(cache.struct[layer], *read, held, s)
        for over, cq, ck in runs:
            rk, ld_k, rv, ld_v = read if over else fresh
            abi.m2_attn_prefill_varlen(q[cq[0]:], H * D, rk[ck[0]:], ld_k, rv[ck[0]:], ld_v, b["attn"][cq[0]:], H * D,
                                       H, Hkv, D, [c - cq[0] for c in cq], [c - ck[0] for c in ck], self.scale, s)
        self._output(b, out, s)

    def decode(self, x, cache: Kv4Cache, layer: int, b: dict, kv_len, out, stream=None) -> None:
        """x, out [nseq][hidden] bf16: one token of every sequence; kv_len = cache.pos + 1 (device int32).
        Appends and attends; the caller advances.  Can be captured."""
        self._check("DeviceAttention.decode", cache.nseq, x, out, kv_len, cache, b)
        s = stream if stream is not None else torch.cuda.current_stream()
        H, Hkv, D = self.H, self.Hkv, self.D
        q, k, v = self._project(x, b, cache.pos, s)
        abi.m2_kv4_append(cache.struct[layer], k, Hkv * D, v, self.n_qkv, range(cache.nseq + 1), cache.pos, s)
        abi.m2_attn_decode_kv4(cache.struct[layer], q, H * D, b["attn"], H * D, H, kv_len, self.scale, b["ws"],
                               b["ws"].numel(), s)
        self._output(b, out, s)

    def tree(self, x, cu_nodes, parent, row_pos, cache: Kv4Cache, layer: int, b: dict, out, stream=None) -> None:
        """x, out [T][hidden] bf16: the nodes of every sequence's tree of drafted tokens, rows cu_nodes[i] ..
        cu_nodes[i+1]-1 of sequence i; parent and row_pos device int32 [T]: each node's parent, and its position (the
        context's tokens + its depth).  The nodes' keys and values go behind the context (pages for them reserved
        before) and are attended to there; ``Kv4Cache.keep`` then keeps the accepted ones.  Can be captured."""
        _check_nodes("DeviceAttention.tree", cu_nodes, cache.nseq, parent)
        T = cu_nodes[-1]
        self._check("DeviceAttention.tree", T, x, out, row_pos, cache, b)
        if "tree_ws" not in b:
            raise abi.M2Error("DeviceAttention.tree", abi.M2_ERR_WORKSPACE)
        if T == 0:
            return
        s = stream if stream is not None else torch.cuda.current_stream()
        H, Hkv, D = self.H, self.Hkv, self.D
        q, k, v = self._project(x, b, row_pos, s)
        abi.m2_kv4_append(cache.struct[layer], k, Hkv * D, v, self.n_qkv, cu_nodes, cache.pos, s)
        abi.m2_attn_tree_kv4(cache.struct[layer], q, H * D, b["attn"], H * D, H, cu_nodes, parent, cache.pos, self.scale,
                             b["tree_ws"], b["tree_ws"].numel(), s)
        self._output(b, out, s)
