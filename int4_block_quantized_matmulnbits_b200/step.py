"""Quantized linears and the decoder-shaped passes that chain them.

The decoders of "Mega-ASR -- INT4 ONNX (GPTQ-calibrated)" and "Qwen3-ASR-0.6B
-- ONNX for the browser" spend ~95% of their work in MatMulNBits
("Compression vs original"): per token, 28 layers x 7 projections plus the
lm_head (decoder_step), and the same projections over all prompt tokens in
decoder_init / decoder_prefill.  These classes hold the packed weights in HBM
and issue the library calls of one such pass; every call is one CUDA kernel
of libmnb, optionally captured into a CUDA graph.
"""
from __future__ import annotations

import contextlib

import torch

from . import (MNB_FLAG_PDL, mnb_dequantize, mnb_embed_gather, mnb_gemm, mnb_gemv, mnb_gemv_argmax,
               mnb_gemv_argmax_workspace_bytes, mnb_gemv_chain, mnb_gemv_chain_plan, mnb_gemv_chain_workspace_bytes,
               mnb_gemv_swiglu, mnb_matmul, mnb_packed_sizes, mnb_paged_attention, mnb_paged_attention_workspace_bytes,
               mnb_paged_tables, mnb_quantize_rtn, mnb_rope_append)


class QLinear:
    """One MatMulNBits weight [N, K]: packed uint8 [N, K/2], scales [N, K/bs], zp or None."""

    def __init__(self, N, K, bs, has_zp=True, scale_dtype=torch.float16, device="cuda", name=""):
        self.N, self.K, self.bs, self.has_zp, self.name = N, K, bs, has_zp, name
        pb, sb, zb = mnb_packed_sizes(N, K, bs, scale_dtype, has_zp)
        self.packed = torch.empty((N, K // 2), dtype=torch.uint8, device=device)
        self.scales = torch.empty((N, K // bs), dtype=scale_dtype, device=device)
        self.zp = torch.empty((N, (K // bs + 1) // 2), dtype=torch.uint8, device=device) if has_zp else None
        self.nbytes = pb + sb + zb

    @classmethod
    def quantize(cls, W, bs, has_zp=True, scale_dtype=torch.float16, name="", stream=None):
        """RTN-quantize an fp32 [N, K] device tensor with mnb_quantize_rtn."""
        N, K = W.shape
        q = cls(N, K, bs, has_zp, scale_dtype, W.device, name)
        mnb_quantize_rtn(W.contiguous(), N, K, bs, has_zp, q.packed, q.scales, q.zp, stream)
        return q

    def dequantize(self, dtype=torch.float16, stream=None):
        out = torch.empty((self.N, self.K), dtype=dtype, device=self.packed.device)
        mnb_dequantize(self.packed, self.scales, self.zp, self.N, self.K, self.bs, out, stream)
        return out

    def gemv(self, X, Y, flags=0, stream=None):
        mnb_gemv(X, self.packed, self.scales, self.zp, Y, X.shape[0], self.N, self.K, self.bs, flags, stream)

    def gemv_swiglu(self, X, Y, flags=0, stream=None):
        mnb_gemv_swiglu(X, self.packed, self.scales, self.zp, Y, X.shape[0], self.N, self.K, self.bs, flags, stream)

    def gemv_argmax(self, X, Y, ids, max_out, workspace, flags=0, stream=None):
        mnb_gemv_argmax(X, self.packed, self.scales, self.zp, Y, X.shape[0], self.N, self.K, self.bs, ids, max_out,
                        workspace, flags, stream)

    def gemm(self, X, Y, flags=0, stream=None):
        mnb_gemm(X, self.packed, self.scales, self.zp, Y, X.shape[0], self.N, self.K, self.bs, flags, stream)

    def matmul(self, X, Y, flags=0, stream=None):
        mnb_matmul(X, self.packed, self.scales, self.zp, Y, X.shape[0], self.N, self.K, self.bs, flags, stream)


def concat_linears(parts, name=""):
    """One QLinear whose rows are the rows of `parts` in order.

    Projections that read the same input (q, k, v; gate, up) are one
    MatMulNBits over their row-concatenated weights: the packed rows, scales and
    zero points are per row, so concatenation changes no stored value, and the
    outputs come out concatenated in the same order."""
    K, bs, has_zp = parts[0].K, parts[0].bs, parts[0].has_zp
    assert all(p.K == K and p.bs == bs and p.has_zp == has_zp for p in parts)
    N = sum(p.N for p in parts)
    q = QLinear(N, K, bs, has_zp, parts[0].scales.dtype, parts[0].packed.device, name)
    torch.cat([p.packed for p in parts], dim=0, out=q.packed)
    torch.cat([p.scales for p in parts], dim=0, out=q.scales)
    if has_zp:
        torch.cat([p.zp for p in parts], dim=0, out=q.zp)
    q.parts = [(p.name, p.N) for p in parts]
    return q


def swiglu_interleave(gate, up, name=""):
    """One QLinear [2I, K] for mnb_gemv_swiglu: rows in groups of 16, the 8 gate
    rows 8j..8j+7 followed by the 8 up rows of the same outputs.  Every stored
    quantity is per row, so interleaving changes no stored value."""
    assert gate.N == up.N and gate.K == up.K and gate.bs == up.bs and gate.has_zp == up.has_zp
    assert gate.N % 8 == 0
    I = gate.N
    q = QLinear(2 * I, gate.K, gate.bs, gate.has_zp, gate.scales.dtype, gate.packed.device, name)

    def inter(a, b, out):
        g = a.reshape(I // 8, 8, *a.shape[1:])
        u = b.reshape(I // 8, 8, *b.shape[1:])
        out.copy_(torch.stack([g, u], dim=1).reshape(2 * I, *a.shape[1:]))

    inter(gate.packed, up.packed, q.packed)
    inter(gate.scales, up.scales, q.scales)
    if gate.has_zp:
        inter(gate.zp, up.zp, q.zp)
    q.swiglu = True   # a decode pass runs it through mnb_gemv_swiglu: N / 2 outputs
    return q


def fuse_decoder(linears, swiglu=False):
    """Per layer [q, k, v, o, gate, up, down] -> [qkv, o, gate_up, down]; others kept.
    swiglu=True stores gate/up interleaved for the fused SwiGLU epilogue."""
    out, i = [], 0
    while i < len(linears):
        names = [l.name.rstrip("0123456789") for l in linears[i:i + 7]]
        if names == ["q", "k", "v", "o", "gate", "up", "down"]:
            L = linears[i:i + 7]
            layer = L[0].name[1:]
            gu = swiglu_interleave(L[4], L[5], f"gate_up{layer}") if swiglu else \
                concat_linears(L[4:6], f"gate_up{layer}")
            out += [concat_linears(L[0:3], f"qkv{layer}"), L[3], gu, L[6]]
            i += 7
        else:
            out.append(linears[i])
            i += 1
    return out


def _on(stream):
    """A context in which torch works on `stream`: None (the current one), a Stream, or a handle as the library's calls
    take it."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


class PagedCache:
    """Keys and values of a decoder's layers in pages, for up to `requests` requests at once.

    The requests' lengths, their block table and the list of free pages live on the
    device and advance there, so a captured step can be replayed token after token:
    begin() hands out the pages and slots of the step's new tokens (mnb_paged_tables),
    layer() appends one layer's keys and values (mnb_rope_append) and attends over them
    (mnb_paged_attention), end() makes the new lengths current.  All layers share the
    table; each has a pool of its own, [pages, page_size, Hkv, D].

    max_len: the tokens that a request may hold; a step that would give it more is
    refused for that request (status 2) and leaves it as it is.  cos, sin: fp32
    [max_len or more, rot_dim / 2] (None: no rotation).  norms: per layer a pair
    of fp32 [D] RMS-norm weights of q and k, or None.  status: the device word that the
    three calls report to; check() reads it.

    A row's pages are not handed back while the others go on: restore() of the state
    that state() gave before the first step makes all rows and pages free again.
    """

    def __init__(self, layers, requests, Hq, Hkv, D, max_len, page_size=16, pages=None, dtype=torch.float16,
                 cos=None, sin=None, norms=None, eps=1e-6, scale=None, device="cuda"):
        self.requests, self.Hq, self.Hkv, self.D = requests, Hq, Hkv, D
        self.page_size, self.cos, self.sin, self.norms, self.eps = page_size, cos, sin, norms, eps
        self.scale = D ** -0.5 if scale is None else scale
        blocks = -(-max_len // page_size)
        self.max_len, self._room = max_len, blocks * page_size
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin go together")
        for name, t in (("cos", cos), ("sin", sin)):
            if t is not None and t.shape[0] < max_len:   # positions without an angle would be dropped
                raise ValueError(f"{name} has {t.shape[0]} rows for max_len = {max_len}")
        self.pages = requests * blocks if pages is None else pages
        self.k, self.v = ([torch.zeros((self.pages, page_size, Hkv, D), dtype=dtype, device=device)
                           for _ in range(layers)] for _ in range(2))

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)

        self.table, self.lens, self.new_lens = i32(requests, blocks), i32(requests), i32(requests)
        self.cu_new, self.one, self.status = i32(requests + 1), i32(requests) + 1, i32(1)
        self.free = torch.arange(self.pages, dtype=torch.int32, device=device)
        self.start, self.next = i32(1), i32(1)
        # a decode step's slots and positions, and its rotated queries
        self.slots, self.positions = i32(requests), i32(requests)
        self.q = torch.zeros((requests, Hq, D), dtype=dtype, device=device)
        self.ws = torch.zeros((mnb_paged_attention_workspace_bytes(requests, Hq, Hkv, D, dtype),), dtype=torch.uint8,
                              device=device)
        self._own_slots = self._decode = False   # of the step that begin() has begun: see there

    launches_per_step = 1            # begin(); end() is two copies
    launches_per_layer = 2

    def begin(self, new=None, slots=None, positions=None, flags=0, stream=None):
        """Pages and slots of new [requests] more tokens a request (None: one each, a decode step), the slots and
        positions of the new tokens in buffers of the caller's then.  The new tokens stand one request behind the
        other: with a request that gets none or several, row b is not request b's, so layer() takes decode steps only,
        and append() without slots only steps whose slots are in the cache's own buffers."""
        if (slots is None) != (positions is None):
            raise ValueError("slots and positions go together")
        self._own_slots = self._decode = False
        own, decode = slots is None, new is None and slots is None
        slots, positions = (self.slots, self.positions) if own else (slots, positions)
        lens, new, over = self.lens, self.one if new is None else new, None
        if self.max_len < self._room:
            # The tables know whole pages only: requests that would pass max_len inside their last page are shown to
            # them as full (five small launches of torch's for a max_len that is no multiple of page_size).
            with _on(stream):
                over = lens.long() + new > self.max_len
                lens = lens.masked_fill(over, self._room)
        mnb_paged_tables(lens, new, self.table, self.page_size, self.pages, self.free, self.start, self.new_lens,
                         self.cu_new, slots, positions, self.next, self.status, flags, stream)
        if over is not None:
            with _on(stream):
                self.new_lens.copy_(torch.where(over, self.lens, self.new_lens))
        self._own_slots, self._decode = own, decode

    def append(self, layer, q, k, v, q_out, slots=None, positions=None, flags=0, stream=None):
        """q [T, Hq, D] normed and rotated into q_out, k and v [T, Hkv, D] into the layer's pools."""
        if (slots is None) != (positions is None):
            raise ValueError("slots and positions go together")
        if slots is None and not self._own_slots:
            raise RuntimeError("append() without slots: begin() has put none into the cache's own buffers")
        slots, positions = (self.slots, self.positions) if slots is None else (slots, positions)
        qw, kw = (None, None) if self.norms is None else self.norms[layer]
        mnb_rope_append(q, k, v, self.k[layer], self.v[layer], slots, positions, self.cos, self.sin, q_out, qw, kw,
                        self.eps, self.status, flags, stream)

    def layer(self, layer, q, k, v, out, flags=0, stream=None):
        """One layer of a decode step: out [requests, Hq, D] from this step's q, k and v."""
        if not self._decode:
            raise RuntimeError("layer() outside a decode step: it follows begin() without new tokens or slots given")
        self.append(layer, q, k, v, self.q, flags=flags, stream=stream)
        mnb_paged_attention(self.q, self.k[layer], self.v[layer], self.table, self.new_lens, self.scale, out, self.ws,
                            None, self.status, flags, stream)

    def end(self, stream=None):
        """The step's lengths and free-list position become current."""
        with _on(stream):
            self.lens.copy_(self.new_lens)
            self.start.copy_(self.next)
        self._own_slots = self._decode = False

    def state(self, stream=None):
        """Lengths, free-list position and status, to be given to restore(): steps in between are then undone (their
        pages go back to the list; the rows they wrote are written again by the next steps).  Both in order with the
        steps of `stream`."""
        with _on(stream):
            return [t.clone() for t in (self.lens, self.start, self.status)]

    def restore(self, state, stream=None):
        with _on(stream):
            for t, was in zip((self.lens, self.start, self.status), state):
                t.copy_(was)

    def check(self, stream=None):
        """Raises if a step since the last check met a bad index, a request without room or an empty free list.
        Waits for the steps of `stream` (None: for the whole device, on whichever streams they run)."""
        if stream is None and self.status.is_cuda:
            torch.cuda.synchronize(self.status.device)
        with _on(stream):
            word = int(self.status.item())
            self.status.zero_()
        if stream is None and self.status.is_cuda:
            torch.cuda.synchronize(self.status.device)   # cleared before a later step on another stream reports
        if word:
            raise RuntimeError(f"paged cache: status {word} (1 a bad index, 2 a length without room, 4 no free page)")


class Pass:
    """A chain of MatMulNBits calls with one X / Y buffer pair per linear.

    kind = "gemv" (decode step, M <= 32), "gemm" (prefill) or "matmul" (any M:
    mnb_matmul picks the kernel).  With pdl=True each
    launch may overlap the tail of the previous one (weights stream early, X is
    read after the previous kernel completes).  An optional int8 embedding
    gather of M token ids runs first, as in a decode step.

    attention: a PagedCache for M requests.  The pass is then a decode step whose
    attention runs too: after each layer's v (or fused qkv) projection, q, k and v
    go through PagedCache.layer, whose result is the input of that layer's o
    projection, and every run appends one token to each request.
    """

    def __init__(self, linears, M, kind="gemv", act_dtype=torch.float16, pdl=True, embed=None, greedy=False,
                 chain=False, waits=None, attention=None):
        self.linears, self.M, self.kind, self.pdl = list(linears), M, kind, pdl
        dev = self.linears[0].packed.device
        # one flat buffer each for all inputs and all outputs (views per linear,
        # 16-byte aligned), so a step's inputs and outputs move in one copy each
        xs = [M * l.K for l in self.linears]
        ys = [M * (l.N // 2 if getattr(l, "swiglu", False) else l.N) for l in self.linears]
        self.x_flat = torch.zeros((sum(xs),), dtype=act_dtype, device=dev)
        self.y_flat = torch.zeros((sum(ys),), dtype=act_dtype, device=dev)
        self.X, self.Y = [], []
        ox = oy = 0
        for l, nx, ny in zip(self.linears, xs, ys):
            self.X.append(self.x_flat[ox:ox + nx].view(M, l.K))
            self.Y.append(self.y_flat[oy:oy + ny].view(M, ny // M))
            ox, oy = ox + nx, oy + ny
        for t in self.X + self.Y:
            assert t.data_ptr() % 16 == 0
        self.embed = embed   # (table, row_scales, ids[M], out[M, D]) or None
        self.graph = None
        # greedy=True: the last linear (the lm_head) also picks each token's id
        self.greedy = greedy and kind == "gemv"
        if self.greedy:
            self.ids = torch.zeros((M,), dtype=torch.int32, device=dev)
            self.max_out = torch.zeros((M,), dtype=torch.float32, device=dev)
            self.ws = torch.zeros((mnb_gemv_argmax_workspace_bytes(M),), dtype=torch.uint8, device=dev)
        # chain=True: all GEMVs in one persistent launch (mnb_gemv_chain).  waits[i]
        # = 1 makes linear i read its X only after linears 0..i-1 are complete
        # (default: every linear waits, the dependencies of separate launches)
        self.chain = None
        if chain:
            assert kind == "gemv" and not self.greedy
            assert not any(getattr(l, "swiglu", False) for l in self.linears)
            n = len(self.linears)
            waits = [1] * n if waits is None else list(waits)
            tasks = [(x, l.packed, l.scales, l.zp, y, l.N, l.K, w)
                     for l, x, y, w in zip(self.linears, self.X, self.Y, waits)]
            plan = mnb_gemv_chain_plan(tasks, M, self.linears[0].bs)
            self.chain = (plan, plan.to(dev),
                          torch.zeros((mnb_gemv_chain_workspace_bytes(n),), dtype=torch.uint8, device=dev))

        self.attention = attention
        if attention is not None:
            assert self.chain is None and attention.requests == M and attention.q.dtype == act_dtype
            self.layers = self._attention_layers()   # {index of the v or qkv projection: (layer, q, k, v, out)}

    def _attention_layers(self):
        c, at, found = self.attention, {l.name: i for i, l in enumerate(self.linears)}, {}
        nq, nk = c.Hq * c.D, c.Hkv * c.D
        for layer in range(len(c.k)):
            if f"qkv{layer}" in at:
                last = at[f"qkv{layer}"]
                q, k, v = self.Y[last].split([nq, nk, nk], dim=1)
            else:
                q, k, v = (self.Y[at[f"{n}{layer}"]] for n in "qkv")
                last = max(at[f"{n}{layer}"] for n in "qkv")
            o = at[f"o{layer}"]
            assert last < o and self.linears[o].K == nq
            heads = [t.view(self.M, -1, c.D) for t in (q, k, v, self.X[o])]
            assert [t.shape[1] for t in heads] == [c.Hq, c.Hkv, c.Hkv, c.Hq]
            found[last] = (layer, *heads)
        return found

    @property
    def weight_bytes(self):
        return sum(l.nbytes for l in self.linears)

    @property
    def flops(self):
        return sum(2 * self.M * l.N * l.K for l in self.linears)

    @property
    def launches(self):
        n = 1 if self.chain is not None else len(self.linears)
        if self.attention is not None:
            n += self.attention.launches_per_step + len(self.layers) * self.attention.launches_per_layer
        return n + (1 if self.embed is not None else 0)

    def run(self, stream=None):
        if self.embed is not None:
            table, rs, ids, out = self.embed
            mnb_embed_gather(table, rs, table.shape[0], table.shape[1], ids, ids.shape[0], out,
                             None, stream)
        flags = MNB_FLAG_PDL if self.pdl else 0
        if self.chain is not None:
            mnb_gemv_chain(*self.chain, flags, stream)
            return
        last = len(self.linears) - 1
        if self.attention is not None:
            self.attention.begin(flags=0, stream=stream)   # after the copies that ended the last step
        for i, (l, x, y) in enumerate(zip(self.linears, self.X, self.Y)):
            if self.kind == "gemv":
                if self.greedy and i == last:
                    l.gemv_argmax(x, y, self.ids, self.max_out, self.ws, flags, stream)
                elif getattr(l, "swiglu", False):
                    l.gemv_swiglu(x, y, flags, stream)
                else:
                    l.gemv(x, y, flags, stream)
            elif self.kind == "matmul":
                l.matmul(x, y, flags, stream)
            else:
                l.gemm(x, y, flags, stream)
            if self.attention is not None and i in self.layers:
                self.attention.layer(*self.layers[i], flags=flags, stream=stream)
        if self.attention is not None:
            self.attention.end(stream)

    def capture(self):
        """Capture run() into a CUDA graph (replayed with replay())."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            state = None if self.attention is None else self.attention.state()
            self.run(s)          # warm-up outside the graph (first-use attribute setup)
            if state is not None:
                self.attention.restore(state)   # the warm-up's tokens are no step of the user's
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            self.run(s)
        self.graph = g
        return g

    def replay(self):
        self.graph.replay()
