"""The operators of a paged key-value cache, as measured cases.

Three operators stand between the q|k|v projections of a decoder layer and its
o projection, next to the int4 matmuls of this package:

  tables   block tables, slots and positions of a step's new tokens, from the
           requests' lengths and a list of free pages;
  append   RMS norm and rotary embedding of the new tokens' q and k, and k and v
           written into their slots of the cache;
  attn     attention of one new token per request over its pages, with the
           log-sum-exp of its scores.

`run` computes a case in plain torch operations (own = False) or with the
package's kernels (own = True).
"""
import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's bookkeeping: one new token for each of 64 requests
        dict(name="tables_decode_64", op="tables", B=64, max_ctx=4096, max_new=1, page=16),
        # a prefill batch's: prompts of up to 1024 new tokens behind cached ones
        dict(name="tables_prefill_256", op="tables", B=256, max_ctx=2048, max_new=1024, page=16),
        # the smallest call: the one token of a decode step of the 1.7B-shaped decoder (16 q heads, 8 KV heads of 128)
        dict(name="append_decode_1", op="append", T=1, Hq=16, Hkv=8, D=128, R=128, page=16, dtype="f16", norm=True,
             heads_first=False, pad=0),
        # its prefill over 1024 prompt tokens
        dict(name="append_prefill_1024", op="append", T=1024, Hq=16, Hkv=8, D=128, R=128, page=16, dtype="f16",
             norm=True, heads_first=False, pad=0),
        # fp32 tensors, an odd number of tokens, some of them padding, half of each head rotated, no norm
        dict(name="append_f32_8191", op="append", T=8191, Hq=12, Hkv=12, D=64, R=32, page=24, dtype="f32",
             norm=False, heads_first=True, pad=37),
        # one request behind the 390 audio tokens of a 30 s clip: latency counts
        dict(name="attn_1x390", op="attn", B=1, Hq=16, Hkv=8, D=128, page=16, max_len=390, even=True, dtype="f16",
             heads_first=False),
        # a decode batch of 16 ragged requests
        dict(name="attn_16x1k", op="attn", B=16, Hq=16, Hkv=8, D=128, page=16, max_len=1024, even=False, dtype="f16",
             heads_first=False),
        # a full server: 64 ragged requests of up to 8192 tokens
        dict(name="attn_64x8k", op="attn", B=64, Hq=16, Hkv=8, D=128, page=16, max_len=8192, even=False, dtype="f16",
             heads_first=False),
        # one request with a long context
        dict(name="attn_1x32k", op="attn", B=1, Hq=16, Hkv=8, D=128, page=32, max_len=32768, even=True, dtype="f16",
             heads_first=False),
        # fp32 cache, ragged
        dict(name="attn_f32_8x2k", op="attn", B=8, Hq=16, Hkv=8, D=128, page=16, max_len=2048, even=False,
             dtype="f32", heads_first=False),
        # heads of 64 without sharing, heads before slots in a page, pages of 24
        dict(name="attn_mha64_40x1500", op="attn", B=40, Hq=16, Hkv=16, D=64, page=24, max_len=1500, even=True,
             dtype="f16", heads_first=True),
        # 16 query heads on each of two KV heads of 256
        dict(name="attn_gqa16_24x4k", op="attn", B=24, Hq=32, Hkv=2, D=256, page=64, max_len=4001, even=False,
             dtype="f16", heads_first=True),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn"])
    if op == "tables":
        return dict(op=op, B=_log(rng, 1, 256), max_ctx=_log(rng, 1, 8192), max_new=_log(rng, 1, 1024),
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128]))
    Hkv, G = rng.choice([1, 2, 4, 8, 12, 16]), rng.choice([1, 2, 3, 4, 6, 8, 16])
    while Hkv * G > 64:
        G = rng.choice([1, 2, 3, 4])
    D = rng.choice([64, 64, 80, 96, 128, 128, 256])
    dtype, heads_first = rng.choice(["f16", "f16", "f32"]), rng.random() < 0.5
    es = 2 if dtype == "f16" else 4
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    if op == "append":
        T = _log(rng, 1, 8191)
        while T * (Hkv * G + 2 * Hkv) * D * es > 8191 * 36 * 64 * 4:
            T //= 2
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 16 * 8]), page=page, dtype=dtype,
                    norm=rng.random() < 0.6, heads_first=heads_first, pad=rng.choice([0, 0, T // 5]))
    B, max_len = _log(rng, 1, 64), _log(rng, 1, 32768)
    while B * max_len * Hkv * D * es > 64 * 4096 * 8 * 128 * 2 or B * max_len * Hkv * G * D > 64 * 4096 * 16 * 128:
        B, max_len = max(1, B // 2), max(1, max_len * 3 // 4)
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, max_len=max_len, even=rng.random() < 0.4,
                dtype=dtype, heads_first=heads_first)


# ------------------------------------------------------------------ the inputs

def _lengths(case):
    """The requests' lengths of an attention case: all of them max_len, or ragged up to it (the longest is max_len)."""
    B, n = case["B"], case["max_len"]
    if case["even"]:
        return [n] * B
    # evenly spread over 1..n, in a fixed order that is neither sorted nor periodic
    return [max(1, n * (1 + (i * 7919) % B) // B) for i in range(B)]


def _table_lengths(case):
    B = case["B"]
    ctx = [(case["max_ctx"] * ((i * 7919 + 3) % B)) // B for i in range(B)]
    new = [1 + ((case["max_new"] - 1) * ((i * 104729 + 1) % B)) // max(1, B - 1) for i in range(B)]
    return ctx, new


def _cache(shape, heads_first, dtype, gen):
    """A pool [pages, page, Hkv, D] of values of earlier tokens; heads_first: stored as [pages, Hkv, page, D]."""
    P, ps, H, D = shape
    if heads_first:
        c = torch.empty((P, H, ps, D), dtype=dtype, device="cuda").normal_(generator=gen)
        return c.permute(0, 2, 1, 3)
    return torch.empty((P, ps, H, D), dtype=dtype, device="cuda").normal_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    st = dict(case)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def perm(n):
        return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)

    if case["op"] == "tables":
        ctx, new = _table_lengths(case)
        shift = seed % case["B"]       # another seed: the same lengths in another order
        ctx, new = ctx[shift:] + ctx[:shift], new[shift:] + new[:shift]
        ps, B = case["page"], case["B"]
        width = -(-(case["max_ctx"] + case["max_new"]) // ps)
        held = [-(-c // ps) for c in ctx]
        need = sum(-(-(c + n) // ps) for c, n in zip(ctx, new)) - sum(held)
        pages = sum(held) + need + 64
        order = perm(pages)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        o = 0
        for b in range(B):
            table[b, :held[b]] = order[o:o + held[b]]
            o += held[b]
        T = sum(new)
        st.update(ctx=i32(ctx), new=i32(new), table=table, pages=pages, free=order[o:].contiguous(), start=i32([0]),
                  T=T, seq=i32([0] * B), cu=i32([0] * (B + 1)), slots=torch.zeros(T, dtype=torch.int32, device="cuda"),
                  pos=torch.zeros(T, dtype=torch.int32, device="cuda"), next=i32([0]))
        return st

    dt = _DT[case["dtype"]]
    Hq, H, D, ps = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] == "append":
        T, R = case["T"], case["R"]
        P = -(-T // ps) + 3
        top = max(4096, T)
        # q | k | v as the fused projection leaves them
        qkv = torch.empty((T, (Hq + 2 * H) * D), dtype=dt, device="cuda").normal_(generator=gen)
        q, k, v = qkv.split([Hq * D, H * D, H * D], dim=1)
        inv = 1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        angle = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * inv
        slots = perm(P * ps)[:T].clone()
        if case["pad"]:
            slots[T - case["pad"]:] = -1               # padding behind the last request
        st.update(q=q.view(T, Hq, D), k=k.view(T, H, D), v=v.view(T, H, D), cos=angle.cos().float(),
                  sin=angle.sin().float(), slots=slots, kept=torch.arange(T - case["pad"], device="cuda"),
                  pos=torch.randint(0, top, (T,), generator=gen, device="cuda", dtype=torch.int32),
                  k_cache=_cache((P, ps, H, D), case["heads_first"], dt, gen),
                  v_cache=_cache((P, ps, H, D), case["heads_first"], dt, gen),
                  q_out=torch.empty((T, Hq, D), dtype=dt, device="cuda"), qw=None, kw=None)
        if case["norm"]:
            st.update(qw=1 + 0.1 * torch.empty(D, device="cuda").normal_(generator=gen),
                      kw=1 + 0.1 * torch.empty(D, device="cuda").normal_(generator=gen))
        return st

    B, lens = case["B"], _lengths(case)
    shift = seed % B
    lens = lens[shift:] + lens[:shift]
    held = [-(-n // ps) for n in lens]
    P = sum(held) + 5
    order = perm(P)
    table = torch.full((B, max(held)), -1, dtype=torch.int32, device="cuda")
    o = 0
    for b in range(B):
        table[b, :held[b]] = order[o:o + held[b]]
        o += held[b]
    # normed and rotated q and k have entries of about 1; a factor makes some keys stand out, as trained heads do
    st.update(lens=i32(lens), table=table, scale=D ** -0.5,
              q=(2.0 * torch.empty((B, Hq, D), device="cuda").normal_(generator=gen)).to(dt),
              k_cache=_cache((P, ps, H, D), case["heads_first"], dt, gen),
              v_cache=_cache((P, ps, H, D), case["heads_first"], dt, gen),
              out=torch.empty((B, Hq, D), dtype=dt, device="cuda"), lse=torch.empty((B, Hq), device="cuda"))
    if own:
        import int4_block_quantized_matmulnbits_b200 as mnb

        st["ws"] = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(B, Hq, H, D, dt), dtype=torch.uint8,
                               device="cuda")
    return st


# ------------------------------------------------------------------- the passes

def run(st):
    return {"tables": _run_tables, "append": _run_append, "attn": _run_attn}[st["op"]](st)


def _run_tables(st):
    if own:
        import int4_block_quantized_matmulnbits_b200 as mnb

        mnb.mnb_paged_tables(st["ctx"], st["new"], st["table"], st["page"], st["pages"], st["free"], st["start"],
                             st["seq"], st["cu"], st["slots"], st["pos"], st["next"])
        return [st[n] for n in ("table", "seq", "cu", "slots", "pos", "next")]
    ps, T, i32 = st["page"], st["T"], torch.int32
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    seq = ctx + new
    had = (ctx + ps - 1) // ps
    need = (seq + ps - 1) // ps - had
    cu = torch.cat([torch.zeros_like(ctx[:1]), new.cumsum(0)])
    end = need.cumsum(0)
    # the j-th column of row b is a new page where had <= j < had + need
    j = torch.arange(table.shape[1], device="cuda")[None, :] - had[:, None]
    taken = (j >= 0) & (j < need[:, None])
    src = (st["start"].long() + (end - need)[:, None] + j).clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(taken, st["free"][src], table))
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[row] + t - cu[row]
    slots = table[row, pos // ps].long() * ps + pos % ps
    return [table, seq.to(i32), cu.to(i32), slots.to(i32), pos.to(i32), (st["start"] + end[-1:]).to(i32)]


def _turn(x, w, cos, sin, R, eps=1e-6):
    """RMS norm (w not None), then the rotary embedding of the first R entries, halves paired."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], dim=-1)


def _run_append(st):
    if own:
        import int4_block_quantized_matmulnbits_b200 as mnb

        mnb.mnb_rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], st["pos"],
                            st["cos"], st["sin"], st["q_out"], st["qw"], st["kw"], 1e-6)
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    dt, R, ps = st["q"].dtype, st["R"], st["page"]
    pos, kept = st["pos"].long(), st["kept"]
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    slot = st["slots"][kept].long()
    st["k_cache"][slot // ps, slot % ps] = _turn(st["k"], st["kw"], cos, sin, R).to(dt)[kept]
    st["v_cache"][slot // ps, slot % ps] = st["v"][kept]
    return [_turn(st["q"], st["qw"], cos, sin, R).to(dt), st["k_cache"], st["v_cache"]]


def _run_attn(st):
    if own:
        import int4_block_quantized_matmulnbits_b200 as mnb

        mnb.mnb_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["scale"],
                                st["out"], st["ws"], st["lse"])
        return [st["out"], st["lse"]]
    B, Hq, H, D, ps = (st[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    n = st["max_len"]
    at = torch.arange(n, device="cuda")
    page, off = st["table"][:, at // ps].clamp(min=0).long(), (at % ps)[None, :]
    live = at[None, :] < st["lens"][:, None]                                             # [B, n]
    q = st["q"].float().view(B, H, Hq // H, D)
    k = st["k_cache"][page, off].float()                                                 # [B, n, H, D]
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]                             # [B, H, G, n]
    del k
    s = s.masked_fill(~live[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = st["v_cache"][page, off].float() * live[:, :, None, None]
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / l
    lse = (m + torch.log(l)).view(B, Hq)
    return [o.view(B, Hq, D).to(st["q"].dtype), lse]


# --------------------------------------------------------------- bytes and flops

def work(case):
    if case["op"] == "tables":
        ctx, new = _table_lengths(case)
        ps, B, T = case["page"], case["B"], sum(new)
        need = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        # lengths in, lengths and offsets out, pages from the list into the table, slots and positions out
        return dict(bytes=4 * (2 * B + 2 * B + 1 + 2 * need + 2 * T + 2), flops=4 * (T + B))
    es, Hq, H, D = (2 if case["dtype"] == "f16" else 4), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        T, R = case["T"], case["R"]
        kept = T - case["pad"]
        rows = min(T, max(4096, T))
        moved = 2 * T * Hq * D * es + 4 * kept * H * D * es + 8 * T + rows * R * 4
        return dict(bytes=moved, flops=T * (Hq + H) * (3 * R + (4 * D if case["norm"] else 0)))
    lens = _lengths(case)
    tot = sum(lens)
    table = sum(-(-n // case["page"]) for n in lens)
    return dict(bytes=tot * H * D * 2 * es + 2 * case["B"] * Hq * D * es + 4 * (table + case["B"] * (1 + Hq)),
                flops=4 * tot * Hq * D)


# ----------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        ps = case["page"]
        table, free = st["table"].cpu().numpy().copy(), st["free"].cpu().numpy()
        seq, cu, slots, pos, at = [], [0], [], [], 0
        for b, (c, n) in enumerate(zip(st["ctx"].tolist(), st["new"].tolist())):
            for j in range(-(-c // ps), -(-(c + n) // ps)):
                table[b, j] = free[at]
                at += 1
            for p in range(c, c + n):
                slots.append(int(table[b, p // ps]) * ps + p % ps)
                pos.append(p)
            seq.append(c + n)
            cu.append(cu[-1] + n)
        return [torch.from_numpy(np.asarray(x, dtype=np.int32)) for x in (table, seq, cu, slots, pos, [at])]
    if case["op"] == "append":
        R, ps = case["R"], case["page"]
        outs = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / case["D"] + 1e-6) * w.double()
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous())
            turn = torch.complex(st["cos"].double(), st["sin"].double())[st["pos"].long()][:, None]
            z = z * turn
            outs.append(torch.cat([z.real, z.imag, x[..., R:]], dim=-1))
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        n = case["T"] - case["pad"]
        s = st["slots"][:n].long()
        kc[s.div(ps, rounding_mode="floor"), s.remainder(ps)] = outs[1][:n]
        vc[s.div(ps, rounding_mode="floor"), s.remainder(ps)] = st["v"][:n].double()
        return [outs[0], kc, vc]
    B, Hq, H, D, ps = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    out, lse = torch.empty((B, Hq, D), dtype=torch.float64, device="cuda"), torch.empty((B, Hq), dtype=torch.float64,
                                                                                       device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        pages = st["table"][b, :-(-n // ps)].long()
        k = st["k_cache"][pages].reshape(-1, H, D)[:n].double()
        v = st["v_cache"][pages].reshape(-1, H, D)[:n].double()
        s = torch.einsum("hgd,nhd->hgn", st["q"][b].double().view(H, Hq // H, D), k) * st["scale"]
        z = torch.logsumexp(s, dim=-1)
        out[b] = torch.einsum("hgn,nhd->hgd", torch.exp(s - z[..., None]), v).reshape(Hq, D)
        lse[b] = z.reshape(Hq)
    return [out, lse]
