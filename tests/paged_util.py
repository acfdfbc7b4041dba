"""Plain 64-bit definitions of the paged cache's operators, on the CPU, and inputs for their tests."""
import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


def tables_ref(ctx, new, table, page, num_pages, free, start, T):
    """mnb_paged_tables by its definition, request by request; returns (table, seq, cu, slots, pos, next, status)."""
    table = table.copy()
    width = table.shape[1]
    slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int64)
    seq, cu, status, taken, out_of_pages = [], [0], 0, 0, False
    avail = len(free) - start
    if not 0 <= start <= len(free):
        avail, status = 0, 4
    asked = 0   # pages asked for so far, granted or not
    for b, (c, n) in enumerate(zip(ctx, new)):
        first = cu[-1]
        cu.append(min(first + max(n, 0), 2 ** 31 - 1))   # int32: the sum stops there
        if c < 0 or n < 0 or c + n > width * page or cu[-1] > T:
            status |= 2
            seq.append(max(c, 0))
            continue
        need = ceil_div(c + n, page) - ceil_div(c, page)
        asked += need
        if need and asked > avail:
            out_of_pages = True
            status |= 4
            seq.append(c)
            continue
        for j in range(need):
            table[b, ceil_div(c, page) + j] = free[start + taken + j]
        taken += need
        seq.append(c + n)
        for i in range(n):
            p = c + i
            pg = table[b, p // page]
            pos[first + i] = p
            if 0 <= pg < num_pages:
                slots[first + i] = int(pg) * page + p % page
            else:
                status |= 1
    assert not out_of_pages or asked > avail
    return table, np.array(seq, np.int64), np.array(cu, np.int64), slots, pos, start + taken, status


def turn_ref(x, w, eps, cos, sin, pos):
    """RMS norm (w not None) and half-paired rotary embedding of x [T, H, D] in float64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos is None:
        return x
    h = cos.shape[1]
    c, s = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * h:]], -1)


def attn_ref(q, k_cache, v_cache, table, lens, scale):
    """(out, lse, spread, reach) in float64: spread = sum_j p_j |v_j| per output, reach = the largest
    |scale| sum_d |q_d k_d| of a row, the quantities that the rounding errors scale with."""
    B, Hq, D = q.shape
    P, ps, H, _ = k_cache.shape
    G = Hq // H
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64)
    spread, reach = torch.zeros_like(out), torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        j = torch.arange(n)
        page = table[b, (j // ps)].long()
        ok = (page >= 0) & (page < P)
        page, off = page[ok], (j % ps)[ok]
        if not len(page):
            continue
        k = k_cache[page, off].double()   # [n, H, D]
        v = v_cache[page, off].double()
        for i in range(Hq):
            s = (k[:, i // G] @ q[b, i].double()) * scale
            lse[b, i] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, i])
            out[b, i] = p @ v[:, i // G]
            spread[b, i] = p @ v[:, i // G].abs()
            reach[b, i] = (k[:, i // G].abs() @ q[b, i].double().abs()).max() * abs(scale)
    return out, lse, spread, reach


def attn_tolerance(out, lse, spread, reach, dtype, n_max, D):
    """Bounds on |out - ref| and |lse - ref|, from the arithmetic of the kernel:
      score      D fp32 products and sums, the scaling: (D + 4) 2^-24 of reach, as an absolute error of the exponent;
      p          exponential of a difference of magnitude up to 2 reach + 1: 2^-24 of that, 2^-22 for ex2 itself;
      sums       over n keys in fp32: at most (n + 64) 2^-24 of the sum of magnitudes (o and l each);
      fp16 only  p rounded to fp16 before the product with v: 2^-11;
      output     one rounding: half a step of its type, and half the smallest subnormal of fp16."""
    s = (D + 4) * 2.0 ** -24 * reach + (2 * reach + 16) * 2.0 ** -23 + 2.0 ** -21
    e = 2 * s + 2 * (n_max + 64) * 2.0 ** -24 + (2.0 ** -11 if dtype == torch.float16 else 0.0)
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -24
    t_out = u * out.abs() + (e * (1 + u))[..., None] * spread + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    t_lse = s + (n_max + 64) * 2.0 ** -24 + lse.abs() * 2.0 ** -22 + 2.0 ** -22
    return t_out, t_lse


def pool(gen, P, ps, H, D, dtype, heads_first=False, fill=None):
    """A cache [P, ps, H, D] on the CPU, stored heads first if asked; random unless `fill` is given."""
    shape = (P, H, ps, D) if heads_first else (P, ps, H, D)
    c = torch.randn(shape, generator=gen).to(dtype) if fill is None else torch.full(shape, fill, dtype=dtype)
    return c.permute(0, 2, 1, 3) if heads_first else c


def paged_case(seed, lens, Hq, Hkv, D, ps, dtype, heads_first=False, poison=True, q_scale=2.0):
    """q, caches, table, lens of one attention call on the CPU.  With poison, everything behind a request's length --
    unused pages, the rest of its last page, unused table entries -- holds NaN or a page id far outside the pool."""
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    held = [ceil_div(max(n, 0), ps) for n in lens]
    P = sum(held) + 2
    order = torch.randperm(P, generator=gen)
    width = max(held + [1]) + 1
    table = torch.full((B, width), 2 ** 31 - 1 if poison else -1, dtype=torch.int32)
    k, v = (pool(gen, P, ps, Hkv, D, dtype, heads_first) for _ in range(2))
    used = torch.zeros(P, ps, dtype=torch.bool)
    o = 0
    for b, n in enumerate(lens):
        pages = order[o:o + held[b]]
        o += held[b]
        table[b, :held[b]] = pages.int()
        j = torch.arange(max(n, 0))
        used[pages[j // ps], j % ps] = True
    if poison:
        k[~used] = float("nan")
        v[~used] = float("nan")
    q = (torch.randn(B, Hq, D, generator=gen) * q_scale).to(dtype)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32)


def on_dev(t, dev):
    """A copy on the device that keeps the strides' order."""
    if t.dim() == 4 and not t.is_contiguous():
        return t.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3)
    return t.to(dev)
