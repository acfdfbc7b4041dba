"""GPU parity of the paged key-value cache's operators against their 64-bit definitions."""
import numpy as np
import pytest
import torch

from tests.paged_util import (attn_ref, attn_tolerance, ceil_div, on_dev, paged_case, pool, tables_ref, turn_ref)

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module")
def mnb(cuda_dev):
    import int4_block_quantized_matmulnbits_b200 as m

    return m


def _i32(x, dev):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(dev)


# ------------------------------------------------------------------- tables

def run_tables(mnb, dev, ctx, new, table, page, num_pages, free, start, T, extra=0):
    """The call's outputs as numpy arrays (table, seq, cu, slots, pos, next, status)."""
    B = len(ctx)
    d = dict(table=_i32(table, dev), seq=_i32([77] * B, dev), cu=_i32([77] * (B + 1), dev), slots=_i32([77] * T, dev),
             pos=_i32([77] * T, dev), next=_i32([77], dev), status=_i32([0], dev))
    mnb.mnb_paged_tables(_i32(ctx, dev), _i32(new, dev), d["table"], page, num_pages, _i32(free, dev),
                         _i32([start], dev), d["seq"], d["cu"], d["slots"], d["pos"], d["next"], d["status"])
    torch.cuda.synchronize()
    return [d[n].cpu().numpy() for n in ("table", "seq", "cu", "slots", "pos", "next", "status")]


def check_tables(mnb, dev, ctx, new, page, width, free, start, T, num_pages, table=None, status=0):
    B = len(ctx)
    rng = np.random.default_rng(B * 31 + T)
    if table is None:
        table = rng.integers(0, num_pages, (B, width)).astype(np.int32)
    got = run_tables(mnb, dev, ctx, new, table, page, num_pages, free, start, T)
    ref = tables_ref(ctx, new, table, page, num_pages, free, start, T)
    assert ref[6] == status
    for name, g, r in zip(("table", "seq", "cu", "slots", "pos", "next", "status"), got, ref):
        assert np.array_equal(np.asarray(g).reshape(-1), np.asarray(r).reshape(-1)), name


@pytest.mark.parametrize("B,page,max_ctx,max_new", [(1, 16, 0, 1), (1, 16, 390, 1), (64, 16, 4096, 1), (7, 1, 50, 9),
                                                    (33, 24, 700, 65), (513, 16, 200, 30), (4096, 8, 60, 3),
                                                    (5, 128, 1000, 2000)])
def test_tables(mnb, cuda_dev, B, page, max_ctx, max_new):
    rng = np.random.default_rng(B + page)
    ctx = rng.integers(0, max_ctx + 1, B).tolist()
    new = rng.integers(0, max_new + 1, B).tolist()
    width = ceil_div(max_ctx + max_new, page)
    need = sum(ceil_div(c + n, page) - ceil_div(c, page) for c, n in zip(ctx, new))
    P = 5 * B + need + 11
    free = rng.permutation(P)[:need + 9]
    for T in (sum(new), sum(new) + 37):   # exact, and padded
        check_tables(mnb, cuda_dev, ctx, new, page, width, free, 4, T, P)


def test_tables_free_list_runs_out(mnb, cuda_dev):
    # 3 pages free: the second request needs two more than are left, the third needs none, the fourth one
    ctx, new = [0, 16, 5, 16], [32, 33, 3, 1]
    check_tables(mnb, cuda_dev, ctx, new, 16, 8, np.arange(50, 55), 2, 69, 100, status=4)
    check_tables(mnb, cuda_dev, [3], [1], 16, 8, [], 0, 1, 10, status=0)    # an empty list that nobody needs
    check_tables(mnb, cuda_dev, [3], [1], 16, 8, [1, 2], 3, 1, 10, status=4)   # a start behind the list
    check_tables(mnb, cuda_dev, [0, 3], [1, 1], 16, 8, [1, 2], -1, 2, 10, status=4)


def test_tables_refuses_requests(mnb, cuda_dev):
    big = 2 ** 31 - 1
    check_tables(mnb, cuda_dev, [-1, 4, 120, 0], [2, -3, 9, 5], 16, 8, np.arange(20), 0, 16, 30, status=2)
    check_tables(mnb, cuda_dev, [big, 4, big, 0], [1, big, big, 2], 16, 8, np.arange(20), 0, 16, 30, status=2)
    check_tables(mnb, cuda_dev, [0, 0], [10, 10], 16, 8, np.arange(20), 0, 15, 30, status=2)   # T too small


def test_tables_page_ids_outside_the_pool(mnb, cuda_dev):
    table = np.array([[3, 999, 0, 0], [-5, 1, 0, 0]], np.int32)
    check_tables(mnb, cuda_dev, [17, 3], [20, 14], 16, 4, [2, 40, 1], 0, 34, 10, table=table, status=1)


def test_tables_no_requests(mnb, cuda_dev):
    check_tables(mnb, cuda_dev, [], [], 16, 3, [1, 2], 1, 5, 10)


# ------------------------------------------------------------------- append

def append_case(seed, T, Hq, H, D, R, ps, dtype, norm, heads_first, pad=0, top=500):
    gen = torch.Generator().manual_seed(seed)
    P = ceil_div(max(T, 1), ps) + 2
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=gen).to(dtype)
    slots = torch.randperm(P * ps, generator=gen)[:T].int()
    if pad:
        slots[T - pad:] = -1
    ang = torch.rand(top, R // 2, generator=gen, dtype=torch.float64) * 1e4
    c = dict(qkv=qkv, slots=slots, pos=torch.randint(0, top, (T,), generator=gen).int(),
             cos=ang.cos().float() if R else None, sin=ang.sin().float() if R else None,
             qw=1 + 0.2 * torch.randn(D, generator=gen) if norm else None,
             kw=1 + 0.2 * torch.randn(D, generator=gen) if norm else None,
             kc=pool(gen, P, ps, H, D, dtype, heads_first), vc=pool(gen, P, ps, H, D, dtype, heads_first))
    return c


def split_qkv(qkv, Hq, H, D):
    T = qkv.shape[0]
    q, k, v = qkv.split([Hq * D, H * D, H * D], 1)
    return q.view(T, Hq, D), k.view(T, H, D), v.view(T, H, D)


def turn_tolerance(x, w, ref, dtype, D):
    """Of the normed and rotated rows: the mean of squares (D + 2 roundings, halved by the root), root, quotient, the
    products with 1/rms and w, the rotation's two products and their sum: at most D/2 + 8 roundings of 2^-24 of the
    sum of the two products' magnitudes (at most sqrt(2) of the pair, here: the row's largest entry twice); then the
    output's rounding and half of fp16's smallest subnormal."""
    rowmax = ref.abs().amax(-1, keepdim=True) * 2 ** 0.5
    u = 2.0 ** -11 if dtype == F16 else 2.0 ** -24
    return u * ref.abs() + 2 * (D / 2 + 8) * 2.0 ** -24 * rowmax + (2.0 ** -25 if dtype == F16 else 0.0)


def check_append(mnb, dev, c, Hq, H, D, dtype, eps=1e-6, in_place=False, status=0):
    qkv = c["qkv"].to(dev)
    q, k, v = split_qkv(qkv, Hq, H, D)
    T = qkv.shape[0]
    kc, vc = on_dev(c["kc"], dev), on_dev(c["vc"], dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    q_out = q if in_place else torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    dv = {n: None if c[n] is None else c[n].to(dev) for n in ("slots", "pos", "cos", "sin", "qw", "kw")}
    mnb.mnb_rope_append(q, k, v, kc, vc, dv["slots"], dv["pos"], dv["cos"], dv["sin"], q_out, dv["qw"], dv["kw"], eps,
                        st)
    torch.cuda.synchronize()
    assert int(st) == status
    qr, kr, vr = split_qkv(c["qkv"], Hq, H, D)
    P, ps = c["kc"].shape[:2]
    top = c["cos"].shape[0] if c["cos"] is not None else 1
    pos_ok = torch.ones(T, dtype=torch.bool) if c["cos"] is None else (c["pos"] >= 0) & (c["pos"] < top)
    pos = c["pos"].clamp(0, top - 1)
    ref = turn_ref(qr, c["qw"], eps, c["cos"], c["sin"], pos)
    ref[~pos_ok] = 0
    d = (q_out.cpu().double() - ref).abs()
    assert bool((d <= turn_tolerance(qr, c["qw"], ref, dtype, D)).all()), float(d.max())
    keep = pos_ok & (c["slots"] >= 0) & (c["slots"] < P * ps)
    s = c["slots"][keep].long()
    kref, krow = c["kc"].double(), turn_ref(kr, c["kw"], eps, c["cos"], c["sin"], pos)[keep]
    touched = torch.zeros(P, ps, dtype=torch.bool)
    touched[s // ps, s % ps] = True
    d = (kc.cpu()[s // ps, s % ps].double() - krow).abs()
    assert bool((d <= turn_tolerance(kr, c["kw"], krow, dtype, D)).all()), float(d.max()) if d.numel() else 0
    assert torch.equal(kc.cpu()[~touched], c["kc"][~touched])       # every other row as it was
    vref = c["vc"].clone()
    vref[s // ps, s % ps] = vr[keep]
    assert torch.equal(vc.cpu(), vref)
    assert kref.shape == kc.shape


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("T,Hq,H,D,R,ps,norm,heads_first,pad", [
    (1, 16, 8, 128, 128, 16, True, False, 0),
    (37, 16, 8, 128, 128, 16, True, True, 5),
    (1001, 3, 1, 64, 32, 24, False, False, 100),
    (5, 2, 2, 80, 40, 1, True, True, 0),
    (9, 4, 2, 256, 256, 7, True, False, 9),
    (130, 6, 3, 8, 8, 16, True, False, 1),
    (64, 2, 2, 96, 0, 16, True, False, 0),
    (64, 8, 1, 200, 72, 32, False, True, 2),
])
def test_append(mnb, cuda_dev, T, Hq, H, D, R, ps, norm, heads_first, pad, dtype):
    c = append_case(T + D, T, Hq, H, D, R, ps, dtype, norm, heads_first, pad)
    check_append(mnb, cuda_dev, c, Hq, H, D, dtype)


def test_append_in_place_and_one_norm(mnb, cuda_dev):
    c = append_case(3, 21, 4, 2, 128, 64, 16, F16, True, False)
    c["qw"] = None
    check_append(mnb, cuda_dev, c, 4, 2, 128, F16, in_place=True)


def test_append_bad_slots_and_positions(mnb, cuda_dev):
    c = append_case(4, 40, 4, 2, 64, 64, 16, F16, True, False)
    c["slots"][3], c["slots"][7] = -2, 2 ** 31 - 1
    c["pos"][11], c["pos"][12] = -1, 500
    check_append(mnb, cuda_dev, c, 4, 2, 64, F16, status=1)


def test_append_keys_and_values_alone(mnb, cuda_dev):
    c = append_case(5, 33, 0, 2, 64, 0, 16, F32, False, True)
    _, k, v = split_qkv(c["qkv"].to(cuda_dev), 0, 2, 64)
    kc, vc = on_dev(c["kc"], cuda_dev), on_dev(c["vc"], cuda_dev)
    mnb.mnb_rope_append(None, k, v, kc, vc, c["slots"].to(cuda_dev), None, None, None, None)
    s = c["slots"].long()
    for got, was, rows in ((kc, c["kc"], k), (vc, c["vc"], v)):
        ref = was.clone()
        ref[s // 16, s % 16] = rows.cpu()
        assert torch.equal(got.cpu(), ref)


# ---------------------------------------------------------------- attention

@pytest.fixture(params=["by sizes", "1x4x1", "2x12x1", "5x3x1", "8x4x1", "3x2x5", "1x5x7", "8x12x2"])
def shape(mnb, request):
    """Each test with the launch shape that its sizes choose, and with others: CTAs of a cluster, warps, clusters."""
    given = [0, 0, 0] if request.param == "by sizes" else map(int, request.param.split("x"))
    assert mnb._lib.mnb_tune_paged_attention(*given) == 0
    yield request.param
    mnb._lib.mnb_tune_paged_attention(0, 0, 0)


def run_attn(mnb, dev, case, scale, ws=None, lse=True, status=None):
    q, k, v, table, lens = case
    out = torch.full_like(q, float("nan"), device=dev)
    ls = torch.full(q.shape[:2], float("nan"), device=dev) if lse else None
    if ws is None:
        ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(q.shape[0], q.shape[1], k.shape[2], q.shape[2],
                                                                 q.dtype), dtype=torch.uint8, device=dev)
    mnb.mnb_paged_attention(q.to(dev), on_dev(k, dev), on_dev(v, dev), table.to(dev), lens.to(dev), scale, out, ws, ls,
                            status)
    torch.cuda.synchronize()
    return out.cpu(), None if ls is None else ls.cpu()


def assert_attn(out, lse, case, scale):
    q, k, v, table, lens = case
    ref, rl, spread, reach = attn_ref(q, k, v, table, lens, scale)
    t_out, t_lse = attn_tolerance(ref, rl, spread, reach, q.dtype, max([1] + lens.tolist()), q.shape[2])
    assert bool(torch.isfinite(out.float()).all())
    d = (out.double() - ref).abs()
    assert bool((d <= t_out).all()), f"out off by {float((d - t_out).max()):.3g} more than allowed"
    if lse is not None:
        none = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), none) and bool((lse[none] < 0).all())
        d = (lse.double() - rl).abs()[~none]
        assert bool((d <= t_lse[~none]).all()), float(d.max())


CASES = [
    # lens, Hq, Hkv, D, page, heads_first
    ([1], 1, 1, 64, 16, False),
    ([0, 1, 2, 0], 4, 2, 128, 16, False),
    ([390], 16, 8, 128, 16, False),
    ([16, 17, 15, 64, 63, 65, 33], 16, 8, 128, 16, False),
    ([5, 1000, 0, 77, 1], 4, 4, 64, 24, True),
    ([100, 41], 6, 2, 80, 1, False),
    ([255, 3], 12, 4, 96, 7, True),
    ([300, 129, 0], 8, 1, 256, 32, False),
    ([700, 1], 32, 2, 256, 64, True),
    ([211, 90], 17, 1, 128, 16, False),      # 17 query heads on one KV head
    ([211, 90], 40, 1, 64, 16, False),
    ([50], 3, 3, 8, 16, False),
    ([4096], 2, 1, 128, 128, False),
    ([9000], 8, 8, 64, 16, False),           # cut over all SMs
    ([9000, 1, 0, 4500], 5, 1, 40, 16, True),
    (list(range(0, 300)), 2, 2, 64, 16, False),
    ([333, 17, 250], 6, 2, 200, 16, True),
    ([333, 17, 250], 3, 1, 72, 48, False),
    ([100, 9], 10, 1, 24, 5, False),
    ([257, 300, 128] * 8, 32, 2, 256, 16, False),   # the largest partial results, in clusters
    ([64] * 97, 4, 2, 128, 16, False),
]


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(mnb, cuda_dev, shape, i, dtype):
    lens, Hq, H, D, ps, heads_first = CASES[i]
    case = paged_case(i, lens, Hq, H, D, ps, dtype, heads_first)
    scale = D ** -0.5
    out, lse = run_attn(mnb, cuda_dev, case, scale)
    assert_attn(out, lse, case, scale)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_attention_many_requests(mnb, cuda_dev, shape, dtype):
    rng = np.random.default_rng(5)
    case = paged_case(9, rng.integers(0, 9, 4096).tolist(), 2, 1, 64, 4, dtype)
    out, lse = run_attn(mnb, cuda_dev, case, 0.125)
    assert_attn(out, lse, case, 0.125)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("scale,q_scale", [(0.0, 1.0), (-0.1, 2.0), (1.0, 8.0), (0.088, 100.0)])
def test_attention_scales(mnb, cuda_dev, shape, scale, q_scale, dtype):
    """No scale at all (the mean of v), a negative one, and scores of hundreds (one key holds nearly all)."""
    case = paged_case(11, [500, 33, 1], 4, 2, 128, 16, dtype, q_scale=q_scale)
    out, lse = run_attn(mnb, cuda_dev, case, scale)
    assert_attn(out, lse, case, scale)


def test_attention_small_probabilities_count(mnb, cuda_dev, shape):
    """One key of weight 1 and 20000 of weight 2^-20: together 2^-6 of the sum, none lost to fp16's range."""
    n, D = 20001, 64
    q, k, v, table, lens = paged_case(12, [n], 1, 1, D, 16, F16)
    q.zero_()
    q[0, 0, 0] = 1.0
    j = torch.arange(n)
    page, off = table[0, j // 16].long(), j % 16
    k[page, off] = 0
    v[page, off] = 1.0
    k[page[777], off[777], 0, 0] = 20 * np.log(2.0)
    v[page[777], off[777]] = 0.0
    case = (q, k, v, table, lens)
    out, lse = run_attn(mnb, cuda_dev, case, 1.0)
    assert_attn(out, lse, case, 1.0)
    assert abs(float(out[0, 0, 0]) - 20000 / (20000 + 2.0 ** 20)) < 2e-4


def test_attention_bad_pages_and_lengths(mnb, cuda_dev, shape):
    case = paged_case(13, [100, 64, 40, 16], 4, 2, 64, 16, F16)
    q, k, v, table, lens = case
    table[0, 1], table[1, 0], table[3, 0] = -1, 10 ** 9, k.shape[0]     # a request without any page left, too
    st = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out, lse = run_attn(mnb, cuda_dev, case, 0.1, status=st)
    assert_attn(out, lse, case, 0.1)
    assert int(st) == 1 and float(lse[3].max()) == float("-inf") and bool((out[3] == 0).all())
    case = paged_case(14, [100, 64], 4, 2, 64, 16, F16)
    q, k, v, table, lens = case
    table[table == 2 ** 31 - 1] = 0
    width = table.shape[1] * 16
    k[torch.isnan(k)], v[torch.isnan(v)] = 0.5, 0.25
    st.zero_()
    bad = torch.tensor([2 ** 31 - 1, -7], dtype=torch.int32)
    out, lse = run_attn(mnb, cuda_dev, (q, k, v, table, bad), 0.1, status=st)
    assert_attn(out, lse, (q, k, v, table, torch.tensor([width, 0], dtype=torch.int32)), 0.1)
    assert int(st) == 2


def test_attention_without_lse_and_strided_views(mnb, cuda_dev, shape):
    """q inside a fused product, out inside a wider buffer that stays as it is around it."""
    case = paged_case(15, [100, 257, 3], 4, 2, 128, 16, F16)
    q, k, v, table, lens = case
    wide_q = torch.randn(3, 8, 128).to(F16).to(cuda_dev)
    wide_q[:, 2:6] = q.to(cuda_dev)
    wide_o = torch.full((3, 6, 136), 7.0, dtype=F16, device=cuda_dev)
    tab = torch.zeros(3, table.shape[1] + 5, dtype=torch.int32, device=cuda_dev)
    tab[:, :table.shape[1]] = table.to(cuda_dev)
    ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(3, 4, 2, 128), dtype=torch.uint8, device=cuda_dev)
    mnb.mnb_paged_attention(wide_q[:, 2:6], on_dev(k, cuda_dev), on_dev(v, cuda_dev), tab[:, :table.shape[1]],
                            lens.to(cuda_dev), 0.09, wide_o[:, 1:5, :128], ws)
    o = wide_o.cpu()
    assert_attn(o[:, 1:5, :128], None, case, 0.09)
    assert bool((o[:, 0] == 7).all() and (o[:, 5] == 7).all() and (o[:, :, 128:] == 7).all())


def test_attention_one_workspace_for_all_and_same_bits(mnb, cuda_dev):
    """One workspace, calls of other sizes, types and layouts between two equal ones: equal bits, counters zero."""
    ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(1, 32, 2, 256), dtype=torch.uint8, device=cuda_dev)
    first = None
    for rep in range(2):
        for i in (13, 8, 15, 3, 14):
            lens, Hq, H, D, ps, hf = CASES[i]
            for dtype in (F16, F32):
                case = paged_case(i, lens, Hq, H, D, ps, dtype, hf)
                out, lse = run_attn(mnb, cuda_dev, case, D ** -0.5, ws)
                assert_attn(out, lse, case, D ** -0.5)
                if i == 13 and dtype == F16:
                    if first is None:
                        first = (out, lse)
                    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert int(ws[:1024].sum()) == 0


def test_attention_on_two_streams_at_once(mnb, cuda_dev):
    """Calls that overlap on two streams, a workspace each: the bits of the same calls one after the other."""
    mnb._lib.mnb_tune_paged_attention(4, 4, 3)      # groups, so that the workspaces are used
    try:
        cases = [paged_case(20 + i, [n, 300], 8, 2, 128, 16, F16) for i, n in enumerate((4000, 2500))]
        want = [run_attn(mnb, cuda_dev, c, 0.1) for c in cases]
        dev = [[on_dev(t, cuda_dev) for t in c] for c in cases]
        ws = [torch.zeros(mnb.mnb_paged_attention_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device=cuda_dev)
              for _ in cases]
        streams = [torch.cuda.Stream() for _ in cases]
        outs = [[torch.empty(2, 8, 128, dtype=F16, device=cuda_dev) for _ in range(30)] for _ in cases]
        torch.cuda.synchronize()
        for r in range(30):
            for (q, k, v, table, lens), w, s, o in zip(dev, ws, streams, outs):
                mnb.mnb_paged_attention(q, k, v, table, lens, 0.1, o[r], w, stream=s)
        torch.cuda.synchronize()
        for (ref, _), o in zip(want, outs):
            assert all(torch.equal(x.cpu(), ref) for x in o)
    finally:
        mnb._lib.mnb_tune_paged_attention(0, 0, 0)


def test_attention_offsets_beyond_32_bits(mnb, cuda_dev, shape):
    """Pages more than 2^31 elements into the pool."""
    ps, H, D = 16, 8, 128
    P = (2 ** 31) // (ps * H * D) + 40
    kv = torch.empty(P, ps, H, D, dtype=F16, device=cuda_dev)
    case = paged_case(16, [150, 40], 16, H, D, ps, F16, poison=False)
    q, k, v, table, lens = case
    far = P - 1 - torch.arange(k.shape[0])       # the small pool's pages, at the far end
    kv[far.to(cuda_dev)] = k.to(cuda_dev)
    table = torch.where(table >= 0, P - 1 - table, table)
    out = torch.empty(q.shape, dtype=F16, device=cuda_dev)
    ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(2, 16, H, D), dtype=torch.uint8, device=cuda_dev)
    mnb.mnb_paged_attention(q.to(cuda_dev), kv, kv, table.to(cuda_dev), lens.to(cuda_dev), 0.088, out, ws)
    assert_attn(out.cpu(), None, (q, k, k, P - 1 - table, lens), 0.088)
    # and a row written there
    x = torch.randn(2, H, D).to(F16).to(cuda_dev)
    slots = torch.tensor([P * ps - 1, (P - 2) * ps], dtype=torch.int32, device=cuda_dev)
    mnb.mnb_rope_append(None, x, x, kv, kv, slots, None, None, None, None)
    assert torch.equal(kv[P - 1, ps - 1], x[0]) and torch.equal(kv[P - 2, 0], x[1])


# ------------------------------------------------------------ all three together

def decode_setup(dev, B, Hq, H, D, ps, dtype, steps, prompt):
    P = sum(ceil_div(n + steps, ps) for n in prompt) + 3
    gen = torch.Generator().manual_seed(B)
    top = max(prompt) + steps + 1
    ang = torch.arange(top, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    width = ceil_div(max(prompt) + steps, ps)
    st = dict(free=torch.randperm(P, generator=gen).int().to(dev), start=_i32([0], dev), next=_i32([0], dev),
              table=torch.full((B, width), -1, dtype=torch.int32, device=dev), ctx=_i32([0] * B, dev),
              seq=_i32([0] * B, dev), cu=_i32([0] * (B + 1), dev), cos=ang.cos().float().to(dev),
              sin=ang.sin().float().to(dev), qw=(1 + 0.1 * torch.randn(D, generator=gen)).to(dev),
              kw=(1 + 0.1 * torch.randn(D, generator=gen)).to(dev), status=_i32([0], dev), P=P,
              kc=torch.full((P, ps, H, D), float("nan"), dtype=dtype, device=dev),
              vc=torch.full((P, ps, H, D), float("nan"), dtype=dtype, device=dev))
    return st, gen


@pytest.mark.parametrize("dtype", [F16, F32])
def test_prompt_and_decode_steps(mnb, cuda_dev, dtype):
    """Prompts, then steps of one token per request: tables, append and attention fed by one another, against the
    attention over all rows so far computed from scratch in 64 bits (over the rows that the cache holds)."""
    B, Hq, H, D, ps, steps = 5, 4, 2, 64, 16, 20
    prompt = [31, 16, 1, 90, 47]
    st, gen = decode_setup(cuda_dev, B, Hq, H, D, ps, dtype, steps, prompt)
    ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(B, Hq, H, D, dtype), dtype=torch.uint8, device=cuda_dev)
    ks, vs = [[] for _ in range(B)], [[] for _ in range(B)]
    for step in range(steps):
        new = prompt if step == 0 else [1] * B
        T = sum(new)
        qkv = torch.randn(T, (Hq + 2 * H) * D, generator=gen).to(dtype)
        q, k, v = split_qkv(qkv.to(cuda_dev), Hq, H, D)
        slots, pos = torch.empty(T, dtype=torch.int32, device=cuda_dev), torch.empty(T, dtype=torch.int32, device=cuda_dev)
        q_out = torch.empty(T, Hq, D, dtype=dtype, device=cuda_dev)
        mnb.mnb_paged_tables(st["ctx"], _i32(new, cuda_dev), st["table"], ps, st["P"], st["free"], st["start"],
                             st["seq"], st["cu"], slots, pos, st["next"], st["status"], mnb.MNB_FLAG_PDL)
        mnb.mnb_rope_append(q, k, v, st["kc"], st["vc"], slots, pos, st["cos"], st["sin"], q_out, st["qw"], st["kw"],
                            1e-6, st["status"], mnb.MNB_FLAG_PDL)
        last = st["cu"][1:].long() - 1          # each request's newest token
        ql = q_out[last].contiguous()
        out, lse = torch.empty(B, Hq, D, dtype=dtype, device=cuda_dev), torch.empty(B, Hq, device=cuda_dev)
        mnb.mnb_paged_attention(ql, st["kc"], st["vc"], st["table"], st["seq"], D ** -0.5, out, ws, lse, st["status"],
                                mnb.MNB_FLAG_PDL)
        st["start"], st["next"], st["ctx"], st["seq"] = st["next"], st["start"], st["seq"], st["ctx"]
        torch.cuda.synchronize()
        # the rows that should be in the cache
        kr = turn_ref(split_qkv(qkv, Hq, H, D)[1], st["kw"].cpu(), 1e-6, st["cos"].cpu(), st["sin"].cpu(), pos.cpu())
        o = 0
        for b in range(B):
            ks[b].append(kr[o:o + new[b]].to(dtype))
            vs[b].append(split_qkv(qkv, Hq, H, D)[2][o:o + new[b]])
            o += new[b]
        lens = [sum(len(x) for x in ks[b]) for b in range(B)]
        assert st["ctx"].cpu().tolist() == lens and int(st["status"]) == 0
        width = ceil_div(max(lens), ps)
        kd, vd = torch.zeros(B * width, ps, H, D, dtype=dtype), torch.zeros(B * width, ps, H, D, dtype=dtype)
        for b in range(B):
            kd[b * width:(b + 1) * width].view(-1, H, D)[:lens[b]] = torch.cat(ks[b])
            vd[b * width:(b + 1) * width].view(-1, H, D)[:lens[b]] = torch.cat(vs[b])
        tab = torch.arange(B * width, dtype=torch.int32).view(B, width)
        # the cached keys are half a step of their type from the reference's keys before rounding, which are then
        # rounded too: at most one step apart, |ds| <= 2u reach and as much again in p
        ref, rl, spread, reach = attn_ref(ql.cpu(), kd, vd, tab, lens, D ** -0.5)
        t_out, t_lse = attn_tolerance(ref, rl, spread, reach, dtype, max(lens), D)
        u = 2.0 ** -11 if dtype == F16 else 2.0 ** -24
        more = 2 * u * reach + (D / 2 + 8) * 2.0 ** -22 * reach
        assert bool(((out.cpu().double() - ref).abs() <= t_out + 2 * more[..., None] * spread).all())
        assert bool(((lse.cpu().double() - rl).abs() <= t_lse + more).all())


def test_captured_step_follows_its_lengths(mnb, cuda_dev):
    """The three launches captured once and replayed on another stream: lengths, tables and slots move on the device."""
    B, Hq, H, D, ps, steps = 3, 4, 2, 128, 16, 40
    st, gen = decode_setup(cuda_dev, B, Hq, H, D, ps, F16, steps, [20, 1, 33])
    for n in ("kc", "vc"):
        st[n].copy_(torch.randn(st[n].shape, generator=gen).to(F16))
    one = _i32([1] * B, cuda_dev)
    slots, pos = _i32([0] * B, cuda_dev), _i32([0] * B, cuda_dev)
    qkv = torch.zeros(B, (Hq + 2 * H) * D, dtype=F16, device=cuda_dev)
    q, k, v = split_qkv(qkv, Hq, H, D)
    q_out, out = torch.empty(B, Hq, D, dtype=F16, device=cuda_dev), torch.empty(B, Hq, D, dtype=F16, device=cuda_dev)
    ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(B, Hq, H, D), dtype=torch.uint8, device=cuda_dev)

    def step(flags=0):
        mnb.mnb_paged_tables(st["ctx"], one, st["table"], ps, st["P"], st["free"], st["start"], st["seq"], st["cu"],
                             slots, pos, st["next"], st["status"], flags)
        mnb.mnb_rope_append(q, k, v, st["kc"], st["vc"], slots, pos, st["cos"], st["sin"], q_out, st["qw"], st["kw"],
                            1e-6, st["status"], flags)
        mnb.mnb_paged_attention(q_out, st["kc"], st["vc"], st["table"], st["seq"], 0.09, out, ws, None, st["status"],
                                flags)

    def reset():
        st["ctx"].zero_(), st["start"].zero_(), st["table"].fill_(-1)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(mnb.MNB_FLAG_PDL)
        st["ctx"].copy_(st["seq"])
        st["start"].copy_(st["next"])
    inputs = [torch.randn(qkv.shape, generator=gen).to(F16).to(cuda_dev) for _ in range(steps)]
    results = []
    for captured in (True, False):
        reset()
        outs = []
        for x in inputs:
            qkv.copy_(x)
            if captured:
                g.replay()
            else:
                step()
                st["ctx"].copy_(st["seq"])
                st["start"].copy_(st["next"])
            outs.append(out.clone())
        results.append(torch.stack(outs))
        assert st["ctx"].cpu().tolist() == [steps] * B
    torch.cuda.synchronize()
    assert int(st["status"]) == 0
    assert torch.equal(results[0], results[1])
    lens = st["seq"].cpu()
    case = (q_out.cpu(), st["kc"].cpu(), st["vc"].cpu(), st["table"].cpu(), lens)
    assert_attn(out.cpu(), None, case, 0.09)


@pytest.mark.parametrize("fused,kind,dtype", [(True, "gemv", F16), (False, "gemv", F16), (False, "matmul", F32)])
def test_pass_with_attention(mnb, cuda_dev, fused, kind, dtype):
    """step.Pass with a PagedCache: two layers, three requests, prompts and then captured steps.  Each step's o inputs
    against the 64-bit attention over all q, k and v that the projections have put out so far."""
    from int4_block_quantized_matmulnbits_b200 import step

    M, hidden, Hq, H, D, ps, layers, steps = 3, 256, 4, 2, 64, 16, 2, 20
    gen = torch.Generator().manual_seed(7)
    sdt = F16 if dtype == F16 else F32
    lin = []
    for layer in range(layers):
        for name, N, K in (("q", Hq * D, hidden), ("k", H * D, hidden), ("v", H * D, hidden), ("o", hidden, Hq * D)):
            W = (torch.randn(N, K, generator=gen) * 0.06).to(cuda_dev)
            lin.append(step.QLinear.quantize(W, 32, True, sdt, name=f"{name}{layer}"))
        if fused:
            lin[-4:] = [step.concat_linears(lin[-4:-1], f"qkv{layer}"), lin[-1]]
    prompt = [5, 33, 16]
    ang = torch.rand(64, D // 2, generator=gen, dtype=torch.float64) * 100
    cos, sin = ang.cos().float().to(cuda_dev), ang.sin().float().to(cuda_dev)
    norms = [tuple((1 + 0.2 * torch.randn(D, generator=gen)).to(cuda_dev) for _ in range(2)) for _ in range(layers)]
    cache = step.PagedCache(layers, M, Hq, H, D, 64, ps, dtype=dtype, cos=cos, sin=sin, norms=norms)
    p = step.Pass(lin, M, kind, dtype, attention=cache)
    assert p.launches == len(lin) + 1 + 2 * layers
    x = torch.randn(p.x_flat.shape, generator=gen).to(dtype)
    p.x_flat.copy_(x)
    p.capture()
    assert cache.lens.cpu().tolist() == [0] * M and int(cache.start) == 0   # its warm-up left no token behind
    # the prompts
    T = sum(prompt)
    slots, pos = torch.empty(T, dtype=torch.int32, device=cuda_dev), torch.empty(T, dtype=torch.int32, device=cuda_dev)
    cache.begin(_i32(prompt, cuda_dev), slots, pos)
    ks, vs = [], []                   # per layer, per request: the rows of the cache so far
    for layer in range(layers):
        qkv = torch.randn(T, (Hq + 2 * H) * D, generator=gen).to(dtype)
        q, k, v = split_qkv(qkv.to(cuda_dev), Hq, H, D)
        cache.append(layer, q, k, v, torch.empty_like(q, memory_format=torch.contiguous_format), slots, pos)
        kr = turn_ref(k.cpu(), norms[layer][1].cpu(), 1e-6, cos.cpu(), sin.cpu(), pos.cpu()).to(dtype)
        ks.append(list(kr.split(prompt))), vs.append(list(v.cpu().split(prompt)))
    cache.end()
    for i in range(steps):
        x = torch.randn(p.x_flat.shape, generator=gen).to(dtype)
        p.x_flat.copy_(x)
        p.replay()
        torch.cuda.synchronize()
        cache.check()
        at = torch.tensor([n + i for n in prompt])
        assert cache.lens.cpu().tolist() == (at + 1).tolist()
        for last, (layer, q, k, v, out) in p.layers.items():
            kr = turn_ref(k.cpu(), norms[layer][1].cpu(), 1e-6, cos.cpu(), sin.cpu(), at).to(dtype)
            qr = turn_ref(q.cpu(), norms[layer][0].cpu(), 1e-6, cos.cpu(), sin.cpu(), at).to(dtype)
            for b in range(M):
                ks[layer][b] = torch.cat([ks[layer][b], kr[b:b + 1]])
                vs[layer][b] = torch.cat([vs[layer][b], v[b:b + 1].cpu()])
            width = ceil_div(max(prompt) + i + 1, ps)
            kd, vd = torch.zeros(M * width, ps, H, D, dtype=dtype), torch.zeros(M * width, ps, H, D, dtype=dtype)
            for b in range(M):
                kd[b * width:(b + 1) * width].view(-1, H, D)[:at[b] + 1] = ks[layer][b]
                vd[b * width:(b + 1) * width].view(-1, H, D)[:at[b] + 1] = vs[layer][b]
            tab = torch.arange(M * width, dtype=torch.int32).view(M, width)
            ref, rl, spread, reach = attn_ref(qr, kd, vd, tab, at + 1, D ** -0.5)
            t_out, _ = attn_tolerance(ref, rl, spread, reach, dtype, int(at.max()) + 1, D)
            # q and k each within a step (2 u) of the reference's rounding: |ds| <= 4 u reach, as much again in p
            u = 2.0 ** -11 if dtype == F16 else 2.0 ** -24
            more = 4 * u * reach + 2 * (D / 2 + 8) * 2.0 ** -22 * reach
            assert bool(((out.cpu().double() - ref).abs() <= t_out + 2 * more[..., None] * spread).all())


def test_cache_steps_on_a_stream_by_its_handle(mnb, cuda_dev):
    """begin, layer and end on a side stream given as a Stream and as its handle: the lengths advance there."""
    from int4_block_quantized_matmulnbits_b200 import step

    cache = step.PagedCache(1, 2, 2, 1, 64, 64)
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, h, 64, generator=gen).to(F16).to(cuda_dev) for h in (2, 1, 1))
    out = torch.empty(2, 2, 64, dtype=F16, device=cuda_dev)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        st = s if i % 2 else s.cuda_stream
        cache.begin(stream=st)
        cache.layer(0, q, k, v, out, stream=st)
        cache.end(st)
    torch.cuda.synchronize()
    cache.check()
    assert cache.lens.cpu().tolist() == [20, 20]
    # equal keys: every probability 1/20, the output is v
    assert float((out.float() - v.float()).abs().max()) <= 2.0 ** -10 * float(v.abs().max())


def test_cache_that_is_full_says_so(mnb, cuda_dev):
    from int4_block_quantized_matmulnbits_b200 import step

    cache = step.PagedCache(1, 2, 2, 1, 64, max_len=32, page_size=16, pages=3)
    x = torch.zeros(2, 2, 64, dtype=F16, device=cuda_dev)
    out = torch.empty_like(x)
    for i in range(18):
        cache.begin()
        cache.layer(0, x, x[:, :1], x[:, :1], out)
        cache.end()
    # the fourth page is missing: the second request stands still at 16 tokens, the first goes on
    assert cache.lens.cpu().tolist() == [18, 16]
    with pytest.raises(RuntimeError, match="status 4"):
        cache.check()
    cache.check()
