"""Paged attention where its values are delicate: outputs that cancel, and NaN or infinities in live rows."""
import pytest
import torch

from tests.paged_util import attn_ref, attn_tolerance, paged_case
from tests.test_gpu_paged import F16, F32, mnb, run_attn  # noqa: F401  (mnb: a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["by sizes", "1x4x1", "8x4x1", "3x2x5"])
def shape(mnb, request):  # noqa: F811
    """The launch shape that the sizes choose, and others: CTAs of a cluster, warps, clusters."""
    given = [0, 0, 0] if request.param == "by sizes" else map(int, request.param.split("x"))
    assert mnb._lib.mnb_tune_paged_attention(*given) == 0
    yield request.param
    mnb._lib.mnb_tune_paged_attention(0, 0, 0)


def two_keys(n, at, G, D, ps, seed, dtype):
    """G query heads on one KV head, q_i = a_i e_0, and n keys of which two count: scores 0 and -a_i, all others below
    -6000 (weight 0 exactly).  Their values are c and -c e^a for columns of heads' own a: the output of head i is nearly
    nothing in the columns d % G == i, so what its probabilities lose shows there."""
    gen = torch.Generator().manual_seed(seed)
    q, k, v, table, lens = paged_case(seed, [n], G, 1, D, ps, dtype)
    a = (0.1 + 3.5 * torch.rand(G, generator=gen)).to(dtype)
    q.zero_()
    q[0, :, 0] = a
    j = torch.arange(n)
    page, off = table[0, j // ps].long(), j % ps
    k[page, off, 0, 0] = -60000.0
    c = 0.05 * (1 + torch.rand(D, generator=gen, dtype=torch.float64))
    for key, score, val in ((at[0], 0.0, c), (at[1], -1.0, -c * torch.exp(a.double()).repeat(D // G))):
        k[page[key], off[key], 0, 0] = score
        v[page[key], off[key], 0] = val.to(dtype)
    return (q, k, v, table, lens), a


@pytest.mark.parametrize("n,at", [(2, (0, 1)), (2, (1, 0)), (16, (3, 12)), (500, (130, 131)), (500, (0, 499)),
                                  (9000, (4100, 4107))])
@pytest.mark.parametrize("G,D", [(1, 64), (2, 128), (4, 80), (8, 128), (8, 256), (16, 64)])
def test_fp16_probabilities_keep_fp32s_bits(mnb, cuda_dev, shape, G, D, n, at):  # noqa: F811
    check_two_keys(mnb, cuda_dev, n, at, G, D, F16)


@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (8, 256)])
def test_fp32_probabilities_of_a_long_request(mnb, cuda_dev, shape, G, D):  # noqa: F811
    """However long the request, keys without weight add zeros exactly: the bound does not grow with it."""
    check_two_keys(mnb, cuda_dev, 9000, (4100, 4107), G, D, F32)


def check_two_keys(mnb, cuda_dev, n, at, G, D, dtype):  # noqa: F811
    """|out - ref| from the arithmetic: the scores' products and sums are exact (one product is not zero); scaling by
    log2 e, the product and the difference to the maximum: three roundings of at most a log2 e + 16; 2^-22 for the
    exponential; a probability as two fp16 numbers: 2^-21 of it; at most 16 sums of terms that are not zero at 2^-23 each;
    the quotient 2^-23.  All of it times the sum of magnitudes: (3 (1.45 a + 16) 2^-24 + 2^-22 + 2^-21 + 17 2^-23) of it,
    below (1.1 a + 24) 2^-22.  Then the output's own rounding."""
    (q, k, v, table, lens), a = two_keys(n, at, G, D, 16, n + D, dtype)
    case = (q, k, v, table, lens)
    out, lse = run_attn(mnb, cuda_dev, case, 1.0)
    ref, rl, spread, _ = attn_ref(*case, 1.0)
    u, least = (2.0 ** -11, 2.0 ** -25) if dtype == F16 else (2.0 ** -24, 0.0)
    bound = u * ref.abs() + ((1.1 * a.double() + 24) * 2.0 ** -22)[None, :, None] * spread + least
    d = (out.double() - ref).abs()
    assert bool((d <= bound).all()), f"off by {float((d / spread).max()):.3g} of the sum of magnitudes"
    assert float((lse.double() - rl).abs().max()) <= 5 * 2.0 ** -22 * 4


# lens, Hq, Hkv, D, page, request and key that are spoilt
SPOILT = [([1], 2, 1, 64, 16, 0, 0), ([40, 390], 4, 2, 128, 16, 1, 0), ([40, 390], 4, 2, 128, 16, 1, 389),
          ([300, 7], 16, 2, 80, 24, 0, 150), ([2500], 6, 1, 256, 32, 0, 1111)]


def spoil(i, dtype, what, value):
    """A case with `value` in one entry of one live row, and the (request, query head, column) places it reaches."""
    lens, Hq, H, D, ps, b, key = SPOILT[i]
    q, k, v, table, n = paged_case(i, lens, Hq, H, D, ps, dtype)
    h, e, G = H - 1, D // 2 + 1, Hq // H
    hit = torch.zeros(q.shape, dtype=torch.bool)
    if what == "query":
        q[b, h * G, e] = value
        hit[b, h * G] = True
    else:
        cache = k if what == "key" else v
        cache[table[b, key // ps].long(), key % ps, h, e] = value
        if what == "key":
            hit[b, h * G:(h + 1) * G] = True
        else:
            hit[b, h * G:(h + 1) * G, e] = True
    return (q, k, v, table, n), hit


def clean(case):
    """The same case with the spoilt entries 0: places that they do not reach have these results."""
    q, k, v, table, n = [t.clone() for t in case]
    live = torch.zeros(k.shape[:2], dtype=torch.bool)
    for r in range(len(n)):
        j = torch.arange(int(n[r]))
        live[table[r, j // k.shape[1]].long(), j % k.shape[1]] = True
    for t in (k, v):
        rows = t[live]
        rows[~torch.isfinite(rows)] = 0
        t[live] = rows
    q[~torch.isfinite(q)] = 0
    return q, k, v, table, n


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("i", range(len(SPOILT)))
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_nan_in_a_live_row_is_seen(mnb, cuda_dev, shape, what, i, dtype):  # noqa: F811
    """A NaN among a head's scores makes its output NaN, one among its values the output's column; the rest is, bit for
    bit, what it is without.  (Heads that share a KV head decide together when their maxima move: beside a query of NaN
    the others are within their rounding errors, twice, of what they were.)"""
    case, hit = spoil(i, dtype, what, float("nan"))
    out, lse = run_attn(mnb, cuda_dev, case, 0.1)
    without = clean(case)
    want, wl = run_attn(mnb, cuda_dev, without, 0.1)
    gone = hit.all(-1)
    assert torch.equal(torch.isnan(out), hit)
    if what != "query":
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~gone], wl[~gone])
    else:
        q, lens = without[0], without[4].tolist()
        t_out, t_lse = attn_tolerance(*attn_ref(*without, 0.1), dtype, max(lens), q.shape[2])
        assert bool(((out - want).abs().double() <= 2 * t_out)[~hit].all())
        assert bool(((lse - wl).abs().double() <= 2 * t_lse)[~gone].all())


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("i", range(len(SPOILT)))
@pytest.mark.parametrize("what,value", [("query", float("nan")), ("key", float("nan")), ("key", float("inf"))])
def test_lse_of_scores_without_a_sum(mnb, cuda_dev, shape, what, value, i, dtype):  # noqa: F811
    """Where a score is NaN or +inf there is no sum of exponentials: lse and out are NaN, not the -inf and zeros of a
    request without keys."""
    case, hit = spoil(i, dtype, what, value)
    case[0][..., case[0].shape[2] // 2 + 1].abs_().add_(1.0)     # times infinity: +inf
    out, lse = run_attn(mnb, cuda_dev, case, 0.1)
    assert torch.equal(torch.isnan(lse), hit.all(-1)) and torch.equal(torch.isnan(out), hit)
    assert bool(torch.isfinite(lse[~hit.all(-1)]).all())


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("i", range(len(SPOILT)))
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_value_in_a_live_row(mnb, cuda_dev, shape, value, i, dtype):
    """p times infinity, p > 0, is infinite: the output's column has it, no other place is touched."""
    case, hit = spoil(i, dtype, "value", value)
    case[0].mul_(0.25)   # no weight near 0
    out, lse = run_attn(mnb, cuda_dev, case, 0.1)
    want, wl = run_attn(mnb, cuda_dev, clean(case), 0.1)
    assert bool((out[hit].float() == value).all())
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, wl)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_scores_of_minus_infinity_have_no_weight(mnb, cuda_dev, shape, dtype):
    """Keys whose score is -inf count as if they were not there; a request that has no other is an empty one."""
    lens, D, ps = [70, 33], 64, 16
    q, k, v, table, n = paged_case(3, lens, 2, 1, D, ps, dtype)
    q[..., 0] = 1.0
    for b, keys in ((0, range(0, 64)), (1, range(33))):
        for j in keys:
            k[table[b, j // ps].long(), j % ps, 0, 0] = float("-inf")
    out, lse = run_attn(mnb, cuda_dev, (q, k, v, table, n), 0.1)
    pages = table[0, torch.arange(64, 70) // ps].long()
    s = torch.einsum("hd,nd->hn", q[0].double(), k[pages, torch.arange(64, 70) % ps, 0].double()) * 0.1
    p = torch.softmax(s, -1) @ v[pages, torch.arange(64, 70) % ps, 0].double()
    # six keys: 2^-11 for the output's rounding in fp16, and far below 2^-15 for the rest in fp32
    assert float((out[0].double() - p).abs().max()) <= (2.0 ** -10 if dtype == F16 else 2.0 ** -15) * float(v[torch.isfinite(v)].abs().max())
    assert float((lse[0].double() - torch.logsumexp(s, -1)).abs().max()) <= 2.0 ** -15
    assert bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())
