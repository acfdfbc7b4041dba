"""step.PagedCache at the end of its room and on other streams than the current one."""
import pytest
import torch

from int4_block_quantized_matmulnbits_b200 import step
from tests.paged_util import attn_ref

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.mark.parametrize("rotate", [True, False])
def test_cache_whose_max_len_is_inside_a_page(cuda_dev, rotate):
    """Room for 30 tokens in pages of 16: 30 steps are granted and attended over, captured ones among them; the next is
    refused as a length without room and leaves the request and its rows as they are."""
    gen = torch.Generator().manual_seed(30)
    ang = torch.rand(30, 32, generator=gen) * 6
    c = step.PagedCache(1, 1, 2, 1, 64, max_len=30, page_size=16, device=cuda_dev,
                        **(dict(cos=ang.cos().to(cuda_dev), sin=ang.sin().to(cuda_dev)) if rotate else {}))
    q, k, v = (torch.empty(1, h, 64, dtype=F16, device=cuda_dev) for h in (2, 1, 1))
    out = torch.empty(1, 2, 64, dtype=F16, device=cuda_dev)

    def one():
        c.begin()
        c.layer(0, q, k, v, out)
        c.end()

    def check_out(n):
        assert c.lens.tolist() == [n]
        ref, _, spread, _ = attn_ref(c.q.cpu(), c.k[0].cpu(), c.v[0].cpu(), c.table.cpu(), [n], c.scale)
        # 2^-11 for the output; 2^-15 of the magnitudes is far more than 30 keys' fp32 sums can lose
        assert bool(((out.cpu().double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -15 * spread + 2.0 ** -25).all())

    g = None
    for i in range(30):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        if i < 10:
            one()
            continue
        if g is None:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
        g.replay()
    c.check()
    check_out(30)
    rows = c.k[0].clone()
    for again in (g.replay, one):
        again()
        assert c.lens.tolist() == [30] and torch.equal(c.k[0], rows)
        with pytest.raises(RuntimeError, match="status 2"):
            c.check()


def full_step(cache, stream, busy):
    """A step on `stream` that a full cache refuses, behind some milliseconds of other work there."""
    x = torch.zeros(1, 2, 64, dtype=F16, device=cache.lens.device)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(20):
            busy @ busy
    cache.begin(stream=stream)
    cache.layer(0, x, x[:, :1], x[:, :1], x, stream=stream)
    cache.end(stream)


@pytest.mark.parametrize("how", ["stream", "handle", "none"])
def test_check_waits_for_the_steps_stream(cuda_dev, how):
    """A refused step on a side stream, still running when check() is called: check() sees it, once."""
    c = step.PagedCache(1, 1, 2, 1, 64, max_len=16, page_size=16, device=cuda_dev)
    c.lens.fill_(16)
    busy, s = torch.zeros(4096, 4096, device=cuda_dev), torch.cuda.Stream()
    given = dict(stream=[s], handle=[s.cuda_stream], none=[])[how]
    for _ in range(2):
        full_step(c, s, busy)
        with pytest.raises(RuntimeError, match="status 2"):
            c.check(*given)
        c.check(*given)


def test_state_and_restore_on_the_steps_stream(cuda_dev):
    """state() behind a step that is still running holds its lengths, restore() undoes what follows it."""
    c = step.PagedCache(1, 1, 2, 1, 64, max_len=64, page_size=16, device=cuda_dev)
    busy, s = torch.zeros(4096, 4096, device=cuda_dev), torch.cuda.Stream()
    full_step(c, s, busy)
    was = c.state(s)
    full_step(c, s, busy)
    c.restore(was, s)
    s.synchronize()
    assert c.lens.tolist() == [1] and was[0].tolist() == [1] and int(c.start) == 1
    c.check(s)


def test_restore_of_the_empty_state_frees_all(cuda_dev):
    """A cache with pages for one batch only serves the next after restore(): the same steps, the same bits."""
    gen = torch.Generator().manual_seed(5)
    c = step.PagedCache(1, 2, 2, 1, 64, max_len=32, page_size=16, device=cuda_dev)
    empty = c.state()
    xs = [[torch.randn(2, h, 64, generator=gen).to(F16).to(cuda_dev) for h in (2, 1, 1)] for _ in range(32)]
    runs = []
    for _ in range(2):
        outs = []
        for q, k, v in xs:
            out = torch.empty(2, 2, 64, dtype=F16, device=cuda_dev)
            c.begin()
            c.layer(0, q, k, v, out)
            c.end()
            outs.append(out)
        c.check()
        runs.append(torch.stack(outs))
        assert int(c.start) == c.pages == 4      # every page is taken
        c.restore(empty)
    assert torch.equal(runs[0], runs[1])
