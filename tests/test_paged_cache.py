"""step.PagedCache's own bookkeeping, on the CPU, with fakes of the library's calls."""
import pytest
import torch

from int4_block_quantized_matmulnbits_b200 import step


@pytest.fixture
def calls(monkeypatch):
    """The library calls that a cache has made, by name."""
    made = []
    for name in ("mnb_paged_tables", "mnb_rope_append", "mnb_paged_attention"):
        monkeypatch.setattr(step, name, lambda *a, name=name: made.append(name))
    return made


def cache(**kw):
    return step.PagedCache(1, 3, 2, 1, 64, **{**dict(max_len=32, device="cpu"), **kw})


def rows(T=3):
    q, k = torch.zeros(T, 2, 64, dtype=torch.float16), torch.zeros(T, 1, 64, dtype=torch.float16)
    return q, k, k


def test_layer_takes_decode_steps_only(calls):
    """The rows of a step that gives a request no token, or several, are not the requests' rows: nothing is launched."""
    c, out = cache(), torch.zeros(3, 2, 64, dtype=torch.float16)
    new, slots = torch.tensor([1, 0, 1], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for begin in (lambda: None, lambda: c.begin(new), lambda: c.begin(new, slots, slots),
                  lambda: c.begin(slots=slots, positions=slots)):
        begin()
        del calls[:]
        with pytest.raises(RuntimeError, match="decode step"):
            c.layer(0, *rows(), out)
        assert calls == []
    c.begin()
    c.layer(0, *rows(), out)
    assert calls == ["mnb_paged_tables", "mnb_rope_append", "mnb_paged_attention"]
    c.end()
    with pytest.raises(RuntimeError, match="decode step"):   # the step is over
        c.layer(0, *rows(), out)


def test_append_without_slots_needs_this_steps(calls):
    """Slots of an earlier step would be written over."""
    c, slots = cache(), torch.zeros(3, dtype=torch.int32)
    q, k, v = rows()
    c.begin()
    c.append(0, q, k, v, q)
    c.end()
    c.begin(torch.ones(3, dtype=torch.int32), slots, slots)
    del calls[:]
    with pytest.raises(RuntimeError, match="own buffers"):
        c.append(0, q, k, v, q)
    assert calls == []
    c.append(0, q, k, v, q, slots, slots)
    c.begin(torch.tensor([1, 0, 1], dtype=torch.int32))     # packed into the cache's buffers: rows 0 and 1
    c.append(0, q, k, v, q)
    for f in (lambda: c.begin(slots=slots), lambda: c.begin(positions=slots), lambda: c.append(0, q, k, v, q, slots)):
        with pytest.raises(ValueError, match="go together"):
            f()


def test_a_begin_that_fails_begins_no_step(calls, monkeypatch):
    c = cache()
    c.begin()

    def fails(*a):
        raise RuntimeError("refused")

    monkeypatch.setattr(step, "mnb_paged_tables", fails)
    with pytest.raises(RuntimeError, match="refused"):
        c.begin()
    with pytest.raises(RuntimeError, match="decode step"):
        c.layer(0, *rows(), torch.zeros(3, 2, 64, dtype=torch.float16))


def test_max_len_inside_a_page(monkeypatch):
    """max_len = 30 in pages of 16, whose tables have room for 32: a request that would hold 31 is shown to them as
    full, so that they refuse it, and keeps its length; the others are not touched."""
    c, seen = cache(max_len=30, page_size=16), []

    def tables(lens, new, *a):      # as the library does it, but for pages and slots
        seen.append(lens.tolist())
        a[5].copy_(torch.where(lens.long() + new > 32, lens, lens + new))

    monkeypatch.setattr(step, "mnb_paged_tables", tables)
    c.lens.copy_(torch.tensor([29, 30, 7]))
    c.begin()
    assert seen == [[29, 32, 7]] and c.new_lens.tolist() == [30, 30, 8] and c.lens.tolist() == [29, 30, 7]
    c.begin(torch.tensor([2, 0, 2 ** 31 - 1], dtype=torch.int32), c.slots, c.positions)
    assert seen[1] == [32, 30, 32] and c.new_lens.tolist() == [29, 30, 7]
    whole = cache(max_len=32, page_size=16)      # nothing to hide here
    whole.lens.fill_(31)
    whole.begin()
    assert seen[2] == [31, 31, 31]


def test_every_position_has_an_angle():
    """Without, the append would drop keys while the lengths go on."""
    angles = torch.zeros(30, 32)
    assert cache(max_len=30, cos=angles, sin=angles).max_len == 30
    for kw in (dict(cos=angles[:29], sin=angles[:29]), dict(cos=angles, sin=angles[:29])):
        with pytest.raises(ValueError, match="29 rows for max_len = 30"):
            cache(max_len=30, **kw)
    with pytest.raises(ValueError, match="go together"):
        cache(max_len=30, cos=angles)
