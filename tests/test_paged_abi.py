"""Refusals of the paged cache's entry points, without a GPU: the C ABI with addresses that are never used, and the
binding's checks of tensors."""
import struct

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = 0, -1, -2, -3, -4
F32, F16 = 0, 1
A = 1 << 20


@pytest.fixture(scope="module")
def mnb():
    import int4_block_quantized_matmulnbits_b200 as m

    return m


CACHE = dict(k=A, v=A, num_pages=10, page_size=16, num_heads=8, head_dim=128, page_stride=16 * 8 * 128,
             slot_stride=8 * 128, head_stride=128, dtype=F16, reserved=0)


def cache(**kw):
    assert set(kw) <= set(CACHE)
    return [0 if v is None else v for v in {**CACHE, **kw}.values()]


# the argument structs of mnb.h as struct formats
CACHE_FMT = "PPqqqqqqqii"
FMT = dict(tables="@11P7q", append="@11P" + CACHE_FMT + "12qfi", attention="@7P" + CACHE_FMT + "8qNfi")


def call(fn, fmt, fields, kw, flags):
    assert set(kw) <= set(fields)
    vals = []
    for v in {**fields, **kw}.values():
        vals += v if isinstance(v, list) else [0 if v is None else v]
    return fn(struct.pack(FMT[fmt], *vals), flags, None)


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=2), INVALID), (dict(num_pages=0), SHAPE),
              (dict(page_size=0), SHAPE), (dict(num_pages=2 ** 20, page_size=2 ** 12), SHAPE),
              (dict(num_heads=0), SHAPE), (dict(num_heads=5000), SHAPE), (dict(head_dim=100), SHAPE),
              (dict(head_dim=264), SHAPE), (dict(head_dim=0), SHAPE), (dict(k=A + 8), ALIGN),
              (dict(page_stride=-8), SHAPE), (dict(slot_stride=1028), ALIGN), (dict(head_stride=2 ** 31 + 8), SHAPE),
              (dict(dtype=F32, head_stride=130), ALIGN)]


def tables(mnb, flags=0, **kw):
    d = dict(ctx=A, new=A + 64, free=A, start=A, table=A, seq=A + 128, cu=A, slots=A, pos=A, next=A + 4, status=None,
             B=4, T=4, page=16, pages=10, nfree=10, stride=8, blocks=8)
    return call(mnb._lib.mnb_paged_tables, "tables", d, kw, flags)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(nfree=-1), INVALID), (dict(B=4097), UNSUPPORTED),
    (dict(page=0), SHAPE), (dict(pages=0), SHAPE), (dict(page=2 ** 16, pages=2 ** 15), SHAPE), (dict(blocks=0), SHAPE),
    (dict(stride=7), SHAPE), (dict(blocks=2 ** 27, stride=2 ** 27), SHAPE), (dict(T=2 ** 30 + 1), SHAPE),
    (dict(flags=2), INVALID), (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID),
    (dict(seq=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(free=None), INVALID),
    (dict(start=None), INVALID), (dict(next=None), INVALID), (dict(slots=A + 2), ALIGN), (dict(status=A + 1), ALIGN),
    (dict(next=A), INVALID), (dict(seq=A), INVALID), (dict(seq=A + 64), INVALID)])
def test_tables_refusals(mnb, kw, rc):
    assert tables(mnb, **kw) == rc
    assert "mnb_paged_tables" in mnb.mnb_last_error()


def append(mnb, c=None, flags=0, **kw):
    d = dict(q=A, k=A, v=A, o=A + 4096, slots=A, pos=A, cos=A, sin=A, qw=A, kw=A, status=None, cache=c or cache(),
             qt=4096, qh=128, kt=4096, kh=128, vt=4096, vh=128, ot=2048, oh=128, T=4, Hq=16, R=128, num_pos=100,
             eps=1e-6, reserved=0)
    return call(mnb._lib.mnb_rope_append, "append", d, kw, flags)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(R=-8), INVALID), (dict(R=12), SHAPE), (dict(R=136), SHAPE),
    (dict(num_pos=0), SHAPE), (dict(T=2 ** 30 + 1), SHAPE), (dict(Hq=4097), SHAPE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(flags=4), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(cos=None), INVALID), (dict(sin=None), INVALID),
    (dict(q=A + 8), ALIGN), (dict(kw=A + 4), ALIGN), (dict(pos=A + 2), ALIGN), (dict(qt=4100), ALIGN),
    (dict(vh=-128), SHAPE), (dict(oh=0), SHAPE), (dict(ot=64), SHAPE), (dict(o=A, ot=2048), INVALID)])
def test_append_refusals(mnb, kw, rc):
    assert append(mnb, **kw) == rc
    assert "mnb_rope_append" in mnb.mnb_last_error()


def test_append_refuses_rows_on_one_another(mnb):
    for kw in (dict(head_stride=64), dict(slot_stride=0), dict(page_stride=120)):
        assert append(mnb, cache(**kw)) == SHAPE
    assert append(mnb, T=0) == OK


def attention(mnb, c=None, flags=0, **kw):
    d = dict(q=A, out=A, lse=None, table=A, lens=A, ws=A, status=None, cache=c or cache(), qb=2048, qh=128, ob=2048,
             oh=128, stride=8, blocks=8, B=4, Hq=16, nws=1 << 30, scale=0.1, reserved=0)
    return call(mnb._lib.mnb_paged_attention, "attention", d, kw, flags)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(B=4097), UNSUPPORTED), (dict(Hq=12), SHAPE),
    (dict(Hq=4104), SHAPE), (dict(blocks=0), SHAPE), (dict(stride=4), SHAPE), (dict(blocks=2 ** 27, stride=2 ** 27), SHAPE),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(flags=8), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(ws=None), INVALID), (dict(q=A + 2), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(ws=A + 4), ALIGN), (dict(lse=A + 2), ALIGN), (dict(lens=A + 1), ALIGN),
    (dict(qh=132), ALIGN), (dict(ob=-8), SHAPE), (dict(oh=64), SHAPE), (dict(ob=0), SHAPE), (dict(nws=100), INVALID)])
def test_attention_refusals(mnb, kw, rc):
    assert attention(mnb, **kw) == rc
    assert "mnb_paged_attention" in mnb.mnb_last_error()


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_cache_refusals(mnb, kw, rc):
    assert append(mnb, cache(**kw)) == rc
    assert attention(mnb, cache(**kw)) == rc


def test_nothing_to_do(mnb):
    assert attention(mnb, B=0) == OK
    for fn in (mnb._lib.mnb_paged_tables, mnb._lib.mnb_rope_append, mnb._lib.mnb_paged_attention):
        assert fn(None, 0, None) == INVALID      # no arguments


def test_formats_are_the_structs_layout(tmp_path):
    """Sizes and a late offset of the argument structs, as a C compiler lays them out, against the formats above."""
    import os
    import subprocess

    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "mnb.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", '
                   "sizeof(mnb_paged_tables_args), sizeof(mnb_rope_append_args), sizeof(mnb_paged_attention_args), "
                   "offsetof(mnb_paged_tables_args, B), offsetof(mnb_rope_append_args, q_token_stride), "
                   "offsetof(mnb_paged_attention_args, scale)); return 0; }")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-I", inc, str(src), "-o", str(tmp_path / "s")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "s")]).split()]
    assert got == [struct.calcsize(f) for f in (*FMT.values(), "@11P", "@11P" + CACHE_FMT, "@7P" + CACHE_FMT + "8qN")]


def test_workspace_bytes(mnb):
    f = mnb.mnb_paged_attention_workspace_bytes
    assert f(1, 16, 8, 128) > 0 and f(64, 16, 8, 128) == f(1, 16, 8, 128)
    assert f(1, 32, 2, 256, torch.float32) > 0
    for bad in ((-1, 16, 8, 128), (4097, 16, 8, 128), (1, 15, 8, 128), (1, 16, 0, 128), (1, 16, 8, 100),
                (1, 16, 8, 264), (1, 8192, 8, 128), (1, 4, 8, 128)):
        assert f(*bad) == 0


def test_binding_refuses_tensors(mnb):
    """Tensors on the CPU, of other types, shapes or strides never reach a kernel."""
    i = torch.zeros(4, dtype=torch.int32)
    kv, q = torch.zeros(3, 16, 2, 64, dtype=torch.float16), torch.zeros(4, 4, 64, dtype=torch.float16)
    tab, ws = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(mnb.MnbError, match="current CUDA device"):
        mnb.mnb_paged_attention(q, kv, kv, tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="current CUDA device"):
        mnb.mnb_paged_tables(i, i, tab, 16, 3, i, i[:1], i, torch.zeros(5, dtype=torch.int32), i, i, i[:1])
    with pytest.raises(mnb.MnbError, match="current CUDA device"):
        mnb.mnb_rope_append(q, q[:, :2], q[:, 2:], kv, kv, i, None, None, None, q)
    with pytest.raises(mnb.MnbError, match="fp16 or fp32"):
        mnb.mnb_paged_attention(q, kv.bfloat16(), kv.bfloat16(), tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="v_cache has shape"):
        mnb.mnb_paged_attention(q, kv, kv[:2], tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="v_cache is torch.float32"):
        mnb.mnb_paged_attention(q, kv, kv.float(), tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="q has shape"):
        mnb.mnb_paged_attention(q[0], kv, kv, tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="k_cache's strides"):
        mnb.mnb_paged_attention(q, kv, kv.transpose(1, 2).contiguous().transpose(1, 2), tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="k has shape"):
        mnb.mnb_rope_append(None, q, kv[0, :4], kv, kv, i, None, None, None, None)
    with pytest.raises(mnb.MnbError, match="v_cache's last dimension"):
        mnb.mnb_paged_attention(q, kv, kv.transpose(1, 3).contiguous().transpose(1, 3), tab, i, 0.1, q, ws)
    with pytest.raises(mnb.MnbError, match="cu_new has shape"):
        mnb.mnb_paged_tables(i, i, tab, 16, 3, i, i[:1], i, i, i, i, i[:1])
    with pytest.raises(mnb.MnbError, match="go together"):
        mnb.mnb_rope_append(None, q, q, kv, kv, i, None, None, None, q)


def test_tuning_hook_checks_its_argument(mnb):
    f = mnb._lib.mnb_tune_paged_attention
    for bad in ((-1, 0, 0), (9, 0, 0), (0, -1, 0), (0, 13, 0), (0, 0, -1), (0, 0, 33)):
        assert f(*bad) == INVALID
    assert f(0, 0, 0) == OK


def test_binding_takes_other_objects_for_what_they_are(mnb):
    i, kv = torch.zeros(4, dtype=torch.int32), torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    for bad in (None, 7, "x", [1, 2]):
        assert mnb._binding.paged_attention(bad, kv, kv, i, i, 0.1, kv, kv, None, None, 0, None) is None
        assert mnb._binding.rope_append(bad, kv, kv, bad, kv, i, None, None, None, None, None, None, 0.0, None, 0, None) is None
        assert mnb._binding.paged_tables(bad, i, i, 1, 1, i, i, i, i, i, i, i, None, 0, None) is None
    with pytest.raises(TypeError):
        mnb._binding.paged_attention(1, 2)
