"""Refusals of the prefill step's entry points that need no GPU: every check
of host-visible arguments returns before a CUDA call."""
import ctypes

import pytest

ARG, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from paged_mla_decode_04_gb300 import _build
    import paged_mla_decode_04_gb300 as m
    return m.load_library(_build.build())


@pytest.fixture(scope="module")
def mem():
    """Host memory that stands for device pointers; no accepted call is made with it."""
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 1023) // 1024 * 1024
    mem.buf = buf
    return base


def pool(mem, **kw):
    import paged_mla_decode_04_gb300 as m
    d = dict(data=mem, num_layers=2, num_pages=4, page_size=16, dtype=0, kv_scale=1.0)
    d.update(kw)
    return bytes(m._Pool(d["data"], d["num_layers"], d["num_pages"], d["page_size"], d["dtype"], d["kv_scale"]))


TABLES = ["context_lens", "new_lens", "batch", "page_size", "num_pages", "free_pages", "free_count", "free_capacity",
          "block_table", "max_blocks", "slot_mapping", "positions", "max_tokens", "q_indptr", "page_indptr", "page_ids",
          "max_page_ids", "state", "workspace", "stream"]


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), ARG), (dict(num_pages=0), ARG), (dict(max_blocks=0), ARG), (dict(free_capacity=-1), ARG),
    (dict(max_tokens=-1), ARG), (dict(max_page_ids=-1), ARG), (dict(page_size=48), UNSUPPORTED),
    (dict(max_blocks=1 << 27, page_size=16), ARG), (dict(batch=1 << 16, max_blocks=1 << 15), ARG), (dict(context_lens=None), ARG), (dict(new_lens=None), ARG),
    (dict(free_pages=None), ARG), (dict(free_count=None), ARG), (dict(block_table=None), ARG),
    (dict(slot_mapping=None), ARG), (dict(q_indptr=None), ARG), (dict(state=None), ARG), (dict(page_indptr=None), ARG),
    (dict(page_ids=None), ARG)])
def test_extend_tables(lib, mem, bad, code):
    a = {n: mem for n in TABLES}
    a.update(batch=2, page_size=16, num_pages=4, free_capacity=4, max_blocks=4, max_tokens=4, max_page_ids=4, stream=None)
    a.update(bad)
    assert lib.mla_extend_tables(*[a[n] for n in TABLES]) == code


ROPE = ["pool", "layer", "rows", "slot_mapping", "n", "positions", "num_axes", "pair_axis", "cos_sin", "max_position",
        "interleaved", "norm_weight", "norm_eps", "q_rope", "q_pitch", "q_out", "q_out_pitch", "num_heads", "workspace",
        "stream"]


def rope(lib, mem, **kw):
    a = {n: mem for n in ROPE}
    a.update(pool=pool(mem), layer=0, n=3, num_axes=1, pair_axis=None, max_position=8, interleaved=1,
             norm_eps=1e-6, q_rope=mem, q_out=mem + 8192, q_pitch=64, q_out_pitch=64, num_heads=2, stream=None)
    a.update(kw)
    return lib.mla_rope_write(*[a[n] for n in ROPE])


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(num_axes=0), dict(num_axes=5), dict(max_position=0), dict(pair_axis=bytes([1] * 32)), dict(layer=2),
    dict(layer=-1), dict(pool=None), dict(rows=None, q_rope=None), dict(slot_mapping=None), dict(positions=None),
    dict(cos_sin=None), dict(norm_eps=-1.0), dict(norm_eps=float("nan")), dict(q_out=None), dict(q_pitch=60),
    dict(q_pitch=68), dict(q_out_pitch=32), dict(num_heads=0)])
def test_rope_write(lib, mem, bad):
    assert rope(lib, mem, **bad) == ARG


def test_rope_write_alignment_and_overlap(lib, mem):
    for name in ("rows", "cos_sin", "norm_weight", "q_rope", "q_out"):
        assert rope(lib, mem, **{name: mem + 8}) == ARG
    # rows of the source shifted by less than a row, by a whole row, or at another pitch
    assert rope(lib, mem, q_rope=mem, q_out=mem + 64, q_pitch=192, q_out_pitch=192) == ARG
    assert rope(lib, mem, q_rope=mem, q_out=mem + 384, q_pitch=192, q_out_pitch=192) == ARG
    assert rope(lib, mem, q_rope=mem + 64, q_out=mem, q_pitch=192, q_out_pitch=192) == ARG
    assert rope(lib, mem, q_rope=mem, q_out=mem, q_pitch=64, q_out_pitch=128) == ARG
    assert rope(lib, mem, n=0) == 0
    bad = pool(mem, dtype=1, kv_scale=0.0)
    assert rope(lib, mem, pool=bad) == ARG


PREFILL = ["pool", "layer", "q", "q_indptr", "page_indptr", "page_ids", "max_blocks", "context_lens", "batch", "q_rows",
           "max_kv_tokens", "num_heads", "w_uk", "w_uv", "softmax_scale", "window", "workspace", "workspace_bytes", "out",
           "lse", "stream"]


@pytest.mark.parametrize("bad,code", [
    (dict(pool=None), ARG), (dict(layer=2), ARG), (dict(window=-1), ARG), (dict(batch=-1), ARG), (dict(q_rows=-1), ARG),
    (dict(max_kv_tokens=-1), ARG), (dict(max_kv_tokens=1 << 31), ARG), (dict(num_heads=0), ARG),
    (dict(num_heads=1025), ARG), (dict(q_rows=1 << 28, num_heads=16), ARG), (dict(softmax_scale=0.0), ARG),
    (dict(softmax_scale=float("nan")), ARG), (dict(q=None), ARG), (dict(q_indptr=None), ARG), (dict(page_ids=None, page_indptr=None), ARG),
    (dict(context_lens=None), ARG), (dict(w_uk=None), ARG), (dict(w_uv=None), ARG), (dict(out=None), ARG),
    (dict(page_indptr=None, max_blocks=0), ARG), (dict(page_indptr=None, max_blocks=1 << 28), ARG),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=1000), WORKSPACE)])
def test_prefill(lib, mem, bad, code):
    a = {n: mem for n in PREFILL}
    a.update(pool=pool(mem), layer=0, max_blocks=4, batch=2, q_rows=8, max_kv_tokens=64, num_heads=4,
             softmax_scale=0.07, window=0, workspace_bytes=1 << 14, stream=None)
    a.update(bad)
    assert lib.mla_prefill(*[a[n] for n in PREFILL]) == code


def test_prefill_alignment_and_empty_calls(lib, mem):
    def call(**kw):
        a = {n: mem for n in PREFILL}
        a.update(pool=pool(mem), layer=0, max_blocks=4, batch=2, q_rows=8, max_kv_tokens=64, num_heads=4,
                 softmax_scale=0.07, window=0, workspace_bytes=1 << 14, stream=None)
        a.update(kw)
        return lib.mla_prefill(*[a[n] for n in PREFILL])
    for name in ("q", "w_uk", "w_uv"):
        assert call(**{name: mem + 8}) == ARG
    assert call(out=mem + 16) == ARG
    assert call(workspace=mem + 16) == WORKSPACE
    assert call(batch=0) == 0 and call(q_rows=0) == 0


def test_prefill_workspace_size(lib):
    size = lib.mla_prefill_workspace_size
    for bad in [(-1, 8, 64, 4, 0), (2, -1, 64, 4, 0), (2, 8, -1, 4, 0), (2, 8, 64, 0, 0), (2, 8, 64, 4, -1),
                (2, 8, 1 << 31, 4, 0), (2, 1 << 28, 64, 16, 0), (2, 8, 64, 1025, 0)]:
        assert size(*bad) == 0
    # 512 bytes a head and row, all heads by default, never more than there are
    assert size(2, 8, 64, 4, 0) == size(2, 8, 64, 4, 4) == size(2, 8, 64, 4, 9) > size(2, 8, 64, 4, 1) > 0
    rows = 1000 * 128
    assert abs(size(1, 8, rows - 16, 8, 8) - size(1, 8, rows - 16, 8, 7) - rows * 512) < 1 << 20
    # the default keeps keys and values within 8 GiB, beside the rows themselves and the partial sums
    assert size(1, 8, 1 << 20, 128, 0) <= (8 << 30) + (1 << 20) * 1152 + (64 << 20)
    assert size(0, 0, 0, 1, 0) > 0


@pytest.mark.parametrize("batch,q_rows,max_kv", [(1, 1, 1), (3, 700, 100), (2, 64, 2000)])
def test_prefill_workspace_grows_with_heads(lib, batch, q_rows, max_kv):
    # A call finds the most heads that fit, then cuts its heads into equal passes: fewer
    # heads a pass must never need more room.
    sizes = [lib.mla_prefill_workspace_size(batch, q_rows, max_kv, 1024, h) for h in range(1, 1025)]
    assert all(a < b for a, b in zip(sizes, sizes[1:]))


def test_compiled_binding(lib):
    import paged_mla_decode_04_gb300 as m
    b = m._step()
    for name, n in (("extend_tables", 15), ("rope_write", 15), ("prefill", 18), ("bind", 3)):
        with pytest.raises(TypeError, match="%d arguments expected" % n):
            getattr(b, name)()
    with pytest.raises(ValueError, match="entry point"):
        b.bind(0, 0, 0)
