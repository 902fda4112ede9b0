"""The workspace of extend_tables and rope_write, of which the kernels write the status word."""
import pytest
import torch

from test_step_library import ROPE, TABLES, WORKSPACE, lib, mem, pool  # noqa: F401


def tables_call(lib, mem, **kw):  # noqa: F811
    a = {n: mem for n in TABLES}
    a.update(batch=2, page_size=16, num_pages=4, free_capacity=4, max_blocks=4, max_tokens=4, max_page_ids=4, stream=None, **kw)
    return lib.mla_extend_tables(*[a[n] for n in TABLES])


def rope_call(lib, mem, **kw):  # noqa: F811
    a = {n: mem for n in ROPE}
    a.update(pool=pool(mem), layer=0, n=3, num_axes=1, pair_axis=None, max_position=8, interleaved=1, norm_eps=1e-6,
             q_rope=mem, q_out=mem + 8192, q_pitch=64, q_out_pitch=64, num_heads=2, stream=None, **kw)
    return lib.mla_rope_write(*[a[n] for n in ROPE])


@pytest.mark.parametrize("offset", [1, 2, 4, 16, 128, 255])
@pytest.mark.parametrize("call", [tables_call, rope_call])
def test_misaligned_workspaces_are_refused(lib, mem, call, offset):  # noqa: F811
    assert call(lib, mem, workspace=mem + offset) == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("short", [0, 1, 3, 255])
def test_short_workspaces_are_refused(short):
    import paged_mla_decode_04_gb300 as m
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.full((10,), 7, dtype=torch.int64, device="cuda")
    tables = dict(context_lens=i(0, 20), new_lens=i(3, 5), free_pages=i(0, 1, 2, 3, 4, 5), free_count=i(6),
                  block_table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), page_size=16, num_pages=6,
                  slot_mapping=slots, q_indptr=i(0, 0, 0), state=i(0, 0))
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros(8, 64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        m.extend_tables(**tables, workspace=ws[:short])
    with pytest.raises(ValueError, match="workspace"):
        m.rope_write(None, 0, None, None, i(0, 1, 2), cs, q_rope=q, workspace=ws[:short])
    torch.cuda.synchronize()
    assert (slots == 7).all() and (q == 1).all()
    # 256 bytes are enough: page 5 and the cached page's rest, and a bad position in the status word
    m.extend_tables(**tables, workspace=ws)
    m.rope_write(None, 0, None, None, i(0, 1, 9), cs, q_rope=q, workspace=ws)
    assert m.get_error(ws) == m.STATUS_BAD_PAGE | m.STATUS_BAD_POSITION  # (request 1's cached pages are -1)
    with pytest.raises(m.MlaError, match="WORKSPACE"):
        m.extend_tables(**tables, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")[4:])


@pytest.mark.gpu
def test_as_many_tokens_as_an_int_holds():
    """Slots for 2^31 - 1 tokens, of which 4,000 requests (two launches) use 8,000: the others are pad entries."""
    import paged_mla_decode_04_gb300 as m
    B, most = 4000, (1 << 31) - 1
    z = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.full((most,), 7, dtype=torch.int64, device="cuda")
    table, state, indptr = torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), z(2), z(B + 1)
    m.extend_tables(z(B), z(B, 2), torch.arange(B, dtype=torch.int32, device="cuda"), z(1, B), table, 16, B, slots, indptr, state)
    assert state.tolist() == [0, B] and indptr[-1] == 2 * B
    want = (torch.arange(B - 1, -1, -1, device="cuda")[:, None] * 16 + torch.arange(2, device="cuda")).flatten()
    assert torch.equal(slots[:2 * B], want)
    for part in slots[2 * B:].split(1 << 28):
        assert bool((part == -1).all())
