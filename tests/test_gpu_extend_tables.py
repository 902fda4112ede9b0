"""Page tables of a step built on the GPU (extend_tables): every output equals
a plain one-page-after-another construction exactly."""
import numpy as np
import pytest
import torch

import step_ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def make(rng, ctx, new, ps, width=None, spare=5, count=None):
    held = [-(-max(c, 0) // ps) for c in ctx]
    total = [max(c, 0) + max(n, 0) for c, n in zip(ctx, new)]
    blocks = [-(-t // ps) for t in total]
    num_pages = sum(max(a, b) for a, b in zip(blocks, held)) + spare + 1
    width = width or max(blocks + [1])
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(ctx), width), -7, np.int32)  # -7: must stay
    k = 0
    for b, h in enumerate(held):
        h = min(h, width)
        table[b, :h] = perm[k:k + h]
        k += h
    free = perm[k:]
    return dict(ctx=np.array(ctx, np.int32), new=np.array(new, np.int32), table=table, free=free,
                count=len(free) if count is None else count, ps=ps, num_pages=num_pages)


class Device:
    def __init__(self, lib, c, max_tokens, max_ids, csr=True, positions=True):
        d = "cuda"
        self.lib, self.c, self.csr = lib, c, csr
        B = len(c["ctx"])
        self.ctx = torch.from_numpy(c["ctx"]).to(d)
        self.new = torch.from_numpy(c["new"]).to(d)
        self.free = torch.from_numpy(c["free"].copy()).to(d)
        self.count = torch.tensor([c["count"]], dtype=I32, device=d)
        self.table = torch.from_numpy(c["table"].copy()).to(d)
        self.slots = torch.full((max_tokens,), 99, dtype=torch.int64, device=d)
        self.pos = torch.full((max_tokens,), 99, dtype=I32, device=d) if positions else None
        self.indptr = torch.full((B + 1,), 99, dtype=I32, device=d)
        self.pind = torch.full((B + 1,), 99, dtype=I32, device=d) if csr else None
        self.ids = torch.full((max_ids,), 99, dtype=I32, device=d) if csr else None
        self.state = torch.full((2,), 99, dtype=I32, device=d)
        self.ws = torch.zeros(256, dtype=torch.uint8, device=d)

    def call(self, count=None, state=None):
        self.lib.extend_tables(self.ctx, self.new, self.free, self.count if count is None else count, self.table,
                               self.c["ps"], self.c["num_pages"], self.slots, self.indptr,
                               self.state if state is None else state, positions=self.pos, page_indptr=self.pind,
                               page_ids=self.ids, workspace=self.ws)
        torch.cuda.synchronize()

    def check(self, ref, state=True):
        assert np.array_equal(self.table.cpu().numpy(), ref["table"])
        assert np.array_equal(self.slots.cpu().numpy(), ref["slots"])
        assert np.array_equal(self.indptr.cpu().numpy(), ref["indptr"])
        if self.pos is not None:
            assert np.array_equal(self.pos.cpu().numpy(), ref["positions"])
        if state:
            assert np.array_equal(self.state.cpu().numpy(), ref["state"])
        if self.csr:
            assert np.array_equal(self.pind.cpu().numpy(), ref["page_indptr"])
            got, n = self.ids.cpu().numpy(), min(len(ref["ids"]), self.ids.numel())
            assert np.array_equal(got[:n], ref["ids"][:n]) and (got[n:] == 99).all()
        assert self.lib.get_error(self.ws) == ref["status"]


def reference(c, max_tokens, max_ids=None):
    return step_ref.extend_tables(c["ctx"], c["new"], c["free"], c["count"], c["table"], c["ps"], c["num_pages"],
                                  max_tokens, max_ids)


def run(lib, c, max_tokens=None, max_ids=None, **kw):
    n = int(np.maximum(c["new"], 0).sum())
    max_tokens = n + 3 if max_tokens is None else max_tokens
    full = reference(c, max_tokens)
    max_ids = len(full["ids"]) + 2 if max_ids is None else max_ids
    d = Device(lib, c, max_tokens, max_ids, **kw)
    d.call()
    d.check(reference(c, max_tokens, max_ids if kw.get("csr", True) else None))
    return d


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_edges_of_pages(lib, ps):
    edges = [0, 1, ps - 1, ps, ps + 1, 2 * ps, 5 * ps + 3]
    ctx = [c for c in edges for _ in edges]
    new = [n for _ in edges for n in edges]
    run(lib, make(np.random.default_rng(ps), ctx, new, ps))


@pytest.mark.parametrize("batch,new_hi", [(1, 1), (1, 5000), (3, 2000), (128, 1), (700, 9), (1024, 1), (1025, 3), (3000, 2), (3840, 1),
                                          (3841, 3), (9000, 2)])
def test_batches_of_both_launch_forms(lib, batch, new_hi):
    rng = np.random.default_rng(batch + new_hi)
    ctx = rng.integers(0, 400, batch)
    new = rng.integers(0 if batch > 1 else new_hi, new_hi + 1, batch)
    run(lib, make(rng, ctx.tolist(), new.tolist(), 16))


def test_long_tables(lib):
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 131072, 40)
    run(lib, make(rng, ctx.tolist(), rng.integers(0, 70, 40).tolist(), 64))


def test_outputs_that_are_not_asked_for(lib):
    rng = np.random.default_rng(6)
    run(lib, make(rng, [5, 100, 0], [3, 0, 40], 16), csr=False)
    run(lib, make(rng, [5, 100, 0], [3, 0, 40], 16), positions=False)


def test_empty_batch_and_no_tokens(lib):
    rng = np.random.default_rng(7)
    run(lib, make(rng, [], [], 16, width=1))
    d = run(lib, make(rng, [30, 0, 16], [0, 0, 0], 16))
    assert (d.slots.cpu() == -1).all()


@pytest.mark.parametrize("count", [0, 1, 2, 7, 11, 12, 20])
@pytest.mark.parametrize("many", [False, True])
def test_pages_that_do_not_suffice(lib, count, many):
    """A refused request takes nothing, those behind it that need pages neither; those that need none are served."""
    ctx, new = [15, 3, 16, 40, 0, 7], [1, 4, 40, 7, 150, 1]
    if many:  # past the one-block form
        ctx, new = ctx + [16] * 1500, new + [4] * 1500
    run(lib, make(np.random.default_rng(8), ctx, new, 16, count=count))


def test_bad_lengths_are_refused_alone(lib):
    ctx, new = [3, -1, 20, 100, 5, 64], [4, 2, -5, 29, 6, 64]
    c = make(np.random.default_rng(9), ctx, new, 16, width=8)  # 129 and 128 tokens of room 128
    run(lib, c)


def test_bad_page_ids(lib):
    c = make(np.random.default_rng(10), [20, 5, 0], [4, 30, 3], 16)
    c["table"][0, 1] = c["num_pages"]       # the page that request 0's tokens go to
    c["free"] = c["free"].copy()
    c["free"][c["count"] - 2] = -3          # the second page handed out
    run(lib, c)


@pytest.mark.parametrize("max_tokens,max_ids", [(0, 0), (5, 3), (30, 1), (4097, 2)])
def test_short_output_arrays(lib, max_tokens, max_ids):
    run(lib, make(np.random.default_rng(11), [20, 5, 0], [14, 30, 3], 16), max_tokens=max_tokens, max_ids=max_ids)


def test_count_beyond_the_stack_is_its_length(lib):
    c = make(np.random.default_rng(12), [1], [100], 16)
    c["count"] = len(c["free"]) + 50
    run(lib, c)


def test_count_updated_in_place_over_captured_steps(lib):
    """free_count and state share memory; a graph of one step, replayed, hands out further pages each time."""
    rng = np.random.default_rng(13)
    B, ps, steps = 9, 16, 40
    ctx0 = rng.integers(0, 50, B).astype(np.int32)
    c = make(rng, (ctx0 + steps).tolist(), [0] * B, ps, spare=0)
    c["table"][:] = -1
    perm = rng.permutation(c["num_pages"]).astype(np.int32)
    k = 0
    for b in range(B):
        h = -(-int(ctx0[b]) // ps)
        c["table"][b, :h] = perm[k:k + h]
        k += h
    c.update(ctx=ctx0, new=np.ones(B, np.int32), free=perm[k:], count=len(perm) - k)
    d = Device(lib, c, B + 2, int(c["table"].size))
    state = torch.tensor([c["count"], 0], dtype=I32, device="cuda")
    before = d.table.clone()
    d.call(count=state, state=state)  # loads the kernels
    d.table.copy_(before)
    state[0] = c["count"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.extend_tables(d.ctx, d.new, d.free, state, d.table, ps, c["num_pages"], d.slots, d.indptr, state,
                          positions=d.pos, page_indptr=d.pind, page_ids=d.ids, workspace=d.ws)
        d.ctx.add_(d.new)
    for _ in range(steps):
        ref = reference(c, B + 2)
        g.replay()
        torch.cuda.synchronize()
        d.ids[len(ref["ids"]):] = 99
        d.check(ref, state=False)
        assert state.cpu().tolist() == ref["state"].tolist()
        c.update(ctx=c["ctx"] + 1, table=ref["table"], count=int(ref["state"][0]))
    assert len(set(c["table"][c["table"] >= 0].tolist())) == int((c["table"] >= 0).sum())  # no page twice


def test_refusals(lib):
    c = make(np.random.default_rng(14), [3, 4], [1, 1], 16)
    d = Device(lib, c, 4, 4)
    call = lambda **k: lib.extend_tables(**{**dict(  # noqa: E731
        context_lens=d.ctx, new_lens=d.new, free_pages=d.free, free_count=d.count, block_table=d.table, page_size=16,
        num_pages=c["num_pages"], slot_mapping=d.slots, q_indptr=d.indptr, state=d.state), **k})
    for bad in [dict(new_lens=d.new[:1]), dict(block_table=d.table[:1]), dict(slot_mapping=d.slots[:, None]),
                dict(positions=d.pos[:2]), dict(q_indptr=d.indptr[:2]), dict(page_indptr=d.pind),
                dict(state=d.state[:1]), dict(context_lens=d.ctx.long()), dict(new_lens=d.new.cpu()),
                dict(slot_mapping=d.slots.int())]:
        with pytest.raises(ValueError):
            call(**bad)
    for bad in [dict(page_size=17), dict(num_pages=0)]:
        with pytest.raises(lib.MlaError):
            call(**bad)
