"""Chunk attention over the paged cache (prefill) against a plain 64-bit form.

Every output is held to the bound that the kernel's roundings allow (see
step_ref.prefill); over all outputs the errors also have to be as small as
independent roundings are: each rounding to bf16 is at most 2^-8 / sqrt(3) =
2.3e-3 of the value in the root mean square, values, weights and output are one
each, and the keys' give scores of standard deviation 1 an error of 1.9e-3,
which moves weights in the sum and their normaliser: sqrt(3 * 2.3^2 + (2 *
1.9)^2) = 5.5e-3 of the norm (bounded by 6e-3 below, scaled by the scores'
deviation where a test makes it larger)."""
import numpy as np
import pytest
import torch

import step_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Case:
    """Requests of ctx cached and new tokens on randomly permuted pages of layer 1."""

    def __init__(self, lib, ctx, new, heads=4, ps=64, fp8=False, window=0, seed=0, q_std=1.0, extra_rows=3, csr=False,
                 heads_per_pass=0, spare_kv=0):
        g = torch.Generator("cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.lib, self.ctx_h, self.new_h, self.window, self.ps, self.fp8 = lib, ctx, new, window, ps, fp8
        total = [c + n for c, n in zip(ctx, new)]
        blocks = [-(-t // ps) for t in total]
        self.num_pages = sum(blocks) + 5
        perm = torch.randperm(self.num_pages, generator=g, device="cuda").to(torch.int32)
        width = max(blocks + [1])
        self.table = torch.full((len(ctx), width), -1, dtype=torch.int32, device="cuda")
        k, ind = 0, [0]
        for b, m in enumerate(blocks):
            self.table[b, :m] = perm[k:k + m]
            k += m
            ind.append(k)
        self.ids = perm[:k].contiguous()
        self.pind = torch.tensor(ind, dtype=torch.int32, device="cuda")
        data = r(2, self.num_pages, ps, 576)
        self.scale_kv = 0.02 if fp8 else 1.0
        data = (data / 0.02).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else data.to(torch.bfloat16)
        self.pool = lib.KVPool(data, self.scale_kv)
        self.T = sum(new) + extra_rows
        self.q = (r(self.T, heads, 192) * q_std).to(torch.bfloat16)
        self.w_uk = (r(heads, 128, 512) * 512 ** -0.5).to(torch.bfloat16)
        self.w_uv = (r(heads, 512, 128) * 512 ** -0.5).to(torch.bfloat16)
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.indptr = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.scale = 192 ** -0.5
        self.max_kv = sum(t - (max(0, c + 1 - window) if window else 0) for t, c, n in zip(total, ctx, new) if n) + spare_kv
        self.heads, self.csr = heads, csr
        self.ws = lib.alloc_prefill_workspace(len(ctx), self.T, self.max_kv, heads, heads_per_pass)
        self.out = torch.full((self.T, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, heads), 7.0, device="cuda")

    def run(self, **kw):
        pages = dict(page_indptr=self.pind, page_ids=self.ids) if self.csr else dict(block_table=self.table)
        self.lib.prefill(self.pool, 1, self.q, self.indptr, self.ctx, self.scale, self.w_uk, self.w_uv, self.ws, self.out,
                         self.max_kv, **{**pages, "window": self.window, "lse": self.lse, **kw})
        torch.cuda.synchronize()
        return self

    def values(self):
        d = self.pool.data[1]
        return f64(d.view(torch.float8_e4m3fn) if self.fp8 else d) * self.scale_kv

    def reference(self):
        vals, table = self.values(), self.table.cpu().numpy()
        return step_ref.prefill(lambda b, at: vals[table[b][at // self.ps], at % self.ps], f64(self.q),
                                self.indptr.cpu().numpy(), self.ctx.cpu().numpy(), f64(self.w_uk), f64(self.w_uv),
                                self.scale, self.window, lambda n, m: self.latent() and n <= (56 if m >= 3000 else 32))

    def latent(self):
        """Calls of this size attend requests of up to 32 new tokens (56 over 3,000 positions) in the latent space."""
        size, few = self.max_kv * self.heads, self.T <= 8 * len(self.ctx)
        return self.heads in (16, 32, 64, 128) and (
            size >= 200000 or few and (size >= 100000 or len(self.ctx) * self.heads >= 400))

    def check(self, norm=6e-3, status=0):
        ref, lse, tol, tol_lse = self.reference()
        n = int(self.indptr[-1])
        got, got_lse = f64(self.out), f64(self.lse)
        assert (got[n:] == 7.0).all() and (got_lse[n:] == 7.0).all()  # rows behind the last request
        bad = np.abs(got[:n] - ref[:n]) > tol[:n]
        assert not bad.any(), "rows %s" % np.unique(np.argwhere(bad)[:, 0])[:20]
        assert (np.abs(got_lse[:n] - lse[:n]) <= tol_lse[:n]).all()
        if n:
            assert np.linalg.norm(got[:n] - ref[:n]) <= norm * np.linalg.norm(ref[:n])
        assert self.lib.get_error(self.ws) == status
        return self


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


EDGES = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_lengths(lib, ps, fp8):
    """Chunks about every block and tile edge, with nothing and with something cached."""
    ctx = [0] * len(EDGES) + [(37 * i) % 200 for i in range(len(EDGES))]
    Case(lib, ctx, EDGES * 2, heads=2, ps=ps, fp8=fp8, seed=ps).run().check()


@pytest.mark.parametrize("ps", [32, 128])
def test_context_lengths(lib, ps):
    ctx = [0, 1, 15, 16, 17, 100, 126, 127, 128, 129, 240, 255, 256, 257, 383, 384, 385, 1000]
    Case(lib, ctx, [3] * len(ctx), heads=3, ps=ps, seed=ps).run().check()


@pytest.mark.parametrize("heads", [1, 2, 5, 16, 33, 128])
def test_head_counts(lib, heads):
    Case(lib, [70, 0, 300], [40, 1, 131], heads=heads, seed=heads).run().check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 127, 128, 129, 200, 500, 100000])
@pytest.mark.parametrize("fp8", [False, True])
def test_windows(lib, window, fp8):
    Case(lib, [0, 5, 130, 700, 411], [300, 1, 257, 140, 3], heads=2, window=window, fp8=fp8, seed=window).run().check()


def test_window_beyond_the_length_is_none(lib):
    a = Case(lib, [200, 0], [150, 300]).run()
    b = Case(lib, [200, 0], [150, 300])
    b.window = 10000
    b.run()
    assert torch.equal(bits(a.out), bits(b.out)) and torch.equal(bits(a.lse), bits(b.lse))


@pytest.mark.parametrize("q_std,norm", [(6.0, 3e-2), (0.0, 6e-3)])
@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_and_equal_scores(lib, q_std, norm, fp8):
    """Scores of standard deviation 6 (their key roundings weigh six times as much); equal scores give the mean."""
    c = Case(lib, [400, 0], [200, 140], heads=4, q_std=q_std, fp8=fp8).run().check(norm)
    if q_std == 0.0:
        i = np.arange(200) + 401
        assert np.abs(f64(c.lse)[:200] - np.log(i)[:, None]).max() <= 1e-6 * np.log(600)


def test_growing_scores_move_the_reference_maximum(lib):
    """Keys whose scores climb by hundreds along the positions: O is rescaled at every step."""
    c = Case(lib, [0], [700], heads=2, q_std=1.0)
    ramp = torch.linspace(0, 60, 700, device="cuda")
    flat = c.pool.data[1].view(-1, 576)
    at = torch.arange(700, device="cuda")
    slots = c.table[0].long()[at // c.ps] * c.ps + at % c.ps
    flat[slots, 512:] = 0
    flat[slots, 512] = ramp.to(torch.bfloat16)
    c.q[:, :, 128:] = 0
    c.q[:, :, 128] = 60.0
    c.run().check()


def test_many_requests(lib):
    rng = np.random.default_rng(3)
    n = 700
    ctx = rng.integers(0, 90, n).tolist()
    new = rng.integers(0, 4, n).tolist()
    Case(lib, ctx, new, heads=1, ps=16).run().check()


@pytest.mark.parametrize("ctx,new,heads,window,fp8", [
    ([9000], [1], 2, 0, False), ([9000], [130], 1, 0, True), ([5000], [256], 2, 0, False), ([7000], [257], 2, 0, False),
    ([3000], [512], 3, 0, False), ([6000], [700], 2, 0, True), ([4000, 100, 2500], [20, 300, 513], 1, 0, False),
    ([6000, 50], [300, 10], 2, 2500, False), ([0], [2500], 1, 0, False)])
def test_few_items_are_cut_along_the_keys(lib, ctx, new, heads, window, fp8):
    """Tiles whose keys several clusters share: all partial sums joined, rows before a piece's keys among them."""
    c = Case(lib, ctx, new, heads=heads, window=window, fp8=fp8).run().check()
    assert int(c.ws[:20].view(torch.int32)[4]) > 0 or heads * len(ctx) > 2  # (tiles were split)
    out = c.out.clone()
    c.run()
    assert torch.equal(bits(c.out), bits(out))  # the same order of sums each time
    b = Case(lib, ctx, new, heads=heads, window=window, fp8=fp8, heads_per_pass=1).run().check()
    assert b.T == c.T


def test_nan_in_cut_tiles(lib):
    args = dict(ctx=[8000], new=[140], heads=1)
    a = Case(lib, **args).run()
    b = Case(lib, **args)
    pos = 8050
    b.pool.data[1].view(-1, 576)[int(b.table[0, pos // b.ps]) * b.ps + pos % b.ps, 9] = float("nan")
    b.run()
    assert torch.isnan(b.out[50:140].float()).all() and torch.equal(bits(a.out[:50]), bits(b.out[:50]))

def test_no_new_tokens_and_empty_batch(lib):
    c = Case(lib, [10, 50], [0, 0]).run().check()
    assert (c.out == 7).all()
    c = Case(lib, [], [], extra_rows=0).run()
    Case(lib, [10, 50, 3], [0, 7, 0]).run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_csr_without_a_page(lib, fp8):
    """Requests without tokens, cached or new, and an empty list of ids; where one has tokens it is refused."""
    c = Case(lib, [0, 0], [0, 0], csr=True, fp8=fp8).run().check()
    assert c.ids.numel() == 0 and (c.out == 7).all()
    c = Case(lib, [0, 0], [0, 3], csr=True, fp8=fp8)
    c.ids = c.ids[:0]
    c.run()
    assert torch.isnan(c.out[:3].float()).all() and (c.out[3:] == 7).all()
    assert lib.get_error(c.ws) == lib.STATUS_BAD_LENGTH


@pytest.mark.parametrize("fp8", [False, True])
def test_csr_lists_equal_block_tables(lib, fp8):
    a = Case(lib, [333, 0, 12], [100, 300, 1], fp8=fp8).run()
    b = Case(lib, [333, 0, 12], [100, 300, 1], fp8=fp8, csr=True).run()
    assert torch.equal(bits(a.out), bits(b.out)) and torch.equal(bits(a.lse), bits(b.lse))


@pytest.mark.parametrize("per_pass", [1, 2, 3, 4, 5])
def test_heads_per_pass_change_nothing(lib, per_pass):
    a = Case(lib, [333, 0, 12], [100, 300, 1], heads=5).run().check()
    b = Case(lib, [333, 0, 12], [100, 300, 1], heads=5, heads_per_pass=per_pass).run()
    assert torch.equal(bits(a.out), bits(b.out)) and torch.equal(bits(a.lse), bits(b.lse))


def test_twice_the_same_and_spare_capacity_and_no_lse(lib):
    a = Case(lib, [500, 64], [300, 257], heads=6).run()
    out = a.out.clone()
    a.out.fill_(7.0)
    a.run(lse=None)
    assert torch.equal(bits(a.out), bits(out))
    b = Case(lib, [500, 64], [300, 257], heads=6, spare_kv=5000).run()
    assert torch.equal(bits(b.out), bits(out))


def test_page_order_and_other_layers_do_not_matter(lib):
    a = Case(lib, [200, 90], [100, 60]).run()
    b = Case(lib, [200, 90], [100, 60])
    perm = torch.randperm(b.num_pages, device="cuda")
    moved = torch.empty_like(b.pool.data)
    moved[:, perm] = b.pool.data
    moved[0] = float("nan")
    b.pool = lib.KVPool(moved)
    b.table = torch.where(b.table >= 0, perm[b.table.clamp(min=0).long()].to(torch.int32), b.table)
    b.run()
    assert torch.equal(bits(a.out), bits(b.out))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 40])
def test_nan_that_nobody_attends_changes_nothing(lib, fp8, window):
    """NaN in spare pages, behind the last token, before the window, and in the queries behind the last request."""
    args = dict(ctx=[100, 21, 300], new=[40, 5, 150], heads=2, fp8=fp8, window=window)
    a = Case(lib, **args).run()
    b = Case(lib, **args)
    used = torch.zeros(b.num_pages * b.ps, dtype=torch.bool, device="cuda")
    for r, (c, n) in enumerate(zip(args["ctx"], args["new"])):
        at = torch.arange(max(0, c + 1 - window) if window else 0, c + n, device="cuda")
        used[b.table[r].long()[at // b.ps] * b.ps + at % b.ps] = True
    flat = b.pool.data[1].view(-1, 576)
    flat[~used] = 0x7F if fp8 else float("nan")
    b.q[int(b.indptr[-1]):] = float("nan")
    b.run()
    assert torch.equal(bits(a.out), bits(b.out)) and torch.equal(bits(a.lse), bits(b.lse))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [3, 511])
@pytest.mark.parametrize("window", [0, 30])
def test_nan_reaches_the_rows_that_attend_it_only(lib, value, dim, window):
    """A bad c_kv row of a new token: the rows before it (causal) and, with a window, far behind it stay as they were."""
    args = dict(ctx=[70, 200], new=[140, 30], heads=2, window=window)
    a = Case(lib, **args).run()
    b = Case(lib, **args)
    pos = 70 + 50  # token 50 of request 0
    flat = b.pool.data[1].view(-1, 576)
    flat[int(b.table[0, pos // b.ps]) * b.ps + pos % b.ps, dim] = value
    b.run()
    hit = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    hit[50:50 + window if window else 140] = True
    assert torch.isnan(b.out[hit].float()).all()
    assert torch.equal(bits(a.out[~hit]), bits(b.out[~hit]))


def test_infinite_rope_value_of_weight_zero(lib):
    """-inf as a score is a weight of zero: a rope value of -inf against a positive query."""
    c = Case(lib, [90], [20], heads=2)
    c.q[:, :, 128:] = 0
    c.q[:, :, 130] = 1.0
    pos = 33
    c.pool.data[1].view(-1, 576)[int(c.table[0, pos // c.ps]) * c.ps + pos % c.ps, 514] = -float("inf")
    c.run().check()


def test_bad_pages_read_as_zero(lib):
    c = Case(lib, [100, 60], [30, 10], ps=16)
    good = c.table.clone()
    c.table[0, 2] = c.num_pages
    c.table[1, 0] = -5
    c.run()
    assert c.lib.get_error(c.ws, clear=True) == c.lib.STATUS_BAD_PAGE
    got = c.out.clone()
    c.table = good
    flat = c.pool.data[1]
    flat[good[0, 2].long()] = 0
    flat[good[1, 0].long()] = 0
    c.run().check()
    assert torch.equal(bits(got), bits(c.out))


@pytest.mark.parametrize("csr", [False, True])
def test_bad_lengths_give_nan_rows_of_their_request_alone(lib, csr):
    args = dict(ctx=[100, 60, 30, 9], new=[30, 10, 300, 2], csr=csr)
    a = Case(lib, **args).run()
    b = Case(lib, **args)
    b.ctx[0] = -1
    b.ctx[2] = 400  # 700 tokens do not fit the 330 of its pages
    b.run()
    assert lib.get_error(b.ws) == lib.STATUS_BAD_LENGTH
    bad = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    bad[0:30] = True
    bad[40:340] = True
    assert torch.isnan(b.out[bad].float()).all() and torch.isnan(b.lse[bad]).all()
    assert torch.equal(bits(a.out[~bad]), bits(b.out[~bad]))


def test_capacity_below_the_lengths(lib):
    """max_kv_tokens too small: the requests that do not fit are NaN, the others right."""
    c = Case(lib, [100, 60], [30, 10])
    a = Case(lib, [100, 60], [30, 10]).run()
    c.max_kv = 130
    c.ctx[1] = 118  # fits its pages' 128, not the rows left
    c.run()
    assert lib.get_error(c.ws) == lib.STATUS_BAD_LENGTH
    assert torch.equal(bits(c.out[:30]), bits(a.out[:30])) and torch.isnan(c.out[30:40].float()).all()


def test_row_pointers_outside_the_queries(lib):
    c = Case(lib, [100, 60, 5], [30, 10, 4], extra_rows=0)
    a = Case(lib, [100, 60, 5], [30, 10, 4], extra_rows=0).run()
    c.indptr[2] = c.T + 100   # request 1 ends, request 2 starts outside
    c.run()
    assert lib.get_error(c.ws) == lib.STATUS_BAD_LENGTH
    assert torch.equal(bits(c.out[:30]), bits(a.out[:30])) and (c.out[30:] == 7).all()


def test_graph_replay_with_changed_lengths(lib):
    """A captured call of fixed capacity, replayed with other lengths, tables and chunk splits."""
    rng = np.random.default_rng(5)
    B, T, most = 6, 400, 2500
    c = Case(lib, [400] * B, [20] * B, heads=3, ps=32, extra_rows=T - 20 * B)
    c.max_kv = most
    c.ws = lib.alloc_prefill_workspace(B, T, most, 3)
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.prefill(c.pool, 1, c.q, c.indptr, c.ctx, c.scale, c.w_uk, c.w_uv, c.ws, c.out, most, block_table=c.table,
                    lse=c.lse)
    for _ in range(4):
        new = rng.multinomial(rng.integers(1, T), np.ones(B) / B)
        new[rng.integers(0, B)] = 0
        ctx = [int(rng.integers(0, 420 - n)) if n < 420 else 0 for n in new]
        c.indptr.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
        c.ctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        c.q.normal_()
        c.q.copy_(c.q)
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("heads,ctx,new,window,fp8", [
    (16, [4000, 3000, 5000, 100, 2000], [1, 64, 7, 300, 65], 0, False),
    (16, [4000, 3000, 5000, 100, 2000], [1, 64, 9, 300, 65], 0, True),
    (16, [9000, 63, 64, 0, 4000], [8, 1, 64, 40, 16], 0, False),
    (16, [9000, 3000, 4500, 0, 4000], [33, 700, 5, 64, 2], 3500, False),
    (16, [9000, 3000, 4500, 5000, 200], [33, 12, 5, 64, 2], 70, False),
    (32, [2500, 1, 3900], [10, 64, 3], 0, False),
    (64, [1100, 2100], [5, 64], 0, True),
    (128, [900, 800, 10], [3, 130, 64], 0, False),
    (128, [1700], [1], 0, False),
    (16, [4000, 2935, 2935, 2967, 5000], [56, 32, 33, 33, 57], 0, True),
    (16, [4000, 9000, 5000], [56, 50, 32], 2900, False),
    (64, [3300], [50], 0, False),
    (64, [60, 0, 17, 100, 64, 63, 200], [1, 1, 2, 9, 1, 1, 1], 0, True),
    (128, [1000], [5], 600, False)])
def test_small_requests_in_the_latent_space(lib, heads, ctx, new, window, fp8):
    """Few new tokens over long caches, alone and beside chunks; every token group, partly filled ones among them."""
    c = Case(lib, ctx, new, heads=heads, window=window, fp8=fp8, seed=heads, spare_kv=0 if not window else 20000)
    assert c.latent()
    c.run().check()
    assert int(c.ws[:32].view(torch.int32)[7]) > 0
    out = c.out.clone()
    c.run()
    assert torch.equal(bits(out), bits(c.out))


def test_small_requests_with_csr_and_passes_and_no_lse(lib):
    args = dict(ctx=[4500, 3000, 5000, 100], new=[1, 64, 7, 300], heads=16)
    a = Case(lib, **args).run().check()
    b = Case(lib, **args, csr=True, heads_per_pass=3)
    assert a.latent()
    b.run(lse=None)
    # (requests 0 and 2 are attended in the latent space; 64 and 300 tokens' keys may be cut elsewhere with other heads a pass)
    for r in (slice(0, 1), slice(65, 72)):
        assert torch.equal(bits(a.out[r]), bits(b.out[r]))
    assert (b.lse == 7).all()
    b.run().check()


def test_many_small_requests_past_the_room_for_them(lib):
    """More groups than the latent form has room for: the others are expanded."""
    n = 1100
    new = [1 + (i % 7 == 0) for i in range(n)]
    c = Case(lib, [11] * n, new, heads=16, ps=16, extra_rows=2)
    assert c.latent()
    c.run()
    assert int(c.ws[:32].view(torch.int32)[7]) == 2048  # (pairs of groups, a pair a request: 1,024 of the 1,100)
    vals, table, m = c.values(), c.table.cpu().numpy(), sum(new)
    tols = []
    for form in (lambda n, m: True, lambda n, m: False):  # (which requests are expanded is the plan's choice)
        ref, _, tol, _ = step_ref.prefill(lambda b, at: vals[table[b][at // c.ps], at % c.ps], f64(c.q),
                                          c.indptr.cpu().numpy(), c.ctx.cpu().numpy(), f64(c.w_uk), f64(c.w_uv),
                                          c.scale, 0, form)
        tols.append(tol)
    assert (np.abs(f64(c.out)[:m] - ref[:m]) <= np.maximum(*tols)[:m]).all()
    assert lib.get_error(c.ws) == 0


def test_nan_and_bad_requests_among_small_ones(lib):
    args = dict(ctx=[4000, 3000, 6000, 50], new=[6, 40, 64, 20], heads=16)
    a = Case(lib, **args).run()
    b = Case(lib, **args)
    pos = 3000 + 20
    b.pool.data[1].view(-1, 576)[int(b.table[1, pos // b.ps]) * b.ps + pos % b.ps, 77] = float("nan")
    used = torch.zeros(b.num_pages, dtype=torch.bool, device="cuda")
    used[b.table[b.table >= 0].long()] = True
    b.pool.data[1][~used] = float("nan")
    b.run()
    hit = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    hit[6 + 20:6 + 40] = True
    assert torch.isnan(b.out[hit].float()).all()
    assert torch.equal(bits(a.out[~hit]), bits(b.out[~hit])) and lib.get_error(b.ws) == 0
    c = Case(lib, **args)
    c.ctx[3] = 5000  # more than its pages hold
    ref, _, tol, _ = a.reference()
    c.run()
    assert lib.get_error(c.ws) == lib.STATUS_BAD_LENGTH
    assert torch.isnan(c.out[110:130].float()).all() and (np.abs(f64(c.out) - ref) <= tol)[:110].all()


def test_graph_replay_of_mixed_steps(lib):
    """A captured call whose requests change between small and large, present and absent."""
    rng = np.random.default_rng(6)
    B, T, H, most = 5, 500, 16, 16000
    c = Case(lib, [3000] * B, [40] * B, heads=H, ps=64, extra_rows=T - 40 * B)
    c.max_kv = most
    c.ws = lib.alloc_prefill_workspace(B, T, most, H)
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.prefill(c.pool, 1, c.q, c.indptr, c.ctx, c.scale, c.w_uk, c.w_uv, c.ws, c.out, most, block_table=c.table,
                    lse=c.lse)
    for new in ([1, 1, 1, 1, 1], [300, 0, 64, 65, 3], [0, 0, 0, 0, 0], [0, 400, 0, 0, 1], [20, 30, 40, 50, 60]):
        ctx = [int(rng.integers(0, 3040 - n)) for n in new]
        c.indptr.copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
        c.ctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.check()

@pytest.mark.parametrize("heads,ctx,new,fp8,latent", [
    (16, [4000, 3500, 9000], [20, 1, 55], False, True), (128, [4000], [3], False, True), (32, [4000, 3100], [40, 9], True, True),
    (2, [4000, 500], [300, 64], False, False), (16, [3000], [200], True, False)])
def test_nearly_as_exact_as_the_results_own_rounding(lib, heads, ctx, new, fp8, latent):
    """Normal values, scores of standard deviation 1. Rounded to bf16, a value is off by 1.67e-3 (root mean square,
    taken from the reference itself below).
    Expanded, only the keys add to it: 128 of 192 products a score, so 1.67e-3 sqrt(2 / 3) = 1.36e-3 of each weight,
    together sqrt(1.67^2 + 1.36^2) = 1.29 of the rounding. In the latent space the pair of queries leaves half of
    that, 0.7e-3, and the weights' two roundings 1.1e-3 / sqrt(2): 1.19. Bounded by 1.4 of it."""
    c = Case(lib, ctx, new, heads=heads, fp8=fp8, seed=7).run()
    assert (int(c.ws[:32].view(torch.int32)[7]) > 0) == latent
    ref, _, _, _ = c.reference()
    n = sum(new)
    own = f64(torch.from_numpy(ref[:n]).to(torch.bfloat16)) - ref[:n]
    assert np.linalg.norm(f64(c.out)[:n] - ref[:n]) <= 1.4 * np.linalg.norm(own)


def test_most_heads_and_a_workspace_cut_to_fit_half(lib):
    """1024 heads, at once and in two passes with a workspace sized for one head more than a pass has."""
    a = Case(lib, [40, 3], [20, 1], heads=1024).run().check()
    b = Case(lib, [40, 3], [20, 1], heads=1024, heads_per_pass=513)
    guard = torch.full((b.ws.numel() + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    guard[:256] = 0
    size = b.ws.numel()
    b.ws = guard[:size]
    b.run()
    assert torch.equal(bits(a.out), bits(b.out)) and bool((guard[size:] == 0x5a).all())


@pytest.mark.parametrize("heads,per_pass,new", [(2, 0, 1), (16, 2, 113)])
def test_rows_past_32_bit_offsets(lib, heads, per_pass, new):
    """A request behind one of 3.84 million tokens, whose gathered rows take 4.4 GB. The long one's pages are one
    page over and over, so that with one new token it is attention over that page's 128 rows."""
    long = 30000 * 128
    c = Case(lib, [200], [30], heads=heads, ps=128)
    one = Case(lib, [127], [1], heads=heads, ps=128)
    c.max_kv = long + 230
    ref, lse, tol, tol_lse = c.reference()
    one.pool, one.table = c.pool, c.table[:, 1:2].contiguous()
    one.w_uk, one.w_uv = c.w_uk, c.w_uv
    ref1, lse1, _, tol1 = one.reference()
    table = torch.empty(2, long // 128, dtype=torch.int32, device="cuda")
    table[0] = c.table[0, 1]
    table[1, :2] = c.table[0]
    c.q = torch.cat([one.q[:1].expand(new, heads, 192), c.q])
    c.T = c.q.shape[0]
    c.table, c.ctx = table, torch.tensor([long - new, 200], dtype=torch.int32, device="cuda")
    c.indptr = torch.tensor([0, new, new + 30], dtype=torch.int32, device="cuda")
    c.ws = lib.alloc_prefill_workspace(2, c.T, c.max_kv, heads, per_pass)
    c.out, c.lse = c.out.new_empty(c.T, heads, 128), c.lse.new_empty(c.T, heads)
    c.run()
    assert lib.get_error(c.ws) == 0
    assert (np.abs(f64(c.out[new:new + 30]) - ref[:30]) <= tol[:30]).all()
    assert (np.abs(f64(c.lse[new:new + 30]) - lse[:30]) <= tol_lse[:30]).all()
    # (the last row attends the page 30,000 times, in pieces of at most 400 steps: their sums add 400 2^-23 to its lse)
    got = f64(c.out[new - 1])
    assert np.linalg.norm(got - ref1[0]) <= 6e-3 * np.linalg.norm(ref1[0])
    assert (np.abs(f64(c.lse[new - 1]) - lse1[0] - np.log(30000)) <= tol1[0] + 400 * 2.0 ** -23).all()


def test_on_another_stream_beside_a_second_call(lib):
    """Two calls at once on two streams, each with a workspace of its own."""
    a = Case(lib, [500, 64], [300, 257], heads=6, seed=1)
    b = Case(lib, [10, 640], [500, 57], heads=6, seed=2)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for c, stream in ((a, s), (b, t)):
            lib.prefill(c.pool, 1, c.q, c.indptr, c.ctx, c.scale, c.w_uk, c.w_uv, c.ws, c.out, c.max_kv,
                        block_table=c.table, lse=c.lse, stream=stream)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_equals_the_absorbed_path(lib, fp8):
    """decode_q on absorbed queries followed by uv_project computes the same; each is within its tolerance (1e-2 and
    4e-2 of the largest value for the absorbed form, whose queries are rounded to bf16 as well)."""
    H, n = 16, 5
    c = Case(lib, [300, 77, 0], [n] * 3, heads=H, fp8=fp8, extra_rows=0).run()
    q = c.q.view(3, n, H, 192).float()
    q_abs = torch.cat([torch.einsum("bnhd,hdc->bnhc", q[..., :128], c.w_uk.float()), q[..., 128:]], -1)
    ws = lib.alloc_workspace_q(3, n, H)
    lat = torch.empty(3, n, H, 512, dtype=torch.bfloat16, device="cuda")
    lib.plan_q(c.ctx, n, H, c.ps, 0, ws)
    lib.decode_q(c.pool, 1, q_abs.to(torch.bfloat16), c.ctx, c.scale, ws, lat, block_table=c.table)
    y = torch.empty(3 * n, H, 128, dtype=torch.bfloat16, device="cuda")
    lib.uv_project(lat.view(3 * n, H, 512), c.w_uv, y)
    torch.cuda.synchronize()
    assert np.abs(f64(y) - f64(c.out)).max() <= (5e-2 if fp8 else 2e-2) * np.abs(f64(y)).max()


def test_refusals(lib):
    c = Case(lib, [100, 60], [30, 10])
    call = lambda **k: lib.prefill(**{**dict(  # noqa: E731
        pool=c.pool, layer=1, q=c.q, q_indptr=c.indptr, context_lens=c.ctx, softmax_scale=c.scale, w_uk=c.w_uk,
        w_uv=c.w_uv, workspace=c.ws, out=c.out, max_kv_tokens=c.max_kv, block_table=c.table), **k})
    for bad in [dict(q=c.q[:, :, :128]), dict(q=c.q.float()), dict(q=c.q[:, ::2]), dict(out=c.out[:5]),
                dict(lse=c.lse[:5]), dict(q_indptr=c.indptr[:2]), dict(w_uk=c.w_uv), dict(w_uv=c.w_uk),
                dict(block_table=None), dict(block_table=c.table[:1]), dict(context_lens=c.ctx.long())]:
        with pytest.raises(ValueError):
            call(**bad)
    for bad in [dict(layer=2), dict(window=-1), dict(softmax_scale=0.0), dict(workspace=c.ws[:4096]),
                dict(max_kv_tokens=10 * c.max_kv + 5000), dict(max_kv_tokens=-1), dict(workspace=c.ws[8:])]:
        with pytest.raises(lib.MlaError):
            call(**bad)
    torch.cuda.synchronize()
    assert (c.out == 7).all()
