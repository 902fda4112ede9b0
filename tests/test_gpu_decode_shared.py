"""decode_shared against its definition in 64 bits: each request over all its positions
by its own pages, whatever is shared."""
import math

import pytest
import torch

from shared_ref import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def run(lib, c, clusters=0, csr=False, ws=None, out=None, lse=None, plan=True, stream=None):
    ws = lib.alloc_workspace_shared(c.batch, c.q_len, c.heads, c.prefix.numel()) if ws is None else ws
    out = torch.full((c.batch, c.q_len, c.heads, 512), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((c.batch, c.q_len, c.heads), 7.0, device="cuda") if lse is None else lse
    if plan:
        lib.plan_shared(c.ctx, c.indptr, c.prefix, c.q_len, c.heads, c.page, ws, num_clusters=clusters, stream=stream)
    kw = dict(block_table=c.table)
    if csr:
        n = [(int(x) + c.q_len + c.page - 1) // c.page for x in c.ctx]
        ids = torch.cat([c.table[b, :k] for b, k in enumerate(n)])
        ptr = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        kw = dict(page_indptr=ptr, page_ids=ids.contiguous())
    lib.decode_shared(lib.KVPool(c.pool, c.scale), c.layer, c.q, c.prefix.numel(), c.softmax_scale, ws, out, lse=lse,
                      stream=stream, **kw)
    return out, lse, ws


def verify(lib, c, **kw):
    out, lse, ws = run(lib, c, **kw)
    torch.cuda.synchronize()
    assert lib.get_error(ws) == 0
    check(c, out, lse)
    pads = [b for b in range(c.batch) if b not in c.real()]
    assert bool((out[pads] == 7).all()) and bool((lse[pads] == 7).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("page", [16, 64])
def test_prefix_lengths(lib, fp8, prefix, page):
    verify(lib, Case([(5, prefix)], [0, 1, 40, 127, 130], page=page, fp8=fp8, seed=prefix))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [1, 3, 16, 24, 48, 64, 128, 200, 256, 300])
def test_heads(lib, fp8, heads):
    verify(lib, Case([(7, 150)], [3, 77, 200, 0, 31, 64, 129], heads=heads, page=32, fp8=fp8, seed=heads))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,heads", [(2, 16), (3, 32), (5, 64), (2, 128), (3, 128), (17, 16), (130, 4)])
def test_several_query_positions(lib, fp8, q_len, heads):
    verify(lib, Case([(3, 100), (2, 200)], [3, 130, 0, 64, 127], heads=heads, q_len=q_len, page=64, fp8=fp8, seed=q_len))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups", [[(1, 50)], [(1, 0), (1, 9)], [(0, 10), (3, 70), (0, 5), (1, 33), (2, 0), (4, 200), (0, 0)],
                                    [(2, 20)] * 20, [(40, 333), (3, 1), (40, 64)]])
def test_groups(lib, fp8, groups):
    n = sum(k for k, _ in groups)
    verify(lib, Case(groups, [(37 * i) % 150 for i in range(n)], page=16, fp8=fp8, seed=n, before=2, after=3))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("clusters", [1, 2, 3, 7, 20, 0])
@pytest.mark.parametrize("page", [16, 128])
def test_schedules(lib, fp8, clusters, page):
    verify(lib, Case([(20, 700), (9, 1100)], [(91 * i) % 400 for i in range(29)], heads=32, page=page, fp8=fp8), clusters=clusters)


@pytest.mark.parametrize("fp8", [False, True])
def test_page_lists(lib, fp8):
    c = Case([(6, 210), (3, 40)], [5, 90, 0, 33, 64, 100, 7, 8, 9], heads=24, page=32, fp8=fp8)
    a, la, ws = run(lib, c)
    b, lb, ws2 = run(lib, c, csr=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert lib.get_error(ws) == 0 and lib.get_error(ws2) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prefix(lib, fp8):
    verify(lib, Case([(6, 20011)], [0, 700, 1, 130, 64, 1000], heads=128, page=64, fp8=fp8))


def test_large_batch(lib):
    verify(lib, Case([(500, 130), (400, 64), (311, 0)], [(7 * i) % 90 for i in range(1211)], heads=8, page=16))


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_softmax(lib, fp8):
    verify(lib, Case([(9, 900)], [200, 3, 0, 500, 64, 64, 1, 2, 300], heads=16, page=64, fp8=fp8, q_std=4.0))


def test_rising_scores(lib):
    """Each position's score above all before it: the running maximum moves with every block."""
    c = Case([(4, 1500)], [300, 0, 77, 128], heads=16, page=64)
    ramp = torch.zeros(512, device="cuda")
    ramp[0] = 1.0
    for b in c.real():
        n = int(c.ctx[b]) + 1
        for t0 in range(0, n, c.page):
            j = int(c.full[b, t0 // c.page])
            t = torch.arange(t0, t0 + c.page, device="cuda")
            for pool in (c.clean, c.pool):
                pool[c.layer, j, :, 0] = (t / 16.0).to(torch.bfloat16)
    c.pool[c.layer][~c.used] = math.nan
    c.q[..., 0] = 16.0
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("heads", [16, 128])
def test_a_requests_nan_stays_its_own(lib, heads):
    c = Case([(6, 200)], [30, 140, 0, 65, 7, 300], heads=heads, page=16)
    want, want_lse, _ = run(lib, c)
    hurt = {1: math.nan, 3: math.inf, 4: -math.inf}
    for b, x in hurt.items():
        t = int(c.ctx[b]) - 2
        c.pool[c.layer, int(c.full[b, t // c.page]), t % c.page, 40] = x
        if b == 1:
            c.pool[c.layer, int(c.full[b, t // c.page]), t % c.page] = x
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == 0
    for b in range(c.batch):
        if b not in hurt:
            assert torch.equal(out[b], want[b]) and torch.equal(lse[b], want_lse[b])
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())


def test_a_later_querys_row_stays_unseen(lib):
    """Of several query positions the earlier ones do not see the later ones' rows."""
    c = Case([(3, 100)], [30, 125, 64], heads=32, q_len=4, page=16)
    want, want_lse, _ = run(lib, c)
    for b in range(3):
        t = int(c.ctx[b]) + 2
        c.pool[c.layer, int(c.full[b, t // c.page]), t % c.page] = math.nan
    out, lse, _ = run(lib, c)
    assert torch.equal(out[:, :2], want[:, :2]) and torch.equal(lse[:, :2], want_lse[:, :2])
    assert bool(out[:, 2:].isnan().all()) and bool(lse[:, 2:].isnan().all())


def test_same_as_decode(lib):
    """On batches that share nothing, and next to mla_decode on the same tables."""
    c = Case([(6, 256)], [30, 140, 0, 65, 7, 300], heads=16, page=64)
    out, lse, _ = run(lib, c)
    pool = lib.KVPool(c.clean, c.scale)
    ws = lib.alloc_workspace(c.batch, c.heads)
    plain, plain_lse = torch.empty_like(out[:, 0]), torch.empty_like(lse[:, 0])
    lib.plan(c.ctx, c.heads, c.page, 0, ws)
    lib.decode(pool, c.layer, c.q[:, 0].contiguous(), c.ctx, c.softmax_scale, ws, plain, block_table=c.full, lse=plain_lse)
    assert (out[:, 0].float() - plain.float()).norm() <= 1e-2 * plain.float().norm()
    assert (lse[:, 0] - plain_lse).abs().max() <= 2e-3 * plain_lse.abs().max()


def test_prefix_longer_than_a_request(lib):
    """The prefix ends where the shortest request's cached tokens do."""
    c = Case([(4, 64)], [0, 30, 200, 9], heads=16, page=16)
    longer = c.prefix + 50  # (request 0 has 64 cached)
    c.prefix = longer
    verify(lib, c)


def test_same_bits_again(lib):
    c = Case([(20, 700), (9, 1100)], [(91 * i) % 400 for i in range(29)], heads=32, page=32)
    a, la, ws = run(lib, c)
    for _ in range(3):
        b, lb, _ = run(lib, c, ws=ws, plan=False)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_pages_and_lengths(lib):
    c = Case([(3, 64)], [20, 40, 33], heads=16, page=16)
    good, good_lse, _ = run(lib, c)
    c.table[1, 5] = 1 << 20  # positions 80 .. 95 of request 1
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == lib.STATUS_BAD_PAGE
    rows = c.rows(1)
    rows[80:96] = 0
    ref, ref_lse, bound, lse_bound = c.reference(1, rows)
    assert bool(((out[1].double() - ref).abs() <= bound).all()) and bool(((lse[1].double() - ref_lse).abs() <= lse_bound).all())
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    # a table too narrow for a length
    c = Case([(3, 64)], [20, 40, 33], heads=16, page=16)
    c.table = c.table[:, :6].contiguous()
    _, _, ws = run(lib, c)
    assert lib.get_error(ws, clear=True) == lib.STATUS_BAD_PAGE
    # lengths out of range count as none
    c = Case([(1, 0), (1, 0), (1, 0)], [20, 0, 33], heads=16, page=16)
    for bad in (-5, 1 << 29, (1 << 31) - 1):
        c2 = c.ctx.clone()
        c2[1] = bad
        saved, c.ctx = c.ctx, c2
        out, lse, ws = run(lib, c)
        c.ctx = saved
        assert lib.get_error(ws) == lib.STATUS_BAD_LENGTH
        check(c, out, lse)
    # groups out of order
    for ptr in ([0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 2, 4]):
        c.indptr = torch.tensor(ptr, dtype=torch.int32, device="cuda")
        out, lse, ws = run(lib, c)
        assert lib.get_error(ws) == lib.STATUS_BAD_LENGTH
        assert bool((out == 7).all()) and bool((lse == 7).all())


def test_plan_of_another_call(lib):
    c = Case([(3, 64)], [20, 40, 33], heads=16, page=16)
    _, _, ws = run(lib, c)
    out = torch.full((c.batch, 1, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    d = Case([(2, 64), (1, 64)], [20, 40, 33], heads=16, page=16)
    big = torch.zeros(lib.workspace_size_shared(c.batch, 1, 16, 2), dtype=torch.uint8, device="cuda")
    run(lib, d, ws=big, out=out, plan=False)  # no plan at all
    assert lib.get_error(big, clear=True) == lib.STATUS_PLAN_MISMATCH
    run(lib, c, ws=big)
    run(lib, d, ws=big, out=out, plan=False)
    assert lib.get_error(big, clear=True) == lib.STATUS_PLAN_MISMATCH
    assert bool((out == 7).all())


def test_empty_calls(lib):
    c = Case([(0, 64)], [0], heads=16, page=16, after=2)
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == 0 and bool((out == 7).all())


def test_without_lse(lib):
    c = Case([(3, 64), (4, 900)], [20, 40, 33, 5, 6, 7, 400], heads=16, page=16)
    out, lse, ws = run(lib, c)
    out2 = torch.zeros_like(out)
    lib.decode_shared(lib.KVPool(c.pool), c.layer, c.q, 2, c.softmax_scale, ws, out2, block_table=c.table)
    assert torch.equal(out, out2)


def test_replayed_with_other_lengths(lib):
    """Plan and decode captured once; replayed with other lengths, groups and pad requests."""
    cases = [Case([(5, 333), (4, 80)], [(41 * i + k) % 200 for i in range(9)], heads=32, page=32, seed=k) for k in range(3)]
    cases.append(Case([(2, 100), (3, 17)], [9, 130, 0, 64, 65], heads=32, page=32, seed=9, before=1, after=3))
    width = max(c.table.shape[1] for c in cases)
    pages = max(c.pool.shape[1] for c in cases)
    z = cases[0]
    pool = torch.zeros(2, pages, 32, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((9, width), -1, dtype=torch.int32, device="cuda")
    ctx, indptr, prefix, q = z.ctx.clone(), z.indptr.clone(), z.prefix.clone(), z.q.clone()
    ws = lib.alloc_workspace_shared(9, 1, 32, 2)
    out, lse = torch.zeros(9, 1, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 1, 32, device="cuda")

    def load(c):
        pool[:, :c.pool.shape[1]] = c.pool
        table.fill_(-1)
        table[:, :c.table.shape[1]] = c.table
        for a, b in ((ctx, c.ctx), (indptr, c.indptr), (prefix, c.prefix), (q, c.q)):
            a.copy_(b)
        out.fill_(7)
        lse.fill_(7)

    def step():
        lib.plan_shared(ctx, indptr, prefix, 1, 32, 32, ws)
        lib.decode_shared(lib.KVPool(pool), 1, q, 2, z.softmax_scale, ws, out, block_table=table, lse=lse)

    load(z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c in cases + cases[:1]:
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        assert lib.get_error(ws) == 0
        check(c, out, lse)
        pads = [b for b in range(9) if b not in c.real()]
        assert bool((out[pads] == 7).all())


def test_two_streams_with_workspaces_of_their_own(lib):
    a = Case([(12, 900)], [(41 * i) % 200 for i in range(12)], heads=32, page=32, seed=1)
    b = Case([(7, 500), (3, 900)], [(51 * i) % 300 for i in range(10)], heads=16, page=16, seed=2, fp8=True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [run(lib, c, stream=s) for _ in range(3) for c, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for c, (out, lse, ws) in zip((a, b) * 3, got):
        assert lib.get_error(ws) == 0
        check(c, out, lse)


def test_refusals(lib):
    c = Case([(3, 64)], [20, 40, 33], heads=16, page=16)
    out, lse, ws = run(lib, c)
    pool = lib.KVPool(c.pool)
    ok = dict(q=c.q, num_prefixes=1, softmax_scale=0.1, workspace=ws, out=out, block_table=c.table)

    def call(**kw):
        a = {**ok, **kw}
        lib.decode_shared(pool, a.pop("layer", 1), **a)

    call()
    for bad in (dict(q=c.q[:, 0]), dict(q=c.q.float()), dict(q=c.q.cpu()), dict(out=out[:2]), dict(lse=lse[:, :, :3]),
                dict(block_table=c.table[:2]), dict(block_table=None), dict(block_table=c.table.long()),
                dict(q=c.q.transpose(1, 2)), dict(out=out.float())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(layer=2), dict(layer=-1), dict(softmax_scale=0.0), dict(softmax_scale=math.nan),
                dict(workspace=ws[:1024]), dict(num_prefixes=-1), dict(workspace=ws[16:])):
        with pytest.raises(lib.MlaError):
            call(**bad)
    plan = dict(context_lens=c.ctx, prefix_indptr=c.indptr, prefix_lens=c.prefix, q_len=1, num_heads=16, page_size=16, workspace=ws)
    for bad in (dict(prefix_indptr=c.indptr[:1]), dict(context_lens=c.ctx.long()), dict(prefix_lens=c.prefix.cpu())):
        with pytest.raises(ValueError):
            lib.plan_shared(**{**plan, **bad})
    for bad in (dict(q_len=0), dict(num_heads=0), dict(num_heads=1025), dict(page_size=48), dict(workspace=ws[:4096]),
                dict(num_clusters=-1)):
        with pytest.raises(lib.MlaError):
            lib.plan_shared(**{**plan, **bad})
    with pytest.raises(lib.MlaError):
        lib.workspace_size_shared(-1, 1, 16, 1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,q_len", [(96, 1), (160, 1), (32, 3), (100, 1), (72, 2), (255, 1), (85, 3)])
@pytest.mark.parametrize("prefix,own", [(1500, 60), (130, 700)])
def test_requests_across_tiles(lib, fp8, heads, q_len, prefix, own):
    """Row counts of which a tile leaves some over: tiles filled up, or of whole requests."""
    c = Case([(7, prefix), (3, prefix // 2)], [own - 9 * b for b in range(7)] + [5, 0, own], heads=heads, q_len=q_len, page=32,
             fp8=fp8, seed=heads)
    verify(lib, c)
    _, _, ws = run(lib, c)
    r = heads * q_len
    if prefix == 1500:  # tiles: full ones
        assert int(ws.view(torch.int32)[8]) == -(-7 * r // 256) + -(-3 * r // 256)


@pytest.mark.parametrize("heads,q_len", [(1, 1), (16, 1), (32, 3), (128, 1), (160, 1), (128, 3)])
@pytest.mark.parametrize("groups,own", [([(9, 5000)], 300), ([(3, 100), (1, 900), (0, 5), (5, 64)], 1000), ([(1, 40000)], 0),
                                        ([(60, 2500)], 600), ([(2, 700)] * 30, 40), ([(8, 65536)], 100)])
@pytest.mark.parametrize("clusters", [0, 1, 5])
def test_schedule_has_each_position_once(lib, heads, q_len, groups, own, clusters):
    """The plan read back: tiles of all rows, their segments' positions, and each block of a
    tile in one item of one cluster, with partial sums of its own where there are several."""
    page, r = 32, heads * q_len
    copy = min(page, 64)
    which = [g for g, (k, _) in enumerate(groups) for _ in range(k)]
    ctx = [groups[g][1] + own * (7 * b % 11) // 11 for b, g in enumerate(which)]
    starts = [sum(k for k, _ in groups[:g]) for g in range(len(groups) + 1)]
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = lib.alloc_workspace_shared(len(ctx), q_len, heads, len(groups))
    lib.plan_shared(torch.tensor(ctx, **i32), torch.tensor(starts, **i32), torch.tensor([p for _, p in groups], **i32), q_len, heads,
                    page, ws, num_clusters=clusters)
    torch.cuda.synchronize()
    assert lib.get_error(ws) == 0
    head = ws[:256].view(torch.int32).tolist()
    num_clusters, num_tiles, num_items, num_split = head[7:11]
    most_tiles = len(ctx) * r // (256 // r * r if r <= 256 else 256) + min(len(groups), len(ctx))
    at, records = 256, []
    for size, count in ((32, len(groups)), (32, most_tiles), (32, most_tiles * (2 + (254 + r) // r)), (96, num_items)):
        records.append(ws[at:at + size * count].view(torch.int32).reshape(count, size // 4).tolist())
        at = -(-(at + size * count) // 256) * 256
    _, tiles, segments, items = records
    assert num_tiles <= most_tiles and 1 <= num_clusters and (clusters == 0 or num_clusters <= clusters)

    row = 0
    for row0, rows, seg0, segs, blocks, shared, *_ in tiles[:num_tiles]:
        assert row0 == row and 1 <= rows <= 256
        row += rows
        g = which[row0 // r]
        first, count = starts[g], groups[g][0]
        assert row <= (first + count) * r  # (of one group)
        prefix = groups[g][1] if count > 1 else 0
        assert shared == -(-prefix // 128)
        own_segments = segments[seg0:seg0 + segs]
        if prefix:
            assert own_segments.pop(0) == [first, 0, rows, 0, 0, 0, prefix, prefix]
        b, upto, done = row0 // r, 0, shared
        for owner, row_lo, row_hi, block0, tok0, tok_lo, tok_hi, base in own_segments:
            assert (owner, row_lo, block0, tok_lo, base) == (b, upto, done, prefix, ctx[b])
            assert row_hi == min((b + 1) * r - row0, rows)
            assert tok0 == prefix // copy * copy and tok_hi == ctx[b] + (row0 + row_hi - 1 - b * r) // heads + 1
            done += -(-(tok_hi - tok0) // 128)
            b, upto = b + 1, row_hi
        assert upto == rows and done == blocks
    assert row == len(ctx) * r

    parts, split, n = [], 0, 0
    for row0, rows, seg0, segs, blocks, shared, *_ in tiles[:num_tiles]:
        mine = []
        while n < num_items and items[n][4] == row0:
            mine.append(items[n])
            n += 1
        assert [i[0] for i in mine] + [blocks] == [0] + [i[1] for i in mine]
        split += len(mine) > 1
        for begin, end, part, _, _, item_rows, seg, seg_last, prefix_end, row_lo, row_hi, *rest in mine:
            assert begin < end and item_rows == rows and seg_last == seg0 + segs - 1 and prefix_end == shared
            assert (part >= 0) == (len(mine) > 1)
            parts += [part] if part >= 0 else []
            assert rest[5:] == segments[seg] and segments[seg][3] <= begin and (seg == seg_last or segments[seg + 1][3] > begin)
            last = max(k for k in range(seg0, seg0 + segs) if segments[k][3] < end)
            want = (0, rows) if begin < shared else (segments[seg][1], segments[last][2])
            assert (row_lo, row_hi) == want
    assert n == num_items and split == num_split and sorted(parts) == list(range(len(parts)))
    assert [i[3] for i in items] == sorted(i[3] for i in items) and items[-1][3] < num_clusters


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_aligned_to_16_bytes_only(lib, fp8):
    c = Case([(5, 300)], [5, 130, 0, 64, 127], heads=48, page=32, fp8=fp8, seed=4)
    want, _, _ = run(lib, c)
    room = torch.zeros(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    c.q = room[8:].view(c.q.shape).copy_(c.q)
    assert c.q.data_ptr() % 32 == 16
    verify(lib, c)
    assert torch.equal(run(lib, c)[0], want)
    with pytest.raises(lib.MlaError):
        c.q = room[4:-4].view(c.q.shape)
        run(lib, c)


@pytest.mark.parametrize("fp8", [False, True])
def test_pool_beyond_32_bit_offsets(lib, fp8):
    c = Case([(4, 700)], [5, 130, 0, 64], heads=32, page=128, fp8=fp8, seed=6, layers=1)
    want, _, _ = run(lib, c)
    n, pages = c.pool.shape[1], (1 << 32) // (128 * 576 * (1 if fp8 else 2)) + 200
    pool = torch.empty(1, pages, 128, 576, dtype=c.pool.dtype, device="cuda")
    pool[0, pages - n:] = c.pool[0]
    valid = (c.table >= 0) & (c.table < n)
    c.pool, c.table = pool, torch.where(valid, c.table + (pages - n), c.table)
    assert torch.equal(run(lib, c)[0], want)


def test_lengths_of_a_garbled_batch_stay_in_the_workspace(lib):
    """Every length the largest that counts: more blocks than 32 bits hold (plan alone)."""
    batch = 8192
    i32 = dict(dtype=torch.int32, device="cuda")
    size = lib.workspace_size_shared(batch, 1, 1, 1)
    room = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = room[:size]
    ws[:256].zero_()
    lib.plan_shared(torch.full((batch,), (1 << 29) - 1, **i32), torch.tensor([0, batch], **i32), torch.tensor([1000], **i32), 1, 1, 64,
                    ws)
    torch.cuda.synchronize()
    head = ws[:256].view(torch.int32).tolist()
    assert lib.get_error(ws) == 0 and head[8] == 32 and head[9] <= 32 + head[7]
    assert bool((room[size:] == 0x5A).all())
