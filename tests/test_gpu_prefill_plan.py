"""What the chunk attention's plan decides, read from the workspace's header, and calls that
its other tests do not make."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import Case, bits, f64

pytestmark = pytest.mark.gpu
CLUSTERS, PIECE_STEPS, LEAST_PIECE, WAVES = 76, 6, 3, 4


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def tiles(ctx, new, window):
    """(rows, key steps of 128) of each tile of 512 query rows."""
    out = []
    for c, n in zip(ctx, new):
        lo = max(0, c + 1 - window) if window else 0
        for i in range(0, n, 512):
            rows = min(512, n - i)
            end = c + i + 1 - lo
            begin = max(0, end - window) // 16 * 16 if window else 0
            out.append((rows, -(-(end + rows - 1 - begin) // 128)))
    return out


def split(ctx, new, heads, window):
    """Tiles that are cut along their keys, and the entries of all tiles: the least piece of P steps with which the pieces
    of all heads run in w waves, for the w that takes least, if that beats the whole tiles by a tenth."""
    t = tiles(ctx, new, window)
    total = sum(c + n for c, n in zip(ctx, new))  # (tiles are cut where there are more than six steps)
    if not len(t) * heads < WAVES * CLUSTERS or total <= 768:
        return 0, len(t)
    longest = max(s for _, s in t)
    least, per = 0.9 * max(longest + PIECE_STEPS, 1.1 * sum(s + PIECE_STEPS for _, s in t) * heads / CLUSTERS), 0
    for w in range(1, WAVES + 1):
        room = min(w * CLUSTERS // heads, 2 * CLUSTERS)
        fits = [p for p in range(LEAST_PIECE, max(longest, LEAST_PIECE) + 1) if sum(max(1, -(-s // p)) for _, s in t) <= room]
        if room > len(t) and fits and w * (fits[0] + PIECE_STEPS) < least and fits[0] < longest:
            least, per = w * (fits[0] + PIECE_STEPS), fits[0]
    pieces = [max(1, -(-s // per)) if per else 1 for _, s in t]
    assert sum(p * r for p, (r, _) in zip(pieces, t) if p > 1) <= 2 * CLUSTERS * 512 // heads  # (partial rows)
    return sum(p > 1 for p in pieces), sum(pieces)


@pytest.mark.parametrize("ctx,new,heads,window,some", [
    ([9000], [1], 2, 0, True), ([9000], [130], 1, 0, True), ([5000], [256], 2, 0, True), ([7000], [257], 2, 0, True),
    ([3000], [512], 3, 0, True), ([6000], [700], 2, 0, True), ([4000, 100, 2500], [20, 300, 513], 1, 0, True),
    ([6000, 50], [300, 10], 2, 2500, True), ([0], [2500], 1, 0, True), ([9000], [130], 70, 0, False),
    ([400], [300], 2, 0, False), ([6000], [600], 40, 0, False), ([100] * 30, [20] * 30, 8, 0, False)])
def test_tiles_are_cut_where_it_pays(lib, ctx, new, heads, window, some):
    c = Case(lib, ctx, new, heads=heads, window=window)
    assert not c.latent()
    c.run()
    header = c.ws[:32].view(torch.int32).tolist()
    want = split(ctx, new, heads, window)
    assert (want[0] > 0) == some and (header[4], header[2]) == want


def test_rows_before_the_first_request(lib):
    """q_indptr that starts behind row 0: the rows before it stay as they were, in both paths."""
    for heads, ctx, new in ((3, [100, 700], [40, 300]), (16, [9000, 4500], [5, 200])):
        a, b = (Case(lib, ctx, new, heads=heads) for _ in range(2))
        a.run()
        b.q = torch.cat([torch.full_like(b.q[:7], float("nan")), b.q])
        b.out, b.lse = (torch.cat([t[:1].expand(7, *t.shape[1:]), t]).contiguous() for t in (b.out, b.lse))
        b.T += 7
        b.indptr += 7
        b.ws = lib.alloc_prefill_workspace(len(ctx), b.T, b.max_kv, heads)
        b.run()
        assert torch.equal(bits(b.out[7:]), bits(a.out)) and torch.equal(bits(b.lse[7:]), bits(a.lse))
        assert (b.out[:7] == 7).all() and (b.lse[:7] == 7).all() and lib.get_error(b.ws) == 0


@pytest.mark.parametrize("n", [200, 300, 700])
def test_many_requests_each_of_its_own_scale(lib, n):
    """The plan in one launch with the gather and in two; values of one size or zero in each request, of many in all."""
    rng = np.random.default_rng(n)
    ctx, new = rng.integers(0, 60, n).tolist(), rng.integers(1, 4, n).tolist()
    c = Case(lib, ctx, new, heads=2, ps=16)
    c.w_uk.zero_()
    flat = c.pool.data[1].view(-1, 576)
    for b in range(n):
        at = torch.arange(ctx[b] + new[b], device="cuda")
        rows = c.table[b].long()[at // 16] * 16 + at % 16
        flat[rows, :512] *= 0.0 if b % 9 == 5 else 2.0 ** int(rng.integers(-40, 40))
    c.run().check()
    ref, got, start = c.reference()[0], f64(c.out), c.indptr.cpu().numpy()
    for b in range(n):
        r, g = ref[start[b]:start[b + 1]], got[start[b]:start[b + 1]]
        assert np.linalg.norm(g - r) <= 4e-3 * np.linalg.norm(r)  # (own rounding 1.67e-3 on average, half a step at most)
    # the same workspace again for values of usual sizes
    d = Case(lib, ctx, new, heads=2, ps=16)
    e = Case(lib, ctx, new, heads=2, ps=16)
    e.ws = c.ws
    d.run()
    e.run()
    assert torch.equal(bits(d.out), bits(e.out)) and torch.equal(bits(d.lse), bits(e.lse))


@pytest.mark.parametrize("window", [1, 2, 0])
def test_lse_of_rows_without_values(lib, window):
    """c_kv zero and queries zero: lse is the log of the number of attended positions, to the bounds of other rows."""
    c = Case(lib, [170, 60], [56, 300], heads=3, window=window, q_std=0.0)
    c.pool.data[1].view(-1, 576)[:, :512] = 0
    c.run().check()
    assert not c.out[:356].any()
