"""Chunk attention (prefill) far from values of size one and scores of a few units:
values of any scale, softmax weights far below a row's largest, infinite and large
scores, expanded and in the latent space alike."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import Case, bits, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def groups(c):
    """Row groups that the call attended in the latent space."""
    return int(c.ws[:32].view(torch.int32)[7])


def slot(c, b, pos):
    return int(c.table[b, pos // c.ps]) * c.ps + pos % c.ps


def check(c, norm=6e-3):
    """Case.check; the reference is made once and returned."""
    made = c.reference()
    c.reference = lambda: made
    c.check(norm)
    return made[0]


def exact_enough(c, ref, n, factor=1.4):
    """Nearly as exact as the result's own rounding to bf16 is: rows together, and no row far off by itself.

    The roundings that add to it (keys, or the latent path's pairs of queries and its weights) make it 1.29 times that in
    the norm over all rows (test_nearly_as_exact_as_the_results_own_rounding). One row's 128 values of a head share their
    weights' errors, of which few may count: their deviation is 1.36e-3, and six of it are 5 times the own rounding's
    1.67e-3, with the latter in all sqrt(5^2 + 1) = 5.1 times; 6 are allowed."""
    got = f64(c.out)[:n]
    own = f64(torch.from_numpy(ref[:n]).to(torch.bfloat16)) - ref[:n]
    size = np.abs(ref[:n]).max(-1, keepdims=True)  # (each row and head in units of its own largest value)
    size[size == 0] = 1
    assert np.linalg.norm((got - ref[:n]) / size) <= factor * np.linalg.norm(own / size)
    err, unit = np.linalg.norm(got - ref[:n], axis=-1), np.linalg.norm(ref[:n], axis=-1)
    assert (err <= 6 * 1.67e-3 * unit + 1e-300).all()


# heads, cached, new, e4m3: expanded with split tiles, with two streams, many heads; in the latent space
FORMS = [(2, [4000, 500], [300, 64], False), (3, [200], [600], True), (16, [3000], [200], False),
         (16, [9000, 4500], [20, 1], False), (128, [2000], [3], True)]


@pytest.mark.parametrize("power", [-50, -35, -20, -12, 12, 16, 30, 50])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_values_of_any_scale(lib, form, power):
    """w_uv times a power of two: the result times it, as exact as ever."""
    heads, ctx, new, fp8 = FORMS[form]
    c = Case(lib, ctx, new, heads=heads, fp8=fp8, seed=form)
    c.w_uv.mul_(2.0 ** power)
    exact_enough(c, check(c.run()), sum(new))
    assert (groups(c) > 0) == (form >= 3)


@pytest.mark.parametrize("power", [-40, -20, 15, 40])
@pytest.mark.parametrize("form", [0, 2, 3])
def test_cached_rows_of_any_scale(lib, form, power):
    """c_kv times a power of two and w_uk divided by it: the scores stay, the result grows."""
    heads, ctx, new, fp8 = FORMS[form]
    c = Case(lib, ctx, new, heads=heads, seed=form)
    c.pool.data[..., :512].mul_(2.0 ** power)
    c.w_uk.mul_(2.0 ** -power)
    exact_enough(c, check(c.run()), sum(new))


@pytest.mark.parametrize("nats", [0.0, 8.0, 12.0, 14.0, 16.0, 17.0, 20.0, 25.0, 30.0])
@pytest.mark.parametrize("heads,ctx,new", [(2, 2000, 30), (2, 700, 400), (1, 9000, 130), (16, 2000, 200)])
def test_a_first_key_without_value_takes_nearly_all_weight(lib, heads, ctx, new, nats):
    """An attention sink: c_kv of the first position is zero and its score `nats` above the others' mean. The result is
    made of the other weights alone, however small they are, and is as exact as without the sink."""
    c = Case(lib, [ctx], [new], heads=heads, seed=3)
    flat = c.pool.data[1].view(-1, 576)
    flat[:, 512] = 0
    s = slot(c, 0, 0)
    flat[s] = 0
    flat[s, 512] = nats / c.scale / 8
    c.q[:, :, 128] = 8
    exact_enough(c, check(c.run()), new)
    assert groups(c) == 0


@pytest.mark.parametrize("nats", [8.0, 14.0, 17.0, 25.0])
@pytest.mark.parametrize("heads,new", [(16, 20), (128, 3)])
def test_such_a_key_in_the_latent_space(lib, heads, new, nats):
    """The same there, where each half of a score is rounded to fp16 before the sum, as in decode: half a step of a
    score x in log2 units is 2^-11 x at most, and that factor is common to all of a row's result."""
    c = Case(lib, [13000 if heads == 16 else 4000], [new], heads=heads, seed=3)
    flat = c.pool.data[1].view(-1, 576)
    flat[:, 512] = 0
    s = slot(c, 0, 0)
    flat[s] = 0
    flat[s, 512] = nats / c.scale / 8
    c.q[:, :, 128] = 8
    ref = check(c.run(), 2e-2)
    assert groups(c) > 0
    common = 2.0 ** -11 * nats  # (nats: 2^-11 x log2 units times ln 2)
    assert np.linalg.norm(f64(c.out)[:new] - ref[:new]) <= (1.4 * 1.67e-3 + common) * np.linalg.norm(ref[:new])


@pytest.mark.parametrize("heads,ctx,new,window", [
    (2, [0], [700], 0), (2, [500], [200], 0), (1, [6000], [150], 0), (2, [3000], [513], 1200), (16, [900, 17], [120, 300], 0),
    (16, [9000, 4000], [20, 300], 0)])
@pytest.mark.parametrize("step", [0.02, 0.06, -0.02, 0.5])
def test_values_that_grow_or_shrink_along_the_positions(lib, heads, ctx, new, window, step):
    """c_kv times 2^(step x position), up to 2^+-40: rows see values of many sizes at once, and a row's result depends
    on those that it attends alone. Scores come from the rope part (w_uk is zero), so that they stay of a few units."""
    c = Case(lib, ctx, new, heads=heads, window=window, seed=9)
    c.w_uk.zero_()
    flat = c.pool.data[1].view(-1, 576)
    for b, n in enumerate(a + m for a, m in zip(ctx, new)):
        at = torch.arange(n, device="cuda")
        rows = c.table[b].long()[at // c.ps] * c.ps + at % c.ps
        power = torch.clamp((at - n // 2) * step, -40, 40).floor()
        flat[rows, :512] *= torch.exp2(power).to(torch.bfloat16)[:, None]
    exact_enough(c, check(c.run()), sum(new))


@pytest.mark.parametrize("big", [2.0 ** 30, 2.0 ** 55])
@pytest.mark.parametrize("heads,ctx,new", [(2, 100, 300), (1, 5000, 120), (16, 13000, 30)])
def test_one_huge_row_changes_those_that_attend_it_only(lib, heads, ctx, new, big):
    args = dict(ctx=[ctx, 90], new=[new, 40], heads=heads, seed=4)
    a, b = Case(lib, **args), Case(lib, **args)
    for c in (a, b):
        c.w_uk.zero_()
    pos = ctx + 20
    b.pool.data[1].view(-1, 576)[slot(b, 0, pos), :512] *= big
    a.run()
    b.run()
    hit = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    hit[20:new] = True
    assert torch.equal(bits(a.out[~hit]), bits(b.out[~hit])) and torch.equal(bits(a.lse[~hit]), bits(b.lse[~hit]))
    exact_enough(b, check(b), new + 40)


def test_zero_values(lib):
    """All values zero, and half of them: zero results, the same lse."""
    c = Case(lib, [300], [200], heads=2)
    c.w_uv.zero_()
    c.run().check()
    assert not c.out[:200].any()
    c = Case(lib, [300], [200], heads=2)
    c.w_uv[0].zero_()
    c.run().check()
    assert not c.out[:200, 0].any() and c.out[:200, 1].any()


# heads, cached, new, in the latent space
SCORES = [(2, [90], [20], False), (2, [2000], [300], False), (16, [13000], [20], True), (16, [9000, 4000], [33, 2], True),
          (128, [2000], [5], True)]


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [514, 570])
@pytest.mark.parametrize("heads,ctx,new,latent", SCORES)
def test_infinite_rope_value(lib, heads, ctx, new, latent, value, dim):
    """A score of -inf is a weight of zero; one of +inf gives NaN to the rows that attend it and to no others."""
    args = dict(ctx=ctx, new=new, heads=heads, seed=5)
    a, b = Case(lib, **args), Case(lib, **args)
    for c in (a, b):
        c.q[:, :, 128:] = 0
        c.q[:, :, 128 + dim - 512] = 1.0
    pos = ctx[0] + new[0] // 2
    b.pool.data[1].view(-1, 576)[slot(b, 0, pos), dim] = value
    a.run()
    b.run()
    assert (groups(b) > 0) == latent
    if value < 0:
        b.check()
        return
    hit = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    hit[new[0] // 2:new[0]] = True
    assert torch.isnan(b.out[hit].float()).all() and torch.isnan(b.lse[hit]).all()
    assert torch.equal(bits(a.out[~hit]), bits(b.out[~hit])) and torch.equal(bits(a.lse[~hit]), bits(b.lse[~hit]))


@pytest.mark.parametrize("heads,ctx,new", [(2, [0], [40]), (16, [0, 13000], [1, 3])])
def test_a_row_whose_only_score_is_minus_infinity(lib, heads, ctx, new):
    """Position 0 attends itself alone: no weight at all is NaN, as in a plain softmax, and has no finite lse."""
    c = Case(lib, ctx, new, heads=heads)
    c.q[:, :, 128:] = 0
    c.q[:, :, 130] = 1.0
    c.pool.data[1].view(-1, 576)[slot(c, 0, 0), 514] = -float("inf")
    c.run()
    assert (groups(c) > 0) == (heads == 16)
    assert torch.isnan(c.out[0].float()).all() and not torch.isfinite(c.lse[0]).any()
    assert torch.isfinite(c.out[1:sum(new)].float()).all() and torch.isfinite(c.lse[1:sum(new)]).all()


@pytest.mark.parametrize("q_std", [6.0, 0.0])
@pytest.mark.parametrize("heads,ctx,new,latent", SCORES)
def test_peaked_and_equal_scores(lib, heads, ctx, new, latent, q_std):
    c = Case(lib, ctx, new, heads=heads, q_std=q_std).run().check(3e-2 if q_std else 6e-3)
    assert (groups(c) > 0) == latent


@pytest.mark.parametrize("heads,ctx,new,latent", SCORES)
def test_growing_scores(lib, heads, ctx, new, latent):
    """Scores that climb by hundreds along the positions. In the latent space each half of a score is off by up to 2^-11
    of it, which the bounds of every output hold; all outputs together are then off by as much."""
    c = Case(lib, ctx, new, heads=heads)
    for b, n in enumerate(a + m for a, m in zip(ctx, new)):
        at = torch.arange(n, device="cuda")
        flat = c.pool.data[1].view(-1, 576)
        slots = c.table[b].long()[at // c.ps] * c.ps + at % c.ps
        flat[slots, 512:] = 0
        flat[slots, 512] = torch.linspace(0, 60, n, device="cuda").to(torch.bfloat16)
    c.q[:, :, 128:] = 0
    c.q[:, :, 128] = 60.0
    c.run().check(0.3 if latent else 6e-3)
    assert (groups(c) > 0) == latent
