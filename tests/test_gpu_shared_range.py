"""decode_shared at the ends of what it takes: weights far below a row's largest, lengths out of
range in a group of several requests, infinite scores, and workspaces that hold another call's plan."""
import math

import pytest
import torch

from shared_ref import CKV, Case, check
from test_gpu_decode_shared import lib, run  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nats", [8.0, 12.0, 17.4, 20.0])
def test_many_small_weights_beside_a_large_one(lib, fp8, nats):  # noqa: F811
    """One position far above 60,000 others, whose values it does not share: what they add up to is there.

    In f16 (e4m3 pools) a weight is off by 2^-11 of itself or by 2^-25. The largest weight of a row is 2^7 or more
    there and in the sum, so that the second is 2^-32 of the sum at most, for each position."""
    c = Case([(3, 60000)], [0, 40, 700], heads=16, page=64, fp8=fp8, seed=1, layers=1)
    key = 8.0  # (of the dims behind the value's; exact in either type)
    c.clean[..., CKV:] = 0
    c.clean[..., :CKV] = c.clean[..., :CKV] & 0x7F if fp8 else c.clean[..., :CKV].abs()  # (of one sign: what is lost shows)
    first = c.clean[0, int(c.full[0, 0]), 0]
    first[:CKV] = 0
    top = torch.tensor([key / c.scale], device="cuda")
    first[CKV] = top.to(torch.float8_e4m3fn).view(torch.uint8)[0] if fp8 else top[0]
    c.pool[0][c.used] = c.clean[0][c.used]
    c.q.zero_()
    c.q[..., CKV] = nats / c.softmax_scale / key
    out, lse, ws = run(lib, c, clusters=1)  # (with more each has a largest weight of its own)
    assert lib.get_error(ws) == 0
    for b in c.real():
        ref, ref_lse, bound, lse_bound = c.reference(b)
        bound = bound + (2.0 ** -32 * c.rows(b)[:, :CKV].abs().sum(0) if fp8 else 0)
        d = (out[b].double() - ref).abs()
        assert bool((d <= bound).all()), (b, (d / bound).max().item(), out[b, 0, 0, 0].item(), ref[0, 0, 0].item())
        assert bool(((lse[b].double() - ref_lse).abs() <= lse_bound).all())


@pytest.mark.parametrize("prefix", [-1, -(1 << 31), 1 << 29, (1 << 31) - 1])
def test_prefix_lengths_out_of_range_count_as_none(lib, prefix):  # noqa: F811
    c = Case([(3, 0), (2, 100)], [200, 300, 250, 5, 9], heads=16, page=16, seed=2)
    c.prefix = torch.tensor([prefix, 100], dtype=torch.int32, device="cuda")
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == lib.STATUS_BAD_LENGTH
    check(c, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,heads", [(1, 16), (3, 32)])
@pytest.mark.parametrize("where", [[0], [1], [2], [1, 2]])
@pytest.mark.parametrize("bad", [-1, 1 << 29, (1 << 31) - 1])
def test_a_cached_length_out_of_range_is_its_own_requests(lib, fp8, q_len, heads, where, bad):  # noqa: F811
    """The others keep the prefix (of which they have no table entries of their own); the request itself has the
    prefix and its new tokens."""
    c = Case([(3, 203), (2, 90)], [20, 40, 133, 7, 60], heads=heads, q_len=q_len, page=16, fp8=fp8, seed=3)
    lengths = c.ctx.clone()
    c.ctx[where] = bad
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == lib.STATUS_BAD_LENGTH
    c.ctx = lengths
    c.ctx[where] = 203
    check(c, out, lse)


def test_a_group_without_a_length_in_range(lib):  # noqa: F811
    c = Case([(2, 0), (2, 64)], [30, 50, 7, 60], heads=16, page=16, seed=4)
    c.prefix = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    lengths = c.ctx.clone()
    c.ctx[:2] = torch.tensor([-3, 1 << 30], dtype=torch.int32, device="cuda")
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == lib.STATUS_BAD_LENGTH
    c.ctx = lengths
    c.ctx[:2] = 0
    check(c, out, lse)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("at", [-5, 0, 1])
def test_an_infinity_that_is_seen(lib, sign, at):  # noqa: F811
    """In a cached row, the first new token's and the second's, with scores of either infinity."""
    c = Case([(3, 100)], [30, 125, 64], heads=32, q_len=3, page=16, seed=6)
    c.q[1, ..., 7] = sign * c.q[1, ..., 7].abs().clamp(min=0.5)
    want, want_lse, _ = run(lib, c)
    t = int(c.ctx[1]) + at
    c.pool[c.layer, int(c.full[1, t // c.page]), t % c.page, 7] = math.inf
    out, lse, ws = run(lib, c)
    assert lib.get_error(ws) == 0
    others = [0, 2]
    assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])
    first = max(at, 0)  # query position that sees it
    assert torch.equal(out[1, :first], want[1, :first]) and torch.equal(lse[1, :first], want_lse[1, :first])
    bad = out[1, first:].isnan()
    if sign > 0:
        assert bool(bad.all()) and bool(lse[1, first:].isnan().all())
        return
    assert bool(bad[..., 7].all()) == (at < 1) and not bool(bad[..., :7].any() or bad[..., 8:].any())
    lat = torch.cat([c.rows(1)[:t], c.rows(1)[t + 1:]])  # as without the position
    ref, ref_lse, bound, lse_bound = c.reference(1, lat)
    keep = [x for x in range(CKV) if x != 7 or at == 1]
    assert bool(((out[1].double() - ref).abs() <= bound)[first:][..., keep].all())
    assert bool(((lse[1].double() - ref_lse).abs() <= lse_bound)[first:].all())


def test_plans_of_other_calls_in_the_same_workspace(lib):  # noqa: F811
    """A plan of mla_decode whose record reads, word by word, as one for this call; and one after the other."""
    c = Case([(20, 64)], [20, 40, 33, 5, 0], heads=16, q_len=16, page=16, seed=5)
    ws = torch.zeros(max(lib.workspace_size_shared(20, 16, 16, 1), lib.workspace_size_q(20, 16, 16)), dtype=torch.uint8, device="cuda")
    lib.plan(c.ctx, 16, 16, 1, ws, num_clusters=16)  # heads, page size, window, clusters: q_len, heads, prefixes, page size
    torch.cuda.synchronize()
    words = ws[:256].view(torch.int32).tolist()
    assert words[1:6] == [20, 16, 16, 1, 16] and words[6] != 0 and words[7] <= 36
    out, lse, _ = run(lib, c, ws=ws, plan=False)
    assert lib.get_error(ws, clear=True) == lib.STATUS_PLAN_MISMATCH
    assert bool((out == 7).all()) and bool((lse == 7).all())
    run(lib, c, ws=ws, out=out, lse=lse)
    assert lib.get_error(ws) == 0
    check(c, out, lse)
    # the other way round: what mla_decode_q's plan left as its q_len does not stay beside this plan
    lib.plan_q(c.ctx, 16, 16, 16, 1, ws)
    lib.plan_shared(c.ctx, c.indptr, c.prefix, 16, 16, 16, ws)
    torch.cuda.synchronize()
    words = ws[:256].view(torch.int32).tolist()
    assert words[11] == 0
    run(lib, c, ws=ws, plan=False, out=out, lse=lse)
    assert lib.get_error(ws) == 0
    check(c, out, lse)
