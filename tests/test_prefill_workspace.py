"""Sizes of the chunk attention's workspace: one that a larger call was given does for
every smaller one, so that a server allocates once, for its largest step."""
import random

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def size():
    from paged_mla_decode_04_gb300 import _build
    import paged_mla_decode_04_gb300 as m
    return m.load_library(_build.build()).mla_prefill_workspace_size


def log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("heads", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("per_pass", [0, 1, 5, 1024])
def test_smaller_calls_need_no_more(size, heads, per_pass):
    """Fewer requests, rows and positions, each of them or all. (Keys and values of all heads stay below the 8 GiB where
    the default takes fewer at a time.)"""
    rng = random.Random(heads)
    for _ in range(2000):
        batch, rows = log_uniform(rng, 1, 400), log_uniform(rng, 1, 20000)
        kv = log_uniform(rng, 1, (8 << 30) // (heads * 520) - 64 * batch - 1000)
        less = lambda x: rng.choice([x, log_uniform(rng, 1, x)])  # noqa: E731
        small = (less(batch), less(rows), less(kv))
        assert 0 < size(*small, heads, per_pass) <= size(batch, rows, kv, heads, per_pass), (small, batch, rows, kv)


def test_the_latent_space_comes_with_fewer_rows(size):
    """1,000 rows of 32 requests are too many for it at 1,000 positions and 16 heads, 256 are not and need more room."""
    assert size(32, 1000, 1000, 16, 0) >= size(32, 256, 1000, 16, 0) >= size(32, 200, 1000, 16, 1)
    assert size(32, 256, 1000, 16, 0) > size(32, 256, 1000, 17, 16) + (20 << 20)  # (17 heads have no latent path)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,ctx,new", [(16, 23, [8] * 32), (16, 25, [1, 13] * 16), (32, 20, [3] * 32)])
def test_a_smaller_step_in_a_larger_ones_workspace(heads, ctx, new):
    import paged_mla_decode_04_gb300 as lib
    from test_gpu_prefill import Case, bits
    args = dict(ctx=[ctx] * 32, new=new, heads=heads)
    a = Case(lib, **args, extra_rows=0).run().check()
    b = Case(lib, **args, extra_rows=0)
    assert int(a.ws[:32].view(torch.int32)[7]) > 0  # (in the latent space)
    b.ws = lib.alloc_prefill_workspace(32, 1000, b.max_kv, heads)
    b.run()
    assert torch.equal(bits(a.out), bits(b.out)) and torch.equal(bits(a.lse), bits(b.lse))


@pytest.mark.gpu
def test_a_workspace_without_room_for_the_latent_space():
    """The call does without it, as long as one head's keys and values fit."""
    import paged_mla_decode_04_gb300 as lib
    from test_gpu_prefill import Case, f64
    args = dict(ctx=[23] * 32, new=[8] * 32, heads=16, extra_rows=0)
    a = Case(lib, **args).run().check()
    b = Case(lib, **args)
    n = lib.prefill_workspace_size(32, b.T, b.max_kv, 17, 1)  # (17 heads have no latent path; one at a time)
    assert n < a.ws.numel()
    guard = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    guard[:256] = 0
    b.ws = guard[:n]
    b.latent = lambda: False
    b.run().check()
    assert int(b.ws[:32].view(torch.int32)[7]) == 0 and bool((guard[n:] == 0x5a).all())
    b.ws = guard[:n - 256]
    b.out.fill_(7)
    with pytest.raises(lib.MlaError, match="WORKSPACE"):
        b.run()
    torch.cuda.synchronize()
    assert (b.out == 7).all()
    assert np.abs(f64(a.out)).max() > 0.1
