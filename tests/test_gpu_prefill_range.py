"""Chunk attention (prefill) far from scores of a few units:
softmax weights far below a row's largest."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import Case, f64

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


@pytest.mark.parametrize("nats", [0.0, 8.0, 12.0, 14.0, 16.0])
@pytest.mark.parametrize("heads,ctx,new", [(2, 2000, 30), (2, 700, 400), (1, 9000, 130), (16, 2000, 200)])
def test_a_first_key_without_value_takes_nearly_all_weight(lib, heads, ctx, new, nats):
    """An attention sink: c_kv of the first position is zero and its score `nats` above the others' mean. The result is
    made of the other weights alone, which are small, and is as exact as without the sink."""
    c = Case(lib, [ctx], [new], heads=heads, seed=3)
    flat = c.pool.data[1].view(-1, 576)
    flat[:, 512] = 0
    s = slot(c, 0, 0)
    flat[s] = 0
    flat[s, 512] = nats / c.scale / 8
    c.q[:, :, 128] = 8
    exact_enough(c, check(c.run()), new)
    assert groups(c) == 0
