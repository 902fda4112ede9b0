"""Rotary latent write (rope_write) against a plain 64-bit form.

Tolerances: the kernel computes in fp32 (a product pair: three roundings of
2^-24 of the terms; the norm: 512 squares summed, at most (512 / 32 + 5 + 4)
roundings, and rsqrt, 2 units) and rounds once. So a bf16 value is within
2^-8 |ref| + (fp32 error) (1 + 2^-8) of the reference, an e4m3 value within
max(2^-4 |ref|, 2^-10) in units of the scale plus the same."""
import numpy as np
import pytest
import torch

import step_ref

pytestmark = pytest.mark.gpu
F32 = step_ref.F32_HALF
LIMIT = 5000
AXES = {1: [0] * 32, 2: [0, 1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12, 4: [3, 2, 1, 0] * 8}


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def table():
    inv = 10000.0 ** (-np.arange(32) / 32)
    a = np.arange(LIMIT)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Case:
    def __init__(self, lib, n, heads, ps=16, fp8=False, axes=1, norm=True, q_dim=192, out_dim=192, seed=0, in_place=False,
                 pads=()):
        g = torch.Generator("cuda")
        g.manual_seed(seed)
        self.lib, self.n, self.heads, self.axes, self.fp8 = lib, n, heads, axes, fp8
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        pages = n // ps + 3
        data = r(2, pages, ps, 576)
        self.scale = 0.0173 if fp8 else 1.0
        if fp8:
            data = (data.float() * 30).to(torch.float8_e4m3fn).view(torch.uint8)
        self.pool = lib.KVPool(data, self.scale)
        self.rows = r(n, 576)
        self.slots = torch.randperm(pages * ps, generator=g, device="cuda")[:n].contiguous()
        for i in pads:
            self.slots[i] = -1
        self.weight = (1 + 0.2 * r(512).float()).to(torch.bfloat16) if norm else None
        self.cos_sin = torch.from_numpy(table()).cuda()
        self.pos = torch.randint(0, LIMIT, (axes, n), generator=g, device="cuda", dtype=torch.int32)
        self.q_all = r(n, heads, q_dim)
        self.q = self.q_all[:, :, q_dim - 64:]
        self.o_all = self.q_all if in_place else r(n, heads, out_dim)
        self.o = self.o_all[:, :, self.o_all.shape[2] - 64:]

    def run(self, interleaved=True, layer=1, **kw):
        args = dict(norm_weight=self.weight, q_rope=self.q, q_out=self.o, pair_axis=AXES[self.axes],
                    interleaved=interleaved)
        args.update(kw)
        self.before = (self.pool.data.clone(), self.q_all.clone(), self.o_all.clone())
        self.lib.rope_write(self.pool, layer, self.rows, self.slots, self.pos, self.cos_sin, **args)
        torch.cuda.synchronize()

    def check(self, interleaved=True, layer=1, skip=()):
        """Every value of the pool and of the outputs; rows in `skip` and everything else as before."""
        cs, pos = self.cos_sin.cpu().numpy(), self.pos.cpu().numpy()
        take = [i for i in range(self.n) if i not in skip and int(self.slots[i]) >= 0]
        q_ref, q_mag = step_ref.rotate(f64(self.before[1])[..., -64:], pos, AXES[self.axes], cs, interleaved)
        o_ref = f64(self.before[2])
        got = f64(self.o_all)
        for i in range(self.n):
            if i in take:
                tol = step_ref.BF16_HALF * np.abs(q_ref[i]) + 3 * F32 * q_mag[i] * 1.01
                assert (np.abs(got[i, :, -64:] - q_ref[i]) <= tol).all()
                assert np.array_equal(got[i, :, :-64], o_ref[i, :, :-64])
            else:
                assert np.array_equal(got[i], o_ref[i])
        rows = f64(self.rows)
        w = None if self.weight is None else f64(self.weight)
        c = step_ref.norm(rows[:, :512], w, 1e-6)
        kr, k_mag = step_ref.rotate(rows[:, 512:], pos, AXES[self.axes], cs, interleaved)
        ref = np.concatenate([c, kr], 1)
        err = np.concatenate([np.abs(c) * (25 + 6) * F32 if w is not None else 0 * c, 3 * F32 * k_mag], 1)
        old = self.before[0].view(torch.int16 if not self.fp8 else torch.uint8).cpu().numpy()
        new = self.pool.data.view(torch.int16 if not self.fp8 else torch.uint8).cpu().numpy()
        vals = f64(self.pool.data.view(torch.float8_e4m3fn)) if self.fp8 else f64(self.pool.data)
        vals = vals[layer].reshape(-1, 576)
        touched = np.zeros(old.shape[1] * old.shape[2], bool)
        for i in take:
            s = int(self.slots[i])
            touched[s] = True
            if self.fp8:
                x = np.clip(ref[i] / self.scale, -448, 448)
                tol = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10) + (err[i] / self.scale + np.abs(x) * F32) * 1.1
                assert (np.abs(vals[s] - x) <= tol).all()
            else:
                assert (np.abs(vals[s] - ref[i]) <= step_ref.BF16_HALF * np.abs(ref[i]) + err[i] * 1.01).all()
        assert np.array_equal(new[1 - layer], old[1 - layer])
        assert np.array_equal(new[layer].reshape(-1, 576)[~touched], old[layer].reshape(-1, 576)[~touched])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("fp8", [False, True])
def test_axes_and_layouts(lib, interleaved, axes, fp8):
    c = Case(lib, 37, 16, fp8=fp8, axes=axes, seed=axes)
    c.run(interleaved)
    c.check(interleaved)


@pytest.mark.parametrize("n,heads", [(1, 1), (1, 128), (2, 16), (3, 7), (8, 33), (9, 128), (130, 5), (700, 40)])
@pytest.mark.parametrize("q_dim,out_dim", [(192, 192), (64, 576)])
def test_sizes(lib, n, heads, q_dim, out_dim):
    c = Case(lib, n, heads, ps=64, q_dim=q_dim, out_dim=out_dim, seed=n)
    c.run(False)
    c.check(False)


@pytest.mark.parametrize("interleaved", [True, False])
def test_in_place(lib, interleaved):
    c = Case(lib, 50, 24, in_place=True)
    c.run(interleaved, q_out=None)
    c.check(interleaved)


def test_without_norm_the_c_kv_part_is_kv_writes(lib):
    c = Case(lib, 40, 8, norm=False)
    c.run()
    c.check()
    flat = c.pool.data[1].reshape(-1, 576)
    assert torch.equal(flat[c.slots][:, :512], c.rows[:, :512])


@pytest.mark.parametrize("fp8", [False, True])
def test_position_zero_equals_kv_write(lib, fp8):
    """No turn and no norm: the same bytes as the plain latent write."""
    c = Case(lib, 33, 4, norm=False, fp8=fp8)
    c.pos.zero_()
    other = lib.KVPool(c.pool.data.clone(), c.scale)
    lib.kv_write(other, 1, c.rows, c.slots)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.pool.data.view(torch.uint8), other.data.view(torch.uint8))
    assert torch.equal(c.o.contiguous(), c.q.contiguous())


def test_a_turn_keeps_lengths_and_differences(lib):
    """The scores of two turned vectors depend on the distance of their positions only."""
    n = 64
    c = Case(lib, n, 1, norm=False, q_dim=64, out_dim=64)
    c.q_all[:] = c.q_all[0].clone()
    c.rows[:] = c.rows[0].clone()
    c.pos[0] = torch.arange(n, device="cuda", dtype=torch.int32) * 70
    c.run(False)
    q = f64(c.o)[:, 0]
    k = f64(c.pool.data[1].reshape(-1, 576)[c.slots])[:, 512:]
    s = q @ k.T
    bound = 4 * step_ref.BF16_HALF * np.abs(f64(c.q_all[0, 0])).max() * np.abs(f64(c.rows[0])).max() * 64
    for d in range(0, 60, 7):
        x = np.diagonal(s, d)
        assert np.ptp(x) <= bound
    assert np.ptp(s) > bound  # the positions matter at all


def test_pad_rows_and_bad_slots_and_positions(lib):
    c = Case(lib, 20, 8, pads=(0, 7, 19))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    c.pos[0, 3] = -1        # a pad row by its position
    c.run(workspace=ws)
    c.check(skip=(3,))
    assert lib.get_error(ws) == 0
    c = Case(lib, 20, 8)
    c.pos[0, 4] = LIMIT     # beyond the table: skipped
    c.run(workspace=ws)
    c.check(skip=(4,))
    assert lib.get_error(ws, clear=True) == lib.STATUS_BAD_POSITION
    c = Case(lib, 4, 8)
    keep = c.pool.data.clone()
    c.slots[:] = c.pool.data.shape[1] * c.pool.data.shape[2]
    c.run(workspace=ws)
    assert torch.equal(c.pool.data, keep) and lib.get_error(ws) == lib.STATUS_BAD_SLOT


def test_rows_alone_and_queries_alone(lib):
    c = Case(lib, 21, 16)
    keep = c.o_all.clone()
    c.run(q_rope=None, q_out=None)
    assert torch.equal(c.o_all, keep)
    d = Case(lib, 21, 16)
    d.run()
    assert torch.equal(c.pool.data, d.pool.data)
    e = Case(lib, 21, 16)
    pool = e.pool.data.clone()
    lib.rope_write(None, 0, None, None, e.pos, e.cos_sin, q_rope=e.q, q_out=e.o)
    torch.cuda.synchronize()
    assert torch.equal(e.o_all, d.o_all) and torch.equal(e.pool.data, pool)


def test_offsets_past_32_bits(lib):
    """Slots of a layer that starts beyond 4 GB, and queries whose last rows lie beyond 2^31 elements."""
    c = Case(lib, 70, 3, ps=128)
    c.run()
    pages = 31000
    pool = torch.empty(2, pages, 128, 576, dtype=torch.bfloat16, device="cuda")
    pool[1, -2:] = 0
    first = (pages - 1) * 128 + 20
    slots = torch.arange(first, first + 70, device="cuda")
    n, heads = 90000, 128
    q = torch.empty(n, heads, 192, dtype=torch.bfloat16, device="cuda")
    q[-70:, :3] = c.q_all
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos[-70:] = c.pos[0]
    assert q[-70:].storage_offset() + q.stride(0) * (n - 70) > 2 ** 31
    want = torch.empty(70, 3, 64, dtype=torch.bfloat16, device="cuda")
    lib.rope_write(None, 0, None, None, c.pos[0].contiguous(), c.cos_sin, q_rope=c.q, q_out=want)
    lib.rope_write(lib.KVPool(pool), 1, c.rows, slots, c.pos[0].contiguous(), c.cos_sin, norm_weight=c.weight)
    lib.rope_write(None, 0, None, None, pos, c.cos_sin, q_rope=q[:, :, 128:])
    small = torch.zeros(2, 2, 128, 576, dtype=torch.bfloat16, device="cuda")
    lib.rope_write(lib.KVPool(small), 1, c.rows, slots - (pages - 2) * 128, c.pos[0].contiguous(), c.cos_sin,
                   norm_weight=c.weight)
    torch.cuda.synchronize()
    assert small[1].any() and torch.equal(pool[1, -2:].view(torch.int16), small[1].view(torch.int16))
    assert torch.equal(q[-70:, :3, 128:].view(torch.int16), want.view(torch.int16))
    assert torch.equal(q[-70:, :3, :128].view(torch.int16), c.q_all[:, :, :128].view(torch.int16))


def test_nan_and_infinity_stay_in_their_row(lib):
    c = Case(lib, 10, 4)
    c.rows[3, 100] = float("inf")
    c.rows[5, 520] = float("nan")
    c.run()
    got = c.pool.data[1].reshape(-1, 576)[c.slots].float()
    assert torch.isnan(got[5, 512 + 8]) and torch.isfinite(got[5, :512]).all()
    assert torch.isfinite(got[[0, 1, 2, 4, 6, 7, 8, 9]]).all() and torch.isfinite(c.o_all.float()).all()


def test_on_another_stream_and_in_a_graph(lib):
    c, d = Case(lib, 64, 16), Case(lib, 64, 16)
    c.run()
    d.before = None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        d.lib.rope_write(d.pool, 1, d.rows, d.slots, d.pos, d.cos_sin, norm_weight=d.weight, q_rope=d.q, q_out=d.o)
    d.rows.mul_(2)  # changed in place between capture and replay: unit scale undoes a factor of two
    d.rows[:, 512:].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o_all, d.o_all)
    a, b = c.pool.data[1].float(), d.pool.data[1].float()
    assert (a - b).abs().max() <= 2 ** -7 * a.abs().max()  # the norm's epsilon moves a rounding at most


def test_refusals(lib):
    c = Case(lib, 6, 4)
    call = lambda **k: lib.rope_write(**{**dict(  # noqa: E731
        pool=c.pool, layer=0, rows=c.rows, slot_mapping=c.slots, positions=c.pos, cos_sin=c.cos_sin), **k})
    for bad in [dict(rows=None), dict(rows=c.rows[:5]), dict(slot_mapping=None), dict(slot_mapping=c.slots[:2]),
                dict(positions=c.pos[:, :3]), dict(cos_sin=c.cos_sin[:, :32]), dict(norm_weight=c.rows[0, :100]),
                dict(pair_axis=[0] * 31), dict(pair_axis=[1] * 32), dict(q_out=c.o), dict(q_rope=c.q[:3]),
                dict(q_rope=c.q[:, ::2][:, :2].transpose(0, 1)), dict(q_rope=c.q.float()),
                dict(q_rope=c.q, q_out=c.o[:, :2]), dict(positions=c.pos.long())]:
        with pytest.raises(ValueError):
            call(**bad)
    wide = torch.zeros(6, 4, 192, dtype=torch.bfloat16, device="cuda")
    for bad in [dict(layer=2), dict(norm_weight=c.weight, norm_eps=-1.0),
                dict(q_rope=wide[:, :, 0:64], q_out=wide[:, :, 32:96]),       # shares elements with its source
                dict(q_rope=wide[:, :, 4:68])]:                               # not 16-byte aligned
        with pytest.raises(lib.MlaError):
            call(**bad)
    call(q_rope=wide[:, :, 0:64], q_out=wide[:, :, 64:128])                   # beside it is fine
