"""Serving steps as a user runs them: extend_tables, rope_write and prefill one
after the other on the same buffers, captured as one CUDA graph and replayed with
other lengths; single tokens at the end also by plan, decode and uv_project. Every
part is held to a plain 64-bit form on the cache as the part before left it."""
import numpy as np
import pytest
import torch

import step_ref

pytestmark = pytest.mark.gpu
B, H, PS, MAX_T, MAX_BLOCKS, PAGES, LIMIT = 4, 16, 32, 200, 25, 70, 1000


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Engine:
    def __init__(self, lib, fp8):
        g = torch.Generator("cuda")
        g.manual_seed(11)
        self.lib, self.fp8, d, i32 = lib, fp8, "cuda", torch.int32
        self.scale_kv = 0.02 if fp8 else 1.0
        self.pool = lib.KVPool(torch.zeros(2, PAGES, PS, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device=d),
                               self.scale_kv)
        r = lambda *s: torch.randn(s, generator=g, device=d)  # noqa: E731
        self.w_uk = (r(H, 128, 512) * 512 ** -0.5).to(torch.bfloat16)
        self.w_uv = (r(H, 512, 128) * 512 ** -0.5).to(torch.bfloat16)
        self.norm = (1 + 0.1 * r(512)).to(torch.bfloat16)
        inv = 10000.0 ** (-np.arange(32) / 32)
        ang = np.arange(LIMIT)[:, None] * inv
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
        self.free = torch.randperm(PAGES, generator=g, device=d).to(i32)
        self.state = torch.tensor([PAGES, 0], dtype=i32, device=d)
        self.table = torch.full((B, MAX_BLOCKS), -1, dtype=i32, device=d)
        self.ctx = torch.zeros(B, dtype=i32, device=d)
        self.new = torch.zeros(B, dtype=i32, device=d)
        self.slots = torch.full((MAX_T,), -1, dtype=torch.int64, device=d)
        self.pos = torch.full((MAX_T,), -1, dtype=i32, device=d)
        self.indptr = torch.zeros(B + 1, dtype=i32, device=d)
        self.rows = torch.zeros(MAX_T, 576, dtype=torch.bfloat16, device=d)
        self.q = torch.zeros(MAX_T, H, 192, dtype=torch.bfloat16, device=d)
        self.out = torch.zeros(MAX_T, H, 128, dtype=torch.bfloat16, device=d)
        self.scale = 192 ** -0.5
        self.max_kv = B * MAX_BLOCKS * PS
        self.ws = lib.alloc_prefill_workspace(B, MAX_T, self.max_kv, H)

    def step(self):
        lib = self.lib
        lib.extend_tables(self.ctx, self.new, self.free, self.state, self.table, PS, PAGES, self.slots, self.indptr,
                          self.state, positions=self.pos, workspace=self.ws)
        lib.rope_write(self.pool, 1, self.rows, self.slots, self.pos, self.cos_sin, norm_weight=self.norm,
                       q_rope=self.q[:, :, 128:], workspace=self.ws)
        lib.prefill(self.pool, 1, self.q, self.indptr, self.ctx, self.scale, self.w_uk, self.w_uv, self.ws, self.out,
                    self.max_kv, block_table=self.table)

    def cache(self):
        """The cache's codes, in units of its scale."""
        d = self.pool.data[1]
        return f64(d.view(torch.float8_e4m3fn) if self.fp8 else d)


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_of_prompts_chunks_and_single_tokens(lib, fp8):
    e = Engine(lib, fp8)
    e.step()  # no tokens: loads the kernels, changes nothing
    torch.cuda.synchronize()
    assert int(e.state[0]) == PAGES and not e.pool.data.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.step()
    rng = np.random.default_rng(3)
    ctx = np.zeros(B, np.int32)
    for new in ([100, 0, 37, 1], [60, 45, 0, 90], [1, 130, 64, 1], [1, 1, 1, 1]):
        new = np.array(new, np.int32)
        T = int(new.sum())
        e.ctx.copy_(torch.from_numpy(ctx))
        e.new.copy_(torch.from_numpy(new))
        e.rows.copy_(torch.from_numpy(rng.standard_normal((MAX_T, 576)).astype(np.float32)))
        e.q.copy_(torch.from_numpy(rng.standard_normal((MAX_T, H, 192)).astype(np.float32)))
        e.out.fill_(5.0)
        raw_q, free, count, table, old = f64(e.q), e.free.cpu().numpy(), int(e.state[0]), e.table.cpu().numpy(), e.cache()
        graph.replay()
        torch.cuda.synchronize()
        assert lib.get_error(e.ws) == 0
        # places
        ref = step_ref.extend_tables(ctx, new, free, count, table, PS, PAGES, MAX_T)
        assert np.array_equal(e.table.cpu().numpy(), ref["table"]) and np.array_equal(e.slots.cpu().numpy(), ref["slots"])
        assert np.array_equal(e.pos.cpu().numpy(), ref["positions"]) and np.array_equal(e.indptr.cpu().numpy(), ref["indptr"])
        assert e.state.cpu().tolist() == ref["state"].tolist()
        # the latent rows: written at those places alone, and right
        cache, flat = e.cache(), e.cache().reshape(-1, 576)
        slots, pos = ref["slots"][:T], ref["positions"][None, :T]
        cs = e.cos_sin.cpu().numpy()
        rows = f64(e.rows)[:T]
        c = step_ref.norm(rows[:, :512], f64(e.norm), 1e-6)
        kr, _ = step_ref.rotate(rows[:, 512:], pos, [0] * 32, cs, True)
        want = np.concatenate([c, kr], 1) / e.scale_kv
        half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) if fp8 else 2.0 ** -8 * np.abs(want)
        size = np.abs(rows).max() * 4 / e.scale_kv  # (fp32 errors, of the larger terms)
        assert (np.abs(flat[slots] - np.clip(want, -448, 448) if fp8 else flat[slots] - want) <= half + size * 2.0 ** -19).all()
        untouched = np.ones(PAGES * PS, bool)
        untouched[slots] = False
        assert np.array_equal(flat[untouched], old.reshape(-1, 576)[untouched])
        # the queries: rotated, pad rows left
        q = f64(e.q)
        qr, mag = step_ref.rotate(raw_q[:T, :, 128:], pos, [0] * 32, cs, True)
        assert (np.abs(q[:T, :, 128:] - qr) <= 2.0 ** -8 * np.abs(qr) + mag * 2.0 ** -22).all()
        assert np.array_equal(q[T:], raw_q[T:]) and np.array_equal(q[:, :, :128], raw_q[:, :, :128])
        # attention over the cache as it is now
        at_scale, tab = cache * e.scale_kv, ref["table"]
        out, _, tol, _ = step_ref.prefill(lambda b, at: at_scale[tab[b][at // PS], at % PS], q, ref["indptr"], ctx,
                                          f64(e.w_uk), f64(e.w_uv), e.scale, 0)
        got = f64(e.out)
        assert (np.abs(got[:T] - out[:T]) <= tol[:T]).all() and (got[T:] == 5.0).all()
        ctx = ctx + new
    # The last step's single tokens once more, by the decode path.
    last = torch.from_numpy(ctx - 1).cuda()
    q = e.q[:B].float()
    q_abs = torch.cat([torch.einsum("bhd,hdc->bhc", q[..., :128], e.w_uk.float()), q[..., 128:]], -1).to(torch.bfloat16)
    ws = lib.alloc_workspace(B, H)
    lat = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(B, H, 128, dtype=torch.bfloat16, device="cuda")
    lib.plan(last, H, PS, 0, ws)
    lib.decode(e.pool, 1, q_abs, last, e.scale, ws, lat, block_table=e.table)
    lib.uv_project(lat, e.w_uv, y, ws)
    torch.cuda.synchronize()
    assert lib.get_error(ws) == 0
    assert np.abs(f64(y) - f64(e.out)[:B]).max() <= (5e-2 if fp8 else 2e-2) * np.abs(f64(y)).max()


def test_pages_run_out_in_a_step(lib):
    """The refused request's tokens are pad rows to the write; its attention reads what is there and harms nobody."""
    e = Engine(lib, False)
    e.state[0] = 5  # pages of 32
    e.new.copy_(torch.tensor([64, 33, 70, 20], dtype=torch.int32))
    e.rows.normal_()
    e.q.normal_()
    before = e.pool.data.clone()
    e.step()
    torch.cuda.synchronize()
    assert lib.get_error(e.ws, clear=True) & lib.STATUS_NO_PAGES
    assert e.state.cpu().tolist() == [1, 2]                        # requests 0 and 1 took four pages, 2 needs three
    slots = e.slots.cpu().numpy()
    assert (slots[:97] >= 0).all() and (slots[97:187] == -1).all()  # nor is request 3 served past the refused one
    assert torch.equal(e.pool.data[0], before[0])
    assert torch.isfinite(e.out[:97].float()).all()
    # the scheduler gives pages back and runs the refused ones again
    e.free[:8] = torch.tensor([p for p in range(PAGES) if p not in e.table[:2].cpu().numpy()][:8], dtype=torch.int32)
    e.state[0] = 8
    e.ctx.copy_(torch.tensor([64, 33, 0, 0], dtype=torch.int32))
    e.new.copy_(torch.tensor([0, 0, 70, 20], dtype=torch.int32))
    e.step()
    torch.cuda.synchronize()
    assert lib.get_error(e.ws) == 0 and e.state.cpu().tolist() == [4, 4]
