"""The compact store: bytes as written, values as read, pad rows, slots out of range; and
a prefix's way from its rows through the store into a pool that decode_shared attends."""
import math

import pytest
import torch

from shared_ref import BF16_HALF, Case, check, store_row, store_values

pytestmark = pytest.mark.gpu
ROWS = {"e4m3": 656, "e2m1": 416}


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def rows_of(n, seed=0, kind="normal"):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    x = torch.randn(n, 576, generator=g, device="cuda")
    if kind == "wide":
        x *= torch.exp2(torch.randint(-120, 120, (n, 576), generator=g, device="cuda").float())
    elif kind == "small":  # down to bf16's subnormal values
        x *= torch.exp2(torch.randint(-140, -110, (n, 1), generator=g, device="cuda").float())
    elif kind == "ties":  # halfway between codes, and zeros
        x = torch.randint(-24, 25, (n, 576), generator=g, device="cuda") / 4.0
        x[:, 0::32] = 6.0
        x[n // 2:, 32:64] = 0
    return x.to(torch.bfloat16)


def same_bytes(a, b, codes):
    """Equal bytes, but that a code of zero may have either sign where nothing fixes it, and any NaN scale is one."""
    assert a.shape == b.shape
    if codes == "e4m3":
        sa, sb = a[:, 512:528].contiguous().view(torch.float32), b[:, 512:528].contiguous().view(torch.float32)
        ca, cb, ra, rb = a[:, :512], b[:, :512], a[:, 528:], b[:, 528:]
        nan = sb.isnan().repeat_interleave(128, 1)
    else:
        sa, sb = a[:, 256:288].contiguous().view(torch.bfloat16), b[:, 256:288].contiguous().view(torch.bfloat16)
        ca, cb, ra, rb = a[:, :256], b[:, :256], a[:, 288:], b[:, 288:]
        nan = sb.isnan().repeat_interleave(16, 1)
    assert torch.equal(sa.isnan(), sb.isnan()) and torch.equal(sa.nan_to_num(), sb.nan_to_num())
    assert torch.equal(ra, rb)
    assert torch.equal(ca.masked_fill(nan, 0), cb.masked_fill(nan, 0))


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 33, 500, 5003])
@pytest.mark.parametrize("page", [16, 128])
def test_write(lib, codes, n, page):
    pages = n // page + 2
    store = lib.alloc_quant_pool(2, pages, page, codes)
    store.data.fill_(0x5A)
    slots = torch.randperm(pages * page, device="cuda")[:n].contiguous()
    rows = rows_of(n, n)
    want = store.data.clone()
    want[1].view(-1, ROWS[codes])[slots] = store_row(rows, codes)
    lib.quant_write(store, 1, rows, slots)
    assert torch.equal(store.data, want)


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
@pytest.mark.parametrize("kind", ["wide", "small", "ties"])
def test_write_of_other_sizes(lib, codes, kind):
    n = 700
    store = lib.alloc_quant_pool(1, 50, 16, codes)
    rows = rows_of(n, 3, kind)
    slots = torch.arange(n, device="cuda")
    lib.quant_write(store, 0, rows, slots)
    same_bytes(store.data[0].view(-1, ROWS[codes])[:n], store_row(rows, codes), codes)
    assert torch.equal(store_values(store.data[0].view(-1, ROWS[codes])[:n])[:, 512:], rows[:, 512:].double())


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
@pytest.mark.parametrize("power", [0, -60, -70, -120, 100])
def test_every_quotient(lib, codes, power):
    """Every significand that a value can have over every one that its group's largest can have, down to quotients
    that round to zero: the code of the IEEE quotient."""
    size = 128 if codes == "e4m3" else 32
    low = 20 if codes == "e4m3" else 6
    x = (1 + torch.arange(128, dtype=torch.float64) / 128)[None, :] * 2.0 ** -torch.arange(low, dtype=torch.float64)[:, None]
    x = x.flatten()
    per = size - 1
    x = torch.cat([x, x[:-x.numel() % per]]).view(-1, per)
    top = 2 * (1 + torch.arange(128, dtype=torch.float64) / 128)
    groups = torch.cat([top[:, None, None].expand(-1, x.shape[0], 1), x[None].expand(128, -1, -1)], 2).reshape(-1, size)
    groups[::2, 1:] *= -1
    n = -(-groups.shape[0] * size // 512)
    flat = torch.zeros(n * 512, dtype=torch.float64)
    flat[:groups.numel()] = groups.flatten()
    rows = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    rows[:, :512] = (flat.view(n, 512) * 2.0 ** power).to(torch.bfloat16).cuda()
    store = lib.alloc_quant_pool(1, n // 16 + 1, 16, codes)
    lib.quant_write(store, 0, rows, torch.arange(n, device="cuda"))
    same_bytes(store.data[0].view(-1, ROWS[codes])[:n], store_row(rows, codes), codes)


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_infinities_and_nan(lib, codes):
    n, size = 40, 128 if codes == "e4m3" else 32
    rows = rows_of(n, 5)
    rows[3, 130], rows[4, 7], rows[5, 511], rows[6, 520] = math.inf, -math.inf, math.nan, math.nan
    rows[7, :512] = 0
    store = lib.alloc_quant_pool(1, 4, 16, codes)
    slots = torch.arange(n, device="cuda")
    back = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    lib.quant_write(store, 0, rows, slots)
    lib.quant_read(store, 0, slots, rows=back)
    bad = torch.zeros(n, 576, dtype=torch.bool, device="cuda")
    for r, d in ((3, 130), (4, 7), (5, 511)):
        bad[r, d // size * size:d // size * size + size] = True
    bad[6, 520] = True
    assert torch.equal(back.isnan(), bad)
    assert bool((back[7, :512] == 0).all())
    same_bytes(store.data[0].view(-1, ROWS[codes])[:n], store_row(rows, codes), codes)


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_error_of_a_value(lib, codes):
    """e4m3: half a step of 3 mantissa bits, 2^-4 of the value, or of the smallest code (2^-9 of the scale);
    e2m1: at most a step of 2 at the top, 1 of a scale, which is off by 2^-8 of itself (six of them at the top)."""
    n = 2000
    rows = rows_of(n, 8)
    store = lib.alloc_quant_pool(1, n // 16, 16, codes)
    back = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, device="cuda")
    lib.quant_write(store, 0, rows, slots)
    lib.quant_read(store, 0, slots, rows=back)
    x, y = rows[:, :512].double(), back[:, :512].double()
    if codes == "e4m3":
        a = x.view(n, 4, 128).abs().amax(-1, keepdim=True).expand(-1, -1, 128).flatten(1) / 448
        bound = torch.maximum(x.abs() * 2.0 ** -4, a * 2.0 ** -10)
    else:
        a = x.view(n, 16, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32).flatten(1) / 6
        bound = a * (1 + 6 * BF16_HALF) * (1 + BF16_HALF)
    assert bool(((y - x).abs() <= bound * (1 + 1e-6) + BF16_HALF * (x.abs() + bound)).all())
    assert torch.equal(rows[:, 512:], back[:, 512:])


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
@pytest.mark.parametrize("into", ["rows", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 5, 8, 31, 32, 33, 1000, 4099])
def test_read(lib, codes, into, n):
    page = 32
    pages = n // page + 2
    store = lib.alloc_quant_pool(2, pages, page, codes)
    every = torch.arange(pages * page, device="cuda")
    lib.quant_write(store, 1, rows_of(pages * page, n), every)
    g = torch.Generator("cuda")
    g.manual_seed(n)
    slots = torch.randint(0, pages * page, (n,), generator=g, device="cuda")  # (some twice)
    value = store_values(store.data[1].view(-1, ROWS[codes])[slots])
    if into == "rows":
        back = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
        lib.quant_read(store, 1, slots, rows=back)
        assert torch.equal(back, value.float().to(torch.bfloat16))  # (products of 8 bits or fewer and 24: one rounding to fp32)
        return
    to = torch.randperm(pages * page, generator=g, device="cuda")[:n].contiguous()
    if into == "bf16":
        pool = lib.KVPool(torch.full((3, pages, page, 576), 7.0, dtype=torch.bfloat16, device="cuda"))
        want = pool.data.clone()
        want[2].view(-1, 576)[to] = value.float().to(torch.bfloat16)
    else:
        pool = lib.KVPool(torch.full((3, pages, page, 576), 7, dtype=torch.uint8, device="cuda"), 1 / 48)
        want = pool.data.clone()
        q = (value.float() / torch.tensor(pool.kv_scale, dtype=torch.float32, device="cuda")).clamp(-448, 448)
        want[2].view(-1, 576)[to] = q.to(torch.float8_e4m3fn).view(torch.uint8)
    lib.quant_read(store, 1, slots, pool=pool, pool_layer=2, pool_slots=to)
    assert torch.equal(pool.data, want)


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_every_code_reads_as_it_stands(lib, codes):
    store = lib.alloc_quant_pool(1, 1, 16, codes)
    flat = store.data[0].view(-1, ROWS[codes])
    every = torch.arange(256, dtype=torch.uint8, device="cuda")
    flat[:, :256] = every
    if codes == "e4m3":
        flat[:, 256:512] = every
        flat[:, 512:528] = torch.tensor([0.5, 3.0, 2.0 ** -9, 1.7], device="cuda").view(torch.uint8)
    else:
        flat[:, 256:288] = (torch.arange(16, device="cuda") * 0.37 + 0.1).to(torch.bfloat16).view(torch.uint8)
    back = torch.zeros(16, 576, dtype=torch.bfloat16, device="cuda")
    lib.quant_read(store, 0, torch.arange(16, device="cuda"), rows=back)
    want = store_values(flat).float().to(torch.bfloat16)
    assert torch.equal(back.isnan(), want.isnan()) and torch.equal(back.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_pad_rows_and_slots_out_of_range(lib, codes):
    n, last = 20, 4 * 16 - 1
    ws = lib.alloc_workspace(1, 16)
    store = lib.alloc_quant_pool(2, 4, 16, codes)
    store.data.fill_(0x21)
    rows = rows_of(n, 2)
    slots = torch.arange(n, device="cuda") + 3
    slots[4], slots[9] = -1, -(1 << 62)
    slots[7] = last
    keep = slots >= 0
    want = store.data.clone()
    want[0].view(-1, ROWS[codes])[slots[keep]] = store_row(rows, codes)[keep]
    lib.quant_write(store, 0, rows, slots, workspace=ws)
    assert lib.get_error(ws) == 0 and torch.equal(store.data, want)
    back = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.quant_read(store, 0, slots, rows=back, workspace=ws)
    value = store_values(want[0].view(-1, ROWS[codes])[slots.clamp(min=0)]).float().to(torch.bfloat16)
    assert torch.equal(back, torch.where(keep[:, None], value, 7.0)) and lib.get_error(ws) == 0
    pool = lib.KVPool(torch.full((1, 4, 16, 576), 7.0, dtype=torch.bfloat16, device="cuda"))
    to = torch.arange(n, device="cuda") + 30
    to[0], to[1] = -1, 4 * 16
    lib.quant_read(store, 0, slots, pool=pool, pool_slots=to, workspace=ws)
    assert lib.get_error(ws, clear=True) == lib.STATUS_BAD_SLOT
    expect = torch.full_like(pool.data, 7.0)
    ok = keep.clone()
    ok[:2] = False
    expect[0].view(-1, 576)[to[ok]] = value[ok]
    assert torch.equal(pool.data, expect)
    for bad in (4 * 16, 1 << 40):
        slots[2] = bad
        keep[2] = False
        before = store.data.clone()
        lib.quant_write(store, 0, rows, slots, workspace=ws)
        assert lib.get_error(ws, clear=True) == lib.STATUS_BAD_SLOT and torch.equal(store.data, before)
        back.fill_(7.0)
        lib.quant_read(store, 0, slots, rows=back, workspace=ws)
        assert lib.get_error(ws, clear=True) == lib.STATUS_BAD_SLOT
        assert torch.equal(back, torch.where(keep[:, None], value, 7.0))
        lib.quant_read(store, 0, slots, rows=back)  # without a status word: skipped in silence
    assert bool((store.data[1] == 0x21).all())


def test_rows_beyond_32_bit_offsets(lib):
    """Slots whose bytes lie beyond 2^31 and 2^32."""
    pages = (1 << 32) // (656 * 128) + 20
    store = lib.alloc_quant_pool(1, pages, 128)
    slots = torch.tensor([5, (1 << 31) // 656 + 1, (1 << 32) // 656 + 1, pages * 128 - 1], device="cuda")
    rows = rows_of(4, 12)
    lib.quant_write(store, 0, rows, slots)
    flat = store.data[0].view(-1, 656)
    assert torch.equal(flat[slots], store_row(rows, "e4m3"))
    back = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    lib.quant_read(store, 0, slots, rows=back)
    assert torch.equal(back, store_values(flat[slots]).float().to(torch.bfloat16))


def test_captured_and_replayed(lib):
    store = lib.alloc_quant_pool(1, 8, 16, "e2m1")
    rows, slots = rows_of(50, 1), torch.arange(50, device="cuda")
    back = torch.zeros(50, 576, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.quant_write(store, 0, rows, slots)
        lib.quant_read(store, 0, slots, rows=back)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.quant_write(store, 0, rows, slots)
        lib.quant_read(store, 0, slots, rows=back)
    for seed in (2, 3):
        rows.copy_(rows_of(50, seed))
        slots.copy_(torch.randperm(128, device="cuda")[:50])
        g.replay()
        assert torch.equal(back, store_values(store_row(rows, "e2m1")).float().to(torch.bfloat16))


@pytest.mark.parametrize("codes,fp8", [("e4m3", False), ("e2m1", False), ("e4m3", True)])
def test_a_prefix_from_the_store_into_decode(lib, codes, fp8):
    """As a service uses them: a prefix's rows into the store as they are computed, read back into pages of the
    pool when a batch comes for it, the requests' own tokens written beside it, one call for all."""
    page, prefix, n, own, layer = 32, 500, 6, [0, 40, 7, 130, 64, 33], 1
    c = Case([(n, prefix)], own, heads=16, page=page, fp8=fp8, seed=4)
    ws = lib.alloc_workspace_shared(n, 1, 16, 1)
    pool = lib.KVPool(torch.zeros_like(c.pool), c.scale)
    at = torch.arange(prefix, device="cuda")
    prefix_rows = c.rows(0)[:prefix].to(torch.bfloat16)
    store = lib.alloc_quant_pool(3, 40, page, codes)
    kept = torch.randperm(40 * page, device="cuda")[:prefix].contiguous()
    for t0 in range(0, prefix, 200):  # in chunks of a prompt
        lib.quant_write(store, 2, prefix_rows[t0:t0 + 200].contiguous(), kept[t0:t0 + 200].contiguous(), workspace=ws)
    slots = c.full[0, at // page].long() * page + at % page
    lib.quant_read(store, 2, kept, pool=pool, pool_layer=layer, pool_slots=slots, workspace=ws)
    rest = prefix % page
    for b in range(n):
        if b and rest:  # the page that the prefix ends in
            pool.data[layer, c.full[b, prefix // page].long(), :rest] = pool.data[layer, c.full[0, prefix // page].long(), :rest]
        t = torch.arange(prefix, prefix + own[b] + 1, device="cuda")
        new = c.rows(b)[prefix:].to(torch.bfloat16)
        lib.kv_write(pool, layer, new, c.full[b, t // page].long() * page + t % page, ws)
    out = torch.zeros(n, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, 1, 16, device="cuda")
    lib.plan_shared(c.ctx, c.indptr, c.prefix, 1, 16, page, ws)
    lib.decode_shared(pool, layer, c.q, 1, c.softmax_scale, ws, out, block_table=c.table, lse=lse)
    assert lib.get_error(ws) == 0
    c.clean = pool.data
    check(c, out, lse)


def test_refusals(lib):
    store = lib.alloc_quant_pool(2, 4, 16)
    rows, slots = rows_of(5), torch.arange(5, device="cuda")
    pool = lib.KVPool(torch.zeros(1, 2, 16, 576, dtype=torch.bfloat16, device="cuda"))
    lib.quant_write(store, 0, rows[:0], slots[:0])
    lib.quant_read(store, 0, slots[:0], rows=rows[:0])
    for bad in (dict(rows=rows[:, :512]), dict(rows=rows.float()), dict(rows=rows.cpu()), dict(slots=slots.int()),
                dict(slots=slots[:4]), dict(rows=rows[::2])):
        with pytest.raises(ValueError):
            lib.quant_write(store, 0, bad.get("rows", rows), bad.get("slots", slots))
    for data in (torch.zeros(2, 4, 16, 600, dtype=torch.uint8, device="cuda"), store.data.cpu(), store.data[0], store.data.int(),
                 store.data[:, ::2]):
        with pytest.raises(ValueError):
            lib.quant_write(lib.QuantPool(data), 0, rows, slots)
    for kw in (dict(), dict(rows=rows, pool=pool, pool_slots=slots), dict(rows=rows, pool_slots=slots), dict(rows=rows[:4]),
               dict(pool=pool, pool_slots=slots[:3])):
        with pytest.raises(ValueError):
            lib.quant_read(store, 0, slots, **kw)
    for layer in (-1, 2):
        with pytest.raises(lib.MlaError):
            lib.quant_write(store, layer, rows, slots)
        with pytest.raises(lib.MlaError):
            lib.quant_read(store, layer, slots, rows=rows)
    with pytest.raises(lib.MlaError):
        lib.quant_read(store, 0, slots, pool=pool, pool_layer=1, pool_slots=slots)
    with pytest.raises(lib.MlaError):
        lib.quant_write(lib.QuantPool(torch.zeros(1, 4, 48, 656, dtype=torch.uint8, device="cuda")), 0, rows, slots)
    with pytest.raises(ValueError):
        lib.alloc_quant_pool(1, 1, 16, "int4")
