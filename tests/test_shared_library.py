"""Refusals of the shared-prefix and compact-store entry points that need no GPU, and the
plain forms that their GPU tests compare with."""
import ctypes

import pytest
import torch

import shared_ref

ARG, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from paged_mla_decode_04_gb300 import _build
    import paged_mla_decode_04_gb300 as m
    return m.load_library(_build.build())


@pytest.fixture(scope="module")
def mem():
    """Host memory that stands for device pointers; no accepted call is made with it."""
    buf = ctypes.create_string_buffer(1 << 16)
    mem.buf = buf
    return (ctypes.addressof(buf) + 1023) // 1024 * 1024


class Store(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int) for n in ("num_layers", "num_pages", "page_size", "format")]


def store(mem, **kw):
    return bytes(Store(**{**dict(data=mem, num_layers=2, num_pages=4, page_size=16, format=0), **kw}))


def pool(mem, **kw):
    import paged_mla_decode_04_gb300 as m
    d = {**dict(data=mem, num_layers=2, num_pages=4, page_size=16, dtype=0, kv_scale=1.0), **kw}
    return bytes(m._Pool(*[d[n] for n in ("data", "num_layers", "num_pages", "page_size", "dtype", "kv_scale")]))


def test_workspace_size_refuses(lib):
    for bad in [(-1, 1, 16, 1), (4, 0, 16, 1), (4, 1, 0, 1), (4, 1, 1025, 1), (4, 1, 16, -1), (1 << 20, 2, 1024, 1), ((1 << 22) + 1, 1, 1, 1), (4, 1, 16, (1 << 22) + 1),
                (1, 1 << 20, 1024, 1)]:
        assert lib.mla_decode_workspace_size_shared(*bad) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), ARG), (dict(q_len=0), ARG), (dict(num_heads=0), ARG), (dict(num_heads=1025), ARG), (dict(num_prefixes=-1), ARG),
    (dict(num_clusters=-1), ARG), (dict(page_size=48), UNSUPPORTED), (dict(context_lens=None), ARG),
    (dict(prefix_indptr=None), ARG), (dict(prefix_lens=None), ARG), (dict(workspace=None), WORKSPACE),
    (dict(workspace=8), WORKSPACE)])
def test_plan(lib, mem, bad, code):
    a = dict(context_lens=mem, prefix_indptr=mem, prefix_lens=mem, batch=2, num_prefixes=1, q_len=1, num_heads=16, page_size=16,
             num_clusters=0, workspace=mem, workspace_bytes=1 << 14, stream=None)
    a.update(bad)
    if a["workspace"] == 8:
        a["workspace"] = mem + 8
    assert lib.mla_decode_plan_shared(*a.values()) == code


@pytest.mark.parametrize("bad,code", [
    (dict(pool=None), ARG), (dict(pool="page"), ARG), (dict(layer=2), ARG), (dict(layer=-1), ARG), (dict(batch=-1), ARG),
    (dict(q_len=0), ARG), (dict(num_heads=0), ARG), (dict(num_prefixes=-1), ARG), (dict(softmax_scale=0.0), ARG),
    (dict(softmax_scale=float("nan")), ARG), (dict(q=None), ARG), (dict(q=8), ARG), (dict(out=None), ARG), (dict(out=16), ARG),
    (dict(page_ids=None), ARG), (dict(max_blocks=0), ARG), (dict(workspace=None), WORKSPACE), (dict(workspace=8), WORKSPACE),
    (dict(pool="rows"), UNSUPPORTED), (dict(batch=0), 0), (dict(num_prefixes=0), 0)])
def test_decode(lib, mem, bad, code):
    a = dict(pool=pool(mem), layer=0, q=mem, page_indptr=None, page_ids=mem, max_blocks=4, batch=2, q_len=1, num_heads=16,
             num_prefixes=1, softmax_scale=0.1, workspace=mem, out=mem, lse=None, stream=None)
    a.update(bad)
    if a["pool"] in ("page", "rows"):
        a["pool"] = pool(mem, page_size=48) if a["pool"] == "page" else pool(mem, num_pages=1 << 27)
    for k in ("q", "out", "workspace"):
        if isinstance(a[k], int) and a[k] < 64:
            a[k] += mem
    assert lib.mla_decode_shared(*a.values()) == code


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), ARG), (dict(pool=None), ARG), (dict(pool="format"), ARG), (dict(pool="page"), ARG), (dict(pool="align"), ARG),
    (dict(layer=2), ARG), (dict(rows=None), ARG), (dict(rows=8), ARG), (dict(slots=None), ARG), (dict(workspace=8), WORKSPACE),
    (dict(n=0), 0)])
def test_write(lib, mem, bad, code):
    a = dict(pool=store(mem), layer=0, rows=mem, slots=mem, n=3, workspace=None, stream=None)
    a.update(bad)
    odd = {"format": dict(format=2), "page": dict(page_size=8), "align": dict(data=mem + 8)}
    if a["pool"] in odd:
        a["pool"] = store(mem, **odd[a["pool"]])
    for k in ("rows", "workspace"):
        if a[k] == 8:
            a[k] = mem + 8
    assert lib.mla_quant_write(*a.values()) == code


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), ARG), (dict(pool=None), ARG), (dict(layer=-1), ARG), (dict(slots=None), ARG), (dict(rows=None), ARG),
    (dict(rows=8), ARG), (dict(into=0), ARG), (dict(into=0, rows=None), ARG), (dict(into=0, rows=None, into_slots=1, into_layer=2), ARG),
    (dict(into_slots=1), ARG), (dict(workspace=8), WORKSPACE), (dict(n=0), 0), (dict(n=0, rows=None), 0)])
def test_read(lib, mem, bad, code):
    a = dict(pool=store(mem), layer=0, slots=mem, n=3, into=None, into_layer=0, into_slots=None, rows=mem, workspace=None, stream=None)
    a.update(bad)
    if a["into"] == 0:
        a["into"] = pool(mem)
    if a["into_slots"] == 1:
        a["into_slots"] = mem
    for k in ("rows", "workspace"):
        if a[k] == 8:
            a[k] = mem + 8
    assert lib.mla_quant_read(*a.values()) == code


def test_compiled_binding(lib):
    import paged_mla_decode_04_gb300 as m
    b = m._step()
    for name, n in (("plan_shared", 9), ("decode_shared", 13), ("quant_write", 6), ("quant_read", 10), ("bind_shared", 5)):
        with pytest.raises(TypeError, match="%d arguments expected" % n):
            getattr(b, name)()
    with pytest.raises(ValueError, match="entry point"):
        b.bind_shared(0, 0, 0, 0, 0)


@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_plain_store(codes):
    """The tests' own form: known codes, ties to even, and a value's error."""
    rows = torch.zeros(2, 576, dtype=torch.bfloat16)
    if codes == "e4m3":
        rows[0, :4] = torch.tensor([448.0, 17.0, 19.0, -2.0 ** -9])  # 17 and 19: between 16, 18 and 20 (mantissas 0, 1, 2)
        data = shared_ref.store_row(rows, codes)
        assert data.shape == (2, 656)
        assert data[0, :4].tolist() == [0x7E, 0x58, 0x5A, 0x81]
        assert data[0, 512:516].view(torch.float32).item() == 1.0
    else:
        rows[0, :8] = torch.tensor([6.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, -5.0])
        data = shared_ref.store_row(rows, codes)
        assert data.shape == (2, 416)
        code = [7, 0, 2, 10, 4, 4, 6, 14]  # each tie to the even code
        assert data[0, :4].tolist() == [code[2 * i] | code[2 * i + 1] << 4 for i in range(4)]
        assert data[0, 256:258].view(torch.bfloat16).item() == 1.0
    assert torch.equal(shared_ref.store_values(data)[1], torch.zeros(576, dtype=torch.float64))


def test_plain_decode():
    """One request of a group against a softmax over rows gathered one by one; tables that name no page are not used."""
    c = shared_ref.Case([(3, 20)], [5, 0, 30], heads=2, q_len=2, page=16, device="cpu")
    out, lse, bound, _ = c.reference(2)
    rows = [c.pool[1, int(c.table[2 if t >= 20 else 0, t // 16]), t % 16].double() for t in range(20 + 30 + 2)]
    for i in range(2):
        k = torch.stack(rows[:51 + i])
        w = torch.softmax(c.q[2, i].double() @ k.T * c.softmax_scale, -1)
        assert torch.allclose(out[i], w @ k[:, :512], atol=1e-12)
    assert bool((bound > 0).all()) and bool(c.pool.isnan().any()) and not bool(out.isnan().any())
