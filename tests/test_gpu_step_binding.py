"""The compiled binding of the prefill step's calls: what it refuses, what it accepts
beside plain tensors and integers, and calls from several threads at once."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import paged_mla_decode_04_gb300 as m
    m.load_library()
    return m


def tables(**kw):
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    a = dict(context_lens=i(0, 20), new_lens=i(3, 5), free_pages=i(0, 1, 2, 3, 4, 5), free_count=i(6),
             block_table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), page_size=16, num_pages=6,
             slot_mapping=torch.zeros(10, dtype=torch.int64, device="cuda"), q_indptr=i(0, 0, 0), state=i(0, 0))
    a["block_table"][1, :2] = i(1, 2)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,error", [
    (dict(page_size="16"), TypeError), (dict(page_size=None), TypeError), (dict(num_pages=1.5), TypeError),
    (dict(num_pages=1 << 40), ValueError), (dict(num_pages=1 << 70), OverflowError),
    (dict(context_lens=[0, 20]), ValueError), (dict(new_lens=None), ValueError), (dict(state=7), ValueError),
    (dict(slot_mapping=torch.zeros(10, dtype=torch.int64)), ValueError), (dict(workspace=b"x"), ValueError),
    (dict(stream=5), AttributeError)])
def test_arguments_of_other_kinds_are_refused(lib, bad, error):
    a = tables(**bad)
    with pytest.raises(error):
        lib.extend_tables(**a)
    torch.cuda.synchronize()
    if isinstance(a["slot_mapping"], torch.Tensor) and a["slot_mapping"].is_cuda:
        assert not a["slot_mapping"].any()


def test_layouts_and_devices(lib):
    """Strided tensors, other types and sparse ones are refused, a zero-size list is not."""
    for bad in (dict(context_lens=torch.zeros(4, dtype=torch.int32, device="cuda")[::2]),
                dict(free_pages=torch.zeros(6, dtype=torch.int64, device="cuda")),
                dict(block_table=torch.zeros(4, 2, dtype=torch.int32, device="cuda").t()),
                dict(q_indptr=torch.zeros(3, dtype=torch.int32, device="meta"))):
        with pytest.raises(ValueError):
            lib.extend_tables(**tables(**bad))
    with pytest.raises((ValueError, RuntimeError)):
        lib.extend_tables(**tables(state=torch.zeros(2, dtype=torch.int32, device="cuda").to_sparse()))
    a = tables(page_indptr=torch.zeros(3, dtype=torch.int32, device="cuda"),
               page_ids=torch.zeros(0, dtype=torch.int32, device="cuda"))
    lib.extend_tables(**a)
    assert a["page_indptr"].tolist() == [0, 1, 3]


def test_numpy_integers_and_parameters(lib):
    a = tables(page_size=np.int64(16), num_pages=np.int32(6))
    a["slot_mapping"] = torch.nn.Parameter(a["slot_mapping"], requires_grad=False)
    lib.extend_tables(**a)
    # request 0 gets page 5 from the top of the stack, request 1 goes on in its page 2
    assert a["slot_mapping"].tolist() == [80, 81, 82, 36, 37, 38, 39, 40, -1, -1]
    assert a["state"].tolist() == [5, 2] and a["q_indptr"].tolist() == [0, 3, 8]


def test_threads_at_once(lib):
    """Four threads, each with a stream, a cache and a workspace of its own, make the same calls."""
    g = torch.Generator("cuda")
    g.manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    H, n = 16, 37
    q, w_uk, w_uv, rows = r(n, H, 192), r(H, 128, 512) * 0.04, r(H, 512, 128) * 0.04, r(n, 576)
    cos_sin = torch.rand(64, 64, generator=g, device="cuda")
    outs, errors = [], []
    sets = []
    for k in range(4):
        pool = lib.KVPool(torch.zeros(1, 6, 16, 576, dtype=torch.bfloat16, device="cuda"))
        a = tables(context_lens=torch.zeros(1, dtype=torch.int32, device="cuda"),
                   new_lens=torch.full((1,), n, dtype=torch.int32, device="cuda"),
                   block_table=torch.full((1, 4), -1, dtype=torch.int32, device="cuda"),
                   q_indptr=torch.zeros(2, dtype=torch.int32, device="cuda"),
                   slot_mapping=torch.zeros(n, dtype=torch.int64, device="cuda"),
                   positions=torch.zeros(n, dtype=torch.int32, device="cuda"))
        sets.append((pool, a, lib.alloc_prefill_workspace(1, n, 64, H), torch.cuda.Stream(),
                     torch.zeros(n, H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)))
    torch.cuda.synchronize()

    def work(pool, a, ws, stream, out, turned):
        try:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    lib.extend_tables(**a)
                    lib.rope_write(pool, 0, rows, a["slot_mapping"], a["positions"], cos_sin, q_rope=q[:, :, 128:],
                                   q_out=turned[:, :, 128:])
                    turned[:, :, :128] = q[:, :, :128]
                    lib.prefill(pool, 0, turned, a["q_indptr"], a["context_lens"], 192 ** -0.5, w_uk, w_uv, ws, out, 64,
                                block_table=a["block_table"])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    outs = [s[4] for s in sets]
    assert outs[0].float().std() > 0.05
    for s in sets:
        assert torch.equal(s[4].view(torch.int16), outs[0].view(torch.int16)) and lib.get_error(s[2]) == 0
