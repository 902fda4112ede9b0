"""Timed cases of decode over a shared prefix and of a compact latent store.

Three operators that serving many requests behind one long prefix (a system
prompt, a document, a set of examples) needs:

  shared   decode_shared: absorbed MLA decode of a batch whose requests share
           their first positions in groups; a group's prefix is attended once
           for all its requests, each request's own positions by itself.
  write    quant_write: latent rows into a paged store of e4m3 codes with an
           fp32 scale for each 128 dims (656 bytes a token instead of 1,152).
  read     quant_read: rows of such a store, or of one with 4-bit codes and a
           scale for each 32 dims (416 bytes), back as bf16 rows or into the
           pages of a decode pool (bf16 or e4m3).

Every case is a dict of plain values; `prepare` makes its inputs from a seed,
`run` makes one pass: the plain torch form, or (where `own` is true) the
library's own call on the same inputs. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

CKV, ROPE, ROW = 512, 64, 576
E4M3_ROW, E2M1_ROW = 656, 416
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # what the 4-bit codes 0 to 7 stand for; 8 to 15 are their negatives


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest call: two requests behind a few shared pages, 16 heads
        {"name": "shared_two", "kind": "shared", "batch": 2, "q_len": 1, "heads": 16, "page": 16, "fp8": False,
         "prefixes": 1, "prefix_lo": 96, "prefix_hi": 96, "own_lo": 5, "own_hi": 40},
        # a decode step of a chat service: one system prompt, uneven conversations
        {"name": "shared_chat", "kind": "shared", "batch": 64, "q_len": 1, "heads": 16, "page": 64, "fp8": False,
         "prefixes": 1, "prefix_lo": 4096, "prefix_hi": 4096, "own_lo": 1, "own_hi": 1500},
        # several applications in one batch, each with a prompt of its own length
        {"name": "shared_groups", "kind": "shared", "batch": 90, "q_len": 1, "heads": 32, "page": 32, "fp8": False,
         "prefixes": 5, "prefix_lo": 700, "prefix_hi": 6001, "own_lo": 1, "own_hi": 2048},
        # a step that checks two drafted tokens a request, e4m3 pool
        {"name": "shared_drafts", "kind": "shared", "batch": 40, "q_len": 3, "heads": 32, "page": 128, "fp8": True,
         "prefixes": 1, "prefix_lo": 3001, "prefix_hi": 3001, "own_lo": 64, "own_hi": 1024},
        # many questions about one document, 128 heads
        {"name": "shared_document", "kind": "shared", "batch": 8, "q_len": 1, "heads": 128, "page": 64, "fp8": False,
         "prefixes": 1, "prefix_lo": 65536, "prefix_hi": 65536, "own_lo": 16, "own_hi": 200},
        # many samples of one long prompt, 128 heads: the largest product
        {"name": "shared_samples", "kind": "shared", "batch": 128, "q_len": 1, "heads": 128, "page": 64, "fp8": False,
         "prefixes": 1, "prefix_lo": 8192, "prefix_hi": 8192, "own_lo": 1, "own_hi": 512},
        # the new tokens of a decode step
        {"name": "write_step", "kind": "write", "tokens": 128, "page": 64},
        # a prompt as it is computed
        {"name": "write_prompt", "kind": "write", "tokens": 8191, "page": 16},
        # a batch of long prompts
        {"name": "write_bulk", "kind": "write", "tokens": 131072, "page": 64},
        # the tail of a prefix, 4-bit codes
        {"name": "read_tail", "kind": "read", "tokens": 33, "page": 16, "codes": "e2m1", "into": "rows"},
        # a prefix brought back into the pages of a decode pool
        {"name": "read_prefix", "kind": "read", "tokens": 8192, "page": 64, "codes": "e4m3", "into": "bf16"},
        # a long document from 4-bit codes
        {"name": "read_document", "kind": "read", "tokens": 131072, "page": 64, "codes": "e2m1", "into": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "write", "read"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "write":
        return {"kind": kind, "tokens": _log(rng, 1, 131072), "page": page}
    if kind == "read":
        return {"kind": kind, "tokens": _log(rng, 1, 131072), "page": page, "codes": rng.choice(["e4m3", "e2m1"]),
                "into": rng.choice(["rows", "bf16", "e4m3"])}
    heads, q_len = rng.choice([8, 16, 24, 32, 64, 128]), rng.choice([1, 1, 2, 4])
    prefix, own_hi = _log(rng, 16, 65536), _log(rng, 1, 4096)
    # rows x positions of no draw outgrow the largest listed case's
    most = min(256, 120_000_000 // (heads * q_len * (prefix + own_hi)), 300_000 // own_hi)
    batch = _log(rng, 1, max(1, most))
    prefixes = min(batch, rng.choice([1, 1, 1, 2, 3, 6]))
    return {"kind": kind, "batch": batch, "q_len": q_len, "heads": heads, "page": page, "fp8": rng.random() < 0.4,
            "prefixes": prefixes, "prefix_lo": prefix if prefixes == 1 else rng.randint(1, prefix), "prefix_hi": prefix,
            "own_lo": rng.randint(0, own_hi), "own_hi": own_hi}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Each prefix's length and number of requests, and each request's own cached tokens; the same for every seed, so that work() knows them."""
    b, g = case["batch"], case["prefixes"]
    lo, hi = case["prefix_lo"], case["prefix_hi"]
    prefix = [hi if i == 0 else lo + round(((i * 0.6180339887498949) % 1.0) * (hi - lo)) for i in range(g)]
    share = [1.0 + (i * 0.7548776662466927) % 1.0 for i in range(g)]  # uneven groups
    ends = [round(b * sum(share[:i + 1]) / sum(share)) for i in range(g)]
    lo, hi = case["own_lo"], case["own_hi"]
    mine = [lo + round(((i * 0.6180339887498949 + 0.5) % 1.0) ** 2 * (hi - lo)) for i in range(b)]
    return prefix, [e - s for s, e in zip([0] + ends, ends)], mine


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = {"case": case, "kind": case["kind"]}
    if own:
        import paged_mla_decode_04_gb300 as lib
        s["lib"] = lib
    {"shared": _prepare_shared, "write": _prepare_write, "read": _prepare_read}[case["kind"]](case, s, gen, dev)
    return s


def _normal(gen, dev, *shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    out.normal_(0.0, std, generator=gen)
    return out


def _pool(gen, dev, fp8, pages, page, layers=1):
    """A latent pool of normal values, and its scale; e4m3 codes as bytes."""
    pool = _normal(gen, dev, layers, pages, page, ROW)
    if not fp8:
        return pool, 1.0
    return (pool.float() * 64).to(torch.float8_e4m3fn).view(torch.uint8), 1.0 / 64


def _prepare_shared(case, s, gen, dev):
    page, h, ql = case["page"], case["heads"], case["q_len"]
    prefix, sizes, mine = _lengths(case)
    which = [g for g, n in enumerate(sizes) for _ in range(n)]
    ctx = [prefix[g] + m for g, m in zip(which, mine)]
    # a prefix's whole pages are the group's, the page that it ends in is each request's own copy
    whole = [p // page for p in prefix]
    blocks = [(c + ql + page - 1) // page for c in ctx]
    total = sum(whole) + sum(n - whole[g] for n, g in zip(blocks, which))
    ids = torch.randperm(total + 16, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(ctx), max(blocks)), -1, dtype=torch.int32, device=dev)
    at, first = 0, []
    for w in whole:
        first.append(at)
        at += w
    for b, g in enumerate(which):
        table[b, :whole[g]] = ids[first[g]:first[g] + whole[g]]
        table[b, whole[g]:blocks[b]] = ids[at:at + blocks[b] - whole[g]]
        at += blocks[b] - whole[g]
    s["pool"], s["scale"] = _pool(gen, dev, case["fp8"], total + 16, page, layers=2)
    head = {}
    for b, g in enumerate(which):
        rest = prefix[g] % page
        if rest:
            head.setdefault(g, table[b, whole[g]].long())
            s["pool"][1, table[b, whole[g]].long(), :rest] = s["pool"][1, head[g], :rest]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    i32 = {"dtype": torch.int32, "device": dev}
    s["table"], s["ctx"] = table, torch.tensor(ctx, **i32)
    s["indptr"], s["prefix"] = torch.tensor(starts, **i32), torch.tensor(prefix, **i32)
    s["longest_prefix"], s["most_requests"], s["longest_own"] = max(prefix), max(sizes), max(mine) + ql
    s["q"] = _normal(gen, dev, len(ctx), ql, h, ROW)
    s["softmax_scale"] = (128 + ROPE) ** -0.5
    s["out"] = torch.zeros(len(ctx), ql, h, CKV, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(len(ctx), ql, h, dtype=torch.float32, device=dev)
    if own:
        # the step's plan, made once from the lengths and used by every layer's call
        lib = s["lib"]
        s["kv"] = lib.KVPool(s["pool"], s["scale"])
        s["ws"] = lib.alloc_workspace_shared(len(ctx), ql, h, len(prefix))
        lib.plan_shared(s["ctx"], s["indptr"], s["prefix"], ql, h, page, s["ws"])


def _prepare_write(case, s, gen, dev):
    n, page = case["tokens"], case["page"]
    pages = (n + page - 1) // page + 4
    store = torch.randint(0, 256, (1, pages, page, E4M3_ROW), dtype=torch.uint8, generator=gen, device=dev)
    store[..., :CKV] &= 0x77  # (rows that this call leaves hold finite values)
    _scales(store).copy_(torch.rand(1, pages, page, 4, generator=gen, device=dev) * 0.02 + 0.001)
    _rope(store).normal_(generator=gen)
    s["store"] = store
    # latent rows after their norm: sizes differ from dim to dim and from token to token
    size = torch.exp(0.5 * torch.randn(CKV, generator=gen, device=dev))
    rows = torch.randn(n, ROW, generator=gen, device=dev)
    rows[:, :CKV] *= size * torch.exp(0.3 * torch.randn(n, 1, generator=gen, device=dev))
    s["rows"] = rows.to(torch.bfloat16)
    s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:n].contiguous()
    if own:
        s["qp"] = s["lib"].QuantPool(store)


def _prepare_read(case, s, gen, dev):
    n, page = case["tokens"], case["page"]
    pages = (n + page - 1) // page + 4
    x = _normal(gen, dev, 1, pages, page, CKV).float()
    if case["codes"] == "e4m3":
        store = torch.zeros(1, pages, page, E4M3_ROW, dtype=torch.uint8, device=dev)
        g = x.unflatten(-1, (4, 128))
        scale = g.abs().amax(-1) / 448
        store[..., :CKV] = (g / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
        _scales(store).copy_(scale)
    else:
        store = torch.zeros(1, pages, page, E2M1_ROW, dtype=torch.uint8, device=dev)
        g = x.unflatten(-1, (16, 32))
        scale = (g.abs().amax(-1) / 6).to(torch.bfloat16)
        middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
        code = torch.bucketize((g / scale[..., None].float()).abs(), middle) + 8 * (g < 0)
        code = code.flatten(-2).to(torch.uint8)
        store[..., :256] = code[..., 0::2] | (code[..., 1::2] << 4)
        _scales(store).copy_(scale)
    _rope(store).normal_(generator=gen)
    s["store"] = store
    s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:n].contiguous()
    if case["into"] == "rows":
        s["rows"] = torch.zeros(n, ROW, dtype=torch.bfloat16, device=dev)
    else:
        s["pool"], s["scale"] = _pool(gen, dev, case["into"] == "e4m3", pages, page)
        s["to"] = torch.randperm(pages * page, generator=gen, device=dev)[:n].contiguous()
    if own:
        lib = s["lib"]
        s["qp"] = lib.QuantPool(store)
        if case["into"] != "rows":
            s["kv"] = lib.KVPool(s["pool"], s["scale"])


def _codes8(store):
    return store[..., :CKV].view(torch.float8_e4m3fn)


def _scales(store):
    if store.shape[-1] == E4M3_ROW:
        return store[..., CKV:CKV + 16].view(torch.float32)
    return store[..., 256:288].view(torch.bfloat16)


def _rope(store):
    return store[..., -2 * ROPE:].view(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"shared": _own_shared, "write": _own_write, "read": _own_read}[s["kind"]](s)
    return {"shared": _plain_shared, "write": _plain_write, "read": _plain_read}[s["kind"]](s)


def _own_shared(s):
    s["lib"].decode_shared(s["kv"], 1, s["q"], s["case"]["prefixes"], s["softmax_scale"], s["ws"], s["out"],
                           block_table=s["table"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_write(s):
    s["lib"].quant_write(s["qp"], 0, s["rows"], s["slots"])
    return _write_out(s)


def _write_out(s):
    return {"codes": _codes8(s["store"]), "scales": _scales(s["store"]), "rope": _rope(s["store"])}


def _own_read(s):
    if s["case"]["into"] == "rows":
        s["lib"].quant_read(s["qp"], 0, s["slots"], rows=s["rows"])
    else:
        s["lib"].quant_read(s["qp"], 0, s["slots"], pool=s["kv"], pool_layer=0, pool_slots=s["to"])
    return _read_out(s)


def _read_out(s):
    if s["case"]["into"] == "rows":
        return s["rows"]
    return s["pool"].view(torch.float8_e4m3fn) if s["case"]["into"] == "e4m3" else s["pool"]


# ------------------------------------------------------------------ plain forms

def _latent(s, ids, offset):
    got = s["pool"][1][ids.long().clamp(min=0), offset]
    return got.view(torch.float8_e4m3fn).float() * s["scale"] if s["case"]["fp8"] else got.float()


def _part(q, rows, seen, scale):
    """Scores' maximum, sum of weights and weighted rows of q [n, r, 576] over rows [n, t, 576] where seen [n, r or 1, t]."""
    x = (q @ rows.transpose(1, 2)).mul_(scale)
    x.masked_fill_(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(top).exp_()
    return top, x.sum(-1, keepdim=True), x @ rows[..., :CKV]


def _plain_shared(s):
    case, dev = s["case"], s["q"].device
    b, ql, h, page = case["batch"], case["q_len"], case["heads"], case["page"]
    ctx, starts, prefix = s["ctx"].long(), s["indptr"].long(), s["prefix"].long()
    # the prefixes, one batch entry a group
    t = torch.arange(s["longest_prefix"], device=dev)
    rows = _latent(s, s["table"][starts[:-1].clamp(max=b - 1)][:, t // page], t % page)
    seen = t[None, :] < prefix[:, None]
    rows = torch.where(seen[:, :, None], rows, 0.0)
    i = torch.arange(s["most_requests"], device=dev)
    real = i[None, :] < (starts[1:] - starts[:-1])[:, None]
    q = s["q"][(starts[:-1, None] + i).clamp(max=b - 1)].float()
    top1, sum1, acc1 = (x.unflatten(1, (-1, ql * h))[real] for x in _part(q.flatten(1, 3), rows, seen[:, None], s["softmax_scale"]))
    # each request's own positions
    mine = prefix.repeat_interleave(starts[1:] - starts[:-1], output_size=b)
    at = mine[:, None] + torch.arange(s["longest_own"], device=dev)
    here = at < (ctx + ql)[:, None]
    blocks = (at // page).clamp(max=s["table"].shape[1] - 1)
    rows = torch.where(here[:, :, None], _latent(s, s["table"].gather(1, blocks), at % page), 0.0)
    last = (ctx[:, None] + torch.arange(ql, device=dev)).repeat_interleave(h, 1)
    top2, sum2, acc2 = _part(s["q"].float().flatten(1, 2), rows, at[:, None, :] <= last[:, :, None], s["softmax_scale"])
    top = torch.maximum(top1, top2)
    f1, f2 = (top1 - top).exp(), (top2 - top).exp()
    total = sum1 * f1 + sum2 * f2
    s["out"].copy_(((acc1 * f1 + acc2 * f2) / total).view(b, ql, h, CKV))
    s["lse"].copy_((top + total.log()).view(b, ql, h))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_write(s):
    rows, store = s["rows"].float(), s["store"]
    g = rows[:, :CKV].unflatten(1, (4, 128))
    scale = g.abs().amax(-1) / 448
    code = torch.where(scale[..., None] > 0, g / scale[..., None], 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    flat = store[0].view(-1, E4M3_ROW)
    flat[s["slots"]] = torch.cat([code.flatten(1).view(torch.uint8), scale.view(torch.uint8),
                                  s["rows"][:, CKV:].contiguous().view(torch.uint8)], 1)
    return _write_out(s)


def _plain_read(s):
    case = s["case"]
    row = s["store"][0].view(-1, s["store"].shape[-1])[s["slots"]]
    if case["codes"] == "e4m3":
        value = _codes8(row).float().unflatten(1, (4, 128)) * _scales(row)[..., None]
    else:
        code = torch.stack([row[:, :256] & 15, row[:, :256] >> 4], -1).flatten(1).int()
        level = torch.tensor(LEVELS + [-x for x in LEVELS], device=row.device)
        value = level[code].unflatten(1, (16, 32)) * _scales(row).float()[..., None]
    value = torch.cat([value.flatten(1), _rope(row).float()], 1)
    if case["into"] == "rows":
        s["rows"].copy_(value)
    elif case["into"] == "bf16":
        s["pool"][0].view(-1, ROW)[s["to"]] = value.to(torch.bfloat16)
    else:
        s["pool"][0].view(-1, ROW)[s["to"]] = (value / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _read_out(s)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "write": _exact_write, "read": _exact_read}[case["kind"]](case, s)


def _exact_shared(case, s):
    """One request after another over all the positions that its tokens see, by its own block table."""
    _, _, mine = _lengths(case)
    ctx = s["ctx"].tolist()
    ql, h = case["q_len"], case["heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    for b, c in enumerate(ctx):
        pages = s["table"][b, :(c + ql + case["page"] - 1) // case["page"]].long()
        got = s["pool"][1][pages].flatten(0, 1)[:c + ql]
        lat = (got.view(torch.float8_e4m3fn).float() if case["fp8"] else got).double() * s["scale"]
        score = torch.einsum("ihd,td->iht", s["q"][b].double(), lat) * s["softmax_scale"]
        for i in range(ql):
            score[i, :, c + i + 1:] = -math.inf
        lse[b] = torch.logsumexp(score, -1)
        out[b] = torch.einsum("iht,td->ihd", torch.exp(score - lse[b][..., None]), lat[:, :CKV])
    return {"out": out, "lse": lse}


def _exact_write(case, s):
    x = s["rows"].double()
    codes, scales, rope = (v.double() for v in _write_out(s).values())
    at = (s["slots"] // case["page"], s["slots"] % case["page"])
    groups = x[:, :CKV].reshape(-1, 4, 128)
    scale = torch.linalg.vector_norm(groups, ord=math.inf, dim=-1) / 448
    codes[0][at] = (groups / scale.clamp(min=1e-300)[..., None]).reshape(-1, CKV)
    scales[0][at] = scale
    rope[0][at] = x[:, CKV:]
    return {"codes": codes, "scales": scales, "rope": rope}


def _exact_read(case, s):
    store, page = s["store"][0], case["page"]
    row = store[s["slots"] // page, s["slots"] % page]
    if case["codes"] == "e4m3":
        v = _codes8(row).float().double().reshape(-1, 4, 128)
    else:
        half = torch.empty(row.shape[0], CKV, dtype=torch.int64, device=row.device)
        half[:, 0::2] = row[:, :256].long() % 16
        half[:, 1::2] = row[:, :256].long() // 16
        mag = half % 8
        # exponent and mantissa of a code: 0 and 1/2 below, (1 + m / 2) 2^(e - 1) from e = 1 on
        v = torch.where(mag < 2, mag / 2.0, (1 + (mag % 2) / 2.0) * 2.0 ** (mag // 2 - 1).double()).double()
        v = torch.where(half >= 8, -v, v).reshape(-1, 16, 32)
    v = torch.cat([(v * _scales(row).double()[..., None]).reshape(-1, CKV), _rope(row).double()], 1)
    if case["into"] == "rows":
        return v
    pool = (s["pool"].view(torch.float8_e4m3fn).float() if case["into"] == "e4m3" else s["pool"]).double()
    pool[0][s["to"] // page, s["to"] % page] = (v / s["scale"]).clamp(-448, 448) if case["into"] == "e4m3" else v
    return pool


# ------------------------------------------------------------------ work

def work(case):
    if case["kind"] == "write":
        return {"bytes": case["tokens"] * (2 * ROW + E4M3_ROW + 8), "flops": case["tokens"] * CKV * 2}
    if case["kind"] == "read":
        n = case["tokens"]
        source = E4M3_ROW if case["codes"] == "e4m3" else E2M1_ROW
        target = {"rows": 2 * ROW, "bf16": 2 * ROW + 8, "e4m3": ROW + 8}[case["into"]]
        return {"bytes": n * (source + target + 8), "flops": n * CKV}
    h, ql = case["heads"], case["q_len"]
    prefix, sizes, mine = _lengths(case)
    which = [g for g, n in enumerate(sizes) for _ in range(n)]
    rows = sum(p for p, n in zip(prefix, sizes) if n) + sum(mine) + len(mine) * ql
    pairs = sum(ql * (prefix[g] + m) + ql * (ql + 1) // 2 for g, m in zip(which, mine)) * h
    q_rows = len(mine) * ql * h
    pages = sum((p + case["page"] - 1) // case["page"] for p in prefix) + sum(m // case["page"] + 1 for m in mine)
    return {"bytes": rows * ROW * (1 if case["fp8"] else 2) + q_rows * (ROW + CKV + 2) * 2 + pages * 4,
            "flops": pairs * 2 * (ROW + CKV)}
