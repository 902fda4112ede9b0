"""Timed cases of a chunked-prefill step on a paged MLA latent cache.

Three operators that a serving step runs one after the other:

  tables   extend_tables: block tables, slot map, positions and CSR page lists
           of the step's new tokens, built on the GPU from request lengths and
           a stack of free pages.
  rope     rope_write: RMS norm of the new latent rows, rotary positions with
           one to three axes on their rope part and on the queries' rope part,
           and the write into the paged cache (bf16 or e4m3).
  prefill  prefill: causal attention of a ragged chunk of new tokens per
           request over the paged cache, in the 192/128 multi-head form.

Every case is a dict of plain values; `prepare` makes its inputs from a seed,
`run` makes one pass: the plain torch form, or (where `own` is true) the
library's own call on the same inputs. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

CKV, ROPE, ROW = 512, 64, 576
NOPE, VDIM, QK = 128, 128, 192
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 128: a slot each, a new page for few
        {"name": "tables_decode", "kind": "tables", "batch": 128, "page": 64, "ctx_lo": 256, "ctx_hi": 8192,
         "new_lo": 1, "new_hi": 1},
        # a step that mixes prompt chunks with single tokens, small pages
        {"name": "tables_mixed", "kind": "tables", "batch": 61, "page": 16, "ctx_lo": 0, "ctx_hi": 4096,
         "new_lo": 1, "new_hi": 1500},
        # a thousand long requests: the CSR list of over a million pages is what counts
        {"name": "tables_long", "kind": "tables", "batch": 1024, "page": 64, "ctx_lo": 32768, "ctx_hi": 131072,
         "new_lo": 1, "new_hi": 4},
        # the smallest call: two requests' tokens of a 16-head decode step
        {"name": "rope_two", "kind": "rope", "tokens": 2, "heads": 16, "page": 16, "fp8": False, "axes": 1,
         "interleaved": True, "norm": True, "out_dim": 576},
        # a decode step of 128 requests, 128 heads: rope part of the absorbed query
        {"name": "rope_decode", "kind": "rope", "tokens": 128, "heads": 128, "page": 64, "fp8": False, "axes": 1,
         "interleaved": True, "norm": True, "out_dim": 576},
        # a prompt with images: three position axes, rotated halves
        {"name": "rope_images", "kind": "rope", "tokens": 16384, "heads": 16, "page": 64, "fp8": False, "axes": 3,
         "interleaved": False, "norm": True, "out_dim": 192},
        # prompt chunks into an e4m3 cache, 128 heads
        {"name": "rope_fp8", "kind": "rope", "tokens": 8191, "heads": 128, "page": 64, "fp8": True, "axes": 1,
         "interleaved": True, "norm": True, "out_dim": 192},
        # the smallest chunk: two short requests, 16 heads, small pages
        {"name": "prefill_tiny", "kind": "prefill", "batch": 2, "heads": 16, "page": 16, "fp8": False,
         "ctx_lo": 37, "ctx_hi": 61, "new_lo": 1, "new_hi": 5, "window": 0},
        # a mixed step: chunks of one to some hundred tokens over uneven caches
        {"name": "prefill_ragged", "kind": "prefill", "batch": 24, "heads": 16, "page": 64, "fp8": False,
         "ctx_lo": 512, "ctx_hi": 4096, "new_lo": 1, "new_hi": 511, "window": 0},
        # fresh prompts, nothing cached before
        {"name": "prefill_prompts", "kind": "prefill", "batch": 3, "heads": 16, "page": 64, "fp8": False,
         "ctx_lo": 0, "ctx_hi": 0, "new_lo": 4500, "new_hi": 8192, "window": 0},
        # a window over an e4m3 cache, 128 heads
        {"name": "prefill_window", "kind": "prefill", "batch": 4, "heads": 128, "page": 64, "fp8": True,
         "ctx_lo": 5000, "ctx_hi": 8192, "new_lo": 300, "new_hi": 1024, "window": 4096},
        # the next chunk of a long prompt, 128 heads
        {"name": "prefill_chunk", "kind": "prefill", "batch": 1, "heads": 128, "page": 64, "fp8": False,
         "ctx_lo": 14336, "ctx_hi": 14336, "new_lo": 2048, "new_hi": 2048, "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["tables", "rope", "prefill", "prefill"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "tables":
        hi = _log(rng, 64, 131072)
        new = _log(rng, 1, 2048)
        return {"kind": kind, "batch": _log(rng, 1, 1024 if new < 64 else 64), "page": max(page, 32) if hi > 16384 else page,
                "ctx_lo": rng.randint(0, hi), "ctx_hi": hi, "new_lo": rng.randint(1, new), "new_hi": new}
    if kind == "rope":
        heads = rng.choice([8, 16, 32, 64, 128])
        return {"kind": kind, "tokens": _log(rng, 1, 8192), "heads": heads, "page": page,
                "fp8": rng.random() < 0.4, "axes": rng.choice([1, 2, 3]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.7, "out_dim": rng.choice([192, 576])}
    heads = rng.choice([8, 16, 32, 64, 128])
    batch = _log(rng, 1, 16)
    most = 4096 * 16 // (heads * batch)  # new tokens a request, so that no draw outgrows the listed chunk
    new = _log(rng, 1, max(2, min(2048, most)))
    ctx = _log(rng, 16, 12000 if batch <= 4 else 4096)
    return {"kind": kind, "batch": batch, "heads": heads, "page": page, "fp8": rng.random() < 0.4,
            "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "new_lo": rng.randint(1, new), "new_hi": new,
            "window": rng.choice([0, 0, _log(rng, 1, 8192)])}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Context and new-token lengths, spread over their ranges; the same for every seed, so that work() knows them."""
    b = case["batch"]
    f = [((i * 0.6180339887498949 + 0.5) % 1.0) for i in range(b)]
    g = [((i * 0.7548776662466927 + 0.25) % 1.0) for i in range(b)]
    ctx = [case["ctx_lo"] + round(x * (case["ctx_hi"] - case["ctx_lo"])) for x in f]
    # new tokens spread over their logarithm: many small chunks, few large ones
    lo, hi = case["new_lo"], case["new_hi"]
    new = [min(hi, max(lo, round(lo * (hi / lo) ** x))) for x in g]
    new[0] = hi
    return ctx, new


def _pages(ctx_end, page, gen, dev, spare=16):
    """A block table whose rows hold the pages of ctx_end[b] tokens, in random order, and the pages left over."""
    ends = torch.tensor(ctx_end, device=dev)
    blocks = (ends + page - 1) // page
    total = sum((e + page - 1) // page for e in ctx_end)
    perm = torch.randperm(total + spare, generator=gen, device=dev).to(torch.int32)
    width = max(1, max((e + page - 1) // page for e in ctx_end))
    table = torch.full((len(ctx_end), width), -1, dtype=torch.int32, device=dev)
    at = torch.arange(width, device=dev)[None, :] < blocks[:, None]
    table[at] = perm[:total]
    return table, perm[total:], total + spare


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = {"case": case, "kind": case["kind"]}
    if own:
        import paged_mla_decode_04_gb300 as lib
        s["lib"] = lib
    {"tables": _prepare_tables, "rope": _prepare_rope, "prefill": _prepare_prefill}[case["kind"]](case, s, gen, dev)
    return s


def _normal(gen, dev, *shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    out.normal_(0.0, std, generator=gen)
    return out


def _prepare_tables(case, s, gen, dev):
    page, (ctx, new) = case["page"], _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    need = sum((t + page - 1) // page - (c + page - 1) // page for t, c in zip(total, ctx))
    table, left, s["num_pages"] = _pages(ctx, page, gen, dev, spare=need + 16)
    width = max((t + page - 1) // page for t in total)
    wide = torch.full((len(ctx), width), -1, dtype=torch.int32, device=dev)
    wide[:, : table.shape[1]] = table
    s["table"] = wide
    s["free"] = left.contiguous()
    s["count"] = torch.tensor([left.numel()], dtype=torch.int32, device=dev)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
    s["max_tokens"] = sum(new) + 7  # a few pad rows, as a captured step of fixed size has
    s["max_ids"] = sum((t + page - 1) // page for t in total)
    b = len(ctx)
    s["slots"] = torch.zeros(s["max_tokens"], dtype=torch.int64, device=dev)
    s["positions"] = torch.zeros(s["max_tokens"], dtype=torch.int32, device=dev)
    s["indptr"] = torch.zeros(b + 1, dtype=torch.int32, device=dev)
    s["page_indptr"] = torch.zeros(b + 1, dtype=torch.int32, device=dev)
    s["ids"] = torch.zeros(s["max_ids"], dtype=torch.int32, device=dev)
    s["state"] = torch.zeros(2, dtype=torch.int32, device=dev)


def _prepare_rope(case, s, gen, dev):
    n, h, page = case["tokens"], case["heads"], case["page"]
    pages = (n + page - 1) // page + 4
    if case["fp8"]:
        pool = torch.empty(1, pages, page, ROW, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s["pool"] = (pool.float() * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale"] = 1.0 / 64
    else:
        s["pool"] = _normal(gen, dev, 1, pages, page, ROW)
        s["scale"] = 1.0
    s["rows"] = _normal(gen, dev, n, ROW)
    s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:n].contiguous()
    s["weight"] = (1 + 0.1 * _normal(gen, dev, CKV).float()).to(torch.bfloat16) if case["norm"] else None
    limit = 32768
    inv = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=dev) / 32)
    angle = torch.arange(limit, dtype=torch.float64, device=dev)[:, None] * inv
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["positions"] = torch.randint(0, limit, (case["axes"], n), generator=gen, device=dev, dtype=torch.int32)
    s["pair_axis"] = {1: [0] * 32, 2: [0] * 16 + [1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12}[case["axes"]]
    s["pair_axis_dev"] = torch.tensor(s["pair_axis"], device=dev)
    s["q"] = _normal(gen, dev, n, h, ROPE)
    # the other dims of the queries are in place before; the call fills the last 64
    s["q_all"] = _normal(gen, dev, n, h, case["out_dim"])
    s["q_out"] = s["q_all"][:, :, case["out_dim"] - ROPE:]
    if own:
        s["kv"] = s["lib"].KVPool(s["pool"], s["scale"])


def _prepare_prefill(case, s, gen, dev):
    page, h, (ctx, new) = case["page"], case["heads"], _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    s["table"], _, pages = _pages(total, page, gen, dev)
    pool = torch.empty(2, pages, page, ROW, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    if case["fp8"]:
        s["pool"] = (pool.float() * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale"] = 1.0 / 64
    else:
        s["pool"], s["scale"] = pool, 1.0
    s["q"] = _normal(gen, dev, sum(new), h, QK)
    s["w_uk"] = _normal(gen, dev, h, NOPE, CKV, std=CKV ** -0.5)
    s["w_uv"] = _normal(gen, dev, h, CKV, VDIM, std=CKV ** -0.5)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    s["indptr"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["longest"], s["most_new"] = max(total), max(new)
    s["softmax_scale"] = QK ** -0.5
    s["out"] = torch.zeros(sum(new), h, VDIM, dtype=torch.bfloat16, device=dev)
    w = case["window"]
    s["max_kv"] = sum(t - (max(0, c + 1 - w) if w else 0) for t, c in zip(total, ctx))
    if own:
        s["kv"] = s["lib"].KVPool(s["pool"], s["scale"])
        s["ws"] = s["lib"].alloc_prefill_workspace(len(ctx), sum(new), s["max_kv"], h)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "prefill": _own_prefill}[s["kind"]](s)
    return {"tables": _plain_tables, "rope": _plain_rope, "prefill": _plain_prefill}[s["kind"]](s)


def _own_tables(s):
    s["lib"].extend_tables(s["ctx"], s["new"], s["free"], s["count"], s["table"], s["case"]["page"], s["num_pages"],
                           s["slots"], s["indptr"], s["state"], positions=s["positions"],
                           page_indptr=s["page_indptr"], page_ids=s["ids"])
    return _tables_out(s)


def _tables_out(s):
    return {"table": s["table"], "slots": s["slots"], "positions": s["positions"], "indptr": s["indptr"],
            "page_indptr": s["page_indptr"], "ids": s["ids"], "state": s["state"]}


def _own_rope(s):
    s["lib"].rope_write(s["kv"], 0, s["rows"], s["slots"], s["positions"], s["cos_sin"], norm_weight=s["weight"],
                        norm_eps=EPS, q_rope=s["q"], q_out=s["q_out"], pair_axis=s["pair_axis"],
                        interleaved=s["case"]["interleaved"])
    return _rope_out(s)


def _rope_out(s):
    pool = s["pool"].view(torch.float8_e4m3fn) if s["case"]["fp8"] else s["pool"]
    return {"pool": pool, "q": s["q_all"]}


def _own_prefill(s):
    s["lib"].prefill(s["kv"], 1, s["q"], s["indptr"], s["ctx"], s["softmax_scale"], s["w_uk"], s["w_uv"], s["ws"],
                     s["out"], s["max_kv"], block_table=s["table"], window=s["case"]["window"])
    return s["out"]


# ------------------------------------------------------------------ plain forms

def _plain_tables(s):
    page, dev = s["case"]["page"], s["ctx"].device
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    held = (ctx + page - 1) // page
    blocks = (ctx + new + page - 1) // page
    need = blocks - held
    upto = need.cumsum(0)
    base = upto - need
    count = s["count"].long()
    served = (upto <= count) | (need == 0)
    # new pages come off the top of the stack, in the order of requests and blocks
    j = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (j >= held[:, None]) & (j < blocks[:, None]) & served[:, None]
    at = (count - 1 - base[:, None] - (j - held[:, None])).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][at], table))
    s["state"][0] = (count - torch.where(upto <= count, upto, 0).max())[0]
    s["state"][1] = torch.where(served, len(ctx), torch.arange(len(ctx), device=dev)).min()
    ends = new.cumsum(0)
    s["indptr"][0] = 0
    s["indptr"][1:] = ends
    t = torch.arange(s["max_tokens"], device=dev)
    who = torch.searchsorted(ends, t, right=True)
    real = who < len(ctx)
    who = who.clamp(max=len(ctx) - 1)
    real &= served[who]
    pos = ctx[who] + t - (ends - new)[who]
    id_ = s["table"][who, (pos // page).clamp(max=table.shape[1] - 1)].long()
    s["slots"].copy_(torch.where(real, id_ * page + pos % page, -1))
    s["positions"].copy_(torch.where(real, pos, -1))
    listed_ = torch.where(served, blocks, held)
    csr = listed_.cumsum(0)
    s["page_indptr"][0] = 0
    s["page_indptr"][1:] = csr
    k = torch.arange(s["max_ids"], device=dev)
    who = torch.searchsorted(csr, k, right=True).clamp(max=len(ctx) - 1)
    s["ids"].copy_(torch.where(k < csr[-1], s["table"][who, (k - (csr - listed_)[who]).clamp(max=table.shape[1] - 1)], s["ids"]))
    return _tables_out(s)


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_rope(s):
    case = s["case"]
    where = s["positions"].long()[s["pair_axis_dev"]].T            # [tokens, 32]
    pair = torch.arange(32, device=where.device)
    cos, sin = s["cos_sin"][where, pair], s["cos_sin"][where, 32 + pair]
    rows = s["rows"].float()
    ckv = rows[:, :CKV]
    if case["norm"]:
        ckv = ckv * torch.rsqrt(ckv.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat([ckv, _rotate(rows[:, CKV:], cos, sin, case["interleaved"])], 1)
    flat = s["pool"][0].view(-1, ROW)
    if case["fp8"]:
        flat[s["slots"]] = (row / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        flat[s["slots"]] = row.to(torch.bfloat16)
    s["q_out"].copy_(_rotate(s["q"].float(), cos[:, None], sin[:, None], case["interleaved"]))
    return _rope_out(s)


def _plain_prefill(s):
    case, dev = s["case"], s["q"].device
    page, h = case["page"], case["heads"]
    ctx, starts = s["ctx"].long(), s["indptr"].long()
    n = s["longest"]
    kpos = torch.arange(n, device=dev)
    end = ctx + starts[1:] - starts[:-1]
    have = kpos[None, :] < end[:, None]
    ids = s["table"].long()[:, (kpos // page)].clamp(min=0)
    if case["fp8"]:
        rows = s["pool"][1].view(torch.float8_e4m3fn).view(torch.uint8)[ids, kpos % page].view(torch.float8_e4m3fn).float() * s["scale"]
    else:
        rows = s["pool"][1][ids, kpos % page].float()
    rows = torch.where(have[:, :, None], rows, 0.0)
    ckv, kr = rows[:, None, :, :CKV], rows[:, None, :, CKV:]
    k = torch.cat([ckv @ s["w_uk"].float().transpose(1, 2), kr.expand(-1, h, -1, -1)], -1)   # [B, H, n, 192]
    v = ckv @ s["w_uv"].float()                                                               # [B, H, n, 128]
    i = torch.arange(s["most_new"], device=dev)
    real = i[None, :] < (end - ctx)[:, None]
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().transpose(1, 2)                                                   # [B, H, new, 192]
    qpos = ctx[:, None] + i
    seen = kpos[None, None, :] <= qpos[:, :, None]
    if case["window"]:
        seen &= kpos[None, None, :] > qpos[:, :, None] - case["window"]
    x = (q @ k.transpose(2, 3)).mul_(s["softmax_scale"])
    x.masked_fill_(~seen[:, None], float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    y = (x @ v).div_(x.sum(-1, keepdim=True))
    s["out"][row[real]] = y.transpose(1, 2)[real].to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if case["kind"] == "tables":
        return None
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["kind"] == "rope" else _exact_prefill(case, s)


def _as_complex(x, interleaved):
    """The 32 rotated pairs of the last 64 values, as complex numbers."""
    x = x.double()
    return torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :32], x[..., 32:])


def _from_complex(z, interleaved):
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _exact_rope(case, s):
    n, il = case["tokens"], case["interleaved"]
    turn = torch.empty(n, 32, dtype=torch.complex128, device=s["q"].device)
    for j, axis in enumerate(s["pair_axis"]):
        at = s["cos_sin"][s["positions"][axis].long()].double()
        turn[:, j] = torch.complex(at[:, j].contiguous(), at[:, 32 + j].contiguous())
    row = s["rows"].double()
    if case["norm"]:
        size = torch.linalg.vector_norm(row[:, :CKV], dim=1, keepdim=True)
        row[:, :CKV] *= s["weight"].double() / (size * size / CKV + EPS).sqrt()
    row[:, CKV:] = _from_complex(_as_complex(row[:, CKV:], il) * turn, il)
    pool = (s["pool"].view(torch.float8_e4m3fn).float() if case["fp8"] else s["pool"]).double()
    flat = pool.view(-1, ROW)
    flat[s["slots"]] = (row / s["scale"]).clamp(-448, 448) if case["fp8"] else row
    q = s["q_all"].double()
    q[:, :, -ROPE:] = _from_complex(_as_complex(s["q"], il) * turn[:, None], il)
    return {"pool": pool, "q": q}


def _exact_prefill(case, s):
    """One request and eight heads at a time, over the positions that its rows can see."""
    pairs = sum(_pairs(case)) * case["heads"]
    if pairs > 6e9:
        return None  # over the time that a check in 64 bits may take
    ctx, new = _lengths(case)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    r0 = 0
    for b, (c, m) in enumerate(zip(ctx, new)):
        first = max(0, c + 1 - case["window"]) if case["window"] else 0
        at = torch.arange(first, c + m, device=out.device)
        pages = s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")]
        lat = s["pool"][1][pages, at % case["page"]]
        lat = (lat.view(torch.float8_e4m3fn).float() if case["fp8"] else lat).double() * s["scale"]
        mine = torch.arange(c, c + m, device=out.device)[:, None]
        hide = at[None, :] > mine
        if case["window"]:
            hide |= at[None, :] < mine + 1 - case["window"]
        for h0 in range(0, case["heads"], 8):
            hs = slice(h0, h0 + 8)
            q = s["q"][r0:r0 + m, hs].double()
            key = torch.einsum("tc,hdc->htd", lat[:, :CKV], s["w_uk"][hs].double())
            x = torch.einsum("mhd,htd->hmt", q[:, :, :NOPE], key) + torch.einsum("mhd,td->hmt", q[:, :, NOPE:], lat[:, CKV:])
            p = torch.softmax((x * s["softmax_scale"]).masked_fill(hide, -math.inf), -1)
            out[r0:r0 + m, hs] = torch.einsum("hmt,tc,hcd->mhd", p, lat[:, :CKV], s["w_uv"][hs].double()) if m < 64 else \
                torch.einsum("hmt,htd->mhd", p, torch.einsum("tc,hcd->htd", lat[:, :CKV], s["w_uv"][hs].double()))
        r0 += m
    return out


# ------------------------------------------------------------------ work

def _pairs(case):
    """Attended (query, position) pairs of each request, for one head."""
    got = []
    for c, m in zip(*_lengths(case)):
        w = case["window"] or c + m
        got.append(sum(min(c + i + 1, w) for i in range(m)))
    return got


def work(case):
    if case["kind"] == "tables":
        ctx, new = _lengths(case)
        page = case["page"]
        blocks = sum((c + n + page - 1) // page for c, n in zip(ctx, new))
        fresh = blocks - sum((c + page - 1) // page for c in ctx)
        # lengths in, two row pointers out; slots and positions out; the CSR list in and out; new pages in and out
        return {"bytes": len(ctx) * 16 + (sum(new) + 7) * 12 + blocks * 8 + fresh * 4, "flops": 0}
    if case["kind"] == "rope":
        n, h = case["tokens"], case["heads"]
        angles = 256 * n + 4 * n * case["axes"]
        return {"bytes": n * (ROW * 2 + ROW * (1 if case["fp8"] else 2) + 8) + angles + n * h * ROPE * 4,
                "flops": n * (h + 1) * 32 * 6 + n * CKV * 4}
    h = case["heads"]
    ctx, new = _lengths(case)
    w = case["window"]
    kv = [c + m - (max(0, c + 1 - w) if w else 0) for c, m in zip(ctx, new)]
    flops = 0.0
    for pairs, m, t in zip(_pairs(case), new, kv):
        # keys and values of every head made once and attended in 192/128 dims, or
        # the queries brought into the latent space and attended in 576/512 dims
        flops += h * min(t * 2 * CKV * (NOPE + VDIM) + pairs * 2 * (QK + VDIM),
                         m * 2 * CKV * (NOPE + VDIM) + pairs * 2 * (ROW + CKV))
    return {"bytes": sum(kv) * ROW * (1 if case["fp8"] else 2) + sum(new) * h * (QK + VDIM) * 2 + h * CKV * (NOPE + VDIM) * 2,
            "flops": flops}
