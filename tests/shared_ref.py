"""Decode over shared prefixes and the compact store in 64 bits (torch, any device), and
the bounds of what the kernels' roundings may change.

A rounding to bf16 is off by at most 2^-8 of the value (half a step), one to f16 by
2^-11, to e4m3 by 2^-4."""
from __future__ import annotations

import math

import torch

CKV, ROW = 512, 576
BF16_HALF, F16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


class Case:
    """A batch of groups [(requests, prefix length)] with own lengths (cached positions
    behind the prefix, one a request). Every row of the pool that nothing attends, and
    every table entry that is not used, holds what would be noticed: NaN, and page ids
    out of range."""

    def __init__(self, groups, own, heads=16, q_len=1, page=16, fp8=False, seed=0, before=0, after=0, device="cuda",
                 q_std=1.0, layers=2):
        g = torch.Generator(device)
        g.manual_seed(seed)
        self.page, self.heads, self.q_len, self.fp8, self.layer = page, heads, q_len, fp8, layers - 1
        which = [i for i, (n, _) in enumerate(groups) for _ in range(n)]
        own = list(own) + [own[-1]] * (len(which) - len(own))
        ctx = [groups[i][1] + m for i, m in zip(which, own)]
        self.which, self.pads = which, (before, after)
        B = before + len(which) + after
        blocks = [(c + q_len + page - 1) // page for c in ctx]
        width = max(blocks, default=1)
        whole = [p // page for _, p in groups]
        pages = sum(whole) + sum(b - whole[i] for b, i in zip(blocks, which)) + 3
        ids = torch.randperm(pages, generator=g, device=device).tolist()
        values = torch.randn(layers, pages, page, ROW, generator=g, device=device)
        if fp8:
            self.scale = 1.0 / 32
            pool = (values / self.scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            none = 0x7F
        else:
            self.scale = 1.0
            pool = values.to(torch.bfloat16)
            none = math.nan
        used = torch.zeros(pages, page, dtype=torch.bool)
        table = [[-1 - 7 * b if b % 2 else 1 << 30] * width for b in range(B)]
        full = [[-1] * width for _ in range(B)]
        shared = [[ids.pop() for _ in range(w)] for w in whole]
        head = {}
        for k, (i, c) in enumerate(zip(which, ctx)):
            b, p = before + k, groups[i][1]
            mine = [ids.pop() for _ in range(blocks[k] - whole[i])]
            full[b][:blocks[k]] = shared[i] + mine
            for j in shared[i]:
                used[j] = True
            for t in range(whole[i] * page, c + q_len):
                used[mine[t // page - whole[i]], t % page] = True
            rest = p % page
            if rest:  # the page that a prefix ends in is each request's own copy
                if i in head:
                    pool[:, mine[0], :rest] = pool[:, head[i], :rest]
                else:
                    head[i] = mine[0]
            alone = groups[i][0] == 1 or (k == 0 or which[k - 1] != i)
            # (of pages that end within the prefix only the group's first request's entries are used)
            table[b][0 if alone else whole[i]:blocks[k]] = full[b][0 if alone else whole[i]:blocks[k]]
            if not alone and rest:  # nor, of its own copy, the rows before the prefix's end
                used[mine[0], :rest] = False
        self.clean = pool.clone()
        pool[:, ~used.to(device)] = none
        self.pool, self.used = pool, used.to(device)
        i32 = dict(dtype=torch.int32, device=device)
        self.table, self.full = torch.tensor(table, **i32).view(B, width), torch.tensor(full, **i32).view(B, width)
        self.ctx = torch.tensor([7] * before + ctx + [5] * after, **i32)
        starts = [before]
        for n, _ in groups:
            starts.append(starts[-1] + n)
        self.indptr, self.prefix = torch.tensor(starts, **i32), torch.tensor([p for _, p in groups], **i32)
        self.q = (q_std * torch.randn(B, q_len, heads, ROW, generator=g, device=device)).to(torch.bfloat16)
        self.softmax_scale = 192 ** -0.5

    @property
    def batch(self):
        return self.ctx.numel()

    def real(self):
        return range(self.pads[0], self.batch - self.pads[1])

    def rows(self, b):
        """What request b attends, in 64 bits: [positions, 576]."""
        n = int(self.ctx[b]) + self.q_len
        got = self.clean[self.layer][self.full[b, :(n + self.page - 1) // self.page].long()].flatten(0, 1)[:n]
        return (got.view(torch.float8_e4m3fn).float() if self.fp8 else got).double() * self.scale

    def reference(self, b, rows=None):
        """out, lse of request b [q_len, heads, ...] and the bounds of their errors."""
        lat = self.rows(b) if rows is None else rows
        q = self.q[b].double()
        n = lat.shape[0]
        score = torch.einsum("ihd,td->iht", q, lat) * self.softmax_scale
        size = torch.einsum("ihd,td->iht", q.abs(), lat.abs()) * self.softmax_scale
        last = n - self.q_len + torch.arange(self.q_len, device=q.device)
        seen = torch.arange(n, device=q.device)[None, :] <= last[:, None]
        score = score.masked_fill(~seen[:, None, :], -math.inf)
        lse = torch.logsumexp(score, -1)
        w = torch.exp(score - lse[..., None])
        out = torch.einsum("iht,td->ihd", w, lat[:, :CKV])
        mass = torch.einsum("iht,td->ihd", w, lat[:, :CKV].abs())
        # A score is a sum of 576 products and what the tiles add, each addition off by at
        # most 2^-23 of the sum of the sizes; then scaled, exponentiated (2^-22 each).
        es = (size.masked_fill(~seen[:, None, :], 0).amax(-1) * 600 * 2.0 ** -23 + 2.0 ** -20)[..., None]
        # Weights are rounded for the product (bf16; f16 for fp8 pools), the result once more.
        half = F16_HALF if self.fp8 else BF16_HALF
        return out, lse, BF16_HALF * out.abs() + (half + 2 * es) * mass * 1.01 + 1e-30, es[..., 0] + F32_HALF * 4 * lse.abs()


def check(case, out, lse, requests=None):
    off, norm, most = 0.0, 0.0, 0.0
    for b in case.real() if requests is None else requests:
        ref, ref_lse, bound, lse_bound = case.reference(b)
        d = (out[b].double() - ref).abs()
        assert bool((d <= bound).all()), (b, (d / bound).max().item())
        off, norm = off + d.square().sum().item(), norm + ref.square().sum().item()
        if lse is not None:
            e = (lse[b].double() - ref_lse).abs()
            assert bool((e <= lse_bound).all()), (b, e.max().item())
            most = max(most, (e / (1 + ref_lse.abs())).max().item())
    # Independent roundings (the weights', the result's) have 0.41 of half a step each in
    # the mean square: together 0.58 of it, of the result's norm.
    assert off <= (BF16_HALF ** 2) * norm, math.sqrt(off / max(norm, 1e-300))
    assert most <= 1e-5, most


# ------------------------------------------------------------------ compact store

def store_row(rows, codes):
    """Bytes of quantised rows [n, 576] bf16: IEEE fp32 divisions, as documented."""
    x = rows[:, :CKV].float()
    if codes == "e4m3":
        g = x.view(-1, 4, 128)
        top = g.abs().amax(-1)
        scale = torch.where(top.isfinite(), top / torch.full_like(top, 448), math.nan)  # (by a number torch multiplies by its inverse)
        q = torch.where(scale[..., None] > 0, g / scale[..., None], 0.0)
        code = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
        scale = scale.contiguous().view(torch.uint8)
    else:
        g = x.view(-1, 16, 32)
        top = g.abs().amax(-1)
        scale = torch.where(top.isfinite(), top / torch.full_like(top, 6), math.nan).to(torch.bfloat16)
        s = scale.float()[..., None]
        q = torch.where(s > 0, g / s, 0.0).flatten(1)
        mag = q.abs().double()
        levels = LEVELS.to(x.device)
        near = (mag[..., None] - levels).abs()
        # the nearest level, of two the one with an even code
        least = near.amin(-1, keepdim=True)
        tied = near == least
        even = tied & (torch.arange(8, device=x.device) % 2 == 0)
        pick = torch.where(tied.sum(-1) > 1, even.int().argmax(-1), tied.int().argmax(-1))
        c = (pick + 8 * torch.signbit(q)).to(torch.uint8)
        code = c[:, 0::2] | (c[:, 1::2] << 4)
        scale = scale.contiguous().view(torch.uint8)
    return torch.cat([code, scale.flatten(1), rows[:, CKV:].contiguous().view(torch.uint8)], 1)


def store_values(data):
    """What stored rows [n, row bytes] stand for, in 64 bits."""
    if data.shape[1] == 656:
        v = data[:, :CKV].contiguous().view(torch.float8_e4m3fn).double().view(-1, 4, 128)
        scale = data[:, CKV:CKV + 16].contiguous().view(torch.float32).double()
    else:
        c = torch.stack([data[:, :256] & 15, data[:, :256] >> 4], -1).flatten(1).long()
        v = LEVELS.to(data.device)[c & 7] * torch.where(c >= 8, -1.0, 1.0)
        v = v.view(-1, 16, 32)
        scale = data[:, 256:288].contiguous().view(torch.bfloat16).double()
    rope = data[:, -128:].contiguous().view(torch.bfloat16).double()
    return torch.cat([(v * scale[..., None]).flatten(1), rope], 1)
