"""Plain 64-bit (numpy, CPU) forms of the prefill step's operators, and the
bounds of what the kernels' roundings may change.

A rounding to bf16 is off by at most 2^-8 of the value (half a step), one to
e4m3 by 2^-4 (2^-10 absolute below the smallest normal value)."""
from __future__ import annotations

import numpy as np
import torch

CKV, ROPE, ROW, NOPE, VDIM, QK = 512, 64, 576, 128, 128, 192
BF16_HALF = 2.0 ** -8
F32_HALF = 2.0 ** -24


def extend_tables(ctx, new, free, count, table, ps, num_pages, max_tokens, max_ids=None):
    """One request after another, one page after another."""
    B, width = table.shape
    table = table.copy()
    count = min(max(int(count), 0), len(free))
    slots = np.full(max_tokens, -1, np.int64)
    pos = np.full(max_tokens, -1, np.int32)
    indptr, pind, ids = [0], [0], []
    taken, asked, refused, status = 0, 0, B, 0
    t = 0
    for b in range(B):
        L, n = int(ctx[b]), int(new[b])
        room = width * ps
        ok = L >= 0 and n >= 0 and L + n <= room
        held = -(-L // ps) if 0 <= L <= room else 0
        need = -(-(L + max(n, 0)) // ps) - held if ok else 0
        served = ok and (need == 0 or asked + need <= count)
        if not ok:
            status |= 0x10
        elif not served:
            refused = min(refused, b)
            status |= 0x20
        if served:
            for k in range(need):
                p = int(free[count - 1 - asked - k])
                if not 0 <= p < num_pages:
                    p, status = -1, status | 0x1
                table[b, held + k] = p
            if need:
                taken = asked + need
        asked += need
        for i in range(max(n, 0)):
            if served and t < max_tokens:
                p = int(table[b, (L + i) // ps])
                if 0 <= p < num_pages:
                    slots[t], pos[t] = p * ps + (L + i) % ps, L + i
                else:
                    status |= 0x1
            t += 1
        indptr.append(t)
        blocks = held + (need if served else 0)
        ids += list(table[b, :blocks])
        pind.append(pind[-1] + blocks)
    if t > max_tokens or (max_ids is not None and len(ids) > max_ids):
        status |= 0x10
    return dict(table=table, slots=slots, positions=pos, indptr=np.array(indptr, np.int32),
                page_indptr=np.array(pind, np.int32), ids=np.array(ids, np.int32),
                state=np.array([count - taken, refused], np.int32), status=status)


def rotate(x, positions, pair_axis, cos_sin, interleaved):
    """x [n, ..., 64] turned by the table's angles; positions [axes, n]."""
    x = x.astype(np.float64)
    out = x.copy()
    mag = np.zeros_like(x)
    for j in range(32):
        p = np.clip(positions[pair_axis[j]], 0, len(cos_sin) - 1)  # (rows out of range are not compared)
        shape = (-1,) + (1,) * (x.ndim - 2)
        c, s = cos_sin[p, j].astype(np.float64).reshape(shape), cos_sin[p, 32 + j].astype(np.float64).reshape(shape)
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + 32)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
        m = np.abs(x[..., a]) + np.abs(x[..., b])
        mag[..., a] = mag[..., b] = m
    return out, mag  # mag bounds the terms of each value (|cos|, |sin| <= 1)


def norm(ckv, weight, eps):
    ckv = ckv.astype(np.float64)
    if weight is None:
        return ckv
    return ckv / np.sqrt((ckv ** 2).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)


def prefill(rows_of, q, indptr, ctx, w_uk, w_uv, scale, window, latent=lambda n, m: False):
    """rows_of(b, positions) -> latent rows [m, 576] in float64. Returns out
    [T, H, 128], lse [T, H] and the largest change that the kernel's roundings
    can make to each output (and to lse): keys, values, softmax weights and
    output are rounded to bf16 (2^-8 of each), products summed in fp32 over at
    most 576 + n terms (2^-24 each, doubled for the approximate 2^x).
    latent(n, m): whether a request of n new tokens over m positions is attended in the latent space:
    there the query brought into it (512 dims) and the latent output are rounded
    to bf16 instead of keys and values, and each half of a score to fp16 (2^-11)."""
    T, H, _ = q.shape
    out, lse = np.zeros((T, H, VDIM)), np.zeros((T, H))
    tol, tol_lse = np.zeros((T, H, VDIM)), np.zeros((T, H))
    wk, wv = torch.from_numpy(w_uk), torch.from_numpy(w_uv)
    for b in range(len(ctx)):
        r0, r1, L = int(indptr[b]), int(indptr[b + 1]), int(ctx[b])
        n = r1 - r0
        if n <= 0:
            continue
        lo = max(0, L + 1 - window) if window else 0
        at = np.arange(lo, L + n)
        lat = torch.from_numpy(rows_of(b, at))
        qb = torch.from_numpy(q[r0:r1]).transpose(0, 1)                      # [H, n, 192]
        k = torch.cat([lat[None, :, :CKV] @ wk.transpose(1, 2), lat[None, :, CKV:].expand(H, -1, -1)], 2)
        v = lat[None, :, :CKV] @ wv
        s = qb @ k.transpose(1, 2) * scale
        mag = (qb[:, :, :NOPE].abs() @ k[:, :, :NOPE].abs().transpose(1, 2)) * scale
        mag_all = (qb.abs() @ k.abs().transpose(1, 2)) * scale
        # An fp32 sum of m products is off by at most m 2^-24 of the sum of their sizes (not of the sum itself, which
        # may cancel): 512 products for a key or value, 192 for a score.
        k_sum = lat[None, :, :CKV].abs() @ wk.abs().transpose(1, 2)
        v_sum = lat[None, :, :CKV].abs() @ wv.abs()
        ds = mag * BF16_HALF + mag_all * 2 * QK * F32_HALF
        ds += (qb[:, :, :NOPE].abs() @ k_sum.transpose(1, 2)) * scale * CKV * F32_HALF
        if latent(n, len(at)):
            qa = qb[:, :, :NOPE] @ wk                                         # [H, n, 512]
            c_abs, r_abs = lat[:, :CKV].abs(), lat[:, CKV:].abs()
            whole = qa.abs() @ c_abs.T + qb[:, :, NOPE:].abs() @ r_abs.T       # of both halves' sizes
            qa_sum = (qb[:, :, :NOPE].abs() @ wk.abs()) @ c_abs.T
            ds = scale * ((qa.abs() @ c_abs.T) * BF16_HALF + whole * (2.0 ** -11 + 1152 * F32_HALF) * (1 + BF16_HALF) +
                          qa_sum * NOPE * F32_HALF)
        mine = torch.arange(L, L + n)[:, None]
        hide = torch.from_numpy(at)[None, :] > mine
        if window:
            hide |= torch.from_numpy(at)[None, :] <= mine - window
        s = s.masked_fill(hide, float("-inf"))
        ds = ds.masked_fill(hide | torch.isinf(s), 0.0)
        p = torch.softmax(s, -1)
        o = p @ v
        d = ds.amax(-1, keepdim=True)
        # weights off by a factor within e^(+-d) each before normalising, 2^-8 by their rounding
        # (also in their sum's place), values by 2^-8, all of it relative to sum p |v|
        weight = torch.expm1(2 * d) + 2 * BF16_HALF + (len(at) + 64) * 2 * F32_HALF
        e = (p @ v.abs()) * (weight * (1 + BF16_HALF) + BF16_HALF) + o.abs() * BF16_HALF + (p @ v_sum) * CKV * F32_HALF
        if latent(n, len(at)):
            # Latent sums off like the values' above, rounded, then multiplied into 128 dims.
            c_abs = lat[:, :CKV].abs()
            d_lat = (p @ c_abs) * weight + (p @ lat[:, :CKV]).abs() * BF16_HALF * (1 + weight)
            e = d_lat @ wv.abs() + o.abs() * BF16_HALF + ((p @ c_abs) @ wv.abs()) * CKV * F32_HALF
        out[r0:r1] = o.transpose(0, 1).numpy()
        tol[r0:r1] = e.transpose(0, 1).numpy() * 1.01
        ls = torch.logsumexp(s, -1)
        lse[r0:r1] = ls.T.numpy()
        tol_lse[r0:r1] = (d[..., 0] + (len(at) + 64) * F32_HALF + ls.abs() * 4 * F32_HALF).T.numpy() * 1.01
    return out, lse, tol, tol_lse
