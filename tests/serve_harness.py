"""Plain 64-bit forms of the serving calls (page plans, appends, attention over
the paged cache in original order) and the error bounds they are compared by.
Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a rounding step


def plan_reference(table, have, new, free, n_free, page, n_pages, capacity):
    """Python lists in, (table, slots, positions, starts, seq_lens, n_free) out;
    the plan that changes nothing where the step does not fit."""
    need = [-(-(h + n) // page) + (-h // page) for h, n in zip(have, new)]
    wide = max(-(-(h + n) // page) for h, n in zip(have, new))
    table = [list(r) for r in table]
    if (sum(need) > n_free or sum(new) > capacity or wide > len(table[0]) or min(have) < 0
            or min(new) < 0 or max(h + n for h, n in zip(have, new)) > 2 ** 31 - 1):
        return table, [-1] * capacity, [-1] * capacity, [0] * (len(have) + 1), list(have), n_free
    stack = list(free[:n_free])
    slots, positions, starts = [], [], [0]
    for row, h, n, m in zip(table, have, new, need):
        first = -(-h // page)
        for j in range(m):
            pg = stack.pop()
            row[first + j] = pg if 0 <= pg < n_pages else -1
        for pos in range(h, h + n):
            pg = row[pos // page]
            slots.append(pg * page + pos % page if 0 <= pg < n_pages else -1)
            positions.append(pos)
        starts.append(starts[-1] + n)
    pad = [-1] * (capacity - len(slots))
    return (table, slots + pad, positions + pad, starts, [h + n for h, n in zip(have, new)],
            len(stack))


def rows_of(pool, table, b, h, T):
    """Rows of positions 0..T-1 of unit (b, h) in fp64 (CPU)."""
    P = pool.shape[2]
    pos = np.arange(T)
    pages = table[b, pos // P].astype(np.int64)
    return pool[pages, h, pos % P]


def attend_reference(q, k_pool, v_pool, table, lens, q_lens):
    """fp64 out [tokens][Hq][d], lse [tokens][Hq] and, for the bounds, the
    weighted sum of |v| and the largest sum |q_e k_e| / sqrt(d) over the keys
    a query sees.  Keys a query does not see are left out, not weighted 0."""
    q = q.detach().cpu().double().numpy()
    kp, vp = k_pool.detach().cpu().double().numpy(), v_pool.detach().cpu().double().numpy()
    table = table.detach().cpu().numpy()
    Hkv, d = kp.shape[1], kp.shape[3]
    n_tok, Hq = sum(q_lens), q.shape[1]
    G = Hq // Hkv
    out, mag = np.zeros((n_tok, Hq, d)), np.zeros((n_tok, Hq, d))
    lse, dot = np.zeros((n_tok, Hq)), np.zeros((n_tok, Hq))
    t0 = 0
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (T, n) in enumerate(zip(lens, q_lens)):
            for h in range(Hkv if n else 0):
                k, v = rows_of(kp, table, b, h, T), rows_of(vp, table, b, h, T)
                qs = q[t0:t0 + n, h * G:(h + 1) * G]
                s = np.einsum("igd,kd->igk", qs, k) / math.sqrt(d)
                a = np.einsum("igd,kd->igk", np.abs(qs), np.abs(k)) / math.sqrt(d)
                for i in range(n):
                    seen = T - n + i + 1
                    x = s[i, :, :seen]
                    top = x.max(axis=1, keepdims=True)
                    w = np.exp(x - np.where(np.isinf(top), 0, top))
                    mass = w.sum(axis=1, keepdims=True)
                    w = w / mass
                    sl = (t0 + i, slice(h * G, (h + 1) * G))
                    out[sl], mag[sl] = w @ v[:seen], w @ np.abs(v[:seen])
                    lse[sl] = top[:, 0] + np.log(mass[:, 0])
                    dot[sl] = a[i, :, :seen].max(axis=1)
            t0 += n
    return out, lse, mag, dot


def attend_bounds(out, lse, mag, dot, dtype, T, d, weight=None):
    """Error bounds from the arithmetic.  A score is d exact (bf16) or rounded
    products added in fp32, at most 2^-23 relative an addition, then one
    scaling: |ds| <= (d + 4) 2^-23 dot.  2^x is taken to within 2^-20.  A
    weight is then off by ds + 2^-20 relative, and by a rounding to the
    storage type on the way to the product with the values (bf16; `weight`:
    the rounding of a weight where it is another).  The mass
    and the output add T terms in fp32 (T 2^-23).  The output divides by the
    mass, so both errors count, and is rounded once."""
    w = (d + 4) * 2.0 ** -23 * dot + 2.0 ** -20 + T * 2.0 ** -23
    rounded = U[torch.bfloat16] if dtype == torch.bfloat16 else 0.0
    if weight is not None:
        rounded = weight
    tol_out = (2 * w[..., None] + rounded) * mag * 1.01 + U[dtype] * np.abs(out) + 1e-30
    tol_lse = w + 2.0 ** -22 * (1 + np.abs(lse))
    return tol_out, tol_lse


def assert_attend(got_out, got_lse, ref, dtype, T, d, weight=None):
    out, lse, mag, dot = ref
    tol_out, tol_lse = attend_bounds(out, lse, mag, dot, dtype, T, d, weight)
    err = np.abs(got_out.detach().cpu().double().numpy()[:len(out)] - out)
    assert (err <= tol_out).all(), f"out: {np.nanmax(err / tol_out)} of the bound, {np.isnan(err).sum()} NaN"
    err = np.abs(got_lse.detach().cpu().double().numpy()[:len(out)] - lse)
    assert (err <= tol_lse).all(), f"lse: {np.nanmax(err / tol_lse)} of the bound, {np.isnan(err).sum()} NaN"


def random_table(lens, page, seed, spare=3):
    """A block table over a shuffled pool; the entries behind a sequence's
    pages name no page."""
    rng = np.random.default_rng(seed)
    need = [-(-T // page) for T in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(need) + 2), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), sum(need) + spare
