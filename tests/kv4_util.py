"""Plain float64 forms of the 4-bit cache's operators, for the tests (no test
functions here).  They work on numpy copies of the pool's bytes and share no
code with the library."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "fp8": torch.float8_e4m3fn}
# Largest relative error of one rounding to nearest.
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24, "fp8": 2.0 ** -4}
# Half of the spacing of the smallest values (FP8's is 2^-9).
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0, "fp8": 2.0 ** -10}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def hold(y):
    """Codes [..., D] and the fp32 step and middle [...] of rows y (float32),
    in the header's fp32 steps."""
    y = np.asarray(y, dtype=np.float32)
    lo, hi = y.min(-1), y.max(-1)
    half = np.float32(0.5)
    step = (hi * half - lo * half) * np.float32(2.0 / 15.0)
    step = np.where(step < np.float32(2.0 ** -126), np.float32(0), step)
    mid = (lo.astype(np.float64) + 8.0 * step.astype(np.float64)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(step > 0, np.float32(1) / step, np.float32(0)).astype(np.float32)
    c = np.rint((y - mid[..., None]) * inv[..., None])
    return (np.clip(c, -8, 7) + 8).astype(np.uint8), step, mid


class Held:
    """The pool's content: codes [pages, Hk, page, D] and params
    [pages, Hk, page, 2] (scale, mid as float64) for K (0) and V (1)."""

    def __init__(self, cache):
        D, page = cache.D, cache.page_size
        raw = cache.pool.cpu().numpy()
        P, Hk, nb, _ = raw.shape
        self.codes, self.params = [], []
        for kv in range(2):
            b = raw[..., kv * 8 * D:(kv + 1) * 8 * D].reshape(P, Hk, nb, 16, D // 2)
            c = np.stack([b & 15, b >> 4], -1).reshape(P, Hk, page, D)
            at = 16 * D + 64 * kv
            w = np.ascontiguousarray(raw[..., at:at + 64]).view(np.uint16).astype(np.uint32) << 16
            self.codes.append(c)
            self.params.append(w.view(np.float32).astype(np.float64).reshape(P, Hk, page, 2))

    def rows(self, kv, pages, page, n):
        """(codes - 8, scale, mid) of the first n rows of a list of pages: [Hk, n, ...]."""
        j = np.arange(n)
        p = np.asarray(pages)[j // page]
        c = self.codes[kv][p, :, j % page].astype(np.float64) - 8
        s = self.params[kv][p, :, j % page]
        return c.transpose(1, 0, 2), s[..., 0].T, s[..., 1].T


def attend(cache, q, Hq, table, lens, starts, scale, dtype):
    """out, lse, the weights added to each row, and error bounds.

    The bound for out counts: one rounding of the output; the weights that
    multiply V, rounded to fp16 (2^-11 relative, at least 2^-25 of the largest
    weight times V scale) or held in two fp16 parts (2^-21); and the relative
    error of each weight, exp(d) - 1 with d the error of a logit: D + 16
    roundings of 2^-23 each (the matrix unit may truncate) of the sum of |terms|.
    Codes that enter a product as fp16 subnormal numbers (c * 2^-24, exponent
    field 2^-14; all types but fp32, and V for bf16 and FP8 only) are aligned by
    that field, so a product of 16 terms keeps 2^-23 of the largest other
    operand x 2^-14, which is 2^-13 of that operand in steps of the code."""
    T, Hk, D, page = q.shape[0], cache.Hk, cache.D, cache.page_size
    G = Hq // Hk
    held = Held(cache)
    out = np.zeros((T, Hk, G, D))
    lse = np.full((T, Hk, G), -np.inf)
    bound = np.zeros_like(out)
    lse_bound = np.zeros_like(lse)
    add = np.zeros((cache.num_pages, Hk, page))
    add_bound = np.zeros_like(add)
    part = 2.0 ** -11 if dtype in ("bf16", "fp8") else 2.0 ** -21
    x = f64(q)[:, :Hq * D].reshape(T, Hk, G, D)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        pages = table[b]
        ck, sk, mk = held.rows(0, pages, page, n)
        cv, sv, mv = held.rows(1, pages, page, n)
        k = ck * sk[..., None] + mk[..., None]
        v = cv * sv[..., None] + mv[..., None]
        nq = starts[b + 1] - starts[b]
        for i in range(nq):
            t, sees = starts[b] + i, n - nq + i + 1
            if sees <= 0:
                continue
            s = slice(0, sees)
            w = np.einsum("hgd,hnd->hgn", x[t], k[:, s]) * scale
            terms = np.einsum("hgd,hnd->hgn", np.abs(x[t]),
                              np.abs(ck[:, s]) * sk[:, s, None] + np.abs(mk[:, s, None])) * abs(scale)
            d = (D + 16) * 2.0 ** -23 * terms + 2.0 ** -22 * (1 + np.abs(w).max())
            if dtype != "fp32":
                d += D / 16 * 2.0 ** -13 * np.abs(x[t]).max((1, 2))[:, None, None] * (
                    sk[:, None, s] * abs(scale))
            top = w.max(-1, keepdims=True)
            e = np.exp(w - top)
            total = e.sum(-1, keepdims=True)
            p = e / total
            rel = np.expm1(2 * d.max(-1, keepdims=True)) + (sees + 16) * 2.0 ** -24
            lse[t] = (top + np.log(total))[..., 0]
            lse_bound[t] = rel[..., 0] + 2.0 ** -22 * np.abs(lse[t])
            out[t] = np.einsum("hgn,hnd->hgd", p, v[:, s])
            mag = np.einsum("hgn,hnd->hgd", p, np.abs(cv[:, s]) * sv[:, s, None])
            mids = np.einsum("hgn,hn->hg", p, np.abs(mv[:, s]))[..., None]
            floor = (2.0 ** -25 if part == 2.0 ** -11 else 2.0 ** -35) * 8
            least = floor * sees * sv[:, s].max(-1)[:, None, None] / total
            # A sum may be taken over the codes c themselves with 8 times the
            # weights taken off: its terms are then up to |c - 8| + 8 in size,
            # and each addition rounds (or truncates) at 2^-23 of that.
            eights = 8 * np.einsum("hgn,hn->hg", p, sv[:, s])[..., None]
            bound[t] = (part * mag + least + rel * (mag + mids)
                        + (sees + 16) * 2.0 ** -23 * (mag + eights + mids)
                        + (2.0 ** -13 / 8 * eights if part == 2.0 ** -11 else 0.0))
            j = np.arange(sees)
            at = np.asarray(pages)[j // page]
            add[at, :, j % page] += p.sum(1).T
            add_bound[at, :, j % page] += (p * rel).sum(1).T
    bound += HALF_STEP[dtype] * (np.abs(out) + bound) + TINY[dtype]
    return (out.reshape(T, Hq * D), lse.reshape(T, Hq), add, bound.reshape(T, Hq * D),
            lse_bound.reshape(T, Hq), add_bound)


def evict(scores, table, lens, page, budget, recent):
    """The kept rows of each sequence and head, by a stable sort."""
    B, Hk = len(lens), scores.shape[1]
    kept = np.full((B, Hk, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(Hk):
            j = np.arange(n)
            s = scores[np.asarray(table[b])[j // page], h, j % page] if n else np.zeros(0)
            new = j >= n - recent
            rank = np.where(np.isnan(s), -np.inf, s)
            order = np.lexsort((j, np.isnan(s), -rank, ~new))  # the last key goes first
            keep = np.sort(order[:min(n, budget)])
            kept[b, h, :len(keep)] = keep
    return kept


def fill(cache, seed, spread=1.0):
    """Random rows in every slot of a cache: keys and values as codes with
    parameters of different sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool, D = cache.pool, cache.D
    pool[..., :16 * D] = torch.randint(0, 256, pool[..., :16 * D].shape, generator=g,
                                       device="cuda", dtype=torch.uint8)
    shape = pool.shape[:3] + (32, 1)
    scale = torch.exp(spread * torch.randn(shape, generator=g, device="cuda")) * 0.2
    mid = 0.2 * torch.randn(shape, generator=g, device="cuda") * scale
    pool[..., 16 * D:] = torch.cat([scale, mid], -1).bfloat16().view(torch.uint8).flatten(3)
