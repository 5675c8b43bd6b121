"""Plain 64-bit forms of the serving operators (routing from logits, the paged cache, attention over it), written
request by request and token by token, with the error bounds the GPU tests hold the kernels to."""
from __future__ import annotations

import numpy as np

WIDTH, VALUE = 576, 512


def route(z, bias, *, k, score="sigmoid", groups=1, keep=1, gscore="top2", renorm=True, scale=1.0):
    """(ids ascending [T][k], weights [T][k]) of fp64 logits z [T][E]."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    T, E = z.shape
    ids, ws = np.empty((T, k), np.int32), np.empty((T, k))
    for t in range(T):
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-z[t]))
        else:
            m = z[t].max()
            if m == np.inf:
                e = (z[t] == np.inf).astype(np.float64)
            elif m == -np.inf:
                e = np.zeros(E)
            else:
                e = np.exp(z[t] - m)
            s = e / e.sum() if e.sum() > 0 else e
        u = s + (bias.astype(np.float64) if bias is not None else 0.0)
        u = np.where(np.isnan(u), -np.inf, u)
        size, open_ = E // groups, range(groups)
        if keep < groups:
            gs = []
            for g in range(groups):
                part = sorted(u[g * size:(g + 1) * size], reverse=True)
                with np.errstate(invalid="ignore"):
                    v = part[0] + part[1] if gscore == "top2" else part[0]
                gs.append(-np.inf if np.isnan(v) else v)
            open_ = sorted(range(groups), key=lambda g: (-gs[g], g))[:keep]
        cand = [e for e in range(E) if e // size in set(open_)]
        pick = sorted(sorted(cand, key=lambda e: (-u[e], e))[:k])
        w = s[pick]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        ids[t], ws[t] = pick, scale * w
    return ids, ws


NO_PAGES, TABLE_FULL, TOKENS, BAD_PAGE = 8, 16, 32, 64


def step(page, max_pages, n_pages, n_tokens, new, seq, held, table, free, count):
    """One step of the cache's bookkeeping, request by request; returns a dict of the outputs (fresh arrays)."""
    B = len(new)
    table, free, status = table.copy(), list(free), 0
    if not 0 <= count <= n_pages:
        status |= BAD_PAGE
        count = min(max(count, 0), n_pages)
    fine = [0 <= held[b] <= max_pages for b in range(B)]
    h = [held[b] if fine[b] else 0 for b in range(B)]
    for b in range(B):
        if new[b] < 0:
            for i in range(h[b]):
                if count < n_pages:
                    free[count] = table[b][i]
                    count += 1
                else:
                    status |= BAD_PAGE
    out = dict(seq_out=np.zeros(B, np.int32), held_out=np.zeros(B, np.int32), q_start=np.zeros(B + 1, np.int32),
               position=[], slot=[])
    asked_pages = asked_tokens = 0
    avail = count
    for b in range(B):
        add, need = 0, 0
        if new[b] >= 0:
            pages = -(-(seq[b] + new[b]) // page)
            if not (fine[b] and seq[b] >= 0 and seq[b] <= h[b] * page and pages <= max_pages):
                status |= TABLE_FULL
            else:
                add, need = new[b], max(0, pages - h[b])
                asked_pages += need
                asked_tokens += add
                refuse = False
                if need and asked_pages > avail:
                    status |= NO_PAGES
                    refuse = True
                if add and asked_tokens > n_tokens:
                    status |= TOKENS
                    refuse = True
                if refuse:
                    add, need = 0, 0
        elif not fine[b]:
            status |= TABLE_FULL
        out["q_start"][b + 1] = out["q_start"][b] + add
        for i in range(need):
            count -= 1
            table[b][h[b] + i] = free[count]
        for i in range(add):
            pos = seq[b] + i
            pg = table[b][pos // page]
            out["position"].append(pos)
            if 0 <= pg < n_pages:
                out["slot"].append(pg * page + pos % page)
            else:
                out["slot"].append(-1)
                status |= BAD_PAGE
        if new[b] >= 0:
            out["seq_out"][b], out["held_out"][b] = seq[b] + add, h[b] + need
    out.update(table=table, free=np.array(free, np.int32), count_out=count, status=status,
               position=np.array(out["position"], np.int32), slot=np.array(out["slot"], np.int32))
    return out


def attention(q, cache, table, q_start, seq, scale, eps, *, sel=None, tiny=0.0):
    """out, lse and the error bounds of both.  q [N][H][576], cache [n_pages][rows][576] fp64 (rows >= page size),
    eps: the step of the type (torch.finfo(t).eps), tiny: the spacing of its subnormal numbers.

    Bounds, with p the weights and A = sum p |v|:
    * a score is a sum of 576 exact products in fp32 (each addition off by at most 2^-23 of the running magnitude, as the
      tensor cores may truncate) and one product with the scale, itself rounded: ds = 580 * 2^-23 * scale * sum |q k|;
    * a weight is exp2 of it (relative 2^-21: 2 ulp, and the argument's own rounding 2^-23 * (|s| log2 e + 16)) and is
      rounded to the type (eps / 2; below the type's normal range half of `tiny`, relative to the largest weight, which is
      at least 1/2): dp = 2 ds + 2^-21 + 2^-22 * (1.5 |s| + 16) + eps / 2;
    * the same errors without the rounding, and those of summing n weights (2^-23 n), are in the denominator;
    * the products with v sum in fp32 (2^-23 n), and the result is rounded (eps / 2).
    """
    N, H = q.shape[0], q.shape[1]
    page = cache.page
    out, lse = np.zeros((N, H, VALUE)), np.full((N, H), -np.inf)
    tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    done = np.zeros(N, bool)
    for b in range(len(seq)):
        T = q_start[b + 1] - q_start[b]
        for i in range(T):
            n = q_start[b] + i
            done[n] = True
            last = min(seq[b] - T + i, seq[b] - 1)
            keys = range(last + 1) if sel is None else [s for s in sel[n] if 0 <= s <= last]
            keys = [s for s in keys if s // page < table.shape[1] and 0 <= table[b][s // page] < cache.n_pages]
            if not keys:
                continue
            kv = np.stack([cache.row(table[b][s // page], s % page) for s in keys])
            raw = kv @ q[n].T                                   # [keys][H]
            s = scale * raw
            ds = 580 * 2.0 ** -23 * abs(scale) * (np.abs(kv) @ np.abs(q[n].T)).max(0)
            m = s.max(0)
            e = np.exp(s - m)
            l = e.sum(0)
            p = e / l
            o, A = p.T @ kv[:, :VALUE], p.T @ np.abs(kv[:, :VALUE])
            exp_err = 2 * ds + 2.0 ** -21 + 2.0 ** -22 * (1.5 * np.abs(s).max(0) + 16)
            count = 2.0 ** -23 * (len(keys) + 64)
            rel = 2 * exp_err + eps / 2 + 2 * count
            out[n], lse[n] = o, m + np.log(l)
            tol[n] = rel[:, None] * A * 1.05 + eps / 2 * np.abs(o) * 1.05 + tiny * np.abs(kv[:, :VALUE]).sum(0) + tiny
            tol_lse[n] = exp_err + count + 2.0 ** -22 * np.abs(lse[n]) + 2.0 ** -22
    return out, lse, tol, tol_lse, done


class Cache:
    """fp64 view of a paged cache [n_pages][page_stride] elements."""

    def __init__(self, flat, page, stride):
        self.flat, self.page, self.stride = flat, page, stride
        self.n_pages = flat.size // stride

    def row(self, page, r):
        a = page * self.stride + r * WIDTH
        return self.flat[a:a + WIDTH]


def pages_of(n, page):
    return -(-n // page)


