"""Plain 64-bit forms of the serving operators, and their inputs, for the tests.
They follow the definitions of include/gdn_serve.h token by token."""

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- tables


def tables(ctx, new, rows, T_total, page, table, counts, free, state):
    """Lists in, lists out; table, counts, free and state are updated."""
    cap, num_rows, max_blocks = len(free), len(counts), len(table[0]) if table else 0
    head, left = (state[0] % cap if cap else 0), state[1]
    cu, kv, slots, pos, refused, back = [0], [], [-1] * T_total, [0] * T_total, 0, []
    need_sum = taken = 0
    for n, (c, x) in enumerate(zip(ctx, new)):
        row = n if rows is None else rows[n]
        inside = 0 <= row < num_rows
        owned = counts[row] if inside else 0
        first, last = cu[-1], min(cu[-1] + max(x, 0), T_total)
        cu.append(last)
        add = last - first
        if x < 0:
            kv.append(0)
            if inside:
                back += table[row][:owned]
                table[row][:owned] = [-1] * owned
                counts[row] = 0
            continue
        blocks = -(-(c + add) // page)
        fine = inside and blocks <= max_blocks and -(-c // page) <= owned
        need = max(0, blocks - owned) if fine else 0
        need_sum += need
        if need and need_sum > left:
            fine = False
        if not fine:
            refused += 1
            kv.append(c)
        else:
            for j in range(need):
                table[row][owned + j] = free[(head + need_sum - need + j) % cap]
            counts[row] = owned + need
            taken += need
            kv.append(c + add)
        for i in range(add):
            pos[first + i] = c + i
            if fine:
                entry = table[row][(c + i) // page]
                slots[first + i] = entry * page + (c + i) % page if entry >= 0 else -1
    for i, p in enumerate(back):
        free[(head + left + i) % cap] = p
    state[:] = [(head + taken) % cap if cap else 0, left - taken + len(back), refused]
    return cu, kv, slots, pos


# ---------------------------------------------------------------- the cache


def nearest_e4m3(x):
    """float64 values to the nearest e4m3 value, ties to even; Inf and NaN to NaN."""
    y = np.where(np.isfinite(x), x, 0.0)
    unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.where(np.isfinite(x), np.rint(y / unit) * unit, np.nan)


def page_scale(amax):
    """The smallest power of two s >= 2^-100 with amax / s <= 448."""
    e = -100
    while math.ldexp(448.0, e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def tokens_of(v):
    """Values' pages [.., page / 16, dv, 16] as [.., page, dv]."""
    return v.transpose(-1, -2).flatten(-3, -2)


def packed(v):
    return v.unflatten(-2, (-1, 16)).transpose(-1, -2)


def write(x, slots, codes, scales):
    """x [T, H, d] into codes [pages, H, page, d] (values the codes stand for before the scale) and scales, float64
    numpy arrays that are updated."""
    page = codes.shape[2]
    runs = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * page:
            runs.setdefault(s // page, []).append(t)
    for p, ts in runs.items():
        a = slots[ts[0]] % page
        for h in range(x.shape[1]):
            part = x[ts, h]
            need = page_scale(np.max(np.where(np.isfinite(part), np.abs(part), 0.0)))
            if a == 0:
                now = need
                codes[p, h] = 0
            else:
                now = max(need, scales[p, h])
                codes[p, h] = nearest_e4m3(codes[p, h] * (scales[p, h] / now))
            codes[p, h, a:a + len(ts)] = nearest_e4m3(part / now)
            scales[p, h] = now


def attention(q, k, v, scale, first_pos, seen):
    """q [L, G, dk], k [S, dk], v [S, dv] of one request and key/value head in float64 (a token outside `seen` is left
    out); row i sees the tokens up to first_pos + i.  Returns (o, sum_j p_j |v_j|, largest sum |q||k| of a row)."""
    L, S = q.shape[0], k.shape[0]
    if not S:
        none = torch.zeros((L, q.shape[1], v.shape[1]), dtype=q.dtype, device=q.device)
        return none, none, none[..., :1]
    vis = seen[None, :] & (torch.arange(S, device=q.device)[None, :]
                           <= first_pos + torch.arange(L, device=q.device)[:, None])
    x = torch.einsum("lgd,sd->lgs", q, k) * scale
    x = torch.where(vis[:, None, :], x, torch.tensor(-math.inf, dtype=x.dtype, device=x.device))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    p = torch.where(vis[:, None, :], p, 0.0)
    total = p.sum(-1, keepdim=True)
    some = vis.any(-1)[:, None, None]
    p = torch.where(some, p / total, 0.0)
    # a NaN value reaches the rows that see its token and no others
    bad = torch.isnan(v)
    o = p @ torch.where(bad, 0.0, v)
    hit = (vis.to(v.dtype) @ bad.to(v.dtype)) > 0
    o = torch.where(hit[:, None, :], math.nan, o)
    return o, p @ torch.where(bad, 0.0, v.abs()), (q.abs() @ torch.nan_to_num(k.abs()).T).amax(-1, keepdim=True) * abs(scale)


# ---------------------------------------------------------------- the pool


def pool(q, k, v, g, beta, states, slots, cu, commit, q_scale, eps):
    """float64 tensors; returns o, states and the same of the recurrence of magnitudes (for error bounds)."""
    if eps > 0:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps) for x in (q, k))
    T, hk, dk = q.shape
    H, dv = v.shape[1:]
    share = torch.arange(H, device=q.device) // (H // hk)
    a = torch.exp(g) if g.dim() == 3 else torch.exp(g)[:, :, None].expand(-1, -1, dk)
    out, o, big_o = states.clone(), torch.full((T, H, dv), math.nan, dtype=q.dtype, device=q.device), None
    big_o, big_states = o.clone(), states.abs()
    for n, slot in enumerate(slots):
        if not 0 <= slot < states.shape[0]:
            continue
        S, M = states[slot].clone(), states[slot].abs()
        keep = cu[n + 1] - cu[n] if commit is None else commit[n]
        for i, t in enumerate(range(cu[n], cu[n + 1])):
            kt, qt = k[t][share], q[t][share] * q_scale
            S, M = S * a[t][..., None], M * a[t][..., None]
            u = beta[t][:, None] * (v[t] - (S * kt[..., None]).sum(1))
            m = beta[t][:, None] * (v[t].abs() + (M * kt.abs()[..., None]).sum(1))
            S, M = S + kt[..., None] * u[:, None], M + kt.abs()[..., None] * m[:, None]
            o[t], big_o[t] = (S * qt[..., None]).sum(1), (M * qt.abs()[..., None]).sum(1)
            if i + 1 == min(keep, cu[n + 1] - cu[n]):
                out[slot], big_states[slot] = S, M
    return o, out, big_o, big_states


# ---------------------------------------------------------------- inputs


class Server:
    """A paged cache filled through float64 writes of random keys and values, and its plain contents."""

    def __init__(self, kv_lens, page, hkv, dk, dv, seed=0, spare=3, device="cpu", rows=False):
        gen = torch.Generator().manual_seed(seed)
        self.page, self.kv_lens, self.device = page, list(kv_lens), device
        n = len(self.kv_lens)
        blocks = [-(-x // page) for x in self.kv_lens]
        pages = sum(blocks) + spare
        order = torch.randperm(pages, generator=gen).tolist()
        self.max_blocks = max([1] + blocks) + 1
        self.rows = torch.randperm(n + 2, generator=gen)[:n].to(torch.int32) if rows else None
        self.table = torch.full((n + 2 if rows else n, self.max_blocks), -1, dtype=torch.int32)
        for i, b in enumerate(blocks):
            row = int(self.rows[i]) if rows else i
            self.table[row, :b] = torch.tensor([order.pop() for _ in range(b)], dtype=torch.int32)
        # codes over the whole range of the format, scales of several powers of two
        self.k = (torch.randn((pages, hkv, page, dk), generator=gen) * 60).clamp(-448, 448).to(E4M3)
        self.v = (torch.randn((pages, hkv, page, dv), generator=gen) * 60).clamp(-448, 448).to(E4M3)
        self.ks = torch.exp2(torch.randint(-8, -4, (pages, hkv), generator=gen).float())
        self.vs = torch.exp2(torch.randint(-8, -4, (pages, hkv), generator=gen).float())

    def to(self, device):
        """(k_cache, v_cache, k_scale, v_scale, table, kv_lens, rows) as the library takes them."""
        vc = packed(self.v.float()).to(E4M3).contiguous()
        return (self.k.to(device), vc.to(device), self.ks.to(device), self.vs.to(device), self.table.to(device),
                torch.tensor(self.kv_lens, dtype=torch.int32, device=device),
                None if self.rows is None else self.rows.to(device))

    def reference(self, q, lens, scale, device="cpu"):
        """o, sum p|v| and the largest sum |q||k| for q [T, H, dk] (float64)."""
        T, H, dk = q.shape
        hkv, dv, pages = self.k.shape[1], self.v.shape[3], self.k.shape[0]
        G = H // hkv
        f = lambda t: t.float().to(device, torch.float64)
        o, mag, big = (torch.zeros((T, H, w), dtype=torch.float64, device=device) for w in (dv, dv, 1))
        t = 0
        for n, L in enumerate(lens):
            S = min(max(self.kv_lens[n], 0), self.table.shape[1] * self.page)
            row = n if self.rows is None else int(self.rows[n])
            entries = self.table[row][:-(-S // self.page)].tolist() if 0 <= row < self.table.shape[0] else []
            seen = torch.zeros(S, dtype=torch.bool, device=device)
            k = torch.zeros((hkv, S, dk), dtype=torch.float64, device=device)
            v = torch.zeros((hkv, S, dv), dtype=torch.float64, device=device)
            for b, p in enumerate(entries):
                if 0 <= p < pages:
                    w = min(self.page, S - b * self.page)
                    sl = slice(b * self.page, b * self.page + w)
                    seen[sl] = True
                    k[:, sl] = f(self.k[p, :, :w]) * f(self.ks[p])[:, None, None]
                    v[:, sl] = f(self.v[p, :, :w]) * f(self.vs[p])[:, None, None]
            for h in range(hkv if L else 0):
                hs = slice(h * G, (h + 1) * G)
                o[t:t + L, hs], mag[t:t + L, hs], big[t:t + L, hs] = attention(q[t:t + L, hs], k[h], v[h], scale, S - L, seen)
            t += L
        return o, mag, big
