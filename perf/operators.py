"""The serving operators beside the gated delta-rule layer, as they are timed and checked.

Four operators of one serving step of a stack that mixes delta-rule layers
(fixed-size states) with attention layers (a cache that grows):

  tables     block tables, slot map, positions and packed offsets of a step,
             from the requests' lengths (gdn_batch_tables)
  write      keys and values into the paged 8-bit cache, one scale for each
             page and head (gdn_cache_write)
  attention  causal attention over that cache, one to many new tokens for each
             request (gdn_cache_attention)
  pool       the delta rule's recurrent form on a pool of states, one or a few
             tokens for each request (gdn_decode_pool)

run() computes a case in plain torch operations, or, with `own`, through the
library.
"""

import math
import zlib

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXPONENT = -100  # of a page's scale


def listed():
    return [
        # one decode step of a busy server: each request adds a token, a few have ended
        dict(name="tables_decode_512", op="tables", n=512, page=64, max_ctx=16384, lo=1, hi=1, ended=9),
        # admission of 64 prompts of 512 to 16384 tokens
        dict(name="tables_prompts_64", op="tables", n=64, page=128, max_ctx=0, lo=512, hi=16384, ended=0),
        # such a step's new keys and values, one behind what each request holds
        dict(name="write_decode_512", op="write", n=512, max_ctx=16384, lo=1, hi=1, hkv=8, dk=128, dv=128, page=64,
             dtype="bf16"),
        # one prompt of 65536 tokens
        dict(name="write_prompt_64k", op="write", n=1, max_ctx=0, lo=65536, hi=65536, hkv=8, dk=128, dv=128, page=64,
             dtype="bf16"),
        # one user, one token, a long context: latency
        dict(name="attn_one_64k", op="attention", n=1, ctx_lo=65535, ctx_hi=65535, lo=1, hi=1, heads=32, hkv=8, dk=128,
             dv=128, page=64, dtype="bf16"),
        # decode of 64 requests of very different lengths
        dict(name="attn_decode_64", op="attention", n=64, ctx_lo=511, ctx_hi=16383, lo=1, hi=1, heads=32, hkv=8,
             dk=128, dv=128, page=64, dtype="bf16"),
        # drafted tokens being verified, full precision, odd lengths
        dict(name="attn_verify_f32", op="attention", n=23, ctx_lo=0, ctx_hi=4097, lo=1, hi=5, heads=12, hkv=4, dk=64,
             dv=64, page=128, dtype="f32"),
        # a chunk of a long prompt beside short requests
        dict(name="attn_chunk_16k", op="attention", n=3, ctx_lo=16001, ctx_hi=16384, lo=1021, hi=2048, heads=32,
             hkv=8, dk=128, dv=128, page=64, dtype="bf16"),
        # two whole prompts of 8192 tokens
        dict(name="attn_prompt_8k", op="attention", n=2, ctx_lo=0, ctx_hi=0, lo=8192, hi=8192, heads=32, hkv=8,
             dk=128, dv=128, page=64, dtype="bf16"),
        # one user, one token: latency
        dict(name="pool_one", op="pool", n=1, spare=7, lo=1, hi=1, heads=32, hk=32, dk=128, dv=128, dtype="bf16",
             head_gate=False, norm=False),
        # decode of 512 requests, keys and queries shared by two value heads
        dict(name="pool_decode_512", op="pool", n=512, spare=64, lo=1, hi=1, heads=32, hk=16, dk=128, dv=128,
             dtype="bf16", head_gate=False, norm=True),
        # drafted tokens being verified, one gate per head, full precision
        dict(name="pool_verify_f32", op="pool", n=45, spare=3, lo=1, hi=7, heads=12, hk=4, dk=64, dv=128, dtype="f32",
             head_gate=True, norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "attention", "attention", "pool"])
    if op == "tables":
        prompts = rng.random() < 0.5
        n = _log(rng, 1, 64) if prompts else _log(rng, 1, 512)
        hi = _log(rng, 2, 16384) if prompts else rng.randint(1, 4)
        return dict(op=op, n=n, page=rng.choice([64, 128, 256]), max_ctx=_log(rng, 1, 16384), lo=rng.randint(0, 1),
                    hi=hi, ended=rng.randint(0, n // 4))
    if op == "write":
        prompts = rng.random() < 0.5
        n = _log(rng, 1, 8) if prompts else _log(rng, 1, 512)
        hi = _log(rng, 5, 8192) if prompts else rng.randint(1, 4)
        return dict(op=op, n=n, max_ctx=_log(rng, 1, 16384 if n > 8 else 2048), lo=rng.randint(0, 1), hi=hi,
                    hkv=rng.choice([1, 2, 3, 4, 8]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    page=rng.choice([64, 128, 256]), dtype=rng.choice(["bf16", "f32"]))
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8])
        heads = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        kind = rng.choice(["decode", "verify", "chunk"])
        n = _log(rng, 1, 64) if kind == "decode" else _log(rng, 1, 24) if kind == "verify" else _log(rng, 1, 3)
        lo, hi = (1, 1) if kind == "decode" else (1, rng.randint(2, 8)) if kind == "verify" else (0, _log(rng, 9, 2048))
        return dict(op=op, n=n, ctx_lo=0, ctx_hi=_log(rng, 3, 4096 if kind == "chunk" else 16384), lo=lo, hi=hi,
                    heads=heads, hkv=hkv, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    page=rng.choice([64, 128, 256]), dtype="bf16" if rng.random() < 0.7 else "f32")
    hk = rng.choice([1, 2, 4, 8, 16])
    heads = min(32, hk * rng.choice([1, 2, 3, 4]))
    heads -= heads % hk
    many = rng.random() < 0.5
    return dict(op=op, n=_log(rng, 1, 512) if many else _log(rng, 1, 64), spare=rng.randint(0, 9),
                lo=rng.randint(0, 1), hi=rng.randint(1, 2) if many else rng.randint(2, 8), heads=heads, hk=hk,
                dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f32"]),
                head_gate=rng.random() < 0.4, norm=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _requests(case):
    """Tokens held and new tokens of each request (CPU): the case's alone, so that all its inputs are of one size.
    Where there is a range, one request has its upper end; -1 new tokens: the request has ended."""
    gen = torch.Generator().manual_seed(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    n = case["n"]

    def lengths(lo, hi):
        x = torch.randint(lo, hi + 1, (n,), generator=gen)
        x[int(torch.randint(0, n, (1,), generator=gen))] = hi
        return x

    if "max_ctx" in case:
        ctx = torch.randint(0, case["max_ctx"] + 1, (n,), generator=gen)
    else:
        ctx = lengths(case.get("ctx_lo", 0), case.get("ctx_hi", 0))
    new = lengths(case["lo"], case["hi"])
    new[torch.randperm(n, generator=gen)[:case.get("ended", 0)]] = -1
    return ctx, new


def _offsets(lens):
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(lens, 0).to(torch.int32)
    return cu


def _paged(gen, total, page, extra):
    """A block table for requests of `total` tokens, pages in random order, -1 where a row ends; the number of pages."""
    blocks = (total + page - 1) // page
    used = int(blocks.sum())
    pages = used + extra
    order = torch.randperm(pages, generator=gen)
    cols = max(1, int(blocks.max()))
    live = torch.arange(cols)[None, :] < blocks[:, None]
    table = torch.full((total.numel(), cols), -1, dtype=torch.int32)
    table[live] = order[:used].to(torch.int32)
    return table, pages


def _cache(dev_gen, pages, heads, inner, bits):
    """Codes of unit normal values and power-of-two scales for each page and head."""
    exps = torch.randint(-7, -4, (pages, heads), generator=dev_gen, device=DEV)
    codes = torch.empty((pages, heads) + inner, dtype=E4M3, device=DEV)
    step = max(1, (1 << 27) // (heads * math.prod(inner)))
    for a in range(0, pages, step):  # in parts: the normal values take four times the codes' room
        x = torch.randn((min(step, pages - a), heads) + inner, generator=dev_gen, device=DEV)
        codes[a:a + step] = (x * bits).to(E4M3)
    return codes, torch.exp2(exps.float())


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator().manual_seed(seed * 7919 + 11)
    dev = torch.Generator(device=DEV).manual_seed(seed * 104729 + 5)

    def randn(*shape):
        return torch.randn(shape, generator=dev, device=DEV)

    ctx, new = _requests(case)
    order = torch.randperm(case["n"], generator=gen)
    ctx, new = ctx[order], new[order]
    if op == "tables":
        n, page = case["n"], case["page"]
        total = ctx + new.clamp(min=0)
        cols = max(1, int((total.max() + page - 1) // page))
        table, _ = _paged(gen, ctx, page, 0)
        table = torch.nn.functional.pad(table, (0, cols - table.shape[1]), value=-1) if cols > table.shape[1] else table
        owned = (ctx + page - 1) // page
        used, need = int(owned.sum()), int(((total + page - 1) // page).sum())
        pages = need + 3 + n // 2
        # every row of the server's table has a request or is idle; the step's requests come in any order
        rows = torch.randperm(n + 5, generator=gen)[:n]
        full = torch.full((n + 5, table.shape[1]), -1, dtype=torch.int32)
        full[rows] = table
        counts = torch.zeros(n + 5, dtype=torch.int32)
        counts[rows] = owned.to(torch.int32)
        free = torch.full((pages,), -1, dtype=torch.int32)
        head = int(torch.randint(0, pages, (1,), generator=gen))
        left = pages - used
        free[(head + torch.arange(left)) % pages] = (used + torch.randperm(left, generator=gen)).to(torch.int32)
        d = dict(ctx=ctx.to(torch.int32), new=new.to(torch.int32), rows=rows.to(torch.int32), table=full, counts=counts,
                 free=free, ring=torch.tensor([head, left, 0], dtype=torch.int32))
        s = {k: v.to(DEV) for k, v in d.items()}
        s.update(op=op, page=page, tokens=int(new.clamp(min=0).sum()))
        return s
    tokens, cu = int(new.sum()), _offsets(new)
    if op == "write":
        page, hkv, t = case["page"], case["hkv"], _type(case)
        # the pool holds the pages that the step touches, full or partly filled before it
        first = ctx // page
        table, pages = _paged(gen, ctx + new - first * page, page, 2)
        seq = torch.repeat_interleave(torch.arange(case["n"]), new)
        pos = torch.arange(tokens) - cu[:-1].long()[seq] + (ctx - first * page)[seq]
        slots = table[seq, pos // page].long() * page + pos % page
        kc, ks = _cache(dev, pages, hkv, (page, case["dk"]), 24.0)
        vc, vs = _cache(dev, pages, hkv, (page // 16, case["dv"], 16), 24.0)
        # a few channels carry much larger values, so pages' scales differ and some of them grow
        wide = torch.exp(1.5 * randn(1, hkv, 1))
        return dict(op=op, page=page, slots=slots.to(torch.int32).to(DEV), kc=kc, ks=ks, vc=vc, vs=vs,
                    k=(randn(tokens, hkv, case["dk"]) * wide).to(t), v=randn(tokens, hkv, case["dv"]).to(t))
    if op == "attention":
        page, hkv, t = case["page"], case["hkv"], _type(case)
        table, pages = _paged(gen, ctx + new, page, 2)
        kc, ks = _cache(dev, pages, hkv, (page, case["dk"]), 64.0)
        vc, vs = _cache(dev, pages, hkv, (page // 16, case["dv"], 16), 64.0)
        return dict(op=op, page=page, kc=kc, ks=ks, vc=vc, vs=vs, table=table.to(DEV),
                    kv_lens=(ctx + new).to(torch.int32).to(DEV), cu=cu.to(DEV),
                    q=randn(tokens, case["heads"], case["dk"]).to(t), scale=case["dk"] ** -0.5,
                    max_new=int(new.max()), max_kv=int((ctx + new).max()))
    n, h, hk, dk, dv, t = case["n"], case["heads"], case["hk"], case["dk"], case["dv"], _type(case)
    slots = torch.randperm(n + case["spare"], generator=gen)[:n]
    # of drafted tokens some are already known to be kept, the others are only tried
    keep = (torch.rand(n, generator=gen) * (new + 1)).long().clamp(max=new) if case["hi"] > 1 else None
    q, k = randn(tokens, hk, dk), randn(tokens, hk, dk)
    if not case["norm"]:
        q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    z = randn(tokens, h) if case["head_gate"] else randn(tokens, h, dk)
    return dict(op=op, q=q.to(t), k=k.to(t), v=randn(tokens, h, dv).to(t),
                g=-torch.log1p(torch.exp(2.0 * z)) if case["head_gate"] else torch.log(0.9 + 0.1 * torch.sigmoid(z)),
                beta=torch.sigmoid(randn(tokens, h)), states=0.02 * randn(n + case["spare"], h, dk, dv),
                slots=slots.to(torch.int32).to(DEV), cu=cu.to(DEV) if case["hi"] > 1 or case["lo"] < 1 else None,
                keep=None if keep is None else keep.to(torch.int32).to(DEV), q_scale=dk ** -0.5,
                eps=1e-6 if case["norm"] else 0.0, longest=int(new.max()))


# ---------------------------------------------------------------- plain forms


def _plain_tables(s):
    page, tokens = s["page"], s["tokens"]
    table, counts, free, ring = s["table"], s["counts"], s["free"], s["ring"]
    cap, cols = free.numel(), table.shape[1]
    ctx, new, rows = s["ctx"].long(), s["new"].long(), s["rows"].long()
    head, left = ring[0].long(), ring[1].long()
    owned = counts[rows].long()
    ended = new < 0
    grow = torch.where(ended, 0, new)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(grow, 0)]).clamp(max=tokens)
    grow = cu[1:] - cu[:-1]
    base = torch.maximum(owned, (ctx + page - 1) // page)
    last = (ctx + grow + page - 1) // page
    need = torch.where(ended | (last > cols), 0, (last - base).clamp(min=0))
    upto = torch.cumsum(need, 0)
    fine = ~ended & (last <= cols) & ((need == 0) | (upto <= left))
    taken = torch.where(fine & (need > 0), upto, 0).max()
    given = torch.where(ended, owned, 0)
    before = torch.cumsum(given, 0) - given
    kv = torch.where(fine, ctx + grow, ctx)
    kv = torch.where(ended, 0, kv)
    # pages that come back go to the ring's end
    at = torch.arange(cols, device=DEV)
    back = ended[:, None] & (at[None, :] < owned[:, None])
    goes = (head + left + before[:, None] + at[None, :]) % cap
    old = table[rows]
    free[goes[back]] = old[back]
    # pages that are needed come from its start
    j = at[None, :] - base[:, None]
    add = fine[:, None] & (j >= 0) & (j < need[:, None])
    comes = (head + (upto - need)[:, None] + j) % cap
    fresh = torch.where(add, free[torch.where(add, comes, 0)], old)
    fresh = torch.where(back, -1, fresh)
    table[rows] = fresh
    counts[rows] = torch.where(ended, 0, torch.where(fine, base + need, owned)).int()
    refused = (~fine & ~ended).sum()
    ring.copy_(torch.stack([(head + taken) % cap, left - taken + given.sum(), refused]))
    t = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=rows.numel() - 1)
    pos = t - cu[seq] + ctx[seq]
    at_page = fresh[seq, (pos // page).clamp(max=cols - 1)].long()
    slot = torch.where((t < cu[-1]) & fine[seq] & (at_page >= 0), at_page * page + pos % page, -1)
    return dict(cu=cu.int(), kv_lens=kv.int(), slots=slot.int(), positions=torch.where(t < cu[-1], pos, 0).int(),
                table=table, counts=counts, free=free, ring=ring)


def _scale_of(amax):
    """The smallest power of two with amax / scale <= 448 (not below 2^-100)."""
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    e = torch.where(m > 0.5, e, e - 1).clamp(min=MIN_EXPONENT)
    return torch.exp2(torch.where(amax > 0, e, MIN_EXPONENT).double()).float()


def _codes(x):
    return torch.where(torch.isfinite(x), x, float("nan")).to(E4M3)


def _tokens(v):
    """The values' pages [.., page / 16, dv, 16] as [.., page, dv]."""
    return v.transpose(-1, -2).flatten(-3, -2)


def _packed(v):
    """[.., page, dv] as the cache holds values."""
    return v.unflatten(-2, (-1, 16)).transpose(-1, -2)


def _plain_write_one(x, cache, scales, slots, page, across):
    """`across`: the cache is that of the values."""
    x = x.float()
    pages, heads = scales.shape
    at, off = slots.long() // page, slots.long() % page
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    amax = torch.zeros((pages, heads), device=DEV).scatter_reduce_(0, at[:, None].expand(-1, heads), top, "amax")
    first = torch.full((pages,), page, device=DEV, dtype=torch.long).scatter_reduce_(0, at, off, "amin")
    touched = (first < page).nonzero()[:, 0]
    first, was = first[touched], scales[touched]
    need = _scale_of(amax[touched])
    now = torch.where((first == 0)[:, None], need, torch.maximum(need, was))
    held = cache.view(torch.uint8)[touched].view(E4M3).float()
    held = _tokens(held) if across else held
    held = held * (was / now)[:, :, None, None]
    held = torch.where((first == 0)[:, None, None, None], 0.0, held)
    where = torch.full((pages,), 0, device=DEV, dtype=torch.long)
    where[touched] = torch.arange(touched.numel(), device=DEV)
    held = held.to(E4M3).view(torch.uint8)
    held[where[at], :, off] = _codes(x / now[where[at]][:, :, None]).view(torch.uint8)
    cache.view(torch.uint8)[touched] = _packed(held) if across else held
    scales[touched] = now


def _plain_write(s):
    _plain_write_one(s["k"], s["kc"], s["ks"], s["slots"], s["page"], False)
    _plain_write_one(s["v"], s["vc"], s["vs"], s["slots"], s["page"], True)
    return dict(kc=s["kc"], ks=s["ks"], vc=s["vc"], vs=s["vs"])


def _plain_attention(s):
    q, kv_lens, cu = s["q"], s["kv_lens"].long(), s["cu"].long()
    tokens, heads, dk = q.shape
    hkv, longest = s["kc"].shape[1], s["max_new"]
    n, group = kv_lens.numel(), heads // hkv
    page = s["page"]
    cols = (s["max_kv"] + page - 1) // page
    table = s["table"][:, :cols].long()
    at = table.clamp(min=0)
    k = s["kc"].view(torch.uint8)[at].view(E4M3).float() * s["ks"][at][..., None, None]
    v = _tokens(s["vc"].view(torch.uint8)[at].view(E4M3).float()) * s["vs"][at][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * page, dk)
    v = v.permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * page, -1)
    lens = cu[1:] - cu[:-1]
    i = torch.arange(longest, device=DEV)
    padded = q.float()[(cu[:-1, None] + i[None, :]).clamp(max=tokens - 1)]
    padded = padded.reshape(n, longest, hkv, group, dk).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * longest, dk)
    x = (padded @ k.transpose(2, 3).contiguous()) * s["scale"]
    j = torch.arange(cols * page, device=DEV)
    sees = j[None, None, :] <= (kv_lens - lens)[:, None, None] + i[None, :, None]
    sees = (sees & (j[None, None, :] < kv_lens[:, None, None]))[:, None, None]
    x = torch.where(sees, x.view(n, hkv, group, longest, -1), float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    total = x.sum(-1, keepdim=True)
    x = (x.view(n, hkv, group * longest, -1) @ v).view(n, hkv, group, longest, -1)
    x = torch.where(total > 0, x / total, 0.0)
    t = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return x.permute(0, 3, 1, 2, 4).reshape(n, longest, heads, -1)[seq, t - cu[seq]].to(q.dtype)


def _plain_pool(s):
    q, k, v, g, beta, states, at = s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["slots"].long()
    tokens, hk, dk = q.shape
    heads = v.shape[1]
    n = at.numel()
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=DEV)
    lens = cu[1:] - cu[:-1]
    keep = lens if s["keep"] is None else s["keep"].long()
    q, k, v = q.float(), k.float(), v.float()
    if s["eps"] > 0:
        q, k = (x / torch.sqrt(x.square().sum(-1, keepdim=True) + s["eps"]) for x in (q, k))
    q, k = ((x * f).repeat_interleave(heads // hk, 1) for x, f in ((q, s["q_scale"]), (k, 1.0)))
    alpha = torch.exp(g if g.dim() == 3 else g[:, :, None].expand(-1, -1, dk))
    state, kept = states[at], states[at]
    o = torch.zeros((tokens, heads, v.shape[2]), device=DEV)
    for i in range(s["longest"]):  # the recurrence itself
        live = i < lens
        t = (cu[:-1] + i).clamp(max=tokens - 1)
        decayed = state * alpha[t][..., None]
        u = beta[t][..., None] * (v[t] - (decayed * k[t][..., None]).sum(2))
        state = torch.where(live[:, None, None, None], decayed + k[t][..., None] * u[:, :, None, :], state)
        kept = torch.where((i < keep)[:, None, None, None], state, kept)
        out = (state * q[t][..., None]).sum(2)
        o[t[live]] = out[live]
    states[at] = kept
    return dict(o=o.to(s["q"].dtype), states=states)


# ---------------------------------------------------------------- one pass


def run(state):
    s = state
    if own:
        import gated_delta_rule_linear_amd as gdn

        if s["op"] == "tables":
            cu, kv_lens, slots, positions = gdn.gdn_batch_tables(s["ctx"], s["new"], s["tokens"], s["page"], s["table"],
                                                                 s["counts"], s["free"], s["ring"], rows=s["rows"])
            return dict(cu=cu, kv_lens=kv_lens, slots=slots, positions=positions, table=s["table"], counts=s["counts"],
                        free=s["free"], ring=s["ring"])
        if s["op"] == "write":
            gdn.gdn_cache_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
            return dict(kc=s["kc"], ks=s["ks"], vc=s["vc"], vs=s["vs"])
        if s["op"] == "attention":
            return gdn.gdn_cache_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["kv_lens"],
                                           s["cu"], scale=s["scale"], max_new=s["max_new"], max_kv=s["max_kv"])
        o = gdn.gdn_decode_pool(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["slots"], cu_seqlens=s["cu"],
                                commit=s["keep"], q_scale=s["q_scale"], l2_eps=s["eps"])
        return dict(o=o, states=s["states"])
    return {"tables": _plain_tables, "write": _plain_write, "attention": _plain_attention, "pool": _plain_pool}[s["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, n = case["op"], case["n"]
    ctx, new = _requests(case)
    ended, new = new < 0, new.clamp(min=0)
    tokens = int(new.sum())
    if op == "tables":
        # lengths, rows, counts, ring in; offsets, lengths, counts and two values for each token out; a page that a
        # request gets or gives back is read in one place and written in another
        held = (ctx + case["page"] - 1) // case["page"]
        pages = int(((ctx + new + case["page"] - 1) // case["page"] - held).sum() + held[ended].sum())
        return dict(bytes=4 * (7 * n + 2 * tokens + 2 * pages + 7), flops=0)
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "write":
        d = case["hkv"] * (case["dk"] + case["dv"])
        return dict(bytes=tokens * d * (size + 1) + 4 * tokens, flops=3 * tokens * d)
    if op == "attention":
        d = case["dk"] + case["dv"]
        pairs = int((new * ctx + new * (new + 1) // 2).sum())
        held = int((ctx + new)[new > 0].sum())
        return dict(bytes=held * case["hkv"] * d + tokens * case["heads"] * d * size, flops=2 * pairs * case["heads"] * d)
    h, dk, dv = case["heads"], case["dk"], case["dv"]
    token = size * (2 * case["hk"] * dk + 2 * h * dv) + 4 * h * (1 + (1 if case["head_gate"] else dk))
    return dict(bytes=8 * int((new > 0).sum()) * h * dk * dv + tokens * token, flops=7 * tokens * h * dk * dv)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_write_one(x, cache, scales, slots, page, across):
    codes = cache.double().cpu()
    codes = codes.permute(0, 1, 2, 4, 3).flatten(2, 3) if across else codes
    scales, x = scales.double().cpu(), x.double().cpu()
    slots = slots.cpu().tolist()
    runs = {}
    for t, s in enumerate(slots):
        runs.setdefault(s // page, []).append(t)
    for p, ts in runs.items():
        a = slots[ts[0]] % page
        part = x[ts]
        amax = part.abs().amax(-1).amax(0)
        need = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(min=MIN_EXPONENT))
        if a == 0:
            codes[p] = 0
            now = need
        else:
            now = torch.maximum(need, scales[p])
            codes[p] = _nearest(codes[p] * (scales[p] / now)[:, None, None])
        codes[p, :, a:a + len(ts)] = _nearest(part / now[None, :, None]).transpose(0, 1)
        scales[p] = now
    return codes.unflatten(2, (-1, 16)).permute(0, 1, 2, 4, 3).contiguous() if across else codes, scales


def _nearest(x):
    """x to the nearest value with three bits behind the leading one, exponents -6 to 8, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return torch.round(x / unit) * unit


def exact(case, seed):
    op = case["op"]
    if op == "tables" or (op == "write" and case["n"] * case["hi"] > 20000):
        return None
    s = prepare(case, seed)
    if op == "write":
        kc, ks = _exact_write_one(s["k"], s["kc"], s["ks"], s["slots"], s["page"], False)
        vc, vs = _exact_write_one(s["v"], s["vc"], s["vs"], s["slots"], s["page"], True)
        return dict(kc=kc, ks=ks, vc=vc, vs=vs)
    if op == "attention":
        cu, kv_lens, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
        tokens, heads, dk = s["q"].shape
        hkv, page, dv = s["kc"].shape[1], s["page"], s["vc"].shape[3]
        o = torch.zeros((tokens, heads, dv), dtype=torch.float64, device=DEV)
        for n, length in enumerate(kv_lens):
            a, b = cu[n], cu[n + 1]
            if b == a:
                continue
            pages = table[n][:-(-length // page)]
            for h in range(hkv):
                keys = torch.cat([s["kc"][p, h].double() * s["ks"][p, h].double() for p in pages])[:length]
                values = torch.cat([s["vc"][p, h].double().permute(0, 2, 1).flatten(0, 1) * s["vs"][p, h].double()
                                    for p in pages])[:length]
                for head in range(h * (heads // hkv), (h + 1) * (heads // hkv)):
                    x = s["q"][a:b, head].double() @ keys.T * s["scale"]
                    future = torch.triu(torch.ones_like(x, dtype=torch.bool), diagonal=length - (b - a) + 1)
                    o[a:b, head] = torch.softmax(x.masked_fill(future, float("-inf")), -1) @ values
        return o
    q, k, v, g, beta, states = (s[x].double() for x in ("q", "k", "v", "g", "beta", "states"))
    tokens, hk, dk = q.shape
    heads, n = v.shape[1], s["slots"].numel()
    at = s["slots"].long()
    starts = list(range(n + 1)) if s["cu"] is None else s["cu"].tolist()
    lens = [b - a for a, b in zip(starts, starts[1:])]
    kept = lens if s["keep"] is None else s["keep"].tolist()
    if s["eps"] > 0:
        q = q / (q.pow(2).sum(-1, keepdim=True) + s["eps"]).pow(0.5)
        k = k / (k.pow(2).sum(-1, keepdim=True) + s["eps"]).pow(0.5)
    share = torch.arange(heads, device=DEV) // (heads // hk)
    o = torch.zeros((tokens, heads, v.shape[2]), dtype=torch.float64, device=DEV)
    state = states[at]
    for i in range(max(lens)):
        who = torch.tensor([m for m in range(n) if lens[m] > i], device=DEV)
        t = torch.tensor([starts[m] + i for m in range(n) if lens[m] > i], device=DEV)
        S = state[who]
        S = S * (torch.exp(g[t])[..., None] if g.dim() == 3 else torch.exp(g[t])[..., None, None])
        key, query = k[t][:, share], q[t][:, share] * s["q_scale"]
        u = (v[t] - torch.matmul(key[:, :, None, :], S)[:, :, 0]) * beta[t][..., None]
        S = S + key[..., None] * u[:, :, None, :]
        o[t] = torch.matmul(query[:, :, None, :], S)[:, :, 0]
        state[who] = S
        save = torch.tensor([j for j, m in enumerate(who.tolist()) if kept[m] == i + 1], dtype=torch.long, device=DEV)
        states[at[who[save]]] = S[save]
    return dict(o=o, states=states)
