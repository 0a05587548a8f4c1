"""Operators around the gated delta-rule layer, trained and served, as they are timed and checked.

  norm        queries and keys normalised for each head and rotated by their
              positions, as gdn_prefill, gdn_cache_write and the cache attention
              take them (gdn_qk_norm)
  norm_back   its gradients, behind gdn_prefill_backward (gdn_qk_norm_backward)
  scan        the gated linear recurrence h_t = e^g_t h_{t-1} + x_t of every
              channel over packed sequences (gdn_scan)
  scan_train  the recurrence and its gradients (gdn_scan, gdn_scan_backward)
  scan_pool   the recurrence on a pool of states, one or a few tokens for each
              request (gdn_scan_pool)
  prefix      attention over the paged 8-bit cache for requests that share the
              pages of a long beginning (gdn_cache_attention_prefix)

run() computes a case in plain torch operations, or, with `own`, through the
library.
"""

import math
import zlib

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of 64 requests in front of exact attention, at far positions: latency
        dict(name="norm_decode_64", op="norm", n=64, lo=1, hi=1, max_ctx=65536, heads=32, hk=8, d=128, kind="rms",
             weights=True, rotary=128, interleaved=False, fused=True, dtype="bf16"),
        # what gdn_prefill takes of a prompt of 65536 tokens: unit vectors, sliced from the projection's output
        dict(name="norm_prompt_64k", op="norm", n=1, lo=65536, hi=65536, max_ctx=0, heads=32, hk=32, d=128, kind="l2",
             weights=False, rotary=0, interleaved=False, fused=True, dtype="bf16"),
        # a training step on four sequences of 8192 tokens, shared key heads
        dict(name="norm_back_8k", op="norm_back", n=4, lo=8192, hi=8192, max_ctx=0, heads=32, hk=8, d=128, kind="rms",
             weights=True, rotary=128, interleaved=False, fused=True, dtype="bf16"),
        # full precision, odd lengths, half of the channels rotated as neighbouring pairs
        dict(name="norm_back_f32", op="norm_back", n=7, lo=0, hi=1021, max_ctx=4097, heads=12, hk=4, d=64, kind="rms",
             weights=True, rotary=32, interleaved=True, fused=False, dtype="f32"),
        # one prompt of 65536 tokens, as wide as 32 heads of 128
        dict(name="scan_prompt_64k", op="scan", n=1, lo=65536, hi=65536, channels=4096, mix=False, init=False,
             dtype="bf16"),
        # chunks of prompts, of 8 requests and of very different lengths, that go on from states, full precision
        dict(name="scan_chunks_f32", op="scan", n=8, lo=1, hi=2047, channels=1028, mix=True, init=True, dtype="f32"),
        # a training step on four sequences of 8192 tokens
        dict(name="scan_train_8k", op="scan_train", n=4, lo=8192, hi=8192, channels=4096, mix=True, init=False,
             dtype="bf16"),
        # packed short sequences, some without a token, full precision, states at both ends
        dict(name="scan_train_f32", op="scan_train", n=23, lo=0, hi=509, channels=516, mix=False, init=True,
             dtype="f32"),
        # decode of 512 requests
        dict(name="scan_pool_512", op="scan_pool", n=512, lo=1, hi=1, spare=64, channels=4096, mix=False, dtype="bf16"),
        # drafted tokens of 45 requests being verified, full precision
        dict(name="scan_pool_f32", op="scan_pool", n=45, lo=1, hi=7, spare=3, channels=1536, mix=True, dtype="f32"),
        # decode of 64 requests behind a common beginning of 16384 tokens
        dict(name="prefix_decode_64", op="prefix", groups=1, each=64, prefix_lo=16384, prefix_hi=16384, own_hi=1023, lo=1,
             hi=1, heads=32, hkv=8, dk=128, dv=128, page=64, dtype="bf16"),
        # drafted tokens of four groups of 6 requests, full precision, odd lengths, one group without a common page
        dict(name="prefix_verify_f32", op="prefix", groups=4, each=6, prefix_lo=0, prefix_hi=4224, own_hi=517, lo=1, hi=5,
             heads=12, hkv=4, dk=64, dv=64, page=128, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "scan", "scan_train", "scan_pool", "prefix", "prefix"])
    dtype = "bf16" if rng.random() < 0.6 else "f32"
    if op in ("norm", "norm_back"):
        d = rng.choice([64, 128])
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        n = _log(rng, 1, 512)
        return dict(op=op, n=n, lo=rng.randint(0, 1), hi=max(1, _log(rng, 1, 16384) // n), max_ctx=_log(rng, 1, 1 << 20),
                    heads=hk * rng.choice([1, 2, 3, 4]), hk=hk, d=d, kind=rng.choice(["l2", "rms", "rms", "none"]),
                    weights=rng.random() < 0.6, rotary=rng.choice([0, 16, d // 2, d, d]), interleaved=rng.random() < 0.4,
                    fused=rng.random() < 0.6, dtype=dtype)
    if op in ("scan", "scan_train"):
        n = _log(rng, 1, 128)
        return dict(op=op, n=n, lo=rng.randint(0, 1), hi=max(2, _log(rng, 2, 16384) // n), channels=4 * _log(rng, 1, 1024),
                    mix=rng.random() < 0.5, init=rng.random() < 0.5, dtype=dtype)
    if op == "scan_pool":
        return dict(op=op, n=_log(rng, 1, 512), lo=rng.randint(0, 1), hi=rng.randint(1, 8), spare=rng.randint(0, 9),
                    channels=4 * _log(rng, 1, 1024), mix=rng.random() < 0.5, dtype=dtype)
    hkv = rng.choice([1, 2, 4, 8])
    groups = _log(rng, 1, 8)
    return dict(op=op, groups=groups, each=max(1, _log(rng, 1, 64) // groups), prefix_lo=0,
                prefix_hi=_log(rng, 3, 16384 // groups), own_hi=_log(rng, 1, 1024), lo=rng.randint(0, 1),
                hi=rng.choice([1, 1, 2, 5, 8, 33]), heads=hkv * rng.choice([1, 2, 3, 4, 7, 8]), hkv=hkv,
                dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), page=rng.choice([64, 128, 256]), dtype=dtype)


# ---------------------------------------------------------------- inputs


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _between(gen, lo, hi, n):
    """n numbers from lo to hi, one of them hi.  Sizes come from the case alone, so that all its inputs are of one size."""
    x = torch.randint(lo, hi + 1, (n,), generator=gen)
    x[int(torch.randint(0, n, (1,), generator=gen))] = hi
    return x


def _sizes(case):
    """New tokens of each request; with a common beginning also the tokens that each group shares (whole pages) and those
    that each request holds of its own before the step."""
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    gen = torch.Generator().manual_seed(zlib.crc32(text.encode()))
    if case["op"] != "prefix":
        return _between(gen, case["lo"], case["hi"], case["n"])
    n, page = case["groups"] * case["each"], case["page"]
    new = _between(gen, case["lo"], case["hi"], n)
    shared = _between(gen, case["prefix_lo"], case["prefix_hi"], case["groups"]) // page * page
    return new, shared, _between(gen, 0, case["own_hi"], n)


def _offsets(lens):
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(lens, 0).to(torch.int32)
    return cu


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator().manual_seed(seed * 7919 + 13)
    dev = torch.Generator(device=DEV).manual_seed(seed * 104729 + 7)

    def randn(*shape):
        return torch.randn(shape, generator=dev, device=DEV)

    t = _type(case)
    new, shared, held = _sizes(case) if op == "prefix" else (_sizes(case), None, None)
    tokens, cu = int(new.sum()), _offsets(new)
    if op in ("norm", "norm_back"):
        heads, hk, d = case["heads"], case["hk"], case["d"]
        # a projection's output: channels of different sizes; in one tensor with the values, or of its own
        width = 0.3 * torch.exp(0.5 * randn(heads + 2 * hk, d))
        x = torch.empty((tokens, heads + 2 * hk, d), dtype=t, device=DEV)
        for a in range(0, tokens, 16384):  # in parts: the normal values take twice the room
            x[a:a + 16384] = randn(min(16384, tokens - a), heads + 2 * hk, d) * width
        q, k = x[:, :heads], x[:, heads:heads + hk]
        if not case["fused"]:
            q, k = q.contiguous(), k.contiguous()
        ctx = torch.randint(0, case["max_ctx"] + 1, (case["n"],), generator=gen)
        seq = torch.repeat_interleave(torch.arange(case["n"]), new)
        positions = torch.arange(tokens) - cu[:-1].long()[seq] + ctx[seq]
        r = case["rotary"]
        f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r) if r else None
        s = dict(op=op, q=q, k=k, kind=case["kind"], eps=1e-6, scale=d ** -0.5, interleaved=case["interleaved"],
                 positions=positions.to(torch.int32).to(DEV) if r else None, freq=f.float().to(DEV) if r else None,
                 wq=1 + 0.2 * randn(d) if case["weights"] else None, wk=1 + 0.2 * randn(d) if case["weights"] else None)
        if op == "norm_back":
            s.update(gq=randn(tokens, heads, d).to(t), gk=randn(tokens, hk, d).to(t))
        return s
    if op in ("scan", "scan_train", "scan_pool"):
        n, c = case["n"], case["channels"]
        # decays by channel and token, down to a quarter a token; the slowest channels look back over some 1000 tokens
        g = torch.log(0.75 + 0.25 * torch.sigmoid(1 + randn(tokens, c) + 1.5 * randn(c)))
        s = dict(op=op, x=randn(tokens, c).to(t), g=g, mix=case["mix"], cu=cu.to(DEV), longest=int(new.max()))
        if op == "scan_pool":
            slots = torch.randperm(n + case["spare"], generator=gen)[:n]
            # of drafted tokens some are already known to be kept, the others are only tried
            keep = (torch.rand(n, generator=gen) * (new + 1)).long().clamp(max=new) if case["hi"] > 1 else None
            single = case["lo"] == case["hi"] == 1
            s.update(states=randn(n + case["spare"], c), slots=slots.to(torch.int32).to(DEV),
                     keep=None if keep is None else keep.to(torch.int32).to(DEV), cu=None if single else s["cu"])
            return s
        s["init"] = randn(n, c) if case["init"] else None
        if op == "scan_train":
            s.update(gh=randn(tokens, c).to(t), gf=randn(n, c) if case["init"] else None)
        return s
    groups, each, page, hkv = case["groups"], case["each"], case["page"], case["hkv"]
    total = shared.repeat_interleave(each) + held + new
    # pages in random order; those of a group's beginning stand in the rows of all its requests
    common, blocks = shared // page, (total + page - 1) // page
    first = common.repeat_interleave(each)
    used = int(common.sum() + (blocks - first).sum())
    pages = used + 2
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    cols = max(1, int(blocks.max()))
    at = torch.arange(cols)[None, :]
    table = torch.full((groups * each, cols), -1, dtype=torch.int32)
    rows = torch.full((groups, cols), -1, dtype=torch.int32)
    rows[at < common[:, None]] = order[:int(common.sum())]
    table[:] = rows.repeat_interleave(each, 0)
    table[(at >= first[:, None]) & (at < blocks[:, None])] = order[int(common.sum()):used]

    def cache(*inner):
        exps = torch.randint(-7, -4, (pages, hkv), generator=dev, device=DEV)
        codes = (64.0 * randn(pages, hkv, *inner)).clamp(-448, 448).to(E4M3)
        return codes, torch.exp2(exps.float())

    kc, ks = cache(page, case["dk"])
    vc, vs = cache(page // 16, case["dv"], 16)
    return dict(op=op, page=page, kc=kc, ks=ks, vc=vc, vs=vs, table=table.to(DEV), kv_lens=total.to(torch.int32).to(DEV),
                cu=cu.to(DEV), groups=(torch.arange(groups + 1) * each).to(torch.int32).to(DEV),
                shared=shared.to(torch.int32).to(DEV), q=randn(tokens, case["heads"], case["dk"]).to(t),
                scale=case["dk"] ** -0.5, max_new=int(new.max()), max_kv=int(total.max()), max_prefix=int(shared.max()))


# ---------------------------------------------------------------- plain forms


def _factor(x, kind, eps):
    """The norm's factor of x (fp32) for each head."""
    if kind == "none":
        return torch.ones_like(x[..., :1])
    square = x.square()
    return torch.rsqrt((square.sum(-1, keepdim=True) if kind == "l2" else square.mean(-1, keepdim=True)) + eps)


def _turn(x, s, back=False):
    """x rotated by its positions, or back."""
    if s["freq"] is None:
        return x
    angle = (s["positions"].double()[:, None] * s["freq"].double()[None, :])[:, None, :]
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    n = -n if back else n
    r = 2 * s["freq"].numel()
    if s["interleaved"]:
        u, w = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([u * c - w * n, u * n + w * c], -1).flatten(-2)
    else:
        u, w = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([u * c - w * n, u * n + w * c], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_norm(s):
    out = []
    for x, weight, scale in ((s["q"], s["wq"], s["scale"]), (s["k"], s["wk"], 1.0)):
        z = x.float()
        z = z * _factor(z, s["kind"], s["eps"])
        z = z if weight is None else z * weight
        out.append((_turn(z, s) * scale).to(x.dtype))
    return dict(q=out[0], k=out[1])


def _plain_norm_back(s):
    out = {}
    for name, x, weight, scale, grad in (("q", s["q"], s["wq"], s["scale"], s["gq"]), ("k", s["k"], s["wk"], 1.0, s["gk"])):
        z = x.float()
        r = _factor(z, s["kind"], s["eps"])
        unit = z * r
        dz = _turn(grad.float() * scale, s, back=True)
        if weight is not None:
            out["w" + name] = (dz * unit).sum((0, 1))
            dz = dz * weight
        if s["kind"] != "none":
            inner = (dz * unit).sum(-1, keepdim=True)
            dz = r * (dz - unit * (inner if s["kind"] == "l2" else inner / x.shape[-1]))
        out[name] = dz.to(x.dtype)
    return out


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dim 0: twice as many tokens in each step.  Changes a and b."""
    step = 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _starts(s):
    """Sequences that have a token, their first and their last one."""
    cu = s["cu"].long()
    some = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    return some, cu[some], cu[some + 1] - 1


def _plain_states(s):
    """Decays, h (fp32) and final states."""
    x, g = s["x"].float(), s["g"]
    n = s["cu"].numel() - 1
    some, first, last = _starts(s)
    a = torch.exp(g)
    b = -torch.expm1(g) * x if s["mix"] else x.clone()
    init = torch.zeros((n, x.shape[1]), device=DEV) if s["init"] is None else s["init"]
    b[first] += a[first] * init[some]
    cut = a.clone()
    cut[first] = 0
    h = _doubling(cut, b)
    final = init.clone()
    final[some] = h[last]
    return a, h, final, init


def _plain_scan(s):
    _, h, final, _ = _plain_states(s)
    return dict(h=h.to(s["x"].dtype), final=final)


def _plain_scan_train(s):
    a, h, final, init = _plain_states(s)
    x = s["x"]
    some, first, last = _starts(s)
    d_init = torch.zeros_like(init) if s["gf"] is None else s["gf"].clone()
    # the gradient of h_t, which runs the other way
    d = s["gh"].float().clone()
    d[last] += d_init[some]
    after = torch.zeros_like(a)
    after[:-1] = a[1:]
    after[last] = 0
    d = _doubling(after.flip(0), d.flip(0)).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = init[some]
    if s["mix"]:
        before -= x.float()
    dg = a * d * before
    dx = -torch.expm1(s["g"]) * d if s["mix"] else d
    d_init[some] = a[first] * d[first]
    return dict(h=h.to(x.dtype), final=final, dx=dx.to(x.dtype), dg=dg, d_init=d_init)


def _plain_scan_pool(s):
    x, g, states, at = s["x"].float(), s["g"], s["states"], s["slots"].long()
    n = at.numel()
    cu = torch.arange(n + 1, device=DEV) if s["cu"] is None else s["cu"].long()
    lens = cu[1:] - cu[:-1]
    keep = lens if s["keep"] is None else s["keep"].long()
    a = torch.exp(g)
    b = -torch.expm1(g) * x if s["mix"] else x
    state, kept, h = states[at], states[at], torch.zeros_like(x)
    for i in range(s["longest"]):  # the recurrence itself
        live = i < lens
        t = (cu[:-1] + i).clamp(max=max(0, x.shape[0] - 1))
        state = torch.where(live[:, None], a[t] * state + b[t], state)
        kept = torch.where((i < keep)[:, None], state, kept)
        h[t[live]] = state[live]
    states[at] = kept
    return dict(h=h.to(s["x"].dtype), states=states)


def _plain_prefix(s):
    """Every request over all of its tokens."""
    q, kv_lens, cu = s["q"], s["kv_lens"].long(), s["cu"].long()
    tokens, heads, dk = q.shape
    hkv, longest, page = s["kc"].shape[1], s["max_new"], s["page"]
    n, group = kv_lens.numel(), heads // hkv
    cols = (s["max_kv"] + page - 1) // page
    at = s["table"][:, :cols].long().clamp(min=0)
    k = s["kc"].view(torch.uint8)[at].view(E4M3).float() * s["ks"][at][..., None, None]
    v = s["vc"].view(torch.uint8)[at].view(E4M3).float().transpose(-1, -2).flatten(-3, -2) * s["vs"][at][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(n, hkv, dk, cols * page)
    v = v.permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * page, -1)
    lens = cu[1:] - cu[:-1]
    i = torch.arange(longest, device=DEV)
    rows = q.float()[(cu[:-1, None] + i[None, :]).clamp(max=tokens - 1)]
    rows = rows.reshape(n, longest, hkv, group, dk).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * longest, dk)
    x = (rows @ k) * s["scale"]
    j = torch.arange(cols * page, device=DEV)
    sees = j[None, None, :] <= (kv_lens - lens)[:, None, None] + i[None, :, None]
    x = torch.where(sees[:, None, None], x.view(n, hkv, group, longest, -1), float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    x = (x.view(n, hkv, group * longest, -1) @ v).view(n, hkv, group, longest, -1) / total
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), lens, output_size=tokens)
    return x.permute(0, 3, 1, 2, 4).reshape(n, longest, heads, -1)[seq, torch.arange(tokens, device=DEV) - cu[seq]].to(q.dtype)


# ---------------------------------------------------------------- one pass


def run(state):
    s = state
    if own:
        import gated_delta_rule_linear_amd as gdn

        kinds = dict(none=gdn.GDN_NORM_NONE, l2=gdn.GDN_NORM_L2, rms=gdn.GDN_NORM_RMS)
        if s["op"] == "norm":
            q, k = gdn.gdn_qk_norm(s["q"], s["k"], norm=kinds[s["kind"]], eps=s["eps"], q_weight=s["wq"], k_weight=s["wk"],
                                   positions=s["positions"], inv_freq=s["freq"], interleaved=s["interleaved"],
                                   q_scale=s["scale"])
            return dict(q=q, k=k)
        if s["op"] == "norm_back":
            dq, dk, dwq, dwk = gdn.gdn_qk_norm_backward(s["q"], s["k"], s["gq"], s["gk"], norm=kinds[s["kind"]],
                                                        eps=s["eps"], q_weight=s["wq"], k_weight=s["wk"],
                                                        positions=s["positions"], inv_freq=s["freq"],
                                                        interleaved=s["interleaved"], q_scale=s["scale"])
            return dict(q=dq, k=dk) if dwq is None else dict(wq=dwq, q=dq, wk=dwk, k=dk)
        mix = dict(mix=s["mix"]) if "mix" in s else {}
        if s["op"] == "scan":
            h, final = gdn.gdn_scan(s["x"], s["g"], s["cu"], initial_state=s["init"], **mix)
            return dict(h=h, final=final)
        if s["op"] == "scan_train":
            kept = gdn.gdn_scan_checkpoints(s["x"])
            h, final = gdn.gdn_scan(s["x"], s["g"], s["cu"], initial_state=s["init"], checkpoints=kept, **mix)
            dx, dg, d_init = gdn.gdn_scan_backward(s["x"], s["g"], s["cu"], s["gh"], initial_state=s["init"],
                                                   d_final_state=s["gf"], checkpoints=kept, **mix)
            return dict(h=h, final=final, dx=dx, dg=dg, d_init=d_init)
        if s["op"] == "scan_pool":
            h = gdn.gdn_scan_pool(s["x"], s["g"], s["states"], s["slots"], cu_seqlens=s["cu"], commit=s["keep"], **mix)
            return dict(h=h, states=s["states"])
        return gdn.gdn_cache_attention_prefix(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["kv_lens"],
                                              s["cu"], s["groups"], s["shared"], scale=s["scale"], max_new=s["max_new"],
                                              max_kv=s["max_kv"], max_prefix=s["max_prefix"])
    return dict(norm=_plain_norm, norm_back=_plain_norm_back, scan=_plain_scan, scan_train=_plain_scan_train,
                scan_pool=_plain_scan_pool, prefix=_plain_prefix)[s["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    new, shared, held = _sizes(case) if op == "prefix" else (_sizes(case), None, None)
    tokens, size = int(new.sum()), 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_back"):
        x = tokens * (case["heads"] + case["hk"]) * case["d"]
        small = 4 * (tokens if case["rotary"] else 0) + 2 * case["rotary"] + 8 * case["d"] * case["weights"]
        if op == "norm":
            return dict(bytes=2 * size * x + small, flops=6 * x)
        return dict(bytes=3 * size * x + small + 8 * case["d"] * case["weights"], flops=14 * x)
    if op in ("scan", "scan_train", "scan_pool"):
        c, n = case["channels"], case["n"]
        x = tokens * c
        if op == "scan":
            return dict(bytes=x * (4 + 2 * size) + 4 * n * c * (1 + case["init"]), flops=3 * x)
        if op == "scan_train":
            # g, x and the gradient of h are read once, h and two gradients written
            return dict(bytes=x * (8 + 4 * size) + 4 * n * c * (2 + 2 * case["init"]), flops=9 * x)
        return dict(bytes=x * (4 + 2 * size) + 8 * int((new > 0).sum()) * c, flops=3 * x)
    each, d = case["each"], case["dk"] + case["dv"]
    own_tokens = (held + new)[new > 0]
    some = (new.view(-1, each) > 0).any(1)
    ctx = shared.repeat_interleave(each) + held
    pairs = int((new * ctx + new * (new + 1) // 2).sum())
    return dict(bytes=int(shared[some].sum() + own_tokens.sum()) * case["hkv"] * d + tokens * case["heads"] * d * size,
                flops=2 * pairs * case["heads"] * d)


# ---------------------------------------------------------------- the definitions in 64 bits


def _matrices(s, d):
    """The rotation of each token as cosines and sines, and the partner and sign of every channel."""
    r = 0 if s["freq"] is None else 2 * s["freq"].numel()
    ch = torch.arange(d, device=DEV)
    half = r // 2
    if s["interleaved"]:
        pair, low, partner = ch // 2, ch % 2 == 0, torch.where(ch % 2 == 0, ch + 1, ch - 1)
    else:
        pair, low, partner = ch % max(half, 1), ch < half, torch.where(ch < half, ch + half, ch - half)
    on = ch < r
    pair, partner = torch.where(on, pair, 0), torch.where(on, partner, ch)
    if r == 0:
        return torch.ones((1, d), dtype=torch.float64, device=DEV), torch.zeros((1, d), dtype=torch.float64, device=DEV), partner
    angle = s["positions"].double()[:, None] * s["freq"].double()[pair][None, :]
    c = torch.where(on, torch.cos(angle), 1.0)
    n = torch.where(on, torch.sin(angle) * torch.where(low, -1.0, 1.0), 0.0)
    return c, n, partner


def _exact_norm(s, back):
    out = {}
    for name, weight, scale in (("q", s["wq"], s["scale"]), ("k", s["wk"], 1.0)):
        x = s[name]
        heads, d = x.shape[1:]
        c, n, partner = _matrices(s, d)
        w = torch.ones(d, dtype=torch.float64, device=DEV) if weight is None else weight.double()
        y, dw = torch.empty(x.shape, dtype=torch.float64, device=DEV), torch.zeros(d, dtype=torch.float64, device=DEV)
        for h in range(heads):
            z = x[:, h].double()
            norm = z.pow(2).sum(-1, keepdim=True) / (1 if s["kind"] == "l2" else d) + s["eps"]
            r = torch.ones_like(norm) if s["kind"] == "none" else norm.pow(-0.5)
            if not back:
                z = z * r * w
                y[:, h] = scale * (c * z + n * z[:, partner])
                continue
            g = scale * s["g" + name][:, h].double()
            g = c * g + (n * g)[:, partner]  # the transposed rotation
            dw += (g * z * r).sum(0)
            g = g * w
            if s["kind"] != "none":
                g = r * g - r.pow(3) * z * (g * z).sum(-1, keepdim=True) / (1 if s["kind"] == "l2" else d)
            y[:, h] = g
        if back and weight is not None:
            out["w" + name] = dw
        out[name] = y
    return out


def _exact_scan(s, train):
    x, g, cu = s["x"].double(), s["g"].double(), s["cu"].tolist()
    n, c = len(cu) - 1, x.shape[1]
    a = torch.exp(g)
    b = (1 - a) * x if s["mix"] else x
    final = torch.zeros((n, c), dtype=torch.float64, device=DEV) if s["init"] is None else s["init"].double().clone()
    h, before = torch.empty_like(x), torch.empty_like(x) if train else None
    for m in range(n):
        state = final[m]
        for t in range(cu[m], cu[m + 1]):
            if train:
                before[t] = state
            state = torch.addcmul(b[t], a[t], state)
            h[t] = state
        final[m] = state
    out = dict(h=h, final=final)
    if not train:
        return out
    d_init = torch.zeros((n, c), dtype=torch.float64, device=DEV) if s["gf"] is None else s["gf"].double().clone()
    d = s["gh"].double()
    for m in range(n):
        for t in reversed(range(cu[m], cu[m + 1])):
            d[t] += d_init[m]
            d_init[m] = a[t] * d[t]
    out.update(dx=d * (1 - a) if s["mix"] else d, dg=d * a * (before - x if s["mix"] else before), d_init=d_init)
    return out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("norm", "norm_back"):
        return _exact_norm(s, op == "norm_back")
    if op in ("scan", "scan_train"):
        return _exact_scan(s, op == "scan_train")
    if op == "scan_pool":
        x, g, states, n = s["x"].double(), s["g"].double(), s["states"].double(), s["slots"].numel()
        starts = list(range(n + 1)) if s["cu"] is None else s["cu"].tolist()
        kept = [starts[m + 1] - starts[m] for m in range(n)] if s["keep"] is None else s["keep"].tolist()
        h = torch.empty_like(x)
        for m, slot in enumerate(s["slots"].tolist()):
            state = states[slot].clone()
            for i, t in enumerate(range(starts[m], starts[m + 1])):
                a = torch.exp(g[t])
                state = a * state + ((1 - a) * x[t] if s["mix"] else x[t])
                h[t] = state
                if i + 1 == kept[m]:
                    states[slot] = state
        return dict(h=h, states=states)
    cu, kv_lens, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["table"].long()
    tokens, heads, _ = s["q"].shape
    hkv, page, dv = s["kc"].shape[1], s["page"], s["vc"].shape[3]
    o = torch.zeros((tokens, heads, dv), dtype=torch.float64, device=DEV)
    for n, length in enumerate(kv_lens):
        a, b = cu[n], cu[n + 1]
        if b == a:
            continue
        at = table[n, :-(-length // page)]
        keys = s["kc"].view(torch.uint8)[at].view(E4M3).double() * s["ks"][at].double()[:, :, None, None]
        values = s["vc"].view(torch.uint8)[at].view(E4M3).double() * s["vs"][at].double()[:, :, None, None, None]
        keys = keys.transpose(0, 1).flatten(1, 2)[:, :length]
        values = values.permute(1, 0, 2, 4, 3).flatten(1, 3)[:, :length]
        future = torch.triu(torch.ones((b - a, length), dtype=torch.bool, device=DEV), diagonal=length - (b - a) + 1)
        for head in range(heads):
            h = head // (heads // hkv)
            x = s["q"][a:b, head].double() @ keys[h].T * s["scale"]
            o[a:b, head] = torch.softmax(x.masked_fill(future, float("-inf")), -1) @ values[h]
    return o
