"""GPU parity of the calls of include/gdn_stack.h with plain 64-bit forms (tests/stack_reference.py): queries and keys
normalised and rotated, the gated linear recurrence, and their gradients; the calls together with the layer's."""

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_linear_amd as gdn
import serve_reference as serve
import stack_reference as ref
from helpers import TOL, log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return None if t is None else t.detach().cpu().double()


def close(name, got, want, bound, dtype):
    """Within the bound of the arithmetic and half a step of the output's type of everything (of what is below the type's
    normal numbers, of the smallest of them)."""
    got, want, bound = f64(got), f64(want), bound.double()
    tiny = torch.finfo(dtype).tiny
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{name}: not finite elsewhere"
    limit = bound + ref.half_step(dtype) * (want.abs() + bound) + ref.half_step(dtype) * tiny
    fine = torch.isfinite(want)
    over = ((got - want).abs() / limit)[fine]
    worst = float(over.max()) if over.numel() else 0.0
    log(f"  {name}: {worst:.3f} of the bound")
    assert worst <= 1.0, f"{name}: {worst:.3f} times the bound"


# ---------------------------------------------------------------- norm and rotation


def norm_case(T, H, hk, d, norm, weights, rotary, interleaved, dtype, strided, seed, far=100000):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    wide = (r(T, H + 2 * hk, d) * torch.exp(r(H + 2 * hk, 1))).to(dtype).cuda()
    q, k = wide[:, :H], wide[:, H:H + hk]
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(-far, far, (T,), generator=gen).to(torch.int32)
    freq = (10000.0 ** (-torch.arange(0, rotary, 2).double() / max(rotary, 1))).float()
    return dict(q=q, k=k if hk else None, norm=norm, eps=1e-5, q_weight=(1 + 0.3 * r(d)).cuda() if weights else None,
                k_weight=(1 + 0.3 * r(d)).cuda() if weights else None, positions=pos.cuda() if rotary else None,
                inv_freq=freq.cuda() if rotary else None, interleaved=interleaved, q_scale=0.37)


def norm_reference(a, kind):
    return (f64(a[kind]), a["norm"], a["eps"], f64(a[kind + "_weight"]),
            None if a["positions"] is None else a["positions"].cpu(), f64(a["inv_freq"]), a["interleaved"],
            a["q_scale"] if kind == "q" else 1.0)


NORMS = [(1, 1, 1, 64, 2, True, 64, False, True), (1, 32, 8, 128, 2, True, 128, False, True),
         (3, 4, 2, 128, 1, False, 0, False, False), (7, 5, 3, 64, 0, True, 32, True, True),
         (129, 12, 4, 64, 2, True, 32, True, False), (65, 3, 1, 128, 2, False, 64, False, True),
         (500, 9, 9, 128, 1, False, 128, True, True), (33, 40, 0, 64, 2, True, 8, False, False),
         (33, 17, 2, 128, 0, False, 16, False, True), (2, 70, 33, 128, 2, True, 120, False, True),
         (9001, 2, 1, 64, 2, True, 64, False, True), (12, 6, 6, 64, 2, True, 56, True, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", NORMS)
def test_norm(case, dtype):
    log(f"norm {case} {dtype}")
    a = norm_case(*case[:-1], dtype, case[-1], seed=sum(map(int, case)))
    q, k = gdn.gdn_qk_norm(**a)
    for kind, got in (("q", q), ("k", k)):
        if a[kind] is None:
            assert got is None
            continue
        want, bound = ref.qk_norm(*norm_reference(a, kind)[:1], *norm_reference(a, kind)[1:])
        close(kind, got, want, bound, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", NORMS)
def test_norm_backward(case, dtype):
    log(f"norm backward {case} {dtype}")
    a = norm_case(*case[:-1], dtype, case[-1], seed=sum(map(int, case)))
    gen = torch.Generator().manual_seed(99)
    g = {s: None if a[s] is None else torch.randn(a[s].shape, generator=gen).to(dtype).cuda() for s in "qk"}
    need = gdn.gdn_qk_norm_backward_workspace_bytes(case[0], case[1], case[2], case[3])
    space = torch.full((need // 4,), float("nan"), device="cuda")  # what a workspace held before does not matter
    rest = {s: v for s, v in a.items() if s not in "qk"}
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_backward(a["q"], a["k"], g["q"], g["k"], workspace=space, **rest)
    for kind, got, dw in (("q", dq, dwq), ("k", dk, dwk)):
        if a[kind] is None:
            continue
        x, *more = norm_reference(a, kind)
        want, bound, weight, weight_bound = ref.qk_norm_backward(x, f64(g[kind]), *more)
        close("d" + kind, got, want, bound, dtype)
        if a[kind + "_weight"] is None:
            assert dw is None
        else:
            close("dw" + kind, dw, weight, weight_bound, F32)


def test_norm_backward_into_slices():
    a = norm_case(77, 6, 2, 64, 2, True, 64, False, BF16, True, seed=5)
    g = [torch.randn(s, device="cuda").to(BF16) for s in ((77, 6, 64), (77, 2, 64))]
    rest = {s: v for s, v in a.items() if s not in "qk"}
    plain = gdn.gdn_qk_norm_backward(a["q"], a["k"], *g, **rest)
    whole = torch.full((77, 10, 64), 3.0, dtype=BF16, device="cuda")
    got = gdn.gdn_qk_norm_backward(a["q"], a["k"], *g, dq=whole[:, :6], dk=whole[:, 6:8], **rest)
    assert torch.equal(whole[:, :6], plain[0]) and torch.equal(whole[:, 6:8], plain[1])
    assert bool((whole[:, 8:] == 3.0).all())
    assert torch.equal(got[2], plain[2]) and torch.equal(got[3], plain[3])
    # in the place of the outputs' gradients, and without the weights'
    over = gdn.gdn_qk_norm_backward(a["q"], a["k"], *g, dq=g[0], dk=g[1], want_d_weights=False, **rest)
    assert torch.equal(g[0], plain[0]) and torch.equal(g[1], plain[1]) and over[2] is None and over[3] is None


def test_norm_in_place():
    a = norm_case(300, 8, 4, 128, 2, True, 128, False, BF16, False, seed=6)
    want = gdn.gdn_qk_norm(**a)
    got = gdn.gdn_qk_norm(**a, q_out=a["q"], k_out=a["k"])
    assert got[0] is a["q"] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,T", [(BF16, 30001), (F32, 15000)])
def test_norm_larger_than_the_caches(dtype, T):
    # (as the first half and the second by themselves, which are not)
    H, hk, d = 32, 8, 128
    x = torch.randn((T, H + hk, d), device="cuda").to(dtype)
    dy = torch.randn((T, H + hk, d), device="cuda").to(dtype)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    kw = dict(norm=gdn.GDN_NORM_RMS, q_weight=torch.rand(d, device="cuda") + 0.5, inv_freq=torch.rand(32, device="cuda"))
    assert T * (H + hk) * d * x.element_size() > 1 << 28
    half = T // 2
    whole = gdn.gdn_qk_norm(x[:, :H], x[:, H:], positions=pos, **kw)
    g = dy[:, :H].contiguous(), dy[:, H:].contiguous()
    back = gdn.gdn_qk_norm_backward(x[:, :H], x[:, H:], *g, positions=pos, **kw)
    for sl in (slice(0, half), slice(half, T)):
        part = gdn.gdn_qk_norm(x[sl, :H], x[sl, H:], positions=pos[sl], **kw)
        assert torch.equal(part[0], whole[0][sl]) and torch.equal(part[1], whole[1][sl])
        part = gdn.gdn_qk_norm_backward(x[sl, :H], x[sl, H:], g[0][sl], g[1][sl], positions=pos[sl], **kw)
        assert torch.equal(part[0], back[0][sl]) and torch.equal(part[1], back[1][sl])


@pytest.mark.parametrize("position", [0, 1, (1 << 20) + 1, (1 << 31) - 1, -(1 << 31)])
def test_norm_far_positions(position):
    a = norm_case(4, 2, 1, 128, 0, False, 128, False, F32, True, seed=7)
    a["positions"] = i32([position] * 4)
    q, _ = gdn.gdn_qk_norm(**a)
    close("q", q, *ref.qk_norm(*norm_reference(a, "q")), F32)


def test_norm_of_nothing_and_of_zeros():
    a = norm_case(0, 4, 2, 64, 2, True, 64, False, BF16, False, seed=8)
    q, k = gdn.gdn_qk_norm(**a)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    rest = {s: v for s, v in a.items() if s not in "qk"}
    out = gdn.gdn_qk_norm_backward(a["q"], a["k"], q, k, **rest)
    assert bool((out[2] == 0).all()) and bool((out[3] == 0).all())
    z = torch.zeros((5, 3, 64), device="cuda")
    for norm in (0, 1, 2):
        assert bool((gdn.gdn_qk_norm(z, norm=norm)[0] == 0).all())
        dq, _, _, _ = gdn.gdn_qk_norm_backward(z, None, z + 1, None, norm=norm, eps=1e-6)
        # r = 1 / sqrt(eps), a thousand, where there is a norm
        close("dq", dq, torch.full((5, 3, 64), 1e3 if norm else 1.0, dtype=torch.float64), torch.full((5, 3, 64), 32e3 * ref.E32), F32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_nan_stays_where_it_is(interleaved):
    a = norm_case(6, 4, 2, 64, 2, True, 32, interleaved, F32, False, seed=9)
    want, _ = gdn.gdn_qk_norm(**a)
    a["q"][2, 1, 5] = math.nan
    a["q"][3, 0, 40] = math.inf
    got, _ = gdn.gdn_qk_norm(**a)
    touched = torch.zeros((6, 4), dtype=torch.bool)
    touched[2, 1] = touched[3, 0] = True
    assert torch.equal(got[~touched.cuda()], want[~touched.cuda()]) and bool(torch.isnan(got[2, 1]).all())
    # without a norm a channel that is not rotated keeps to itself, one that is reaches its partner
    a["norm"] = gdn.GDN_NORM_NONE
    got, _ = gdn.gdn_qk_norm(**a)
    assert int(torch.isinf(got[3, 0]).sum()) == 1 and int(torch.isnan(got[3, 0]).sum()) == 0
    assert int(torch.isnan(got[2, 1]).sum()) == 2


@pytest.mark.parametrize("norm", [gdn.GDN_NORM_L2, gdn.GDN_NORM_RMS])
def test_norm_large_magnitudes(norm):
    # a head normalises as long as its sum of squares is a number of fp32, however large a channel is, and to 0 from there on
    x = torch.zeros((4, 1, 128), device="cuda")
    x[0, 0, 5] = 1.8e19  # 3.24e38
    x[1] = 1.6e18        # 128 times 2.56e36: 3.28e38
    x[2, 0, 5] = 1.9e19  # 3.61e38
    x[3] = 1.7e18        # 3.70e38
    y, _ = gdn.gdn_qk_norm(x, norm=norm, eps=1e-6)
    want, bound = ref.qk_norm(f64(x), norm, 1e-6, None, None, None, False, 1.0)
    close("y", y[:2], want[:2], bound[:2], F32)
    assert bool((y[2:] == 0).all())
    dx, _, _, _ = gdn.gdn_qk_norm_backward(x, None, torch.ones_like(x), None, norm=norm, eps=1e-6)
    assert bool(torch.isfinite(dx).all()) and bool((dx[2:] == 0).all())


# ---------------------------------------------------------------- the recurrence


def scan_case(lens, C, mix, init, dtype, seed, extra=0, slow=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    T, n = sum(lens) + extra, len(lens)
    g = torch.log(0.7 + 0.3 * torch.sigmoid(r(T, C) + 2 * r(C))) if slow else -5 * torch.rand((T, C), generator=gen)
    return dict(x=r(T, C).to(dtype).cuda(), g=g.cuda(), cu_seqlens=i32([0] + list(np.cumsum(lens))), mix=mix,
                initial_state=r(n, C).cuda() if init else None), (r(T, C).to(dtype).cuda(), r(n, C).cuda() if init else None)


def scan_reference(a):
    return f64(a["x"]), f64(a["g"]), a["cu_seqlens"].tolist(), a["mix"], f64(a["initial_state"])


LENS = [[1], [0], [2, 0, 0, 7], [63, 64, 65], [1] * 150, [0] * 130 + [5] + [0] * 90 + [3, 0], [700], [513, 2, 0, 129, 1],
        [8] * 40, [3000], [1, 1023, 64, 0, 0, 960], [16, 112, 128, 256, 1]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("lens,C", [(l, c) for l, c in zip(LENS, [4, 8, 252, 256, 260, 516, 64, 1028, 12, 20, 300, 1024])])
def test_scan(lens, C, mix, dtype):
    init = len(lens) % 2 == 0 or C > 500
    log(f"scan {lens[:6]} x{len(lens)} C={C} mix={mix} init={init} {dtype}")
    a, _ = scan_case(lens, C, mix, init, dtype, seed=len(lens) + C, extra=3 * (C % 8 == 4))
    h = torch.full_like(a["x"], 7.0)
    out, final = gdn.gdn_scan(**a, h=h)
    assert out is h
    want = ref.scan(*scan_reference(a))
    end = sum(lens)
    close("h", h[:end], want["h"][:end], want["bound"][:end], dtype)
    assert bool((h[end:] == 7.0).all())
    close("final", final, want["final"], want["final_bound"], F32)
    for m, length in enumerate(lens):
        if length == 0:
            assert torch.equal(f64(final[m]), want["final"][m])
    again, none = gdn.gdn_scan(**a, output_final_state=False)
    assert none is None and torch.equal(again[:end], h[:end])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("lens,C", [(l, c) for l, c in zip(LENS, [4, 8, 252, 256, 260, 516, 64, 1028, 12, 20, 300, 1024])])
def test_scan_backward(lens, C, mix, dtype):
    init = len(lens) % 2 == 0 or C > 500
    log(f"scan backward {lens[:6]} x{len(lens)} C={C} mix={mix} init={init} {dtype}")
    a, (dh, df) = scan_case(lens, C, mix, init, dtype, seed=len(lens) + C, extra=3 * (C % 8 == 4))
    kept = gdn.gdn_scan_checkpoints(a["x"])
    gdn.gdn_scan(**a, checkpoints=kept)
    space = torch.full((gdn.gdn_scan_backward_workspace_bytes(*a["x"].shape) // 4,), float("nan"), device="cuda")
    outs = [gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df, checkpoints=c, workspace=space) for c in (None, kept)]
    end = sum(lens)
    assert all(torch.equal(x[:end] if i < 2 else x, y[:end] if i < 2 else y) for i, (x, y) in enumerate(zip(*outs)))
    want = ref.scan_backward(*scan_reference(a), f64(dh), f64(df))
    dx, dg, d_init = outs[0]
    close("dx", dx[:end], want["dx"][:end], want["dx_bound"][:end], dtype)
    close("dg", dg[:end], want["dg"][:end], want["dg_bound"][:end], F32)
    close("d_init", d_init, want["d_init"], want["d_init_bound"], F32)
    assert gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df, want_d_initial_state=False)[2] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_fast_decays_and_long(dtype):
    # products of decays far below fp32's smallest number
    for lens, C in (([5000, 37], 8), ([300], 260)):
        a, (dh, df) = scan_case(lens, C, True, True, dtype, seed=3, slow=False)
        h, final = gdn.gdn_scan(**a)
        want = ref.scan(*scan_reference(a))
        close("h", h, want["h"], want["bound"], dtype)
        close("final", final, want["final"], want["final_bound"], F32)
        back = ref.scan_backward(*scan_reference(a), f64(dh), f64(df))
        dx, dg, d_init = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
        close("dx", dx, back["dx"], back["dx_bound"], dtype)
        close("dg", dg, back["dg"], back["dg_bound"], F32)
        close("d_init", d_init, back["d_init"], back["d_init_bound"], F32)


def test_scan_borders_of_the_gate():
    # no decay at all (sums), and decays of 0 (each token by itself)
    T, C = 400, 8
    x = torch.randn((T, C), device="cuda")
    cu = i32([0, T])
    h, _ = gdn.gdn_scan(x, torch.zeros_like(x), cu)
    mags = f64(x).abs().cumsum(0)
    steps = torch.arange(1, T + 1).double()[:, None]
    close("sums", h, f64(x).cumsum(0), steps * 8 * ref.E32 * mags, F32)
    assert bool((gdn.gdn_scan(x, torch.zeros_like(x), cu, mix=True, initial_state=torch.full((1, C), 2.0, device="cuda"))[0] == 2).all())
    g = torch.full_like(x, -math.inf)
    for mix in (False, True):
        h, final = gdn.gdn_scan(x, g, cu, mix=mix)
        assert torch.equal(h, x) and torch.equal(final[0], x[-1])
        dx, dg, d0 = gdn.gdn_scan_backward(x, g, cu, x, mix=mix)
        assert torch.equal(dx, x) and bool((dg == 0).all()) and bool((d0 == 0).all())


def test_scan_nan_and_inf_stay_in_their_sequence():
    lens, C = [100, 70, 0, 300, 9], 12
    for bad in (math.nan, math.inf):
        a, (dh, df) = scan_case(lens, C, False, True, F32, seed=12)
        want, final = gdn.gdn_scan(**a)
        back = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
        a["x"][130, 3] = bad  # sequence 1
        a["initial_state"][3, 5] = bad
        dh[140, 2] = bad
        got, got_final = gdn.gdn_scan(**a)
        off = torch.zeros_like(want, dtype=torch.bool)
        off[130:170, 3] = True
        off[170:470, 5] = True
        assert torch.equal(got[~off], want[~off]) and bool((~torch.isfinite(got[off])).all())
        assert torch.equal(torch.isinf(got[off]), torch.full_like(got[off], bad == math.inf, dtype=torch.bool))
        assert int((~torch.isfinite(got_final)).sum()) == 2 and not math.isfinite(float(got_final[1, 3]))
        dx, dg, d0 = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
        off[:] = False
        off[100:141, 2] = True
        assert torch.equal(dx[~off], back[0][~off]) and bool((~torch.isfinite(dx[off])).all())
        off[131:170, 3] = off[170:470, 5] = True
        assert torch.equal(dg[~off], back[1][~off])
        assert not math.isfinite(float(d0[1, 2])) and int((~torch.isfinite(d0)).sum()) == 1


def same_places(name, got, want, sure=None):
    """Infinities, with their signs, and NaN stand where they stand in `want` (looked at where `sure` says so)."""
    got, want = (f64(t) if sure is None else f64(t)[sure] for t in (got, want))
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), f"{name}: infinite elsewhere"
    assert torch.equal(got[inf], want[inf]), f"{name}: infinite with the other sign"


def scan_places(a, dh, df, dtype, reference):
    """Both calls against the 64-bit form, finite values and others; `reference`: the arguments of the 64-bit form."""
    kept = gdn.gdn_scan_checkpoints(a["x"])
    h, final = gdn.gdn_scan(**a, checkpoints=kept)
    want = ref.scan(*reference)
    back = ref.scan_backward(*reference, f64(dh), f64(df))
    # dg is an infinite gradient times h_{t-1} (- x_t), or an infinite state times a gradient.  A finite factor below its error
    # may be 0 or of the other sign: fp32's h_{t-1} is off by 2^-24 of its magnitude at least, so that with `mix` and behind a
    # decay of e^-20 it is x_{t-1} itself, whose difference to an equal x_t (of bf16, one of some 256) is 0, and 0 Inf is NaN,
    # where 64 bits keep 2e-9 Inf.  (That such a dg is not finite is asked all the same, by close.)
    x = f64(a["x"])
    past = want["before"] - x if a["mix"] else want["before"]
    past_bound = ref.E32 * (want["off"] + (want["big"] + x.abs() if a["mix"] else 0))
    beyond = lambda value, bound: ~torch.isfinite(value) | (value.abs() > bound)
    sure = beyond(past, past_bound) & beyond(back["dx"], back["dx_bound"])
    for c in (kept, None):
        dx, dg, d_init = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df, checkpoints=c)
        for name, got, w in (("h", h, want["h"]), ("final", final, want["final"]), ("dx", dx, back["dx"]), ("d_init", d_init, back["d_init"])):
            same_places(name, got, w)
        same_places("dg", dg, back["dg"], sure)
        close("h", h, want["h"], want["bound"], dtype)
        close("final", final, want["final"], want["final_bound"], F32)
        close("dx", dx, back["dx"], back["dx_bound"], dtype)
        close("dg", dg, back["dg"], back["dg_bound"], F32)
        close("d_init", d_init, back["d_init"], back["d_init_bound"], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [False, True])
def test_scan_infinities_behind_fast_decays(dtype, mix):
    # decays whose product over a wave's tokens, over a tile's or over none leaves fp32's range: an infinite state, or an
    # infinite gradient from behind, stays infinite through all tiles and groups of its sequence
    lens, C = [1500, 0, 300, 450], 260
    a, (dh, df) = scan_case(lens, C, mix, True, dtype, seed=31)
    gen = torch.Generator().manual_seed(32)
    speed = torch.tensor([0.01, 0.3, 0.9, 2.0, 5.0, 20.0, 80.0])[torch.arange(C) % 7]
    a["g"] = (-speed * (0.9 + 0.1 * torch.rand((sum(lens), C), generator=gen))).cuda()
    kind = (torch.arange(C) // 7 % 7).cuda()
    for n, first in ((0, 0), (3, 1800)):
        a["initial_state"][n, kind == 0] = math.inf
        a["x"][first + 40, kind == 1] = -math.inf
        a["initial_state"][n, kind == 2] = -math.inf
        a["x"][first + 200, kind == 2] = math.inf
        df[n, kind == 3] = math.inf
        dh[first + lens[n] - 33, kind == 4] = -math.inf
        a["initial_state"][n, kind == 5] = math.nan
    scan_places(a, dh, df, dtype, scan_reference(a))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("gate", [-math.inf, -1e4])
def test_scan_decays_of_zero(dtype, mix, gate):
    # two tokens with a decay of 0: what is finite ends there, to the last bit, in whatever tile it is looked at, and
    # what is infinite becomes NaN
    T, C = 1300, 260
    a, (dh, df) = scan_case([T], C, mix, True, dtype, seed=33)
    a["g"][100] = a["g"][1111] = gate
    a["initial_state"][0, 0:64] = math.inf
    a["initial_state"][0, 64:128] = 1e30
    a["x"][:, 64:128] = 0
    df[0, 128:192] = -math.inf
    df[0, 192:256] = 1e30
    dh[:, 192:256] = 0
    x, g, cu, mix, init = scan_reference(a)
    scan_places(a, dh, df, dtype, (x, g.clamp(min=-1e4), cu, mix, init))
    h, _ = gdn.gdn_scan(**a)
    dx, _, d_init = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
    assert bool(torch.isinf(h[:100, :64]).all()) and bool(torch.isnan(h[100:, :64]).all()) and bool((h[100:, 64:128] == 0).all())
    assert bool(torch.isnan(dx[:1111, 128:192]).all()) and bool((dx[:1111, 192:256] == 0).all()) and bool((d_init[:, 192:256] == 0).all())


def test_scan_past_32_bits():
    # more than 2^32 elements: a part of the channels is as by itself
    T, C = 1100003, 4096
    x = torch.randn((T, C), device="cuda", dtype=BF16)
    g = torch.empty((T, C), device="cuda").uniform_(-0.3, 0.0)
    cu = i32([0, 700001, T])
    h, final = gdn.gdn_scan(x, g, cu, mix=True)
    for c in (0, C - 8):
        part, last = gdn.gdn_scan(x[:, c:c + 8].contiguous(), g[:, c:c + 8].contiguous(), cu, mix=True)
        assert torch.equal(part, h[:, c:c + 8]) and torch.equal(last, final[:, c:c + 8])
    dx, dg, d0 = gdn.gdn_scan_backward(x, g, cu, h, mix=True)
    for c in (0, C - 8):
        part = gdn.gdn_scan_backward(*(t[:, c:c + 8].contiguous() for t in (x, g)), cu, h[:, c:c + 8].contiguous(), mix=True)
        assert all(torch.equal(p, w[:, c:c + 8]) for p, w in zip(part, (dx, dg, d0)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [False, True])
def test_scan_in_place(dtype, mix):
    a, (dh, df) = scan_case([700, 0, 3, 601, 64], 260, mix, True, dtype, seed=16, extra=5)
    end, x = 1368, a["x"].clone()
    want, final = gdn.gdn_scan(**a)
    back = gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
    h, got = gdn.gdn_scan(**{**a, "x": x}, h=x)
    assert h is x and torch.equal(x[:end], want[:end]) and torch.equal(x[end:], a["x"][end:]) and torch.equal(got, final)
    # dx over d_h, by the library's own entry point
    lib, (T, C) = gdn._load(), a["x"].shape
    dx, dg, d0 = dh.clone(), torch.full_like(a["g"], 7.0), torch.empty_like(df)
    space = torch.empty(gdn.gdn_scan_backward_workspace_bytes(T, C), dtype=torch.uint8, device="cuda")
    st = lib.gdn_scan_backward(a["x"].data_ptr(), a["g"].data_ptr(), a["cu_seqlens"].data_ptr(), 5, T, C, mix,
                               a["initial_state"].data_ptr(), None, dx.data_ptr(), df.data_ptr(), dx.data_ptr(), dg.data_ptr(),
                               d0.data_ptr(), gdn._dtype_code(dx), space.data_ptr(), space.numel(),
                               torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK
    assert torch.equal(dx[:end], back[0][:end]) and torch.equal(dg[:end], back[1][:end]) and torch.equal(d0, back[2])
    assert torch.equal(dx[end:], dh[end:]) and bool((dg[end:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_pool_in_place(dtype):
    a, _ = scan_case([3, 1, 0, 5], 516, True, False, dtype, seed=17)
    cu, slots = a["cu_seqlens"], i32([2, 0, 1, 4])
    pools = [torch.ones((5, 516), device="cuda") for _ in range(2)]
    want = gdn.gdn_scan_pool(a["x"], a["g"], pools[0], slots, cu_seqlens=cu, mix=True)
    got = gdn.gdn_scan_pool(a["x"], a["g"], pools[1], slots, cu_seqlens=cu, mix=True, h=a["x"])
    assert got is a["x"] and torch.equal(got, want) and torch.equal(*pools)


def test_norm_of_one_token_of_an_odd_row():
    # one token: how far the next would be does not matter
    wide = torch.randn((1, 8 * 64 + 3), device="cuda").to(BF16)
    q = wide.as_strided((1, 8, 64), (515, 64, 1))
    assert torch.equal(gdn.gdn_qk_norm(q)[0], gdn.gdn_qk_norm(q.contiguous())[0])


def test_scan_offsets_that_are_none():
    # outputs are then no one's, but nothing outside the arrays is touched and the call ends
    a, (dh, df) = scan_case([300, 300], 64, False, True, F32, seed=13)
    for cu in ([0, 700, 600], [500, 20, 600], [-5, 9, 1 << 30], [0, 0, -7], [9, 9, 9]):
        a["cu_seqlens"] = i32(cu)
        gdn.gdn_scan(**a)
        gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,C,lens,commit,mix", [
    (1, 4, None, False, False), (3, 260, None, False, True), (65, 1024, None, True, False),
    (5, 256, [1, 0, 7, 3, 2], True, True), (4, 1300, [2, 9, 1, 1], False, False)])
def test_scan_pool(dtype, n, C, lens, commit, mix):
    gen = torch.Generator().manual_seed(n + C)
    r = lambda *s: torch.randn(s, generator=gen)
    cu = list(range(n + 1)) if lens is None else [0] + [int(v) for v in np.cumsum(lens)]
    T = cu[-1]
    x, g, states = r(T, C).to(dtype).cuda(), -torch.rand((T, C), generator=gen).cuda(), r(n + 3, C).cuda()
    slots = torch.randperm(n + 3, generator=gen)[:n].tolist()
    if n > 2:
        slots[1] = -4 if n % 2 else n + 9
    keep = [int(v) for v in torch.randint(-1, 5, (n,), generator=gen)] if commit else None
    want, bound, after, after_bound = ref.scan_pool(f64(x), f64(g), f64(states), slots, cu, keep, mix)
    was, h = states.clone(), torch.full_like(x, 7.0)
    gdn.gdn_scan_pool(x, g, states, i32(slots), cu_seqlens=None if lens is None else i32(cu),
                      commit=None if keep is None else i32(keep), mix=mix, h=h)
    skipped = torch.isnan(want)
    assert bool((h.cpu()[skipped] == 7.0).all())
    close("h", torch.where(skipped, 0.0, f64(h)), torch.where(skipped, 0.0, want), bound, dtype)
    close("states", states, after, after_bound, F32)
    for s in range(n + 3):
        if s not in slots or (keep is not None and keep[slots.index(s)] <= 0):
            assert torch.equal(states[s], was[s])


def test_scan_pool_goes_on_from_scan():
    # a prompt with gdn_scan, then tokens one by one on a pool: as the whole sequence at once
    a, _ = scan_case([137], 512, True, False, F32, seed=14)
    x, g = a["x"], a["g"]
    whole, final = gdn.gdn_scan(**a)
    h, state = gdn.gdn_scan(x[:100], g[:100], i32([0, 100]), mix=True)
    pool = torch.zeros((3, 512), device="cuda")
    pool[1] = state[0]
    rows = [gdn.gdn_scan_pool(x[t:t + 1], g[t:t + 1], pool, i32([1]), mix=True) for t in range(100, 137)]
    want = ref.scan(*scan_reference(a))
    close("h", torch.cat([h] + rows), want["h"], want["bound"], F32)
    close("state", pool[1:2], want["final"], want["final_bound"], F32)
    assert bool((pool[0] == 0).all()) and bool((pool[2] == 0).all())


# ---------------------------------------------------------------- attention behind a common beginning


def shared_server(groups, page, hkv, dk, dv, seed, rows=True):
    """groups: [(tokens of the beginning, [(own tokens before the step, new tokens), ...])]; a paged cache in which the
    whole pages of a group's beginning are the same.  Returns (server, new tokens, group offsets, beginnings)."""
    kv = [p + own + new for p, reqs in groups for own, new in reqs]
    server = serve.Server(kv, page, hkv, dk, dv, seed=seed, rows=rows)
    n = 0
    for p, reqs in groups:
        at = [n + i if server.rows is None else int(server.rows[n + i]) for i in range(len(reqs))]
        for row in at[1:]:
            server.table[row, :p // page] = server.table[at[0], :p // page]
        n += len(reqs)
    sizes = [len(reqs) for _, reqs in groups]
    return server, [new for _, reqs in groups for _, new in reqs], [0] + [int(x) for x in np.cumsum(sizes)], [p for p, _ in groups]


@pytest.fixture(params=["1", "0", None], ids=["shared", "apart", "planned"])
def share(request, monkeypatch):
    """The beginnings read once, by each request, or as the library plans."""
    if request.param is None:
        monkeypatch.delenv("GDN_PREFIX_SHARE", raising=False)
    else:
        monkeypatch.setenv("GDN_PREFIX_SHARE", request.param)
    return request.param


@pytest.fixture
def always(monkeypatch):
    monkeypatch.setenv("GDN_PREFIX_SHARE", "1")


def prefix_check(server, lens, offsets, shared, H, dtype, seed=0, extra=2, **kw):
    gen = torch.Generator().manual_seed(seed + 100)
    dk, dv, T = server.k.shape[3], server.v.shape[3], sum(lens)
    q = torch.randn((T + extra, H, dk), generator=gen).to(dtype).cuda()
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    cu = i32([0] + [int(x) for x in np.cumsum(lens)])
    o = torch.full((T + extra, H, dv), 7.0, dtype=dtype, device="cuda")
    need = gdn.gdn_cache_attention_prefix_workspace_bytes(
        len(lens), len(shared), T + extra, kw.get("max_new", 0), kw.get("max_kv", 0), kw.get("max_prefix", 0), server.page,
        server.table.shape[1], H, server.k.shape[1], dk, dv)
    space = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    got = gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv_lens, cu, i32(offsets), i32(shared), rows=rows, o=o,
                                         workspace=space, **kw)
    assert got is o and bool((o[T:] == 7.0).all())
    scale = kw.get("scale", dk ** -0.5)
    want, mag, big = server.reference(q[:T].double(), lens, scale, "cuda")
    got = o[:T].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    # Scores: dk + 4 fp32 roundings of sum |q||k| (three of them for each of the split parts of fp32 q), and the
    # exponential and its argument in base 2.  p is off by twice that (numerator and denominator), the sums over S tokens
    # by at most S roundings each of sum p|v|; p itself is rounded once to the type's bf16 parts (three: 2^-24), o once to
    # its type.  A part's factor in the join is an exponential more: 8 roundings of p are added for it.
    S = max([1] + [int(x) for x in server.kv_lens])
    parts, half = (3, ref.E32) if dtype == F32 else (1, ref.E16)
    score = (parts * (dk + 4) + 16) * ref.E32 * big
    tol = (2 * score + 2 * (S + 64) * ref.E32 + half + 16 * ref.E32) * mag + half * want.abs() + 1e-30
    err = torch.nan_to_num((got - want).abs() / tol, nan=0.0).max().item() if T else 0.0
    log(f"  behind a common beginning: largest error / tolerance {err:.3f}")
    assert err <= 1.0, err
    return q, o


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("page,hkv,G", [(64, 2, 1), (128, 1, 7), (256, 2, 4), (64, 1, 20)])
def test_prefix(always, dtype, dk, dv, page, hkv, G):
    groups = [(1300, [(5, 1), (64, 1), (0, 1), (300, 2)]), (0, [(10, 1), (700, 1)]), (257, [(1, 3)]),
              (64, [(63, 1), (1, 0), (128, 40)]), (page - 1, [(3, 1), (9, 1)])]
    log(f"prefix page={page} H_kv={hkv} G={G} dk={dk} dv={dv} {dtype}")
    prefix_check(*shared_server(groups, page, hkv, dk, dv, seed=dk + page), hkv * G, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hints", [{}, dict(max_new=1, max_kv=10240, max_prefix=9000), dict(max_new=1, max_kv=64, max_prefix=64),
                                   dict(max_new=4000, max_prefix=100000)])
def test_prefix_long(share, dtype, hints):
    groups = [(9000, [(i * 37 % 700, 1) for i in range(40)])]
    prefix_check(*shared_server(groups, 64, 2, 128, 128, seed=3), 8, dtype, **hints)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("groups", [
    [(4096, [(0, 300), (17, 1), (0, 129)])], [(1000, [(0, 1)] * 3), (2000, [(5, 2)] * 2), (3000, [(9, 200), (0, 7)])],
    [(640, [(0, 1)] * 33), (64, [(0, 33), (0, 1)])], [(300, [(0, 0), (0, 0)]), (300, [(1, 1), (2, 0), (3, 5)])],
    [(70, [(0, 1), (0, 1)])] * 70, [(6000, [(3000, 1), (1, 1), (9000, 1)])]])
def test_prefix_of_many_and_few_rows(share, dtype, groups):
    prefix_check(*shared_server(groups, 64, 1, 64, 64, seed=4), 4, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefix_of_more_groups_than_lanes(always, dtype):
    # groups of many rows, of few, without a beginning, and without a request that takes part, in turn
    groups = [[(1100, [(i % 5, 1)] * 9), (700, [(3, 1)] * 2), (0, [(5, 1)] * 10), (640, [(1, 1)] * 11)][i % 4] for i in range(131)]
    server, lens, offsets, shared = shared_server(groups, 64, 1, 64, 64, seed=18)
    for g in range(3, 131, 8):
        shared[g] = 1 << 20
    prefix_check(server, lens, offsets, shared, 4, dtype)


def test_prefix_requests_that_take_no_part(share):
    # of the second group one request holds less than the beginning and one has been refused (it holds fewer tokens than it
    # adds); requests behind the last group are in none
    server, lens, offsets, shared = shared_server([(640, [(0, 1), (70, 2)]), (700, [(5, 1), (5, 1), (40, 3), (0, 1)]),
                                                   (500, [(0, 1), (1, 1)])], 64, 2, 64, 64, seed=5)
    server.kv_lens[3], server.kv_lens[4] = 333, 2
    prefix_check(server, lens, offsets[:3], shared[:2], 6, BF16)
    # a length of the beginning that no request holds, or below zero
    prefix_check(server, lens, offsets, [10 ** 9, -5, 500], 6, BF16)
    # no group, and groups of one: gdn_cache_attention itself
    for offs, lengths in ([[0], []], [list(range(9)), [64] * 8]):
        q, o = prefix_check(server, lens, offs, lengths, 6, BF16, extra=0)
        kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
        cu = i32([0] + [int(x) for x in np.cumsum(lens)])
        assert torch.equal(gdn.gdn_cache_attention(q, kc, vc, ks, vs, table, kv_lens, cu, rows=rows), o)


@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_prefix_requests_without_a_row(share, bad):
    # the first and the last request of a group have no row of the table: they see nothing, and the others all they hold
    server, lens, offsets, shared = shared_server([(640, [(4, 1), (70, 2), (0, 1), (9, 1)]), (200, [(0, 1), (5, 70)])], 64, 2, 64,
                                                  64, seed=14)
    for n in (0, 3, 4):
        server.rows[n] = bad
    prefix_check(server, lens, offsets, shared, 6, BF16)


def test_prefix_lengths_past_the_table(share):
    # requests that say to hold more than the table has room for hold what it has
    server, lens, offsets, shared = shared_server([(640, [(4, 1), (0, 2), (10, 1)]), (128, [(500, 1), (7, 1)])], 64, 2, 64, 64,
                                                  seed=15)
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    room = server.table.shape[1] * 64
    shared = [room, 128]
    q = torch.randn((sum(lens), 4, 64), device="cuda").to(BF16)
    cu, most = i32([0] + [int(x) for x in np.cumsum(lens)]), kv_lens.clamp(max=room)
    outs = []
    for kv in (most.clone(), most.clone()):
        kv[1] = room if not outs else 1 << 30
        outs.append(gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv, cu, i32(offsets), i32(shared), rows=rows))
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefix_bad_pages_and_nan(share, dtype):
    groups = [(1024, [(100, 1), (0, 1), (30, 70)]), (128, [(0, 1), (64, 2)])]
    for what in ("gone", "all gone", "nan value", "nan key", "past"):
        server, lens, offsets, shared = shared_server(groups, 64, 2, 64, 64, seed=6, rows=False)
        if what == "gone":
            server.table[:3, 4] = -1
            server.table[1, 16] = 10 ** 6
        elif what == "all gone":
            server.table[:3, :16] = -3
            server.table[1, 16:] = -1
            server.table[3:, :2] = 10 ** 6
        elif what == "nan value":
            page = int(server.table[0, 7])
            server.v[page, 1, 13, 5] = math.nan
            server.v[int(server.table[4, 2]), 0, 63, 9] = math.nan
        elif what == "nan key":
            server.k[int(server.table[0, 2]), 0, 3, 1] = math.nan
        else:
            server.table = server.table[:, :9].contiguous()  # of the beginning too there is no more than the table has
            server.kv_lens = [min(x, 9 * 64) for x in server.kv_lens]
            shared = [512, 128]
        prefix_check(server, lens, offsets, shared, 6, dtype)


def test_prefix_rows_that_see_nothing(share):
    server, lens, offsets, shared = shared_server([(128, [(3, 1), (0, 1)])], 64, 1, 64, 64, seed=7, rows=False)
    server.rows = torch.tensor([5, -1], dtype=torch.int32)
    _, o = prefix_check(server, lens, offsets, shared, 2, BF16)
    assert bool((o[:2] == 0).all())


def test_prefix_infinite_queries(share):
    # a row whose scores are all -Inf is NaN, as without a common beginning
    server, lens, offsets, shared = shared_server([(320, [(10, 1), (99, 1), (5, 1)])], 64, 1, 64, 64, seed=8, rows=False)
    server.k[..., 0] = 8.0
    kc, vc, ks, vs, table, kv_lens, _ = server.to("cuda")
    q = torch.randn((3, 40, 64), device="cuda")
    q[1, 7, 0], q[2, 39, 0] = -math.inf, math.inf
    o = gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv_lens, i32([0, 1, 2, 3]), i32(offsets), i32(shared))
    bad = torch.zeros((3, 40), dtype=torch.bool, device="cuda")
    bad[1, 7] = bad[2, 39] = True
    assert bool(torch.isnan(o[bad]).all()) and bool(torch.isfinite(o[~bad]).all())


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_prefix_scale(always, scale):
    prefix_check(*shared_server([(700, [(100, 1), (0, 3), (64, 1)])], 64, 2, 64, 64, seed=9), 6, BF16, scale=scale)


def test_prefix_offsets_that_are_none(always):
    # outputs are then no one's, but nothing outside the arrays is touched and the call ends
    server, lens, offsets, shared = shared_server([(640, [(9, 1)] * 4), (128, [(9, 2)] * 3)], 64, 2, 64, 64, seed=10)
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    q = torch.randn((sum(lens), 4, 64), device="cuda").to(BF16)
    good = [0] + [int(x) for x in np.cumsum(lens)]
    for offs, cu in (([5, 2, 7], good), ([-9, 3, 1 << 30], good), ([0, 9, -1], good), ([3, 3, 3], good), ([0, 4, 7], [9, 3, 3, 1, 50, 2, 0, -4]),
                     ([7, 4, 0], [0, 900, 3, 5, 5, 5, 7, 1 << 30])):
        gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv_lens, i32(cu), i32(offs), i32(shared), rows=rows)
        torch.cuda.synchronize()
    gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, i32([-5, 1 << 30, 0, 7, -(1 << 31), 700, 3]), i32(good), i32(offsets),
                                   i32(shared), rows=rows)
    torch.cuda.synchronize()


def test_prefix_equals_requests_apart(monkeypatch):
    # for the same call both ways: a call that the plan reads apart gives gdn_cache_attention's bits
    server, lens, offsets, shared = shared_server([(640, [(9, 1)] * 4)], 64, 2, 64, 64, seed=12)
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    q = torch.randn((4, 4, 64), device="cuda").to(BF16)
    cu = i32([0, 1, 2, 3, 4])
    plain = gdn.gdn_cache_attention(q, kc, vc, ks, vs, table, kv_lens, cu, rows=rows, max_new=1, max_kv=650)
    got = []
    for how in ("1", "0", None):
        monkeypatch.delenv("GDN_PREFIX_SHARE", raising=False)
        if how:
            monkeypatch.setenv("GDN_PREFIX_SHARE", how)
        got.append(gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv_lens, cu, i32(offsets), i32(shared), rows=rows,
                                                  max_new=1, max_kv=650, max_prefix=640))
    assert torch.equal(got[1], plain) and torch.equal(got[2], plain)
    # each rounds p and o of its own sums
    assert float((got[0].double() - plain.double()).norm() / plain.double().norm()) <= 2 * ref.E16


def test_prefix_two_graphs_and_other_streams(share):
    server, lens, offsets, shared = shared_server([(3000, [(i, 1) for i in range(20)]), (640, [(0, 70), (9, 1)])], 64, 2, 128, 128,
                                                  seed=11)
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    cu, go, pl = i32([0] + [int(x) for x in np.cumsum(lens)]), i32(offsets), i32(shared)
    q = torch.randn((sum(lens), 8, 128), device="cuda").to(BF16)

    def call(stream=None):
        return gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv_lens, cu, go, pl, rows=rows, stream=stream)

    want = call().clone()
    side = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [call(s) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(call())
    for rep in range(4):
        junk = torch.randn(1 << 20, device="cuda")
        assert torch.isfinite((junk * 2).sum()).item()
        for g, o in zip(graphs, outs):
            o.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want), rep


def test_a_server_behind_one_prompt(share):
    """Steps of a server: a prompt written once, its pages put into the rows of twelve requests, then tokens of each: tables,
    norm and rotation, cache write, attention behind the prompt, recurrence on a pool."""
    torch.manual_seed(31)
    page, hkv, H, d, n, P, C = 64, 2, 8, 64, 12, 1000, 256
    pages, blocks = 64, 24
    kc = torch.zeros((pages, hkv, page, d), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros((pages, hkv, page // 16, d, 16), dtype=torch.float8_e4m3fn, device="cuda")
    ks, vs = (torch.ones((pages, hkv), device="cuda") for _ in range(2))
    table, counts = i32([[-1] * blocks] * (n + 1)), i32([0] * (n + 1))
    free, state = i32(list(range(pages))), i32([0, pages, 0])
    freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()
    norm = dict(norm=gdn.GDN_NORM_RMS, q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"),
                inv_freq=freq)
    wide = lambda T: torch.randn((T, H + 2 * hkv, d), device="cuda").to(BF16)

    def step(ctx, new, T, rows):
        cu, kv, slots, pos = gdn.gdn_batch_tables(i32(ctx), i32(new), T, page, table, counts, free, state, rows=i32(rows))
        x = wide(T)
        q, k = gdn.gdn_qk_norm(x[:, :H], x[:, H:H + hkv], positions=pos, **norm)
        gdn.gdn_cache_write(k, x[:, H + hkv:].contiguous(), slots, kc, vc, ks, vs)
        return q, cu, kv

    step([0], [P], P, [n])  # the prompt, in the last row
    whole = P // page
    table[:n, :whole] = table[n, :whole]
    counts[:n] = whole
    pool = torch.randn((n + 2, C), device="cuda")
    groups, shared = i32([0, n]), i32([whole * page])
    for turn in range(3):
        held = [whole * page + turn * 2] * n
        q, cu, kv = step(held, [2] * n, 2 * n, list(range(n)))
        kw = dict(rows=i32(list(range(n))), max_new=2, max_kv=1024)
        o = gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, kv, cu, groups, shared, max_prefix=P, **kw)
        plain = gdn.gdn_cache_attention(q, kc, vc, ks, vs, table, kv, cu, **kw)
        # two roundings of bf16 apart: each rounds p and o of its own sums
        assert float((o.double() - plain.double()).norm() / plain.double().norm()) <= 2 * ref.E16
        y = o.reshape(2 * n, -1)[:, :C].contiguous()
        before = pool.clone()
        commit = kv - i32(held)
        g = -torch.rand((2 * n, C), device="cuda")
        h = gdn.gdn_scan_pool(y, g, pool, i32(list(range(n))), cu_seqlens=cu, commit=commit)
        want, bound, after, after_bound = ref.scan_pool(f64(y), f64(g), f64(before), list(range(n)), list(range(0, 2 * n + 1, 2)),
                                                        [2] * n, False)
        close("h", h, want, bound, BF16)
        close("pool", pool, after, after_bound, F32)
    assert int(state[2]) == 0


# ---------------------------------------------------------------- the calls together


def _calls():
    """Every call on fixed inputs; returns their outputs."""
    n = norm_case(200, 8, 2, 128, 2, True, 128, False, BF16, True, seed=21)
    rest = {s: v for s, v in n.items() if s not in "qk"}
    gq, gk = torch.randn((200, 8, 128), device="cuda").to(BF16), torch.randn((200, 2, 128), device="cuda").to(BF16)
    a, (dh, df) = scan_case([400, 0, 3, 250], 516, True, True, BF16, seed=22)
    pool, was = torch.empty((9, 516), device="cuda"), torch.randn((9, 516), device="cuda")
    slots = i32([3, 8, 0])

    def calls():
        out = list(gdn.gdn_qk_norm(**n))
        out += gdn.gdn_qk_norm_backward(n["q"], n["k"], gq, gk, **rest)
        kept = gdn.gdn_scan_checkpoints(a["x"])
        out += gdn.gdn_scan(**a, checkpoints=kept)
        out += gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df, checkpoints=kept)
        out += gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)
        pool.copy_(was)
        out += [gdn.gdn_scan_pool(a["x"][:3], a["g"][:3], pool, slots, mix=True), pool]
        return out

    return calls


def test_graphs_replay_every_call():
    calls = _calls()
    eager = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(calls())
    for rep in range(4):
        junk = torch.randn(1 << 20, device="cuda")
        assert torch.isfinite((junk * 2).sum()).item()
        for g, got in zip(graphs, outs):
            for t in got:
                t.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            for i, (x, y) in enumerate(zip(got, eager)):
                assert torch.equal(x, y), f"replay {rep}: output {i} differs from the eager call"


def test_other_streams_and_repeats_give_the_same_bits():
    calls = _calls()
    want = [t.clone() for t in calls()]
    for rep in range(3):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = calls()
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_scans_on_two_streams_at_once():
    a, (dh, df) = scan_case([9000], 1024, False, True, BF16, seed=23)
    want = [t.clone() for t in gdn.gdn_scan(**a)] + [t.clone() for t in gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:  # of each call its own workspace
        got.append(gdn.gdn_scan(**a, stream=s) + gdn.gdn_scan_backward(**a, d_h=dh, d_final_state=df, stream=s))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_a_training_step():
    """Unit queries and keys into the layer, the recurrence behind it, and the gradients back through all three: against
    differences of the same forward calls in full precision."""
    torch.manual_seed(30)
    T, H, d = 150, 2, 64
    lens = [80, 0, 70]
    cu = i32([0, 80, 80, 150])
    r = lambda *s: torch.randn(s, device="cuda")
    p = dict(q=r(T, H, d), k=r(T, H, d), v=r(T, H, d), g=-torch.rand((T, H, d), device="cuda"), beta=torch.sigmoid(r(T, H)),
             gate=-torch.rand((T, H * d), device="cuda"))
    dy = r(T, H * d)
    norm = dict(norm=gdn.GDN_NORM_L2, eps=1e-6, q_scale=d ** -0.5)

    def forward(p):
        q, k = gdn.gdn_qk_norm(p["q"], p["k"], **norm)
        o, _ = gdn.gdn_prefill(q, k, p["v"], p["g"], p["beta"], cu)
        y, _ = gdn.gdn_scan(o.view(T, H * d), p["gate"], cu, mix=True)
        return q, k, o, y

    q, k, o, y = forward(p)
    dx, dgate, _ = gdn.gdn_scan_backward(o.view(T, H * d), p["gate"], cu, dy, mix=True)
    dqn, dkn, dv, dg, dbeta, _ = gdn.gdn_prefill_backward(q, k, p["v"], p["g"], p["beta"], cu, dx.view(T, H, d))
    dq, dk, _, _ = gdn.gdn_qk_norm_backward(p["q"], p["k"], dqn, dkn, **norm)
    got = dict(q=dq, k=dk, v=dv, g=dg, beta=dbeta, gate=dgate)
    for name in got:
        # along the gradient itself, so that the difference is large against fp32's noise: the two halves of a central
        # difference of step e carry E32-sized noise of |y||dy|, over 2 e |gradient|
        direction = got[name] / got[name].norm()
        e = 2e-3 * float(p[name].norm()) / 10
        ends = [float((forward({**p, name: p[name] + s * e * direction})[3].double() * dy.double()).sum()) for s in (1, -1)]
        slope, want = (ends[0] - ends[1]) / (2 * e), float(got[name].double().norm())
        log(f"  {name}: gradient {want:.6f}, difference {slope:.6f}")
        assert abs(slope - want) <= 2e-2 * want, name


def test_binding_refusals(always):
    x = torch.zeros((4, 2, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    for kw in (dict(q=x[:, :, :32]), dict(q=x.transpose(0, 1)), dict(q=x[..., ::2]), dict(k=x[:3]), dict(positions=i32([0] * 4)),
               dict(inv_freq=w[:32]), dict(q_weight=w[:32]), dict(q_out=x[:3]), dict(k_out=x), dict(q_weight=w.cpu()),
               dict(k=x, k_out=x[:, :1])):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_qk_norm(**{**dict(q=x), **kw})
    for kw in (dict(q=x.to(BF16), k=x), dict(q_weight=w.double()), dict(q=x.half())):
        with pytest.raises(TypeError):
            gdn.gdn_qk_norm(**{**dict(q=x), **kw})
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm(x, positions=i32([0] * 4), inv_freq=torch.ones(6, device="cuda"))  # 12 channels
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm(x, eps=0.0)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_backward(x, None, x, None, q_weight=w, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_backward(x, x, x, x, dq=torch.empty((4, 3, 64), device="cuda"))
    y, cu = torch.zeros((9, 8), device="cuda"), i32([0, 9])
    s = torch.zeros((1, 8), device="cuda")
    for kw in (dict(g=y[:8]), dict(x=y[:, :6], g=y[:, :6]), dict(initial_state=s[:, :4]), dict(final_state=s[:0]),
               dict(h=y.t()), dict(checkpoints=y[0, :1]), dict(workspace=torch.empty(1 << 16))):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_scan(**{**dict(x=y, g=y, cu_seqlens=cu), **kw})
    for kw in (dict(g=y.to(BF16)), dict(cu_seqlens=cu.long()), dict(initial_state=s.to(BF16)), dict(x=y.half())):
        with pytest.raises(TypeError):
            gdn.gdn_scan(**{**dict(x=y, g=y, cu_seqlens=cu), **kw})
    with pytest.raises(gdn.GdnError):
        gdn.gdn_scan(y[:, :6].contiguous(), y[:, :6].contiguous(), cu)  # channels in fours
    with pytest.raises(gdn.GdnError):
        gdn.gdn_scan(y, y, cu, initial_state=s, final_state=s)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_scan(y, y, cu, workspace=torch.empty(1, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        gdn.gdn_scan_backward(y, y, cu, y.to(BF16))
    with pytest.raises((ValueError, gdn.GdnError)):
        gdn.gdn_scan_pool(y, y, s, cu)
    server, lens, offsets, shared = shared_server([(128, [(3, 1), (0, 1)])], 64, 1, 64, 64, seed=7, rows=False)
    kc, vc, ks, vs, table, kv_lens, _ = server.to("cuda")
    q = torch.randn((2, 2, 64), device="cuda")
    fine = dict(block_table=table, kv_lens=kv_lens, cu_seqlens=i32([0, 1, 2]), group_offsets=i32(offsets),
                prefix_lens=i32(shared))
    for kw in (dict(group_offsets=i32([0])), dict(cu_seqlens=i32([0, 1])), dict(prefix_lens=i32([1, 2])), dict(o=q[:1]),
               dict(workspace=torch.empty(4, device="cuda")), dict(max_prefix=-1), dict(group_offsets=i32([0, 2]).cpu())):
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, **{**fine, **kw})
    with pytest.raises(TypeError):
        gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, **{**fine, "prefix_lens": i32([1]).long()})


def test_validation_of_group_offsets(monkeypatch):
    # one offset in the middle is past the requests
    monkeypatch.setenv("GDN_VALIDATE", "1")
    server, lens, offsets, shared = shared_server([(128, [(3, 1), (0, 1)]), (0, [(0, 1)])], 64, 1, 64, 64, seed=7, rows=False)
    kc, vc, ks, vs, table, kv_lens, _ = server.to("cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_cache_attention_prefix(torch.randn((3, 2, 64), device="cuda"), kc, vc, ks, vs, table, kv_lens, i32([0, 1, 2, 3]),
                                       i32([0, 1 << 20, 3]), i32(shared))
    assert e.value.status == gdn.GDN_ERR_DOMAIN


def test_validation_mode(monkeypatch):
    monkeypatch.setenv("GDN_VALIDATE", "1")
    y = torch.zeros((9, 8), device="cuda")
    s, good = torch.zeros((4, 8), device="cuda"), i32([0, 4, 9])
    gdn.gdn_scan(y, y, good)
    gdn.gdn_scan(y, y, i32([0, 4, 8]))
    behind = y.clone()
    behind[8] = math.nan
    gdn.gdn_scan(y, behind, i32([0, 4, 8]))
    gdn.gdn_scan_pool(y, y, s, i32([3, 1]), cu_seqlens=good)
    bad = y.clone()
    bad[3, 2] = 1e-3
    nan = y.clone()
    nan[8, 7] = math.nan
    for kw in (dict(cu_seqlens=i32([0, 5, 4])), dict(cu_seqlens=i32([1, 4, 9])), dict(cu_seqlens=i32([0, 4, 10])), dict(g=bad),
               dict(g=nan)):
        for call in (gdn.gdn_scan, lambda **k: gdn.gdn_scan_backward(**k, d_h=y)):
            with pytest.raises(gdn.GdnError) as e:
                call(**{**dict(x=y, g=y, cu_seqlens=good), **kw})
            assert e.value.status == gdn.GDN_ERR_DOMAIN
    server, lens, offsets, shared = shared_server([(128, [(3, 1), (0, 1)]), (0, [(0, 1)])], 64, 1, 64, 64, seed=7, rows=False)
    kc, vc, ks, vs, table, kv_lens, _ = server.to("cuda")
    q = torch.randn((3, 2, 64), device="cuda")
    other = table.clone()
    other[1, 1] = table[2, 0]
    fine = dict(block_table=table, kv_lens=kv_lens, cu_seqlens=i32([0, 1, 2, 3]), group_offsets=i32(offsets),
                prefix_lens=i32(shared))
    gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, **fine)
    gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, **{**fine, "block_table": other, "prefix_lens": i32([64, 0])})
    for kw in (dict(group_offsets=i32([0, 2, 4])), dict(group_offsets=i32([1, 2, 3])), dict(group_offsets=i32([0, 2, 1])),
               dict(prefix_lens=i32([-1, 0])), dict(block_table=other), dict(cu_seqlens=i32([0, 2, 1, 3]))):
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_cache_attention_prefix(q, kc, vc, ks, vs, **{**fine, **kw})
        assert e.value.status == gdn.GDN_ERR_DOMAIN
    for kw in (dict(slots=i32([1, 1])), dict(cu_seqlens=i32([0, 4, 8])), dict(g=nan)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_scan_pool(**{**dict(x=y, g=y, states=s, slots=i32([3, 1]), cu_seqlens=good), **kw})
        assert e.value.status == gdn.GDN_ERR_DOMAIN


def test_a_training_step_against_64_bits():
    """The calls of test_a_training_step against float64's automatic differentiation of the definitions, by sequence and
    head, so that no part of a gradient can be missing: each part is as near as the layer's gradients are held to in full
    precision, for each of the three calls that it goes through."""
    gen = torch.Generator().manual_seed(31)
    T, H, d, lens = 150, 2, 64, [80, 0, 70]
    r = lambda *s: torch.randn(s, generator=gen)
    p = dict(q=r(T, H, d), k=r(T, H, d), v=r(T, H, d), g=-torch.rand((T, H, d), generator=gen), beta=torch.sigmoid(r(T, H)),
             gate=-torch.rand((T, H * d), generator=gen))
    dy = r(T, H * d)
    leaves = {n: t.double().requires_grad_() for n, t in p.items()}
    unit = lambda x: x * (x.square().sum(-1, keepdim=True) + 1e-6).rsqrt()
    qn, kn = unit(leaves["q"]) * d ** -0.5, unit(leaves["k"])
    alpha, decay, y, first = leaves["g"].exp(), leaves["gate"].exp(), [], 0
    for length in lens:
        S, h = torch.zeros((H, d, d), dtype=torch.float64), torch.zeros(H * d, dtype=torch.float64)
        for t in range(first, first + length):
            S = alpha[t][:, :, None] * S
            gap = leaves["v"][t] - (S * kn[t][:, :, None]).sum(1)
            S = S + leaves["beta"][t][:, None, None] * kn[t][:, :, None] * gap[:, None, :]
            o = (S * qn[t][:, :, None]).sum(1).reshape(H * d)
            h = decay[t] * h + (1 - decay[t]) * o
            y.append(h)
        first += length
    y = torch.stack(y)
    (y * dy.double()).sum().backward()

    a, cu = {n: t.cuda() for n, t in p.items()}, i32([0, 80, 80, 150])
    norm = dict(norm=gdn.GDN_NORM_L2, eps=1e-6, q_scale=d ** -0.5)
    q, k = gdn.gdn_qk_norm(a["q"], a["k"], **norm)
    o, _ = gdn.gdn_prefill(q, k, a["v"], a["g"], a["beta"], cu)
    o = o.view(T, H * d)
    h, _ = gdn.gdn_scan(o, a["gate"], cu, mix=True)
    dx, dgate, _ = gdn.gdn_scan_backward(o, a["gate"], cu, dy.cuda(), mix=True)
    dqn, dkn, dv, dg, dbeta, _ = gdn.gdn_prefill_backward(q, k, a["v"], a["g"], a["beta"], cu, dx.view(T, H, d))
    dq, dk, _, _ = gdn.gdn_qk_norm_backward(a["q"], a["k"], dqn, dkn, **norm)
    for name, got, want in [("y", h, y)] + [(n, t, leaves[n].grad) for n, t in dict(q=dq, k=dk, v=dv, g=dg, beta=dbeta, gate=dgate).items()]:
        got, want = f64(got).reshape(T, H, -1), want.detach().reshape(T, H, -1)
        for lo, hi in ((0, 80), (80, 150)):
            for head in range(H):
                x, w = got[lo:hi, head], want[lo:hi, head]
                off = float((x - w).abs().max() / w.abs().max())
                log(f"  {name} tokens {lo} to {hi}, head {head}: {off:.2e}")
                assert off <= 3 * TOL[F32], name
