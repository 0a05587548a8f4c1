"""The calls of include/gdn_stack.h on the host, without a GPU: exports, refusals with the documented status codes before
any memory is touched, workspace sizes, the binding's own checks, and the plain 64-bit forms that the GPU tests compare
with (pinned by properties and differences that do not go through the library)."""

import ctypes
import math

import pytest
import torch

import gated_delta_rule_linear_amd as gdn
import stack_reference as ref

OK, INVALID, UNSUPPORTED, DOMAIN, OOM, HIPERR = range(6)
BAD = ctypes.c_void_p(0x1001)   # misaligned; never dereferenced because validation rejects it first
FAKE = ctypes.c_void_p(0x1000)  # aligned, and never dereferenced either
NUL = None
MANY = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return gdn.load_library()


def test_exports(lib):
    names = gdn.exported_symbols_in_header(gdn.STACK_HEADER)
    assert {"gdn_qk_norm", "gdn_qk_norm_backward", "gdn_qk_norm_backward_workspace_bytes", "gdn_scan", "gdn_scan_backward",
            "gdn_scan_pool", "gdn_scan_checkpoint_bytes", "gdn_scan_workspace_bytes",
            "gdn_scan_backward_workspace_bytes", "gdn_cache_attention_prefix",
            "gdn_cache_attention_prefix_workspace_bytes"} == set(names)
    for n in names:
        assert hasattr(lib, n) and n in gdn.__all__ and hasattr(gdn, n), n


def _norm(lib, q=FAKE, qs=512, k=FAKE, ks=256, T=5, H=4, hk=2, d=128, norm=2, eps=1e-6, wq=NUL, wk=NUL, pos=FAKE, freq=FAKE,
          rot=128, pairs=0, scale=1.0, qo=FAKE, ko=FAKE, dt=1):
    return lib.gdn_qk_norm(q, qs, k, ks, T, H, hk, d, norm, eps, wq, wk, pos, freq, rot, pairs, scale, qo, ko, dt, None)


NORM = [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(H=-1), INVALID), (dict(hk=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(H=1 << 20), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
    (dict(norm=3), UNSUPPORTED), (dict(norm=-1), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=1e-42), INVALID), (dict(eps=math.inf), INVALID), (dict(eps=math.nan), INVALID), (dict(scale=math.nan), INVALID),
    (dict(rot=12), INVALID), (dict(rot=-8), INVALID), (dict(rot=136), INVALID), (dict(pos=NUL), INVALID),
    (dict(freq=NUL), INVALID), (dict(freq=BAD), INVALID), (dict(pos=BAD), INVALID), (dict(wq=BAD), INVALID),
    (dict(wk=BAD), INVALID), (dict(q=BAD), INVALID), (dict(k=NUL), INVALID), (dict(qs=511), INVALID),
    (dict(qs=516), INVALID), (dict(ks=248), INVALID), (dict(qs=1 << 62), INVALID)]


@pytest.mark.parametrize("kw,want", NORM + [(dict(qo=NUL), INVALID), (dict(ko=BAD), INVALID),
                                            (dict(T=0, q=NUL, pos=NUL), OK), (dict(H=0, hk=0, q=NUL, k=NUL), OK)])
def test_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def _norm_back(lib, q=FAKE, qs=512, k=FAKE, ks=256, gq=FAKE, gk=FAKE, T=5, H=4, hk=2, d=128, norm=2, eps=1e-6, wq=NUL,
               wk=NUL, pos=FAKE, freq=FAKE, rot=128, pairs=0, scale=1.0, dq=FAKE, dqs=512, dk=FAKE, dks=256, dwq=NUL, dwk=NUL,
               dt=1, ws=NUL, wb=0):
    return lib.gdn_qk_norm_backward(q, qs, k, ks, gq, gk, T, H, hk, d, norm, eps, wq, wk, pos, freq, rot, pairs, scale, dq,
                                    dqs, dk, dks, dwq, dwk, dt, ws, wb, None)


@pytest.mark.parametrize("kw,want", NORM + [
    (dict(gq=NUL), INVALID), (dict(gk=BAD), INVALID), (dict(dq=NUL), INVALID), (dict(dk=BAD), INVALID),
    (dict(dqs=504), INVALID), (dict(dks=257), INVALID), (dict(dwq=BAD), INVALID), (dict(dwq=FAKE), INVALID),
    (dict(dwk=FAKE, ws=FAKE, wb=16), INVALID), (dict(dwk=FAKE, ws=BAD, wb=MANY), INVALID),
    (dict(T=0, q=NUL, pos=NUL, gq=NUL), OK), (dict(H=0, hk=0, q=NUL, k=NUL), OK)])
def test_norm_backward_refusals(lib, kw, want):
    assert _norm_back(lib, **kw) == want


def _scan(lib, x=FAKE, g=FAKE, cu=FAKE, n=2, T=9, C=64, mix=0, s0=NUL, s1=NUL, h=FAKE, ck=NUL, dt=1, ws=FAKE, wb=MANY):
    return lib.gdn_scan(x, g, cu, n, T, C, mix, s0, s1, h, ck, dt, ws, wb, None)


SCAN = [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(C=0), INVALID), (dict(C=-4), INVALID), (dict(C=6), UNSUPPORTED),
    (dict(T=(1 << 31) - 1, C=1 << 10), UNSUPPORTED), (dict(T=1 << 29, C=4), UNSUPPORTED),
    (dict(T=1 << 20, C=1 << 19), UNSUPPORTED), (dict(T=0, C=(1 << 31) - 4), UNSUPPORTED), (dict(n=-1), INVALID), (dict(n=0), INVALID), (dict(dt=7), UNSUPPORTED),
    (dict(x=BAD), INVALID), (dict(g=NUL), INVALID), (dict(cu=NUL), INVALID), (dict(cu=BAD), INVALID), (dict(s0=BAD), INVALID),
    (dict(ck=BAD), INVALID), (dict(ws=NUL), INVALID), (dict(ws=BAD), INVALID), (dict(wb=64), INVALID)]


@pytest.mark.parametrize("kw,want", SCAN + [
    (dict(h=NUL), INVALID), (dict(s1=BAD), INVALID), (dict(s0=FAKE, s1=FAKE), INVALID),
    (dict(s0=FAKE, s1=ctypes.c_void_p(0x1000 + 2 * 64 * 4 - 16)), INVALID), (dict(n=0, T=0, x=NUL, cu=NUL), OK)])
def test_scan_refusals(lib, kw, want):
    assert _scan(lib, **kw) == want


def _scan_back(lib, x=FAKE, g=FAKE, cu=FAKE, n=2, T=9, C=64, mix=0, s0=NUL, ck=NUL, dh=FAKE, df=NUL, dx=FAKE, dg=FAKE,
               d0=NUL, dt=1, ws=FAKE, wb=MANY):
    return lib.gdn_scan_backward(x, g, cu, n, T, C, mix, s0, ck, dh, df, dx, dg, d0, dt, ws, wb, None)


@pytest.mark.parametrize("kw,want", SCAN + [
    (dict(dh=NUL), INVALID), (dict(dx=BAD), INVALID), (dict(dg=NUL), INVALID), (dict(df=BAD), INVALID),
    (dict(d0=BAD), INVALID), (dict(df=FAKE, d0=FAKE), INVALID), (dict(n=0, T=0, x=NUL, cu=NUL), OK)])
def test_scan_backward_refusals(lib, kw, want):
    assert _scan_back(lib, **kw) == want


def _pool(lib, x=FAKE, g=FAKE, states=FAKE, slots=FAKE, cu=NUL, commit=NUL, n=3, T=3, ns=8, C=64, mix=0, h=FAKE, dt=1):
    return lib.gdn_scan_pool(x, g, states, slots, cu, commit, n, T, ns, C, mix, h, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(ns=-1), INVALID), (dict(C=0), INVALID), (dict(C=5), UNSUPPORTED),
    (dict(dt=9), UNSUPPORTED), (dict(T=4), INVALID), (dict(n=0, T=4, cu=FAKE), INVALID),
    (dict(n=1 << 20, T=1 << 20, C=4096), UNSUPPORTED), (dict(x=BAD), INVALID), (dict(g=NUL), INVALID),
    (dict(states=NUL), INVALID), (dict(h=BAD), INVALID), (dict(slots=NUL), INVALID), (dict(cu=BAD), INVALID),
    (dict(commit=BAD), INVALID), (dict(n=0, T=0, x=NUL), OK), (dict(ns=0, states=NUL), OK)])
def test_scan_pool_refusals(lib, kw, want):
    assert _pool(lib, **kw) == want


def _prefix(lib, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, rows=NUL, kv=FAKE, cu=FAKE, go=FAKE, pl=FAKE, n=4,
            groups=2, T=4, max_new=0, max_kv=0, max_prefix=0, pages=5, page=64, nr=4, mb=4, scale=0.1, o=FAKE, H=4, hkv=2, dk=64,
            dv=64, dt=1, ws=FAKE, wb=MANY):
    return lib.gdn_cache_attention_prefix(q, kc, vc, ks, vs, table, rows, kv, cu, go, pl, n, groups, T, max_new, max_kv,
                                          max_prefix, pages, page, nr, mb, scale, o, H, hkv, dk, dv, dt, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(groups=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(max_new=-1), INVALID), (dict(max_kv=-1), INVALID), (dict(max_prefix=-1), INVALID), (dict(mb=-1), INVALID),
    (dict(H=5), INVALID), (dict(hkv=0), INVALID), (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(dt=5), UNSUPPORTED), (dict(n=0), INVALID), (dict(T=1 << 30, H=64), UNSUPPORTED),
    (dict(nr=-1), INVALID), (dict(pages=-1), INVALID), (dict(scale=math.inf), INVALID), (dict(q=BAD), INVALID),
    (dict(o=NUL), INVALID), (dict(kv=NUL), INVALID), (dict(cu=BAD), INVALID), (dict(rows=BAD), INVALID),
    (dict(table=NUL), INVALID), (dict(kc=BAD), INVALID), (dict(vs=NUL), INVALID), (dict(go=NUL), INVALID),
    (dict(go=BAD), INVALID), (dict(pl=NUL), INVALID), (dict(ws=NUL), INVALID), (dict(wb=16), INVALID),
    (dict(T=0, n=0, q=NUL, go=NUL), OK)])
def test_prefix_refusals(lib, monkeypatch, kw, want):
    monkeypatch.setenv("GDN_PREFIX_SHARE", "1")  # (so small a call would not be planned to need a workspace)
    assert _prefix(lib, **kw) == want


def test_prefix_workspace_sizes(monkeypatch):
    monkeypatch.delenv("GDN_PREFIX_SHARE", raising=False)
    size = gdn.gdn_cache_attention_prefix_workspace_bytes
    sizes = (64, 1024, 32, 8, 128, 128)
    plain = gdn.gdn_cache_attention_workspace_bytes(8, 8, 1, 9000, *sizes)
    assert size(8, 8, 8, 1, 9000, 4096, *sizes) == plain and size(8, 0, 8, 1, 9000, 4096, *sizes) == plain
    # one new token of each: little to save, then much; and forced either way
    assert size(8, 1, 8, 1, 1100, 1024, *sizes) == gdn.gdn_cache_attention_workspace_bytes(8, 8, 1, 1100, *sizes)
    assert size(64, 1, 64, 1, 17000, 16384, *sizes) > gdn.gdn_cache_attention_workspace_bytes(64, 64, 1, 17000, *sizes)
    # 256 new tokens keep the matrix cores busy by themselves
    assert size(8, 1, 2048, 256, 17000, 16384, *sizes) == gdn.gdn_cache_attention_workspace_bytes(8, 2048, 256, 17000, *sizes)
    monkeypatch.setenv("GDN_PREFIX_SHARE", "1")
    assert size(8, 1, 8, 1, 1100, 1024, *sizes) > gdn.gdn_cache_attention_workspace_bytes(8, 8, 1, 1100, *sizes)
    assert size(8, 8, 8, 1, 9000, 4096, *sizes) == plain
    monkeypatch.setenv("GDN_PREFIX_SHARE", "0")
    assert size(64, 1, 64, 1, 17000, 16384, *sizes) == gdn.gdn_cache_attention_workspace_bytes(64, 64, 1, 17000, *sizes)
    # more rows than a grid has workgroups are not joined, whatever is asked for
    monkeypatch.setenv("GDN_PREFIX_SHARE", "1")
    apart = gdn.gdn_cache_attention_workspace_bytes(8192, 1 << 20, 64, 17000, *sizes)
    assert size(8192, 1, 1 << 20, 64, 17000, 16384, *sizes) == apart
    assert size(8192, 1, 1 << 18, 32, 17000, 16384, *sizes) > gdn.gdn_cache_attention_workspace_bytes(8192, 1 << 18, 32, 17000, *sizes)
    monkeypatch.delenv("GDN_PREFIX_SHARE")
    assert size(8, 1, 0, 1, 9000, 4096, *sizes) == 0 and size(8, -1, 8, 1, 9000, 4096, *sizes) == 0


def test_workspace_sizes():
    assert gdn.gdn_qk_norm_backward_workspace_bytes(-1, 4, 2, 64) == 0
    assert gdn.gdn_qk_norm_backward_workspace_bytes(10, 4, 2, 65) == 0
    assert 0 < gdn.gdn_qk_norm_backward_workspace_bytes(1 << 30, 64, 8, 128) <= 1 << 21
    for f in (gdn.gdn_scan_checkpoint_bytes, gdn.gdn_scan_workspace_bytes, gdn.gdn_scan_backward_workspace_bytes):
        assert f(-1, 64) == 0 and f(100, 6) == 0 and f(100, 0) == 0
        assert f(65536, 4096) <= 65536 * 4096  # a small part of the inputs' 6 bytes an element


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm(x)
    with pytest.raises(TypeError):
        gdn.gdn_qk_norm(x.half())
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_backward(x, None, x, None)
    y = torch.zeros(3, 64)
    with pytest.raises(ValueError):
        gdn.gdn_scan(y, y, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.gdn_scan_backward(y, y, torch.zeros(2, dtype=torch.int32), y)
    with pytest.raises(ValueError):
        gdn.gdn_scan_pool(y, y, y, torch.zeros(3, dtype=torch.int32))


# ---------------------------------------------------------------- the plain forms themselves


def _difference(f, x, direction, step=1e-5):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_norm_gradients_match_differences(norm, interleaved):
    gen = torch.Generator().manual_seed(norm)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, dy, w, d = r(5, 3, 64), r(5, 3, 64), r(64), r(5, 3, 64)
    pos, freq = torch.tensor([0, 1, -7, 1000, 123456]), torch.rand(16, generator=gen, dtype=torch.float64)
    f = lambda x, w: (ref.qk_norm(x, norm, 1e-6, w, pos, freq, interleaved, 0.3)[0] * dy).sum()
    dx, _, dw, _ = ref.qk_norm_backward(x, dy, norm, 1e-6, w, pos, freq, interleaved, 0.3)
    assert abs(_difference(lambda v: f(v, w), x, d) - (dx * d).sum()) < 1e-7
    e = r(64)
    assert abs(_difference(lambda v: f(x, v), w, e) - (dw * e).sum()) < 1e-7


def test_reference_rotation_keeps_angles_between_positions():
    gen = torch.Generator().manual_seed(1)
    q, k = (torch.randn((1, 1, 64), generator=gen, dtype=torch.float64).expand(4, 1, 64) for _ in range(2))
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    for pairs in (False, True):
        a, _ = ref.turned(q, torch.tensor([3, 10, 1000, 50000]), freq, pairs)
        b, _ = ref.turned(k, torch.tensor([0, 7, 997, 49997]), freq, pairs)
        dots = (a * b).sum(-1)
        assert (dots - dots[0]).abs().max() < 1e-9
        back, _ = ref.turned(a, torch.tensor([3, 10, 1000, 50000]), freq, pairs, back=True)
        assert (back - q).abs().max() < 1e-9


@pytest.mark.parametrize("mix", [False, True])
def test_reference_scan_gradients_match_differences(mix):
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    cu = [0, 5, 5, 6, 17]
    x, g, init, dh, df = r(17, 3), -r(17, 3).abs(), r(4, 3), r(17, 3), r(4, 3)

    def f(x, g, init):
        o = ref.scan(x, g, cu, mix, init)
        return (o["h"] * dh).sum() + (o["final"] * df).sum()

    b = ref.scan_backward(x, g, cu, mix, init, dh, df)
    for name, got, args in (("x", b["dx"], lambda v: (v, g, init)), ("g", b["dg"], lambda v: (x, v, init)),
                            ("init", b["d_init"], lambda v: (x, g, v))):
        at = dict(x=x, g=g, init=init)[name]
        d = r(*at.shape)
        assert abs(_difference(lambda v: f(*args(v)), at, d) - (got * d).sum()) < 1e-7, name


def test_reference_scan_is_the_recurrence():
    x, g = torch.tensor([[1.0], [2.0], [4.0]], dtype=torch.float64), torch.log(torch.tensor([[0.5], [0.5], [0.25]], dtype=torch.float64))
    o = ref.scan(x, g, [0, 3], False, torch.tensor([[8.0]], dtype=torch.float64))
    assert torch.allclose(o["h"][:, 0], torch.tensor([5.0, 4.5, 5.125], dtype=torch.float64))
    o = ref.scan(x, g, [0, 1, 3], True, None)
    assert torch.allclose(o["h"][:, 0], torch.tensor([0.5, 1.0, 3.25], dtype=torch.float64))
