"""The serving calls on the host, without a GPU: exports, refusals with the
documented status codes before any memory is touched, workspace sizes, the
binding's own checks, and the plain 64-bit forms that the GPU tests compare
with (pinned by properties that do not go through the library)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_linear_amd as gdn
import serve_reference as ref

OK, INVALID, UNSUPPORTED, DOMAIN, OOM, HIPERR = range(6)
BAD = ctypes.c_void_p(0x1001)   # misaligned; never dereferenced because validation rejects it first
FAKE = ctypes.c_void_p(0x1000)  # aligned, and never dereferenced either
NUL = None


@pytest.fixture(scope="module")
def lib():
    return gdn.load_library()


def test_exports(lib):
    names = gdn.exported_symbols_in_header(gdn.SERVE_HEADER)
    assert set(names) == {"gdn_batch_tables", "gdn_batch_tables_workspace_bytes", "gdn_cache_write",
                          "gdn_cache_attention", "gdn_cache_attention_workspace_bytes", "gdn_decode_pool"}
    for n in names:
        assert hasattr(lib, n) and n in gdn.__all__ and hasattr(gdn, n), n


def _tables(lib, ctx=FAKE, new=FAKE, rows=NUL, n=4, T=10, page=64, table=FAKE, nr=4, mb=8, counts=FAKE, free=FAKE,
            pages=9, state=FAKE, cu=FAKE, kv=FAKE, slots=FAKE, pos=FAKE, ws=FAKE, wb=1 << 20):
    return lib.gdn_batch_tables(ctx, new, rows, n, T, page, table, nr, mb, counts, free, pages, state, cu, kv, slots, pos,
                                ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(nr=-1), INVALID),
    (dict(mb=-1), INVALID), (dict(pages=-1), INVALID), (dict(page=32), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
    (dict(ctx=NUL), INVALID), (dict(new=BAD), INVALID), (dict(rows=BAD), INVALID), (dict(table=NUL), INVALID),
    (dict(counts=BAD), INVALID), (dict(free=NUL), INVALID), (dict(state=NUL), INVALID), (dict(cu=NUL), INVALID),
    (dict(kv=NUL), INVALID), (dict(slots=NUL), INVALID), (dict(pos=BAD), INVALID), (dict(ws=NUL), INVALID),
    (dict(wb=4), INVALID)])
def test_tables_refusals(lib, kw, want):
    assert _tables(lib, **kw) == want


def _write(lib, k=FAKE, v=FAKE, slots=FAKE, T=3, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=4, page=64, hkv=2, dk=64,
           dv=128, dt=1):
    return lib.gdn_cache_write(k, v, slots, T, kc, vc, ks, vs, pages, page, hkv, dk, dv, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(pages=-1), INVALID), (dict(hkv=0), INVALID),
    (dict(hkv=40000), INVALID), (dict(dt=2), UNSUPPORTED), (dict(dk=96), UNSUPPORTED), (dict(dv=32), UNSUPPORTED),
    (dict(page=16), UNSUPPORTED), (dict(pages=(1 << 25) + 1), UNSUPPORTED), (dict(k=BAD), INVALID),
    (dict(v=NUL), INVALID), (dict(kc=BAD), INVALID), (dict(vc=NUL), INVALID), (dict(slots=NUL), INVALID),
    (dict(ks=BAD), INVALID), (dict(vs=NUL), INVALID), (dict(T=0, k=NUL), OK), (dict(pages=0, kc=NUL), OK)])
def test_write_refusals(lib, kw, want):
    assert _write(lib, **kw) == want


def _attention(lib, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, rows=NUL, kv=FAKE, cu=FAKE, n=2, T=4,
               max_new=0, max_kv=0, pages=5, page=64, nr=2, mb=4, scale=0.1, o=FAKE, H=4, hkv=2, dk=64, dv=64, dt=1,
               ws=FAKE, wb=1 << 30):
    return lib.gdn_cache_attention(q, kc, vc, ks, vs, table, rows, kv, cu, n, T, max_new, max_kv, pages, page, nr, mb,
                                   scale, o, H, hkv, dk, dv, dt, ws, wb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(max_new=-1), INVALID),
    (dict(max_kv=-1), INVALID), (dict(mb=-1), INVALID), (dict(H=5), INVALID), (dict(H=0), INVALID),
    (dict(hkv=0), INVALID), (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(dt=5), UNSUPPORTED), (dict(n=0), INVALID), (dict(T=1 << 30, H=64), UNSUPPORTED), (dict(nr=-1), INVALID),
    (dict(pages=-1), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(q=BAD), INVALID),
    (dict(o=NUL), INVALID), (dict(kv=NUL), INVALID), (dict(cu=BAD), INVALID), (dict(rows=BAD), INVALID),
    (dict(table=NUL), INVALID), (dict(kc=BAD), INVALID), (dict(vc=NUL), INVALID), (dict(ks=NUL), INVALID),
    (dict(vs=BAD), INVALID), (dict(T=0, n=0, q=NUL), OK), (dict(mb=4096, ws=NUL), INVALID),
    (dict(mb=4096, wb=16), INVALID)])
def test_attention_refusals(lib, kw, want):
    assert _attention(lib, **kw) == want


def _pool(lib, q=FAKE, k=FAKE, v=FAKE, g=FAKE, head=0, beta=FAKE, states=FAKE, slots=FAKE, cu=NUL, commit=NUL, n=3, T=3,
          ns=8, qs=1.0, eps=0.0, o=FAKE, H=4, hk=2, dk=64, dv=128, dt=1):
    return lib.gdn_decode_pool(q, k, v, g, head, beta, states, slots, cu, commit, n, T, ns, qs, eps, o, H, hk, dk, dv, dt,
                               None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(ns=-1), INVALID), (dict(H=3), INVALID), (dict(H=0), INVALID),
    (dict(hk=0), INVALID), (dict(dt=9), UNSUPPORTED), (dict(dk=32), UNSUPPORTED), (dict(dv=96), UNSUPPORTED),
    (dict(qs=math.nan), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.inf), INVALID), (dict(T=4), INVALID),
    (dict(n=0, T=4, cu=FAKE), INVALID), (dict(n=1 << 28, T=1 << 28, H=64, hk=64), UNSUPPORTED), (dict(q=BAD), INVALID),
    (dict(k=NUL), INVALID), (dict(v=BAD), INVALID), (dict(states=NUL), INVALID), (dict(o=BAD), INVALID),
    (dict(g=NUL), INVALID), (dict(beta=BAD), INVALID), (dict(slots=NUL), INVALID), (dict(cu=BAD), INVALID),
    (dict(commit=BAD), INVALID), (dict(n=0, T=0, q=NUL), OK), (dict(ns=0, states=NUL), OK)])
def test_pool_refusals(lib, kw, want):
    assert _pool(lib, **kw) == want


def test_workspace_sizes():
    assert gdn.gdn_batch_tables_workspace_bytes(-1, 4) == 0
    assert gdn.gdn_batch_tables_workspace_bytes(5, 4) > 0
    size = gdn.gdn_cache_attention_workspace_bytes
    assert size(1, 1, 0, 65536, 64, 1024, 32, 8, 128, 128) > 0   # a long cache and one row: cut into parts
    assert size(1, 0, 0, 65536, 64, 1024, 32, 8, 128, 128) == 0
    assert size(1, 1, 0, 65536, 63, 1024, 32, 8, 128, 128) == 0
    assert size(1, 1, 0, 0, 64, 1024, 32, 8, 128, 128) == size(1, 1, 0, 65536, 64, 1024, 32, 8, 128, 128)


def test_attention_workspace_of_last_tiles():
    # Tiles past a multiple of 512 workgroups are cut into parts.  One request that is such a multiple has none.
    size = gdn.gdn_cache_attention_workspace_bytes
    for T in (2048, 4096, 8192):
        for hint in (0, T):
            assert size(1, T, hint, 32768, 64, 512, 32, 8, 128, 128) == 0
            assert size(1, T + 1, hint, 32768, 64, 512, 32, 8, 128, 128) > 0
    # heads that do not divide 512: 312 tiles of 36 heads are 21 x 512 + 480, 313 are 22 x 512 + 4
    assert size(1, 4992, 0, 131072, 64, 2048, 288, 36, 128, 128) == 0
    # one tile's 36 workgroups cut into 14 parts, of at most two tiles' 32 tokens
    assert 0 < size(1, 5008, 0, 131072, 64, 2048, 288, 36, 128, 128) <= 14 * 32 * 288 * (128 + 2) * 4 + 512


def test_attention_workspace_is_bounded():
    # of few rows at most 16384 workgroups of 16 rows, of many at most 1024 of 128 and as many that they share a tile with
    rng = np.random.RandomState(7)
    most = (16384 * 16 + 2 * 1024 * 128) * (128 + 2) * 4 + 2048
    for _ in range(20000):
        hkv, G = int(rng.choice([1, 2, 3, 5, 8, 12, 16, 36, 40, 100, 300])), int(rng.choice([1, 2, 4, 7, 8, 16]))
        n = int(2 ** rng.uniform(0, 9))
        T = max(n, int(2 ** rng.uniform(0, 14)))
        blocks = int(2 ** rng.uniform(0, 12))
        hint = int(rng.choice([0, 1, 5, T // n, T]))
        assert gdn.gdn_cache_attention_workspace_bytes(n, T, hint, 0, 64, blocks, hkv * G, hkv, 128, 128) <= most, \
            (n, T, hint, blocks, hkv, G)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        gdn.gdn_cache_write(k, k, torch.zeros(3, dtype=torch.int32), torch.zeros(1, 2, 64, 64, dtype=ref.E4M3),
                            torch.zeros(1, 2, 4, 64, 16, dtype=ref.E4M3), torch.ones(1, 2), torch.ones(1, 2))
    with pytest.raises(ValueError):
        gdn.gdn_decode_pool(k, k, k, torch.zeros(3, 2, 64), torch.zeros(3, 2), torch.zeros(4, 2, 64, 64),
                            torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.gdn_cache_attention(k.half(), *[None] * 7)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_batch_tables(i, i, 0, 64, torch.zeros(3, 4, dtype=torch.int32), i, i, i)


def test_binding_refuses_a_stream_of_another_device():
    # else the call would run on its own device's current stream, not ordered behind the stream it was given
    class Stream:
        device_index = 1

    with pytest.raises(ValueError):
        gdn.serve._On(0, Stream())
    Stream.device_index = 0
    try:
        gdn.serve._On(0, Stream())
    except ValueError:
        pytest.fail("a stream of the same device is refused")
    except (AssertionError, RuntimeError):
        pass  # without a device


# ---------------------------------------------------------------- the plain forms themselves


def test_reference_rounding_matches_the_format():
    # every e4m3 value is its own nearest, midpoints go to the even code, and torch's conversion agrees
    codes = torch.arange(256, dtype=torch.uint8).view(ref.E4M3).double().numpy()
    fine = codes[np.isfinite(codes)]
    assert np.array_equal(ref.nearest_e4m3(fine), fine)
    x = np.random.RandomState(0).standard_normal(20000) * np.exp2(np.random.RandomState(1).uniform(-12, 7, 20000))
    x = x.astype(np.float32).astype(np.float64)
    assert np.array_equal(ref.nearest_e4m3(x), torch.tensor(x, dtype=torch.float32).to(ref.E4M3).double().numpy())
    up = np.sort(np.unique(np.abs(fine)))
    mid = (up[1:] + up[:-1]) / 2
    assert np.array_equal(ref.nearest_e4m3(mid), torch.tensor(mid, dtype=torch.float32).to(ref.E4M3).double().numpy())


@pytest.mark.parametrize("amax,want", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.00003, 2.0), (1.0, 2.0 ** -8),
                                       (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (3e38, 2.0 ** 120), (1e-40, 2.0 ** -100)])
def test_reference_scale(amax, want):
    assert ref.page_scale(float(np.float32(amax))) == want


def test_reference_tables_keep_the_pages():
    # whatever is taken, refused and given back, every page is in one row or in the ring, once
    rng = np.random.RandomState(3)
    for _ in range(50):
        n, page, pages = rng.randint(1, 9), 64, rng.randint(1, 40)
        blocks = rng.randint(1, 9)
        counts = [0] * n
        table = [[-1] * blocks for _ in range(n)]
        free, state = list(rng.permutation(pages)), [int(rng.randint(pages)), pages, 0]
        free = [int(x) for x in np.roll(free, state[0])]
        ctx = [0] * n
        for _ in range(6):
            new = [int(x) for x in rng.randint(-1, 200, n)]
            cu, kv, slots, pos = ref.tables(ctx, new, None, max(0, sum(x for x in new if x > 0)), page, table, counts, free, state)
            held = [table[r][j] for r in range(n) for j in range(counts[r])]
            ring = [free[(state[0] + i) % pages] for i in range(state[1])]
            assert sorted(held + ring) == list(range(pages))
            assert all(0 <= s for n_ in range(n) if kv[n_] > ctx[n_] for s in slots[cu[n_]:cu[n_ + 1]])
            ctx = kv
