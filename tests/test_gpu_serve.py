"""GPU parity of the serving calls with plain 64-bit forms (tests/serve_reference.py):
batch tables, the paged 8-bit cache, attention over it, the delta rule on a pool
of states, and the calls together as a server makes them."""

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_linear_amd as gdn
import serve_reference as ref
from gated_delta_rule_linear_amd import inputs
from helpers import log, np64

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -24  # half a step of fp32, relative
EPS16 = 2.0 ** -8   # of bf16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- tables


def _tables_case(seed, n, page, blocks, pages, lo, hi, enders=0, look=0, odd_rows=False, null_rows=False):
    """Requests with contexts that fit their pages; pages in the ring's middle."""
    r = np.random.RandomState(seed)
    num_rows = n if null_rows else n + 3
    rows = list(range(n)) if null_rows else [int(x) for x in r.permutation(num_rows)[:n]]
    counts, table = [0] * num_rows, [[-1] * blocks for _ in range(num_rows)]
    order = [int(x) for x in r.permutation(pages)]
    ctx = []
    for row in rows:
        own = int(min(r.randint(0, blocks + 1), max(0, len(order) - 2)))
        for j in range(own):
            table[row][j] = order.pop()
        counts[row] = own
        ctx.append(int(r.randint(max(0, (own - 1 - look)) * page, own * page + 1)) if own else 0)
    head = int(r.randint(pages)) if pages else 0
    free = [-7] * pages
    for i, p in enumerate(order):
        free[(head + i) % pages] = p
    new = [int(x) for x in r.randint(lo, hi + 1, n)]
    for i in r.permutation(n)[:enders]:
        new[i] = -int(r.randint(1, 5))
    if odd_rows and n > 2:
        rows[0], rows[1] = -1, num_rows + 5
    return ctx, new, None if null_rows else rows, table, counts, free, [head, len(order), 0]


TABLES = [
    dict(n=1, page=64, blocks=4, pages=5, lo=1, hi=1), dict(n=0, page=64, blocks=4, pages=5, lo=1, hi=1),
    dict(n=7, page=128, blocks=3, pages=40, lo=0, hi=3, enders=2, look=2),
    dict(n=70, page=64, blocks=6, pages=150, lo=0, hi=300, enders=9, look=1, odd_rows=True),  # pages run out
    dict(n=33, page=256, blocks=2, pages=200, lo=0, hi=700, null_rows=True),                   # rows run out of room
    dict(n=5, page=64, blocks=3, pages=0, lo=1, hi=9),                                         # no page at all
    dict(n=1025, page=64, blocks=3, pages=4000, lo=1, hi=2, enders=100),                       # two turns of the sums
    dict(n=5000, page=64, blocks=2, pages=9000, lo=0, hi=4, enders=500, odd_rows=True),        # a second launch
    dict(n=64, page=64, blocks=300, pages=21000, lo=512, hi=16384),                            # prompts
    dict(n=3, page=64, blocks=0, pages=4, lo=0, hi=2),                                         # rows without room
]


@pytest.mark.parametrize("case", TABLES)
@pytest.mark.parametrize("extra", [0, 5, -3])
def test_tables(case, extra):
    log(f"tables {case} T_total {extra:+d}")
    ctx, new, rows, table, counts, free, state = _tables_case(n_seed(case), **case)
    T = max(0, sum(x for x in new if x > 0) + extra)
    d = dict(table=i32(table).reshape(len(counts), -1), counts=i32(counts), free=i32(free), state=i32(state))
    for again in range(2):
        got = gdn.gdn_batch_tables(i32(ctx), i32(new), T, case["page"], d["table"], d["counts"], d["free"], d["state"],
                                   rows=None if rows is None else i32(rows))
        want = ref.tables(ctx, new, rows, T, case["page"], table, counts, free, state)
        for name, x, y in zip(("cu_seqlens", "kv_lens", "slots", "positions"), got, want):
            assert x.tolist() == y, (name, again)
        assert d["counts"].tolist() == counts and d["free"].tolist() == free and d["state"].tolist() == state
        assert d["table"].tolist() == table


def n_seed(case):
    return case["n"] * 31 + case["page"] + case["hi"]


def test_tables_called_again():
    # one page, held by a request that ends: the other is refused, and finds it free in the next call with the same
    # lengths; from then on, as always where none is refused, a repeat changes nothing
    for extra in (0, 3000):  # in one launch and in two
        ctx, new, T = [64, 0], [-1, 5], 5 + extra
        table, counts, free, state = [[0], [-1]], [1, 0], [-9], [0, 0, 0]
        d = [i32(table), i32(counts), i32(free), i32(state)]
        seen = []
        for _ in range(3):
            got = gdn.gdn_batch_tables(i32(ctx), i32(new), T, 64, *d)
            want = ref.tables(ctx, new, None, T, 64, table, counts, free, state)
            assert [x.tolist() for x in got] == list(want) and [x.tolist() for x in d] == [table, counts, free, state]
            seen.append([x.tolist() for x in list(got) + d])
        assert seen[0][2][:5] == [-1] * 5 and seen[0][7] == [0, 1, 1] and seen[0][1] == [0, 0]
        assert seen[1][2][:5] == [0, 1, 2, 3, 4] and seen[1][7] == [0, 0, 0] and seen[1][4] == [[-1], [0]]
        assert seen[2] == seen[1]


def test_tables_long_request():
    # one request of 2^20 tokens: positions and slots far from zero
    T, page = 1 << 20, 64
    pages = T // page + 3
    table, counts = torch.full((1, T // page), -1, dtype=torch.int32, device="cuda"), i32([0])
    ring = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).contiguous()
    cu, kv, slots, pos = gdn.gdn_batch_tables(i32([0]), i32([T]), T, page, table, counts, ring, i32([pages - 1, pages, 0]))
    assert cu.tolist() == [0, T] and kv.tolist() == [T] and counts.tolist() == [T // page]
    assert torch.equal(pos, torch.arange(T, dtype=torch.int32, device="cuda"))
    at = torch.cat([ring[-1:], ring[:-1]])[:T // page]
    assert torch.equal(table[0], at)
    assert torch.equal(slots.view(-1, page), at[:, None] * page + torch.arange(page, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- cache write


def _write_check(k, v, slots, kc, vc, ks, vs):
    """Runs the call and the plain form on copies and compares every code and scale."""
    kr, vr = kc.float().double().cpu().numpy(), ref.tokens_of(vc.float()).double().cpu().numpy()
    ksr, vsr = ks.double().cpu().numpy(), vs.double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref.write(np64(k), slots, kr, ksr)
        ref.write(np64(v), slots, vr, vsr)
    gdn.gdn_cache_write(k, v, i32(slots), kc, vc, ks, vs)
    assert np.array_equal(ks.double().cpu().numpy(), ksr) and np.array_equal(vs.double().cpu().numpy(), vsr)
    assert np.array_equal(kc.float().double().cpu().numpy(), kr, equal_nan=True)
    assert np.array_equal(ref.tokens_of(vc.float()).double().cpu().numpy(), vr, equal_nan=True)


def _pool_of_pages(gen, pages, hkv, page, dk, dv):
    kc = (torch.randn((pages, hkv, page, dk), generator=gen) * 50).clamp(-448, 448).to(ref.E4M3).cuda()
    vc = (torch.randn((pages, hkv, page // 16, dv, 16), generator=gen) * 50).clamp(-448, 448).to(ref.E4M3).cuda()
    ks, vs = (torch.exp2(torch.randint(-9, -3, (pages, hkv), generator=gen).float()).cuda() for _ in range(2))
    return kc, vc, ks, vs


@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write(page, dk, dv, dtype):
    log(f"write page={page} dk={dk} dv={dv} {dtype}")
    gen = torch.Generator().manual_seed(page + dk + 2 * dv)
    hkv, pages = 3, 14
    cache = _pool_of_pages(gen, pages, hkv, page, dk, dv)
    order = torch.randperm(pages, generator=gen).tolist()
    slots = []
    # runs of one token, at a page's start, its end, inside, whole pages and a skipped one
    for a, b in [(0, 1), (page - 1, page), (5, 6), (0, page), (17, 49), (16, 32), (0, 20), (page - 30, page), (3, 3),
                 (33, 63), (0, page - 1)]:
        p = order.pop()
        slots += [p * page + i for i in range(a, b)] + ([-1] if a == 17 else [])
    slots += [pages * page, -5, 2 ** 31 - 1]
    T = len(slots)
    k = (torch.randn((T, hkv, dk), generator=gen) * torch.exp2(torch.randint(-6, 6, (T, 1, 1), generator=gen).float()))
    v = (torch.randn((T, hkv, dv), generator=gen) * torch.exp2(torch.randint(-6, 6, (T, 1, 1), generator=gen).float()))
    _write_check(k.to(dtype).cuda(), v.to(dtype).cuda(), slots, *cache)


@pytest.mark.parametrize("T,hkv", [(1, 1), (511, 8), (4097, 2)])
def test_write_sizes(T, hkv):
    # single tokens of many requests (T = 511) and long runs
    gen = torch.Generator().manual_seed(T)
    page, pages = 64, 520 if T == 511 else T // 64 + 3
    cache = _pool_of_pages(gen, pages, hkv, page, 128, 128)
    order = torch.randperm(pages, generator=gen)
    if T == 511:
        slots = (order[:T] * page + torch.randint(0, page, (T,), generator=gen)).tolist()
    else:
        i = torch.arange(T) + 7
        slots = (order[i // page] * page + i % page).tolist()
    k, v = (torch.randn((T, hkv, 128), generator=gen).bfloat16().cuda() for _ in range(2))
    _write_check(k, v, slots, *cache)


@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("longest", [6, 90, 700])
def test_write_many_runs(page, longest):
    # runs of all lengths, some over several pages, so many that a workgroup takes more than one of them
    gen = torch.Generator().manual_seed(page + longest)
    hkv, slots = 8, []
    T, pages = (1500, 640) if longest == 6 else (2900, 150)
    order = torch.randperm(pages, generator=gen).tolist()
    while len(slots) < T:
        n = int(torch.randint(1, longest + 1, (1,), generator=gen))
        at = int(torch.randint(0, page, (1,), generator=gen))
        while n:
            m = min(n, page - at)
            p = order.pop()
            slots += [p * page + at + i for i in range(m)]
            n, at = n - m, 0
    cache = _pool_of_pages(gen, pages, hkv, page, 64, 64)
    k, v = (torch.randn((len(slots), hkv, 64), generator=gen).bfloat16().cuda() for _ in range(2))
    _write_check(k, v, slots, *cache)


def test_write_values_at_the_borders():
    # zeros, subnormals, the largest values, Inf and NaN, ties between codes, a scale that grows by 2^200
    gen = torch.Generator().manual_seed(4)
    cache = _pool_of_pages(gen, 6, 2, 64, 64, 64)
    cache[2][2:4] = 2.0 ** -100
    k = torch.randn((9, 2, 64), generator=gen)
    k[0] = 0.0
    k[1] = 1e-40
    k[2] = 3e38
    k[3, :, 3] = math.inf
    k[4, 0, 5] = math.nan
    k[5, :, 7] = -math.inf
    k[6] = torch.arange(64).float() + 0.5  # ties
    k[7] = math.nan
    k[8] = 448 * 2.0 ** 40
    slots = [0, 65, 2 * 64 + 9, 3 * 64, 3 * 64 + 1, 3 * 64 + 2, 4 * 64, 5 * 64, 5 * 64 + 1]
    _write_check(k.cuda(), k.clone().cuda(), slots, *cache)


def test_write_leaves_the_rest():
    gen = torch.Generator().manual_seed(9)
    cache = _pool_of_pages(gen, 5, 2, 64, 128, 64)
    before = [t.clone() for t in cache]
    k, v = torch.randn(3, 2, 128).cuda(), torch.randn(3, 2, 64).cuda()
    gdn.gdn_cache_write(k, v, i32([2 * 64 + 8, 2 * 64 + 9, -1]), *cache)
    keep = [0, 1, 3, 4]
    for a, b in zip(cache, before):
        assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))


def test_write_and_read_far_into_a_large_cache():
    # byte offsets past 2^32 in both caches: 70000 pages of 64 tokens x 8 heads x 128
    pages, hkv, page = 70000, 8, 64
    kc = torch.zeros((pages, hkv, page, 128), dtype=torch.uint8, device="cuda").view(ref.E4M3)
    vc = torch.zeros((pages, hkv, page // 16, 128, 16), dtype=torch.uint8, device="cuda").view(ref.E4M3)
    ks, vs = (torch.ones((pages, hkv), device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(2)
    k, v = (torch.randn((70, hkv, 128), generator=gen).bfloat16().cuda() for _ in range(2))
    at = [pages - 1, pages - 7]
    slots = [at[i // page] * page + i % page for i in range(70)]
    gdn.gdn_cache_write(k, v, i32(slots), kc, vc, ks, vs)
    small = [kc[at].clone(), vc[at].clone(), ks[at].clone(), vs[at].clone()]
    q = torch.randn((1, 16, 128), generator=gen).bfloat16().cuda()
    far = gdn.gdn_cache_attention(q, kc, vc, ks, vs, i32([at]), i32([70]), i32([0, 1]))
    near = gdn.gdn_cache_attention(q, *small, i32([[0, 1]]), i32([70]), i32([0, 1]))
    assert torch.equal(far, near)
    assert (k - (small[0].float() * small[2][..., None, None]).transpose(1, 2).reshape(-1, hkv, 128)[:70]).abs().max() \
        <= k.abs().max() * 2.0 ** -4


# ---------------------------------------------------------------- attention


def _attention_check(server, lens, H, dtype, seed=0, scale=None, T_extra=0, **kw):
    gen = torch.Generator().manual_seed(seed + 100)
    dk, dv = server.k.shape[3], server.v.shape[3]
    T = sum(lens)
    q = torch.randn((T + T_extra, H, dk), generator=gen).to(dtype)
    scale = dk ** -0.5 if scale is None else scale
    cu = i32([0] + list(np.cumsum(lens)))
    kc, vc, ks, vs, table, kv_lens, rows = server.to("cuda")
    o = torch.full((T + T_extra, H, dv), 7.0, dtype=dtype, device="cuda")
    got = gdn.gdn_cache_attention(q.cuda(), kc, vc, ks, vs, table, kv_lens, cu, rows=rows, scale=scale, o=o, **kw)
    assert got is o and torch.all(o[T:] == 7.0)  # rows behind the last request
    want, mag, big = server.reference(q[:T].double().cuda(), lens, scale, "cuda")
    got = o[:T].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    # Scores: dk + 4 fp32 roundings of sum |q||k| (three of them for each of the
    # split parts of fp32 q), and the exponential and its argument in base 2.  p
    # is off by twice that (numerator and denominator), the sums over S tokens by
    # at most S roundings each of sum p|v|; p itself is rounded once to the
    # type's bf16 parts (three: 2^-24), o once to its type.
    S = max([1] + [int(x) for x in server.kv_lens])
    parts, half = (3, EPS32) if dtype == torch.float32 else (1, EPS16)
    score = (parts * (dk + 4) + 8) * EPS32 * big
    tol = (2 * score + 2 * (S + 64) * EPS32 + half + 16 * EPS32) * mag + half * want.abs() + 1e-30
    bad = (got - want).abs() > torch.where(torch.isnan(want), math.inf, tol)
    err = torch.nan_to_num((got - want).abs() / tol, nan=0.0).max().item() if T else 0.0
    log(f"  attention: largest error / tolerance {err:.3f}")
    assert not bad.any(), err
    return o


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("page,hkv,group", [(64, 2, 1), (128, 1, 7), (256, 2, 4), (64, 1, 20)])
def test_attention(dtype, dk, dv, page, hkv, group):
    kv = [1, 63, 64, 65, 300, 0, 1027, 129]
    lens = [1, 5, 1, 65, 17, 0, 1, 40]
    log(f"attention kv={kv} new={lens} page={page} H_kv={hkv} G={group} dk={dk} dv={dv} {dtype}")
    _attention_check(ref.Server(kv, page, hkv, dk, dv, seed=dk + page, rows=True), lens, hkv * group, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("max_kv", [0, 20000, 100])
def test_attention_parts(dtype, max_kv):
    # one token each, caches of very different lengths: cut into parts and joined
    log(f"attention in parts {dtype} max_kv={max_kv}")
    _attention_check(ref.Server([20000, 1, 0, 511, 8193], 64, 2, 128, 128, seed=5), [1, 1, 1, 1, 1], 8, dtype,
                     max_new=1, max_kv=max_kv)


@pytest.mark.parametrize("lens,kv", [([700], [700]), ([300, 1, 129], [5000, 4096, 129]), ([1, 600, 1], [1000, 600, 3]),
                                     ([257], [9000])])
@pytest.mark.parametrize("dtype,dk,dv", [(torch.bfloat16, 128, 128), (torch.bfloat16, 64, 128),
                                         (torch.float32, 128, 64), (torch.float32, 64, 64)])
def test_attention_prompts(lens, kv, dtype, dk, dv):
    log(f"attention prompts new={lens} kv={kv} {dtype} dk={dk} dv={dv}")
    _attention_check(ref.Server(kv, 64, 2, dk, dv, seed=kv[0]), lens, 8, dtype, max_new=max(lens), max_kv=max(kv))


@pytest.mark.parametrize("lens,kv,hints", [
    ([1027], [4000], {}), ([500, 1, 530, 3], [3100, 5000, 3700, 40], dict(max_new=530, max_kv=5000)),
    # few held tokens in front of them, and none
    ([1027], [4000], dict(max_new=1027, max_kv=1027)), ([1040], [1040], dict(max_new=1, max_kv=9000))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_last_tiles_in_parts(lens, kv, hints, dtype):
    # a few more tiles of rows than the device holds at once, over a long cache
    log(f"attention: last tiles in parts new={lens} kv={kv} {hints} {dtype}")
    _attention_check(ref.Server(kv, 64, 16, 64, 64, seed=23), lens, 64, dtype, T_extra=3, **hints)


def test_attention_last_tiles_with_offsets_that_are_none():
    # offsets that start below 0 or decrease: nothing outside o is written, and the workspace is enough
    s = ref.Server([4000, 300], 64, 16, 64, 64, seed=23)
    kc, vc, ks, vs, table, kv_lens, _ = s.to("cuda")
    q = torch.randn((1030, 64, 64)).bfloat16().cuda()
    need = gdn.gdn_cache_attention_workspace_bytes(2, 1030, 0, 0, 64, table.shape[1], 64, 16, 64, 64)
    for cu in ([-5000, 1030, 1030], [0, 1030, 7], [900, 20, 1030], [-3, 10 ** 9, -7], [2000, 2000, 2000]):
        ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
        room = torch.full((1030 + 64, 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_cache_attention(q, kc, vc, ks, vs, table, kv_lens, i32(cu), o=room[:1030], workspace=ws[:need])
        assert torch.all(ws[need:] == 77) and torch.all(room[1030:] == 7.0)


@pytest.mark.parametrize("lens,kv,hints", [([2, 1, 70, 0], [9000, 5, 300, 7], dict(max_new=1, max_kv=64)),
                                           ([2, 3], [9000, 40000], dict(max_new=1)),
                                           ([1, 1], [9000, 40000], dict(max_new=500)),
                                           ([300], [700], dict(max_new=1, max_kv=1)), ([5], [70000], dict())])
def test_attention_hints_are_only_hints(lens, kv, hints):
    log(f"attention new={lens} kv={kv} hints {hints}")
    _attention_check(ref.Server(kv, 128, 2, 64, 64, seed=11), lens, 8, torch.bfloat16, **hints)


@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [3, 70, 1, 200]])
def test_attention_rows_that_see_nothing(lens):
    # more new tokens than tokens held, an empty cache, a padded batch
    log(f"attention: rows without a token {lens}")
    o = _attention_check(ref.Server([0, 64, 2, 9], 64, 1, 64, 64, seed=8), lens, 4, torch.bfloat16, T_extra=6)
    assert torch.all(o[:lens[0]] == 0)


@pytest.mark.parametrize("lens", [[1, 1, 1], [2, 130, 90]])
def test_attention_bad_pages(lens):
    # entries outside the pool, and a request whose row is outside the table, are left out
    s = ref.Server([300, 513, 200], 64, 2, 64, 128, seed=3, rows=True)
    s.table[int(s.rows[0]), 1] = -1
    s.table[int(s.rows[1]), 0] = 10 ** 9
    s.table[int(s.rows[1]), 8] = s.k.shape[0]
    s.rows[2] = 40
    o = _attention_check(s, lens, 4, torch.bfloat16)
    assert torch.all(o[sum(lens[:2]):] == 0)


def test_attention_length_past_the_table():
    s = ref.Server([190], 64, 1, 64, 64, seed=3)
    s.table = s.table[:, :2].contiguous()
    s.kv_lens = [10 ** 6]
    _attention_check(s, [1], 2, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[1, 1], [6, 9], [100, 120]])
def test_attention_nan(dtype, lens):
    # NaN in keys or values of a token reaches the rows that see it, and codes behind the last token reach none
    s = ref.Server([150, 200], 64, 2, 128, 128, seed=6)
    c = s.v.view(torch.uint8)
    last = s.table[0, 2]
    c[last, :, 150 - 128:] = 0x7f
    s.k.view(torch.uint8)[last, :, 150 - 128:] = 0xff
    p = s.table[1]
    c[p[3], 1, 199 - 192, 5] = 0xff        # the last token's value, one channel
    c[p[3], 0, 195 - 192, 17] = 0x7f
    c[p[1], 1, 3, 100] = 0x7f              # a token in the middle
    log(f"attention NaN {dtype} {lens}")
    o = _attention_check(s, lens, 8, dtype)
    assert not torch.isnan(o[:lens[0]]).any()
    k = s.k.view(torch.uint8)
    k[p[3], 0, 197 - 192, 9] = 0x7f        # a key: every channel of the rows that see it
    want = torch.isnan(s.reference(torch.randn((sum(lens), 8, 128), dtype=torch.float64), lens, 0.1)[0])
    kc, vc, ks, vs, table, kv_lens, _ = s.to("cuda")
    o = gdn.gdn_cache_attention(torch.randn((sum(lens), 8, 128)).to(dtype).cuda(), kc, vc, ks, vs, table, kv_lens,
                                i32([0, lens[0], sum(lens)]))
    assert torch.equal(torch.isnan(o).cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("kv,rise", [(200, 1), (200, 2), (700, 1), (700, 4), (3000, 1), (3000, 3)])
def test_attention_far_apart_scores(dtype, dk, dv, kv, rise):
    # Up to tile `rise` of 64 tokens, scores of every other 16 tokens are so far below the others' that their
    # exponentials are 0 (they are all the tokens that one lane has of a row); then the maximum rises, once.
    log(f"attention: scores far apart kv={kv} rise={rise} {dtype} dk={dk} dv={dv}")
    s = ref.Server([kv], 64, 1, dk, dv, seed=kv)
    s.ks[:] = 1.0
    k = torch.zeros((s.k.shape[0], 1, 64, dk))
    low = (torch.arange(64) // 16) % 2 == 1
    for b, page in enumerate(s.table[0, :-(-kv // 64)].tolist()):
        k[page, 0, :, 0] = torch.where(low, -448.0, 0.0) if b < rise else 8.0   # rows with q0 > 0
        k[page, 0, :, 1] = torch.where(low, 0.0, -448.0) if b < rise else 8.0   # q1 > 0: the other 16 tokens
    s.k = k.to(ref.E4M3)
    _attention_check(s, [60], 4, dtype, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,kv,hints", [([1, 1, 1, 1], [3000, 70, 0, 64], {}), ([3, 1, 2, 1], [130, 70, 1, 64], {}),
                                           ([70, 90, 1, 33], [3000, 90, 0, 1000], {}),
                                           ([200, 40], [3000, 9000], dict(max_new=200, max_kv=9000))])
def test_attention_infinite_queries(dtype, lens, kv, hints):
    # Inf in a query: its scores are Inf, -Inf or both, and the row NaN, unless it sees no token; other rows are as ever
    log(f"attention: Inf in queries new={lens} kv={kv} {dtype}")
    s = ref.Server(kv, 64, 2, 64, 64, seed=sum(kv))
    k = s.k.float()
    k[..., 0] = k[..., 0].abs().clamp(min=1.0)  # of one sign
    s.k = k.to(ref.E4M3)
    s.table[0, 0] = -1
    gen = torch.Generator().manual_seed(sum(lens))
    T, H = sum(lens), 8
    q = torch.randn((T, H, 64), generator=gen)
    odd = torch.rand((T, H), generator=gen) < 0.5
    ends = torch.tensor(np.cumsum(lens)) - 1
    odd[ends, 0], odd[ends, 1], odd[ends, 2] = True, True, False
    q[..., 0] = torch.where(odd, torch.where(torch.rand((T, H), generator=gen) < 0.7, -math.inf, math.inf), q[..., 0])
    q[ends, 0, 0] = -math.inf
    q = q.to(dtype).cuda()
    want, mag, _ = s.reference(q.double(), lens, 0.125, "cuda")
    kc, vc, ks, vs, tab, kv_lens, _ = s.to("cuda")
    o = gdn.gdn_cache_attention(q, kc, vc, ks, vs, tab, kv_lens, i32([0] + list(np.cumsum(lens))), scale=0.125, **hints)
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    # the other rows: p and o rounded to bf16 (or 2^-24, with the sums' roundings), scores below 2^5 off by their sums
    eps = EPS16 if dtype == torch.bfloat16 else EPS32 * (max(kv) + 64)
    calm = ~odd.cuda()
    assert ((o.double() - want).abs()[calm] <= (3 * eps + 2 * 200 * EPS32 * 2 ** 6) * (mag + want.abs())[calm] + 1e-30).all()


def _gaps(s, gaps):
    """Without the pages of these blocks of the first request."""
    row = 0 if s.rows is None else int(s.rows[0])
    s.table[row, gaps] = -1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("gaps", [[7], [8], [0], [60], [61], [62], [63], [64], [65], [3, 4, 59, 66, 67, 100, 129],
                                  list(range(20, 90))])
def test_attention_prompt_with_gaps(dtype, dk, dv, gaps):
    # pages left out of the tiles that every row sees whole, at even and odd tiles and around every 64th
    log(f"attention: a chunk with gaps {gaps} {dtype} dk={dk} dv={dv}")
    for kv, lens, hints in (([9000], [150], {}), ([9000, 300], [150, 40], dict(max_new=150, max_kv=9000))):
        s = ref.Server(kv, 64, 1, dk, dv, seed=gaps[0])
        _gaps(s, gaps)
        _attention_check(s, lens, 4, dtype, **hints)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,gaps", [(64, []), (128, [1, 5]), (256, [0])])
def test_attention_prompt_nan_early(dtype, page, gaps):
    # NaN codes in tiles that every row sees whole: a value's channel, and a key (every channel of its head)
    log(f"attention: NaN early {dtype} page={page} gaps={gaps}")
    for where in ("value", "key"):
        s = ref.Server([5000, 700], page, 2, 128, 128, seed=page)
        codes = (s.v if where == "value" else s.k).view(torch.uint8)
        codes[s.table[0, gaps].long(), 0, 5, 3] = 0xff  # in a page that is left out it reaches none
        _gaps(s, gaps)
        codes[int(s.table[0, 3]), 1, 9, 77] = 0x7f
        lens = [150, 60]
        want = torch.isnan(s.reference(torch.ones((210, 8, 128), dtype=torch.float64), lens, 0.1)[0])
        kc, vc, ks, vs, tab, kv_lens, _ = s.to("cuda")
        q = torch.randn((210, 8, 128), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        o = gdn.gdn_cache_attention(q, kc, vc, ks, vs, tab, kv_lens, i32([0, 150, 210]))
        assert want.any() and not want.all() and torch.equal(torch.isnan(o).cpu(), want)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scale(scale):
    _attention_check(ref.Server([150, 20], 64, 2, 64, 64, seed=1), [1, 20], 4, torch.float32, scale=scale)


@pytest.mark.parametrize("max_kv", [0, 40000])
def test_attention_one_long_request_among_many(max_kv):
    # enough workgroups without parts, and one cache of several parts beside short ones
    log(f"attention: 40000 tokens beside 35 short requests, max_kv={max_kv}")
    kv = [1 + 7 * i for i in range(35)] + [40000]
    _attention_check(ref.Server(kv, 256, 8, 64, 64, seed=19), [1] * 36, 8, torch.bfloat16, max_new=1, max_kv=max_kv)


def test_attention_of_nothing():
    # no tokens, no requests, no pages, no table: rows that are there are 0
    def call(T, n, pages, rows, blocks, cu):
        kc = torch.zeros((pages, 2, 64, 64), dtype=torch.uint8, device="cuda").view(ref.E4M3)
        vc = torch.zeros((pages, 2, 4, 64, 16), dtype=torch.uint8, device="cuda").view(ref.E4M3)
        ks, vs = (torch.ones((pages, 2), device="cuda") for _ in range(2))
        table = torch.zeros((rows, blocks), dtype=torch.int32, device="cuda")
        return gdn.gdn_cache_attention(torch.ones((T, 4, 64), device="cuda"), kc, vc, ks, vs, table, i32([7] * n), i32(cu))

    assert call(0, 0, 2, 1, 1, [0]).shape == (0, 4, 64)
    assert call(0, 2, 2, 2, 1, [0, 0, 0]).shape == (0, 4, 64)
    for T, pages, rows, blocks in ((1, 0, 1, 1), (40, 0, 1, 1), (1, 2, 0, 1), (40, 2, 0, 1), (1, 2, 1, 0), (40, 2, 1, 0)):
        assert torch.count_nonzero(call(T, 1, pages, rows, blocks, [0, T])) == 0


def test_attention_many_requests():
    r = np.random.RandomState(0)
    kv = [int(x) for x in r.randint(0, 200, 300)]
    lens = [int(min(x, y)) for x, y in zip(kv, r.randint(0, 4, 300))]
    log("attention: 300 requests")
    _attention_check(ref.Server(kv, 64, 1, 64, 64, seed=2), lens, 3, torch.bfloat16)


# ---------------------------------------------------------------- pool


def _pool_inputs(lens, H, hk, dk, dv, dtype, head_gate, slots, extra, seed, unit):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q, k = torch.randn((T, hk, dk), generator=gen), torch.randn((T, hk, dk), generator=gen)
    if unit:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    v = torch.randn((T, H, dv), generator=gen)
    g = -torch.nn.functional.softplus(3 * torch.randn((T, H) if head_gate else (T, H, dk), generator=gen))
    beta = torch.sigmoid(torch.randn((T, H), generator=gen))
    states = 0.1 * torch.randn((max([-1] + slots) + 1 + extra, H, dk, dv), generator=gen)
    return [x.to(dtype) for x in (q, k, v)] + [g, beta, states]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("H,hk,head_gate,eps,commit", [(4, 4, False, 0.0, None), (6, 2, True, 1e-6, [1, 0, 4, 2, -3, 1]),
                                                       (3, 1, False, 1e-6, [9, 1, 2, 1, 3, 1])])
def test_pool(dtype, dk, dv, H, hk, head_gate, eps, commit):
    lens, slots = [1, 0, 4, 2, 3, 7], [5, 0, 3, -1, 8, 1]
    log(f"pool lens={lens} H={H} H_k={hk} dk={dk} dv={dv} {dtype} head_gate={head_gate} eps={eps} commit={commit}")
    args = _pool_inputs(lens, H, hk, dk, dv, dtype, head_gate, slots, 2, dk + H, eps == 0.0)
    cu = [0] + [int(x) for x in np.cumsum(lens)]
    _pool_check(args, slots, cu, commit, eps, skipped=3)


def _pool_check(args, slots, cu, commit, eps, skipped=None, null_cu=False):
    d = [t.cuda() for t in args]
    dtype, dk, T = args[0].dtype, args[0].shape[2], args[0].shape[0]
    o = torch.full((T, args[2].shape[1], args[2].shape[2]), 3.0, dtype=dtype, device="cuda")
    gdn.gdn_decode_pool(*d, i32(slots), cu_seqlens=None if null_cu else i32(cu),
                        commit=None if commit is None else i32(commit), q_scale=0.7, l2_eps=eps, o=o)
    wo, ws, bo, bs = ref.pool(*[t.double().cuda() for t in args], slots, cu, commit, 0.7, eps)
    # Each token adds at most dk + 16 fp32 roundings of the recurrence of
    # magnitudes (sums over dk rows, the gate's exponential, the norms' factors);
    # the hardware exponential is good to 2 steps plus its argument's |g| / ln 2.
    steps = max([1] + [b - a for a, b in zip(cu, cu[1:])])
    c = steps * (dk + 16 + 2 * 2 * args[3].abs().max().item()) * EPS32
    got_o, got_s = o.double(), d[5].double()
    for n, slot in enumerate(slots):
        if n == skipped:
            assert torch.all(o[cu[n]:cu[n + 1]] == 3.0)
            wo[cu[n]:cu[n + 1]], bo[cu[n]:cu[n + 1]] = 3.0, 0.0
    half = EPS16 if dtype == torch.bfloat16 else 0.0
    eo = ((got_o - wo).abs() / (c * bo + half * wo.abs() + 1e-30)).max().item() if T else 0.0
    es = ((got_s - ws).abs() / (c * bs + 1e-30)).max().item()
    log(f"  pool: error / tolerance o {eo:.3f} states {es:.3f}")
    assert eo <= 1 and es <= 1
    untouched = [s for s in range(args[5].shape[0]) if s not in [x for n, x in enumerate(slots) if cu[n + 1] > cu[n]]]
    assert torch.equal(d[5][untouched].cpu(), args[5][untouched])


@pytest.mark.parametrize("N,H", [(1, 1), (1, 32), (129, 8)])
def test_pool_one_token_each(N, H):
    slots = [int(x) for x in np.random.RandomState(N).permutation(N + 3)[:N]]
    args = _pool_inputs([1] * N, H, H, 128, 128, torch.bfloat16, False, slots, 1, N, True)
    _pool_check(args, slots, list(range(N + 1)), None, 0.0, null_cu=True)


def test_pool_leaves_rows_behind_the_last_offset():
    # a batch padded to a fixed number of tokens: rows behind the offsets, and those of a skipped slot, keep what o held
    args = _pool_inputs([2, 1, 1, 3], 4, 2, 64, 64, torch.bfloat16, False, [1, 0, 2, 3], 0, 5, True)
    d = [t.cuda() for t in args]
    o = torch.full((7, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    before = d[5].clone()
    assert gdn.gdn_decode_pool(*d, i32([1, 9, 0]), cu_seqlens=i32([0, 2, 3, 4]), q_scale=0.7, o=o) is o
    assert torch.all(o[2:3] == 7.0) and torch.all(o[4:] == 7.0) and not torch.any(o[[0, 1, 3]] == 7.0)
    assert torch.equal(d[5][2:], before[2:])


def test_pool_many_tokens():
    # longer than a server's steps: the same recurrence
    args = _pool_inputs([200, 33], 2, 1, 64, 64, torch.float32, True, [1, 0], 0, 7, False)
    _pool_check(args, [1, 0], [0, 200, 233], [150, 33], 1e-6)


def test_pool_and_write_of_nothing():
    f = torch.ones
    q, v, g, b = (f((2, 2, 64), device="cuda") for _ in range(4))
    states, kept = (f((1, 2, 64, 64), device="cuda") for _ in range(2))
    o = torch.full((2, 2, 64), 7.0, device="cuda")
    gdn.gdn_decode_pool(q, q, v, -g, b[:, :, 0].contiguous(), states, i32([-1, 5]), o=o)  # no such states
    gdn.gdn_decode_pool(q, q, v, -g, b[:, :, 0].contiguous(), states[:0], i32([0, 0]), o=o)
    gdn.gdn_decode_pool(q[:0], q[:0], v[:0], -g[:0], b[:0, :, 0].contiguous(), states, i32([0]), cu_seqlens=i32([0, 0]))
    gdn.gdn_decode_pool(q, q, v, -g, b[:, :, 0].contiguous(), states, i32([0]), cu_seqlens=i32([0, 0]), o=o)
    assert torch.equal(states, kept) and torch.all(o == 7.0)
    cache = _pool_of_pages(torch.Generator().manual_seed(1), 2, 2, 64, 64, 64)
    before = [t.clone() for t in cache]
    gdn.gdn_cache_write(q[:0], v[:0], i32([]), *cache)
    gdn.gdn_cache_write(q, v, i32([0, 1]), *(t[:0] for t in cache))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(cache, before))


def test_pool_equals_decode():
    # one token each, slots in order, unit keys: gdn_decode's step
    S0, draws = inputs.make_decode_steps(9, 4, 128, 128, 1, dtype=torch.bfloat16, seed=3, device="cuda")
    x = draws[0]
    a, b = S0.clone(), S0.clone()
    o1 = gdn.gdn_decode(x.q, x.k, x.v, x.g, x.beta, a)
    o2 = gdn.gdn_decode_pool(x.q, x.k, x.v, x.g, x.beta, b, i32(list(range(9))))
    assert (a - b).abs().max() <= 1e-5 * a.abs().max()
    assert (o1.float() - o2.float()).abs().max() <= 2 * EPS16 * o1.float().abs().max()


def test_pool_nan_stays_in_its_request():
    args = _pool_inputs([2, 2], 2, 2, 64, 64, torch.float32, False, [0, 1], 1, 7, True)
    d = [t.cuda() for t in args]
    clean = [t.clone() for t in d]
    o1 = gdn.gdn_decode_pool(*clean, i32([0, 1]), cu_seqlens=i32([0, 2, 4]))
    d[1][1, 0, 3] = math.nan
    o2 = gdn.gdn_decode_pool(*d, i32([0, 1]), cu_seqlens=i32([0, 2, 4]))
    assert torch.isnan(o2[1, 0]).all() and torch.equal(o1[2:], o2[2:]) and torch.equal(o1[:, 1], o2[:, 1])
    assert torch.equal(o1[0], o2[0]) and torch.equal(clean[5][1:], d[5][1:])


# ---------------------------------------------------------------- together, and how calls are made


class _Engine:
    """A server of two requests' worth of layers: a delta-rule layer and an attention layer."""

    def __init__(self, rows, pages=64, page=64, max_blocks=16, H=4, hkv=2, d=64):
        z = lambda *s, **k: torch.zeros(s, device="cuda", **k)
        self.page, self.H, self.hkv, self.d = page, H, hkv, d
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.counts, self.state = z(rows, dtype=torch.int32), i32([0, pages, 0])
        self.ring = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.kc = z(pages, hkv, page, d, dtype=torch.uint8).view(ref.E4M3)
        self.vc = z(pages, hkv, page // 16, d, 16, dtype=torch.uint8).view(ref.E4M3)
        self.ks, self.vs = z(pages, hkv), z(pages, hkv)
        self.states = z(rows, H, d, d)

    def tokens(self, T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        bf = torch.bfloat16
        return dict(q=unit(r(T, self.H, self.d)).to(bf), k=unit(r(T, self.H, self.d)).to(bf), v=r(T, self.H, self.d).to(bf),
                    g=torch.log(0.9 + 0.1 * torch.sigmoid(r(T, self.H, self.d))), beta=torch.sigmoid(r(T, self.H)),
                    aq=r(T, self.H, self.d).to(bf), ak=r(T, self.hkv, self.d).to(bf), av=r(T, self.hkv, self.d).to(bf))

    def step(self, ctx, new, rows, x, T, prompt=False):
        cu, kv, slots, pos = gdn.gdn_batch_tables(ctx, new, T, self.page, self.table, self.counts, self.ring, self.state,
                                                  rows=rows)
        if prompt:
            first = self.states[rows.long()]
            o1, last = gdn.gdn_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, initial_state=first)
            self.states[rows.long()] = last
        else:
            o1 = gdn.gdn_decode_pool(x["q"], x["k"], x["v"], x["g"], x["beta"], self.states, rows, cu_seqlens=cu)
        gdn.gdn_cache_write(x["ak"], x["av"], slots, self.kc, self.vc, self.ks, self.vs)
        o2 = gdn.gdn_cache_attention(x["aq"], self.kc, self.vc, self.ks, self.vs, self.table, kv, cu, rows=rows)
        return o1, o2, kv


def test_a_server_runs():
    # prompts, decode steps, drafted tokens, one request ends and another takes its row: every attention output
    # against the tokens' own keys and values, within the cache's rounding, and the states against gdn_prefill
    e = _Engine(4)
    held = {}
    plan = [([0, 2], [130, 64], True), ([0, 2], [1, 1], False), ([2, 0], [3, 1], False), ([0], [-1], False),
            ([0, 2], [70, 1], False), ([3, 2, 0], [5, 1, 2], False)]
    for i, (rows, new, prompt) in enumerate(plan):
        ctx = [0 if r not in held else held[r]["aq"].shape[0] for r in rows]
        T = sum(x for x in new if x > 0)
        x = e.tokens(T, i)
        ended = [r for r, n_ in zip(rows, new) if n_ < 0]
        o1, o2, kv = e.step(i32(ctx), i32(new), i32(rows), x, T, prompt)
        t = 0
        for r, n_ in zip(rows, new):
            if n_ < 0:
                held.pop(r, None)
                e.states[r] = 0
                continue
            part = {k: v[t:t + n_] for k, v in x.items()}
            held[r] = {k: torch.cat([held[r][k], part[k]]) if r in held else part[k] for k in part}
            k, v = held[r]["ak"].double(), held[r]["av"].double()
            first = k.shape[0] - n_
            for h in range(e.H):
                j = h // (e.H // e.hkv)
                want, mag, _ = ref.attention(part["aq"][:, h:h + 1].double(), k[:, j], v[:, j], e.d ** -0.5, first,
                                             torch.ones(k.shape[0], dtype=torch.bool, device="cuda"))
                err = (o2[t:t + n_, h].double() - want[:, 0]).abs().max().item()
                # the cache's values are off by half a step of 3 mantissa bits of the page's largest
                assert err <= 2.0 ** -4 * 2 * v[:, j].abs().max().item(), (i, r, h, err)
            one = {k_: held[r][k_].contiguous() for k_ in held[r]}
            S = gdn.gdn_prefill(one["q"], one["k"], one["v"], one["g"], one["beta"], i32([0, k.shape[0]]))
            assert (S[0][first:].float() - o1[t:t + n_].float()).abs().max() <= 2e-2 * S[0].float().abs().max()
            assert (S[1][0] - e.states[r]).abs().max() <= 2e-2 * S[1].abs().max()
            t += n_
        assert e.state.tolist()[2] == 0
    log("  a server's steps agree with whole-sequence forms")


def test_a_server_runs_out_of_pages():
    # A request is refused: its state and its cache stay as they were, the other's go on, and when pages have come back
    # it takes the same tokens and has the state of a request that was never refused.
    e = _Engine(2, pages=3, max_blocks=4)
    rows = i32([0, 1])
    x0 = e.tokens(160, 0)
    e.step(i32([0, 0]), i32([100, 60]), rows, x0, 160, prompt=True)
    assert e.state.tolist()[1:] == [0, 0]

    def decode(ctx, new, x, T):
        cu, kv, slots, _ = gdn.gdn_batch_tables(i32(ctx), i32(new), T, e.page, e.table, e.counts, e.ring, e.state, rows=rows)
        took = kv - i32(ctx)
        before = e.states.clone()
        gdn.gdn_decode_pool(x["q"], x["k"], x["v"], x["g"], x["beta"], e.states, rows, cu_seqlens=cu, commit=took)
        if T:  # the same by the prompts' way
            _, last = gdn.gdn_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, initial_state=before)
            last = torch.where((took > 0)[:, None, None, None], last, before)
            assert (last - e.states).abs().max() <= 2e-2 * last.abs().max()
        gdn.gdn_cache_write(x["ak"], x["av"], slots, e.kc, e.vc, e.ks, e.vs)
        o = gdn.gdn_cache_attention(x["aq"], e.kc, e.vc, e.ks, e.vs, e.table, kv, cu, rows=rows)
        return took.tolist(), o

    x1, kept, page = e.tokens(6, 1), e.states.clone(), int(e.table[1, 0])
    held = [t[page].clone() for t in (e.kc, e.vc, e.ks, e.vs)]
    assert decode([100, 60], [1, 5], x1, 6)[0] == [1, 0] and e.state.tolist()[2] == 1
    assert torch.equal(e.states[1], kept[1]) and not torch.equal(e.states[0], kept[0])
    assert all(torch.equal(a.view(torch.uint8), b[page].view(torch.uint8)) for a, b in zip(held, (e.kc, e.vc, e.ks, e.vs)))
    none = {k: v[:0] for k, v in x1.items()}
    kept = e.states.clone()
    assert decode([101, 60], [-1, 0], none, 0)[0] == [-101, 0] and torch.equal(e.states, kept)
    later = {k: v[1:].contiguous() for k, v in x1.items()}
    took, o = decode([0, 60], [0, 5], later, 5)
    assert took == [0, 5] and e.state.tolist()[2] == 0 and torch.equal(e.states[0], kept[0])
    whole = {k: torch.cat([x0[k][100:], later[k]]).contiguous() for k in later}
    S = gdn.gdn_prefill(whole["q"], whole["k"], whole["v"], whole["g"], whole["beta"], i32([0, 65]))[1]
    assert (S[0] - e.states[1]).abs().max() <= 2e-2 * S.abs().max()
    k, v = whole["ak"].double(), whole["av"].double()
    for h in range(e.H):
        j = h // (e.H // e.hkv)
        want, _, _ = ref.attention(later["aq"][:, h:h + 1].double(), k[:, j], v[:, j], e.d ** -0.5, 60,
                                   torch.ones(65, dtype=torch.bool, device="cuda"))
        # keys and values are off by half a step of 3 mantissa bits of the page's largest
        assert (o[:, h].double() - want[:, 0]).abs().max() <= 2.0 ** -4 * 2 * v[:, j].abs().max()


def _calls():
    """Every serving call on inputs of its own: (name, function, tensors it updates)."""
    gen = torch.Generator().manual_seed(5)
    ctx, new, rows, table, counts, free, state = _tables_case(3, 40, 64, 5, 250, 0, 90, enders=4)
    tb = [i32(table), i32(counts), i32(free), i32(state)]
    T = sum(x for x in new if x > 0)
    a = (i32(ctx), i32(new), i32(rows))
    yield "tables", lambda: gdn.gdn_batch_tables(a[0], a[1], T, 64, *tb, rows=a[2]), tb
    cache = list(_pool_of_pages(gen, 9, 2, 64, 128, 128))
    k, v = (torch.randn((70, 2, 128), generator=gen).bfloat16().cuda() for _ in range(2))
    slots = i32([64 * 3 + 5 + i for i in range(59)] + [64 * 7 + i for i in range(11)])
    yield "write", lambda: [gdn.gdn_cache_write(k, v, slots, *cache)] and [], cache
    s = ref.Server([3000, 40, 700], 64, 2, 128, 128, seed=2)
    kc, vc, ks, vs, tab, kv_lens, _ = s.to("cuda")
    for name, lens in (("decode", [1, 1, 1]), ("mixed", [300, 1, 2])):
        q = torch.randn((sum(lens), 8, 128), generator=gen).bfloat16().cuda()
        cu = i32([0] + list(np.cumsum(lens)))
        yield f"attention {name}", lambda q=q, cu=cu: [gdn.gdn_cache_attention(q, kc, vc, ks, vs, tab, kv_lens, cu,
                                                                               max_kv=3000)], []
    d = [t.cuda() for t in _pool_inputs([1, 3, 0, 2], 4, 2, 128, 128, torch.bfloat16, False, [2, 0, 1, 4], 1, 3, True)]
    sl, cu4 = i32([2, 0, 1, 4]), i32([0, 1, 4, 4, 6])
    yield "pool", lambda: [gdn.gdn_decode_pool(*d, sl, cu_seqlens=cu4)], [d[5]]


def _restore(tensors, saved):
    for t, s in zip(tensors, saved):
        t.view(torch.uint8).copy_(s.view(torch.uint8))


def test_graphs_replay_every_call():
    for name, fn, state in _calls():
        saved = [t.clone() for t in state]
        eager = [t.clone() for t in fn()]
        after = [t.clone() for t in state]
        _restore(state, saved)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fn()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = fn()
        for rep in range(3):
            _restore(state, saved)
            for t in outs:
                t.zero_()
            assert torch.isfinite(torch.randn(1 << 18, device="cuda").sum()).item()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(list(outs) + state, eager + after):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (name, rep)
        log(f"  {name}: 3 replays equal the eager call")


def test_other_streams_and_repeats_give_the_same_bits():
    for name, fn, state in _calls():
        saved = [t.clone() for t in state]
        first = [t.clone() for t in fn()] + [t.clone() for t in state]
        for rep in range(2):
            _restore(state, saved)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                again = list(fn()) + state
            stream.synchronize()
            for x, y in zip(again, first):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (name, rep)


def test_two_attentions_at_once():
    # two streams, each with a workspace of its own, on the same cache
    s = ref.Server([20000, 5000], 64, 2, 128, 128, seed=2)
    kc, vc, ks, vs, tab, kv_lens, _ = s.to("cuda")
    qs = [torch.randn((2, 8, 128), device="cuda").bfloat16() for _ in range(2)]
    call = lambda q, **k: gdn.gdn_cache_attention(q, kc, vc, ks, vs, tab, kv_lens, i32([0, 1, 2]), **k)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = [call(q, stream=st) for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- refusals on the device


def test_binding_refusals():
    s = ref.Server([64], 64, 2, 64, 64)
    kc, vc, ks, vs, tab, kv_lens, _ = s.to("cuda")
    q = torch.zeros((1, 4, 64), device="cuda")
    for bad in (dict(q=q.half()), dict(kc=kc.view(torch.uint8)), dict(vc=ref.tokens_of(s.v).cuda()), dict(ks=ks.double()),
                dict(tab=tab.long()), dict(q=q.transpose(0, 1)), dict(kv=kv_lens.cpu()), dict(q=q[:, :3].contiguous()),
                dict(cu=i32([0]))):
        a = dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, tab=tab, kv=kv_lens, cu=i32([0, 1])) | bad
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_cache_attention(*a.values())
    long = torch.zeros((1, 2000), dtype=torch.int32, device="cuda")
    with pytest.raises(gdn.GdnError):
        gdn.gdn_cache_attention(q, kc, vc, ks, vs, long, kv_lens, i32([0, 1]), workspace=torch.empty(16, device="cuda"))
    for bad in (torch.empty(1 << 20), torch.empty((2048, 512), device="cuda").t()):  # not on the device; not in one piece
        with pytest.raises(ValueError):
            gdn.gdn_cache_attention(q, kc, vc, ks, vs, long, kv_lens, i32([0, 1]), workspace=bad)
        with pytest.raises(ValueError):
            gdn.gdn_batch_tables(i32([0]), i32([1]), 1, 64, long, i32([0]), i32([0]), i32([0, 1, 0]), workspace=bad)


def test_validation_mode(monkeypatch):
    monkeypatch.setenv("GDN_VALIDATE", "1")
    one = torch.zeros((2, 1, 64), device="cuda")
    cache = _pool_of_pages(torch.Generator().manual_seed(0), 3, 1, 64, 64, 64)
    gdn.gdn_cache_write(one, one, i32([5, 6]), *cache)
    for slots in ([5, 7], [6, 5], [5, 5]):
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_cache_write(one, one, i32(slots), *cache)
        assert e.value.status == gdn.GDN_ERR_DOMAIN
    s = ref.Server([100, 30], 64, 2, 64, 64)
    kc, vc, ks, vs, tab, kv, _ = s.to("cuda")
    q = torch.zeros((3, 4, 64), device="cuda")
    gdn.gdn_cache_attention(q, kc, vc, ks, vs, tab, kv, i32([0, 2, 3]))
    odd = ks.clone()
    odd[int(s.table[0, 1])] *= 1.5
    for bad in (dict(ks=odd), dict(kv=i32([-1, 30])), dict(kv=i32([100, 300])), dict(cu=i32([0, 2, 4])),
                dict(cu=i32([0, 2, 1])), dict(cu=i32([1, 2, 3]))):
        a = dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, tab=tab, kv=kv, cu=i32([0, 2, 3])) | bad
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_cache_attention(*a.values())
        assert e.value.status == gdn.GDN_ERR_DOMAIN
    args = [t.cuda() for t in _pool_inputs([1, 1], 2, 2, 64, 64, torch.float32, True, [0, 1], 0, 1, True)]
    gdn.gdn_decode_pool(*args, i32([1, -1]))
    for kw in (dict(slots=[1, 1]), dict(slots=[0, 1], cu=[0, 2, 1]), dict(slots=[0, 1], cu=[0, 1, 1])):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_decode_pool(*args, i32(kw["slots"]), cu_seqlens=i32(kw["cu"]) if "cu" in kw else None)
    args[3][0, 0] = 0.5
    with pytest.raises(gdn.GdnError):
        gdn.gdn_decode_pool(*args, i32([0, 1]))
    tb = lambda: [i32([[-1] * 4] * 2), i32([0, 0]), i32([0, 1, 2]), i32([0, 3, 0])]
    gdn.gdn_batch_tables(i32([0, 0]), i32([1, 2]), 3, 64, *tb(), rows=i32([1, 0]))
    for ctx, rows, state in (([-1, 0], [0, 1], [0, 3, 0]), ([0, 0], [1, 1], [0, 3, 0]), ([0, 0], [0, 2], [0, 3, 0]),
                             ([0, 0], [0, 1], [3, 3, 0]), ([0, 0], [0, 1], [0, 4, 0])):
        t = tb()
        t[3] = i32(state)
        with pytest.raises(gdn.GdnError):
            gdn.gdn_batch_tables(i32(ctx), i32([1, 1]), 2, 64, *t, rows=i32(rows))


def test_validation_of_new_lengths(monkeypatch):
    # more new tokens than T_total: the call would cut them; those of ended requests are none
    monkeypatch.setenv("GDN_VALIDATE", "1")
    for new, T, fine in (([1, 2], 3, True), ([1, 2], 2, False), ([-5, 3], 3, True), ([2 ** 31 - 1, 2 ** 31 - 1], 9, False)):
        t = [i32([[-1] * 4] * 2), i32([0, 0]), i32([0, 1, 2]), i32([0, 3, 0])]
        call = lambda: gdn.gdn_batch_tables(i32([0, 0]), i32(new), T, 64, *t)
        if fine:
            assert call()[0].tolist()[-1] == T
            continue
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == gdn.GDN_ERR_DOMAIN and t[1].tolist() == [0, 0]
