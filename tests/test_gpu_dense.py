"""Dense attention to an encoder's states and over a paged cache, and the cache's write and
read, against definitions in 64 bits. Tolerances: tests/dense_util.py derives them."""
import pytest
import torch

from block_sparse_online_b200 import solattn
from tests import dense_util as du

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, mul=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * mul).to(dtype)


# ------------------------------------------------------------------ the cache


@pytest.mark.parametrize("kind", [None, I8, E4], ids=["16", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", [  # (new tokens, lengths, Hkv, page, d)
    ([1], [1], 1, 16, 64),
    ([1, 0, 1, 1], [5, 0, 16, 33], 3, 16, 128),
    ([17, 40, 1], [17, 129, 700], 4, 64, 128),
    ([700], [1000], 5, 128, 64),
    ([33, 0], [64, 10], 2, 32, 64),
], ids=str)
def test_append_and_read(shape, dtype, kind):
    ns, lens, Hkv, page, d = shape
    g = gen(3 + len(ns))
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, dtype, kind)
    total = sum(ns) + 2  # two rows behind the last sequence
    x = [rnd(g, total, Hkv, d, mul=m, dtype=dtype) for m in (1.0, 0.03)]
    x[0][0, 0] = 0  # a row of zeros
    x[1][0, Hkv - 1, 1:] = 0  # one element: its code is TOP
    # rows whose ratios x TOP / amax lie on the border of two codes, for either kind, with exact and with rounded scales
    i = torch.arange(d, device="cuda")
    border = (i % 127 * 2 + 1) / 256, (17 + i % 8 * 2) / 64, 3.0 / 2.0 ** (i % 9 + 2)
    x[0][sum(ns) - 1, 0] = border[0].to(dtype)
    x[0][sum(ns) - 1, 0, 0] = 127 / 128
    x[1][sum(ns) - 1, 0] = border[(len(ns) + d // 64) % 2 + 1].to(dtype)
    x[1][sum(ns) - 1, 0, 0] = 7 / 8 if (len(ns) + d // 64) % 2 == 0 else 1.0
    before = [t.clone() if t is not None else None for t in (k, v, ks, vs)]
    cache = solattn.PagedCache(k, v, ks, vs)
    st = solattn.alloc_status()
    cu, length = du.cu_of(ns), du.ints(lens)
    solattn.solattn_cache_append(cache, x[0], x[1], table, cu, length, workspace=st)
    outs = [torch.full_like(x[0], 7.0), torch.full_like(x[0], 7.0)]
    solattn.solattn_cache_read(cache, table, cu, length, outs[0], outs[1], workspace=st)
    assert solattn.solattn_get_status(st) == 0
    for which, (pages, scale, was, was_s) in enumerate(((k, ks, before[0], before[2]), (v, vs, before[1], before[3]))):
        touched = torch.zeros(pages.shape[0], page, dtype=torch.bool, device="cuda")
        t = 0
        for b, (n, L) in enumerate(zip(ns, lens)):
            for i in range(n):
                pos = L - n + i
                at, row = int(table[b, pos // page]), pos % page
                touched[at, row] = True
                new = x[which][t + i]
                if kind is None:
                    assert torch.equal(pages[at, :, row], new)
                    assert torch.equal(outs[which][t + i], new)
                else:
                    codes, sc = du.quantise(new, kind)
                    assert torch.equal(pages.view(torch.uint8)[at, :, row].contiguous().view(kind).double(), codes)
                    assert torch.equal(scale[at, :, row], sc)
                    # one rounding of the 32-bit product code * scale
                    assert torch.equal(outs[which][t + i], (codes.float() * sc[:, None]).to(dtype))
            t += n
        assert (outs[which][t:] == 7).all()
        same = ~touched[:, None, :, None].expand_as(pages)
        raw = (lambda y: y.view(torch.int16) if kind is None else y.view(torch.uint8))
        assert torch.equal(raw(pages)[same], raw(was)[same])
        if kind is not None:
            keep = ~touched[:, None, :].expand_as(scale)
            assert torch.equal(scale.view(torch.int32)[keep], was_s.view(torch.int32)[keep])


@pytest.mark.parametrize("kind", [I8, E4], ids=["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_append_extreme_rows(dtype, kind):
    """Every magnitude of the type, subnormal to largest; rows with an infinity or NaN read back as NaN."""
    d, g = 64, gen(5)
    fi = torch.finfo(dtype)
    amax = [fi.max, fi.max / 3, fi.tiny, fi.smallest_normal * fi.eps, 1e30 if dtype == BF else 6e4, 1.0, 3.0, float("inf"),
            float("nan")]
    x = torch.rand(len(amax), 1, d, generator=g, device="cuda", dtype=torch.float64) * 2 - 1
    x[:, 0, 0] = 1
    x = (x * torch.tensor([a if a == a and a != float("inf") else 1.0 for a in amax], device="cuda", dtype=torch.float64)[:, None, None]).to(dtype)
    x[-2, 0, 5], x[-1, 0, 6] = float("inf"), float("nan")
    n = len(amax)
    k = torch.zeros(1, 1, 16, d, device="cuda").to(kind)
    ks = torch.zeros(1, 1, 16, device="cuda")
    cache = solattn.PagedCache(k, k.clone(), ks, ks.clone())
    table, cu, length = du.ints([[0]]), du.cu_of([n]), du.ints([n])
    solattn.solattn_cache_append(cache, x, x, table, cu, length)
    codes, sc = du.quantise(x[:-2], kind)
    got = k.view(torch.uint8)[0, 0, :n - 2].view(kind).double()
    assert torch.equal(got, codes[:, 0])
    assert torch.equal(ks[0, 0, :n - 2], sc[:, 0])
    assert ks[0, 0, n - 2:n].isnan().all()
    out = torch.empty_like(x)
    solattn.solattn_cache_read(cache, table, cu, length, out, torch.empty_like(x))
    assert out[-2:].isnan().all() and not out[:-2].isnan().any()


def test_append_strided_and_bad_pages():
    g, d, Hkv, page = gen(9), 128, 2, 16
    k, v, ks, vs, table = du.make_cache(g, [20, 40], Hkv, page, d, BF, E4)
    # a fused projection's output: keys and values interleaved in one row
    qkv = rnd(g, 12, 3 * Hkv, d)
    nk, nv = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    cache = solattn.PagedCache(k, v, ks, vs)
    st = solattn.alloc_status()
    table2 = table.clone()
    table2[1, 2] = k.shape[0]  # outside the cache: positions 32..39 of sequence 1
    before = k.clone()
    solattn.solattn_cache_append(cache, nk, nv, table2, du.cu_of([2, 10]), du.ints([20, 40]), workspace=st)
    assert solattn.solattn_get_status(st) == solattn.SOLATTN_ETABLE
    codes, sc = du.quantise(nk, E4)
    for i, pos in enumerate(range(18, 20)):
        at = int(table[0, pos // page])
        assert torch.equal(k.view(torch.uint8)[at, :, pos % page].view(E4).double(), codes[i])
    for i, pos in enumerate(range(30, 32)):
        at = int(table[1, pos // page])
        assert torch.equal(k.view(torch.uint8)[at, :, pos % page].view(E4).double(), codes[2 + i])
    same = torch.ones_like(before, dtype=torch.bool)
    same[int(table[0, 1]), :, 2:4] = False
    same[int(table[1, 1]), :, 14:16] = False
    assert torch.equal(k.view(torch.uint8)[same], before.view(torch.uint8)[same])


# ------------------------------------------------------------------ attention over the cache

PAGED = [  # (new tokens, lengths, H, Hkv, page, d, causal)
    ([1], [1], 1, 1, 16, 64, True),
    ([1], [77], 2, 2, 16, 128, True),
    ([1, 1, 0, 1], [1, 300, 7, 1025], 16, 4, 64, 128, True),
    ([1, 1], [4097, 15], 24, 3, 128, 128, False),
    ([2, 1], [130, 128], 12, 4, 32, 64, True),
    ([5, 3], [5, 259], 6, 2, 16, 128, True),
    ([1], [20000], 4, 2, 64, 128, True),
    ([1] * 40, [1 + 37 * i for i in range(40)], 8, 8, 16, 64, True),
    ([40], [40], 4, 1, 16, 128, True),
    ([130, 0, 257], [130, 5, 1000], 3, 3, 16, 64, True),
    ([300], [1111], 10, 2, 128, 128, False),
    ([1560], [5000], 2, 2, 64, 128, False),
    ([129, 1, 640], [700, 300, 640], 8, 2, 16, 128, True),
    ([200], [333], 14, 2, 32, 128, True),
]


def run_paged(ns, lens, H, Hkv, page, d, causal, dtype, kind, seed=1, mul=1.0, qmul=2.0, max_new=None):
    g = gen(seed)
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, dtype, kind, mul=mul)
    total = sum(ns)
    q = rnd(g, total + 3, H, d, mul=qmul, dtype=dtype)
    out = torch.full_like(q, 5.0)
    cache = solattn.PagedCache(k, v, ks, vs)
    ws = solattn.alloc_paged_workspace(cache, len(ns), H, total + 3)
    solattn.solattn_paged_forward(q, cache, table, du.cu_of(ns), du.ints(lens), max_new=max(ns) if max_new is None else max_new,
                                  causal=causal, out=out, workspace=ws)
    assert solattn.solattn_get_status(ws) == 0
    assert (out[total:] == 5).all()  # rows behind the last sequence are left alone
    want, bound = du.paged_oracle(q[:total], k, v, ks, vs, table, ns, lens, causal, dtype)
    du.check(out[:total], want, bound)
    return out


@pytest.mark.parametrize("case", PAGED, ids=[str(i) for i in range(len(PAGED))])
@pytest.mark.parametrize("dtype,kind", [(BF, None), (FP, None), (BF, I8), (FP, E4), (BF, E4), (FP, I8)],
                         ids=["bf16", "fp16", "bf16-int8", "fp16-e4m3", "bf16-e4m3", "fp16-int8"])
def test_paged(case, dtype, kind):
    run_paged(*case, dtype, kind)


@pytest.mark.parametrize("max_new", [0, 1, 5, 100000])
def test_paged_max_new_does_not_change_the_result(max_new):
    run_paged([70, 1, 9], [300, 40, 200], 4, 2, 16, 128, True, BF, None, max_new=max_new)


@pytest.mark.parametrize("kind", [None, I8, E4], ids=["16", "int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("mul,qmul", [(1e-4, 2.0), (30.0, 20.0), (1.0, 0.0)])
def test_paged_magnitudes(n, kind, mul, qmul):
    """Caches of tiny and large values; logits so large that the softmax is a choice; equal logits."""
    run_paged([n, n], [999, 257], 4, 2, 32, 128, True, BF, kind, mul=mul, qmul=qmul)


@pytest.mark.parametrize("n", [1, 150, 400])
def test_paged_8bit_scales_far_apart(n):
    """Value scales that grow along the sequence by many orders, and rows of zeros among them."""
    g, d, page, L = gen(21), 128, 16, 700
    k, v, ks, vs, table = du.make_cache(g, [L], 1, page, d, BF, I8)
    pos = torch.arange(L, device="cuda")
    at = table[0].long()[pos // page]
    vs[at, 0, pos % page] *= torch.exp2((pos // 50).float() * 3 - 20)
    zero = pos % 7 == 0
    vs[at[zero], 0, pos[zero] % page] = 0
    v[at[zero], 0, pos[zero] % page] = 0
    q = rnd(g, n, 4, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    out = solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n)
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
    du.check(out, want, bound)


@pytest.mark.parametrize("n,H", [(1, 2), (300, 2), (400, 32)])
@pytest.mark.parametrize("kind", [None, I8], ids=["16", "int8"])
def test_paged_bad_pages_read_as_zeros(n, H, kind):
    g, d, page, L = gen(31), 64, 16, 400
    k, v, ks, vs, table = du.make_cache(g, [L], 2, page, d, BF, kind)
    bad = table.clone()
    bad[0, 3], bad[0, 7] = -5, 1 << 20
    q = rnd(g, n, H, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    ws = solattn.alloc_paged_workspace(cache, 1, H, n)
    out = solattn.solattn_paged_forward(q, cache, bad, du.cu_of([n]), du.ints([L]), max_new=n, causal=False, workspace=ws)
    assert solattn.solattn_get_status(ws) == solattn.SOLATTN_ETABLE
    for p in (3, 7):
        k[int(table[0, p])] = 0
        v[int(table[0, p])] = 0
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], False, BF)
    du.check(out, want, bound)


@pytest.mark.parametrize("n", [1, 130])
def test_paged_bad_lengths_are_cut_and_reported(n):
    g, d, page = gen(32), 64, 16
    k, v, ks, vs, table = du.make_cache(g, [64, 64], 1, page, d, BF, None)
    q = rnd(g, 2 * n, 1, d)
    cache = solattn.PagedCache(k, v)
    for length in ([65, 10], [-3, 64], [1 << 30, 64]):
        ws = solattn.alloc_paged_workspace(cache, 2, 1, 2 * n)
        out = solattn.solattn_paged_forward(q, cache, table, du.cu_of([n, n]), du.ints(length), max_new=n, causal=False, workspace=ws)
        assert solattn.solattn_get_status(ws) == solattn.SOLATTN_ETABLE
        cut = [min(max(x, 0), 64) for x in length]
        want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n, n], cut, False, BF)
        du.check(out, want, bound)
    ws = solattn.alloc_paged_workspace(cache, 2, 1, 2 * n)
    solattn.solattn_paged_forward(q, cache, table, du.ints([0, 5 * n, 2 * n]), du.ints([64, 64]), max_new=n, causal=False, workspace=ws)
    assert solattn.solattn_get_status(ws) == solattn.SOLATTN_ETABLE


@pytest.mark.parametrize("n", [1, 300])
def test_paged_offsets_past_32_bits(n):
    """A pool of over 2^32 elements: the sequence's pages lie at both ends of it."""
    d, page, Hkv, pool = 128, 128, 8, 34000
    assert pool * Hkv * page * d > 1 << 32
    g = gen(41)
    k = torch.empty(pool, Hkv, page, d, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty(pool, Hkv, page, device="cuda")
    vs = torch.empty_like(ks)
    ids = [pool - 1, 0, pool - 7, 33333]
    for i in ids:
        for x, s in ((k, ks), (v, vs)):
            c, sc = du.quantise(rnd(g, Hkv, page, d), I8)
            x[i], s[i] = c.to(I8), sc
    table, L = du.ints([ids]), 4 * page - 3
    q = rnd(g, n, Hkv, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    out = solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n)
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
    du.check(out, want, bound)
    new = rnd(g, 2, Hkv, d)
    outs = torch.empty_like(new), torch.empty_like(new)
    solattn.solattn_cache_append(cache, new, new, du.ints([[pool - 2]]), du.cu_of([2]), du.ints([2]))
    solattn.solattn_cache_read(cache, du.ints([[pool - 2]]), du.cu_of([2]), du.ints([2]), *outs)
    codes, sc = du.quantise(new, I8)
    assert torch.equal(outs[0], (codes.float() * sc[..., None]).to(BF)) and torch.equal(outs[0], outs[1])


# ------------------------------------------------------------------ attention to an encoder's states

CROSS = [  # (B, H, Hkv, Nq, Nk, d, lens)
    (1, 2, 2, 1024, 77, 64, None),
    (1, 1, 1, 1, 1, 64, None),
    (3, 4, 2, 1, 300, 128, [300, 0, 129]),
    (2, 8, 1, 2, 65, 128, None),
    (1, 2, 2, 300, 769, 128, None),
    (3, 2, 2, 257, 256, 128, [0, 256, 13]),
    (2, 6, 2, 129, 128, 64, [128, 1]),
    (1, 2, 1, 4096, 512, 128, None),
    (1, 5, 1, 100, 4096, 128, None),
    (4, 3, 3, 1000, 33, 64, [33, 2, 0, 16]),
    (2, 2, 2, 5, 0, 64, None),
    (1, 14, 2, 50, 640, 64, None),
]


@pytest.mark.parametrize("case", CROSS, ids=[str(i) for i in range(len(CROSS))])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_cross(case, dtype, layout):
    B, H, Hkv, Nq, Nk, d, lens = case
    g = gen(7)

    def heads(n, h, mul=1.0):
        x = rnd(g, B, n, h, d, mul=mul, dtype=dtype).transpose(1, 2)
        return x if layout == "bnhd" else x.contiguous()

    q, k, v = heads(Nq, H, 2.0), heads(Nk, Hkv), heads(Nk, Hkv)
    if lens is not None:
        for b, L in enumerate(lens):  # padding may hold anything
            k[b, :, L:] = float("nan")
            v[b, :, L:] = float("inf")
    ws = solattn.alloc_cross_workspace(B, H, Hkv, Nq, Nk, d)
    out = solattn.solattn_cross(q, k, v, key_len=None if lens is None else du.ints(lens), workspace=ws)
    assert solattn.solattn_get_status(ws) == 0
    assert out.stride() == q.stride()
    want, bound = du.cross_oracle(q, k, v, lens, dtype)
    du.check(out, want, bound)


@pytest.mark.parametrize("Nq", [3, 200, 2000])
def test_cross_broadcast_and_slices(Nq):
    """Keys expanded over the batch, values cut out of a fused projection, a wide output."""
    g, B, H, Nk, d = gen(8), 3, 2, 190, 128
    q = rnd(g, B, H, Nq, d)
    k = rnd(g, 1, H, Nk, d).expand(B, H, Nk, d)
    v = rnd(g, B, Nk, 2, H, d)[:, :, 1].transpose(1, 2)
    wide = torch.full((B, Nq, 3 * H, d), 9.0, dtype=BF, device="cuda")
    out = wide[:, :, H:2 * H].transpose(1, 2)
    solattn.solattn_cross(q, k, v, out=out)
    want, bound = du.cross_oracle(q, k, v, None, BF)
    du.check(out, want, bound)
    assert (wide[:, :, :H] == 9).all() and (wide[:, :, 2 * H:] == 9).all()


def test_cross_bad_lengths_are_cut_and_reported():
    g = gen(10)
    q, k, v = (rnd(g, 2, 2, n, 64) for n in (40, 50, 50))
    ws = solattn.alloc_cross_workspace(2, 2, 2, 40, 50, 64)
    out = solattn.solattn_cross(q, k, v, key_len=du.ints([1000, -1]), workspace=ws)
    assert solattn.solattn_get_status(ws) == solattn.SOLATTN_ETABLE
    want, bound = du.cross_oracle(q, k, v, [50, 0], BF)
    du.check(out, want, bound)


@pytest.mark.parametrize("Nq", [4, 400, 20000])
def test_masked_infinities_and_nan_in_values(Nq):
    """A NaN among the keys that a row sees reaches that row; a score of -inf is a key without weight."""
    g = gen(12)
    q, k, v = rnd(g, 1, 1, Nq, 64), rnd(g, 1, 1, 200, 64), rnd(g, 1, 1, 200, 64)
    v[0, 0, 150, 3] = float("nan")
    out = solattn.solattn_cross(q, k, v)
    assert out[..., 3].isnan().all() and not out[..., :3].isnan().any()
    k[0, 0, 150] = 0
    q[..., 0] = 1.0
    k[0, 0, 150, 0] = -float("inf")  # weight 0
    v[0, 0, 150, 3] = 1.0
    out = solattn.solattn_cross(q, k, v)
    keep = torch.arange(200, device="cuda") != 150
    want, bound = du.cross_oracle(q, k[:, :, keep], v[:, :, keep], None, BF)
    du.check(out, want, bound)
    for at in (0, 70, 199):  # a NaN in a key that every row sees: its scores are NaN, and so are the rows
        kk = k.clone()
        kk[0, 0, at, 7] = float("nan")
        assert solattn.solattn_cross(q, kk, v).isnan().all()


# ------------------------------------------------------------------ many rows with every kind of edge

BIG_CROSS = [  # (B, H, Hkv, Nq, Nk, d, lens): enough products for the tile kernel
    (3, 6, 2, 3000, 200, 64, [200, 0, 13]),
    (2, 4, 4, 2000, 769, 128, [769, 130]),
    (4, 8, 8, 2500, 33, 64, [33, 2, 0, 16]),
    (1, 16, 16, 4097, 77, 128, None),
    (2, 3, 1, 6333, 128, 128, [128, 64]),
    (1, 2, 2, 50000, 17, 128, None),
    (3, 7, 1, 1999, 320, 64, [1, 320, 65]),
]


@pytest.mark.parametrize("case", BIG_CROSS, ids=[str(i) for i in range(len(BIG_CROSS))])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_cross_many_rows(case, dtype):
    B, H, Hkv, Nq, Nk, d, lens = case
    g = gen(13)
    q = rnd(g, B, Nq, H, d, mul=2.0, dtype=dtype).transpose(1, 2)
    k, v = rnd(g, B, Hkv, Nk, d, dtype=dtype), rnd(g, B, Nk, Hkv, d, dtype=dtype).transpose(1, 2)
    if lens is not None:
        for b, L in enumerate(lens):
            k[b, :, L:] = float("inf")
            v[b, :, L:] = float("nan")
    ws = solattn.alloc_cross_workspace(B, H, Hkv, Nq, Nk, d)
    key_len = None if lens is None else du.ints(lens)
    out = solattn.solattn_cross(q, k, v, key_len=key_len, workspace=ws)
    for _ in range(4):
        assert torch.equal(out, solattn.solattn_cross(q, k, v, key_len=key_len, workspace=ws))
    assert solattn.solattn_get_status(ws) == 0
    want, bound = du.cross_oracle(q, k, v, lens, dtype)
    du.check(out, want, bound)


BIG_PAGED = [
    ([700, 1, 0, 300], [900, 1, 5, 300], 6, 2, 16, 128, True),
    ([513, 200], [513, 1000], 10, 2, 32, 64, True),
    ([257, 700], [3000, 700], 5, 5, 128, 64, False),
    ([2000], [2000], 3, 1, 64, 128, True),
    ([130] * 9, [130 + 61 * i for i in range(9)], 16, 4, 16, 64, True),
]


@pytest.mark.parametrize("case", BIG_PAGED, ids=[str(i) for i in range(len(BIG_PAGED))])
@pytest.mark.parametrize("dtype,kind", [(BF, None), (FP, None), (BF, I8), (FP, E4), (BF, E4), (FP, I8)],
                         ids=["bf16", "fp16", "bf16-int8", "fp16-e4m3", "bf16-e4m3", "fp16-int8"])
def test_paged_many_rows(case, dtype, kind):
    run_paged(*case, dtype, kind)


@pytest.mark.parametrize("Nq", [30, 3000])
def test_cross_more_query_heads_than_half_a_tile(Nq):
    g = gen(14)
    q, k, v = rnd(g, 1, 130, Nq, 64), rnd(g, 1, 1, 100, 64), rnd(g, 1, 1, 100, 64)
    want, bound = du.cross_oracle(q, k, v, None, BF)
    du.check(solattn.solattn_cross(q, k, v), want, bound)


def test_more_sequences_than_are_searched_at_once():
    """1100 sequences, single tokens and none: write, attend, read back."""
    B, Hkv, H, d, page = 1100, 1, 2, 64, 16
    ns = [i % 3 != 1 and 1 or 0 for i in range(B)]
    lens = [max(n, (7 * i) % 40) for i, n in enumerate(ns)]
    g = gen(15)
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, BF, I8)
    cache = solattn.PagedCache(k, v, ks, vs)
    total = sum(ns)
    new = rnd(g, total, Hkv, d), rnd(g, total, Hkv, d)
    cu, length = du.cu_of(ns), du.ints(lens)
    ws = solattn.alloc_paged_workspace(cache, B, H, total)
    solattn.solattn_cache_append(cache, *new, table, cu, length, workspace=ws)
    back = solattn.solattn_cache_read(cache, table, cu, length, torch.empty_like(new[0]), torch.empty_like(new[1]), workspace=ws)
    for x, y in zip(new, back):
        codes, sc = du.quantise(x, I8)
        assert torch.equal(y, (codes.float() * sc[..., None]).to(BF))
    q = rnd(g, total, H, d)
    out = solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=1, workspace=ws)
    assert solattn.solattn_get_status(ws) == 0
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens, True, BF)
    du.check(out, want, bound)


# ------------------------------------------------------------------ together, streams, graphs


@pytest.mark.parametrize("kind", [None, I8, E4], ids=["16", "int8", "e4m3"])
def test_streaming_steps(kind):
    """Chunks of a growing sequence: append, attend (causal, then to all), cross attention, read back."""
    g, H, Hkv, d, page, steps = gen(51), 4, 2, 128, 32, [100, 1, 37, 1]
    total = sum(steps)
    pool = -(-total // page) + 1
    base = torch.zeros(pool, Hkv, page, d, device="cuda", dtype=BF)
    k, v = (base.clone(), base.clone()) if kind is None else (base.to(kind), base.to(kind))
    ks, vs = (None, None) if kind is None else (torch.zeros(pool, Hkv, page, device="cuda"), torch.zeros(pool, Hkv, page, device="cuda"))
    cache = solattn.PagedCache(k, v, ks, vs)
    table = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)[None, :].contiguous()
    text = rnd(g, 1, Hkv, 77, d), rnd(g, 1, Hkv, 77, d)
    ws = solattn.alloc_paged_workspace(cache, 1, H, max(steps))
    rows = [[], []]
    L = 0
    for n in steps:
        L += n
        cu, length = du.cu_of([n]), du.ints([L])
        new = rnd(g, n, Hkv, d), rnd(g, n, Hkv, d)
        q = rnd(g, n, H, d)
        solattn.solattn_cache_append(cache, *new, table, cu, length, workspace=ws)
        o = solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=n, causal=True, workspace=ws)
        x = solattn.solattn_cross(o.transpose(0, 1)[None], *text, workspace=ws)
        back = solattn.solattn_cache_read(cache, table, cu, length, torch.empty_like(new[0]), torch.empty_like(new[1]), workspace=ws)
        for i in range(2):
            rows[i].append(back[i])
        want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
        du.check(o, want, bound)
        want, bound = du.cross_oracle(o.transpose(0, 1)[None], *text, None, BF)
        du.check(x, want, bound)
    everything = torch.empty(total, Hkv, d, dtype=BF, device="cuda"), torch.empty(total, Hkv, d, dtype=BF, device="cuda")
    solattn.solattn_cache_read(cache, table, du.cu_of([total]), du.ints([total]), *everything, workspace=ws)
    assert torch.equal(everything[0], torch.cat(rows[0])) and torch.equal(everything[1], torch.cat(rows[1]))
    assert solattn.solattn_get_status(ws) == 0


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("kind", [None, E4], ids=["16", "e4m3"])
def test_repeatable_and_captured(n, kind):
    """Two calls agree bit for bit; a captured graph replays on new lengths and inputs, on another stream."""
    g, H, Hkv, d, page = gen(61), 8, 2, 128, 64
    lens = [3000, 1, 700]
    ns = [n, 1, n]
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, BF, kind)
    cache = solattn.PagedCache(k, v, ks, vs)
    q = rnd(g, sum(ns), H, d)
    cu, length = du.cu_of(ns), du.ints(lens)
    ws = solattn.alloc_paged_workspace(cache, 3, H, sum(ns))
    a = solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=n, workspace=ws)
    b = solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=n, workspace=ws)
    assert torch.equal(a, b)
    other = torch.cuda.Stream()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=n, out=out, workspace=ws)
    lens2 = [2500, 1, 699]
    length.copy_(du.ints(lens2))
    q.copy_(rnd(g, sum(ns), H, d))
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(3):
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens2, True, BF)
    du.check(out, want, bound)
    assert solattn.solattn_get_status(ws) == 0


def test_explicit_stream_and_two_at_once():
    """Calls on two streams with a workspace each."""
    g = gen(71)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    xs, outs = [], []
    for i in range(2):
        xs.append([rnd(g, 2, 4, n, 128) for n in (3000, 600, 600)])
    torch.cuda.synchronize()
    wss = [solattn.alloc_cross_workspace(2, 4, 4, 3000, 600, 128) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = [solattn.solattn_cross(*x, workspace=w, stream=s) for x, w, s in zip(xs, wss, streams)]
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        want, bound = du.cross_oracle(*x, None, BF)
        du.check(o, want, bound)


def test_short_call_path_agrees_with_the_long_one(monkeypatch):
    """The binding's short call path (every tensor given, current stream) and the Python way make the same call."""
    g = gen(81)
    q, k, v = rnd(g, 2, 4, 300, 64), rnd(g, 2, 2, 90, 64), rnd(g, 2, 2, 90, 64)
    ws = solattn.alloc_cross_workspace(2, 4, 2, 300, 90, 64)
    kp, vp, ks, vs, table = du.make_cache(g, [70, 33], 2, 16, 64, BF, E4)
    cache = solattn.PagedCache(kp, vp, ks, vs)
    pq, new = rnd(g, 5, 4, 64), rnd(g, 5, 2, 64)
    cu, length = du.cu_of([2, 3]), du.ints([70, 33])
    pws = solattn.alloc_paged_workspace(cache, 2, 4, 5)

    def calls():
        out, po = torch.empty_like(q), torch.empty_like(pq)
        rows = torch.empty_like(new), torch.empty_like(new)
        solattn.solattn_cross(q, k, v, key_len=du.ints([90, 7]), out=out, workspace=ws)
        solattn.solattn_cache_append(cache, new, new, table, cu, length, workspace=pws)
        solattn.solattn_paged_forward(pq, cache, table, cu, length, max_new=3, causal=True, out=po, workspace=pws)
        solattn.solattn_cache_read(cache, table, cu, length, *rows, workspace=pws)
        return out, po, *rows

    short = calls()
    monkeypatch.setattr(solattn, "_fast", None)
    for a, b in zip(short, calls()):
        assert torch.equal(a, b)
    monkeypatch.undo()
    # what the short path does not take is refused in words
    bad = torch.empty(2, 4, 300, 64, device="cuda")
    with pytest.raises(ValueError):
        solattn.solattn_cross(q, k, v, out=bad, workspace=ws)
    with pytest.raises(ValueError):
        solattn.solattn_cross(q, k, v[:, :, :50], out=torch.empty_like(q), workspace=ws)
    with pytest.raises(solattn.SolAttnError):
        solattn.solattn_cross(q, k, v, out=torch.empty_like(q), workspace=ws[:512])
    with pytest.raises(ValueError):
        solattn.solattn_paged_forward(pq, cache, table.long(), cu, length, max_new=1, out=torch.empty_like(pq), workspace=pws)
    with pytest.raises(ValueError):
        solattn.solattn_paged_forward(pq, cache, table, cu[:2], length, max_new=1, out=torch.empty_like(pq), workspace=pws)
    with pytest.raises(solattn.SolAttnError):
        solattn.solattn_paged_forward(pq, cache, table, cu, length, max_new=-1, out=torch.empty_like(pq), workspace=pws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [None, I8, E4], ids=["16", "int8", "e4m3"])
def test_repeated_passes_agree(d, kind):
    """Many passes of a batch of chunks give the same bits: no buffer is overwritten before it has been read."""
    g, H, Hkv, page = gen(91), 8, 4, 32
    ns, lens = [700, 1300, 65, 1], [1500, 4400, 700, 2000]
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, BF, kind)
    cache = solattn.PagedCache(k, v, ks, vs)
    q = rnd(g, sum(ns), H, d)
    cu, length = du.cu_of(ns), du.ints(lens)
    ws = solattn.alloc_paged_workspace(cache, len(ns), H, sum(ns))
    outs = [torch.empty_like(q) for _ in range(2)]
    solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=1300, causal=False, out=outs[0], workspace=ws)
    for _ in range(60):
        solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=1300, causal=False, out=outs[1], workspace=ws)
        assert torch.equal(outs[0], outs[1])
    assert solattn.solattn_get_status(ws) == 0
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens, False, BF)
    du.check(outs[1], want, bound)
