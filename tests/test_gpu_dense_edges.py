"""Masks, infinities and magnitudes at which the dense attention's kernels could differ from the definition,
in the rows kernel and in the tile kernel: each test names the kernel that it means and checks that it ran.
Tolerances: tests/dense_util.py derives them."""
import pytest
import torch

from block_sparse_online_b200 import solattn
from tests import dense_util as du

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn
KINDS = [(BF, None), (FP, None), (BF, I8), (FP, E4)]
KIND_IDS = ["bf16", "fp16", "bf16-int8", "fp16-e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, mul=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * mul).to(dtype)


def run_on(kernel, call):
    """call(), which has to launch `kernel` ("rows" or "tile") and not the other."""
    for _ in range(3):  # (activity records may be lost; a result is the same every time)
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
            result = call()
            torch.cuda.synchronize()
        names = " ".join(e.key for e in p.key_averages())
        ran = {k for k in ("rows", "tile") if f"{k}_kernel" in names}
        if ran:
            break
    assert ran == {kernel}, (ran, names)
    return result


# ------------------------------------------------------------------ columns without weight


@pytest.mark.parametrize("kernel,n", [("rows", 15), ("tile", 1000)])
@pytest.mark.parametrize("dtype,kind", KINDS, ids=KIND_IDS)
def test_causal_rows_in_front_of_the_sequence_are_zero(kernel, n, dtype, kind):
    """More new tokens than the sequence has keys: reported, and the tokens without a key are zeros."""
    g, H, d, page = gen(1), 16, 128, 16
    ns, lens = [n, n], [10, n]
    k, v, ks, vs, table = du.make_cache(g, lens, H, page, d, dtype, kind)
    q = rnd(g, 2 * n, H, d, dtype=dtype)
    cache = solattn.PagedCache(k, v, ks, vs)
    ws = solattn.alloc_paged_workspace(cache, 2, H, 2 * n)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of(ns), du.ints(lens), max_new=n,
                                                               causal=True, workspace=ws))
    assert solattn.solattn_get_status(ws) == solattn.SOLATTN_ETABLE
    assert (out[:n - 10] == 0).all()
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens, True, dtype)
    du.check(out, want, bound)


def cross_inputs(seed, n, Nk, dtype, d=64):
    """q, k, v of 16 heads; element 0 of every query is 1 and of every key 0."""
    g = gen(seed)
    q, k, v = (rnd(g, 1, 16, m, d, dtype=dtype) for m in (n, Nk, Nk))
    q[..., 0], k[..., 0] = 1.0, 0.0
    return q, k, v


@pytest.mark.parametrize("kernel,n", [("rows", 5), ("tile", 2000)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Nk", [50, 300])
def test_scores_of_minus_infinity(kernel, n, dtype, Nk):
    """A row whose scores are all -inf is zero; with one finite score it is that key's value."""
    q, k, v = cross_inputs(2, n, Nk, dtype)
    k[..., 0] = -float("inf")
    out = run_on(kernel, lambda: solattn.solattn_cross(q, k, v))
    assert (out == 0).all()
    for at in (0, Nk - 1):
        kk = k.clone()
        kk[:, :, at, 0] = 0.0
        out = solattn.solattn_cross(q, kk, v)
        # weight 1 and a sum of 1: the value itself, after the last rounding of it and of P
        want = v[:, :, at:at + 1].expand_as(out).double()
        du.check(out, want, want.abs() * (du.EPS[dtype] + 1.5e-4))


@pytest.mark.parametrize("kernel,n", [("rows", 5), ("tile", 2000)])
@pytest.mark.parametrize("at", [0, 5, 6, 7, 14, 15, 62, 63, 64, 70, 79, 127, 130, 134])
def test_a_score_of_infinity_makes_the_row_nan(kernel, n, at):
    q, k, v = cross_inputs(3, n, 300, BF)
    k[:, :, at, 0] = float("inf")
    assert run_on(kernel, lambda: solattn.solattn_cross(q, k, v)).isnan().all()


@pytest.mark.parametrize("kernel,n", [("rows", 5), ("tile", 2000)])
@pytest.mark.parametrize("score", [-8192.0, -1200.0, -float("inf")])
def test_huge_values_of_keys_without_weight(kernel, n, score):
    """A key hundreds of powers of two below the others has no weight, however large its value: 2^(1.44 score / 8)
    times 2^127 is below 2^-88."""
    for at in (14, 71, 128 + 6, 299):  # in a row's first step, in later ones, in the ragged last one
        q, k, v = cross_inputs(4, n, 300, BF)
        k[:, :, at, 0] = score
        v[:, :, at] = 2.0 ** 127
        out = run_on(kernel, lambda: solattn.solattn_cross(q, k, v))
        if score == -float("inf"):
            k[:, :, at, 0] = -8192.0
        want, bound = du.cross_oracle(q, k, v, None, BF)
        du.check(out, want, bound)


@pytest.mark.parametrize("kernel,n", [("rows", 12), ("tile", 1000)])
def test_huge_values_of_later_keys(kernel, n):
    """Causal: a token's row does not see the large value of a token behind it."""
    g, H, d, page = gen(5), 16, 64, 16
    k, v, _, _, table = du.make_cache(g, [n], H, page, d, BF, None)
    v[int(table[0, 0]), :, 7] = 2.0 ** 120
    q = rnd(g, n, H, d, mul=0.5)
    cache = solattn.PagedCache(k, v)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([n]), max_new=n))
    want, bound = du.paged_oracle(q, k, v, None, None, table, [n], [n], True, BF)
    du.check(out, want, bound)


# ------------------------------------------------------------------ scales of 8-bit rows


@pytest.mark.parametrize("kernel,n", [("rows", 3), ("tile", 1000)])
@pytest.mark.parametrize("kind", [I8, E4], ids=["int8", "e4m3"])
@pytest.mark.parametrize("which", ["all", "mixed", "mixed_large"])
def test_negative_scales(kernel, n, kind, which):
    """x = code * scale whatever the scale's sign, for keys and for values."""
    g, H, d, page, L = gen(6), 8, 128, 32, 1300
    k, v, ks, vs, table = du.make_cache(g, [L], H, page, d, BF, kind)
    for s in (ks, vs):
        sign = -1.0 if which == "all" else torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        s.mul_(sign)
        if which == "mixed_large":  # the negative ones far above the others
            s.mul_(torch.where(s < 0, 2.0 ** (12 if s is vs else 1), 1.0))
    q = rnd(g, n, H, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n))
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
    du.check(out, want, bound)


# ------------------------------------------------------------------ lengths out of range, written and read


@pytest.mark.parametrize("kind", [None, I8], ids=["16", "int8"])
@pytest.mark.parametrize("cu,lens,total", [
    ([0, 12], [64], 10),               # behind the packed rows: cut to 10 tokens, positions 54 .. 63
    ([0, 4, 1 << 30], [20, 64], 10),
    ([-5, 3, 10], [40, 64], 10),       # in front of them: cut to [0, 3)
    ([0, 7, 4, 4], [64, 30, 33], 10),  # descending: the second and third sequence are empty
    ([0, 5, 10], [1 << 30, 65], 10),   # longer than the table
    ([0, 5, 10], [-1, 64], 10),        # no keys at all: nothing is written
    ([0, 10], [3], 10),                # more new tokens than keys: those in front of the sequence are dropped
], ids=str)
def test_cache_lengths_are_cut_as_the_attention_cuts_them(cu, lens, total, kind):
    """What append writes is where the attention looks for it, what cannot be written is left alone, and either
    call reports it."""
    g, Hkv, d, page = gen(7), 2, 64, 16
    B, width = len(lens), 4
    pages = [torch.randn(B * width, Hkv, page, d, generator=g, device="cuda") for _ in range(2)]
    if kind is None:
        k, v, ks, vs = pages[0].to(BF), pages[1].to(BF), None, None
    else:
        k, v = ((x * 20).to(kind) for x in pages)
        ks, vs = (torch.rand(B * width, Hkv, page, generator=g, device="cuda") for _ in range(2))
    cache = solattn.PagedCache(k, v, ks, vs)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).reshape(B, width)
    new = rnd(g, total, Hkv, d), rnd(g, total, Hkv, d)
    want = [x.clone() for x in (k, v)], [None if x is None else x.clone() for x in (ks, vs)]
    rows = {}
    for b in range(B):  # as the attention cuts them
        lo = min(max(cu[b], 0), total)
        hi = max(min(max(cu[b + 1], 0), total), lo)
        L = min(max(lens[b], 0), width * page)
        for i in range(lo, hi):
            if L - (hi - i) >= 0:
                rows[i] = (int(table[b, (L - (hi - i)) // page]), (L - (hi - i)) % page)
    for i, (at, r) in rows.items():
        for w in range(2):
            if kind is None:
                want[0][w][at, :, r] = new[w][i]
            else:
                codes, sc = du.quantise(new[w][i], kind)
                want[0][w][at, :, r] = codes.to(kind)
                want[1][w][at, :, r] = sc
    st = solattn.alloc_status()
    args = table, du.ints(cu), du.ints(lens)
    solattn.solattn_cache_append(cache, *new, *args, workspace=st)
    assert solattn.solattn_get_status(st) == solattn.SOLATTN_ETABLE
    for got, x in zip((k, v), want[0]):
        assert torch.equal(got, x)
    if kind is not None:
        for got, x in zip((ks, vs), want[1]):
            assert torch.equal(got, x)
    out = torch.full_like(new[0], 7.0), torch.full_like(new[1], 7.0)
    st = solattn.alloc_status()
    solattn.solattn_cache_read(cache, *args, *out, workspace=st)
    assert solattn.solattn_get_status(st) == solattn.SOLATTN_ETABLE
    for w in range(2):
        for i in range(total):
            if i in rows:
                at, r = rows[i]
                x = want[0][w][at, :, r]
                x = x if kind is None else (x.float() * want[1][w][at, :, r][..., None]).to(BF)
                assert torch.equal(out[w][i], x)
            else:
                assert (out[w][i] == 7).all()


# ------------------------------------------------------------------ 8-bit rows whose scales differ


def paged_oracle8(q, k, v, ks, vs, table, ns, lens, causal, dtype):
    """As du.paged_oracle, with a bound that knows of the keys that a row SEES alone. P times the value's scale is rounded
    to fp16 in units in which the row's largest such product is at least 1: a product below 2^-14 of that is off by at
    most 2^-25, so the row by 2^-25 max_j (w_j |scale_j|) sum_j |code_j|, j over the keys that it sees."""
    total, H, d = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    G = H // Hkv
    o = torch.zeros(total, H, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    t0 = 0
    for b, (n, L) in enumerate(zip(ns, lens)):
        if n == 0:
            continue
        kk, _, _ = du.cached(k, ks, table[b], page, L)
        vv, codes, _ = du.cached(v, vs, table[b], page, L)
        pos = torch.arange(L, device=q.device)
        scale = vs[table[b].long()[pos // page], :, pos % page].double().abs().t()  # [Hkv, L]
        i = torch.arange(n, device=q.device)
        limit = L - n + i + 1 if causal else torch.full_like(i, L)
        seen = pos[None, :] < limit[:, None]
        for h in range(H):
            x, g = q[t0:t0 + n, h].double(), h // G
            o[t0:t0 + n, h], tight = du.attend(x, kk[g], vv[g], limit, codes=torch.zeros_like(codes[g]), dtype=dtype, ptype=FP)
            s = torch.where(seen, x @ kk[g].t() / d ** 0.5, torch.tensor(-float("inf"), dtype=torch.float64, device=q.device))
            most = (torch.softmax(s, 1) * scale[g]).amax(1, keepdim=True)
            bound[t0:t0 + n, h] = tight + 2.0 ** -25 * most * (seen.double() @ codes[g].abs())
        t0 += n
    return o, bound


def check8(kernel, n, L, kind, causal, change, H=8, dtype=BF, seed=8, qmul=2.0):
    """One sequence of L keys, n new tokens, with `change(k, v, ks, vs, at, row)` applied to the cache (at, row: the page and
    the row of each position)."""
    g, d, page = gen(seed), 128, 16
    k, v, ks, vs, table = du.make_cache(g, [L], H, page, d, dtype, kind)
    pos = torch.arange(L, device="cuda")
    q = rnd(g, n, H, d, mul=qmul, dtype=dtype)
    change(q, k, v, ks, vs, table[0].long()[pos // page], pos % page)
    cache = solattn.PagedCache(k, v, ks, vs)
    ws = solattn.alloc_paged_workspace(cache, 1, H, n)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n,
                                                               causal=causal, workspace=ws))
    assert solattn.solattn_get_status(ws) == 0
    want, bound = paged_oracle8(q, k, v, ks, vs, table, [n], [L], causal, dtype)
    # the bound means something: an output of zeros would fail in nearly every row that the type can hold (fp16 ends at 2^-24)
    size = want.abs().amax(2)
    told = size > (2.0 ** -18 if dtype == FP else 0.0)
    assert told.double().mean() > 0.5 and (size > 4 * bound.amax(2))[told].double().mean() > 0.9
    du.check(out, want, bound)


KERNELS = [("rows", 15), ("tile", 1000)]


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [I8, E4], ids=["int8", "e4m3"])
@pytest.mark.parametrize("up", [14, 30, 60])
@pytest.mark.parametrize("where", [9, -2])
def test_a_later_tokens_scale_leaves_a_row_alone(kernel, n, kind, up, where):
    """Causal: the value scale of one token is 2^14 to 2^60 times the others'. The tokens in front of it do not see it."""
    def change(q, k, v, ks, vs, at, row):
        vs[at[where], :, row[where]] *= 2.0 ** up
    check8(kernel, n, n, kind, True, change)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [I8, E4], ids=["int8", "e4m3"])
@pytest.mark.parametrize("where", [0, 200, 699])
def test_a_large_scale_without_weight_costs_the_others_nothing(kernel, n, kind, where):
    """A value scale 2^30 times the others', of a key whose score is 2^70 below theirs."""
    def change(q, k, v, ks, vs, at, row):
        q[..., 0] = 1.0
        codes = k.view(torch.uint8)
        zero, low = torch.tensor([0.0, -112.0], device="cuda").to(kind).view(torch.uint8)
        codes[..., 0] = zero
        codes[at[where], :, row[where]] = zero
        codes[at[where], :, row[where], 0] = low
        ks[at[where], :, row[where]] = 70 / 1.4427 * 128 ** 0.5 / 112
        vs[at[where], :, row[where]] *= 2.0 ** 30
    check8(kernel, n, 1400, kind, False, change, qmul=0.5)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [I8, E4], ids=["int8", "e4m3"])
@pytest.mark.parametrize("step", [3, -3])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_scales_that_grow_or_shrink(kernel, n, kind, step, dtype):
    """Value scales that change eightfold every 70 keys, zeros among them, within fp16's range for fp16."""
    def change(q, k, v, ks, vs, at, row):
        pos = torch.arange(len(at), device="cuda")
        e = (pos // 70) * step
        e = e - (e.max() + e.min()) // 2 - (6 if dtype == FP else 0)
        vs[at, :, row] *= torch.exp2(e.float().clamp(-24, 12 if dtype == FP else 40))[:, None]
        zero = pos % 7 == 0
        zero[:2] = False
        vs[at[zero], :, row[zero]] = 0
        v.view(torch.uint8)[at[zero], :, row[zero]] = 0
    check8(kernel, n, 1000, kind, True, change, dtype=dtype)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("e", [-98, -60, -20, 20, 60, 90])
def test_caches_of_any_magnitude(kernel, n, e):
    def change(q, k, v, ks, vs, at, row):
        vs.mul_(2.0 ** e)
    check8(kernel, n, 1000, I8, True, change)


@pytest.mark.parametrize("kernel,n", KERNELS)
def test_scales_at_both_ends_of_the_range(kernel, n):
    """Neighbouring keys 2^180 apart: the small ones count in the sum of weights though their values vanish."""
    def change(q, k, v, ks, vs, at, row):
        pos = torch.arange(len(at), device="cuda")
        vs[at, :, row] *= torch.exp2(torch.where((pos // 150) % 2 == 0, -80.0, 95.0))[:, None]
    check8(kernel, n, 1000, I8, True, change)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [None, I8, E4], ids=["16", "int8", "e4m3"])
@pytest.mark.parametrize("up", [20, 45, 100])
def test_a_tokens_large_queries_leave_the_others_alone(kernel, n, kind, up):
    """The queries of one token are 2^20 to 2^100 times the others' (bf16 queries meet 8-bit keys as fp16)."""
    g, H, d, page, L = gen(9), 8, 128, 16, 1300
    k, v, ks, vs, table = du.make_cache(g, [L], H, page, d, BF, kind)
    q = rnd(g, n, H, d, mul=2.0)
    at = n // 2
    q[at] *= 2.0 ** up
    cache = solattn.PagedCache(k, v, ks, vs)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n, causal=False))
    rest = torch.arange(n, device="cuda") != at
    limit = torch.full((n - 1,), L, device="cuda")
    for h in range(H):
        kk, _, _ = du.cached(k, ks, table[0], page, L)
        vv, codes, cmax = du.cached(v, vs, table[0], page, L)
        want, bound = du.attend(q[rest, h].double(), kk[h], vv[h], limit, codes=None if codes is None else codes[h], cmax=cmax,
                                ptype=FP if kind is not None else BF)
        du.check(out[rest, h], want, bound)
        # and the token itself chooses one key
        best = (q[at, h].double() @ kk[h].t()).argmax()
        du.check(out[at, h], vv[h, best], vv[h, best].abs() * (2.0 ** -7 + 1.5e-4))


# ------------------------------------------------------------------ the tile kernel at the ends of its ranges


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("dtype,kind", [(BF, None), (FP, None), (BF, I8), (BF, E4), (FP, I8)],
                         ids=["bf16", "fp16", "bf16-int8", "bf16-e4m3", "fp16-int8"])
@pytest.mark.parametrize("mul,qmul", [(1e-4, 2.0), (30.0, 20.0), (1.0, 0.0)])
def test_magnitudes(kernel, n, dtype, kind, mul, qmul):
    """Caches of tiny and large values; logits so large that the softmax is a choice; equal logits."""
    g, H, d, page = gen(10), 8, 128, 32
    ns, lens = [n, n], [n + 999, n + 257]
    k, v, ks, vs, table = du.make_cache(g, lens, H, page, d, dtype, kind, mul=mul)
    q = rnd(g, 2 * n, H, d, mul=qmul, dtype=dtype)
    cache = solattn.PagedCache(k, v, ks, vs)
    ws = solattn.alloc_paged_workspace(cache, 2, H, 2 * n)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of(ns), du.ints(lens), max_new=n, workspace=ws))
    assert solattn.solattn_get_status(ws) == 0
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens, True, dtype)
    du.check(out, want, bound)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [None, I8], ids=["16", "int8"])
def test_offsets_past_32_bits(kernel, n, kind):
    """A pool of over 2^32 elements: the sequence's pages lie at both ends of it."""
    d, page, Hkv, pool = 128, 128, 8, 34000
    assert pool * Hkv * page * d > 1 << 32
    g = gen(11)
    k, v = (torch.empty(pool, Hkv, page, d, dtype=kind or BF, device="cuda") for _ in range(2))
    ks, vs = (None, None) if kind is None else (torch.empty(pool, Hkv, page, device="cuda") for _ in range(2))
    ids = [pool - 1, 0, pool - 7, 33333, 16500, 1, pool - 2, 32800, 5]
    for i in ids:
        for x, s in ((k, ks), (v, vs)):
            r = rnd(g, Hkv, page, d)
            if kind is None:
                x[i] = r
            else:
                c, sc = du.quantise(r, kind)
                x[i], s[i] = c.to(kind), sc
    table, L = du.ints([ids]), len(ids) * page - 3
    q = rnd(g, n, Hkv, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    out = run_on(kernel, lambda: solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n))
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
    du.check(out, want, bound)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [None, E4], ids=["16", "e4m3"])
def test_sequences_that_share_pages(kernel, n, kind):
    """Sequences behind one prefix: the first pages of each table row are the same; and a table far wider than any of
    them needs, whose other entries name no page."""
    g, H, Hkv, d, page = gen(12), 16, 8, 128, 16
    prefix, ns = 160, [n, 1, n // 2]
    lens = [prefix + x for x in ns]
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, BF, kind)
    table[1:, :prefix // page] = table[0, :prefix // page]
    wide = torch.full((3, 8192), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rnd(g, sum(ns), H, d)
    cache = solattn.PagedCache(k, v, ks, vs)
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, ns, lens, True, BF)
    for t in (table, wide):
        ws = solattn.alloc_paged_workspace(cache, 3, H, sum(ns))
        call = lambda: solattn.solattn_paged_forward(q, cache, t, du.cu_of(ns), du.ints(lens), max_new=n, workspace=ws)  # noqa: E731
        out = run_on(kernel, call) if t is table else call()
        assert solattn.solattn_get_status(ws) == 0
        du.check(out, want, bound)


@pytest.mark.parametrize("kernel,n", KERNELS)
@pytest.mark.parametrize("kind", [None, I8], ids=["16", "int8"])
def test_two_graphs_with_one_workspace(kernel, n, kind):
    """Two captured calls that share a workspace, replayed in turn on one stream over new lengths and queries."""
    g, H, Hkv, d, page = gen(13), 8, 8, 128, 64
    lens = [n + 2000, n + 1, n + 700]
    ns = [n, 1, n]
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, BF, kind)
    cache = solattn.PagedCache(k, v, ks, vs)
    q = [rnd(g, sum(ns), H, d) for _ in range(2)]
    outs = [torch.empty_like(x) for x in q]
    cu, length = du.cu_of(ns), du.ints(lens)
    ws = solattn.alloc_paged_workspace(cache, 3, H, sum(ns))
    run_on(kernel, lambda: solattn.solattn_paged_forward(q[0], cache, table, cu, length, max_new=n, out=outs[0], workspace=ws))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            solattn.solattn_paged_forward(q[i], cache, table, cu, length, max_new=n, causal=i == 0, out=outs[i], workspace=ws)
    lens2 = [x - 1 if x > n else x for x in lens]
    length.copy_(du.ints(lens2))
    q[0].copy_(rnd(g, sum(ns), H, d))
    torch.cuda.synchronize()
    for _ in range(4):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert solattn.solattn_get_status(ws) == 0
    for i in range(2):
        want, bound = du.paged_oracle(q[i], k, v, ks, vs, table, ns, lens2, i == 0, BF)
        du.check(outs[i], want, bound)


def test_a_tile_that_takes_longer_than_a_wait_may():
    """2^28 keys (one page, named over and over) for as many tiles as there are SMs: a block is busy with its tile for
    more than the two seconds of an ordinary wait. (Equal scores: each row is the mean of the page's values, as far as sums of
    2^28 terms in 32 bits tell.)"""
    g, d, page, L = gen(14), 64, 128, 1 << 28
    n = 256 * torch.cuda.get_device_properties(0).multi_processor_count
    k, v = torch.zeros(1, 1, page, d, dtype=BF, device="cuda"), torch.ones(1, 1, page, d, dtype=BF, device="cuda")
    q = rnd(g, n, 1, d)
    table = torch.zeros(1, L // page, dtype=torch.int32, device="cuda")
    cache = solattn.PagedCache(k, v)
    ws = solattn.alloc_paged_workspace(cache, 1, 1, n)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out = solattn.solattn_paged_forward(q, cache, table, du.cu_of([n]), du.ints([L]), max_new=n, causal=False, workspace=ws)
    end.record()
    torch.cuda.synchronize()
    assert solattn.solattn_get_status(ws) == 0
    assert start.elapsed_time(end) > 2000, "too quick to show anything: more keys"
    assert (out > 0).all() and out.isfinite().all()
