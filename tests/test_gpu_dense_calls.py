"""Calls of the dense attention and cache entry points in ways that a user may make them: streams of their own, no
workspace, at once with other work."""
import pytest
import torch

from block_sparse_online_b200 import solattn
from tests import dense_util as du

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, mul=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * mul).to(dtype)


def overwrite(need):
    """What the caller does next on its own stream: buffers of the workspace's size, filled with ones."""
    for _ in range(4):
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)


@pytest.mark.parametrize("n", [3, 900])
def test_streams_without_workspaces(n):
    """Two streams, no workspace and no output given, split items (so that parts live in the workspace), while the
    current stream takes and fills buffers of the same size."""
    g = gen(101)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    xs = [[rnd(g, 1, 4, m, 128) for m in (n, 5000, 5000)] for _ in range(2)]
    need = solattn.solattn_cross_workspace_size(1, 4, 4, n, 5000, 128)
    overwrite(need)
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)  # about a millisecond: the call is still queued while the next lines run
            outs.append(solattn.solattn_cross(*x, stream=s))
            overwrite(need)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want = [du.cross_oracle(*x, None, BF) for x in xs]
    for i, o in enumerate(outs):
        du.check(o, *want[i % 2])


@pytest.mark.parametrize("n", [1, 300])
def test_paged_stream_without_workspaces(n):
    """Append, attend and read back on a stream of their own."""
    g, H, Hkv, d, page, L = gen(102), 4, 2, 128, 32, 3000
    k, v, ks, vs, table = du.make_cache(g, [L], Hkv, page, d, BF, torch.int8)
    cache = solattn.PagedCache(k, v, ks, vs)
    cu, length = du.cu_of([n]), du.ints([L])
    q, new = rnd(g, n, H, d), (rnd(g, n, Hkv, d), rnd(g, n, Hkv, d))
    need = solattn.solattn_paged_workspace_size(1, H, Hkv, n, d)
    back = torch.empty_like(new[0]), torch.empty_like(new[1])
    overwrite(need)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
    solattn.solattn_cache_append(cache, *new, table, cu, length, stream=s)
    overwrite(256)
    out = solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=n, stream=s)
    overwrite(need)
    solattn.solattn_cache_read(cache, table, cu, length, *back, stream=s)
    overwrite(256)
    torch.cuda.synchronize()
    want, bound = du.paged_oracle(q, k, v, ks, vs, table, [n], [L], True, BF)
    du.check(out, want, bound)
    for x, y in zip(new, back):
        codes, sc = du.quantise(x, torch.int8)
        assert torch.equal(y, (codes.float() * sc[..., None]).to(BF))


def test_operator_stream_without_workspace():
    """The routed operator's call the same way, against its own result on the current stream."""
    g = gen(103)
    q, k, v = (rnd(g, 1, 4, 4096, 128) for _ in range(3))
    want, kept, _ = solattn.solattn_forward(q, k, v, 128, 128, 2.0)
    need = solattn.solattn_workspace_size(1, 4, 4096, 128, 128, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
    out, kept2, _ = solattn.solattn_forward(q, k, v, 128, 128, 2.0, stream=s)
    overwrite(need)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kept, kept2)


def test_everything_given_on_a_stream():
    """With every tensor given a call takes the short path on a given stream too: it is queued there, not on the current one."""
    g, H, d, page, L, n = gen(104), 4, 128, 16, 300, 5
    q, k, v = (rnd(g, 1, H, m, d) for m in (n, L, L))
    kp, vp, ks, vs, table = du.make_cache(g, [L], H, page, d, BF, torch.int8)
    cache = solattn.PagedCache(kp, vp, ks, vs)
    cu, length = du.cu_of([n]), du.ints([L])
    pq, new = rnd(g, n, H, d), rnd(g, n, H, d)
    outs = [torch.zeros_like(x) for x in (q, pq, new, new)]
    ws, pws = solattn.alloc_cross_workspace(1, H, H, n, L, d), solattn.alloc_paged_workspace(cache, 1, H, n)
    s = torch.cuda.Stream()

    def calls():
        solattn.solattn_cross(q, k, v, out=outs[0], workspace=ws, stream=s)
        solattn.solattn_cache_append(cache, new, new, table, cu, length, workspace=pws, stream=s)
        solattn.solattn_paged_forward(pq, cache, table, cu, length, n, True, outs[1], pws, s)
        solattn.solattn_cache_read(cache, table, cu, length, outs[2], outs[3], workspace=pws, stream=s)

    torch.cuda.synchronize()
    calls()  # loads the kernels
    torch.cuda.synchronize()
    assert not any(bool((x == 0).all()) for x in outs)
    for x in outs:
        x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(500_000_000)  # about a quarter of a second
    calls()
    torch.cuda.current_stream().synchronize()
    early = [bool((x == 0).all()) for x in outs]
    s.synchronize()
    assert all(early) and solattn.solattn_get_status(ws) == 0 and solattn.solattn_get_status(pws) == 0
    want, bound = du.cross_oracle(q, k, v, None, BF)
    du.check(outs[0], want, bound)
    want, bound = du.paged_oracle(pq, kp, vp, ks, vs, table, [n], [L], True, BF)
    du.check(outs[1], want, bound)
    codes, sc = du.quantise(new, torch.int8)
    for x in outs[2:]:
        assert torch.equal(x, (codes.float() * sc[..., None]).to(BF))
