"""The bounds-checked build (libsolattn_debug.so) on the dense attention and the cache: on valid inputs of every path no
check fires, and outputs, pages and scales equal the release build's bit for bit."""
import os

import pytest
import torch

from block_sparse_online_b200 import solattn
from tests import dense_util as du

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(solattn.DEBUG_LIB_PATH):
        from block_sparse_online_b200 import build
        build.build(debug=True)
    yield
    solattn.load_library()  # back to the release build


def both(call, ws):
    """call() with each build: equal results, status 0."""
    got = []
    for path in (None, solattn.DEBUG_LIB_PATH):
        solattn.load_library(path) if path else solattn.load_library()
        got.append([x.clone() for x in call()])
        assert solattn.solattn_get_status(ws) == 0, path
    solattn.load_library()
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(3, 4, 2, 7, 300, 128, [300, 0, 129]), (1, 2, 2, 3, 0, 64, None), (2, 6, 2, 3000, 200, 64, [200, 13]),
                                   (1, 8, 8, 2048, 769, 128, None)], ids=str)
def test_cross(shape, dtype):
    B, H, Hkv, Nq, Nk, d, lens = shape
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(B, h, n, d, generator=g, device="cuda").to(dtype) for h, n in ((H, Nq), (Hkv, Nk), (Hkv, Nk)))
    ws = solattn.alloc_cross_workspace(B, H, Hkv, Nq, Nk, d)
    both(lambda: [solattn.solattn_cross(q, k, v, key_len=None if lens is None else du.ints(lens), workspace=ws)], ws)


@pytest.mark.parametrize("dtype,kind", [(BF, None), (FP, None), (BF, I8), (FP, E4)], ids=["bf16", "fp16", "bf16-int8", "fp16-e4m3"])
@pytest.mark.parametrize("shape", [([1, 1, 0, 1], [1, 300, 7, 5025], 16, 4, 64, 128), ([5, 3], [5, 259], 6, 2, 16, 64),
                                   ([700, 1, 0, 300], [900, 1, 5, 3000], 16, 8, 16, 128), ([2000], [2000], 6, 2, 128, 64)], ids=str)
def test_cache_and_attention(shape, dtype, kind):
    ns, lens, H, Hkv, page, d = shape
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v, ks, vs, table = du.make_cache(g, lens, Hkv, page, d, dtype, kind)
    cache = solattn.PagedCache(k, v, ks, vs)
    total = sum(ns) + 2
    cu, length = du.cu_of(ns), du.ints(lens)
    q = torch.randn(total, H, d, generator=g, device="cuda").to(dtype)
    new = [torch.randn(total, Hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2)]
    ws = solattn.alloc_paged_workspace(cache, len(ns), H, total)

    def call():
        solattn.solattn_cache_append(cache, *new, table, cu, length, workspace=ws)
        outs = [torch.zeros_like(new[0]), torch.zeros_like(new[1])]
        solattn.solattn_cache_read(cache, table, cu, length, *outs, workspace=ws)
        for causal in (True, False):
            outs.append(solattn.solattn_paged_forward(q, cache, table, cu, length, max_new=max(ns), causal=causal, workspace=ws,
                                                      out=torch.zeros_like(q)))
        return outs + [x for x in (k, v, ks, vs) if x is not None]

    both(call, ws)
