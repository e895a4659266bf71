"""Calls of the dense attention's and the cache's binding that have to be refused before the library sees
them (no GPU needed: tensors are stand-ins)."""
import pytest
import torch

from block_sparse_online_b200 import solattn
from tests.test_host_streams import ints, log, on_gpu, paged_cache, rows  # noqa: F401 (log is a fixture)


@pytest.mark.parametrize("bytes_", [0, 4, 64, 255])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8])
def test_a_status_word_needs_its_256_bytes(log, bytes_, dtype):  # noqa: F811
    """The library takes it by its address alone: a shorter buffer would be written behind its end."""
    short = on_gpu(torch.zeros(bytes_, dtype=dtype))
    args = ints(0, 1)[None], ints(0, 4), ints(9)
    with pytest.raises(ValueError, match="workspace"):
        solattn.solattn_cache_append(paged_cache(), rows(4, 2, 64), rows(4, 2, 64), *args, workspace=short)
    with pytest.raises(ValueError, match="workspace"):
        solattn.solattn_cache_read(paged_cache(), *args, rows(4, 2, 64), rows(4, 2, 64), workspace=short)
    assert log["launch"] == []
    solattn.solattn_cache_append(paged_cache(), rows(4, 2, 64), rows(4, 2, 64), *args, workspace=on_gpu(torch.zeros(256, dtype=dtype)))
    assert log["launch"] == [11]


@pytest.mark.parametrize("name", ["dense_common", "rows_kernel", "tile_kernel", "cache_kernel", "attn_kernel"])
def test_kernels_have_the_debug_builds_checks(name):
    """libsolattn_debug.so promises checks of the indices before an access, in every kernel."""
    src = open(solattn.library_path().rsplit("/", 1)[0] + f"/csrc/{name}.cuh").read()
    assert "SOLATTN_DCHECK" in src
