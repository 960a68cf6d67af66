"""Paged cache without a GPU: what its binding needs of torch, and limits the C calls state."""
import os
import subprocess
import sys

import pytest

from free_block_sparse_mean_b200 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_package_imports_with_a_torch_that_has_no_cuda():
    """Such a torch lacks the CUDA functions of torch._C: they are only looked up by a call."""
    code = ("import torch\n"
            "for name in [x for x in dir(torch._C) if x.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import free_block_sparse_mean_b200 as sa\n"
            "print(sa.sparse_attn_tree_fwd.__name__)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == "sparse_attn_tree_fwd"


@pytest.mark.parametrize("layers", [1, 3])
def test_one_array_as_both_caches_is_not_moved_in(layers):
    """Keys and values are moved by threads of their own: in one array they would overtake each other."""
    p = 1 << 20
    cache = _lib.SaCache(pages=4, page_size=16, Hkv=2, d=64, dtype=_lib.SA_BF16, page_stride=2048, token_stride=128,
                         head_stride=64)
    step = _lib.SaStep(R=2, n=8, width=3, max_new=4, words=0, starts=p, lens=p, granted=None, table=p, mask=None)
    assert _lib.load().sparse_attn_cache_accept(p, p, cache, layers, 8192, step, p, 4, p, None) == 1
