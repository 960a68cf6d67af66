"""Paged cache without a GPU: what its binding needs of torch, and limits the C calls state."""
import os
import subprocess
import sys

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
