"""The host parts (block allocator, prefix cache) of the package on a torch
build without CUDA, which lacks torch's private CUDA attributes."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from paged_kv_cache_64_gb300 import api, build
build.build()
a = api.BlockAllocator(4, 16)
a.add(1)
assert a.append(1, 17)[0] == list(range(17))
assert api.PrefixCachePool(4, 16).lookup([1, 2, 3]) == 0
assert api.int4_pool_shape(4, 2, 16, 128) == (4, 2, 1088)
print("imported")
"""


def test_import_and_host_parts():
    done = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                          timeout=600)
    assert done.returncode == 0 and done.stdout.endswith("imported\n"), done.stderr[-2000:]
