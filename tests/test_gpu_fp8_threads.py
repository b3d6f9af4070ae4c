"""8-bit products from several host threads and after calls of other sizes."""
import subprocess
import sys
import threading

import pytest
import torch

from conftest import ROOT
from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _product(M, E, N, K, seed):
    """A call without an output of its own, and its result."""
    g = torch.Generator().manual_seed(seed)
    a, sa = B.fp8_quantize(torch.randn(M, K, generator=g).to(DEV))
    w, sw = B.fp8_quantize_weight(torch.randn(E, N, K, generator=g).to(DEV))
    out = torch.empty((M, N), device=DEV)
    if E == 1:
        return lambda: B.fp8_linear(a, sa, w[0], sw[0], out=out)
    off = torch.linspace(0, M, E + 1).int().to(DEV)
    return lambda: B.fp8_grouped_gemm(a, sa, w, sw, off, out=out)


def test_threads_with_different_numbers_of_groups():
    """What a kernel may take of shared memory is set for all calls: one thread's
    does not take it away from another's (their sizes grow with the groups)."""
    calls = [_product(4, 1, 256, 256, 1), _product(16, 1024, 128, 128, 2), _product(300, 1, 512, 128, 3),
             _product(4000, 20, 512, 128, 4)]
    want = [c().clone() for c in calls]
    failed = []

    def loop(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            try:
                for _ in range(3000):
                    out = calls[i]()
                torch.cuda.current_stream().synchronize()
                if not torch.equal(out, want[i]):
                    failed.append((i, "result"))
            except B.NVFP4Error as e:
                failed.append((i, str(e)))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert B.nvfp4moe_last_device_status() == 0


ORDER = """
import sys
import torch
sys.path.insert(0, %r)
from nvfp4_block_scaled_05_gb300 import binding as B
def product(M, E, N, K):
    g = torch.Generator().manual_seed(M)
    a, sa = B.fp8_quantize(torch.randn(M, K, generator=g).cuda())
    w, sw = B.fp8_quantize_weight(torch.randn(1, N, K, generator=g).cuda())
    if E == 1:
        return B.fp8_linear(a, sa, w[0], sw[0], out_dtype=torch.float32)
    off = torch.linspace(0, M, E + 1).int().cuda()
    return B.fp8_grouped_gemm(a, sa, w.repeat(E, 1, 1), sw.repeat(E, 1, 1), off, out_dtype=torch.float32)
shapes = [(1, 1, 4096, 7168), (12, 256, 1024, 7168), (12, 1024, 1024, 7168), (30, 1, 2048, 4096), (20, 1, 4096, 4096)]
if sys.argv[1] == "1":
    shapes.reverse()
out = {s: product(*s).cpu() for s in shapes}
assert B.nvfp4moe_last_device_status() == 0
torch.save(out, sys.argv[2])
"""


def test_the_bits_of_a_product_do_not_depend_on_the_calls_before_it(tmp_path):
    """In a process of its own each, products of many and of few groups in either order."""
    got = []
    for order in "01":
        path = str(tmp_path / order)
        subprocess.run([sys.executable, "-c", ORDER % ROOT, order, path], check=True, timeout=300)
        got.append(torch.load(path))
    for shape, a in got[0].items():
        assert torch.equal(a, got[1][shape]), shape
