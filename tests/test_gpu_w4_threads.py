"""mla_linear_w4 from several host threads at once: the library promises that its calls are safe there."""
import os
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from launch_util import launches_of  # noqa: E402
from test_gpu_w4 import DEV, _weight  # noqa: E402

from mla_latent_kv_absorb_gb300 import binding  # noqa: E402

pytestmark = pytest.mark.gpu


def _job(n, k):
    """(arguments of the call, its output, what it launches, everything that has to stay)."""
    w, _ = _weight(1, n, k, "int4", 128, False, n)
    x = torch.randn(1, k, generator=torch.Generator().manual_seed(k)).bfloat16().to(DEV)
    out = torch.empty(1, n, dtype=torch.bfloat16, device=DEV)
    stream = torch.cuda.Stream()
    launch, = launches_of(lambda: binding.mla_linear_w4(x, w, out))
    args = (1, x.data_ptr(), k, k, w._ref, out.data_ptr(), n, n, stream.cuda_stream)
    return args, out, launch, (w, x, stream)


def test_the_limit_of_shared_memory_goes_by_the_kernel():
    """A kernel's limit of dynamic shared memory is the process's, not the call's: calls of the same
    kernel that need different amounts must set the same, or one thread's launch fails where another
    has lowered it in between."""
    large, small = _job(1536, 7168)[2], _job(4096, 4096)[2]
    assert large.name == small.name and large.smem > small.smem
    assert large.most_smem == small.most_smem >= large.smem


def test_products_from_two_threads():
    """Two such products called over and over from two threads on two streams: every call succeeds and
    gives the bits of a call alone."""
    jobs = [_job(1536, 7168), _job(4096, 4096)]
    call, status, wants = binding.lib().mla_linear_w4, [0, 0], []
    for args, out, _, _ in jobs:
        assert call(*args) == binding.MLA_OK
        torch.cuda.synchronize()
        wants.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(i):
        args = jobs[i][0]
        start.wait()
        for _ in range(20000):
            status[i] = call(*args) or status[i]

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [binding.MLA_OK] * 2
    for (_, out, _, _), want in zip(jobs, wants):
        assert torch.equal(out, want)
