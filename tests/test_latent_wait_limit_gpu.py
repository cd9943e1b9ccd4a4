"""The latent attention's bounded waits, exercised without faulting the GPU.

In a test-only build (-DMTPATTN_WAIT_CYCLES=200000, about 0.1 ms of SM clocks, and -DMTPATTN_TEST_STALL, which
makes the fetch leave out the first block of keys of the first unit) the wait for that block runs out: its CTA
raises its abort flag, every role winds down (waiting, again with a limit, for its own copies and products in
flight), the tensor memory is freed and the call reports MTPATTN_ERR_TIMEOUT in its status word. The join then
follows no note that the CTA did not leave, whatever stands in the workspace. A second call returns the same way,
and the product library, on the same workspace, gives what it gave before. It runs in a child process, so that the
test build's kernels stay out of the other tests' process.
"""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = textwrap.dedent("""
    import ctypes, sys
    import torch
    sys.path.insert(0, {root!r})
    from paged_fp8_speculative_gb300 import _lib, api
    from tests.test_latent_gpu import Batch

    stall = _lib.load({path!r})
    for lens, nodes, heads in (([30000, 700], [4, 2], 16), ([100], [3], 5), ([9000, 8000], [1, 1], 128)):
        b = Batch(lens, nodes, heads, seed=3)
        want = b.run()
        b.check(want)
        size = api.mtp_latent_attn_workspace_size(len(lens), b.total, heads, b.bt.shape[1])
        d = torch.full((1,), 0.75, device="cuda")
        for fill in (0x00, 0x01, 0x7F, 0xFF):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            out = torch.zeros_like(want)
            b.status.zero_()
            rc = stall.mtp_latent_attn_fwd(
                b.q.data_ptr(), b.q.stride(0), b.q.stride(1), b.cache.data_ptr(), b.cache.shape[0], b.bt.data_ptr(),
                b.bt.shape[1], b.sl.data_ptr(), b.cu.data_ptr(), None, len(lens), b.total, heads, d.data_ptr(),
                ctypes.c_float(b.scale), ws.data_ptr(), ws.numel(), out.data_ptr(), out.stride(0), out.stride(1),
                b.status.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
            assert rc == 0, rc
            torch.cuda.synchronize()                      # the call returned
            assert b.status.item() & api.ERR_TIMEOUT, b.status.item()
            assert torch.equal(b.run(workspace=ws), want)
    print("latent wait-limit test ok")
""")


def test_a_wait_that_runs_out_returns_the_timeout_status():
    from paged_fp8_speculative_gb300 import build
    path = os.path.join(build.BUILD, "libmtpattn_stall_latent.so")
    build.build(extra_flags=("-DMTPATTN_WAIT_CYCLES=200000", "-DMTPATTN_TEST_STALL=1"), lib_path=path)
    r = subprocess.run([sys.executable, "-c", _CHILD.format(root=ROOT, path=path)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "latent wait-limit test ok" in r.stdout
