"""The tree attention's bounded waits, exercised without faulting the GPU.

In a test-only build (-DMTPATTN_WAIT_CYCLES=200000, about 0.1 ms of SM clocks, and
-DMTPATTN_TEST_STALL, which makes CTA 0's V producer skip its first half tile) the widening warps'
wait for those codes runs out: the CTA raises its abort flag, every role winds down (waiting, again
with a limit, for its own copies and products in flight), the tensor memory is freed and the call
reports MTPATTN_ERR_TIMEOUT in its status word.  The join then follows no note that the CTA did not
leave, whatever stands in the workspace.  A second call returns the same way, and the product
library, on the same workspace, gives what it gave before.  It runs in a child process, so that the test
build's kernels stay out of the other tests' process.
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
    from tests.test_tree_attn_gpu import Batch, check, run

    stall = _lib.load({path!r})
    for lens, nodes in (([30000, 700], [20, 5]), ([100], [3])):
        batch = Batch(lens, nodes, 1, 16, seed=3)
        want = run(batch)
        check(want, batch)
        a = batch.device()
        q, bt, n = a["q"], a["block_tables"], len(lens)
        size = api.mtp_tree_attn_workspace_size(n, q.shape[0], 16, 1, bt.shape[1])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for fill in (0x00, 0x01, 0x7F, 0xFF):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            out = torch.zeros_like(q)
            status.zero_()
            rc = stall.mtp_tree_attn_fwd(
                q.data_ptr(), q.stride(0), q.stride(1), a["k_cache"].data_ptr(), a["v_cache"].data_ptr(),
                a["k_cache"].shape[0], bt.data_ptr(), bt.shape[1], a["seq_lens"].data_ptr(),
                a["cu_seqlens_q"].data_ptr(), a["tree_mask"].data_ptr(), n, q.shape[0], 16, 1,
                a["k_descale"].data_ptr(), a["v_descale"].data_ptr(), ctypes.c_float(a["softmax_scale"]),
                ws.data_ptr(), ws.numel(), out.data_ptr(), out.stride(0), out.stride(1), status.data_ptr(),
                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
            assert rc == 0, rc
            torch.cuda.synchronize()                      # the call returned
            assert status.item() & api.ERR_TIMEOUT, status.item()
            assert torch.equal(run(batch, workspace=ws), want)
    print("tree wait-limit test ok")
""")


def test_a_wait_that_runs_out_returns_the_timeout_status():
    from paged_fp8_speculative_gb300 import build
    path = os.path.join(build.BUILD, "libmtpattn_stall_tree.so")
    build.build(extra_flags=("-DMTPATTN_WAIT_CYCLES=200000", "-DMTPATTN_TEST_STALL=1"), lib_path=path)
    r = subprocess.run([sys.executable, "-c", _CHILD.format(root=ROOT, path=path)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "tree wait-limit test ok" in r.stdout
