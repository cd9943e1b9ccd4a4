"""Buffers that are taken as bytes from their first one on (workspaces, what the streaming read goes over): a tensor
whose elements are not all there, one after the other, is refused before anything is launched."""
from __future__ import annotations

import pytest
import torch

from paged_fp8_speculative_gb300 import api

I32 = dict(dtype=torch.int32)
SEVERAL = [torch.zeros(1, dtype=torch.uint8).expand(1 << 30),            # one byte that stands for many
           torch.zeros(1 << 16, dtype=torch.uint8)[::2], torch.zeros(64, 64).t()]


def calls():
    kv, table, lens = torch.zeros(5, 16, 2, 256, dtype=torch.uint8), torch.zeros(2, 2, **I32), torch.zeros(2, **I32)
    cu, q, one = torch.zeros(3, **I32), torch.zeros(3, 4, 256, dtype=torch.bfloat16), torch.ones(1)
    latent = torch.zeros(5, 16, 576, dtype=torch.uint8)
    return {
        "verify": lambda ws: api.mtp_verify_attn_fwd(q, kv, kv, table, lens, cu, one, one, 0.1, num_segments=2, workspace=ws),
        "tree": lambda ws: api.mtp_tree_attn_fwd(q, kv, kv, table, lens, cu, torch.zeros(3, dtype=torch.int64), one, one, 0.1,
                                                 workspace=ws),
        "latent": lambda ws: api.mtp_latent_attn_fwd(torch.zeros(3, 4, 576, dtype=torch.bfloat16), latent, table, lens, cu, one,
                                                     0.1, workspace=ws),
        "resize": lambda ws: api.mtp_cache_resize(kv, kv, table, lens, torch.zeros(5, **I32), lens, workspace=ws),
        "fork": lambda ws: api.mtp_cache_fork(kv, kv, table, lens, torch.zeros(5, **I32), lens, lens, workspace=ws),
    }


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("which", range(len(SEVERAL)))
def test_workspaces(name, which):
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        calls()[name](SEVERAL[which])


def test_streaming_read():
    with pytest.raises(ValueError, match="buf must be contiguous"):
        api.mtpattn_stream_read(torch.zeros(1).expand(1 << 20), torch.zeros(8, **I32), blocks=8)
    for sink in (torch.zeros(7, **I32), torch.zeros(1, **I32).expand(8), torch.zeros(8)):
        with pytest.raises(ValueError, match="sink"):
            api.mtpattn_stream_read(torch.zeros(1 << 10), sink, blocks=8)
