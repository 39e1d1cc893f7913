"""Tensors of no rows, whatever strides they carry, in the calls that take T rows."""
import numpy as np
import pytest
import torch

import __graft_entry__
from sparse_kv_cache_retrieval_gb300 import binding as B

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()


def test_an_empty_tensor_has_no_strides(monkeypatch):
    empty = torch.from_numpy(np.zeros((0, 8, 128), np.float32)).to(torch.bfloat16)
    assert empty.stride() == (0, 0, 0)
    B._device()
    monkeypatch.setattr(B, "_device", lambda: -1)           # the device of a tensor on the host
    assert B._rows("q", empty, 0, 8, 128, None, -1) == (0, 1024)
    ws = torch.zeros(B.spc_kv4_chunk_attn_workspace_size(0, 1, 8, 8, 128) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    B.spc_kv4_chunk_attn(empty, FAKE, FAKE, FAKE, FAKE, 0, 1, 8, 8, 128, 2, 16, 2, 0.1, None, None, ws, stream=0)
    for t in (empty[:, :4], empty[..., :64], empty.float()):
        with pytest.raises(ValueError):
            B._rows("q", t, 0, 8, 128, None, -1)
