"""What the binding takes for an address, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_mla_attention_indexer_b200 import build as sml_build, sml


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sml_build.build()
    sml.lib()


def test_addresses_are_tensors_ints_or_none():
    t = torch.zeros(4)
    assert sml._p(t) == t.data_ptr() and sml._p(4096) == 4096 and sml._p(None) is None


@pytest.mark.parametrize("bad", [b"\0" * 512, bytearray(512), "0x1000", 1.5, np.zeros(64, np.uint8), (ctypes.c_char * 64)()],
                         ids=lambda x: type(x).__name__)
def test_a_host_object_is_not_an_address(bad):
    """It raises before the library is called: ctypes would pass a bytes object's host address on."""
    with pytest.raises(AttributeError):
        sml._p(bad)
    p = sml.Problem(num_requests=1, num_tokens=1, num_heads=16, topk=1, rope_dim=64, max_pages=1, max_ctx=64, sm_scale=1.0,
                    cu_q=0x1000, ctx_len=0x1000, block_table=0x1000)
    ws = torch.empty(256, dtype=torch.uint8)
    with pytest.raises(AttributeError):
        sml.sml_paged_mla_decode(p, bad, torch.zeros(64 * 656, dtype=torch.uint8), None, None, ws)
    with pytest.raises(AttributeError):
        sml.sml_latent_cache_read(torch.zeros(0, dtype=torch.int32), torch.zeros(64 * 656, dtype=torch.uint8), bad)
