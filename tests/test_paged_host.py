"""The whole-cache operators' argument checks and the oracle's block rules, without a GPU."""
import ctypes

import numpy as np
import pytest

from oracle import blocks as OB, formats as F
from sparse_mla_attention_indexer_b200 import build as sml_build, sml, synth


@pytest.fixture(scope="module")
def L():
    sml_build.build()
    return sml.lib()


def _problem(**kw):
    base = dict(num_requests=2, num_tokens=3, num_heads=16, topk=2048, rope_dim=64, max_pages=4, max_ctx=256, ssmax=0,
                sm_scale=0.04, ssmax_s=0.4, ssmax_s_index=0.4, cu_q=0x1000, ctx_len=0x2000, block_table=0x3000)
    base.update(kw)
    return ctypes.byref(sml.Problem(**base))


LAT = sml.Cache(0x10000, 4, 0, 0.0)


def refused(code, want, *parts):
    assert code == want, (code, sml.sml_last_error())
    for part in parts:
        assert part in sml.sml_last_error(), sml.sml_last_error()


def test_stage_constant_and_workspace_size(L):
    import re
    assert int(re.search(r"#define SML_STAGE_PAGED (\d+)", open(sml.HEADER, encoding="utf-8").read()).group(1)) == \
        sml.SML_STAGE_PAGED
    sizes = [L.sml_workspace_size(_problem(num_heads=h), sml.SML_STAGE_PAGED) for h in (16, 32, 64, 128)]
    assert all(s > 0 and s % 256 == 0 for s in sizes)
    # neither the batch nor the context enters it
    big = _problem(num_requests=65535, num_tokens=65535, max_ctx=1 << 30, max_pages=1 << 24)
    assert L.sml_workspace_size(big, sml.SML_STAGE_PAGED) == sizes[0]
    assert L.sml_workspace_size(_problem(), 6) == 0 and "stage" in sml.sml_last_error()


def test_paged_attention_refuses_without_cuda(L):
    args = (0x1000, LAT, 0, 0x2000, 0x3000, 0x100, 1 << 40, None)
    refused(L.sml_paged_mla_decode(_problem(num_heads=24), *args), sml.SML_ERR_UNSUPPORTED, "num_heads")
    refused(L.sml_paged_mla_decode(None, *args), sml.SML_ERR_INVALID_ARG, "problem is NULL")
    refused(L.sml_paged_mla_decode(_problem(), 0x1008, sml.Cache(0x10001, 0, 9, 0.0), -1, 0x2004, None, None, 0, None),
            sml.SML_ERR_INVALID_ARG, "q NULL or not 16-B", "latent.base", "latent.num_pages", "latent.format", "window < 0",
            "out NULL or not 16-B", "lse is NULL", "workspace is NULL")
    refused(L.sml_paged_mla_decode(_problem(), 0x1000, LAT, 0, 0x2000, 0x3000, 0x100, 1000, None),
            sml.SML_ERR_WORKSPACE, "needs")
    refused(L.sml_paged_mla_decode(_problem(), 0x1000, LAT, 0, 0x2000, 0x3000, 0x180, 1 << 40, None),
            sml.SML_ERR_WORKSPACE, "256-B")
    refused(L.sml_paged_mla_decode(_problem(), 0x1000, sml.Cache(0x10000, 1 << 26, 0, 0.0), 0, 0x2000, 0x3000, 0x100,
                                   1 << 40, None), sml.SML_ERR_UNSUPPORTED, "exceed int32")
    refused(L.sml_paged_mla_decode(_problem(), 0x1000, sml.Cache(0x10000, 4, sml.SML_LATENT_E4M3, 0.0), 0, 0x2000,
                                   0x3000, 0x100, 1 << 40, None), sml.SML_ERR_INVALID_ARG, "latent.scale")


def test_block_attention_refuses_without_cuda(L):
    refused(L.sml_block_mla_decode(_problem(), 0x1000, LAT, None, None, 0, 0x2000, 0x3000, 0x100, 1 << 40, None),
            sml.SML_ERR_INVALID_ARG, "blocks is NULL", "blocks_len is NULL", "max_blocks < 1")
    refused(L.sml_block_mla_decode(_problem(), 0x1000, LAT, 0x10, 0x20, (1 << 24) + 1, 0x2000, 0x3000, 0x100, 1 << 40,
                                   None), sml.SML_ERR_UNSUPPORTED, "max_blocks > 2^24")


def test_block_selection_refuses_without_cuda(L):
    index, pool = sml.Cache(0x10000, 129, 0, 0.0), sml.Cache(0x20000, 2, 0, 0.0)
    refused(L.sml_block_keys_write(index, 0x1002, 3, pool, 0x80, None), sml.SML_ERR_INVALID_ARG, "pages NULL or not 4-B",
            "fewer rows", "workspace not 256-B")
    refused(L.sml_block_keys_write(sml.Cache(None, 0, 1, 0.0), None, -1, pool, None, None), sml.SML_ERR_INVALID_ARG,
            "n < 0", "index_cache.base", "index_cache.num_pages", "index_cache.format")
    assert L.sml_block_keys_write(sml.Cache(0x10000, 128, 0, 0.0), None, 0, pool, None, None) == sml.SML_OK
    refused(L.sml_block_scores(_problem(), 0x1001, None, 0x1004, sml.Cache(0x10000, 1, 2, 0.0), None, None, None),
            sml.SML_ERR_INVALID_ARG, "iq8", "iq_scale", "iw", "block_cache.format", "scores")
    refused(L.sml_block_topk(_problem(), None, 2049, None, None, 0x10, None), sml.SML_ERR_INVALID_ARG, "scores",
            "num_blocks", "blocks is NULL", "blocks_len is NULL", "workspace not 256-B")
    refused(L.sml_block_topk(_problem(), 0x10, 0, 0x10, 0x10, None, None), sml.SML_ERR_UNSUPPORTED, "num_blocks")


def test_reading_back_refuses_without_cuda(L):
    refused(L.sml_latent_cache_read(None, 5, LAT, 0x1008, 0x1004, 0x10, None), sml.SML_ERR_INVALID_ARG, "slot",
            "c NULL or not 16-B", "k_pe not 16-B", "workspace not 256-B")
    refused(L.sml_indexer_k_cache_read(0x1000, -2, sml.Cache(0x10000, 1 << 26, 0, 0.0), None, None, None),
            sml.SML_ERR_INVALID_ARG, "n < 0", "k NULL", "exceed int32")
    assert L.sml_latent_cache_read(None, 0, LAT, None, None, None, None) == sml.SML_OK
    assert L.sml_indexer_k_cache_read(None, 0, LAT, None, None, None) == sml.SML_OK


def test_oracle_block_key_of_equal_and_opposite_keys():
    """64 equal keys give that key; 32 and their negatives give zero under scale 1."""
    page = np.zeros(F.INDEXER_PAGE_BYTES, dtype=np.uint8)
    codes = synth.to_e4m3(np.linspace(-448, 448, 128, dtype=np.float32))
    page[:8192] = np.tile(codes, 64)
    page[8192:] = np.full(64, 0.5, dtype="<f4").view(np.uint8)
    pool, bad = OB.block_keys(page, [0, -1], np.full(F.INDEXER_PAGE_BYTES, 9, dtype=np.uint8))
    assert not bad and np.array_equal(pool[:128], codes) and pool[8192:8196].view("<f4")[0] == np.float32(0.5)
    assert (pool[128:8192] == 9).all()
    page[:8192].reshape(64, 128)[::2] ^= 0x80
    pool, _ = OB.block_keys(page, [0], pool)
    assert (F.decode_e4m3(pool[:128]) == 0).all() and pool[8192:8196].view("<f4")[0] == 1


def test_oracle_block_selection():
    assert list(OB.block_topk_row(np.array([3., 1, 2, 9]), 193, 3)) == [0, 2, 3]      # candidates 0..2, then block 3
    assert list(OB.block_topk_row(np.array([3., 1, 2, 9]), 192, 3)) == [0, 1, 2]      # candidates 0..1
    assert list(OB.block_topk_row(np.array([np.nan, 1, 1]), 193, 2)) == [1, 3]
    assert list(OB.block_topk_row(np.array([5.]), 64, 4)) == [0] and len(OB.block_topk_row(np.array([5.]), 0, 4)) == 0
    assert list(OB.block_positions([2, 0], 130)) == [128, 129] + list(range(64))
