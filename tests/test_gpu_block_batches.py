"""Block attention, block selection and the whole block path for batches of many query tokens:
the sizes where the attention's plan changes (32 tokens, one CTA a token, a thread a token), a
prompt's chunk, and the calls in a row.  Bounds: tests/paged_cases.py and, for scores and
selections, tests/test_gpu_blocks.py."""
import numpy as np
import pytest
import torch

from oracle import blocks as OB, dsa
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC
from tests.test_gpu_blocks import block_pool, check_scores, check_topk, dev, run_topk
from tests.test_gpu_paged import run_blocks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


def sampled(T):
    return sorted({0, 1, 31, 32, 33, T // 3, T // 2, 607, 608, 609, 1215, T - 2, T - 1} & set(range(T)))


@pytest.mark.parametrize("fmt,heads", [("fp8_ds_mla", 16), ("fp8_ds_mla", 128), ("e4m3", 32), ("bf16", 64)])
@pytest.mark.parametrize("T", [32, 33, 38, 149, 608, 609, 1217])
def test_listed_blocks_of_many_tokens(T, fmt, heads):
    """Lists of 0 to 7 blocks in any order, some of one token far longer than the others'."""
    first = T // 3
    wl = synth.make_workload(f"bb/{fmt}/{heads}/{T}", [first + 900, T - first + 300], [first, T - first], heads,
                             latent_format=fmt, layers=(("l", 64, False, None),))
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    rng = synth.stream(T, "bb/lists")
    k = 30
    blocks, count = np.full((T, k), -1, np.int32), np.zeros(T, np.int32)
    for t in range(T):
        have = (int(n_all[t]) + 63) // 64
        count[t] = min(have, k) if t in (first // 2, T - 1) else rng.integers(0, min(have, 7) + 1)
        blocks[t, :count[t]] = rng.permutation(have)[:count[t]]
    out, lse = run_blocks(PC.spoil_unused(wl), blocks, count)
    assert np.isfinite(out).all() and np.array_equal(np.isfinite(lse).all(1), count > 0)
    for t in sampled(T):
        PC.check(f"T {T} token {t}", out[t], lse[t],
                 PC.expect(wl, 0, t, OB.block_positions(blocks[t, :count[t]], int(n_all[t]))))


@pytest.mark.parametrize("T,pages,k", [(609, 40, 32), (2048, 1000, 32), (2048, 1025, 2048), (1000, 17000, 45)])
def test_selection_for_many_tokens(T, pages, k):
    """Every row against the oracle's order, with ties in it."""
    wl = synth.make_workload(f"bb/sel/{T}", [T], [T], 16)
    wl.ctx_len = np.array([pages * 64], np.int32)
    wl.block_table = np.zeros((1, pages), np.int32)
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    scores = np.round(synth.stream(T, "bb/scores").standard_normal((T, pages), dtype=np.float32) * 64) / 64
    blocks, count, status = run_topk(wl, scores, k)
    assert status == (sml.SML_OK, 0)
    check_topk(wl, scores, k, blocks, count, n_all)


@pytest.mark.parametrize("heads", [16, 128])
def test_a_prompts_chunk_over_selected_blocks(heads):
    """2,048 new tokens behind 6,144: the keys of every full page, scores, the 32 best blocks and
    the attention over them, in a row on one stream, each checked on what the step before it gave."""
    wl = synth.make_workload(f"bb/prompt/{heads}", [8192], [2048], heads, ssmax=True)
    dw = DeviceWorkload(wl)
    p, lay, T, k = dw.problem(0), dw.layers[0], wl.T, 32
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    full = wl.block_table[0, :wl.ctx_len[0] // 64].astype(np.int32)
    pool, pages = dev(block_pool(wl.num_pages)), dev(full)
    scores = torch.full((T, wl.max_pages), 123.0, device="cuda")
    blocks = torch.empty(T, k, dtype=torch.int32, device="cuda")
    count = torch.empty(T, dtype=torch.int32, device="cuda")
    out = torch.full((T, heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, heads), float("nan"), device="cuda")
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    sml.sml_block_keys_write(dw.index_cache, pages, pool, ws)
    sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, pool, scores, ws)
    sml.sml_block_topk(p, scores, blocks, count, ws)
    sml.sml_block_mla_decode(p, lay.q, dw.latent, blocks, count, out, lse, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    hp, hs = pool.cpu().numpy(), scores.cpu().numpy()
    assert np.array_equal(hp, OB.block_keys(wl.index_cache, full, block_pool(wl.num_pages))[0])
    check_scores(wl, hp, hs, n_all, tokens=range(0, T, 97))
    hb, hc = blocks.cpu().numpy(), count.cpu().numpy()
    check_topk(wl, hs, k, hb, hc, n_all)
    ho, hl = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(ho).all() and np.isfinite(hl).all()
    for t in sampled(T)[::1 if heads == 16 else 3]:
        PC.check(f"token {t}", ho[t], hl[t], PC.expect(wl, 0, t, OB.block_positions(hb[t, :hc[t]], int(n_all[t]))))
