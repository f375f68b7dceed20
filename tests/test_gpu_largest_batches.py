"""The largest batches (65,535 query tokens, 65,535 requests), and calls whose first launch in a
process is captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import dsa
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


@pytest.mark.parametrize("lens,qs,window", [([65535], [65535], 100), ([1 + (i * 7) % 150 for i in range(65535)], [1] * 65535, 0),
                                            ([70000, 3], [65534, 1], 64)], ids=["one", "each", "two"])
def test_paged_attention_of_65535_tokens(lens, qs, window):
    """Every request reads the same pages; queries repeat every 97 tokens."""
    wl = synth.make_workload("largest", [64 * max(-(-n // 64) for n in lens)], [1], 16, layers=(("l", 64, False, None),))
    wl.ctx_len = np.array(lens, np.int32)
    wl.cu_q = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    wl.block_table = np.repeat(wl.block_table, len(lens), 0)
    x = synth.to_bf16_bits(synth.stream(0, "largest/q").standard_normal((97, 16, 576), dtype=np.float32))
    wl.layers[0].q = x[np.arange(wl.T) % 97]
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    out = torch.full((wl.T, 16, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((wl.T, 16), float("nan"), device="cuda")
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    sml.sml_paged_mla_decode(p, dw.layers[0].q, dw.latent, out, lse, ws, window=window)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    for t in (0, 1, 607, 608, 32767, 32768, 65533, 65534):
        n = int(n_all[t])
        PC.check(f"token {t}", out[t].float().cpu().numpy(), lse[t].cpu().numpy(),
                 PC.expect(wl, 0, t, np.arange(max(0, n - window) if window else 0, n)))


CAPTURED = """
import torch
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
wl = synth.make_workload("captured", [5000, 777, 64], [1, 3, 1], 32)
dw = DeviceWorkload(wl)
p, lay, d = dw.problem(0), dw.layers[0], "cuda"
ws = torch.zeros(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device=d)
pool = torch.zeros(-(-wl.num_pages // 64) * synth.INDEX_PAGE, dtype=torch.uint8, device=d)
pages = torch.arange(wl.num_pages, dtype=torch.int32, device=d)
slot = torch.arange(300, dtype=torch.int32, device=d)
made = [torch.zeros(s, dtype=t, device=d) for s, t in (
    ((wl.T, 32, 512), torch.bfloat16), ((wl.T, 32), torch.float32), ((wl.T, 32, 512), torch.bfloat16), ((wl.T, 32), torch.float32),
    ((wl.T, wl.max_pages), torch.float32), ((wl.T, 9), torch.int32), ((wl.T,), torch.int32), ((300, 512), torch.bfloat16),
    ((300, 128), torch.bfloat16))]
out, lse, bout, blse, scores, blocks, count, c, k = made
def calls():
    sml.sml_paged_mla_decode(p, lay.q, dw.latent, out, lse, ws)
    sml.sml_block_keys_write(dw.index_cache, pages, pool, ws)
    sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, pool, scores, ws)
    sml.sml_block_topk(p, scores, blocks, count, ws)
    sml.sml_block_mla_decode(p, lay.q, dw.latent, blocks, count, bout, blse, ws)
    sml.sml_latent_cache_read(slot, dw.latent, c)
    sml.sml_indexer_k_cache_read(slot, dw.index_cache, k)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in made]
for t in made:
    t.zero_()
calls()
torch.cuda.synchronize()
assert sml.sml_read_device_status(ws) == (0, 0)
assert all(t.view(torch.uint8).any() for t in made)
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, made))
"""


def test_first_calls_of_a_process_may_be_captured():
    subprocess.run([sys.executable, "-c", CAPTURED], cwd=ROOT, check=True, timeout=300)
