"""What follows a wait that gives up in the attention over the whole cache and in the block scores:
every CTA winds down, the status word says SML_FAULT_TIMEOUT, and the next calls are right.

The library is built again with waits of a few polls (SML_WAIT_POLLS), so that they give up where
they stand: one poll at the first loads, hundreds in the middle of a piece, at its output or at the
next request's keys, wherever a warp comes to wait for longer.  Nothing is withheld: every load and
product that a CTA has begun completes, and is waited for before the CTA ends."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from oracle import blocks as OB, dsa
from sparse_mla_attention_indexer_b200 import build, sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC
from tests.test_gpu_blocks import check_scores, dev, scored

pytestmark = pytest.mark.gpu

POLLS = [1, 8, 40, 150, 600]


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """Path of the library for each number of polls (0: as it is)."""
    build.build()
    out = tmp_path_factory.mktemp("give_up")
    ours = ("paged", "blocks")

    def compile_one(job):
        polls, name = job
        obj = str(out / f"{name}{polls}.o")
        subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, f"-DSML_WAIT_POLLS={polls}", "-c",
                        os.path.join(build.CSRC, name + ".cu"), "-o", obj], check=True)
        return obj

    jobs = [(p, n) for p in POLLS for n in ours]
    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as ex:
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
    rest = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources()
            if os.path.basename(s)[:-3] not in ours]
    paths = {0: build.LIB}
    for p in POLLS:
        paths[p] = str(out / f"libsml{p}.so")
        subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-o", paths[p], *rest, *(objs[p, n] for n in ours)], check=True)
    old = sml._lib, sml.LIB_PATH
    yield paths
    sml._lib, sml.LIB_PATH = old


def use(libs, polls):
    sml._lib, sml.LIB_PATH = None, libs[polls]
    sml.lib()


def timed_out(ws, polls):
    """Reads the status: it has to be a timeout with one poll (no load is there at once)."""
    code, bits = sml.sml_read_device_status(ws)
    assert (code, bits) in ((sml.SML_ERR_TIMEOUT, sml.SML_FAULT_TIMEOUT), (sml.SML_OK, 0))
    assert polls > 1 or code == sml.SML_ERR_TIMEOUT
    return code == sml.SML_ERR_TIMEOUT


# One long piece for a CTA, several short ones, empty ones between; every format and head group.
@pytest.mark.parametrize("lens,qs", [([9000], [150]), ([300, 64, 1, 2000, 700], [40, 3, 1, 60, 50]), ([40000, 130], [1, 2])])
@pytest.mark.parametrize("fmt,heads", [("fp8_ds_mla", 16), ("fp8_ds_mla", 64), ("e4m3", 128), ("bf16", 16), ("bf16", 64)])
def test_paged_attention_gives_up_and_recovers(libs, fmt, heads, lens, qs):
    wl = synth.make_workload(f"giveup/{fmt}/{heads}/{len(lens)}", lens, qs, heads, latent_format=fmt,
                             layers=(("l", 64, False, None),))
    dw = DeviceWorkload(wl)
    p, q = dw.problem(0), dw.layers[0].q
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    use(libs, 0)
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    out = torch.empty(wl.T, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(wl.T, heads, device="cuda")
    sample = sorted({0, wl.T // 2, wl.T - 1})
    want = {t: PC.expect(wl, 0, t, np.arange(int(n_all[t]))) for t in sample}
    for polls in POLLS:
        use(libs, polls)
        for _ in range(3):
            sml.sml_paged_mla_decode(p, q, dw.latent, out, lse, ws)
            if not timed_out(ws, polls):
                for t in sample:
                    PC.check(f"{polls} polls, token {t}", out[t].float().cpu().numpy(), lse[t].cpu().numpy(), want[t])
        use(libs, 0)
        sml.sml_paged_mla_decode(p, q, dw.latent, out, lse, ws)
        assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
        for t in sample:
            PC.check(f"after {polls} polls, token {t}", out[t].float().cpu().numpy(), lse[t].cpu().numpy(), want[t])


@pytest.mark.parametrize("heads", [16, 128])
def test_block_attention_gives_up_and_recovers(libs, heads):
    wl = synth.make_workload(f"giveup/blocks/{heads}", [5000, 700], [50, 20], heads, layers=(("l", 64, False, None),))
    dw = DeviceWorkload(wl)
    p, q = dw.problem(0), dw.layers[0].q
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    blocks = np.stack([np.arange(9, dtype=np.int32)] * wl.T)
    count = np.arange(wl.T, dtype=np.int32) % 10                   # some of them none
    d_blocks, d_count = dev(blocks), dev(count)
    use(libs, 0)
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    out = torch.empty(wl.T, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(wl.T, heads, device="cuda")
    for polls in POLLS:
        use(libs, polls)
        for _ in range(3):
            sml.sml_block_mla_decode(p, q, dw.latent, d_blocks, d_count, out, lse, ws)
            timed_out(ws, polls)
        use(libs, 0)
        sml.sml_block_mla_decode(p, q, dw.latent, d_blocks, d_count, out, lse, ws)
        assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
        for t in (0, 9, 58, wl.T - 1):
            PC.check(f"after {polls} polls, token {t}", out[t].float().cpu().numpy(), lse[t].cpu().numpy(),
                     PC.expect(wl, 0, t, OB.block_positions(blocks[t, :count[t]], int(n_all[t]))))


@pytest.mark.parametrize("lens,qs", [([8300], [1]), ([9000, 9000, 500, 8300, 20000], [40, 300, 5, 30, 600])])
def test_block_scores_give_up_and_recover(libs, lens, qs):
    """One request and token a CTA, and CTAs that go from one request's keys to the next's."""
    use(libs, 0)
    wl, pool = scored(f"giveup/scores/{len(lens)}", lens, qs)
    dw = DeviceWorkload(wl)
    p, lay, d_pool = dw.problem(0), dw.layers[0], dev(pool)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    scores = torch.empty(wl.T, wl.max_pages, device="cuda")
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    for polls in POLLS:
        use(libs, polls)
        for _ in range(3):
            sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, d_pool, scores, ws)
            timed_out(ws, polls)
        use(libs, 0)
        scores.fill_(123.0)
        sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, d_pool, scores, ws)
        assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
        check_scores(wl, pool, scores.cpu().numpy(), n_all, tokens=sorted({0, wl.T // 2, wl.T - 1}))
