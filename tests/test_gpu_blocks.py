"""Block keys, block scores and block selection on the GPU against the oracle, the chain they
form with the attention, and cached rows read back."""
import numpy as np
import pytest
import torch

from oracle import blocks as OB, dsa, formats as F
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC, parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def status_ws():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    return ws


def block_pool(num_pages, fill=0):
    return np.full(-(-num_pages // 64) * F.INDEXER_PAGE_BYTES, fill, dtype=np.uint8)


@pytest.mark.parametrize("num_pages,n", [(1, 1), (64, 64), (65, 40), (3000, 2500)])
def test_block_keys_bytes(num_pages, n):
    index = synth._fill_index(0, f"bk/{num_pages}", num_pages)
    index.reshape(num_pages, -1)[0, :8192] = 0                       # an all-zero page: scale 1
    rng = synth.stream(0, f"bk/pages/{num_pages}")
    pages = rng.permutation(num_pages)[:n].astype(np.int32)
    pages[n // 2:n // 2 + 1] = -1
    pages[:1] = 0
    start = rng.integers(0, 256, block_pool(num_pages).size, dtype=np.uint8)
    want, bad = OB.block_keys(index, pages, start)
    assert not bad
    pool, ws = dev(start), status_ws()
    sml.sml_block_keys_write(dev(index), dev(pages), pool, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    assert np.array_equal(pool.cpu().numpy(), want)


def test_block_keys_bad_pages_twice_listed_and_empty():
    index = synth._fill_index(0, "bk/bad", 70)
    pages = np.array([3, 70, 3, -1, -5, 69], dtype=np.int32)
    want, bad = OB.block_keys(index, pages, block_pool(70, 7))
    assert bad
    pool, ws = dev(block_pool(70, 7)), status_ws()
    sml.sml_block_keys_write(dev(index), dev(pages), pool, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_ERR_DEVICE_FAULT, sml.SML_FAULT_PAGE)
    assert np.array_equal(pool.cpu().numpy(), want)
    sml.sml_block_keys_write(dev(index), torch.empty(0, dtype=torch.int32, device="cuda"), pool)
    assert np.array_equal(pool.cpu().numpy(), want)


def scored(name, lens, qs, **kw):
    """A workload with its block pool filled by the oracle."""
    wl = synth.make_workload(name, lens, qs, 16, **kw)
    used = [p for r in range(wl.B) for p in wl.block_table[r, :OB.candidates(wl.ctx_len[r])]]
    pool, _ = OB.block_keys(wl.index_cache, np.array(used, dtype=np.int64), block_pool(wl.num_pages, 0xFF))
    return wl, pool


def run_scores(wl, pool, vis=None):
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    if vis is not None:
        dw.vis = torch.from_numpy(vis).cuda()
        p.vis_len = dw.vis.data_ptr()
    lay = dw.layers[0]
    scores = torch.full((wl.T, wl.max_pages), 123.0, device="cuda")
    ws = status_ws()
    sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, dev(pool), scores, ws)
    return scores.cpu().numpy(), sml.sml_read_device_status(ws)


def check_scores(wl, pool, got, n_all, tokens=None):
    """Exact FP8 products; 128 of them, then 64 weighted heads, are summed in fp32: at most
    (128 + 64 + 4) roundings of 2^-24 of the summed terms' size, and as much again for the order."""
    v = wl.view(0)
    req = dsa.request_of_tokens(wl.cu_q)
    for t in range(wl.T) if tokens is None else tokens:
        n = int(n_all[t])
        c = dsa.ssmax_factor(wl.ssmax, wl.ssmax_s_index, n) if n else 0.0
        want, _ = OB.block_scores_row(v.iq8[t], v.iq_scale[t], v.iw[t], pool, wl.block_table[req[t]], n, c)
        pages = wl.block_table[req[t], :OB.candidates(n)].astype(np.int64)
        k_abs = np.abs(F.indexer_keys(pool, pages // 64, pages % 64))
        q_abs = np.abs(F.decode_e4m3(v.iq8[t])) * float(v.iq_scale[t])
        size = abs(c) * (np.abs(v.iw[t])[:, None] * (q_abs @ k_abs.T)).sum(0)
        d = np.abs(got[t, :len(want)] - want)
        assert (d <= 2 * 196 * 2.0 ** -24 * size).all(), f"token {t}: {d.max():.3e}"
        assert (got[t, len(want):] == 123.0).all(), f"token {t}: entries past the candidates written"


@pytest.mark.parametrize("lens,qs,ssmax", [([1, 64, 65, 128, 129, 8200, 3000], [1] * 7, False),
                                           ([700, 5, 8193, 260], [5, 5, 2, 70], True),
                                           ([20000], [1], True), ([130], [130], False)])
def test_block_scores(lens, qs, ssmax):
    wl, pool = scored(f"bs/{len(lens)}/{lens[0]}", lens, qs, ssmax=ssmax)
    got, status = run_scores(wl, pool)
    assert status == (sml.SML_OK, 0)
    check_scores(wl, pool, got, dsa.visible_lengths(wl.cu_q, wl.ctx_len))


def test_block_scores_of_a_long_chunk_are_the_same_every_time():
    """A prompt's chunk: CTAs of sixteen tokens, which take their queries and weights through
    buffers that are filled again while others are read; ten runs, one after the other and
    overlapping, give the same bits."""
    wl, pool = scored("bs/chunk", [20000, 700], [2900, 100], ssmax=True)
    dw = DeviceWorkload(wl)
    p, lay, ws, d_pool = dw.problem(0), dw.layers[0], status_ws(), dev(pool)
    runs = [torch.full((wl.T, wl.max_pages), 123.0, device="cuda") for _ in range(10)]
    for i, scores in enumerate(runs):
        sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, d_pool, scores, ws)
        if i < 4:
            torch.cuda.synchronize()
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    for scores in runs[1:]:
        assert torch.equal(scores, runs[0])
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    check_scores(wl, pool, runs[0].cpu().numpy(), n_all, tokens=list(range(0, wl.T, 41)) + list(range(2880, 2920)))


def test_block_scores_keep_nan():
    """A NaN in a block key's codes or scale gives that block NaN for every token, one in a query
    every block of that token; the rest is as without."""
    wl, pool = scored("bs/nan", [1000, 700], [2, 3])
    code, scale = [int(wl.block_table[0, j]) for j in (3, 7)]
    pool[code // 64 * F.INDEXER_PAGE_BYTES + code % 64 * 128 + 77] = 0xFF
    at = scale // 64 * F.INDEXER_PAGE_BYTES + F.INDEXER_KEYS_BYTES + scale % 64 * 4
    pool[at:at + 4] = np.frombuffer(np.float32(np.nan).tobytes(), dtype=np.uint8)
    wl.layers[0].iq8[3, 40, 5] = 0x7F
    got, status = run_scores(wl, pool)
    assert status == (sml.SML_OK, 0)
    assert np.isnan(got[:2, [3, 7]]).all()
    assert np.isnan(got[3, :OB.candidates(699)]).all()
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    check_scores(wl, pool, got, n_all, tokens=[2, 4])
    clean = np.delete(np.arange(OB.candidates(999)), [3, 7])
    want, _ = run_scores(wl, np.where(pool == 0xFF, 0, pool).astype(np.uint8))
    assert np.array_equal(got[0, clean], want[0, clean])


def test_block_scores_given_lengths_and_bad_pages():
    wl, pool = scored("bs/vis", [700, 1000], [3, 2])
    vis = np.array([0, 65, 700, 64, 513], dtype=np.int32)
    got, status = run_scores(wl, pool, vis)
    assert status == (sml.SML_OK, 0)
    check_scores(wl, pool, got, vis)
    wl.block_table[1, 2] = 64 * (pool.size // F.INDEXER_PAGE_BYTES)
    wl.block_table[1, 5] = -1
    got, status = run_scores(wl, pool, vis)
    assert status == (sml.SML_ERR_DEVICE_FAULT, sml.SML_FAULT_PAGE)
    assert np.isnan(got[4, [2, 5]]).all() and np.isfinite(got[4, [0, 1, 3, 4, 6, 7]]).all()
    assert (got[3] == 123.0).all()


def run_topk(wl, scores, k, vis=None):
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    if vis is not None:
        dw.vis = torch.from_numpy(vis).cuda()
        p.vis_len = dw.vis.data_ptr()
    blocks = torch.full((wl.T, k), 77, dtype=torch.int32, device="cuda")
    count = torch.full((wl.T,), 77, dtype=torch.int32, device="cuda")
    ws = status_ws()
    sml.sml_block_topk(p, dev(scores), blocks, count, ws)
    return blocks.cpu().numpy(), count.cpu().numpy(), sml.sml_read_device_status(ws)


def check_topk(wl, scores, k, blocks, count, n_all):
    for t in range(wl.T):
        want = OB.block_topk_row(scores[t], int(n_all[t]), k)
        assert count[t] == len(want), t
        assert np.array_equal(blocks[t, :len(want)], want), f"token {t}"
        assert (blocks[t, len(want):] == -1).all(), t


@pytest.mark.parametrize("k", [1, 2, 32, 33, 513, 2048])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_block_topk(k, kind):
    lens = [1, 64, 65, 2048, 2049, 33000, 140000, 70000]
    wl = synth.make_workload(f"bt/{k}", [64] * 8, [1] * 8, 16)
    wl.ctx_len = np.array(lens, dtype=np.int32)
    wl.block_table = np.zeros((8, 2200), dtype=np.int32)
    rng = synth.stream(k, "bt/" + kind)
    scores = rng.standard_normal((8, 2200), dtype=np.float32)
    if kind == "ties":
        scores = np.round(scores * 2) / 2
        scores[scores == 0] = rng.choice([0.0, -0.0], (scores == 0).sum())
    if kind == "special":
        scores[:, ::7] = np.nan
        scores[:, 1::5] = np.inf
        scores[:, 2::3] = -np.inf
        scores[5] = 0.0
    blocks, count, status = run_topk(wl, scores, k)
    assert status == (sml.SML_OK, 0)
    check_topk(wl, scores, k, blocks, count, np.array(lens))


def test_block_topk_long_rows():
    """A million positions and more: 16,383 candidates, and 40,000."""
    wl = synth.make_workload("bt/long", [64, 64], [1, 1], 16)
    wl.ctx_len = np.array([1 << 20, 2560001], dtype=np.int32)
    wl.block_table = np.zeros((2, 40001), dtype=np.int32)
    scores = synth.stream(0, "bt/long").standard_normal((2, 40001), dtype=np.float32)
    scores[1, 30000:30050] = 9.0                                   # more equal ones than are taken
    for k in (45, 2048):
        blocks, count, status = run_topk(wl, scores, k)
        assert status == (sml.SML_OK, 0)
        check_topk(wl, scores, k, blocks, count, wl.ctx_len)


@pytest.mark.parametrize("pages", [900, 1024, 1025, 16384, 16385])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "outlier", "tiny", "few", "close", "clustered"])
def test_block_topk_of_every_distribution(pages, kind):
    """Rows whose candidates leave the threshold's search nothing to go by, or too much: behind the
    candidates the row holds larger scores, which do not count."""
    lens = [64 * pages, 64 * pages - 63, 64 * (pages * 2 // 3) + 1, 40 * 64, 33 * 64 + 1]
    wl = synth.make_workload(f"btd/{pages}", [64] * 5, [1] * 5, 16)
    wl.ctx_len = np.array(lens, dtype=np.int32)
    wl.block_table = np.zeros((5, pages), dtype=np.int32)
    rng = synth.stream(pages, "btd/" + kind)
    x = rng.standard_normal((5, pages)).astype(np.float32)
    if kind == "equal":
        x[:] = -3.5
    if kind in ("rising", "falling"):
        x = np.sort(x, 1)[:, ::1 if kind == "rising" else -1].copy()
    if kind == "outlier":   # one key far above the others, one far below
        x[:, 5], x[:, 9] = 3e38, -3e38
    if kind == "tiny":
        x *= np.float32(2.0 ** -140)   # subnormal, of either sign, and zeros
    if kind == "few":
        x[:, :] = np.nan
        x[:, 3:pages:pages // 40] = 1.0
    if kind == "close":     # a few last bits apart
        x = (np.float32(1.0).view(np.uint32) + rng.integers(0, 40, x.shape).astype(np.uint32)).view(np.float32)
    if kind == "clustered":   # all of the best next to one another
        x[:, 20:20 + pages // 8] += 50.0
    for t, n in enumerate(lens):
        x[t, (n - 1) // 64:] = np.inf
    for k in (2, 31, 45, 300, 1000):
        blocks, count, status = run_topk(wl, x, k)
        assert status == (sml.SML_OK, 0)
        check_topk(wl, x, k, blocks, count, np.array(lens))


def test_block_topk_given_lengths_and_bad_requests():
    wl = synth.make_workload("bt/vis", [700, 1000, 300], [3, 2, 1], 16)
    scores = synth.stream(0, "bt/vis").standard_normal((6, wl.max_pages), dtype=np.float32)
    vis = np.array([0, 65, 700, 64, 513, 300], dtype=np.int32)
    blocks, count, status = run_topk(wl, scores, 5, vis)
    assert status == (sml.SML_OK, 0)
    check_topk(wl, scores, 5, blocks, count, vis)
    vis[1] = 701                                                   # more than the request holds
    blocks, count, status = run_topk(wl, scores, 5, vis)
    assert status == (sml.SML_ERR_DEVICE_FAULT, sml.SML_FAULT_LENGTHS)
    vis[1] = 0
    check_topk(wl, scores, 5, blocks, count, vis)


def test_a_decode_layer_over_selected_blocks():
    """Keys of every full page, scores, selection and attention in a row, each checked on what
    the step before it produced; then the same in a captured graph."""
    wl = synth.make_workload("chain", [5000, 777, 64, 12000], [1, 3, 1, 2], 32, ssmax=True)
    dw = DeviceWorkload(wl)
    p, lay, k = dw.problem(0), dw.layers[0], 9
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    full = np.array([pg for r in range(wl.B) for pg in wl.block_table[r, :wl.ctx_len[r] // 64]], dtype=np.int32)
    pool = dev(block_pool(wl.num_pages))
    scores = torch.full((wl.T, wl.max_pages), 123.0, device="cuda")
    blocks = torch.empty(wl.T, k, dtype=torch.int32, device="cuda")
    count = torch.empty(wl.T, dtype=torch.int32, device="cuda")
    out = torch.empty(wl.T, 32, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(wl.T, 32, device="cuda")
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    pages = dev(full)

    def layer():
        sml.sml_block_keys_write(dw.index_cache, pages, pool, ws)
        sml.sml_block_scores(p, lay.iq8, lay.iq_scale, lay.iw, pool, scores, ws)
        sml.sml_block_topk(p, scores, blocks, count, ws)
        sml.sml_block_mla_decode(p, lay.q, dw.latent, blocks, count, out, lse, ws)

    def check():
        assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
        hp, hs = pool.cpu().numpy(), scores.cpu().numpy()
        assert np.array_equal(hp, OB.block_keys(wl.index_cache, full, block_pool(wl.num_pages))[0])
        check_scores(wl, hp, hs, n_all)
        hb, hc = blocks.cpu().numpy(), count.cpu().numpy()
        check_topk(wl, hs, k, hb, hc, n_all)
        ho, hl = out.float().cpu().numpy(), lse.cpu().numpy()
        for t in range(wl.T):
            n = int(n_all[t])
            PC.check(f"token {t}", ho[t], hl[t], PC.expect(wl, 0, t, OB.block_positions(hb[t, :hc[t]], n)))

    layer()
    check()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        layer()
    for b in (pool, blocks, count, out, lse):
        b.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    check()


# ---- reading back -------------------------------------------------------------------

FORMATS = {"fp8_ds_mla": (synth._fill_latent, 656), "e4m3": (synth.plain_pool, 576), "bf16": (synth.bf16_pool, 1152)}


def wrap(fmt, pool):
    t = dev(pool)
    return {"fp8_ds_mla": t, "e4m3": sml.E4M3Latent(t, synth.PLAIN_SCALE), "bf16": sml.Bf16Latent(t)}[fmt]


def oracle_pool(fmt, pool):
    return {"fp8_ds_mla": pool, "e4m3": F.PlainE4M3Pool(pool, synth.PLAIN_SCALE), "bf16": F.Bf16Pool(pool)}[fmt]


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("n,pages,rope", [(1, 1, True), (2, 1, False), (63, 2, True), (5001, 97, True), (5001, 97, False)])
def test_latent_rows_read_back(fmt, n, pages, rope):
    """Code times scale, both exact in float64 and their product rounded to fp32, then to bf16: the
    same two roundings here, so the bits are equal."""
    pool = FORMATS[fmt][0](0, f"rd/{fmt}", pages)
    slot = synth.stream(n, "rd/slot").integers(0, pages * 64, n).astype(np.int32)      # some named twice
    slot[::5] = -1 if n > 4 else slot[::5]
    c = torch.full((n, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    pe = torch.full((n, 64), 7.0, dtype=torch.bfloat16, device="cuda") if rope else None
    ws = status_ws()
    sml.sml_latent_cache_read(dev(slot), wrap(fmt, pool), c, pe, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    there = slot >= 0
    want_c, want_pe = OB.read_latent(oracle_pool(fmt, pool), slot[there])
    seven = synth.to_bf16_bits(np.float32([7.0]))[0]
    for got, want in ((c, want_c),) + (((pe, want_pe),) if rope else ()):
        got = bits(got)
        assert np.array_equal(got[there], synth.to_bf16_bits(want.astype(np.float32)))
        assert (got[~there] == seven).all()


def test_indexer_keys_read_back_and_bad_slots():
    pool = synth._fill_index(0, "rd/index", 40)
    slot = synth.stream(0, "rd/islot").integers(0, 40 * 64, 1003).astype(np.int32)
    slot[[5, 700]] = -1
    k = torch.full((1003, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = status_ws()
    sml.sml_indexer_k_cache_read(dev(slot), dev(pool), k, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    there = slot >= 0
    assert np.array_equal(bits(k)[there], synth.to_bf16_bits(OB.read_indexer_k(pool, slot[there]).astype(np.float32)))
    before = k.clone()
    slot[3], slot[900] = 40 * 64, -2
    sml.sml_indexer_k_cache_read(dev(slot), dev(pool), k, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_ERR_DEVICE_FAULT, sml.SML_FAULT_PAGE)
    assert torch.equal(k, before)
    c = torch.full((1003, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lat = synth._fill_latent(0, "rd/bad", 40)
    sml.sml_latent_cache_read(dev(slot), dev(lat), c, None, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_ERR_DEVICE_FAULT, sml.SML_FAULT_PAGE)
    assert bool((c[[3, 5, 700, 900]] == 7).all())
    sml.sml_latent_cache_read(torch.empty(0, dtype=torch.int32, device="cuda"), dev(lat), None, None, ws)
    sml.sml_indexer_k_cache_read(torch.empty(0, dtype=torch.int32, device="cuda"), dev(pool), None, ws)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_written_rows_read_back_within_half_a_step(fmt):
    """New rows written by the cache writers and read back: off by half an E4M3 step of the value
    (2^-4), or of the subnormal step under the block's scale (2^-10 s), then half a bf16 step
    (2^-8); a bf16 pool returns the very bits."""
    n, pages = 300, 6
    bits_in = synth.producer_rows(11, "rt/c", n, 512, spread=False)
    x = torch.from_numpy(bits_in.view(np.int16)).view(torch.bfloat16).cuda()
    pe = torch.from_numpy(synth.producer_rows(11, "rt/pe", n, 64, spread=False).view(np.int16)).view(torch.bfloat16).cuda()
    slot = dev(synth.producer_slots(11, "rt/slot", n, pages))
    pool = wrap(fmt, np.zeros(pages * 64 * FORMATS[fmt][1], dtype=np.uint8))
    c2, pe2 = torch.empty_like(x), torch.empty_like(pe)
    sml.sml_latent_cache_write(x, pe, slot, pool)
    sml.sml_latent_cache_read(slot, pool, c2, pe2)
    if fmt == "bf16":
        assert torch.equal(c2, x) and torch.equal(pe2, pe)
        return
    if fmt == "fp8_ds_mla":
        assert torch.equal(pe2, pe)
        s = (x.double().view(n, 4, 128).abs().amax(-1) / 448).repeat_interleave(128, 1)
    else:
        s = torch.full_like(x.double(), synth.PLAIN_SCALE)
    d = (c2.double() - x.double()).abs()
    assert bool((d <= x.double().abs() * (2.0 ** -4 + 1.07 * 2.0 ** -8) + 1.01 * 2.0 ** -10 * s).all())
