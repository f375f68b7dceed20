"""MLA over the whole paged cache, a window of it, and listed blocks, on the GPU against the
float64 oracle, with bounds derived from the arithmetic (tests/paged_cases.py)."""
import numpy as np
import pytest
import torch

from oracle import blocks as OB, dsa, formats as F
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


def buffers(T, H):
    """Outputs that start as NaN, so that an unwritten value shows."""
    return (torch.full((T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda"),
            torch.full((T, H), float("nan"), device="cuda"))


def workspace(p):
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    ws[256 + 4 * 65536:] = 0xFF        # nothing behind the header has to start at zero
    return ws


def host(t):
    return t.float().cpu().numpy()


def paged(wl, layer_i=0, window=0):
    dw = DeviceWorkload(wl)
    p = dw.problem(layer_i)
    out, lse = buffers(wl.T, wl.num_heads)
    ws = workspace(p)
    sml.sml_paged_mla_decode(p, dw.layers[layer_i].q, dw.latent, out, lse, ws, window=window)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    return host(out), host(lse)


def check_all(name, wl, out, lse, window=0, layer_i=0, tokens=None):
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    for t in range(wl.T) if tokens is None else tokens:
        n = int(n_all[t])
        PC.check(f"{name} token {t} (n {n})", out[t], lse[t],
                 PC.expect(wl, layer_i, t, np.arange(max(0, n - window) if window else 0, n)))


EDGES = [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 1000, 2047]


@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3", "bf16"])
@pytest.mark.parametrize("heads,rope", [(16, 64), (32, 0), (64, 64)])
def test_every_length_around_the_page_and_tile_edges(fmt, heads, rope):
    wl = synth.make_workload(f"paged/{fmt}/{heads}", EDGES, [1] * len(EDGES), heads, latent_format=fmt,
                             layers=(("l", rope, False, None),), extra_pages=3)
    out, lse = paged(PC.spoil_unused(wl))
    check_all(fmt, wl, out, lse)


@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "bf16"])
def test_several_new_tokens_all_heads_and_ssmax(fmt):
    wl = synth.make_workload(f"paged/q/{fmt}", [5, 700, 66, 1500], [5, 2, 3, 1], 128, ssmax=True, latent_format=fmt,
                             layers=(("l", 64, False, None),))
    out, lse = paged(PC.spoil_unused(wl))
    check_all(fmt, wl, out, lse)


@pytest.mark.parametrize("window", [1, 63, 64, 65, 130, 1999])
@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "bf16"])
def test_window(fmt, window):
    wl = synth.make_workload(f"paged/w/{fmt}", [1, 64, 70, 129, 900, 2500], [1, 2, 3, 1, 4, 2], 16, latent_format=fmt,
                             layers=(("l", 64, False, None),))
    out, lse = paged(wl, window=window)
    check_all(f"{fmt} window {window}", wl, out, lse, window=window)


def test_rows_before_the_window_may_hold_nan():
    wl = synth.make_workload("paged/wnan", [1000], [1], 16, layers=(("l", 64, False, None),))
    n, w = 1000, 100
    want = PC.expect(wl, 0, 0, np.arange(n - w, n))
    rows = wl.latent.reshape(-1, 656)
    pos = np.arange(n - w)
    rows[wl.block_table[0, pos // 64].astype(np.int64) * 64 + pos % 64] = 0xFF
    out, lse = paged(PC.spoil_unused(wl), window=w)
    PC.check("nan before the window", out[0], lse[0], want)


def test_one_long_request_is_split_over_every_cta():
    wl = synth.make_workload("paged/long", [60011], [1], 32, layers=(("l", 64, False, None),))
    out, lse = paged(wl)
    check_all("long", wl, out, lse)


def test_many_requests_and_a_long_one_among_them():
    lens = [1 + (i * 37) % 200 for i in range(400)]
    lens[123] = 20000
    wl = synth.make_workload("paged/many", lens, [1] * 400, 16, layers=(("l", 64, False, None),))
    out, lse = paged(wl)
    check_all("many", wl, out, lse, tokens=list(range(0, 400, 17)) + [122, 123, 124, 399])


def test_more_tokens_than_threads():
    wl = synth.make_workload("paged/prefill", [2500, 40, 3], [2400, 40, 1], 16, layers=(("l", 64, False, None),))
    out, lse = paged(wl)
    check_all("prefill", wl, out, lse, tokens=[0, 1, 63, 64, 1023, 1024, 1025, 2047, 2399, 2400, 2439, 2440])


def _peaked(wl, layer_i, gain):
    """Queries times `gain` (a power of two: exact in bf16), so that few keys carry the softmax."""
    x = torch.from_numpy(wl.layers[layer_i].q.view(np.int16)).view(torch.bfloat16)
    wl.layers[layer_i].q = (x * gain).view(torch.int16).numpy().view(np.uint16)
    return wl


@pytest.mark.parametrize("gain", [0.0, 2.0 ** -20, 16.0, 1024.0])
@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3", "bf16"])
def test_flat_and_peaked_softmax(fmt, gain):
    """From equal weights to one key that takes all, with the largest logits in any tile (the
    running maximum has to rise more than once)."""
    wl = _peaked(synth.make_workload(f"paged/peak/{fmt}", [777, 1300], [1, 2], 16, latent_format=fmt,
                                     layers=(("l", 64, False, None),)), 0, gain)
    out, lse = paged(wl)
    check_all(f"{fmt} gain {gain}", wl, out, lse)


@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3", "bf16"])
def test_smallest_and_largest_queries(fmt):
    """Heads of zeros, of bf16's smallest magnitudes among zeros, and of magnitudes near its largest
    (kept finite by sm_scale)."""
    wl = synth.make_workload(f"paged/extreme/{fmt}", [200], [1], 16, latent_format=fmt, layers=(("l", 64, False, None),))
    q = (wl.layers[0].q.astype(np.uint32) << 16).view(np.float32)
    q[0, 0] = 0.0
    q[0, 1] *= np.float32(2.0 ** -126)
    q[0, 1, ::3] = 0.0
    q[0, 2] = np.where(np.arange(576) == 7, np.float32(2.0 ** -133), 0.0)
    q[0, 3] *= np.float32(2.0 ** 120)
    q[0, 4:] *= np.float32(2.0 ** 118)
    wl.layers[0].q = synth.to_bf16_bits(q)
    wl.sm_scale = float(np.float32(2.0 ** -122))
    out, lse = paged(wl)
    check_all(fmt, wl, out, lse)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3", "bf16"])
def test_infinities_and_nan_in_a_query_stay_in_their_head(fmt, heads):
    wl = synth.make_workload(f"paged/inf/{fmt}", [700, 130], [1, 2], heads, latent_format=fmt, layers=(("l", 64, False, None),))
    q = wl.layers[0].q.reshape(-1, heads, 576)
    want = [PC.expect(wl, 0, t, np.arange(int(n))) for t, n in enumerate(dsa.visible_lengths(wl.cu_q, wl.ctx_len))]
    q[:, 1, 7], q[:, 3, 300], q[:, 6, 560], q[:, 10, 0] = 0x7f80, 0x7fc0, 0x7fc0, 0xff80
    out, lse = paged(wl)
    bad = [1, 3, 6, 10]
    assert np.isnan(out[:, bad]).all() and np.isnan(lse[:, bad]).all()
    good = [h for h in range(heads) if h not in bad]   # (heads share scale exponents: not the same bits as without)
    for t in range(wl.T):
        PC.check(f"token {t}", out[t, good], lse[t, good], [x[good] for x in want[t]])


def test_rising_logits():
    """Keys that grow along the context: every tile raises the running maximum."""
    wl = synth.make_workload("paged/rise", [1500], [1], 16, latent_format="bf16", layers=(("l", 64, False, None),))
    rows = wl.latent.reshape(-1, 1152).view("<u2")
    pos = np.arange(1500)
    at = wl.block_table[0, pos // 64].astype(np.int64) * 64 + pos % 64
    vals = (rows[at].astype(np.uint32) << 16).view(np.float32)
    q = (wl.layers[0].q[0, 0].astype(np.uint32) << 16).view(np.float32)
    vals = 0.01 * vals + (pos[:, None] / 100.0) * (q / np.abs(q).max())[None]
    rows[at] = synth.to_bf16_bits(vals.astype(np.float32))
    out, lse = paged(wl)
    check_all("rising", wl, out, lse)


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -14, 2.0 ** 20])
def test_block_scales_far_from_one(scale):
    """Latents whose block scales lie far outside half precision's range."""
    wl = synth.make_workload("paged/scales", [300, 130], [1, 1], 16, layers=(("l", 64, False, None),))
    sc = np.ascontiguousarray(wl.latent.reshape(-1, 656)[:, 512:528]).view("<f4")
    with np.errstate(over="ignore"):                                # rows nobody holds
        wl.latent.reshape(-1, 656)[:, 512:528] = (sc * np.float32(scale)).view(np.uint8).reshape(-1, 16)
    wl.sm_scale = float(np.float32(wl.sm_scale / max(1.0, scale)))
    out, lse = paged(wl)
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    for t in range(2):
        PC.check(f"scale {scale}", out[t], lse[t], PC.expect(wl, 0, t, np.arange(int(n_all[t]))))


def test_given_visible_and_ssmax_lengths():
    wl = synth.make_workload("paged/vis", [500, 300, 200], [2, 3, 1], 16, ssmax=True, layers=(("l", 64, False, None),))
    dw = DeviceWorkload(wl)
    vis = np.array([0, 129, 0, 0, 64, 200], dtype=np.int32)
    nss = np.array([5, 1000, 1, 7, 64, 100000], dtype=np.int32)
    d_vis, d_nss = torch.from_numpy(vis).cuda(), torch.from_numpy(nss).cuda()
    p = sml.make_problem(num_heads=16, topk=1, rope_dim=64, cu_q=dw.cu_q, ctx_len=dw.ctx_len, block_table=dw.block_table,
                         max_ctx=500, ssmax=True, sm_scale=wl.sm_scale, num_tokens=6, vis_len=d_vis, ssmax_len=d_nss)
    out, lse = buffers(6, 16)
    ws = workspace(p)
    sml.sml_paged_mla_decode(p, dw.layers[0].q, dw.latent, out, lse, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    out, lse = host(out), host(lse)
    for t in range(6):
        PC.check(f"vis {vis[t]}", out[t], lse[t], PC.expect(wl, 0, t, np.arange(vis[t]), n=int(vis[t]), nss=int(nss[t])))


def _blocks_case(name, lens, qs, heads, k, fmt, seed=0, **kw):
    wl = synth.make_workload(name, lens, qs, heads, latent_format=fmt, layers=(("l", kw.pop("rope", 64), False, None),), **kw)
    rng = synth.stream(seed, name + "/blocks")
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    blocks = np.full((wl.T, k), -1, dtype=np.int32)
    count = np.zeros(wl.T, dtype=np.int32)
    for t in range(wl.T):
        have = (int(n_all[t]) + 63) // 64
        count[t] = min(have, int(rng.integers(0, k + 1)) if t else k)
        blocks[t, :count[t]] = rng.permutation(have)[:count[t]]      # in any order
    return wl, blocks, count


def run_blocks(wl, blocks, count, expect_bits=0):
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    out, lse = buffers(wl.T, wl.num_heads)
    ws = workspace(p)
    sml.sml_block_mla_decode(p, dw.layers[0].q, dw.latent, torch.from_numpy(blocks).cuda(),
                             torch.from_numpy(count).cuda(), out, lse, ws)
    assert sml.sml_read_device_status(ws)[1] == expect_bits
    return host(out), host(lse)


@pytest.mark.parametrize("fmt,heads,rope,k", [("fp8_ds_mla", 16, 64, 7), ("e4m3", 32, 64, 8), ("bf16", 64, 0, 5),
                                              ("fp8_ds_mla", 128, 0, 1), ("bf16", 16, 64, 33)])
def test_listed_blocks(fmt, heads, rope, k):
    wl, blocks, count = _blocks_case(f"blk/{fmt}/{k}", [1, 64, 65, 640, 3001], [1, 1, 2, 3, 2], heads, k, fmt, rope=rope,
                                     ssmax=True)
    out, lse = run_blocks(PC.spoil_unused(wl), blocks, count)
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    for t in range(wl.T):
        n = int(n_all[t])
        PC.check(f"token {t} blocks {blocks[t, :count[t]]}", out[t], lse[t],
                 PC.expect(wl, 0, t, OB.block_positions(blocks[t, :count[t]], n)))


def test_a_block_listed_twice_counts_twice():
    wl, blocks, count = _blocks_case("blk/twice", [640], [1], 16, 4, "fp8_ds_mla")
    blocks[0] = [3, 3, 9, 0]
    count[0] = 4
    out, lse = run_blocks(wl, blocks, count)
    PC.check("twice", out[0], lse[0], PC.expect(wl, 0, 0, OB.block_positions(blocks[0], 640)))


def test_bad_blocks_counts_and_pages_are_masked_and_reported():
    wl, blocks, count = _blocks_case("blk/bad", [640, 300, 200], [1, 1, 1], 16, 4, "fp8_ds_mla")
    blocks[0] = [10, 2, -1, 5]          # 640 positions: blocks 0..9
    count[:] = [4, 4, 3]
    blocks[1] = [0, 1, 2, 4]
    blocks[2] = [3, 0, 1, -1]
    out, lse = run_blocks(wl, blocks, count, expect_bits=sml.SML_FAULT_INDEX)
    for t, good in enumerate(([2, 5], [0, 1, 2, 4], [3, 0, 1])):
        n = int(wl.ctx_len[t])
        PC.check(f"token {t}", out[t], lse[t], PC.expect(wl, 0, t, OB.block_positions(good, n)))
    count[1] = 9                        # more than a row holds: its four are read
    count[2] = -3                       # none
    out, lse = run_blocks(wl, blocks, count, expect_bits=sml.SML_FAULT_INDEX | sml.SML_FAULT_TOPK_LEN)
    PC.check("clamped", out[1], lse[1], PC.expect(wl, 0, 1, OB.block_positions(blocks[1], 300)))
    assert not out[2].any() and np.isneginf(lse[2]).all()
    page = wl.block_table[0, 5].copy()
    for bad in (wl.num_pages, -1):
        wl.block_table[0, 5] = bad
        out, lse = run_blocks(wl, blocks, np.array([4, 4, 3], np.int32), expect_bits=sml.SML_FAULT_INDEX | sml.SML_FAULT_PAGE)
        PC.check("bad page", out[0], lse[0], PC.expect(wl, 0, 0, OB.block_positions([2], 640)))
    wl.block_table[0, 5] = page


def test_bad_lengths_give_empty_rows_and_are_reported():
    wl = synth.make_workload("paged/badlen", [300, 200, 100], [1, 2, 1], 16, layers=(("l", 64, False, None),))
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    dw.ctx_len[1] = 301                 # past max_ctx
    out, lse = buffers(4, 16)
    ws = workspace(p)
    sml.sml_paged_mla_decode(p, dw.layers[0].q, dw.latent, out, lse, ws)
    code, bits = sml.sml_read_device_status(ws)
    assert code == sml.SML_ERR_DEVICE_FAULT and bits == sml.SML_FAULT_LENGTHS
    out, lse = host(out), host(lse)
    for t, r in ((0, 0), (3, 2)):
        PC.check(f"request {r}", out[t], lse[t], PC.expect(wl, 0, t, np.arange(int(wl.ctx_len[r]))))
    assert not out[1:3].any() and np.isneginf(lse[1:3]).all()


def test_captured_replayed_and_on_another_stream():
    """Two calls with different inputs that share a workspace, captured in one graph on a side
    stream and replayed with changed queries."""
    a = synth.make_workload("paged/graph/a", [900, 4000, 65], [1, 1, 1], 16, layers=(("l", 64, False, None),))
    b = synth.make_workload("paged/graph/b", [3000], [2], 16, latent_format="bf16", layers=(("l", 64, False, None),))
    da, db = DeviceWorkload(a), DeviceWorkload(b)
    pa, pb = da.problem(0), db.problem(0)
    ws = max((workspace(pa), workspace(pb)), key=lambda w: w.numel())
    oa, la = buffers(a.T, 16)
    ob, lb = buffers(b.T, 16)
    q = torch.zeros_like(da.layers[0].q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        sml.sml_paged_mla_decode(pa, q, da.latent, oa, la, ws)       # first launches outside the capture
        sml.sml_paged_mla_decode(pb, db.layers[0].q, db.latent, ob, lb, ws, window=1000)
    with torch.cuda.graph(g, stream=s):
        sml.sml_paged_mla_decode(pa, q, da.latent, oa, la, ws)
        sml.sml_paged_mla_decode(pb, db.layers[0].q, db.latent, ob, lb, ws, window=1000)
    for rep in range(3):
        q.copy_(da.layers[0].q)
        oa.fill_(float("nan"))
        ob.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check_all(f"replay {rep} a", a, host(oa), host(la))
        check_all(f"replay {rep} b", b, host(ob), host(lb), window=1000)
        q.zero_()
        g.replay()
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)


def test_same_call_twice_gives_the_same_bits():
    wl = synth.make_workload("paged/bits", [5000, 30000, 7], [1, 3, 1], 32, layers=(("l", 64, False, None),))
    first, second = paged(wl), paged(wl)
    assert np.array_equal(first[0], second[0]) and np.array_equal(first[1], second[1])


def test_paged_and_sparse_attention_agree_where_the_selection_is_everything():
    """n <= topk: the sparse path over all positions, the paged path and the blocks path over all
    blocks are the same attention."""
    wl = synth.make_workload("paged/sparse", [1900, 130], [2, 1], 32)
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    idx, ln, so, sl = dw.outputs()
    lay = dw.layers[0]
    wsl = dw.workspace()
    sml.sml_run_layer(p, lay.q, lay.iq8, lay.iq_scale, lay.iw, dw.latent, dw.index_cache, None, None, idx, ln, so, sl, wsl)
    out, lse = paged(wl)
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    want = [PC.expect(wl, 0, t, np.arange(int(n_all[t]))) for t in range(wl.T)]
    for t in range(wl.T):
        PC.check("paged", out[t], lse[t], want[t])
        PC.check("sparse", so[t].cpu().numpy(), sl[t].cpu().numpy(), want[t])
    all_blocks = np.tile(np.arange(30, dtype=np.int32), (3, 1))
    count = ((n_all + 63) // 64).astype(np.int32)
    out, lse = run_blocks(wl, all_blocks, count)
    for t in range(wl.T):
        PC.check("blocks", out[t], lse[t], want[t])


def _with_scales(name, heads, change, lens=(128 + 64 * 9, 1500)):
    """A workload whose block scales are change(scales [rows, 4], ids of each request's rows), with
    so many tokens that a CTA walks a whole token's tiles."""
    wl = synth.make_workload(f"paged/{name}", list(lens), [70, 80], heads, layers=(("l", 64, False, None),))
    rows = wl.latent.reshape(-1, 656)
    sc = np.ascontiguousarray(rows[:, 512:528]).view("<f4")
    ids = [wl.block_table[r, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64 for r, n in enumerate(lens)]
    with np.errstate(over="ignore", invalid="ignore"):
        sc = change(sc, ids).astype("<f4")
    rows[:, 512:528] = sc.view(np.uint8).reshape(-1, 16)
    return wl, ids


def _check_any_scales(name, wl):
    out, lse = paged(PC.spoil_unused(wl))
    for t, n in enumerate(dsa.visible_lengths(wl.cu_q, wl.ctx_len)):
        if t % 9 and t != wl.T - 1:
            continue
        PC.check(f"{name} token {t}", out[t], lse[t], PC.expect(wl, 0, t, np.arange(int(n)), any_scales=True))


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("spread", [3, 7])
def test_block_scales_of_different_magnitude(spread, heads):
    """The four blocks of a row 2^spread apart from their neighbours, and rows scaled by up to
    2^spread either way."""
    rng = synth.stream(spread, "paged/spread")

    def change(sc, ids):
        return sc * np.exp2(rng.uniform(-spread, spread, (len(sc), 1))) * np.exp2(spread * (np.arange(4) - 3.0))
    _check_any_scales(f"spread {spread}", _with_scales(f"spread/{spread}", heads, change, (300, 1100))[0])


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("early", [0.0, 2.0 ** -126, 2.0 ** -30, 2.0 ** -10, 2.0 ** 10])
def test_one_blocks_scales_change_after_the_first_keys(early, heads):
    """In a request's first 128 keys one block is zeros, or far below or above what it is later:
    the other blocks' weights keep their bits."""
    def change(sc, ids):
        for r, i in enumerate(ids):
            sc[i[:128], 2 * r + 1] *= np.float32(early)
            if early == 2.0 ** -126:
                sc[i[:128], 2 * r + 1] = np.float32(early)
        return sc
    _check_any_scales(f"early {early}", _with_scales(f"early/{heads}", heads, change)[0])


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("at", [0, 5, 300])
@pytest.mark.parametrize("seen", [True, False])
def test_one_key_with_a_large_block(seen, at, heads):
    """One key with a block 2^12 above the others, of ordinary logit (it takes over that block's
    output, the other blocks keep their bits) or far below (no block may lose any)."""
    wl, ids = _with_scales(f"large/{heads}", heads, lambda sc, ids: sc)
    rows = wl.latent.reshape(-1, 656)
    sc = np.ascontiguousarray(rows[:, 512:528]).view("<f4")
    pe = np.zeros((len(rows), 64), np.float32)
    for r, i in enumerate(ids):
        sc[i[at], 3 * r] *= np.float32(2.0 ** 12)
        pe[i[at], 0] = 0.0 if seen else -40.0 / wl.sm_scale
    rows[:, 512:528] = sc.view(np.uint8).reshape(-1, 16)
    rows[:, 528:] = synth.to_bf16_bits(pe).astype("<u2").view(np.uint8).reshape(-1, 128)
    q = F.decode_bf16(wl.layers[0].q).astype(np.float32)
    q[..., 512:] = 0.0
    q[..., 512] = 1.0
    for t, r in enumerate(dsa.request_of_tokens(wl.cu_q)):
        q[t, :, 128 * 3 * r:128 * 3 * r + 128] = 0.0   # the large block does not enter the logits
    wl.layers[0].q = synth.to_bf16_bits(q)
    _check_any_scales(f"large {seen} {at}", wl)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("small", [2.0 ** -126, 2.0 ** -24])
def test_all_scales_grow_after_keys_that_take_the_weight(small, heads):
    """128 keys of tiny scale that every query prefers, before ordinary ones: the output is the
    ordinary keys', whose weights are a millionth of the sum, with their bits."""
    def change(sc, ids):
        for i in ids:
            sc[i[:128]] = np.float32(small)
        return sc
    wl, ids = _with_scales(f"sink/{heads}", heads, change)
    rows = wl.latent.reshape(-1, 656)
    pe = np.zeros((len(rows), 64), np.float32)
    for i in ids:
        pe[i[:128], 0] = 14.0 / wl.sm_scale
    rows[:, 528:] = synth.to_bf16_bits(pe).astype("<u2").view(np.uint8).reshape(-1, 128)
    q = F.decode_bf16(wl.layers[0].q).astype(np.float32)
    q[..., 512:] = 0.0
    q[..., 512] = 1.0
    wl.layers[0].q = synth.to_bf16_bits(q)
    _check_any_scales(f"sink {small}", wl)


def test_pages_past_four_gigabytes():
    """A pool of 4.4 GB whose last pages hold the rows: offsets that do not fit 32 bits."""
    wl = synth.make_workload("paged/far", [700, 130], [1, 1], 16, layers=(("l", 64, False, None),))
    far = 105000
    dw = DeviceWorkload(wl)
    pool = torch.empty((far + wl.num_pages) * synth.LATENT_PAGE, dtype=torch.uint8, device="cuda")
    assert far * synth.LATENT_PAGE > 2 ** 32
    pool[far * synth.LATENT_PAGE:] = dw.latent
    table = dw.block_table + far
    p = sml.make_problem(num_heads=16, topk=1, rope_dim=64, cu_q=dw.cu_q, ctx_len=dw.ctx_len, block_table=table,
                         max_ctx=700, sm_scale=wl.sm_scale, num_tokens=2)
    out, lse = buffers(2, 16)
    ws = workspace(p)
    sml.sml_paged_mla_decode(p, dw.layers[0].q, pool, out, lse, ws)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    check_all("far", wl, host(out), host(lse))
    slot = torch.tensor([far * 64 + 5, (far + 3) * 64 + 63], dtype=torch.int32, device="cuda")
    c = torch.empty(2, 512, dtype=torch.bfloat16, device="cuda")
    near = torch.empty_like(c)
    sml.sml_latent_cache_read(slot, pool, c)
    sml.sml_latent_cache_read(slot - far * 64, dw.latent, near)
    assert torch.equal(c.view(torch.int16), near.view(torch.int16))      # an unused row may hold NaN


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace and outputs."""
    works = [synth.make_workload(f"paged/streams/{i}", lens, qs, 32, layers=(("l", 64, False, None),))
             for i, (lens, qs) in enumerate((([9000, 130, 64], [1, 2, 1]), ([40000], [3])))]
    dws = [DeviceWorkload(w) for w in works]
    ps = [d.problem(0) for d in dws]
    wss = [workspace(p) for p in ps]
    bufs = [[buffers(w.T, 32) for _ in range(4)] for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    for rep in range(4):
        for d, p, ws, b, st in zip(dws, ps, wss, bufs, streams):
            with torch.cuda.stream(st):
                sml.sml_paged_mla_decode(p, d.layers[0].q, d.latent, *b[rep], ws)
    torch.cuda.synchronize()
    for w, ws, b in zip(works, wss, bufs):
        assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
        check_all("stream", w, host(b[0][0]), host(b[0][1]))
        for out, lse in b[1:]:
            assert torch.equal(out, b[0][0]) and torch.equal(lse, b[0][1])


@pytest.mark.parametrize("T", [1, 31, 32, 33, 100, 148, 149, 700])
def test_every_way_to_share_the_tiles(T):
    """Batches around the borders of the plan: one warp's batch, one CTA a token, more tokens than
    CTAs; equal lengths (whole tokens) and one long request among short ones (equal ranges)."""
    for long in (0, 9000):
        lens = [130 + 64 * (t % 3) for t in range(T)]
        lens[T // 2] = max(lens[T // 2], long)
        wl = synth.make_workload(f"paged/share/{T}/{long}", lens, [1] * T, 16, layers=(("l", 64, False, None),))
        out, lse = paged(wl)
        check_all(f"T {T} long {long}", wl, out, lse, tokens=sorted({0, T // 2, T - 1, T // 3, max(0, T // 2 - 1)}))


def test_one_workspace_for_both_kinds_of_attention():
    """A workspace large enough for both serves the sparse layer and the paged calls in turn (the
    top-k counters in it stay zero)."""
    wl = synth.make_workload("paged/ws", [140000, 900], [1, 2], 16)
    dw = DeviceWorkload(wl)
    p, lay = dw.problem(0), dw.layers[0]
    size = max(sml.sml_workspace_size(p, sml.SML_STAGE_LAYER), sml.sml_workspace_size(p, sml.SML_STAGE_PAGED))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    first = None
    for _ in range(3):
        idx, ln, so, sl = dw.outputs()
        sml.sml_run_layer(p, lay.q, lay.iq8, lay.iq_scale, lay.iw, dw.latent, dw.index_cache, None, None, idx, ln, so, sl, ws)
        out, lse = buffers(wl.T, 16)
        sml.sml_paged_mla_decode(p, lay.q, dw.latent, out, lse, ws, window=3000)
        now = [t.clone() for t in (idx, ln, so, sl, out, lse)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    check_all("after the sparse layer", wl, host(out), host(lse), window=3000)
