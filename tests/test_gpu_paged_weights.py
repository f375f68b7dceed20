"""The softmax weights of the FP8 pools' attention: many small ones behind a dominant key, on
the GPU against the float64 oracle.

The logits come through the RoPE key alone (the query's latent dims are 0), so that they do not
depend on the latents, which have a common offset: weights that are lost do not average out.

Bounds, from the arithmetic that include/sml.h promises (u = 2^-8, half a bf16 step):

* the output's rounding u |out|; each weight of 8 significant bits, three roundings to half
  precision on the way: (u + 3 * 2^-11) A, A = sum_i p_i |c_i|;
* the small weights together, whatever the number of keys: 1/224 of the row sum, as mass put on a
  tile's mean |c|, the largest over the context (tiles are 128 positions from the first page on,
  however the context is cut).  It stands for a sum of random roundings, at most 2^-14 each in units
  of which the largest weight is 56 or more: six deviations of 64,000 of them are 6 * 253 * 2^-14 / 56
  = 1/600, and weights alike, 500 tiles of half a step 2^-14 each, 1/1,800.  fp8_ds_mla: in units of
  the block's scale exponent, at most 4 of its largest scale (a weight of at most 224 sets it to lie
  above 56);
* the logits' sums: as in tests/paged_cases.py.  The log-sum-exp: those, the weights' own sum in fp32
  (n / 128 terms in a thread, 2^-24 each) and 2^-20 (1 + |lse|) for log2 and exp2.
"""
import functools

import numpy as np
import pytest
import torch

from oracle import dsa, formats as F
from sparse_mla_attention_indexer_b200 import sml, synth
from sparse_mla_attention_indexer_b200.device import DeviceWorkload
from tests import paged_cases as PC, parity

pytestmark = pytest.mark.gpu

ROW = {"fp8_ds_mla": 656, "e4m3": 576, "bf16": 1152}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


def put_rows(wl, at, c, k_pe):
    """Pool rows `at` with latents c [n, 512] and RoPE keys k_pe [n, 64], quantised as the pool is."""
    rows = wl.latent.reshape(-1, ROW[wl.latent_format])
    if wl.latent_format == "fp8_ds_mla":
        codes, scale = synth.quantise_rows(c.astype(np.float32), 128)
        rows[at, :512] = codes
        rows[at, 512:528] = scale.astype("<f4").view(np.uint8).reshape(-1, 16)
        rows[at, 528:] = synth.to_bf16_bits(k_pe.astype(np.float32)).astype("<u2").view(np.uint8).reshape(-1, 128)
    elif wl.latent_format == "e4m3":
        rows[at] = synth.to_e4m3(np.concatenate([c, k_pe], 1).astype(np.float32) / np.float32(synth.PLAIN_SCALE))
    else:
        x = np.concatenate([c, k_pe], 1).astype(np.float32)
        rows[at] = synth.to_bf16_bits(x).astype("<u2").view(np.uint8).reshape(-1, 1152)


def rows_of(wl, r, positions):
    return wl.block_table[r, positions // 64].astype(np.int64) * 64 + positions % 64


@functools.lru_cache(maxsize=2)
def latents(n, seed=0):
    return synth.stream(seed, f"weights/latents/{n}").normal(1.0, 1.0, (n, 512)).astype(np.float32)


def sink_case(fmt, heads, n, new, sigma, at=0):
    """One request of n tokens, `new` of them queries: key `at` holds a share of the softmax that
    differs by head (0.5, 0.65 and 0.8 of it, every fourth head none above the others), the other
    keys are alike (sigma = 0) or spread with that deviation."""
    wl = synth.make_workload(f"weights/{fmt}/{heads}/{new}", [n], [new], heads, latent_format=fmt,
                             layers=(("l", 64, False, None),))
    rng = synth.stream(1, f"weights/{fmt}/{n}/{sigma}")
    pe = np.zeros((n, 64))
    pe[:, 32:] = rng.standard_normal((n, 32)) if sigma else 0.0
    pe[at] = 0.0
    pe[at, :32] = 1.0
    put_rows(wl, rows_of(wl, 0, np.arange(n)), latents(n), pe)
    share = np.array([0.5, 0.65, 0.8, 0.0])[np.arange(heads) % 4]
    z = np.maximum(np.log(n * np.exp(sigma ** 2 / 2) * np.maximum(share, 1e-9) / (1 - share)), 0.0)
    wl.sm_scale = float(np.float32(1 / 32.0))
    q = np.zeros((new, heads, 576), np.float32)
    q[:, :, 512:544] = z[None, :, None]                       # 32 dims of 1 times 1 / 32
    q[:, :, 544:] = sigma * 32.0 / 32 ** 0.5
    wl.layers[0].q = synth.to_bf16_bits(q)
    return wl


def tile_mean(x):
    """Largest mean over tiles of 128 rows of x [n, d]."""
    pad = np.pad(x, ((0, -len(x) % 128), (0, 0)))
    return pad.reshape(-1, 128, x.shape[1]).mean(1).max(0)


def check_token(name, wl, out, lse, t, n, c, k_pe, scales):
    q = F.decode_bf16(wl.layers[0].q[t])
    keys = np.concatenate([c[:n], k_pe[:n]], 1)
    z = wl.sm_scale * (q[:, 512:] @ k_pe[:n].T)
    top = z.max(1, keepdims=True)
    p = np.exp(z - top)
    l = p.sum(1, keepdims=True)
    p /= l
    want, want_lse = p @ c[:n], (top + np.log(l))[:, 0]
    A = p @ np.abs(c[:n])
    d = 576 * 2.0 ** -23 * wl.sm_scale * (np.abs(q) @ np.abs(keys).T).max(1)
    tol = 2 * d[:, None] * ((p * (1 - p)) @ np.abs(c[:n])) + PC.U * np.abs(want) + (PC.U + 3 * 2.0 ** -11) * A * 1.01
    if wl.latent_format == "fp8_ds_mla":
        codes = np.abs(c[:n].reshape(n, 4, 128)) / scales[:n, :, None]
        tol += 4 / 224 * (scales[:n].max(0)[:, None] * tile_mean(codes.reshape(n, 512)).reshape(4, 128)).reshape(1, 512)
    elif wl.latent_format == "e4m3":
        tol += tile_mean(np.abs(c[:n]))[None] / 224
    ltol = d + (n / 128 + 8) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(want_lse))
    PC.check(f"{name} token {t} (n {n})", out[t], lse[t], (want, want_lse, tol, ltol))


def run(wl, window=0):
    dw = DeviceWorkload(wl)
    p = dw.problem(0)
    out = torch.full((wl.T, wl.num_heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((wl.T, wl.num_heads), float("nan"), device="cuda")
    ws = torch.empty(sml.sml_workspace_size(p, sml.SML_STAGE_PAGED), dtype=torch.uint8, device="cuda")
    sml.sml_workspace_init(ws)
    sml.sml_paged_mla_decode(p, dw.layers[0].q, dw.latent, out, lse, ws, window=window)
    assert sml.sml_read_device_status(ws) == (sml.SML_OK, 0)
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check_tokens(name, wl, out, lse, tokens):
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    pos = np.arange(int(wl.ctx_len[0]))
    pages, rows = F.physical(wl.block_table[0], pos)
    c, k_pe = F.latent_rows(parity.oracle_latent(wl), pages, rows)
    scales = PC.block_scales(wl, pages, rows) if wl.latent_format == "fp8_ds_mla" else None
    for t in tokens:
        check_token(name, wl, out, lse, t, int(n_all[t]), c, k_pe, scales)


# More tokens than CTAs a head group (148, or 37 of 128 heads): the first and the last token are one
# piece; 32: pieces of some 14,000 and 56,000 keys; 1: every CTA a piece.
@pytest.mark.parametrize("sigma", [0.0, 0.5])
@pytest.mark.parametrize("n,new", [(64000, 150), (64000, 32), (20000, 150), (41000, 1)])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3"])
def test_a_dominant_key_before_a_long_tail(fmt, heads, n, new, sigma):
    new = new if heads == 16 or new < 100 else 38
    wl = sink_case(fmt, heads, n, new, sigma)
    out, lse = run(wl)
    check_tokens(f"{fmt} {heads} heads sigma {sigma}", wl, out, lse, sorted({0, new // 2, new - 1}))


@pytest.mark.parametrize("sigma", [1.0, 3.0])
@pytest.mark.parametrize("at", [0, 9000, 39990])
@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3", "bf16"])
def test_a_dominant_key_anywhere_among_spread_ones(fmt, at, sigma):
    """Weights over many binades, the dominant key first, in the middle and near the end."""
    wl = sink_case(fmt, 16, 40000, 150, sigma, at=at)
    out, lse = run(wl)
    check_tokens(f"{fmt} sigma {sigma} at {at}", wl, out, lse, [0, 149])


@pytest.mark.parametrize("fmt", ["fp8_ds_mla", "e4m3"])
def test_several_dominant_keys_and_steps_between_levels(fmt):
    """Stretches of keys 0, 6, 13, 30 and 60 octaves below the largest, in a mixed order, with
    a key at the top of every 1,777."""
    n, new = 30000, 150
    wl = sink_case(fmt, 16, n, new, 0.0)
    pe = np.zeros((n, 64))
    levels = np.array([13, 30, 6, 60, 13, 6, 0, 6, 30, 60, 13, 6], np.float64)
    step = levels[np.arange(n) * len(levels) // n]
    pe[:, 0] = -step * np.log(2.0) / 8
    pe[::1777, 0] = 0.0
    put_rows(wl, rows_of(wl, 0, np.arange(n)), latents(n), pe)
    q = np.zeros((new, 16, 576), np.float32)
    q[:, :, 512] = 8.0 * 32 * np.linspace(0.25, 1, 16)[None]
    wl.layers[0].q = synth.to_bf16_bits(q)
    out, lse = run(wl)
    check_tokens(f"{fmt} levels", wl, out, lse, [0, 75, 149])


def check_block_scales(name, wl, out, lse, tokens):
    """Against less than the contract for fp8_ds_mla allows: a weight within 2^-15 of V_b = the largest
    p_hi / pmax_h sc_ib of the heads that share an exponent (4, or 8 of 32 heads and more) over all keys
    (the contract: over pmax_h so far), times its head's pmax_h and its code, and the other terms of the
    module's bounds."""
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    pages, rows = F.physical(wl.block_table[0], np.arange(int(wl.ctx_len[0])))
    c_all, pe_all = F.latent_rows(wl.latent, pages, rows)
    sc_all = PC.block_scales(wl, pages, rows)
    for t in tokens:
        n = int(n_all[t])
        c, pe, sc = c_all[:n], pe_all[:n], sc_all[:n]
        q = F.decode_bf16(wl.layers[0].q[t])
        z = wl.sm_scale * (q[:, 512:] @ pe.T)
        top = z.max(1, keepdims=True)
        e = np.exp(z - top)                                      # p / pmax
        p = e / e.sum(1, keepdims=True)
        want, want_lse = p @ c, (top + np.log(e.sum(1, keepdims=True)))[:, 0]
        share = 4 if wl.num_heads == 16 else 8
        V = np.repeat((e[:, :, None] * sc[None]).max(1).reshape(-1, share, 4).max(1), share, 0)   # [H, 4]
        codes = np.abs(c.reshape(n, 4, 128) / sc[:, :, None]).sum(0)                            # [4, 128]
        d = 576 * 2.0 ** -23 * wl.sm_scale * (np.abs(q[:, 512:]) @ np.abs(pe).T).max(1)
        A = p @ np.abs(c)
        tol = 2 * d[:, None] * ((p * (1 - p)) @ np.abs(c)) + PC.U * np.abs(want) + (PC.U + 3 * 2.0 ** -11) * A * 1.01
        tol += (2.0 ** -15 * p.max(1)[:, None, None] * V[:, :, None] * codes[None]).reshape(-1, 512)
        ltol = d + (n / 128 + 8) * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(want_lse))
        PC.check(f"{name} token {t}", out[t], lse[t], (want, want_lse, tol, ltol))


def rising_case(heads, octaves, who, fall, gradual):
    """160 queries of one request of 2,208 tokens (16 tiles and more in a piece); the logits of the heads
    `who` rise by `octaves` a tile, the others' are level; from the fifth tile on, block 1's scales are
    2^-fall of what they were (gradual: reached over ten tiles)."""
    n, new = 2048 + 160, 160
    wl = synth.make_workload(f"weights/rise/{heads}", [n], [new], heads, layers=(("l", 64, False, None),))
    tile = np.arange(n) // 128
    pe = np.zeros((n, 64))
    pe[:, :8] = tile[:, None] / 16
    put_rows(wl, rows_of(wl, 0, np.arange(n)), latents(n), pe)
    rows = wl.latent.reshape(-1, 656)
    at = rows_of(wl, 0, np.arange(n))
    sc = np.ascontiguousarray(rows[at, 512:528]).view("<f4")
    sc[:, 1] *= np.exp2(-fall * (np.clip((tile - 3) / 10, 0, 1) if gradual else tile >= 4)).astype(np.float32)
    rows[at, 512:528] = sc.view(np.uint8)
    q = np.zeros((new, heads, 576), np.float32)
    q[:, who, 512:520] = octaves                                  # 8 dims, 1/16 a tile, times 2 ln 2
    wl.layers[0].q = synth.to_bf16_bits(q)
    wl.sm_scale = float(np.float32(2 * np.log(2.0)))
    return wl


@pytest.mark.parametrize("gradual", [False, True])
@pytest.mark.parametrize("fall", [8, 16, 40])
@pytest.mark.parametrize("octaves", [2, 3, 8])
@pytest.mark.parametrize("heads", [16, 64])
def test_logits_rise_while_one_blocks_scales_fall(heads, octaves, fall, gradual):
    """The exponent of a block's weights follows its scales down however slowly every M_h rises."""
    wl = rising_case(heads, octaves, slice(None), fall, gradual)
    out, lse = run(wl)
    check_block_scales(f"octaves {octaves} fall {fall}", wl, out, lse, [0, 80, 159])


@pytest.mark.parametrize("fall", [8, 16, 40])
@pytest.mark.parametrize("heads", [16, 64])
def test_one_head_rises_while_one_blocks_scales_fall(heads, fall):
    """One head of every four rises by 3 octaves a tile and does not take the others' bits, nor they its."""
    wl = rising_case(heads, 3, slice(1, None, 4), fall, False)
    out, lse = run(wl)
    check_block_scales(f"one head, fall {fall}", wl, out, lse, [0, 80, 159])


def shared_exponent_term(p, sc, codes, share):
    """What the weights of an fp8_ds_mla token (one piece) may be off by in all, [H, 512]: six deviations of
    roundings that differ from key to key, each at most 2^-13 of the unit 2^(M_h + eb_b) of its tile.
    2^M_h is at most 1 / 56 of the head's largest p so far, 2^eb_b at most 1 / 56 of the largest product
    (a weight of at most 440 times the block's scale) that the heads which share it have had since eb was
    last looked at: from then on, 8 octaves of M_h, 10 of a head's largest p (M_h follows within 2)."""
    H, n = p.shape
    starts = np.arange(0, n, 128)
    top = np.maximum(np.stack([p[:, a:a + 128].max(1) for a in starts], 1), 1e-300)          # [H, tiles]
    run = np.maximum.accumulate(top, 1)
    prod = np.stack([(p[:, a:a + 128, None] / run[:, i, None, None] * sc[None, a:a + 128]).max(1)
                     for i, a in enumerate(starts)], 1)                                      # [H, tiles, 4]
    prod = prod.reshape(-1, share, len(starts), 4).max(1)                                     # [quarters, tiles, 4]
    tol = np.zeros((H, 4, 128))
    for g in range(len(prod)):
        heads = slice(g * share, (g + 1) * share)
        since, looked = 0, run[heads, 0]
        for i, a in enumerate(starts):
            if (run[heads, i] > looked * 2.0 ** 10).any():
                since, looked = i, run[heads, i]
            unit = run[heads, i, None] / 56 * prod[g, since:i + 1].max(0) * 440 / 56           # [share, 4]
            tol[heads] += (2.0 ** -13 * unit[:, :, None]) ** 2 * (codes[a:a + 128] ** 2).sum(0).reshape(4, 128)
    return 6 * np.sqrt(tol).reshape(H, 512)


@pytest.mark.parametrize("large", [8, 16, 30])
@pytest.mark.parametrize("heads", [16, 64])
def test_heads_that_fall_do_not_hold_a_blocks_exponent(heads, large):
    """Half of the heads that share an exponent attend to the first keys, the others' logits rise by 5
    octaves a tile; one block's scales are 2^large larger in two tiles of the middle.  The rising heads'
    outputs, which come from the last tiles, keep their bits."""
    n, new = 2048 + 160, 160
    wl = synth.make_workload(f"weights/held/{heads}", [n], [new], heads, layers=(("l", 64, False, None),))
    tile = np.arange(n) // 128
    pe = np.zeros((n, 64))
    pe[:, :8] = tile[:, None] / 16
    put_rows(wl, rows_of(wl, 0, np.arange(n)), latents(n), pe)
    rows, at = wl.latent.reshape(-1, 656), rows_of(wl, 0, np.arange(n))
    sc = np.ascontiguousarray(rows[at, 512:528]).view("<f4")
    sc[(tile == 5) | (tile == 6), 2] *= np.float32(2.0 ** large)
    rows[at, 512:528] = sc.view(np.uint8)
    q = np.zeros((new, heads, 576), np.float32)
    q[:, ::2, 512:520], q[:, 1::2, 512:520] = -6, 5
    wl.layers[0].q = synth.to_bf16_bits(q)
    wl.sm_scale = float(np.float32(2 * np.log(2.0)))
    out, lse = run(wl)
    n_all = dsa.visible_lengths(wl.cu_q, wl.ctx_len)
    pages, rws = F.physical(wl.block_table[0], np.arange(n))
    c, pe = F.latent_rows(wl.latent, pages, rws)
    sc = PC.block_scales(wl, pages, rws)
    for t in (0, new - 1):
        m = int(n_all[t])
        want, want_lse, tol, ltol = PC.expect(wl, 0, t, np.arange(m))
        z = wl.sm_scale * (F.decode_bf16(wl.layers[0].q[t])[:, 512:] @ pe[:m].T)
        p = np.exp(z - want_lse[:, None])
        A = p @ np.abs(c[:m])
        d = (ltol - 2.0 ** -20 * (1 + np.abs(want_lse)))[:, None]
        tol = 2 * d * ((p * (1 - p)) @ np.abs(c[:m])) + PC.U * np.abs(want) + (PC.U + 3 * 2.0 ** -11) * A * 1.01
        tol += shared_exponent_term(p, sc[:m], c[:m] / np.repeat(sc[:m], 128, 1), 4 if heads == 16 else 8)
        PC.check(f"large {large} token {t}", out[t], lse[t], (want, want_lse, tol, ltol + (m / 128 + 8) * 2.0 ** -24))
