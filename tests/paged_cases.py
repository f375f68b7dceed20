"""Inputs, expected values and error bounds shared by the tests of the whole-cache operators.

Bounds of the attention's outputs, from its arithmetic (u = 2^-8, half a bf16 step relative
to the value):

* the output is rounded to bf16 once: u |out|;
* each softmax weight has at least 8 significant bits when it enters its product (u relative,
  plus 2^-11 for each rounding to half precision on the way: of the weight, of the scale it is
  multiplied with, and of the product); the same weights unrounded are summed for the
  denominator, so an output is off by at most (u + 3 * 2^-11) A, A = sum_i p_i |c_i|;
* a weight far below the largest keeps only an absolute error: half of E4M3's subnormal step
  (2^-10) in each of its two terms against a largest weight-times-scale of at least 28 (an
  output's keys share it within the spread of their block scales, a factor 4 for these inputs):
  2^-9 / 28 * 4 <= 2^-11.8 of the largest p, times sum_i |c_i|;
* a logit is a sum in fp32 of up to 576 products: off by at most d = 576 * 2^-23 of the summed terms'
  size (2^-23, not 2^-24: the tensor cores may cut instead of round).  A softmax weight then moves by
  p_i |d_i - mean d| <= 2 d p_i (1 - p_i), the output by 2 d sum_i p_i (1 - p_i) |c_i|, and the
  log-sum-exp by d, plus 2^-20 (1 + |lse|) for log2, exp2 and the sum of the weights.
"""
import numpy as np

from oracle import dsa, formats as F, mla
from tests import parity

U = 2.0 ** -8


def block_scales(wl, pages, rows):
    """[n, 4] block scales of rows of an fp8_ds_mla pool."""
    return np.ascontiguousarray(wl.latent.reshape(-1, 656)[pages * 64 + rows, 512:528]).view("<f4").astype(np.float64)


def small_weight_term(p, scales, c):
    """The third bound for block scales of any spread, [H, 512].  Four heads (eight of 32 heads and
    more) share a scale 2^eb for each block, set to put their largest weight of a 128-key tile,
    p' sc_b / 2^eb_b with p' = p / 2^M_h, into (56, 112] by powers of two, raised for a tile above it;
    M_h puts the largest p' of a tile into (56, 112] too.  So 2^M_h <= pmax_h / 56 and 2^eb_b <=
    112 / 56 V_b, V_b the largest p_hi / (pmax_h of the tile) sc_ib of those heads over the tiles,
    and half of E4M3's subnormal step in each of two terms is 2^-9 2^(M_h + eb_b) <=
    2^-9 / 28 pmax_h V_b for a code of one."""
    H, n = p.shape
    w = np.zeros((H, 4))
    for a in range(0, n, 128):
        top = np.maximum(p[:, a:a + 128].max(1), 1e-300)
        w = np.maximum(w, (p[:, a:a + 128, None] / top[:, None, None] * scales[None, a:a + 128]).max(1))
    heads = 4 if H == 16 else 8
    V = np.repeat(w.reshape(-1, heads, 4).max(1), heads, 0)
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.nan_to_num(np.abs(c.reshape(n, 4, 128)) / scales[:, :, None]).sum(0)
    return 2.0 ** -9 / 28 * p.max(1)[:, None] * (V[:, :, None] * codes[None]).reshape(H, 512)


def expect(wl, layer_i, t, positions, n=None, nss=None, any_scales=False):
    """(out, lse, out bound, lse bound) of token t over logical positions, in float64.
    any_scales: the third bound as small_weight_term has it."""
    v = wl.view(layer_i)
    r = int(dsa.request_of_tokens(wl.cu_q)[t])
    if n is None:
        n = int(dsa.visible_lengths(wl.cu_q, wl.ctx_len)[t])
    q = F.decode_bf16(v.q[t])
    H = q.shape[0]
    if len(positions) == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    pages, rows = F.physical(wl.block_table[r], positions)
    c, k_pe = F.latent_rows(parity.oracle_latent(wl), pages, rows)
    scale = wl.sm_scale * dsa.ssmax_factor(wl.ssmax, wl.ssmax_s, n if nss is None else nss)
    out, lse = mla.attend(q, c, k_pe, v.rope_dim, scale)
    keys = np.concatenate([c, k_pe], 1)[:, :q.shape[1]]
    p = np.exp(scale * (q @ keys.T) - lse[:, None])
    A = p @ np.abs(c)
    d = 576 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(keys).T).max(1)
    tol = 2 * d[:, None] * ((p * (1 - p)) @ np.abs(c)) + U * np.abs(out) + (U + 3 * 2.0 ** -11) * A * 1.01
    if any_scales:
        tol += small_weight_term(p, block_scales(wl, pages, rows), c)
    else:
        tol += 2.0 ** -11.8 * p.max(1)[:, None] * np.abs(c).sum(0)[None]
    return out, lse, tol, d + 2.0 ** -20 * (1 + np.abs(lse))


def check(name, got_out, got_lse, want):
    out, lse, tol, ltol = want
    got_out, got_lse = got_out.astype(np.float64), got_lse.astype(np.float64)
    assert np.isfinite(got_out).all(), name
    assert np.array_equal(np.isfinite(got_lse), np.isfinite(lse)), f"{name}: finiteness of lse"
    over = np.abs(got_out - out) - tol
    assert (over <= 0).all(), f"{name}: out off by up to {np.abs(got_out - out).max():.3e}, {(over > 0).sum()} beyond"
    fin = np.isfinite(lse)
    d = np.abs(got_lse[fin] - lse[fin])
    assert (d <= ltol[fin]).all(), f"{name}: lse off by {d.max():.3e}, allowed {ltol[fin].min():.3e}"


def spoil_unused(wl, positions_kept=None):
    """NaN codes, NaN scales and NaN RoPE keys (0xFF bytes) in every row of the pool that no
    request holds, the rows behind each request's last token among them."""
    row = {"e4m3": 576, "bf16": 1152}.get(wl.latent_format, 656)
    lat = wl.latent.reshape(wl.num_pages * 64, row)
    held = np.zeros(wl.num_pages * 64, dtype=bool)
    for r in range(wl.B):
        pos = np.arange(int(wl.ctx_len[r]))
        held[wl.block_table[r, pos // 64].astype(np.int64) * 64 + pos % 64] = True
    lat[~held] = 0xFF
    return wl
