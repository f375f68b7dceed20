"""Queries whose dims differ by many octaves, on the GPU against the float64 oracle: the FP8 pools'
two E4M3 terms of a query are exact down to 2^-2 s_h, and within 2^-10 s_h below that, s_h the power
of two at or above amax_h / 448 (include/sml.h).

A logit is then off by at most scale 2^-10 s_h sum |k_d| over the dims below 2^-2 s_h, on top of the
bounds of tests/paged_cases.py: e of that moves a weight by at most p_i (1 - p_i) (exp(2 e) - 1) and
the log-sum-exp by e.  The dims above the rest meet keys of 0, so that the logits are the others'."""
import numpy as np
import pytest

from oracle import dsa, formats as F
from sparse_mla_attention_indexer_b200 import sml, synth
from tests import paged_cases as PC, parity
from tests.test_gpu_paged_weights import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_mla_attention_indexer_b200 import build
    build.build()
    sml.lib()


def check_all(name, wl, shared):
    """shared: whether the latent and the RoPE query have one scale (plain E4M3) or the latter none."""
    out, lse = run(wl)
    rope = wl.layers[0].rope_dim
    for t, n in enumerate(dsa.visible_lengths(wl.cu_q, wl.ctx_len)):
        want, want_lse, tol, ltol = PC.expect(wl, 0, t, np.arange(int(n)))
        r = int(dsa.request_of_tokens(wl.cu_q)[t])
        pages, rows = F.physical(wl.block_table[r], np.arange(int(n)))
        c, pe = F.latent_rows(parity.oracle_latent(wl), pages, rows)
        q = np.abs(F.decode_bf16(wl.layers[0].q[t]))
        part = q if shared else q[:, :512]
        keys = np.abs(np.concatenate([c, pe], 1)[:, :part.shape[1]])
        s = np.exp2(np.ceil(np.log2(part.max(1, keepdims=True) / 448)))
        e = wl.sm_scale * 2.0 ** -10 * (s * (part < s / 4)) @ keys.T if wl.latent_format != "bf16" else np.zeros((len(q), 1))
        e = e.max(1)
        z = wl.sm_scale * (F.decode_bf16(wl.layers[0].q[t]) @ np.concatenate([c, pe], 1)[:, :512 + rope].T)
        p = np.exp(z - want_lse[:, None])
        tol = tol + np.expm1(2 * e)[:, None] * ((p * (1 - p)) @ np.abs(c))
        PC.check(f"{name} token {t}", out[t], lse[t], (want, want_lse, tol, ltol + e))


@pytest.mark.parametrize("octaves", [6, 10, 13])
@pytest.mark.parametrize("fmt,heads", [("fp8_ds_mla", 16), ("fp8_ds_mla", 64), ("e4m3", 16), ("e4m3", 32), ("bf16", 16)])
def test_one_dim_far_above_the_others(fmt, heads, octaves):
    wl = synth.make_workload(f"query/{fmt}/{heads}", [700, 130], [1, 2], heads, latent_format=fmt,
                             layers=(("l", 64, False, None),))
    rows = wl.latent.reshape(wl.num_pages * 64, -1)
    size = 2 if fmt == "bf16" else 1
    for dim in (5, 400):                                          # 400: of the last block
        rows[:, size * dim:size * (dim + 1)] = 0
    q = F.decode_bf16(wl.layers[0].q)
    top = np.abs(q).max(2)
    q[:, ::2, 5], q[:, 1::2, 400] = top[:, ::2] * 2.0 ** octaves, -top[:, 1::2] * 2.0 ** octaves
    wl.layers[0].q = synth.to_bf16_bits(q.astype(np.float32))
    check_all(f"{fmt} {heads} heads, {octaves} octaves", wl, fmt == "e4m3")


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("octaves", [-10, 10])
def test_latent_and_rope_queries_of_different_size(octaves, heads):
    """Plain E4M3: the latent and the RoPE query share a scale; the larger one meets keys of 0."""
    wl = synth.make_workload(f"query/rope/{heads}", [700, 130], [1, 2], heads, latent_format="e4m3",
                             layers=(("l", 64, False, None),))
    rows = wl.latent.reshape(-1, 576)
    q = F.decode_bf16(wl.layers[0].q)
    if octaves > 0:
        rows[:, 512:] = 0
        q[..., 512:] *= 2.0 ** octaves
    else:
        rows[:, :512:2] = 0                                       # every other latent dim, so that an output is left
        q[..., :512:2] *= 2.0 ** -octaves
    wl.layers[0].q = synth.to_bf16_bits(q.astype(np.float32))
    check_all(f"rope by {octaves} octaves", wl, True)
