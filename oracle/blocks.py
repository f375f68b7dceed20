"""Selection of whole 64-token pages and reading cached rows back, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* block key of a page: the mean of its 64 dequantised indexer keys, stored as a
  key is (``oracle.producers``: E4M3 codes and one fp32 scale, decided in
  float32), in the row of the page's number of a pool in the indexer layout;
* block score of page j of token t: the indexer's score (``oracle.dsa``) with
  the block key in the key's place, for the pages j < (n_t - 1) // 64 that lie
  wholly before the page of the token's newest position;
* block selection: the k - 1 best of those pages (larger score first, NaN last,
  -0.0 equal to +0.0, ties to the lower page), ascending, then the page of the
  newest position;
* reading back: a cached row's values, code times scale, in float64.

vLLM blog "vLLM 首日支持 Mistral Large 4", section "实现细节 / 模型架构" (the
indexer and its FP8 cache); the pages print no block selection.
"""
from __future__ import annotations

import numpy as np

from . import dsa, formats as F, producers as PR

ROWS = F.PAGE_TOKENS


def block_keys(index_pool, pages, block_pool):
    """The block pool after writing the keys of ``pages`` (-1 skips; a page
    outside the pool is skipped and reported), and whether one was reported."""
    out = block_pool.copy()
    num_pages = index_pool.size // F.INDEXER_PAGE_BYTES
    bad = False
    for p in np.asarray(pages, dtype=np.int64):
        if p == -1:
            continue
        if p < 0 or p >= num_pages:
            bad = True
            continue
        keys = F.indexer_keys(index_pool, np.full(ROWS, p), np.arange(ROWS))
        codes, scale = PR.quantise_block((keys.sum(axis=0) / ROWS).astype(np.float32))
        base, row = (p // ROWS) * F.INDEXER_PAGE_BYTES, p % ROWS
        out[base + row * F.INDEXER_DIM:base + (row + 1) * F.INDEXER_DIM] = codes
        at = base + F.INDEXER_KEYS_BYTES + 4 * row
        out[at:at + 4] = np.frombuffer(np.float32(scale).tobytes(), dtype=np.uint8)
    return out, bad


def candidates(n):
    """Pages wholly before the page of position n - 1."""
    return max(0, (int(n) - 1) // ROWS)


def block_scores_row(q8_t, q_scale_t, w_t, block_pool, bt_row, n, c_t):
    """(scores, size of the summed terms) of one token's candidate pages."""
    pages = np.asarray(bt_row[:candidates(n)], dtype=np.int64)
    k = F.indexer_keys(block_pool, pages // ROWS, pages % ROWS)
    relu = np.maximum(F.decode_e4m3(q8_t) * float(q_scale_t) @ k.T, 0.0)
    w = np.asarray(w_t, dtype=np.float64)[:, None]
    return c_t * (w * relu).sum(axis=0), abs(c_t) * (np.abs(w) * relu).sum(axis=0)


def block_topk_row(scores, n, k):
    """Selected pages of one token that sees n positions."""
    if n < 1:
        return np.empty(0, dtype=np.int64)
    c = candidates(n)
    return np.append(dsa.topk_row(np.asarray(scores)[:c], k - 1), c)


def block_positions(blocks, n):
    """Positions the listed blocks hold, those at or past n left out."""
    pos = (np.asarray(blocks, dtype=np.int64)[:, None] * ROWS + np.arange(ROWS)).reshape(-1)
    return pos[pos < n]


def read_latent(pool, slot):
    """(c [n, 512], k_pe [n, 64]) of the rows slot (all >= 0), in float64."""
    s = np.asarray(slot, dtype=np.int64)
    return F.latent_rows(pool, s // ROWS, s % ROWS)


def read_indexer_k(pool, slot):
    s = np.asarray(slot, dtype=np.int64)
    return F.indexer_keys(pool, s // ROWS, s % ROWS)
