// Absorbed-query MLA over a paged latent cache: every visible token of a
// request, the last `window` of them, or the 64-token blocks listed for each
// query token.  Split over the cache's length, then a log-sum-exp join.
//
// vLLM blog "vLLM 首日支持 Mistral Large 4": highlights list (MLA, KV LoRA rank
// 512, RoPE dim 64); section on DSpark (sliding-window MLA draft layers over a
// bf16 cache).  For token t, head h:
//   z_i = sm_scale * c_t * (q_nope . c_hat_i + q_pe . k_pe_i)
//   out = sum_i softmax(z)_i c_hat_i,   lse = ln sum_i exp(z_i)
// over the positions i that the token attends to, in one pass over the rows
// with a running exponent and sum per head.
//
// A unit is (query token, group of 16 heads, or 32 of 32 heads and more, tile of
// two pages = 128 keys).  One CTA per SM works out its range of them from the
// device's lengths (plan_range) and walks it:
//   * warp 18 looks up pages and loads them by TMA, 64 rows x 128 B a box in the
//     128-B swizzle, into two tile buffers (one of bf16), a quarter of the
//     latent dims at a time;
//   * warp 16 issues S^T = C Q^T (keys as M, heads as N: 16 or 32 heads as M
//     would waste half of the smallest M and more), straight from the E4M3 codes,
//     the bf16 query split into two E4M3 terms; one accumulator per block
//     scale, RoPE apart in bf16;
//   * warps 0-15 read S^T (thread = key x a quarter of the heads), scale, take
//     2^(z - M_h) and write the weights, block scale folded in, as two E4M3
//     terms, the second times 2^4 (bf16 pools: two bf16 terms);
//   * warp 17 issues O^T += C^T W^T, the tile read MN-major, and frees the tile a
//     quarter of the dims at a time.
// The latent is never converted, and every wait is bounded: one that gives up
// sets SML_FAULT_TIMEOUT and the CTA winds down.
//
// What bounds it, and what it measured (B200, 6.57 TB/s copy):
//   * 16 heads, 32 contexts of 8K to 64K tokens: HBM.  146 us for 787 MB, 5.4
//     TB/s; bf16 rows of the same batch 226 us, 93 % of the copy rate.  A tile
//     takes 2.0 us against 1.9 of a 148th of that rate; the rest is what stands
//     before and after the loop (first loads, uneven finish, join).
//   * 128 heads, 32 tokens of 60,000 (four groups of 32 heads, which read a tile
//     from L2 after the first): 945 us, 566 TFLOP/s of the attention's own.  The
//     two buffers' cycle bounds it, and probably shared memory under it: of 3,500
//     to 3,900 cycles a tile the products' operands take 1,930 by the rate of
//     products timed alone (their operands' bytes / 128 B, 52 cycles at N = 64
//     whatever their majors; no counter shows it), TMA's writes 660 and the weights
//     400, and each slows the others (PV takes 2,900 cycles from its first product
//     to its last).  Issue 46 %, L2 35 %.  Twice the
//     heads a product would read the tile half as often, but 64 heads' O and
//     logits do not fit in TMEM, nor a third buffer beside the query and the
//     weights (224 KB); weights handed to PV in two waves, two loading warps, and
//     raising M_h further at a time changed nothing.
//   * few tiles a CTA (selected blocks, one short context): the chain of first
//     loads, first tile, output and join, 14 us at least.  Code that a CTA runs
//     once or twice costs what it takes to fetch, 0.5 to 0.9 us for 2 to 3 KB of
//     it unrolled, so there a lane works for all (rebase, the row sums).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "ptx.cuh"
#include "sml_internal.cuh"

namespace sml {
namespace {

constexpr int kKT = 128;                 // keys per tile: two pages
// A tile's latent dims arrive, enter QK^T and PV and are freed in quarters of
// 128, block part_block(p) as the p-th.  The scales and the RoPE keys come with
// the second: the products left when the last part lands are then four, and
// with 32 heads, whose weights for the first two output blocks lie where the
// RoPE keys were, those are read by then.
constexpr int kParts = 4, kRopePart = 1;
__host__ __device__ constexpr int part_block(int part) { return (part + 3) & 3; }
constexpr int kLatBlock = kKT * 128;     // one 128-B wide block of a tile
constexpr int kSoftmaxWarps = 16;        // warps 0-15
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kWarpQk = 16, kWarpPv = 17, kWarpLoad = 18;
constexpr int kThreads = 608;
constexpr uint32_t kColO = 256;          // TMEM: logits from column 0, O from here
constexpr float kNoM = -1e30f;            // M_h before a head's first key: any logit is far above it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
template <int kHU>
constexpr int kGroupBf = 2 * kHU * 2 * 8;  // bytes of an 8-key group of bf16 weights

struct Params {
  int B, T, H, rope_dim, max_ctx, max_pages, ssmax;
  float sm_scale, ssmax_s;
  const int32_t* cu_q;
  const int32_t* ctx_len;
  const int32_t* block_table;
  const int32_t* vis_len;
  const int32_t* ssmax_len;
  const uint16_t* q;
  const uint8_t* latent;
  int64_t latent_pages;
  float latent_scale;
  PagedSel sel;
  uint16_t* out;
  float* lse;
  PagedWs ws;
  int32_t* status;
};

// What query token t attends to: np pages (page k is logical page first_page +
// k, or the k-th listed block) of request r, positions [lo, n) of them.
struct Tok {
  int r, n, nss, lo, np;
  bool ok, len_bad;
};

// Every load of a token's lengths in one round: with equal query counts its
// request is t B / T, which the request's own offsets confirm; else a binary
// search and a second round.
__device__ __forceinline__ Tok token_at(const Params& P, int t) {
  Tok k;
  k.r = (int)((unsigned)((long long)t * P.B) / (unsigned)P.T);   // t, B, T <= 65535
  Req rq = load_request(P.cu_q, P.ctx_len, k.r, P.T, P.max_ctx, P.max_pages, P.vis_len != nullptr);
  const int vis = P.vis_len ? __ldg(P.vis_len + t) : 0, ssl = P.ssmax_len ? __ldg(P.ssmax_len + t) : 0;
  const int len = P.sel.blocks ? __ldg(P.sel.blocks_len + t) : 0;
  if (!(rq.q0 <= t && t - rq.q0 < rq.Q)) {
    k.r = request_of(P.cu_q, P.B, t);
    rq = load_request(P.cu_q, P.ctx_len, k.r, P.T, P.max_ctx, P.max_pages, P.vis_len != nullptr);
  }
  k.ok = rq.ok && t >= rq.q0 && t - rq.q0 < rq.Q;
  if (P.vis_len) {
    k.ok = k.ok && vis >= 0 && vis <= rq.L;
    k.n = k.ok ? vis : 0;
  } else {
    k.n = k.ok ? rq.L - rq.Q + (t - rq.q0) + 1 : 0;
  }
  k.nss = max(1, P.ssmax_len ? ssl : k.n);
  k.lo = P.sel.window > 0 && k.n > P.sel.window ? k.n - P.sel.window : 0;
  k.len_bad = P.sel.blocks && k.ok && (len < 0 || len > P.sel.max_blocks);
  k.np = !P.sel.blocks ? (k.n + SML_PAGE_TOKENS - 1) / SML_PAGE_TOKENS - k.lo / SML_PAGE_TOKENS
         : k.ok        ? max(0, min(len, P.sel.max_blocks))
                       : 0;
  return k;
}

__device__ __forceinline__ int tiles_of(const Tok& k) { return max(1, (k.np + 1) / 2); }

// Logical and physical page of the k-th and the l-th page of token t (physical
// -1: masked, and reported where asked); the loads of both overlap.
struct Page {
  int lg, ph;
};
__device__ __forceinline__ void pages_at(const Params& P, const Tok& tk, int t, int k, bool report_k, Page& a, int l,
                                         bool report_l, Page& b) {
  const bool ka = k < tk.np, kb = l < tk.np;
  a.lg = tk.lo / SML_PAGE_TOKENS + k;
  b.lg = tk.lo / SML_PAGE_TOKENS + l;
  bool va = ka, vb = kb;
  if (P.sel.blocks) {
    const int32_t* list = P.sel.blocks + (size_t)t * P.sel.max_blocks;
    const int all = (tk.n + SML_PAGE_TOKENS - 1) / SML_PAGE_TOKENS;
    a.lg = ka ? __ldg(list + k) : 0;
    b.lg = kb ? __ldg(list + l) : 0;
    va = ka && a.lg >= 0 && a.lg < all;
    vb = kb && b.lg >= 0 && b.lg < all;
    if ((ka && !va && report_k) || (kb && !vb && report_l)) raise_fault(P.status, SML_FAULT_INDEX);
  }
  const int32_t* table = P.block_table + (size_t)tk.r * P.max_pages;
  a.ph = va ? __ldg(table + a.lg) : -1;
  b.ph = vb ? __ldg(table + b.lg) : -1;
  const bool pa = a.ph >= 0 && a.ph < P.latent_pages, pb = b.ph >= 0 && b.ph < P.latent_pages;
  if ((va && !pa && report_k) || (vb && !pb && report_l)) raise_fault(P.status, SML_FAULT_PAGE);
  if (!pa) a.ph = -1;
  if (!pb) b.ph = -1;
  if (!va) a.lg = 0;
  if (!vb) b.lg = 0;
}

// This CTA's range [ub, ue) of its head group's tiles, and the token t0 that it
// starts in (tok0: that token's first tile).
struct Range {
  long long total, ub, ue, tok0;
  int used, t0;
  int m;   // > 0: m CTAs to every token, see share
};
struct PlanSmem {
  long long part[32];   // per warp of the block
  int longest[32];
  long long tok0;
  int t0, base;
  Tok tok[32];          // tokens base to base + 31: a small batch's, else those from where the range starts
};

// a / b of non-negative numbers, in 32 bits where both fit (a 64-bit division
// is a long routine, and several stand at the start of every CTA).
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int cta_of(long long total, int used, long long u) { return (int)div_ll((u + 1) * used - 1, total); }

// Two ways to share the tiles.  (1) Equal contiguous ranges, as few as give the
// same longest one; a range may hold the ends of two tokens.  (2) m = cpg / T
// CTAs to every token, each an equal piece of it: no CTA has more than one piece,
// but the longest token decides.  A piece costs about as much as three tiles
// more (its query, its first tile, its output), and joining split tokens two.
// 128 heads (37 CTAs a head group), 32 tokens: over 32 selected blocks, selection
// included, 56 us with whole tokens and 71 with equal ranges; over 60,000 tokens
// of context equal ranges are 4 % faster.
__device__ __forceinline__ void share(Range& R, int T, int cpg, int gi, int longest) {
  const long long most = div_ll(R.total + cpg - 1, cpg);
  R.m = T <= cpg ? (int)((unsigned)cpg / (unsigned)T) : 0;
  if (R.m > 0 && (longest + R.m - 1) / R.m + 3 + (R.m > 1 ? 2 : 0) <= most + 8) {
    R.used = R.m * T;
    R.t0 = (int)((unsigned)gi / (unsigned)R.m);
    return;   // the range follows from token t0's tiles, see piece
  }
  R.m = 0;
  R.used = (int)div_ll(R.total + most - 1, most);
  R.ub = gi < R.used ? div_ll(R.total * gi, R.used) : 0;
  R.ue = gi < R.used ? div_ll(R.total * (gi + 1), R.used) : 0;
}
// Way (2): this CTA's piece of token t0, which has nt tiles (nt < m: some of the
// m CTAs have none).
__device__ __forceinline__ void piece(Range& R, int gi, int nt) {
  const int m = min(R.m, nt), i = gi - R.t0 * R.m;
  R.tok0 = 0;
  R.ub = gi < R.used && i < m ? div_ll((long long)nt * i, m) : 0;
  R.ue = gi < R.used && i < m ? div_ll((long long)nt * (i + 1), m) : 0;
}
// The CTAs that hold a token whose first tile is tok0, of nt tiles.
__device__ __forceinline__ int2 holders(const Range& R, int nt) {
  if (R.m > 0) return make_int2(R.t0 * R.m, R.t0 * R.m + min(R.m, nt) - 1);
  return make_int2(cta_of(R.total, R.used, R.tok0), cta_of(R.total, R.used, R.tok0 + nt - 1));
}

// Token t's lengths, from shared memory where they are there.
__device__ __forceinline__ Tok token_of(const Params& P, const PlanSmem& S, int t) {
  const unsigned i = t - S.base;
  return i < 32 ? S.tok[i] : token_at(P, t);
}

// Every thread of the block calls it.  Up to 32 tokens: each warp for itself, 1.6
// us from the first load to the range (1.3 where one warp plans for all, which
// changed nothing in all; with the scan over the block below, 1 us more).
__device__ __forceinline__ Range plan_range(const Params& P, int gi, PlanSmem& S) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Range R;
  if (P.T <= 32) {
    const Tok tk = token_at(P, min(lane, P.T - 1));
    if (warp == 0) S.tok[lane] = tk;
    if (threadIdx.x == 0) S.base = 0;
    const int mine = lane < P.T ? tiles_of(tk) : 0;   // at most 2^23 each
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    R.total = __shfl_sync(0xffffffffu, upto, 31);
    share(R, P.T, P.ws.cpg, gi, __reduce_max_sync(0xffffffffu, mine));
    if (R.m > 0) {
      piece(R, gi, __shfl_sync(0xffffffffu, mine, min(R.t0, P.T - 1)));
      __syncthreads();
      return R;
    }
    const unsigned in = __ballot_sync(0xffffffffu, upto - mine <= R.ub && R.ub < upto);
    R.t0 = __ffs(in) - 1;
    R.tok0 = __shfl_sync(0xffffffffu, upto - mine, R.t0);
    __syncthreads();
    return R;
  }
  // A thread a token, or a few: their tiles, summed over the block.
  const int per = (P.T + kThreads - 1) / kThreads, a = min(P.T, (int)threadIdx.x * per), b = min(P.T, a + per);
  const Tok own = token_at(P, min(a, P.T - 1));
  long long mine = 0;
  int longest = 0;
  for (int t = a; t < b; ++t) {
    const int nt = tiles_of(t == a ? own : token_at(P, t));
    mine += nt;
    longest = max(longest, nt);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) {
    S.part[warp] = upto;
    S.longest[warp] = longest;
  }
  __syncthreads();
  R.total = 0;
  long long before = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? S.part[w] : 0;
    R.total += S.part[w];
    longest = max(longest, S.longest[w]);
  }
  share(R, P.T, P.ws.cpg, gi, longest);
  const long long first = before + upto - mine;   // first tile of token a
  if (R.m == 0 && first <= R.ub && R.ub < first + mine) {
    long long at = first;
    for (int t = a; t < b; ++t) {
      const int nt = tiles_of(t == a ? own : token_at(P, t));
      if (R.ub < at + nt) {
        S.t0 = t;
        S.tok0 = at;
        break;
      }
      at += nt;
    }
  }
  __syncthreads();
  if (R.m == 0) {
    R.t0 = S.t0;
    R.tok0 = S.tok0;
  }
  // The range's own tokens stay in shared memory where a thread holds one each
  // (a load round less at every token's start).
  if (threadIdx.x == 0) S.base = per == 1 ? R.t0 : P.T;
  if (per == 1 && a < b && (unsigned)(a - R.t0) < 32) S.tok[a - R.t0] = own;
  __syncthreads();
  if (R.m > 0) piece(R, gi, tiles_of(token_of(P, S, min(R.t0, P.T - 1))));
  return R;
}

// ---- the attention kernel -------------------------------------------------------

// Latent formats of the kernel's template parameter.
constexpr int kFmtDsMla = SML_LATENT_FP8_DS_MLA, kFmtPlain = SML_LATENT_E4M3, kFmtBf16 = SML_LATENT_BF16;
template <int kFmt>
struct Fmt {
  static constexpr bool kDs = kFmt == kFmtDsMla, kPlain = kFmt == kFmtPlain, kBf = kFmt == kFmtBf16;
  static constexpr int kBufs = kBf ? 1 : 2;        // tile buffers (a bf16 tile is 144 KB)
  static constexpr uint32_t kPageBytes = kBf ? SML_LATENT_BF16_PAGE_BYTES : kPlain ? SML_LATENT_E4M3_PAGE_BYTES : SML_LATENT_PAGE_BYTES;
  static constexpr int kBlocks = kBf ? 8 : 4;      // 128-B wide blocks of a tile's latents
  static constexpr int kSets = kDs ? 4 : 1;        // weight sets: one per block scale
  // Logit accumulators: one per block scale, and RoPE's.  Both query terms'
  // columns stand side by side (one MMA of twice the width costs about as much
  // as one: 42 cycles at N = 32, 49 at 64), except those of the last block
  // where 32 heads would leave no room for them beside O: they are summed.
  static constexpr bool split_terms(int heads, int b) { return !kBf && !(kDs && heads == 32 && b == 3); }
  static constexpr uint32_t col_block(int heads, int b) { return kDs ? 2 * heads * b : 0; }
  static constexpr uint32_t col_rope(int heads) { return heads == 32 ? 224 : 128; }
  static constexpr int kPeX = kBf ? 2 * SML_LATENT_DIM : kPlain ? SML_LATENT_DIM : SML_LATENT_DIM + 16;
};

template <int kFmt, int kHU>
struct __align__(1024) Smem {
  using F = Fmt<kFmt>;
  static constexpr int kSetBytes = kKT * 2 * kHU * (F::kBf ? 2 : 1);   // both terms of one weight set
  // With 32 heads per unit the weight sets of a tile's first two output blocks
  // live where its RoPE keys were: those are dead once the tile's logits are done.
  static constexpr bool kOverlay = F::kDs && kHU == 32;
  static constexpr int kOwnSets = kOverlay ? 2 : F::kSets;
  __device__ __forceinline__ uint32_t set_addr(int b, int buf) const {
    if (F::kSets == 1) return ptx::smem_u32(pb[0]);
    if (!kOverlay) return ptx::smem_u32(pb[b]);
    return b == part_block(0)   ? ptx::smem_u32(pe[buf])
           : b == part_block(1) ? ptx::smem_u32(pe[buf]) + kSetBytes
                                : ptx::smem_u32(pb[b == part_block(2) ? 0 : 1]);
  }
  uint8_t lat[F::kBufs][F::kBlocks][kLatBlock];   // [buffer][block][128 keys x 128 B], SW128
  uint8_t pe[F::kBufs][kKT * 128];                // [buffer][128 keys x 128 B] RoPE keys, SW128
  uint8_t q8[1024 * kHU];   // E4M3: [block] 2 kHU rows (high, then low term) x 128 B, SW128; bf16: 8 blocks of kHU rows
  uint8_t qpe[(F::kPlain ? 2 : 1) * kHU * 128];   // RoPE query, SW128 (plain E4M3: high, then low term)
  uint8_t pb[kOwnSets][kSetBytes];                // weight sets: 8-key x 16-B core matrices
  float sc[F::kDs ? F::kBufs : 1][kKT][4];        // [buffer][key] block scales
  __align__(8) float xmax[4][4][kHU / 4];                      // [head quarter][key quarter][head]
  __align__(16) float xscale[4][4][4];            // [head quarter][key quarter][block]
  float mlook[16][kHU / 4], ebtop[16][4];         // [warp][head], [warp][block]: see rebase
  __align__(8) float nm[16][kHU / 4], fac[16][kHU / 4];   // [warp][head] -M_h, and what O scales by
  __align__(8) float xsum[4][4][kHU / 4];
  float qs[kHU];                                  // power-of-two query scale per head
  int4 rows[4];                                   // [tile % 4] valid rows {lo, hi} of each page of the tile
  uint64_t full[F::kBufs][kParts], lat_free[F::kBufs][kParts];   // per quarter of the latent dims
  uint64_t q_ready, s_full, s_free, p_full, pv_done, o_free, drain[2];
  uint32_t tmem_base;
  int abort;
  PlanSmem plan;
};

// A piece of a token in this CTA's range: tiles [j0, j0 + ne) of it (ne = 0:
// the token attends to nothing).
struct Seg {
  Tok tk;
  int t, j0, ne;
  bool whole;
  size_t part;   // its first row in the partials
};
struct Walk {
  long long u, ue;
  int t, j0;
};
__device__ __forceinline__ bool walk_next(const Params& P, const PlanSmem& ts, Walk& w, int slot, int heads, Seg& s) {
  if (w.u >= w.ue) return false;
  s.t = w.t;
  s.tk = token_of(P, ts, w.t);
  const int nt = tiles_of(s.tk), nj = (int)min((long long)(nt - w.j0), w.ue - w.u);
  s.j0 = w.j0;
  s.ne = s.tk.np > 0 ? nj : 0;
  s.whole = w.j0 == 0 && nj == nt;
  s.part = (size_t)(slot + (w.j0 == 0)) * heads;
  w.u += nj;
  ++w.t;
  w.j0 = 0;
  return true;
}

// Cursor over the tiles of the range, in order: tile jj of the seg-th piece
// that has any, the k-th tile overall.
struct Cur {
  Walk w;
  int ne, jj, seg, k;
  bool valid;
};
__device__ __forceinline__ void cur_seek(Cur& c, const Params& P, const PlanSmem& ts) {
  Seg s;
  c.jj = 0;
  c.valid = false;
  while (walk_next(P, ts, c.w, 0, 0, s)) {
    c.ne = s.ne;
    if (s.ne > 0) {
      c.valid = true;
      return;
    }
  }
}
__device__ __forceinline__ void cur_next(Cur& c, const Params& P, const PlanSmem& ts) {
  ++c.k;
  if (++c.jj < c.ne) return;
  ++c.seg;
  cur_seek(c, P, ts);
}

// Byte address of (row, 16-B chunk) in a 128-B-swizzled tile of 128-B rows.
__device__ __forceinline__ uint32_t sw128(uint32_t base, int row, int chunk) {
  return base + (row >> 3) * 1024 + (row & 7) * 128 + ((chunk ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_b32(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}

__device__ __forceinline__ void st_b16(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"((uint16_t)a) : "memory");
}

__device__ __forceinline__ uint32_t f2_to_e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) & 0xffffu;
}
// Two floats -> E4M3 codes of the nearest values; x becomes the residuals.
__device__ __forceinline__ uint32_t split_e4m3x2(float& x0, float& x1) {
  const uint32_t c = f2_to_e4m3x2(x0, x1);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
  const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h));
  x0 -= r.x;
  x1 -= r.y;
  return c;
}
// Two weights (at most 448) in half precision as two E4M3 terms, hi + 2^-4 lo:
// eight significant bits, as many as a bf16 has, where the sparse attention's
// three terms carry twelve.  A third would not fit: 32 heads' O of three terms, 384
// columns, and their logits, 256, are more than tensor memory's 512.  The three
// roundings to half precision before (of the weight, the scale and their product,
// 2^-11 each) let one instruction split two heads' weights; all of it is 1.4 x
// 2^-8 of a weight at most.  x - hi is exact in half precision and at most 16, so lo stays within 256; the
// epilogue gives lo's columns of O their 2^-4.  (hi without the conversion back,
// by Veltkamp's splitting in half precision, measured the same.)
//
// Weights below 2^-6 keep lo's subnormal step, 2^-13, and a long context behind a
// dominant key holds tens of thousands of them, which add up: alike, they would
// all be rounded the same way, or to nothing.  So lo is rounded with a dither, an
// offset of less than half a step that depends on the key's row of the tile
// (dither_of): 128 weights alike are off by at most half a step in all, others at
// random, and one that is a tenth of a step is a step at a tenth of the rows.
__device__ __forceinline__ uint32_t half2_to_e4m3x2(__half2 x) {
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, __NV_E4M3) & 0xffffu;
}
constexpr float kLoScale = 16.f;
__device__ __forceinline__ __half2 dither_of(int row) {   // (2 bitrev(row) - 127) / 256 of lo's step 2^-9
  return __float2half2_rn((float)(2 * (int)(__brev((uint32_t)row) >> 25) - 127) * 0x1p-17f);
}
__device__ __forceinline__ void split2_e4m3x2(__half2 x, __half2 dither, uint32_t& hi, uint32_t& lo) {
  hi = half2_to_e4m3x2(x);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3);
  lo = half2_to_e4m3x2(__hfma2(__hsub2_rn(x, *reinterpret_cast<const __half2*>(&h)), __float2half2_rn(kLoScale), dither));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e: 0 below the smallest normal number, at most 2^127.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __int_as_float((127 + min(e, 127)) << 23); }

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort));
}
// AND of a flag over the softmax threads (named barrier 5): a wait that gave up
// ends all of them together instead of leaving some blocked at a barrier.
__device__ __forceinline__ bool softmax_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 5, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(kSoftmaxThreads)
      : "memory");
  return r != 0;
}
// OR of a flag over the four warps of one head quarter (named barrier 1 +
// quarter; also a barrier for them).
__device__ __forceinline__ bool group_any(int hq, bool v) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"((uint32_t)v), "r"(1 + hq)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int hq) { asm volatile("bar.sync %0, 128;" ::"r"(1 + hq) : "memory"); }

// Column (and query row) of head h's term among 2 heads columns: each head
// quarter's high terms, then its low terms, so that one thread's are adjacent.
template <int kHU>
__device__ __forceinline__ int split_col(int h, int term) {
  constexpr int kHT = kHU / 4;
  return (h / kHT) * (2 * kHT) + term * kHT + h % kHT;
}

__device__ __forceinline__ void tmem_ldn(uint32_t a, uint32_t (&r)[16]) { ptx::tmem_ld16(a, r); }
__device__ __forceinline__ void tmem_stn(uint32_t a, const uint32_t (&r)[16]) { ptx::tmem_st16(a, r); }
__device__ __forceinline__ void tmem_ldn(uint32_t a, uint32_t (&r)[4]) { ptx::tmem_ld4(a, r); }
__device__ __forceinline__ void tmem_ldn(uint32_t a, uint32_t (&r)[8]) { ptx::tmem_ld8(a, r); }
__device__ __forceinline__ void tmem_stn(uint32_t a, const uint32_t (&r)[8]) { ptx::tmem_st8(a, r); }

// Stage the query of (token t, head group g); thread = head x 1 / kPer of its
// latent dims and RoPE dims.  E4M3 pools: q = s_h (hi + lo), both E4M3, s_h the
// power of two with amax_h <= 448 s_h.  A bf16 has 8 significant bits, four in
// each term, and lo's step is 2^-9: exact wherever |q| >= 2^-2 s_h; below, within
// half that step, 2^-10 s_h, 2^-17.8 of amax_h or less (2^-8.8 of an element 2^-9
// of the largest, a bf16's own rounding; 2^-5 of one 2^-13 of it).  RoPE: bf16 as
// given (fp8_ds_mla), or split the same way (plain E4M3).  bf16 pools: the bf16
// query as given.
template <int kFmt, int kHU>
__device__ __forceinline__ void stage_query(const Params& P, Smem<kFmt, kHU>& S, int t, int g, int tid) {
  using F = Fmt<kFmt>;
  constexpr int kPer = kSoftmaxThreads / kHU;          // threads a head: 32 or 16
  constexpr int kChunks = SML_LATENT_DIM / kPer / 16;   // 16-dim chunks a thread: 1 or 2
  const int h = tid / kPer, p = tid % kPer;
  const uint16_t* qh = P.q + ((size_t)t * P.H + g * kHU + h) * (SML_LATENT_DIM + P.rope_dim);
  const uint32_t q0 = ptx::smem_u32(S.q8), qp = ptx::smem_u32(S.qpe);
  if constexpr (F::kBf) {
    const int nc = P.rope_dim ? 72 : 64;
    for (int c = p; c < nc; c += kPer) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(qh) + c);
      st_v4(c < 64 ? sw128(q0 + (c >> 3) * (kHU * 128), h, c & 7) : sw128(qp, h, c - 64), v.x, v.y, v.z, v.w);
    }
    if (p == 0) S.qs[h] = 1.f;
  } else {
    uint4 v[2 * kChunks];
#pragma unroll
    for (int i = 0; i < 2 * kChunks; ++i) v[i] = __ldcg(reinterpret_cast<const uint4*>(qh) + 2 * kChunks * p + i);
    constexpr int kPe = 64 / kPer / 2;   // pairs of RoPE dims a thread: 1 or 2
    uint32_t pv[kPe] = {};
    if (P.rope_dim) {
#pragma unroll
      for (int i = 0; i < kPe; ++i) pv[i] = __ldcg(reinterpret_cast<const uint32_t*>(qh + SML_LATENT_DIM) + kPe * p + i);
    }
    // amax as the largest bit pattern without sign
    uint32_t m2 = 0;
    auto amax2 = [&](uint32_t w) { m2 = __vmaxu2(m2, w & 0x7fff7fffu); };
#pragma unroll
    for (int i = 0; i < 2 * kChunks; ++i) {
      amax2(v[i].x);
      amax2(v[i].y);
      amax2(v[i].z);
      amax2(v[i].w);
    }
    if (F::kPlain) {
#pragma unroll
      for (int i = 0; i < kPe; ++i) amax2(pv[i]);
    }
#pragma unroll
    for (int o = 1; o < kPer; o <<= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    const int amax = max((int)(m2 & 0xffffu), (int)(m2 >> 16));
    // 448 = 1.75 * 2^8; 2^-e2 stays finite (a query that small gives logits of 0 either way)
    const int e2 = max((amax >> 7) - 127 - 8 + ((amax & 127) > 96), -120);
    const float inv = __int_as_float((127 - e2) << 23);
    if (p == 0) S.qs[h] = amax < 0x7f80 ? __int_as_float((127 + e2) << 23) : NAN;   // infinities would be clipped
    auto split2 = [&](uint32_t w, uint32_t& hi, uint32_t& lo) {
      float x0 = __uint_as_float(w << 16) * inv, x1 = __uint_as_float(w & 0xffff0000u) * inv;
      hi = split_e4m3x2(x0, x1);
      lo = f2_to_e4m3x2(x0, x1);
    };
    auto split4 = [&](uint32_t wa, uint32_t wb, uint32_t& hi, uint32_t& lo) {
      uint32_t h2, l2;
      split2(wa, hi, lo);
      split2(wb, h2, l2);
      hi |= h2 << 16;
      lo |= l2 << 16;
    };
    // dims [16 kChunks p, ..) -> block p / (kPer / 4), 16-B chunks kChunks (p % (kPer / 4)) ..
    const int blk = p / (kPer / 4);
    const uint32_t qb = q0 + blk * (2 * kHU * 128);
    const bool split = F::split_terms(kHU, blk);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      uint32_t hw[4], lw[4];
      split4(v[2 * c].x, v[2 * c].y, hw[0], lw[0]);
      split4(v[2 * c].z, v[2 * c].w, hw[1], lw[1]);
      split4(v[2 * c + 1].x, v[2 * c + 1].y, hw[2], lw[2]);
      split4(v[2 * c + 1].z, v[2 * c + 1].w, hw[3], lw[3]);
      const int chunk = kChunks * (p % (kPer / 4)) + c;
      st_v4(sw128(qb, split ? split_col<kHU>(h, 0) : h, chunk), hw[0], hw[1], hw[2], hw[3]);
      st_v4(sw128(qb, split ? split_col<kHU>(h, 1) : h + kHU, chunk), lw[0], lw[1], lw[2], lw[3]);
    }
    if (P.rope_dim) {
#pragma unroll
      for (int i = 0; i < kPe; ++i) {
        const int at = kPe * p + i;   // pair of dims
        if (F::kPlain) {
          uint32_t hi, lo;
          split2(pv[i], hi, lo);
          st_b16(sw128(qp, split_col<kHU>(h, 0), at >> 3) + 2 * (at & 7), hi);
          st_b16(sw128(qp, split_col<kHU>(h, 1), at >> 3) + 2 * (at & 7), lo);
        } else {
          st_b32(sw128(qp, h, at >> 2) + 4 * (at & 3), pv[i]);
        }
      }
    }
  }
}

// Weights are capped at 440 (E4M3's largest value is 448; the margin covers the
// approximate 2^x and log2) and set to at most 112.  bf16 weights need no such
// range: M_h only keeps them within 2^16.
template <int kFmt>
constexpr float kCap = kFmt == kFmtBf16 ? 16.f : 8.78135971f;    // log2(440)
template <int kFmt>
constexpr float kHead = kFmt == kFmtBf16 ? 0.f : 6.80735492f;    // log2(112)
constexpr float kFar = 50.f;   // a block scale 2^kFar above 2^eb raises eb whatever its key's weight: lk stays finite

// log2 of a key's largest block scale, relative to 2^eb of its block.
__device__ __forceinline__ float log_rel(const float (&sc)[4], const float (&ebf)[4]) {
  const float top = fmaxf(fmaxf(sc[0] * ebf[0], sc[1] * ebf[1]), fmaxf(sc[2] * ebf[2], sc[3] * ebf[3]));
  return lg2(fminf(fmaxf(top, 0x1p-60f), 0x1p100f));
}

// The exponents that the weights of a tile need, for the four warps of a head
// quarter (its heads, this thread's key), and what has been summed up so far in
// units of the new ones.  A lane works out one head's, or one block's, and all
// read it back: this code is run once in a while, and fetched for it (with every
// thread working out all of them, unrolled, a pass took 0.9 us more).
//
// A head whose largest softmax weight of the tile is above 2^limit takes the
// integer M_h that puts it in (56, 112]: headroom of 4 for later tiles, and the
// dominant weights keep all eight bits.  Then the same for each block's weight
// times scale, over the quarter's heads: eb rises where a product passes the cap,
// and else, once some M_h has risen by kLook octaves since the last look (mlook),
// falls to what this tile's largest product needs, so that scales that fall while
// logits rise keep their bits.  Heads whose logits fall do not hold it.  (A look at
// every rise takes 4 to 7 % more time in the verification step, after 4 octaves 2
// to 5 %, after 8 1 %.)  What O holds grows as eb falls: within kFall octaves of
// the largest eb so far (ebtop, less what every M_h has risen by since) O stays
// below 2^112, 2^30 keys of 440 x 448 each.  O scales by powers of two, exactly.
//
// In: z the logits + lk; out: z less M_h.  last: the tile whose PV O waits for;
// -1 where O holds nothing yet.  False: that wait gave up (every warp takes part
// in the barriers all the same).
template <int kFmt, int kHU, int kHP>
__device__ __forceinline__ bool rebase(Smem<kFmt, kHU>& S, float2 (&z)[kHP], float2 (&nM)[kHP], float2 (&lrow)[kHP],
                                       const float (&scv)[4], float (&ebf)[4], float& lk, uint32_t T0, int last) {
  using F = Fmt<kFmt>;
  constexpr int kHT = kHU / 4, kFirst = 1000;
  constexpr float kLook = 8.f, kFall = 64.f;
  constexpr float kLimit = F::kDs ? kHead<kFmt> + 1.f : kCap<kFmt>;   // (the block's scale may come on top)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp & 3, hq = warp >> 2;
  // this thread's latent dim of output block 0, this quarter's heads
  const uint32_t o_addr = T0 + kColO + 2 * kHT * hq + ((uint32_t)(32 * q4) << 16);
  bool ok = true;
  if constexpr (F::kDs) {
#pragma unroll
    for (int i = 0; i < kHP; ++i) z[i] = __fadd2_rn(z[i], make_float2(-lk, -lk));
  }
#pragma unroll
  for (int i = 0; i < kHP; ++i) {
    const float a = ptx::warp_max_f32(z[i].x), b = ptx::warp_max_f32(z[i].y);
    if (lane == 0) *reinterpret_cast<float2*>(&S.xmax[hq][q4][2 * i]) = make_float2(a, b);
  }
  group_sync(hq);
  bool look = false;   // whether some M_h has risen by kLook octaves since eb was looked at (or is new)
  {
    const int h = lane % kHT;
    const float e = fmaxf(fmaxf(S.xmax[hq][0][h], S.xmax[hq][1][h]), fmaxf(S.xmax[hq][2][h], S.xmax[hq][3][h]));
    float neg = S.nm[warp][h];
    const bool was = neg != -kNoM;
    int by = 0;
    if (e + neg > kLimit) {
      const float Mn = ceilf(e - kHead<kFmt>);
      by = (int)fminf(Mn + neg, 500.f);   // a positive integer (of a head without M_h: any)
      neg = -Mn;
    }
    __syncwarp();   // every lane has read the old one
    if (lane < kHT) {
      S.nm[warp][h] = neg;
      S.fac[warp][h] = was ? pow2(-by) : 1.f;
    }
    if constexpr (F::kDs) look = __any_sync(0xffffffffu, -neg - S.mlook[warp][h] >= kLook);
    const bool any = __any_sync(0xffffffffu, was && by > 0);   // (also makes the stores visible to the warp)
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kHP; ++i) {
      nM[i] = *reinterpret_cast<const float2*>(&S.nm[warp][2 * i]);
      lrow[i] = __fmul2_rn(lrow[i], *reinterpret_cast<const float2*>(&S.fac[warp][2 * i]));
      z[i] = __fadd2_rn(z[i], nM[i]);
    }
    if (any && last >= 0) ok = warp_wait(&S.pv_done, last & 1, &S.abort);   // the last tile's PV accumulates into O
    if (any && last >= 0 && ok) {
      ptx::tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t ov[2 * kHT];
        tmem_ldn(o_addr + 2 * kHU * b, ov);
        ptx::tmem_wait_ld(ov);
#pragma unroll
        for (int i = 0; i < kHT; ++i) {
          const float fi = S.fac[warp][i];
          ov[i] = __float_as_uint(__uint_as_float(ov[i]) * fi);
          ov[kHT + i] = __float_as_uint(__uint_as_float(ov[kHT + i]) * fi);
        }
        tmem_stn(o_addr + 2 * kHU * b, ov);
      }
      ptx::tmem_wait_st();
    }
  }
  if constexpr (F::kDs) {
    float u = -kFar;
#pragma unroll
    for (int i = 0; i < kHP; ++i) u = fmaxf(u, fmaxf(z[i].x, z[i].y));
    if (look || group_any(hq, u + lk > kCap<kFmt>)) {
      float v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) v[b] = ptx::warp_max_f32(u + lg2(scv[b]));
      if (lane == 0) *reinterpret_cast<float4*>(S.xscale[hq][q4]) = make_float4(v[0], v[1], v[2], v[3]);
      group_sync(hq);
      const int b = lane & 3;
      const float t = fmaxf(fmaxf(S.xscale[hq][0][b], S.xscale[hq][1][b]), fmaxf(S.xscale[hq][2][b], S.xscale[hq][3][b]));
      const float was = b & 2 ? (b & 1 ? ebf[3] : ebf[2]) : (b & 1 ? ebf[1] : ebf[0]);
      const int eb = 127 - (int)(__float_as_uint(was) >> 23);
      const int fit = (int)ceilf(fminf(fmaxf(t - kHead<kFmt>, -126.f), 126.f));
      // what every M_h has risen by (a head without one, or with an infinite one, aside)
      const float mh = -S.nm[warp][lane % kHT], ml = S.mlook[warp][lane % kHT], gone = mh - ml;
      const int rise = __reduce_min_sync(0xffffffffu, ml != kNoM && gone < (float)kFirst ? (int)gone : kFirst);
      const float top = S.ebtop[warp][b] - (float)rise;
      const int to = rise == kFirst               ? fit
                     : t - (float)eb > kCap<kFmt> ? max(fit, eb)
                     : t > -INFINITY              ? max(min(fit, eb), (int)(top - kFall))
                                                  : eb;   // (scales of 0: nothing to fit)
      __syncwarp();   // every lane has read the old ones
      if (lane < kHT) S.mlook[warp][lane] = mh;
      if (lane < 4) S.ebtop[warp][b] = rise == kFirst ? (float)to : fmaxf(top, (float)to);
      const float now = pow2(-to);
#pragma unroll
      for (int i = 0; i < 4; ++i) ebf[i] = __shfl_sync(0xffffffffu, now, i);
      const bool moved = last >= 0 && __any_sync(0xffffffffu, to != eb);
      if (moved) ok = ok && warp_wait(&S.pv_done, last & 1, &S.abort);
      if (moved && ok) {
        const float f = pow2(eb - to);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, i);
          uint32_t ov[2 * kHT];
          tmem_ldn(o_addr + 2 * kHU * i, ov);
          ptx::tmem_wait_ld(ov);
#pragma unroll
          for (int h = 0; h < 2 * kHT; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * fi);
          tmem_stn(o_addr + 2 * kHU * i, ov);
        }
        ptx::tmem_wait_st();
      }
      lk = log_rel(scv, ebf);
    }
#pragma unroll
    for (int i = 0; i < kHP; ++i) z[i] = __fadd2_rn(z[i], make_float2(lk, lk));
  }
  return ok;
}

template <int kFmt, int kHU>
__global__ void __launch_bounds__(kThreads, 1)
paged_mla_kernel(const __grid_constant__ CUtensorMap row_map, const __grid_constant__ CUtensorMap scale_map,
                 const __grid_constant__ Params P) {
  using F = Fmt<kFmt>;
  using Sm = Smem<kFmt, kHU>;
  constexpr int kBufs = F::kBufs, kHT = kHU / 4;   // kHT: heads per softmax thread
  extern __shared__ uint8_t smem_raw[];
  Sm& S = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = (int)blockIdx.x % P.ws.hg, gi = (int)blockIdx.x / P.ws.hg;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBufs * kParts; ++i) {
      ptx::mbar_init(&S.full[0][0] + i, 1);
      ptx::mbar_init(&S.lat_free[0][0] + i, 1);
    }
    ptx::mbar_init(&S.q_ready, kSoftmaxWarps);
    ptx::mbar_init(&S.s_full, 1);
    ptx::mbar_init(&S.s_free, kSoftmaxWarps);
    ptx::mbar_init(&S.p_full, kSoftmaxWarps);
    ptx::mbar_init(&S.pv_done, 1);
    ptx::mbar_init(&S.o_free, kSoftmaxWarps);
    ptx::mbar_init(&S.drain[0], 1);
    ptx::mbar_init(&S.drain[1], 1);
    S.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kWarpQk) {
    ptx::tmem_alloc(&S.tmem_base, 512);
    ptx::tmem_relinquish();
  }
  if (warp == kWarpLoad && lane == 0) {
    ptx::prefetch_tensormap(&row_map);
    if (F::kDs) ptx::prefetch_tensormap(&scale_map);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::griddep_wait();
  // this CTA holds its tensor memory: a dependent grid cannot starve it
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  volatile int* abort = &S.abort;
  const uint32_t T0 = S.tmem_base;
  const PlanSmem& ts = S.plan;
  const Range R = plan_range(P, gi, S.plan);
  const int slot = (g * P.ws.cpg + gi) * 2;
  if (warp == kWarpPv) {
    // the token that this CTA continues, and the CTAs that hold it
    int4 rec = make_int4(-1, 0, 0, 0);
    if (R.ub > R.tok0 && R.ub < R.ue) {
      const int2 h = holders(R, tiles_of(token_of(P, ts, R.t0)));
      rec = make_int4(R.t0, h.x, h.y, gi);
    }
    if (lane == 0) P.ws.join[g * P.ws.cpg + gi] = rec;
  }
  const Walk begin = {R.ub, R.ue, R.t0, (int)(R.ub - R.tok0)};

  if (warp == kWarpLoad) {
    // ================= producer: page ids, then TMA =================
    Walk w = begin;
    Seg s;
    int k = 0, begun = 0;   // tiles so far, and parts of the next one
    bool ok = true;
    const bool rope = P.rope_dim != 0;
    constexpr int kPartBlocks = F::kBlocks / kParts;
    constexpr uint32_t kPartBytes = kPartBlocks * SML_PAGE_TOKENS * 128;   // of one page
    const uint32_t rope_bytes = kPartBytes + (F::kDs ? SML_PAGE_TOKENS * 16 : 0) + (rope ? SML_PAGE_TOKENS * 128 : 0);
    while (ok && walk_next(P, ts, w, slot, kHU, s)) {
      if (lane == 0 && g == 0) {
        if (!s.tk.ok) raise_fault(P.status, SML_FAULT_LENGTHS);
        if (s.tk.len_bad) raise_fault(P.status, SML_FAULT_TOPK_LEN);
      }
      Page pg = {0, -1}, pn = {0, -1};   // pages 2 (j0 + 16 i) + lane, and 32 on
      for (int jj = 0; jj < s.ne; ++jj, ++k) {
        const int buf = k % kBufs, two = 2 * (jj & 15), k0 = 2 * (s.j0 + jj) + lane;
        if (jj == 0) {
          pages_at(P, s.tk, s.t, k0, lane < 2 * s.ne, pg, k0 + 32, lane + 32 < 2 * s.ne, pn);
        } else if (two == 0) {
          pg = pn;
          Page none;
          pages_at(P, s.tk, s.t, k0 + 32, lane + 32 < 2 * (s.ne - jj), pn, s.tk.np, false, none);
        }
        const int p0 = __shfl_sync(0xffffffffu, pg.ph, two), p1 = __shfl_sync(0xffffffffu, pg.ph, two + 1);
        const int l0 = __shfl_sync(0xffffffffu, pg.lg, two), l1 = __shfl_sync(0xffffffffu, pg.lg, two + 1);
        // While the tile's buffer is still in use its pages go to L2 (one head
        // group asks for all): 32 contexts of 8K to 64K tokens take 148 us, 158
        // without; two tiles ahead 153, four 207.
        if (g == 0 && k >= kBufs && lane < 2) {
          const int ph = lane == 0 ? p0 : p1;
          if (ph >= 0) ptx::bulk_prefetch_l2(P.latent + (size_t)ph * F::kPageBytes, F::kPageBytes);
        }
        const uint32_t pages = (p0 >= 0) + (p1 >= 0);
        for (int part = 0; part < kParts; ++part) {
          begun = part;
          if (k >= kBufs) ok = warp_wait(&S.lat_free[buf][part], ((k / kBufs) - 1) & 1, abort);
          if (!ok) break;
          if (lane == 0) {
            const bool with_rope = part == kRopePart;
            if (with_rope) {
              int4 r;   // valid rows of each page: none of one that is not loaded
              r.x = max(0, s.tk.lo - l0 * SML_PAGE_TOKENS);
              r.y = p0 >= 0 ? min(SML_PAGE_TOKENS, s.tk.n - l0 * SML_PAGE_TOKENS) : 0;
              r.z = max(0, s.tk.lo - l1 * SML_PAGE_TOKENS);
              r.w = p1 >= 0 ? min(SML_PAGE_TOKENS, s.tk.n - l1 * SML_PAGE_TOKENS) : 0;
              S.rows[k & 3] = r;   // last read by the softmax of tile k - 4
            }
            uint64_t* bar = &S.full[buf][part];
            ptx::mbar_arrive_expect_tx(bar, pages * (with_rope ? rope_bytes : kPartBytes));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int ph = half ? p1 : p0, y = ph * SML_PAGE_TOKENS, off = half * SML_PAGE_TOKENS * 128;
              if (ph < 0) continue;
#pragma unroll
              for (int b = 0; b < kPartBlocks; ++b)
                ptx::tma_load_2d(S.lat[buf][part_block(part) * kPartBlocks + b] + off, &row_map, bar,
                                 128 * (part_block(part) * kPartBlocks + b), y);
              if (with_rope && F::kDs)
                ptx::tma_load_2d(&S.sc[F::kDs ? buf : 0][half * SML_PAGE_TOKENS][0], &scale_map, bar, SML_LATENT_DIM, y);
              if (with_rope && rope) ptx::tma_load_2d(S.pe[buf] + off, &row_map, bar, F::kPeX, y);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        begun = 0;
      }
    }
    if (!ok) *abort = 1;
    // nothing of this CTA's in flight when its shared memory goes away
    for (int part = 0; part < kParts; ++part) {
      const int n = k + (part < begun);   // loads of this part so far
      for (int i = max(0, n - kBufs); i < n; ++i)
        ptx::mbar_wait(&S.full[i % kBufs][part], (i / kBufs) & 1, nullptr, 100000u);
    }
    __syncwarp();
  } else if (warp == kWarpQk) {
    // ================= QK^T issuer =================
    constexpr uint32_t id_q1 = F::kBf ? ptx::idesc_f16(kHU, 1, 0, 0) : ptx::idesc_f16(kHU, 0, 0, 0);
    constexpr uint32_t id_q2 = ptx::idesc_f16(2 * kHU, 0, 0, 0);   // both terms
    constexpr uint32_t id_pe = ptx::idesc_f16(kHU, 1, 0, 0);
    const uint32_t q0 = ptx::smem_u32(S.q8), qp = ptx::smem_u32(S.qpe);
    // One part of a tile's QK^T: 128 latent dims, and with the second the RoPE dims.
    auto issue_qk = [&](int buf, int part) {
      if constexpr (F::kBf) {
        // S^T = C . Q^T + K_pe . Q_pe^T, 16 dims per step
#pragma unroll
        for (int bb = 0; bb < 2; ++bb)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int b = 2 * part_block(part) + bb;
            ptx::mma_bf(T0, ptx::sdesc_sw128(ptx::smem_u32(S.lat[buf][b]) + 32 * kk),
                        ptx::sdesc_sw128(q0 + b * (kHU * 128) + 32 * kk), id_q1, (part | bb | kk) != 0);
          }
      } else {
        // S_b^T = C_b . [Qhi_b; Qlo_b]^T, 32 dims per step (plain E4M3: one sum over the blocks)
        const int b = part_block(part);
        const bool split = F::split_terms(kHU, b);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int term = 0; term < (split ? 1 : 2); ++term)
            ptx::mma_f8(T0 + F::col_block(kHU, b), ptx::sdesc_sw128(ptx::smem_u32(S.lat[buf][b]) + 32 * kk),
                        ptx::sdesc_sw128(q0 + (2 * b + term) * (kHU * 128) + 32 * kk), split ? id_q2 : id_q1,
                        F::kDs ? (kk | term) != 0 : (part | kk) != 0);
      }
      const uint32_t pe0 = ptx::smem_u32(S.pe[buf]);
      if (part == kRopePart && P.rope_dim) {
        if constexpr (F::kPlain) {
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            ptx::mma_f8(T0, ptx::sdesc_sw128(pe0 + 32 * kk), ptx::sdesc_sw128(qp + 32 * kk), id_q2, true);
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_bf(T0 + (F::kDs ? F::col_rope(kHU) : 0), ptx::sdesc_sw128(pe0 + 32 * kk), ptx::sdesc_sw128(qp + 32 * kk),
                        id_pe, F::kBf || kk > 0);
        }
      }
      if (part == kParts - 1) ptx::mma_commit(&S.s_full);
    };
    // One elected lane issues, from code with the buffer and part known at
    // compile time, so that the descriptors are constants off a uniform base.
    Cur c;
    c.w = begin;
    c.seg = c.k = 0;
    cur_seek(c, P, ts);
    bool ok = true;
    for (; c.valid; cur_next(c, P, ts)) {
      const int buf = c.k % kBufs;
      if (c.jj == 0) ok = warp_wait(&S.q_ready, c.seg & 1, abort);                    // the piece's query is staged
      if (ok && c.k > 0) ok = warp_wait(&S.s_free, (c.k - 1) & 1, abort);             // the last tile's S has been read
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        ok = ok && warp_wait(&S.full[buf][part], (c.k / kBufs) & 1, abort);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          if (buf == 0) issue_qk(0, part);
          else issue_qk(kBufs - 1, part);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok) *abort = 1;
    // every MMA issued has finished before TMEM is released
    if (ptx::elect_one()) ptx::mma_commit(&S.drain[0]);
    __syncwarp();
    ptx::mbar_wait(&S.drain[0], 0, nullptr, 100000u);
    __syncwarp();
  } else if (warp == kWarpPv) {
    // ================= PV issuer =================
    constexpr uint32_t id_pv = F::kBf ? ptx::idesc_f16(2 * kHU, 1, 1, 1) : ptx::idesc_f16(2 * kHU, 0, 1, 1);
    // O_b^T (+)= C_b^T . [Bhi_b; Blo_b]^T for the four 128-dim output blocks,
    // each freeing its part of the tile.  A: the tile read MN-major (dims
    // contiguous; 8-key swizzle atoms 1,024 B apart; of a bf16 tile the two
    // 64-dim atoms of an output block 16 KB apart).  B: 8-key x 16-B core
    // matrices, along the heads 128 B apart.
    constexpr int kKeysPerStep = F::kBf ? 16 : 32;
    constexpr uint32_t kGroup = 2 * kHU * (F::kBf ? 2 : 1) * 8;   // bytes of an 8-key group of a weight set
    auto issue_pv = [&](int buf, bool first) {
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const int b = part_block(part);
        const uint32_t set = S.set_addr(b, buf);
#pragma unroll
        for (int st = 0; st < kKT / kKeysPerStep; ++st) {
          const uint64_t bd = ptx::sdesc(set + st * (kKeysPerStep / 8) * kGroup, kGroup, 128, 0);
          const uint32_t d = T0 + kColO + 2 * kHU * b;
          if constexpr (F::kBf)
            ptx::mma_bf(d, ptx::sdesc(ptx::smem_u32(S.lat[buf][2 * b]) + 2048 * st, 16384, 1024, 2), bd, id_pv, st > 0 || !first);
          else
            ptx::mma_f8(d, ptx::sdesc(ptx::smem_u32(S.lat[buf][b]) + 4096 * st, 16384, 1024, 2), bd, id_pv, st > 0 || !first);
        }
        ptx::mma_commit(&S.lat_free[buf][part]);
      }
      ptx::mma_commit(&S.pv_done);
    };
    Cur c;
    c.w = begin;
    c.seg = c.k = 0;
    cur_seek(c, P, ts);
    bool ok = true;
    for (; c.valid; cur_next(c, P, ts)) {
      const int buf = c.k % kBufs;
      if (c.jj == 0 && c.seg > 0) ok = warp_wait(&S.o_free, (c.seg - 1) & 1, abort);  // the last piece's O has been read
      ok = ok && warp_wait(&S.p_full, c.k & 1, abort);                                // weights written, masked rows zeroed
      if (!ok) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        if (buf == 0) issue_pv(0, c.jj == 0);
        else issue_pv(kBufs - 1, c.jj == 0);
      }
      __syncwarp();
    }
    if (!ok) *abort = 1;
    if (ptx::elect_one()) ptx::mma_commit(&S.drain[1]);
    __syncwarp();
    ptx::mbar_wait(&S.drain[1], 0, nullptr, 100000u);
    __syncwarp();
  } else if (warp < kSoftmaxWarps) {
    // ================= softmax =================
    // TMEM lane quarter (keys, and latent dims in the epilogue) and head
    // quarter: this thread owns key (or dim) `row` for heads kHT hq ..
    const int q4 = warp & 3, hq = warp >> 2, row = 32 * q4 + lane, tid = threadIdx.x;
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    const __half2 dither = dither_of(row);
    auto stage = [&](const Seg& s) {
      stage_query<kFmt, kHU>(P, S, s.t, g, tid);
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.q_ready);
    };
    Walk w = begin;
    Seg s;
    int k = 0;
    bool ok = true, staged = false;
    while (walk_next(P, ts, w, slot, kHU, s)) {
      // every softmax thread is done with the last piece: its S.qs and S.xsum
      ok = softmax_all(ok);
      if (!ok) break;
      const size_t orow = (size_t)s.t * P.H + g * kHU;
      if (s.ne == 0) {
        // nothing to attend to (always a whole token)
        for (int i = tid; i < kHU * SML_LATENT_DIM / 8; i += kSoftmaxThreads)
          reinterpret_cast<uint4*>(P.out + orow * SML_LATENT_DIM)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tid < kHU) P.lse[orow + tid] = -INFINITY;
        continue;
      }
      if (!staged) stage(s);
      staged = false;
      ok = softmax_all(ok);   // S.qs visible to every softmax thread
      // logits in log2 units, so that p = 2^(z - M)
      const float zscale = P.sm_scale * (P.ssmax ? P.ssmax_s * logf((float)s.tk.nss) : 1.f) * kLog2e *
                           (F::kPlain ? P.latent_scale : 1.f);
      // Two heads to an instruction (add / fma.f32x2): the scale of their
      // logits, -M_h and this key row's share of the row sum, in units of 2^M_h.
      constexpr int kHP = kHT / 2;
      float2 qz[kHP], nM[kHP], lrow[kHP];
#pragma unroll
      for (int i = 0; i < kHP; ++i) {
        qz[i] = make_float2(S.qs[kHT * hq + 2 * i] * zscale, S.qs[kHT * hq + 2 * i + 1] * zscale);
        nM[i] = make_float2(-kNoM, -kNoM);
        lrow[i] = make_float2(0.f, 0.f);
      }
      if (lane < kHT) {
        S.nm[warp][lane] = -kNoM;
        S.mlook[warp][lane] = kNoM;
      }
      // A block's scales enter the weights relative to 2^eb, so that every block
      // uses E4M3's range whatever its magnitude; the output is multiplied back.
      float ebf[4] = {1.f, 1.f, 1.f, 1.f};   // 2^-eb
      for (int jj = 0; jj < s.ne; ++jj, ++k) {
        const int buf = k % kBufs;
        ok = ok && warp_wait(&S.full[buf][kRopePart], (k / kBufs) & 1, abort) && warp_wait(&S.s_full, k & 1, abort);
        ptx::tc_fence_after();
        const int4 rr = S.rows[k & 3];
        const int prow = row & 63;
        const bool valid = row < 64 ? prow >= rr.x && prow < rr.y : prow >= rr.z && prow < rr.w;
        const bool partial = (rr.x | rr.z) != 0 || rr.y != SML_PAGE_TOKENS || rr.w != SML_PAGE_TOKENS;
        // z = zscale (s_h sum_b scale_b (S_b,hi + S_b,lo) + S_pe) + lk, with lk
        // the logarithm of the key's largest block scale: 2^(z - M_h) bounds the
        // key's weights.  Block scales are taken relative to 2^eb, see above.
        float scv[4] = {1.f, 1.f, 1.f, 1.f};
        float lk = 0.f, rk = 1.f;   // and rk = 2^-lk
        float2 z[kHP];
        if constexpr (F::kDs) {
          const float4 f = *reinterpret_cast<const float4*>(S.sc[buf][row]);
          scv[0] = f.x;
          scv[1] = f.y;
          scv[2] = f.z;
          scv[3] = f.w;
          if (partial && !valid) scv[0] = scv[1] = scv[2] = scv[3] = 0.f;
          lk = log_rel(scv, ebf);
          rk = ex2(-lk);
          float2 acc[kHP];
#pragma unroll
          for (int i = 0; i < kHP; ++i) acc[i] = make_float2(0.f, 0.f);
          auto add = [&](const uint32_t* v, float sc) {   // acc += sc v, kHT values
            const float2 s2 = make_float2(sc, sc);
#pragma unroll
            for (int i = 0; i < kHP; ++i)
              acc[i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, acc[i]);
          };
#pragma unroll
          for (int b = 0; b < 4; b += 2) {   // two blocks at a time: their loads overlap
            uint32_t v[2][2 * kHT], w[kHT];
            tmem_ldn(T0 + F::col_block(kHU, b) + 2 * kHT * hq + lane_off, v[0]);
            if (F::split_terms(kHU, b + 1)) tmem_ldn(T0 + F::col_block(kHU, b + 1) + 2 * kHT * hq + lane_off, v[1]);
            else tmem_ldn(T0 + F::col_block(kHU, b + 1) + kHT * hq + lane_off, w);
            ptx::tmem_wait_ld();
            ptx::reg_fence(v[0]);
            if (F::split_terms(kHU, b + 1)) ptx::reg_fence(v[1]);
            else ptx::reg_fence(w);
            add(v[0], scv[b]);
            add(v[0] + kHT, scv[b]);
            if (F::split_terms(kHU, b + 1)) {
              add(v[1], scv[b + 1]);
              add(v[1] + kHT, scv[b + 1]);
            } else {
              add(w, scv[b + 1]);
            }
          }
          const float2 lk2 = make_float2(lk, lk), zs2 = make_float2(zscale, zscale);
          if (P.rope_dim) {
            uint32_t v[kHT];
            tmem_ldn(T0 + F::col_rope(kHU) + kHT * hq + lane_off, v);
            ptx::tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < kHP; ++i)
              z[i] = __ffma2_rn(acc[i], qz[i],
                                __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), zs2, lk2));
          } else {
#pragma unroll
            for (int i = 0; i < kHP; ++i) z[i] = __ffma2_rn(acc[i], qz[i], lk2);
          }
        } else {
          uint32_t v[F::kBf ? kHT : 2 * kHT];
          tmem_ldn(T0 + (F::kBf ? kHT : 2 * kHT) * hq + lane_off, v);
          ptx::tmem_wait_ld(v);
#pragma unroll
          for (int i = 0; i < kHP; ++i) {
            float2 x = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            if constexpr (!F::kBf)
              x = __fadd2_rn(x, make_float2(__uint_as_float(v[kHT + 2 * i]), __uint_as_float(v[kHT + 2 * i + 1])));
            z[i] = __fmul2_rn(x, qz[i]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.s_free);   // S read: the next tile's QK^T may overwrite it
        if (partial && !valid) {
#pragma unroll
          for (int i = 0; i < kHP; ++i) z[i] = make_float2(-INFINITY, -INFINITY);
        }
        // The weights 2^(z - M_h) must stay within E4M3's 448.  One above the
        // cap, or a head without M_h yet, sends the quarter's four warps through
        // the exact update (a vote: rare after the first tile).
        float2 d[kHP];
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < kHP; ++i) {
          d[i] = __fadd2_rn(z[i], nM[i]);
          most = fmaxf(most, fmaxf(d[i].x, d[i].y));
        }
        if (F::kDs) most = fmaxf(most, lk - kFar);
        if (group_any(hq, most > kCap<kFmt> || !ok)) {
          if (group_any(hq, !ok)) {   // a wait that gave up ends the quarter's warps together
            ok = false;
            break;
          }
          ok = rebase<kFmt, kHU>(S, z, nM, lrow, scv, ebf, lk, T0, jj > 0 ? k - 1 : -1);
          if (!ok) {
            *abort = 1;
            continue;   // the next vote ends the quarter's warps
          }
          rk = ex2(-lk);
#pragma unroll
          for (int i = 0; i < kHP; ++i) d[i] = z[i];
        }
        // the last tile's PV reads the weights (of the piece before: its epilogue waited)
        if (jj > 0) {
          ok = warp_wait(&S.pv_done, (k - 1) & 1, abort);
          if (!ok) {
            *abort = 1;
            continue;   // the next vote ends the quarter's warps
          }
        }
        // p: the weights times this key's largest scale
#pragma unroll
        for (int i = 0; i < kHP; ++i) {
          d[i] = make_float2(ex2(d[i].x), ex2(d[i].y));
          lrow[i] = __ffma2_rn(d[i], make_float2(rk, rk), lrow[i]);
        }
        // weights: keys by [high | low] terms of each head quarter
        if constexpr (F::kBf) {
          const uint32_t pb = ptx::smem_u32(S.pb[0]) + (row >> 3) * kGroupBf<kHU> + (row & 7) * 16 + hq * (kHT / 4) * 128;
          uint32_t hi[kHT / 2], lo[kHT / 2];
#pragma unroll
          for (int i = 0; i < kHT / 2; ++i) {
            const __nv_bfloat162 hv = __floats2bfloat162_rn(d[i].x, d[i].y);
            const float2 hf = __bfloat1622float2(hv);
            const __nv_bfloat162 lv = __floats2bfloat162_rn(d[i].x - hf.x, d[i].y - hf.y);
            hi[i] = *reinterpret_cast<const uint32_t*>(&hv);
            lo[i] = *reinterpret_cast<const uint32_t*>(&lv);
          }
          if constexpr (kHT == 4) {
            st_v4(pb, hi[0], hi[1], lo[0], lo[1]);
          } else {
            st_v4(pb, hi[0], hi[1], hi[2], hi[3]);
            st_v4(pb + 128, lo[0], lo[1], lo[2], lo[3]);
          }
        } else {
          __half2 p2[kHP];
#pragma unroll
          for (int i = 0; i < kHP; ++i) p2[i] = __floats2half2_rn(d[i].x, d[i].y);
          const uint32_t off = (row >> 3) * (kHU * 16) + (row & 7) * 16 + ((2 * kHT * hq) >> 4) * 128 + ((2 * kHT * hq) & 15);
#pragma unroll
          for (int b = 0; b < F::kSets; ++b) {
            const uint32_t pb = off + S.set_addr(b, buf);
            const __half2 sc2 = __float2half2_rn(F::kDs ? scv[b] * ebf[b] * rk : 1.f);   // at most 1
            uint32_t hi[kHT / 4], lo[kHT / 4];
#pragma unroll
            for (int i = 0; i < kHT / 4; ++i) {
              uint32_t h01, l01, h23, l23;
              split2_e4m3x2(F::kDs ? __hmul2_rn(p2[2 * i], sc2) : p2[2 * i], dither, h01, l01);
              split2_e4m3x2(F::kDs ? __hmul2_rn(p2[2 * i + 1], sc2) : p2[2 * i + 1], dither, h23, l23);
              hi[i] = h01 | (h23 << 16);
              lo[i] = l01 | (l23 << 16);
            }
            if constexpr (kHT == 4) st_v2(pb, hi[0], lo[0]);
            else st_v4(pb, hi[0], hi[1], lo[0], lo[1]);
          }
        }
        // A masked row may hold anything, and 0 x NaN is NaN in the product:
        // it is zeroed (QK^T, done with this tile, only ever spoiled that
        // row's own logits).
        if (partial && !valid) {
#pragma unroll
          for (int b = hq; b < F::kBlocks; b += 4) {
            const uint32_t a = ptx::smem_u32(S.lat[buf][b]) + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) st_v4(a + 16 * c, 0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.p_full);
      }
      // the next piece's query, before this one's epilogue: its first QK^T is
      // issued ahead of the PV that the epilogue waits for
      {
        Walk peek = w;
        Seg nx;
        while (ok && walk_next(P, ts, peek, slot, kHU, nx)) {
          if (nx.ne > 0) {
            stage(nx);
            staged = true;
            break;
          }
        }
      }
      // ---- epilogue ----
      ok = ok && warp_wait(&S.pv_done, (k - 1) & 1, abort);
      if (!ok) *abort = 1;
      ok = softmax_all(ok);
      if (!ok) break;
      ptx::tc_fence_after();
      // Row sums over the keys: halving the heads with each exchange, a lane is
      // left with head lane / (32 / kHT); then a lane a head, see rebase.
      float v[kHT];
#pragma unroll
      for (int i = 0; i < kHP; ++i) {
        v[2 * i] = lrow[i].x;
        v[2 * i + 1] = lrow[i].y;
      }
#pragma unroll
      for (int n = kHT / 2, o = 16; o > 0; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < (n > 0 ? n : 1); ++i) {
          const float mine = n > 0 && up ? v[i + n] : v[i], other = n > 0 && !up ? v[i + n] : v[i];
          v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
        }
      }
      if (lane % (32 / kHT) == 0) S.xsum[hq][q4][lane / (32 / kHT)] = v[0];
      group_sync(hq);
      {
        const int h = lane % kHT;
        const float l = S.xsum[hq][0][h] + S.xsum[hq][1][h] + S.xsum[hq][2][h] + S.xsum[hq][3][h];
        if (lane < kHT) {
          S.fac[warp][h] = l > 0.f ? (F::kPlain ? P.latent_scale : 1.f) / l : l == 0.f ? 0.f : l;   // NaN stays
          if (q4 == 0) {
            const float lse = l == 0.f ? -INFINITY : (log2f(l) - S.nm[warp][h]) * kLn2;
            if (s.whole) P.lse[orow + kHT * hq + h] = lse;
            else P.ws.part_lse[s.part + kHT * hq + h] = lse;
          }
        }
        __syncwarp();
      }
      float osc[kHT];
#pragma unroll
      for (int h = 0; h < kHT; ++h) osc[h] = S.fac[warp][h];
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {   // (not unrolled: its code is run once a piece, and fetched for it)
        uint32_t ov[2 * kHT];
        tmem_ldn(T0 + kColO + 2 * kHU * b + 2 * kHT * hq + lane_off, ov);
        ptx::tmem_wait_ld(ov);
        const int dim = 128 * b + row;
        const float back = 1.f / (b == 0 ? ebf[0] : b == 1 ? ebf[1] : b == 2 ? ebf[2] : ebf[3]);   // a power of two
#pragma unroll
        for (int h = 0; h < kHT; ++h) {
          const float o = fmaf(__uint_as_float(ov[kHT + h]), F::kBf ? 1.f : 1.f / kLoScale, __uint_as_float(ov[h])) * osc[h] * back;
          if (s.whole) {
            const __nv_bfloat16 r = __float2bfloat16_rn(o);
            P.out[(orow + kHT * hq + h) * SML_LATENT_DIM + dim] = *reinterpret_cast<const uint16_t*>(&r);
          } else {
            P.ws.part_out[(s.part + kHT * hq + h) * SML_LATENT_DIM + dim] = o;
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.o_free);
    }
    if (!ok) *abort = 1;
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && S.abort) raise_fault(P.status, SML_FAULT_TIMEOUT);
  if (warp == kWarpQk) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(S.tmem_base, 512);
  }
}

// out = sum_i exp(lse_i - lse) O_i, lse = ln sum_i exp(lse_i) over the pieces
// of one token that several CTAs hold.  The CTAs that continue a token share its
// output, join_blocks(heads) blocks each: a head's 512 dims are cut into chunks
// of 256 / G columns of four dims, and G groups of threads add up every G-th
// piece, four loads in flight each, issued before the weights are known.  (With a
// block a head and CTA, at most eight of them at work, 128 heads in nine pieces
// took 8 us more; with chunks of four columns 148 pieces 10 us more.)
constexpr int kJoinThreads = 256, kMaxPieces = 1024;
constexpr int join_blocks(int heads) { return heads / 4; }

__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(int H, int heads, PagedWs ws, uint16_t* __restrict__ out, float* __restrict__ lse) {
  __shared__ float part[kMaxPieces];
  __shared__ float4 sums[kJoinThreads];
  const int c = blockIdx.x, g = c / ws.cpg, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int4 rec = __ldcg(ws.join + c);
  if (rec.x < 0) return;
  const int n = rec.z - rec.y + 1, idx = rec.w - rec.y - 1;   // pieces, and this CTA's place among the joiners
  int G = 1;   // (then a chunk is two heads, one a warp: each warp has its own part of `part`)
  while (4 * G < n && G < 16) G *= 2;
  const int cols = kJoinThreads / G, chunks = heads * (SML_LATENT_DIM / 4) / cols, grp = tid / cols;
  float* const lw = part + (G == 1 ? 4 * (tid >> 5) : 0);
  for (int k = idx * gridDim.y + blockIdx.y; k < chunks; k += (n - 1) * gridDim.y) {
    const int f = k * cols + tid % cols, hl = f / (SML_LATENT_DIM / 4), col = f % (SML_LATENT_DIM / 4);
    auto row = [&](int i) { return (size_t)((g * ws.cpg + rec.y + i) * 2 + (i == 0)) * heads + hl; };
    float4 v[4];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * G;
        v[u] = i < n ? __ldcg(reinterpret_cast<const float4*>(ws.part_out + row(i) * SML_LATENT_DIM) + col)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load(grp);
    for (int i = G == 1 ? lane : tid; i < n; i += kJoinThreads) lw[i] = __ldcg(ws.part_lse + row(i));
    __syncthreads();
    // Maximum and denominator, each warp for itself.  NaN stays; -inf adds nothing.
    float m = -INFINITY, den = 0.f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, lw[i]);
    m = ptx::warp_max_f32(m);
    for (int i = lane; i < n; i += 32) den += lw[i] == -INFINITY ? 0.f : expf(lw[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp;;) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * G;
        const float w = i < n && lw[i] != -INFINITY ? expf(lw[i] - m) : 0.f;
        o.x = fmaf(w, v[u].x, o.x);
        o.y = fmaf(w, v[u].y, o.y);
        o.z = fmaf(w, v[u].z, o.z);
        o.w = fmaf(w, v[u].w, o.w);
      }
      i0 += 4 * G;
      if (i0 >= n) break;
      load(i0);
    }
    // the groups of a warp, then what the warps hold
    for (int x = 16; x >= cols; x /= 2) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    sums[tid] = o;
    __syncthreads();
    if (grp == 0) {
      for (int wide = max(cols, 32), i = wide; i < kJoinThreads; i += wide) {
        const float4 x = sums[i + tid];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
      const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;   // NaN stays
      const size_t orow = (size_t)rec.x * H + g * heads + hl;
      const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      reinterpret_cast<uint2*>(out + orow * SML_LATENT_DIM)[col] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      if (col == 0) lse[orow] = den == 0.f ? -INFINITY : m + logf(den);
    }
    __syncthreads();   // part and sums are read
  }
}

template <int kFmt, int kHU>
cudaError_t launch_unit(const CUtensorMap& rows, const CUtensorMap& scales, const Params& P, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<kFmt, kHU>) + 1024;
  auto kernel = paged_mla_kernel<kFmt, kHU>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(P.ws.hg * P.ws.cpg), dim3(kThreads), smem, stream, 0, rows, scales, P);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_join_kernel, dim3(P.ws.hg * P.ws.cpg, join_blocks(kHU)), dim3(kJoinThreads), 0, stream, 0, P.H, kHU, P.ws, P.out,
                    P.lse);
}

template <int kFmt>
cudaError_t launch_format(const CUtensorMap& rows, const CUtensorMap& scales, const Params& P, cudaStream_t stream) {
  return P.H == 16 ? launch_unit<kFmt, 16>(rows, scales, P, stream) : launch_unit<kFmt, 32>(rows, scales, P, stream);
}

}  // namespace

int paged_heads(const sml_problem& p) { return p.num_heads == 16 ? 16 : 32; }

PagedWs paged_plan(const sml_problem& p) {
  PagedWs w = {};
  w.hg = p.num_heads / paged_heads(p);
  const int cpg = device_sm_count() / w.hg;
  w.cpg = cpg < 1 ? 1 : cpg > kMaxPieces ? kMaxPieces : cpg;   // a token has at most cpg pieces
  return w;
}

cudaError_t launch_paged_mla(const sml_problem& p, const uint16_t* q, const sml_cache& latent, const PagedSel& sel,
                             uint16_t* out, float* lse, const PagedWs& ws, int32_t* status, cudaStream_t stream) {
  Params P;
  P.B = p.num_requests;
  P.T = p.num_tokens;
  P.H = p.num_heads;
  P.rope_dim = p.rope_dim;
  P.max_ctx = p.max_ctx;
  P.max_pages = p.max_pages;
  P.ssmax = p.ssmax;
  P.sm_scale = p.sm_scale;
  P.ssmax_s = p.ssmax_s;
  P.cu_q = p.cu_q;
  P.ctx_len = p.ctx_len;
  P.block_table = p.block_table;
  P.vis_len = p.vis_len;
  P.ssmax_len = p.ssmax_len;
  P.q = q;
  P.latent = static_cast<const uint8_t*>(latent.base);
  P.latent_pages = latent.num_pages;
  P.latent_scale = latent.format == SML_LATENT_E4M3 ? latent.scale : 1.f;
  P.sel = sel;
  P.out = out;
  P.lse = lse;
  P.ws = ws;
  P.status = status;
  // The pool as rows of bytes: one box is a 128-B column of a page's 64 rows
  // (a row's last box may reach past its end: zeros), or its 64 x 4 block scales.
  const auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t row = latent.format == SML_LATENT_BF16   ? SML_LATENT_BF16_ROW_BYTES
                         : latent.format == SML_LATENT_E4M3 ? SML_LATENT_E4M3_ROW_BYTES
                                                            : SML_LATENT_ROW_BYTES;
  const cuuint64_t dims[2] = {row, (cuuint64_t)latent.num_pages * SML_PAGE_TOKENS}, strides[1] = {row};
  const cuuint32_t box[2] = {128, SML_PAGE_TOKENS}, sbox[2] = {16, SML_PAGE_TOKENS}, one[2] = {1, 1};
  CUtensorMap rows, scales;
  if (enc(&rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(latent.base), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(latent.base), dims, strides, sbox, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (latent.format == SML_LATENT_BF16) return launch_format<kFmtBf16>(rows, scales, P, stream);
  if (latent.format == SML_LATENT_E4M3) return launch_format<kFmtPlain>(rows, scales, P, stream);
  return launch_format<kFmtDsMla>(rows, scales, P, stream);
}

}  // namespace sml
