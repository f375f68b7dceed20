// Selection of whole 64-token pages: one key per page (the mean of its indexer
// keys), the indexer's score of it for every query token, and the best pages
// of each token.
//
// vLLM blog "vLLM 首日支持 Mistral Large 4", section "实现细节 / 模型架构": the
// sparse indexer reads an FP8 cache with one scale per key.  The block keys are
// held the same way (E4M3 codes and one fp32 scale), 132 B per page in place of
// the 8,448 B of the page's own keys.
#include <cuda_fp8.h>
#include <math.h>

#include "ptx.cuh"
#include "sml_internal.cuh"

namespace sml {
namespace {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float2 e4m3x2_f(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ---- block keys ---------------------------------------------------------------
// One CTA per page.  Warp w sums keys 8 w .. 8 w + 7, lane l dims 4 l .. 4 l + 3,
// in 64 bits: a code times its scale is exact there (28 bits), and so is the sum
// of 64 such products while their scales lie within 2^5 of each other, so that
// the stored bytes do not depend on the order of the summation.  8.4 KB a page:
// 512 pages take 3.7 us, launch included.
constexpr int kKeyWarps = 8;

__global__ void __launch_bounds__(32 * kKeyWarps)
block_keys_kernel(const uint8_t* __restrict__ index, long long num_pages, const int32_t* __restrict__ pages, int n,
                  uint8_t* __restrict__ block, int32_t* status) {
  __shared__ double sum[kKeyWarps][SML_INDEX_DIM];
  __shared__ float red[SML_INDEX_DIM / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::griddep_wait();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int pg = __ldg(pages + i);
    if (pg < 0 || pg >= num_pages) {
      if (pg != -1 && threadIdx.x == 0) raise_fault(status, SML_FAULT_PAGE);
      continue;
    }
    const uint8_t* src = index + (size_t)pg * SML_INDEX_PAGE_BYTES;
    constexpr int kPer = SML_PAGE_TOKENS / kKeyWarps;
    uint32_t code[kPer];
    float sc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int row = warp * kPer + k;
      code[k] = __ldcg(reinterpret_cast<const uint32_t*>(src + row * SML_INDEX_DIM) + lane);
      sc[k] = __ldcg(reinterpret_cast<const float*>(src + SML_PAGE_TOKENS * SML_INDEX_DIM) + row);
    }
    double a[4] = {0., 0., 0., 0.};
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float2 x = e4m3x2_f(code[k]), y = e4m3x2_f(code[k] >> 16);
      a[0] += (double)x.x * sc[k];
      a[1] += (double)x.y * sc[k];
      a[2] += (double)y.x * sc[k];
      a[3] += (double)y.y * sc[k];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[warp][4 * lane + j] = a[j];
    __syncthreads();
    float mean = 0.f;
    if (threadIdx.x < SML_INDEX_DIM) {
      double s = 0.;
#pragma unroll
      for (int w = 0; w < kKeyWarps; ++w) s += sum[w][threadIdx.x];
      mean = (float)(s / SML_PAGE_TOKENS);
      float m = fabsf(mean);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) red[warp] = m;
    }
    __syncthreads();
    if (threadIdx.x < SML_INDEX_DIM) {
      const float amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
      const float s = amax > 0.f ? __fdiv_rn(amax, kE4m3Max) : 1.f;
      uint8_t* dst = block + (size_t)(pg / SML_PAGE_TOKENS) * SML_INDEX_PAGE_BYTES;
      const int row = pg % SML_PAGE_TOKENS;
      dst[row * SML_INDEX_DIM + threadIdx.x] = __nv_cvt_float_to_fp8(__fdiv_rn(mean, s), __NV_SATFINITE, __NV_E4M3);
      if (threadIdx.x == 0) reinterpret_cast<float*>(dst + SML_PAGE_TOKENS * SML_INDEX_DIM)[row] = s;
    }
  }
}

// ---- what the scores and the selection share ------------------------------------
struct Batch {
  int B, T, max_ctx, max_pages, ssmax;
  float s_index;
  const int32_t* cu_q;
  const int32_t* ctx_len;
  const int32_t* block_table;
  const int32_t* vis_len;
  const int32_t* ssmax_len;
  int32_t* status;
};

Batch batch_of(const sml_problem& p, int32_t* status) {
  return Batch{p.num_requests, p.num_tokens, p.max_ctx,  p.max_pages, p.ssmax,     p.ssmax_s_index,
               p.cu_q,         p.ctx_len,    p.block_table, p.vis_len, p.ssmax_len, status};
}

// Request and visible length (0 when the lengths are bad) of token t: with
// equal query counts its request is t B / T, else a binary search finds it.
__device__ __forceinline__ int visible_of(const Batch& b, int t, int* r, bool* bad) {
  *r = (int)((unsigned)((long long)t * b.B) / (unsigned)b.T);
  Req rq = load_request(b.cu_q, b.ctx_len, *r, b.T, b.max_ctx, b.max_pages, b.vis_len != nullptr);
  if (!(rq.q0 <= t && t - rq.q0 < rq.Q)) {
    *r = request_of(b.cu_q, b.B, t);
    rq = load_request(b.cu_q, b.ctx_len, *r, b.T, b.max_ctx, b.max_pages, b.vis_len != nullptr);
  }
  *bad = !(rq.ok && t >= rq.q0 && t - rq.q0 < rq.Q);
  if (*bad) return 0;
  const int n = visible_len(b.vis_len, rq, t, bad);
  return *bad ? 0 : n;
}

// ---- block scores ---------------------------------------------------------------
// A CTA scores one tile of 128 blocks for up to kChunk consecutive tokens: the
// blocks' keys are gathered once per request into shared memory (K-major rows
// of 128 B, 128-B swizzle), then for each token the 64 x 128 query comes by
// TMA and one D[128 blocks, 64 heads] = K Q^T runs on kind::f8f6f4 (exact E4M3
// products, fp32 sums in TMEM).  Warps 0-3 gather the keys and reduce D over
// the heads (thread = block); warp 4 loads queries up to four ahead and issues the
// MMAs, so the product of the next token overlaps the reduction of the last.
// 2,048 queries of 511 blocks take 24.8 us for 21 MB (3.3 us) and products that
// the tensor cores would do in 6 at this shape: 8 us before the first product and
// after the last, then 0.3 us a token and tile on each SM.  Shared memory's pipe
// is what that takes: the weights (16 loads of 16 B a warp), the products'
// operands and TMA's queries, about 510 of 560 cycles; without the reduction's
// arithmetic and weights it is 19 us in all.  Two tiles of blocks to each weight
// read: 22.3 us here, but 13.4 instead of 11.9 for 512 queries.
constexpr int kTileBlocks = 128, kChunk = 64, kEpiThreads = 128, kScoreThreads = kEpiThreads + 32;
constexpr int kQBufs = 4;
constexpr int kQueryBytes = SML_INDEX_HEADS * SML_INDEX_DIM;

struct __align__(1024) ScoreSmem {
  uint8_t key[kTileBlocks * SML_INDEX_DIM];
  uint8_t q[kQBufs][kQueryBytes];
  __align__(16) float w[kQBufs][SML_INDEX_HEADS];
  int nb[kChunk], req[kChunk];   // of the CTA's tokens: candidate blocks, request
  float fac[kChunk];             // and query scale times SSMax factor
  uint64_t q_full[kQBufs], acc_full[2], acc_free[2], key_full, drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort));
}
// AND of a flag over the epilogue warps (named barrier 1).
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(kEpiThreads)
      : "memory");
  return r != 0;
}

// ReLU that keeps a NaN, so that a page with a NaN key ranks last.
__device__ __forceinline__ float relu(uint32_t x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(__uint_as_float(x)));
  return y;
}

__global__ void __launch_bounds__(kScoreThreads, 4)
block_scores_kernel(const __grid_constant__ CUtensorMap qmap, Batch b, int chunk, const float* __restrict__ iq_scale,
                    const float* __restrict__ iw, const uint8_t* __restrict__ block, long long rows,
                    float* __restrict__ scores) {
  extern __shared__ uint8_t raw[];
  ScoreSmem& S = *reinterpret_cast<ScoreSmem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.y * chunk, nt = min(chunk, b.T - t0), j0 = blockIdx.x * kTileBlocks;
  if (tid == 0) {
    for (int i = 0; i < kQBufs; ++i) ptx::mbar_init(&S.q_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&S.acc_full[i], 2);   // the products' commit, and warp 4's own arrival
      ptx::mbar_init(&S.acc_free[i], 4);
    }
    ptx::mbar_init(&S.key_full, 4);
    ptx::mbar_init(&S.drain, 1);
    S.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 4) {
    ptx::tmem_alloc(&S.tmem_base, 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::griddep_wait();
  // this CTA holds its tensor memory: a dependent grid cannot starve it
  if (tid == 0) ptx::griddep_launch_dependents();
  bool any = false;
  if (tid < nt) {
    int r;
    bool bad;
    const float sq = __ldg(iq_scale + t0 + tid);
    const int ssl = b.ssmax_len ? __ldg(b.ssmax_len + t0 + tid) : 0;
    const int n = visible_of(b, t0 + tid, &r, &bad), nb = n > 0 ? (n - 1) / SML_PAGE_TOKENS : 0;
    if (bad && blockIdx.x == 0) raise_fault(b.status, SML_FAULT_LENGTHS);
    S.nb[tid] = nb;
    S.req[tid] = r;
    S.fac[tid] = sq * (b.ssmax ? b.s_index * logf((float)max(1, b.ssmax_len ? ssl : n)) : 1.f);
    any = nb > j0;
  }
  const bool work = __syncthreads_or(any);   // some token of the CTA has candidates in this tile
  volatile int* abort = &S.abort;
  const uint32_t T0 = S.tmem_base;
  if (work && warp == 4) {
    // ---- queries and products; tokens k = 0, 1, ... of those with candidates here ----
    constexpr uint32_t id = ptx::idesc_f16(SML_INDEX_HEADS, 0, 0, 0);
    const uint32_t key0 = ptx::smem_u32(S.key), q0 = ptx::smem_u32(S.q[0]);
    auto next = [&](int i) {
      while (i < nt && S.nb[i] <= j0) ++i;
      return i;
    };
    int at = next(0), loaded = 0;   // the next token to load, and loads so far
    auto load = [&]() {
      if (at >= nt) return;
      if (lane == 0) {
        const int buf = loaded % kQBufs;
        ptx::mbar_arrive_expect_tx(&S.q_full[buf], kQueryBytes + SML_INDEX_HEADS * 4);
        ptx::tma_load_2d(S.q[buf], &qmap, &S.q_full[buf], 0, (t0 + at) * SML_INDEX_HEADS);
        ptx::bulk_load(S.w[buf], iw + (size_t)(t0 + at) * SML_INDEX_HEADS, SML_INDEX_HEADS * 4, &S.q_full[buf]);
      }
      __syncwarp();
      ++loaded;
      at = next(at + 1);
    };
#pragma unroll 1
    for (int i = 0; i < kQBufs; ++i) load();
    bool ok = true;
    int k = 0, runs = 0, last = -1;
    for (int i = next(0); i < nt && ok; i = next(i + 1), ++k) {
      if (S.req[i] != last) {
        ok = warp_wait(&S.key_full, runs & 1, abort);
        last = S.req[i];
        ++runs;
      }
      if (ok && k >= 2) {
        // token k - 2 is reduced: its D is free, and its query and weights make
        // room for token k + 2
        ok = warp_wait(&S.acc_free[k & 1], ((k >> 1) - 1) & 1, abort);
        if (ok && loaded == k + 2) load();
      }
      ok = ok && warp_wait(&S.q_full[k % kQBufs], (k / kQBufs) & 1, abort);
      if (!ok) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < SML_INDEX_DIM / 32; ++kk)
          ptx::mma_f8(T0 + (k & 1) * SML_INDEX_HEADS, ptx::sdesc_sw128(key0 + 32 * kk),
                      ptx::sdesc_sw128(q0 + (k % kQBufs) * kQueryBytes + 32 * kk), id, kk > 0);
        ptx::mma_commit(&S.acc_full[k & 1]);
        // This warp has waited for the query and its weights: its arrival passes
        // them on (a wait of every reducing warp for them costs 1.3 us at 2,048
        // queries).
        ptx::mbar_arrive(&S.acc_full[k & 1]);
      }
      __syncwarp();
    }
    if (!ok) *abort = 1;
    for (int i = max(0, loaded - kQBufs); i < loaded; ++i)
      ptx::mbar_wait(&S.q_full[i % kQBufs], (i / kQBufs) & 1, nullptr, 100000u);
    if (ptx::elect_one()) ptx::mma_commit(&S.drain);
    __syncwarp();
    ptx::mbar_wait(&S.drain, 0, nullptr, 100000u);
    __syncwarp();
  } else if (work) {
    // ---- keys, then the reduction over the heads ----
    const int j = j0 + tid;
    const uint32_t key0 = ptx::smem_u32(S.key);
    bool ok = true, there = false;
    float sb = 0.f;
    int k = 0, last = -1;
    // (A wait that gives up still goes on to the next request's barrier, or the end.)
    for (int i = 0; i < nt; ++i) {
      if (S.nb[i] <= j0) continue;
      if (S.req[i] != last) {
        // Every product with the last request's keys is done: each was waited
        // for below.  Blocks past the request's last candidate hold zeros.
        last = S.req[i];
        int most = S.nb[i];
        for (int x = i + 1; x < nt && S.req[x] == last; ++x) most = max(most, S.nb[x]);
        const int pg = j < most ? __ldg(b.block_table + (size_t)last * b.max_pages + j) : -1;
        there = pg >= 0 && pg < rows;
        if (j < most && !there) raise_fault(b.status, SML_FAULT_PAGE);
        auto page_of = [&](int pg) { return block + (size_t)(pg / SML_PAGE_TOKENS) * SML_INDEX_PAGE_BYTES; };
        const int own = there ? pg : 0;
        sb = __ldcg(reinterpret_cast<const float*>(page_of(own) + SML_PAGE_TOKENS * SML_INDEX_DIM) + own % SML_PAGE_TOKENS);
        // eight lanes a key, so that a load touches four lines (a thread a key: 32,
        // and 4 us more before the first product)
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int pk = __shfl_sync(0xffffffffu, there ? pg : -1, 4 * c + (lane >> 3));
          v[c] = pk >= 0 ? __ldcg(reinterpret_cast<const uint4*>(page_of(pk) + pk % SML_PAGE_TOKENS * SML_INDEX_DIM) + (lane & 7))
                         : make_uint4(0, 0, 0, 0);
        }
        ok = epi_all(ok);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int row = 32 * warp + 4 * c + (lane >> 3);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(key0 + row * 128 + (((lane & 7) ^ (row & 7)) << 4)),
                       "r"(v[c].x), "r"(v[c].y), "r"(v[c].z), "r"(v[c].w)
                       : "memory");
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.key_full);
      }
      const int acc = k & 1;
      ok = ok && warp_wait(&S.acc_full[acc], (k >> 1) & 1, abort);
      if (!ok) {
        *abort = 1;
        continue;
      }
      ptx::tc_fence_after();
      const uint32_t d = T0 + ((uint32_t)(32 * warp) << 16) + acc * SML_INDEX_HEADS;
      uint32_t v0[32], v1[32];
      ptx::tmem_ld32(d, v0);
      ptx::tmem_ld32(d + 32, v1);
      ptx::tmem_wait_ld(v0, v1);
      const float4* w = reinterpret_cast<const float4*>(S.w[k % kQBufs]);
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 wa = w[c], wb = w[8 + c];
        s[0] = fmaf(wa.x, relu(v0[4 * c]), s[0]);
        s[1] = fmaf(wa.y, relu(v0[4 * c + 1]), s[1]);
        s[2] = fmaf(wa.z, relu(v0[4 * c + 2]), s[2]);
        s[3] = fmaf(wa.w, relu(v0[4 * c + 3]), s[3]);
        s[0] = fmaf(wb.x, relu(v1[4 * c]), s[0]);
        s[1] = fmaf(wb.y, relu(v1[4 * c + 1]), s[1]);
        s[2] = fmaf(wb.z, relu(v1[4 * c + 2]), s[2]);
        s[3] = fmaf(wb.w, relu(v1[4 * c + 3]), s[3]);
      }
      const float sum = (s[0] + s[1]) + (s[2] + s[3]);
      // D and the weights have been read: the arrival lets the next product and
      // TMA overwrite them.  Loads of the weights that are only issued may still
      // be on their way; the proxy fence puts them before TMA's writes.  The
      // score is stored after it: the fence would wait for that too.
      ptx::fence_proxy_async();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.acc_free[acc]);
      if (j < S.nb[i]) scores[(size_t)(t0 + i) * b.max_pages + j] = there ? sum * S.fac[i] * sb : NAN;
      ++k;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && S.abort) raise_fault(b.status, SML_FAULT_TIMEOUT);
  if (warp == 4) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(S.tmem_base, 128);
  }
}

// ---- block selection --------------------------------------------------------------
// Order-preserving key: larger score, larger key; -0.0 as +0.0; NaN lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// One CTA per token; warp w owns the row's entries [32 c w, 32 c (w + 1)), c
// steps of one entry a lane, so that loads are coalesced and a ballot a step
// gives every kept entry its place in ascending order.
//
// The threshold is the k-th largest key.  A bound below it first: of A warps'
// entries each warp's j-th largest thread maximum, j = ceil(k / A), has at least
// j A >= k keys at or above the smallest of those.  A histogram of 512 equal
// steps from there to the largest key leaves a few keys in the threshold's step,
// and up to three more split that step again; one whose step holds exactly the
// keys still wanted is the last.  (Histograms of the keys' own 8-bit digits, all
// keys in the first one and every warp scanning each, took 14.9 us for four rows
// of 16,375 entries and 5.5 us for 32 of 512 to 1,024, where this takes 8.3 and
// 4.1 to 4.4.)  What is left is a chain: lengths, loads, the bound, one or two
// histograms, the places, 0.3 to 0.8 us each.
// kReg > 0: rows of up to kReg entries a thread, read once into registers (1 where
// that holds a row: 43.6 us for 2,048 rows of 1,000, 45.8 with 16); 0: rows of
// any length, read from L1/L2 in every pass (40,000 entries: 36 us).
constexpr int kTopThreads = 1024, kTopWarps = kTopThreads / 32, kBins = 512, kMaxJ = 8;

template <int kReg>
__global__ void __launch_bounds__(kTopThreads)
block_topk_kernel(Batch b, const float* __restrict__ scores, int k, int32_t* __restrict__ blocks,
                  int32_t* __restrict__ blocks_len) {
  static_assert(kReg < 32, "a bit a step");
  __shared__ __align__(16) int hist[4][kBins];   // one per round, so that no round waits to clear another's
  __shared__ uint2 top[kTopWarps];
  __shared__ int2 part[kTopWarps];
  __shared__ int4 found;
  ptx::griddep_wait();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int r;
  bool bad;
  const int n = visible_of(b, t, &r, &bad), nb = n > 0 ? (n - 1) / SML_PAGE_TOKENS : 0;
  if (bad && tid == 0) raise_fault(b.status, SML_FAULT_LENGTHS);
  const float* row = scores + (size_t)t * b.max_pages;
  int32_t* dst = blocks + (size_t)t * k;
  const int take = min(k - 1, nb);
  const int len = n > 0 ? take + 1 : 0;
  for (int i = len + tid; i < k; i += kTopThreads) dst[i] = -1;
  if (tid == 0) {
    blocks_len[t] = len;
    if (n > 0) dst[take] = nb;
  }
  if (take == nb) {
    for (int i = tid; i < nb; i += kTopThreads) dst[i] = i;
    return;
  }
  if (take == 0) return;
  const int c = (nb + kTopThreads - 1) / kTopThreads, i0 = warp * c * 32 + lane;
  const int steps = i0 < nb ? min(c, (nb - i0 + 31) / 32) : 0;   // of this lane
  uint32_t reg[kReg > 0 ? kReg : 1];
  if constexpr (kReg > 0) {
#pragma unroll
    for (int u = 0; u < kReg; ++u) reg[u] = u < steps ? __float_as_uint(__ldg(row + i0 + 32 * u)) : 0u;   // all in flight
#pragma unroll
    for (int u = 0; u < kReg; ++u) {
      if (u >= c) break;
      reg[u] = u < steps ? order_key(__uint_as_float(reg[u])) : 0u;
    }
  }
  // f(step, key, whether there is one) for every step, by whole warps
  auto each = [&](auto&& f) {
    if constexpr (kReg > 0) {
#pragma unroll
      for (int u = 0; u < kReg; ++u) {
        if (u >= c) break;
        f(u, reg[u], u < steps);
      }
    } else {
      for (int u = 0; u < c; ++u) f(u, u < steps ? order_key(__ldg(row + i0 + 32 * u)) : 0u, u < steps);
    }
  };
  for (int i = tid; i < 4 * kBins; i += kTopThreads) (&hist[0][0])[i] = 0;
  uint32_t low = 0, base;
  {
    uint32_t mx = 0;   // (an entry that is not there, 0, is below any other and at least a NaN)
    each([&](int, uint32_t key, bool) { mx = max(mx, key); });
    const int full = nb / (32 * c);   // warps whose entries are all there
    const int j = full > 0 ? (take + full - 1) / full : kMaxJ + 1;
    uint32_t first = __reduce_max_sync(0xffffffffu, mx), at = j <= kMaxJ ? first : 0u;
    for (int i = 1; i < j && j <= kMaxJ; ++i) {   // (one of equal maxima at a time)
      const unsigned eq = __ballot_sync(0xffffffffu, mx == at);
      if (lane == __ffs(eq) - 1) mx = 0;
      at = __reduce_max_sync(0xffffffffu, mx);
    }
    if (lane == 0) top[warp] = make_uint2(first, warp < full || j > kMaxJ ? at : 0xffffffffu);
    __syncthreads();
    const uint2 x = top[lane];
    low = __reduce_min_sync(0xffffffffu, x.y);
    base = __reduce_max_sync(0xffffffffu, x.x) - low;
  }
  int shift = max(0, 32 - __clz(base) - 9);   // base, so far: the largest key less low
  uint32_t width = 0xffffffffu;               // of the step that holds the threshold, less one
  base = 0;
  int need = take;   // keys still wanted among those in [low + base, low + base + width]
  bool all = false;
#pragma unroll 1
  for (int round = 0;; ++round) {
    int* h = hist[round];
    each([&](int, uint32_t key, bool there) {
      const uint32_t x = key - low - base;
      if (there && key >= low && x <= width) atomicAdd(&h[x >> shift], 1);
    });
    __syncthreads();
    if (warp == 0) {   // lane l: steps 16 l .. 16 l + 15; above = keys in larger steps
      constexpr int kPer = kBins / 32;
      int cnt[kPer], sum = 0;
#pragma unroll
      for (int u = 0; u < kPer; u += 4) {
        const int4 x = *reinterpret_cast<const int4*>(&h[kPer * lane + u]);
        cnt[u] = x.x;
        cnt[u + 1] = x.y;
        cnt[u + 2] = x.z;
        cnt[u + 3] = x.w;
        sum += x.x + x.y + x.z + x.w;
      }
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += y;
      }
      above -= sum;
      if (above < need && above + sum >= need) {
        int step = -1, left = 0, have = 0;
#pragma unroll
        for (int u = kPer - 1; u >= 0; --u) {
          if (step < 0 && above + cnt[u] >= need) {
            step = kPer * lane + u;
            left = need - above;
            have = cnt[u];
          }
          above += cnt[u];
        }
        found = make_int4(step, left, have, 0);
      }
    }
    __syncthreads();
    const int4 got = found;
    base += (uint32_t)got.x << shift;
    width = (1u << shift) - 1;
    need = got.y;
    all = got.z == need;   // every key of this step: the threshold is its smallest key
    if (all || shift == 0) break;
    shift = max(0, shift - 9);
  }
  // keep every key above the threshold and the first `need` equal to it (all:
  // every key at or above it)
  const uint32_t thr = low + base;
  const uint32_t surely = all ? thr : thr + 1;   // (no key is 2^32 - 1)
  int2 mine = make_int2(0, 0);           // this warp's: kept for sure, equal to the threshold
  uint32_t sure_steps = 0, tie_steps = 0;   // kReg: this lane's steps of either kind
  each([&](int u, uint32_t key, bool there) {
    if constexpr (kReg > 0) {
      if (key >= thr) tie_steps |= 1u << u;
      if (key >= surely) sure_steps |= 1u << u;
    } else {
      mine.x += there && key >= surely;
      mine.y += there && key >= thr && key < surely;
    }
  });
  if constexpr (kReg > 0) {
    const uint32_t there = (1u << steps) - 1;
    sure_steps &= there;
    tie_steps &= there & ~sure_steps;
    mine = make_int2(__popc(sure_steps), __popc(tie_steps));
  }
  mine.x = __reduce_add_sync(0xffffffffu, mine.x);
  mine.y = __reduce_add_sync(0xffffffffu, mine.y);
  if (lane == 0) part[warp] = mine;
  __syncthreads();
  if (mine.x + mine.y == 0) return;   // (no barrier follows)
  const int2 p = lane < warp ? part[lane] : make_int2(0, 0);
  int kept = __reduce_add_sync(0xffffffffu, p.x), ties = __reduce_add_sync(0xffffffffu, p.y);
  const unsigned below = (1u << lane) - 1;
  auto place = [&](int u, bool is_sure, bool is_tie) {   // kept, ties: before this step's entries
    const unsigned sure = __ballot_sync(0xffffffffu, is_sure), tie = __ballot_sync(0xffffffffu, is_tie);
    const int t0 = ties + __popc(tie & below);
    if (is_sure || (is_tie && t0 < need)) dst[kept + __popc(sure & below) + (all ? 0 : min(t0, need))] = i0 + 32 * u;
    kept += __popc(sure);
    ties += __popc(tie);
  };
  if constexpr (kReg > 0) {
    for (unsigned left = __reduce_or_sync(0xffffffffu, sure_steps | tie_steps); left; left &= left - 1) {
      const int u = __ffs(left) - 1;
      place(u, sure_steps >> u & 1, tie_steps >> u & 1);
    }
  } else {
    each([&](int u, uint32_t key, bool there) { place(u, there && key >= surely, there && key >= thr && key < surely); });
  }
}

}  // namespace

cudaError_t launch_block_keys(const sml_cache& index, const int32_t* pages, int n, const sml_cache& block,
                              int32_t* status, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  const int cap = device_sm_count() * 8;
  return launch_pdl(block_keys_kernel, dim3(n < cap ? n : cap), dim3(32 * kKeyWarps), 0, stream, 0,
                    static_cast<const uint8_t*>(index.base), (long long)index.num_pages, pages, n,
                    static_cast<uint8_t*>(const_cast<void*>(block.base)), status);
}

cudaError_t launch_block_scores(const sml_problem& p, const uint8_t* iq8, const float* iq_scale, const float* iw,
                                const sml_cache& block, float* scores, int32_t* status, cudaStream_t stream) {
  // Tokens per CTA: as many as leave about four CTAs for every SM, which is
  // what shared memory and TMEM hold, so that a tile's keys are read for as few
  // CTAs as fill the device.
  const int tiles = (p.max_pages + kTileBlocks - 1) / kTileBlocks;
  const long long ctas = 4ll * device_sm_count();
  long long chunk = ((long long)p.num_tokens * tiles + ctas - 1) / ctas;
  chunk = chunk < 1 ? 1 : chunk > kChunk ? kChunk : chunk;
  const int chunks = (int)((p.num_tokens + chunk - 1) / chunk);
  const auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap qmap;   // the queries as [T * 64 rows][128 B]: one box = the 64 heads of a token
  const cuuint64_t dims[2] = {SML_INDEX_DIM, (cuuint64_t)p.num_tokens * SML_INDEX_HEADS}, strides[1] = {SML_INDEX_DIM};
  const cuuint32_t box[2] = {SML_INDEX_DIM, SML_INDEX_HEADS}, one[2] = {1, 1};
  if (enc(&qmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(iq8), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(ScoreSmem) + 1024;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(block_scores_kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(block_scores_kernel, dim3(tiles, chunks), dim3(kScoreThreads), smem, stream, 0, qmap,
                    batch_of(p, status), (int)chunk, iq_scale, iw, static_cast<const uint8_t*>(block.base),
                    (long long)block.num_pages * SML_PAGE_TOKENS, scores);
}

cudaError_t launch_block_topk(const sml_problem& p, const float* scores, int k, int32_t* blocks, int32_t* blocks_len,
                              int32_t* status, cudaStream_t stream) {
  constexpr int kReg = 16;   // rows of up to 16,384 blocks (a million positions) stay in registers
  auto kernel = p.max_pages <= kTopThreads          ? block_topk_kernel<1>
                : p.max_pages <= kReg * kTopThreads ? block_topk_kernel<kReg>
                                                    : block_topk_kernel<0>;
  return launch_pdl(kernel, dim3(p.num_tokens), dim3(kTopThreads), 0, stream, 0, batch_of(p, status), scores, k, blocks,
                    blocks_len);
}

}  // namespace sml
