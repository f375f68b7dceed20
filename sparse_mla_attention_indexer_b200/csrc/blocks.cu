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
// in 64 bits: a code times its scale is exact there, and the sum of 64 such
// products is exact unless their scales lie more than 2^8 apart, so the stored
// bytes do not depend on the order of the summation.
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

// Request and visible length (0 when the lengths are bad) of token t.
__device__ __forceinline__ int visible_of(const Batch& b, int t, int* r, bool* bad) {
  const int guess = (int)((long long)t * b.B / b.T);
  *r = __ldg(b.cu_q + guess) <= t && t < __ldg(b.cu_q + guess + 1) ? guess : request_of(b.cu_q, b.B, t);
  const Req rq = load_request(b.cu_q, b.ctx_len, *r, b.T, b.max_ctx, b.max_pages, b.vis_len != nullptr);
  *bad = !(rq.ok && t >= rq.q0 && t - rq.q0 < rq.Q);
  if (*bad) return 0;
  const int n = visible_len(b.vis_len, rq, t, bad);
  return *bad ? 0 : n;
}

// ---- block scores ---------------------------------------------------------------
// One CTA per (token, 32 blocks); eight threads per block, eight heads each.
constexpr int kScoreThreads = 256, kScoreBlocks = 32;

__global__ void __launch_bounds__(kScoreThreads)
block_scores_kernel(Batch b, const uint8_t* __restrict__ iq8, const float* __restrict__ iq_scale,
                    const float* __restrict__ iw, const uint8_t* __restrict__ block, long long rows,
                    float* __restrict__ scores) {
  __shared__ __half q[SML_INDEX_HEADS][SML_INDEX_DIM + 2];
  __shared__ float key[kScoreBlocks][SML_INDEX_DIM + 1];
  ptx::griddep_wait();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  const int t = blockIdx.x, tid = threadIdx.x;
  int r;
  bool bad;
  const int n = visible_of(b, t, &r, &bad), nb = n > 0 ? (n - 1) / SML_PAGE_TOKENS : 0;
  if (bad && blockIdx.y == 0 && tid == 0) raise_fault(b.status, SML_FAULT_LENGTHS);
  if ((int)blockIdx.y * kScoreBlocks >= nb) return;
  for (int i = tid; i < SML_INDEX_HEADS * SML_INDEX_DIM / 2; i += kScoreThreads) {
    const float2 v = e4m3x2_f(reinterpret_cast<const uint16_t*>(iq8 + (size_t)t * SML_INDEX_HEADS * SML_INDEX_DIM)[i]);
    q[2 * i / SML_INDEX_DIM][2 * i % SML_INDEX_DIM] = __float2half(v.x);
    q[2 * i / SML_INDEX_DIM][2 * i % SML_INDEX_DIM + 1] = __float2half(v.y);
  }
  const float c = b.ssmax ? b.s_index * logf((float)ssmax_len_of(b.ssmax_len, t, n)) : 1.f;
  for (int j0 = blockIdx.y * kScoreBlocks; j0 < nb; j0 += gridDim.y * kScoreBlocks) {
    __syncthreads();
    const int j = j0 + tid / 8, part = tid % 8;
    const int pg = j < nb ? __ldg(b.block_table + (size_t)r * b.max_pages + j) : -1;
    const bool there = pg >= 0 && pg < rows;
    const uint8_t* src = block + (size_t)(there ? pg / SML_PAGE_TOKENS : 0) * SML_INDEX_PAGE_BYTES;
    const int row = there ? pg % SML_PAGE_TOKENS : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = e4m3x2_f(reinterpret_cast<const uint16_t*>(src + row * SML_INDEX_DIM + 16 * part)[i]);
      key[tid / 8][16 * part + 2 * i] = v.x;
      key[tid / 8][16 * part + 2 * i + 1] = v.y;
    }
    __syncthreads();
    float sum = 0.f;
    for (int h = part; h < SML_INDEX_HEADS; h += 8) {
      float dot = 0.f;
#pragma unroll 16
      for (int d = 0; d < SML_INDEX_DIM; ++d) dot = fmaf(__half2float(q[h][d]), key[tid / 8][d], dot);
      sum = fmaf(iw[(size_t)t * SML_INDEX_HEADS + h], fmaxf(dot, 0.f), sum);
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (part == 0 && j < nb) {
      const float sb = reinterpret_cast<const float*>(src + SML_PAGE_TOKENS * SML_INDEX_DIM)[row];
      if (!there) raise_fault(b.status, SML_FAULT_PAGE);
      scores[(size_t)t * b.max_pages + j] = there ? sum * (__ldg(iq_scale + t) * c) * sb : NAN;
    }
  }
}

// ---- block selection --------------------------------------------------------------
// Order-preserving key: larger score, larger key; -0.0 as +0.0; NaN lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// One CTA per token: the k-th largest key of the row by four rounds of an 8-bit
// histogram, then one ordered pass that keeps every larger key and the first
// of the equal ones.  A row is read five times, from L1/L2 after the first.
constexpr int kTopThreads = 512;

__global__ void __launch_bounds__(kTopThreads)
block_topk_kernel(Batch b, const float* __restrict__ scores, int k, int32_t* __restrict__ blocks,
                  int32_t* __restrict__ blocks_len) {
  __shared__ int hist[256];
  __shared__ int warp_take[kTopThreads / 32], warp_tie[kTopThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
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
  uint32_t prefix = 0;   // the threshold key's leading bits found so far
  int need = take;       // keys still wanted among those that share them
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kTopThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nb; i += kTopThreads) {
      const uint32_t key = order_key(__ldg(row + i));
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  int out = 0, ties = 0;   // taken, and equal to the threshold, before this step
  for (int i0 = 0; i0 < nb; i0 += kTopThreads) {
    const int i = i0 + tid;
    const uint32_t key = i < nb ? order_key(__ldg(row + i)) : 0u;
    const bool above = i < nb && key > prefix, tie = i < nb && key == prefix;
    const unsigned tmask = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_tie[warp] = __popc(tmask);
    __syncthreads();
    int tb = ties, tsum = 0;
    for (int w = 0; w < kTopThreads / 32; ++w) {
      tb += w < warp ? warp_tie[w] : 0;
      tsum += warp_tie[w];
    }
    const bool keep = above || (tie && tb + __popc(tmask & ((1u << lane) - 1)) < need);
    const unsigned kmask = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) warp_take[warp] = __popc(kmask);
    __syncthreads();
    int ob = out, osum = 0;
    for (int w = 0; w < kTopThreads / 32; ++w) {
      ob += w < warp ? warp_take[w] : 0;
      osum += warp_take[w];
    }
    if (keep) dst[ob + __popc(kmask & ((1u << lane) - 1))] = i;
    out += osum;
    ties += tsum;
    __syncthreads();
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
  const int tiles = (p.max_pages + kScoreBlocks - 1) / kScoreBlocks;
  return launch_pdl(block_scores_kernel, dim3(p.num_tokens, tiles < 65535 ? tiles : 65535), dim3(kScoreThreads), 0,
                    stream, 0, batch_of(p, status), iq8, iq_scale, iw, static_cast<const uint8_t*>(block.base),
                    (long long)block.num_pages * SML_PAGE_TOKENS, scores);
}

cudaError_t launch_block_topk(const sml_problem& p, const float* scores, int k, int32_t* blocks, int32_t* blocks_len,
                              int32_t* status, cudaStream_t stream) {
  return launch_pdl(block_topk_kernel, dim3(p.num_tokens), dim3(kTopThreads), 0, stream, 0, batch_of(p, status), scores,
                    k, blocks, blocks_len);
}

}  // namespace sml
