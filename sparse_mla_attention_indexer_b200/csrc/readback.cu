// Cached rows back as bf16: the counterparts of the cache writers.  Each value
// is dequantised in fp32 (code times scale) and rounded to bf16 once; a bf16
// pool's values are copied.
//
// Streaming copies with a little arithmetic, bound by the bytes in flight: a
// warp takes two rows and issues every load of both before it uses any.  Lane
// l holds latent values [16 l, 16 l + 16) of a row (one 16-B load of codes, two
// 16-B stores), lanes 0..7 the RoPE key.  30,720 fp8_ds_mla rows: 10.5 us for 55
// MB, 5.3 TB/s (one or four rows a warp: slower); their indexer keys 4.1 us for 12.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "sml_internal.cuh"

namespace sml {
namespace {

constexpr int kWarps = 8;
constexpr int kRowsPerWarp = 2;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two E4M3 codes times s, as two bf16.
__device__ __forceinline__ uint32_t dequant2(uint32_t two, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x * s, f.y * s);
}
__device__ __forceinline__ uint4 dequant8(uint32_t lo, uint32_t hi, float s) {
  return make_uint4(dequant2(lo, s), dequant2(lo >> 16, s), dequant2(hi, s), dequant2(hi >> 16, s));
}

__device__ __forceinline__ bool slot_ok(int s, long long slots, int lane, int32_t* status) {
  if (s >= 0 && s < slots) return true;
  if (s != -1 && lane == 0) raise_fault(status, SML_FAULT_PAGE);
  return false;
}

template <int kFormat>
__global__ void __launch_bounds__(32 * kWarps)
latent_read_kernel(const int32_t* __restrict__ slot, int n, const uint8_t* __restrict__ cache, long long slots,
                   float scale, uint4* __restrict__ c, uint4* __restrict__ kpe, int32_t* status) {
  constexpr bool kBf = kFormat == SML_LATENT_BF16, kPlain = kFormat == SML_LATENT_E4M3;
  constexpr int kRow = kBf ? SML_LATENT_BF16_ROW_BYTES : kPlain ? SML_LATENT_E4M3_ROW_BYTES : SML_LATENT_ROW_BYTES;
  constexpr int kPe = kBf ? 2 * SML_LATENT_DIM : kPlain ? SML_LATENT_DIM : SML_LATENT_DIM + 16;
  ptx::griddep_wait();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long step = (long long)gridDim.x * kWarps * kRowsPerWarp;
  for (long long i0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRowsPerWarp; i0 < n; i0 += step) {
    int s[kRowsPerWarp];
    bool ok[kRowsPerWarp];
    uint4 v0[kRowsPerWarp], v1[kRowsPerWarp], pe[kRowsPerWarp];
    float sc[kRowsPerWarp];
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      s[u] = i0 + u < n ? __ldg(slot + i0 + u) : -1;
      ok[u] = slot_ok(s[u], slots, lane, status);
    }
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      if (!ok[u]) continue;
      const uint8_t* row = cache + (size_t)s[u] * kRow;
      if (kBf) {
        v0[u] = __ldcg(reinterpret_cast<const uint4*>(row) + lane);
        v1[u] = __ldcg(reinterpret_cast<const uint4*>(row) + 32 + lane);
      } else {
        v0[u] = __ldcg(reinterpret_cast<const uint4*>(row) + lane);
        sc[u] = kPlain ? scale : __ldcg(reinterpret_cast<const float*>(row + SML_LATENT_DIM) + (lane >> 3));
      }
      if (kpe && lane < 8) {
        if (kPlain) {
          const uint2 p = __ldcg(reinterpret_cast<const uint2*>(row + kPe) + lane);
          pe[u].x = p.x;
          pe[u].y = p.y;
        } else {
          pe[u] = __ldcg(reinterpret_cast<const uint4*>(row + kPe) + lane);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      if (!ok[u]) continue;
      uint4* dst = c + (size_t)(i0 + u) * (SML_LATENT_DIM / 8);
      if (kBf) {
        dst[lane] = v0[u];
        dst[32 + lane] = v1[u];
      } else {
        dst[2 * lane] = dequant8(v0[u].x, v0[u].y, sc[u]);
        dst[2 * lane + 1] = dequant8(v0[u].z, v0[u].w, sc[u]);
      }
      if (kpe && lane < 8)
        kpe[(size_t)(i0 + u) * (SML_ROPE_DIM / 8) + lane] = kPlain ? dequant8(pe[u].x, pe[u].y, scale) : pe[u];
    }
  }
}

// Eight lanes per key, 16 values each; four keys per warp.
__global__ void __launch_bounds__(32 * kWarps)
indexer_k_read_kernel(const int32_t* __restrict__ slot, int n, const uint8_t* __restrict__ cache, long long slots,
                      uint4* __restrict__ k, int32_t* status) {
  ptx::griddep_wait();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  const int part = threadIdx.x & 7;
  const long long step = (long long)gridDim.x * kWarps * 4;
  for (long long i = (long long)blockIdx.x * kWarps * 4 + (threadIdx.x >> 3); i < n; i += step) {
    const int s = __ldg(slot + i);
    if (!slot_ok(s, slots, part, status)) continue;
    const uint8_t* page = cache + (size_t)(s / SML_PAGE_TOKENS) * SML_INDEX_PAGE_BYTES;
    const int row = s % SML_PAGE_TOKENS;
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(page + row * SML_INDEX_DIM) + part);
    const float sc = __ldcg(reinterpret_cast<const float*>(page + SML_PAGE_TOKENS * SML_INDEX_DIM) + row);
    uint4* dst = k + (size_t)i * (SML_INDEX_DIM / 8) + 2 * part;
    dst[0] = dequant8(v.x, v.y, sc);
    dst[1] = dequant8(v.z, v.w, sc);
  }
}

int row_grid(int n, int per_cta) {
  const int want = (n + per_cta - 1) / per_cta, cap = device_sm_count() * 8;
  return want < cap ? want : cap;
}

}  // namespace

cudaError_t launch_latent_read(const int32_t* slot, int n, const sml_cache& cache, void* c, void* kpe,
                               int32_t* status, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  auto kernel = cache.format == SML_LATENT_BF16   ? latent_read_kernel<SML_LATENT_BF16>
                : cache.format == SML_LATENT_E4M3 ? latent_read_kernel<SML_LATENT_E4M3>
                                                  : latent_read_kernel<SML_LATENT_FP8_DS_MLA>;
  return launch_pdl(kernel, dim3(row_grid(n, kWarps * kRowsPerWarp)), dim3(32 * kWarps), 0, stream, 0, slot, n,
                    static_cast<const uint8_t*>(cache.base), (long long)cache.num_pages * SML_PAGE_TOKENS, cache.scale,
                    static_cast<uint4*>(c), static_cast<uint4*>(kpe), status);
}

cudaError_t launch_indexer_k_read(const int32_t* slot, int n, const sml_cache& cache, void* k, int32_t* status,
                                  cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  return launch_pdl(indexer_k_read_kernel, dim3(row_grid(n, kWarps * 4)), dim3(32 * kWarps), 0, stream, 0, slot, n,
                    static_cast<const uint8_t*>(cache.base), (long long)cache.num_pages * SML_PAGE_TOKENS,
                    static_cast<uint4*>(k), status);
}

}  // namespace sml
