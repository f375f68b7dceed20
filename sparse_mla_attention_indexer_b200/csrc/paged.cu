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
// with a running maximum and sum per head.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "ptx.cuh"
#include "sml_internal.cuh"

namespace sml {
namespace {

constexpr int kHU = 16;            // heads per unit
constexpr int kThreads = 256;
constexpr int kMaxThreads = 1024;
constexpr int kRowF = 577;         // floats per staged row (odd: no bank conflicts)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  int format;
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

// Request of token t: with equal query counts it is t B / T, which two loads
// confirm; else a binary search.
__device__ __forceinline__ int find_request(const Params& P, int t) {
  const int guess = (int)((long long)t * P.B / P.T);
  if (__ldg(P.cu_q + guess) <= t && t < __ldg(P.cu_q + guess + 1)) return guess;
  return request_of(P.cu_q, P.B, t);
}

__device__ __forceinline__ Tok token_at(const Params& P, int t) {
  Tok k;
  k.r = find_request(P, t);
  const Req rq = load_request(P.cu_q, P.ctx_len, k.r, P.T, P.max_ctx, P.max_pages, P.vis_len != nullptr);
  k.ok = rq.ok && t >= rq.q0 && t - rq.q0 < rq.Q;
  bool bad = false;
  k.n = k.ok ? visible_len(P.vis_len, rq, t, &bad) : 0;
  k.ok = k.ok && !bad;
  if (!k.ok) k.n = 0;
  k.nss = ssmax_len_of(P.ssmax_len, t, k.n);
  k.lo = P.sel.window > 0 && k.n > P.sel.window ? k.n - P.sel.window : 0;
  k.len_bad = false;
  if (P.sel.blocks) {
    const int len = k.ok ? __ldg(P.sel.blocks_len + t) : 0;
    k.len_bad = len < 0 || len > P.sel.max_blocks;
    k.np = max(0, min(len, P.sel.max_blocks));
  } else {
    k.np = (k.n + SML_PAGE_TOKENS - 1) / SML_PAGE_TOKENS - k.lo / SML_PAGE_TOKENS;
  }
  return k;
}

__device__ __forceinline__ int tiles_of(const Tok& k) { return max(1, (k.np + 1) / 2); }

// Logical and physical page of the k-th page of token t (physical -1: masked,
// and reported by the one thread that asks with report set).
__device__ __forceinline__ int page_at(const Params& P, const Tok& tk, int t, int k, bool report, int* logical) {
  *logical = 0;
  if (k >= tk.np) return -1;
  int lg = tk.lo / SML_PAGE_TOKENS + k;
  if (P.sel.blocks) {
    lg = __ldg(P.sel.blocks + (size_t)t * P.sel.max_blocks + k);
    if (lg < 0 || lg >= (tk.n + SML_PAGE_TOKENS - 1) / SML_PAGE_TOKENS) {
      if (report) raise_fault(P.status, SML_FAULT_INDEX);
      return -1;
    }
  }
  *logical = lg;
  const int ph = __ldg(P.block_table + (size_t)tk.r * P.max_pages + lg);
  if (ph < 0 || ph >= P.latent_pages) {
    if (report) raise_fault(P.status, SML_FAULT_PAGE);
    return -1;
  }
  return ph;
}

// This CTA's range of its head group's tiles, and the token it starts in.
struct Range {
  long long total, ub, ue, tok0;   // tok0: first tile of token t0
  int used, t0;
};
struct PlanSmem {
  long long part[kMaxThreads / 32];
  long long tok0;
  int t0;
};

__device__ __forceinline__ long long range_begin(long long total, int used, int i) { return total * i / used; }
__device__ __forceinline__ int cta_of(long long total, int used, long long u) { return (int)(((u + 1) * used - 1) / total); }

template <int kN>
__device__ Range plan_range(const Params& P, int gi, PlanSmem& S) {
  const int per = (P.T + kN - 1) / kN, a = min(P.T, (int)threadIdx.x * per), b = min(P.T, a + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine = 0;
  for (int t = a; t < b; ++t) mine += tiles_of(token_at(P, t));
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) S.part[warp] = upto;
  __syncthreads();
  Range R;
  R.total = 0;
  long long before = 0;
  for (int w = 0; w < kN / 32; ++w) {
    before += w < warp ? S.part[w] : 0;
    R.total += S.part[w];
  }
  // as few CTAs as give the same longest range
  const long long most = (R.total + P.ws.cpg - 1) / P.ws.cpg;
  R.used = (int)((R.total + most - 1) / most);
  R.ub = gi < R.used ? range_begin(R.total, R.used, gi) : 0;
  R.ue = gi < R.used ? range_begin(R.total, R.used, gi + 1) : 0;
  const long long first = before + upto - mine;   // first tile of token a
  if (first <= R.ub && R.ub < first + mine) {
    long long at = first;
    for (int t = a; t < b; ++t) {
      const int nt = tiles_of(token_at(P, t));
      if (R.ub < at + nt) {
        S.t0 = t;
        S.tok0 = at;
        break;
      }
      at += nt;
    }
  }
  __syncthreads();
  R.t0 = S.t0;
  R.tok0 = S.tok0;
  return R;
}

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float e4m3_f(uint8_t v) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)v, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// Value d of the row at `row` (512 latent values, then 64 RoPE values).
__device__ __forceinline__ float row_value(const Params& P, const uint8_t* row, int d) {
  if (P.format == SML_LATENT_BF16) return bf16_f(reinterpret_cast<const uint16_t*>(row)[d]);
  if (P.format == SML_LATENT_E4M3) return e4m3_f(row[d]) * P.latent_scale;
  if (d < SML_LATENT_DIM) return e4m3_f(row[d]) * reinterpret_cast<const float*>(row + SML_LATENT_DIM)[d >> 7];
  return bf16_f(reinterpret_cast<const uint16_t*>(row + SML_LATENT_DIM + 16)[d - SML_LATENT_DIM]);
}

struct Smem {
  float row[SML_PAGE_TOKENS][kRowF];
  float q[kHU][kRowF];
  float p[kHU][SML_PAGE_TOKENS];
  float fac[kHU];
  PlanSmem plan;
};

__global__ void __launch_bounds__(kThreads) paged_mla_kernel(const Params P) {
  extern __shared__ uint8_t raw[];
  Smem& S = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x;
  const int g = (int)blockIdx.x % P.ws.hg, gi = (int)blockIdx.x / P.ws.hg;
  ptx::griddep_wait();
  if (tid == 0) ptx::griddep_launch_dependents();
  const Range R = plan_range<kThreads>(P, gi, S.plan);
  const int slot = (g * P.ws.cpg + gi) * 2;
  if (tid == 0) {
    // the token to join at this CTA: the one it continues, if the CTA before began it
    int4 rec = make_int4(-1, 0, 0, 0);
    if (gi < R.used && R.ub > R.tok0) {
      const int i0 = cta_of(R.total, R.used, R.tok0);
      if (i0 == gi - 1)
        rec = make_int4(R.t0, i0, cta_of(R.total, R.used, R.tok0 + tiles_of(token_at(P, R.t0)) - 1), 0);
    }
    P.ws.join[g * P.ws.cpg + gi] = rec;
  }
  const int D = SML_LATENT_DIM + P.rope_dim, rowb = P.format == SML_LATENT_BF16  ? SML_LATENT_BF16_ROW_BYTES
                                                     : P.format == SML_LATENT_E4M3 ? SML_LATENT_E4M3_ROW_BYTES
                                                                                   : SML_LATENT_ROW_BYTES;
  long long u = R.ub;
  int j0 = (int)(R.ub - R.tok0);
  for (int t = R.t0; u < R.ue; ++t, j0 = 0) {
    const Tok tk = token_at(P, t);
    const int nt = tiles_of(tk), j1 = (int)min((long long)nt, j0 + (R.ue - u));
    u += j1 - j0;
    if (tid == 0) {
      if (!tk.ok) raise_fault(P.status, SML_FAULT_LENGTHS);
      if (tk.len_bad) raise_fault(P.status, SML_FAULT_TOPK_LEN);
    }
    __syncthreads();
    for (int i = tid; i < kHU * D; i += kThreads)
      S.q[i / D][i % D] = bf16_f(P.q[((size_t)t * P.H + g * kHU + i / D) * D + i % D]);
    const float zscale = P.sm_scale * (P.ssmax ? P.ssmax_s * logf((float)tk.nss) : 1.f) * kLog2e;
    float m = -INFINITY, l = 0.f, acc[2][kHU];
#pragma unroll
    for (int h = 0; h < kHU; ++h) acc[0][h] = acc[1][h] = 0.f;
    for (int k = 2 * j0; k < min(tk.np, 2 * j1); ++k) {
      int lg;
      const int ph = page_at(P, tk, t, k, tid == 0, &lg);
      if (ph < 0) continue;
      __syncthreads();
      const int lo = max(0, tk.lo - lg * SML_PAGE_TOKENS), hi = min(SML_PAGE_TOKENS, tk.n - lg * SML_PAGE_TOKENS);
      for (int i = tid; i < SML_PAGE_TOKENS * D; i += kThreads) {
        const int row = i / D, d = i % D;
        S.row[row][d] =
            row >= lo && row < hi ? row_value(P, P.latent + ((size_t)ph * SML_PAGE_TOKENS + row) * rowb, d) : 0.f;
      }
      __syncthreads();
      // thread = (head, keys kk, kk + 16, ...)
      const int h = tid >> 4, kk = tid & 15;
      float z[4], mt = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = kk + 16 * i;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(S.q[h][d], S.row[key][d], s);
        z[i] = key >= lo && key < hi ? s * zscale : -INFINITY;
        mt = fmaxf(mt, z[i]);
      }
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float f = m == -INFINITY ? 0.f : exp2f(m - mt);
      l *= f;
      m = mt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = z[i] == -INFINITY ? 0.f : exp2f(z[i] - m);
        l += p;
        S.p[h][kk + 16 * i] = p;
      }
      if (kk == 0) S.fac[h] = f;
      __syncthreads();
#pragma unroll
      for (int hh = 0; hh < kHU; ++hh) {
        acc[0][hh] *= S.fac[hh];
        acc[1][hh] *= S.fac[hh];
      }
      for (int key = 0; key < SML_PAGE_TOKENS; ++key) {
        const float v0 = S.row[key][tid], v1 = S.row[key][tid + kThreads];
#pragma unroll
        for (int hh = 0; hh < kHU; ++hh) {
          acc[0][hh] = fmaf(S.p[hh][key], v0, acc[0][hh]);
          acc[1][hh] = fmaf(S.p[hh][key], v1, acc[1][hh]);
        }
      }
    }
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __syncthreads();
    const bool whole = j0 == 0 && j1 == nt;
    const size_t prow = (size_t)(slot + (j0 == 0)) * kHU;
    if ((tid & 15) == 0) {
      const int h = tid >> 4;
      S.fac[h] = l > 0.f ? 1.f / l : 0.f;
      const float lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      if (whole) P.lse[(size_t)t * P.H + g * kHU + h] = lse;
      else P.ws.part_lse[prow + h] = lse;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHU; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float o = acc[i][h] * S.fac[h];
        const int d = tid + i * kThreads;
        if (whole) {
          const __nv_bfloat16 b = __float2bfloat16_rn(o);
          P.out[((size_t)t * P.H + g * kHU + h) * SML_LATENT_DIM + d] = *reinterpret_cast<const uint16_t*>(&b);
        } else {
          P.ws.part_out[(prow + h) * SML_LATENT_DIM + d] = o;
        }
      }
  }
}

// out = sum_i exp(lse_i - lse) O_i, lse = ln sum_i exp(lse_i) over the pieces
// of one token that several CTAs hold.  One block per (CTA, head of its unit);
// only the CTA after the one that begins a split token has something to join.
__global__ void __launch_bounds__(128) paged_join_kernel(int H, PagedWs ws, uint16_t* __restrict__ out,
                                                         float* __restrict__ lse) {
  const int c = blockIdx.x, hl = blockIdx.y, g = c / ws.cpg;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int4 rec = __ldcg(ws.join + c);
  if (rec.x < 0) return;
  auto row = [&](int i) { return (size_t)((g * ws.cpg + i) * 2 + (i == rec.y)) * kHU + hl; };
  float m = -INFINITY;
  for (int i = rec.y; i <= rec.z; ++i) m = fmaxf(m, __ldcg(ws.part_lse + row(i)));
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int i = rec.y; i <= rec.z && m != -INFINITY; ++i) {
    const float w = expf(__ldcg(ws.part_lse + row(i)) - m);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(ws.part_out + row(i) * SML_LATENT_DIM) + threadIdx.x);
    den += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const size_t orow = (size_t)rec.x * H + g * kHU + hl;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  reinterpret_cast<uint2*>(out + orow * SML_LATENT_DIM)[threadIdx.x] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (threadIdx.x == 0) lse[orow] = den > 0.f ? m + logf(den) : -INFINITY;
}

}  // namespace

int paged_heads(const sml_problem&) { return kHU; }

PagedWs paged_plan(const sml_problem& p) {
  PagedWs w = {};
  w.hg = p.num_heads / kHU;
  w.cpg = device_sm_count() / w.hg > 0 ? device_sm_count() / w.hg : 1;
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
  P.format = latent.format;
  P.latent_scale = latent.scale;
  P.sel = sel;
  P.out = out;
  P.lse = lse;
  P.ws = ws;
  P.status = status;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(paged_mla_kernel), sizeof(Smem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_mla_kernel, dim3(ws.hg * ws.cpg), dim3(kThreads), sizeof(Smem), stream, 0, P);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_join_kernel, dim3(ws.hg * ws.cpg, kHU), dim3(128), 0, stream, 0, p.num_heads, ws, out, lse);
}

}  // namespace sml
