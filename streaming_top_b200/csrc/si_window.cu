// Attention of prompts through a sliding window with sinks.
//
// One warp per (sequence, query, head): it walks the visible keys with the
// running maximum and sum of the softmax, every lane holding D / 32 dims.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "si_internal.h"

namespace si {
namespace {

struct RowParams {
  const uint8_t *q, *k, *v;
  const float *ks, *vs;
  const int32_t *table, *lens;
  uint8_t* out;
  float* lse;
  int B, L, H, H_kv, page, max_pages, n_pages, window, n_sink;
  float scale;
};

template <bool HALF>
__device__ __forceinline__ float load16(const uint8_t* p, size_t i) {
  if (HALF) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float load8(const uint8_t* p, size_t i) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <int D, bool HALF, bool PAGED>
__global__ void __launch_bounds__(128) row_attention_kernel(const RowParams p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.L * p.H) return;
  const int h = static_cast<int>(row % p.H);
  const int i = static_cast<int>(row / p.H % p.L), b = static_cast<int>(row / p.H / p.L);
  const int g = h / (p.H / p.H_kv);
  long long len = p.lens ? p.lens[b] : p.L;
  long long pos;
  if (PAGED) {
    pos = len - p.L + i;
    len = min(len, static_cast<long long>(p.max_pages) * p.page);
  } else {
    len = min(max(len, 0ll), static_cast<long long>(p.L));
    pos = i < len ? i : -1;
  }
  float q[N], acc[N], m = -INFINITY, sum = 0.f;
  for (int d = 0; d < N; ++d) {
    q[d] = load16<HALF>(p.q, static_cast<size_t>(row) * D + d * 32 + lane);
    acc[d] = 0.f;
  }
  const long long stop = min(pos + 1, len);
  long long first = p.window ? max(pos - p.window + 1, 0ll) : 0;
  for (long long j = p.window ? 0 : first; j < stop; ++j) {
    if (j >= p.n_sink && j < first) j = first;
    if (j >= stop) break;
    float kv[N], vv[N];
    if (PAGED) {
      const int id = p.table[static_cast<size_t>(b) * p.max_pages + j / p.page];
      if (id < 0 || id >= p.n_pages) continue;
      const size_t ph = static_cast<size_t>(id) * p.H_kv + g, at = (ph * p.page + j % p.page) * D;
      for (int d = 0; d < N; ++d) {
        kv[d] = load8(p.k, at + d * 32 + lane) * p.ks[ph];
        vv[d] = load8(p.v, at + d * 32 + lane) * p.vs[ph];
      }
    } else {
      const size_t at = ((static_cast<size_t>(b) * p.L + j) * p.H_kv + g) * D;
      for (int d = 0; d < N; ++d) {
        kv[d] = load16<HALF>(p.k, at + d * 32 + lane);
        vv[d] = load16<HALF>(p.v, at + d * 32 + lane);
      }
    }
    float s = 0.f;
    for (int d = 0; d < N; ++d) s += q[d] * kv[d];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= p.scale;
    const float mn = fmaxf(m, s), c = m == mn ? 1.f : __expf(m - mn), e = s == mn ? 1.f : __expf(s - mn);
    m = mn;
    sum = sum * c + e;
    for (int d = 0; d < N; ++d) acc[d] = acc[d] * c + e * vv[d];
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  for (int d = 0; d < N; ++d) {
    const size_t at = static_cast<size_t>(row) * D + d * 32 + lane;
    if (HALF) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(acc[d] * inv);
    else reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[d] * inv);
  }
  if (p.lse && lane == 0) p.lse[row] = sum > 0.f ? m + logf(sum) : -INFINITY;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <bool PAGED>
si_status launch_rows(const RowParams& p, int D, int dtype, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.B) * p.L * p.H;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  const bool half = dtype == SI_DTYPE_FP16;
  if (D == 128) {
    if (half) row_attention_kernel<128, true, PAGED><<<grid, 128, 0, s>>>(p);
    else row_attention_kernel<128, false, PAGED><<<grid, 128, 0, s>>>(p);
  } else {
    if (half) row_attention_kernel<64, true, PAGED><<<grid, 128, 0, s>>>(p);
    else row_attention_kernel<64, false, PAGED><<<grid, 128, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "row_attention_kernel launch");
}

}  // namespace
}  // namespace si

using namespace si;

extern "C" {

si_status si_window_attention(const void* q, const void* k, const void* v, const int32_t* lens, int B, int S, int H,
                              int H_kv, int D, int window, int n_sink, float scale, int dtype, void* out, float* lse,
                              void* stream, const si_options* opt) {
  if (!k || !v) return fail(SI_ERR_INVALID_ARGUMENT, "k and v must be non-null device pointers");
  si_status st = check_attention(q, out, lse, B, S, H, H_kv, D, scale, dtype, n_sink);
  if (st != SI_OK) return st;
  if (window < 1) return fail(SI_ERR_INVALID_ARGUMENT, "window must be >= 1 (got %d)", window);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(lens, 4))
    return fail(SI_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned; lens 4-byte aligned");
  int* err = nullptr;
  st = error_word(opt, &err);
  if (st != SI_OK) return st;
  RowParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.lens = lens;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.B = B;
  p.L = S;
  p.H = H;
  p.H_kv = H_kv;
  p.window = window;
  p.n_sink = n_sink;
  p.scale = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(D));
  return launch_rows<false>(p, D, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
