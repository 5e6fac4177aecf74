// The paged 8-bit K/V cache: appending rows, and the management of its pages
// (room for new tokens, forks, freeing, compaction).
//
// A page holds `page` tokens of a sequence for every key/value head as e4m3
// codes, with one fp32 scale per page and head (value = code * scale).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "si_internal.h"

namespace cg = cooperative_groups;

namespace si {
namespace {

// ------------------------------------------------------------------ append
//
// One block per (sequence, touched page, head, K or V): it reads the page's
// new rows once into registers (8 vectors of 16 bytes a thread), takes their
// amax, fixes the page's scale and writes the codes; no row is read twice.
// Bound by HBM bandwidth: 3 bytes an element (2 in, 1 out).  The scale is a
// power of two, so that a growing scale shifts the older codes' exponents and
// re-encoding them is exact down to e4m3's subnormals.

struct AppendParams {
  const uint8_t *k, *v;  // [B, L, H_kv, D] 16-bit
  uint8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  const int32_t *table, *lens, *n_new;
  int L, H_kv, page, max_pages, n_pages, slots;
};

// The least power of two s with amax <= 448 s = 1.75 * 2^8 s; 0 for amax 0;
// never below the least normal number, so that 1 / s is finite.
__device__ __forceinline__ float power_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8;  // biased exponent of s
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

template <bool HALF>
__device__ __forceinline__ float2 to_float2(uint32_t u) {
  if (HALF) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

constexpr int AP_VECS = 8;

// The largest finite magnitude of a thread's own vectors, where they hold an
// infinity or NaN.  A call: in line, 8 prompts of 2048 to 4096 tokens took 35 for 31 us.
template <int D, bool HALF>
__device__ __noinline__ uint32_t finite_top(const uint8_t* rows, int cnt, size_t stride) {
  constexpr uint32_t LIMIT = HALF ? 0x7C00u : 0x7F80u;
  constexpr int VROW = D / 8;
  uint32_t top = 0;
#pragma unroll 1
  for (int vec = threadIdx.x; vec / VROW < cnt; vec += blockDim.x) {
    const uint4 y = *reinterpret_cast<const uint4*>(rows + (vec / VROW) * stride + (vec % VROW) * 16);
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo16 = w[i] & 0x7FFFu, hi16 = (w[i] >> 16) & 0x7FFFu;
      top = max(top, max(lo16 < LIMIT ? lo16 : 0u, hi16 < LIMIT ? hi16 : 0u));
    }
  }
  return top;
}

template <int D, bool HALF>
__global__ void __launch_bounds__(256, 4) cache_append_kernel(const AppendParams p) {
  constexpr int VROW = D / 8;  // 16-byte input vectors of a row
  __shared__ uint32_t s_amax[8];
  long long u = blockIdx.x;
  const int h = static_cast<int>(u % p.H_kv);
  u /= p.H_kv;
  const bool val = u & 1;
  u >>= 1;
  const int slot = static_cast<int>(u % p.slots), b = static_cast<int>(u / p.slots);
  const long long len = p.lens[b];
  const long long nn = p.n_new ? min(max(p.n_new[b], 0), p.L) : p.L;
  const long long start = len > 0 ? len : 0, stop = len + nn;  // tokens written: [start, stop)
  const int shift = 31 - __clz(p.page);  // (a power of two)
  const long long pg = (start >> shift) + slot, t0 = pg << shift;
  const long long lo = max(start, t0), hi = min(stop, t0 + p.page);
  if (lo >= hi || pg >= p.max_pages) return;
  const int id = p.table[static_cast<size_t>(b) * p.max_pages + pg];
  if (id < 0 || id >= p.n_pages) return;
  const int off = static_cast<int>(lo - t0), cnt = static_cast<int>(hi - lo);
  const size_t ph = static_cast<size_t>(id) * p.H_kv + h;
  float* scale = (val ? p.v_scale : p.k_scale) + ph;
  uint8_t* codes = (val ? p.v_pages : p.k_pages) + ph * p.page * D;
  const uint8_t* rows = (val ? p.v : p.k) + ((static_cast<size_t>(b) * p.L + (lo - len)) * p.H_kv + h) * (D * 2);
  const float old = off > 0 ? *scale : 0.f;

  uint4 x[AP_VECS];
#pragma unroll
  for (int j = 0; j < AP_VECS; ++j) {
    const int vec = threadIdx.x + j * blockDim.x, row = vec / VROW;
    x[j] = make_uint4(0, 0, 0, 0);
    if (row < cnt)
      x[j] = __ldcs(reinterpret_cast<const uint4*>(rows + static_cast<size_t>(row) * p.H_kv * (D * 2) + (vec % VROW) * 16));
  }
  // the largest magnitude: 16-bit patterns without their sign order as their values
  constexpr uint32_t LIMIT = HALF ? 0x7C00u : 0x7F80u;  // infinity; NaN above
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < AP_VECS; ++j)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                                 __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu)));
  top = max(top & 0xFFFFu, top >> 16);
  if (top >= LIMIT)  // not finite
    top = finite_top<D, HALF>(rows, cnt, static_cast<size_t>(p.H_kv) * (D * 2));
  const float amax = to_float2<HALF>(top).x;
  const uint32_t wm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));  // non-negative: bits order as values
  if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = wm;
  __syncthreads();
  uint32_t am = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x) >> 5; ++i) am = max(am, s_amax[i]);
  const float fresh = power_scale(__uint_as_float(am));
  const float s = fmaxf(fresh, old);
  if (threadIdx.x == 0) *scale = s;
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;  // an exact reciprocal, or a true division
  const float inv = s > 0.f ? (pow2 ? __frcp_rn(s) : 1.f) : 1.f;
  if (s > old && off > 0) {
    // the older codes under the grown (power of two) scale
    for (int i = threadIdx.x; i < off * (D / 16); i += blockDim.x) {
      uint4* at = reinterpret_cast<uint4*>(codes) + i;
      const uint4 c = *at;
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint32_t r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = decode2(w[q]), g = decode2(w[q] >> 16);
        r[q] = encode4(f.x * old * inv, f.y * old * inv, g.x * old * inv, g.y * old * inv);
      }
      *at = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  if (pow2) {
#pragma unroll
    for (int j = 0; j < AP_VECS; ++j) {
      const int vec = threadIdx.x + j * blockDim.x, row = vec / VROW;
      if (row < cnt) {
        const float2 a = to_float2<HALF>(x[j].x), b = to_float2<HALF>(x[j].y), c = to_float2<HALF>(x[j].z),
                     d = to_float2<HALF>(x[j].w);
        *reinterpret_cast<uint2*>(codes + static_cast<size_t>(off + row) * D + (vec % VROW) * 8) =
            make_uint2(encode4(a.x * inv, a.y * inv, b.x * inv, b.y * inv), encode4(c.x * inv, c.y * inv, d.x * inv, d.y * inv));
      }
    }
  } else {
#pragma unroll 1
    for (int i = threadIdx.x; i < cnt * (D / 4); i += blockDim.x) {
      const int row = i / (D / 4), at = i % (D / 4);
      const uint2 w = *reinterpret_cast<const uint2*>(rows + static_cast<size_t>(row) * p.H_kv * (D * 2) + at * 8);
      const float2 a = to_float2<HALF>(w.x), b = to_float2<HALF>(w.y);
      *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(off + row) * D + at * 4) = encode4(a.x / s, a.y / s, b.x / s, b.y / s);
    }
  }
}

// ------------------------------------------------------------------ pages
//
// Each call plans in one launch of one cluster: its blocks scan a slice of
// refs each, exchange their counts through distributed shared memory, and so
// agree on the n-th free page without atomics whose order could change the
// result.  Bytes move in a second launch over the whole GPU, driven by the
// plan's list of (from, to) pages, which nothing else of the call reads.

constexpr int PG_CTAS = 8, PG_T = 1024, PG_W = PG_T / 32;
constexpr int PG_MAX_ROWS = 8192;

struct PageParams {
  int32_t *table, *lens, *refs;
  const int32_t *src, *dst, *n_new;
  int32_t *status;
  int32_t *list;        // scratch: free pages in order
  int32_t *from, *to;   // scratch: pages to copy
  int32_t *count;       // scratch: how many
  int n, n_seq, max_pages, n_pages, page, share;
};

struct PlanShared {
  int cnt[PG_CTAS][2];  // per block of the cluster: free pages, used pages
  long long warp[PG_W];  // block_prefix
};

// Exclusive prefix of v over the block's threads; *sum the total.  All threads call it.
template <typename T>
__device__ T block_prefix(T v, long long* warp_sums, T* sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();  // the last call's warp_sums have been read
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  if (w == 0) {
    T t = static_cast<T>(warp_sums[lane]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) t += u;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  *sum = static_cast<T>(warp_sums[PG_W - 1]);
  return static_cast<T>(w ? warp_sums[w - 1] : 0) + inc - v;
}

// Slice [lo, hi) of n that block r of the cluster scans.
__device__ __forceinline__ void slice(int n, int r, int* lo, int* hi) {
  const long long per = (n + PG_CTAS - 1) / PG_CTAS;
  *lo = static_cast<int>(min(static_cast<long long>(n), per * r));
  *hi = static_cast<int>(min(static_cast<long long>(n), per * (r + 1)));
}

// Counts the free pages of this block's slice and gives the count to every
// block of the cluster (complete after the next cluster barrier).
__device__ void count_free(cg::cluster_group& cl, PlanShared* S, const int32_t* refs, int n_pages) {
  int lo, hi, c = 0;
  slice(n_pages, cl.block_rank(), &lo, &hi);
  for (int i = lo + threadIdx.x; i < hi; i += PG_T) c += refs[i] <= 0;
  int sum;
  block_prefix(c, S->warp, &sum);
  if (threadIdx.x < PG_CTAS) {
    PlanShared* o = cl.map_shared_rank(S, threadIdx.x);
    o->cnt[cl.block_rank()][0] = sum;
    o->cnt[cl.block_rank()][1] = hi - lo - sum;
  }
}

// Writes the i-th pages (from `first` on, up to `most`) of this block's slice
// whose state is `want_free` and whose id is in [from_id, to_id) into list[],
// in ascending order.
__device__ void list_pages(PlanShared* S, const int32_t* refs, int lo, int hi, bool want_free, int first, int most,
                           int32_t* list) {
  for (int base = lo; base < hi && first < most; base += PG_T) {
    const int i = base + threadIdx.x;
    const int is = i < hi && (refs[i] <= 0) == want_free;
    int sum;
    const int at = first + block_prefix(is, S->warp, &sum);
    if (is && at < most) list[at] = i;
    first += sum;
  }
}

// Leading entries of a row (up to `most`) that are pages, counted by a warp;
// `first` is the row's entry at the lane.
__device__ int leading_pages(const int32_t* row, int first, int most, int n_pages) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < most; base += 32) {
    const int j = base + lane;
    const int id = j < most ? (base ? row[j] : first) : -1;
    const uint32_t bad = __ballot_sync(0xFFFFFFFFu, id < 0 || id >= n_pages);
    if (bad) return base + __ffs(bad) - 1;
  }
  return most;
}

// Reserve (FORK false): need[i] new pages for row i.  Fork: need[i] copied
// pages for pair i.  Both: validate and count the needs, spread over the
// cluster; prefix them in order; list as many free pages as are needed; hand
// them out.  need, held and the lengths live in every block's shared memory.
// Bound by the latency of dependent loads, so what does not depend on another
// load is under way with it.
template <bool FORK>
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_T, 1) page_plan_kernel(const PageParams p) {
  extern __shared__ int dyn[];
  __shared__ PlanShared S;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), lane = threadIdx.x & 31;
  const int gw = rank * PG_W + (threadIdx.x >> 5), n_gw = PG_CTAS * PG_W;
  int* need = dyn;            // [n] pages to hand out; -1: status 2
  int* held = dyn + p.n;      // [n] reserve: pages held; fork: pages of the child
  int* tok = dyn + 2 * p.n;   // [n] fork: tokens of the child
  int* dsts = dyn + 3 * p.n;  // [n] fork: the destinations
  if (FORK)
    for (int i = threadIdx.x; i < p.n; i += PG_T) dsts[i] = p.dst[i];
  cl.sync();                  // every block runs before any writes into another's shared memory
  count_free(cl, &S, p.refs, p.n_pages);  // (its barriers also order dsts)
  for (int i = gw; i < p.n; i += n_gw) {
    int nd = 0, hd = 0, tk = 0;
    if (FORK) {
      const int s = p.src[i], d = dsts[i];
      bool ok = s >= 0 && s < p.n_seq && d >= 0 && d < p.n_seq;
      bool twice = false;
      if (ok) {
        const int32_t* row = p.table + static_cast<size_t>(s) * p.max_pages;
        const int first = lane < p.max_pages ? row[lane] : -1;
        const int d0 = p.table[static_cast<size_t>(d) * p.max_pages], d_len = p.lens[d];
        tk = max(p.lens[s], 0);
        ok = d_len == 0 && (d0 < 0 || d0 >= p.n_pages);
        for (int j = lane; j < i; j += 32) twice |= dsts[j] == d;
        const int most = static_cast<int>(min(static_cast<long long>(p.max_pages), (static_cast<long long>(tk) + p.page - 1) / p.page));
        hd = leading_pages(row, first, most, p.n_pages);
        tk = static_cast<int>(min(static_cast<long long>(tk), static_cast<long long>(hd) * p.page));
        nd = p.share ? (tk % p.page ? 1 : 0) : hd;
      }
      if (__any_sync(0xFFFFFFFFu, twice) || !ok) {
        nd = -1;
        hd = tk = 0;
      }
    } else {
      const int32_t* row = p.table + static_cast<size_t>(i) * p.max_pages;
      const int add = p.n_new[i], len = p.lens[i], first = lane < p.max_pages ? row[lane] : -1;
      if (add > 0) {
        hd = leading_pages(row, first, p.max_pages, p.n_pages);
        const long long want = (max(static_cast<long long>(len) + add, 0ll) + p.page - 1) / p.page;
        nd = want > p.max_pages ? -1 : static_cast<int>(max(want - hd, 0ll));
      }
    }
    if (lane < PG_CTAS) {
      *cl.map_shared_rank(need + i, lane) = nd;
      *cl.map_shared_rank(held + i, lane) = hd;
      if (FORK) *cl.map_shared_rank(tok + i, lane) = tk;
    }
  }
  cl.sync();
  int free_before = 0, n_free = 0;
  for (int r = 0; r < PG_CTAS; ++r) {
    free_before += r < rank ? S.cnt[r][0] : 0;
    n_free += S.cnt[r][0];
  }
  // need[i] -> where its pages begin in the list; entries that fail get -1 - status
  int total = 0;       // pages handed out
  long long run = 0;   // needs before this chunk, failed ones among them
  for (int base = 0; base < p.n; base += PG_T) {
    const int i = base + threadIdx.x;
    const int nd = i < p.n ? need[i] : 0;
    long long sum;
    const long long at = run + block_prefix<long long>(max(nd, 0), S.warp, &sum);
    const bool fits = nd <= 0 || at + nd <= n_free;
    int good;
    block_prefix(nd > 0 && fits ? nd : 0, S.warp, &good);
    if (i < p.n) need[i] = nd < 0 ? -3 : fits ? static_cast<int>(nd ? at : 0) : -2;
    if (i < p.n && rank == 0) p.status[i] = nd < 0 ? 2 : fits ? 0 : 1;
    total += good;
    run += sum;
  }
  {
    int lo, hi;
    slice(p.n_pages, rank, &lo, &hi);
    list_pages(&S, p.refs, lo, hi, true, free_before, total, p.list);
  }
  cl.sync();  // the list is complete, refs have been read, status rows decided everywhere
  if (FORK && rank == 0 && threadIdx.x == 0) *p.count = total;
  for (int i = gw; i < p.n; i += n_gw) {
    const int at = need[i];
    if (at < 0) continue;
    if (FORK) {
      const int hd = held[i], tk = tok[i];
      const int full = p.share ? tk / p.page : 0;  // shared pages; the rest of the hd pages are copied
      const int32_t* from = p.table + static_cast<size_t>(p.src[i]) * p.max_pages;
      int32_t* row = p.table + static_cast<size_t>(p.dst[i]) * p.max_pages;
      for (int j = lane; j < p.max_pages; j += 32) {
        int id = -1;
        if (j < full) {
          id = from[j];
          atomicAdd(p.refs + id, 1);
        } else if (j < hd) {
          id = p.list[at + j - full];
          p.refs[id] = 1;
          p.from[at + j - full] = from[j];
          p.to[at + j - full] = id;
        }
        row[j] = id;
      }
      if (lane == 0) p.lens[p.dst[i]] = tk;
    } else {
      const int hd = held[i];
      int32_t* row = p.table + static_cast<size_t>(i) * p.max_pages;
      const int add = p.n_new[i];
      if (add <= 0) continue;
      const int want = static_cast<int>((max(static_cast<long long>(p.lens[i]) + add, 0ll) + p.page - 1) / p.page);
      for (int j = hd + lane; j < want; j += 32) {
        const int id = p.list[at + j - hd];
        row[j] = id;
        p.refs[id] = 1;
      }
    }
  }
}

// Compaction: U pages in use; the i-th free page below U takes the i-th used
// page from U on.
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_T, 1)
    compact_plan_kernel(const PageParams p, int32_t* used, int32_t* moved) {
  __shared__ PlanShared S;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank();
  cl.sync();
  count_free(cl, &S, p.refs, p.n_pages);
  cl.sync();
  int U = 0;
  for (int r = 0; r < PG_CTAS; ++r) U += S.cnt[r][1];
  // holes: free pages below U, movers: used pages from U on, each block's
  // share counted in its slice of [0, U) and [U, n_pages)
  int lo, hi, sum_h, sum_m, c = 0, m = 0;
  slice(p.n_pages, rank, &lo, &hi);
  for (int i = lo + threadIdx.x; i < hi; i += PG_T) {
    const bool is = p.refs[i] > 0;
    c += i < U && !is;
    m += i >= U && is;
    moved[i] = is ? i : -1;
  }
  block_prefix(c, S.warp, &sum_h);
  block_prefix(m, S.warp, &sum_m);
  cl.sync();  // the first counts have been read everywhere
  if (threadIdx.x < PG_CTAS) {
    PlanShared* o = cl.map_shared_rank(&S, threadIdx.x);
    o->cnt[rank][0] = sum_h;
    o->cnt[rank][1] = sum_m;
  }
  cl.sync();
  int h0 = 0, m0 = 0, total = 0;
  for (int r = 0; r < PG_CTAS; ++r) {
    h0 += r < rank ? S.cnt[r][0] : 0;
    m0 += r < rank ? S.cnt[r][1] : 0;
    total += S.cnt[r][0];
  }
  list_pages(&S, p.refs, lo, min(hi, max(U, lo)), true, h0, total, p.to);
  list_pages(&S, p.refs, max(lo, min(U, hi)), hi, false, m0, total, p.from);
  cl.sync();
  const int t = rank * PG_T + threadIdx.x, nt = PG_CTAS * PG_T;
  if (t == 0) {
    *used = U;
    *p.count = total;
  }
  for (int i = t; i < total; i += nt) {
    const int a = p.from[i], b = p.to[i];
    moved[a] = b;
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  cl.sync();
  const long long entries = static_cast<long long>(p.n_seq) * p.max_pages;
  for (long long i = t; i < entries; i += nt) {
    const int id = p.table[i];
    if (id >= U && id < p.n_pages) p.table[i] = moved[id];
  }
}

__global__ void cache_free_kernel(int32_t* table, int32_t* lens, int32_t* refs, const int32_t* rows, int n_seq,
                                  int max_pages, int n_pages) {
  const int r = rows[blockIdx.x];
  if (r < 0 || r >= n_seq) return;
  // an entry is taken by exchange, so that a row named twice is freed once
  for (int j = threadIdx.x; j < max_pages; j += blockDim.x) {
    const int id = atomicExch(table + static_cast<size_t>(r) * max_pages + j, -1);
    if (id >= 0 && id < n_pages) atomicSub(refs + id, 1);
  }
  if (threadIdx.x == 0) lens[r] = 0;
}

// Copies the listed pages: K, V and their scales.  A unit is up to 16 KB of
// one page of K or V (256 threads x 4 vectors), so that a few pages still
// spread over the GPU.
constexpr int CP_T = 256, CP_VECS = 4;

__global__ void __launch_bounds__(CP_T) copy_pages_kernel(uint4* k, uint4* v, float* ks, float* vs, const int32_t* from,
                                                         const int32_t* to, const int32_t* count, int vecs, int heads) {
  const int n = *count;
  const int parts = (vecs + CP_T * CP_VECS - 1) / (CP_T * CP_VECS);
  const long long units = 2ll * n * parts;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int part = static_cast<int>(u % parts);
    const long long w = u / parts;
    const int i = static_cast<int>(w >> 1);
    const size_t a = from[i], b = to[i];
    uint4* pool = w & 1 ? v : k;
    const uint4* s = pool + a * vecs;
    uint4* d = pool + b * vecs;
    uint4 x[CP_VECS];
#pragma unroll
    for (int j = 0; j < CP_VECS; ++j) {
      const int at = part * CP_T * CP_VECS + j * CP_T + threadIdx.x;
      if (at < vecs) x[j] = __ldcs(s + at);
    }
#pragma unroll
    for (int j = 0; j < CP_VECS; ++j) {
      const int at = part * CP_T * CP_VECS + j * CP_T + threadIdx.x;
      if (at < vecs) __stcs(d + at, x[j]);
    }
    if (part == 0) {
      float* sc = w & 1 ? vs : ks;
      for (int h = threadIdx.x; h < heads; h += CP_T) sc[b * heads + h] = sc[a * heads + h];
    }
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

si_status launch_copy_pages(const si_cache* c, const PageParams& p, cudaStream_t stream) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const int vecs = c->H_kv * c->page * (c->D / 16);
  copy_pages_kernel<<<n_sm * 8, CP_T, 0, stream>>>(static_cast<uint4*>(c->k_pages), static_cast<uint4*>(c->v_pages),
                                                    c->k_scale, c->v_scale, p.from, p.to, p.count, vecs, c->H_kv);
  e = cudaGetLastError();
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "copy_pages_kernel launch");
}

si_status check_pages(const si_cache* c, const void* table, const void* refs, int n_seq, int max_pages) {
  si_status st = check_cache(c);
  if (st != SI_OK) return st;
  if (!table || !refs) return fail(SI_ERR_INVALID_ARGUMENT, "table and refs must be non-null device pointers");
  if (n_seq < 1 || max_pages < 1) return fail(SI_ERR_INVALID_ARGUMENT, "n_seq and max_pages must be >= 1");
  if (n_seq > PG_MAX_ROWS) return fail(SI_ERR_UNSUPPORTED, "n_seq must be at most %d (got %d)", PG_MAX_ROWS, n_seq);
  return SI_OK;
}

bool ints_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}

// Shared memory of the plan: four ints for each of n entries.
template <bool FORK>
si_status launch_plan(PageParams& p, const si_cache* c, cudaStream_t stream) {
  // scratch: the free list, and for a fork the copies' ends and their count
  void* ws = nullptr;
  const size_t ints = static_cast<size_t>(p.n_pages) * (FORK ? 3 : 1) + 1;
  si_status st = scratch_alloc(&ws, ints * 4, stream, FORK ? "cache fork plan" : "cache reserve plan");
  if (st != SI_OK) return st;
  p.list = static_cast<int32_t*>(ws);
  p.count = p.list + p.n_pages;
  p.from = p.count + 1;
  p.to = p.from + p.n_pages;
  const size_t smem = static_cast<size_t>(p.n) * 4 * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(page_plan_kernel<FORK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PG_MAX_ROWS * 4 * static_cast<int>(sizeof(int)));
  if (e == cudaSuccess) {
    page_plan_kernel<FORK><<<PG_CTAS, PG_T, smem, stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) st = cuda_fail(e, "page plan launch");
  if (st == SI_OK && FORK) st = launch_copy_pages(c, p, stream);
  cudaFreeAsync(ws, stream);
  return st;
}

}  // namespace

si_status check_cache(const si_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale)
    return fail(SI_ERR_INVALID_ARGUMENT, "the cache and its pages and scales must be non-null");
  if (c->n_pages < 1 || c->H_kv < 1 || c->page < 1 || c->D < 1)
    return fail(SI_ERR_INVALID_ARGUMENT, "n_pages, H_kv, page and D must be >= 1");
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(SI_ERR_INVALID_ARGUMENT, "pages must be 16-byte aligned, scales 4-byte aligned");
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return fail(SI_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", c->page);
  if (c->D != 64 && c->D != 128) return fail(SI_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", c->D);
  if (static_cast<double>(c->n_pages) * c->H_kv * c->page > 2147483647.0)
    return fail(SI_ERR_UNSUPPORTED, "n_pages * H_kv * page must fit in 31 bits");
  return SI_OK;
}

}  // namespace si

using namespace si;

extern "C" {

si_status si_cache_append(const si_cache* c, const void* k, const void* v, const int32_t* table, const int32_t* lens,
                          const int32_t* n_new, int B, int L, int max_pages, int dtype, void* stream) {
  si_status st = check_cache(c);
  if (st != SI_OK) return st;
  if (!k || !v || !table || !lens) return fail(SI_ERR_INVALID_ARGUMENT, "k, v, table and lens must be non-null");
  if (B < 1 || L < 1 || max_pages < 1) return fail(SI_ERR_INVALID_ARGUMENT, "B, L and max_pages must be >= 1");
  if (!aligned(k, 16) || !aligned(v, 16) || !ints_aligned({table, lens, n_new}))
    return fail(SI_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned; table, lens and n_new 4-byte");
  if (dtype != SI_DTYPE_BF16 && dtype != SI_DTYPE_FP16)
    return fail(SI_ERR_UNSUPPORTED, "k and v are bf16 or fp16 (dtype %d)", dtype);
  AppendParams p;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_pages = static_cast<uint8_t*>(c->k_pages);
  p.v_pages = static_cast<uint8_t*>(c->v_pages);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.table = table;
  p.lens = lens;
  p.n_new = n_new;
  p.L = L;
  p.H_kv = c->H_kv;
  p.page = c->page;
  p.max_pages = max_pages;
  p.n_pages = c->n_pages;
  // pages that L rows touch at most, the first of them from its last slot on
  p.slots = static_cast<int>((static_cast<long long>(L) + c->page - 2) / c->page + 1);
  const double blocks = 2.0 * B * p.slots * c->H_kv;
  if (blocks > 2147483647.0) return fail(SI_ERR_UNSUPPORTED, "B * L * H_kv is too large for one call");
  const unsigned grid = static_cast<unsigned>(blocks);
  const int threads = std::max(32, c->page * c->D / (8 * AP_VECS));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = dtype == SI_DTYPE_FP16;
  if (c->D == 128) {
    if (half) cache_append_kernel<128, true><<<grid, threads, 0, s>>>(p);
    else cache_append_kernel<128, false><<<grid, threads, 0, s>>>(p);
  } else {
    if (half) cache_append_kernel<64, true><<<grid, threads, 0, s>>>(p);
    else cache_append_kernel<64, false><<<grid, threads, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "cache_append_kernel launch");
}

si_status si_cache_reserve(const si_cache* c, int32_t* table, const int32_t* lens, int32_t* refs, const int32_t* n_new,
                           int n_seq, int max_pages, int32_t* status, void* stream) {
  si_status st = check_pages(c, table, refs, n_seq, max_pages);
  if (st != SI_OK) return st;
  if (!lens || !n_new || !status) return fail(SI_ERR_INVALID_ARGUMENT, "lens, n_new and status must be non-null");
  if (!ints_aligned({table, lens, refs, n_new, status}))
    return fail(SI_ERR_INVALID_ARGUMENT, "int32 arrays must be 4-byte aligned");
  PageParams p = {};
  p.table = table;
  p.lens = const_cast<int32_t*>(lens);
  p.refs = refs;
  p.n_new = n_new;
  p.status = status;
  p.n = p.n_seq = n_seq;
  p.max_pages = max_pages;
  p.n_pages = c->n_pages;
  p.page = c->page;
  return launch_plan<false>(p, c, static_cast<cudaStream_t>(stream));
}

si_status si_cache_fork(const si_cache* c, int32_t* table, int32_t* lens, int32_t* refs, const int32_t* src,
                        const int32_t* dst, int n, int n_seq, int max_pages, int share, int32_t* status, void* stream) {
  si_status st = check_pages(c, table, refs, n_seq, max_pages);
  if (st != SI_OK) return st;
  if (n < 0) return fail(SI_ERR_INVALID_ARGUMENT, "n must be >= 0 (got %d)", n);
  if (n == 0) return SI_OK;
  if (n > PG_MAX_ROWS) return fail(SI_ERR_UNSUPPORTED, "n must be at most %d (got %d)", PG_MAX_ROWS, n);
  if (!lens || !src || !dst || !status) return fail(SI_ERR_INVALID_ARGUMENT, "lens, src, dst and status must be non-null");
  if (!ints_aligned({table, lens, refs, src, dst, status}))
    return fail(SI_ERR_INVALID_ARGUMENT, "int32 arrays must be 4-byte aligned");
  PageParams p = {};
  p.table = table;
  p.lens = lens;
  p.refs = refs;
  p.src = src;
  p.dst = dst;
  p.status = status;
  p.n = n;
  p.n_seq = n_seq;
  p.max_pages = max_pages;
  p.n_pages = c->n_pages;
  p.page = c->page;
  p.share = share != 0;
  return launch_plan<true>(p, c, static_cast<cudaStream_t>(stream));
}

si_status si_cache_free(int32_t* table, int32_t* lens, int32_t* refs, const int32_t* rows, int n, int n_seq,
                        int max_pages, int n_pages, void* stream) {
  if (!table || !lens || !refs || (n > 0 && !rows))
    return fail(SI_ERR_INVALID_ARGUMENT, "table, lens, refs and rows must be non-null device pointers");
  if (n < 0 || n_seq < 1 || max_pages < 1 || n_pages < 1)
    return fail(SI_ERR_INVALID_ARGUMENT, "n must be >= 0; n_seq, max_pages and n_pages >= 1");
  if (!ints_aligned({table, lens, refs, rows}))
    return fail(SI_ERR_INVALID_ARGUMENT, "int32 arrays must be 4-byte aligned");
  if (n == 0) return SI_OK;
  cache_free_kernel<<<n, 128, 0, static_cast<cudaStream_t>(stream)>>>(table, lens, refs, rows, n_seq, max_pages,
                                                                      n_pages);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "cache_free_kernel launch");
}

si_status si_cache_compact(const si_cache* c, int32_t* table, int32_t* refs, int n_seq, int max_pages, int32_t* used,
                           int32_t* moved, void* stream) {
  si_status st = check_pages(c, table, refs, n_seq, max_pages);
  if (st != SI_OK) return st;
  if (!used || !moved) return fail(SI_ERR_INVALID_ARGUMENT, "used and moved must be non-null device pointers");
  if (!ints_aligned({table, refs, used, moved}))
    return fail(SI_ERR_INVALID_ARGUMENT, "int32 arrays must be 4-byte aligned");
  PageParams p = {};
  p.table = table;
  p.refs = refs;
  p.n_seq = n_seq;
  p.max_pages = max_pages;
  p.n_pages = c->n_pages;
  p.page = c->page;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  st = scratch_alloc(&ws, (static_cast<size_t>(p.n_pages) * 2 + 1) * 4, s, "cache compaction plan");
  if (st != SI_OK) return st;
  p.count = static_cast<int32_t*>(ws);
  p.from = p.count + 1;
  p.to = p.from + p.n_pages;
  compact_plan_kernel<<<PG_CTAS, PG_T, 0, s>>>(p, used, moved);
  const cudaError_t e = cudaGetLastError();
  st = e == cudaSuccess ? launch_copy_pages(c, p, s) : cuda_fail(e, "compact_plan_kernel launch");
  cudaFreeAsync(ws, s);
  return st;
}

}  // extern "C"
