// Attention of prompts through a sliding window with sinks: whole tiles of
// queries against the keys of their band.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i with
// j > i - window or j < n_sink; lse_i the log of the sum.
//
// What bounds it: a query row reads and writes 4 D bytes and computes 4 D flops
// a visible key, so up to a window of some 240 keys HBM decides, above it the
// tensor cores and, as much, the exponentials (16 a clock and SM against 4096
// products: a 128 x 128 tile takes 1024 clocks in either unit at D = 128).
//
// One CTA an SM, persistent over items, the longest first.  An item is a block
// of positions of one sequence and key/value head, as two tiles of 128 query
// rows: a row is (position, head), with all H / H_kv heads of a position next
// to each other, so that shared heads share the keys that the item loads, and
// its positions span few keys beyond the window.  Key tiles (KT keys) start at
// the band's first key.  Per key tile and query tile:
//   S = Q K^T      tcgen05 kind::f16, M = 128 rows, N = KT keys, into TMEM
//   softmax        a thread a row: running maximum and sum in registers, P
//                  rounded to the inputs' type over S in TMEM (the product takes
//                  operands of one type; the sum is of the unrounded weights:
//                  0.0023 of the outputs' size off in bf16, 0.0016 by their own
//                  rounding; fp16 0.00026 and 0.00020.  A second product with
//                  what the rounding leaves would double the PV time)
//   O += P V       A = P from TMEM, B = V read along dims (MN-major)
// O stays in TMEM; it is rescaled only when a row's maximum grows by more than
// 2^8 (P is then at most 256), which after the first tiles hardly happens.
// The two query tiles alternate on the tensor cores, each one's softmax under
// the other's products.  Key tiles of 64 keep two S buffers a query tile, of
// 128 one.
//
// P is 0 where a key is masked, but 0 * NaN would reach the sums: two warps look
// through the value tiles that some row does not see whole.  Values that no row
// of the item sees (padding, later tokens) are cleared where they are not
// finite; where some row does see one, the item is done again key by key.
//
// Warps: 0 TMA, 1 MMA issue, 2-3 value check, 4-7 and 8-11 softmax and
// epilogue of the two query tiles.  Every wait is bounded; on expiry
// SI_ERR_TIMEOUT is recorded, copies and MMAs in flight are drained and the
// kernel exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "si_internal.h"
#include "si_ptx.cuh"

namespace si {
namespace {

constexpr int W_THREADS = 384;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int W_FEW = 16;  // up to so many sinks take a small tile of their own

enum { WERR_Q = 61, WERR_K = 62, WERR_V = 63, WERR_S = 64, WERR_P = 65, WERR_O = 66, WERR_SCAN = 67, WERR_DRAIN = 68 };

struct WindowParams {
  const uint8_t *q, *k, *v;
  const int32_t* lens;
  uint8_t* out;
  float* lse;
  int* err;
  int B, S, H, H_kv, G, P;  // P positions a query tile
  int window, n_sink, blocks, wide_out, band_keys, band_sinks;
  int items;  // B * H_kv * blocks: no more than rows
  int withhold;  // test: block 0 leaves out a load of its second item
  float scale_log2;
  uint64_t wait_limit_ns;
};

// An item: positions p0 .. p0 + 2 P - 1 of sequence b, key/value head h.  Its
// key tiles: n_sink_tiles over keys [0, sink_end), then main tiles from key
// k_start on.  Query tile m uses the sinks' tiles and the main tiles [lo, hi).
struct Item {
  int b, h, p0, len, k_start, sink_end, sink_keys, n_sink_tiles, tiles, lo[2], hi[2];
  __device__ __forceinline__ bool uses(int m, int u) const {
    return hi[m] > lo[m] && (u < n_sink_tiles || (u - n_sink_tiles >= lo[m] && u - n_sink_tiles < hi[m]));
  }
};

template <int KT>
__device__ __forceinline__ Item item_of(const WindowParams& p, int n) {
  Item it;
  const int bh = n % (p.B * p.H_kv);
  it.b = bh / p.H_kv;
  it.h = bh % p.H_kv;
  it.p0 = (p.blocks - 1 - n / (p.B * p.H_kv)) * 2 * p.P;  // late positions see the most keys
  it.len = p.lens ? min(max(p.lens[it.b], 0), p.S) : p.S;
  it.k_start = max(0, it.p0 - p.window + 1);
  it.sink_end = min(p.n_sink, it.k_start);
  it.sink_keys = it.sink_end <= W_FEW ? W_FEW : KT;
  it.n_sink_tiles = (it.sink_end + it.sink_keys - 1) / it.sink_keys;
  const int k_end = min(it.p0 + 2 * p.P, it.len);
  const int main_tiles = it.p0 < it.len ? (k_end - it.k_start + KT - 1) / KT : 0;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int a = it.p0 + m * p.P, e = min(a + p.P, it.len);
    // (sinks that lie past k_start are seen from everywhere)
    it.lo[m] = a < it.len && p.n_sink <= it.k_start ? (max(0, a - p.window + 1) - it.k_start) / KT : 0;
    it.hi[m] = a < it.len ? (e - it.k_start + KT - 1) / KT : 0;
  }
  it.tiles = main_tiles ? main_tiles + it.n_sink_tiles : 0;
  return it;
}

__device__ __forceinline__ void window_error(const WindowParams& p, volatile int* abort, int where) {
  atomicCAS(p.err, 0, static_cast<int>(SI_ERR_TIMEOUT));
  atomicCAS(p.err + 1, 0, where);
  *abort = 1;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 4-D tiled load: (dim, head, position, sequence).
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int x, int h, int s, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(h), "r"(s), "r"(b)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A's rows on the lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand, 128-byte swizzle: atoms of 8 K-rows x 64 values; lbo bytes
// between atoms along N.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* v) {
  tmem_st16(addr, v);
  tmem_st16(addr + 16, v + 16);
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes a lane: whole sectors.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (HALF) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Two packed values times f.
template <bool HALF>
__device__ __forceinline__ uint32_t scale2(uint32_t v, float f) {
  float2 t;
  if constexpr (HALF) t = __half22float2(*reinterpret_cast<const __half2*>(&v));
  else t = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  return pack2<HALF>(t.x * f, t.y * f);
}

template <bool HALF>
__device__ __forceinline__ float load16(const uint8_t* p, size_t i) {
  if (HALF) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// A row by a warp, key by key, each lane D / 32 dims: for items that hold
// values that are not finite where some of their rows do not see them.
template <int D, bool HALF>
__device__ __noinline__ void row_by_keys(const WindowParams& p, const Item& it, int pos, int head) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const size_t row = (static_cast<size_t>(it.b) * p.S + pos) * p.H + head;
  float q[N], acc[N], m = -INFINITY, sum = 0.f;
  for (int d = 0; d < N; ++d) {
    q[d] = load16<HALF>(p.q, row * D + d * 32 + lane);
    acc[d] = 0.f;
  }
  const int first = max(pos - p.window + 1, 0);
  for (int j = 0; j <= pos; ++j) {
    if (j >= p.n_sink && j < first) j = first;
    const size_t at = ((static_cast<size_t>(it.b) * p.S + j) * p.H_kv + it.h) * D;
    float s = 0.f;
    for (int d = 0; d < N; ++d) s = fmaf(q[d], load16<HALF>(p.k, at + d * 32 + lane), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= p.scale_log2;
    // as by tiles: scores of -infinity weigh nothing, of +infinity NaN
    const float mn = fmaxf(m, s), off = mn == -INFINITY ? 0.f : mn, c = ex2(m - off), e = ex2(s - off);
    m = mn;
    sum = fmaf(sum, c, e);
    for (int d = 0; d < N; ++d) acc[d] = fmaf(e, load16<HALF>(p.v, at + d * 32 + lane), acc[d] * c);
  }
  for (int d = 0; d < N; ++d) {
    const size_t at = row * D + d * 32 + lane;
    if (HALF) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(acc[d] / sum);
    else reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[d] / sum);
  }
  if (p.lse && lane == 0) p.lse[row] = (m + log2f(sum)) * LN2;
}

template <int D, int KT>
struct WindowShape {
  static constexpr int HALVES = D / 64;        // 128-byte column blocks of a row
  static constexpr int QT = 128 * D * 2;       // a query tile
  static constexpr int TILE = KT * D * 2;      // a K or V tile
  static constexpr int NK = 65536 / TILE;      // K slots
  static constexpr int NV = KT == 128 && D == 128 ? 3 : NK;  // V slots: a V tile is held until both query tiles are through with it
  static constexpr int NSB = 128 / KT;         // S buffers of a query tile
};

template <int D, int KT>
struct WindowCtrl {
  using Sh = WindowShape<D, KT>;
  uint64_t q_full, q_empty;
  uint64_t k_full[Sh::NK], k_empty[Sh::NK], v_full[Sh::NV], v_empty[Sh::NV], v_ok[Sh::NV];
  uint64_t s_full[2][2], p_full[2][2], o_step[2][2], o_empty[2], scanned[2], rows_done[2], done;
  uint32_t tmem_slot;
  int abort;
  int again[2];  // number + 1 of an item that has to be done key by key (two items in turn)
};

// Low n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, bool HALF, int KT>
__global__ void __launch_bounds__(W_THREADS, 1)
    window_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k_few,
                            const __grid_constant__ CUtensorMap tm_v_few, const WindowParams p) {
  using Sh = WindowShape<D, KT>;
  constexpr int NK = Sh::NK, NV = Sh::NV, NSB = Sh::NSB;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + 2 * Sh::QT;
  uint8_t* v_s = k_s + NK * Sh::TILE;
  auto* C = reinterpret_cast<WindowCtrl<D, KT>*>(v_s + NV * Sh::TILE);
  volatile int* abort = &C->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = p.wait_limit_ns;
  if (tid == 0) {
    mbar_init(&C->q_full, 1);
    mbar_init(&C->q_empty, 1);
    for (int s = 0; s < NK; ++s) {
      mbar_init(&C->k_full[s], 1);
      mbar_init(&C->k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&C->v_full[s], 1);
      mbar_init(&C->v_empty[s], 1);
      mbar_init(&C->v_ok[s], 2);
    }
    for (int m = 0; m < 2; ++m) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&C->s_full[m][s], 1);
        mbar_init(&C->p_full[m][s], 4);
      }
      for (int s = 0; s < 2; ++s) mbar_init(&C->o_step[m][s], 1);
      mbar_init(&C->o_empty[m], 4);
      mbar_init(&C->scanned[m], 2);
      mbar_init(&C->rows_done[m], 8);
      C->again[m] = 0;
    }
    mbar_init(&C->done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&C->tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C->tmem_slot;
  // TMEM columns: S (and P over it) of query tile m at 128 m, O at 256 + 128 m

  // 384 threads x 168 registers at launch = 128 x 88 + 256 x 208
  if (warp < 4) regs_dec<88>();
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      uint32_t slots[2] = {0, 0}, phases[2] = {0, 0}, n_it = 0, any = 0, last = 0;  // K, V
      bool stop = false;
      for (int n = blockIdx.x; n < p.items && !stop; n += gridDim.x) {
        const Item it = item_of<KT>(p, n);
        if (!it.tiles) continue;
        if (!mbar_wait_bounded(&C->q_empty, (n_it & 1u) ^ 1u, abort, limit)) {
          window_error(p, abort, WERR_Q);
          break;
        }
        ++n_it;
        mbar_arrive_expect_tx(&C->q_full, 2 * p.P * p.G * D * 2);
        for (int m = 0; m < 2; ++m)
          for (int c = 0; c < Sh::HALVES; ++c)
            tma_load_4d(q_s + m * Sh::QT + c * 16384, &tm_q, &C->q_full, c * 64, it.h * p.G, it.p0 + m * p.P, it.b);
        for (int u = 0; u < it.tiles; ++u) {
          const bool sink = u < it.n_sink_tiles, few = sink && it.sink_keys == W_FEW;
          const int key0 = sink ? u * it.sink_keys : it.k_start + (u - it.n_sink_tiles) * KT;
          const uint32_t bytes = few ? W_FEW * D * 2 : Sh::TILE;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t slot = slots[kv], phase = phases[kv];
            uint64_t* full = kv ? &C->v_full[slot] : &C->k_full[slot];
            if (!mbar_wait_bounded(kv ? &C->v_empty[slot] : &C->k_empty[slot], phase ^ 1u, abort, limit)) {
              window_error(p, abort, kv ? WERR_V : WERR_K);
              stop = true;
              break;
            }
            if (!(p.withhold && blockIdx.x == 0 && n_it == 2 && u + kv == 0)) {
              mbar_arrive_expect_tx(full, bytes);
              const CUtensorMap* tm = kv ? (few ? &tm_v_few : &tm_v) : (few ? &tm_k_few : &tm_k);
              for (int c = 0; c < Sh::HALVES; ++c)
                tma_load_4d((kv ? v_s : k_s) + slot * Sh::TILE + c * (KT * 128), tm, full, c * 64, it.h, key0, it.b);
              any |= 1u << (slot + 16 * kv);
              last = (last & ~(1u << (slot + 16 * kv))) | (phase << (slot + 16 * kv));
            }
            if (++slots[kv] == (kv ? NV : NK)) {
              slots[kv] = 0;
              phases[kv] ^= 1u;
            }
          }
          if (stop) break;
        }
      }
      // every copy issued has landed before the CTA can exit
      bool ok = !n_it || mbar_wait_timed(&C->q_full, (n_it - 1) & 1u, limit);
      for (int s = 0; s < NK; ++s)
        if ((any >> s) & 1u) ok = mbar_wait_timed(&C->k_full[s], (last >> s) & 1u, limit) && ok;
      for (int s = 0; s < NV; ++s)
        if ((any >> (16 + s)) & 1u) ok = mbar_wait_timed(&C->v_full[s], (last >> (16 + s)) & 1u, limit) && ok;
      if (!ok) window_error(p, abort, WERR_DRAIN);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp walks the tiles and one lane issues: loop state and
    // descriptors stay the same in all lanes, in uniform registers.
    constexpr uint32_t FMT = HALF ? 0 : 1;
    constexpr uint32_t IDESC_S = idesc_f32acc(FMT, FMT, 128, KT), IDESC_FEW = idesc_f32acc(FMT, FMT, 128, W_FEW);
    constexpr uint32_t IDESC_O = idesc_f32acc(FMT, FMT, 128, D) | (1u << 16);  // V MN-major
    const uint64_t qd = sdesc_kmajor_sw128(smem_u32(q_s)), kd = sdesc_kmajor_sw128(smem_u32(k_s));
    const uint64_t vd = sdesc_mn(smem_u32(v_s), KT * 128);
    uint32_t kslot = 0, kphase = 0, vslot = 0, vphase = 0, n_it = 0;
    uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, ni[2] = {0, 0};  // S tiles, P tiles, items of a query tile
    bool stop = false;
    auto await = [&](uint64_t* bar, uint32_t parity, int where) {
      const bool got = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort, limit));
      if (!got && lane == 0) window_error(p, abort, where);
      return got;
    };
    for (int n = blockIdx.x; n < p.items && !stop; n += gridDim.x) {
      const Item it = item_of<KT>(p, n);
      const int tiles = __reduce_max_sync(0xFFFFFFFFu, it.tiles), sinks = __reduce_max_sync(0xFFFFFFFFu, it.n_sink_tiles);
      const bool few_sinks = __all_sync(0xFFFFFFFFu, it.sink_keys == W_FEW);
      int from[2], to[2];  // main tiles of a query tile
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        from[m] = sinks + __reduce_max_sync(0xFFFFFFFFu, it.lo[m]);
        to[m] = sinks + __reduce_max_sync(0xFFFFFFFFu, it.hi[m]);
      }
      if (!tiles) continue;
      if (!await(&C->q_full, n_it & 1u, WERR_Q)) break;
      ++n_it;
      bool begun[2] = {false, false};
      for (int step = 0; step < tiles + NSB; ++step) {
        const int u = step - NSB;  // the tile of this step's PV
        if (u >= 0 && !(await(&C->v_full[vslot], vphase, WERR_V) && await(&C->v_ok[vslot], vphase, WERR_V))) {
          stop = true;
          break;
        }
        if (step < tiles && !await(&C->k_full[kslot], kphase, WERR_K)) {
          stop = true;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (u >= 0 && to[m] > from[m] && (u < sinks || (u >= from[m] && u < to[m]))) {
            const uint32_t sb = np[m] % NSB;
            if (!await(&C->p_full[m][sb], (np[m] / NSB) & 1u, WERR_P) ||
                (!begun[m] && !await(&C->o_empty[m], (ni[m] & 1u) ^ 1u, WERR_P))) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + 256 + m * 128, a = tmem + m * 128 + sb * KT;
            const uint64_t vs = vd + vslot * (Sh::TILE >> 4);
            if (u < sinks && few_sinks) {
              if (elect_one()) mma_f16_ts(d, a, vs, IDESC_O, begun[m]);
            } else if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk) mma_f16_ts(d, a + kk * 8, vs + kk * (2048 >> 4), IDESC_O, begun[m] || kk != 0);
            }
            if (elect_one()) mma_commit(&C->o_step[m][np[m] & 1]);
            if (!begun[m]) ++ni[m];
            begun[m] = true;
            ++np[m];
          }
          if (step < tiles && to[m] > from[m] && (step < sinks || (step >= from[m] && step < to[m]))) {
            const uint32_t sb = nq[m] % NSB;
            const uint32_t idesc = step < sinks && few_sinks ? IDESC_FEW : IDESC_S;
            const uint32_t d = tmem + m * 128 + sb * KT;
            const uint64_t a = qd + m * (Sh::QT >> 4), b = kd + kslot * (Sh::TILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_bf16(d, a + ((kk >> 2) * 16384 + (kk & 3) * 32 >> 4), b + ((kk >> 2) * (KT * 128) + (kk & 3) * 32 >> 4),
                         idesc, kk != 0);
              mma_commit(&C->s_full[m][sb]);
            }
            ++nq[m];
          }
        }
        if (stop) break;
        if (u >= 0) {
          if (elect_one()) mma_commit(&C->v_empty[vslot]);
          if (++vslot == NV) {
            vslot = 0;
            vphase ^= 1u;
          }
        }
        if (step < tiles) {
          if (elect_one()) {
            mma_commit(&C->k_empty[kslot]);
            if (step == tiles - 1) mma_commit(&C->q_empty);
          }
          if (++kslot == NK) {
            kslot = 0;
            kphase ^= 1u;
          }
        }
      }
    }
    if (elect_one()) {
      mma_commit(&C->done);
      if (!mbar_wait_timed(&C->done, 0, limit)) window_error(p, abort, WERR_DRAIN);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ value check
    constexpr uint32_t EXP = HALF ? 0x7C007C00u : 0x7F807F80u, CARRY = HALF ? 0x04000400u : 0x00800080u;
    uint32_t slot = 0, phase = 0, n_it = 0;
    bool stop = false;
    for (int n = blockIdx.x; n < p.items && !stop; n += gridDim.x) {
      const Item it = item_of<KT>(p, n);
      if (!it.tiles) continue;
      const int last = min(it.p0 + 2 * p.P, it.len) - 1;  // the item's last position
      // the rows of the item before the last one have been written: again[] is free
      if (!mbar_wait_warp(&C->rows_done[n_it & 1], ((n_it >> 1) & 1u) ^ 1u, abort, limit)) {
        if (lane == 0) window_error(p, abort, WERR_SCAN);
        break;
      }
      for (int u = 0; u < it.tiles; ++u) {
        if (!mbar_wait_warp(&C->v_full[slot], phase, abort, limit)) {
          if (lane == 0) window_error(p, abort, WERR_V);
          stop = true;
          break;
        }
        const bool sink = u < it.n_sink_tiles, few = sink && it.sink_keys == W_FEW;
        const int keys = few ? W_FEW : KT;
        const int key0 = sink ? u * it.sink_keys : it.k_start + (u - it.n_sink_tiles) * KT;
        const int seen = sink ? it.sink_end : last + 1;  // keys from here on: seen by no row
        // every row of both query tiles sees the whole tile
        const bool all = key0 + keys <= seen && it.p0 + 2 * p.P <= it.len &&
                         (sink || (key0 + keys - 1 <= it.p0 && (key0 > last - p.window || key0 + keys <= p.n_sink)));
        if (!all) {
          // a thread a key (two with 128), its row's 16-byte chunks from a
          // place of its own on, so that the lanes meet no bank twice
          uint8_t* tile = v_s + slot * Sh::TILE;
#pragma unroll 1
          for (int key = tid - 64; key < keys; key += 64) {
            uint32_t acc = 0;
#pragma unroll
            for (int i = 0; i < Sh::HALVES * 8; ++i) {
              const uint4 x = *(reinterpret_cast<const uint4*>(tile + (i >> 3) * (KT * 128) + key * 128) + ((i + key) & 7));
              // an exponent of ones carries into the sign's place
              acc |= ((x.x & EXP) + CARRY) | ((x.y & EXP) + CARRY) | ((x.z & EXP) + CARRY) | ((x.w & EXP) + CARRY);
            }
            if (acc & 0x80008000u) {
              if (key0 + key >= seen) {
#pragma unroll 1
                for (int i = 0; i < Sh::HALVES * 8; ++i)
                  *(reinterpret_cast<uint4*>(tile + (i >> 3) * (KT * 128) + key * 128) + (i & 7)) = make_uint4(0, 0, 0, 0);
              } else {
                *reinterpret_cast<volatile int*>(&C->again[n_it & 1]) = static_cast<int>(n_it + 1);
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // cleared values are read by the MMA
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->v_ok[slot]);
        if (++slot == NV) {
          slot = 0;
          phase ^= 1u;
        }
      }
      if (lane == 0) mbar_arrive(&C->scanned[n_it & 1]);
      ++n_it;
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue of a query tile
    regs_inc<208>();
    const int m = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float ninf = -__int_as_float(0x7f800000);
    const int i_pos = row / p.G, head_of = row % p.G;
    const bool used = row < p.P * p.G;
    uint32_t ns = 0, n_it = 0;
    for (int n = blockIdx.x; n < p.items; n += gridDim.x) {
      const Item it = item_of<KT>(p, n);
      const int pos = it.p0 + m * p.P + i_pos;
      const bool live = used && pos < it.len;
      const int low = pos - p.window;  // the last key before the window
      float mref = ninf, l = 0.f;
      int count = 0;
      bool fail = false;
      for (int u = 0; u < it.tiles; ++u) {
        if (!it.uses(m, u)) continue;
        const uint32_t sb = ns % NSB;
        const bool got = mbar_wait_bounded(&C->s_full[m][sb], (ns / NSB) & 1u, abort, limit);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          if (lane == 0) window_error(p, abort, WERR_S);
          fail = true;
          break;
        }
        ++ns;
        tc_fence_after();
        const bool sink = u < it.n_sink_tiles, few = sink && it.sink_keys == W_FEW;
        const int key0 = sink ? u * it.sink_keys : it.k_start + (u - it.n_sink_tiles) * KT;
        const int keys = few ? W_FEW : KT;
        // columns c <= b and (c > a or c < e) are seen
        const int b = !live ? -1 : sink ? it.sink_end - 1 - key0 : pos - key0;
        const int a = sink ? -1 : low - key0, e = sink ? 0 : p.n_sink - key0;
        const bool masked = __any_sync(0xFFFFFFFFu, !(b >= keys - 1 && (a < 0 || e >= keys)));
        const uint32_t st = base + m * 128 + sb * KT;
        auto bits = [&](int c) { return low_bits(b + 1 - 32 * c) & (~low_bits(a + 1 - 32 * c) | low_bits(e - 32 * c)); };
        // one tile of NC columns; false: a wait ran out
        auto tile = [&](auto cols) -> bool {
          constexpr int NC = decltype(cols)::value, CH = (NC + 31) / 32, CW = NC / CH;  // chunks of CW columns
          float x[NC];
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if constexpr (CW == 16) tmem_ld16(st, *reinterpret_cast<uint32_t(*)[16]>(x));
            else tmem_ld32(st + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
          }
          tmem_ld_wait();
          uint32_t none = 0;  // chunks of which no row of the warp sees anything
          if (masked) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const uint32_t full = CW == 16 ? 0xFFFFu : ~0u, see = bits(c) & full;
              if (__all_sync(0xFFFFFFFFu, see == full)) continue;
              if (__all_sync(0xFFFFFFFFu, see == 0)) none |= 1u << c;
#pragma unroll
              for (int i = 0; i < CW; ++i) x[CW * c + i] = (see >> i) & 1u ? x[CW * c + i] : ninf;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < NC - 4; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
          mx[0] = max3(mx[0], x[NC - 4], x[NC - 3]);
          mx[1] = max3(mx[1], x[NC - 2], x[NC - 1]);
          const float mt = max3(max3(mx[0], mx[1], mx[2]), mx[3], ninf) * p.scale_log2;
          // a new reference where the maximum left the old one's reach
          const bool grow = mref != ninf && mt > mref + 8.f;
          if (count > 0 && __any_sync(0xFFFFFFFFu, grow)) {
            // O so far, after its last product; rows that do not grow keep it
            const bool got_o = mbar_wait_bounded(&C->o_step[m][ns & 1], ((ns - 2) >> 1) & 1u, abort, limit);  // product ns - 2
            if (!__all_sync(0xFFFFFFFFu, got_o)) {
              if (lane == 0) window_error(p, abort, WERR_O);
              return false;
            }
            tc_fence_after();
            const float f = grow ? ex2(mref - mt) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t x[32];
              tmem_ld32(base + 256 + m * 128 + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
              tmem_st32(base + 256 + m * 128 + 32 * c, x);
            }
          }
          if (grow || mref == ninf) mref = mt;
          const float off = mref == ninf ? 0.f : mref;
          const float2 sc = make_float2(p.scale_log2, p.scale_log2), sub = make_float2(-off, -off);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint32_t w[CW / 2];
            if ((none >> c) & 1u) {
#pragma unroll
              for (int i = 0; i < CW / 2; ++i) w[i] = 0;
            } else {
#pragma unroll
              for (int i = 0; i < CW / 2; ++i) {
                float2 t = fma2(make_float2(x[CW * c + 2 * i], x[CW * c + 2 * i + 1]), sc, sub);
                t = make_float2(ex2(t.x), ex2(t.y));
                sum[i & 1] = add2(sum[i & 1], t);
                w[i] = pack2<HALF>(t.x, t.y);
              }
            }
            // P lies over S, whose columns have all been read
            if constexpr (CW == 16) tmem_st8(st, w);
            else tmem_st16(st + 16 * c, w);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          return true;
        };
        const bool ok = few ? tile(std::integral_constant<int, W_FEW>{}) : tile(std::integral_constant<int, KT>{});
        if (!ok) {
          fail = true;
          break;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->p_full[m][sb]);
        ++count;
      }
      if (fail) break;
      // ---- the item's rows
      bool again = false;
      if (it.tiles) {
        bool got = mbar_wait_bounded(&C->scanned[n_it & 1], (n_it >> 1) & 1u, abort, limit);
        if (got && count) got = mbar_wait_bounded(&C->o_step[m][(ns - 1) & 1], ((ns - 1) >> 1) & 1u, abort, limit);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          if (lane == 0) window_error(p, abort, WERR_SCAN);
          break;
        }
        tc_fence_after();
        again = *reinterpret_cast<volatile int*>(&C->again[n_it & 1]) == static_cast<int>(n_it + 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->rows_done[n_it & 1]);
        ++n_it;
      }
      const bool write = used && pos < p.S && !(again && live);
      const size_t at = (static_cast<size_t>(it.b) * p.S + pos) * p.H + it.h * p.G + head_of;
      const float inv = live ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32], w[16];
        if (count) {
          tmem_ld32(base + 256 + m * 128 + 32 * c, x);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          w[i >> 1] = live ? pack2<HALF>(__uint_as_float(x[i]) * inv, __uint_as_float(x[i + 1]) * inv) : 0u;
        if (write) {
          uint8_t* dst = p.out + (at * D + 32 * c) * 2;
          if (p.wide_out) {
            store32(dst, w);
            store32(dst + 32, w + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
      }
      if (count) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->o_empty[m]);
      }
      if (write && p.lse) p.lse[at] = live ? (mref + log2f(l)) * LN2 : ninf;
      if (again) {
        for (int r = quad; r < p.P * p.G; r += 4) {
          const int rp = it.p0 + m * p.P + r / p.G;
          if (rp < it.len) row_by_keys<D, HALF>(p, it, rp, it.h * p.G + r % p.G);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ narrow bands
//
// Where all keys of an item's two query tiles, sinks included, are at most 256
// (window 128 with 8 heads a key/value head: 176), the whole item is one step:
// S of a query tile takes up to 256 TMEM columns, one softmax pass needs no
// running state, P lies over the first half of S and O over the second.  The
// streaming form above spends its time there on the steps' hand-offs: QK
// products of 64 columns cost as much as of 128 (the query tile has to be read
// for either), and a query tile takes four steps.  Q, K and V have one buffer:
// Q and K are free once both S are there, so the next item's arrive during the
// softmax, V's during the next QK.
//
// Window 128, 4 sinks, 64 query and 8 key/value heads, D = 128, 16,384
// positions: 186 to 193 us from one GPU to another (3.3 to 3.2 TB/s of 6.5, 24 %
// of the bf16 rate), 171 us where calls in a row leave their inputs in L2; the
// streaming form 276 us.  What is left is latency: a query tile's QK, softmax, PV
// and epilogue follow one another (1.3, 4, 1.4 and 2.7 thousand clocks), and with
// O over S only two fit into tensor memory.  Without the stores it takes 34 us
// less, without the exponentials 18.  Tried and not faster, each against this
// form in the same run: two warpgroups a query tile that share its columns (232
// to 193 us) or take items in turn (194 to 193), a share of the exponentials on
// the FMA units (177 to 194 against 177, inputs in L2).

struct BandItem {
  int b, h, p0, len, k_start, sink_end;
};

__device__ __forceinline__ BandItem band_item(const WindowParams& p, int n) {
  BandItem it;
  const int bh = n % (p.B * p.H_kv);
  it.b = bh / p.H_kv;
  it.h = bh % p.H_kv;
  it.p0 = n / (p.B * p.H_kv) * 2 * p.P;
  it.len = p.lens ? min(max(p.lens[it.b], 0), p.S) : p.S;
  it.k_start = max(0, it.p0 - p.window + 1);
  it.sink_end = min(p.n_sink, it.k_start);
  return it;
}

constexpr int BAND_KEYS = 256;   // columns of S
constexpr int BAND_STAGE = 4096; // a warp's rows on their way out: 32 rows x 64 dims

struct BandCtrl {
  uint64_t qk_full, qk_empty, v_full, v_empty, v_ok;
  uint64_t s_full[2], p_full[2], o_full[2], t_empty[2], checked, done;
  uint32_t tmem_slot;
  int abort, again;
};

template <int D, bool HALF>
__global__ void __launch_bounds__(W_THREADS, 1)
    band_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k_sink,
                          const __grid_constant__ CUtensorMap tm_v_sink, const WindowParams p) {
  constexpr int HALVES = D / 64, QT = 128 * D * 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int keys = p.band_keys, s16 = p.band_sinks;  // columns; those of the sinks, in front
  const int plane = keys * 128;                      // 64 dims of all keys
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + 2 * QT;
  uint8_t* v_s = k_s + HALVES * plane;
  uint8_t* o_s = v_s + HALVES * plane;
  auto* C = reinterpret_cast<BandCtrl*>(o_s + 8 * BAND_STAGE);
  volatile int* abort = &C->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = p.wait_limit_ns;
  if (tid == 0) {
    mbar_init(&C->qk_full, 1);
    mbar_init(&C->qk_empty, 1);
    mbar_init(&C->v_full, 1);
    mbar_init(&C->v_empty, 1);
    mbar_init(&C->v_ok, 2);
    for (int m = 0; m < 2; ++m) {
      mbar_init(&C->s_full[m], 1);
      mbar_init(&C->p_full[m], 4);
      mbar_init(&C->o_full[m], 1);
      mbar_init(&C->t_empty[m], 4);
    }
    mbar_init(&C->checked, 8);
    mbar_init(&C->done, 1);
    *abort = 0;
    C->again = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&C->tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C->tmem_slot;
  // items of this CTA, all with the same steps (padding's too: skipping it cost
  // the others 9 %, 197 against 180 us in one run): number i waits for parity i & 1

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      uint32_t i = 0, n_qk = 0, n_v = 0;  // items; loads issued
      for (int n = blockIdx.x; n < p.items; n += gridDim.x, ++i) {
        const BandItem it = band_item(p, n);
        if (!mbar_wait_bounded(&C->qk_empty, (i & 1u) ^ 1u, abort, limit)) {
          window_error(p, abort, WERR_Q);
          break;
        }
        if (!(p.withhold && blockIdx.x == 0 && i == 1)) {
          mbar_arrive_expect_tx(&C->qk_full, 2 * p.P * p.G * D * 2 + keys * D * 2);
          for (int c = 0; c < HALVES; ++c) {
            for (int m = 0; m < 2; ++m)
              tma_load_4d(q_s + m * QT + c * 16384, &tm_q, &C->qk_full, c * 64, it.h * p.G, it.p0 + m * p.P, it.b);
            if (s16) tma_load_4d(k_s + c * plane, &tm_k_sink, &C->qk_full, c * 64, it.h, 0, it.b);
            tma_load_4d(k_s + c * plane + s16 * 128, &tm_k, &C->qk_full, c * 64, it.h, it.k_start, it.b);
          }
          ++n_qk;
        }
        if (!mbar_wait_bounded(&C->v_empty, (i & 1u) ^ 1u, abort, limit)) {
          window_error(p, abort, WERR_V);
          break;
        }
        mbar_arrive_expect_tx(&C->v_full, keys * D * 2);
        for (int c = 0; c < HALVES; ++c) {
          if (s16) tma_load_4d(v_s + c * plane, &tm_v_sink, &C->v_full, c * 64, it.h, 0, it.b);
          tma_load_4d(v_s + c * plane + s16 * 128, &tm_v, &C->v_full, c * 64, it.h, it.k_start, it.b);
        }
        ++n_v;
      }
      // every copy issued has landed before the CTA can exit, whatever ended the loop
      bool ok = !n_qk || mbar_wait_timed(&C->qk_full, (n_qk - 1) & 1u, limit);
      if (n_v) ok = mbar_wait_timed(&C->v_full, (n_v - 1) & 1u, limit) && ok;
      if (!ok) window_error(p, abort, WERR_DRAIN);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t FMT = HALF ? 0 : 1;
    const uint32_t idesc_s = idesc_f32acc(FMT, FMT, 128, 0) | (static_cast<uint32_t>(keys >> 3) << 17);
    constexpr uint32_t IDESC_O = idesc_f32acc(FMT, FMT, 128, D) | (1u << 16);  // V MN-major
    const uint64_t qd = sdesc_kmajor_sw128(smem_u32(q_s)), kd = sdesc_kmajor_sw128(smem_u32(k_s));
    const uint64_t vd = sdesc_mn(smem_u32(v_s), plane);
    auto await = [&](uint64_t* bar, uint32_t parity, int where) {
      const bool got = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort, limit));
      if (!got && lane == 0) window_error(p, abort, where);
      return got;
    };
    uint32_t i = 0;
    bool stop = false;
    for (int n = blockIdx.x; n < p.items && !stop; n += gridDim.x, ++i) {
      const uint32_t par = i & 1u;
      if (!await(&C->qk_full, par, WERR_Q)) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (!await(&C->t_empty[m], par ^ 1u, WERR_O)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16(tmem + m * 256, qd + (m * QT + (kk >> 2) * 16384 + (kk & 3) * 32 >> 4),
                     kd + ((kk >> 2) * plane + (kk & 3) * 32 >> 4), idesc_s, kk != 0);
          mma_commit(&C->s_full[m]);
          if (m == 1) mma_commit(&C->qk_empty);
        }
      }
      if (stop || !await(&C->v_ok, par, WERR_V)) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (!await(&C->p_full[m], par, WERR_P)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          for (int kk = 0; kk < keys / 16; ++kk)
            mma_f16_ts(tmem + m * 256 + 128, tmem + m * 256 + kk * 8, vd + kk * (2048 >> 4), IDESC_O, kk != 0);
          mma_commit(&C->o_full[m]);
          if (m == 1) mma_commit(&C->v_empty);
        }
      }
    }
    if (elect_one()) {
      mma_commit(&C->done);
      if (!mbar_wait_timed(&C->done, 0, limit)) window_error(p, abort, WERR_DRAIN);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ value check
    constexpr uint32_t EXP = HALF ? 0x7C007C00u : 0x7F807F80u, CARRY = HALF ? 0x04000400u : 0x00800080u;
    uint32_t i = 0;
    for (int n = blockIdx.x; n < p.items; n += gridDim.x, ++i) {
      const BandItem it = band_item(p, n);
      const int last = min(it.p0 + 2 * p.P, it.len) - 1;
      // the last item's verdict has been read, this one's values are here
      const bool got = mbar_wait_bounded(&C->checked, (i & 1u) ^ 1u, abort, limit) &&
                       mbar_wait_bounded(&C->v_full, i & 1u, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) window_error(p, abort, WERR_V);
        break;
      }
#pragma unroll 1
      for (int r = tid - 64; r < keys; r += 64) {
        uint32_t acc = 0;
#pragma unroll
        for (int c = 0; c < HALVES * 8; ++c) {
          const uint4 x = *(reinterpret_cast<const uint4*>(v_s + (c >> 3) * plane + r * 128) + ((c + r) & 7));
          // an exponent of ones carries into the sign's place
          acc |= ((x.x & EXP) + CARRY) | ((x.y & EXP) + CARRY) | ((x.z & EXP) + CARRY) | ((x.w & EXP) + CARRY);
        }
        if (acc & 0x80008000u) {
          const bool seen = r < s16 ? r < it.sink_end : it.k_start + r - s16 <= last;
          if (seen) {
            *reinterpret_cast<volatile int*>(&C->again) = static_cast<int>(i + 1);
          } else {
#pragma unroll 1
            for (int c = 0; c < HALVES * 8; ++c)
              *(reinterpret_cast<uint4*>(v_s + (c >> 3) * plane + r * 128) + (c & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // cleared values are read by the MMA
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->v_ok);
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue of a query tile
    const int m = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t st = tmem + (static_cast<uint32_t>(quad * 32) << 16) + m * 256;
    const float ninf = -__int_as_float(0x7f800000);
    const int i_pos = row / p.G, head_of = row % p.G;
    const bool used = row < p.P * p.G;
    uint8_t* stage = o_s + (warp - 4) * BAND_STAGE;
    const int chunks = (keys + 63) / 64;
    uint32_t i = 0;
    for (int n = blockIdx.x; n < p.items; n += gridDim.x, ++i) {
      const BandItem it = band_item(p, n);
      const int pos = it.p0 + m * p.P + i_pos;
      const uint32_t par = i & 1u;
      const bool live = used && pos < it.len;
      // seen: columns up to b that lie behind a, or before e; of the sinks' columns those before sink_end
      const int b = pos - it.k_start + s16, a = b - p.window, e = p.n_sink - it.k_start + s16;
      auto bits = [&](int c) {
        const uint32_t main = low_bits(b + 1 - 32 * c) & (~low_bits(a + 1 - 32 * c) | low_bits(e - 32 * c)) & ~low_bits(s16 - 32 * c);
        return live ? main | low_bits(it.sink_end - 32 * c) : 0u;
      };
      bool got = mbar_wait_bounded(&C->s_full[m], par, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) window_error(p, abort, WERR_S);
        break;
      }
      tc_fence_after();
      // One pass, 64 columns at a time: P relative to a whole power of two, taken
      // from the first columns that are seen; where a later column exceeds it by
      // more than 2^8, what was written is scaled, which a power of two does
      // without rounding (but where fp16 weights become subnormal: by 2^-25 at most).
      float ref = ninf;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 sc = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const uint32_t see[2] = {bits(2 * c), bits(2 * c + 1)};
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = 0;
        if (__any_sync(0xFFFFFFFFu, (see[0] | see[1]) != 0)) {
          float x[64];
          tmem_ld32(st + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld32(st + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (!__all_sync(0xFFFFFFFFu, see[h] == ~0u)) {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[32 * h + k] = (see[h] >> k) & 1u ? x[32 * h + k] : ninf;
            }
          float mx[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) mx[j] = max3(x[j], x[8 + j], x[16 + j]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx[j] = max3(mx[j], x[24 + j], x[32 + j]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx[j] = max3(max3(mx[j], x[40 + j], x[48 + j]), x[56 + j], ninf);
          const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * p.scale_log2;
          const bool grow = ref != ninf && mt > ref + 8.f;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float to = ceilf(mt), f = grow ? ex2(ref - to) : 1.f;
            if (grow) ref = to;
            tmem_st_wait();  // the weights of the columns before are there
#pragma unroll
            for (int k = 0; k < 2; ++k) sum[k] = make_float2(sum[k].x * f, sum[k].y * f);
#pragma unroll 1
            for (int o = 0; o < 2 * c; ++o) {
              uint32_t y[16];
              tmem_ld16(st + 16 * o, y);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = scale2<HALF>(y[k], f);
              tmem_st16(st + 16 * o, y);
            }
            tmem_st_wait();
          }
          if (ref == ninf) ref = ceilf(mt);
          const float off = ref == ninf ? 0.f : ref;
          const float2 sub = make_float2(-off, -off);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (__any_sync(0xFFFFFFFFu, (see[g >> 1] >> (16 * (g & 1))) & 0xFFFFu)) {
#pragma unroll
              for (int k = 8 * g; k < 8 * g + 8; ++k) {
                float2 t = fma2(make_float2(x[2 * k], x[2 * k + 1]), sc, sub);
                t = make_float2(ex2(t.x), ex2(t.y));
                sum[k & 1] = add2(sum[k & 1], t);
                w[k] = pack2<HALF>(t.x, t.y);
              }
            }
        }
        tmem_st32(st + 32 * c, w);  // behind the columns that are still to be read
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->p_full[m]);
      const float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      const size_t at = (static_cast<size_t>(it.b) * p.S + pos) * p.H + it.h * p.G + head_of;
      if (p.lse && used && pos < p.S) p.lse[at] = live ? (ref + log2f(l)) * LN2 : ninf;
      got = mbar_wait_bounded(&C->o_full[m], par, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) window_error(p, abort, WERR_O);
        break;
      }
      tc_fence_after();
      const bool again = *reinterpret_cast<volatile int*>(&C->again) == static_cast<int>(i + 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->checked);
      // O leaves TMEM at once, so that the next S can come; then 64 dims at a
      // time through shared memory, so that whole lines go out
      const float inv = live ? 1.f / l : 0.f;
      const bool write = used && pos < p.S && !(again && live);
      const uint32_t writes = __ballot_sync(0xFFFFFFFFu, write);
      uint32_t w[D / 2];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float x[32];
        tmem_ld32(st + 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) w[c * 16 + k] = live ? pack2<HALF>(x[2 * k] * inv, x[2 * k + 1] * inv) : 0u;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->t_empty[m]);
      uint8_t* out = p.out + (static_cast<size_t>(it.b) * p.S + it.p0) * p.H * (D * 2);  // the item's first row
      const uint32_t rel = static_cast<uint32_t>((m * p.P + i_pos) * p.H + it.h * p.G + head_of);
#pragma unroll
      for (int c = 0; c < HALVES; ++c) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(w[c * 32 + 4 * j], w[c * 32 + 4 * j + 1], w[c * 32 + 4 * j + 2], w[c * 32 + 4 * j + 3]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j * 4 + (lane >> 3), ch = lane & 7;
          const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
          const uint32_t to = __shfl_sync(0xFFFFFFFFu, rel, r);
          if ((writes >> r) & 1u)
            __stcs(reinterpret_cast<uint4*>(out + static_cast<size_t>(to) * (D * 2) + c * 128) + ch, x);
        }
      }
      if (again) {
        const Item full{it.b, it.h, it.p0, it.len, 0, 0, 0, 0, 0, {0, 0}, {0, 0}};
        for (int r = quad; r < p.P * p.G; r += 4) {
          const int rp = it.p0 + m * p.P + r / p.G;
          if (rp < it.len) row_by_keys<D, HALF>(p, full, rp, it.h * p.G + r % p.G);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Map of [B, S, heads, D] rows: boxes of 64 dims x heads x positions.
si_status map_rows(CUtensorMap* m, bool half, const void* base, const WindowParams& p, int D, int heads, int box_heads,
                   int box_pos) {
  const uint64_t row = static_cast<uint64_t>(heads) * D * 2;
  const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(p.S),
                            static_cast<uint64_t>(p.B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, row, row * p.S};
  const uint32_t box[4] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_pos), 1};
  return encode_tmap(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides,
                     box, 128);
}

template <typename Kernel>
si_status launch_tiles(Kernel kernel, size_t smem, const WindowParams& p, int D, bool half, int keys, int few, int n_sm,
                       cudaStream_t stream) {
  CUtensorMap tm_q, tm_k, tm_v, tm_k_few, tm_v_few;
  si_status st = map_rows(&tm_q, half, p.q, p, D, p.H, p.G, p.P);
  if (st == SI_OK) st = map_rows(&tm_k, half, p.k, p, D, p.H_kv, 1, keys);
  if (st == SI_OK) st = map_rows(&tm_v, half, p.v, p, D, p.H_kv, 1, keys);
  if (st == SI_OK) st = map_rows(&tm_k_few, half, p.k, p, D, p.H_kv, 1, few);
  if (st == SI_OK) st = map_rows(&tm_v_few, half, p.v, p, D, p.H_kv, 1, few);
  if (st != SI_OK) return st;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) {
    kernel<<<std::min(p.items, n_sm), W_THREADS, smem, stream>>>(tm_q, tm_k, tm_v, tm_k_few, tm_v_few, p);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "window attention launch");
}

template <int D, bool HALF, int KT>
si_status launch_window(const WindowParams& p, int n_sm, cudaStream_t stream) {
  using Sh = WindowShape<D, KT>;
  constexpr size_t smem = 1024 + 2 * Sh::QT + (Sh::NK + Sh::NV) * Sh::TILE + sizeof(WindowCtrl<D, KT>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  // the kernel's register split has to fit the registers it is launched with,
  // a property of the build: its warps would wait for the rest forever
  static std::atomic<int> built{0};
  int regs = built.load();
  if (regs == 0) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, window_attention_kernel<D, HALF, KT>);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(window_attention_kernel)");
    built.store(regs = a.numRegs);
  }
  if (regs * W_THREADS < 128 * 88 + 256 * 208)
    return fail(SI_ERR_CUDA, "window_attention_kernel was built with %d registers a thread", regs);
  return launch_tiles(window_attention_kernel<D, HALF, KT>, smem, p, D, HALF, KT, W_FEW, n_sm, stream);
}

template <int D, bool HALF>
si_status launch_window_tiles(WindowParams& p, int n_sm, cudaStream_t stream) {
  const long long sinks = (static_cast<long long>(p.n_sink) + 15) / 16 * 16;
  const long long keys = sinks + (2ll * p.P + p.window - 1 + 15) / 16 * 16;
  if (keys <= BAND_KEYS) {
    p.band_keys = static_cast<int>(keys);
    p.band_sinks = static_cast<int>(sinks);
    constexpr size_t most = 1024 + 2 * 128 * D * 2 + 2 * BAND_KEYS * D * 2 + 8 * BAND_STAGE + sizeof(BandCtrl);
    static_assert(most <= 227 * 1024, "shared memory of a CTA");
    const size_t smem = 1024 + 2 * 128 * D * 2 + 2 * p.band_keys * D * 2 + 8 * BAND_STAGE + sizeof(BandCtrl);
    return launch_tiles(band_attention_kernel<D, HALF>, smem, p, D, HALF, p.band_keys - p.band_sinks,
                        std::max(p.band_sinks, 16), n_sm, stream);
  }
  // A query tile sees window + P - 1 keys.  Tiles of 64 keys waste fewer columns
  // at the band's ends and keep two S buffers, but their QK takes as long as
  // that of 128.  16,384 positions, 64 heads, P = 16, tiles of 64 against 128:
  // window 256 369 and 398 us, 384 424 and 428, 512 519 and 485, 2048 672 and 482
  // (8192 positions, 32 heads); window 128 with a head each (P = 128) 357 and 383.
  if (p.window + p.P <= 400) return launch_window<D, HALF, 64>(p, n_sm, stream);
  return launch_window<D, HALF, 128>(p, n_sm, stream);
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
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  WindowParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.lens = lens;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.err = err;
  p.B = B;
  p.S = S;
  p.H = H;
  p.H_kv = H_kv;
  p.G = H / H_kv;
  p.P = 128 / p.G;
  p.window = std::min(window, S);
  p.n_sink = std::min(n_sink, S);
  p.blocks = static_cast<int>((static_cast<long long>(S) + 2 * p.P - 1) / (2 * p.P));
  p.items = B * H_kv * p.blocks;
  p.wide_out = aligned(out, 32);
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(D))) * LOG2E;
  // an item that is done again key by key holds up its CTA's other warps for 13 to 15 us a visible key
  const uint64_t most_keys = std::min(static_cast<uint64_t>(p.window) + p.n_sink, static_cast<uint64_t>(S));
  p.wait_limit_ns = kDefaultWaitLimitNs + most_keys * 40000;
  p.withhold = take_withheld_load(&p.wait_limit_ns);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = dtype == SI_DTYPE_FP16;
  if (D == 128) return half ? launch_window_tiles<128, true>(p, n_sm, s) : launch_window_tiles<128, false>(p, n_sm, s);
  return half ? launch_window_tiles<64, true>(p, n_sm, s) : launch_window_tiles<64, false>(p, n_sm, s);
}

}  // extern "C"
