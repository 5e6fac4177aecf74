// Attention over the paged 8-bit K/V cache: the last L tokens of each
// sequence against everything they see of it.
//
// What bounds it: every visible token costs 2 D bytes of HBM a key/value head
// and 4 D flops a query row.  With up to some 64 rows a head the bytes decide,
// so the kernel is built to read each page once, at full rate, and never to
// touch a code with an ALU:
//   S^T[token, row] = K[token, :] . q[row, :]     A = 128 cached tokens (e4m3, as TMA brings them), B = q
//   O^T[dim, row]   = sum_token V[token, dim] P   A = V read along dims (MN-major), B = P
// Both are tcgen05 kind::f8f6f4 products with the tokens (or dims) on the 128
// lanes and the few query rows on N, so no lane of the tensor core's M is
// padding.  q and the softmax weights, which have more bits than e4m3, enter
// as sums of e4m3 terms (two carry 8 bits, bf16's own precision; three the 11
// of fp16): q = 2^x (t0 + t1 / 16 [+ t2 / 256]), each term the rounded rest.  The
// terms stand side by side on N, so that the cached tile, whose reading bounds a
// product with so few columns, is read once for all of them, and their
// columns are added up when the accumulator is read.  With x from the row's
// largest magnitude (224 .. 448) bf16's terms are exact down to 2^-13 of it, then
// off by 2^-21 of it at most (fp16: 2^-14, 2^-25).
//
// P carries the value scales: P = 256 exp2(s - m) v_scale / v_ref, where m is the
// largest of s + log2(v_scale / v_ref) over what the row sees of the tile (with
// the scale's power of two; v_ref the tile's largest scale).  So P is 128 or more
// where weight times scale is largest, whichever of the two makes it so, and a
// tile far below the running maximum keeps its precision.  A weight is rounded by
// 2^-8 of itself (fp16: 2^-11), where weight times scale is below 2^-14 of the
// tile's largest by 2^-21 of that at most (fp16: 2^-25).  The sum takes the
// weights themselves, unrounded, and the running state joins tiles as usual; both in fp32.
//
// Work: tiles of 128 tokens.  All CTAs get equal runs of consecutive tiles of
// the whole batch (sequence, head, rows, tile), whatever its lengths; a unit
// (sequence, head, row chunk) that a run's border cuts leaves partial results
// (maximum, sum, unnormalised O) in one of its CTA's two slots, which a second
// kernel joins.  Where a unit has few tiles at most, units are not cut and no
// second kernel is launched.
//
// Measured (D = 128 unless said; bytes are those of the visible codes): 64
// sequences of 4096 to 8192 tokens, 64 / 8 heads: 150 to 160 us from one GPU to
// another, 5.4 to 5.1 TB/s of 6.5; 16 of 8192 to 16,384 tokens, four queries each,
// 32 / 8 heads, D = 64, fp16: 111 us, 1.9 TB/s; one of 262,143 tokens, 64 / 1 heads:
// 75 us, 0.89 TB/s; windows of 128 tokens and 4 sinks in 128 sequences: 33 us.
// With eight rows a head a tile takes 2700 clocks in each of an SM's two CTAs, near
// the 1400 that its bytes need; with more rows, or few tiles a CTA, the hand-offs
// between the warps (a tile's S, maximum, P, O) are what is left.  The joining
// kernel takes some 20 of the 75 us of the long sequence (64 of its blocks work,
// each on 148 partial results in turn), 8 of the 150 and of the 111.
//
// Warps: 0 schedules (walks the tiles, reads page table and scales ahead,
// publishes tile descriptors) and loads pages by TMA; 1 issues the MMAs; 2-3
// split the queries into terms; the rest do the softmax: two or four
// warpgroups take a share of the rows each, a thread one token (and later one
// dim).
// Every wait is bounded; on expiry SI_ERR_TIMEOUT is recorded, copies and MMAs
// in flight are drained and the kernel exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "si_internal.h"
#include "si_ptx.cuh"

namespace si {
namespace {

constexpr int C_TILE = 128;      // tokens of a tile
constexpr int C_ND = 8;          // tile descriptors in flight
// Units of at most this many tiles are not cut: the second kernel costs more
// than their length.  64 query and 8 key/value heads, cut against whole: 1000
// tokens (8 tiles) 22 and 18 us a sequence, 45 and 38 us for 64 of them; 2000
// tokens (16 tiles) 21.5 and 27.
constexpr int C_WHOLE = 8;
constexpr int C_MAX_CTAS = 512;  // of a launch
constexpr int C_FAR = 80;  // value scales of a tile further apart than 2^C_FAR count as that far
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

enum { CERR_SLOT = 41, CERR_DESC = 42, CERR_FULL = 43, CERR_Q = 44, CERR_S = 45, CERR_P = 46, CERR_O = 47,
       CERR_X = 48, CERR_DRAIN = 49 };

enum { F_FIRST = 1, F_LAST = 2, F_MASK = 4 };  // of the CTA's segment of a unit; not every row sees every token

struct CacheParams {
  const uint8_t* q;
  const float *ks, *vs;
  const int32_t *table, *lens;
  uint8_t* out;
  float* lse;
  float* part;       // partial results: [2 * CTAs] slots of rows x (D + 2) floats
  int4* meta;        // [CTAs]: the unit that begins in the CTA and goes on, the CTAs it spans, its slot
  int* err;
  long long rows_total;  // rows of the pools
  int B, L, H, H_kv, G, page, max_pages, n_pages, window, n_sink, chunks, cut;
  int withhold;  // test: block 0 leaves out the keys of its second tile
  float scale_log2;
  uint64_t wait_limit_ns;
};

// A tile, as the scheduler publishes it.
struct TileDesc {
  int flags, b, h, row0, rows, vslot, vparity;
  int p_lo, p_hi;       // positions of the sequence's first and last query
  int pages;            // bit j: page j of the tile is there
  int seg;              // 0: the CTA's first segment of a unit, 1: a later one (its slot)
  int left;             // the unit's tiles behind this one
  float vref;
  int tok[8];           // a page's first token
  float ks[8];          // its key scale
  float rv[8], lr[8];   // value scale / v_ref = 2^lr rv / 256, rv in (128, 256]
};

// The visible pages of a sequence: sink_pages from 0 on, then those from `first`
// on.  Its tiles take them in this order, 128 tokens' worth each, so that the
// sinks share a tile with the window.
struct Span {
  int first, sink_pages, pages, tiles;
  int p_lo, p_hi;
};

// Tokens of a sequence: what lies beyond its row of the table is not there.
__device__ __forceinline__ long long tokens_of(const CacheParams& p, int b) {
  return min(static_cast<long long>(p.lens[b]), static_cast<long long>(p.max_pages) * p.page);
}

__device__ __forceinline__ Span span_of(const CacheParams& p, int b) {
  Span s;
  const long long len = tokens_of(p, b);
  const long long p_lo = len - p.L, p_hi = len - 1;
  // visible tokens: [0, sink) and [lo, hi)
  const long long hi = max(len, 0ll);
  const long long lo = p.window ? min(max(p_lo - p.window + 1, 0ll), hi) : 0;
  const long long sink = p.window ? min(static_cast<long long>(p.n_sink), hi) : 0;
  s.first = static_cast<int>(lo / p.page);
  s.sink_pages = min(static_cast<int>((sink + p.page - 1) / p.page), s.first);
  s.pages = static_cast<int>((hi + p.page - 1) / p.page) - s.first + s.sink_pages;
  s.tiles = max((s.pages * p.page + C_TILE - 1) / C_TILE, 1);  // an empty unit still writes its rows
  s.p_lo = static_cast<int>(max(p_lo, -(1ll << 30)));
  s.p_hi = static_cast<int>(p_hi < 0 ? -1 : p_hi);
  return s;
}

// part * total / n, by a 32-bit division where that is enough.
__device__ __forceinline__ long long share(long long total, unsigned part, unsigned n) {
  const unsigned long long x = static_cast<unsigned long long>(total) * part;
  return x >> 32 ? static_cast<long long>(x / n) : static_cast<long long>(static_cast<uint32_t>(x) / n);
}

__device__ __forceinline__ void cache_error(const CacheParams& p, volatile int* abort, int where) {
  atomicCAS(p.err, 0, static_cast<int>(SI_ERR_TIMEOUT));
  atomicCAS(p.err + 1, 0, where);
  *abort = 1;
}

// Matrix descriptors: `type` 2 = 128-byte swizzle, 4 = 64-byte, 0 = none.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t type) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1u) << 46 |
         static_cast<uint64_t>(type) << 61;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"(addr));
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(addr));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
  } else {
    static_assert(N == 32, "columns");
    tmem_ld32(addr, *reinterpret_cast<uint32_t(*)[32]>(v));
  }
}

// The largest of a value over the warp (NaN loses).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Term i of a sum of e4m3 terms is stored times TERM_UP^i: what a term leaves is
// at most 1/16 of it, and so keeps off the codes' subnormal numbers for longer.
constexpr float TERM_UP = 16.f;

// What four codes leave of v[0..3], for the next term.
__device__ __forceinline__ void take_off(float (&v)[4], uint32_t codes) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
  v[0] = (v[0] - fa.x) * TERM_UP;
  v[1] = (v[1] - fa.y) * TERM_UP;
  v[2] = (v[2] - fb.x) * TERM_UP;
  v[3] = (v[3] - fb.y) * TERM_UP;
}

// Sizes of an instantiation: R query rows of a unit (8, 16, 32 or 64).
template <int D, int R, bool HALF>
struct CacheShape {
  static constexpr int TERMS = HALF ? 3 : 2;   // e4m3 terms of q and of P
  static constexpr int N = (TERMS * R + 15) / 16 * 16;  // the MMAs' N: term i of row r is column i R + r
  static constexpr int CTAS = R <= 16 ? 2 : 1; // per SM
  // Softmax warpgroups, each with a share of the rows.  Eight rows a thread at
  // most (sixteen of 64): with 32 the unrolled loop no longer fits the
  // instruction cache, and 2 warpgroups wait more than they issue.
  static constexpr int WG = R >= 32 ? 4 : 2;
  static constexpr int HC = R / WG;            // rows of a thread
  static constexpr int THREADS = 128 + 128 * WG;
  // With sixteen rows a thread the softmax warps take registers from the others
  // (96 a thread spill in the tile loop: 86 for 77 us with 262,143 tokens).
  static constexpr bool SPLIT = HC > 8;
  static constexpr int REGS_FEW = 64, REGS_MANY = 104, REGS = 96;
  static_assert(!SPLIT || 128 * REGS_FEW + 128 * WG * REGS_MANY <= THREADS * REGS, "registers of a launch");
  static constexpr int SLOT = C_TILE * D;      // a K or V tile
  static constexpr int Q = N * D;              // one q buffer
  static constexpr int P = N * C_TILE;         // one P buffer
  static constexpr int SLOTS = CTAS == 2 ? (D == 128 ? (R == 16 && HALF ? 4 : 5) : 10) : (R == 32 || D == 64 ? 10 : 8);
  static constexpr int TMEM = 4 * N <= 64 ? 64 : 4 * N <= 128 ? 128 : 4 * N <= 256 ? 256 : 512;  // S and O, two buffers each
  static_assert(4 * N <= 512 / CTAS, "tensor memory");
};

template <int D, int R, bool HALF>
struct CacheCtrl {
  using Sh = CacheShape<D, R, HALF>;
  uint64_t full[Sh::SLOTS], empty[Sh::SLOTS];
  uint64_t d_full[C_ND], d_empty[C_ND];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], xbar, done;
  int k_flags[Sh::SLOTS];             // flags of the tile whose keys a slot holds
  TileDesc desc[C_ND];
  alignas(16) float qs[2][R];         // score scale of a row
  alignas(16) int pos[2][R];          // a row's position; -1: sees nothing
  alignas(16) int low[2][R];          // tokens at or below are before its window
  alignas(16) int out[2][R];          // its row of the output
  alignas(16) float red[2][R][4];     // per row and quadrant of lanes: the tile's maximum
  alignas(16) float sum[R][4];        // the same: the unit's sum
  alignas(16) float fa[2][R], fb[2][R];  // per row: factors of the state and of the tile's O
  alignas(16) float col[4 * Sh::WG][3][Sh::HC];  // per warp: its rows' maxima in the tile, factors of the state, of the tile
  uint16_t nan_bits[2][C_TILE][D / 16];  // dims whose value is NaN, for tokens that only some rows see
  int nan_tok[2][8], nan_tile[2];     // first tokens of such a tile's pages, and its number
  long long scan[Sh::THREADS / 32];
  int b0;                             // the sequence in which the run starts,
  long long before0;                  // and the tiles of one (head, chunk) in the sequences before it
  uint32_t tmem_slot;
  int abort;
};

template <int D, int R, bool HALF>
__global__ void __launch_bounds__((CacheShape<D, R, HALF>::THREADS), (CacheShape<D, R, HALF>::CTAS))
    cache_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const CacheParams p) {
  using Sh = CacheShape<D, R, HALF>;
  constexpr int N = Sh::N, TERMS = Sh::TERMS, NS = Sh::SLOTS, HC = Sh::HC, WG = Sh::WG, C_THREADS = Sh::THREADS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kv_s = smem;
  uint8_t* q_s = kv_s + NS * Sh::SLOT;
  uint8_t* p_s = q_s + 2 * Sh::Q;
  auto* C = reinterpret_cast<CacheCtrl<D, R, HALF>*>(p_s + 2 * Sh::P);
  volatile int* abort = &C->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = p.wait_limit_ns;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&C->full[s], 1);
      mbar_init(&C->empty[s], 1);
    }
    for (int s = 0; s < C_ND; ++s) {
      mbar_init(&C->d_full[s], 1);
      mbar_init(&C->d_empty[s], 2 + 4 * WG);  // two q warps, the softmax warps
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&C->q_full[s], 2);
      mbar_init(&C->q_empty[s], 1 + 4 * WG);  // the MMAs' commit, the softmax warps
      mbar_init(&C->s_full[s], 1);
      mbar_init(&C->p_full[s], 4 * WG);
      mbar_init(&C->o_full[s], 1);
      C->nan_tile[s] = -1;
    }
    mbar_init(&C->xbar, 4 * WG);
    mbar_init(&C->done, 1);
    *abort = 0;
    if (p.cut) p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) tmem_alloc(&C->tmem_slot, Sh::TMEM);

  // ---- this CTA's run of tiles
  const int HN = p.H_kv * p.chunks;
  long long total = 0, start = 0, stop_at = 0;
  int n_cta = static_cast<int>(gridDim.x);
  if (p.cut) {
    // prefix of the sequences' tiles over the block's threads; false: past the last one
    long long before = 0, tiles = 0, run = 0;
    auto scan = [&](int base) {
      const int b = base + tid;
      tiles = b < p.B ? span_of(p, b).tiles : 0;
      long long inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      __syncthreads();  // the last sums have been read
      if (lane == 31) C->scan[warp] = inc;
      __syncthreads();
      before = run;
#pragma unroll
      for (int w = 0; w < C_THREADS / 32; ++w) {
        const long long v = C->scan[w];
        if (w < warp) before += v;
        run += v;
      }
      before += inc - tiles;
    };
    for (int base = 0; base < p.B; base += C_THREADS) scan(base);
    total = run * HN;
    n_cta = static_cast<int>(min(static_cast<long long>(gridDim.x), total));  // (every sequence has a tile)
    if (static_cast<int>(blockIdx.x) < n_cta) {
      start = share(total, blockIdx.x, n_cta);
      stop_at = share(total, blockIdx.x + 1, n_cta);
    }
    // the sequence in which the run starts (the scan of a small batch is still at hand)
    if (p.B > C_THREADS) run = 0;
    for (int base = 0; base < p.B; base += C_THREADS) {
      if (p.B > C_THREADS) scan(base);
      if (start < stop_at && tiles > 0 && before * HN <= start && start < (before + tiles) * HN) {
        C->b0 = base + tid;
        C->before0 = before;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C->tmem_slot;

  // n_tiles of this CTA, the first at tile k0 of unit (b0, hn0)
  long long n_tiles = 0;
  int b0 = 0, hn0 = 0, k0 = 0;
  long long u_stop = 0;  // whole units: the run's end
  if (p.cut) {
    n_tiles = stop_at - start;
    if (n_tiles > 0) {
      b0 = C->b0;
      const int t = span_of(p, b0).tiles;
      const long long in_b = start - C->before0 * HN;
      hn0 = static_cast<int>(in_b / t);
      k0 = static_cast<int>(in_b % t);
    }
  } else {
    const long long U = static_cast<long long>(p.B) * HN;
    const long long u0 = U * blockIdx.x / n_cta;
    u_stop = U * (blockIdx.x + 1) / n_cta;
    if (u0 < u_stop) {
      b0 = static_cast<int>(u0 / HN);
      hn0 = static_cast<int>(u0 % HN);
      for (long long u = u0; u < u_stop;) {
        const int b = static_cast<int>(u / HN);
        const long long e = min(u_stop, (b + 1ll) * HN);
        n_tiles += (e - u) * span_of(p, b).tiles;
        u = e;
      }
    }
  }

  if constexpr (Sh::SPLIT) {
    if (warp < 4) regs_dec<Sh::REGS_FEW>();
    else regs_inc<Sh::REGS_MANY>();
  }
  if (warp == 0) {
    // ------------------------------------------------------------ scheduler and TMA
    const int npg = C_TILE / p.page, group = 32 / npg;  // pages of a tile; tiles that the warp looks up at once
    const int gi = lane / npg, pj = lane % npg;
    int b = b0, hn = hn0, k = k0;
    Span sp = n_tiles ? span_of(p, b) : Span{};
    uint32_t slot = 0, phase = 0, any = 0, last_par = 0;
    long long t = 0;
    int seg = 0;
    bool stop = false;
    while (t < n_tiles && !stop) {
      // up to `group` tiles of this unit: lane (gi, pj) looks up page pj of tile k + gi
      const int h = hn / p.chunks, row0 = (hn % p.chunks) * R;
      const int cnt = static_cast<int>(min(static_cast<long long>(min(group, sp.tiles - k)), n_tiles - t));
      const int kk = k + gi;
      const int nth = kk * npg + pj;  // of the sequence's visible pages
      const int pg = nth < sp.sink_pages ? nth : sp.first + nth - sp.sink_pages;
      const int tok = pg * p.page;
      bool there = gi < cnt && nth < sp.pages;
      int id = -1;
      if (there) id = p.table[static_cast<size_t>(b) * p.max_pages + pg];
      there = there && id >= 0 && id < p.n_pages;
      const size_t ph = static_cast<size_t>(there ? id : 0) * p.H_kv + h;
      const float ks = there ? p.ks[ph] : 0.f, vs = there ? p.vs[ph] : 0.f;
      // coordinates past the pool read zeros
      const int y = there ? static_cast<int>(ph * p.page) : static_cast<int>(p.rows_total);
      const uint32_t there_bits = __ballot_sync(0xFFFFFFFFu, there);
      // pages that every row sees whole
      const uint32_t clear_bits = __ballot_sync(
          0xFFFFFFFFu, tok + p.page - 1 <= sp.p_lo && (!p.window || tok > static_cast<long long>(sp.p_hi) - p.window ||
                                                       static_cast<long long>(tok) + p.page <= p.n_sink));
      float vref = vs;
      for (int o = npg >> 1; o; o >>= 1) vref = fmaxf(vref, __shfl_xor_sync(0xFFFFFFFFu, vref, o));
      // the scale's power of two goes into the scores, the rest into the weights
      float rv = vref > 0.f ? vs / vref * 256.f : 0.f;
      const uint32_t rv_bits = __float_as_uint(rv);
      const int e = max(static_cast<int>(rv_bits >> 23) - 135 + ((rv_bits & 0x7FFFFFu) != 0), -C_FAR);
      const float lr = static_cast<float>(e);
      rv *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      for (int i = 0; i < cnt; ++i, ++t) {
        const int ds = static_cast<int>(t % C_ND);
        if (!mbar_wait_warp(&C->d_empty[ds], (static_cast<uint32_t>(t / C_ND) & 1u) ^ 1u, abort, limit)) {
          if (lane == 0) cache_error(p, abort, CERR_DESC);
          stop = true;
          break;
        }
        TileDesc& d = C->desc[ds];
        uint32_t vslot = slot + 1, vphase = phase;
        if (vslot == NS) {
          vslot = 0;
          vphase ^= 1u;
        }
        if (gi == i) {
          d.tok[pj] = tok;
          d.ks[pj] = ks;
          d.rv[pj] = rv;
          d.lr[pj] = lr;
          if (pj == 0) {
            const uint32_t pages = (there_bits >> (gi * npg)) & ((1u << npg) - 1u);
            const bool every = pages == (1u << npg) - 1u && ((clear_bits >> (gi * npg)) & ((1u << npg) - 1u)) == (1u << npg) - 1u;
            const bool first = t == 0 || kk == 0, last = t == n_tiles - 1 || kk == sp.tiles - 1;
            d.flags = (first ? F_FIRST : 0) | (last ? F_LAST : 0) | (every ? 0 : F_MASK);
            d.b = b;
            d.h = h;
            d.row0 = row0;
            d.rows = min(R, p.L * p.G - row0);
            d.vslot = static_cast<int>(vslot);
            d.vparity = static_cast<int>(vphase);
            d.p_lo = sp.p_lo;
            d.p_hi = sp.p_hi;
            d.pages = static_cast<int>(pages);
            d.seg = seg;
            d.left = sp.tiles - 1 - kk;
            d.vref = vref;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->d_full[ds]);
        for (int kv = 0; kv < 2; ++kv) {
          if (!mbar_wait_warp(&C->empty[slot], phase ^ 1u, abort, limit)) {
            if (lane == 0) cache_error(p, abort, CERR_SLOT);
            stop = true;
            break;
          }
          if (!(p.withhold && blockIdx.x == 0 && t == 1 && kv == 0)) {
            if (lane == 0) {
              if (kv == 0) C->k_flags[slot] = d.flags;
              mbar_arrive_expect_tx(&C->full[slot], Sh::SLOT);
            }
            __syncwarp();
            if (gi == i) tma_load_2d(kv_s + slot * Sh::SLOT + pj * p.page * D, kv ? &tm_v : &tm_k, &C->full[slot], 0, y);
            any |= 1u << slot;
            last_par = (last_par & ~(1u << slot)) | (phase << slot);
          }
          if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (stop) break;
      }
      k += cnt;
      if (k == sp.tiles) {
        k = 0;
        seg = 1;
        if (++hn == HN) {
          hn = 0;
          ++b;
          if (b < p.B && t < n_tiles) sp = span_of(p, b);
        }
      }
    }
    __syncwarp();
    // every copy issued has landed before the CTA can exit
    if (lane == 0)
      for (int s = 0; s < NS; ++s)
        if (((any >> s) & 1u) && !mbar_wait_timed(&C->full[s], (last_par >> s) & 1u, limit))
          cache_error(p, abort, CERR_DRAIN);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    // S(t) needs no wait for its TMEM buffer: P(t - 2), which has been waited
    // for, was written after S(t - 2) had been read.  Nor does O(t - 1): a warp
    // writes its part of P(t - 1) after it has read O(t - 3).
    constexpr uint32_t IDESC_S = idesc_f32acc(0, 0, 128, N);
    constexpr uint32_t IDESC_O = idesc_f32acc(0, 0, 128, N) | (1u << 15) | (1u << 16);  // V and P MN-major
    constexpr uint32_t SW = D == 128 ? 2 : 4, ATOM = 8 * D;  // 8 rows of D bytes
    const uint64_t kd = sdesc(smem_u32(kv_s), 16, ATOM, SW), qd = sdesc(smem_u32(q_s), 16, ATOM, SW);
    // With D = 64 the upper half of M reads the next 8-token group (LBO = one
    // atom): lanes 64-127 of O hold nothing of use.
    const uint64_t vd = sdesc(smem_u32(kv_s), ATOM, ATOM, SW), pd = sdesc(smem_u32(p_s), 128, 2048, 0);
    auto await = [&](uint64_t* bar, uint32_t parity, int where) {
      const bool got = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort, limit));
      if (!got && lane == 0) cache_error(p, abort, where);
      return got;
    };
    uint32_t n_unit = 0, slot = 0, phase = 0, vslot = 0, vphase = 0;
    for (long long t = 0; t <= n_tiles; ++t) {
      uint32_t next_v = 0, next_vphase = 0;
      if (t < n_tiles) {
        const uint32_t sb = t & 1;
        if (!await(&C->full[slot], phase, CERR_FULL)) break;
        const int flags = *reinterpret_cast<volatile int*>(&C->k_flags[slot]);
        if (flags & F_FIRST) {
          ++n_unit;
          if (!await(&C->q_full[(n_unit - 1) & 1], ((n_unit - 1) >> 1) & 1u, CERR_Q)) break;
        }
        tc_fence_after();
        const uint64_t k = kd + slot * (Sh::SLOT >> 4), q = qd + ((n_unit - 1) & 1) * (Sh::Q >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) mma_f8(tmem + sb * N, k + kk * 2, q + kk * 2, IDESC_S, kk != 0);
          mma_commit(&C->s_full[sb]);
          mma_commit(&C->empty[slot]);
          if (flags & F_LAST) mma_commit(&C->q_empty[(n_unit - 1) & 1]);
        }
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
        next_v = slot;
        next_vphase = phase;
        if (++slot == NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      if (t > 0) {
        const uint32_t ob = (t - 1) & 1, ph = static_cast<uint32_t>((t - 1) >> 1) & 1u;
        if (!await(&C->full[vslot], vphase, CERR_FULL) || !await(&C->p_full[ob], ph, CERR_P)) break;
        tc_fence_after();
        const uint64_t v = vd + vslot * (Sh::SLOT >> 4), q = pd + ob * (Sh::P >> 4);
        if (elect_one()) {
          // 32 tokens a step
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8(tmem + (2 + ob) * N, v + kk * (2 * D), q + kk * 32, IDESC_O, kk != 0);
          mma_commit(&C->o_full[ob]);
          mma_commit(&C->empty[vslot]);
        }
      }
      vslot = next_v;
      vphase = next_vphase;
    }
    if (elect_one()) {
      mma_commit(&C->done);
      if (!mbar_wait_timed(&C->done, 0, limit)) cache_error(p, abort, CERR_DRAIN);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ queries into e4m3 terms
    uint32_t n_unit = 0;
    for (long long t = 0; t < n_tiles; ++t) {
      const int ds = static_cast<int>(t % C_ND);
      if (!mbar_wait_warp(&C->d_full[ds], static_cast<uint32_t>(t / C_ND) & 1u, abort, limit)) {
        if (lane == 0) cache_error(p, abort, CERR_DESC);
        break;
      }
      const TileDesc& d = C->desc[ds];
      const int flags = d.flags, b = d.b, h = d.h, row0 = d.row0, rows = d.rows;
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->d_empty[ds]);
      if (!(flags & F_FIRST)) continue;
      const uint32_t qb = n_unit & 1;
      if (!mbar_wait_warp(&C->q_empty[qb], ((n_unit >> 1) & 1u) ^ 1u, abort, limit)) {
        if (lane == 0) cache_error(p, abort, CERR_Q);
        break;
      }
      ++n_unit;
      const long long len = tokens_of(p, b);
      // eight lanes a row, four rows at a time, the loads of several steps under way together
      constexpr int EL = D / 8, STEPS = R / 8 < 2 ? 1 : R == 32 ? 4 : 2;  // a lane's dims
      const int sub = lane & 7;
#pragma unroll 1
      for (int r0 = (warp - 2) * 4 + (lane >> 3); r0 - (lane >> 3) < rows; r0 += 8 * STEPS) {
        uint4 raw[STEPS][EL / 8];
        int row_i[STEPS], out_at[STEPS];
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          const int row = row0 + min(r0 + 8 * j, rows - 1), i = row / p.G, g = row - i * p.G;
          row_i[j] = i;
          out_at[j] = (b * p.L + i) * p.H + h * p.G + g;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(out_at[j]) * D + sub * EL) * 2);
#pragma unroll
          for (int e = 0; e < EL / 8; ++e) raw[j][e] = src[e];
        }
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          const int r = r0 + 8 * j;
          float v[EL], amax = 0.f;
#pragma unroll
          for (int e = 0; e < EL / 2; ++e) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(raw[j])[e];
            float2 f;
            if constexpr (HALF) f = __half22float2(*reinterpret_cast<const __half2*>(&w));
            else f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          // 2^x, so that amax / 2^x is in [224, 448]: the exponent as it stands in a float
          const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - ((__float_as_uint(amax) & 0x7FFFFFu) > 0x600000u ? 7 : 8);
          const int exb = min(max(ex, 1), 253);
          const float sc = __uint_as_float(static_cast<uint32_t>(exb) << 23);
          const float inv = __uint_as_float(static_cast<uint32_t>(254 - exb) << 23);
#pragma unroll
          for (int e = 0; e < EL; ++e) v[e] *= inv;
          if (r < rows) {
            // rows of D bytes, 16-byte chunks swizzled within 8-row atoms (R is a
            // multiple of 8: all terms of a row swizzle alike)
            const int byte = sub * EL;
            const int chunk = D == 128 ? (byte >> 4) ^ (r & 7) : (byte >> 4) ^ ((r >> 1) & 3);
            uint8_t* dst = q_s + qb * Sh::Q + r * D + chunk * 16 + (byte & 15);
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              uint32_t c[EL / 4];
#pragma unroll
              for (int e = 0; e < EL / 4; ++e) {
                float(&x)[4] = *reinterpret_cast<float(*)[4]>(v + 4 * e);
                c[e] = e4m3x4(x[0], x[1], x[2], x[3]);
                if (term + 1 < TERMS) take_off(x, c[e]);
              }
              if constexpr (EL == 16) *reinterpret_cast<uint4*>(dst + term * R * D) = make_uint4(c[0], c[1], c[2], c[3]);
              else *reinterpret_cast<uint2*>(dst + term * R * D) = make_uint2(c[0], c[1]);
            }
            if (sub == 0) {
              const long long pos = len - p.L + row_i[j];
              const int ps = static_cast<int>(pos < 0 ? -1 : pos);
              // e4m3 has no infinity: a row that holds one scores NaN
              C->qs[qb][r] = amax <= 3.402823466e38f ? sc * p.scale_log2 : __int_as_float(0x7fc00000);
              C->pos[qb][r] = ps;
              C->low[qb][r] = p.window && p.window <= ps ? ps - p.window : -1;
              C->out[qb][r] = out_at[j];
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read by the MMA
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->q_full[qb]);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int part = (warp - 4) >> 2, quad = warp & 3, c0 = part * HC;  // its rows, and its share of a value row
    const int me = quad * 32 + lane;  // the token of a tile, and the dim of O
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const float ninf = -__int_as_float(0x7f800000);
    const int page_of = me / p.page;
    float m = ninf;  // lane c: running maximum of row c0 + c
    float l[HC], acc[HC];
    float(*col)[HC] = C->col[warp - 4];
    uint32_t n_unit = 0, n_x = 0;

    // the softmax warps meet (bounded)
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->xbar);
      const bool got = mbar_wait_bounded(&C->xbar, n_x & 1u, abort, limit);
      ++n_x;
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) cache_error(p, abort, CERR_X);
        return false;
      }
      return true;
    };
    // the sum of a row's terms
    auto load_terms = [&](uint32_t addr, float (&v)[HC]) {
      float t[TERMS - 1][HC];
      tmem_ld<HC>(addr, v);
#pragma unroll
      for (int i = 1; i < TERMS; ++i) tmem_ld<HC>(addr + i * R, t[i - 1]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 1; i < TERMS; ++i)
#pragma unroll
        for (int c = 0; c < HC; c += 2) {
          const float f = i == 1 ? 1.f / TERM_UP : 1.f / (TERM_UP * TERM_UP);
          const float2 x = fma2(make_float2(t[i - 1][c], t[i - 1][c + 1]), make_float2(f, f), make_float2(v[c], v[c + 1]));
          v[c] = x.x;
          v[c + 1] = x.y;
        }
    };
    // joins tile j's O into the state
    auto join = [&](long long j, int qb) -> bool {
      const uint32_t ob = j & 1, ph = static_cast<uint32_t>(j >> 1) & 1u;
      const bool got = mbar_wait_bounded(&C->o_full[ob], ph, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) cache_error(p, abort, CERR_O);
        return false;
      }
      tc_fence_after();
      float o[HC];
      load_terms(tmem + lanes + (2 + ob) * N + c0, o);
#pragma unroll
      for (int c = 0; c < HC; c += 2) {
        const float2 fa = *reinterpret_cast<const float2*>(&C->fa[ob][c0 + c]), fb = *reinterpret_cast<const float2*>(&C->fb[ob][c0 + c]);
        const float2 x = fma2(make_float2(o[c], o[c + 1]), fb, mul2(make_float2(acc[c], acc[c + 1]), fa));
        acc[c] = x.x;
        acc[c + 1] = x.y;
      }
      if (C->nan_tile[ob] == static_cast<int>(j) && me < D) {
        // a value that is NaN reaches the rows that see its token, in its dim
#pragma unroll 1
        for (int k = 0; k < C_TILE; ++k)
          if ((C->nan_bits[ob][k][me >> 4] >> (me & 15)) & 1u) {
            const int tok = C->nan_tok[ob][k / p.page] + k % p.page;
#pragma unroll
            for (int c = 0; c < HC; ++c)
              if (tok <= C->pos[qb][c0 + c] && (tok > C->low[qb][c0 + c] || tok < p.n_sink))
                acc[c] = __int_as_float(0x7fc00000);
          }
      }
      return true;
    };

    for (long long t = 0; t < n_tiles; ++t) {
      const int ds = static_cast<int>(t % C_ND);
      bool got = mbar_wait_bounded(&C->d_full[ds], static_cast<uint32_t>(t / C_ND) & 1u, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) cache_error(p, abort, CERR_DESC);
        break;
      }
      const TileDesc& d = C->desc[ds];
      const int flags = d.flags, tok = d.tok[page_of] + me % p.page;
      const float ks = d.ks[page_of], rv = d.rv[page_of], lr = d.lr[page_of], vref = d.vref;
      if (flags & F_FIRST) {
        ++n_unit;
        got = mbar_wait_bounded(&C->q_full[(n_unit - 1) & 1], ((n_unit - 1) >> 1) & 1u, abort, limit);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          if (lane == 0) cache_error(p, abort, CERR_Q);
          break;
        }
        m = ninf;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          l[c] = 0.f;
          acc[c] = 0.f;
        }
      }
      const int qb = (n_unit - 1) & 1;
      const uint32_t sb = t & 1, ph = static_cast<uint32_t>(t >> 1) & 1u;
      got = mbar_wait_bounded(&C->s_full[sb], ph, abort, limit);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        if (lane == 0) cache_error(p, abort, CERR_S);
        break;
      }
      tc_fence_after();
      float s[HC];
      load_terms(tmem + lanes + sb * N + c0, s);
      // log2 of weight times value scale, before the mask: a row's own scale may be 0
#pragma unroll
      for (int c = 0; c < HC; c += 2) {
        const float2 q2 = *reinterpret_cast<const float2*>(&C->qs[qb][c0 + c]);
        const float2 x = fma2(mul2(make_float2(s[c], s[c + 1]), make_float2(ks, ks)), q2, make_float2(lr, lr));
        s[c] = x.x;
        s[c + 1] = x.y;
      }
      if (flags & F_MASK) {
        const bool there = (d.pages >> page_of) & 1;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          const bool see = there && tok <= C->pos[qb][c0 + c] && (tok > C->low[qb][c0 + c] || tok < p.n_sink);
          s[c] = see ? s[c] : ninf;
        }
      }
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        const float w = warp_max(s[c]);
        if (lane == 0) C->red[sb][c0 + c][quad] = w;
      }
      if (!meet()) break;
      // a lane a row: the tile's maximum, the state's factor and the tile's (one of them is 1)
      if (lane < HC) {
        const float4 r = *reinterpret_cast<const float4*>(C->red[sb][c0 + lane]);
        const float mt = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w));
        const float f = mt == m ? 1.f : ex2(-fabsf(m - mt));
        const bool up = mt > m;
        const float fa = up ? f : 1.f, fb = up ? 1.f : f;
        m = fmaxf(m, mt);
        col[0][lane] = mt == ninf ? 0.f : -mt;
        col[1][lane] = fa;
        col[2][lane] = fb;
        if (quad == 0) {
          C->fa[sb][c0 + lane] = fa;
          C->fb[sb][c0 + lane] = fb * vref * (1.f / 256.f);
        }
      }
      __syncwarp();
      const float ilr = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(lr)) << 23);  // 2^-lr: the sum is of weights alone
      // P in half precision (11 bits), then its terms, the row of a token
      // contiguous along N in groups of 16
#pragma unroll
      for (int c = 0; c < HC; c += 4) {
        const float4 mt = *reinterpret_cast<const float4*>(&col[0][c]), fa = *reinterpret_cast<const float4*>(&col[1][c]),
                     fb = *reinterpret_cast<const float4*>(&col[2][c]);
        // two rows at once
        auto pair = [&](int i, float2 m2, float2 a2, float2 b2) -> __half2 {
          float2 e = add2(make_float2(s[c + i], s[c + i + 1]), m2);
          e = make_float2(ex2(e.x), ex2(e.y));
          const float2 n = fma2(mul2(e, make_float2(ilr, ilr)), b2, mul2(make_float2(l[c + i], l[c + i + 1]), a2));
          l[c + i] = n.x;
          l[c + i + 1] = n.y;
          const float2 v = mul2(e, make_float2(rv, rv));
          return __floats2half2_rn(v.x, v.y);
        };
        __half2 x = pair(0, make_float2(mt.x, mt.y), make_float2(fa.x, fa.y), make_float2(fb.x, fb.y));
        __half2 y = pair(2, make_float2(mt.z, mt.w), make_float2(fa.z, fa.w), make_float2(fb.z, fb.w));
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const uint32_t qx = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
          const uint32_t qy = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(y), __NV_SATFINITE, __NV_E4M3);
          const int at = term * R + c0 + c;
          *reinterpret_cast<uint32_t*>(p_s + sb * Sh::P + (at >> 4) * 2048 + me * 16 + (at & 15)) = qx | (qy << 16);
          if (term + 1 < TERMS) {
            const __half2 up = __float2half2_rn(TERM_UP), dn = __float2half2_rn(-TERM_UP);  // exact: what is left has fewer bits
            x = __hfma2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(qx), __NV_E4M3)), dn, __hmul2(x, up));
            y = __hfma2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(qy), __NV_E4M3)), dn, __hmul2(y, up));
          }
        }
      }
      if (flags & F_MASK) {
        // Values of tokens that no row sees may hold anything; 0 * NaN would
        // reach the sums.  They are cleared; of tokens that some rows see, NaN
        // codes are cleared and noted.
        const bool any = tok <= d.p_hi && (!p.window || tok > static_cast<long long>(d.p_lo) - p.window || tok < p.n_sink);
        const bool all = tok <= d.p_lo && (!p.window || tok > static_cast<long long>(d.p_hi) - p.window || tok < p.n_sink);
        got = mbar_wait_bounded(&C->full[d.vslot], d.vparity, abort, limit);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          if (lane == 0) cache_error(p, abort, CERR_FULL);
          break;
        }
        // each warpgroup takes a share of the row's chunks; the lanes begin at
        // different ones, so that they meet no bank twice
        constexpr int CH = D / 16 / WG;
        uint4* row = reinterpret_cast<uint4*>(kv_s + d.vslot * Sh::SLOT + me * D);
        uint32_t found = 0;
        if (!any) {
          // (pages that are not there arrived as zeros)
          if ((d.pages >> page_of) & 1) {
#pragma unroll
            for (int i = 0; i < CH; ++i) row[part * CH + ((i + me) & (CH - 1))] = make_uint4(0, 0, 0, 0);
          }
        } else if (!all) {
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            // chunk i of the share, wherever the swizzle put it
            const int chunk = part * CH + i;
            const int at = D == 128 ? chunk ^ (me & 7) : chunk ^ ((me >> 1) & 3);
            const uint4 x = row[at];
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, hit = 0, bits = 0;
            // a code of ones but for its sign carries into the sign's place
#pragma unroll
            for (int q = 0; q < 4; ++q) hit |= ((w[q] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            if (hit) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (((w[q] >> (8 * e)) & 0x7Fu) == 0x7Fu) {
                    bits |= 1u << (q * 4 + e);
                    w[q] &= ~(0xFFu << (8 * e));
                  }
              row[at] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            found |= bits;
            if (p.L > 1) C->nan_bits[sb][me][chunk] = static_cast<uint16_t>(bits);
          }
        }
        if (p.L > 1) {
          if (any == all) {
#pragma unroll
            for (int i = 0; i < CH; ++i) C->nan_bits[sb][me][part * CH + i] = 0;
          }
          if (me % p.page == 0) C->nan_tok[sb][page_of] = tok;
          if (found) C->nan_tile[sb] = static_cast<int>(t);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // P (and cleared values) are read by the MMA
      tc_fence_before();                                             // S and the O before have been read
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->p_full[sb]);
      if (!(flags & F_FIRST) && !join(t - 1, qb)) break;
      if (flags & F_LAST) {
        // the sums over the tokens, then the unit's rows or a partial result
        if (!meet()) break;  // ab of this tile is visible
        if (!join(t, qb)) break;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          float v = l[c];
#pragma unroll
          for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
          if (lane == 0) C->sum[c0 + c][quad] = v;
        }
        if (!meet()) break;
        const int b = d.b, h = d.h, row0 = d.row0, rows = d.rows;
        const bool begins = d.seg || k0 == 0, whole = begins && d.left == 0;
        float* left = p.part + (static_cast<size_t>(blockIdx.x) * 2 + d.seg) * R * (D + 2);
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          const int r = c0 + c;
          if (r < rows && me < D) {
            const float4 v = *reinterpret_cast<const float4*>(C->sum[r]);
            const float sum = (v.x + v.y) + (v.z + v.w);
            if (whole) {
              const size_t at = static_cast<size_t>(C->out[qb][r]) * D + me;
              const float o = acc[c] * (sum == 0.f ? 0.f : 1.f / sum);
              if constexpr (HALF) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(o);
              else reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
            } else {
              left[r * D + me] = acc[c];
            }
          }
        }
        if (quad == 0 && lane < HC && c0 + lane < rows) {
          const int r = c0 + lane;
          const float4 v = *reinterpret_cast<const float4*>(C->sum[r]);
          const float sum = (v.x + v.y) + (v.z + v.w);
          if (!whole) {
            left[R * D + r] = m;
            left[R * D + R + r] = sum;
          } else if (p.lse) {
            p.lse[C->out[qb][r]] = sum == 0.f ? ninf : (m + log2f(sum)) * LN2;
          }
        }
        if (begins && !whole && me == 0 && part == 0) {
          // the unit goes on in the next CTAs: the joining kernel starts from here
          const long long end = stop_at - 1 + d.left;  // its last tile; CTA c holds tiles from c * total / n_cta on
          const int last_cta = static_cast<int>(((end + 1) * n_cta - 1) / total);
          p.meta[blockIdx.x] = make_int4(b, h * p.chunks + row0 / R, last_cta - static_cast<int>(blockIdx.x) + 1, d.seg);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&C->q_empty[qb]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&C->d_empty[ds]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Sh::TMEM);
}

// Joins the partial results of the units that begin in CTA c and go on: a
// block per (c, row), a thread per dim.
template <int D, int R, bool HALF>
__global__ void __launch_bounds__(128) cache_join_kernel(const CacheParams p) {
  __shared__ float w[C_MAX_CTAS];
  __shared__ float red[4];
  const int4 u = p.meta[blockIdx.x];
  if (u.x < 0) return;
  const int b = u.x, h = u.y / p.chunks, row0 = (u.y % p.chunks) * R, n = u.z, r = blockIdx.y;
  if (row0 + r >= p.L * p.G) return;
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr size_t SLOT = static_cast<size_t>(R) * (D + 2);
  const float* first = p.part + (static_cast<size_t>(blockIdx.x) * 2 + u.w) * SLOT;
  const float* rest = p.part + static_cast<size_t>(blockIdx.x) * 2 * SLOT;  // CTA c + s, slot 0
  float mx = -__int_as_float(0x7f800000);
  for (int s = tid; s < n; s += 128) {
    const float m = (s ? rest + 2 * s * SLOT : first)[R * D + r];
    w[s] = m;
    mx = fmaxf(mx, m);
  }
  mx = warp_max(mx);
  if (lane == 0) red[tid >> 5] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  float sum = 0.f;
  for (int s = tid; s < n; s += 128) {
    const float f = w[s] == mx ? 1.f : ex2(w[s] - mx);
    w[s] = f;
    sum = fmaf(f, (s ? rest + 2 * s * SLOT : first)[R * D + R + r], sum);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) red[tid >> 5] = sum;
  __syncthreads();
  sum = (red[0] + red[1]) + (red[2] + red[3]);
  const int row = row0 + r, i = row / p.G, g = row % p.G;
  const size_t at = (static_cast<size_t>(b) * p.L + i) * p.H + h * p.G + g;
  if (tid < D) {
    float acc = w[0] * first[r * D + tid];
#pragma unroll 8
    for (int s = 1; s < n; ++s) acc = fmaf(w[s], rest[2 * s * SLOT + r * D + tid], acc);
    const float o = acc * (sum == 0.f ? 0.f : 1.f / sum);
    if constexpr (HALF) reinterpret_cast<__half*>(p.out)[at * D + tid] = __float2half_rn(o);
    else reinterpret_cast<__nv_bfloat16*>(p.out)[at * D + tid] = __float2bfloat16_rn(o);
  }
  if (tid == 0 && p.lse) p.lse[at] = sum == 0.f ? -__int_as_float(0x7f800000) : (mx + log2f(sum)) * LN2;
}

template <int D, int R, bool HALF>
si_status launch_cache(CacheParams& p, const si_cache* c, int n_sm, const si_options* opt, cudaStream_t stream) {
  using Sh = CacheShape<D, R, HALF>;
  CUtensorMap tm_k, tm_v;
  p.rows_total = static_cast<long long>(c->n_pages) * c->H_kv * c->page;
  const uint64_t dims[2] = {D, static_cast<uint64_t>(p.rows_total)}, stride = D;
  const uint32_t box[2] = {D, static_cast<uint32_t>(c->page)};
  si_status st = encode_tmap(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c->k_pages, dims, &stride, box, D);
  if (st == SI_OK) st = encode_tmap(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c->v_pages, dims, &stride, box, D);
  if (st != SI_OK) return st;
  if constexpr (Sh::SPLIT) {
    // the register split has to fit the registers of the launch, a property of
    // the build: its warps would wait for the rest forever
    static std::atomic<int> built{0};
    int regs = built.load();
    if (regs == 0) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, cache_attention_kernel<D, R, HALF>);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(cache_attention_kernel)");
      built.store(regs = a.numRegs);
    }
    if (regs < Sh::REGS) return fail(SI_ERR_CUDA, "cache_attention_kernel was built with %d registers a thread", regs);
  }
  p.chunks = (p.L * p.G + R - 1) / R;
  // the tiles that a sequence can have at most
  long long pages = p.max_pages;
  if (p.window)
    pages = std::min(pages, (static_cast<long long>(p.window) + p.L - 2) / p.page + 2 +
                                (static_cast<long long>(p.n_sink) + p.page - 1) / p.page);
  const long long tiles = (pages * p.page + C_TILE - 1) / C_TILE;
  p.cut = tiles > C_WHOLE;
  const long long units = static_cast<long long>(p.B) * p.H_kv * p.chunks;
  const long long most = std::min(n_sm * Sh::CTAS, C_MAX_CTAS);
  const int grid = static_cast<int>(p.cut ? most : std::min(units, most));
  void* own = nullptr;
  if (p.cut) {
    const size_t need = static_cast<size_t>(grid) * (sizeof(int4) + 2 * sizeof(float) * R * (D + 2));
    void* ws = opt && opt->workspace && opt->workspace_bytes >= need && aligned(opt->workspace, 16) ? opt->workspace : nullptr;
    if (!ws) {
      st = scratch_alloc(&own, need, stream, "cache attention partial results");
      if (st != SI_OK) return st;
      ws = own;
    }
    p.meta = static_cast<int4*>(ws);
    p.part = reinterpret_cast<float*>(p.meta + grid);
  }
  const size_t smem = 1024 + Sh::SLOTS * Sh::SLOT + 2 * (Sh::Q + Sh::P) + sizeof(CacheCtrl<D, R, HALF>);
  static_assert(1024 + Sh::SLOTS * Sh::SLOT + 2 * (Sh::Q + Sh::P) + sizeof(CacheCtrl<D, R, HALF>) <=
                    (Sh::CTAS == 2 ? 113 * 1024 : 227 * 1024), "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(cache_attention_kernel<D, R, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e == cudaSuccess) {
    cache_attention_kernel<D, R, HALF><<<grid, Sh::THREADS, smem, stream>>>(tm_k, tm_v, p);
    if (p.cut) cache_join_kernel<D, R, HALF><<<dim3(grid, std::min(R, p.L * p.G)), 128, 0, stream>>>(p);
    e = cudaGetLastError();
  }
  if (own) cudaFreeAsync(own, stream);
  return e == cudaSuccess ? SI_OK : cuda_fail(e, "cache_attention_kernel launch");
}

template <int D, bool HALF>
si_status launch_cache_rows(CacheParams& p, const si_cache* c, int n_sm, const si_options* opt, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.L) * p.G;
  if (rows <= 8) return launch_cache<D, 8, HALF>(p, c, n_sm, opt, stream);
  if (rows <= 16) return launch_cache<D, 16, HALF>(p, c, n_sm, opt, stream);
  // (three terms of 64 rows do not fit into tensor memory)
  if (rows <= 32 || HALF) return launch_cache<D, 32, HALF>(p, c, n_sm, opt, stream);
  return launch_cache<D, HALF ? 32 : 64, HALF>(p, c, n_sm, opt, stream);
}

}  // namespace

si_status check_attention(const void* q, const void* out, const float* lse, int B, int L, int H, int H_kv, int D,
                          float scale, int dtype, int n_sink) {
  if (!q || !out) return fail(SI_ERR_INVALID_ARGUMENT, "q and out must be non-null device pointers");
  if (B < 1 || L < 1 || H < 1 || H_kv < 1) return fail(SI_ERR_INVALID_ARGUMENT, "B, the length, H and H_kv must be >= 1");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return fail(SI_ERR_INVALID_ARGUMENT, "q and out must be 16-byte aligned; lse 4-byte aligned");
  if (!(scale >= 0.f) || std::isinf(scale)) return fail(SI_ERR_INVALID_ARGUMENT, "scale must be finite and >= 0 (0 = 1/sqrt(D))");
  if (n_sink < 0) return fail(SI_ERR_INVALID_ARGUMENT, "n_sink must be >= 0 (got %d)", n_sink);
  if (D != 64 && D != 128) return fail(SI_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", D);
  if (dtype != SI_DTYPE_BF16 && dtype != SI_DTYPE_FP16)
    return fail(SI_ERR_UNSUPPORTED, "q, k and v are bf16 or fp16 (dtype %d)", dtype);
  if (H % H_kv != 0 || H / H_kv > 128)
    return fail(SI_ERR_UNSUPPORTED, "H must be a multiple of H_kv, at most 128 times it (got %d, %d)", H, H_kv);
  if (static_cast<double>(B) * L * H > 2147483647.0)
    return fail(SI_ERR_UNSUPPORTED, "the query rows (B * length * H) must fit in 31 bits");
  return SI_OK;
}


}  // namespace si

using namespace si;

extern "C" {

si_status si_cache_attention(const void* q, const si_cache* c, const int32_t* table, const int32_t* lens, int B, int L,
                             int H, int max_pages, int window, int n_sink, float scale, int dtype, void* out,
                             float* lse, void* stream, const si_options* opt) {
  si_status st = check_cache(c);
  if (st != SI_OK) return st;
  if (!table || !lens) return fail(SI_ERR_INVALID_ARGUMENT, "table and lens must be non-null device pointers");
  st = check_attention(q, out, lse, B, L, H, c->H_kv, c->D, scale, dtype, n_sink);
  if (st != SI_OK) return st;
  if (max_pages < 1 || window < 0) return fail(SI_ERR_INVALID_ARGUMENT, "max_pages must be >= 1 and window >= 0");
  if (!aligned(table, 4) || !aligned(lens, 4))
    return fail(SI_ERR_INVALID_ARGUMENT, "table and lens must be 4-byte aligned");
  int* err = nullptr;
  st = error_word(opt, &err);
  if (st != SI_OK) return st;
  if (static_cast<long long>(max_pages) * c->page > 0x7FFFFFFFll - 2 * C_TILE)
    return fail(SI_ERR_UNSUPPORTED, "max_pages * page must stay below 2^31 - %d", 2 * C_TILE);
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  CacheParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.table = table;
  p.lens = lens;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.err = err;
  p.B = B;
  p.L = L;
  p.H = H;
  p.H_kv = c->H_kv;
  p.G = H / c->H_kv;
  p.page = c->page;
  p.max_pages = max_pages;
  p.n_pages = c->n_pages;
  p.window = window;
  p.n_sink = n_sink;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(c->D))) * LOG2E;
  p.wait_limit_ns = kDefaultWaitLimitNs;
  p.withhold = take_withheld_load(&p.wait_limit_ns);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = dtype == SI_DTYPE_FP16;
  if (c->D == 128) return half ? launch_cache_rows<128, true>(p, c, n_sm, opt, s) : launch_cache_rows<128, false>(p, c, n_sm, opt, s);
  return half ? launch_cache_rows<64, true>(p, c, n_sm, opt, s) : launch_cache_rows<64, false>(p, c, n_sm, opt, s);
}

size_t si_cache_attention_workspace_size(int D) {
  // the largest of any number of rows: 64 rows and one CTA an SM
  int dev = 0, n_sm = 0;
  if (D < 1 || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return static_cast<size_t>(std::min(2 * n_sm, C_MAX_CTAS)) * sizeof(int4) +
         static_cast<size_t>(std::min(n_sm, C_MAX_CTAS)) * 2 * sizeof(float) * 64 * (static_cast<size_t>(D) + 2);
}

}  // extern "C"
