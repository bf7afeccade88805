// One decode step of attention over a paged 8-bit KV cache, sm_100a: bf16
// queries, e4m3 codes with a power-of-two scale per (position, K/V head), as
// fa_cache_append writes them.
//
//     x_j = scale log2(e) <q, k_j>,  p_j = 2^(x_j - m),  O = sum p_j v_j / sum p_j
// over the positions j of the sequence (or of its window), with the running
// reference m and the rescaling of "Flash Attention" (karlkratz.de), "Tiling".
//
// Bound by the codes' bytes: each K/V row is read once per (sequence, K/V head)
// and serves H / Hkv query heads.  What the kernel is built around:
//   * all tiles (128 positions) of all sequences form one list, cut into as many
//     equal ranges as the GPU holds CTAs per head group, so lengths and batch size
//     leave no SM idle.  The CTAs of one range's K/V heads are neighbours: they walk
//     the same pages, whose rows of different heads are neighbours in memory.  A
//     sequence that crosses a range's border leaves fp32 partials for the join;
//   * a producer warp looks up a tile's pages, a lane each, and issues one TMA box
//     per page and tensor and one bulk copy of the page's scale bytes; it runs ahead
//     over sequence borders;
//   * four consumer warps take 32 positions of a tile each, on warp-level MMAs with
//     the POSITIONS as the 16 rows of S^T = K Q^T and the features as the rows of O^T
//     = V^T P^T, so that up to 8 query heads fill the 8 columns and none of the tensor
//     work is padding at H / Hkv = 8;
//   * codes become f16 pairs with the conversion instruction, two per word of four
//     codes, and m16n8k16 multiplies f16: every e4m3 value is exact in it, and P keeps 11
//     bits.  For K any order of the features will do, as long as Q has the same: a lane
//     reads 16 codes of a row at once;
//   * for V^T, ldmatrix.trans on pairs of features hands a lane the codes (f, j), (f +
//     1, j), (f, j + 1), (f + 1, j + 1); swapping the middle two gives the pairs of rows
//     f and f + 1: 8-bit data is transposed by the 16-bit instruction;
//   * P goes from the accumulator layout to the operand layout with movmatrix.
// Rounding: q is scaled by a power of two per head so that its largest element is in
// [2^7, 2^8), exact in f16 down to 2^-24 of it.  P times the V scales is rounded to
// f16, with a power of two near the V scales taken out, like m; where the scales that a warp
// meets are too far apart for f16 it is split into two bf16 terms.  Sums, maxima and
// statistics are fp32.
//
// Measured on a B200 (GPU time): 64 sequences of 512 to 8192 positions, 64 heads on 8,
// d = 128, 16-token pages, 632 MB: 101 us, 6.25 TB/s (95% of a copy's 6.57); one
// sequence of 100000, 206 MB: 40 us, of which 8 us are the start, the last merge and the
// join.  Beyond 8 heads a K/V head, and for d = 64, the consumers' latency and not the
// memory bounds it (64 heads on 4: 67 us for 290 MB; with Q's fragments in registers the
// two blocks of positions had to go one after the other: 77 us).  The two bf16 terms: 115 us
// for the 100 of the 64 sequences where each begins with a V row of zeros (one warp in
// four walks its sequences that way), 70 for 61 at d = 64.  What did not pay:
//   * a grid of (sequence, chunk) with two CTAs per SM, codes converted with integer
//     shifts (7 operations a word): 161 us;
//   * e4m3 operands for S^T with m16n8k32 and q split in two: 129 us (the instruction is
//     converted and multiplied as f16 on this GPU, at four times the instructions);
//   * S^T on tcgen05 into tensor memory, a lane per position for the softmax: 108 us, 7.5
//     instead of 6.4 us for a short sequence, 28.3 instead of 27.5 us for one head a K/V
//     head: the product's round trip through barriers and tensor memory costs a tile
//     more than the conversions of K do;
//   * three CTAs per SM with more than 8 heads a K/V head: spilled registers, 122 us;
//   * two accumulator chains for S^T: the same time; ranges cut to 32 positions instead
//     of whole tiles: 1% slower (a tile that a border cuts is walked twice).
//
// A row whose scale byte is 255 (NaN) makes the heads that see it NaN.  A
// sequence with no position gets O = 0, LSE = -inf, and so does one with a
// length outside its table row or a page index outside the pool, which is
// reported (kDevBadInput); page 0 is read in such a page's place.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kConsumers = 4;
constexpr int kWarpKeys = kTileKeys / kConsumers;
constexpr int kThreads = (kConsumers + 1) * 32;
// The reference m is only moved when a score passes it by more than kLazy (log2
// units): p <= 2^kLazy, and P * 2^(15 - kLazy) stays inside f16.
constexpr float kLazy = 6.f;
constexpr int kPShift = 9;
// Scores are held with q's power of two still in them, up to 2^24 times K's scale (up to 2^120): another
// 2^-kKShift keeps the largest finite, and the smallest (K's scale 2^-126) above fp32's subnormals' end.
constexpr int kKShift = 20;
// P times the V scales goes to f16, in a unit of 2^kVUp times the largest V scale of its first 32 rows,
// as long as every scale that a warp meets in a sequence is at most that unit and at least 2^-kVSpan
// of it.  What a product loses is then below 2^(kVSpan - 34) of its own V row, however small that
// is beside the others.  From the first scale outside on the products are sums of two bf16 terms,
// which have fp32's range, and the unit follows the largest scale (up to 2^32, so that the range serves
// both ways).  A first token with V rows some 2^-7 of the others' stays inside.
constexpr int kVUp = 4;
constexpr int kVSpan = 14;
constexpr int kVCap = 127 + 32;
constexpr int kBarBytes = 192;

template <int D, int NT>
struct Cfg8 {
  static constexpr int kTileBytes = kTileKeys * D;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kCtas = NT == 2 ? 2 : D == 128 ? 3 : 4;   // per SM
  static constexpr int kStages = NT == 2 ? (D == 128 ? 3 : 4) : (D == 128 ? 2 : 3);
  static constexpr bool kSharedQ = NT == 2;                      // Q's fragments in shared memory (registers)
  static constexpr int kRounds = NT == 1 ? 2 : D / 32;                  // the merge goes through in slices of the features
  static constexpr int kSlice = D / kRounds;
  static constexpr int kORow = kSlice + 4;
  static constexpr int kOffScale = kStages * kStageBytes;        // [stage][256] scale bytes
  static constexpr int kOffMerge = kOffScale + kStages * 2 * kTileKeys;
  static constexpr int kOffML = kOffMerge + kConsumers * 8 * NT * kORow * 4;  // [2][4 warps][16 heads] reference, sum
  static constexpr int kOffBar = kOffML + 2 * kConsumers * 16 * 4;
  static constexpr int kSmemBytes = kOffBar + kBarBytes;
  static_assert(kCtas * (kSmemBytes + 1024) <= 227 * 1024, "CTAs per SM");
  static_assert(kStages <= 4, "barrier block");
  static_assert(!kSharedQ || NT * (D / 16) * 256 <= kConsumers * 8 * NT * kORow * 4, "Q fits in the merge's place");
};

struct Bars8 {
  uint64_t full[4], empty[4];
  int bad[4];   // the stage's tile has a page outside the pool
  int abort;
  int first_b, first_off;  // where this CTA's range begins
  int sums[kConsumers + 1];
  int rows[16];  // pool rows of the tile's boxes
};
static_assert(sizeof(Bars8) <= kBarBytes, "barrier block");

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// one lane of the converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an f16 pair that holds e4m3 values as a bf16 pair (exact)
__device__ __forceinline__ uint32_t bf16_of_f16(uint32_t x) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return pack_bf16x2(v.x, v.y);
}
// codes 0, 2 and codes 1, 3 of a word as f16 pairs
__device__ __forceinline__ void f16_pairs(uint32_t w, uint32_t& even, uint32_t& odd) {
  asm("{\n\t.reg .b32 p;\n\t.reg .b16 lo, hi;\n\t"
      "prmt.b32 p, %2, 0, 0x3120;\n\t"
      "mov.b32 {lo, hi}, p;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(even), "=r"(odd)
      : "r"(w));
}
// codes 0, 1 and codes 2, 3
__device__ __forceinline__ void f16_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

// the same, and whether any thread passes true
__device__ __forceinline__ bool any_consumer(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(kConsumers * 32)
      : "memory");
  return r != 0;
}

// tile row that fragment row g (0..7) stands for: with 128-byte rows, neighbouring
// fragment rows sit 4 rows apart, so the 8 lanes of a 128-bit shared-memory phase
// (two fragment rows, four 16-byte units each) hit 8 different units of the
// swizzled line; with 64-byte rows two neighbouring rows fill a line already
template <int D>
__device__ __forceinline__ int key_of(int g) {
  return D == 128 ? (g >> 1) | ((g & 1) << 2) : g;
}
// byte offset of 16-byte unit u of tile row r (TMA's 128-byte swizzle; 64-byte for d = 64)
template <int D>
__device__ __forceinline__ uint32_t unit_off(int r, int u) {
  return D == 128 ? static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4))
                  : static_cast<uint32_t>(r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Bounded wait.  Unlike wait_bar it keeps no record per launch: a launch that a
// captured graph replays has one epoch, and a replay after one that gave up has to
// run as any other.
__device__ __forceinline__ bool wait_ring(uint64_t* bar, uint32_t parity, Bars8* bars, const DevCtl& ctl, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* gave_up = &bars->abort;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 15) == 0) {
      if (*gave_up) return false;
      if (globaltimer_ns() - t0 > ctl.limit_ns) {
        *gave_up = 1;
        atomicCAS(ctl.status, 0, kDevTimeout | site);
        return false;
      }
    }
  }
}

// The visible part of a sequence: positions [lo, len), in tiles from base on.
struct Seq {
  int len, lo, base, tiles;
};
__device__ __forceinline__ Seq sequence(const Decode8Args& a, int b) {
  Seq s;
  s.len = a.seqlens[b];
  if (s.len < 0 || s.len > a.max_pages * a.page_size) s.len = 0;  // max_pages * page_size <= 2^30 (host check)
  s.lo = a.window < 0 ? 0 : max(0, s.len - 1 - a.window);
  s.base = s.lo & ~(kTileKeys - 1);
  s.tiles = (s.len - s.base + kTileKeys - 1) / kTileKeys;
  return s;
}

// This CTA's walk: up to `left` tiles from tile `off` of sequence b on, sequence by sequence.
struct Walk {
  int b, off, left;
  Seq s;
  int n;  // tiles of the current segment
  __device__ __forceinline__ bool next(const Decode8Args& a) {  // the segment at (b, off); false at the end
    while (left > 0) {
      s = sequence(a, b);
      n = min(s.tiles - off, left);
      if (n > 0) return true;
      ++b;
      off = 0;
    }
    return false;
  }
  __device__ __forceinline__ void done() {
    left -= n;
    ++b;
    off = 0;
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg8<D, NT>::kCtas)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const Decode8Args a, const DevCtl ctl) {
  using C = Cfg8<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicCAS(ctl.status, 0, kDevTimeout | 0xC4);
    return;
  }
  Bars8* bars = reinterpret_cast<Bars8*>(smem + C::kOffBar);
  const int warp = warp_id();
  const int lane = lane_id();
  const int hkv = blockIdx.x / a.hgroups;
  const int hg = blockIdx.x % a.hgroups;
  const int G = a.H / a.Hkv;
  const int h0 = hkv * G + hg * (8 * NT);
  const int gv = min(8 * NT, G - hg * (8 * NT));
  const int P = a.page_size;

  if (threadIdx.x == 0) {
    bars->abort = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], kConsumers);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  wait_for_previous_kernel();
  // ---- where this CTA's range of tiles begins ----
  Walk walk;
  const int range = blockIdx.y;
  if (a.ranges == 0) {  // one sequence per CTA
    walk.b = range;
    walk.off = 0;
    walk.left = sequence(a, range).tiles;
    __syncthreads();
  } else {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += sequence(a, b).tiles;
    int cum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, cum, o);
      if (lane >= o) cum += x;
    }
    if (lane == 31) bars->sums[warp] = cum;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i <= kConsumers; ++i) {
      if (i < warp) cum += bars->sums[i];
      total += bars->sums[i];
    }
    cum -= mine;  // tiles before this thread's sequences
    const int len = max(1, (total + a.ranges - 1) / a.ranges);
    const long long begin = static_cast<long long>(range) * len;
    walk.left = static_cast<int>(max(0LL, min(static_cast<long long>(len), total - begin)));
    if (begin >= cum && begin < cum + mine) {  // one thread, if the range is not empty
      int b = b0, t = sequence(a, b).tiles;
      while (begin >= cum + t) {
        cum += t;
        t = sequence(a, ++b).tiles;
      }
      bars->first_b = b;
      bars->first_off = static_cast<int>(begin) - cum;
      if (blockIdx.x == 0) a.borders[range] = make_int4(b, cum, t, len);
    }
    if (threadIdx.x == 0 && blockIdx.x == 0 && walk.left == 0) a.borders[range] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    walk.b = bars->first_b;
    walk.off = bars->first_off;
  }
  const int R = min(P, kTileKeys);  // positions per box

  if (warp == kConsumers) {
    // ===================== producer warp: lane i looks up the page of box i of a tile =====================
    int issued = 0;
    bool going = true;
    while (going && walk.next(a)) {
      const int* table = a.block_table + static_cast<size_t>(walk.b) * a.max_pages;
      const int kbeg = walk.s.base + walk.off * kTileKeys, kend = walk.s.len, lo = walk.s.lo;
      auto page_of = [&](int t) {  // this lane's page of tile t (nothing is read outside [lo, kend))
        const int j = kbeg + t * kTileKeys + lane * R;
        return (lane * R < kTileKeys && j < kend && j + R > lo) ? table[j / P] : 0;
      };
      int next = page_of(0);
      for (int t = 0; t < walk.n; ++t) {
        const int st = issued % C::kStages;
        int page = next;
        if (t + 1 < walk.n) next = page_of(t + 1);
        const bool free = issued < C::kStages ||
                          wait_ring(&bars->empty[st], ((issued / C::kStages) - 1) & 1, bars, ctl, 0xC5);
        if (!__all_sync(0xffffffffu, free)) {
          going = false;
          break;
        }
        const int key0 = kbeg + t * kTileKeys;
        const int nbox = (min(kTileKeys, kend - key0) + R - 1) / R;
        const int b0 = max(0, lo - key0) / R;  // boxes wholly before the window are left out
        const bool mine = lane >= b0 && lane < nbox;
        const bool bad = mine && (page < 0 || page >= a.num_pages);
        if (bad) {
          atomicCAS(ctl.status, 0, kDevBadInput | 0xD2);
          page = 0;
        }
        const bool any_bad = __any_sync(0xffffffffu, bad);
        if (mine) bars->rows[lane] = page * P + ((key0 + lane * R) & (P - 1));
        __syncwarp();
        if (elect_one()) {
          uint64_t* full = &bars->full[st];
          bars->bad[st] = any_bad ? 1 : 0;  // before the arrival, which releases it
          mbar_arrive_expect_tx(full, static_cast<uint32_t>((nbox - b0) * R * (2 * D + 2)));
          uint8_t* ks = smem + st * C::kStageBytes;
          uint8_t* sc = smem + C::kOffScale + st * 2 * kTileKeys;
          for (int i = b0; i < nbox; ++i) {
            const int row = bars->rows[i];
            tma_load_2d(ks + i * R * D, &tmK, full, hkv * D, row);
            tma_load_2d(ks + i * R * D + C::kTileBytes, &tmV, full, hkv * D, row);
            const int slot = row & (P - 1);
            const uint8_t* src = a.kv_scale + (static_cast<size_t>(row - slot) * a.Hkv + hkv * P) * 2 + slot;
            if (P <= kTileKeys) {  // the page's K bytes and V bytes are neighbours
              bulk_load(sc + i * 2 * R, src, 2 * R, full);
            } else {
              bulk_load(sc, src, R, full);
              bulk_load(sc + R, src + P, R, full);
            }
          }
        }
        __syncwarp();  // the rows have been read
        ++issued;
      }
      walk.done();
    }
    // no copy of this CTA may still be writing its shared memory when it exits
    if (lane == 0) drain_ring(bars->full, C::kStages, issued, ctl.limit_ns);
    return;  // the consumers' merges below sync only the four consumer warps
  }

  // ===================== consumers =====================
  // sequences without a visible position, shared out over the ranges
  for (int b = range; b < a.B; b += gridDim.y) {
    if (sequence(a, b).tiles != 0) continue;
    if (threadIdx.x == 0 && a.seqlens[b] != 0) atomicCAS(ctl.status, 0, kDevBadInput | 0xD1);
    const size_t row = static_cast<size_t>(b) * a.H + h0;
    for (int i = threadIdx.x; i < gv * D / 8; i += kConsumers * 32)
      st_global_v4(static_cast<__nv_bfloat16*>(a.O) + row * D + i * 8, 0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < gv; i += kConsumers * 32) a.LSE[row + i] = -INFINITY;
  }

  const int g = lane >> 2;  // fragment row (position, feature pair) and column (head)
  const int t4 = lane & 3;
  const int kg = key_of<D>(g);
  const int mi = lane >> 3, rr = lane & 7;
  // lane i looks after the scales of its warp's position i
  const int my_key = warp * kWarpKeys + lane;
  const uint32_t my_scale = static_cast<uint32_t>(my_key / R * 2 * R + my_key % R);
  float* mw = reinterpret_cast<float*>(smem + C::kOffML);  // [4][16]
  float* lw = mw + kConsumers * 16;

  int it = 0;  // tiles so far
  while (walk.next(a)) {
    const int kend = walk.s.len, lo = walk.s.lo;
    const int kbeg = walk.s.base + walk.off * kTileKeys;
    // Q as the B operand: head nt * 8 + g, the features in the order in which a lane holds a K row
    // (its 16-byte units t4 and, for d = 128, t4 + 4): q = (qh + ql / 16) 2^(e - 134)
    uint32_t qb[NT][D / 16][2];  // kSharedQ: on their way to the merge's place, [nt][k step][lane]
    const uint32_t q_at = smem_u32(smem + C::kOffMerge) + lane * 8;
    float qf[NT][2];  // heads 2 t4, 2 t4 + 1: scale_log2 * 2^(e - 134 + kKShift)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool have = nt * 8 + g < gv;
      const uint4* qrow = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(a.Q) +
          (static_cast<size_t>(walk.b) * a.H + h0 + (have ? nt * 8 + g : 0)) * D);
      uint4 raw[D / 32];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {  // half i % 2 (8 features) of unit t4 + 4 (i / 2)
        raw[i] = have ? qrow[(t4 + 4 * (i >> 1)) * 2 + (i & 1)] : make_uint4(0u, 0u, 0u, 0u);
        constexpr uint32_t kAbs = 0x7fff7fffu;
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(raw[i].x & kAbs, raw[i].y & kAbs), __vmaxu2(raw[i].z & kAbs, raw[i].w & kAbs)));
      }
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // exponent of the largest element; at least 9, so that 2^(134 - e) is a normal number
      const int e = max(9, static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7));
      const float up = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // four features = one word of codes
          qb[nt][2 * i + k][0] = pack_f16x2(__uint_as_float(wd[2 * k] << 16) * up, __uint_as_float(wd[2 * k] & 0xffff0000u) * up);
          qb[nt][2 * i + k][1] =
              pack_f16x2(__uint_as_float(wd[2 * k + 1] << 16) * up, __uint_as_float(wd[2 * k + 1] & 0xffff0000u) * up);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int eh = __shfl_sync(0xffffffffu, e, (2 * t4 + i) * 4);
        // kept finite and positive, so that a hidden score stays -inf
        qf[nt][i] = fminf(fmaxf(scalbnf(a.scale_log2, eh - 134 + kKShift), 1.2e-38f), 3e38f);
      }
    }
    // scores are held as t = <q, k> 2^-kKShift with q's power of two still in it: x = t qf
    if constexpr (C::kSharedQ) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          if ((k & 3) == warp)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_at + (nt * (D / 16) + k) * 256), "r"(qb[nt][k][0]),
                         "r"(qb[nt][k][1])
                         : "memory");
      sync_consumers();
    }
    float o[D / 16][NT][4];
    float mt[NT][2], m0[NT][2];  // reference, in t; m0: the same, but 0 while there is none
    float2 l[NT];
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mt[nt][i] = -INFINITY;
        m0[nt][i] = 0.f;
      }
    }
    int unit = -1000;   // V scale byte of the sums' unit: P is multiplied by 2^(byte - unit); negative: no position yet
    bool wide = false;  // two bf16 terms
    int bad = 0;

    bool ok = true;
    for (int t = 0; t < walk.n; ++t, ++it) {
      const int st = it % C::kStages;
      if (!__all_sync(0xffffffffu, wait_ring(&bars->full[st], (it / C::kStages) & 1, bars, ctl, 0xC6))) {
        ok = false;
        break;
      }
      const int key0 = kbeg + t * kTileKeys;
      const uint32_t ks = smem_u32(smem + st * C::kStageBytes) + warp * kWarpKeys * D;
      const uint32_t vs = ks + C::kTileBytes;
      const uint32_t sc = smem_u32(smem + C::kOffScale + st * 2 * kTileKeys) + my_scale;
      bad |= *reinterpret_cast<volatile int*>(&bars->bad[st]);

      // this lane's position: factor of K, byte of V
      const float kf = scale_of(lds_u8(sc)) * (1.f / (1 << kKShift));
      int vbyte = static_cast<int>(lds_u8(sc + R));

      // positions outside [lo, kend) are hidden, whatever their bytes are; their V rows are
      // zeroed, because 0 * NaN would reach the sums
      const bool edge = key0 + kTileKeys > kend || key0 < lo;
      if (edge) {
        const int first = key0 + warp * kWarpKeys;
        if (first + lane >= kend || first + lane < lo) vbyte = unit;
        for (int i = lane; i < kWarpKeys * (D / 16); i += 32) {
          const int r = i / (D / 16);
          if (first + r >= kend || first + r < lo) st_shared_v4(vs + unit_off<D>(r, i % (D / 16)), 0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      // S^T = K Q^T
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          const uint4 ra = lds128(ks + unit_off<D>(u * 16 + kg, t4 + 4 * q));
          const uint4 rb = lds128(ks + unit_off<D>(u * 16 + 8 + kg, t4 + 4 * q));
          const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a0, a1, a2, a3;
            f16_halves(wa[k], a0, a2);
            f16_halves(wb[k], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b0 = qb[nt][4 * q + k][0], b1 = qb[nt][4 * q + k][1];
              if constexpr (C::kSharedQ)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b0), "=r"(b1) : "r"(q_at + (nt * (D / 16) + 4 * q + k) * 256));
              mma_f16(s[u][nt], a0, a1, a2, a3, b0, b1);
            }
          }
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float f = __shfl_sync(0xffffffffu, kf, u * 16 + hh * 8 + kg);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) s[u][nt][2 * hh + i] *= f;
        }
      }
      if (edge) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int key = key0 + warp * kWarpKeys + u * 16 + hh * 8 + kg;
            if (key >= kend || key < lo) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) s[u][nt][2 * hh] = s[u][nt][2 * hh + 1] = -INFINITY;
            }
          }
      }
      float mx[NT][2];
      bool grow = static_cast<uint32_t>(unit - vbyte) > kVSpan;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[nt][i] = fmaxf(fmaxf(s[0][nt][i], s[0][nt][2 + i]), fmaxf(s[1][nt][i], s[1][nt][2 + i]));
          grow |= (mx[nt][i] - mt[nt][i]) * qf[nt][i] > kLazy;
        }
      if (__any_sync(0xffffffffu, grow)) {
        const int top = __reduce_max_sync(0xffffffffu, vbyte);
        if (unit < 0 && top >= 0) unit = min(top + kVUp, kVCap);
        float eal = 1.f;
        wide |= __any_sync(0xffffffffu, vbyte >= 0 && static_cast<uint32_t>(unit - vbyte) > kVSpan);
        if (wide && min(top, kVCap) > unit) {
          eal = __uint_as_float(static_cast<uint32_t>(max(0, 127 + unit - min(top, kVCap))) << 23);
          unit = min(top, kVCap);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = mx[nt][i];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            v = fmaxf(v, mt[nt][i]);
            const float al = (v == -INFINITY) ? 1.f : ex2((mt[nt][i] - v) * qf[nt][i]);
            mt[nt][i] = v;
            m0[nt][i] = (v == -INFINITY) ? 0.f : v;
            if (i == 0) l[nt].x *= al;
            else l[nt].y *= al;
            const float oal = al * eal;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][nt][i] *= oal;
              o[c][nt][2 + i] *= oal;
            }
          }
      }
      // the reference is taken off before the factor: a product's rounding, 2^-24 of the score, would reach the
      // exponent, and from scores of 2^28 on leave f16
      auto probability = [&](float2 t, int nt) {
        const float2 x = fmul2(fadd2(t, make_float2(-m0[nt][0], -m0[nt][1])), make_float2(qf[nt][0], qf[nt][1]));
        return make_float2(ex2(x.x), ex2(x.y));
      };
      // P^T as the B operand, transposed: p * 2^(V byte - unit) * 2^kPShift
      if (!wide) {
        uint32_t pb[2][NT][2];
        const float vf = __uint_as_float(static_cast<uint32_t>(vbyte - unit + 127 + kPShift) << 23);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float f = __shfl_sync(0xffffffffu, vf, u * 16 + hh * 8 + kg);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 p = probability(make_float2(s[u][nt][2 * hh], s[u][nt][2 * hh + 1]), nt);
              l[nt] = fadd2(l[nt], p);
              const float2 pv = fmul2(p, make_float2(f, f));
              pb[u][nt][hh] = movmatrix_t(pack_f16x2(pv.x, pv.y));
            }
          }
        // O^T += V^T P^T: one ldmatrix.trans covers 16 positions x 32 features
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t r[4];
            ldsm_x4_t(vs + unit_off<D>(u * 16 + (mi & 1) * 8 + key_of<D>(rr), 2 * cc + (mi >> 1)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a0, a1, a2, a3;
              f16_pairs(r[2 * i], a0, a1);
              f16_pairs(r[2 * i + 1], a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * cc + i][nt], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
            }
          }
      } else {
        // the same in bf16 (a code is exact in it, too), once for P and once for what its rounding left;
        // one block of 16 positions at a time, because unrolled it made the f16 branch spill (5% slower)
        const float vf = vbyte == 255 ? __uint_as_float(0x7fc00000u)
                                      : __uint_as_float(static_cast<uint32_t>(max(0, vbyte - unit + 127 + kPShift)) << 23);
#pragma unroll 1
        for (int step = 0; step < 4; ++step) {
          const bool second = step & 2, rest = step & 1;  // positions 16 to 31; P's rounding error
          uint32_t w[NT][2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float f = __shfl_sync(0xffffffffu, vf, (second ? 16 : 0) + hh * 8 + kg);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 p = probability(make_float2(second ? s[1][nt][2 * hh] : s[0][nt][2 * hh],
                                                       second ? s[1][nt][2 * hh + 1] : s[0][nt][2 * hh + 1]), nt);
              if (!rest) l[nt] = fadd2(l[nt], p);
              const float2 pv = fmul2(p, make_float2(f, f));
              uint32_t b = pack_bf16x2(pv.x, pv.y);
              if (rest) b = pack_bf16x2(pv.x - __uint_as_float(b << 16), pv.y - __uint_as_float(b & 0xffff0000u));
              w[nt][hh] = movmatrix_t(b);
            }
          }
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t r[4];
            ldsm_x4_t(vs + unit_off<D>((second ? 16 : 0) + (mi & 1) * 8 + key_of<D>(rr), 2 * cc + (mi >> 1)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a0, a1, a2, a3;
              f16_pairs(r[2 * i], a0, a1);
              f16_pairs(r[2 * i + 1], a2, a3);
              a0 = bf16_of_f16(a0), a1 = bf16_of_f16(a1), a2 = bf16_of_f16(a2), a3 = bf16_of_f16(a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_bf16(o[2 * cc + i][nt], a0, a1, a2, a3, w[nt][0], w[nt][1]);
            }
          }
        }
      }
      if (edge) fence_proxy_async_smem();  // the next TMA write of the stage follows the zeros
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->empty[st]);
    }

    // the last tile has been multiplied: the join may be brought up (it waits for this grid's end)
    if (walk.left == walk.n) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- merge the four warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = i == 0 ? l[nt].x : l[nt].y;
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (g == 0) {
          mw[warp * 16 + nt * 8 + 2 * t4 + i] = mt[nt][i] == -INFINITY ? -INFINITY : __fmul_rn(mt[nt][i], qf[nt][i]);
          lw[warp * 16 + nt * 8 + 2 * t4 + i] = v;
        }
      }
    sync_consumers();
    auto head_max = [&](int h) {
      float v = -INFINITY;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) v = fmaxf(v, mw[i * 16 + h]);
      return v;
    };
    float of[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // P's 2^kPShift and the V exponent go out here.  A warp that saw nothing has zeros (or
        // NaN, if all it saw was NaN) and takes them as they are.
        // The product is rounded as the one in mw was (an fma would not round it).
        const float f = scalbnf(ex2(__fmul_rn(m0[nt][i], qf[nt][i]) - head_max(nt * 8 + 2 * t4 + i)), unit - 127 - kPShift);
        of[nt][i] = mt[nt][i] == -INFINITY ? 1.f : f;
      }
    // head and features of this thread in every slice (threads past the last head have none)
    constexpr int kPer = 4;
    static_assert(C::kSlice * 8 * NT / kPer <= kConsumers * 32, "a thread takes four features of one head");
    static_assert(kConsumers * 32 / (C::kSlice / kPer) <= 16, "heads of the statistics block");
    const int h = threadIdx.x / (C::kSlice / kPer);
    const int c0 = threadIdx.x % (C::kSlice / kPer) * kPer;
    const float M = head_max(h);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kConsumers; ++i) {
      const float x = mw[i * 16 + h];
      sum += lw[i * 16 + h] * (x == -INFINITY ? 1.f : ex2(x - M));
    }
    const bool none = bad || sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const bool whole = walk.n == walk.s.tiles;
    const size_t row = static_cast<size_t>(walk.b) * a.H + h0 + h;
    // a partial's slot: the range's first (the sequence began earlier) or second one
    const size_t part = (static_cast<size_t>(range) * 2 + (walk.off == 0 ? 1 : 0)) * a.H + h0 + h;
    if (h < gv && c0 == 0) {
      const float lse = none ? -INFINITY : (M == -INFINITY ? sum : (M + __log2f(sum)) * 0.69314718055994531f);
      if (whole) a.LSE[row] = lse;
      else a.LSEpart[part] = bad ? INFINITY : lse;  // +inf never comes out of a sum: the sequence is not to be used
    }
    float* ob = reinterpret_cast<float*>(smem + C::kOffMerge);
#pragma unroll
    for (int rd = 0; rd < C::kRounds; ++rd) {
      if (rd) sync_consumers();  // the slice before has been read
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < C::kSlice / 16; ++c) {
            const float* x = o[rd * (C::kSlice / 16) + c][nt];
            *reinterpret_cast<float2*>(ob + (warp * 8 * NT + nt * 8 + 2 * t4 + i) * C::kORow + 16 * c + 2 * g) =
                make_float2(x[i] * of[nt][i], x[2 + i] * of[nt][i]);
          }
      sync_consumers();
      if (h < gv) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!none) {
#pragma unroll
          for (int i = 0; i < kConsumers; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(ob + (i * 8 * NT + h) * C::kORow + c0);
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
          }
          v.x *= inv;
          v.y *= inv;
          v.z *= inv;
          v.w *= inv;
        }
        const int f = rd * C::kSlice + c0;
        if (whole) {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + row * D + f) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        } else if (!none) {
          *reinterpret_cast<float4*>(a.Opart + part * D + f) = v;
        }
      }
    }
    // statistics and slice have been read: the next segment may write its own, unless a wait gave up
    if (any_consumer(!ok)) break;
    walk.done();
  }
}

// Joins a sequence that crosses range borders, one CTA per (query head, border):
// the sequence's first border does the work, four warps taking every fourth
// partial, each with a running maximum of its own so that statistics and outputs are
// asked for together.  With M = max LSE_s and w_s = exp(LSE_s - M), O = sum w_s O_s / sum
// w_s and LSE = M + ln sum w_s.  A partial without positions (-inf) has no output; one
// that is not to be used (+inf) makes the row empty.
template <int D>
__global__ void __launch_bounds__(128) decode_fp8_join_kernel(const Decode8Args a) {
  constexpr int kPer = D / 32;
  constexpr int kAhead = 4;
  const int h = blockIdx.x, border = blockIdx.y + 1;
  const int warp = warp_id(), lane = lane_id();
  __shared__ float s_max[4], s_w[4];
  __shared__ float s_acc[4][D];
  wait_for_previous_kernel();  // its partials
  const int4 at = a.borders[border];  // sequence at the border, tiles before it, its tiles, tiles per range
  const int b = at.x, begin = at.y, len = at.w;
  if (b < 0 || begin >= border * len || begin < (border - 1) * len) return;
  const int parts = (begin + at.z - 1) / len - border + 2;
  // slot of partial s: the second one of the range in which the sequence begins, then the first ones
  auto slot = [&](int s) {
    return (s == 0 ? static_cast<size_t>(border - 1) * 2 + 1 : static_cast<size_t>(border - 1 + s) * 2) * a.H + h;
  };
  float M = -INFINITY, wsum = 0.f;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int s0 = warp; s0 < parts; s0 += 4 * kAhead) {
    float ls[kAhead], v[kAhead][kPer];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int s = s0 + 4 * k;
      ls[k] = -INFINITY;
      if (s < parts) {
        ls[k] = __ldcg(a.LSEpart + slot(s));
        const float* op = a.Opart + slot(s) * D + lane * kPer;  // not written where the statistic is infinite: not used then
        if constexpr (kPer == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(op));
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(op));
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) m = fmaxf(m, ls[k]);
    if (m == INFINITY) {  // not to be used; nothing that follows changes it
      M = m;
      break;
    }
    const float base = m == -INFINITY ? 0.f : m;
    const float al = M == -INFINITY ? 1.f : expf(M - base);  // with M = -inf there is nothing, or NaN
    M = m;
    wsum *= al;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] *= al;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (ls[k] == -INFINITY) continue;
      const float wgt = expf(ls[k] - base);
      wsum += wgt;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] += wgt * v[k][i];
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_acc[warp][lane * kPer + i] = acc[i];
  if (lane == 0) {
    s_max[warp] = M;
    s_w[warp] = wsum;
  }
  __syncthreads();
  if (warp == 0) {
    M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const bool bad = M == INFINITY;
    const float base = M == -INFINITY ? 0.f : M;
    float W = 0.f, out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[i] = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = s_max[u] == -INFINITY ? 1.f : expf(s_max[u] - base);
      W += s_w[u] * f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) out[i] += s_acc[u][lane * kPer + i] * f;
    }
    const bool none = bad || W == 0.f;
    const float inv = none ? 0.f : 1.f / W;
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[i] = none ? 0.f : out[i] * inv;
    const size_t row = static_cast<size_t>(b) * a.H + h;
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.O) + row * D + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
    else
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(out[0], out[1]);
    if (lane == 0) a.LSE[row] = none ? -INFINITY : base + logf(W);
  }
}

template <int D, int NT>
cudaError_t launch_nt(const CUtensorMap& tk, const CUtensorMap& tv, const Decode8Args& a, const DevCtl& c,
                      cudaStream_t s) {
  using C = Cfg8<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.Hkv * a.hgroups, a.ranges ? a.ranges : a.B);
  e = launch_behind(decode_fp8_kernel<D, NT>, grid, dim3(kThreads), C::kSmemBytes, s, tk, tv, a, c);
  if (e != cudaSuccess || a.ranges < 2) return e;
  return launch_behind(decode_fp8_join_kernel<D>, dim3(a.H, a.ranges - 1), dim3(128), 0, s, a);
}

}  // namespace

int decode_fp8_ctas_per_sm(int d, int nt) {
  if (d == 128) return nt == 1 ? Cfg8<128, 1>::kCtas : Cfg8<128, 2>::kCtas;
  return nt == 1 ? Cfg8<64, 1>::kCtas : Cfg8<64, 2>::kCtas;
}

cudaError_t launch_decode_fp8(const CUtensorMap& tk, const CUtensorMap& tv, const Decode8Args& a, int d, int nt,
                              const DevCtl& c, cudaStream_t s) {
  if (d == 128) return nt == 1 ? launch_nt<128, 1>(tk, tv, a, c, s) : launch_nt<128, 2>(tk, tv, a, c, s);
  return nt == 1 ? launch_nt<64, 1>(tk, tv, a, c, s) : launch_nt<64, 2>(tk, tv, a, c, s);
}

}  // namespace fa
