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
//   * grid (K/V head x head group, sequence, chunk of positions); the lanes of a
//     producer warp issue one TMA box per page and tensor and one bulk copy of
//     the page's scale bytes, 128 positions a stage, completion on mbarriers;
//   * four consumer warps take 32 positions of a tile each, on warp-level MMAs
//     (m16n8k16, f16 in, fp32 sums) with the POSITIONS as the 16 rows of S^T = K
//     Q^T and the features as the rows of O^T = V^T P^T, so that up to 8 query
//     heads fill the 8 columns and none of the tensor work is padding at H / Hkv
//     = 8 (the heads as rows would leave half of it empty);
//   * e4m3 -> f16 in integer arithmetic: the sign moves to bit 15 and the 7 other
//     bits to 13..7, which is code * 2^-8 exactly, subnormals included, and is
//     finite for every byte.  So what lies behind a sequence's end in a page can
//     be multiplied by a zero probability as it is;
//   * a 32-bit word of four codes gives the f16 pairs (0, 2) and (1, 3).  Along
//     the features of K any order will do, Q is loaded in the same one: a lane
//     reads 16 codes of a row at once.  For V, ldmatrix.trans on pairs of
//     features hands a lane the codes (f, j), (f + 1, j), (f, j + 1), (f + 1, j +
//     1), so the same two pairs are rows f and f + 1 of V^T: 8-bit data is
//     transposed by the 16-bit instruction;
//   * P goes from the accumulator layout to the operand layout with movmatrix.
// Rounding: Q is scaled by a power of two per head so that its largest element
// is in [2^8, 2^9), which is exact in f16 but for elements 2^22 below it; P times
// the V scales is rounded to f16 (11 bits; the running maximum of the V scales'
// exponents is taken out, like m); sums, maxima and statistics are fp32.
//
// A row whose scale byte is 255 (NaN) makes the heads that see it NaN.  A
// sequence with no position gets O = 0, LSE = -inf, and so does one with a
// length outside its table row or a page index outside the pool, which is
// reported (kDevBadInput); page 0 is read in such a page's place.
#include <cuda_bf16.h>

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

template <int D>
struct Cfg8 {
  static constexpr int kTileBytes = kTileKeys * D;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kOffScale = kStages * kStageBytes;        // [stage][256] scale bytes
  static constexpr int kOffBar = kOffScale + kStages * 2 * kTileKeys;
  static constexpr int kOffML = kOffBar + 128;                   // [2][4 warps][16 heads] reference, sum
  static constexpr int kSmemBytes = kOffML + 2 * kConsumers * 16 * 4;
  static constexpr int kORow = D + 4;
  static_assert(kConsumers * 16 * kORow * 4 <= kOffScale, "merge buffer fits in the stages");
};

struct Bars8 {
  uint64_t full[4], empty[4];
  int bad, abort;
};
static_assert(sizeof(Bars8) <= 128 && Cfg8<64>::kStages <= 4 && Cfg8<128>::kStages <= 4, "barrier block");

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
// codes 0, 2 and codes 1, 3 of a word as f16 pairs, each code * 2^-8
__device__ __forceinline__ uint32_t even_codes(uint32_t w) {
  return ((w << 7) & 0x3f803f80u) | ((w << 8) & 0x80008000u);
}
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return ((w >> 1) & 0x3f803f80u) | (w & 0x80008000u); }

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

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

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const Decode8Args a, const DevCtl ctl) {
  using C = Cfg8<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicCAS(ctl.status, 0, kDevTimeout | 0xC4);
    return;
  }
  Bars8* bars = reinterpret_cast<Bars8*>(smem + C::kOffBar);
  const int warp = warp_id();
  const int lane = lane_id();
  const int split = blockIdx.z;
  const int hkv = blockIdx.x / a.hgroups;
  const int hg = blockIdx.x % a.hgroups;
  const int b = blockIdx.y;
  const int G = a.H / a.Hkv;
  const int h0 = hkv * G + hg * (8 * NT);
  const int gv = min(8 * NT, G - hg * (8 * NT));
  const int P = a.page_size;

  const int L = a.seqlens[b];
  const bool bad_len = L < 0 || L > a.max_pages * P;  // max_pages * P <= 2^30 (host check)
  const int lo = a.window < 0 || bad_len ? 0 : max(0, L - 1 - a.window);  // first visible position
  // positions stay below 2^30 and chunks times splits below 2^30 + 2^30 (host checks)
  const int kbeg = (lo & ~(kTileKeys - 1)) + split * a.chunk;
  const int kend = bad_len ? kbeg : static_cast<int>(min(static_cast<long long>(kbeg) + a.chunk, static_cast<long long>(L)));
  const int ntiles = kend > kbeg ? (kend - kbeg + kTileKeys - 1) / kTileKeys : 0;
  if (threadIdx.x == 0) {
    bars->bad = bad_len ? 1 : 0;
    bars->abort = 0;
    if (bad_len) atomicCAS(ctl.status, 0, kDevBadInput | 0xD1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], kConsumers);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int R = min(P, kTileKeys);  // positions per box

  if (warp == kConsumers) {
    // ===================== producer warp: lane i loads box i of a tile =====================
    if (ntiles > 0) {
      const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      auto page_of = [&](int t) {  // this lane's page of tile t (nothing is read outside [lo, kend))
        const int j = kbeg + t * kTileKeys + lane * R;
        return (lane * R < kTileKeys && j < kend && j + R > lo) ? table[j / P] : 0;
      };
      int issued = 0;
      int next = page_of(0);
      for (int t = 0; t < ntiles; ++t) {
        const int st = t % C::kStages;
        int page = next;
        if (t + 1 < ntiles) next = page_of(t + 1);
        const bool free =
            t < C::kStages || wait_ring(&bars->empty[st], ((t / C::kStages) - 1) & 1, bars, ctl, 0xC5);
        if (!__all_sync(0xffffffffu, free)) break;
        const int key0 = kbeg + t * kTileKeys;
        const int nbox = (min(kTileKeys, kend - key0) + R - 1) / R;
        const int b0 = max(0, lo - key0) / R;  // boxes wholly before the window are left out
        const bool mine = lane >= b0 && lane < nbox;
        if (mine && (page < 0 || page >= a.num_pages)) {
          atomicCAS(ctl.status, 0, kDevBadInput | 0xD2);
          *reinterpret_cast<volatile int*>(&bars->bad) = 1;
          page = 0;
        }
        __syncwarp();  // the flag is set before lane 0 arrives
        if (lane == 0)
          mbar_arrive_expect_tx(&bars->full[st], static_cast<uint32_t>((nbox - b0) * R * (2 * D + 2)));
        __syncwarp();
        if (mine) {
          uint8_t* ks = smem + st * C::kStageBytes + lane * R * D;
          uint8_t* sc = smem + C::kOffScale + st * 2 * kTileKeys + lane * 2 * R;
          const int slot = (key0 + lane * R) & (P - 1);
          const int row = page * P + slot;
          tma_load_2d(ks, &tmK, &bars->full[st], hkv * D, row);
          tma_load_2d(ks + C::kTileBytes, &tmV, &bars->full[st], hkv * D, row);
          const uint8_t* src = a.kv_scale + (static_cast<size_t>(page) * a.Hkv + hkv) * 2 * P + slot;
          if (P <= kTileKeys) {  // the page's K bytes and V bytes are neighbours
            bulk_load(sc, src, 2 * R, &bars->full[st]);
          } else {
            bulk_load(sc, src, R, &bars->full[st]);
            bulk_load(sc + R, src + P, R, &bars->full[st]);
          }
        }
        ++issued;
      }
      // no copy of this CTA may still be writing its shared memory when it exits
      if (lane == 0) drain_ring(bars->full, C::kStages, issued, ctl.limit_ns);
    }
    return;  // the consumers' merge below syncs only the four consumer warps
  }

  // ===================== consumers =====================
  const int g = lane >> 2;  // fragment row (position, feature pair) and column (head)
  const int t4 = lane & 3;
  const int kg = key_of<D>(g);
  // Q as the B operand: head nt * 8 + g, in the order in which even_codes / odd_codes
  // hand over the 16-byte units t4 (and t4 + 4) of a K row
  uint32_t qb[NT][D / 16][2];
  float qf[NT][2];  // heads 2 t4, 2 t4 + 1: scale_log2 * 2^8 / (the power of two put into Q)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const bool have = nt * 8 + g < gv;
    const uint4* qrow =
        reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.Q) + (static_cast<size_t>(b) * a.H + h0 + nt * 8 + (have ? g : 0)) * D);
    uint4 raw[D / 32];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {  // features [16 u, 16 u + 16) of unit u = t4 + 4 (i / 2)
      raw[i] = have ? qrow[(t4 + 4 * (i >> 1)) * 2 + (i & 1)] : make_uint4(0u, 0u, 0u, 0u);
      constexpr uint32_t kAbs = 0x7fff7fffu;
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(raw[i].x & kAbs, raw[i].y & kAbs), __vmaxu2(raw[i].z & kAbs, raw[i].w & kAbs)));
    }
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // exponent of the largest element; at least 9, so that 2^(135 - e) is a normal number
    const int e = max(9, static_cast<int>(max(mx & 0xffffu, mx >> 16) >> 7));
    const float up = __uint_as_float(static_cast<uint32_t>(262 - e) << 23);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t wd[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // four features = one word of codes = one k step
        const float f0 = __uint_as_float(wd[2 * k] << 16) * up, f1 = __uint_as_float(wd[2 * k] & 0xffff0000u) * up;
        const float f2 = __uint_as_float(wd[2 * k + 1] << 16) * up, f3 = __uint_as_float(wd[2 * k + 1] & 0xffff0000u) * up;
        qb[nt][2 * i + k][0] = pack_f16x2(f0, f2);
        qb[nt][2 * i + k][1] = pack_f16x2(f1, f3);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int eh = __shfl_sync(0xffffffffu, e, (2 * t4 + i) * 4);
      qf[nt][i] = scalbnf(a.scale_log2, 8 + eh - 135);
    }
  }

  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
  int eref = 0;  // the largest V scale byte so far: P is multiplied by 2^(byte - eref)

  // this lane's four positions of a tile: u * 16 + hh * 8 + kg of its warp's 32
  uint32_t soff[2][2];  // their K scale bytes in the stage's scale block; V's lie R further
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int key = warp * kWarpKeys + u * 16 + hh * 8 + kg;
      soff[u][hh] = static_cast<uint32_t>(key / R * 2 * R + key % R);
    }
  const int mi = lane >> 3, rr = lane & 7;

  for (int t = 0; t < ntiles; ++t) {
    const int st = t % C::kStages;
    if (!__all_sync(0xffffffffu, wait_ring(&bars->full[st], (t / C::kStages) & 1, bars, ctl, 0xC6))) break;
    const int key0 = kbeg + t * kTileKeys;
    const uint32_t ks = smem_u32(smem + st * C::kStageBytes) + warp * kWarpKeys * D;
    const uint32_t vs = ks + C::kTileBytes;
    const uint32_t sc = smem_u32(smem + C::kOffScale + st * 2 * kTileKeys);

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
          const uint32_t a0 = even_codes(wa[k]), a1 = even_codes(wb[k]), a2 = odd_codes(wa[k]), a3 = odd_codes(wb[k]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(s[u][nt], a0, a1, a2, a3, qb[nt][4 * q + k][0], qb[nt][4 * q + k][1]);
        }
      }
    }
    // scores in log2 units; positions outside [lo, kend) are hidden, whatever their bytes are
    const bool edge = key0 + kTileKeys > kend || key0 < lo;
    float kf[2][2];
    uint32_t vb[2][2];
    uint32_t hidden = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        kf[u][hh] = scale_of(lds_u8(sc + soff[u][hh]));
        vb[u][hh] = lds_u8(sc + soff[u][hh] + R);
        if (edge) {
          const int key = key0 + warp * kWarpKeys + u * 16 + hh * 8 + kg;
          if (key >= kend || key < lo) {
            hidden |= 1u << (2 * u + hh);
            vb[u][hh] = 0;
          }
        }
      }
    float mx[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float& x = s[u][nt][2 * hh + i];
            x = (x * kf[u][hh]) * qf[nt][i];
            if (hidden >> (2 * u + hh) & 1u) x = -INFINITY;
            v = fmaxf(v, x);
          }
        mx[nt][i] = v;
        grow |= v > m[nt][i] + kLazy;
      }
    const uint32_t bmax = max(max(vb[0][0], vb[0][1]), max(vb[1][0], vb[1][1]));
    if (__any_sync(0xffffffffu, grow || static_cast<int>(bmax) > eref)) {
      const int en = max(eref, static_cast<int>(__reduce_max_sync(0xffffffffu, bmax)));
      const float eal = __uint_as_float(static_cast<uint32_t>(max(0, 127 + eref - en)) << 23);
      eref = en;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = mx[nt][i];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          v = fmaxf(v, m[nt][i]);
          const float al = (v == -INFINITY) ? 1.f : ex2(m[nt][i] - v);
          m[nt][i] = v;
          l[nt][i] *= al;
          const float oal = al * eal;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[c][nt][i] *= oal;
            o[c][nt][2 + i] *= oal;
          }
        }
    }
    // P^T as the B operand: p * 2^(V byte - eref) * 2^kPShift in f16, transposed
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t vbyte = vb[u][hh];
        const float vf = vbyte == 255u
                             ? __uint_as_float(0x7fc00000u)
                             : __uint_as_float(static_cast<uint32_t>(max(0, static_cast<int>(vbyte) - eref + 127 + kPShift)) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
          const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
          const float p0 = ex2(s[u][nt][2 * hh] - b0), p1 = ex2(s[u][nt][2 * hh + 1] - b1);
          l[nt][0] += p0;
          l[nt][1] += p1;
          pb[u][nt][hh] = movmatrix_t(pack_f16x2(p0 * vf, p1 * vf));
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
          const uint32_t a0 = even_codes(r[2 * i]), a1 = odd_codes(r[2 * i]);
          const uint32_t a2 = even_codes(r[2 * i + 1]), a3 = odd_codes(r[2 * i + 1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * cc + i][nt], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
        }
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->empty[st]);
  }

  // ---- merge the four warps ----
  float* mw = reinterpret_cast<float*>(smem + C::kOffML);  // [4][16]
  float* lw = mw + kConsumers * 16;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = l[nt][i];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g == 0) {
        mw[warp * 16 + nt * 8 + 2 * t4 + i] = m[nt][i];
        lw[warp * 16 + nt * 8 + 2 * t4 + i] = v;
      }
    }
  sync_consumers();  // the statistics are written, and every warp is done reading the stages
  auto head_max = [&](int h) {
    float v = -INFINITY;
#pragma unroll
    for (int i = 0; i < kConsumers; ++i) v = fmaxf(v, mw[i * 16 + h]);
    return v;
  };
  float* ob = reinterpret_cast<float*>(smem) + warp * 8 * NT * C::kORow;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = nt * 8 + 2 * t4 + i;
      const float M = head_max(h);
      // the codes' 2^-8, P's 2^kPShift and the V exponent go out here.  A warp that saw
      // nothing has zeros (or NaN, if all it saw was NaN) and takes them as they are.
      const float f = m[nt][i] == -INFINITY ? 1.f : scalbnf(ex2(m[nt][i] - M), eref - 127 + 8 - kPShift);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        *reinterpret_cast<float2*>(ob + h * C::kORow + 16 * c + 2 * g) = make_float2(o[c][nt][i] * f, o[c][nt][2 + i] * f);
    }
  sync_consumers();
  {
    constexpr int kPer = D * 8 * NT / (kConsumers * 32);  // features per thread
    const int h = threadIdx.x / (D / kPer);
    const int c0 = threadIdx.x % (D / kPer) * kPer;
    if (h < gv) {
      const float M = head_max(h);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kConsumers; ++i) {
        const float mi_ = mw[i * 16 + h];
        sum += lw[i * 16 + h] * (mi_ == -INFINITY ? 1.f : ex2(mi_ - M));
      }
      const bool bad = bars->bad != 0;
      const bool none = bad || sum == 0.f;
      const float inv = none ? 0.f : 1.f / sum;
      const int hq = h0 + h;
      const size_t ri = (static_cast<size_t>(split) * a.B + b) * a.H + hq;
      if (threadIdx.x % (D / kPer) == 0) {
        const float lse = none ? -INFINITY : (M == -INFINITY ? sum : (M + __log2f(sum)) * 0.69314718055994531f);
        if (a.splits == 1) a.LSE[static_cast<size_t>(b) * a.H + hq] = lse;
        else a.LSEpart[ri] = bad ? INFINITY : lse;  // +inf never comes out of a sum: the chunk is not to be used
      }
      if (a.splits == 1 || !none) {
#pragma unroll
        for (int c = 0; c < kPer; c += 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (!none) {
#pragma unroll
            for (int i = 0; i < kConsumers; ++i) {
              const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                                (i * 8 * NT + h) * C::kORow + c0 + c);
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
          if (a.splits == 1) {
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.O) + (static_cast<size_t>(b) * a.H + hq) * D + c0 + c;
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          } else {
            *reinterpret_cast<float4*>(a.Opart + ri * D + c0 + c) = v;
          }
        }
      }
    }
  }
}

// Joins the chunks of one (sequence, query head): four warps take every fourth
// chunk.  With M = max LSE_s and w_s = exp(LSE_s - M), O = sum w_s O_s / sum w_s and
// LSE = M + ln sum w_s.  A chunk without positions (-inf) has no partial output; a
// chunk that is not to be used (+inf) makes the row empty.
template <int D>
__global__ void __launch_bounds__(128) decode_fp8_join_kernel(const Decode8Args a) {
  constexpr int kPer = D / 32;
  const long long rows = static_cast<long long>(a.B) * a.H;
  const long long row = blockIdx.x;
  const int warp = warp_id(), lane = lane_id();
  __shared__ float s_max[4], s_w[4];
  __shared__ float s_acc[4][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials of the kernel before
  float M = -INFINITY;
  for (int s = static_cast<int>(threadIdx.x); s < a.splits; s += 128) M = fmaxf(M, a.LSEpart[s * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_max[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const bool bad = M == INFINITY;
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  float wsum = 0.f;
#pragma unroll 4
  for (int s = warp; s < a.splits; s += 4) {
    const float ls = a.LSEpart[s * rows + row];
    if (ls == -INFINITY || bad) continue;
    const float wgt = expf(ls - base);
    const float* op = a.Opart + (s * rows + row) * D + lane * kPer;
    float v[kPer];
    if constexpr (kPer == 4) {
      const float4 x = *reinterpret_cast<const float4*>(op);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(op);
      v[0] = x.x, v[1] = x.y;
    }
    wsum += wgt;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] += wgt * v[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_acc[warp][lane * kPer + i] = acc[i];
  if (lane == 0) s_w[warp] = wsum;
  __syncthreads();
  if (warp == 0) {
    const float W = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
    const float inv = W == 0.f ? 0.f : 1.f / W;
    float out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = lane * kPer + i;
      out[i] = ((s_acc[0][c] + s_acc[1][c]) + (s_acc[2][c] + s_acc[3][c])) * inv;
    }
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.O) + row * D + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
    else
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(out[0], out[1]);
    if (lane == 0) a.LSE[row] = W == 0.f ? -INFINITY : base + logf(W);
  }
}

template <int D, int NT>
cudaError_t launch_nt(const CUtensorMap& tk, const CUtensorMap& tv, const Decode8Args& a, const DevCtl& c,
                      cudaStream_t s) {
  using C = Cfg8<D>;
  cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.Hkv * a.hgroups, a.B, a.splits);
  decode_fp8_kernel<D, NT><<<grid, kThreads, C::kSmemBytes, s>>>(tk, tv, a, c);
  if ((e = cudaGetLastError()) != cudaSuccess || a.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.B) * a.H));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its start overlaps the end of the kernel before
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_join_kernel<D>, a);
}

}  // namespace

cudaError_t launch_decode_fp8(const CUtensorMap& tk, const CUtensorMap& tv, const Decode8Args& a, int d, int nt,
                              const DevCtl& c, cudaStream_t s) {
  if (d == 128) return nt == 1 ? launch_nt<128, 1>(tk, tv, a, c, s) : launch_nt<128, 2>(tk, tv, a, c, s);
  return nt == 1 ? launch_nt<64, 1>(tk, tv, a, c, s) : launch_nt<64, 2>(tk, tv, a, c, s);
}

}  // namespace fa
