// RMS norm of query and key heads with the rotation by position, in one pass,
// and its backward; bf16 and fp32, d = 64 or 128, sm_100a.
//
// For one row x (d features of one head at one position) with gain w:
//     r = 1 / sqrt(mean(x^2) + eps),   y = x r w
// and, for every pair (first, second) of features with the position's angle
// (c, s) from the caller's tables,
//     out_first = y_first c - y_second s,   out_second = y_second c + y_first s.
// Pairs are (i, i + d/2), or (2i, 2i + 1) when interleaved.  The rotation is
// orthogonal, so with the incoming gradient g and gr = R^T g
//     dw = sum over rows of gr x r,
//     dx = r w gr - x r^3 / d * sum(w gr x).
// The backward recomputes r from x (which it has to read anyway), so the
// forward saves nothing.
//
// Both are bound by the bytes they move (x in, out; x, g in, dx out).  A lane
// holds 16 features of a row, the same 8 of each half, so both elements of a
// pair are in one thread in either layout.  They come in runs of 16 bytes (two
// of 8 bf16, four of 4 fp32), neighbouring lanes' runs next to one another, so
// every access fills whole sectors.  A row takes d / 16 lanes (a warp 4 rows of
// d = 128, 8 of d = 64).  A warp takes the heads of one position, so the angles
// and gains are read once for all of them.  All arithmetic is fp32 (packed
// pairs), each output is rounded once.
//
// Measured on a B200 (GPU time), d = 128, bf16: forward B1 N16384 H32 + 32 (537 MB) 86
// us, 6.2 TB/s; B1 N4096 H64 + 8 out of a packed projection (151 MB) 25.4 us, 5.9 TB/s;
// backward B1 N16384 H32 + 32 (805 MB) 131 us with the gains' sums, 6.1 TB/s.
// fp32: B2 N4096 H32 + 8 forward (335 MB) 58 us, 5.8 TB/s; backward (503 MB) 86 us, 5.9
// TB/s (130 us with a lane's 8 features of a half side by side: 32-byte steps).
#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

// 16 features of one row, in runs of 16 bytes
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a, b;
};
template <>
struct Raw<float> {
  float4 a0, a1, b0, b1;
};

// The first feature of x[j], the lane's j-th pair of neighbouring features (j = 0..7)
template <typename T, int D>
__device__ __forceinline__ constexpr int feature(int j, int sub) {
  return sizeof(T) == 2 ? (j >> 2) * (D / 2) + 8 * sub + 2 * (j & 3) : (j >> 1) * (D / 4) + 4 * sub + 2 * (j & 1);
}

template <int D>
__device__ __forceinline__ void load_row(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p, int sub) {
  r.a = *reinterpret_cast<const uint4*>(p + 8 * sub);
  r.b = *reinterpret_cast<const uint4*>(p + D / 2 + 8 * sub);
}
template <int D>
__device__ __forceinline__ void load_row(Raw<float>& r, const float* p, int sub) {
  r.a0 = *reinterpret_cast<const float4*>(p + 4 * sub);
  r.a1 = *reinterpret_cast<const float4*>(p + D / 4 + 4 * sub);
  r.b0 = *reinterpret_cast<const float4*>(p + D / 2 + 4 * sub);
  r.b1 = *reinterpret_cast<const float4*>(p + 3 * D / 4 + 4 * sub);
}

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// x[0..3]: the run of the first half as pairs of neighbours, x[4..7]: of the second
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float2 (&x)[8]) {
  x[0] = bf2(r.a.x);
  x[1] = bf2(r.a.y);
  x[2] = bf2(r.a.z);
  x[3] = bf2(r.a.w);
  x[4] = bf2(r.b.x);
  x[5] = bf2(r.b.y);
  x[6] = bf2(r.b.z);
  x[7] = bf2(r.b.w);
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float2 (&x)[8]) {
  x[0] = make_float2(r.a0.x, r.a0.y);
  x[1] = make_float2(r.a0.z, r.a0.w);
  x[2] = make_float2(r.a1.x, r.a1.y);
  x[3] = make_float2(r.a1.z, r.a1.w);
  x[4] = make_float2(r.b0.x, r.b0.y);
  x[5] = make_float2(r.b0.z, r.b0.w);
  x[6] = make_float2(r.b1.x, r.b1.y);
  x[7] = make_float2(r.b1.z, r.b1.w);
}

template <int D>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, int sub, const float2 (&x)[8]) {
  uint4 a, b;
  a.x = pack_bf16x2(x[0].x, x[0].y);
  a.y = pack_bf16x2(x[1].x, x[1].y);
  a.z = pack_bf16x2(x[2].x, x[2].y);
  a.w = pack_bf16x2(x[3].x, x[3].y);
  b.x = pack_bf16x2(x[4].x, x[4].y);
  b.y = pack_bf16x2(x[5].x, x[5].y);
  b.z = pack_bf16x2(x[6].x, x[6].y);
  b.w = pack_bf16x2(x[7].x, x[7].y);
  *reinterpret_cast<uint4*>(p + 8 * sub) = a;
  *reinterpret_cast<uint4*>(p + D / 2 + 8 * sub) = b;
}
template <int D>
__device__ __forceinline__ void store_row(float* p, int sub, const float2 (&x)[8]) {
  *reinterpret_cast<float4*>(p + 4 * sub) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  *reinterpret_cast<float4*>(p + D / 4 + 4 * sub) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  *reinterpret_cast<float4*>(p + D / 2 + 4 * sub) = make_float4(x[4].x, x[4].y, x[5].x, x[5].y);
  *reinterpret_cast<float4*>(p + 3 * D / 4 + 4 * sub) = make_float4(x[6].x, x[6].y, x[7].x, x[7].y);
}

// The 8 (c, s) of this lane's pairs, laid out for rotate(): Half: cs[j] belongs to
// the features x[j] and x[4 + j]; interleaved: to the pair x[2j], x[2j + 1] split
// as c[j].x for x[2j], c[j].y for x[2j + 1].
// Ordinary loads: the launch overlaps the end of the kernel before, which may write the tables, and what
// griddepcontrol.wait orders are not the loads of the read-only path.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void load_angles(const float* cos_t, const float* sin_t, int pos, int sub, float2 (&c)[4],
                                            float2 (&s)[4]) {
  const size_t row = static_cast<size_t>(pos) * (D / 2);
  if constexpr (kInter && sizeof(T) == 4) {  // a run holds two pairs: two neighbouring angles
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = feature<T, D>(2 * k, sub) / 2;
      c[k] = *reinterpret_cast<const float2*>(cos_t + row + at);
      s[k] = *reinterpret_cast<const float2*>(sin_t + row + at);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {  // four neighbouring angles each
      const int at = kInter ? feature<T, D>(2 * k, sub) / 2 : feature<T, D>(k, sub);
      const float4 vc = *reinterpret_cast<const float4*>(cos_t + row + at);
      const float4 vs = *reinterpret_cast<const float4*>(sin_t + row + at);
      c[k] = make_float2(vc.x, vc.y);
      c[k + 1] = make_float2(vc.z, vc.w);
      s[k] = make_float2(vs.x, vs.y);
      s[k + 1] = make_float2(vs.z, vs.w);
    }
  }
}

// The rotation (kBack: its transpose) with a gain folded into the angles:
// out = R diag(w) x.  Half: x[j] (first) and x[4 + j] (second), two pairs at a
// time; interleaved: x[j] = (first, second) of pair j.
//   Half:  out[j] = x[j] ca[j] - x[4+j] sb[j], out[4+j] = x[4+j] cb[j] + x[j] sa[j]
//   with ca = c w_first, sb = s w_second, cb = c w_second, sa = s w_first
//   interleaved: out[j] = x[j] * (c w0, c w1) + swap(x[j]) * (-s w1, s w0)
struct Coef {
  float2 p[8], q[8];  // Half: p = ca | cb, q = -sb | sa;  interleaved: p = (c w0, c w1), q = (-s w1, s w0)
};

template <bool kInter, bool kNorm>
__device__ __forceinline__ void make_coef(const float2 (&c)[4], const float2 (&s)[4], const float2 (&w)[8], Coef& k) {
  if constexpr (kInter) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float cj = (j & 1) ? c[j >> 1].y : c[j >> 1].x;
      const float sj = (j & 1) ? s[j >> 1].y : s[j >> 1].x;
      k.p[j] = kNorm ? make_float2(cj * w[j].x, cj * w[j].y) : make_float2(cj, cj);
      k.q[j] = kNorm ? make_float2(-sj * w[j].y, sj * w[j].x) : make_float2(-sj, sj);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k.p[j] = kNorm ? fmul2(c[j], w[j]) : c[j];
      k.p[4 + j] = kNorm ? fmul2(c[j], w[4 + j]) : c[j];
      const float2 ns = make_float2(-s[j].x, -s[j].y);
      k.q[j] = kNorm ? fmul2(ns, w[4 + j]) : ns;
      k.q[4 + j] = kNorm ? fmul2(s[j], w[j]) : s[j];
    }
  }
}

template <bool kInter>
__device__ __forceinline__ void rotate(const float2 (&x)[8], const Coef& k, float2 (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 other = kInter ? make_float2(x[j].y, x[j].x) : x[j < 4 ? j + 4 : j - 4];
    o[j] = ffma2(x[j], k.p[j], fmul2(other, k.q[j]));
  }
}

// gr = R^T g (no gain)
template <bool kInter>
__device__ __forceinline__ void rotate_back(const float2 (&g)[8], const float2 (&c)[4], const float2 (&s)[4],
                                            float2 (&o)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float cj = (j & 1) ? c[j >> 1].y : c[j >> 1].x;
      const float sj = (j & 1) ? s[j >> 1].y : s[j >> 1].x;
      o[j].x = fmaf(g[j].x, cj, g[j].y * sj);
      o[j].y = fmaf(g[j].y, cj, -g[j].x * sj);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = ffma2(g[j], c[j], fmul2(g[4 + j], s[j]));
      o[4 + j] = ffma2(g[4 + j], c[j], fmul2(g[j], make_float2(-s[j].x, -s[j].y)));
    }
  }
}

// this lane's 16 gains in the order of x (rows of T, gains of either type)
template <typename T, int D>
__device__ __forceinline__ void load_gain(const void* w, int w_f32, int sub, float2 (&o)[8]) {
  if (w_f32) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // four features each
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + feature<T, D>(2 * r, sub));
      o[2 * r] = make_float2(v.x, v.y);
      o[2 * r + 1] = make_float2(v.z, v.w);
    }
  } else if constexpr (sizeof(T) == 2) {
    Raw<__nv_bfloat16> r;
    load_row<D>(r, static_cast<const __nv_bfloat16*>(w), sub);
    unpack(r, o);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + feature<T, D>(2 * r, sub));
      o[2 * r] = bf2(v.x);
      o[2 * r + 1] = bf2(v.y);
    }
  }
}

// sum over the d / 16 lanes of a row
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__device__ __forceinline__ float row_rsqrt(const float2 (&x)[8], float eps) {
  float2 q = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) q = ffma2(x[j], x[j], q);
  return rsqrtf(fmaf(row_sum<D>(q.x + q.y), 1.f / D, eps));
}

// position of a token: -1 for padding; one outside the tables is reported and treated as padding
__device__ __forceinline__ int checked_position(const RopeArgs& a, int pos, int lane) {
  if (pos >= a.table) {
    if (lane == 0) atomicCAS(a.status, 0, kDevBadInput | 0xD3);
    pos = -1;
  }
  return pos;
}

// one row of the forward: every lane of the warp comes here, its row valid or not
template <int D, bool kNorm, bool kInter, typename T>
__device__ __forceinline__ void turn_row(const Raw<T>& raw, bool place, const Coef& k, float eps, float2 (&o)[8]) {
  if (place) {  // not padding
    float2 x[8];
    unpack(raw, x);
    float r = 1.f;
    if constexpr (kNorm) r = row_rsqrt<D>(x, eps);
    rotate<kInter>(x, k, o);
    if constexpr (kNorm) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmul2(o[j], make_float2(r, r));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_float2(0.f, 0.f);
  }
}

// ---------------------------------------------------------------------------
// Forward, few rows: a warp takes two groups of rows (4 heads of d = 128, 8 of d = 64) of
// one tensor at one position, both loaded before the first is used; grid (position
// blocks, pairs of groups of q then k).
// ---------------------------------------------------------------------------
template <typename T, int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 && !kInter ? 5 : 4) rope_fwd_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  wait_for_previous_kernel();
  const int lane = lane_id();
  const int token = blockIdx.x * kWarps + warp_id();
  if (token >= a.tokens) return;
  const int sub = lane % kLanes;
  const bool is_q = static_cast<int>(blockIdx.y) < a.q_groups;
  const int pair = is_q ? blockIdx.y : blockIdx.y - a.q_groups;
  const int nh = is_q ? a.H : a.Hkv;
  const int h0 = pair * 2 * kRows + lane / kLanes;
  const int b = token / a.N, n = token - b * a.N;
  const RopeTensor& t = is_q ? a.q : a.k;
  const T* x0 = static_cast<const T*>(t.x) + b * t.sb + n * t.sn;
  T* o0 = static_cast<T*>(t.out) + static_cast<size_t>(token) * nh * D;
  const int pos = checked_position(a, a.positions ? a.positions[token] : n, lane);
  constexpr int kAhead = sizeof(T) == 2 ? 2 : 1;  // registers
  Raw<T> raw[2];
  auto load = [&](int u) {
    raw[u] = {};
    if (pos >= 0 && h0 + u * kRows < nh) load_row<D>(raw[u], x0 + (h0 + u * kRows) * t.sh, sub);
  };
  float2 c[4], s[4], w[8];
  if (pos >= 0) load_angles<T, D, kInter>(a.cos_t, a.sin_t, pos, sub, c, s);
  if (kNorm) load_gain<T, D>(t.w, a.w_f32, sub, w);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u);
  Coef k;
  if (pos >= 0) make_coef<kInter, kNorm>(c, s, w, k);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (u && pair * 2 * kRows + kRows >= nh) break;  // no row of the second group
    if (u >= kAhead) load(u);
    float2 o[8];
    turn_row<D, kNorm, kInter>(raw[u], pos >= 0, k, a.eps, o);
    if (h0 + u * kRows < nh) store_row<D>(o0 + static_cast<size_t>(h0 + u * kRows) * D, sub, o);
  }
}

// ---------------------------------------------------------------------------
// Forward of many rows, and backward: blocks [0, q_blocks) walk the row groups (512 / d
// heads at one position) of q, the others those of k.  Rows and angles of the next
// iterations wait in shared memory, written by asynchronous copies into slots of the
// lane's own (no barrier).
// ---------------------------------------------------------------------------
// kTensors rows per iteration (x; or g and x).  Three stages against two, bf16 d128:
// backward B1 N4096 H64 + 8 39.4 us and 42.4, forward 25.5 and 27.9.
template <typename T, int kTensors>
struct Ring {
  static constexpr int kStages = 3;
  static constexpr int kStep = kWarps * 32 * 16;               // a piece of every lane
  static constexpr int kRow = 16 * sizeof(T) / 16;             // 16-byte pieces of a lane's 16 features
  static constexpr int kPieces = kTensors * kRow;
  static constexpr int kBytes = kStages * (kPieces + 4) * kStep;  // and the angles
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8_l1(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void lds_row(uint32_t addr, Raw<__nv_bfloat16>& r) {
  const float4 a = lds_f4(addr), b = lds_f4(addr + kWarps * 32 * 16);
  r.a = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w));
  r.b = make_uint4(__float_as_uint(b.x), __float_as_uint(b.y), __float_as_uint(b.z), __float_as_uint(b.w));
}
__device__ __forceinline__ void lds_row(uint32_t addr, Raw<float>& r) {
  constexpr int kStep = kWarps * 32 * 16;
  r.a0 = lds_f4(addr);
  r.a1 = lds_f4(addr + kStep);
  r.b0 = lds_f4(addr + 2 * kStep);
  r.b1 = lds_f4(addr + 3 * kStep);
}
// this lane's 16 features of the row at p into its slots from dst on, run by run
template <int D, typename T>
__device__ __forceinline__ void copy_row(uint32_t dst, const T* p, int sub) {
  constexpr int kStep = kWarps * 32 * 16;
  constexpr int kRun = 16 / sizeof(T);
  constexpr int kRuns = 16 / kRun;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) copy16(dst + i * kStep, p + i * (D / kRuns) + kRun * sub);
}

// A warp's walk over row groups, counted through all positions (fewer than 2^32: B N H d
// < 2^40).  In rounds, every warp takes the next `per` groups, so that the GPU reads one
// stretch of memory at a time; what is left for no full round is cut into equal ranges.
// Backward, without the cut (whole ranges of a position): B1 N8192 H40 + 40 d128 101 us for
// 81.  One range per warp and no rounds: H32 + 32 N16384 139 us for 131, d64 133 for 125.
struct Shares {
  unsigned int groups;          // of a position
  unsigned int per, step;       // of a warp's range, of a round
  unsigned int last, last_end;  // this warp's range of the rest
};
struct Walk {
  unsigned int g, end;    // the position's first group in this range, end of the range
  unsigned int ng, nend;  // the range after it (empty: none)
  int rounds;             // full rounds after that one; -1: the rest is given out, too
  int it, its;            // iteration, iterations at this position
  int group;              // first group at this position
  int token, b, n;        // position in [0, B N): b N + n
  int ntoken, nb, nn;     // the next one
  int pos, coming;        // the caller's positions of both (the next one's asked for ahead)
  __device__ __forceinline__ bool more() const { return g < end; }
  static __device__ __forceinline__ int raw_position(const RopeArgs& a, int tok, int n) {
    return a.positions ? a.positions[tok] : n;
  }
  __device__ __forceinline__ void open(const RopeArgs& a, const Shares& w, int raw, int lane) {  // g < end
    pos = checked_position(a, raw, lane);
    its = static_cast<int>(min(end - g, w.groups - group));
    it = 0;
    if (end - g > static_cast<unsigned int>(its)) {
      ntoken = token + 1;
      const bool wrap = n + 1 == a.N;
      nb = b + wrap;
      nn = wrap ? 0 : n + 1;
      coming = raw_position(a, ntoken, nn);
    } else if (ng < nend) {
      ntoken = static_cast<int>(ng / w.groups);
      nb = ntoken / a.N;
      nn = ntoken - nb * a.N;
      coming = raw_position(a, ntoken, nn);
    }
  }
  // the range after [ng, nend)
  __device__ __forceinline__ void after(const Shares& w) {
    if (rounds > 0) {
      ng += w.step;
      nend = ng + w.per;
    } else {
      ng = rounds == 0 ? w.last : nend;
      nend = rounds == 0 ? w.last_end : nend;
    }
    rounds = max(rounds - 1, -1);
  }
  __device__ __forceinline__ void first(const RopeArgs& a, const Shares& w, unsigned int mine, int full, int lane) {
    g = full ? mine * w.per : w.last;
    end = full ? g + w.per : w.last_end;
    rounds = full - 1;
    ng = g;
    nend = end;
    after(w);
    if (!more()) return;
    token = static_cast<int>(g / w.groups);
    b = token / a.N;
    n = token - b * a.N;
    group = static_cast<int>(g - static_cast<unsigned int>(token) * w.groups);
    open(a, w, raw_position(a, token, n), lane);
  }
  __device__ __forceinline__ void next(const RopeArgs& a, const Shares& w, int lane) {
    g += its;
    const bool jump = !more();
    if (jump) {
      g = ng;
      end = nend;
      if (!more()) return;
      after(w);
    }
    token = ntoken;
    b = nb;
    n = nn;
    group = jump ? static_cast<int>(g - static_cast<unsigned int>(token) * w.groups) : 0;
    open(a, w, coming, lane);
  }
};

// An iteration on its way: where its row goes (this lane's), and what it is
template <typename T>
struct Coming {
  T* out;
  unsigned int is;
};
constexpr unsigned int kLive = 1, kPlace = 2, kFresh = 4, kHead = 8;  // there is one; not padding; new angles; a row

// warp `mine`'s shares of the row groups; returns the full rounds
__device__ __forceinline__ int give_shares(Shares& s, const RopeArgs& a, int groups, unsigned int mine,
                                           unsigned int warps) {
  s.groups = groups;
  s.per = a.per;
  s.step = warps * s.per;
  const unsigned int total = static_cast<unsigned int>(a.tokens) * groups;
  const unsigned int full = total / s.step, rest = total - full * s.step;  // rest * warps < 2^32
  s.last = full * s.step + rest * mine / warps;
  s.last_end = full * s.step + rest * (mine + 1) / warps;
  return static_cast<int>(full);
}

// a position's angles into this lane's four slots (as load_angles: cosines, then sines)
template <typename T, int D, bool kInter>
__device__ __forceinline__ void copy_angles(uint32_t dst, const float* cos_t, const float* sin_t, int pos, int sub) {
  constexpr int kStep = kWarps * 32 * 16;
  const size_t row = static_cast<size_t>(pos) * (D / 2);
  if constexpr (kInter && sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = feature<T, D>(2 * k, sub) / 2;
      copy8_l1(dst + (k >> 1) * kStep + (k & 1) * 8, cos_t + row + at);
      copy8_l1(dst + (2 + (k >> 1)) * kStep + (k & 1) * 8, sin_t + row + at);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const int at = kInter ? feature<T, D>(2 * k, sub) / 2 : feature<T, D>(k, sub);
      copy16_l1(dst + (k >> 1) * kStep, cos_t + row + at);
      copy16_l1(dst + (2 + (k >> 1)) * kStep, sin_t + row + at);
    }
  }
}
__device__ __forceinline__ void lds_angles(uint32_t src, float2 (&c)[4], float2 (&s)[4]) {
  constexpr int kStep = kWarps * 32 * 16;
  const float4 c0 = lds_f4(src), c1 = lds_f4(src + kStep), s0 = lds_f4(src + 2 * kStep), s1 = lds_f4(src + 3 * kStep);
  c[0] = make_float2(c0.x, c0.y), c[1] = make_float2(c0.z, c0.w);
  c[2] = make_float2(c1.x, c1.y), c[3] = make_float2(c1.z, c1.w);
  s[0] = make_float2(s0.x, s0.y), s[1] = make_float2(s0.z, s0.w);
  s[2] = make_float2(s1.x, s1.y), s[3] = make_float2(s1.z, s1.w);
}

// The forward at 3 or 4 blocks per SM (120 registers; 5 spill).  Against warps with one
// position each and four rows loaded ahead, bf16 d128: B1 N2048 H32 + 8 7.7 us (9.3), B1
// N4096 H64 + 8 25.4 (27.3), B2 N8192 H32 + 8 57 (60), B1 N8192 H40 + 40 55.6 (60.8), B1
// N16384 H32 + 32 86 (84.4); d64 B4 N4096 H16 + 16 23.4 (29.7).
template <typename T, int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, 4) rope_fwd_rounds_kernel(const RopeArgs a) {
  using R = Ring<T, 1>;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  constexpr int kStep = R::kStep;
  wait_for_previous_kernel();
  const int lane = lane_id(), warp = warp_id();
  const int sub = lane % kLanes;
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
  const int first = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
  const int blocks = is_q ? a.q_blocks : static_cast<int>(gridDim.x) - a.q_blocks;
  const int nh = is_q ? a.H : a.Hkv;
  const RopeTensor& t = is_q ? a.q : a.k;
  Shares share;
  const unsigned int warps = blocks * kWarps, mine = first * kWarps + warp;
  const int full = give_shares(share, a, is_q ? a.q_groups : a.k_groups, mine, warps);
  const uint32_t rows_at = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t angles_at = rows_at + R::kStages * R::kRow * kStep;
  float2 w[8];
  if (kNorm) load_gain<T, D>(t.w, a.w_f32, sub, w);
  Walk ahead;
  ahead.first(a, share, mine, full, lane);
  int ahead_row = 0, ahead_unit = 0, h = 0;  // slots; head of this lane's row
  const T* xp = nullptr;
  T* op = nullptr;
  // the copies of one iteration, as one group (which may be empty)
  auto fetch = [&]() {
    Coming<T> c = {nullptr, 0};
    if (ahead.more()) {
      c.is = kLive;
      if (ahead.it == 0) {
        c.is |= kFresh;
        h = ahead.group * kRows + lane / kLanes;
        xp = static_cast<const T*>(t.x) + ahead.b * t.sb + ahead.n * t.sn + h * t.sh;
        op = static_cast<T*>(t.out) + (static_cast<size_t>(ahead.token) * nh + h) * D;
        if (ahead.pos >= 0) copy_angles<T, D, kInter>(angles_at + ahead_unit * 4 * kStep, a.cos_t, a.sin_t, ahead.pos, sub);
        ahead_unit = ahead_unit + 1 == R::kStages ? 0 : ahead_unit + 1;
      }
      if (ahead.pos >= 0) c.is |= kPlace;
      if (h < nh) c.is |= kHead;
      if (ahead.pos >= 0 && h < nh) copy_row<D>(rows_at + ahead_row * R::kPieces * kStep, xp, sub);
      c.out = op;
      h += kRows;
      xp += kRows * t.sh;
      op += kRows * D;
      if (++ahead.it == ahead.its) ahead.next(a, share, lane);
    }
    ahead_row = ahead_row + 1 == R::kStages ? 0 : ahead_row + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
    return c;
  };
  Coming<T> line[R::kStages - 1];
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) line[i] = fetch();
  int row_slot = 0, unit_slot = 0;
  Coef k;
  while (line[0].is & kLive) {
    const Coming<T> at = line[0];
#pragma unroll
    for (int i = 0; i < R::kStages - 2; ++i) line[i] = line[i + 1];
    line[R::kStages - 2] = fetch();
    copies_wait<R::kStages - 1>();  // the oldest group has arrived
    if (at.is & kFresh) {
      float2 c[4], s[4];
      lds_angles(angles_at + unit_slot * 4 * kStep, c, s);
      make_coef<kInter, kNorm>(c, s, w, k);
      unit_slot = unit_slot + 1 == R::kStages ? 0 : unit_slot + 1;
    }
    Raw<T> raw;
    float2 o[8];
    lds_row(rows_at + row_slot * R::kPieces * kStep, raw);  // whatever is there, where the position is padding
    row_slot = row_slot + 1 == R::kStages ? 0 : row_slot + 1;
    turn_row<D, kNorm, kInter>(raw, at.is & kPlace, k, a.eps, o);
    if (at.is & kHead) store_row<D>(at.out, sub, o);
  }
  copies_wait<0>();
}

// The backward: each warp has its own running sum of the gain's gradient; a block writes
// the sum of its warps to partial[block][d].  The registers that the gradient needs leave
// room for 12 warps on an SM, whose own loads would keep only 24 KB in flight.
template <typename T, int D, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, 3) rope_bwd_kernel(const RopeArgs a) {
  using R = Ring<T, kNorm ? 2 : 1>;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kLanes = D / 16;
  constexpr int kRows = 32 / kLanes;
  constexpr int kStep = R::kStep;
  wait_for_previous_kernel();
  const int lane = lane_id(), warp = warp_id();
  const int sub = lane % kLanes;
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
  const int first = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
  const int blocks = is_q ? a.q_blocks : static_cast<int>(gridDim.x) - a.q_blocks;
  const int nh = is_q ? a.H : a.Hkv;
  const RopeTensor& t = is_q ? a.q : a.k;
  Shares share;
  const unsigned int warps = blocks * kWarps, mine = first * kWarps + warp;
  const int full = give_shares(share, a, is_q ? a.q_groups : a.k_groups, mine, warps);
  const uint32_t rows_at = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t angles_at = rows_at + R::kStages * R::kPieces * kStep;
  float2 w[8], acc[8];
  if (kNorm) load_gain<T, D>(t.w, a.w_f32, sub, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = make_float2(0.f, 0.f);

  Walk ahead;
  ahead.first(a, share, mine, full, lane);
  int ahead_row = 0, ahead_unit = 0, h = 0;  // slots; head of this lane's row
  const T* gp = nullptr;
  const T* xp = nullptr;
  T* op = nullptr;
  // the copies of one iteration, as one group (which may be empty)
  auto fetch = [&]() {
    Coming<T> c = {nullptr, 0};
    if (ahead.more()) {
      c.is = kLive;
      if (ahead.it == 0) {
        c.is |= kFresh;
        h = ahead.group * kRows + lane / kLanes;
        gp = static_cast<const T*>(t.g) + ahead.b * t.gb + ahead.n * t.gn + h * t.gh;
        xp = static_cast<const T*>(t.x) + ahead.b * t.sb + ahead.n * t.sn + h * t.sh;
        op = static_cast<T*>(t.out) + (static_cast<size_t>(ahead.token) * nh + h) * D;
        if (ahead.pos >= 0) copy_angles<T, D, kInter>(angles_at + ahead_unit * 4 * kStep, a.cos_t, a.sin_t, ahead.pos, sub);
        ahead_unit = ahead_unit + 1 == R::kStages ? 0 : ahead_unit + 1;
      }
      if (ahead.pos >= 0) c.is |= kPlace;
      if (h < nh) c.is |= kHead;
      if (ahead.pos >= 0 && h < nh) {
        const uint32_t dst = rows_at + ahead_row * R::kPieces * kStep;
        copy_row<D>(dst, gp, sub);
        if (kNorm) copy_row<D>(dst + R::kRow * kStep, xp, sub);
      }
      c.out = op;
      h += kRows;
      gp += kRows * t.gh;
      xp += kRows * t.sh;
      op += kRows * D;
      if (++ahead.it == ahead.its) ahead.next(a, share, lane);
    }
    ahead_row = ahead_row + 1 == R::kStages ? 0 : ahead_row + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
    return c;
  };
  Coming<T> line[R::kStages - 1];
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) line[i] = fetch();
  int row_slot = 0, unit_slot = 0;
  float2 c[4], s[4];
  while (line[0].is & kLive) {
    const Coming<T> at = line[0];
#pragma unroll
    for (int i = 0; i < R::kStages - 2; ++i) line[i] = line[i + 1];
    line[R::kStages - 2] = fetch();
    copies_wait<R::kStages - 1>();
    if (at.is & kFresh) {
      lds_angles(angles_at + unit_slot * 4 * kStep, c, s);
      unit_slot = unit_slot + 1 == R::kStages ? 0 : unit_slot + 1;
    }
    const uint32_t src = rows_at + row_slot * R::kPieces * kStep;
    row_slot = row_slot + 1 == R::kStages ? 0 : row_slot + 1;
    float2 o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_float2(0.f, 0.f);
    if (at.is & kPlace) {  // what a lane without a row holds stays in its row's lanes
      Raw<T> raw;
      float2 g[8], gr[8];
      lds_row(src, raw);
      unpack(raw, g);
      rotate_back<kInter>(g, c, s, gr);
      if constexpr (!kNorm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = gr[j];
      } else {
        float2 x[8];
        lds_row(src + R::kRow * kStep, raw);
        unpack(raw, x);
        const float r = row_rsqrt<D>(x, a.eps);
        float2 dot = make_float2(0.f, 0.f), gx[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          gx[j] = fmul2(gr[j], x[j]);
          dot = ffma2(gx[j], w[j], dot);
        }
        const float m = row_sum<D>(dot.x + dot.y) * (1.f / D) * r * r * r;
        const float2 r2 = make_float2(r, r), m2 = make_float2(-m, -m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (at.is & kHead) acc[j] = ffma2(gx[j], r2, acc[j]);
          o[j] = ffma2(fmul2(gr[j], w[j]), r2, fmul2(x[j], m2));
        }
      }
    }
    if (at.is & kHead) store_row<D>(at.out, sub, o);
  }
  copies_wait<0>();

  if constexpr (kNorm) {
    __shared__ float sums[kWarps][D];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 v = acc[j];
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      if (lane < kLanes) {
        const int f = feature<T, D>(j, sub);
        sums[warp][f] = v.x;
        sums[warp][f + 1] = v.y;
      }
    }
    __syncthreads();
    for (int f = threadIdx.x; f < D; f += kWarps * 32) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += sums[i][f];
      a.partial[static_cast<size_t>(blockIdx.x) * D + f] = v;
    }
  }
}

// dw = sum of the blocks' partial sums, in 64 bits and in a fixed order: grid (q or k,
// 32 features), 32 x 32 threads of one feature and every 32nd block each
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int q_blocks, int blocks,
                                                       void* dwq, void* dwk, int w_f32) {
  __shared__ double sums[32][33];
  const int f = lane_id(), part = warp_id();
  const int lo = blockIdx.x ? q_blocks : 0, hi = blockIdx.x ? blocks : q_blocks;
  const float* p = partial + blockIdx.y * 32 + f;
  double v = 0.0;
  wait_for_previous_kernel();  // its partial sums
#pragma unroll 8
  for (int i = lo + part; i < hi; i += 32) v += static_cast<double>(__ldcg(p + static_cast<size_t>(i) * D));
  sums[f][part] = v;
  __syncthreads();
  v = sums[part][f];  // warp `part` now holds feature `part`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (f == 0) {
    void* out = blockIdx.x ? dwk : dwq;
    const int at = blockIdx.y * 32 + part;
    if (w_f32)
      static_cast<float*>(out)[at] = static_cast<float>(v);
    else
      static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(static_cast<float>(v));
  }
}

template <typename T, int D, bool kNorm, bool kInter>
cudaError_t launch_fwd_k(const RopeArgs& a, cudaStream_t s) {
  if (a.blocks == 0) {
    const dim3 grid((a.tokens + kWarps - 1) / kWarps, a.q_groups + a.k_groups);
    return launch_behind(rope_fwd_kernel<T, D, kNorm, kInter>, grid, dim3(kWarps * 32), 0, s, a);
  }
  constexpr int kBytes = Ring<T, 1>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(rope_fwd_rounds_kernel<T, D, kNorm, kInter>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  return launch_behind(rope_fwd_rounds_kernel<T, D, kNorm, kInter>, dim3(a.blocks), dim3(kWarps * 32), kBytes, s, a);
}

template <typename T, int D>
cudaError_t launch_fwd_d(const RopeArgs& a, cudaStream_t s) {
  const bool norm = a.q.w != nullptr;
  if (norm) return a.interleaved ? launch_fwd_k<T, D, true, true>(a, s) : launch_fwd_k<T, D, true, false>(a, s);
  return a.interleaved ? launch_fwd_k<T, D, false, true>(a, s) : launch_fwd_k<T, D, false, false>(a, s);
}

template <typename T, int D, bool kNorm, bool kInter>
cudaError_t launch_bwd_k(const RopeArgs& a, cudaStream_t s) {
  constexpr int kBytes = Ring<T, kNorm ? 2 : 1>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(rope_bwd_kernel<T, D, kNorm, kInter>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  return launch_behind(rope_bwd_kernel<T, D, kNorm, kInter>, dim3(a.blocks), dim3(kWarps * 32), kBytes, s, a);
}

template <typename T, int D>
cudaError_t launch_bwd_d(const RopeArgs& a, cudaStream_t s) {
  const bool norm = a.q.w != nullptr;
  cudaError_t e = cudaSuccess;
  if (a.blocks == 0) {  // no row: the gains' gradients are still written (zero)
  } else if (norm && a.interleaved) e = launch_bwd_k<T, D, true, true>(a, s);
  else if (norm) e = launch_bwd_k<T, D, true, false>(a, s);
  else if (a.interleaved) e = launch_bwd_k<T, D, false, true>(a, s);
  else e = launch_bwd_k<T, D, false, false>(a, s);
  if (e != cudaSuccess || !norm) return e;
  return launch_behind(rope_dw_kernel<D>, dim3(2, D / 32), dim3(1024), 0, s, a.partial, a.q_blocks, a.blocks, a.dwq, a.dwk,
                       a.w_f32);
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs& a, int d, bool f32, cudaStream_t s) {
  if (f32) return d == 128 ? launch_fwd_d<float, 128>(a, s) : launch_fwd_d<float, 64>(a, s);
  return d == 128 ? launch_fwd_d<__nv_bfloat16, 128>(a, s) : launch_fwd_d<__nv_bfloat16, 64>(a, s);
}

cudaError_t launch_rope_bwd(const RopeArgs& a, int d, bool f32, cudaStream_t s) {
  if (f32) return d == 128 ? launch_bwd_d<float, 128>(a, s) : launch_bwd_d<float, 64>(a, s);
  return d == 128 ? launch_bwd_d<__nv_bfloat16, 128>(a, s) : launch_bwd_d<__nv_bfloat16, 64>(a, s);
}

}  // namespace fa
