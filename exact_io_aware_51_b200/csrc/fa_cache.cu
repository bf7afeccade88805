// Writing new tokens into a paged KV cache and reading cached positions back,
// bf16 or 8-bit pools, d = 64 or 128, sm_100a.
//
// 8-bit rows (one position of one K/V head, d values x): a power-of-two scale
//     s = 2^e,  e the smallest integer >= -126 with max|x| <= 448 * 2^e,
// stored as the byte e + 127, and e4m3 codes round_to_nearest_even(x / s).  A
// power of two costs nothing against an arbitrary scale, because e4m3 is a
// floating-point format (the codes' relative error is 2^-4 either way), and it
// makes x / s exact, needs one byte instead of four, and leaves code * s exact in
// bf16 down to its subnormals.  A row holding an Inf or a NaN gets the byte 255
// (NaN) and NaN codes: the whole row reads back as NaN.  A zero row gets byte 1.
//
// Both directions are bound by the bytes they move.  A lane holds 16 features of
// a row, 8 from each half, so that neighbouring lanes' 16-byte accesses of bf16 and
// 8-byte accesses of codes touch whole 32-byte sectors; a row takes d / 16 lanes, and
// a warp takes 4 (d = 128) or 8 (d = 64) consecutive positions of one head, K and V,
// so the positions' scale bytes, which are neighbours in the pool, are written and
// read together.  One group of positions a warp: two or four, loaded ahead, took
// registers and with them warps away and measured 6 to 20% slower.
//
// Measured on a B200 (GPU time), 8 K/V heads, d = 128, 8-bit: reading back 8 contexts of
// 512 to 8192 positions (354 MB) 56 us, 6.3 TB/s; appending 8 prompts of 0 to 4096
// tokens (101 MB on average) 17.5 us, 5.8 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

struct Unit {
  int b, n, h;  // sequence, position index of this lane's row, K/V head
};

// warp -> (sequence, a.per groups of 512 / d positions, head), heads fastest
template <int D>
__device__ __forceinline__ bool unit_of(const CacheArgs& a, Unit& u) {
  const int kRows = 512 / D * a.per;
  const unsigned int w = blockIdx.x * kWarps + warp_id();
  if (w >= a.units) return false;
  const unsigned int t = w / a.Hkv;
  u.h = w - t * a.Hkv;
  u.b = t / a.groups;
  u.n = static_cast<int>(t - u.b * a.groups) * kRows + lane_id() / (D / 16);
  return true;
}

// pool row (page * page_size + slot) of position `pos`, or -1 (reported) if its page is no page of the pool
__device__ __forceinline__ long long pool_row(const CacheArgs& a, int b, int pos, int* page, int* slot) {
  const int p = pos >> a.page_shift;
  *slot = pos & (a.page_size - 1);
  *page = a.block_table[static_cast<size_t>(b) * a.max_pages + p];
  if (*page < 0 || *page >= a.num_pages) {
    atomicCAS(a.status, 0, kDevBadInput | 0xD2);
    return -1;
  }
  return (static_cast<long long>(*page) << a.page_shift) + *slot;
}

__device__ __forceinline__ size_t scale_index(const CacheArgs& a, int page, int h, int which, int slot) {
  return ((static_cast<size_t>(page) * a.Hkv + h) * 2 + which) * a.page_size + slot;
}

// Largest |x| of the row as a bf16 bit pattern (unsigned order: finite < Inf < NaN)
template <int D>
__device__ __forceinline__ uint32_t row_amax_bits(const uint4& a, const uint4& b) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
  m = __vmaxu2(m, __vmaxu2(__vmaxu2(b.x & kAbs, b.y & kAbs), __vmaxu2(b.z & kAbs, b.w & kAbs)));
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m & 0xffffu, m >> 16);
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int e = static_cast<int>(amax >> 7);  // biased exponent; 448 = 1.75 * 2^8
  if (e == 255) return 255u;
  return static_cast<uint32_t>(max(1, e - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0)));
}

__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, float inv) {
  return pack_e4m3x4(__uint_as_float(lo << 16) * inv, __uint_as_float(lo & 0xffff0000u) * inv,
                     __uint_as_float(hi << 16) * inv, __uint_as_float(hi & 0xffff0000u) * inv);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) cache_append_kernel(const CacheArgs a) {
  wait_for_previous_kernel();
  Unit u;
  if (!unit_of<D>(a, u)) return;
  const int sub = lane_id() % (D / 16);
  const int start = a.start[u.b];
  const int count = a.count ? a.count[u.b] : a.N;
  // a sequence whose new positions do not fit its table row is left out, and reported
  const bool fits = start >= 0 && count >= 0 && count <= a.N &&
                    static_cast<long long>(start) + count <= static_cast<long long>(a.max_pages) * a.page_size;
  if (!fits && lane_id() == 0) atomicCAS(a.status, 0, kDevBadInput | 0xD1);
  if (!fits) return;
  constexpr int kRows = 512 / D;
  const int end = u.n - lane_id() / (D / 16) + a.per * kRows;  // the same for every lane
  for (int first = end - a.per * kRows; first < min(end, count); first += kRows, u.n += kRows) {
    const bool ok = u.n < count;
    uint4 x[2][2];
#pragma unroll
    for (int w = 0; w < 2; ++w) x[w][0] = x[w][1] = make_uint4(0u, 0u, 0u, 0u);
    long long row = -1;
    int page = 0, slot = 0;
    if (ok) {
      const CacheTensor& tk = a.t[0];
      const CacheTensor& tv = a.t[1];
      const uint4* pk = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(tk.x) + u.b * tk.sb +
                                                       u.n * tk.sn + u.h * tk.sh + 8 * sub);
      const uint4* pv = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(tv.x) + u.b * tv.sb +
                                                       u.n * tv.sn + u.h * tv.sh + 8 * sub);
      x[0][0] = pk[0];
      x[0][1] = pk[D / 16];
      x[1][0] = pv[0];
      x[1][1] = pv[D / 16];
      row = pool_row(a, u.b, start + u.n, &page, &slot);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const size_t at = (static_cast<size_t>(row) * a.Hkv + u.h) * D + 8 * sub;
      if constexpr (kFp8) {
        const uint32_t sb = scale_byte(row_amax_bits<D>(x[w][0], x[w][1]));  // every lane of the warp
        // 2^-(byte - 127); NaN for byte 255, so that every code is NaN
        const float inv = sb == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - sb) << 23);
        if (row >= 0) {
          uint2* p = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.t[w].pool) + at);
          p[0] = make_uint2(codes4(x[w][0].x, x[w][0].y, inv), codes4(x[w][0].z, x[w][0].w, inv));
          p[D / 16] = make_uint2(codes4(x[w][1].x, x[w][1].y, inv), codes4(x[w][1].z, x[w][1].w, inv));
          if (sub == 0) a.kv_scale[scale_index(a, page, u.h, w, slot)] = static_cast<uint8_t>(sb);
        }
      } else if (row >= 0) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.t[w].pool) + at);
        p[0] = x[w][0];
        p[D / 16] = x[w][1];
      }
    }
  }
}

// four e4m3 codes times the scale, as two bf16 pairs
__device__ __forceinline__ uint2 values4(uint32_t codes, float scale) {
  uint32_t h0, h1;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(h0), "=r"(h1)
      : "r"(codes));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  if (byte == 0u) return __uint_as_float(0x00400000u);    // 2^-127
  if (byte == 255u) return __uint_as_float(0x7fc00000u);  // NaN
  return __uint_as_float(byte << 23);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const CacheArgs a) {
  wait_for_previous_kernel();
  Unit u;
  if (!unit_of<D>(a, u)) return;
  const int sub = lane_id() % (D / 16);
  const int len = a.start[u.b];  // seqlens
  const bool good = len >= 0 && len <= static_cast<long long>(a.max_pages) * a.page_size;
  if (!good && lane_id() == 0) atomicCAS(a.status, 0, kDevBadInput | 0xD1);
  if (u.n >= a.N) return;
  long long row = -1;
  int page = 0, slot = 0;
  if (good && u.n < len) row = pool_row(a, u.b, u.n, &page, &slot);
  uint4 y[2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w) y[w][0] = y[w][1] = make_uint4(0u, 0u, 0u, 0u);
  if (row >= 0) {
    const size_t at = (static_cast<size_t>(row) * a.Hkv + u.h) * D + 8 * sub;
    if constexpr (kFp8) {
      uint2 c[2][2];
      uint32_t sb[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.t[w].pool) + at);
        c[w][0] = p[0];
        c[w][1] = p[D / 16];
        sb[w] = a.kv_scale[scale_index(a, page, u.h, w, slot)];
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float sc = scale_value(sb[w]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint2 p0 = values4(c[w][i].x, sc), p1 = values4(c[w][i].y, sc);
          y[w][i] = make_uint4(p0.x, p0.y, p1.x, p1.y);
        }
      }
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.t[w].pool) + at);
        y[w][0] = p[0];
        y[w][1] = p[D / 16];
      }
    }
  }
  const size_t to = ((static_cast<size_t>(u.b) * a.N + u.n) * a.Hkv + u.h) * D + 8 * sub;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.t[w].out) + to);
    p[0] = y[w][0];
    p[D / 16] = y[w][1];
  }
}

template <int D>
cudaError_t launch_d(const CacheArgs& a, bool fp8, bool append, cudaStream_t s) {
  const unsigned int blocks = (a.units + kWarps - 1) / kWarps;
  const dim3 grid(blocks), block(kWarps * 32);
  if (append) return launch_behind(fp8 ? cache_append_kernel<D, true> : cache_append_kernel<D, false>, grid, block, 0, s, a);
  return launch_behind(fp8 ? cache_read_kernel<D, true> : cache_read_kernel<D, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_cache(const CacheArgs& a, int d, bool fp8, bool append, cudaStream_t s) {
  return d == 128 ? launch_d<128>(a, fp8, append, s) : launch_d<64>(a, fp8, append, s);
}

}  // namespace fa
