// Rotary positions, and the quantised KV cache written and read back.
//
// Rotation of a pair (a, b) of a head at position p: the pair's step is its
// turns per position as a 64-bit binary fraction, so the phase p * step mod
// 2^64 is exact for every int32 position and the angle 2 pi * phase / 2^64 is
// formed once from its upper 32 bits (error 2^-24 of half a turn, independent
// of p; fp32 position * frequency is off by p * 2^-24 radians instead, a
// hundredth of a turn at a million).  Then
//     a' = a c - b s,  b' = b c + a s,   c, s = factor * cos, sin
// in fp32 with every product and sum rounded on its own, so that the codes of
// a rotated key do not depend on which products a compiler fuses.
//
// Quantisation of 64 values of a head: scale = FP16(fp32(max|x| / qmax)),
// code = rint(fp32(x / scale)) clamped to [-qmax - 1, qmax], qmax = 127 or 7.
//
// All three kernels read their input and write their output once.  A row (token, head) is spread over D / 16 threads; a
// thread holds two runs of 8 values, placed so that in the half layout the
// second run holds the partners of the first (i and i + R / 2):
// loads and stores are 16 bytes wide and a rotation never leaves its thread.
// The angles of a block's tokens are computed once into shared memory and shared
// by all their heads.  Reading back writes twice to four times what it reads: a
// thread takes 16 codes and stores 32 bytes at a time.
//
// Measured (GB300, copy rate 6.78 TB/s): rotation of 8191 x 40 heads of 128 in
// bf16, 168 MB in 31 us, 5.4 TB/s; of a quarter of 4097 x 24 heads of 256 in fp32,
// 201 MB in 38 us, 5.3 TB/s; 8001 tokens of 40 + 8 + 8 heads of 128 written, 214 MB in
// about 44 us, 4.9 TB/s (blocks of one token; no unit is full: issue 68 %, load/store
// 65 %, DRAM 43 %; walking over tokens in registers, with fewer blocks at a time, was
// 40 % slower); 65,521 tokens of 8 heads
// read back, 373 MB in 65 us, 5.8 TB/s.  A call of a few tokens takes 2 to 4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "host.h"
#include "kv_cache.cuh"
#include "nq.h"
#include "ptx.cuh"

namespace nq {
namespace {

constexpr int kRowThreads = 128;   // threads of a block that writes to or reads from the cache
constexpr int kRopeThreads = 256;  // and of one that only rotates
constexpr int kTableMax = 2048;    // angles of a block in shared memory
constexpr int kAppendTable = 512;  // the same, where heads have at most 256 values

struct Rotary {
  const int32_t* positions;
  const unsigned long long* steps;
  int half;          // rotated pairs: R / 2 (0: no rotation)
  int interleaved;
  float factor;
  float sign;        // -1 for the adjoint: the sine's sign
};

// One run of 8 values.
// (32-byte accesses: half the requests; `p` is 32-byte aligned)
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float2 angle_cs(const Rotary& ro, int pos, int i) {
  const unsigned long long phase =
      static_cast<unsigned long long>(static_cast<long long>(pos)) * ro.steps[i];
  const float angle = __fmul_rn(static_cast<float>(static_cast<int>(phase >> 32)),
                                static_cast<float>(3.14159265358979323846 / 2147483648.0));
  return make_float2(__fmul_rn(cosf(angle), ro.factor),
                     ro.sign * __fmul_rn(sinf(angle), ro.factor));
}
__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  const float y = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = x;
  b = y;
}

// The angles of `ntok` tokens from `tok0` into tab[token][pair].
__device__ __forceinline__ void fill_table(const Rotary& ro, long long tok0, int ntok,
                                           float2* tab) {
  for (int e = threadIdx.x; e < ntok * ro.half; e += blockDim.x) {
    const int t = e / ro.half;
    tab[e] = angle_cs(ro, ro.positions[tok0 + t], e - t * ro.half);
  }
}

// The two 8-value runs of thread `lane` of a row: first value of each.  Rotated
// runs come first (half layout: run j and run j + R / 16), the others follow
// in order.  R must be a multiple of 16.
__device__ __forceinline__ void runs_of(int lane, int half, int interleaved, int* first,
                                        int* second) {
  const int rot_lanes = half >> 3;
  if (!interleaved && lane < rot_lanes) {
    *first = 8 * lane;
    *second = 8 * lane + half;
  } else {
    *first = 16 * lane;
    *second = 16 * lane + 8;
  }
}

// Rotates a thread's two runs in place.
__device__ __forceinline__ void rotate_runs(const float2* tab, int lane, int half,
                                            int interleaved, float (&a)[8], float (&b)[8]) {
  if (lane >= (half >> 3)) return;
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate(a[i], b[i], tab[8 * lane + i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate(a[2 * i], a[2 * i + 1], tab[8 * lane + i]);
      rotate(b[2 * i], b[2 * i + 1], tab[8 * lane + 4 + i]);
    }
  }
}

// n / d as umulhi(n, ceil(2^32 / d)), exact for n d < 2^32 (below: at most
// 65535 rows of at most 256 threads); 0 stands for d = 1.
__device__ __forceinline__ int divide(int n, unsigned mul) {
  return mul ? static_cast<int>(__umulhi(static_cast<unsigned>(n), mul)) : n;
}
unsigned divisor(unsigned d) {
  return d == 1 ? 0u : static_cast<unsigned>(((1ull << 32) + d - 1) / d);
}

// The raw 16-byte words of two runs of 8 values.
template <typename T>
struct Raw {
  uint4 w[sizeof(T)];  // bf16: one word a run; fp32: two
  __device__ __forceinline__ void load(const T* x, int i0, int i1) {
    constexpr int n = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      w[i] = __ldcs(reinterpret_cast<const uint4*>(x + i0) + i);
      w[n + i] = __ldcs(reinterpret_cast<const uint4*>(x + i1) + i);
    }
  }
  __device__ __forceinline__ void get(int run, float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t u[4] = {w[run].x, w[run].y, w[run].z, w[run].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = w[2 * run + i];
        v[4 * i] = __uint_as_float(x.x);
        v[4 * i + 1] = __uint_as_float(x.y);
        v[4 * i + 2] = __uint_as_float(x.z);
        v[4 * i + 3] = __uint_as_float(x.w);
      }
    }
  }
};

struct RopeArgs {
  const void* x;
  void* out;
  long long tokens, xs_tok, xs_head, os_tok, os_head;  // strides in elements
  int heads, dim, tok_per_block;
  unsigned tok_mul, lane_mul;  // divide by the rows of a token, the threads of a row
  Rotary ro;
};

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) nq_rope_kernel(const RopeArgs a) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // rows of a thread in flight
  __shared__ float2 tab[kTableMax];
  griddep_wait();
  const long long tok0 = static_cast<long long>(blockIdx.x) * a.tok_per_block;
  const int ntok = static_cast<int>(min(static_cast<long long>(a.tok_per_block), a.tokens - tok0));
  const int lanes = a.dim >> 4, items = ntok * a.heads * lanes;
  Raw<T> raw[U];
  struct Place {
    int t, h, lane, i0, i1;
  };
  auto place = [&](int e) {
    Place p;
    const int row = divide(e, a.lane_mul);
    p.lane = e - row * lanes;
    p.t = divide(row, a.tok_mul);
    p.h = row - p.t * a.heads;
    runs_of(p.lane, a.ro.half, a.ro.interleaved, &p.i0, &p.i1);
    return p;
  };
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + u * kRopeThreads;
      if (e < items) {
        const Place p = place(e);
        raw[u].load(static_cast<const T*>(a.x) + (tok0 + p.t) * a.xs_tok + p.h * a.xs_head, p.i0, p.i1);
      }
    }
  };
  int base = blockIdx.y * (U * kRopeThreads) + threadIdx.x;
  load(base);
  fill_table(a.ro, tok0, ntok, tab);
  __syncthreads();
  while (base < items) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + u * kRopeThreads;
      if (e < items) {
        const Place p = place(e);
        T* y = static_cast<T*>(a.out) + (tok0 + p.t) * a.os_tok + p.h * a.os_head;
        float va[8], vb[8];
        raw[u].get(0, va);
        raw[u].get(1, vb);
        rotate_runs(tab + p.t * a.ro.half, p.lane, a.ro.half, a.ro.interleaved, va, vb);
        store8(y + p.i0, va);
        store8(y + p.i1, vb);
      }
    }
    base += gridDim.y * (U * kRopeThreads);
    load(base);
  }
}

// Any head size, rotated part and stride: a thread per pair or passed value.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) nq_rope_any_kernel(const RopeArgs a) {
  griddep_wait();
  const int per_row = a.dim - a.ro.half;  // half rotated pairs, dim - 2 half values that pass
  const long long n = a.tokens * a.heads * per_row;
  for (long long e = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x; e < n;
       e += static_cast<long long>(gridDim.x) * kRopeThreads) {
    const long long row = e / per_row;
    const int j = static_cast<int>(e - row * per_row);
    const long long t = row / a.heads;
    const int h = static_cast<int>(row - t * a.heads);
    const T* x = static_cast<const T*>(a.x) + t * a.xs_tok + h * a.xs_head;
    T* y = static_cast<T*>(a.out) + t * a.os_tok + h * a.os_head;
    if (j < a.ro.half) {
      const int i0 = a.ro.interleaved ? 2 * j : j;
      const int i1 = a.ro.interleaved ? 2 * j + 1 : j + a.ro.half;
      float u = to_f32(x[i0]), v = to_f32(x[i1]);
      rotate(u, v, angle_cs(a.ro, a.ro.positions[t], j));
      from_f32(u, y + i0);
      from_f32(v, y + i1);
    } else {
      y[j + a.ro.half] = x[j + a.ro.half];
    }
  }
}

struct AppendArgs {
  CacheView c;
  const void *q, *k, *v;
  __nv_bfloat16* q_out;
  const int32_t* slots;
  long long tokens;
  long long qs_tok, qs_head, ks_tok, ks_head, vs_tok, vs_head, os_tok, os_head;
  int q_heads, tok_per_block;
  unsigned tok_mul;
  Rotary ro;
  int* status;
};

// The larger of two magnitudes, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Codes of 8 values in the low bits of c: rint(fp32(x / s)) clamped to [lo, hi].
// k = rint(x * (1 / s)) is that code unless the quotient lies close to a half;
// the remainder x - k s (one rounding) tells: below (1/2 - 6.2e-5) s, the
// rounded quotient (off by 2^-24 of at most 128) is nearest to k too.  Else,
// and for scales below FP16's normal range, whose rounding can take a quotient
// beyond the codes, the division is made and clamped.
__device__ __forceinline__ void codes8(const float (&v)[8], float s, float lo, float hi,
                                       uint32_t (&c)[8]) {
  constexpr float kRound = 12582912.f;  // 1.5 2^23: a sum's low bits are the nearest integer
  const float inv = __frcp_rn(s), most = s * (0.5f - 6.2e-5f);
  bool divide = s < 6.103515625e-05f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fmaf(v[i], inv, kRound);
    divide |= fabsf(fmaf(-(r - kRound), s, v[i])) > most;
    c[i] = __float_as_uint(r);
  }
  if (divide) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = __float_as_uint(fminf(fmaxf(__fdiv_rn(v[i], s), lo), hi) + kRound);
  }
}

// Codes of one run of 8 values (two words of 8-bit codes, one of 4-bit ones)
// to their place in the row's codes.
__device__ __forceinline__ void store_codes(uint8_t* row, int first, int bits, const float (&v)[8],
                                            float s) {
  uint32_t c[8];
  if (s > 0.f && s <= 65504.f) {
    codes8(v, s, bits == 8 ? -128.f : -8.f, bits == 8 ? 127.f : 7.f, c);
  } else {  // a zero group, or one that cannot be held
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 0u;
  }
  if (bits == 8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040),
                         __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    *reinterpret_cast<uint2*>(row + first) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (c[i] & 0xFu) << (4 * i);
    *reinterpret_cast<uint32_t*>(row + (first >> 1)) = w;
  }
}

// Rows of a token: its query heads (rotated to q_out), its key heads (rotated,
// quantised into the cache) and its value heads (quantised).  The threads of
// a row sit in one warp (DIM / 16 of them), so a group's largest magnitude is
// a few shuffles away.
template <typename T, int DIM>
__global__ void __launch_bounds__(kRowThreads) nq_cache_append_kernel(const AppendArgs a) {
  constexpr int kLanes = DIM / 16, kGroups = DIM / 64, kRows = kRowThreads / kLanes;
  __shared__ float2 tab[kAppendTable];
  griddep_wait();
  const long long tok0 = static_cast<long long>(blockIdx.x) * a.tok_per_block;
  const int ntok = static_cast<int>(min(static_cast<long long>(a.tok_per_block), a.tokens - tok0));
  const int units = a.q_heads + 2 * a.c.kv_heads, rows = ntok * units;
  const int lane = threadIdx.x % kLanes;
  struct Place {
    int t, which, h, half, i0, i1;  // which: 0 k, 1 v, 2 q
  };
  auto place = [&](int row) {
    Place p;
    p.t = divide(row, a.tok_mul);
    const int u = row - p.t * units;
    p.which = u < a.q_heads ? 2 : (u - a.q_heads < a.c.kv_heads ? 0 : 1);
    p.h = p.which == 2 ? u : u - a.q_heads - p.which * a.c.kv_heads;
    p.half = p.which == 1 ? 0 : a.ro.half;
    runs_of(lane, p.half, a.ro.interleaved, &p.i0, &p.i1);
    return p;
  };
  // A row's words and slot, asked for a turn ahead: as soon as the words of the
  // turn are unpacked.  (Two rows a thread cost registers, and with them blocks.)
  Raw<T> raw;
  int next_slot = -1;
  auto load = [&](int row) {
    if (row < rows) {
      const Place p = place(row);
      const long long tok = tok0 + p.t;
      const T* x = p.which == 2   ? static_cast<const T*>(a.q) + tok * a.qs_tok + p.h * a.qs_head
                   : p.which == 0 ? static_cast<const T*>(a.k) + tok * a.ks_tok + p.h * a.ks_head
                                  : static_cast<const T*>(a.v) + tok * a.vs_tok + p.h * a.vs_head;
      raw.load(x, p.i0, p.i1);
      next_slot = p.which == 2 ? -1 : __ldg(a.slots + tok);
    }
  };
  int row = blockIdx.y * kRows + threadIdx.x / kLanes;
  load(row);
  fill_table(a.ro, tok0, ntok, tab);
  __syncthreads();
  // Every thread of a warp makes the same number of turns (the shuffles need
  // whole warps): the count goes by the block's first row.
  for (int first = blockIdx.y * kRows; first < rows; first += gridDim.y * kRows) {
    const bool live = row < rows;
    const Place p = place(live ? row : 0);
    const int slot = next_slot;
    float va[8], vb[8];
    raw.get(0, va);
    raw.get(1, vb);
    row += gridDim.y * kRows;
    load(row);
    const long long tok = tok0 + p.t;
    if (live) {
      rotate_runs(tab + p.t * a.ro.half, lane, p.half, a.ro.interleaved, va, vb);
      if (p.which == 2) {
        __nv_bfloat16* y = a.q_out + tok * a.os_tok + p.h * a.os_head;
        store8(y + p.i0, va);
        store8(y + p.i1, vb);
      }
    }
    const bool write = live && p.which != 2;
    if (!__any_sync(0xffffffffu, write)) continue;
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ma = max_nan(ma, fabsf(va[i]));
      mb = max_nan(mb, fabsf(vb[i]));
    }
    float most[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float m = max_nan((p.i0 >> 6) == g ? ma : 0.f, (p.i1 >> 6) == g ? mb : 0.f);
#pragma unroll
      for (int d = kLanes / 2; d >= 1; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
      most[g] = m;
    }
    if (!write) continue;
    if (slot < 0) continue;
    if (slot >= a.c.capacity) {
      if (lane == 0) atomicCAS(a.status, 0, kStatusRange);
      continue;
    }
    const int bits = a.c.bits[p.which];
    const float qmax = bits == 8 ? 127.f : 7.f;
    const long long r = cache_row(a.c, slot, p.h);
    uint8_t* codes = a.c.codes[p.which] + r * (DIM * bits / 8);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const __half sh = __float2half_rn(__fdiv_rn(most[g], qmax));
      const float s = __half2float(sh);
      if ((p.i0 >> 6) == g) s0 = s;
      if ((p.i1 >> 6) == g) s1 = s;
      if (lane == g) {
        a.c.scales[p.which][r * kGroups + g] = __half_as_ushort(sh);
        if (!(s <= 65504.f)) atomicCAS(a.status, 0, kStatusRange);
      }
    }
    store_codes(codes, p.i0, bits, va, s0);
    store_codes(codes, p.i1, bits, vb, s1);
  }
}

struct ReadArgs {
  CacheView c;
  const int32_t* slots;
  long long tokens;
  int tok_per_block;
  unsigned tok_mul;
  bool wide;         // outputs on 32-byte boundaries
  void* out[2];
  int* status;
};

// The fp32 values of 16 codes.
template <int BITS>
__device__ __forceinline__ void values16(const uint32_t* w, float s, float (&v)[16]) {
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = s * static_cast<float>(static_cast<signed char>(w[i >> 2] >> (8 * (i & 3))));
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // codes i and i + 4 of the word, exact in fp16
        const uint32_t h = sub_f16x2((w[k] >> (4 * i) & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);
        v[8 * k + i] = s * half_lo_to_float(h);
        v[8 * k + i + 4] = s * half_hi_to_float(h);
      }
  }
}
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    store32(p, w);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16], bool wide) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * k + i]);
    store_words(p + 8 * k, w, wide);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  store_words(p, w, wide);
}

// A thread's item is 16 codes: 32 bytes of bf16 values, one store, next to its
// neighbours'.  Items of a block: [token][kv head][D / 16].
template <typename T, int DIM, int BITS>
__device__ __forceinline__ void read_rows(const ReadArgs& a, int which) {
  constexpr int U = 8, kRuns = DIM / 16, W = BITS / 2;
  const long long tok0 = static_cast<long long>(blockIdx.x) * a.tok_per_block;
  const int ntok = static_cast<int>(min(static_cast<long long>(a.tok_per_block), a.tokens - tok0));
  const int items = ntok * a.c.kv_heads * kRuns;
  for (int base = threadIdx.x + blockIdx.z * (U * kRowThreads); base < items;
       base += gridDim.z * (U * kRowThreads)) {
    uint32_t w[U][W];
    uint16_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + u * kRowThreads;
#pragma unroll
      for (int i = 0; i < W; ++i) w[u][i] = 0u;
      sc[u] = 0;
      if (e < items) {
        const int row = e / kRuns, run = e % kRuns;
        const int t = divide(row, a.tok_mul), h = row - t * a.c.kv_heads;
        const int slot = __ldg(a.slots + tok0 + t);
        if (slot >= a.c.capacity) {
          atomicCAS(a.status, 0, kStatusRange);
        } else if (slot >= 0) {
          const long long r = cache_row(a.c, slot, h);
          const uint8_t* p = a.c.codes[which] + r * (DIM * BITS / 8) + run * (2 * BITS);
          if constexpr (BITS == 8) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p));
            w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
          } else {
            const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
            w[u][0] = x.x, w[u][1] = x.y;
          }
          sc[u] = __ldg(a.c.scales[which] + r * (DIM / 64) + (run >> 2));
        }
      }
    }
    T* y = static_cast<T*>(a.out[which]) + tok0 * a.c.kv_heads * DIM;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = base + u * kRowThreads;
      if (e >= items) break;
      float v[16];
      values16<BITS>(w[u], __half2float(__ushort_as_half(sc[u])), v);
      store16(y + static_cast<long long>(e) * 16, v, a.wide);
    }
  }
}

// blockIdx.y: keys, values.
template <typename T, int DIM>
__global__ void __launch_bounds__(kRowThreads) nq_cache_read_kernel(const ReadArgs a) {
  griddep_wait();
  if (a.c.bits[blockIdx.y] == 8) read_rows<T, DIM, 8>(a, blockIdx.y);
  else read_rows<T, DIM, 4>(a, blockIdx.y);
}

bool pdl_on() { return env_switch("NQ_PDL", 1) != 0; }

// How the row kernels cut their work: blocks of `tokens` tokens, each cut in
// `parts` over its items (a thread holds `unroll` of them at a time).
struct RowCut {
  int tokens, parts;
  unsigned mul;      // divides a block's row by the rows of a token
};

// A thread's items: up to `unroll`, fewer while there are too few for every
// thread that fits the GPU (`resident` an SM).  Tokens of a block by that; a
// token with more items than its threads take is cut into parts.
RowCut cut_rows(long long tokens, int rows_per_token, int threads_per_row, int unroll, int half,
                int sms, int resident, int threads = kRowThreads, int table = kTableMax) {
  const long long per_token = static_cast<long long>(rows_per_token) * threads_per_row;
  const long long deep = std::max<long long>(
      1, std::min<long long>(unroll, tokens * per_token / (static_cast<long long>(sms) * resident)));
  const long long turn = threads * deep;
  long long n = std::max<long long>(1, turn / per_token);
  if (half > 0) n = std::min<long long>(n, table / half);
  RowCut c;
  c.tokens = static_cast<int>(std::min<long long>(n, 64));
  const long long turns = (c.tokens * per_token + turn - 1) / turn;
  c.parts = static_cast<int>(tokens * per_token < static_cast<long long>(sms) * resident ? std::min<long long>(turns, 64) : 1);
  c.mul = c.tokens == 1 ? 1u : divisor(rows_per_token);  // (one token: every row is of token 0)
  return c;
}

int check_rotary(int dim, int rotary_dim, int layout) {
  if (rotary_dim < 0 || rotary_dim > dim || rotary_dim % 2) return NQ_EINVAL;
  if (layout != NQ_ROPE_HALF && layout != NQ_ROPE_INTERLEAVED) return NQ_EINVAL;
  return NQ_OK;
}

int cuda_rc(cudaError_t e) {
  if (e == cudaSuccess) return NQ_OK;
  (void)cudaGetLastError();
  return NQ_ECUDA;
}

bool mult(long long stride, int elem) { return stride * elem % 16 == 0; }

}  // namespace

int check_cache(const nq_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return NQ_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NQ_EINVAL;
  if ((c->k_bits != 4 && c->k_bits != 8) || (c->v_bits != 4 && c->v_bits != 8)) return NQ_EINVAL;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->pages < 1 || c->pages > INT_MAX / kPage)
    return NQ_EINVAL;
  if (!is_aligned16(c->k_codes) || !is_aligned16(c->v_codes) || !is_aligned16(c->k_scales) ||
      !is_aligned16(c->v_scales))
    return NQ_EALIGN;
  return NQ_OK;
}

}  // namespace nq

using namespace nq;

extern "C" {

int nq_rope_steps(int rotary_dim, double base, int scaling, double scale_factor,
                  double trained_context, uint64_t* steps, float* factor) {
  if (rotary_dim < 2 || rotary_dim % 2 || !(base > 1.0) || !steps || !factor) return NQ_EINVAL;
  if (scaling < NQ_ROPE_PLAIN || scaling > NQ_ROPE_YARN) return NQ_EINVAL;
  if (scaling != NQ_ROPE_PLAIN && !(scale_factor >= 1.0 && std::isfinite(scale_factor)))
    return NQ_EINVAL;
  if (scaling == NQ_ROPE_YARN && !(trained_context > 0.0)) return NQ_EINVAL;
  if (scaling == NQ_ROPE_NTK && rotary_dim < 4) return NQ_EINVAL;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == NQ_ROPE_NTK)
    base *= std::pow(scale_factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == NQ_ROPE_LINEAR) f /= scale_factor;
    if (scaling == NQ_ROPE_YARN) {
      const double keep =
          std::fmin(1.0, std::fmax(0.0, (trained_context * f / two_pi - 1.0) / (32.0 - 1.0)));
      f = f / scale_factor * (1.0 - keep) + f * keep;
    }
    const double turn = f / two_pi * 4294967296.0;  // < 2^32: at most one radian a position
    const double hi = std::floor(turn);
    steps[i] = (static_cast<uint64_t>(hi) << 32) +
               static_cast<uint64_t>(std::nearbyint((turn - hi) * 4294967296.0));
  }
  *factor = scaling == NQ_ROPE_YARN ? static_cast<float>(0.1 * std::log(scale_factor) + 1.0) : 1.f;
  return NQ_OK;
}

int nq_rope(const void* x, void* out, int dtype, int64_t tokens, int heads, int head_dim,
            int rotary_dim, int64_t x_token_stride, int64_t x_head_stride, int64_t out_token_stride,
            int64_t out_head_stride, const int32_t* positions, const uint64_t* steps, int layout,
            float factor, int adjoint, nq_stream_t stream) {
  if (tokens < 0 || tokens > INT_MAX || heads < 1 || heads > 65535 || head_dim < 1 ||
      head_dim > NQ_ROPE_MAX_DIM)
    return NQ_EINVAL;
  if (dtype != NQ_F32 && dtype != NQ_BF16) return NQ_EINVAL;
  if (int rc = check_rotary(head_dim, rotary_dim, layout)) return rc;
  if (tokens == 0) return NQ_OK;
  if (!x || !out || (rotary_dim && (!positions || !steps))) return NQ_EINVAL;
  if (!is_aligned16(x) || !is_aligned16(out) || !is_aligned16(steps)) return NQ_EALIGN;
  RopeArgs a;
  a.x = x;
  a.out = out;
  a.tokens = tokens;
  a.xs_tok = x_token_stride;
  a.xs_head = x_head_stride;
  a.os_tok = out_token_stride;
  a.os_head = out_head_stride;
  a.heads = heads;
  a.dim = head_dim;
  a.ro = Rotary{positions, reinterpret_cast<const unsigned long long*>(steps), rotary_dim / 2,
                layout == NQ_ROPE_INTERLEAVED, factor, adjoint ? -1.f : 1.f};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int elem = dtype == NQ_F32 ? 4 : 2;
  const bool wide = head_dim % 16 == 0 && rotary_dim % 16 == 0 && mult(x_token_stride, elem) &&
                    mult(x_head_stride, elem) && mult(out_token_stride, elem) &&
                    mult(out_head_stride, elem);
  if (!wide) {
    a.tok_per_block = 1;
    const long long n = tokens * heads * (head_dim - rotary_dim / 2);
    const long long blocks = (n + kRopeThreads - 1) / kRopeThreads;
    const dim3 grid(static_cast<unsigned>(blocks < 65536 ? blocks : 65536));
    return cuda_rc(dtype == NQ_F32
                       ? launch(nq_rope_any_kernel<float>, grid, dim3(kRopeThreads), 0, pdl_on(), st, a)
                       : launch(nq_rope_any_kernel<__nv_bfloat16>, grid, dim3(kRopeThreads), 0,
                                pdl_on(), st, a));
  }
  int *status, sms;
  if (int rc = device_status(&status, &sms)) return rc;
  const RowCut cut = cut_rows(tokens, heads, head_dim / 16, elem == 2 ? 4 : 2, rotary_dim / 2, sms, 768,
                              kRopeThreads);
  a.tok_per_block = cut.tokens;
  a.tok_mul = cut.mul;
  a.lane_mul = divisor(head_dim / 16);
  const dim3 grid(static_cast<unsigned>((tokens + cut.tokens - 1) / cut.tokens), cut.parts);
  return cuda_rc(dtype == NQ_F32
                     ? launch(nq_rope_kernel<float>, grid, dim3(kRopeThreads), 0, pdl_on(), st, a)
                     : launch(nq_rope_kernel<__nv_bfloat16>, grid, dim3(kRopeThreads), 0, pdl_on(),
                              st, a));
}

int nq_cache_append(const nq_kv_cache* cache, const void* k, const void* v, int dtype,
                    int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                    int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                    const void* q, void* q_out, int q_heads, int64_t q_token_stride,
                    int64_t q_head_stride, int64_t q_out_token_stride, int64_t q_out_head_stride,
                    const int32_t* positions, const uint64_t* steps, int rotary_dim, int layout,
                    float factor, nq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (tokens < 0 || tokens > INT_MAX || q_heads < 0 || q_heads > 65535) return NQ_EINVAL;
  if (dtype != NQ_F32 && dtype != NQ_BF16) return NQ_EINVAL;
  const int dim = cache->head_dim;
  if (int rc = check_rotary(dim, rotary_dim, layout)) return rc;
  if (rotary_dim % 16) return NQ_EINVAL;
  if (tokens == 0) return NQ_OK;
  if (!k || !v || !slots || (rotary_dim && (!positions || !steps))) return NQ_EINVAL;
  if (q_heads && (!q || !q_out)) return NQ_EINVAL;
  if (!is_aligned16(k) || !is_aligned16(v) || !is_aligned16(steps) ||
      (q_heads && (!is_aligned16(q) || !is_aligned16(q_out))))
    return NQ_EALIGN;
  const int elem = dtype == NQ_F32 ? 4 : 2;
  if (!mult(k_token_stride, elem) || !mult(k_head_stride, elem) || !mult(v_token_stride, elem) ||
      !mult(v_head_stride, elem) ||
      (q_heads && (!mult(q_token_stride, elem) || !mult(q_head_stride, elem) ||
                   !mult(q_out_token_stride, 2) || !mult(q_out_head_stride, 2))))
    return NQ_EALIGN;
  AppendArgs a;
  a.c = cache_view(*cache);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.slots = slots;
  a.tokens = tokens;
  a.qs_tok = q_token_stride;
  a.qs_head = q_head_stride;
  a.ks_tok = k_token_stride;
  a.ks_head = k_head_stride;
  a.vs_tok = v_token_stride;
  a.vs_head = v_head_stride;
  a.os_tok = q_out_token_stride;
  a.os_head = q_out_head_stride;
  a.q_heads = q_heads;
  a.ro = Rotary{positions, reinterpret_cast<const unsigned long long*>(steps), rotary_dim / 2,
                layout == NQ_ROPE_INTERLEAVED, factor, 1.f};
  int sms;
  if (int rc = device_status(&a.status, &sms)) return rc;
  const RowCut cut = cut_rows(tokens, q_heads + 2 * cache->kv_heads, dim / 16, 1, rotary_dim / 2, sms, 1024,
                              kRowThreads, kAppendTable);
  a.tok_per_block = cut.tokens;
  a.tok_mul = cut.mul;
  const dim3 grid(static_cast<unsigned>((tokens + cut.tokens - 1) / cut.tokens), cut.parts);
  void (*kern)(AppendArgs) = nullptr;
  if (dtype == NQ_F32)
    kern = dim == 64    ? nq_cache_append_kernel<float, 64>
           : dim == 128 ? nq_cache_append_kernel<float, 128>
                        : nq_cache_append_kernel<float, 256>;
  else
    kern = dim == 64    ? nq_cache_append_kernel<__nv_bfloat16, 64>
           : dim == 128 ? nq_cache_append_kernel<__nv_bfloat16, 128>
                        : nq_cache_append_kernel<__nv_bfloat16, 256>;
  return cuda_rc(launch(kern, grid, dim3(kRowThreads), 0, pdl_on(),
                        reinterpret_cast<cudaStream_t>(stream), a));
}

int nq_cache_read(const nq_kv_cache* cache, const int32_t* slots, int64_t tokens, void* k_out,
                  void* v_out, int dtype, nq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (tokens < 0 || tokens > INT_MAX || (dtype != NQ_F32 && dtype != NQ_BF16)) return NQ_EINVAL;
  if (tokens == 0) return NQ_OK;
  if (!slots || !k_out || !v_out) return NQ_EINVAL;
  if (!is_aligned16(k_out) || !is_aligned16(v_out)) return NQ_EALIGN;
  ReadArgs a;
  a.c = cache_view(*cache);
  a.slots = slots;
  a.tokens = tokens;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  int sms;
  if (int rc = device_status(&a.status, &sms)) return rc;
  const int dim = cache->head_dim;
  const RowCut cut = cut_rows(tokens, cache->kv_heads, dim / 16, 8, 0, sms, 512);
  a.tok_per_block = cut.tokens;
  a.tok_mul = cut.mul;
  const dim3 grid(static_cast<unsigned>((tokens + cut.tokens - 1) / cut.tokens), 2, cut.parts);
  void (*kern)(ReadArgs) = nullptr;
  if (dtype == NQ_F32)
    kern = dim == 64    ? nq_cache_read_kernel<float, 64>
           : dim == 128 ? nq_cache_read_kernel<float, 128>
                        : nq_cache_read_kernel<float, 256>;
  else
    kern = dim == 64    ? nq_cache_read_kernel<__nv_bfloat16, 64>
           : dim == 128 ? nq_cache_read_kernel<__nv_bfloat16, 128>
                        : nq_cache_read_kernel<__nv_bfloat16, 256>;
  return cuda_rc(launch(kern, grid, dim3(kRowThreads), 0, pdl_on(),
                        reinterpret_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
