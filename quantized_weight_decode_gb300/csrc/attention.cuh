// Shared by the kernels of the attention of drafted tokens over the quantised
// KV cache: arguments, the decode of codes to pairs, the split of the work, small PTX wrappers.
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j   over the keys token t sees:
//   the sequence's committed keys, and the drafted ones its tree bits name,
//   k_j = s c in 64-groups with FP16 scales s and 8- or 4-bit codes c.
//
// The keys' scales stay out of the matrix product: a group's dot product of
// query and (exact) codes is scaled in fp32 afterwards.  What the kernels do
// with the values' scales, and what they round, stands at each.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace nq {

constexpr int kMaxDrafts = 64;       // bits of a tree mask
constexpr float kLazyMax = 8.f;      // log2 by which a logit may pass the running reference

struct AttnArgs {
  CacheView c;
  const __nv_bfloat16* q;
  long long qs_tok, qs_head;         // strides in elements
  __nv_bfloat16* out;                // [total][q_heads][dim]
  float* lse;                        // [total][q_heads] or null
  long long total;
  int q_heads, group;                // group = q_heads / kv_heads
  const int32_t* table;              // [seqs][table_stride], `width` pages a row
  long long table_stride;
  int width;
  const int32_t* lengths;            // [seqs] committed tokens
  const int32_t* starts;             // [seqs + 1] first drafted token, or null: total / seqs each
  const unsigned long long* tree;    // [total] or null: a chain
  int seqs, max_drafts;
  float scale_log2;                  // scale * log2(e)
  int row_tiles, tile_rows;          // row tiles of a (sequence, kv head) at most, rows of one
  int tile_keys, min_stretch;        // keys of a tile, tiles of a block at least
  int blocks;                        // of the attention's grid
  float* part_o;                     // [pieces][tile_rows][dim]
  float2* part_ml;                   // the same without [dim]: (reference, sum)
  int2* unit_blocks;                 // [seqs * kv_heads * row_tiles] blocks of a unit's first and last tile
  int* status;
  unsigned long long wait_ns;        // bound of a wait in the kernel
};

using AttnKernel = void (*)(AttnArgs);
// The many-rows kernel of a head size and code widths.
struct ManyKernel {
  AttnKernel func;
  int threads, smem, max_rows;
};
ManyKernel many_kernel(int dim, int kb, int vb);

// What a sequence's blocks agree on.
struct SeqView {
  int first, drafts;                 // its drafted tokens
  int len, keys;                     // committed keys; committed and drafted
};

// (report: what is wrong with it goes to the status word, by every thread that asks)
__device__ __forceinline__ SeqView seq_view(const AttnArgs& a, int s, bool report = false) {
  SeqView v;
  bool bad = false;
  long long first, n;
  if (a.starts) {
    first = a.starts[s];
    n = static_cast<long long>(a.starts[s + 1]) - first;
  } else {
    n = a.total / a.seqs;
    first = n * s;
  }
  if (first < 0 || n < 0 || n > a.max_drafts || first + n > a.total) {
    bad = true;
    first = 0;
    n = 0;
  }
  long long len = a.lengths[s];
  const long long room = static_cast<long long>(a.width) * kPage;
  if (len < 0 || len + n > room) {
    bad = true;
    len = len < 0 ? 0 : len > room ? room : len;
  }
  v.first = static_cast<int>(first);
  v.drafts = static_cast<int>(n);
  v.len = static_cast<int>(len);
  v.keys = static_cast<int>(len + n > room ? room : len + n);
  if (report && bad) atomicCAS(a.status, 0, kStatusRange);
  return v;
}

// Bits of the drafted keys that drafted token t of the sequence sees.
__device__ __forceinline__ unsigned long long tree_bits(const AttnArgs& a, const SeqView& v, int t) {
  return a.tree ? a.tree[v.first + t] : (2ull << t) - 1ull;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// Two fp32 rounded to bf16: lo in bits 0-15, hi in bits 16-31.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Signed bytes 0 and 2 of w as a bf16 pair, exact: 128 + (c & 127) minus 128
// or 256 -- bit 7 of the byte is the exponent's lowest bit.
__device__ __forceinline__ uint32_t bytes_bf16(uint32_t w) {
  return sub_bf16x2(lop3_and_or(w, 0x007F007Fu, 0x43004300u),
                    lop3_and_or(w, 0x00800080u, 0x43004300u));
}
// (a & mask) ^ x in one instruction.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t x) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The same in fp16, where a byte fits the mantissa: 1024 + (c + 128) - 1152.
__device__ __forceinline__ uint32_t bytes_f16(uint32_t w) {
  return sub_f16x2(and_xor(w, 0x00FF00FFu, 0x64806480u), 0x64806480u);
}
// Signed nibbles 0 (1) of both halves of w as an fp16 pair: 1024 + (c + 8) - 1032,
// or 1024 + 16 (c + 8) over 16 minus 72.
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t w) {
  return sub_f16x2(and_xor(w, 0x000F000Fu, 0x64086408u), 0x64086408u);
}
__device__ __forceinline__ uint32_t nibbles4_f16(uint32_t w) {
  return fma_f16x2(and_xor(w, 0x00F000F0u, 0x64806480u), 0x2C002C00u, 0xD480D480u);
}
// Signed nibbles 0 of both halves of w as a bf16 pair, exact: 128 + (c ^ 8) - 136.
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t w) {
  return sub_bf16x2(and_xor(w, 0x000F000Fu, 0x43084308u), 0x43084308u);
}

// The line of all tiles (of a.tile_keys keys): sequence after sequence, in it unit
// (kv head, row tile) after unit, in it tile after tile (a unit with rows has
// one at least).  The blocks of the grid take equal stretches of it, so ragged
// lengths leave no block with more than another; a unit that several blocks
// share is merged from pieces, and the piece of block b of unit u (numbered
// over the batch) has the place b + u: along the line one of the two grows by
// one.  Computed by whole warps.  The one that a kernel builds with `report` (one
// warp of its first block) looks at every sequence, those without rows among
// them, and reports what is wrong with it.
__device__ __forceinline__ long long divide_long(long long n, long long d) {  // n, d >= 0
  if (((n | d) >> 32) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return n / d;
}
struct Place {
  int seq, row_tiles, tiles;  // of the sequence: units a kv head, tiles a unit
  int unit, tile;
  long long pos;              // where the sequence begins
};
struct Line {
  long long total;
  long long upto;             // tiles of the first 32 sequences, up to that of this lane
  static __device__ __forceinline__ void seq(const AttnArgs& a, int s, int* row_tiles, int* tiles,
                                             bool report = false) {
    const SeqView v = seq_view(a, s, report);
    *row_tiles = (v.drafts * a.group + a.tile_rows - 1) / a.tile_rows;
    *tiles = max(1, (v.keys + a.tile_keys - 1) / a.tile_keys);
  }
  // Tiles of the sequences s0 .. s0 + lane.
  static __device__ __forceinline__ long long scan(const AttnArgs& a, int s0, int lane, bool report = false) {
    long long n = 0;
    if (s0 + lane < a.seqs) {
      int rt, k;
      seq(a, s0 + lane, &rt, &k, report);
      n = static_cast<long long>(rt) * a.c.kv_heads * k;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long m = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += m;
    }
    return n;
  }
  __device__ __forceinline__ Line(const AttnArgs& a, int lane, bool report = false) {
    upto = scan(a, 0, lane, report);
    total = __shfl_sync(0xffffffffu, upto, 31);
    for (int s = 32; s < a.seqs; s += 32) total += __shfl_sync(0xffffffffu, scan(a, s, lane, report), 31);
  }
  __device__ __forceinline__ long long stretch(const AttnArgs& a, int blocks) const {
    const long long n = divide_long(total + blocks - 1, blocks);
    return n < a.min_stretch ? a.min_stretch : n;
  }
  // The place at `pos`, which is less than the total.
  __device__ __forceinline__ Place at(const AttnArgs& a, long long pos, int lane) const {
    long long before = 0, n = upto;
    int s0 = 0;
    unsigned after;
    while ((after = __ballot_sync(0xffffffffu, before + n > pos)) == 0u) {
      before += __shfl_sync(0xffffffffu, n, 31);
      s0 += 32;
      n = scan(a, s0, lane);
    }
    const int k = __ffs(after) - 1;
    Place p;
    p.seq = s0 + k;
    const long long prior = __shfl_sync(0xffffffffu, n, max(k - 1, 0));
    p.pos = before + (k ? prior : 0);
    seq(a, p.seq, &p.row_tiles, &p.tiles);
    p.unit = static_cast<int>(divide_long(pos - p.pos, p.tiles));
    p.tile = static_cast<int>((pos - p.pos) - static_cast<long long>(p.unit) * p.tiles);
    return p;
  }
};
// What the merge has to know of a unit: the blocks of its first and last tile.
__device__ __forceinline__ void note_unit(const AttnArgs& a, long long unit, int tile, int tiles, int all) {
  if (tile == 0) a.unit_blocks[unit].x = blockIdx.x;
  if (tile + tiles == all) a.unit_blocks[unit].y = blockIdx.x;
}

}  // namespace nq
