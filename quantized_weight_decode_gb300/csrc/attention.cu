// Attention of drafted tokens over the quantised KV cache: the kernel for few
// rows, the merge of pieces, and the C entry points.
//
// Few rows (a row is a drafted token's query head of one kv head): the cache
// is read once and everything else is small, so the floor is the stream of
// codes from memory.  Each warp works alone on blocks of 16 keys:
//   S^T[16 keys x 8 rows]   = codes_K[16 x D] . Q^T        (mma m16n8k16, fp16)
//   O^T[D x 8 rows]        += codes_V^T[D x 16] . P^T      (mma m16n8k16, bf16)
// Keys and value channels are the long sides (the MMA's 16-row side), so 5
// rows fill 5 / 8 of the tensor work instead of 5 / 16.  The order of a
// contraction is free, so a thread's 16 bytes of a key are the contraction
// slices of its own fragment (the query is permuted to match), and its 8
// bytes of four values are 8 output channels of its fragment.  A lane copies
// exactly those bytes for itself (asynchronously, several blocks ahead,
// through shared memory): coalesced, free of bank conflicts, with no barrier
// in the loop.  Loading them into registers a block ahead instead kept too
// few bytes in flight: 98 us against 85 for 16 sequences of up to 16 k keys.
//
// Codes, and the queries times a power of two a row, are exact in fp16.  A
// probability times its value group's scale is the sum of two bf16 (2^-17;
// bf16 has the range that a product of a probability and any FP16 scale
// needs); one bf16 alone cost 2.5 us less of 83 and put the error against 64
// bits from 0.0017, the output's own rounding, to 0.0024.  The softmax keeps its
// running reference lazily: it moves only when a logit passes it by 2^8 (one
// vote a block instead of six shuffles); sums and outputs stay in fp32.
//
// Measured (GB300): 16 sequences of up to 16 k keys, 40 query heads of 128 on 8,
// 8 bits: 395 MB in 83 us, 4.8 TB/s.  Copies and arithmetic bound it together:
// the copies alone take 71 us, all but the copies 70, and no unit is full (DRAM
// 62 %, issue 54 %, ALU 47 %).  Five blocks an SM spill: 87 us; three: 82.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "attention.cuh"
#include "host.h"
#include "nq.h"
#include "tcgen05.cuh"

namespace nq {
namespace {

constexpr int kWarpsA = 4;  // warps of a block of the few-rows kernel
constexpr int kKeys = 16;   // keys of a warp's block

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Blocks of an SM: what the registers allow.
constexpr int few_blocks(int dim, int nt) { return dim == 64 ? (nt == 1 ? 5 : 4) : dim == 128 && nt == 1 ? 4 : 2; }

// A warp's blocks of codes and scales on their way through shared memory: a
// lane copies (asynchronously) the very bytes that it will use, so that
// nothing has to be waited for but the lane's own copies.
template <int D, int KB, int VB, int NT>
struct Few {
  static constexpr int G = D / 64;
  static constexpr int KW = KB / 2;  // words of a thread's 16 key codes of a group
  static constexpr int VW = VB / 4;  // words of a thread's 8 value codes of a group
  static constexpr int SB = G == 4 ? 8 : 4;  // bytes that hold a key's scales
  static constexpr int off_v = 2 * G * 32 * KW * 4, off_ks = off_v + 4 * G * 32 * VW * 4;
  static constexpr int off_vs = off_ks + 2 * 32 * SB, kStage = off_vs + 2 * 32 * SB;
  static constexpr int kRoom = (227 * 1024 / few_blocks(D, NT) - 1024) / (kWarpsA * kStage);
  static constexpr int NS = kRoom > 6 ? 6 : kRoom;  // blocks of a warp in flight
  static constexpr int kOut = kWarpsA * 8 * NT * (D + 2) * 4;  // the warps' outputs, at the end
  static constexpr int bytes = NS * kWarpsA * kStage > kOut ? NS * kWarpsA * kStage : kOut;
  static_assert(NS >= 2, "");
};

template <int D, int KB, int VB, int NT>
__global__ void __launch_bounds__(kWarpsA * 32, few_blocks(D, NT)) nq_attn_few_kernel(const AttnArgs a) {
  using F = Few<D, KB, VB, NT>;
  constexpr int G = F::G, KW = F::KW, VW = F::VW, SB = F::SB, NS = F::NS;
  constexpr int R = 8 * NT;          // rows of a block
  extern __shared__ __align__(16) float sm_o[];  // [warps][R][D], then (reference, sum) [warps][R]
  float2* sm_ml = reinterpret_cast<float2*>(sm_o + kWarpsA * R * D);
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 2, r = lane & 3;
  const Line line(a, lane, blockIdx.x == 0 && warp == 0);
  const long long stretch = line.stretch(a, gridDim.x);
  const long long pos_end = min(line.total, (blockIdx.x + 1) * stretch);
  long long pos = blockIdx.x * stretch;
  while (pos < pos_end) {
  const Place pl = line.at(a, pos, lane);
  const SeqView v = seq_view(a, pl.seq);
  const int rows = v.drafts * a.group, head = pl.unit / pl.row_tiles, tile = pl.unit - head * pl.row_tiles;
  const int tiles = static_cast<int>(min(static_cast<long long>(pl.tiles - pl.tile), pos_end - pos));
  const bool whole = tiles == pl.tiles;
  const long long unit = static_cast<long long>(pl.seq) * a.c.kv_heads * a.row_tiles + pl.unit;
  const long long slot = blockIdx.x + unit;
  if (threadIdx.x == 0 && a.unit_blocks) note_unit(a, unit, pl.tile, tiles, pl.tiles);
  pos += tiles;

  // (the first copies go out before anything else is loaded)
  const int32_t* table = a.table + pl.seq * a.table_stride;
  const int pages = a.c.capacity / kPage;
  const int blk_end = min((pl.tile + tiles) * (kPage / kKeys), (v.keys + kKeys - 1) / kKeys);
  int blk = pl.tile * (kPage / kKeys) + warp;

  uint8_t* ring = reinterpret_cast<uint8_t*>(sm_o) + warp * (NS * F::kStage);
  const uint32_t ring_at = smem_addr(ring);
  unsigned oks = 0u;                 // bit i: the page of the block in place i is one of the cache's
  int ahead = blk, place = 0;        // the block to be copied next, and its place
  int page = blk < blk_end ? __ldg(table + blk / (kPage / kKeys)) : 0;
  // Copies block `ahead` (codes and scales of a page that is none are those of page 0).
  auto issue = [&]() {
    if (ahead < blk_end) {
      const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(pages);
      if (!ok && lane == 0) atomicCAS(a.status, 0, kStatusRange);
      const long long row = (static_cast<long long>(ok ? page : 0) * a.c.kv_heads + head) * kPage +
                            (ahead % (kPage / kKeys)) * kKeys;
      oks = (oks & ~(1u << place)) | static_cast<unsigned>(ok) << place;
      const uint32_t to = ring_at + place * F::kStage + lane * 4;
      const uint8_t* kp = a.c.codes[0] + (row + q) * (D * KB / 8) + 16 * r * KB / 8;
      const uint8_t* vp = a.c.codes[1] + (row + 2 * r) * (D * VB / 8) + 8 * q * VB / 8;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int g = 0; g < G; ++g)
          copy_async<KW * 4>(to + lane * (KW * 4 - 4) + (e * G + g) * (32 * KW * 4),
                             kp + 8 * e * (D * KB / 8) + 64 * g * KB / 8);
      const uint8_t* ks = reinterpret_cast<const uint8_t*>(a.c.scales[0] + (row + q) * G);
      const uint8_t* vs = reinterpret_cast<const uint8_t*>(a.c.scales[1] + (row + q) * G);
      if constexpr (G == 1) {  // (the aligned pair that holds it)
        ks -= (q & 1) * 2;
        vs -= (q & 1) * 2;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        copy_async<SB>(to + lane * (SB - 4) + F::off_ks + e * (32 * SB), ks + 8 * e * G * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int g = 0; g < G; ++g)
          copy_async<VW * 4>(to + lane * (VW * 4 - 4) + F::off_v + (e * G + g) * (32 * VW * 4),
                             vp + ((e & 1) + 8 * (e >> 1)) * (D * VB / 8) + 64 * g * VB / 8);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        copy_async<SB>(to + lane * (SB - 4) + F::off_vs + e * (32 * SB), vs + 8 * e * G * 2);
    }
    copy_commit();
    ahead += kWarpsA;
    if (++place == NS) place = 0;
    if (ahead < blk_end) page = __ldg(table + ahead / (kPage / kKeys));
  };
  auto scale_of = [&](const uint8_t* p, int g) {  // of the scales at p
    uint32_t w;
    if constexpr (G == 4) w = reinterpret_cast<const uint32_t*>(p)[g >> 1];
    else w = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (G == 1) return (q & 1) ? half_hi_to_float(w) : half_lo_to_float(w);
    else return (g & 1) ? half_hi_to_float(w) : half_lo_to_float(w);
  };
#pragma unroll 1
  for (int i = 0; i < NS; ++i) issue();

  // Queries as the MMA's B operand, in the order of the key codes: fp16, each
  // row times a power of two that takes its largest magnitude into [2^7, 2^8)
  // (exact but for values 2^-21 below the row's largest, off by 2^-32 of that).
  uint32_t qf[NT][G][4][2];
  float undo[NT][2];                 // the logits' factor of this thread's rows
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int rr = tile * R + 8 * n + q;
    const bool live = rr < rows;
    const int t = live ? rr / a.group : 0, h = head * a.group + (live ? rr - t * a.group : 0);
    const __nv_bfloat16* qp = a.q + (v.first + t) * a.qs_tok + h * a.qs_head + 16 * r;
    uint32_t w[G][8];
    unsigned most = 0u;              // the largest finite magnitude's bits
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[g][i] = 0u;
      if (live) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(qp + 64 * g));
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(qp + 64 * g + 8));
        w[g][0] = x.x, w[g][1] = x.y, w[g][2] = x.z, w[g][3] = x.w;
        w[g][4] = y.x, w[g][5] = y.y, w[g][6] = y.z, w[g][7] = y.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned lo = w[g][i] & 0x7FFFu, hi = (w[g][i] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) most = max(most, lo);
        if (hi < 0x7F80u) most = max(most, hi);
      }
    }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const int ex = most == 0u ? 0 : max(-120, min(120, 134 - static_cast<int>(most >> 7)));
    const float up = __int_as_float((ex + 127) << 23);
    const float down = a.scale_log2 * __int_as_float((127 - ex) << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e) undo[n][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * r + e));
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = KB == 8 ? w[g][2 * j] : w[g][4 * (j >> 1) + (j & 1)];
        const uint32_t hi = KB == 8 ? w[g][2 * j + 1] : w[g][4 * (j >> 1) + (j & 1) + 2];
        qf[n][g][j][0] = cvt_f16x2(__uint_as_float(lo << 16) * up, __uint_as_float(hi << 16) * up);
        qf[n][g][j][1] = cvt_f16x2(__uint_as_float(lo & 0xFFFF0000u) * up, __uint_as_float(hi & 0xFFFF0000u) * up);
      }
  }
  // This thread's rows (two per row block): tree bits, reference, sum, outputs.
  unsigned long long bits[NT][2];
  float m[NT][2], l[NT][2], o[NT][G][4][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = tile * R + 8 * n + 2 * r + e;
      bits[n][e] = rr < rows ? tree_bits(a, v, rr / a.group) : 0ull;
      m[n][e] = -INFINITY;
      l[n][e] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][g][i][2 * e] = o[n][g][i][2 * e + 1] = 0.f;
    }

  while (blk < blk_end) {
    const uint8_t* mine = ring + place * F::kStage;  // (the oldest block's place is the next to be filled)
    copy_wait<NS - 1>();
    // S^T: a group's dot products, then its scales.
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float acc[NT][4];
      uint32_t kw[2][KW];
#pragma unroll
      for (int e = 0; e < 2; ++e) load_words<KW>(mine + (e * G + g) * (32 * KW * 4) + lane * KW * 4, kw[e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t f[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (KB == 8) {
            f[e][0] = bytes_f16(kw[e][j]);
            f[e][1] = bytes_f16(kw[e][j] >> 8);
          } else {
            const uint32_t w = j & 1 ? kw[e][j >> 1] >> 8 : kw[e][j >> 1];
            f[e][0] = nibbles_f16(w);
            f[e][1] = nibbles4_f16(w);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (j == 0) mma_16816_f16_zc(acc[n], f[0][0], f[1][0], f[0][1], f[1][1], qf[n][g][j][0], qf[n][g][j][1]);
          else mma_16816_f16(acc[n], f[0][0], f[1][0], f[0][1], f[1][1], qf[n][g][j][0], qf[n][g][j][1]);
        }
      }
      const float s0 = scale_of(mine + F::off_ks + lane * SB, g);
      const float s1 = scale_of(mine + F::off_ks + (32 + lane) * SB, g);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x[n][0] = fmaf(acc[n][0], s0, x[n][0]);
        x[n][1] = fmaf(acc[n][1], s0, x[n][1]);
        x[n][2] = fmaf(acc[n][2], s1, x[n][2]);
        x[n][3] = fmaf(acc[n][3], s1, x[n][3]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] *= undo[n][i & 1];
    const int key0 = blk * kKeys + q;
    const bool ok = oks >> place & 1u;
    const bool masked = (blk + 1) * kKeys > v.len || !ok;
    // Keys that a row does not see.
    if (masked) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 8 * (i >> 1), d = key - v.len;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool seen = ok && key < v.keys && (d < 0 || (bits[n][i & 1] >> d & 1ull));
          if (!seen) x[n][i] = -INFINITY;
        }
      }
    }
    // Move the references if a logit passes them by far.
    bool far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) far |= x[n][i] > m[n][i & 1] + kLazyMax;
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(x[n][e], x[n][e + 2]);
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          if (top > m[n][e] + kLazyMax) {  // (by row: what another row sees does not matter)
            const float f = ex2(m[n][e] - top);  // 0 from -inf
            m[n][e] = top;
            l[n][e] *= f;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[n][g][i][e] *= f;
                o[n][g][i][2 + e] *= f;
              }
          }
        }
    }
    float p[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[n][i] = masked && x[n][i] == -INFINITY ? 0.f : ex2(x[n][i] - m[n][i & 1]);
        l[n][i & 1] += p[n][i];
      }
    // O^T: probabilities times the value scales as the B operand, per group.
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float s0 = scale_of(mine + F::off_vs + lane * SB, g);
      const float s1 = scale_of(mine + F::off_vs + (32 + lane) * SB, g);
      uint32_t vw[4][VW];
#pragma unroll
      for (int e = 0; e < 4; ++e) load_words<VW>(mine + F::off_v + (e * G + g) * (32 * VW * 4) + lane * VW * 4, vw[e]);
      uint32_t b[NT][2], bl[NT][2];  // probabilities, and what their rounding left
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p0 = p[n][0] * s0, p1 = p[n][1] * s0, p2 = p[n][2] * s1, p3 = p[n][3] * s1;
        if (masked) {  // (a key that is not seen may have any scale, NaN too)
          if (p[n][0] == 0.f) p0 = 0.f;
          if (p[n][1] == 0.f) p1 = 0.f;
          if (p[n][2] == 0.f) p2 = 0.f;
          if (p[n][3] == 0.f) p3 = 0.f;
        }
        const uint32_t h0 = cvt_bf16x2(p0, p1), h1 = cvt_bf16x2(p2, p3);
        b[n][0] = movmatrix_trans(h0);
        b[n][1] = movmatrix_trans(h1);
        bl[n][0] = movmatrix_trans(cvt_bf16x2(p0 - bf16_lo(h0), p1 - bf16_hi(h0)));
        bl[n][1] = movmatrix_trans(cvt_bf16x2(p2 - bf16_lo(h1), p3 - bf16_hi(h1)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t f[2][2];  // [keys 2r.. | 2r + 8..][channel 2i | 2i + 1]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (VB == 8) {
            const uint32_t w = prmt(vw[2 * e][i >> 1], vw[2 * e + 1][i >> 1], i & 1 ? 0x7632 : 0x5410);
            f[e][0] = bytes_bf16(w);
            f[e][1] = bytes_bf16(w >> 8);
          } else {
            const uint32_t w = prmt(vw[2 * e][0], vw[2 * e + 1][0], i & 2 ? 0x7632 : 0x5410);
            f[e][0] = nibbles_bf16(w >> (8 * (i & 1)));
            f[e][1] = nibbles_bf16(w >> (8 * (i & 1) + 4));
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_16816(o[n][g][i], f[0][0], f[0][1], f[1][0], f[1][1], b[n][0], b[n][1]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_16816(o[n][g][i], f[0][0], f[0][1], f[1][0], f[1][1], bl[n][0], bl[n][1]);
      }
    }
    issue();
    blk += kWarpsA;
  }
  copy_wait<0>();
  __syncthreads();  // the rings become the place of the outputs

  // Merge the warps: references and sums, then outputs.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
      const int rr = 8 * n + 2 * r + e;
      if (q == 0) sm_ml[warp * R + rr] = make_float2(m[n][e], l[n][e]);
      float* dst = sm_o + (warp * R + rr) * D + 8 * q;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        *reinterpret_cast<float4*>(dst + 64 * g) =
            make_float4(o[n][g][0][e], o[n][g][0][2 + e], o[n][g][1][e], o[n][g][1][2 + e]);
        *reinterpret_cast<float4*>(dst + 64 * g + 4) =
            make_float4(o[n][g][2][e], o[n][g][2][2 + e], o[n][g][3][e], o[n][g][3][2 + e]);
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (D / 4); e += kWarpsA * 32) {
    const int rr = e / (D / 4), d = (e - rr * (D / 4)) * 4;
    if (tile * R + rr >= rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarpsA; ++w) top = fmaxf(top, sm_ml[w * R + rr].x);
    float sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarpsA; ++w) {
      const float2 ml = sm_ml[w * R + rr];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      // A row that a warp's keys leave empty has a zero sum and zero outputs
      // (NaN if a key it does see is NaN, its reference then still -inf).
      const float4 z = *reinterpret_cast<const float4*>(sm_o + (w * R + rr) * D + d);
      const float k = ml.x == -INFINITY ? ml.y : f * ml.y;
      sum += k;
      y.x = fmaf(f, z.x, y.x);
      y.y = fmaf(f, z.y, y.y);
      y.z = fmaf(f, z.z, y.z);
      y.w = fmaf(f, z.w, y.w);
    }
    const int t = (tile * R + rr) / a.group;
    const int h = head * a.group + (tile * R + rr) - t * a.group;
    const long long id = static_cast<long long>(v.first + t) * a.q_heads + h;
    if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(a.out + id * D + d) =
          make_uint2(cvt_bf16x2(y.x * inv, y.y * inv), cvt_bf16x2(y.z * inv, y.w * inv));
      if (a.lse && d == 0)
        a.lse[id] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
    } else {
      const long long at = slot * a.tile_rows + rr;
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = y;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
    }
  }
  __syncthreads();  // (the next stretch writes here)
  }
}

// Merges the pieces of each row: a block of four warps per row, the pieces in
// turn to the warps, the warps' sums in their order.
template <int D>
__global__ void __launch_bounds__(128) nq_attn_merge_kernel(const AttnArgs a) {
  __shared__ float part[4][D];
  __shared__ float sums[4];
  griddep_wait();
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x / (a.max_drafts * a.group), row = blockIdx.x - head * (a.max_drafts * a.group);
  const SeqView v = seq_view(a, s);
  if (row >= v.drafts * a.group) return;
  const int row_tiles = (v.drafts * a.group + a.tile_rows - 1) / a.tile_rows;
  const int rtile = row / a.tile_rows, n = row - rtile * a.tile_rows;
  const long long slot = static_cast<long long>(s) * a.c.kv_heads * a.row_tiles + head * row_tiles + rtile;
  const int2 blocks = a.unit_blocks[slot];
  if (blocks.x == blocks.y) return;                     // one block had it all
  float top = -INFINITY;
  for (int b = blocks.x + lane; b <= blocks.y; b += 32) top = fmaxf(top, a.part_ml[(slot + b) * a.tile_rows + n].x);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float sum = 0.f, y[D / 32] = {};
#pragma unroll 4
  for (int b = blocks.x + warp; b <= blocks.y; b += 4) {
    const long long at = (slot + b) * a.tile_rows + n;
    const float2 ml = a.part_ml[at];
    // (a piece without keys has a zero sum and zero outputs; NaN where it saw one)
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    sum += ml.x == -INFINITY ? ml.y : f * ml.y;
    const float* z = a.part_o + at * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 w = *reinterpret_cast<const float2*>(z + 64 * i + 2 * lane);
      y[2 * i] = fmaf(f, w.x, y[2 * i]);
      y[2 * i + 1] = fmaf(f, w.y, y[2 * i + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    *reinterpret_cast<float2*>(&part[warp][64 * i + 2 * lane]) = make_float2(y[2 * i], y[2 * i + 1]);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const int t = row / a.group;
  const long long id = static_cast<long long>(v.first + t) * a.q_heads + head * a.group + row - t * a.group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (2 * threadIdx.x < D) {
    const int i = 2 * threadIdx.x;
    const float o0 = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
    const float o1 = (part[0][i + 1] + part[1][i + 1]) + (part[2][i + 1] + part[3][i + 1]);
    *reinterpret_cast<uint32_t*>(a.out + id * D + i) = cvt_bf16x2(o0 * inv, o1 * inv);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[id] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

struct FewKernel {
  AttnKernel func;
  int smem;
};
template <int D, int KB, int VB, int NT>
FewKernel few_of() {
  return FewKernel{nq_attn_few_kernel<D, KB, VB, NT>, Few<D, KB, VB, NT>::bytes};
}
template <int D, int NT>
FewKernel few_kernel_bits(int kb, int vb) {
  if (kb == 8) return vb == 8 ? few_of<D, 8, 8, NT>() : few_of<D, 8, 4, NT>();
  return vb == 8 ? few_of<D, 4, 8, NT>() : few_of<D, 4, 4, NT>();
}
FewKernel few_kernel(int d, int nt, int kb, int vb) {
  if (d == 64) return nt == 1 ? few_kernel_bits<64, 1>(kb, vb) : few_kernel_bits<64, 2>(kb, vb);
  if (d == 128) return nt == 1 ? few_kernel_bits<128, 1>(kb, vb) : few_kernel_bits<128, 2>(kb, vb);
  return few_kernel_bits<256, 1>(kb, vb);
}

struct AttnPlan {
  bool many;
  int nt, row_tiles, tile_rows, tile_keys, min_stretch, blocks;
  size_t bytes, ml_at, units_at;  // of the workspace; words before the (reference, sum) pairs, the units' blocks
};

// At most this many keys over all kv heads take the few-rows kernel to 64 rows.
constexpr int64_t kFewKeys = 16384;

// Which kernel: few rows up to 16 (two of its row blocks), to 32 for heads of
// 64 channels.  Measured on both sides (us, few / many; 8 sequences of 8 k,
// 18 to 36 rows): heads of 128, 48.1 / 44.6 to 67.3 / 50.0; of 256, 47.9 / 45.2 to
// 68.9 / 54.6; of 64, 31.5 / 36.9 to 42.6 / 42.5; at 16 rows 38.6 / 43.1, 38.3 / 41.6
// and 25.7 / 34.7.  Up to 16 k keys over all kv heads the many-rows kernel's
// longer start decides, to 64 rows: one sequence of 2 k, 18 to 64 rows, 13.2 / 13.4 to
// 15.7 / 16.5 (128), 13.5 / 18.8 to 16.0 / 27.0 (256), 11.1 / 12.6 to 12.9 / 15.7 (64).
// (So for heads of 128 the two meet there; for 256 and 64 they would later, which
// was not looked for: one rule for all.)
bool takes_many(int rows, int dim, int64_t keys) {
  if (rows <= (dim == 64 ? 32 : 16)) return false;
  return rows > 64 || keys > kFewKeys;
}

AttnPlan plan_attention(int sms, int seqs, int max_drafts, int q_heads, int kv_heads, int dim,
                        int64_t max_context) {
  AttnPlan p;
  const int rows = max_drafts * (q_heads / kv_heads);
  p.many = takes_many(rows, dim, max_context * seqs * kv_heads);
  if (p.many) {
    const int most = many_kernel(dim, 8, 8).max_rows;
    p.nt = 0;
    p.row_tiles = (rows + most - 1) / most;
    p.tile_rows = ((rows + p.row_tiles - 1) / p.row_tiles + 15) / 16 * 16;
    p.tile_keys = 2 * kPage;
    p.min_stretch = 2;
  } else {
    p.nt = dim < 256 && rows > 8 ? 2 : 1;
    p.tile_rows = 8 * p.nt;
    p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
    p.tile_keys = kPage;
    p.min_stretch = 2;
  }
  // As many blocks as run at once (never more than tiles), each with an equal
  // stretch of all tiles.
  const int64_t units = static_cast<int64_t>(seqs) * kv_heads * p.row_tiles;
  const int64_t tiles = units * ((max_context + max_drafts + p.tile_keys - 1) / p.tile_keys);
  const int64_t at_once = static_cast<int64_t>(sms) * (p.many ? 1 : few_blocks(dim, p.nt));
  p.blocks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(at_once, (tiles + p.min_stretch - 1) / p.min_stretch)));
  const size_t pieces = static_cast<size_t>(p.blocks + units) * p.tile_rows;
  p.ml_at = pieces * dim;
  p.units_at = p.ml_at + pieces * 2;
  p.bytes = p.blocks == 1 ? 0 : (p.units_at + static_cast<size_t>(units) * 2) * sizeof(float);
  return p;
}

// Workspace of every batch of up to `seqs` sequences.  Within one kernel it grows
// with the batch, but a smaller batch may take the few-rows kernel instead, which
// has more blocks: the largest such batch counts too.
size_t workspace_bytes_up_to(int sms, int seqs, int max_drafts, int q_heads, int kv_heads, int dim,
                             int64_t max_context) {
  const AttnPlan p = plan_attention(sms, seqs, max_drafts, q_heads, kv_heads, dim, max_context);
  size_t bytes = p.bytes;
  const int64_t few = max_context > 0 ? kFewKeys / (max_context * kv_heads) : 0;  // sequences
  if (p.many && few >= 1 && few < seqs) {
    const AttnPlan f = plan_attention(sms, static_cast<int>(few), max_drafts, q_heads, kv_heads, dim, max_context);
    bytes = std::max(bytes, f.bytes);
  }
  return bytes;
}

int check_attention(int seqs, int max_drafts, int q_heads, int kv_heads, int dim, int64_t total,
                    int64_t max_context) {
  if (dim != 64 && dim != 128 && dim != 256) return NQ_EINVAL;
  if (seqs < 1 || seqs > 65535 || max_drafts < 1 || max_drafts > kMaxDrafts) return NQ_EINVAL;
  if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads > 65535) return NQ_EINVAL;
  if (total < 0 || total > static_cast<int64_t>(seqs) * max_drafts) return NQ_EINVAL;
  if (max_context < 0 || max_context > INT_MAX - kMaxDrafts) return NQ_EINVAL;
  return NQ_OK;
}

int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return NQ_OK;
  (void)cudaGetLastError();
  return NQ_ECUDA;
}

}  // namespace
}  // namespace nq

using namespace nq;

extern "C" {

int nq_tree_attention_workspace_bytes(int seqs, int max_drafts, int64_t total, int q_heads,
                                      int kv_heads, int head_dim, int64_t max_context,
                                      size_t* bytes) {
  if (!bytes) return NQ_EINVAL;
  if (int rc = check_attention(seqs, max_drafts, q_heads, kv_heads, head_dim, total, max_context))
    return rc;
  int* status;
  int sms;
  if (int rc = device_status(&status, &sms)) return rc;
  *bytes = workspace_bytes_up_to(sms, seqs, max_drafts, q_heads, kv_heads, head_dim, max_context);
  return NQ_OK;
}

int nq_tree_attention(const nq_kv_cache* cache, const void* q, int64_t q_token_stride,
                      int64_t q_head_stride, int64_t total, int q_heads, const int32_t* page_table,
                      int64_t table_stride, int table_width, const int32_t* lengths,
                      const int32_t* starts, const uint64_t* tree, int seqs, int max_drafts,
                      int64_t max_context, float scale, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, nq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_attention(seqs, max_drafts, q_heads, cache->kv_heads, cache->head_dim, total,
                               max_context))
    return rc;
  // (a sequence's keys rounded up to whole tiles stay within an int)
  if (table_width < 0 || table_width > (INT_MAX - 255) / kPage) return NQ_EINVAL;
  if (!starts && total % seqs) return NQ_EINVAL;
  if (!starts && total / seqs > max_drafts) return NQ_EINVAL;
  if (total == 0) return NQ_OK;
  if (!q || !page_table || !lengths || !out) return NQ_EINVAL;
  if (!is_aligned16(q) || !is_aligned16(out) || q_token_stride % 8 || q_head_stride % 8)
    return NQ_EALIGN;
  AttnArgs a;
  int sms;
  if (int rc = device_status(&a.status, &sms)) return rc;
  const int dim = cache->head_dim;
  const AttnPlan p = plan_attention(sms, seqs, max_drafts, q_heads, cache->kv_heads, dim, max_context);
  if (p.bytes > workspace_bytes || (p.bytes && !workspace)) return NQ_EINVAL;
  if (p.bytes && !is_aligned16(workspace)) return NQ_EALIGN;
  a.c = cache_view(*cache);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qs_tok = q_token_stride;
  a.qs_head = q_head_stride;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.total = total;
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.table = page_table;
  a.table_stride = table_stride;
  a.width = table_width;
  a.lengths = lengths;
  a.starts = starts;
  a.tree = reinterpret_cast<const unsigned long long*>(tree);
  a.seqs = seqs;
  a.max_drafts = max_drafts;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.row_tiles = p.row_tiles;
  a.tile_rows = p.tile_rows;
  a.wait_ns = static_cast<unsigned long long>(std::max(1, env_switch("NQ_WAIT_MS", 2000))) * 1000000ULL;
  a.tile_keys = p.tile_keys;
  a.min_stretch = p.min_stretch;
  a.blocks = p.blocks;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (p.bytes ? p.ml_at : 0));
  a.unit_blocks = p.bytes ? reinterpret_cast<int2*>(a.part_o + p.units_at) : nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool pdl = env_switch("NQ_PDL", 1) != 0;
  if (p.many) {
    const ManyKernel k = many_kernel(dim, cache->k_bits, cache->v_bits);
    if (int rc = allow_shared(reinterpret_cast<const void*>(k.func))) return rc;
    if (int rc = rc_of(launch(k.func, dim3(p.blocks), dim3(k.threads), k.smem, pdl, st, a))) return rc;
  } else {
    const FewKernel k = few_kernel(dim, p.nt, cache->k_bits, cache->v_bits);
    if (int rc = allow_shared(reinterpret_cast<const void*>(k.func))) return rc;
    if (int rc = rc_of(launch(k.func, dim3(p.blocks), dim3(kWarpsA * 32), k.smem, pdl, st, a))) return rc;
  }
  if (p.blocks == 1) return NQ_OK;
  AttnKernel merge = dim == 64    ? nq_attn_merge_kernel<64>
                     : dim == 128 ? nq_attn_merge_kernel<128>
                                  : nq_attn_merge_kernel<256>;
  const dim3 merge_grid(static_cast<unsigned>(max_drafts) * q_heads, seqs);
  return rc_of(launch(merge, merge_grid, dim3(128), 0, pdl, st, a));
}

}  // extern "C"
