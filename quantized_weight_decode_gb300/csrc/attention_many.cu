// Attention of drafted tokens over the quantised KV cache: the kernel for many
// rows (trees: drafted tokens x query heads of a kv head), on the
// 5th-generation tensor cores.
//
// With many rows the products weigh as much as the stream of codes: 4 D rows
// operations against 2 D bytes a key at 8 bits.  So each code is decoded once
// for all rows of a block, and both products run on tcgen05 with keys and
// value channels on the M = 128 side and the rows (padded to 16) on the N side:
//   S^T[128 keys x rows]   = codes_K[128 x D] . Q^T     per 64-group, fp32
//   O^T[D x rows]         += V'^T[D x 128] . P'^T       fp32, in tensor memory
// In the softmax a thread holds one key (its tensor-memory lane), so the key's
// scales are registers of the thread: logits are sums of a group's dot product
// times its scale in fp32, and no reduction over the rows is needed.
//
// Everything is fp16 on the tensor cores: codes are exact; queries are bf16
// values times a power of two a row, exact but for values 2^-22 below the row's
// largest (off by 2^-33 of that); values are code times the
// group's scale over a power of two 2^e of the key (one rounding, 2^-11 at
// most), and 2^e goes into the probability, which is rounded once (2^-11 of
// itself, 2^-25 at least).  The reference is kept so that the largest such product
// lies in 2^6 .. 2^14: it moves only when one passes 2^14 (then sums and O are
// scaled), so the fp16 floor is 2^-31 and less of the largest.  A key whose values
// are all zero has e = -24, below any other key's: however probable, it does not raise
// the floor.  Sums of probabilities are fp32, of the unrounded ones.
//
// Warps have roles, joined by barriers in shared memory alone: one copies the
// codes and scales of tiles of 128 keys (two pages, bulk copies into rings),
// two prepare the scales, 8 (16 for heads of 256) decode the codes into fp16
// operand lines, one thread issues the products, 16 (8) do the softmax.  Heads
// of 256 go through the same buffers in two halves of 128 channels.  A tile:
//   S computed -> logits less the references, written back to tensor memory,
//   S free -> vote of the four warps that share rows -> probabilities to shared
//   memory, sums in tensor memory -> O computed beside the next tile's logits.
// The loops are kept rolled and short: with everything unrolled the roles
// thrashed the instruction cache (143 us against 94 for the same work).
//
// Measured (GB300): 8 sequences of up to 16 k keys, trees of up to 16, 40 query
// heads of 128 on 8, 8 bits: 200 MB and 28.5 GFLOP in 86 us, of which the merge
// takes 4 and the start and end of stretches about 8; the chain of hand-overs a
// tile bounds it (1.7 us a tile of 128 keys; with all arithmetic left out, 1.3).
// One tree of 16 over 131 k keys, 24 query heads of 256 on 4: 210 MB in 162 us (two
// row tiles, each decoding all codes).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "attention.cuh"
#include "gemv.cuh"
#include "host.h"
#include "tcgen05.cuh"

namespace nq {
namespace {

constexpr int kThreadsT = 28 * 32;       // (72 registers a thread; fewer, fatter warps were slower: 20 warps 111 us against 94)
constexpr int kCopyWarp = 24, kMmaWarp = 25, kScaleWarp = 26, kScaleWarps = 2;
constexpr int kTileKeys = 128;
constexpr int kBlock = kTileKeys * 128;  // bytes of 128 lines of 64 fp16
constexpr int kTmemCols = 512;
constexpr float kHigh = 14.f, kTop = 6.f;  // log2 of the bound and of a new reference's largest

constexpr int kScaleSlots = 2;     // tiles of scales, raw and prepared (three are no faster)

struct Segment {     // a unit's tiles that a block takes in one go
  SeqView v;
  int seq, head, row0, rows, tile0, tiles, whole, live;
  long long slot, next;
};
template <int G>
struct SmallMem {
  alignas(16) float ref[128];            // minus the rows' references (0 before the first); read 16 bytes at a time
  alignas(16) float undo[128];           // one over the rows' powers of two
  alignas(16) float k[kScaleSlots][kTileKeys][G < 4 ? 2 : 4];     // key groups' scales times the logits' factor
  alignas(16) uint16_t raw[kScaleSlots][2][kTileKeys * G];        // FP16 scales as the cache has them
  alignas(8) uint16_t ratio[kScaleSlots][kTileKeys][G < 4 ? 2 : 4];  // fp16 scales of the value groups over 2^e
  float log2_e[kScaleSlots][kTileKeys];           // e, the power of two of a key's values' scales; -inf: no key
  unsigned char bad[kScaleSlots][kTileKeys];      // value groups whose scale is not finite
  int any_bad[kScaleSlots];
  int top[128];              // the rows' largest of a tile (ordered bits), then by what the reference moved
  float factor[128];         // what a move multiplies sums and outputs by
  unsigned rows[64][4];      // rows that see a drafted key
  unsigned poison[4][4];     // rows that see a value group with a scale that is not finite
  float sum[4][128];
  int id[128];               // row of q, out and lse
  unsigned char set[128];    // rows with a reference
  uint32_t tmem;
  int abort, lost;           // a wait gave up; one for a copy did
  Segment seg[2];
  // Barriers: copies landed (keys, values, scales) and slots free; scales
  // prepared and free; a half of the fp16 keys, of the values, probabilities
  // written; a half of S computed (its keys are free), all of it, S read; a half
  // of O computed, all of it.
  unsigned long long drained;  // after a wait that gave up
  unsigned long long kraw_full[4], kraw_free[4], vraw_full[4], vraw_free[4];
  unsigned long long sraw_full[kScaleSlots], sraw_free[kScaleSlots];
  unsigned long long scales_full[kScaleSlots], scales_free[kScaleSlots];
  unsigned long long k_full, v_full, p_full, k_free, s_full, s_free, v_free, o_full;
};

template <int D, int KB, int VB>
struct Many {
  static constexpr int G = D / 64;
  static constexpr int NH = D == 256 ? 2 : 1;   // halves of 128 channels, decoded and multiplied in turn
  static constexpr int GP = G / NH;             // groups of a half
  // Warps: softmax (groups of four: the tensor-memory lanes of a warp go by its
  // number modulo 4; a group takes every kGroups-th run of 8 rows), decoding,
  // then copies, products, scales (two).  Long heads have fewer rows a block
  // and more codes a key.
  static constexpr int kSoftmaxWarps = D == 256 ? 8 : 16, kDecodeWarps = kCopyWarp - kSoftmaxWarps;
  static constexpr int kGroups = kSoftmaxWarps / 4;
  static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps, kDecodeThreads = 32 * kDecodeWarps;
  // Tensor memory, columns: S of each group, O of each half, sums, logits
  // against the references.
  static constexpr int kMaxRows = D == 64 ? 128 : D == 128 ? 96 : 64;
  static constexpr int kColO = G * kMaxRows, kColL = kColO + NH * kMaxRows, kColY = kColL + kMaxRows;
  static_assert(kColY + kMaxRows <= kTmemCols, "");
  // Bytes of a key's codes and the 16-byte units a decoding thread takes.
  __host__ __device__ static constexpr int row_bytes(int bits) { return D * bits / 8; }
  // Shared memory: a half of the fp16 keys, of the values (two blocks), probabilities,
  // queries, rings of raw codes.
  static constexpr int off_k = 0;
  static constexpr int off_v = off_k + GP * kBlock;
  static constexpr int off_p = off_v + 2 * kBlock;
  static constexpr int off_q = off_p + (kMaxRows > 64 ? 2 : 1) * kBlock;
  static constexpr int off_raw = off_q + G * kMaxRows * 128;
  static constexpr int kSmall = (sizeof(SmallMem<G>) + 127) / 128 * 128;
  static constexpr int kKeySlot = kTileKeys * row_bytes(KB), kValueSlot = kTileKeys * row_bytes(VB);
  static constexpr int kRoom = 227 * 1024 - kSmall - off_raw, kPairs = kRoom / (kKeySlot + kValueSlot);
  static constexpr int NV = kPairs > 4 ? 4 : kPairs;
  static constexpr int NK = kPairs > 4 ? 4 : kPairs + (kPairs < 4 && kRoom - kPairs * (kKeySlot + kValueSlot) >= kKeySlot);
  static constexpr int off_raw_v = off_raw + NK * kKeySlot;
  static constexpr int off_small = off_raw_v + NV * kValueSlot;
  static constexpr int bytes = off_small + kSmall;
  static_assert(NV >= 1 && NK >= 1 && NK <= 4 && NV <= 4, "a tile of codes in flight at least");
  static_assert(off_v % 1024 == 0 && off_p % 1024 == 0 && off_q % 1024 == 0 && off_raw % 128 == 0 &&
                    off_raw_v % 128 == 0 && off_small % 128 == 0 && bytes <= 227 * 1024,
                "operand lines and copies");
};

__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int b) {
  return __int_as_float(b >= 0 ? b : b ^ 0x7FFFFFFF);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Eight codes as fp16, exact.  8 bits: 1024 + (c + 128) minus 1152, in order.
// 4 bits: pairs (c_i, c_{i+4}), 1024 + (c + 8) minus 1032, or 1024 + 16 (c + 8)
// over 16 minus 72.
__device__ __forceinline__ void codes_f16(uint32_t lo, uint32_t hi, uint32_t (&h)[4]) {
  const uint32_t a = lo ^ 0x80808080u, b = hi ^ 0x80808080u;
  h[0] = sub_f16x2(prmt(a, 0x64646464u, 0x4140), 0x64806480u);
  h[1] = sub_f16x2(prmt(a, 0x64646464u, 0x4342), 0x64806480u);
  h[2] = sub_f16x2(prmt(b, 0x64646464u, 0x4140), 0x64806480u);
  h[3] = sub_f16x2(prmt(b, 0x64646464u, 0x4342), 0x64806480u);
}
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  h[0] = nibbles_f16(w);
  h[1] = nibbles4_f16(w);
  h[2] = nibbles_f16(w >> 8);
  h[3] = nibbles4_f16(w >> 8);
}
// The channel that stands at place s of a run of 8 decoded codes.
__device__ __forceinline__ int channel_at(int bits, int s) {
  return bits == 8 ? s : (s >> 1) + 4 * (s & 1);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A bounded wait: the first probe in line, the rest apart (the loops of the
// roles share the instruction cache).
__device__ __noinline__ void wait_on(uint32_t bar, uint32_t par, int* abort, unsigned long long limit, int* status) {
  const Waiter wt{abort, limit, status};
  (void)wt.wait<false>(bar, par);
}
// The same on the barriers of the copies.  A wait that gave up elsewhere does not
// end it: a slot with a copy under way must not be taken for free, nor its
// barrier armed again.  All other waits end then, so these are met within their
// own time (of twice the limit, unless a copy is lost for good).
__device__ __noinline__ void wait_copy_on(uint32_t bar, uint32_t par, int* lost, int* abort, unsigned long long limit,
                                          int* status) {
  const Waiter wt{lost, 2 * limit, status};
  if (!wt.wait<false>(bar, par)) *const_cast<volatile int*>(abort) = 1;
}

// Pairs of fp32.
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  unsigned long long d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(unsigned long long x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A vote of the four softmax warps of a group, their barrier, and that of all softmax warps.
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, %2, 128, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(3 + group)
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(3 + group) : "memory");
}
template <int N>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
}
// The softmax warps tell the products' warp that the queries are in place.
template <int N>
__device__ __forceinline__ void queries_done() {
  asm volatile("barrier.cta.arrive 2, %0;" ::"n"(N + 32) : "memory");
}
template <int N>
__device__ __forceinline__ void queries_wait() {
  asm volatile("barrier.cta.sync 2, %0;" ::"n"(N + 32) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kThreadsT, 1) nq_attn_many_kernel(const AttnArgs a) {
  using C = Many<D, KB, VB>;
  constexpr int G = C::G, NH = C::NH, GP = C::GP;
  using Small = SmallMem<G>;
  static_assert(offsetof(Small, ref) % 16 == 0 && offsetof(Small, undo) % 16 == 0 && offsetof(Small, k) % 16 == 0 && offsetof(Small, raw) % 16 == 0 &&
                    offsetof(Small, ratio) % 8 == 0 && offsetof(Small, kraw_full) % 8 == 0,
                "wide accesses and copies");
  extern __shared__ __align__(1024) uint8_t sm[];
  Small& st = *reinterpret_cast<Small*>(sm + C::off_small);
  const uint32_t sb = smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&st.tmem), kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&st.kraw_full[i]), 1);
      mbar_init(smem_addr(&st.kraw_free[i]), C::kDecodeWarps);
      mbar_init(smem_addr(&st.vraw_full[i]), 1);
      mbar_init(smem_addr(&st.vraw_free[i]), C::kDecodeWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_addr(&st.sraw_full[i]), 1);
      mbar_init(smem_addr(&st.sraw_free[i]), kScaleWarps);
      mbar_init(smem_addr(&st.scales_full[i]), kScaleWarps);
      mbar_init(smem_addr(&st.scales_free[i]), C::kSoftmaxWarps + C::kDecodeWarps);
      st.any_bad[i] = 0;
    }
    mbar_init(smem_addr(&st.drained), 1);
    mbar_init(smem_addr(&st.k_full), C::kDecodeWarps);
    mbar_init(smem_addr(&st.v_full), C::kDecodeWarps);
    mbar_init(smem_addr(&st.p_full), C::kSoftmaxWarps);
    mbar_init(smem_addr(&st.s_full), 1);
    mbar_init(smem_addr(&st.s_free), C::kSoftmaxWarps);
    mbar_init(smem_addr(&st.k_free), 1);
    mbar_init(smem_addr(&st.v_free), 1);
    mbar_init(smem_addr(&st.o_full), 1);
    fence_mbar_init();
    st.abort = st.lost = 0;
  }
  if (D == 64)  // the upper half of O's lanes has no channels: zeros
    for (int e = tid; e < kBlock / 16; e += kThreadsT) st_shared16(sb + C::off_v + kBlock + 16 * e, 0, 0, 0, 0);
  fence_proxy_async_smem();
  const int pages = a.c.capacity / kPage;
  auto wait = [&](unsigned long long& bar, uint32_t par) {
    if (!mbar_try_wait(smem_addr(&bar), par & 1u)) wait_on(smem_addr(&bar), par & 1u, &st.abort, a.wait_ns, a.status);
  };
  auto wait_copy = [&](unsigned long long& bar, uint32_t par) {
    if (!mbar_try_wait(smem_addr(&bar), par & 1u))
      wait_copy_on(smem_addr(&bar), par & 1u, &st.lost, &st.abort, a.wait_ns, a.status);
  };
  auto arrive = [&](unsigned long long& bar) {  // one arrival of a warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&bar));
  };
  griddep_wait();

  // The copies' warp looks ahead: where the next tiles of this block's stretch are.
  long long pos_end = 0;
  auto look_ahead = [&](const Line& line, long long pos, Segment& sg) {
    Segment x;
    x.live = pos < pos_end;
    if (x.live) {
      const Place pl = line.at(a, pos, lane);
      x.v = seq_view(a, pl.seq);
      x.seq = pl.seq;
      x.head = pl.unit / pl.row_tiles;
      x.row0 = (pl.unit - x.head * pl.row_tiles) * a.tile_rows;
      x.rows = min(a.tile_rows, x.v.drafts * a.group - x.row0);
      x.tile0 = pl.tile;
      x.tiles = static_cast<int>(min(static_cast<long long>(pl.tiles - pl.tile), pos_end - pos));
      x.whole = x.tiles == pl.tiles;
      const long long unit = static_cast<long long>(pl.seq) * a.c.kv_heads * a.row_tiles + pl.unit;
      x.slot = blockIdx.x + unit;
      if (lane == 0 && a.unit_blocks) note_unit(a, unit, pl.tile, x.tiles, pl.tiles);
      x.next = pos + x.tiles;
      if (x.v.keys == 0) x.tiles = 0;
    }
    if (lane == 0) sg = x;
    return x.live ? x.next : pos;
  };
  long long ahead = 0;
  if (warp == kCopyWarp) {
    const Line line(a, lane, blockIdx.x == 0);
    const long long stretch = line.stretch(a, gridDim.x);
    pos_end = min(line.total, (blockIdx.x + 1) * stretch);
    ahead = look_ahead(line, blockIdx.x * stretch, st.seg[0]);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = st.tmem;

  unsigned done = 0u;  // tiles of this block so far: the phase of every barrier
  for (int which = 0;; which ^= 1) {
    const Segment& sg = st.seg[which];
    if (!sg.live) break;
    const int tiles = sg.tiles, rows = sg.rows, npad = (rows + 15) & ~15, nch = npad >> 3;
    const int key_begin = sg.tile0 * kTileKeys;
    const int key_end = min(key_begin + tiles * kTileKeys, sg.v.keys);

    if (warp == kCopyWarp) {
      // ---- codes and scales of a tile: its two pages
      const int32_t* table = a.table + sg.seq * a.table_stride;
      const int page_end = (key_end + kPage - 1) / kPage;
      const int head = sg.head;
      int id[2], next[2] = {-1, -1};  // pages of the tile whose values, whose keys come next
      auto fill = [&](unsigned long long* full, unsigned long long* free, unsigned slots, uint32_t bytes, unsigned n,
                      const int (&page)[2], auto copy) {
        const unsigned slot = n % slots;
        if (n >= slots) wait_copy(free[slot], n / slots - 1);
        if (lane == 0) {
          const uint32_t bar = smem_addr(&full[slot]);
          mbar_arrive_expect_tx(bar, bytes * ((page[0] >= 0) + (page[1] >= 0)));
          for (int i = 0; i < 2; ++i)
            if (page[i] >= 0) copy(slot, i, (static_cast<long long>(page[i]) * a.c.kv_heads + head) * kPage, bar);
        }
      };
      // The order of the decoding: keys of a tile before the values of the one before it.
#pragma unroll 1
      for (int t = -1; t < tiles && tiles > 0; ++t) {
        const unsigned n = done + t;
        id[0] = next[0];
        id[1] = next[1];
        if (t + 1 < tiles) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int pg = 2 * (sg.tile0 + t + 1) + i;
            next[i] = pg < page_end ? __ldg(table + pg) : -1;
            if (pg < page_end && static_cast<unsigned>(next[i]) >= static_cast<unsigned>(pages)) {
              next[i] = -1;
              if (lane == 0) atomicCAS(a.status, 0, kStatusRange);
            }
          }
          fill(st.sraw_full, st.sraw_free, kScaleSlots, 2 * kPage * G * 2, n + 1, next,
               [&](unsigned slot, int i, long long row, uint32_t bar) {
#pragma unroll
                 for (int w = 0; w < 2; ++w)
                   bulk_load(smem_addr(&st.raw[slot][w][i * kPage * G]), a.c.scales[w] + row * G, kPage * G * 2, bar);
               });
          fill(st.kraw_full, st.kraw_free, C::NK, C::kKeySlot / 2, n + 1, next,
               [&](unsigned slot, int i, long long row, uint32_t bar) {
                 bulk_load(sb + C::off_raw + slot * C::kKeySlot + i * (C::kKeySlot / 2),
                           a.c.codes[0] + row * C::row_bytes(KB), C::kKeySlot / 2, bar);
               });
        }
        if (t >= 0)
          fill(st.vraw_full, st.vraw_free, C::NV, C::kValueSlot / 2, n, id,
               [&](unsigned slot, int i, long long row, uint32_t bar) {
                 bulk_load(sb + C::off_raw_v + slot * C::kValueSlot + i * (C::kValueSlot / 2),
                           a.c.codes[1] + row * C::row_bytes(VB), C::kValueSlot / 2, bar);
               });
      }
      // (the last stretch of a block needs no second scan)
      if (ahead < pos_end) ahead = look_ahead(Line(a, lane), ahead, st.seg[which ^ 1]);
      else if (lane == 0) st.seg[which ^ 1].live = 0;
    } else if (warp == kMmaWarp) {
      // ---- products
      const uint32_t idesc_s = mma_f16_desc(128, npad, false, false);
      const uint32_t idesc_o = mma_f16_desc(128, npad, true, true);
      auto product_s = [&](unsigned n, int h) {
        wait(st.k_full, n * NH + h);
        if (h == 0 && n > 0) wait(st.s_free, n - 1);
        tcgen05_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int g = 0; g < GP; ++g) {
            const uint64_t ka = smem_desc(sb + C::off_k + g * kBlock, 16, 1024);
            const uint64_t qb = smem_desc(sb + C::off_q + (h * GP + g) * (npad * 128), 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_ss(tmem + (h * GP + g) * C::kMaxRows, ka + 2 * k, qb + 2 * k, idesc_s, k > 0);
          }
          mma_commit(smem_addr(&st.k_free));
          if (h == NH - 1) mma_commit(smem_addr(&st.s_full));
        }
        __syncwarp();
      };
      auto product_o = [&](unsigned n, int h, bool more) {
        if (h == 0) wait(st.p_full, n);
        wait(st.v_full, n * NH + h);
        tcgen05_fence_after();
        if (lane == 0) {
          const uint64_t va = smem_desc(sb + C::off_v, kBlock, 1024), pb = smem_desc(sb + C::off_p, kBlock, 1024);
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_f16_ss(tmem + C::kColO + h * C::kMaxRows, va + 128 * k, pb + 128 * k, idesc_o, more || k > 0);
          mma_commit(smem_addr(&st.v_free));
          if (h == NH - 1) mma_commit(smem_addr(&st.o_full));
        }
        __syncwarp();
      };
      queries_wait<C::kSoftmaxThreads>();
#pragma unroll 1
      for (int t = -1; t < tiles && tiles > 0; ++t) {
        const unsigned n = done + t;  // (t = -1: only the first tile's S)
#pragma unroll 1
        for (int h = 0; h < NH; ++h) {
          if (t + 1 < tiles) product_s(n + 1, h);
          if (t >= 0) product_o(n, h, t > 0);
        }
      }
    } else if (warp >= kScaleWarp) {
      // ---- scales: what the softmax and the decoding need of a key
      const float factor = a.scale_log2;
      const int32_t* table = a.table + sg.seq * a.table_stride;
      for (int t = 0; t < tiles; ++t) {
        const unsigned n = done + t, slot = n % kScaleSlots;
        if (n >= kScaleSlots) wait(st.scales_free[slot], n / kScaleSlots - 1);
        wait_copy(st.sraw_full[slot], n / kScaleSlots);
        bool any = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = (warp - kScaleWarp) * 64 + i * 32 + lane, at = key_begin + t * kTileKeys + key;
          const bool ok = at < key_end && static_cast<unsigned>(__ldg(table + at / kPage)) < static_cast<unsigned>(pages);
          float sv[G], most = 0.f;
          unsigned bad = 0u;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            st.k[slot][key][g] = ok ? __half2float(__ushort_as_half(st.raw[slot][0][key * G + g])) * factor : 0.f;
            sv[g] = ok ? __half2float(__ushort_as_half(st.raw[slot][1][key * G + g])) : 0.f;
            if (!(fabsf(sv[g]) <= 65504.f)) {
              bad |= 1u << g;
              sv[g] = 0.f;
            }
            most = fmaxf(most, fabsf(sv[g]));
          }
          // (without values: the smallest power of FP16, so that the key's probability,
          // which gives nothing to O, leaves the reference to the keys that do)
          const unsigned e = most == 0.f ? 0x33800000u : __float_as_uint(most) & 0x7F800000u;
          st.log2_e[slot][key] = ok ? static_cast<float>(static_cast<int>(e >> 23) - 127) : -INFINITY;
#pragma unroll
          for (int g = 0; g < G; ++g)
            st.ratio[slot][key][g] = __half_as_ushort(__float2half_rn(sv[g] * __uint_as_float(0x7F000000u - e)));
          st.bad[slot][key] = static_cast<unsigned char>(bad);
          any |= bad != 0u;
        }
        if (__any_sync(0xffffffffu, any) && lane == 0) st.any_bad[slot] = 1;
        arrive(st.sraw_free[slot]);
        arrive(st.scales_full[slot]);
      }
    } else if (warp >= C::kSoftmaxWarps) {
      // ---- decoding: codes to fp16 lines
      const int dt = tid - C::kSoftmaxThreads;
      // (half h of the channels of the raw codes at `src`)
      auto decode = [&](auto bits_c, auto values_c, int h, int src, int dst, unsigned slot) {
        constexpr int B = decltype(bits_c)::value;
        constexpr bool kValues = decltype(values_c)::value;
        constexpr int RB = C::row_bytes(B), KU = RB / 16 / NH, CU = 128 / B;       // units a key, codes a unit
        static_assert(kTileKeys * KU % C::kDecodeThreads == 0, "whole units a thread");
        constexpr int kUnits = kTileKeys * KU / C::kDecodeThreads, kStep = C::kDecodeThreads / KU;  // a thread's, keys a turn
        // Eight lanes' stores of 16 bytes have to fall on eight different chunks
        // of a line (chunk c of line r lies at c ^ (r & 7)), their loads too.
        // Units of 16 codes over two groups (KU = 8): four lanes take one key's
        // first group, four the next key's second. Units of 32 codes over two
        // groups: the second group's lanes take their chunks in the order 2 3 0 1.
        constexpr bool kPairs = KU == 8, kTurn = CU == 32 && KU == 4;
        const int key = kPairs ? 2 * (dt >> 4) + (dt >> 2 & 1) : dt / KU;
        const int unit = kPairs ? ((dt >> 1 ^ dt) & 4) + (dt & 3) : dt % KU;
        const int c8 = unit * (CU / 8);
        const bool turn = kTurn && (unit & 2);
        const uint32_t line0 = (sb + dst + (c8 >> 3) * kBlock + key * 128 + (((c8 & 7) ^ (key & 7)) << 4)) ^ (turn ? 32u : 0u);
        const uint8_t* from = sm + src + key * RB + h * (RB / NH) + unit * 16;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const uint4 x = *reinterpret_cast<const uint4*>(from + u * kStep * RB);
          const uint32_t w[4] = {turn ? x.z : x.x, turn ? x.w : x.y, turn ? x.x : x.z, turn ? x.y : x.w};
          uint32_t ratio = 0u;  // (a unit lies in one group)
          if constexpr (kValues) {
            const uint32_t y = st.ratio[slot][key + kStep * u][h * GP + (c8 >> 3)];
            ratio = prmt(y, y, 0x1010);
          }
#pragma unroll
          for (int i = 0; i < CU / 8; ++i) {
            uint32_t f[4];
            if constexpr (B == 8) codes_f16(w[2 * i], w[2 * i + 1], f);
            else codes_f16(w[i], f);
            if constexpr (kValues) {
#pragma unroll
              for (int k = 0; k < 4; ++k) f[k] = mul_f16x2(f[k], ratio);
            }
            st_shared16((line0 ^ (16 * i)) + u * kStep * 128, f[0], f[1], f[2], f[3]);
          }
        }
        fence_proxy_async_smem();
      };
#pragma unroll 1
      for (int t = -1; t < tiles && tiles > 0; ++t) {
        const unsigned n = done + t;  // (t = -1: only the first tile's keys)
#pragma unroll 1
        for (int h = 0; h < NH; ++h) {
          if (t + 1 < tiles) {
            const unsigned slot = (n + 1) % C::NK, m = (n + 1) * NH + h;
            wait_copy(st.kraw_full[slot], (n + 1) / C::NK);
            if (m > 0) wait(st.k_free, m - 1);
            decode(std::integral_constant<int, KB>(), std::false_type(), h, C::off_raw + slot * C::kKeySlot, C::off_k, 0u);
            if (h == NH - 1) arrive(st.kraw_free[slot]);
            arrive(st.k_full);
          }
          if (t >= 0) {
            const unsigned slot = n % C::NV, ss = n % kScaleSlots, m = n * NH + h;
            wait_copy(st.vraw_full[slot], n / C::NV);
            wait(st.scales_full[ss], n / kScaleSlots);
            if (m > 0) wait(st.v_free, m - 1);
            decode(std::integral_constant<int, VB>(), std::true_type(), h, C::off_raw_v + slot * C::kValueSlot, C::off_v, ss);
            if (h == NH - 1) {
              arrive(st.vraw_free[slot]);
              arrive(st.scales_free[ss]);
            }
            arrive(st.v_full);
          }
        }
      }
    } else {
      // ---- softmax
      const int wq = warp & 3, cg = warp >> 2;       // tensor-memory lanes, share of the rows
      const int kt = wq * 32 + lane;                 // this thread's key of a tile (and value channel)
      const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      if (tid < 128) {
        const int rr = sg.row0 + tid, t = rr / a.group;
        st.ref[tid] = 0.f;
        st.id[tid] = (sg.v.first + t) * a.q_heads + sg.head * a.group + rr - t * a.group;
        // rows that see a drafted key, 32 rows a warp
        const unsigned long long bits = tid < rows ? tree_bits(a, sg.v, t) : 0ull;
        for (int d = 0; d < sg.v.drafts; ++d) {
          const unsigned m = __ballot_sync(0xffffffffu, bits >> d & 1ull);
          if (lane == 0) st.rows[d][warp] = m;
        }
      }
      if (tid < 16) st.poison[tid >> 2][tid & 3] = 0u;
      if (tid < 128) st.set[tid] = 0;
      // Queries: runs of 8 channels, each row scaled by a power of two of its own
      // (one for all rows would let a row of huge values take the others' precision).
      {
        constexpr int kRuns = D / 8, kItems = C::kMaxRows * kRuns / C::kSoftmaxThreads;
        static_assert(kRuns <= 32 && C::kSoftmaxThreads % kRuns == 0, "a row's runs lie side by side in a warp");
        uint4 raw[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int e = tid + i * C::kSoftmaxThreads, n = e / kRuns, c = e % kRuns;
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (n < rows) {
            const int rr = sg.row0 + n, t = rr / a.group;
            raw[i] = __ldg(reinterpret_cast<const uint4*>(
                a.q + (sg.v.first + t) * a.qs_tok + (sg.head * a.group + rr - t * a.group) * a.qs_head + 8 * c));
          }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int e = tid + i * C::kSoftmaxThreads, n = e / kRuns, c = e % kRuns;
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          unsigned most = 0u;  // the row's largest finite magnitude
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
            if (lo < 0x7F80u) most = max(most, lo);
            if (hi < 0x7F80u) most = max(most, hi);
          }
#pragma unroll
          for (int k = kRuns / 2; k >= 1; k >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, k));
          // into [2^7, 2^8): exponent field of a bf16
          const int ex = most == 0u ? 0 : max(-120, min(120, 134 - static_cast<int>(most >> 7)));
          const float up = __int_as_float((ex + 127) << 23);
          if (c == 0) st.undo[n] = __int_as_float((127 - ex) << 23);
          if (n < npad) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = __uint_as_float(w[k] << 16) * up;
              f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * up;
            }
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = KB == 8 ? cvt_f16x2(f[2 * k], f[2 * k + 1]) : cvt_f16x2(f[k], f[k + 4]);
            st_shared16(sb + C::off_q + (c >> 3) * (npad * 128) + n * 128 + (((c & 7) ^ (n & 7)) << 4), h[0],
                        h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_smem();
      }
      softmax_sync<C::kSoftmaxThreads>();
      queries_done<C::kSoftmaxThreads>();

      bool unset = false;  // this lane's row (below) has no reference after the tiles so far
      for (int t = 0; t < tiles; ++t) {
        const unsigned n = done + t, slot = n % kScaleSlots;
        wait(st.scales_full[slot], n / kScaleSlots);
        unsigned long long kk[G];
        if constexpr (G == 4) {
          const float4 x = *reinterpret_cast<const float4*>(st.k[slot][kt]);
          const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int g = 0; g < G; ++g) kk[g] = pack2(f[g], f[g]);
        } else {
#pragma unroll
          for (int g = 0; g < G; ++g) kk[g] = pack2(st.k[slot][kt][g], st.k[slot][kt][g]);
        }
        const float log2_e = st.log2_e[slot][kt];
        const float inv_e = log2_e == -INFINITY ? 0.f : __int_as_float((127 - static_cast<int>(log2_e)) << 23);
        const unsigned long long e2 = pack2(log2_e, log2_e), w2 = pack2(inv_e, inv_e);
        wait(st.s_full, n);
        tcgen05_fence_after();
        // Logits (base 2, with the key's power of two) against the references.
        const int key0 = key_begin + t * kTileKeys, draft = key0 + kt - sg.v.len;
        const bool masked = key0 + kTileKeys > sg.v.len;
        float high = -INFINITY;
#pragma unroll 1
        for (int c = cg; c < nch; c += C::kGroups) {
          constexpr int GL = G < 2 ? G : 2;  // groups read at a time
          float y[GL][8];
          unsigned long long z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = 0ull;
#pragma unroll
          for (int g0 = 0; g0 < G; g0 += GL) {
#pragma unroll
            for (int g = 0; g < GL; ++g) tmem_ld8(lanes + (g0 + g) * C::kMaxRows + c * 8, y[g]);
#pragma unroll
            for (int g = 0; g < GL; ++g) tmem_wait_ld(y[g]);
#pragma unroll
            for (int g = 0; g < GL; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) z[i] = fma2(pack2(y[g][2 * i], y[g][2 * i + 1]), kk[g0 + g], z[i]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 u = *reinterpret_cast<const float4*>(st.undo + 8 * c + 4 * i);
            const float4 r = *reinterpret_cast<const float4*>(st.ref + 8 * c + 4 * i);
            unpack2(add2(fma2(z[2 * i], pack2(u.x, u.y), e2), pack2(r.x, r.y)), y[0][4 * i], y[0][4 * i + 1]);
            unpack2(add2(fma2(z[2 * i + 1], pack2(u.z, u.w), e2), pack2(r.z, r.w)), y[0][4 * i + 2], y[0][4 * i + 3]);
          }
          // (a key that is none for every row too: e = -inf does not hide it from a query of NaN)
          if ((masked && draft >= 0) || log2_e == -INFINITY) {
            const unsigned seen = log2_e == -INFINITY ? 0u : st.rows[draft][c >> 2] >> (8 * (c & 3));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (!(seen >> i & 1u)) y[0][i] = -INFINITY;
          }
          tmem_st8(lanes + C::kColY + c * 8, y[0]);
#pragma unroll
          for (int i = 0; i < 8; i += 2) high = fmaxf(high, fmaxf(y[0][i], y[0][i + 1]));
        }
        tcgen05_fence_before();
        arrive(st.s_free);
        tmem_wait_st();
        if (st.any_bad[slot]) {  // rows that see a value group whose scale is not finite
          const unsigned bad = st.bad[slot][kt];
#pragma unroll 1
          for (int c = cg; c < nch; c += C::kGroups) {
            float y[8];
            unsigned m = 0u;
            tmem_ld8(lanes + C::kColY + c * 8, y);
            tmem_wait_ld(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) m |= (y[i] == -INFINITY ? 0u : 1u) << i;
#pragma unroll
            for (int g = 0; g < G; ++g)
              if (bad >> g & 1u) atomicOr(&st.poison[g][c >> 2], m << (8 * (c & 3)));
          }
        }
        // A tile that may hold a row's first key moves the references too (tiles
        // before it may have had none: their pages were not the cache's).
        // The four warps that share rows (one a quarter of the keys) agree among
        // themselves; the groups of warps are not in step.
        const bool move = group_any(cg, high > kHigh || t == 0 || masked || unset);
        if (n > 0) wait(st.o_full, n - 1);
        if (move) {
          const int row = 8 * (cg + C::kGroups * (lane >> 3)) + (lane & 7);  // a lane of the first warp's
          if (wq == 0) st.top[row] = INT_MIN;
          group_sync(cg);
#pragma unroll 1
          for (int c = cg; c < nch; c += C::kGroups) {
            float y[8];
            tmem_ld8(lanes + C::kColY + c * 8, y);
            tmem_wait_ld(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int b = __reduce_max_sync(0xffffffffu, ordered(y[i]));
              if (lane == 0) atomicMax(&st.top[8 * c + i], b);
            }
          }
          group_sync(cg);
          if (wq == 0) {  // (above the reference)
            const float top = from_ordered(st.top[row]);
            float by = 0.f, factor = 1.f;
            if (row < rows && top != -INFINITY && (!st.set[row] || !(top <= kHigh))) {
              by = top - kTop;
              factor = st.set[row] ? ex2(-by) : 0.f;
              st.ref[row] -= by;
              st.set[row] = 1;
            }
            st.top[row] = __float_as_int(by);
            st.factor[row] = factor;
            unset = row < rows && !st.set[row];
          }
          group_sync(cg);
          tcgen05_fence_after();
#pragma unroll 1
          for (int e = 0; e < 2 + NH; ++e) {  // logits, and from the second tile on sums and outputs
            if (e > 0 && t == 0) break;
#pragma unroll 1
            for (int c = cg; c < nch; c += C::kGroups) {
              const uint32_t at = lanes + (e == 0 ? C::kColY : e == 1 ? C::kColL : C::kColO + (e - 2) * C::kMaxRows) + c * 8;
              float o[8];
              tmem_ld8(at, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                o[i] = e == 0 ? o[i] - __int_as_float(st.top[8 * c + i]) : o[i] * st.factor[8 * c + i];
              tmem_st8(at, o);
            }
          }
          tmem_wait_st();
        }
        // Probabilities times the key's power of two: to shared memory; sums without it.
        auto store_p = [&](int c, float (&x)[8], float (&l)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = ex2(x[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            unpack2(fma2(pack2(x[2 * i], x[2 * i + 1]), w2, pack2(l[2 * i], l[2 * i + 1])), l[2 * i], l[2 * i + 1]);
          tmem_st8(lanes + C::kColL + c * 8, l);
          st_shared16(sb + C::off_p + (c >> 3) * kBlock + kt * 128 + (((c & 7) ^ (kt & 7)) << 4),
                      cvt_f16x2(x[0], x[1]), cvt_f16x2(x[2], x[3]), cvt_f16x2(x[4], x[5]), cvt_f16x2(x[6], x[7]));
        };
        if (t == 0) {  // the sums start
          float l[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c = cg; c < nch; c += C::kGroups) tmem_st8(lanes + C::kColL + c * 8, l);
          tmem_wait_st();
        }
#pragma unroll 1
        for (int c = cg; c < nch; c += C::kGroups) {
          float x[8], l[8];
          tmem_ld8(lanes + C::kColY + c * 8, x);
          tmem_ld8(lanes + C::kColL + c * 8, l);
          tmem_wait_ld(x);
          tmem_wait_ld(l);
          store_p(c, x, l);
        }
        fence_proxy_async_smem();
        tmem_wait_st();
        tcgen05_fence_before();
        arrive(st.scales_free[slot]);
        arrive(st.p_full);
      }

      // ---- sums over the keys (lanes), in a fixed order: halving the columns
      // a lane holds at every step, lane i ends with column i of its 32
#pragma unroll 1
      for (int c0 = cg; c0 < nch && tiles > 0; c0 += 4 * C::kGroups) {
        float y[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + C::kGroups * j;
          float l[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (c < nch) {
            tmem_ld8(lanes + C::kColL + c * 8, l);
            tmem_wait_ld(l);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) y[8 * j + i] = l[i];
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
          const bool up = lane & d;
#pragma unroll
          for (int i = 0; i < d; ++i) {
            const float give = up ? y[i] : y[i + d], keep = up ? y[i + d] : y[i];
            y[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        }
        const int c = c0 + C::kGroups * (lane >> 3);
        if (c < nch) st.sum[wq][8 * c + (lane & 7)] = y[0];
      }
      softmax_sync<C::kSoftmaxThreads>();
      // A row's outputs are multiplied by: one over its sum where this block
      // has all its keys; 1 for a piece; nothing seen: 0 (and so the outputs).
      if (tid < rows) {
        const bool none = !st.set[tid];
        const float sum = (st.sum[0][tid] + st.sum[1][tid]) + (st.sum[2][tid] + st.sum[3][tid]);
        st.factor[tid] = none ? 0.f : sg.whole ? 1.f / sum : 1.f;
        st.top[tid] = none;
        if (!sg.whole)
          a.part_ml[sg.slot * a.tile_rows + tid] = none ? make_float2(-INFINITY, 0.f) : make_float2(-st.ref[tid], sum);
        else if (a.lse)
          a.lse[st.id[tid]] = none ? -INFINITY : (log2f(sum) - st.ref[tid]) * 0.693147180559945309f;
      }
      softmax_sync<C::kSoftmaxThreads>();
      if (tiles > 0) wait(st.o_full, done + tiles - 1);
      tcgen05_fence_after();
#pragma unroll 1
      for (int e = cg; e < nch * NH; e += C::kGroups) {
        const int h = e / nch, c = e - h * nch, ch = h * 128 + (kt & ~7) + channel_at(VB, kt & 7);
        float o[8];
        tmem_ld8(lanes + C::kColO + h * C::kMaxRows + c * 8, o);
        tmem_wait_ld(o);
        if (kt >= D) continue;
        const unsigned spoilt = st.poison[ch >> 6][c >> 2] >> (8 * (c & 3));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = 8 * c + i;
          if (n >= rows) break;
          float z = st.top[n] ? 0.f : o[i] * st.factor[n];
          if (spoilt >> i & 1u) z = __int_as_float(0x7FC00000);
          if (sg.whole) a.out[static_cast<long long>(st.id[n]) * D + ch] = __float2bfloat16_rn(z);
          else a.part_o[(sg.slot * a.tile_rows + n) * D + ch] = z;
        }
      }
      tcgen05_fence_before();
    }
    done += tiles;
    __syncthreads();
    tcgen05_fence_after();
  }
  if (st.abort) {
    // A wait gave up: the copies and products still under way have to end
    // before the block does (each again within the limit).
    auto drain = [&](uint32_t bar, uint32_t par) {
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(bar, par & 1u) && global_ns() - t0 < a.wait_ns) {
      }
    };
    if (warp == kCopyWarp && lane == 0) {
      auto ring = [&](unsigned long long* full, unsigned slots) {  // the last copy into each place
        for (unsigned i = 0; i < slots && i < done; ++i) drain(smem_addr(&full[i]), (done - 1 - i) / slots);
      };
      ring(st.kraw_full, C::NK);
      ring(st.vraw_full, C::NV);
      ring(st.sraw_full, kScaleSlots);
    }
    if (warp == kMmaWarp && lane == 0) {
      mma_commit(smem_addr(&st.drained));
      drain(smem_addr(&st.drained), 0u);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int KB, int VB>
ManyKernel of() {
  return ManyKernel{nq_attn_many_kernel<D, KB, VB>, kThreadsT, Many<D, KB, VB>::bytes, Many<D, KB, VB>::kMaxRows};
}
template <int D>
ManyKernel of_bits(int kb, int vb) {
  if (kb == 8) return vb == 8 ? of<D, 8, 8>() : of<D, 8, 4>();
  return vb == 8 ? of<D, 4, 8>() : of<D, 4, 4>();
}

}  // namespace

ManyKernel many_kernel(int dim, int kb, int vb) {
  return dim == 64 ? of_bits<64>(kb, vb) : dim == 128 ? of_bits<128>(kb, vb) : of_bits<256>(kb, vb);
}

}  // namespace nq
