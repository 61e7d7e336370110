// Logits of hidden states under one LM head with, beside it, the low-rank
// adapter each token's request asks for:
//   z_t = x_t W^T + s_a (x_t A_a^T) B_a^T,   a = adapter[t] (a < 0: no adapter).
//
// lora_down forms h_t = s_a x_t A_a^T (r numbers per token) and, for every tile of
// up to 128 tokens, the list of the adapters it asks for, each with the set of its
// token rows.  lora_head_kernel, its programmatic dependent (it
// streams W while lora_down runs), is a persistent warp-specialised tcgen05 GEMM
// over (token tile, vocab tile) units: TMA producer warp, MMA issuer, eight
// epilogue warps.  Between a unit's x W^T k-blocks it runs the products h B_a^T of
// the listed adapters into the same accumulator, with the TMEM lanes of the other
// adapters' tokens disabled: a token takes its own adapter only, whatever values
// the others hold (a NaN in one request's adapter stays in that request), and
// tokens need no sorting; several tiles of mixed tokens are sorted all the same
// (lora_sort, lora_gather), as each tile then asks for fewer adapters.
//
// h is kept as three bf16 numbers, h = h0 + h1 + h2 with h0 = h cut to bf16, h1 =
// h - h0 cut to bf16, h2 the rest: 24 significant bits, all of the fp32 sum.  Each
// multiplies the same B tile in shared memory.  bf16 logits take the first two, the
// second rounded (16 bits, 2^-7 of their own rounding).  Cut, not rounded: a finite h
// then has finite parts, and parts of one sign, none of them 0 (in the place of a 0
// stands h 2^-40), make +-inf of an infinite B as h itself does, where 0 inf or inf -
// inf would be NaN.  The tensor cores cut bits at every
// accumulation step (4e-6 of the result over H = 4096 against 5e-7 for fp32 sums),
// so the accumulator is taken out every few k-blocks (Params::chunk) and summed in
// fp32 registers, while the next ones run into the other accumulator.
//
// An adapter costs the tensor cores the same whether one token asks for it or 128:
// about 170 cycles an MMA whatever its width, two or three MMAs for 16 ranks.  The
// k-blocks of W leave the tensor cores idle where tokens are few, so the adapters'
// stages go between them (all but the first unit's, which has to wait for
// lora_down).
//
// Few tokens: bound by HBM, W and the adapters' B read once.  The vocab tile is
// the multiple of 16 that fills whole waves of SMs best.  1 token, H 4096, V 32768:
// 47.5 us (5.7 TB/s); 48 tokens of 24 adapters of 16 ranks, V 128256: 197 us (6.0
// TB/s).  Many adapters beside a short W (200 tokens of 64 adapters of 32 ranks, H
// 2056, V 50001, bf16 logits: 122 us, 3.6 TB/s): bound by the adapters' MMAs and the
// time to the first of them, 87 us without adapters.  Many tokens (2048 of 4 adapters
// of 64 ranks, H 4096, V 128256): bound by the tensor cores, 1.41 ms for a call by
// itself (1.55 PFLOP/s) and 1.60 ms among others, at the power limit's clocks; a
// library's product x W^T with bf16 logits and no adapters takes 1.11 and 1.31 ms.
#include <cmath>
#include <cstdint>

#include "answer.h"
#include "ptx.cuh"

namespace lmho {
namespace {

constexpr int kMaxBN = 256;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kMaxStages = 8;
constexpr int kEpiWarps = 8;
// Warps: TMA, MMA, two that only give up registers, then the epilogue's.  The launch's
// 168 registers a thread are split so that the epilogue's 128 sums leave it some: with
// 168 there it kept others in local memory, and its reads of those took 20 us of a
// 128 x 224 tile's store.
constexpr int kOtherThreads = 128, kThreads = kOtherThreads + 32 * kEpiWarps;
constexpr int kLaunchRegs = 168, kOtherRegs = 80, kEpiRegs = 208;
static_assert(kOtherThreads * kOtherRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs, "the launch's registers");
constexpr int kRankBlock = 16;        // ranks of one MMA step; a row of h's tile: 16 each of h0, h1, h2, and 16 unused
constexpr int kPitch = 17;            // staging of unaligned rows: 16 columns of 16 rows
constexpr int kStageOut = kEpiWarps * 16 * kPitch * 4;
constexpr int kOutTile = 32 * 4 * kLoraOutRows;  // TMA stores, a warp's: 32 columns
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 227 * 1024;

// Shared-memory descriptor of a K-major bf16 tile written by TMA with 128-byte
// swizzle: rows of 128 bytes, 8-row core groups 1024 bytes apart (SBO), start
// address >> 4 in bits 0-13, LBO field 1 (unused for this layout), bits 46-48
// = 0b001, swizzle mode 2 (128-byte) in bits 61-63.  Tiles are 1024-byte
// aligned, so the base-offset field is 0.  Moving 16 bf16 (32 bytes) along K
// inside the swizzle row adds 2 to the start-address field.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// ---------------------------------------------------------------- the tokens' order
// More than one tile of tokens: in the order of their adapters a tile asks for fewer,
// and an adapter's products cost a tile the same whatever the number of its tokens.
// One block counts the tokens of every adapter, and the adapters of every tile in
// either order; if sorting saves one per tile, the tokens are taken in the stable
// order (a warp places 32 at a time).  Else they stay, and the output can leave by TMA.
// order: the tokens, their adapters, and whether they are sorted.  2048 mixed tokens,
// H 4096, V 32768: with 64 adapters of 16 ranks 704 us as they come and 550 sorted,
// with 4 of 64 ranks 558 and 490; tokens in runs 478, and 490 sorted all the same.
constexpr int kSortThreads = 1024;
constexpr int kSortKeys = 4096;

__global__ void __launch_bounds__(kSortThreads) lora_sort(const int64_t* __restrict__ adapter, int64_t T, int n,
                                                          int tile_rows, int32_t* __restrict__ order) {
  griddep_launch_dependents();
  __shared__ int32_t start[kLoraMaxSort + 1];
  __shared__ uint32_t bits[kSortThreads / 32][kLoraMaxSort / 32];
  __shared__ uint16_t keys[kSortKeys];
  __shared__ int32_t warp_sum[kSortThreads / 32], before, after;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const auto key_of = [&](int64_t t) {  // n: no adapter, or none that there is
    const int64_t a = adapter[t];
    return a >= 0 && a < n ? static_cast<int>(a) : n;
  };
  for (int i = tid; i <= n; i += kSortThreads) start[i] = 0;
  if (tid == 0) before = after = 0;
  __syncthreads();
  for (int64_t t = tid; t < T; t += kSortThreads) atomicAdd(&start[key_of(t)], 1);
  const int words = (n + 31) / 32;
  int mine = 0;
  for (int64_t t0 = static_cast<int64_t>(warp) * tile_rows; t0 < T; t0 += kSortThreads / 32 * tile_rows) {
    for (int i = lane; i < words; i += 32) bits[warp][i] = 0;
    __syncwarp();
    for (int k = lane; k < tile_rows && t0 + k < T; k += 32) {
      const int a = key_of(t0 + k);
      if (a < n) atomicOr(&bits[warp][a >> 5], 1u << (a & 31));
    }
    __syncwarp();
    for (int i = lane; i < words; i += 32) mine += __popc(bits[warp][i]);
    __syncwarp();
  }
  if (mine) atomicAdd(&before, mine);
  __syncthreads();
  // the adapters' first places
  const int per = (n + kSortThreads) / kSortThreads, i0 = tid * per;
  int sum = 0;
  for (int i = i0; i < i0 + per && i <= n; ++i) sum += start[i];
  int upto = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
    if (lane >= off) upto += o;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int at = upto - sum, tiles = 0;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int i = i0; i < i0 + per && i <= n; ++i) {
    const int c = start[i];
    if (i < n && c) tiles += (at + c - 1) / tile_rows - at / tile_rows + 1;
    start[i] = at;
    at += c;
  }
  if (tiles) atomicAdd(&after, tiles);
  __syncthreads();
  const bool sorted = before - after > (T + tile_rows - 1) / tile_rows;
  if (tid == 0) order[2 * T] = sorted;
  if (!sorted) {
    for (int64_t t = tid; t < T; t += kSortThreads) {
      const int key = key_of(t);
      order[t] = static_cast<int32_t>(t);
      order[T + t] = key < n ? key : -1;
    }
    return;
  }
  for (int64_t t0 = 0; t0 < T; t0 += kSortKeys) {
    const int count = static_cast<int>(T - t0 < kSortKeys ? T - t0 : kSortKeys);
    for (int i = tid; i < count; i += kSortThreads) keys[i] = static_cast<uint16_t>(key_of(t0 + i));
    __syncthreads();
    if (warp == 0)
      for (int i = lane; i - lane < count; i += 32) {
        const int key = i < count ? keys[i] : kLoraMaxSort + 1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, key);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int place = i < count ? start[key] : 0;
        __syncwarp();
        if (i < count) {
          if (rank == 0) start[key] = place + __popc(same);
          order[place + rank] = static_cast<int32_t>(t0 + i);
          order[T + place + rank] = key < n ? key : -1;
        }
        __syncwarp();
      }
    __syncthreads();
  }
}

// x in the tokens' order, if they are sorted: a block per row.
__global__ void __launch_bounds__(256) lora_gather(const uint16_t* __restrict__ x, int64_t T, int64_t H,
                                                   const int32_t* __restrict__ order, uint16_t* __restrict__ xs) {
  griddep_launch_dependents();
  griddep_wait();
  if (!order[2 * T]) return;
  const uint4* from = reinterpret_cast<const uint4*>(x + order[blockIdx.x] * H);
  uint4* to = reinterpret_cast<uint4*>(xs + blockIdx.x * H);
  for (int64_t i = threadIdx.x; i < H / 8; i += blockDim.x) to[i] = __ldg(from + i);
}

// ---------------------------------------------------------------- h = s x A^T
// A block per 16 tokens and distinct adapter among them (slots past the last one
// return), then one per tile of 128 tokens for its adapter list.  The 16 x r
// products over H run on mma.sync m16n8k16: 16 warps split H, a lane loads 8
// consecutive numbers of its rows of x and A per 32 of H (which of them is which k of
// an MMA does not matter as long as both operands agree), so every load is 16 bytes
// and the latency of a few of them is the whole kernel.  Rows of tokens with another
// adapter are computed along and dropped.
// h row of token t: for every block of 16 ranks, 16 numbers h0, 16 h1, 16 h2 and 16
// that nothing reads.
constexpr int kDownThreads = 512;
constexpr int kDownWarps = kDownThreads / 32;
constexpr int kGroup = 16;
constexpr int kDownRanks = 32;        // at a time

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kDownThreads) lora_down(const uint16_t* __restrict__ x,
                                                          const uint16_t* __restrict__ A,
                                                          const int64_t* __restrict__ adapter,
                                                          const float* __restrict__ scale, int64_t T, int64_t H,
                                                          int64_t n, int r, int r_blocks, int64_t groups,
                                                          uint16_t* __restrict__ h, LoraTile* __restrict__ plan,
                                                          const int32_t* __restrict__ order, int tile_rows,
                                                          bool two_parts) {
  // The head's kernel starts when every block has said so: with an order, when that
  // and x in it are complete.
  if (order) griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int32_t ids[kBM];
  const auto token_at = [&](int64_t place) { return order ? order[place] : place; };
  const auto id_of = [&](int64_t place) {
    if (place >= T) return -1;
    if (order) return order[T + place];
    const int64_t a = adapter[place];
    return (a >= 0 && a < n) ? static_cast<int32_t>(a) : -1;
  };
  if (blockIdx.x >= groups * kGroup) {
    const int64_t mt = blockIdx.x - groups * kGroup;
    __shared__ uint32_t firsts[kBM / 32];
    if (threadIdx.x < kBM)
      ids[threadIdx.x] = static_cast<int>(threadIdx.x) < tile_rows ? id_of(mt * tile_rows + threadIdx.x) : -1;
    __syncthreads();
    if (threadIdx.x >= kBM) return;
    const int32_t id = ids[threadIdx.x];
    uint32_t rows[kBM / 32] = {};
    bool first = id >= 0;
    for (int k = 0; k < kBM; ++k)
      if (ids[k] == id) {
        rows[k >> 5] |= 1u << (k & 31);
        if (k < static_cast<int>(threadIdx.x)) first = false;
      }
    const uint32_t ball = __ballot_sync(0xFFFFFFFFu, first);
    if (lane == 0) firsts[warp] = ball;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    int pos = __popc(firsts[warp] & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < kBM / 32; ++w) {
      if (w < warp) pos += __popc(firsts[w]);
      total += __popc(firsts[w]);
    }
    if (first) {
      LoraEntry e{};
      e.adapter = id;
      for (int w = 0; w < kBM / 32; ++w) e.skip[w] = ~rows[w];
      plan[mt].e[pos] = e;
    }
    if (threadIdx.x == 0) plan[mt].count = total;
    return;
  }
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / kGroup) * kGroup;
  const int slot = static_cast<int>(blockIdx.x % kGroup);
  __shared__ float part[kDownWarps][kGroup][kDownRanks + 1];
  const int32_t id = id_of(t0 + (lane & (kGroup - 1)));
  if (threadIdx.x < kGroup) ids[threadIdx.x] = id;
  // the slot-th distinct adapter, found by every warp
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
  uint32_t firsts = __ballot_sync(0xFFFFFFFFu, id >= 0 && __ffs(same) - 1 == lane);
  for (int i = 0; i < slot; ++i) firsts &= firsts - 1;
  const int32_t mine = __shfl_sync(0xFFFFFFFFu, id, firsts ? __ffs(firsts) - 1 : 0);
  if (!firsts) return;
  __syncthreads();
  const float s = scale ? scale[mine] : 1.f;
  const int64_t row = static_cast<int64_t>(r_blocks) * 4 * kRankBlock;  // of h
  const int g = lane >> 2, c = lane & 3;
  const int64_t blocks = (H + 31) / 32;
  const int64_t ta = t0 + g < T ? t0 + g : T - 1, tb = t0 + g + 8 < T ? t0 + g + 8 : T - 1;
  const uint16_t* xa = x + token_at(ta) * H + 8 * c;
  const uint16_t* xb = x + token_at(tb) * H + 8 * c;
  for (int q = 0; q < r; q += kDownRanks) {
    const int tiles = (min(r - q, kDownRanks) + 7) / 8;
    const uint16_t* ar = A + (static_cast<int64_t>(mine) * r + q + g) * H + 8 * c;
    float d[kDownRanks / 8][4] = {};
    for (int64_t k = warp; k < blocks; k += kDownWarps) {
      // all of a step's loads before its products, without a branch between them
      const bool in = k * 32 + 8 * c < H;  // H is a multiple of 8
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 w[kDownRanks / 8];
#pragma unroll
      for (int j = 0; j < kDownRanks / 8; ++j)
        w[j] = in && j < tiles ? __ldg(reinterpret_cast<const uint4*>(ar + static_cast<int64_t>(8 * j) * H + k * 32)) : zero;
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(xa + k * 32)) : zero;
      const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(xb + k * 32)) : zero;
#pragma unroll
      for (int j = 0; j < kDownRanks / 8; ++j) {
        mma_16816(d[j], u.x, v.x, u.y, v.y, w[j].x, w[j].y);
        mma_16816(d[j], u.z, v.z, u.w, v.w, w[j].z, w[j].w);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kDownRanks / 8; ++j) {
      part[warp][g][8 * j + 2 * c] = d[j][0];
      part[warp][g][8 * j + 2 * c + 1] = d[j][1];
      part[warp][g + 8][8 * j + 2 * c] = d[j][2];
      part[warp][g + 8][8 * j + 2 * c + 1] = d[j][3];
    }
    __syncthreads();
    const int tok = threadIdx.x / kDownRanks, j = threadIdx.x % kDownRanks;  // 16 x 32 = the block
    if (ids[tok] != mine) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWarps; ++w) v += part[w][tok][j];
    v *= s;
    if (q + j >= r_blocks * kRankBlock) continue;
    uint16_t* to = h + (t0 + tok) * row + (q + j) / kRankBlock * 4 * kRankBlock + j % kRankBlock;
    const float whole = v;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (v == 0.f) v = whole * 0x1p-40f;
      const bool last = two_parts && k == 1;
      const uint32_t b = last ? pack_bf16x2(v, 0.f) & 0xFFFFu : __float_as_uint(v) >> 16;
      const float f = __uint_as_float(b << 16);
      to[k * kRankBlock] = static_cast<uint16_t>(b);
      v = fabsf(f) < INFINITY ? v - f : 0.f;  // every part of a non-finite h is it
    }
  }
}
static_assert(kDownThreads == kGroup * kDownRanks, "a thread per token and rank");

// ---------------------------------------------------------------- the head
struct Params {
  int64_t T, V, n;
  int32_t num_m, num_n, group_m, k_blocks, bn;
  int32_t r_blocks;             // blocks of 16 ranks
  int32_t stages, stage_bytes;
  int32_t chunk;                // k-blocks per accumulator
  int32_t tile_rows;            // tokens of a tile
  int32_t x_bytes;              // of a k-block of x: the rows there are, rounded up to 8
  int32_t a_bytes;              // of its place in a stage
  bool h_kept;                  // a token tile's h stays in shared memory (up to two rank blocks)
  bool pair;                    // a B tile holds both rank blocks, rows of 64 bytes (else one, 32)
  bool tma_out;                 // output by TMA stores
  uint32_t units;
  const int64_t* adapter;
  const LoraTile* plan;
  const int32_t* order;         // of the tokens; null: they stay
  void* out;
  uint64_t timeout_ns;
  uint32_t* status;
};

struct Unit {
  int mt, nt;
};
// Units in groups of group_m token tiles, vocab tiles outer within a group: CTAs
// that run at one time share W tiles in L2.
__device__ __forceinline__ Unit unit_of(const Params& p, uint32_t u) {
  const uint32_t per_group = static_cast<uint32_t>(p.group_m) * p.num_n;
  const uint32_t g = u / per_group, q = u - g * per_group;
  const uint32_t m0 = g * p.group_m, left = p.num_m - m0;
  const uint32_t gm = left < static_cast<uint32_t>(p.group_m) ? left : p.group_m;
  const uint32_t nt = q / gm;
  return Unit{static_cast<int>(m0 + q - nt * gm), static_cast<int>(nt)};
}

// K-major tile of rows of 64 or 32 bytes written by TMA with the swizzle of that
// width: 8-row groups 512 or 256 bytes apart, swizzle mode 4 or 6.
__device__ __forceinline__ uint64_t smem_desc_narrow(uint32_t saddr, bool pair) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>((pair ? 512 : 256) >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(pair ? 4 : 6) << 61;
  return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// One adapter's products of one rank block: h0, h1 and (kTerms 3) h2 by the same B
// tile, in the TMEM lanes whose bit of `skip` is clear.  In one statement: the issuing
// thread moves the operands to uniform registers once.
template <int kTerms>
__device__ __forceinline__ void mma_adapter(uint32_t d, uint64_t dh, uint64_t db, uint32_t idesc, uint4 skip) {
  if constexpr (kTerms == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a1;\n\tsetp.eq.u32 p, 0, 0;\n\tadd.u64 a1, %1, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, %2, %3, {%4, %5, %6, %7}, p;\n\t}"
        ::"r"(d), "l"(dh), "l"(db), "r"(idesc), "r"(skip.x), "r"(skip.y), "r"(skip.z), "r"(skip.w) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a1, a2;\n\tsetp.eq.u32 p, 0, 0;\n\tadd.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, %2, %3, {%4, %5, %6, %7}, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, %2, %3, {%4, %5, %6, %7}, p;\n\t}"
        ::"r"(d), "l"(dh), "l"(db), "r"(idesc), "r"(skip.x), "r"(skip.y), "r"(skip.z), "r"(skip.w) : "memory");
  }
}

// The order of a unit's B tiles, as the producer fills stages with them and the MMA
// thread takes them: with h kept, an adapter's tiles one after the other; else a rank
// block's adapters, whose stages bring that block of h.
struct BOrder {
  int count, tiles;   // adapters; tiles of one, of a rank block each, or of two in a row (pair)
  bool kept;
  int per_stage;
  int q = 0, e = 0;   // the next tile
  __device__ __forceinline__ int stages() const {
    return kept ? (count * tiles + per_stage - 1) / per_stage : tiles * ((count + per_stage - 1) / per_stage);
  }
  // Tiles of the next stage.
  __device__ __forceinline__ int next_stage() const {
    const int left = kept ? (count - e) * tiles - q : count - e;
    return left < per_stage ? left : per_stage;
  }
  __device__ __forceinline__ void next() {
    if (kept) {
      if (++q == tiles) { q = 0; ++e; }
    } else if (++e == count) {
      e = 0;
      ++q;
    }
  }
};

// Eight output values of one row in one 32-byte (fp32) or 16-byte (bf16) store.
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu); }

// TMA stores of a warp's tile: 16-byte piece c of row i lies where the map's
// swizzle (128 bytes for fp32 rows, 64 for bf16) has it.
__device__ __forceinline__ void st_tile(uint8_t* tile, int i, int c, const float* v, float) {
  *reinterpret_cast<float4*>(tile + i * 128 + ((c ^ (i & 7)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st_tile(uint8_t* tile, int i, int c, const float* v, uint16_t) {
  *reinterpret_cast<uint4*>(tile + i * 64 + ((c ^ ((i >> 1) & 3)) << 4)) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* tile, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(tmap), "r"(smem_u32(tile)), "r"(c0), "r"(c1) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// kVec: rows of the output are aligned for store8 and TMA.
template <typename O, bool kVec>
__global__ void __launch_bounds__(kThreads, 1)
    lora_head_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_xs,
                     const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_out, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* h_tiles = smem + p.stages * p.stage_bytes;                               // [r_blocks][16 KB] if kept
  uint8_t* out_tiles = h_tiles + (p.h_kept ? p.r_blocks * kABytes : 0);             // [kEpiWarps][2 KB] if tma_out
  uint8_t* after = out_tiles + (p.tma_out ? kEpiWarps * kOutTile : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(after);  // [kMaxStages]
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* h_full = acc_empty + 2;
  uint64_t* h_empty = h_full + 1;
  uint64_t* drain = h_empty + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  const LoraTile* plan = reinterpret_cast<const LoraTile*>(after + kBarBytes);  // of the unit's token tile
  float* stage_out = reinterpret_cast<float*>(after + kBarBytes + sizeof(LoraTile));  // unaligned rows only
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 32 * kEpiWarps);
    }
    mbar_init(h_full, 1);
    mbar_init(h_empty, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_h);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int b_bytes = p.bn * (p.pair ? 64 : 32);  // of a B tile
  const int per_stage = p.pair ? 2 : 4;           // such tiles in a stage
  const int chunks = (p.k_blocks + p.chunk - 1) / p.chunk;

  const bool other = warp < kOtherThreads / 32;
  if (other) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, last_parity = 0, h_phase = 0;
      bool ok = true;
      auto acquire = [&](uint32_t bytes) -> uint8_t* {
        if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, p.status)) return nullptr;
        mbar_arrive_expect_tx(&full[stage], bytes);
        filled |= 1u << stage;
        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
        return smem + stage * p.stage_bytes;
      };
      auto advance = [&] {
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      };
      // The token tile's adapter list and h tiles, when the tile changes: once the
      // MMAs of the unit before have read theirs.
      int tile = -1;
      const void* map_x = &tm_x;
      if (p.order && p.order[2 * p.T]) {
        map_x = &tm_xs;
        asm volatile("fence.proxy.async.global;" ::: "memory");
      }
      auto load_tile = [&](int mt) -> bool {
        if (mt == tile) return true;
        if (tile < 0) {  // lora_down is complete, and its stores are seen by the copies below
          griddep_wait();
          asm volatile("fence.proxy.async.global;" ::: "memory");
        }
        tile = mt;
        if (!mbar_wait(h_empty, h_phase ^ 1u, p.timeout_ns, p.status)) return false;
        mbar_arrive_expect_tx(h_full, static_cast<uint32_t>(sizeof(LoraTile) + (p.h_kept ? p.r_blocks * p.x_bytes : 0)));
        bulk_load(const_cast<LoraTile*>(plan), p.plan + mt, sizeof(LoraTile), h_full);
        if (p.h_kept)
          for (int q = 0; q < p.r_blocks; ++q)
            tma_load_2d(h_tiles + q * kABytes, &tm_h, q * 4 * kRankBlock, mt * p.tile_rows, h_full);
        h_phase ^= 1u;
        return true;
      };
      for (uint32_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const Unit c = unit_of(p, u);
        // The tile's list is here: its adapters' stages go between the k-blocks.  Else
        // they follow them, and the list is fetched early enough to be there then, and
        // so late that the wait for the unit before is over; the first one waits for
        // lora_down.
        const bool here = c.mt == tile;
        const int when = here || tile < 0 ? p.k_blocks : p.stages + 1 < p.k_blocks ? p.stages + 1 : p.k_blocks;
        BOrder order{here ? plan->count : 0, p.pair ? 1 : p.r_blocks, p.h_kept, per_stage};
        const auto b_stage = [&]() -> bool {
          const int m = order.next_stage();
          uint8_t* sa = acquire(static_cast<uint32_t>(m * b_bytes + (p.h_kept ? 0 : p.x_bytes)));
          if (!sa) return false;
          if (!p.h_kept) tma_load_2d(sa, &tm_h, order.q * 4 * kRankBlock, c.mt * p.tile_rows, &full[stage]);
          for (int i = 0; i < m; ++i, order.next())
            tma_load_3d(sa + p.a_bytes + i * b_bytes, &tm_b, order.q * kRankBlock, c.nt * p.bn, plan->e[order.e].adapter,
                        &full[stage]);
          advance();
          return true;
        };
        const int between = order.stages();
        int due = 0;
        for (int kb = 0; kb < p.k_blocks && ok; ++kb) {
          if (kb == when && !load_tile(c.mt)) { ok = false; break; }
          uint8_t* sa = acquire(static_cast<uint32_t>(p.x_bytes + p.bn * kBK * 2));
          if (!sa) { ok = false; break; }
          tma_load_2d(sa, map_x, kb * kBK, c.mt * p.tile_rows, &full[stage]);
          tma_load_2d(sa + p.a_bytes, &tm_w, kb * kBK, c.nt * p.bn, &full[stage]);
          advance();
          for (due += between; due >= p.k_blocks && ok; due -= p.k_blocks) ok = b_stage();
        }
        if (!ok) break;
        if (!here) {
          if (!load_tile(c.mt) || !mbar_wait(h_full, h_phase ^ 1u, p.timeout_ns, p.status)) break;
          order.count = plan->count;
          const int after = order.stages();
          for (int k = 0; k < after && ok; ++k) ok = b_stage();
        }
      }
      // never leave with copies in flight
      for (int s = 0; s < p.stages; ++s)
        if (filled & (1u << s)) mbar_wait(&full[s], (last_parity >> s) & 1u, p.timeout_ns, p.status);
      if (tile >= 0) mbar_wait(h_full, h_phase ^ 1u, p.timeout_ns, p.status);
      else griddep_wait();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr int kTerms = sizeof(O) == 4 ? 3 : 2;
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(p.bn >> 3) << 17) |
                             (static_cast<uint32_t>(kBM >> 4) << 24);
      // This thread's own instructions between two MMAs delay the tensor cores (a
      // run-time modulo per k-block took 8 % at T = 2048): a k-block costs it a wait,
      // an addition per descriptor, four MMAs and a commit.
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0, h_phase = 0;
      int tile = -1;
      bool ok = true;
      const uint32_t s0 = smem_u32(smem);
      const uint64_t h_desc = smem_desc_sw128(smem_u32(h_tiles));
      const uint64_t dn0 = smem_desc_narrow(s0 + p.a_bytes, p.pair), b_step = static_cast<uint64_t>(b_bytes) >> 4;
      const uint32_t entries = smem_u32(plan->e);
      const uint64_t da0 = smem_desc_sw128(s0), db0 = smem_desc_sw128(s0 + p.a_bytes);
      const uint64_t step = static_cast<uint64_t>(p.stage_bytes) >> 4;
      uint64_t at = 0;  // the stage's offset in a descriptor
      const auto advance = [&] {
        at += step;
        if (++stage == p.stages) {
          stage = 0;
          at = 0;
          phase ^= 1u;
        }
      };
      const int k_blocks = p.k_blocks, chunk = p.chunk;
      for (uint32_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        uint32_t d = 0;
        const int mt = unit_of(p, u).mt;
        const bool here = mt == tile;  // as the producer orders the stages
        BOrder order{here ? plan->count : 0, p.pair ? 1 : p.r_blocks, p.h_kept, per_stage};
        const auto b_stage = [&]() -> bool {
          if (!mbar_wait(&full[stage], phase, p.timeout_ns, p.status)) return false;
          tc_fence_after();
          const int m = order.next_stage();
          uint64_t db = dn0 + at;
          for (int i = 0; i < m; ++i, order.next()) {
            const uint64_t dh = p.h_kept ? h_desc + static_cast<uint64_t>(order.q) * (kABytes >> 4) : da0 + at;
            const uint4 skip = lds128(entries + static_cast<uint32_t>(order.e * sizeof(LoraEntry)));
            mma_adapter<kTerms>(d, dh, db, idesc, skip);
            if (p.pair) mma_adapter<kTerms>(d, dh + (kABytes >> 4), db + 2, idesc, skip);
            db += b_step;
          }
          tc_commit(&empty[stage]);
          advance();
          return true;
        };
        const int between = order.stages();
        int due = 0;
        for (int k0 = 0; k0 < k_blocks && ok; k0 += chunk) {
          if (k0) {  // the chunk before is complete
            tc_commit(&acc_full[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
          }
          if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          d = tmem + static_cast<uint32_t>(acc * kMaxBN);
          const int n = k_blocks - k0 < chunk ? k_blocks - k0 : chunk;
          for (int kb = 0; kb < n && ok; ++kb) {
            if (!mbar_wait(&full[stage], phase, p.timeout_ns, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint64_t da = da0 + at, db = db0 + at;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) tc_mma_bf16(d, da + 2 * k, db + 2 * k, idesc, (kb | k) ? 1u : 0u);
            tc_commit(&empty[stage]);
            advance();
            for (due += between; due >= k_blocks && ok; due -= k_blocks) ok = b_stage();
          }
        }
        if (!ok) break;
        if (!here) {  // the adapters go on in the last chunk's accumulator
          if (!mbar_wait(h_full, h_phase, p.timeout_ns, p.status)) break;
          h_phase ^= 1u;
          tile = mt;
          order.count = plan->count;
          const int after = order.stages();
          for (int k = 0; k < after && ok; ++k) ok = b_stage();
        }
        if (!ok) break;
        // the next unit is another token tile's: its list and h may overwrite these
        if (u + gridDim.x < p.units && unit_of(p, u + gridDim.x).mt != mt) tc_commit(h_empty);
        tc_commit(&acc_full[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      tc_commit(drain);
      mbar_wait(drain, 0, p.timeout_ns, p.status);
    }
  } else if (!other) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ------------------------------------------------------------ epilogue
    // Warp = a quadrant of the TMEM lanes and half of the 32-column blocks.
    const int quad = warp & 3, half = (warp - kOtherThreads / 32) >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const int blocks = (p.bn + 31) / 32, first = half ? (blocks + 1) / 2 : 0;
    const int mine = half ? blocks / 2 : (blocks + 1) / 2;
    float* sw = stage_out + (warp - kOtherThreads / 32) * 16 * kPitch;
    const bool sorted = p.order && p.order[2 * p.T];
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (uint32_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const Unit c = unit_of(p, u);
      const int64_t row0 = static_cast<int64_t>(c.mt) * p.tile_rows + quad * 32;
      const int64_t left = p.T - row0 < p.tile_rows - quad * 32 ? p.T - row0 : p.tile_rows - quad * 32;
      const int rows = static_cast<int>(left < 0 ? 0 : left < 32 ? left : 32);
      const int token = sorted && lane < rows ? p.order[row0 + lane] : static_cast<int>(row0) + lane;
      const bool bad = lane < rows && p.adapter[token] >= p.n;
      float sum[8][16];
#pragma unroll 1
      for (int ch = 0; ch < chunks; ++ch) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[acc], acc_phase, p.timeout_ns, p.status));
        if (!ok) break;
        tc_fence_after();
        if (rows > 0) {
          const uint32_t from = tmem + lane_addr + static_cast<uint32_t>(acc * kMaxBN + first * 32);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (b >= 2 * mine) break;
            uint32_t v[16];
            tmem_ld16(from + b * 16, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[b][k] = ch ? sum[b][k] + __uint_as_float(v[k]) : __uint_as_float(v[k]);
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_empty[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok) break;
      if (rows == 0) continue;
      const int64_t n0 = static_cast<int64_t>(c.nt) * p.bn;
      const int cols = static_cast<int>(p.V - n0 < p.bn ? p.V - n0 : p.bn);  // of the unit
      O* out = static_cast<O*>(p.out) + n0;
      if (kVec && p.tma_out && !sorted) {  // whole 128- or 64-byte pieces of rows, clipped at the last row and column
        constexpr int kRows = kLoraOutRows, kPer = 16 / static_cast<int>(sizeof(O));
        uint8_t* tile = out_tiles + (warp - kOtherThreads / 32) * kOutTile;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b >= mine || (first + b) * 32 >= cols) break;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (bad) {
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[2 * b + k][j] = __int_as_float(0x7FC00000);
            }
          }
#pragma unroll
          for (int part = 0; part < 32 / kRows; ++part) {
            if (part * kRows >= rows) break;
            if (lane == 0) tma_store_read();  // the tile before has left
            __syncwarp();
            if (lane / kRows == part) {
#pragma unroll
              for (int c = 0; c < 32 / kPer; ++c)
                st_tile(tile, lane % kRows, c, &sum[2 * b + c * kPer / 16][c * kPer % 16], O{});
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
              tma_store_2d(&tm_out, tile, static_cast<int32_t>(n0) + (first + b) * 32,
                           static_cast<int32_t>(row0) + part * kRows);
          }
        }
        continue;
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (b >= 2 * mine) break;
        const int c0 = first * 32 + b * 16;
        if (bad) {
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[b][k] = __int_as_float(0x7FC00000);
        }
        if constexpr (kVec) {  // a lane's row, whole sectors
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            if (lane < rows && c0 + k < cols) store8(out + static_cast<int64_t>(token) * p.V + c0 + k, &sum[b][k]);
        } else {          // through shared memory, two rows of 16 columns per store
          const int col = c0 + (lane & 15);
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 16) {
            if (r0 >= rows) break;
            __syncwarp();
            if ((lane & 16) == r0) {
#pragma unroll
              for (int k = 0; k < 16; ++k) sw[(lane & 15) * kPitch + k] = sum[b][k];
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const int i = k + (lane >> 4);
              const int64_t to = __shfl_sync(0xFFFFFFFFu, token, r0 + i);
              if (col < cols && r0 + i < rows) store1(out + to * p.V + col, sw[i * kPitch + (lane & 15)]);
            }
          }
        }
      }
    }
  }
  if (warp >= kOtherThreads / 32 && lane == 0) tma_store_read();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <typename O, bool kVec>
cudaError_t launch_head(const LoraMaps& m, const Params& p, int grid, int smem, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  if (cudaError_t e = ensure_smem_limit(lora_head_kernel<O, kVec>, kSmemMax, done)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_head_kernel<O, kVec>, m.x, m.xs, m.w, m.h, m.b, m.out, p);
}

}  // namespace

namespace {
// The vocab columns of a unit, a multiple of 16 (or of 32 for the TMA stores): the ones
// that cost the fullest SM least, in cycles, with W's k-blocks at an SM's share of
// HBM (23 bytes a cycle) and an adapter's MMA at 170 cycles (equal ones: the widest,
// which re-reads x least).  More than one token tile: bound by the tensor cores, wide
// tiles.
int choose_bn(int64_t T, int64_t H, int64_t V, int64_t n, int64_t r, int num_sms, bool tma_out) {
  const int64_t num_m = (T + kBM - 1) / kBM;
  const int64_t tokens = T < kBM ? T : kBM, sorted = (n - 1) / num_m + 1;
  const int64_t adapters = sorted < tokens ? sorted : tokens;  // of a tile
  int best = kMaxBN;
  double least = 0;
  for (int bn = kMaxBN; bn >= (num_m > 1 ? 192 : 96); bn -= tma_out ? 32 : 16) {
    const int64_t units = num_m * ((V + bn - 1) / bn);
    const double waves = static_cast<double>((units + num_sms - 1) / num_sms);
    const double bytes = 2.0 * bn * (H / num_m + adapters * r / num_m);
    const double cores = 4.0 * ((H + kBK - 1) / kBK) * bn * 0.5 + adapters * 3.0 * ((r + 15) / 16) * 170;
    const double cost = waves * (bytes / 23 > cores ? bytes / 23 : cores);
    if (least == 0 || cost < least * 0.995) {
      least = cost;
      best = bn;
    }
  }
  return best;
}
}  // namespace

LoraConfig lora_config(int64_t T, int64_t H, int64_t V, int64_t n, int64_t r, const void* out, bool out_bf16,
                       int num_sms) {
  LoraConfig c{};
  const uintptr_t at = reinterpret_cast<uintptr_t>(out);
  // Output by TMA stores: more than one token tile (a few rows are stored directly).
  c.vec_out = V % 8 == 0 && (at & (out_bf16 ? 15 : 31)) == 0;
  c.tma_out = T > kBM && c.vec_out;
  c.sorts = T > kBM && n > 1 && n <= kLoraMaxSort;
  c.bn = choose_bn(T, H, V, n, r, num_sms, c.tma_out);
  // Tokens of a tile, rows of x's and h's boxes: the tiles' share (200 tokens of 64
  // adapters are two tiles of 104 and 96).  A TMA store writes whole boxes of rows.
  // The MMA reads 128 rows of shared memory whatever was
  // loaded: past a short batch whatever follows there (a stage is 12 KB of W at least,
  // and the adapter list follows the last one), which ends in TMEM lanes that nothing
  // reads.
  const int64_t num_m = (T + kBM - 1) / kBM, unit = c.tma_out ? kLoraOutRows : 8;
  c.x_rows = static_cast<int>(((T + num_m - 1) / num_m + unit - 1) / unit * unit);
  c.a_bytes = (c.x_rows * kBK * 2 + 1023) / 1024 * 1024;
  c.stage_bytes = c.a_bytes + c.bn * kBK * 2;
  c.smem = 1024 + kBarBytes + static_cast<int>(sizeof(LoraTile)) + (c.tma_out ? kEpiWarps * kOutTile : 0) +
           (c.vec_out ? 0 : kStageOut);
  // h stays where that leaves four stages, else its block comes with every stage of B tiles
  c.r_blocks = static_cast<int>((r + kRankBlock - 1) / kRankBlock);
  c.h_kept = c.r_blocks <= 2 && c.smem + c.r_blocks * kABytes + 4 * c.stage_bytes <= kSmemMax;
  c.pair = c.h_kept && c.r_blocks == 2;
  if (c.h_kept) c.smem += c.r_blocks * kABytes;
  c.stages = (kSmemMax - c.smem) / c.stage_bytes;
  if (c.stages > kMaxStages) c.stages = kMaxStages;
  c.smem += c.stages * c.stage_bytes;
  return c;
}

cudaError_t launch_lora_head(const LoraMaps& m, const LoraArgs& a, const FusedLaunch& L) {
  const LoraConfig& c = a.cfg;
  Params p{};
  p.T = a.T;
  p.V = a.V;
  p.n = a.n;
  p.bn = c.bn;
  p.r_blocks = c.r_blocks;
  p.num_m = static_cast<int32_t>((a.T + kBM - 1) / kBM);
  p.num_n = static_cast<int32_t>((a.V + c.bn - 1) / c.bn);
  p.group_m = p.num_m < kGroupSingle ? p.num_m : kGroupSingle;
  p.k_blocks = static_cast<int32_t>((a.H + kBK - 1) / kBK);
  p.units = static_cast<uint32_t>(p.num_m) * static_cast<uint32_t>(p.num_n);
  p.adapter = a.adapter;
  p.plan = a.plan;
  p.order = c.sorts ? a.order : nullptr;
  p.out = a.out;
  p.timeout_ns = L.timeout_ns;
  p.status = a.status;
  p.tile_rows = c.x_rows;
  p.x_bytes = c.x_rows * kBK * 2;
  p.a_bytes = c.a_bytes;
  p.stage_bytes = c.stage_bytes;
  p.stages = c.stages;
  p.h_kept = c.h_kept;
  p.pair = c.pair;
  p.tma_out = c.tma_out;
  // 8 k-blocks (512 of H) where HBM is the bound and the epilogue waits anyway, 4 for
  // one quadrant of rows (under 1 % longer; 2 took 6 %); 12 for many tokens: 8 took 2
  // to 4 % longer at T = 2048, 16 under 1 % longer than one chunk.  Errors: 2.6e-7,
  // 5e-7, 7e-7 and, with 16, 1e-6 (fp32 sums: 1e-7 to 6e-7).
  p.chunk = a.T <= 32 ? 4 : p.num_m <= 2 ? 8 : 12;
  launch_mark(0, L.stream);
  const int64_t groups = (a.T + kGroup - 1) / kGroup;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * kGroup + p.num_m));
  cfg.blockDim = dim3(kDownThreads);
  cfg.stream = L.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  if (c.sorts) {
    lora_sort<<<1, kSortThreads, 0, L.stream>>>(a.adapter, a.T, static_cast<int>(a.n), c.x_rows, a.order);
    if (cudaError_t e = cudaGetLastError()) return e;
    cfg.numAttrs = 1;
    cudaLaunchConfig_t rows = cfg;
    rows.gridDim = dim3(static_cast<unsigned>(a.T));
    rows.blockDim = dim3(256);
    if (cudaError_t e = cudaLaunchKernelEx(&rows, lora_gather, a.x, a.T, a.H, static_cast<const int32_t*>(a.order), a.xs))
      return e;
  }
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down, a.x, a.A, a.adapter, a.scale, a.T, a.H, a.n, a.r, c.r_blocks,
                                         groups, a.h, a.plan, p.order, c.x_rows, a.out_bf16))
    return e;
  const int grid = static_cast<int>(p.units < static_cast<uint32_t>(L.num_sms) ? p.units : L.num_sms);
  const auto head = a.out_bf16 ? (c.vec_out ? launch_head<uint16_t, true> : launch_head<uint16_t, false>)
                               : (c.vec_out ? launch_head<float, true> : launch_head<float, false>);
  const cudaError_t e = head(m, p, grid, c.smem, L.stream);
  launch_mark(1, L.stream);
  return e;
}

}  // namespace lmho
