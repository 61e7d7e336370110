// Penalties for repeated tokens, biases, a temperature and a grammar mask on
// logits.  For token v of row t, with c the number of times v is in the row's
// output list and `seen` true when it is in the output or the prompt list:
//   z1 = seen ? (z > 0 ? z / repetition : z * repetition) : z
//   z2 = z1 - frequency * c - presence        (where c > 0)
//   z3 = z2 + the row's biases for v
//   out = allowed(v) ? z3 / temperature : -inf
//
// Two launches.  process_stream applies the temperature and the mask to every
// column: bound by HBM (logits read once, result written once), 16 bytes per
// thread and access.  The listed tokens are few next to the vocabulary, so
// process_lists computes their columns again: launched as a programmatic
// dependent, it runs beside the stream on the SM's free threads, waits for the
// stream to complete, and stores.  Per row it marks the lists' tokens in a bitmap of
// the vocabulary in shared memory, numbers the marked tokens by a scan over the
// bitmap's words, counts the output tokens by that number (dense counters whatever
// the vocabulary) and computes the numbered columns side by side.  The lists are
// read once, by asynchronous copies, and kept as 32-bit tokens for the later steps.
// Where lists are long a row gets a cluster of blocks: each marks a share of the
// lists, takes every cluster-th four words of the bitmap from all of them
// (distributed shared memory) and does those words' tokens.  A biased column is
// computed by the thread of its first bias entry.
// That chain of dependent steps is bound by latency, its reads (offsets, lists,
// logits) queueing behind the stream's; what counts is that it ends no later than the
// stream.  256 bf16 rows of 128256 with 3000 listed tokens each take 49 us (4.0 TB/s;
// the stream alone 37), 64 fp32 rows with a mask and 950 tokens 22.5 us (18.4), 37 fp32
// rows of 50001 with 40000 tokens 37 us (10.2), a single row of 128256 with 400 10 us
// (6.1), calls by themselves; in a queue of calls 49.2 and 18.5 us for the first two,
// where copies of as many bytes take 32.8 and 13.5.  With the lists read again for every
// step, 256 threads and 4096 tokens in hand those were 67, 25.6, 42 and 13 us; with the
// tokens found again from the bitmap's bits 54, 25.6, 40 and 13.5.  In one kernel with a
// word per column in shared memory the first two took 78 and 33 us; with the lists
// prepared between the chunks of the stream 143 and 53 (every vector's lookup lengthens
// the chain from its load to its store); with a hash table in the bitmap's place 85 and
// 31.6 (atomics that return a value cost far more than setting bits).
#include <cmath>
#include <cstdint>

#include "answer.h"
#include "ptx.cuh"
#include "rowstats.cuh"

namespace lmho {
namespace {

// ---------------------------------------------------------------- one element
struct RowRule {
  float repetition, frequency, presence, temperature;
  float inverse;  // 1 / temperature, 0: divide by it
};

__device__ __forceinline__ float inverse_of(float temperature) {
  if (temperature == 0.f) return 1.f;
  return fabsf(temperature) > 1e-37f && fabsf(temperature) < 1e37f ? __fdiv_rn(1.f, temperature) : 0.f;
}
__device__ __forceinline__ RowRule rule_of(const ProcessArgs& a, int64_t t) {
  RowRule r{a.repetition ? a.repetition[t] : 1.f, a.frequency ? a.frequency[t] : 0.f, a.presence ? a.presence[t] : 0.f,
            a.temperature ? a.temperature[t] : 0.f, 0.f};
  r.inverse = inverse_of(r.temperature);
  return r;
}

__device__ __forceinline__ float penalised(float z, uint32_t count, const RowRule& r) {
  z = z > 0.f ? __fdiv_rn(z, r.repetition) : __fmul_rn(z, r.repetition);
  if (count) {
    z = __fsub_rn(z, __fmul_rn(r.frequency, static_cast<float>(count)));
    z = __fsub_rn(z, r.presence);
  }
  return z;
}
// z / temperature as z times the rounded reciprocal: one rounding more than the
// division, and one instruction in place of ten on every element.  Temperatures
// whose reciprocal leaves the normal range divide.
__device__ __forceinline__ float scaled(float z, float inverse, float temperature) {
  return inverse != 0.f ? __fmul_rn(z, inverse) : __fdiv_rn(z, temperature);
}

// ---------------------------------------------------------------- the stream
// Each thread pipelines its own vectors: asynchronous copies of the 16-byte
// vector and its mask word run kDepth vectors ahead into slots that only this
// thread reads, so there is no barrier and the bytes in flight (32 KB per SM) take
// no registers; with 5 ahead the lists' reads beside it wait longer (256 bf16 rows
// of 128256 took 4 us more), with 3 the stream itself loses 1 us.  A block works on
// a contiguous range of chunks, a chunk being one vector per thread; the temperature
// of the row after this one is read a row ahead.
constexpr int kStreamThreads = 256;
constexpr int kDepth = 4;
constexpr int kElements = 8;  // of a thread of process_elements

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async8(void* smem, const void* g) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async4(void* smem, const void* g) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
// 32 bytes in one store (sm_100+): eight fp32 of one thread, whole sectors.
__device__ __forceinline__ void st_v8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
__device__ __forceinline__ void st_vec(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st_vec(float* p, const float (&v)[8]) { st_v8(p, v); }

struct StreamSlots {
  uint4 vec[kDepth][kStreamThreads];
  uint32_t mask[kDepth][kStreamThreads];
};

// The row and column of a thread's vector, as it steps through the tensor.
struct Place {
  int64_t t;
  uint32_t c;
  __device__ __forceinline__ Place(int64_t e, uint32_t V) : t(e / V), c(static_cast<uint32_t>(e - t * V)) {}
  // `by` elements on (V + by < 2^32); true when the row is another.
  __device__ __forceinline__ bool step(uint32_t by, uint32_t V) {
    c += by;
    if (c < V) return false;
    const uint32_t rows = V >= by ? 1u : c / V;
    t += rows;
    c -= rows * V;
    return true;
  }
};

// A block's contiguous range of the tensor's 16-byte vectors, which need not begin
// with the rows: the few that hold two rows' ends are taken element by element.
template <typename E, bool kMask>
__global__ void __launch_bounds__(kStreamThreads, 5) process_stream(const E* __restrict__ logits, const ProcessArgs a,
                                                                    int64_t chunks) {
  constexpr int N = Elt<E>::kPerVec;
  constexpr uint32_t kStep = kStreamThreads * N;
  extern __shared__ __align__(16) uint8_t slots_raw[];
  StreamSlots& sl = *reinterpret_cast<StreamSlots*>(slots_raw);
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const uint32_t V = static_cast<uint32_t>(a.V);
  const int64_t total = a.T * a.V, vectors = total / N;
  const int64_t each = (chunks + gridDim.x - 1) / gridDim.x;
  const int64_t first = blockIdx.x * each * kStreamThreads + tid;
  if (blockIdx.x * each >= chunks) return;
  // this thread's whole vectors
  const int64_t left = first < vectors ? (vectors - first + kStreamThreads - 1) / kStreamThreads : 0;
  const int n = static_cast<int>(left < each ? left : each);
  const auto temperature_of = [&](int64_t t) { return a.temperature && t < a.T ? __ldg(a.temperature + t) : 0.f; };
  const auto one = [&](float z, Place at, uint32_t j) {  // an element's result
    at.step(j, V);
    const float temperature = temperature_of(at.t);
    const bool allowed = !kMask || (__ldg(a.mask + at.t * a.mask_words + (at.c >> 5)) >> (at.c & 31)) & 1u;
    return allowed ? scaled(z, inverse_of(temperature), temperature) : -INFINITY;
  };
  Place here(first * N, V), ahead = here;
  const E* src = logits + first * N;
  float* dst = a.out + first * N;
  float temperature = temperature_of(here.t), following = temperature_of(here.t + 1);
  float inverse = inverse_of(temperature);
  const uint32_t* mask_here = kMask ? a.mask + here.t * a.mask_words : nullptr;
  const uint32_t* mask_ahead = mask_here;
  auto issue = [&](int d) {
    cp_async16(&sl.vec[d][tid], src);
    src += kStep;
    if constexpr (kMask) {
      cp_async4(&sl.mask[d][tid], mask_ahead + (ahead.c >> 5));
      if (ahead.step(kStep, V)) mask_ahead = a.mask + ahead.t * a.mask_words;
    }
  };
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k < n) issue(k);
    cp_async_commit();
  }
#pragma unroll 1
  for (int k = 0, d = 0; k < n; ++k, d = d + 1 == kDepth ? 0 : d + 1) {
    cp_async_wait<kDepth - 1>();
    if (here.c + N <= V) {
      float v[N];
      Elt<E>::unpack(sl.vec[d][tid], v);
      if (inverse != 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = __fmul_rn(v[j], inverse);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = scaled(v[j], inverse, temperature);
      }
      if constexpr (kMask) {
        const uint32_t shift = here.c & 31;
        uint32_t bits = sl.mask[d][tid] >> shift;
        if (shift + N > 32)  // odd vocabularies: columns of two words
          bits |= __ldg(mask_here + (here.c >> 5) + 1) << (32 - shift);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (bits >> j) & 1u ? v[j] : -INFINITY;
      }
      st_vec(dst, v);
    } else {
      const E* z = reinterpret_cast<const E*>(&sl.vec[d][tid]);
#pragma unroll 1
      for (int j = 0; j < N; ++j) dst[j] = one(Elt<E>::load_any(z + j), here, j);
    }
    dst += kStep;
    if (here.step(kStep, V)) {
      if constexpr (kMask) mask_here = a.mask + here.t * a.mask_words;
      temperature = V >= kStep ? following : temperature_of(here.t);
      inverse = inverse_of(temperature);
      following = temperature_of(here.t + 1);
    }
    if (k + kDepth < n) issue(d);
    cp_async_commit();
  }
  if (first + static_cast<int64_t>(n) * kStreamThreads == vectors && n < each) {  // the elements past the last vector
    const int64_t e0 = vectors * N;
    for (int j = 0; e0 + j < total; ++j) a.out[e0 + j] = one(Elt<E>::load1(logits + e0 + j), Place(e0, V), j);
  }
}

// Tensors off the 16-byte grid, an element at a time.
template <typename E>
__global__ void __launch_bounds__(kStreamThreads) process_elements(const E* __restrict__ logits, const ProcessArgs a,
                                                                   int64_t per_row) {
  griddep_launch_dependents();
  const int64_t t = blockIdx.x / per_row;
  const float temperature = a.temperature ? a.temperature[t] : 0.f, inverse = inverse_of(temperature);
  const uint32_t* mask = a.mask ? a.mask + t * a.mask_words : nullptr;
  const int64_t c0 = (blockIdx.x - t * per_row) * kElements * kStreamThreads + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kElements; ++k) {
    const int64_t c = c0 + k * kStreamThreads;
    if (c >= a.V) break;
    const bool allowed = !mask || (__ldg(mask + (c >> 5)) >> (c & 31)) & 1u;
    a.out[t * a.V + c] = allowed ? scaled(Elt<E>::load1(logits + t * a.V + c), inverse, temperature) : -INFINITY;
  }
}

// ---------------------------------------------------------------- the lists
// Two blocks of 512 threads and 40 registers, with 80 KB each at a vocabulary of
// 128256, fit an SM beside the stream's two.
constexpr int kT = 512;
constexpr int kBiasList = 512;    // a row's biases kept in shared memory
constexpr int64_t kProcessMaxWords = 8192;  // of a bitmap: 262144 tokens
constexpr int kBatch = 4;         // columns per thread whose loads are in flight together
constexpr int kMaxCluster = 8;
constexpr uint32_t kNoToken = 0xFFFFFFFFu;

// Entries [lo, hi) of row t in a ragged list of `total` entries (offsets that
// are out of range or out of order give an empty or clipped list).
struct Span {
  int64_t lo, hi;
};
__device__ __forceinline__ Span span_of(const int64_t* offsets, int64_t t, int64_t total) {
  if (!offsets) return Span{0, 0};
  int64_t lo = offsets[t], hi = offsets[t + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > total ? total : hi;
  return Span{lo, hi < lo ? lo : hi};
}

// A thread's share of a row's lists on its way through shared memory: tokens
// [lo, hi) of the prompt and the output list end to end, every kT-th of them this
// thread's, by asynchronous copies into slots that only this thread reads.  Two
// halves of `half` tokens: one is worked on while the other is in flight.
struct Tokens {
  const int64_t* prompt;  // the row's
  const int64_t* output;
  int n_prompt, lo, hi;
  int64_t* slots;         // [2 * half]
  int half;               // a multiple of kT

  __device__ __forceinline__ void issue(int base, int64_t* to) const {
    const int end = base + half < hi ? base + half : hi;
    const int mid = n_prompt < end ? n_prompt : end;
    int j = base + threadIdx.x;
    to += threadIdx.x;
#pragma unroll 4
    for (; j < mid; j += kT, to += kT) cp_async8(to, prompt + j);
#pragma unroll 4
    for (; j < end; j += kT, to += kT) cp_async8(to, output + (j - n_prompt));
    cp_async_commit();
  }
  __device__ __forceinline__ void start() const {
    issue(lo, slots);
    issue(lo + half, slots + half);
  }
  // Calls f(place from lo, token) for this thread's tokens.
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    int64_t* at = slots;
    for (int base = lo; base < hi; base += half) {
      cp_async_wait<1>();
      const int end = hi - base < half ? hi - base : half;
#pragma unroll 4
      for (int i = threadIdx.x; i < end; i += kT) f(base - lo + i, at[i]);
      issue(base + 2 * half, at);
      at = at == slots ? slots + half : slots;
    }
    cp_async_wait<0>();
  }
};

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

struct Shared {
  int32_t bias_token[kBiasList];  // token - v0, -1 outside the window
  float bias_value[kBiasList];
  uint32_t warp_sum[kT / 32];
  int repeats;                    // a token of the window has more than one bias
  int any_repeats;                // one of an earlier window
};

// One row's lists, as every helper below takes them.
template <typename E>
struct Row {
  const E* in;
  float* out;
  const uint32_t* mask;
  Span prompt, output, bias;
  RowRule rule;
  const int64_t* bias_tokens;
  const float* bias_values;
  bool bias_kept;  // in sh.bias_token / sh.bias_value
  bool waited;     // for the stream (per thread)

  // the stream's own values of the listed columns come first
  __device__ __forceinline__ void wait() {
    if (!waited) griddep_wait();
    waited = true;
  }
  __device__ __forceinline__ bool allowed(int64_t v) const {
    return !mask || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u);
  }
};

// The biases of the columns: mine(v, at) says whether token v0 + v is this block's
// now, and at which number it is in hand (kUnlisted: it is in no list).  A token's
// first entry computes its column: in hand it replaces the value there, else it is
// stored.  The first of a thread's entries has its logit loaded already.  Where a token
// has several biases every entry looks through the list: up to kBiasList entries here,
// longer lists in repeated_biases.
constexpr uint32_t kUnlisted = 0xFFFFFFFFu;
struct FirstBias {
  int64_t token;
  float value, z;
  bool write;  // the mask allows it
};
template <typename E, class F, class C>
__device__ __forceinline__ void bias_columns(Shared& sh, Row<E>& r, const FirstBias& first, int64_t v0, uint32_t width,
                                             float* value, C&& count_of, F&& mine) {
  if (sh.repeats && !r.bias_kept) return;
  const int64_t b0 = r.bias.lo + threadIdx.x;
  for (int64_t k = b0; k < r.bias.hi; k += kT) {
    const auto token_at = [&](int64_t i) -> uint64_t {
      return r.bias_kept ? static_cast<uint64_t>(static_cast<int64_t>(sh.bias_token[i - r.bias.lo]))
                         : static_cast<uint64_t>(r.bias_tokens[i]) - static_cast<uint64_t>(v0);
    };
    const auto value_at = [&](int64_t i) { return r.bias_kept ? sh.bias_value[i - r.bias.lo] : r.bias_values[i]; };
    const uint64_t v = k == b0 ? static_cast<uint64_t>(first.token) - static_cast<uint64_t>(v0) : token_at(k);
    uint32_t at = kUnlisted;
    if (v >= width || !mine(static_cast<uint32_t>(v), at)) continue;
    float add = k == b0 ? first.value : value_at(k);
    if (sh.repeats) {
      bool earliest = true;
      for (int64_t i = r.bias.lo; i < k && earliest; ++i) earliest = token_at(i) != v;
      if (!earliest) continue;
      for (int64_t i = k + 1; i < r.bias.hi; ++i)
        if (token_at(i) == v) add = __fadd_rn(add, value_at(i));
    }
    const int64_t col = v0 + static_cast<int64_t>(v);
    float z = k == b0 ? first.z : Elt<E>::load1(r.in + col);
    if (at != kUnlisted) z = penalised(z, count_of(at), r.rule);
    z = scaled(__fadd_rn(z, add), r.rule.inverse, r.rule.temperature);
    if (at != kUnlisted) {
      value[at] = z;
    } else if (k == b0 ? first.write : r.allowed(col)) {
      r.wait();
      r.out[col] = z;
    }
  }
}

// The values of `n` listed columns into value[i], the i-th by at(i, token, count);
// a masked token's hand[i] becomes kNoToken (the stream's -inf stays).
template <typename E, class F>
__device__ __forceinline__ void list_values(const Row<E>& r, int64_t v0, uint32_t n, uint32_t* hand, float* value,
                                            F&& at) {
  for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kBatch * kT) {
    uint32_t v[kBatch], c[kBatch];
    float z[kBatch];
    bool write[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t i = i0 + k * kT;
      v[k] = c[k] = 0;
      z[k] = 0.f;
      write[k] = true;
      if (i >= n) continue;
      at(i, v[k], c[k]);
      z[k] = Elt<E>::load1(r.in + v0 + v[k]);
      write[k] = r.allowed(v0 + v[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t i = i0 + k * kT;
      if (i >= n) break;
      value[i] = scaled(penalised(z[k], c[k], r.rule), r.rule.inverse, r.rule.temperature);
      if (!write[k]) hand[i] = kNoToken;
    }
  }
}

// The biased columns of a row whose list is long and has tokens more than once, after
// everything else of the row: the work grows with the lists' lengths (times the rounds
// of `room` / 3 tokens), where a search for every entry's repetitions takes the square
// (60000 biases, one of them repeated: 4.0 ms and 711).  The biased tokens of this
// block's words get numbers as the listed ones do, and by these their output counts,
// whether they are in a list, and the sums of their biases in list order: a warp takes
// the tokens of every kWarps-th word and walks the list 32 entries at a time.
constexpr int kWarps = kT / 32;
constexpr int kWalk = 4;  // entries of a lane in flight
constexpr uint32_t kSeen = 1u << 31, kSummed = 1u << 30;  // above a count (at most kProcessMaxTokens)
static_assert(kProcessMaxTokens < kSummed, "a count's bits");
template <typename E>
__device__ __noinline__ void repeated_biases(const E* logits, const ProcessArgs& a, int64_t t, int rank, int cluster,
                                             uint32_t* maps, int words, int room, uint32_t* warp_sum) {
  const E* in = logits + t * a.V;
  float* out = a.out + t * a.V;
  const uint32_t* mask = a.mask ? a.mask + t * a.mask_words : nullptr;
  const Span prompt = span_of(a.prompt_offsets, t, a.n_prompt), output = span_of(a.output_offsets, t, a.n_output),
             bias = span_of(a.bias_offsets, t, a.n_bias);
  const RowRule rule = rule_of(a, t);
  const uint32_t most = room / 3;
  uint32_t* marked = maps;
  uint32_t* number = maps + words;
  uint32_t* hand = maps + 2 * words;
  uint32_t* count = hand + most;
  float* sum = reinterpret_cast<float*>(count + most);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t v0 = 0; v0 < a.V; v0 += static_cast<int64_t>(words) * 32) {
    const int64_t left = a.V - v0;
    const uint32_t width = static_cast<uint32_t>(left < words * 32 ? left : words * 32);
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += kT) marked[i] = 0;
    __syncthreads();
    for (int64_t k = bias.lo + threadIdx.x; k < bias.hi; k += kT) {
      const uint64_t v = static_cast<uint64_t>(a.bias_tokens[k]) - static_cast<uint64_t>(v0);
      if (v < width && ((v >> 7) & (cluster - 1)) == static_cast<uint32_t>(rank))
        atomicOr(&marked[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    // numbers in the tokens' order: a round is a range of tokens
    const int each = (words + kT - 1) / kT, w0 = threadIdx.x * each, w1 = min(w0 + each, words);
    uint32_t mine = 0;
    for (int i = w0; i < w1; ++i) mine += __popc(marked[i]);
    uint32_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    uint32_t total = 0, base = upto - mine;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += warp_sum[w];
      total += warp_sum[w];
    }
    for (int i = w0; i < w1; ++i) {
      number[i] = base;
      base += __popc(marked[i]);
    }
    __syncthreads();
    for (uint32_t n0 = 0; n0 < total; n0 += most) {
      const uint32_t n = total - n0 < most ? total - n0 : most;
      for (int i = threadIdx.x; i < words; i += kT) {
        uint32_t at = number[i] - n0;
        for (uint32_t bits = marked[i]; bits; bits &= bits - 1, ++at)
          if (at < n) {
            hand[at] = static_cast<uint32_t>(i * 32 + __ffs(bits) - 1);
            count[at] = 0;
          }
      }
      __syncthreads();
      const int64_t first = v0 + hand[0];
      const uint32_t range = hand[n - 1] - hand[0];
      const auto in_round = [&](int64_t token) {
        return static_cast<uint64_t>(token) - static_cast<uint64_t>(first) <= range;
      };
      const auto place_of = [&](int64_t token) -> uint32_t {  // of a token in that range
        const uint32_t v = static_cast<uint32_t>(token - v0), bits = marked[v >> 5], bit = 1u << (v & 31);
        return bits & bit ? number[v >> 5] + __popc(bits & (bit - 1)) - n0 : kUnlisted;
      };
      for (int64_t k = prompt.lo + threadIdx.x; k < prompt.hi; k += kT) {
        const int64_t token = a.prompt[k];
        const uint32_t at = in_round(token) ? place_of(token) : kUnlisted;
        if (at < n) atomicOr(&count[at], kSeen);
      }
      for (int64_t k = output.lo + threadIdx.x; k < output.hi; k += kT) {
        const int64_t token = a.output[k];
        const uint32_t at = in_round(token) ? place_of(token) : kUnlisted;
        if (at < n) atomicAdd(&count[at], 1u);
      }
      for (int64_t k0 = bias.lo; k0 < bias.hi; k0 += 32 * kWalk) {
        int64_t token[kWalk];
#pragma unroll
        for (int j = 0; j < kWalk; ++j) {
          const int64_t k = k0 + 32 * j + lane;
          token[j] = k < bias.hi ? a.bias_tokens[k] : -1;
        }
#pragma unroll
        for (int j = 0; j < kWalk; ++j) {
          const bool may = in_round(token[j]) && ((token[j] >> 5) & (kWarps - 1)) == warp;
          if (!__any_sync(0xFFFFFFFFu, may)) continue;
          const uint32_t at = may ? place_of(token[j]) : kUnlisted;
          const bool ours = at < n;
          uint32_t same = __match_any_sync(0xFFFFFFFFu, ours ? at : kUnlisted);
          if (ours && lane == __ffs(same) - 1) {
            const float* value = a.bias + k0 + 32 * j;
            const bool more = atomicOr(&count[at], kSummed) & kSummed;
            float s = more ? __fadd_rn(sum[at], value[lane]) : value[lane];
            for (same &= same - 1; same; same &= same - 1) s = __fadd_rn(s, value[__ffs(same) - 1]);
            sum[at] = s;
          }
          __syncwarp();
        }
      }
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < n; i += kT) {
        const int64_t v = v0 + hand[i];
        if (mask && !((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u)) continue;
        float z = Elt<E>::load1(in + v);
        const uint32_t c = count[i] & ~(kSeen | kSummed);
        if (c || (count[i] & kSeen)) z = penalised(z, c, rule);
        out[v] = scaled(__fadd_rn(z, sum[i]), rule.inverse, rule.temperature);
      }
      __syncthreads();
    }
  }
}

// Dynamic shared memory, 32-bit words: a bitmap of the listed tokens and the numbers
// of its words' first tokens ([words] each, a multiple of 4; the second is a bitmap of
// the biased tokens first), then [numbered] tokens in hand with their counts and
// their columns' values.  The lists come in through the last two while those are not
// in use; lists of at most [numbered] tokens stay in the last until the values do.
constexpr size_t lists_bytes(int64_t words, int numbered) {
  return static_cast<size_t>(words) * 8 + static_cast<size_t>(numbered) * 8;
}
// A numbered token and its count share a word, 18 bits and 14; longer output lists
// take two words.
constexpr uint32_t kTokenBits = 18, kTokenMask = (1u << kTokenBits) - 1;
constexpr int64_t kPackedCounts = (1 << (32 - kTokenBits)) - 1;
static_assert(kProcessMaxWords * 32 == 1 << kTokenBits, "a window's token fits");

template <typename E, bool kCluster>
__global__ void __launch_bounds__(kT, 3) process_lists(const E* __restrict__ logits,
                                                       const __grid_constant__ ProcessArgs a, int cluster, int numbered) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint32_t maps[];
  const int64_t t = blockIdx.x / cluster;
  const int rank = static_cast<int>(blockIdx.x - t * cluster);
  Row<E> r{logits + t * a.V, a.out + t * a.V, a.mask ? a.mask + t * a.mask_words : nullptr,
           span_of(a.prompt_offsets, t, a.n_prompt), span_of(a.output_offsets, t, a.n_output),
           span_of(a.bias_offsets, t, a.n_bias), rule_of(a, t), a.bias_tokens, a.bias, false, false};
  r.bias_kept = r.bias.hi - r.bias.lo <= kBiasList;
  const int64_t all_words = (a.V + 31) / 32;
  const int words = static_cast<int>(all_words < kProcessMaxWords ? (all_words + 3) & ~3 : kProcessMaxWords);  // of a window
  uint32_t* in_lists = maps;
  uint32_t* number = maps + words;
  uint32_t* in_bias = number;
  uint32_t* hand = maps + 2 * words;
  float* value = reinterpret_cast<float*>(hand + numbered);
  const bool packed = r.output.hi - r.output.lo < kPackedCounts;
  const uint32_t most = packed ? numbered : numbered / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // This block's words of a window's bitmap: every cluster-th four, as the common
  // tokens have low numbers.
  const auto word_at = [&](int j) { return 4 * (rank + (j >> 2) * cluster) + (j & 3); };
  const auto owned = [&](uint32_t v) { return !kCluster || ((v >> 7) & (cluster - 1)) == static_cast<uint32_t>(rank); };

  if (threadIdx.x == 0) sh.repeats = sh.any_repeats = 0;
  // windows of the vocabulary: one up to 262144 tokens
  for (int64_t v0 = 0; v0 < a.V; v0 += static_cast<int64_t>(words) * 32) {
    const int64_t left = a.V - v0;
    const uint32_t width = static_cast<uint32_t>(left < words * 32 ? left : words * 32);
    // this block's share of the lists, to be marked
    const int n_prompt = static_cast<int>(r.prompt.hi - r.prompt.lo);
    const int n_tokens = n_prompt + static_cast<int>(r.output.hi - r.output.lo);
    const int share = (n_tokens + cluster - 1) / cluster, first = rank * share;
    const int64_t* prompt = a.prompt + r.prompt.lo;
    const int64_t* output = a.output + r.output.lo;
    const bool kept = !kCluster && n_tokens <= numbered;  // then in one round, below
    uint32_t* list = reinterpret_cast<uint32_t*>(value);
    const Tokens marked{prompt, output, n_prompt, first, min(first + share, n_tokens),
                            reinterpret_cast<int64_t*>(hand), kCluster ? numbered / 2 : numbered / 4};
    const Tokens counted{prompt, output, n_prompt, n_prompt, n_tokens,
                             reinterpret_cast<int64_t*>(value), numbered / 4};
    marked.start();
    const int64_t b0 = r.bias.lo + threadIdx.x;
    FirstBias bias{b0 < r.bias.hi ? a.bias_tokens[b0] : -1, b0 < r.bias.hi ? a.bias[b0] : 0.f, 0.f, true};
    __syncthreads();
    for (int i = threadIdx.x; i < words / 2; i += kT) reinterpret_cast<uint4*>(maps)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
      sh.any_repeats |= sh.repeats;
      sh.repeats = 0;
    }
    __syncthreads();
    marked.each([&](int j, int64_t token) {
      const uint64_t v = static_cast<uint64_t>(token) - static_cast<uint64_t>(v0);
      if (kept) list[j] = v < width ? static_cast<uint32_t>(v) : kNoToken;
      if (v < width) atomicOr(&in_lists[v >> 5], 1u << (v & 31));
    });
    for (int64_t k = b0; k < r.bias.hi; k += kT) {
      const uint64_t v = static_cast<uint64_t>(k == b0 ? bias.token : a.bias_tokens[k]) - static_cast<uint64_t>(v0);
      if (r.bias_kept) {
        sh.bias_token[k - r.bias.lo] = v < width ? static_cast<int32_t>(v) : -1;
        sh.bias_value[k - r.bias.lo] = k == b0 ? bias.value : a.bias[k];
      }
      if (v >= width) continue;
      const uint32_t bit = 1u << (v & 31);
      if (atomicOr(&in_bias[v >> 5], bit) & bit) sh.repeats = 1;
    }
    if constexpr (kCluster) {
      cluster_sync();
      for (int j = threadIdx.x, i; (i = word_at(j)) < words; j += kT) {
        uint32_t bits[kMaxCluster];
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b) bits[b] = b < cluster ? ld_dsmem_u32(mapa_shared(&in_lists[i], b)) : 0u;
        uint32_t any = 0;
#pragma unroll
        for (int b = 0; b < kMaxCluster; ++b) any |= bits[b];
        in_lists[i] = any;  // the other blocks read other words of this bitmap
      }
      cluster_sync();
    } else {
      __syncthreads();
    }

    if (!kept) counted.start();
    if (bias.token >= v0 && bias.token < v0 + width) {
      bias.z = Elt<E>::load1(r.in + bias.token);
      bias.write = r.allowed(bias.token);
    }

    // Numbers of the marked tokens, in any order: a thread sums every kT-th four
    // words, the block scans the threads' sums.
    const uint4* fours = reinterpret_cast<const uint4*>(in_lists);
    uint32_t mine = 0;
    for (int q = rank + threadIdx.x * cluster; q < words / 4; q += kT * cluster)
      mine += __popc(fours[q].x) + __popc(fours[q].y) + __popc(fours[q].z) + __popc(fours[q].w);
    uint32_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += o;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    uint32_t total = 0, base = upto - mine;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) {
      if (w < warp) base += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    for (int q = rank + threadIdx.x * cluster; q < words / 4; q += kT * cluster) {
      const uint4 b = fours[q];
      uint4 at = make_uint4(base, 0, 0, 0);
      at.y = at.x + __popc(b.x);
      at.z = at.y + __popc(b.y);
      at.w = at.z + __popc(b.z);
      base = at.w + __popc(b.w);
      reinterpret_cast<uint4*>(number)[q] = at;
    }
    __syncthreads();
    const auto number_of = [&](uint32_t v) {
      return number[v >> 5] + __popc(in_lists[v >> 5] & ((1u << (v & 31)) - 1));
    };

    for (uint32_t n0 = 0; n0 == 0 || n0 < total; n0 += most) {
      const uint32_t n = total - n0 < most ? total - n0 : most;
      if (n0 > 0) counted.start();
      if (kept) {  // from the list: repeated tokens store the same
#pragma unroll 4
        for (int j = threadIdx.x; j < n_tokens; j += kT)
          if (list[j] != kNoToken) hand[number_of(list[j])] = list[j];
        __syncthreads();
#pragma unroll 4
        for (int j = n_prompt + threadIdx.x; j < n_tokens; j += kT)
          if (list[j] != kNoToken) atomicAdd(&hand[number_of(list[j])], 1u << kTokenBits);
      } else {  // from the bitmap, and the output list once more
        for (int j = threadIdx.x, i; (i = word_at(j)) < words; j += kT) {
          uint32_t bits = in_lists[i], at = number[i] - n0;
          for (; bits; bits &= bits - 1, ++at)
            if (at < n) hand[at] = static_cast<uint32_t>(i * 32 + __ffs(bits) - 1);
        }
        if (!packed)
          for (uint32_t i = threadIdx.x; i < n; i += kT) hand[most + i] = 0;
        __syncthreads();
        counted.each([&](int, int64_t token) {
          const uint64_t v = static_cast<uint64_t>(token) - static_cast<uint64_t>(v0);
          if (v >= width || !owned(static_cast<uint32_t>(v))) return;
          const uint32_t at = number_of(static_cast<uint32_t>(v)) - n0;
          if (at < n) atomicAdd(packed ? &hand[at] : &hand[most + at], packed ? 1u << kTokenBits : 1u);
        });
      }
      __syncthreads();
      const auto count_of = [&](uint32_t i) { return packed ? hand[i] >> kTokenBits : hand[most + i]; };
      list_values(r, v0, n, hand, value, [&](uint32_t i, uint32_t& v, uint32_t& c) {
        v = hand[i] & kTokenMask;
        c = count_of(i);
      });
      __syncthreads();
      bias_columns(sh, r, bias, v0, width, value, count_of, [&](uint32_t v, uint32_t& at) {
        if (!owned(v)) return false;
        if (!((in_lists[v >> 5] >> (v & 31)) & 1u)) return n0 == 0;
        at = number_of(v) - n0;
        return at < n;
      });
      __syncthreads();
      r.wait();
      for (uint32_t i = threadIdx.x; i < n; i += kT)
        if (hand[i] != kNoToken) r.out[v0 + (hand[i] & kTokenMask)] = value[i];
      __syncthreads();
    }
  }
  r.wait();  // the call is over only when the stream is
  if (!r.bias_kept && (sh.repeats | sh.any_repeats))
    repeated_biases(logits, a, t, rank, cluster, maps, words, 2 * numbered, sh.warp_sum);
}

// ---------------------------------------------------------------- launches
constexpr int kStreamBlocks = 2;      // per SM: a third took 2 us more at 64 x 128256, leaving less to the lists
// A cluster doubles while its blocks have this many tokens each and all rows' blocks
// can be resident: 37 rows of 40000 tokens take 38 us with 4 blocks a row, 48 with 8
// (the last of those 37 clusters found no place until others had ended).
constexpr int64_t kLongLists = 4096;
// Tokens in hand at a time (a multiple of 4 kT): rows with more take another round
// after the stream, 54 us instead of 51 at 256 x 128256 with 4096.
constexpr int kNumbered = 6144, kNumberedCluster = 8192;

// ensure_smem_limit, and the SM's memory split so that all of it may be shared:
// with a split made for this kernel alone, no block of the lists' kernel fits
// beside it and that kernel starts when the stream has ended.
template <class K>
cudaError_t ensure_shared_sm(K kern, int bytes, std::atomic<bool> (&done)[kMaxDevices]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                           cudaSharedmemCarveoutMaxShared))
    return e;
  return ensure_smem_limit(kern, bytes, done);
}

template <typename E, bool kCluster>
cudaError_t launch_lists(const E* logits, const ProcessArgs& a, int cluster, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  const int64_t all = (a.V + 31) / 32, words = all < kProcessMaxWords ? all : kProcessMaxWords;
  const int numbered = kCluster ? kNumberedCluster : kNumbered;
  if (cudaError_t e = ensure_smem_limit(process_lists<E, kCluster>,
                                        static_cast<int>(lists_bytes(kProcessMaxWords, numbered)), done))
    return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T * cluster));
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = lists_bytes((words + 3) & ~3, numbered);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, process_lists<E, kCluster>, logits, a, cluster, numbered);
}

template <typename E>
cudaError_t launch(const E* logits, const ProcessArgs& a, int num_sms, cudaStream_t st) {
  constexpr int N = Elt<E>::kPerVec;
  const bool vectors = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.out) & (4 * N - 1)) == 0;
  const int64_t chunks = (a.T * a.V + kStreamThreads * N - 1) / (kStreamThreads * N);
  const int64_t most = static_cast<int64_t>(num_sms) * kStreamBlocks;
  launch_mark(0, st);
  if (vectors) {
    static std::atomic<bool> done[2][kMaxDevices];
    const auto kernel = a.mask ? process_stream<E, true> : process_stream<E, false>;
    if (cudaError_t e = ensure_shared_sm(kernel, sizeof(StreamSlots), done[a.mask != nullptr])) return e;
    kernel<<<static_cast<unsigned>(chunks < most ? chunks : most), kStreamThreads, sizeof(StreamSlots), st>>>(logits, a,
                                                                                                           chunks);
  } else {
    const int64_t per_row = (a.V + kElements * kStreamThreads - 1) / (kElements * kStreamThreads);
    process_elements<E><<<static_cast<unsigned>(a.T * per_row), kStreamThreads, 0, st>>>(logits, a, per_row);
  }
  cudaError_t e = cudaGetLastError();
  const int64_t tokens = (a.prompt_offsets ? a.n_prompt : 0) + (a.output_offsets ? a.n_output : 0);
  if (e == cudaSuccess && (tokens > 0 || a.bias_offsets)) {
    int cluster = 1;
    while (cluster < kMaxCluster && tokens >= a.T * kLongLists * cluster && 4 * a.T * cluster <= 3 * num_sms) cluster *= 2;
    e = cluster > 1 ? launch_lists<E, true>(logits, a, cluster, st) : launch_lists<E, false>(logits, a, 1, st);
  }
  launch_mark(1, st);
  return e;
}

}  // namespace

cudaError_t launch_logits_process_f32(const float* logits, const ProcessArgs& a, int num_sms, cudaStream_t st) {
  return launch(logits, a, num_sms, st);
}
cudaError_t launch_logits_process_bf16(const uint16_t* logits, const ProcessArgs& a, int num_sms, cudaStream_t st) {
  return launch(logits, a, num_sms, st);
}

}  // namespace lmho
