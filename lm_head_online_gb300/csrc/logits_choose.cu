// Each row's n best tokens with their log-probabilities, and one token drawn
// among them.  For row t of the logits:
//   lse  = ln sum_v exp(z_v);  a token's log-probability is z - lse
//   best = the n tokens of largest z above -inf, ties by the lowest token
//   kept = the first top_k of them, then those whose probability mass before
//          them, renormalised over that prefix, is below top_p
//   token = argmax over the kept of z_j + noise[t, j] (j the rank), ties by rank:
//          with Gumbel noise a draw from the kept tokens' softmax, without noise
//          the best token.
// A row that holds a NaN or +inf has no token (-1) and NaN log-probabilities; a
// row whose logits are all -inf has no token and -inf.
//
// One pass over the logits.  A row is cut into S pieces, one block each, the
// blocks of a row a cluster.  A piece is streamed in steps of 256 threads x U
// 16-byte vectors held in registers.  Each step folds its values into the
// thread's running (max, sum of exp) and sets aside, in shared memory, the
// vectors whose maximum can still be among the n best.  What can: every warp
// takes the k-th largest of its threads' running maxima, k = ceil(n / 8), and the
// least of the block's 8 such values is a bound that at least n different logits
// reach; it is taken anew after 1, 2, 4, 8, ... steps, so a step sets aside a
// handful of vectors and all others cost one comparison.  The warps of a block wait
// for one another only after the first step and at the end.  The vectors' values
// become (value, token) keys once, at the piece's end, against its last bound; a
// row of many equal values or an ascending one overflows the store and is taken
// again step by step, and then the list of keys is sorted and cut to its n best as
// it grows.
// The cluster's first block merges the pieces' (max, sum) in piece order and
// gathers, through distributed shared memory, their keys that reach the largest
// of the pieces' bounds, sorts those (each thread counts the keys above its own)
// and draws.
// Bound by HBM while the logits stream (256 fp32 rows of 128256: 22 us, 6.0 TB/s), then
// by the latency of a row's chain (keys, gather, sort, draw: 9 us).  In a queue of
// calls those rows take 37.2 us with n = 64 (3.5 TB/s), 2048 bf16 rows of 32768 with n
// = 8 38.9 us (3.4 TB/s), 300 bf16 rows of 50001 with n = 20 22 to 25 us.  With a barrier
// of the block in every step the first two were 43 and 41 us.
#include <cmath>
#include <cstdint>

#include "answer.h"
#include "ptx.cuh"
#include "rowstats.cuh"

namespace lmho {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;    // keys of a candidate list
constexpr int kMaxPieces = 16;  // of a cluster
constexpr int kUnroll = 4;                // vectors per thread and step
constexpr int kFull = 512;                // set-aside vectors at which they become keys
constexpr int kStore = kFull + kThreads * kUnroll;  // room for one more step's

// Order of candidates: larger value first, then the lower token.  One 64-bit
// key sorts both: the value's bits made monotone in the high half, the token
// complemented in the low half.  0 is below every key.
__device__ __forceinline__ uint32_t mono_of(float z) {
  z = z == 0.f ? 0.f : z;  // -0 and +0 are one value
  const uint32_t b = __float_as_uint(z);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float z, uint32_t v) {
  return (static_cast<uint64_t>(mono_of(z)) << 32) | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float value_of_mono(uint32_t m) {
  return __uint_as_float((m & 0x80000000u) ? (m & 0x7FFFFFFFu) : ~m);
}
__device__ __forceinline__ float value_of(uint64_t key) { return value_of_mono(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int64_t token_of(uint64_t key) {
  return static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}
constexpr uint32_t kMonoNegInf = 0x007FFFFFu;                                       // mono_of(-inf)
constexpr uint64_t kLowestKey = static_cast<uint64_t>(kMonoNegInf + 1) << 32;       // above every -inf

// Fold of a thread's U vectors, whose maximum is vm, into (m, s).  The difference z - m is
// taken first and then scaled: its two roundings are relative to it, so a term's error
// does not grow with the logits, and the maximum's own term is 1.  (2^(z log2 e - m log2 e)
// in one multiply-add would leave the rounding of m log2 e in every exponent, half an ulp
// of 1.44 m: 8e-7 at 31, nats from 1e8 on, and a sum out of range from 1e10 on.)
template <typename E, int U>
__device__ __forceinline__ void fold(MS& a, const uint4 (&r)[U], float vm) {
  constexpr int N = Elt<E>::kPerVec;
  if (vm > a.m) {
    a.s *= ex2_approx((a.m - vm) * kLog2e);
    a.m = vm;
  }
  const float ref = a.m == -INFINITY ? 0.f : a.m;  // nothing but -inf or NaN so far
  const uint64_t ref2 = f32x2(ref, ref), k2 = f32x2(kLog2e, kLog2e);
  uint64_t acc0 = f32x2(a.s, 0.f), acc1 = f32x2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[N];
    Elt<E>::unpack(r[u], v);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float p, q;
      f32x2_split(mul_f32x2(sub_f32x2(f32x2(v[i], v[i + 1]), ref2), k2), p, q);
      acc0 = add_f32x2(acc0, f32x2(ex2_approx(p), ex2_approx(q)));
      f32x2_split(mul_f32x2(sub_f32x2(f32x2(v[i + 2], v[i + 3]), ref2), k2), p, q);
      acc1 = add_f32x2(acc1, f32x2(ex2_approx(p), ex2_approx(q)));
    }
  }
  float lo, hi;
  f32x2_split(add_f32x2(acc0, acc1), lo, hi);
  a.s = lo + hi;
}

// A row seen as 16-byte vectors on the 16-byte grid: vector q holds the elements
// q N - off .. q N - off + N - 1, those outside the row read as -inf.
template <typename E>
struct RowVecs {
  const E* row;
  const E* grid;
  int64_t V;
  int off;
  __device__ RowVecs(const E* r, int64_t V_) : row(r), V(V_) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(E));
    grid = r - off;
  }
  __device__ int64_t count() const { return (off + V + Elt<E>::kPerVec - 1) / Elt<E>::kPerVec; }
  __device__ uint4 load(int64_t q, int64_t end) const {
    constexpr int N = Elt<E>::kPerVec;
    const int64_t e0 = q * N - off;
    if (q < end && e0 >= 0 && e0 + N <= V) return ldg_stream_v4(grid + q * N);
    uint4 r = neg_inf_vec<E>();
    if (q < end) {
      E* w = reinterpret_cast<E*>(&r);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i >= 0 && e0 + i < V) w[i] = row[e0 + i];
    }
    return r;
  }
};

// Maximum of a vector's values (NaN passed over).
template <typename E> __device__ __forceinline__ float vec_max(const uint4& r);
template <> __device__ __forceinline__ float vec_max<float>(const uint4& r) {
  return fmaxf(max3_f32(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z)), __uint_as_float(r.w));
}
template <> __device__ __forceinline__ float vec_max<uint16_t>(const uint4& r) {
  const uint32_t m = max_bf16x2(max_bf16x2(r.x, r.y), max_bf16x2(r.z, r.w));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}

struct List {
  uint64_t keys[kCap];
  uint64_t thr;     // candidates are the keys >= thr
  int count;
};
struct Shared {
  union {
    struct {
      uint4 vec[kStore];       // vectors set aside, and
      uint32_t at[kStore];     // their index in the row
    } store;
    List all;                  // first block, at the end: the row's keys
  };
  List mine;                   // this piece's keys
  uint64_t sorted[kThreads];
  uint32_t bound[kWarps];
  uint32_t thr_max;
  int stored;
  float wm[kWarps], ws[kWarps];
  float m, s;                            // this piece's
  float pm[kMaxPieces], ps[kMaxPieces];  // first block: every piece's
  uint64_t pthr[kMaxPieces];
  int upto[kMaxPieces];                  // their counts, summed
};

// Sort the list's keys (<= kCap), largest first, leave the n best and raise the bound.
__device__ __noinline__ void compact(List& l, int n) {
  const int c = l.count;
  int size = 32;
  while (size < c) size <<= 1;
  for (int i = c + threadIdx.x; i < size; i += kThreads) l.keys[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
        const uint64_t a = l.keys[lo], b = l.keys[hi];
        if ((a < b) == ((lo & k) == 0)) {
          l.keys[lo] = b;
          l.keys[hi] = a;
        }
      }
      __syncthreads();
    }
  if (threadIdx.x == 0) {
    l.count = c < n ? c : n;
    if (c >= n && l.keys[n - 1] > l.thr) l.thr = l.keys[n - 1];
  }
  __syncthreads();
}

// The k-th largest of the warp's `mine` values (k <= 32).
__device__ __forceinline__ uint32_t warp_kth(uint32_t mine, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;
  for (int i = 0; i < k; ++i) {
    top = __reduce_max_sync(0xFFFFFFFFu, mine);
    if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, mine == top)) - 1) mine = 0;
  }
  return top;
}

__device__ __forceinline__ void append(List& l, uint64_t key, bool want) {
  if (!want) return;
  const int at = atomicAdd(&l.count, 1);
  if (at < kCap) l.keys[at] = key;
}

// The set-aside vectors' values that reach the list's bound become keys; the
// store is empty afterwards.  Every thread of the block, at a point where the
// store is complete.  More keys than the list holds (many equal values, mostly):
// again with the list cut to its n best as it fills.
template <typename E>
__device__ __noinline__ void drain(Shared& sh, int off, int n) {
  constexpr int N = Elt<E>::kPerVec;
  List& l = sh.mine;
  const int total = sh.stored * N, before = l.count;
  const auto key_at = [&](int i) -> uint64_t {
    if (i >= total) return 0;
    const float z = Elt<E>::load_any(reinterpret_cast<const E*>(sh.store.vec) + i);
    return z == z ? key_of(z, static_cast<uint32_t>(static_cast<int64_t>(sh.store.at[i / N]) * N - off + i % N)) : 0;
  };
  __syncthreads();
  const uint64_t thr = l.thr;
  for (int base = 0; base < total; base += kThreads) {
    const uint64_t key = key_at(base + threadIdx.x);
    append(l, key, key >= thr);
  }
  __syncthreads();
  const bool over = l.count > kCap;
  __syncthreads();
  if (over) {
    if (threadIdx.x == 0) l.count = before;
    __syncthreads();
    for (int base = 0; base < total; base += kThreads) {
      if (l.count > kCap - kThreads) compact(l, n);
      __syncthreads();
      const uint64_t key = key_at(base + threadIdx.x);
      append(l, key, key >= l.thr);
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) sh.stored = 0;
  __syncthreads();
}

// The list's n best, largest first, 0 past the last.  Short lists are sorted by
// counting the larger keys.  A longer one is cut by a bound on the n-th best first,
// as in the stream: the least of the warps' k-th largest, which leaves more than
// 256 only where values are equal.  `spare` is another list, not in use.  (48 rows of
// 128256, n = 64, take 23 us; 39 with the network sort for lists of 257 to 1024.)
__device__ __forceinline__ const uint64_t* sort_best(Shared& sh, List& l, List& spare, int n) {
  const List* from = &l;
  if (l.count > kThreads) {
    const int c = l.count, warp = threadIdx.x >> 5;
    uint32_t mine = 0;
    for (int i = threadIdx.x; i < c; i += kThreads) mine = max(mine, static_cast<uint32_t>(l.keys[i] >> 32));
    const uint32_t kth = warp_kth(mine, (n + kWarps - 1) / kWarps);
    if ((threadIdx.x & 31) == 0) sh.bound[warp] = kth;
    if (threadIdx.x == 0) spare.count = 0;
    __syncthreads();
    uint32_t least = sh.bound[0];
    for (int w = 1; w < kWarps; ++w) least = min(least, sh.bound[w]);
    for (int i = threadIdx.x; i < c; i += kThreads) append(spare, l.keys[i], static_cast<uint32_t>(l.keys[i] >> 32) >= least);
    __syncthreads();
    if (spare.count > kThreads) {
      compact(l, n);
      for (int i = l.count + threadIdx.x; i < n; i += kThreads) l.keys[i] = 0;
      __syncthreads();
      return l.keys;
    }
    from = &spare;
  }
  const int c = from->count;
  if (threadIdx.x < kChooseMax) sh.sorted[threadIdx.x] = 0;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < c) {
    const uint64_t mine = from->keys[threadIdx.x];
    int rank = 0;
    for (int i = 0; i < c; ++i) rank += from->keys[i] > mine;
    sh.sorted[rank] = mine;
  }
  __syncthreads();
  return sh.sorted;
}

// Reads of another block's shared memory (cluster addresses).
__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_dsmem_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The outputs of row t, by one warp: keys[0..n) sorted, 0 where there is none.
// Lane l takes the ranks 4 l .. 4 l + 3.
__device__ void choose_row(const uint64_t* keys, const ChooseArgs& a, int64_t t, MS st) {
  constexpr int P = kChooseMax / 32;
  const int lane = threadIdx.x & 31, n = a.n;
  const bool bad = !(st.s < INFINITY);  // NaN or +inf in the row
  const float log_sum = logf(st.s);
  const float fill = bad ? __int_as_float(0x7FC00000) : -INFINITY;
  int kept = n;
  if (a.top_k) {
    const int64_t k = a.top_k[t];
    if (k > 0 && k < n) kept = static_cast<int>(k);
  }
  float z[P], w[P], noise[P];
  bool there[P];
  int64_t tok[P];
  const float top = value_of(keys[0]);
  float mass = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int j = lane * P + i;
    const uint64_t key = j < n ? keys[j] : 0;
    there[i] = !bad && key != 0;
    z[i] = there[i] ? value_of(key) : -INFINITY;
    tok[i] = there[i] ? token_of(key) : -1;
    noise[i] = (a.noise && j < n) ? a.noise[t * n + j] : 0.f;
    w[i] = there[i] && j < kept ? expf(z[i] - top) : 0.f;
    mass += w[i];
    if (j < n) {
      a.best[t * n + j] = tok[i];
      a.best_logprob[t * n + j] = there[i] ? (z[i] - st.m) - log_sum : fill;
    }
  }
  float upto = mass;  // inclusive prefix over the lanes
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
    if (lane >= off) upto += o;
  }
  const float total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  const float p = a.top_p ? a.top_p[t] : 1.f;
  const float limit = p * total;
  float before = upto - mass;
  float score = -INFINITY;
  int pick = n;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int j = lane * P + i;
    if (there[i] && j < kept && (j == 0 || p >= 1.f || before < limit)) {
      const float sc = a.noise ? z[i] + noise[i] : z[i];
      if (pick == n || sc > score) {
        score = sc;
        pick = j;
      }
    }
    before += w[i];
  }
  // the best score, ties by the lowest rank
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const float os = __shfl_xor_sync(0xFFFFFFFFu, score, off);
    const int op = __shfl_xor_sync(0xFFFFFFFFu, pick, off);
    if (op < n && (pick == n || os > score || (os == score && op < pick))) {
      score = os;
      pick = op;
    }
  }
  if (lane == 0) {
    a.token[t] = pick < n ? token_of(keys[pick]) : -1;
    a.logprob[t] = pick < n ? (value_of(keys[pick]) - st.m) - log_sum : fill;
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 4) choose_rows(const E* __restrict__ logits, const ChooseArgs a,
                                                           int S, int64_t piece) {
  constexpr int N = Elt<E>::kPerVec;
  constexpr int U = kUnroll;
  __shared__ Shared sh;
  const int64_t t = blockIdx.x / S;
  const int s = static_cast<int>(blockIdx.x - t * S);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RowVecs<E> row(logits + t * a.V, a.V);
  const int64_t q0 = s * piece;
  const int64_t q1 = q0 + piece < row.count() ? q0 + piece : row.count();
  List& l = sh.mine;
  if (threadIdx.x == 0) {
    l.count = 0;
    l.thr = kLowestKey;
    sh.stored = 0;
  }
  __syncthreads();
  MS st = ms_empty();
  uint64_t thr = kLowestKey;
  // warps that surely have a vector in every lane bound the n best
  const int warps = q1 - q0 >= kThreads ? kWarps : static_cast<int>((q1 - q0) / 32);
  const int k = warps > 0 ? (a.n + warps - 1) / warps : kThreads;
  const int64_t whole0 = row.off > 0, whole1 = (row.off + a.V) / N;
  auto load_step = [&](int64_t q, uint4(&r)[U]) {
    if (q >= whole0 && q + kThreads * U <= (q1 < whole1 ? q1 : whole1)) {  // whole vectors of the piece
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ldg_stream_v4(row.grid + (q + u * kThreads + threadIdx.x) * N);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = row.load(q + u * kThreads + threadIdx.x, q1);
    }
  };
  // Sets aside the step's vectors that reach the bound; the places past the store are
  // lost (and counted).
  auto keep = [&](int64_t q, const uint4(&r)[U], const float(&vm)[U]) {
    const float thr_z = value_of(thr);
    bool full = false;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (vm[u] >= thr_z) {
        const int at = atomicAdd(&sh.stored, 1);
        if (at < kStore) {
          sh.store.vec[at] = r[u];
          sh.store.at[at] = static_cast<uint32_t>(q + u * kThreads + threadIdx.x);
        }
        full |= at >= kFull;
      }
    return full;
  };
  int step = 0;
  uint4 next[U];
  if (q0 < q1) load_step(q0, next);
  for (int64_t q = q0; q < q1; q += kThreads * U) {
    uint4 r[U];
    float vm[U], tm = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = next[u];
    if (q + kThreads * U < q1) load_step(q + kThreads * U, next);  // in flight while this step is worked on
#pragma unroll
    for (int u = 0; u < U; ++u) {
      vm[u] = vec_max<E>(r[u]);
      tm = fmaxf(tm, vm[u]);
    }
    fold<E, U>(st, r, tm);
    ++step;
    if ((step & (step - 1)) == 0 && k <= 32) {
      // A warp's value only ever says that k of its logits reach it, so whichever of
      // the others' values is seen here will do; the first step waits for all of them.
      const uint32_t kth = warp_kth(mono_of(st.m), k);
      if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&sh.bound[warp]) = kth;
      if (step == 1) __syncthreads();
      uint32_t least = *reinterpret_cast<volatile uint32_t*>(&sh.bound[0]);
      for (int w = 1; w < warps; ++w) least = min(least, *reinterpret_cast<volatile uint32_t*>(&sh.bound[w]));
      const uint64_t b = static_cast<uint64_t>(least) << 32;
      thr = b > thr ? b : thr;
    }
    keep(q, r, vm);
  }
  if (threadIdx.x == 0) sh.thr_max = 0;
  __syncthreads();
  // the warps' bounds differ by what each has seen of the others: the largest holds
  if (lane == 0) atomicMax(&sh.thr_max, static_cast<uint32_t>(thr >> 32));
  __syncthreads();
  thr = static_cast<uint64_t>(sh.thr_max) << 32;
  if (threadIdx.x == 0) l.thr = thr;
  if (sh.stored > kStore) {
    // Many equal values, or an ascending row: once more from memory, step by step, the
    // store made into keys whenever it fills.
    __syncthreads();
    if (threadIdx.x == 0) sh.stored = 0;
    __syncthreads();
    for (int64_t q = q0; q < q1; q += kThreads * U) {
      uint4 r[U];
      float vm[U];
      load_step(q, r);
#pragma unroll
      for (int u = 0; u < U; ++u) vm[u] = vec_max<E>(r[u]);
      if (__syncthreads_or(keep(q, r, vm))) {
        drain<E>(sh, row.off, a.n);
        thr = l.thr;
      }
    }
  }
  __syncthreads();
  drain<E>(sh, row.off, a.n);
  st = ms_warp_allreduce(st);
  if (lane == 0) {
    sh.wm[warp] = st.m;
    sh.ws[warp] = st.s;
  }
  __syncthreads();
  st = MS{sh.wm[0], sh.ws[0]};
#pragma unroll
  for (int w = 1; w < kWarps; ++w) st = ms_merge(st, MS{sh.wm[w], sh.ws[w]});

  if (S == 1) {
    const uint64_t* keys = sort_best(sh, l, sh.all, a.n);
    if (warp == 0) choose_row(keys, a, t, st);
    return;
  }
  if (threadIdx.x == 0) {
    sh.m = st.m;
    sh.s = st.s;
  }
  cluster_sync();  // every piece's list is complete
  if (s == 0) {
    List& all = sh.all;
    if (warp == 0) {
      int c = 0;
      if (lane < S) {
        sh.pm[lane] = ld_dsmem_f32(mapa_shared(&sh.m, lane));
        sh.ps[lane] = ld_dsmem_f32(mapa_shared(&sh.s, lane));
        sh.pthr[lane] = ld_dsmem_u64(mapa_shared(&l.thr, lane));
        c = ld_dsmem_s32(mapa_shared(&l.count, lane));
      }
#pragma unroll
      for (int off = 1; off < kMaxPieces; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, c, off);
        if (lane >= off) c += o;
      }
      if (lane < S) sh.upto[lane] = c;
      if (lane == 0) all.count = 0;
    }
    __syncthreads();
    st = ms_empty();
    uint64_t thr = 0;
    for (int p = 0; p < S; ++p) {
      st = ms_merge(st, MS{sh.pm[p], sh.ps[p]});
      thr = sh.pthr[p] > thr ? sh.pthr[p] : thr;
    }
    if (threadIdx.x == 0) all.thr = thr;
    for (int base = 0, p = 0; base < sh.upto[S - 1]; base += kThreads) {
      const int i = base + threadIdx.x;
      uint64_t key = 0;
      if (i < sh.upto[S - 1]) {
        while (i >= sh.upto[p]) ++p;
        key = ld_dsmem_u64(mapa_shared(&l.keys[p ? i - sh.upto[p - 1] : i], p));
      }
      append(all, key, key >= thr);
    }
    __syncthreads();
    const bool over = all.count > kCap;
    __syncthreads();
    if (over) {  // many equal values: 256 at a time
      if (threadIdx.x == 0) all.count = 0;
      __syncthreads();
      for (int base = 0, p = 0; base < sh.upto[S - 1]; base += kThreads) {
        const int i = base + threadIdx.x;
        uint64_t key = 0;
        if (i < sh.upto[S - 1]) {
          while (i >= sh.upto[p]) ++p;
          key = ld_dsmem_u64(mapa_shared(&l.keys[p ? i - sh.upto[p - 1] : i], p));
        }
        append(all, key, key >= all.thr);
        __syncthreads();
        if (all.count > kCap - kThreads) compact(all, a.n);
        __syncthreads();
      }
    }
  }
  cluster_sync();  // the lists have been read
  if (s == 0) {
    const uint64_t* keys = sort_best(sh, sh.all, l, a.n);
    if (warp == 0) choose_row(keys, a, t, st);
  }
}

struct Cut {
  int S;
  int64_t piece;  // vectors
};
// Pieces of a row (a power of two, each of at least one step, a multiple of the
// block's width): about kWant blocks in all, two for every SM.  Rows of 128256 with n = 64
// take 38.3 us at 300 rows in two pieces each, 38.5 at 303, and 38.4 at 304 in one; 36.8
// at 256, 43.8 at 400, 56.0 at 607.
constexpr int64_t kWant = 304;
Cut cut_rows(int64_t T, int64_t V, int per_vec) {
  const int64_t vecs = (V + per_vec - 1) / per_vec + 1;
  int64_t S = 1;
  while (S < kMaxPieces && 2 * S * kThreads * kUnroll <= vecs && T * S < kWant) S *= 2;
  const int64_t each = (vecs + S - 1) / S;
  return Cut{static_cast<int>(S), (each + kThreads - 1) / kThreads * kThreads};
}

template <typename E>
cudaError_t launch(const E* logits, const ChooseArgs& a, cudaStream_t st) {
  const Cut c = cut_rows(a.T, a.V, Elt<E>::kPerVec);
  static std::atomic<bool> wide[kMaxDevices];  // clusters of 16 allowed on the device
  if (c.S > 8) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= kMaxDevices || !wide[dev].load(std::memory_order_acquire)) {
      if (cudaError_t e = cudaFuncSetAttribute(choose_rows<E>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))
        return e;
      if (dev < kMaxDevices) wide[dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T * c.S));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(c.S);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  launch_mark(0, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, choose_rows<E>, logits, a, c.S, c.piece);
  launch_mark(1, st);
  return e;
}

}  // namespace

cudaError_t launch_logits_choose_f32(const float* logits, const ChooseArgs& a, cudaStream_t st) {
  return launch(logits, a, st);
}
cudaError_t launch_logits_choose_bf16(const uint16_t* logits, const ChooseArgs& a, cudaStream_t st) {
  return launch(logits, a, st);
}

}  // namespace lmho
