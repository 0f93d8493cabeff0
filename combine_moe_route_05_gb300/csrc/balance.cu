// The router's balance loss with per-expert counts, and its gradient (sm_103a).
//
// For sequence s of n_s tokens, c_se its entries of expert e and P_se the sum
// over its tokens of p_te (softmax, or sigmoid divided by the row's sum):
//   loss = coef / S' * sum_s E / (K n_s^2) * sum_e c_se P_se,
// S' the sequences that are not empty.  With the counts constant,
//   dloss/dl_tj = coef / S' * E / (K n_s^2) * q_tj (c_sj - sum_e c_se p_te),
// q = p for softmax, sigma (1 - sigma) / sum(sigma) for sigmoid.  Since p sums
// to 1, a constant can be taken off the counts: the backward takes about
// their mean off as an integer, exactly, so that the gradient of an even router is made of
// small differences, not of near-equal sums of counts.
//
// Forward: tokens are cut into equal tiles, one block each.  A tile's part of a
// sequence is a fragment.  A sequence inside one tile is finished there; the
// fragments of one that spans tiles go to slots (two a tile suffice: one for
// the fragment that began in an earlier tile, one for that which goes on into
// the next), and a second kernel, one cluster, adds them up and the loss with
// them.  Every sum has a fixed order (counts are integers), so repeated calls
// give the same bits.
//
// Both passes read the logits once and are bound by HBM at the largest sizes, below
// some 20 MB by the chain of dependent loads around that: offsets, logits, slots.  So
// logits come into L2 before the offsets are known, offsets are read by all threads
// at once and searched in shared memory, and a tile's fragments are worked on
// together.
//
// us (replayed in a graph, logits from HBM; floor: the bytes at the copy rate): 131072
// tokens x 512 experts 51.6 (40.8), the DeepSeek-V3 shape (16384 x 256, sigmoid) packed
// in 9 sequences 13.3 (2.4): 1.2 offsets, 4.7 tiles, 1.5 their sums, 0.5 the hand-over to
// the second kernel, 4 that one.  Backward of the latter, added to another gradient, 11.6
// (6.9), of 8192 x 128 3.7 (1.3).
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 32;       // of a tile's block: one an SM
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTiles = 160;
constexpr int kFrags = 16;       // fragments that a tile works on at a time
constexpr int kRows = kWarps + kFrags - 1;  // rows of sums: warp w's of fragment f is w + f
constexpr int kBwdWarps = 8;     // of a block of the backward
constexpr int kOffBatch = 2048;  // sequences whose offsets are kept in shared memory
constexpr int kJoinWarps = 32;   // of a block of the second kernel
constexpr int kCluster = 8;      // blocks of the second kernel
constexpr int kShare = kMaxTiles / kJoinWarps;  // tiles of one of its warps
constexpr int kJoinRows = kJoinWarps + kMaxTiles;
// Tokens a team sums in registers before it adds them to shared memory.  A sum then
// has 64 + T / (64 * warps of the grid * teams of a warp) + 70 fp32 additions in a row:
// 135 for 131072 tokens of 512 experts, under 1100 for any logits that fit into 284 GB.
constexpr int kFlush = 64;
constexpr float kInf = __builtin_huge_valf();

struct BalArgs {
  const float* logits;   // [T, E]
  const int32_t* idx;    // [T, K] (forward)
  const int32_t* off;    // [S + 1] or NULL: one sequence, all T tokens
  int T, E, K, S;
  int tile, tiles;       // tokens of a tile, tiles
  int stride;            // of a slot: E rounded up to 4
  int vec;               // rows can be read 16 bytes at a time
  float coef;
  uint32_t* flags;
  // forward
  int32_t* cnt;          // [S, E]
  float* prob;           // [S, E] or NULL
  float* loss;           // [1]
  float* slot_p;         // [2 * tiles, stride]
  int32_t* slot_c;       // [2 * tiles, stride]
  float* tile_loss;      // [tiles] of the sequences inside a tile
  int4* spans;           // [tiles] {a fragment that began earlier, the sequence that begins
                         // here and goes on or -1, its length, its last tile}
  int32_t* full;         // [1] sequences that are not empty
  // backward
  const int32_t* bcnt;   // [S, E]
  const float* gloss;    // [1] or NULL: 1
  const float* base;     // [T, E] or NULL
  float* glogits;        // [T, E]
};

// Tokens of sequence s, kept inside [0, T] whatever the offsets hold.
__device__ __forceinline__ int2 range_of(int lo, int hi, int T) {
  lo = min(max(lo, 0), T);
  return make_int2(lo, min(max(hi, lo), T));
}
__device__ __forceinline__ int2 seq_range(const BalArgs& a, int s) {
  return a.off ? range_of(__ldg(a.off + s), __ldg(a.off + s + 1), a.T) : make_int2(0, a.T);
}

template <int LPT>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int LPT>
__device__ __forceinline__ float team_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Column of value i of lane `tl` of a team of LPT lanes: four in a row a lane.
template <int LPT>
__device__ __forceinline__ int col_of(int tl, int i) {
  return (i >> 2) * (4 * LPT) + tl * 4 + (i & 3);
}

template <int LPT, int NV, typename T4, typename T1>
__device__ __forceinline__ void load_row(const T1* row, int E, bool vec, bool live, int tl, T1 fill,
                                         T1 (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of<LPT>(tl, 4 * j);
    if (vec) {
      T4 x{fill, fill, fill, fill};
      if (live && c < E) x = __ldg(reinterpret_cast<const T4*>(row + c));
      v[4 * j] = x.x;
      v[4 * j + 1] = x.y;
      v[4 * j + 2] = x.z;
      v[4 * j + 3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = live && c + i < E ? __ldg(row + c + i) : fill;
    }
  }
}

// As load_row, of a gradient that may be written over in place.
template <int LPT, int NV>
__device__ __forceinline__ void load_base(const float* row, int E, bool vec, bool live, int tl,
                                          float (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of<LPT>(tl, 4 * j);
    if (vec) {
      float4 x{0.0f, 0.0f, 0.0f, 0.0f};
      if (live && c < E) x = *reinterpret_cast<const float4*>(row + c);
      v[4 * j] = x.x;
      v[4 * j + 1] = x.y;
      v[4 * j + 2] = x.z;
      v[4 * j + 3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = live && c + i < E ? row[c + i] : 0.0f;
    }
  }
}

// e^x, 0 below 2^-126: the fast exponential without its subnormal results.
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
// 1 / x to 1 ulp, 0 above 2^126.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^(v - the team's largest) in place of v, and their sum.
template <int LPT, int N>
__device__ __forceinline__ float exponentials(float (&v)[N], bool& infinite) {
  float m = -kInf;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);  // a NaN is not taken, but comes up in the sum
  m = team_max<LPT>(m);
  infinite = m == kInf;
  const float sub = m > -kInf ? m : 0.0f;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = exp_fast(v[i] - sub);
    z += v[i];
  }
  return team_sum<LPT>(z);
}

// Turns a team's logits v into v = p * z and, for the backward of sigmoids, q =
// (see the top) * z, and returns 1 / z.  A logit of -inf is an expert that is
// masked out: p = q = 0.  A row without any other is 0, and so is one with a NaN
// or +inf, which returns `bad`.  exp is the fast one: its error, 2 + 1.2 |x| ulp, falls
// for the softmax on values that are e^x of the row's largest.  `again` loads v
// once more, for a row (`live`) whose sigmoids are all far below 1: those are e^l
// to 1e-9, and normalised from the row's largest they cannot vanish together.
template <int LPT, int NV, bool SIGMOID, bool GRAD, typename F>
__device__ __forceinline__ float probabilities(float (&v)[4 * NV], float (&q)[4 * NV], bool live,
                                               bool& bad, F&& again) {
  constexpr int N = 4 * NV;
  float z = 0.0f;
  if (!SIGMOID) {
    z = exponentials<LPT>(v, bad);
  } else {
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m = fmaxf(m, v[i]);
      const float e = exp_fast(-v[i]), s = reciprocal(1.0f + e);
      if (GRAD) q[i] = s * fminf(e * s, 1.0f);  // 1 - s = e s; 1 where e is infinite (inf * 0)
      v[i] = s;
      z += s;
    }
    z = team_sum<LPT>(z);
    const unsigned votes = __ballot_sync(kFull, m == kInf);
    const int first = (threadIdx.x & 31) / LPT * LPT;
    bad = (votes >> first) & (LPT == 32 ? kFull : (1u << (LPT & 31)) - 1u);
    const bool small = live && z < 1e-9f;
    if (__any_sync(kFull, small)) {
      float w[N];
      bool none;
      again(w);
      const float zw = exponentials<LPT>(w, none);
      if (small) {
        z = zw;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v[i] = w[i];
          if (GRAD) q[i] = w[i];
        }
      }
    }
  }
  bad |= !(z < kInf);
  if (bad) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
      if (GRAD && SIGMOID) q[i] = 0.0f;
    }
  }
  return z > 0.0f && !bad ? 1.0f / z : 0.0f;
}

// Sum over the block's threads, the same in each; `red` holds 32 values.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  return v;
}

// Factor of a sequence of n tokens.
__device__ __forceinline__ float seq_factor(const BalArgs& a, int n) {
  return static_cast<float>(a.E) / (static_cast<float>(a.K) * n) / n;
}

// Sequences of the table that are not empty, and before whose end token t lies (the
// index of the first that ends behind it), by the whole block.  Each offset is
// read once; those of a table of at most kOffBatch sequences stay in `soff`.
struct Table {
  int full, first;
  bool wrong;
};
__device__ __forceinline__ Table read_table(const BalArgs& a, int t, int* soff, int* red) {
  if (!a.off) {
    if (threadIdx.x < 2) soff[threadIdx.x] = threadIdx.x ? a.T : 0;
    __syncthreads();
    return Table{a.T > 0, t < a.T ? 0 : 1, false};
  }
  int full = 0, first = 0, wrong = 0;
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const int lo = __ldg(a.off + s), hi = __ldg(a.off + s + 1);
    const int2 r = range_of(lo, hi, a.T);
    full += r.y > r.x;
    first += hi <= t;
    wrong |= lo < 0 || hi < lo || hi > a.T;
    if (a.S <= kOffBatch) {
      soff[s] = lo;
      if (s == a.S - 1) soff[a.S] = hi;
    }
  }
  full = __reduce_add_sync(kFull, full);
  first = __reduce_add_sync(kFull, first);
  wrong = __reduce_or_sync(kFull, wrong);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    red[warp] = full;
    red[32 + warp] = first;
    red[64 + warp] = wrong;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const bool mine = lane < static_cast<int>(blockDim.x >> 5);
  full = __reduce_add_sync(kFull, mine ? red[lane] : 0);
  first = __reduce_add_sync(kFull, mine ? red[32 + lane] : 0);
  wrong = __reduce_or_sync(kFull, mine ? red[64 + lane] : 0);
  __syncthreads();
  return Table{full, first, wrong != 0};
}

constexpr int64_t kAhead = 128 * 1024;
// Pulls the n bytes from p on into L2, but for what the ends share a 16-byte line
// with: a hint that nothing waits for.
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t n) {
  const uint64_t from = (reinterpret_cast<uint64_t>(p) + 15) & ~uint64_t{15};
  const uint64_t to = (reinterpret_cast<uint64_t>(p) + n) & ~uint64_t{15};
  if (to > from)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from),
                 "r"(static_cast<uint32_t>(to - from))
                 : "memory");
}

// Tokens of a team whose logits it loads before it works on the first of them.
template <int NV>
constexpr int kBatch = NV < 3 ? 4 / NV : 1;

// Counts a token's entries; the later repeats of an expert are dropped.
__device__ __forceinline__ void count_token(const BalArgs& a, unsigned t, int* hist) {
  const int32_t* from = a.idx + static_cast<size_t>(t) * a.K;
  int seen[MOE_MAX_TOPK];
#pragma unroll
  for (int k = 0; k < MOE_MAX_TOPK; ++k) seen[k] = k < a.K ? __ldg(from + k) : -1;
#pragma unroll
  for (int k = 0; k < MOE_MAX_TOPK; ++k) {
    if (k >= a.K) break;
    const int e = seen[k];
    if (e == -1) continue;
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(a.E)) {
      raise_flag(a.flags, MOE_DEVERR_BAD_EXPERT);
      continue;
    }
    bool again = false;
#pragma unroll
    for (int b = 0; b < k; ++b) again |= seen[b] == e;
    if (again) raise_flag(a.flags, MOE_DEVERR_DUP_EXPERT);
    else atomicAdd(hist + e, 1);
  }
}

// Fragments of a tile that are worked on together, in the order of their tokens.
struct Fragments {
  int n;                 // how many
  int seq[kFrags], begin[kFrags], end[kFrags];
  int length[kFrags];    // of the sequence
  int kind[kFrags];      // 0: the whole sequence; 1: it began in an earlier tile; 2: it goes on
  int next_seq, next_token;
  int last_tile;         // of the last one's sequence
};

// Finds the next fragments of tokens [cursor, t1), from sequence s on, by one warp.
// Sequences that overlap (no table) are cut, so that tokens always rise.
__device__ __forceinline__ void find_fragments(const BalArgs& a, const int* soff, int s, int cursor,
                                               int t0, int t1, Fragments* f) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  bool more = true;
  while (more && n < kFrags && s < a.S) {
    const int mine = s + lane;
    int2 r = make_int2(t1, t1);
    if (mine < a.S)
      r = a.S <= kOffBatch ? range_of(soff[mine], soff[mine + 1], a.T) : seq_range(a, mine);
    unsigned some = __ballot_sync(kFull, r.y > r.x && r.x < t1 && r.y > cursor);
    more = __all_sync(kFull, r.x < t1);
    int done = 32;
    while (some != 0 && n < kFrags) {
      const int k = __ffs(some) - 1;
      some &= some - 1;
      const int lo = __shfl_sync(kFull, r.x, k), hi = __shfl_sync(kFull, r.y, k);
      const int begin = max(lo, cursor), end = min(hi, t1);
      if (begin >= end) continue;
      if (lane == 0) {
        f->seq[n] = s + k;
        f->begin[n] = begin;
        f->end[n] = end;
        f->length[n] = hi - lo;
        f->kind[n] = lo < t0 ? 1 : hi > t1 ? 2 : 0;
        f->last_tile = (hi - 1) / a.tile;
      }
      cursor = end;
      if (++n == kFrags) done = k + 1;
    }
    s += done;
  }
  if (lane == 0) {
    f->n = n;
    f->next_seq = n == kFrags ? s : a.S;
    f->next_token = cursor;
  }
}

// A tile: sums of p and counts of its tokens [t0, t1) of each sequence.  Each warp
// takes tokens in a row, so that it meets few sequences, and a block's fragments
// are worked on together: one after the other they would cost some 3 us each.
template <int LPT, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 1) balance_tile_kernel(BalArgs a) {
  // the tile's first logits and routes come into L2 while the kernel in front
  // ends and the offsets are read
  if (threadIdx.x == 0) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int64_t n = min(static_cast<int64_t>(a.tile), static_cast<int64_t>(a.T) - t);
    if (n > 0) {
      prefetch_l2(a.logits + t * a.E, min(n * a.E * 4, kAhead));
      prefetch_l2(a.idx + t * a.K, min(n * a.K * 4, kAhead));
    }
  }
  grid_dependency_wait();
  constexpr int N = 4 * NV, TPW = 32 / LPT, U = kBatch<NV>;
  extern __shared__ float dyn[];
  float* stage = dyn;                                     // [kRows][E]
  int* hist = reinterpret_cast<int*>(dyn + kRows * a.E);  // [kFrags][E]
  __shared__ int soff[kOffBatch + 1];
  __shared__ int ired[96];
  __shared__ float red[32];
  __shared__ Fragments frag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LPT, tl = lane % LPT;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * a.tile,
                                      static_cast<int64_t>(a.T)));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(t0) + a.tile, static_cast<int64_t>(a.T)));
  for (int i = threadIdx.x; i < kFrags * a.E; i += kThreads) hist[i] = 0;
  const Table table = read_table(a, t0, soff, ired);
  if (table.full < a.S) {  // empty sequences
    for (int s = blockIdx.x * kWarps + warp; s < a.S; s += gridDim.x * kWarps) {
      const int2 r = seq_range(a, s);
      if (r.y > r.x) continue;
      const size_t row = static_cast<size_t>(s) * a.E;
      for (int e = lane; e < a.E; e += 32) {
        a.cnt[row + e] = 0;
        if (a.prob) a.prob[row + e] = 0.0f;
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && table.wrong) raise_flag(a.flags, MOE_DEVERR_BAD_LAYOUT);
  float loss = 0.0f;  // the thread's part
  int4 span = make_int4(0, -1, 0, 0);
  int next_seq = table.first, next_token = t0;
  while (next_seq < a.S && next_token < t1) {
    if (warp == 0) find_fragments(a, soff, next_seq, next_token, t0, t1, &frag);
    __syncthreads();
    const int nf = frag.n;
    if (nf == 0) break;
    const int f0 = frag.begin[0], f1 = frag.end[nf - 1];
    const int share = ((f1 - f0 - 1) / (kWarps * TPW) + 1) * TPW;  // tokens of a warp
    const int w0 = min(static_cast<int64_t>(f0) + static_cast<int64_t>(warp) * share,
                       static_cast<int64_t>(f1));
    const int w1 = min(static_cast<int64_t>(w0) + share, static_cast<int64_t>(f1));
    // counts: a thread a token
    for (unsigned t = f0 + threadIdx.x; t < static_cast<unsigned>(f1); t += kThreads) {
      int f = 0;
      while (f + 1 < nf && static_cast<int>(t) >= frag.begin[f + 1]) ++f;
      if (static_cast<int>(t) < frag.end[f]) count_token(a, t, hist + f * a.E);
    }
    for (int f = 0; f < nf; ++f) {
      const int x0 = max(w0, frag.begin[f]), x1 = min(w1, frag.end[f]);
      if (x0 >= x1) continue;
      float acc[N], unused[N];
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = 0.0f;
      bool begun = false;
      int held = 0;
      auto flush = [&]() {
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
          for (int o = LPT; o < 32; o <<= 1) acc[k] += __shfl_xor_sync(kFull, acc[k], o);
          const int c = col_of<LPT>(tl, k);
          if (team == 0 && c < a.E) {
            float* to = stage + (warp + f) * a.E + c;
            *to = begun ? *to + acc[k] : acc[k];
          }
          acc[k] = 0.0f;
        }
        begun = true;
        held = 0;
      };
      const unsigned last = x1;
      for (unsigned base = x0; base < last; base += U * TPW) {
        float v[U][N];
        auto load = [&](int u, float (&to)[N]) {
          const unsigned t = base + u * TPW + team;
          const bool live = t < last;
          load_row<LPT, NV, float4>(a.logits + static_cast<size_t>(live ? t : x0) * a.E, a.E, a.vec,
                                    live, tl, -kInf, to);
          return live;
        };
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) live[u] = load(u, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          bool bad;
          const float inv = probabilities<LPT, NV, SIGMOID, false>(
              v[u], unused, live[u], bad, [&](float (&to)[N]) { load(u, to); });
          if (bad && tl == 0) raise_flag(a.flags, MOE_DEVERR_NONFINITE);
#pragma unroll
          for (int k = 0; k < N; ++k) acc[k] = fmaf(v[u][k], inv, acc[k]);
        }
        held += U;
        if (held >= kFlush) flush();
      }
      flush();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nf * a.E; i += kThreads) {
      const int f = nf == 1 ? 0 : i / a.E, e = i - f * a.E;
      const int first = (frag.begin[f] - f0) / share, end = (frag.end[f] - 1 - f0) / share;
      float p = 0.0f;
#pragma unroll 8
      for (int w = first; w <= end; ++w) p += stage[(w + f) * a.E + e];
      const int c = hist[i];
      hist[i] = 0;
      const int kind = frag.kind[f];
      if (kind == 0) {
        const size_t at = static_cast<size_t>(frag.seq[f]) * a.E + e;
        a.cnt[at] = c;
        if (a.prob) a.prob[at] = p / frag.length[f];
        loss = fmaf(static_cast<float>(c) * p, seq_factor(a, frag.length[f]), loss);
      } else {
        const size_t at = static_cast<size_t>(2 * blockIdx.x + kind - 1) * a.stride + e;
        a.slot_p[at] = p;
        a.slot_c[at] = c;
      }
    }
    if (frag.kind[0] == 1) span.x = 1;
    if (frag.kind[nf - 1] == 2)
      span = make_int4(span.x, frag.seq[nf - 1], frag.length[nf - 1], frag.last_tile);
    next_seq = frag.next_seq;
    next_token = frag.next_token;
    __syncthreads();  // stage, hist and frag are taken up again
  }
  if (gridDim.x > 1) {
    // slots without a fragment: the second kernel asks for them as well, and lines
    // that were written lately it finds in L2
    for (int i = threadIdx.x; i < 2 * a.stride; i += kThreads) {
      const bool head = i < a.stride;
      if (head ? span.x == 0 : span.y < 0) {
        const size_t at = static_cast<size_t>(2 * blockIdx.x) * a.stride + i;
        a.slot_p[at] = 0.0f;
        a.slot_c[at] = 0;
      }
    }
  }
  loss = block_sum(loss, red);
  if (threadIdx.x == 0) {
    if (gridDim.x == 1) {  // every sequence is whole: the loss in the same launch
      *a.loss = table.full > 0 ? a.coef * loss / table.full : 0.0f;
    } else {
      a.tile_loss[blockIdx.x] = loss;
      a.spans[blockIdx.x] = span;
      if (blockIdx.x == 0) *a.full = table.full;
    }
  }
}

// Sequences that span tiles: adds up their slots.  Each block of the cluster has 32 C
// experts, C a lane, each warp kShare tiles at most, whose slots it asks for at once
// with what the tiles noted down.  A warp's tiles hold runs of slots of one sequence
// each; sequence f of those that span tiles has its run of warp w in row w + f, as
// both rise with the tokens, and its sum is that of rows in a row.  Block 0 adds up
// the loss.
template <int C>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kJoinWarps * 32)
    balance_join_kernel(BalArgs a) {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  grid_dependency_wait();
  extern __shared__ float dyn[];
  float* ps = dyn;                                                    // [kJoinRows][32 * C]
  int* cs = reinterpret_cast<int*>(dyn + kJoinRows * 32 * C);         // the same
  __shared__ int item_seq[kMaxTiles], item_length[kMaxTiles], item_first[kMaxTiles],
      item_last[kMaxTiles];
  __shared__ float losses[kJoinWarps], block_loss[kCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x;  // in the one cluster
  const int per = (a.tiles + kJoinWarps - 1) / kJoinWarps;
  const int first = warp * per;
  const int col = (rank * 32 + lane) * C;
  // everything is on its way together
  float x[kShare][2][C];
  int y[kShare][2][C];
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    const bool real = i < per && first + i < a.tiles && col < a.E;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const size_t at = static_cast<size_t>(2 * (first + i) + h) * a.stride + col;
      if (C == 2) {  // the row is padded to four
        float2 p{0.0f, 0.0f};
        int2 c{0, 0};
        if (real) {
          p = __ldcg(reinterpret_cast<const float2*>(a.slot_p + at));
          c = __ldcg(reinterpret_cast<const int2*>(a.slot_c + at));
        }
        x[i][h][0] = p.x;
        x[i][h][C - 1] = p.y;
        y[i][h][0] = c.x;
        y[i][h][C - 1] = c.y;
      } else {
        x[i][h][0] = real ? __ldcg(a.slot_p + at) : 0.0f;
        y[i][h][0] = real ? __ldcg(a.slot_c + at) : 0;
      }
    }
  }
  const int full = __ldcg(a.full);
  float loss = rank == 0 && threadIdx.x < a.tiles ? __ldcg(a.tile_loss + threadIdx.x) : 0.0f;
  // sequences that go on from a tile in front of the warp's, and from any
  int f = -1, items = 0;
  int tails[kShare];
#pragma unroll
  for (int i = 0; i < kShare; ++i)
    tails[i] = i * 32 + lane < a.tiles ? __ldcg(&a.spans[i * 32 + lane].y) : -1;
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    items += __popc(__ballot_sync(kFull, tails[i] >= 0));
    f += __popc(__ballot_sync(kFull, tails[i] >= 0 && i * 32 + lane < first));
  }
  float p[C];
  int c[C];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    p[k] = 0.0f;
    c[k] = 0;
  }
  bool some = false;
  auto keep = [&]() {  // the run of sequence f
    if (some && f >= 0)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        ps[(warp + f) * (32 * C) + lane * C + k] = p[k];
        cs[(warp + f) * (32 * C) + lane * C + k] = c[k];
      }
  };
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    if (i >= per || first + i >= a.tiles) break;
    const int4 span = __ldcg(a.spans + first + i);
    if (span.x) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        p[k] += x[i][0][k];
        c[k] += y[i][0][k];
      }
      some = true;
    }
    if (span.y >= 0) {
      keep();
      ++f;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        p[k] = x[i][1][k];
        c[k] = y[i][1][k];
      }
      some = true;
      if (lane == 0) {
        item_seq[f] = span.y;
        item_length[f] = span.z;
        item_first[f] = warp;
        item_last[f] = min(span.w / per, kJoinWarps - 1);
      }
    }
  }
  keep();
  __syncthreads();
  for (int n = warp; n < items; n += kJoinWarps) {
    const int s = item_seq[n], tokens = item_length[n];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      p[k] = 0.0f;
      c[k] = 0;
    }
#pragma unroll 4
    for (int w = item_first[n]; w <= item_last[n]; ++w)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        p[k] += ps[(w + n) * (32 * C) + lane * C + k];
        c[k] += cs[(w + n) * (32 * C) + lane * C + k];
      }
    float val = 0.0f;
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (col + k < a.E && s < a.S) {
        const size_t at = static_cast<size_t>(s) * a.E + col + k;
        a.cnt[at] = c[k];
        if (a.prob) a.prob[at] = p[k] / tokens;
        val = fmaf(static_cast<float>(c[k]), p[k], val);
      }
    loss = fmaf(val, seq_factor(a, tokens), loss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(kFull, loss, o);
  if (lane == 0) losses[warp] = loss;
  __syncthreads();
  if (warp == 0) {
    loss = losses[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(kFull, loss, o);
  }
  // block 0 runs by now
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                 : "=r"(to)
                 : "r"(smem_addr(block_loss + rank)));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(loss) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
  if (rank == 0 && threadIdx.x == 0) {
    loss = 0.0f;
#pragma unroll
    for (int b = 0; b < kCluster; ++b) loss += block_loss[b];
    *a.loss = full > 0 ? a.coef * loss / full : 0.0f;
  }
}

// Blocks of the backward an SM: four but with the widest rows, a token a warp at a
// time.  Two tokens at a time on three blocks took 12.9 against 11.5 us (DeepSeek-V3
// shape, packed) and 4.2 against 3.6 (Qwen3-30B shape).  The 64 registers of four blocks
// (80 of three) are short for sigmoids: 28 bytes spill at 9 to 128 experts, 84 with three
// vectors a lane (257 to 384), where three blocks have not been tried, 96 with four.
template <int NV>
constexpr int kBwdBlocks = NV < 4 ? 4 : 3;

// Backward: a team of lanes a token, a warp's tokens in a row.
template <int LPT, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdBlocks<NV>) balance_bwd_kernel(BalArgs a) {
  constexpr int N = 4 * NV, TPW = 32 / LPT;
  // about the block's rows come into L2 while the kernel in front ends and the
  // offsets are read
  if (threadIdx.x == 0) {
    const int64_t rows = (static_cast<int64_t>(a.T) - 1) / gridDim.x + 1;
    const int64_t t = blockIdx.x * rows, n = min(rows, a.T - t);
    if (n > 0) {
      prefetch_l2(a.logits + t * a.E, min(n * a.E * 4, kAhead / 2));
      if (a.base) prefetch_l2(a.base + t * a.E, min(n * a.E * 4, kAhead / 2));
    }
  }
  grid_dependency_wait();
  __shared__ int soff[kOffBatch + 1];
  __shared__ int ired[96];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LPT, tl = lane % LPT;
  int lo = 0, hi = a.T;  // tokens of any sequence
  if (a.off) {
    const int2 r = range_of(__ldg(a.off), __ldg(a.off + a.S), a.T);
    lo = r.x;
    hi = r.y;
  }
  float g = a.gloss ? __ldg(a.gloss) : 1.0f;
  const Table table = read_table(a, 0, soff, ired);
  g *= a.coef / max(table.full, 1);
  const int64_t passes = (static_cast<int64_t>(hi) - lo + TPW - 1) / TPW;
  const int64_t W = static_cast<int64_t>(gridDim.x) * kBwdWarps;
  const int64_t per = (passes + W - 1) / W;
  const int64_t w0 = (static_cast<int64_t>(blockIdx.x) * kBwdWarps + warp) * per;
  const int64_t begin = lo + w0 * TPW, end = min(static_cast<int64_t>(hi), begin + per * TPW);
  if (begin >= end) return;
  int2 r = make_int2(0, 0);
  float d[N], factor = 0.0f;  // counts less their mean; the sequence's factor
  const unsigned mates = kFull >> (32 - LPT) << team * LPT;  // the team's lanes
  const float inv_e = 1.0f / static_cast<float>(a.E);
  // the sequence of token t, for tokens in order: most often the next one
  int s = -1;
  auto enter = [&](int t) {
    const bool kept = a.off && a.S <= kOffBatch;
    auto end_of = [&](int n) { return kept ? soff[n + 1] : __ldg(a.off + n + 1); };
    if (!a.off) {
      s = 0;
    } else {
      int x = s + 1, y = a.S;
      if (s >= 0 && x < y && end_of(x) > t) y = x;
      while (x < y) {
        const int mid = (x + y) >> 1;
        if (end_of(mid) > t) y = mid;
        else x = mid + 1;
      }
      s = min(x, a.S - 1);
    }
    r = kept ? range_of(soff[s], soff[s + 1], a.T) : seq_range(a, s);
    int c[N];
    load_row<LPT, NV, int4>(a.bcnt + static_cast<size_t>(s) * a.E, a.E, a.vec, true, tl, 0, c);
    const int n = r.y - r.x;
    // their mean as they are, since entries without an expert are not in them; a
    // team enters together, and max_tokens * K fits into 31 bits
    unsigned sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += c[i];
    if (LPT == 32) {
      sum = __reduce_add_sync(kFull, sum);
    } else {
#pragma unroll
      for (int o = LPT / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mates, sum, o);
    }
    const int mean = __float2int_rn(static_cast<float>(sum) * inv_e);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = static_cast<float>(c[i] - mean);
    factor = n > 0 ? g * seq_factor(a, n) : 0.0f;
  };
  bool entered = false;
  for (int64_t tt = begin; tt < end; tt += TPW) {
    float v[N], o[N], q[N];
    const int64_t t64 = tt + team;
    const bool live = t64 < end;
    const size_t at = static_cast<size_t>(live ? t64 : begin) * a.E;
    auto load = [&](float (&to)[N]) {
      load_row<LPT, NV, float4>(a.logits + at, a.E, a.vec, live, tl, -kInf, to);
    };
    load(v);
    if (a.base) {
      load_base<LPT, NV>(a.base + at, a.E, a.vec, live, tl, o);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = 0.0f;
    }
    if (live && (!entered || t64 >= r.y)) {
      enter(static_cast<int>(t64));
      entered = true;
    }
    __syncwarp();
    bool bad;
    const float inv = probabilities<LPT, NV, SIGMOID, true>(v, q, live, bad, load);
    if (bad && tl == 0) raise_flag(a.flags, MOE_DEVERR_NONFINITE);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) dot = fmaf(v[i], live ? d[i] : 0.0f, dot);
    dot = team_sum<LPT>(dot) * inv;
    const float scale = inv > 0.0f ? factor * inv : 0.0f;  // an infinite factor, too
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(scale * (SIGMOID ? q[i] : v[i]), d[i] - dot, o[i]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col_of<LPT>(tl, 4 * j);
      if (a.vec) {
        if (c < a.E)
          *reinterpret_cast<float4*>(a.glogits + at + c) =
              make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < a.E) a.glogits[at + c + i] = o[4 * j + i];
      }
    }
  }
}

// Lanes a token and 16-byte vectors a lane for E experts: f is called with both
// as constants.
template <typename F>
cudaError_t with_team(int E, F&& f) {
  auto c = [&](auto lanes, auto vecs) { return f(lanes, vecs); };
  if (E <= 8) return c(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
  if (E <= 16) return c(std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
  if (E <= 32) return c(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  if (E <= 64) return c(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  if (E <= 128) return c(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  if (E <= 256) return c(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  if (E <= 384) return c(std::integral_constant<int, 32>{}, std::integral_constant<int, 3>{});
  return c(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
}

bool rows_vec(int E, const void* p) {
  return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

BalArgs bal_args(const moe_handle* h, const float* logits, int T, const int32_t* off, int S,
                 double coef) {
  BalArgs a{};
  a.logits = logits;
  a.off = off;
  a.T = T;
  a.E = h->cfg.num_experts;
  a.K = h->cfg.top_k;
  a.S = S;
  a.stride = (a.E + 3) / 4 * 4;
  a.coef = static_cast<float>(coef);
  a.flags = h->flags;
  return a;
}

}  // namespace

namespace {
size_t tile_shared(int E) { return static_cast<size_t>(kRows + kFrags) * E * sizeof(float); }
size_t join_shared(int C) { return static_cast<size_t>(kJoinRows) * 32 * C * 2 * sizeof(float); }
}  // namespace

BalancePlan balance_plan(int E) {
  BalancePlan p{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t slots = static_cast<size_t>(2 * kMaxTiles) * ((E + 3) / 4 * 4);
  p.slot_p = take(slots * sizeof(float));
  p.slot_c = take(slots * sizeof(int32_t));
  p.tile_loss = take(kMaxTiles * sizeof(float));
  p.spans = take(kMaxTiles * sizeof(int4));
  p.full = take(sizeof(int32_t));
  p.total = o;
  return p;
}

cudaError_t launch_balance(const moe_handle* h, const float* logits, const int32_t* idx, int T,
                           const int32_t* off, int S, double coef, float* loss, int32_t* cnt,
                           float* prob, void* workspace, cudaStream_t s) {
  BalArgs a = bal_args(h, logits, T, off, S, coef);
  const BalancePlan p = balance_plan(a.E);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.idx = idx;
  a.loss = loss;
  a.cnt = cnt;
  a.prob = prob;
  a.slot_p = reinterpret_cast<float*>(ws + p.slot_p);
  a.slot_c = reinterpret_cast<int32_t*>(ws + p.slot_c);
  a.tile_loss = reinterpret_cast<float*>(ws + p.tile_loss);
  a.spans = reinterpret_cast<int4*>(ws + p.spans);
  a.full = reinterpret_cast<int32_t*>(ws + p.full);
  a.vec = rows_vec(a.E, logits);
  // tiles of at least 32 tokens, one to an SM at most; one, and with it one launch,
  // where a block works through all tokens in less than a second launch's time: a
  // token costs it as much as 8 logits and its own (us, softmax, against two launches:
  // 1536 tokens of 8 experts 5.9 and 8.1, 6144 of 8 11.2 and 8.9, 384 of 64 7.4 and
  // 8.5, 768 of 64 9.3 and 8.6, 12288 of 4 17.8 and 8.9).  These are of one sequence; the
  // rule counts neither sequences nor the score, and the one block works on 16 sequences
  // at a time, 11 us each time: 2800 tokens of 8 take 8 us in one sequence, 43 in 64,
  // 1970 in 2800
  int tiles = h->num_sms < kMaxTiles ? h->num_sms : kMaxTiles;
  if ((T - 1) / 32 + 1 < tiles) tiles = (T - 1) / 32 + 1;
  if (static_cast<int64_t>(T) * (a.E + 8) <= 45056) tiles = 1;
  a.tile = T > 0 ? (T - 1) / tiles + 1 : 1;
  a.tiles = T > 0 ? (T - 1) / a.tile + 1 : 1;
  const size_t smem = tile_shared(a.E);
  const bool sigmoid = h->cfg.score_fn == MOE_SCORE_SIGMOID;
  cudaError_t e = with_team(a.E, [&](auto lanes, auto vecs) {
    auto k = sigmoid ? balance_tile_kernel<lanes(), vecs(), true>
                     : balance_tile_kernel<lanes(), vecs(), false>;
    const cudaError_t r = allow_shared_at_launch(h, reinterpret_cast<const void*>(k),
                                                 tile_shared(MOE_MAX_EXPERTS));
    if (r != cudaSuccess) return r;
    return launch_chained(k, dim3(a.tiles), dim3(kThreads), smem, s, false, a);
  });
  if (e != cudaSuccess || a.tiles == 1) return e;
  const bool two = a.E > 32 * kCluster;
  auto join = two ? balance_join_kernel<2> : balance_join_kernel<1>;
  const size_t join_smem = join_shared(two ? 2 : 1);
  e = allow_shared_at_launch(h, reinterpret_cast<const void*>(join), join_smem);
  if (e != cudaSuccess) return e;
  return launch_chained(join, dim3(kCluster), dim3(32 * kJoinWarps), join_smem, s, false, a);
}

cudaError_t launch_balance_bwd(const moe_handle* h, const float* logits, const int32_t* cnt, int T,
                               const int32_t* off, int S, double coef, const float* gloss,
                               const float* base, float* glogits, cudaStream_t s) {
  BalArgs a = bal_args(h, logits, T, off, S, coef);
  a.bcnt = cnt;
  a.gloss = gloss;
  a.base = base;
  a.glogits = glogits;
  a.vec = rows_vec(a.E, logits) && rows_vec(a.E, cnt) && rows_vec(a.E, base) &&
          rows_vec(a.E, glogits);
  if (T == 0) return cudaSuccess;
  const bool sigmoid = h->cfg.score_fn == MOE_SCORE_SIGMOID;
  return with_team(a.E, [&](auto lanes, auto vecs) {
    constexpr int TPW = 32 / lanes();
    auto k = sigmoid ? balance_bwd_kernel<lanes(), vecs(), true>
                     : balance_bwd_kernel<lanes(), vecs(), false>;
    const int64_t blocks = (static_cast<int64_t>(T) + kBwdWarps * TPW - 1) / (kBwdWarps * TPW);
    const int64_t most = static_cast<int64_t>(kBwdBlocks<vecs()>) * h->num_sms;
    return launch_chained(k, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                          dim3(kBwdWarps * 32), 0, s, false, a);
  });
}

}  // namespace moe
