// The router's balance loss with per-expert counts, and its gradient (sm_103a).
//
// For sequence s of n_s tokens, c_se its entries of expert e and P_se the sum
// over its tokens of p_te (softmax, or sigmoid divided by the row's sum):
//   loss = coef / S' * sum_s E / (K n_s^2) * sum_e c_se P_se,
// S' the sequences that are not empty.  With the counts constant,
//   dloss/dl_tj = coef / S' * E / (K n_s^2) * q_tj (c_sj - sum_e c_se p_te),
// q = p for softmax, sigma (1 - sigma) / sum(sigma) for sigmoid.  Since p sums
// to 1, a constant can be taken off the counts: the backward takes the mean
// count off as an integer, exactly, so that the difference of two near-equal
// sums of counts never loses digits.
//
// Forward: tokens are cut into equal tiles, one block each.  A tile's part of a
// sequence is a fragment.  A sequence inside one tile is finished there; the
// fragments of one that spans tiles go to slots (two a tile suffice: one for
// the fragment that began in an earlier tile, one for that which goes on into
// the next) and a second kernel adds them up.  Every sum has a fixed order
// (counts are integers), so repeated calls give the same bits.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTiles = 1024;
constexpr int kOffBatch = 256;   // sequence offsets staged at a time
constexpr int kJoinCols = 32;    // experts of a block of the second kernel
// Tokens a team sums in registers before it adds them to shared memory: bounds
// the number of fp32 additions in a row however long a tile is.
constexpr int kFlush = 64;
constexpr float kInf = __builtin_huge_valf();

struct BalArgs {
  const float* logits;   // [T, E]
  const int32_t* idx;    // [T, K] (forward)
  const int32_t* off;    // [S + 1] or NULL: one sequence, all T tokens
  int T, E, K, S;
  int tile, tiles;       // tokens of a tile, tiles
  int chunks;            // blocks of kJoinCols experts
  int vec;               // rows can be read 16 bytes at a time
  float coef;
  uint32_t* flags;
  // forward
  int32_t* cnt;          // [S, E]
  float* prob;           // [S, E] or NULL
  float* loss;           // [1]
  float* slot_p;         // [2 * tiles, E]
  int32_t* slot_c;       // [2 * tiles, E]
  float* part;           // [S, chunks]
  unsigned* ticket;
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

// First sequence that ends behind token t (S if there is none).
__device__ __forceinline__ int seq_of(const BalArgs& a, int t) {
  if (!a.off) return t < a.T ? 0 : 1;
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.off + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
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

// Turns a team's logits v into p and, for the backward, q (see the top).  A
// logit of -inf is an expert that is masked out: p = q = 0.  A row without any
// other is 0, and so is one with a NaN or +inf, for which `bad` is returned.
// exp is the fast one: its error, 2 + |x| ulp at x <= 0, falls on values that
// are e^x of the row's largest.
template <int LPT, int NV, bool SIGMOID, bool GRAD>
__device__ __forceinline__ bool probabilities(float (&v)[4 * NV], float (&q)[4 * NV]) {
  constexpr int N = 4 * NV;
  float m = -kInf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmaxf(m, v[i]);  // a NaN is not taken: `bad` finds it
    bad |= !(v[i] < kInf);
  }
  m = team_max<LPT>(m);
  float z = 0.0f;
  // sigmoids all far below 1 are e^l to 1e-13, and normalised from the row's
  // largest they cannot vanish together
  const bool scaled = !SIGMOID || m < -30.0f;
  if (scaled) {
    const float sub = m > -kInf ? m : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = __expf(v[i] - sub);
      if (GRAD) q[i] = v[i];
      z += v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = __expf(-fabsf(v[i]));
      const float r = __fdividef(1.0f, 1.0f + e);
      const float s = v[i] >= 0.0f ? r : e * r;
      if (GRAD) q[i] = s * (v[i] >= 0.0f ? e * r : r);
      v[i] = s;
      z += s;
    }
  }
  z = team_sum<LPT>(z);
  // the team's lanes agree: the sum is the same in each, and so is this vote
  const unsigned votes = __ballot_sync(kFull, bad);
  const int first = (threadIdx.x & 31) / LPT * LPT;
  bad = (votes >> first) & (LPT == 32 ? kFull : (1u << (LPT & 31)) - 1u);
  const float inv = z > 0.0f && !bad ? 1.0f / z : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = bad ? 0.0f : v[i] * inv;
    if (GRAD) q[i] = bad ? 0.0f : q[i] * inv;
  }
  return bad;
}

// Sum over the block's threads, the same in each; `red` holds kWarps values.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) v += red[w];
  __syncthreads();
  return v;
}

// Factor of a sequence of n tokens.
__device__ __forceinline__ float seq_factor(const BalArgs& a, int n) {
  return static_cast<float>(a.E) / (static_cast<float>(a.K) * n) / n;
}

// The loss from the sequences' parts, by one block.
__device__ void finish(const BalArgs& a) {
  __shared__ double sums[32];
  __shared__ int full[32];
  double sum = 0.0;
  int n = 0;
  for (int64_t i = threadIdx.x; i < static_cast<int64_t>(a.S) * a.chunks; i += blockDim.x)
    sum += static_cast<double>(__ldcg(a.part + i));
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    const int2 r = seq_range(a, s);
    n += r.y > r.x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, o);
    n += __shfl_xor_sync(kFull, n, o);
  }
  if ((threadIdx.x & 31) == 0) {
    sums[threadIdx.x >> 5] = sum;
    full[threadIdx.x >> 5] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) {
      sum += sums[w];
      n += full[w];
    }
    *a.loss = n > 0 ? static_cast<float>(a.coef * sum / n) : 0.0f;
  }
}

// Fragments of a tile: sums of p and counts of its tokens [t0, t1) of each
// sequence.
template <int LPT, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) balance_tile_kernel(BalArgs a) {
  grid_dependency_wait();
  constexpr int N = 4 * NV, TPW = 32 / LPT;
  extern __shared__ float dyn[];
  float* stage = dyn;                                        // [kWarps][E]
  int* hist = reinterpret_cast<int*>(dyn + kWarps * a.E);    // [E]
  __shared__ int soff[kOffBatch + 1];
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LPT, tl = lane % LPT;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  if (a.off || a.T == 0) {  // empty sequences, and the offsets themselves
    bool wrong = false;
    const int W = gridDim.x * kWarps;
    for (int s = blockIdx.x * kWarps + warp; s < a.S; s += W) {
      const int lo = a.off ? __ldg(a.off + s) : 0, hi = a.off ? __ldg(a.off + s + 1) : 0;
      wrong |= lo < 0 || hi < lo || hi > a.T;
      const int2 r = range_of(lo, hi, a.T);
      if (r.y > r.x) continue;
      const size_t row = static_cast<size_t>(s) * a.E;
      for (int e = lane; e < a.E; e += 32) {
        a.cnt[row + e] = 0;
        if (a.prob) a.prob[row + e] = 0.0f;
      }
      if (lane < a.chunks) a.part[static_cast<size_t>(s) * a.chunks + lane] = 0.0f;
    }
    if (wrong) raise_flag(a.flags, MOE_DEVERR_BAD_LAYOUT);
  }
  const int t0 = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * a.tile,
                                      static_cast<int64_t>(a.T)));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(t0) + a.tile, static_cast<int64_t>(a.T)));
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  const int s0 = seq_of(a, t0);
  bool more = true;
  for (int sb = s0; more && sb < a.S; sb += kOffBatch) {
    const int ns = min(kOffBatch, a.S - sb);
    __syncthreads();
    for (int i = threadIdx.x; i <= ns; i += kThreads)
      soff[i] = a.off ? __ldg(a.off + sb + i) : (i == 0 ? 0 : a.T);
    __syncthreads();
    for (int i = 0; i < ns; ++i) {
      const int s = sb + i;
      const int2 r = range_of(soff[i], soff[i + 1], a.T);
      if (soff[i] >= t1) {
        more = false;
        break;
      }
      const int f0 = max(r.x, t0), f1 = min(r.y, t1);
      if (f0 >= f1) continue;
      // counts: a thread a token, whose later repeats of an expert are dropped
      for (unsigned t = f0 + threadIdx.x; t < static_cast<unsigned>(f1); t += kThreads) {
        const int32_t* entries = a.idx + static_cast<size_t>(t) * a.K;
        int seen[MOE_MAX_TOPK];
#pragma unroll
        for (int k = 0; k < MOE_MAX_TOPK; ++k) {
          if (k >= a.K) break;
          const int e = __ldg(entries + k);
          seen[k] = e;
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
      // sums of p
      float acc[N], v[N], unused[N];
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
            float* to = stage + warp * a.E + c;
            *to = begun ? *to + acc[k] : acc[k];
          }
          acc[k] = 0.0f;
        }
        begun = true;
        held = 0;
      };
      for (unsigned t = f0 + warp * TPW; t < static_cast<unsigned>(f1); t += kWarps * TPW) {
        const bool live = t + team < static_cast<unsigned>(f1);
        load_row<LPT, NV, float4>(a.logits + static_cast<size_t>(live ? t + team : t) * a.E, a.E,
                                  a.vec, live, tl, -kInf, v);
        if (probabilities<LPT, NV, SIGMOID, false>(v, unused) && tl == 0)
          raise_flag(a.flags, MOE_DEVERR_NONFINITE);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += v[k];
        if (++held == kFlush) flush();
      }
      flush();
      __syncthreads();
      const bool whole = r.x >= t0 && r.y <= t1;
      const int slot = 2 * blockIdx.x + (r.x >= t0);
      float val = 0.0f;
      for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) p += stage[w * a.E + e];
        const int c = hist[e];
        hist[e] = 0;
        if (whole) {
          const size_t at = static_cast<size_t>(s) * a.E + e;
          a.cnt[at] = c;
          if (a.prob) a.prob[at] = p / (r.y - r.x);
          val += static_cast<float>(c) * p;
        } else {
          const size_t at = static_cast<size_t>(slot) * a.E + e;
          a.slot_p[at] = p;
          a.slot_c[at] = c;
        }
      }
      if (whole) {
        val = block_sum(val, red) * seq_factor(a, r.y - r.x);
        if (threadIdx.x < a.chunks)
          a.part[static_cast<size_t>(s) * a.chunks + threadIdx.x] = threadIdx.x == 0 ? val : 0.0f;
      } else {
        __syncthreads();  // stage and hist are taken up again
      }
    }
  }
  if (gridDim.x == 1) {  // every sequence is whole: the loss in the same launch
    __syncthreads();
    finish(a);
  }
}

// Sequences that span tiles: block (x, y) adds up the slots of one of them for
// kJoinCols experts, a warp for every blockDim / 32-th slot; the last block to
// end adds up the loss.
__global__ void __launch_bounds__(1024) balance_join_kernel(BalArgs a) {
  grid_dependency_wait();
  __shared__ float ps[32][kJoinCols];
  __shared__ int cs[32][kJoinCols];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // item x is sequence x, or where there are more sequences than tiles the one
  // that goes on from tile x into the next
  int s = blockIdx.x;
  if (a.S > a.tiles) {
    const int64_t next = (static_cast<int64_t>(blockIdx.x) + 1) * a.tile;
    s = next < a.T ? seq_of(a, static_cast<int>(next)) : a.S;
  }
  if (s < a.S) {
    const int2 r = seq_range(a, s);
    const int b0 = r.x / a.tile, b1 = (r.y - 1) / a.tile;
    if (r.y > r.x && b1 > b0 && (a.S <= a.tiles || b0 == static_cast<int>(blockIdx.x))) {
      const int e = blockIdx.y * kJoinCols + lane;
      float p = 0.0f;
      int c = 0;
      if (e < a.E)
#pragma unroll 4
        for (int b = b0 + warp; b <= b1; b += warps) {
          const size_t at = static_cast<size_t>(2 * b + (b == b0)) * a.E + e;
          p += __ldcg(a.slot_p + at);
          c += __ldcg(a.slot_c + at);
        }
      ps[warp][lane] = p;
      cs[warp][lane] = c;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < warps; ++w) {
          p += ps[w][lane];
          c += cs[w][lane];
        }
        float val = 0.0f;
        if (e < a.E) {
          const size_t at = static_cast<size_t>(s) * a.E + e;
          a.cnt[at] = c;
          if (a.prob) a.prob[at] = p / (r.y - r.x);
          val = static_cast<float>(c) * p;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) val += __shfl_xor_sync(kFull, val, o);
        if (lane == 0)
          a.part[static_cast<size_t>(s) * a.chunks + blockIdx.y] = val * seq_factor(a, r.y - r.x);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
    __threadfence();
  }
  __syncthreads();
  if (last) finish(a);
}

// Backward: a team of lanes a token, a warp's tokens in a row.
template <int LPT, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalArgs a) {
  constexpr int N = 4 * NV, TPW = 32 / LPT;
  __shared__ int counts[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = lane / LPT, tl = lane % LPT;
  int full = a.T > 0;
  if (a.off) {  // sequences that are not empty
    full = 0;
    for (int s = threadIdx.x; s < a.S; s += kThreads) {
      const int2 r = seq_range(a, s);
      full += r.y > r.x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) full += __shfl_xor_sync(kFull, full, o);
    if (lane == 0) counts[warp] = full;
    __syncthreads();
    full = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) full += counts[w];
  }
  const float g = a.coef * (a.gloss ? __ldg(a.gloss) : 1.0f) / max(full, 1);
  int lo = 0, hi = a.T;  // tokens of any sequence
  if (a.off) {
    const int2 r = range_of(__ldg(a.off), __ldg(a.off + a.S), a.T);
    lo = r.x;
    hi = r.y;
  }
  const int64_t passes = (static_cast<int64_t>(hi) - lo + TPW - 1) / TPW;
  const int64_t W = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t per = (passes + W - 1) / W;
  const int64_t w0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * per;
  const int64_t begin = lo + w0 * TPW, end = min(static_cast<int64_t>(hi), begin + per * TPW);
  if (begin >= end) return;
  int s = -1;
  int2 r = make_int2(0, 0);
  float d[N], factor = 0.0f;  // counts less their mean; the sequence's factor
  for (int64_t tt = begin; tt < end; tt += TPW) {
    const int t = static_cast<int>(min(tt + team, end - 1));
    const bool live = tt + team < end;
    float v[N], q[N];
    const size_t at = static_cast<size_t>(t) * a.E;
    load_row<LPT, NV, float4>(a.logits + at, a.E, a.vec, live, tl, -kInf, v);
    if (s < 0 || t >= r.y) {
      s = min(seq_of(a, t), a.S - 1);
      r = seq_range(a, s);
      int c[N];
      load_row<LPT, NV, int4>(a.bcnt + static_cast<size_t>(s) * a.E, a.E, a.vec, true, tl, 0, c);
      const int n = r.y - r.x;
      const int mean = static_cast<int>(static_cast<int64_t>(a.K) * n / a.E);
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = static_cast<float>(c[i] - mean);
      factor = n > 0 ? g * seq_factor(a, n) : 0.0f;
    }
    __syncwarp();
    if (probabilities<LPT, NV, SIGMOID, true>(v, q) && tl == 0)
      raise_flag(a.flags, MOE_DEVERR_NONFINITE);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) dot = fmaf(v[i], d[i], dot);
    dot = team_sum<LPT>(dot);
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col_of<LPT>(tl, 4 * j);
      if (a.vec) {
        if (c >= a.E) continue;
        float4 o{0.0f, 0.0f, 0.0f, 0.0f};
        if (a.base) o = *reinterpret_cast<const float4*>(a.base + at + c);
        o.x = fmaf(factor * q[4 * j], d[4 * j] - dot, o.x);
        o.y = fmaf(factor * q[4 * j + 1], d[4 * j + 1] - dot, o.y);
        o.z = fmaf(factor * q[4 * j + 2], d[4 * j + 2] - dot, o.z);
        o.w = fmaf(factor * q[4 * j + 3], d[4 * j + 3] - dot, o.w);
        *reinterpret_cast<float4*>(a.glogits + at + c) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < a.E)
            a.glogits[at + c + i] = fmaf(factor * q[4 * j + i], d[4 * j + i] - dot,
                                         a.base ? a.base[at + c + i] : 0.0f);
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
  if (E <= 16) return c(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  if (E <= 32) return c(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (E <= 64) return c(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (E <= 128) return c(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
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
  a.chunks = (a.E + kJoinCols - 1) / kJoinCols;
  a.coef = static_cast<float>(coef);
  a.flags = h->flags;
  return a;
}

}  // namespace

BalancePlan balance_plan(int E, int S) {
  BalancePlan p{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  p.ticket = take(sizeof(unsigned));
  p.slot_p = take(static_cast<size_t>(2 * kMaxTiles) * E * sizeof(float));
  p.slot_c = take(static_cast<size_t>(2 * kMaxTiles) * E * sizeof(int32_t));
  p.part = take(static_cast<size_t>(S) * ((E + kJoinCols - 1) / kJoinCols) * sizeof(float));
  p.total = o;
  return p;
}

cudaError_t launch_balance(const moe_handle* h, const float* logits, const int32_t* idx, int T,
                           const int32_t* off, int S, double coef, float* loss, int32_t* cnt,
                           float* prob, void* workspace, cudaStream_t s) {
  BalArgs a = bal_args(h, logits, T, off, S, coef);
  const BalancePlan p = balance_plan(a.E, S);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.idx = idx;
  a.loss = loss;
  a.cnt = cnt;
  a.prob = prob;
  a.ticket = reinterpret_cast<unsigned*>(ws + p.ticket);
  a.slot_p = reinterpret_cast<float*>(ws + p.slot_p);
  a.slot_c = reinterpret_cast<int32_t*>(ws + p.slot_c);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.vec = rows_vec(a.E, logits);
  // tiles of at least 8 tokens, four to an SM at most; one, and with it one
  // launch, where a block reads all of the logits in about a launch's time
  int tiles = 4 * h->num_sms < kMaxTiles ? 4 * h->num_sms : kMaxTiles;
  if ((T + 7) / 8 < tiles) tiles = (T + 7) / 8;
  if (static_cast<int64_t>(T) * a.E <= 16384) tiles = 1;
  if (tiles < 1) tiles = 1;
  a.tile = T > 0 ? (T + tiles - 1) / tiles : 1;
  a.tiles = T > 0 ? (T + a.tile - 1) / a.tile : 1;
  const size_t smem = static_cast<size_t>(kWarps + 1) * a.E * sizeof(float);
  const bool sigmoid = h->cfg.score_fn == MOE_SCORE_SIGMOID;
  cudaError_t e = with_team(a.E, [&](auto lanes, auto vecs) {
    auto k = sigmoid ? balance_tile_kernel<lanes(), vecs(), true>
                     : balance_tile_kernel<lanes(), vecs(), false>;
    return launch_chained(k, dim3(a.tiles), dim3(kThreads), smem, s, false, a);
  });
  if (e != cudaSuccess || a.tiles == 1) return e;
  const int items = S < a.tiles ? S : a.tiles;
  int warps = 1;
  while (warps < 32 && warps * items < a.tiles) warps *= 2;
  return launch_chained(balance_join_kernel, dim3(items, a.chunks), dim3(32 * warps), 0, s, false,
                        a);
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
    const int64_t blocks = (static_cast<int64_t>(T) + kWarps * TPW - 1) / (kWarps * TPW);
    const int64_t most = 8LL * h->num_sms;
    k<<<static_cast<unsigned>(blocks < most ? blocks : most), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace moe
