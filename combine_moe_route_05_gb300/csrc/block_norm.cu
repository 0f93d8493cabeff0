// The norms around a block (sm_103a): the block's output rows, or the weighted
// sum of their receive rows, normed, gated and added to the residual stream, and
// the next block's norm of that sum; and the backward.
//
//   c = y + add                      (y: token rows, or sum_k w_k y[pos[t,k]])
//   res' = res_scale * res + gate * (c r_c (w_post + offset))
//   x    = res' r_p (w_pre + offset),    r_v = 1 / sqrt(mean(v^2) + eps)
//
// One pass over the rows: a team of threads (8 to 32 lanes of a warp, or the warps of
// a block, several teams to a block) holds a row in registers, 16 elements a thread,
// and the two sums of squares are its only exchange.  x is made from the sum before
// that is rounded; sums are fp32, each output is rounded once.
//
// Bound by HBM; what stands in its way are the two sums in a row's chain.  Each
// thread therefore copies the vectors that it will need itself into shared memory
// ahead of time (cp.async: no other thread waits for them), so loads go on while
// the team waits for its sums, and the weights, in fp32 with their offset, stay
// there too, once for all teams of a block.  Nothing else that a token needs (row
// positions, scores, the norms' factors) is read in the token's own chain, and no
// division is left in it.  Arithmetic is on pairs of fp32, one instruction for both.
//
// DeepSeek-V3 shape (16384 tokens of 7168, bf16), us against the 457 and 211 of the
// bytes at the copy rate: the combine's sum of 8 rows with shared experts, both norms
// and what the backward needs 738 as plain loads in registers, 672 with the copies
// ahead, 458 with nothing read in the chain, 437 now; the backward 549, 302, 225, 216.
// Token rows alone 150 (141), the backward of 8192 x 2048 with a gate row for 1300
// tokens 41.8 (30.2), of which some 9 are the first rows' and the joins' latency.
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kEpt = 16;           // elements of a row a thread holds
constexpr int kWarpRow = 32 * kEpt;  // widest row of a one-warp team
constexpr int kTeamThreads = 512;  // threads of a block of several teams, at most
// Tokens whose column sums are added up in registers before they are added to a block's
// row: a sum has 1024 + T / (1024 * SMs) + 112 fp32 additions in a row, of which the
// middle part is 17 for 2600000 tokens.
constexpr int kFlush = 1024;
constexpr int kJoinWarps = 16, kJoinCols = 64;  // of the kernel that joins the column sums
constexpr int kJoinLoads = 10;  // of a warp at a time: all of an SM's sums in one
constexpr size_t kShared = 224 * 1024;  // dynamic shared memory of a block, at most
constexpr size_t kSmShared = 228 * 1024;  // of an SM, of which a block takes 1 KB for itself

// ---------------------------------------------------------------------------
// pairs of fp32

using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }
__device__ __forceinline__ float sum_of(F2 a) {
  const float2 v = split(a);
  return v.x + v.y;
}

// A 16-byte vector of a row as pairs (bf16: 4, fp32: 2), and back, rounded.
template <typename Elt>
struct PairTraits;
template <>
struct PairTraits<__nv_bfloat16> {
  static constexpr int P = 4;
  __device__ __forceinline__ static void to(const Vec16& v, F2* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = pair(__uint_as_float(v.u[i] << 16), __uint_as_float(v.u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static Vec16 from(const F2* f) {
    Vec16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = split(f[i]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(a.x, a.y);
      v.u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return v;
  }
};
template <>
struct PairTraits<float> {
  static constexpr int P = 2;
  __device__ __forceinline__ static void to(const Vec16& v, F2* f) {
    f[0] = pair(__uint_as_float(v.u[0]), __uint_as_float(v.u[1]));
    f[1] = pair(__uint_as_float(v.u[2]), __uint_as_float(v.u[3]));
  }
  __device__ __forceinline__ static Vec16 from(const F2* f) {
    const float2 a = split(f[0]), b = split(f[1]);
    return Vec16{{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                  __float_as_uint(b.y)}};
  }
};

// ---------------------------------------------------------------------------
// a thread's own shared memory: vectors on their way, weights

__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most N of the thread's groups of copies are under way.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 16 bytes, or zeros where there is nothing to read (`from` is not read then).
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ Vec16 ld_shared(uint32_t a) {
  Vec16 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3])
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t a, const Vec16& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.u[0]), "r"(v.u[1]),
               "r"(v.u[2]), "r"(v.u[3])
               : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// Shared memory of a block: the weights, 16 bytes a thread of a team in each of
// kWeightSlots rows (teams share them), then the vectors under way in slots of 16
// bytes, `sb` = 16 times the block's threads from one to the next, so that a
// warp's copies land side by side.  (Slots of a thread one behind another, with
// addresses known when compiled, took the backward from 302 to 372 us at the
// DeepSeek-V3 shape.)
constexpr int kWeightSlots = kEpt / 4;  // 16 fp32

// The 16 weights of a team's thread on their way from memory to shared memory: asked
// for ahead of the rows, which the weights would otherwise arrive behind.  Zero
// behind the row's end; the thread's vectors of N elements are tid, tid + threads, ...
template <int N>
struct Weights {
  float4 f[kWeightSlots];
  __device__ __forceinline__ void load(const uint8_t* w, int f32, int tid, int threads, int nvec) {
#pragma unroll
    for (int q = 0; q < kWeightSlots; ++q) {
      const int v = tid + q / (N / 4) * threads;
      f[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (w && v < nvec) {
        const int at = v * (N / 4) + q % (N / 4);
        if (f32) {
          f[q] = __ldg(reinterpret_cast<const float4*>(w) + at);
        } else {
          const uint2 b = __ldg(reinterpret_cast<const uint2*>(w) + at);
          f[q].x = __uint_as_float(b.x);  // spread out when they are kept
          f[q].y = __uint_as_float(b.y);
        }
      }
    }
  }
  // from `to` on, in rows wb bytes apart
  __device__ __forceinline__ void keep(int f32, float offset, uint32_t to, uint32_t wb, int tid,
                                       int threads, int nvec) const {
#pragma unroll
    for (int q = 0; q < kWeightSlots; ++q) {
      float4 x = f[q];
      if (!f32) {
        const uint32_t lo = __float_as_uint(x.x), hi = __float_as_uint(x.y);
        x = make_float4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u),
                        __uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
      }
      const float o = tid + q / (N / 4) * threads < nvec ? offset : 0.0f;
      st_shared(to + q * wb, make_float4(x.x + o, x.y + o, x.z + o, x.w + o));
    }
  }
};
// The weights of the thread's vector i.
template <int N>
__device__ __forceinline__ void kept_weights(uint32_t at, uint32_t wb, int i, F2* f) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const Vec16 v = ld_shared(at + (i * (N / 4) + q) * wb);
    f[2 * q] = pair(__uint_as_float(v.u[0]), __uint_as_float(v.u[1]));
    f[2 * q + 1] = pair(__uint_as_float(v.u[2]), __uint_as_float(v.u[3]));
  }
}

// Which team a thread is in, and where in it: blocks hold whole teams.  WARP: teams
// of a warp, or of half or a quarter of one for the narrowest rows.
template <bool WARP, int MAXT>
struct Team {
  int threads, index, tid;
  float* red;  // two sets of 32 values, taken in turn (teams of several warps)
  int turn = 0;
  unsigned lanes;  // the team's, of its warp
  __device__ __forceinline__ Team(int team_threads, float* sums)
      : threads(team_threads),
        index(threadIdx.x / team_threads),
        tid(threadIdx.x - index * team_threads),
        red(sums + (WARP ? 0 : 64 * index)),
        lanes(kFull) {
    if (!WARP) {
      for (int i = tid; i < 64; i += threads) red[i] = 0.0f;
    } else if (threads < 32) {
      lanes = ((1u << threads) - 1u) << ((threadIdx.x & 31) - tid);
    }
  }
  __device__ __forceinline__ void sync() {
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
  }
  // Sum over the team.  A barrier a sum is enough, and the values behind the last
  // warp's stay zero, so that they are read four at a time.
  __device__ __forceinline__ float sum(float v) {
    if constexpr (WARP) {
      for (int o = threads >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(lanes, v, o);
      return v;
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
      float* set = red + turn;
      turn ^= 32;
      if ((tid & 31) == 0) set[tid >> 5] = v;
      sync();
      float4 a = *reinterpret_cast<const float4*>(set);
#pragma unroll
      for (int w = 4; w < MAXT / 32; w += 4) {
        const float4 b = *reinterpret_cast<const float4*>(set + w);
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      return (a.x + a.y) + (a.z + a.w);
    }
  }
};
constexpr int kRed = 64 * 8;  // eight teams of two warps at most

// ---------------------------------------------------------------------------
// forward

struct NormArgs {
  const uint8_t* y;      // [T, H], [rows, H] with pos, or NULL
  const int32_t* pos;    // [T, K] or NULL (then K = 1)
  const float* cw;       // [T, K] or NULL
  const uint8_t* add;    // [T, H] or NULL
  const uint8_t* res;    // [T, H]
  const uint8_t* gate;   // [groups, H] or NULL
  const uint8_t* w_post; // [H] or NULL
  const uint8_t* w_pre;  // [H] or NULL
  uint8_t* c;            // [T, H] or NULL
  uint8_t* res_out;      // [T, H] or NULL
  uint8_t* x;            // [T, H] or NULL
  float* rstd_post;      // [T] or NULL
  float* rstd_pre;       // [T] or NULL
  int64_t row_bytes;
  int T, H, nvec, K, rows, gate_tokens;
  int units;             // teams; a team takes every units-th token
  int teams, team_threads;  // of a block; of a team
  int w_f32;             // weights in fp32 (else bf16)
  float res_scale, eps, offset, inv_h;
  uint32_t* flags;
};

// A team takes every units-th token, a vector a thread of all its rows at a time.
// KMAX: rows that are summed at most (1: token rows).  AHEAD: tokens whose vectors are
// in shared memory or on their way there.  0: they are loaded when they are needed, as
// not one token's fit (fp32 with 6 and more receive rows, bf16 with 12 and more, at most
// widths; fewer with added rows and gate): 8 fp32 rows, 8192 x 2048, 124 us against 111
// of the bytes, 4096 x 7168 238 and 193; 16 bf16 rows, 8192 x 2048, 126 and 96; 8 with
// added rows and gate, 2048 x 8192, 108 and 65.
template <typename Elt, int KMAX, bool WARP, int MAXT, int AHEAD>
__global__ void __launch_bounds__(MAXT, KMAX == 1 && MAXT <= 512 && sizeof(Elt) == 2 ? 2 : 1)
    block_norm_kernel(NormArgs a) {
  using PT = PairTraits<Elt>;
  constexpr int P = PT::P, N = 2 * P, V = kEpt / N;
  constexpr bool GATHER = KMAX > 1;
  static_assert(!GATHER || AHEAD < 2, "a token's weights are asked for one token ahead");
  __shared__ __align__(16) float red[kRed];
  extern __shared__ __align__(16) uint8_t shared[];
  grid_dependency_wait();
  Team<WARP, MAXT> team(a.team_threads, red);
  const int tid = team.tid, step = team.threads;
  const int unit = blockIdx.x * a.teams + team.index;
  const uint32_t sb = blockDim.x * 16, wb = step * 16;
  const uint32_t wpost = smem_addr(shared) + tid * 16;
  const uint32_t wpre = wpost + (a.w_post ? kWeightSlots * wb : 0);
  const uint32_t ring = smem_addr(shared) + threadIdx.x * 16 +
                        ((a.w_post != nullptr) + (a.w_pre != nullptr)) * kWeightSlots * wb;
  // slots of a vector's rows: the residual stream's, the block's, ...
  const uint32_t add_at = sb * (1 + (a.y ? a.K : 0)), gate_at = add_at + (a.add ? sb : 0);
  const uint32_t vector = gate_at + (a.gate ? sb : 0), token = V * vector;  // bytes
  bool in[V];    // vectors inside the row, and where
  int at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = tid + i * step < a.nvec;
    at[i] = in[i] ? (tid + i * step) * 16 : 0;
  }

  // receive rows and weights of a token's entries, as read
  auto read_entries = [&](int64_t t, const auto* from, auto (&to)[KMAX], auto none) {
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      to[k] = none;
      if (k < a.K && t < a.T) to[k] = __ldg(from + t * a.K + k);
    }
  };
  auto check_entries = [&](int (&p)[KMAX]) {
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (p[k] != -1) p[k] = checked_row(p[k], a.rows, a.flags);
  };
  int p[KMAX], p_read[KMAX];     // rows of the token asked for next, and of the one behind it
  float wk[KMAX], w_read[KMAX];  // weights of the token in work and the one behind it
  auto fetch = [&](int64_t t, int i, uint32_t to) {
    if (t < a.T) {
      const int64_t off = t * a.row_bytes + at[i];
      copy_async(to, a.res + off, in[i]);
      if (GATHER) {
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          if (k >= a.K) break;
          const bool real = in[i] && p[k] >= 0;
          copy_async(to + (k + 1) * sb, a.y + (real ? p[k] * a.row_bytes + at[i] : 0), real);
        }
      } else if (a.y) {
        copy_async(to + sb, a.y + off, in[i]);
      }
      if (a.add) copy_async(to + add_at, a.add + off, in[i]);
      if (a.gate)
        copy_async(to + gate_at,
                   a.gate + (static_cast<unsigned>(t) / static_cast<unsigned>(a.gate_tokens)) *
                                a.row_bytes + at[i],
                   in[i]);
    }
    commit_copies();
  };
  // weights as they count: a dropped entry's row is zeros, and whatever its
  // weight is, it adds nothing
  auto count_weights = [&](const float (&read)[KMAX]) {
#pragma unroll
    for (int k = 0; k < KMAX; ++k) wk[k] = p[k] < 0 ? 0.0f : a.cw ? read[k] : 1.0f;
  };

  // weights ahead of the rows, but where registers are short (bf16 token rows): there
  // the loop came out slower (16384 x 2048 49.3 against 46.5 us; fp32 rows of 1000,
  // 1500 tokens, 9.2 against 11.5)
  constexpr bool EARLY = GATHER || sizeof(Elt) == 4;
  Weights<N> post, pre;
  if (EARLY && team.index == 0) {
    post.load(a.w_post, a.w_f32, tid, step, a.nvec);
    pre.load(a.w_pre, a.w_f32, tid, step, a.nvec);
  }
  if (AHEAD > 0) {
    if (GATHER) {
      read_entries(unit, a.pos, p, -1);
      if (a.cw) read_entries(unit, a.cw, w_read, 0.0f);
      read_entries(unit + static_cast<int64_t>(a.units), a.pos, p_read, -1);
      check_entries(p);
      count_weights(w_read);
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n)
#pragma unroll
      for (int i = 0; i < V; ++i)
        fetch(unit + static_cast<int64_t>(n) * a.units, i, ring + n * token + i * vector);
    if (GATHER) {
      check_entries(p_read);
#pragma unroll
      for (int k = 0; k < KMAX; ++k) p[k] = p_read[k];
    }
  }
  // each thread of the first team for its places in all teams
  if (team.index == 0) {
    if (!EARLY) post.load(a.w_post, a.w_f32, tid, step, a.nvec);
    if (a.w_post) post.keep(a.w_f32, a.offset, wpost, wb, tid, step, a.nvec);
    if (!EARLY) pre.load(a.w_pre, a.w_f32, tid, step, a.nvec);
    if (a.w_pre) pre.keep(a.w_f32, a.offset, wpre, wb, tid, step, a.nvec);
  }
  __syncthreads();
  uint32_t stage = ring;
  for (int64_t t = unit; t < a.T; t += a.units) {
    const int64_t row = t * a.row_bytes;
    if (GATHER) {
      if (AHEAD > 0) {
        read_entries(t + 2 * static_cast<int64_t>(a.units), a.pos, p_read, -1);
        if (a.cw) read_entries(t + a.units, a.cw, w_read, 0.0f);
      } else {
        read_entries(t, a.pos, p, -1);
        if (a.cw) read_entries(t, a.cw, w_read, 0.0f);
        check_entries(p);
        count_weights(w_read);
      }
    }
    F2 c[V][P];
    Vec16 res[V], gate[V];
    F2 ss = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (AHEAD > 0) wait_copies<V * AHEAD - 1>();
      const uint32_t from = stage + i * vector;
      auto get = [&](uint32_t slot, const uint8_t* g, bool real) {
        Vec16 x{};
        if (AHEAD > 0) x = ld_shared(from + slot);
        else if (real) x = ld_vec(g);
        return x;
      };
      res[i] = get(0, a.res + row + at[i], in[i]);
      if (GATHER) {
        Vec16 rows[KMAX];
        if (AHEAD == 0)
#pragma unroll
          for (int k = 0; k < KMAX; ++k)
            rows[k] = get((k + 1) * sb, a.y + p[k] * a.row_bytes + at[i], in[i] && p[k] >= 0);
#pragma unroll
        for (int j = 0; j < P; ++j) c[i][j] = 0;
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          if (k >= a.K) break;
          if (AHEAD > 0) rows[k] = get((k + 1) * sb, nullptr, true);
          F2 f[P];
          PT::to(rows[k], f);
#pragma unroll
          for (int j = 0; j < P; ++j) c[i][j] = fma2(both(wk[k]), f[j], c[i][j]);
        }
      } else if (a.y) {
        PT::to(get(sb, a.y + row + at[i], in[i]), c[i]);
      } else {
        PT::to(res[i], c[i]);
      }
      if (a.add) {
        F2 f[P];
        PT::to(get(add_at, a.add + row + at[i], in[i]), f);
#pragma unroll
        for (int j = 0; j < P; ++j) c[i][j] = add2(c[i][j], f[j]);
      }
      if (a.gate)
        gate[i] = get(gate_at, a.gate + t / a.gate_tokens * a.row_bytes + at[i], in[i]);
      if (a.c && in[i]) st_vec(a.c + row + at[i], PT::from(c[i]));
#pragma unroll
      for (int j = 0; j < P; ++j) ss = fma2(c[i][j], c[i][j], ss);
      if (AHEAD > 0) fetch(t + static_cast<int64_t>(AHEAD) * a.units, i, stage + i * vector);
    }
    if (AHEAD > 0) {
      stage += token;
      if (stage == ring + AHEAD * token) stage = ring;
    }
    if (a.y) {
      float r = 1.0f;
      if (a.w_post) {
        r = 1.0f / sqrtf(team.sum(sum_of(ss)) * a.inv_h + a.eps);
        if (a.rstd_post && tid == 0) a.rstd_post[t] = r;
      }
      ss = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 f[P];
        if (a.w_post) {
          kept_weights<N>(wpost, wb, i, f);
#pragma unroll
          for (int j = 0; j < P; ++j) c[i][j] = mul2(mul2(c[i][j], both(r)), f[j]);
        }
        if (a.gate) {
          PT::to(gate[i], f);
#pragma unroll
          for (int j = 0; j < P; ++j) c[i][j] = mul2(c[i][j], f[j]);
        }
        PT::to(res[i], f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          c[i][j] = fma2(both(a.res_scale), f[j], c[i][j]);
          ss = fma2(c[i][j], c[i][j], ss);
        }
        if (in[i]) st_vec_cs(a.res_out + row + at[i], PT::from(c[i]));
      }
    }
    if (a.x) {
      const float r = 1.0f / sqrtf(team.sum(sum_of(ss)) * a.inv_h + a.eps);
      if (a.rstd_pre && tid == 0) a.rstd_pre[t] = r;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 f[P];
        kept_weights<N>(wpre, wb, i, f);
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = mul2(mul2(c[i][j], both(r)), f[j]);
        if (in[i]) st_vec_cs(a.x + row + at[i], PT::from(f));
      }
    }
    if (GATHER && AHEAD > 0) {
      count_weights(w_read);
      check_entries(p_read);
#pragma unroll
      for (int k = 0; k < KMAX; ++k) p[k] = p_read[k];
    }
  }
}

// ---------------------------------------------------------------------------
// backward

struct NormBwdArgs {
  const uint8_t* gres_out;  // [T, H] or NULL
  const uint8_t* gx;        // [T, H] or NULL
  const uint8_t* res_out;   // [T, H] (with gx)
  const uint8_t* c;         // [T, H] or NULL
  const uint8_t* gate;      // [groups, H] or NULL
  const uint8_t* w_post;    // [H] or NULL
  const uint8_t* w_pre;     // [H] (with gx)
  const float* rstd_post;
  const float* rstd_pre;
  uint8_t* gres;            // [T, H] or NULL
  uint8_t* gy;              // [T, H] or NULL
  uint8_t* ggate;           // [groups, H] or NULL
  float* gw_post;           // [H] or NULL
  float* gw_pre;            // [H] or NULL
  float* part;              // [2, blocks, H] column sums: post, pre
  float* slots;             // [2 * units, H] gate sums of groups that span units
  int64_t row_bytes;
  int T, H, nvec, gate_tokens, groups;
  int chunk, units, blocks; // tokens of a unit (a team), units, blocks
  int teams, team_threads;  // of a block; of a team
  int w_f32;
  float res_scale, offset, inv_h;
};

// Adds a thread's column sums to a row of fp32 sums (or writes them if they are
// the first) and clears them.
template <int V, int P>
__device__ __forceinline__ void flush_sums(F2 (&acc)[V][P], float* to, bool first, int tid,
                                           int step, int nvec) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * step;
#pragma unroll
    for (int j = 0; j < P; j += 2) {
      if (v < nvec) {
        float4* p = reinterpret_cast<float4*>(to + (v * P + j) * 2);
        float4 s{0.0f, 0.0f, 0.0f, 0.0f};
        if (!first) s = *p;
        const float2 x = split(acc[i][j]), y = split(acc[i][j + 1]);
        *p = make_float4(s.x + x.x, s.y + x.y, s.z + y.x, s.w + y.y);
      }
      acc[i][j] = acc[i][j + 1] = 0;
    }
  }
}

// What a backward kernel does about the gate: there is none; a row per token; a row
// per group of tokens.
enum GateKind { kNoGate, kGateRows, kGateGroups };

// A unit (a team) takes `chunk` tokens in a row and holds the column sums of the
// weights' gradients.  D = gres' + r_p (v - h mean(v h)), v = gx w_pre, h = res'
// r_p: the gradient of the residual sum; then the same form behind the gate for c.
// Where a gate row serves a group of tokens, one sum over the group, A = sum D c r_c,
// gives both gradients behind it, the gate's w_post A and w_post's gate A, and the
// row's product with w_post is kept for the group.
//
// AHEAD as in the forward.  With room for one token alone, its vectors are asked for
// in two parts, each as soon as that of the token before is used up (fp32 rows of
// 7168: 98.6 -> 65.6 us for 2048 tokens); with more, at the token's end (sooner,
// between its two sums, took 232 instead of 222 us at the DeepSeek-V3 shape).  -1: as
// 0, and the group's gate row, for which there is no room beside its product with
// w_post, is read again at the group's end (fp32 rows of more than 14336).
template <typename Elt, GateKind GATE, bool WARP, int MAXT, int AHEAD>
__global__ void __launch_bounds__(MAXT, 1) block_norm_bwd_kernel(NormBwdArgs a) {
  using PT = PairTraits<Elt>;
  constexpr int P = PT::P, N = 2 * P, V = kEpt / N, ROWS = GATE == kGateRows ? 5 : 4;
  constexpr bool PARTS = AHEAD == 1;
  constexpr bool KEPT_GATE = AHEAD >= 0;  // of a group
  enum { GRes, Gx, ResOut, C, Gate };
  __shared__ __align__(16) float red[kRed];
  extern __shared__ __align__(16) uint8_t shared[];
  grid_dependency_wait();
  Team<WARP, MAXT> team(a.team_threads, red);
  const int tid = team.tid, step = team.threads;
  const int unit = blockIdx.x * a.teams + team.index;
  const uint32_t sb = blockDim.x * 16, token = ROWS * V * sb, wb = step * 16;  // bytes
  const uint32_t wpost = smem_addr(shared) + tid * 16;
  const uint32_t wpre = wpost + kWeightSlots * wb;
  // of a group: the gate's row, and its product with w_post
  const uint32_t gate_row = smem_addr(shared) + threadIdx.x * 16 + 2 * kWeightSlots * wb;
  const uint32_t gate_w = gate_row + (KEPT_GATE ? V * sb : 0);
  const uint32_t ring = GATE == kGateGroups ? gate_w + kWeightSlots * sb : gate_row;
  bool in[V];    // vectors inside the row, and where
  int at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = tid + i * step < a.nvec;
    at[i] = in[i] ? (tid + i * step) * 16 : 0;
  }
  const int64_t begin64 = static_cast<int64_t>(unit) * a.chunk;
  const int begin = static_cast<int>(begin64 < a.T ? begin64 : a.T);
  const int end = static_cast<int>(begin64 + a.chunk < a.T ? begin64 + a.chunk : a.T);
  auto copy = [&](uint32_t to, int k, int i, const uint8_t* p, int64_t off) {
    copy_async(to + (k * V + i) * sb, p + off + at[i], in[i]);
  };
  // a token's rows of the residual stream and the norm, and those behind them
  auto fetch = [&](bool first, bool second, int64_t off, uint32_t to) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (first && a.gx) {
        copy(to, Gx, i, a.gx, off);
        copy(to, ResOut, i, a.res_out, off);
      }
      if (first && a.gres_out) copy(to, GRes, i, a.gres_out, off);
      if (second && a.c) copy(to, C, i, a.c, off);
      if (second && GATE == kGateRows) copy(to, Gate, i, a.gate, off);
    }
  };
  int64_t row = begin * a.row_bytes;
  float r_pre = a.gx && begin < end ? __ldg(a.rstd_pre + begin) : 0.0f;
  float r_post = a.w_post && begin < end ? __ldg(a.rstd_post + begin) : 1.0f;
  Weights<N> post, pre;
  if (team.index == 0) {
    post.load(a.w_post, a.w_f32, tid, step, a.nvec);
    pre.load(a.gx ? a.w_pre : nullptr, a.w_f32, tid, step, a.nvec);
  }
  if (AHEAD > 0)
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const bool real = n < end - begin;
      if (PARTS) {
        if (real) fetch(true, false, row, ring);
        commit_copies();
      }
      if (real) fetch(!PARTS, true, row + n * a.row_bytes, ring + n * token);
      commit_copies();
    }
  if (team.index == 0) {
    if (a.w_post) post.keep(a.w_f32, a.offset, wpost, wb, tid, step, a.nvec);
    if (a.gx) pre.keep(a.w_f32, a.offset, wpre, wb, tid, step, a.nvec);
  }
  __syncthreads();
  F2 gpost[V][P], gpre[V][P], A[V][P];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) gpost[i][j] = gpre[i][j] = A[i][j] = 0;
  // the block's rows of sums; a team adds to them when it has held kFlush tokens
  // and at the end, the teams in turn
  float* post_row = a.part + static_cast<size_t>(blockIdx.x) * a.H;
  float* pre_row = a.part + static_cast<size_t>(a.blocks + blockIdx.x) * a.H;
  // the token's group: its number and last token + 1
  int group = GATE == kGateGroups ? begin / a.gate_tokens : 0;
  int64_t group_end = (static_cast<int64_t>(group) + 1) * a.gate_tokens;
  bool enters = true, gate_first = true;
  int gate_held = 0;
  uint32_t stage = ring;
  // All teams of a block make the same number of rounds of kFlush tokens; behind
  // each they add their sums to the block's, one after the other.
  const int rounds = (a.chunk - 1) / kFlush + 1;
  for (int round = 0; round < rounds; ++round) {
    const int stop = static_cast<int>(
        min(static_cast<int64_t>(end), begin64 + (round + 1) * static_cast<int64_t>(kFlush)));
    for (int t = static_cast<int>(min(static_cast<int64_t>(end),
                                      begin64 + round * static_cast<int64_t>(kFlush)));
         t < stop; ++t, row += a.row_bytes) {
      auto load = [&](int k, int i, const uint8_t* p, F2* f) {
        Vec16 x{};
        if (AHEAD > 0) x = ld_shared(stage + (k * V + i) * sb);
        else if (in[i]) x = ld_vec(p + row + at[i]);
        PT::to(x, f);
      };
      const float rp = r_pre, r = r_post;
      if (t + 1 < end) {  // the next token's, a row's time ahead
        if (a.gx) r_pre = __ldg(a.rstd_pre + t + 1);
        if (a.w_post) r_post = __ldg(a.rstd_post + t + 1);
      }
      if constexpr (AHEAD > 0) wait_copies<PARTS ? 1 : AHEAD - 1>();
      F2 D[V][P], h[V][P];
      if (a.gx) {
        F2 s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          F2 w[P];
          load(Gx, i, a.gx, D[i]);
          load(ResOut, i, a.res_out, h[i]);
          kept_weights<N>(wpre, wb, i, w);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            h[i][j] = mul2(h[i][j], both(rp));
            gpre[i][j] = fma2(D[i][j], h[i][j], gpre[i][j]);
            D[i][j] = mul2(D[i][j], w[j]);
            s = fma2(D[i][j], h[i][j], s);
          }
        }
        const float m = team.sum(sum_of(s)) * a.inv_h;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          F2 g[P];
#pragma unroll
          for (int j = 0; j < P; ++j) g[j] = 0;
          if (a.gres_out) load(GRes, i, a.gres_out, g);
#pragma unroll
          for (int j = 0; j < P; ++j)
            D[i][j] = fma2(both(rp), fma2(both(-m), h[i][j], D[i][j]), g[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) load(GRes, i, a.gres_out, D[i]);
      }
      if (a.gres) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          F2 o[P];
#pragma unroll
          for (int j = 0; j < P; ++j) o[j] = mul2(both(a.res_scale), D[i][j]);
          if (in[i]) st_vec(a.gres + row + at[i], PT::from(o));
        }
      }
      if (PARTS) {
        if (end - t > 1) fetch(true, false, row + a.row_bytes, stage);
        commit_copies();
        wait_copies<1>();
      }
      if (GATE == kGateGroups && enters) {
        const uint8_t* p = a.gate + group * a.row_bytes;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          Vec16 x{};
          if (in[i]) {
            x = ld_vec(p + at[i]);
            if (group_end < end)  // the next group's, into L2
              asm volatile("prefetch.global.L2 [%0];" ::"l"(p + a.row_bytes + at[i]));
          }
          F2 g[P], w[P];
          PT::to(x, g);
          if (KEPT_GATE) st_shared(gate_row + i * sb, x);
          if (a.w_post) {
            kept_weights<N>(wpost, wb, i, w);
#pragma unroll
            for (int j = 0; j < P; ++j) g[j] = mul2(g[j], w[j]);
          }
#pragma unroll
          for (int q = 0; q < P / 2; ++q) {
            const float2 lo = split(g[2 * q]), hi = split(g[2 * q + 1]);
            st_shared(gate_w + (i * (P / 2) + q) * sb, make_float4(lo.x, lo.y, hi.x, hi.y));
          }
        }
        enters = false;
      }
      if (a.c) {
        F2 s = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          F2 w[P];
          load(C, i, a.c, h[i]);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            h[i][j] = mul2(h[i][j], both(r));
            w[j] = both(1.0f);
          }
          if (GATE == kGateGroups) {
            kept_weights<N>(gate_w, sb, i, w);
#pragma unroll
            for (int j = 0; j < P; ++j) A[i][j] = fma2(D[i][j], h[i][j], A[i][j]);
          } else {
            if (a.w_post) kept_weights<N>(wpost, wb, i, w);
            if (GATE == kGateRows) {
              F2 g[P], o[P];
              load(Gate, i, a.gate, g);
#pragma unroll
              for (int j = 0; j < P; ++j) {
                o[j] = mul2(D[i][j], mul2(h[i][j], w[j]));
                D[i][j] = mul2(D[i][j], g[j]);
              }
              if (a.ggate && in[i]) st_vec(a.ggate + row + at[i], PT::from(o));
            }
            if (a.w_post) {
#pragma unroll
              for (int j = 0; j < P; ++j) gpost[i][j] = fma2(D[i][j], h[i][j], gpost[i][j]);
            }
          }
          if (a.w_post || GATE == kGateGroups) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              D[i][j] = mul2(D[i][j], w[j]);
              s = fma2(D[i][j], h[i][j], s);
            }
          }
        }
        if (a.w_post) {
          const float m = team.sum(sum_of(s)) * a.inv_h;
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j)
              D[i][j] = mul2(both(r), fma2(both(-m), h[i][j], D[i][j]));
        }
      }
      if (a.gy) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (in[i]) st_vec(a.gy + row + at[i], PT::from(D[i]));
      }
      if constexpr (AHEAD > 0) {
        if (end - t > AHEAD) fetch(!PARTS, true, row + AHEAD * a.row_bytes, stage);
        commit_copies();
        stage += token;
        if (stage == ring + AHEAD * token) stage = ring;
      }
      if (GATE == kGateGroups) {
        const bool ends = t + 1 == group_end || t + 1 == a.T;
        if (ends || t + 1 == end || ++gate_held == kFlush) {
          const bool all = ends && group_end - a.gate_tokens >= begin;  // of the group's tokens
          float* slot = a.slots +
                        static_cast<size_t>(2 * unit + (group_end - a.gate_tokens >= begin)) * a.H;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (a.w_post) {
              F2 g[P], w[P];
              Vec16 x{};
              if (KEPT_GATE) x = ld_shared(gate_row + i * sb);
              else if (in[i]) x = ld_vec(a.gate + group * a.row_bytes + at[i]);
              PT::to(x, g);
              kept_weights<N>(wpost, wb, i, w);
#pragma unroll
              for (int j = 0; j < P; ++j) {
                gpost[i][j] = fma2(g[j], A[i][j], gpost[i][j]);
                A[i][j] = mul2(w[j], A[i][j]);
              }
            }
            if (all && a.ggate && in[i]) {
#pragma unroll
              for (int j = 0; j < P; ++j)
                if (!gate_first) {
                  const float2 x =
                      *reinterpret_cast<const float2*>(slot + ((tid + i * step) * P + j) * 2);
                  A[i][j] = add2(A[i][j], pair(x.x, x.y));
                }
              st_vec(a.ggate + group * a.row_bytes + at[i], PT::from(A[i]));
            }
          }
          if (!all && a.ggate) {
            flush_sums(A, slot, gate_first, tid, step, a.nvec);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
              for (int j = 0; j < P; ++j) A[i][j] = 0;
          }
          gate_first = ends;
          gate_held = 0;
          if (ends) {
            ++group;
            group_end += a.gate_tokens;
            enters = true;
          }
        }
      }
    }
    if (a.teams > 1 && round + 1 == rounds) break;
    for (int k = 0; k < a.teams; ++k) {
      if (k > 0) __syncthreads();
      if (k != team.index) continue;
      if (a.gw_post) flush_sums(gpost, post_row, round + k == 0, tid, step, a.nvec);
      if (a.gw_pre) flush_sums(gpre, pre_row, round + k == 0, tid, step, a.nvec);
    }
    if (a.teams > 1) __syncthreads();
  }
  if (a.teams == 1) return;
  // behind the last round the teams' sums meet in shared memory
  wait_copies<0>();
  auto meet = [&](const F2 (&acc)[V][P], float* to) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWeightSlots; ++q) {
      const float2 x = split(acc[q / (P / 2)][q % (P / 2) * 2]);
      const float2 y = split(acc[q / (P / 2)][q % (P / 2) * 2 + 1]);
      st_shared(ring + q * sb, make_float4(x.x, x.y, y.x, y.y));
    }
    __syncthreads();
    const uint32_t first = smem_addr(shared) + 2 * kWeightSlots * wb + (ring - gate_row);
    for (int n = threadIdx.x; n < kWeightSlots * step; n += blockDim.x) {
      const int q = n / step, thread = n - q * step;
      const int v = thread + q / (P / 2) * step;
      if (v >= a.nvec) continue;
      float4* p = reinterpret_cast<float4*>(to + v * N + q % (P / 2) * 4);
      float4 s{0.0f, 0.0f, 0.0f, 0.0f};
      if (rounds > 1) s = *p;
      for (int k = 0; k < a.teams; ++k) {
        const Vec16 x = ld_shared(first + q * sb + k * wb + thread * 16);
        s.x += __uint_as_float(x.u[0]);
        s.y += __uint_as_float(x.u[1]);
        s.z += __uint_as_float(x.u[2]);
        s.w += __uint_as_float(x.u[3]);
      }
      *p = s;
    }
  };
  if (a.gw_post) meet(gpost, post_row);
  if (a.gw_pre) meet(gpre, pre_row);
}

// Joins the units' column sums: row y = 0, 1 of the grid the weights' gradients,
// the rows behind them the gate's, an item for every `share` warps: item i is
// group i, or where there are more groups than units that which goes on from unit
// i into the next.  A group inside one unit is done.
template <typename Elt>
__global__ void __launch_bounds__(32 * kJoinWarps)
    block_norm_join_kernel(NormBwdArgs a, int items, int share) {
  grid_dependency_wait();
  __shared__ float2 ps[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kJoinCols + 2 * lane;
  const int y = blockIdx.y;
  const float* from = nullptr;
  float* out = nullptr;
  int u0 = 0, u1 = a.blocks, stride = 1, head = 0, group = -1;
  if (y < 2) {
    share = kJoinWarps;
    out = y == 0 ? a.gw_post : a.gw_pre;
    if (out) from = a.part + static_cast<size_t>(y) * a.blocks * a.H;
  } else {
    const int item = (y - 2) * (kJoinWarps / share) + warp / share;
    const int64_t next = (static_cast<int64_t>(item) + 1) * a.chunk;
    const bool by_unit = a.groups > a.units;
    if (item < items && !(by_unit && next >= a.T)) {
      group = by_unit ? static_cast<int>(next / a.gate_tokens) : item;
      const int64_t g0 = static_cast<int64_t>(group) * a.gate_tokens;
      const int64_t g1 = min(g0 + a.gate_tokens, static_cast<int64_t>(a.T));
      u0 = static_cast<int>(g0 / a.chunk);
      u1 = static_cast<int>((g1 - 1) / a.chunk) + 1;
      if (u1 - u0 > 1 && !(by_unit && u0 != item)) from = a.slots;
    }
    stride = 2;
    head = 1;
  }
  float2 p{0.0f, 0.0f};
  for (int ub = u0 + warp % share; ub < u1 && from && col < a.H; ub += kJoinLoads * share) {
    float2 x[kJoinLoads];
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {  // all on their way together
      const int u = ub + i * share;
      x[i] = make_float2(0.0f, 0.0f);
      if (u < u1)
        x[i] = __ldcg(reinterpret_cast<const float2*>(
            from + static_cast<size_t>(stride * u + (u == u0 ? head : 0)) * a.H + col));
    }
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      p.x += x[i].x;
      p.y += x[i].y;
    }
  }
  ps[warp][lane] = p;
  __syncthreads();
  if (!from || warp % share != 0 || col >= a.H) return;
#pragma unroll 4
  for (int w = 1; w < share; ++w) {
    p.x += ps[warp + w][lane].x;
    p.y += ps[warp + w][lane].y;
  }
  if (y < 2) {
    out[col] = p.x;
    out[col + 1] = p.y;
  } else {
    Elt* g = reinterpret_cast<Elt*>(a.ggate + group * a.row_bytes) + col;
    g[0] = static_cast<Elt>(p.x);
    g[1] = static_cast<Elt>(p.y);
  }
}

bool one_warp(int H) { return H <= kWarpRow; }

int team_threads(int H) { return H <= 128 ? 8 : H <= 256 ? 16 : (H + kWarpRow - 1) / kWarpRow * 32; }

// Teams of a block for T tokens: as many as it holds, once there is one for every SM.
int teams_of(int T, int H, int num_sms) {
  const int most = kTeamThreads / team_threads(H);
  int n = (T - 1) / num_sms + 1;
  n = most < 1 || n < 1 ? 1 : n < most ? n : most;
  const int per_warp = 32 / team_threads(H);  // whole warps
  return per_warp > 1 ? (n + per_warp - 1) / per_warp * per_warp : n;
}

// Resident blocks per SM of a forward kernel.  There are more kernels and sizes here
// than the table of resident_blocks() holds.
int forward_blocks(void (*kernel)(NormArgs), int threads, size_t shared) {
  struct Entry {
    void (*kernel)(NormArgs);
    int threads;
    size_t shared;
    int per_sm;
  };
  static Entry table[64];
  static int used = 0, next = 0;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (table[i].kernel == kernel && table[i].threads == threads && table[i].shared == shared)
      return table[i].per_sm;
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, shared) !=
          cudaSuccess ||
      per_sm < 1)
    per_sm = 1;
  table[next] = Entry{kernel, threads, shared, per_sm};
  next = (next + 1) % 64;
  if (used < 64) ++used;
  return per_sm;
}

// A kernel, the tokens that it has under way, and its shared memory.
template <typename A>
struct Chosen {
  void (*kernel)(A);
  int ahead;
  size_t shared;
};

size_t kept_bytes(int H, int weights) {
  return static_cast<size_t>(team_threads(H)) * 16 * kWeightSlots * weights;
}
// Shared memory of `rows` rows' vectors in a block of `threads`.
template <typename Elt>
size_t token_bytes(int threads, int rows) {
  return static_cast<size_t>(threads) * kEpt * sizeof(Elt) * rows;
}

// Kernels are made for rows of one warp, for those of up to 512 threads, where a block
// holds as many teams, and for wider ones, whose narrowest has 544.  With a class's
// most and least bytes of what a block keeps and of a token's rows, a kernel is left
// out where one with more tokens under way fits any of its rows, or where it fits none.
struct Bytes {
  size_t kept, token;
  constexpr bool fit(int tokens) const { return kept + tokens * token <= kShared; }
};
template <typename Elt>
constexpr Bytes class_bytes(int team, int threads, int weights, int rows, bool groups) {
  const size_t t = threads, row = kEpt * sizeof(Elt);
  return {static_cast<size_t>(team) * 16 * kWeightSlots * weights +
              (groups ? t * (row + kEpt * sizeof(float)) : 0),
          t * row * rows};
}
constexpr int kWideThreads = kTeamThreads + 32;

// The kernel with the most tokens under way, AHEAD at most, whose shared memory fits
// into `most`.
template <typename Elt, int KMAX, bool WARP, int MAXT, int AHEAD = KMAX == 1 && MAXT < 1024 ? 2 : 1>
Chosen<NormArgs> forward_within(size_t kept, size_t token, size_t most) {
  constexpr auto largest = class_bytes<Elt>(WARP ? 32 : MAXT, MAXT, 2, KMAX + 3, false);
  constexpr auto least =
      class_bytes<Elt>(0, MAXT == 1024 ? kWideThreads : 8, 0, KMAX == 16 ? 10 : 1, false);
  if constexpr (AHEAD == 0 || (AHEAD == 1 && largest.fit(1))) {
    return {block_norm_kernel<Elt, KMAX, WARP, MAXT, AHEAD>, AHEAD, kept + AHEAD * token};
  } else {
    if constexpr (least.fit(AHEAD))
      if (kept + AHEAD * token <= most)
        return {block_norm_kernel<Elt, KMAX, WARP, MAXT, AHEAD>, AHEAD, kept + AHEAD * token};
    return forward_within<Elt, KMAX, WARP, MAXT, AHEAD - 1>(kept, token, most);
  }
}
template <typename Elt, int KMAX>
Chosen<NormArgs> forward_kernel(int H, size_t kept, size_t token, size_t most) {
  return one_warp(H) ? forward_within<Elt, KMAX, true, kTeamThreads>(kept, token, most)
         : team_threads(H) <= kTeamThreads
             ? forward_within<Elt, KMAX, false, kTeamThreads>(kept, token, most)
             : forward_within<Elt, KMAX, false, 1024>(kept, token, most);
}
template <typename Elt>
Chosen<NormArgs> forward_kernel(int H, int kmax, int threads, int rows, int weights) {
  const size_t kept = kept_bytes(H, weights), token = token_bytes<Elt>(threads, rows);
  // two blocks an SM where their registers and one token ahead allow it
  const size_t half = kSmShared / 2 - 1024 - kRed * sizeof(float);
  const bool two = kmax == 1 && sizeof(Elt) == 2 && kept + token <= half;
  return kmax == 1   ? forward_kernel<Elt, 1>(H, kept, token, two ? half : kShared)
         : kmax == 8 ? forward_kernel<Elt, 8>(H, kept, token, kShared)
                     : forward_kernel<Elt, 16>(H, kept, token, kShared);
}

// `gate`: bytes of a group's gate row among `kept`; with them the widest rows need
// more than a block has, and do without.
template <typename Elt, GateKind GATE, bool WARP, int MAXT, int AHEAD = MAXT < 1024 ? 3 : 1>
Chosen<NormBwdArgs> backward_within(size_t kept, size_t gate, size_t token) {
  constexpr int rows = GATE == kGateRows ? 5 : 4;
  constexpr bool groups = GATE == kGateGroups;
  constexpr auto largest = class_bytes<Elt>(WARP ? 32 : MAXT, MAXT, 2, rows, groups);
  constexpr auto least = MAXT == 1024
                             ? class_bytes<Elt>(kWideThreads, kWideThreads, 2, rows, groups)
                             : class_bytes<Elt>(8, 8, 2, rows, groups);
  if constexpr (AHEAD < 0) {
    static_assert(groups && largest.kept - MAXT * kEpt * sizeof(Elt) <= kShared,
                  "both weights and the gate's product with one");
    return {block_norm_bwd_kernel<Elt, GATE, WARP, MAXT, AHEAD>, AHEAD, kept - gate};
  } else if constexpr (largest.fit(AHEAD)) {
    return {block_norm_bwd_kernel<Elt, GATE, WARP, MAXT, AHEAD>, AHEAD, kept + AHEAD * token};
  } else {
    if constexpr (least.fit(AHEAD))
      if (kept + AHEAD * token <= kShared)
        return {block_norm_bwd_kernel<Elt, GATE, WARP, MAXT, AHEAD>, AHEAD, kept + AHEAD * token};
    return backward_within<Elt, GATE, WARP, MAXT, AHEAD - 1>(kept, gate, token);
  }
}
template <typename Elt, GateKind GATE>
Chosen<NormBwdArgs> backward_fitting(int H, size_t kept, size_t gate, size_t token) {
  return one_warp(H) ? backward_within<Elt, GATE, true, kTeamThreads>(kept, gate, token)
         : team_threads(H) <= kTeamThreads
             ? backward_within<Elt, GATE, false, kTeamThreads>(kept, gate, token)
             : backward_within<Elt, GATE, false, 1024>(kept, gate, token);
}
template <typename Elt, GateKind GATE>
Chosen<NormBwdArgs> backward_kernel(int H, int threads) {
  size_t kept = kept_bytes(H, 2);
  const size_t row = GATE == kGateGroups ? token_bytes<Elt>(threads, 1) : 0;
  if (GATE == kGateGroups)  // a gate row and 16 fp32 a thread
    kept += row + static_cast<size_t>(threads) * kEpt * sizeof(float);
  auto c = backward_fitting<Elt, GATE>(
      H, kept, row, token_bytes<Elt>(threads, GATE == kGateRows ? 5 : 4));
  // the teams' sums meet there as well
  const size_t meet = kept + static_cast<size_t>(threads) * kEpt * sizeof(float);
  if (threads > team_threads(H) && c.shared < meet) c.shared = meet;
  return c;
}
template <typename Elt>
Chosen<NormBwdArgs> backward_kernel(GateKind gate, int H, int threads) {
  return gate == kNoGate     ? backward_kernel<Elt, kNoGate>(H, threads)
         : gate == kGateRows ? backward_kernel<Elt, kGateRows>(H, threads)
                             : backward_kernel<Elt, kGateGroups>(H, threads);
}

// Units of the backward for T tokens, at least: the workspace of T serves fewer.
int units_of(int T, int H, int num_sms, int* teams) {
  *teams = teams_of(T, H, num_sms);
  const int blocks = (T - 1) / *teams + 1;
  return *teams * (blocks < num_sms ? blocks : num_sms);
}
}  // namespace

size_t block_norm_workspace(const moe_handle* h, int T, int H, int gate_tokens) {
  int teams;
  const size_t units = units_of(T, H, h->num_sms, &teams);
  const size_t blocks = T < 1 ? 1 : T < h->num_sms ? T : h->num_sms;
  return (2 * blocks + (gate_tokens > 1 ? 2 * units : 0)) * H * sizeof(float);
}

cudaError_t launch_block_norm(const moe_handle* h, const moe_block_norm_args& q, int T,
                              cudaStream_t s) {
  NormArgs a{};
  a.y = static_cast<const uint8_t*>(q.d_y);
  a.pos = q.gather ? h->pos : nullptr;
  a.cw = q.d_cw;
  a.add = static_cast<const uint8_t*>(q.d_add);
  a.res = static_cast<const uint8_t*>(q.d_res);
  a.gate = static_cast<const uint8_t*>(q.d_gate);
  a.w_post = static_cast<const uint8_t*>(q.d_w_post);
  a.w_pre = static_cast<const uint8_t*>(q.d_w_pre);
  a.c = static_cast<uint8_t*>(q.d_c);
  a.res_out = static_cast<uint8_t*>(q.d_res_out);
  a.x = static_cast<uint8_t*>(q.d_x);
  a.rstd_post = q.d_rstd_post;
  a.rstd_pre = q.d_rstd_pre;
  const bool bf16 = q.dtype == MOE_BF16;
  a.row_bytes = static_cast<int64_t>(q.H) * (bf16 ? 2 : 4);
  a.T = T;
  a.H = q.H;
  a.nvec = static_cast<int>(a.row_bytes / 16);
  a.K = h->cfg.top_k;
  a.rows = h->T * h->cfg.top_k + h->cfg.num_experts * (h->pad - 1);
  a.gate_tokens = q.gate_tokens;
  a.w_f32 = q.weight_dtype == MOE_F32;
  a.res_scale = static_cast<float>(q.res_scale);
  a.eps = static_cast<float>(q.eps);
  a.offset = static_cast<float>(q.weight_offset);
  a.inv_h = 1.0f / q.H;
  a.flags = h->flags;
  if (T == 0) return cudaSuccess;
  if (!q.gather) a.K = 1;
  a.teams = teams_of(T, q.H, h->num_sms);
  a.team_threads = team_threads(q.H);
  const int threads = a.teams * a.team_threads;
  const int kmax = !q.gather ? 1 : a.K <= 8 ? 8 : 16;
  const int rows = 1 + (a.y ? a.K : 0) + (a.add != nullptr) + (a.gate != nullptr);
  const int weights = (a.w_post != nullptr) + (a.w_pre != nullptr);
  const auto c = bf16 ? forward_kernel<__nv_bfloat16>(q.H, kmax, threads, rows, weights)
                      : forward_kernel<float>(q.H, kmax, threads, rows, weights);
  const cudaError_t e =
      allow_shared_at_launch(h, reinterpret_cast<const void*>(c.kernel), kShared);
  if (e != cudaSuccess) return e;
  const long long most =
      static_cast<long long>(h->num_sms) * forward_blocks(c.kernel, threads, c.shared);
  const int blocks = (T - 1) / a.teams + 1;
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  a.units = grid * a.teams;
  return launch_chained(c.kernel, dim3(grid), dim3(threads), c.shared, s, false, a);
}

cudaError_t launch_block_norm_bwd(const moe_handle* h, const moe_block_norm_bwd_args& q, int T,
                                  void* workspace, cudaStream_t s) {
  NormBwdArgs a{};
  a.gres_out = static_cast<const uint8_t*>(q.d_gres_out);
  a.gx = static_cast<const uint8_t*>(q.d_gx);
  a.res_out = static_cast<const uint8_t*>(q.d_res_out);
  if (q.d_gate || q.d_w_post) a.c = static_cast<const uint8_t*>(q.d_c);
  a.gate = static_cast<const uint8_t*>(q.d_gate);
  a.w_post = static_cast<const uint8_t*>(q.d_w_post);
  a.w_pre = static_cast<const uint8_t*>(q.d_w_pre);
  a.rstd_post = q.d_rstd_post;
  a.rstd_pre = q.d_rstd_pre;
  a.gres = static_cast<uint8_t*>(q.d_gres);
  a.gy = static_cast<uint8_t*>(q.d_gy);
  a.ggate = static_cast<uint8_t*>(q.d_ggate);
  a.gw_post = q.d_gw_post;
  a.gw_pre = q.d_gw_pre;
  const bool bf16 = q.dtype == MOE_BF16;
  a.row_bytes = static_cast<int64_t>(q.H) * (bf16 ? 2 : 4);
  a.T = T;
  a.H = q.H;
  a.nvec = static_cast<int>(a.row_bytes / 16);
  a.gate_tokens = q.gate_tokens;
  a.groups = T > 0 ? (T - 1) / q.gate_tokens + 1 : 0;
  a.w_f32 = q.weight_dtype == MOE_F32;
  a.res_scale = static_cast<float>(q.res_scale);
  a.offset = static_cast<float>(q.weight_offset);
  a.inv_h = 1.0f / q.H;
  a.units = units_of(T, q.H, h->num_sms, &a.teams);
  a.chunk = T > 0 ? (T - 1) / a.units + 1 : 1;
  // whole groups, where that leaves at most a fifth of the teams without work: none
  // of them has to be joined then
  const int64_t whole = (static_cast<int64_t>(a.chunk - 1) / q.gate_tokens + 1) * q.gate_tokens;
  if (whole * 4 <= static_cast<int64_t>(a.chunk) * 5) a.chunk = static_cast<int>(whole);
  a.blocks = a.units / a.teams;
  a.team_threads = team_threads(q.H);
  a.part = static_cast<float*>(workspace);
  a.slots = a.part + 2 * static_cast<size_t>(a.blocks) * q.H;
  const int threads = a.teams * a.team_threads;
  const GateKind gate = !q.d_gate ? kNoGate : q.gate_tokens == 1 ? kGateRows : kGateGroups;
  const auto k = bf16 ? backward_kernel<__nv_bfloat16>(gate, q.H, threads)
                      : backward_kernel<float>(gate, q.H, threads);
  if (T > 0) {
    cudaError_t e = allow_shared_at_launch(h, reinterpret_cast<const void*>(k.kernel), kShared);
    if (e == cudaSuccess)
      e = launch_chained(k.kernel, dim3(a.blocks), dim3(threads), k.shared, s, false, a);
    if (e != cudaSuccess) return e;
  }
  const bool spans = a.ggate && a.gate_tokens > 1 && a.chunk % a.gate_tokens != 0;
  if (!a.gw_post && !a.gw_pre && !spans) return cudaSuccess;
  const int items = !spans ? 0 : a.groups < a.units ? a.groups : a.units;
  int share = 1;  // warps of an item: eight slots each
  while (share < kJoinWarps && 8 * share * static_cast<int64_t>(a.chunk) < a.gate_tokens) share *= 2;
  const int rows = 2 + (items * share + kJoinWarps - 1) / kJoinWarps;
  if (T == 0) a.blocks = 0;  // sums of nothing
  return launch_chained(bf16 ? block_norm_join_kernel<__nv_bfloat16> : block_norm_join_kernel<float>,
                        dim3((q.H + kJoinCols - 1) / kJoinCols, rows), dim3(32 * kJoinWarps), 0, s,
                        false, a, items, share);
}

}  // namespace moe
