// The norms around a block (sm_103a): the block's output rows, or the weighted
// sum of their receive rows, normed, gated and added to the residual stream, and
// the next block's norm of that sum; and the backward.
//
//   c = y + add                      (y: token rows, or sum_k w_k y[pos[t,k]])
//   res' = res_scale * res + gate * (c r_c (w_post + offset))
//   x    = res' r_p (w_pre + offset),    r_v = 1 / sqrt(mean(v^2) + eps)
//
// One pass over the rows: a team of threads (a warp, or a block) holds a row in
// registers, 16 elements a thread, and the two sums of squares are its only
// exchange.  x is made from the sum before that is rounded; sums are fp32, each
// output is rounded once.
//
// Bound by HBM; what stands in its way are the two sums in a row's chain.  Each
// thread therefore copies the vectors that it will need itself into shared memory
// ahead of time (cp.async: no other thread waits for them), so loads go on while
// the team waits for its sums, and its weights, in fp32 with their offset, stay
// there too.  Arithmetic is on pairs of fp32 (one instruction for both), which
// halves what the issue slots have to do: without it the backward took 52
// instructions an element and ran at half of the copy rate.
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kEpt = 16;           // elements of a row a thread holds
constexpr int kWarpRow = 32 * kEpt;  // widest row of a one-warp team
constexpr int kTeams = 4;          // one-warp teams of a block
// Tokens whose column sums are added up in registers before they go to memory:
// bounds the number of fp32 additions in a row for any T.
constexpr int kFlush = 1024;
constexpr size_t kShared = 226 * 1024;  // dynamic shared memory of a block, at most
constexpr size_t kSmShared = 228 * 1024, kBlockShared = 1024 + 512;  // of an SM; a block's own share

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
__device__ __forceinline__ void st_shared(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// A thread's shared memory is its own slots of 16 bytes, `sb` = 16 times the
// block's threads from one to the next: the copies of a warp land side by side.
// (Slots of a thread one behind another, with addresses known when compiled, took
// the backward from 302 to 372 us at the DeepSeek-V3 shape.)
constexpr int kWeightSlots = kEpt / 4;  // 16 fp32

// Keeps the thread's 16 weights of w from `to` on, zero behind the row's end;
// its vectors of N elements are tid, tid + threads, ...
template <int N>
__device__ __forceinline__ void keep_weights(const uint8_t* w, int f32, float offset, uint32_t to,
                                             uint32_t sb, int tid, int threads, int nvec) {
#pragma unroll
  for (int q = 0; q < kWeightSlots; ++q) {
    const int v = tid + q / (N / 4) * threads;
    float4 f{0.0f, 0.0f, 0.0f, 0.0f};
    if (v < nvec) {
      const int at = v * (N / 4) + q % (N / 4);
      if (f32) {
        f = __ldg(reinterpret_cast<const float4*>(w) + at);
      } else {
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(w) + at);
        f = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                        __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
      }
      f = make_float4(f.x + offset, f.y + offset, f.z + offset, f.w + offset);
    }
    st_shared(to + q * sb, f);
  }
}
// The weights of the thread's vector i.
template <int N>
__device__ __forceinline__ void kept_weights(uint32_t at, uint32_t sb, int i, F2* f) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const Vec16 v = ld_shared(at + (i * (N / 4) + q) * sb);
    f[2 * q] = pair(__uint_as_float(v.u[0]), __uint_as_float(v.u[1]));
    f[2 * q + 1] = pair(__uint_as_float(v.u[2]), __uint_as_float(v.u[3]));
  }
}

// Sum over the team: a warp, or the block, whose warps hand over through `red`
// (two sets of 32 values, taken in turn, so that one barrier a sum is enough;
// zero behind the last warp's, so that they can be read four at a time).
template <bool WARP>
__device__ __forceinline__ float team_sum(float v, float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if constexpr (WARP) return v;
  const int warps = blockDim.x >> 5;
  float* set = red + turn;
  turn ^= 32;
  if ((threadIdx.x & 31) == 0) set[threadIdx.x >> 5] = v;
  __syncthreads();
  float4 a = *reinterpret_cast<const float4*>(set);
  for (int w = 4; w < warps; w += 4) {
    const float4 b = *reinterpret_cast<const float4*>(set + w);
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  }
  return (a.x + a.y) + (a.z + a.w);
}
template <bool WARP>
__device__ __forceinline__ void clear_sums(float* red) {
  if constexpr (!WARP) {
    for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i] = 0.0f;
    __syncthreads();
  }
}

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
  int w_f32;             // weights in fp32 (else bf16)
  float res_scale, eps, offset, inv_h;
  uint32_t* flags;
};

// A team takes every units-th token, a vector a thread of all its rows at a time.
// AHEAD: tokens whose vectors are in shared memory or on their way there (0: they
// are loaded when they are needed).  KMAX: rows that are summed at most (1: token
// rows).
template <int KMAX>
struct NormSlots {  // of one vector's rows
  static constexpr int Res = KMAX, Add = KMAX + 1, Gate = KMAX + 2, Count = KMAX + 3;
};

template <typename Elt, int KMAX, int AHEAD>
constexpr int forward_slots() {
  constexpr int V = kEpt / (2 * PairTraits<Elt>::P);
  return 2 * kWeightSlots + AHEAD * V * NormSlots<KMAX>::Count;
}

template <typename Elt, int KMAX, bool WARP, int MAXT, int AHEAD>
__global__ void __launch_bounds__(MAXT, 1) block_norm_kernel(NormArgs a) {
  using PT = PairTraits<Elt>;
  using Slot = NormSlots<KMAX>;
  constexpr int P = PT::P, N = 2 * P, V = kEpt / N;
  constexpr bool GATHER = KMAX > 1;
  const uint32_t sb = blockDim.x * 16;
  const uint32_t vector = Slot::Count * sb, token = V * vector;  // bytes
  static_assert(!GATHER || AHEAD < 2, "a token's weights are asked for one token ahead");
  __shared__ __align__(16) float red[64];
  extern __shared__ __align__(16) uint8_t own[];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int unit = WARP ? blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (unit >= a.units) return;  // a warp's; a block is always a unit
  const uint32_t wpost = smem_addr(own) + threadIdx.x * 16;
  const uint32_t wpre = wpost + kWeightSlots * sb;
  const uint32_t ring = wpre + kWeightSlots * sb;
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
      copy_async(to + Slot::Res * sb, a.res + off, in[i]);
      if (GATHER) {
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          if (k >= a.K) break;
          const bool real = in[i] && p[k] >= 0;
          copy_async(to + k * sb, a.y + (real ? p[k] * a.row_bytes + at[i] : 0), real);
        }
      } else if (a.y) {
        copy_async(to, a.y + off, in[i]);
      }
      if (a.add) copy_async(to + Slot::Add * sb, a.add + off, in[i]);
      if (a.gate)
        copy_async(to + Slot::Gate * sb,
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
  if (a.w_post) keep_weights<N>(a.w_post, a.w_f32, a.offset, wpost, sb, tid, step, a.nvec);
  if (a.w_pre) keep_weights<N>(a.w_pre, a.w_f32, a.offset, wpre, sb, tid, step, a.nvec);
  clear_sums<WARP>(red);
  int turn = 0;
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
      auto get = [&](int slot, const uint8_t* g, bool real) {
        Vec16 x{};
        if (AHEAD > 0) x = ld_shared(from + slot * sb);
        else if (real) x = ld_vec(g);
        return x;
      };
      res[i] = get(Slot::Res, a.res + row + at[i], in[i]);
      if (GATHER) {
        Vec16 rows[KMAX];
        if (AHEAD == 0)
#pragma unroll
          for (int k = 0; k < KMAX; ++k)
            rows[k] = get(k, a.y + p[k] * a.row_bytes + at[i], in[i] && p[k] >= 0);
#pragma unroll
        for (int j = 0; j < P; ++j) c[i][j] = 0;
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          if (k >= a.K) break;
          if (AHEAD > 0) rows[k] = get(k, nullptr, true);
          F2 f[P];
          PT::to(rows[k], f);
#pragma unroll
          for (int j = 0; j < P; ++j) c[i][j] = fma2(both(wk[k]), f[j], c[i][j]);
        }
      } else if (a.y) {
        PT::to(get(0, a.y + row + at[i], in[i]), c[i]);
      } else {
        PT::to(res[i], c[i]);
      }
      if (a.add) {
        F2 f[P];
        PT::to(get(Slot::Add, a.add + row + at[i], in[i]), f);
#pragma unroll
        for (int j = 0; j < P; ++j) c[i][j] = add2(c[i][j], f[j]);
      }
      if (a.gate)
        gate[i] = get(Slot::Gate, a.gate + t / a.gate_tokens * a.row_bytes + at[i], in[i]);
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
        r = 1.0f / sqrtf(team_sum<WARP>(sum_of(ss), red, turn) * a.inv_h + a.eps);
        if (a.rstd_post && tid == 0) a.rstd_post[t] = r;
      }
      ss = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 f[P];
        if (a.w_post) {
          kept_weights<N>(wpost, sb, i, f);
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
        if (in[i]) st_vec(a.res_out + row + at[i], PT::from(c[i]));
      }
    }
    if (a.x) {
      const float r = 1.0f / sqrtf(team_sum<WARP>(sum_of(ss), red, turn) * a.inv_h + a.eps);
      if (a.rstd_pre && tid == 0) a.rstd_pre[t] = r;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 f[P];
        kept_weights<N>(wpre, sb, i, f);
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = mul2(mul2(c[i][j], both(r)), f[j]);
        if (in[i]) st_vec(a.x + row + at[i], PT::from(f));
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

// A unit (a team) takes `chunk` tokens in a row and holds the column sums of the
// weights' gradients, and of the gate's while the tokens of its group last.
// D = gres' + r_p (v - h mean(v h)), v = gx w_pre, h = res' r_p: the gradient of
// the residual sum; then the same form behind the gate for c.  AHEAD as in the
// forward.
template <typename Elt, bool GATE, int AHEAD>
constexpr int backward_slots() {
  constexpr int V = kEpt / (2 * PairTraits<Elt>::P);
  return 2 * kWeightSlots + AHEAD * V * (GATE ? 5 : 4);
}

template <typename Elt, bool GATE, bool WARP, int MAXT, int AHEAD>
__global__ void __launch_bounds__(MAXT, 1) block_norm_bwd_kernel(NormBwdArgs a) {
  using PT = PairTraits<Elt>;
  constexpr int P = PT::P, N = 2 * P, V = kEpt / N, ROWS = GATE ? 5 : 4;
  const uint32_t sb = blockDim.x * 16, token = ROWS * V * sb;  // bytes
  enum { GRes, Gx, ResOut, C, Gate };
  __shared__ __align__(16) float red[64];
  extern __shared__ __align__(16) uint8_t own[];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int unit = WARP ? blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (unit >= a.units) return;  // a warp's; a block is always a unit
  const uint32_t wpost = smem_addr(own) + threadIdx.x * 16;
  const uint32_t wpre = wpost + kWeightSlots * sb;
  const uint32_t ring = wpre + kWeightSlots * sb;
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
  // the gate's row of a token, for tokens in order: its offset and last token + 1
  struct Group {
    int64_t row, end;
  };
  auto group_of = [&](int t) {
    const int64_t g = t / a.gate_tokens;
    return Group{g * a.row_bytes, (g + 1) * a.gate_tokens};
  };
  Group asked = GATE ? group_of(begin) : Group{0, 0}, group = asked;
  int64_t off = begin * a.row_bytes;  // of the row asked for next
  int next = begin;
  auto fetch = [&](uint32_t to) {
    if (next < end) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        auto copy = [&](int k, const uint8_t* p, int64_t o) {
          copy_async(to + (k * V + i) * sb, p + o + at[i], in[i]);
        };
        if (a.gx) {
          copy(Gx, a.gx, off);
          copy(ResOut, a.res_out, off);
        }
        if (a.gres_out) copy(GRes, a.gres_out, off);
        if (a.c) copy(C, a.c, off);
        if (GATE) copy(Gate, a.gate, asked.row);
      }
      off += a.row_bytes;
      ++next;
      if (GATE && next == asked.end) {
        asked.row += a.row_bytes;
        asked.end += a.gate_tokens;
      }
    }
    commit_copies();
  };
  if (AHEAD > 0)
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) fetch(ring + n * token);
  float r_pre = a.gx && begin < end ? __ldg(a.rstd_pre + begin) : 0.0f;
  float r_post = a.w_post && begin < end ? __ldg(a.rstd_post + begin) : 1.0f;
  if (a.w_post) keep_weights<N>(a.w_post, a.w_f32, a.offset, wpost, sb, tid, step, a.nvec);
  if (a.gx) keep_weights<N>(a.w_pre, a.w_f32, a.offset, wpre, sb, tid, step, a.nvec);
  clear_sums<WARP>(red);
  F2 gpost[V][P], gpre[V][P], ggate[V][P];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) gpost[i][j] = gpre[i][j] = ggate[i][j] = 0;
  float* post_row = a.part + static_cast<size_t>(unit) * a.H;
  float* pre_row = a.part + static_cast<size_t>(a.units + unit) * a.H;
  bool first = true, gate_first = true;
  int held = 0, gate_held = 0, turn = 0;
  uint32_t stage = ring;
  int64_t row = begin * a.row_bytes;
  for (int t = begin; t < end; ++t, row += a.row_bytes) {
    auto load = [&](int k, int i, const uint8_t* p, int64_t o, F2* f) {
      Vec16 x{};
      if (AHEAD > 0) x = ld_shared(stage + (k * V + i) * sb);
      else if (in[i]) x = ld_vec(p + o + at[i]);
      PT::to(x, f);
    };
    const float rp = r_pre, r = r_post;
    if (t + 1 < end) {  // the next token's, a row's time ahead
      if (a.gx) r_pre = __ldg(a.rstd_pre + t + 1);
      if (a.w_post) r_post = __ldg(a.rstd_post + t + 1);
    }
    if (AHEAD > 0) wait_copies<AHEAD - 1>();
    F2 D[V][P], h[V][P];
    if (a.gx) {
      F2 s = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 w[P];
        load(Gx, i, a.gx, row, D[i]);
        load(ResOut, i, a.res_out, row, h[i]);
        kept_weights<N>(wpre, sb, i, w);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          h[i][j] = mul2(h[i][j], both(rp));
          gpre[i][j] = fma2(D[i][j], h[i][j], gpre[i][j]);
          D[i][j] = mul2(D[i][j], w[j]);
          s = fma2(D[i][j], h[i][j], s);
        }
      }
      const float m = team_sum<WARP>(sum_of(s), red, turn) * a.inv_h;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 g[P];
#pragma unroll
        for (int j = 0; j < P; ++j) g[j] = 0;
        if (a.gres_out) load(GRes, i, a.gres_out, row, g);
#pragma unroll
        for (int j = 0; j < P; ++j)
          D[i][j] = fma2(both(rp), fma2(both(-m), h[i][j], D[i][j]), g[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) load(GRes, i, a.gres_out, row, D[i]);
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
    if (a.c) {
      F2 s = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        F2 w[P];
        load(C, i, a.c, row, h[i]);
#pragma unroll
        for (int j = 0; j < P; ++j) h[i][j] = mul2(h[i][j], both(r));
        if (a.w_post) kept_weights<N>(wpost, sb, i, w);
        if (GATE) {
          F2 g[P];
          load(Gate, i, a.gate, group.row, g);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            ggate[i][j] = fma2(D[i][j], a.w_post ? mul2(h[i][j], w[j]) : h[i][j], ggate[i][j]);
            D[i][j] = mul2(D[i][j], g[j]);
          }
        }
        if (a.w_post) {
#pragma unroll
          for (int j = 0; j < P; ++j) {
            gpost[i][j] = fma2(D[i][j], h[i][j], gpost[i][j]);
            D[i][j] = mul2(D[i][j], w[j]);
            s = fma2(D[i][j], h[i][j], s);
          }
        }
      }
      if (a.w_post) {
        const float m = team_sum<WARP>(sum_of(s), red, turn) * a.inv_h;
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
    if (AHEAD > 0) {
      fetch(stage);
      stage += token;
      if (stage == ring + AHEAD * token) stage = ring;
    }
    if (GATE) {
      const int64_t g0 = group.end - a.gate_tokens;
      const bool ends = t + 1 == group.end || t + 1 == a.T;
      if (a.ggate) {
        float* slot = a.slots + static_cast<size_t>(2 * unit + (g0 >= begin)) * a.H;
        if (ends && g0 >= begin) {  // all of the group's tokens
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (in[i]) {
#pragma unroll
              for (int j = 0; j < P; ++j)
                if (!gate_first) {
                  const float2 x =
                      *reinterpret_cast<const float2*>(slot + ((tid + i * step) * P + j) * 2);
                  ggate[i][j] = add2(ggate[i][j], pair(x.x, x.y));
                }
              st_vec(a.ggate + group.row + at[i], PT::from(ggate[i]));
            }
#pragma unroll
            for (int j = 0; j < P; ++j) ggate[i][j] = 0;
          }
          gate_first = true;
          gate_held = 0;
        } else if (ends || t + 1 == end || ++gate_held == kFlush) {
          flush_sums(ggate, slot, gate_first, tid, step, a.nvec);
          gate_first = ends;
          gate_held = 0;
        }
      }
      if (ends) {
        group.row += a.row_bytes;
        group.end += a.gate_tokens;
      }
    }
    if (++held == kFlush) {
      if (a.gw_post) flush_sums(gpost, post_row, first, tid, step, a.nvec);
      if (a.gw_pre) flush_sums(gpre, pre_row, first, tid, step, a.nvec);
      first = false;
      held = 0;
    }
  }
  if (a.gw_post) flush_sums(gpost, post_row, first, tid, step, a.nvec);
  if (a.gw_pre) flush_sums(gpre, pre_row, first, tid, step, a.nvec);
}

// Joins the units' column sums: row y = 0, 1 of the grid the weights'
// gradients; row 2 + i the gate's of group i, or where there are more groups than
// units of the one that goes on from unit i into the next; a group inside one
// unit is done.
template <typename Elt>
__global__ void __launch_bounds__(1024) block_norm_join_kernel(NormBwdArgs a) {
  grid_dependency_wait();
  __shared__ float ps[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int y = blockIdx.y;
  float* out = nullptr;
  const float* from = a.part;
  int u0 = 0, u1 = a.units, stride = 1, head = 0;
  int group = 0;
  if (y < 2) {
    out = y == 0 ? a.gw_post : a.gw_pre;
    from += static_cast<size_t>(y) * a.units * a.H;
    if (!out) return;
  } else {
    const int64_t next = (static_cast<int64_t>(y - 2) + 1) * a.chunk;
    if (a.groups > a.units && next >= a.T) return;
    group = a.groups > a.units ? static_cast<int>(next / a.gate_tokens) : y - 2;
    const int64_t g0 = static_cast<int64_t>(group) * a.gate_tokens;
    const int64_t g1 = min(g0 + a.gate_tokens, static_cast<int64_t>(a.T));
    u0 = static_cast<int>(g0 / a.chunk);
    u1 = static_cast<int>((g1 - 1) / a.chunk) + 1;
    if (u1 - u0 < 2 || (a.groups > a.units && u0 != y - 2)) return;
    from = a.slots;
    stride = 2;
    head = 1;
  }
  float p = 0.0f;
  if (col < a.H)
#pragma unroll 4
    for (int u = u0 + warp; u < u1; u += warps)
      p += __ldcg(from + static_cast<size_t>(stride * u + (u == u0 ? head : 0)) * a.H + col);
  ps[warp][lane] = p;
  __syncthreads();
  if (warp != 0 || col >= a.H) return;
  for (int w = 1; w < warps; ++w) p += ps[w][lane];
  if (y < 2)
    out[col] = p;
  else
    reinterpret_cast<Elt*>(a.ggate + group * a.row_bytes)[col] = static_cast<Elt>(p);
}

bool one_warp(int H) { return H <= kWarpRow; }

int team_threads(int H) { return (H + kWarpRow - 1) / kWarpRow * 32; }

// Tokens of a unit and units of the backward: as many threads an SM as its
// registers hold.
int bwd_units_per_sm(int H) {
  return one_warp(H) ? 16 : 512 / team_threads(H) < 1 ? 1 : 512 / team_threads(H);
}

void bwd_units(int T, int H, int num_sms, int* chunk, int* units) {
  const int most = bwd_units_per_sm(H) * num_sms;
  int n = T < most ? T : most;
  if (n < 1) n = 1;
  *chunk = (T + n - 1) / n;
  if (*chunk < 1) *chunk = 1;
  n = (T + *chunk - 1) / *chunk;
  if (n < 1) n = 1;
  *units = n;
}

// Largest dynamic shared memory for a kernel that takes more than the default.
template <typename K>
cudaError_t allow_shared(K k) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kShared));
}

// A kernel, the tokens that it has under way, and its shared memory.
template <typename A>
struct Chosen {
  void (*kernel)(A);
  int ahead;
  size_t shared;
};

template <typename Elt, int KMAX, bool WARP, int MAXT, int AHEAD>
Chosen<NormArgs> forward(int threads) {
  return {block_norm_kernel<Elt, KMAX, WARP, MAXT, AHEAD>, AHEAD,
          static_cast<size_t>(threads) * forward_slots<Elt, KMAX, AHEAD>() * 16};
}

// The kernel with the most tokens under way whose shared memory fits into `most`.
template <typename Elt, int KMAX, bool WARP, int MAXT>
Chosen<NormArgs> forward_within(int threads, size_t most) {
  if constexpr (KMAX == 1 && MAXT < 1024) {
    const auto two = forward<Elt, KMAX, WARP, MAXT, 2>(threads);
    if (two.shared <= most) return two;
  }
  const auto one = forward<Elt, KMAX, WARP, MAXT, 1>(threads);
  return one.shared <= most ? one : forward<Elt, KMAX, WARP, MAXT, 0>(threads);
}
template <typename Elt, int KMAX>
Chosen<NormArgs> forward_kernel(int H, int threads, size_t most) {
  return one_warp(H)      ? forward_within<Elt, KMAX, true, 32 * kTeams>(threads, most)
         : threads <= 512 ? forward_within<Elt, KMAX, false, 512>(threads, most)
                          : forward_within<Elt, KMAX, false, 1024>(threads, most);
}
template <typename Elt>
Chosen<NormArgs> forward_kernel(int kmax, int H, int threads, size_t most) {
  return kmax == 1   ? forward_kernel<Elt, 1>(H, threads, most)
         : kmax == 8 ? forward_kernel<Elt, 8>(H, threads, most)
                     : forward_kernel<Elt, 16>(H, threads, most);
}

template <typename Elt, bool GATE, bool WARP, int MAXT, int AHEAD>
Chosen<NormBwdArgs> backward(int threads) {
  return {block_norm_bwd_kernel<Elt, GATE, WARP, MAXT, AHEAD>, AHEAD,
          static_cast<size_t>(threads) * backward_slots<Elt, GATE, AHEAD>() * 16};
}
template <typename Elt, bool GATE, bool WARP, int MAXT>
Chosen<NormBwdArgs> backward_within(int threads, size_t most) {
  if constexpr (MAXT < 1024) {
    const auto three = backward<Elt, GATE, WARP, MAXT, 3>(threads);
    if (three.shared <= most) return three;
    const auto two = backward<Elt, GATE, WARP, MAXT, 2>(threads);
    if (two.shared <= most) return two;
  }
  return backward<Elt, GATE, WARP, MAXT, 0>(threads);
}
template <typename Elt, bool GATE>
Chosen<NormBwdArgs> backward_kernel(int H, int threads, size_t most) {
  return one_warp(H)      ? backward_within<Elt, GATE, true, 32 * kTeams>(threads, most)
         : threads <= 512 ? backward_within<Elt, GATE, false, 512>(threads, most)
                          : backward_within<Elt, GATE, false, 1024>(threads, most);
}

// Shared memory for every kernel that the choices above can make.
template <typename Elt, bool WARP, int MAXT>
cudaError_t allow_team() {
  cudaError_t e = cudaSuccess;
  auto allow = [&](const auto& c) {
    if (e == cudaSuccess) e = allow_shared(c.kernel);
  };
  allow(forward<Elt, 1, WARP, MAXT, 0>(MAXT));
  allow(forward<Elt, 1, WARP, MAXT, 1>(MAXT));
  allow(forward<Elt, 8, WARP, MAXT, 0>(MAXT));
  allow(forward<Elt, 8, WARP, MAXT, 1>(MAXT));
  allow(forward<Elt, 16, WARP, MAXT, 0>(MAXT));
  allow(forward<Elt, 16, WARP, MAXT, 1>(MAXT));
  allow(backward<Elt, false, WARP, MAXT, 0>(MAXT));
  allow(backward<Elt, true, WARP, MAXT, 0>(MAXT));
  if constexpr (MAXT < 1024) {
    allow(forward<Elt, 1, WARP, MAXT, 2>(MAXT));
    allow(backward<Elt, false, WARP, MAXT, 2>(MAXT));
    allow(backward<Elt, false, WARP, MAXT, 3>(MAXT));
    allow(backward<Elt, true, WARP, MAXT, 2>(MAXT));
    allow(backward<Elt, true, WARP, MAXT, 3>(MAXT));
  }
  return e;
}
template <typename Elt>
cudaError_t allow_all() {
  cudaError_t e = allow_team<Elt, true, 32 * kTeams>();
  if (e == cudaSuccess) e = allow_team<Elt, false, 512>();
  return e == cudaSuccess ? allow_team<Elt, false, 1024>() : e;
}

}  // namespace

// Once for a device: the first call of a process loads the kernels.
cudaError_t prepare_block_norm_kernels() {
  static std::mutex mu;
  static uint64_t done[4];  // a bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  uint64_t* word = dev < 256 ? done + dev / 64 : nullptr;
  if (word && (*word >> (dev % 64) & 1)) return cudaSuccess;
  e = allow_all<__nv_bfloat16>();
  if (e == cudaSuccess) e = allow_all<float>();
  if (e == cudaSuccess && word) *word |= uint64_t{1} << (dev % 64);
  return e;
}

size_t block_norm_workspace(const moe_handle* h, int T, int H, int gate_tokens) {
  const int most = bwd_units_per_sm(H) * h->num_sms;  // grows with T, unlike the units in use
  const size_t units = T < 1 ? 1 : T < most ? T : most;
  return 2 * units * (gate_tokens > 1 ? 2 : 1) * H * sizeof(float);
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
  const bool warp = one_warp(q.H);
  const int threads = warp ? 32 * kTeams : team_threads(q.H);
  const int kmax = !q.gather ? 1 : a.K <= 8 ? 8 : 16;
  const auto c = bf16 ? forward_kernel<__nv_bfloat16>(kmax, q.H, threads, kShared)
                      : forward_kernel<float>(kmax, q.H, threads, kShared);
  const long long teams = warp ? kTeams : 1;
  const long long most = teams * h->num_sms *
                         resident_blocks(reinterpret_cast<const void*>(c.kernel), threads, c.shared);
  a.units = static_cast<int>(T < most ? T : most);
  c.kernel<<<static_cast<unsigned>((a.units + teams - 1) / teams), threads, c.shared, s>>>(a);
  return cudaGetLastError();
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
  bwd_units(T, q.H, h->num_sms, &a.chunk, &a.units);
  a.part = static_cast<float*>(workspace);
  a.slots = a.part + 2 * static_cast<size_t>(a.units) * q.H;
  const bool warp = one_warp(q.H);
  a.blocks = warp ? (a.units + kTeams - 1) / kTeams : a.units;
  const int threads = warp ? 32 * kTeams : team_threads(q.H);
  const bool gated = q.d_gate != nullptr;
  const int blocks_per_sm = warp ? 16 / kTeams : bwd_units_per_sm(q.H);
  const size_t most = kSmShared / blocks_per_sm - kBlockShared;
  using B = __nv_bfloat16;
  const auto k = bf16 ? (gated ? backward_kernel<B, true>(q.H, threads, most)
                               : backward_kernel<B, false>(q.H, threads, most))
                      : (gated ? backward_kernel<float, true>(q.H, threads, most)
                               : backward_kernel<float, false>(q.H, threads, most));
  if (T > 0) {
    k.kernel<<<a.blocks, threads, k.shared, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const bool spans = a.ggate && a.gate_tokens > 1;
  if (!a.gw_post && !a.gw_pre && !spans) return cudaSuccess;
  const int join_rows = 2 + (!spans ? 0 : a.groups < a.units ? a.groups : a.units);
  if (T == 0) a.units = 0;  // sums of nothing
  return launch_chained(bf16 ? block_norm_join_kernel<B> : block_norm_join_kernel<float>,
                        dim3((q.H + 31) / 32, join_rows), dim3(1024), 0, s, false, a);
}

}  // namespace moe
