// Gated expert activation of receive rows with expert dropout and the routed
// score (sm_103a): hs = w * m * a(g) * u, and its backward.
//
// The activation is a(g) = g * sigmoid(c(g)) with c(g) = g (SiLU) or
// c(g) = 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU in its tanh form, since
// (1 + tanh z) / 2 = sigmoid(2 z)), so one exponential and one reciprocal
// serve the value and the derivative a' = s + g c' s (1 - s).  1 - s is taken
// as e^-c * s, which keeps its relative accuracy where s is near 1; below
// c = -87.3 the sigmoid, under 2^-126, is 0 (the fast division's result for a
// denominator above 2^126), and a' with it.
//
// The dropout mask is never stored: Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) of the counter
// (i div 8, t*K + k, offset) under the key `seed` gives 128 bits for the 8
// elements i of a row's 16-byte bf16 vector, 16 bits each; an element is
// dropped when its 16 bits are below p * 2^16.  The counter names the entry
// (t, k) and not its receive row, so the mask survives another layout or
// padding of the same routing.  16 bits an element instead of 32 halve the
// generator's work, about 60 instructions a vector.
//
// Products and sums are fp32 and each output is rounded once.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kActThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

struct ActArgs {
  const uint8_t* gu;    // [rows, 2I]: gate, up
  const uint8_t* ghs;   // [rows, I] (backward)
  const float* rw;      // [rows] or NULL
  uint8_t* out;         // hs [rows, I] (forward) or ggu [rows, 2I] (backward)
  float* gw;            // [T, K] or NULL (backward)
  const int32_t* off_end;  // off_e + E: rows in segments
  const int32_t* recv_token;
  const int32_t* recv_k;
  const int32_t* pos;
  const int64_t* rng;   // {seed, offset} when drop > 0
  int64_t half_bytes;   // I elements
  int nvec;             // 16-byte vectors of I elements
  int rows;             // receive rows of the tensors
  int T, K;
  uint32_t drop;        // dropped 16-bit values, in the high half
  float keep_scale;     // 2^16 / (2^16 - drop)
  uint32_t* flags;
};

// Byte of a row's 16-byte vector v.  32 bits hold it (I is at most 2^26), which
// the backward uses; the forward is faster with 64 (DeepSeek-V3 shape with
// dropout: forward 241 against 248 us, backward 412 against 398).
__device__ __forceinline__ int64_t byte_of(int v) { return static_cast<int64_t>(v) * 16; }

__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(p1 >> 32) ^ c.y ^ k0, static_cast<uint32_t>(p1),
                   static_cast<uint32_t>(p0 >> 32) ^ c.w ^ k1, static_cast<uint32_t>(p0));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// Whether each element of the row vector v (N elements) of entry `ent` is
// kept; drop16: the dropped values in the high half of a word, so that a high
// half is compared in place and a low half after one shift.
template <int N>
__device__ __forceinline__ void kept_elements(bool (&kept)[N], int v, uint32_t ent,
                                              uint32_t drop16, uint2 key, uint2 offset) {
  const uint32_t oct = N == 8 ? v : v >> 1;
  const uint4 r = philox(make_uint4(oct, ent, offset.x, offset.y), key.x, key.y);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const uint32_t word = N == 8 ? w[j / 2] : ((v & 1) ? w[2 + j / 2] : w[j / 2]);
    kept[j] = (word << 16) >= drop16;
    kept[j + 1] = word >= drop16;
  }
}

template <bool FAST>
__device__ __forceinline__ float exp_neg(float c) {
  return FAST ? __expf(-c) : expf(-c);
}

// The gate's value a(g).
template <int ACT, bool FAST>
__device__ __forceinline__ float gate_value(float g) {
  constexpr float kR = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  const float c = ACT == MOE_ACT_GELU ? kR * g * (1.0f + 0.044715f * (g * g)) : g;
  return g * __fdividef(1.0f, 1.0f + exp_neg<FAST>(c));
}

// The gate's sigmoid s and one-minus-sigmoid q at c(g), and c'(g).
template <int ACT, bool FAST>
__device__ __forceinline__ void gate_terms(float g, float& s, float& q, float& dc) {
  constexpr float kR = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  float c = g;
  dc = 1.0f;
  if (ACT == MOE_ACT_GELU) {
    // bounded, so that c' stays finite beside the 0 that it multiplies at
    // saturation (from |g| = 1.9e19 on its square is infinite in fp32)
    const float g2 = fminf(g * g, 1e30f);
    c = kR * g * (1.0f + 0.044715f * g2);
    dc = kR * (1.0f + 0.134145f * g2);
  }
  const float e = exp_neg<FAST>(c);
  s = __fdividef(1.0f, 1.0f + e);
  q = fminf(e * s, 1.0f);  // infinity times 0: 1
}

// The entry t*K + k of receive row r, -1 for a pad row.
__device__ __forceinline__ int entry_of(const ActArgs& a, int r) {
  const int t = __ldg(a.recv_token + r), k = __ldg(a.recv_k + r);
  if (static_cast<unsigned>(t) < static_cast<unsigned>(a.T) &&
      static_cast<unsigned>(k) < static_cast<unsigned>(a.K))
    return t * a.K + k;
  if (t != -1) raise_flag(a.flags, MOE_DEVERR_BAD_LAYOUT);
  return -1;
}

__device__ __forceinline__ int rows_in_segments(const ActArgs& a) {
  const int n = *a.off_end;
  if (n >= 0 && n <= a.rows) return n;
  if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(a.flags, MOE_DEVERR_BAD_LAYOUT);
  return n < 0 ? 0 : a.rows;
}

__device__ __forceinline__ uint2 split64(int64_t v) {
  return make_uint2(static_cast<uint32_t>(v),
                    static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
}

// Vectors of a row that a warp loads before it works on the first of them:
// with one, a warp waits out the memory's latency for every 32 vectors
// (forward 385 us on the DeepSeek-V3 shape with dropout, a thread per vector
// and a 64-bit division for each).
constexpr int kAhead = 2;

// Forward: a warp per piece of kPiece vectors of a row.
constexpr int kPiece = 256;

template <typename Elt, int ACT, bool DROP>
__global__ void __launch_bounds__(kActThreads) act_rows_kernel(ActArgs a) {
  using VT = VecTraits<Elt>;
  constexpr int N = VT::N;
  constexpr bool kFast = N == 8;
  const int lane = threadIdx.x & 31;
  const int pieces = (a.nvec + kPiece - 1) / kPiece;
  const int64_t total = static_cast<int64_t>(rows_in_segments(a)) * pieces;
  uint2 key{}, offset{};
  if (DROP) {
    key = split64(a.rng[0]);
    offset = split64(a.rng[1]);
  }
  const int64_t W = static_cast<int64_t>(gridDim.x) * (kActThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5);
       i < total; i += W) {
    const int r = pieces == 1 ? static_cast<int>(i) : static_cast<int>(i / pieces);
    const int v0 =
        pieces == 1 ? 0 : static_cast<int>(i - static_cast<int64_t>(r) * pieces) * kPiece;
    const int end = min(v0 + kPiece, a.nvec);
    const uint8_t* row = a.gu + static_cast<int64_t>(r) * 2 * a.half_bytes;
    uint8_t* out = a.out + static_cast<int64_t>(r) * a.half_bytes;
    const int ent = entry_of(a, r);
    const float w = a.rw ? __ldg(a.rw + r) : 1.0f;
    const float ws = DROP ? w * a.keep_scale : w;
    if (ent < 0) {  // a pad row
      const float zero[N] = {};
      for (int v = v0 + lane; v < end; v += 32) st_vec(out + byte_of(v), VT::from_f32(zero));
      continue;
    }
    for (int v = v0 + lane; v < end; v += 32 * kAhead) {
      Vec16 gv[kAhead], uv[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (v + 32 * k < end) {
          gv[k] = ld_stream(row + byte_of(v + 32 * k));
          uv[k] = ld_stream(row + a.half_bytes + byte_of(v + 32 * k));
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (v + 32 * k >= end) continue;
        float g[N], u[N];
        VT::to_f32(gv[k], g);
        VT::to_f32(uv[k], u);
        bool kept[N];
        if (DROP) kept_elements<N>(kept, v + 32 * k, ent, a.drop, key, offset);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float o = gate_value<ACT, kFast>(g[j]) * u[j] * ws;
          g[j] = !DROP || kept[j] ? o : 0.0f;
        }
        st_vec_cs(out + byte_of(v + 32 * k), VT::from_f32(g));
      }
    }
  }
}

// Backward: one warp per receive row; the score gradient is the row's sum, if
// it is asked for (GW).  With dropout the issue slots bind nearly as much as
// memory (some 40 instructions an element with GELU), and registers beside them:
// 65536 rows of 2048, bf16, with score gradient: SiLU 197 us with 10 blocks an SM,
// 200 with 12 and 204 where the compiler chose, GELU 227, 209 and 214 (either
// without dropout: 197).  With 12 blocks GELU with dropout and score gradient
// spills 16 bytes.  A warp per 64 vectors of a row (without GW) was
// slower with dropout (SiLU 196 -> 211, GELU 212 -> 252).
template <typename Elt, int ACT, bool DROP, bool GW>
__global__ void __launch_bounds__(kActThreads, ACT == MOE_ACT_GELU ? 12 : 10)
    act_rows_bwd_kernel(ActArgs a) {
  using VT = VecTraits<Elt>;
  constexpr int N = VT::N;
  constexpr bool kFast = N == 8;
  const int lane = threadIdx.x & 31;
  const int nrows = rows_in_segments(a);
  uint2 key{}, offset{};
  if (DROP) {
    key = split64(a.rng[0]);
    offset = split64(a.rng[1]);
  }
  if (GW) {  // entries without a receive row
    const int64_t n = static_cast<int64_t>(a.T) * a.K;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kActThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kActThreads)
      if (__ldg(a.pos + i) < 0) a.gw[i] = 0.0f;
  }
  const int64_t W = static_cast<int64_t>(gridDim.x) * (kActThreads / 32);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5);
       i < nrows; i += W) {
    const int r = static_cast<int>(i);
    const uint8_t* grow = a.gu + static_cast<int64_t>(r) * 2 * a.half_bytes;
    const uint8_t* drow = a.ghs + static_cast<int64_t>(r) * a.half_bytes;
    uint8_t* orow = a.out + static_cast<int64_t>(r) * 2 * a.half_bytes;
    const int ent = entry_of(a, r);
    const float w = a.rw ? __ldg(a.rw + r) : 1.0f;
    const float ws = DROP ? w * a.keep_scale : w;
    float dot = 0.0f;
    if (ent < 0) {  // a pad row
      const float zero[N] = {};
      for (int v = lane; v < 2 * a.nvec; v += 32) st_vec(orow + v * 16, VT::from_f32(zero));
      continue;
    }
    for (int v = lane; v < a.nvec; v += 32) {
      float g[N], u[N], d[N];
      VT::to_f32(ld_vec(grow + v * 16), g);
      VT::to_f32(ld_vec(grow + a.half_bytes + v * 16), u);
      VT::to_f32(ld_vec(drow + v * 16), d);
      bool kept[N];
      if (DROP) kept_elements<N>(kept, v, ent, a.drop, key, offset);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float s, q, dc;
        gate_terms<ACT, kFast>(g[j], s, q, dc);
        const float dw = d[j] * ws;
        const float act = g[j] * s;
        const float da = s + act * q * dc;
        const bool live = !DROP || kept[j];
        if (GW) dot = live ? fmaf(d[j] * act, u[j], dot) : dot;
        g[j] = live ? dw * u[j] * da : 0.0f;
        u[j] = live ? dw * act : 0.0f;
      }
      st_vec(orow + v * 16, VT::from_f32(g));
      st_vec(orow + a.half_bytes + v * 16, VT::from_f32(u));
    }
    if (GW) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(kFull, dot, off);
      if (lane == 0) a.gw[ent] = DROP ? dot * a.keep_scale : dot;
    }
  }
}

ActArgs act_args(const moe_handle* h, int I, int dtype, const float* rw, double p,
                 const int64_t* rng) {
  ActArgs a{};
  a.rw = rw;
  a.off_end = h->off_e + h->cfg.num_experts;
  a.recv_token = h->recv_token;
  a.recv_k = h->recv_k;
  a.pos = h->pos;
  a.rng = rng;
  a.half_bytes = static_cast<int64_t>(I) * (dtype == MOE_BF16 ? 2 : 4);
  a.nvec = static_cast<int>(a.half_bytes / 16);
  a.rows = h->T * h->cfg.top_k + h->cfg.num_experts * (h->pad - 1);
  a.T = h->T;
  a.K = h->cfg.top_k;
  a.drop = dropped_of(p) << 16;
  a.keep_scale = static_cast<float>(65536.0 / (65536.0 - dropped_of(p)));
  a.flags = h->flags;
  return a;
}

template <typename Elt, int ACT, bool DROP>
cudaError_t launch_t(const moe_handle* h, const ActArgs& a, bool bwd, cudaStream_t s) {
  auto k = !bwd   ? act_rows_kernel<Elt, ACT, DROP>
           : a.gw ? act_rows_bwd_kernel<Elt, ACT, DROP, true>
                  : act_rows_bwd_kernel<Elt, ACT, DROP, false>;
  const long long items =
      static_cast<long long>(a.rows) * (bwd ? 1 : (a.nvec + kPiece - 1) / kPiece);
  const long long blocks = (items + kActThreads / 32 - 1) / (kActThreads / 32);
  // a block per kActThreads / 32 items, not one wave of resident blocks: the
  // SMs take blocks at their own pace (DeepSeek-V3 shape with dropout: forward
  // 251 against 258 us, backward 394 against 417, at blocks of 256 threads)
  const long long most = 1 << 30;
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  k<<<grid < 1 ? 1 : grid, kActThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename Elt>
cudaError_t launch_d(const moe_handle* h, const ActArgs& a, int act, bool bwd, cudaStream_t s) {
  if (act == MOE_ACT_GELU)
    return a.drop ? launch_t<Elt, MOE_ACT_GELU, true>(h, a, bwd, s)
                  : launch_t<Elt, MOE_ACT_GELU, false>(h, a, bwd, s);
  return a.drop ? launch_t<Elt, MOE_ACT_SILU, true>(h, a, bwd, s)
                : launch_t<Elt, MOE_ACT_SILU, false>(h, a, bwd, s);
}

}  // namespace

uint32_t dropped_of(double p) { return static_cast<uint32_t>(std::nearbyint(p * 65536.0)); }

cudaError_t launch_act_rows(const moe_handle* h, const void* gu, int I, int dtype, int act,
                            const float* rw, double p, const int64_t* rng, void* hs,
                            cudaStream_t s) {
  ActArgs a = act_args(h, I, dtype, rw, p, rng);
  a.gu = static_cast<const uint8_t*>(gu);
  a.out = static_cast<uint8_t*>(hs);
  if (h->T == 0) return cudaSuccess;
  return dtype == MOE_BF16 ? launch_d<__nv_bfloat16>(h, a, act, false, s)
                           : launch_d<float>(h, a, act, false, s);
}

cudaError_t launch_act_rows_bwd(const moe_handle* h, const void* ghs, const void* gu, int I,
                                int dtype, int act, const float* rw, double p, const int64_t* rng,
                                void* ggu, float* gw, cudaStream_t s) {
  ActArgs a = act_args(h, I, dtype, rw, p, rng);
  a.gu = static_cast<const uint8_t*>(gu);
  a.ghs = static_cast<const uint8_t*>(ghs);
  a.out = static_cast<uint8_t*>(ggu);
  a.gw = gw;
  if (h->T == 0) return cudaSuccess;
  return dtype == MOE_BF16 ? launch_d<__nv_bfloat16>(h, a, act, true, s)
                           : launch_d<float>(h, a, act, true, s);
}

}  // namespace moe
