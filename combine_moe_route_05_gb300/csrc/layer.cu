// A whole MoE layer for a few tokens (sm_103a): routing, then two kernels that
// stream the reached experts' weights once.
//
//   up:    a[t,k,i] = act(<w13_e[i], x_t>) * <w13_e[I + i], x_t>     (bf16)
//   down:  y[t,k,n] = <w2_e[n], a[t,k]>                              (fp32)
//          out[t]   = round(sum_k w[t,k] y[t,k] + sum_j y[t, K + j])
//
// With at most 128 tokens each expert sees a handful, so the layer is bound by
// reading its weights; the kernels are matrix-vector products with the
// weights as the 16-row operand of mma.m16n8k16 and the expert's tokens as its
// 8 columns.  Weights go from global memory straight into the operand
// registers: a lane loads 16 contiguous bytes of its two rows, and since the
// order of the k index is free as long as both operands agree, those bytes
// are its operand registers of two (bf16) or four (e4m3) products, with the
// same 16 bytes (e4m3: 32) of its column's token beside them.
//
// In the up kernel rows 0..7 of the 16 are gate rows and rows 8..15 the up
// rows of the same 8 outputs, so a lane's accumulators hold gate and up of one
// output and the activation needs no exchange.
//
// A block's 8 warps split k and add their partial sums in shared memory in
// warp order.  In the down kernel the last block to finish an output tile
// (16 rows of w2, over all experts) adds the experts' fp32 rows in k order,
// so the result does not depend on the order in which blocks run.
//
// Every block groups the (t, k) entries by expert itself, in shared memory.
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxEntries = MOE_LAYER_MAX_TOKENS * (MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED);
constexpr int kMaxExperts = MOE_MAX_EXPERTS + MOE_LAYER_MAX_SHARED;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint16_t kNone = 0xffff;

struct LayerArgs {
  const uint8_t* x;      // [T, H] bf16
  const int32_t* idx;    // [T, K]
  const float* w;        // [T, K]
  const int32_t* live;   // live tokens or NULL
  const uint8_t* w13;    // [E + S, 2I, H]
  const uint8_t* w2;     // [E + S, H, I]
  const float* s13;      // block scales of e4m3 weights
  const float* s2;
  __nv_bfloat16* a;      // [T (K + S), I]
  float* y;              // [T (K + S), H]
  int32_t* done;         // finished experts per output tile
  __nv_bfloat16* out;    // [T, H]
  int T, K, S, E, H, I;
  uint32_t* flags;
};

// The entries (t, k) grouped by expert; entry t (K + S) + k, shared expert j
// as k = K + j.
struct Groups {
  uint16_t order[kMaxEntries];  // entries, grouped
  uint16_t rank[kMaxEntries];   // place within its expert, kNone: dropped
  int cnt[kMaxExperts];
  int start[kMaxExperts];
  uint16_t slot_expert[kMaxExperts];  // experts with entries
  int warp_sum[kWarps];
  int nslots;
  int tokens;
};

__device__ __forceinline__ int expert_of(const LayerArgs& a, int entry) {
  const int k = entry % (a.K + a.S);
  return k < a.K ? __ldg(a.idx + entry / (a.K + a.S) * a.K + k) : a.E + k - a.K;
}

__device__ void group_entries(const LayerArgs& a, Groups& g) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_exp = a.E + a.S;
  for (int e = tid; e < n_exp; e += kThreads) g.cnt[e] = 0;
  const int tokens = a.live ? min(max(*a.live, 0), a.T) : a.T;
  const int n = tokens * (a.K + a.S);
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int e = expert_of(a, i);
    const int k = i % (a.K + a.S);
    bool ok = static_cast<unsigned>(e) < static_cast<unsigned>(n_exp) && (k >= a.K || e < a.E);
    uint32_t bad = ok || e == -1 ? 0u : MOE_DEVERR_BAD_EXPERT;
    for (int j = 0; j < min(k, a.K) && ok && k < a.K; ++j)
      if (expert_of(a, i - k + j) == e) {
        ok = false;
        bad = MOE_DEVERR_DUP_EXPERT;
      }
    if (bad && blockIdx.x == 0) raise_flag(a.flags, bad);
    g.rank[i] = ok ? static_cast<uint16_t>(atomicAdd(&g.cnt[e], 1)) : kNone;
  }
  __syncthreads();
  // exclusive scan of counts (low 16 bits) and of experts with entries (high)
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    const int c = e < n_exp ? g.cnt[e] : 0;
    own[j] = sum;
    sum += c + (c ? 0x10000 : 0);
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) g.warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int wv = 0; wv < warp; ++wv) base += g.warp_sum[wv];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    if (e < n_exp) {
      const int at = base + own[j];
      g.start[e] = at & 0xffff;
      if (g.cnt[e]) g.slot_expert[at >> 16] = static_cast<uint16_t>(e);
    }
  }
  if (tid == kThreads - 1) {
    g.nslots = (base + sum) >> 16;
    g.tokens = tokens;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads)
    if (g.rank[i] != kNone) g.order[g.start[expert_of(a, i)] + g.rank[i]] = static_cast<uint16_t>(i);
  __syncthreads();
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 values as bf16 (exact).
__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu),
                                                  __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// acc[nt] += 16 weight rows x 8 columns over this warp's share of k.
// row0 / row1: the lane's weight rows (lane / 4 and lane / 4 + 8); col[nt]: the
// lane's token row of tile nt or NULL; sc0 / sc1: block scales of the rows'
// 128-row block (e4m3).  Steps of 32 (e4m3: 64) k are dealt out to the warps.
template <int NT, bool FP8>
__device__ __forceinline__ void dot_rows(float (&acc)[NT][4], const uint8_t* row0,
                                         const uint8_t* row1, const uint8_t* const (&col)[NT],
                                         const float* sc0, const float* sc1, int kd, int warp) {
  constexpr int kStep = FP8 ? 64 : 32;
  constexpr int U = NT == 1 ? 4 : 2;
  constexpr int X = FP8 ? 2 : 1;  // 16-byte token vectors per weight vector
  const int t = threadIdx.x & 3;
  const Vec16 zero{};
  for (int s0 = warp; s0 * kStep < kd; s0 += kWarps * U) {
    Vec16 w0[U], w1[U], xv[U][NT][X];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int o = (s0 + u * kWarps) * kStep + t * (kStep / 4);
      w0[u] = o < kd ? ld_stream(row0 + static_cast<int64_t>(o) * (FP8 ? 1 : 2)) : zero;
      w1[u] = o < kd ? ld_stream(row1 + static_cast<int64_t>(o) * (FP8 ? 1 : 2)) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int o = (s0 + u * kWarps) * kStep + t * (kStep / 4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int v = 0; v < X; ++v)
          xv[u][nt][v] = o < kd && col[nt] ? ld_vec(col[nt] + o * 2 + v * 16) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!FP8) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < 4; q += 2)
            mma_bf16(acc[nt], w0[u].u[q], w1[u].u[q], w0[u].u[q + 1], w1[u].u[q + 1],
                     xv[u][nt][0].u[q], xv[u][nt][0].u[q + 1]);
      } else {
        const int s = s0 + u * kWarps;
        if (s * kStep >= kd) continue;
        const float f0 = __ldg(sc0 + s / 2), f1 = __ldg(sc1 + s / 2);
        float part[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[nt][j] = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a0 = bf16x2_of_e4m3x2(w0[u].u[q]), a2 = bf16x2_of_e4m3x2(w0[u].u[q] >> 16);
          const uint32_t a1 = bf16x2_of_e4m3x2(w1[u].u[q]), a3 = bf16x2_of_e4m3x2(w1[u].u[q] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16(part[nt], a0, a1, a2, a3, xv[u][nt][q / 2].u[q % 2 * 2],
                     xv[u][nt][q / 2].u[q % 2 * 2 + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][0] = fmaf(f0, part[nt][0], acc[nt][0]);
          acc[nt][1] = fmaf(f0, part[nt][1], acc[nt][1]);
          acc[nt][2] = fmaf(f1, part[nt][2], acc[nt][2]);
          acc[nt][3] = fmaf(f1, part[nt][3], acc[nt][3]);
        }
      }
    }
  }
}

// The warps' partial sums added in warp order; warp nt returns true with tile
// nt's sums in acc.
template <int NT>
__device__ __forceinline__ bool sum_warps(float (&acc)[NT][4], float (&sum)[4], float* red,
                                          int warp, int lane) {
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[((warp * NT + nt) * 4 + j) * 32 + lane] = acc[nt][j];
  __syncthreads();
  if (warp >= NT) return false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sum[j] = 0.0f;
    for (int wv = 0; wv < kWarps; ++wv) sum[j] += red[((wv * NT + warp) * 4 + j) * 32 + lane];
  }
  return true;
}

__device__ __forceinline__ float act_value(float g, int act) {
  const float c = act == MOE_ACT_GELU
                      ? 1.5957691216057308f * g * (1.0f + 0.044715f * g * g) : g;
  return c < -80.0f ? g * 0.0f : g * __fdividef(1.0f, 1.0f + __expf(-c));
}

constexpr int kNT = 4;  // column tiles of 8 tokens handled at once

// One unit: 16 weight rows of one expert against its tokens, kNT * 8 at a
// time; store(sum, token column, lane row) takes the results.
template <bool FP8, typename Col, typename Store>
__device__ __forceinline__ void unit_products(const Groups& g, int e, const uint8_t* row0,
                                              const uint8_t* row1, const float* sc0,
                                              const float* sc1, int kd, float* red, Col col_of,
                                              Store store) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cnt = g.cnt[e], start = g.start[e];
  for (int c0 = 0; c0 < cnt;) {
    auto pass = [&](auto tiles) {
      constexpr int NT = decltype(tiles)::value;
      float acc[NT][4] = {}, sum[4];
      const uint8_t* col[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = c0 + nt * 8 + (lane >> 2);
        col[nt] = c < cnt ? col_of(g.order[start + c]) : nullptr;
      }
      dot_rows<NT, FP8>(acc, row0, row1, col, sc0, sc1, kd, warp);
      if (sum_warps<NT>(acc, sum, red, warp, lane)) {
        const int c = c0 + warp * 8 + 2 * (lane & 3);
        if (c < cnt) store(g.order[start + c], sum[0], sum[2]);
        if (c + 1 < cnt) store(g.order[start + c + 1], sum[1], sum[3]);
      }
      c0 += NT * 8;
    };
    if (cnt - c0 <= 8) pass(std::integral_constant<int, 1>{});
    else if (cnt - c0 <= 16) pass(std::integral_constant<int, 2>{});
    else pass(std::integral_constant<int, kNT>{});
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 2) layer_up_kernel(LayerArgs a, int act) {
  grid_dependency_wait();
  __shared__ Groups g;
  __shared__ float red[kWarps * kNT * 4 * 32];
  group_entries(a, g);
  const int lane = threadIdx.x & 31;
  const int tiles2 = (a.H + 15) / 16;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < tiles2; i += gridDim.x * kThreads) a.done[i] = 0;
  const int tiles = a.I / 8;
  const int units = g.nslots * tiles;
  const int KS = a.K + a.S;
  constexpr int kEb = FP8 ? 1 : 2;
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  for (int u = u0; u < u1; ++u) {
    const int e = g.slot_expert[u / tiles], i0 = u % tiles * 8;
    const int64_t base = static_cast<int64_t>(e) * 2 * a.I;
    const uint8_t* row0 = a.w13 + (base + i0 + (lane >> 2)) * a.H * kEb;
    const uint8_t* row1 = row0 + static_cast<int64_t>(a.I) * a.H * kEb;
    const int kb = (a.H + 127) / 128, rb = (2 * a.I + 127) / 128;
    const float* sc = a.s13 + static_cast<int64_t>(e) * rb * kb;
    unit_products<FP8>(
        g, e, row0, row1, sc + static_cast<int64_t>(i0 / 128) * kb,
        sc + static_cast<int64_t>((a.I + i0) / 128) * kb, a.H, red,
        [&](int entry) { return a.x + static_cast<int64_t>(entry / KS) * a.H * 2; },
        [&](int entry, float gate, float up) {
          a.a[static_cast<int64_t>(entry) * a.I + i0 + (lane >> 2)] =
              __float2bfloat16_rn(act_value(gate, act) * up);
        });
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 2) layer_down_kernel(LayerArgs a) {
  grid_dependency_wait();
  __shared__ Groups g;
  __shared__ float red[kWarps * kNT * 4 * 32];
  __shared__ int last;
  group_entries(a, g);
  const int lane = threadIdx.x & 31;
  const int tiles = (a.H + 15) / 16;
  const int units = g.nslots * tiles;
  const int KS = a.K + a.S;
  constexpr int kEb = FP8 ? 1 : 2;
  if (units == 0) {  // no expert reached: zero rows
    const int64_t n = static_cast<int64_t>(g.tokens) * a.H;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      a.out[i] = __float2bfloat16_rn(0.0f);
    return;
  }
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  for (int u = u0; u < u1; ++u) {
    const int e = g.slot_expert[u / tiles], n0 = u % tiles * 16;
    const int r0 = n0 + (lane >> 2);
    const bool second = r0 + 8 < a.H;  // H is a multiple of 8
    const uint8_t* row0 = a.w2 + (static_cast<int64_t>(e) * a.H + r0) * a.I * kEb;
    const uint8_t* row1 = second ? row0 + static_cast<int64_t>(8) * a.I * kEb : row0;
    const int kb = (a.I + 127) / 128, rb = (a.H + 127) / 128;
    const float* sc = a.s2 + (static_cast<int64_t>(e) * rb + n0 / 128) * kb;
    unit_products<FP8>(
        g, e, row0, row1, sc, sc, a.I, red,
        [&](int entry) {
          return reinterpret_cast<const uint8_t*>(a.a + static_cast<int64_t>(entry) * a.I);
        },
        [&](int entry, float lo, float hi) {
          float* y = a.y + static_cast<int64_t>(entry) * a.H + r0;
          y[0] = lo;
          if (second) y[8] = hi;
        });
    // the last expert's block of this tile adds the experts' rows
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done + u % tiles, 1) == g.nslots - 1;
    __syncthreads();
    if (last) {
      __threadfence();
      const int width = min(16, a.H - n0);
      for (int i = threadIdx.x; i < g.tokens * 16; i += kThreads) {
        const int t = i / 16, n = i % 16;
        if (n >= width) continue;
        float v = 0.0f;
        for (int k = 0; k < KS; ++k) {
          if (g.rank[t * KS + k] == kNone) continue;
          const float yv = __ldcg(a.y + static_cast<int64_t>(t * KS + k) * a.H + n0 + n);
          v = fmaf(k < a.K ? __ldg(a.w + t * a.K + k) : 1.0f, yv, v);
        }
        a.out[static_cast<int64_t>(t) * a.H + n0 + n] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace

LayerPlan layer_plan(int T, int K, int S, int H, int I) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t entries = static_cast<size_t>(T) * (K + S);
  LayerPlan p;
  p.a = 0;
  p.y = up(entries * I * sizeof(__nv_bfloat16));
  p.done = p.y + up(entries * H * sizeof(float));
  p.total = p.done + up(static_cast<size_t>((H + 15) / 16) * sizeof(int32_t));
  return p;
}

cudaError_t launch_layer(const moe_handle* h, const moe_layer_args& q, int T, void* workspace,
                         cudaStream_t s) {
  const int K = h->cfg.top_k;
  if (T == 0) return cudaSuccess;
  if (q.d_logits) {
    const cudaError_t e = launch_route_topk(h, q.d_logits, q.d_bias, T, q.d_idx, q.d_w, s, q.d_live);
    if (e != cudaSuccess) return e;
  }
  const LayerPlan p = layer_plan(T, K, q.num_shared, q.H, q.I);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LayerArgs a{};
  a.x = static_cast<const uint8_t*>(q.d_x);
  a.idx = q.d_idx;
  a.w = q.d_w;
  a.live = q.d_live;
  a.w13 = static_cast<const uint8_t*>(q.d_w13);
  a.w2 = static_cast<const uint8_t*>(q.d_w2);
  a.s13 = q.d_s13;
  a.s2 = q.d_s2;
  a.a = reinterpret_cast<__nv_bfloat16*>(ws + p.a);
  a.y = reinterpret_cast<float*>(ws + p.y);
  a.done = reinterpret_cast<int32_t*>(ws + p.done);
  a.out = static_cast<__nv_bfloat16*>(q.d_out);
  a.T = T;
  a.K = K;
  a.S = q.num_shared;
  a.E = h->cfg.num_experts;
  a.H = q.H;
  a.I = q.I;
  a.flags = h->flags;
  const bool fp8 = q.weight_dtype == MOE_E4M3;
  const dim3 grid(2 * h->num_sms), block(kThreads);
  cudaError_t e = fp8 ? launch_chained(layer_up_kernel<true>, grid, block, 0, s, false, a, q.act)
                      : launch_chained(layer_up_kernel<false>, grid, block, 0, s, false, a, q.act);
  if (e != cudaSuccess) return e;
  return fp8 ? launch_chained(layer_down_kernel<true>, grid, block, 0, s, false, a)
             : launch_chained(layer_down_kernel<false>, grid, block, 0, s, false, a);
}

}  // namespace moe
