// The norms around a block (sm_103a): the block's output rows, or the weighted
// sum of their receive rows, normed, gated and added to the residual stream, and
// the next block's norm of that sum; and the backward.
//
//   c = y + add                      (y: token rows, or sum_k w_k y[pos[t,k]])
//   res' = res_scale * res + gate * (c r_c (w_post + offset))
//   x    = res' r_p (w_pre + offset),    r_v = 1 / sqrt(mean(v^2) + eps)
//
// One pass over the rows: a team of threads holds a row in registers, 16
// elements a thread, and the two sums of squares are its only exchange.  x is
// made from the sum before that is rounded; sums are fp32, each output is
// rounded once.
#include <type_traits>

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

struct NormArgs {
  const uint8_t* y;      // [T, H], [rows, H] with pos, or NULL
  const int32_t* pos;    // [T, K] or NULL
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
  int w_f32;             // weights in fp32 (else bf16)
  float res_scale, eps, offset, inv_h;
  uint32_t* flags;
};

// N weights from column c on, with the offset that the stored ones lack.
template <int N>
__device__ __forceinline__ void load_weights(const uint8_t* w, int f32, int c, float offset,
                                             float (&f)[N]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w) + (c + i) / 4);
      f[i] = v.x;
      f[i + 1] = v.y;
      f[i + 2] = v.z;
      f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(w) + (c + i) / 4);
      f[i] = __uint_as_float(v.x << 16);
      f[i + 1] = __uint_as_float(v.x & 0xffff0000u);
      f[i + 2] = __uint_as_float(v.y << 16);
      f[i + 3] = __uint_as_float(v.y & 0xffff0000u);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] += offset;
}

// Sum over the team: a warp, or the block, whose warps hand over through `red`
// (two sets of 32 values, taken in turn, so that one barrier a sum is enough).
template <bool WARP>
__device__ __forceinline__ float team_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* set = red[turn];
  turn ^= 1;
  if (lane == 0) set[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? set[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <typename Elt, int KMAX, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_kernel(NormArgs a) {
  using VT = VecTraits<Elt>;
  constexpr int N = VT::N, V = kEpt / N;
  __shared__ float red[2][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int t = WARP ? blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.T) return;
  int turn = 0;
  const int64_t row = static_cast<int64_t>(t) * a.row_bytes;
  float c[V][N];
  Vec16 res[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * step;
    if (v < a.nvec) res[i] = ld_vec(a.res + row + v * 16);
  }
  float ss = 0.0f;
  if (a.y) {
    int p[KMAX > 0 ? KMAX : 1];
    float wk[KMAX > 0 ? KMAX : 1];
    if (KMAX > 0) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k) {
        p[k] = -1;
        wk[k] = 1.0f;
        if (k < a.K) {
          p[k] = checked_row(__ldg(a.pos + static_cast<size_t>(t) * a.K + k), a.rows, a.flags);
          if (a.cw) wk[k] = __ldg(a.cw + static_cast<size_t>(t) * a.K + k);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * step;
#pragma unroll
      for (int j = 0; j < N; ++j) c[i][j] = 0.0f;
      if (v >= a.nvec) continue;
      if (KMAX > 0) {
        Vec16 in[KMAX > 0 ? KMAX : 1];
#pragma unroll
        for (int k = 0; k < KMAX; ++k)
          if (p[k] >= 0) in[k] = ld_stream(a.y + static_cast<int64_t>(p[k]) * a.row_bytes + v * 16);
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          if (p[k] < 0) continue;
          float f[N];
          VT::to_f32(in[k], f);
#pragma unroll
          for (int j = 0; j < N; ++j) c[i][j] = fmaf(wk[k], f[j], c[i][j]);
        }
      } else {
        VT::to_f32(ld_vec(a.y + row + v * 16), c[i]);
      }
      if (a.add) {
        float f[N];
        VT::to_f32(ld_vec(a.add + row + v * 16), f);
#pragma unroll
        for (int j = 0; j < N; ++j) c[i][j] += f[j];
      }
      if (a.c) st_vec(a.c + row + v * 16, VT::from_f32(c[i]));
#pragma unroll
      for (int j = 0; j < N; ++j) ss = fmaf(c[i][j], c[i][j], ss);
    }
    float r = 1.0f;
    if (a.w_post) {
      r = 1.0f / sqrtf(team_sum<WARP>(ss, red, turn) * a.inv_h + a.eps);
      if (a.rstd_post && tid == 0) a.rstd_post[t] = r;
    }
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * step;
      if (v >= a.nvec) continue;
      float f[N];
      if (a.w_post) {
        load_weights<N>(a.w_post, a.w_f32, v * N, a.offset, f);
#pragma unroll
        for (int j = 0; j < N; ++j) c[i][j] *= r * f[j];
      }
      if (a.gate) {
        VT::to_f32(ld_vec(a.gate + static_cast<int64_t>(t / a.gate_tokens) * a.row_bytes + v * 16),
                   f);
#pragma unroll
        for (int j = 0; j < N; ++j) c[i][j] *= f[j];
      }
      VT::to_f32(res[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        c[i][j] = fmaf(a.res_scale, f[j], c[i][j]);
        ss = fmaf(c[i][j], c[i][j], ss);
      }
      st_vec(a.res_out + row + v * 16, VT::from_f32(c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (tid + i * step >= a.nvec) continue;
      VT::to_f32(res[i], c[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) ss = fmaf(c[i][j], c[i][j], ss);
    }
  }
  if (!a.x) return;
  const float r = 1.0f / sqrtf(team_sum<WARP>(ss, red, turn) * a.inv_h + a.eps);
  if (a.rstd_pre && tid == 0) a.rstd_pre[t] = r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * step;
    if (v >= a.nvec) continue;
    float f[N];
    load_weights<N>(a.w_pre, a.w_f32, v * N, a.offset, f);
#pragma unroll
    for (int j = 0; j < N; ++j) c[i][j] *= r * f[j];
    st_vec(a.x + row + v * 16, VT::from_f32(c[i]));
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
  int T, H, nvec, gate_tokens;
  int chunk, units, blocks; // tokens of a unit (a team), units, blocks
  int w_f32;
  float res_scale, offset, inv_h;
};

// Adds a thread's column sums to a row of fp32 sums (or writes them if they are
// the first) and clears them.
template <int N, int V>
__device__ __forceinline__ void flush_sums(float (&acc)[V][N], float* to, bool first, int tid,
                                           int step, int nvec) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * step;
    if (v < nvec) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        float4* p = reinterpret_cast<float4*>(to + v * N + j);
        float4 s{0.0f, 0.0f, 0.0f, 0.0f};
        if (!first) s = *p;
        s.x += acc[i][j];
        s.y += acc[i][j + 1];
        s.z += acc[i][j + 2];
        s.w += acc[i][j + 3];
        *p = s;
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.0f;
  }
}

// A unit (a team) takes `chunk` tokens in a row and holds the column sums of the
// weights' gradients, and of the gate's while the tokens of its group last.
// D = gres' + r_p (v - h mean(v h)), v = gx w_pre, h = res' r_p: the gradient of
// the residual sum; then the same form behind the gate for c.
template <typename Elt, bool GATE, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_bwd_kernel(NormBwdArgs a) {
  using VT = VecTraits<Elt>;
  constexpr int N = VT::N, V = kEpt / N;
  __shared__ float red[2][32];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int unit = WARP ? blockIdx.x * kTeams + (threadIdx.x >> 5) : blockIdx.x;
  if (unit >= a.units) return;  // a warp's; a block is always a unit
  int turn = 0;
  float gpost[V][N], gpre[V][N], ggate[V][N];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) gpost[i][j] = gpre[i][j] = ggate[i][j] = 0.0f;
  const int64_t begin64 = static_cast<int64_t>(unit) * a.chunk;
  const int begin = static_cast<int>(begin64 < a.T ? begin64 : a.T);
  const int end = static_cast<int>(begin64 + a.chunk < a.T ? begin64 + a.chunk : a.T);
  float* post_row = a.part + static_cast<size_t>(unit) * a.H;
  float* pre_row = a.part + static_cast<size_t>(a.units + unit) * a.H;
  bool first = true, gate_first = true;
  int held = 0, gate_held = 0;
  for (int t = begin; t < end; ++t) {
    const int64_t row = static_cast<int64_t>(t) * a.row_bytes;
    float D[V][N], h[V][N];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * step;
#pragma unroll
      for (int j = 0; j < N; ++j) D[i][j] = 0.0f;
      if (v < a.nvec && a.gres_out) VT::to_f32(ld_vec(a.gres_out + row + v * 16), D[i]);
    }
    if (a.gx) {
      const float r = __ldg(a.rstd_pre + t);
      float vv[V][N];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v >= a.nvec) continue;
        float w[N];
        VT::to_f32(ld_vec(a.gx + row + v * 16), vv[i]);
        VT::to_f32(ld_vec(a.res_out + row + v * 16), h[i]);
        load_weights<N>(a.w_pre, a.w_f32, v * N, a.offset, w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i][j] *= r;
          gpre[i][j] = fmaf(vv[i][j], h[i][j], gpre[i][j]);
          vv[i][j] *= w[j];
          s = fmaf(vv[i][j], h[i][j], s);
        }
      }
      s = team_sum<WARP>(s, red, turn) * a.inv_h;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * step < a.nvec)
#pragma unroll
          for (int j = 0; j < N; ++j) D[i][j] = fmaf(r, fmaf(-s, h[i][j], vv[i][j]), D[i][j]);
    }
    if (a.gres) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v >= a.nvec) continue;
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = a.res_scale * D[i][j];
        st_vec(a.gres + row + v * 16, VT::from_f32(o));
      }
    }
    const float r = a.w_post ? __ldg(a.rstd_post + t) : 1.0f;
    s = 0.0f;
    if (a.c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v >= a.nvec) continue;
        float w[N], g[N];
        VT::to_f32(ld_vec(a.c + row + v * 16), h[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[i][j] *= r;
          w[j] = 1.0f;
        }
        if (a.w_post) load_weights<N>(a.w_post, a.w_f32, v * N, a.offset, w);
        if (GATE) {
          VT::to_f32(ld_vec(a.gate + static_cast<int64_t>(t / a.gate_tokens) * a.row_bytes + v * 16),
                     g);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            ggate[i][j] = fmaf(D[i][j], h[i][j] * w[j], ggate[i][j]);
            D[i][j] *= g[j];
          }
        }
        if (a.w_post) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            gpost[i][j] = fmaf(D[i][j], h[i][j], gpost[i][j]);
            D[i][j] *= w[j];
            s = fmaf(D[i][j], h[i][j], s);
          }
        }
      }
      if (a.w_post) {
        s = team_sum<WARP>(s, red, turn) * a.inv_h;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (tid + i * step < a.nvec)
#pragma unroll
            for (int j = 0; j < N; ++j) D[i][j] = r * fmaf(-s, h[i][j], D[i][j]);
      }
    }
    if (a.gy) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * step < a.nvec) st_vec(a.gy + row + (tid + i * step) * 16, VT::from_f32(D[i]));
    }
    if (GATE && a.ggate) {
      const int group = t / a.gate_tokens;
      const int64_t g0 = static_cast<int64_t>(group) * a.gate_tokens;
      const int64_t g1 = min(g0 + a.gate_tokens, static_cast<int64_t>(a.T));
      const bool ends = t + 1 == g1;
      float* slot = a.slots + static_cast<size_t>(2 * unit + (g0 >= begin)) * a.H;
      if (ends && g0 >= begin) {  // all of the group's tokens
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int v = tid + i * step;
          if (v < a.nvec) {
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (!gate_first) ggate[i][j] += slot[v * N + j];
            st_vec(a.ggate + group * a.row_bytes + v * 16, VT::from_f32(ggate[i]));
          }
#pragma unroll
          for (int j = 0; j < N; ++j) ggate[i][j] = 0.0f;
        }
        gate_first = true;
        gate_held = 0;
      } else if (ends || t + 1 == end || ++gate_held == kFlush) {
        flush_sums<N, V>(ggate, slot, gate_first, tid, step, a.nvec);
        gate_first = ends;
        gate_held = 0;
      }
    }
    if (++held == kFlush) {
      if (a.gw_post) flush_sums<N, V>(gpost, post_row, first, tid, step, a.nvec);
      if (a.gw_pre) flush_sums<N, V>(gpre, pre_row, first, tid, step, a.nvec);
      first = false;
      held = 0;
    }
  }
  if (a.gw_post) flush_sums<N, V>(gpost, post_row, first, tid, step, a.nvec);
  if (a.gw_pre) flush_sums<N, V>(gpre, pre_row, first, tid, step, a.nvec);
}

// Joins the units' column sums: row y = 0, 1 of the grid the weights'
// gradients; row 2 + u the gate's of a group that begins in unit u and goes on
// behind it.
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
    const int u = y - 2;
    const int64_t begin = static_cast<int64_t>(u) * a.chunk, next = begin + a.chunk;
    if (next >= a.T) return;
    group = static_cast<int>(next / a.gate_tokens);
    const int64_t g0 = static_cast<int64_t>(group) * a.gate_tokens;
    if (g0 < begin || g0 >= next) return;  // begins elsewhere
    const int64_t g1 = min(g0 + a.gate_tokens, static_cast<int64_t>(a.T));
    from = a.slots;
    u0 = u;
    u1 = static_cast<int>((g1 - 1) / a.chunk) + 1;
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

}  // namespace

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
  auto pick = [&](auto elt, auto kmax) {
    using Elt = decltype(elt);
    constexpr int K = decltype(kmax)::value;
    return warp ? block_norm_kernel<Elt, K, true, 32 * kTeams>
           : threads <= 512 ? block_norm_kernel<Elt, K, false, 512>
                            : block_norm_kernel<Elt, K, false, 1024>;
  };
  auto with = [&](auto elt) {
    return !q.gather ? pick(elt, std::integral_constant<int, 0>{})
           : a.K <= 8 ? pick(elt, std::integral_constant<int, 8>{})
                      : pick(elt, std::integral_constant<int, 16>{});
  };
  auto k = bf16 ? with(__nv_bfloat16{}) : with(float{});
  k<<<warp ? (T + kTeams - 1) / kTeams : T, threads, 0, s>>>(a);
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
  auto pick = [&](auto elt, auto gated) {
    using Elt = decltype(elt);
    constexpr bool G = decltype(gated)::value;
    return warp ? block_norm_bwd_kernel<Elt, G, true, 32 * kTeams>
           : threads <= 512 ? block_norm_bwd_kernel<Elt, G, false, 512>
                            : block_norm_bwd_kernel<Elt, G, false, 1024>;
  };
  using B = __nv_bfloat16;
  const bool gated = q.d_gate != nullptr;
  auto k = bf16 ? (gated ? pick(B{}, std::true_type{}) : pick(B{}, std::false_type{}))
                : (gated ? pick(float{}, std::true_type{}) : pick(float{}, std::false_type{}));
  if (T > 0) {
    k<<<a.blocks, threads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const bool spans = a.ggate && a.gate_tokens > 1;
  if (!a.gw_post && !a.gw_pre && !spans) return cudaSuccess;
  const int join_rows = spans ? 2 + a.units : 2;
  if (T == 0) a.units = 0;  // sums of nothing
  return launch_chained(bf16 ? block_norm_join_kernel<B> : block_norm_join_kernel<float>,
                        dim3((q.H + 31) / 32, join_rows), dim3(1024), 0, s, false, a);
}

}  // namespace moe
