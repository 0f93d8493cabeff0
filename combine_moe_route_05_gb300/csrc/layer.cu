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
  __nv_bfloat16* a;      // [2][T (K + S), I]: high and low parts
  float* y;              // [T (K + S), H]
  uint32_t* kept;        // [T] bit k: entry (t, k) has an expert
  __nv_bfloat16* out;    // [T, H]
  int T, K, S, E, H, I;
  int act;
  uint32_t* flags;
};

// ---------------------------------------------------------------------------
// entries (t, k) grouped by expert

// Shared-memory tables of a block.  Entry n = t (K + S) + k, the shared expert
// j as k = K + j; experts are numbered shared first, so that their many
// tokens do not come last.
struct Groups {
  uint16_t* order;        // entries, grouped
  uint16_t* rank;         // an entry's place within its expert, kNone: dropped
  uint16_t* slot_expert;  // experts with entries
  int* cnt;               // per expert
  int* start;
  int* head;              // warp sums, number of slots
  int tokens, nslots;
};

__host__ __device__ constexpr size_t up16(size_t b) { return (b + 15) / 16 * 16; }

__host__ __device__ constexpr size_t groups_bytes(int T, int KS, int n_exp) {
  return 2 * up16(2ull * T * KS) + up16(2ull * n_exp) + 2 * up16(4ull * n_exp) + 64;
}

__device__ __forceinline__ int expert_of(const LayerArgs& a, int entry) {
  const int t = entry / (a.K + a.S), k = entry - t * (a.K + a.S);
  if (k >= a.K) return k - a.K;
  const int e = __ldcg(a.idx + t * a.K + k);
  return static_cast<unsigned>(e) < static_cast<unsigned>(a.E) ? e + a.S : e == -1 ? -1 : -2;
}

__device__ void group_entries(const LayerArgs& a, Groups& g, uint8_t* smem) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_exp = a.E + a.S, KS = a.K + a.S;
  g.order = reinterpret_cast<uint16_t*>(smem);
  smem += up16(2ull * a.T * KS);
  g.rank = reinterpret_cast<uint16_t*>(smem);
  smem += up16(2ull * a.T * KS);
  g.slot_expert = reinterpret_cast<uint16_t*>(smem);
  smem += up16(2ull * n_exp);
  g.cnt = reinterpret_cast<int*>(smem);
  smem += up16(4ull * n_exp);
  g.start = reinterpret_cast<int*>(smem);
  smem += up16(4ull * n_exp);
  g.head = reinterpret_cast<int*>(smem);

  for (int e = tid; e < n_exp; e += kThreads) g.cnt[e] = 0;
  g.tokens = a.live ? min(max(__ldcg(a.live), 0), a.T) : a.T;
  const int n = g.tokens * KS;
  // an entry's expert, checked, in `order` until the entries are placed
  for (int i = tid; i < n; i += kThreads) {
    const int e = expert_of(a, i);
    if (e == -2 && blockIdx.x == 0) raise_flag(a.flags, MOE_DEVERR_BAD_EXPERT);
    g.order[i] = e >= 0 ? static_cast<uint16_t>(e) : kNone;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const uint16_t e = g.order[i];
    bool ok = e != kNone;
    if (ok && e >= a.S) {  // a repeated expert of the token counts once
      bool seen = false;
      for (int j = i / KS * KS; j < i; ++j) seen |= g.order[j] == e;
      if (seen) {
        ok = false;
        if (blockIdx.x == 0) raise_flag(a.flags, MOE_DEVERR_DUP_EXPERT);
      }
    }
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
  if (lane == 31) g.head[warp] = inc;
  // the entries' experts, before `order` takes the entries
  constexpr int kMine = MOE_LAYER_MAX_TOKENS * (MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED) / kThreads;
  uint16_t mine[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (tid + j * kThreads < n) mine[j] = g.order[tid + j * kThreads];
  __syncthreads();
  int base = inc - sum;
  for (int wv = 0; wv < warp; ++wv) base += g.head[wv];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    if (e < n_exp) {
      const int at = base + own[j];
      g.start[e] = at & 0xffff;
      if (g.cnt[e]) g.slot_expert[at >> 16] = static_cast<uint16_t>(e);
    }
  }
  if (tid == kThreads - 1) g.head[kWarps] = (base + sum) >> 16;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kThreads;
    if (i < n && g.rank[i] != kNone) g.order[g.start[mine[j]] + g.rank[i]] = static_cast<uint16_t>(i);
  }
  g.nslots = g.head[kWarps];
  __syncthreads();
}

// ---------------------------------------------------------------------------
// matrix products on lane-private queues

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

// Asynchronous copies of 16 and 4 bytes into shared memory; !valid writes
// zeros and reads nothing.  Weights pass by L1, tokens are kept in it.
__device__ __forceinline__ void copy16_stream(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_keep(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ Vec16 lds16(uint32_t p) {
  Vec16 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3])
               : "r"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}

// Shape of a kernel: MT tiles of 16 weight rows by NT tiles of 8 tokens,
// STEPS steps of 64 bytes of a weight row per stage of the queue.
template <int MT_, int NT_, int STEPS_, int STAGES_, bool FP8_, bool UP_>
struct Shape {
  static constexpr int MT = MT_, NT = NT_, kSteps = STEPS_, kStages = STAGES_;
  static constexpr bool FP8 = FP8_, UP = UP_;
  static constexpr int kRows = UP ? 8 * MT : 16 * MT;     // outputs of a tile
  static constexpr int kParts = UP ? 1 : 2;               // x; high and low part of a
  static constexpr int kVec = FP8 ? 2 : 1;                // token vectors beside a weight vector
  static constexpr int kSlots = 2 * MT + NT * kVec * kParts;
  static constexpr int kStepBytes = kThreads * (16 * kSlots + (FP8 ? 8 * MT : 0));
  static constexpr int kStageBytes = kSteps * kStepBytes;
  static constexpr size_t kRedBytes = static_cast<size_t>(kWarps) * MT * NT * 4 * 32 * 4;
  static_assert(kStages * kStageBytes + kRedBytes +
                        groups_bytes(MOE_LAYER_MAX_TOKENS, MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED,
                                     kMaxExperts) <= 227 * 1024, "shared memory budget");
  static size_t smem(const LayerArgs& a) {
    return kStages * kStageBytes + kRedBytes + groups_bytes(a.T, a.K + a.S, a.E + a.S);
  }
};

// Tile `tile` of the outputs for tokens [c0, c0 + 8 NT) of the expert in slot
// `slot`; q = slot * tiles + tile.
struct Job {
  int q, slot, tile, c0;
};

template <typename S>
struct Kernel {
  const LayerArgs& a;
  const Groups& g;
  uint32_t fifo;  // shared-memory address of this thread's queue
  int tiles, kd, stages, nq;
  int lane, warp;
  int team;       // warps that share a job and split its k
  int first_q, stride_q, part;

  __device__ Kernel(const LayerArgs& args, const Groups& groups, uint8_t* smem)
      : a(args), g(groups), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    fifo = smem_addr(smem) + threadIdx.x * 16;
    kd = S::UP ? a.H : a.I;
    tiles = ((S::UP ? a.I : a.H) + S::kRows - 1) / S::kRows;
    constexpr int kPer = S::kSteps * (S::FP8 ? 64 : 32);
    stages = (kd + kPer - 1) / kPer;
    nq = g.nslots * tiles;
    team = 1;
    while (team < kWarps && nq * team < 4 * kWarps * static_cast<int>(gridDim.x) && team < stages) team *= 2;
    first_q = blockIdx.x + gridDim.x * (warp / team);
    stride_q = gridDim.x * (kWarps / team);
    part = warp % team;
  }

  __device__ __forceinline__ bool valid(const Job& j) const { return j.q < nq; }
  __device__ __forceinline__ Job at(int q) const {
    const int slot = q / tiles;
    return Job{q, slot, q - slot * tiles, 0};
  }
  __device__ __forceinline__ Job next(Job j) const {
    j.c0 += 8 * S::NT;
    return j.c0 < g.cnt[g.slot_expert[j.slot]] ? j : at(j.q + stride_q);
  }

  // Where the next copies of this warp come from.
  struct Cursor {
    Job j;
    int stage;
    const uint8_t* row;   // the lane's first weight row
    const float* scale;   // its block scales
    int col[S::NT];       // the lane's entry (up: token) per token tile, -1: none
    int first_row;
  };

  __device__ __forceinline__ void open(Cursor& c) const {
    if (!valid(c.j)) return;
    const int p = g.slot_expert[c.j.slot];
    const int e = p < a.S ? a.E + p : p - a.S;
    constexpr int kEb = S::FP8 ? 1 : 2;
    c.first_row = c.j.tile * S::kRows;
    const int rows = S::UP ? 2 * a.I : a.H;
    c.row = (S::UP ? a.w13 : a.w2) +
            (static_cast<int64_t>(e) * rows + c.first_row + (lane >> 2)) * kd * kEb;
    if (S::FP8)
      c.scale = (S::UP ? a.s13 : a.s2) +
                static_cast<int64_t>(e) * ((rows + 127) / 128) * ((kd + 127) / 128);
    const int cnt = g.cnt[p], at = g.start[p];
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) {
      const int n = c.j.c0 + nt * 8 + (lane >> 2);
      c.col[nt] = n < cnt ? (S::UP ? g.order[at + n] / (a.K + a.S) : g.order[at + n]) : -1;
    }
  }
  __device__ __forceinline__ Cursor begin() const {
    Cursor c;
    c.j = at(first_q);
    c.stage = part;
    if (part >= stages) c.j.q = nq;  // more warps than stages
    open(c);
    return c;
  }
  __device__ __forceinline__ void advance(Cursor& c) const {
    c.stage += team;
    if (c.stage < stages) return;
    c.stage = part;
    c.j = next(c.j);
    open(c);
  }

  __device__ __forceinline__ void copy_weights(const Cursor& c, int slot) const {
    if (!valid(c.j)) return;
    constexpr int kEb = S::FP8 ? 1 : 2;
    const int64_t half = static_cast<int64_t>(S::UP ? a.I : 8) * kd * kEb;
#pragma unroll
    for (int st = 0; st < S::kSteps; ++st) {
      const uint32_t dst = fifo + slot * S::kStageBytes + st * S::kStepBytes;
      const int step = c.stage * S::kSteps + st;
      const int o = step * 64 + (lane & 3) * 16;
      const bool in = o < kd * kEb;
#pragma unroll
      for (int mt = 0; mt < S::MT; ++mt) {
        const int r = c.first_row + mt * (S::UP ? 8 : 16);  // outputs are whole 8-row groups
        const uint8_t* p = c.row + static_cast<int64_t>(mt * (S::UP ? 8 : 16)) * kd * kEb + o;
        const bool row_ok = r < (S::UP ? a.I : a.H);
        const bool ok0 = in && row_ok;
        const bool ok1 = S::UP ? ok0 : in && r + 8 < a.H;
        copy16_stream(dst + (2 * mt) * kThreads * 16, ok0 ? p : c.row, ok0);
        copy16_stream(dst + (2 * mt + 1) * kThreads * 16, ok1 ? p + half : c.row, ok1);
        if (S::FP8) {
          const int kb = (kd + 127) / 128;
          const bool ok = row_ok && step * 64 < kd;
          const float* s0 = c.scale + static_cast<int64_t>(r / 128) * kb + step / 2;
          const float* s1 = S::UP ? c.scale + static_cast<int64_t>((a.I + r) / 128) * kb + step / 2 : s0;
          const uint32_t sd = dst - threadIdx.x * 16 + S::kSlots * kThreads * 16 +
                              (mt * kThreads + threadIdx.x) * 8;
          // also where this lane's bytes lie behind the row's end: the scale
          // is for the sums it receives
          copy4(sd, ok ? s0 : c.scale, ok);
          copy4(sd + 4, ok ? s1 : c.scale, ok);
        }
      }
    }
  }
  __device__ __forceinline__ void copy_tokens(const Cursor& c, int slot) const {
    if (!valid(c.j)) return;
    const uint8_t* src = S::UP ? a.x : reinterpret_cast<const uint8_t*>(a.a);
    const int64_t low = static_cast<int64_t>(a.T) * (a.K + a.S) * kd * 2;
#pragma unroll
    for (int st = 0; st < S::kSteps; ++st) {
      const uint32_t dst = fifo + slot * S::kStageBytes + st * S::kStepBytes +
                           2 * S::MT * kThreads * 16;
      // bytes of a bf16 row
      const int o = ((c.stage * S::kSteps + st) * 64 + (lane & 3) * 16) * (S::FP8 ? 2 : 1);
      const bool in = o < kd * 2;
#pragma unroll
      for (int nt = 0; nt < S::NT; ++nt) {
        const bool ok = in && c.col[nt] >= 0;
        const uint8_t* p = ok ? src + static_cast<int64_t>(c.col[nt]) * kd * 2 + o : src;
#pragma unroll
        for (int h = 0; h < S::kParts; ++h)
#pragma unroll
          for (int v = 0; v < S::kVec; ++v)
            copy16_keep(dst + ((nt * S::kParts + h) * S::kVec + v) * kThreads * 16,
                        ok ? p + h * low + v * 16 : src, ok);
      }
    }
  }

  // acc += the products of one step of the queue's slot.
  __device__ __forceinline__ void products(float (&acc)[S::MT][S::NT][4], int slot, int step) const {
    const uint32_t at = fifo + slot * S::kStageBytes + step * S::kStepBytes;
    Vec16 b[S::NT][S::kParts][S::kVec];
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
      for (int h = 0; h < S::kParts; ++h)
#pragma unroll
        for (int v = 0; v < S::kVec; ++v)
          b[nt][h][v] = lds16(at + (2 * S::MT + (nt * S::kParts + h) * S::kVec + v) * kThreads * 16);
#pragma unroll
    for (int mt = 0; mt < S::MT; ++mt) {
      const Vec16 w0 = lds16(at + (2 * mt) * kThreads * 16);
      const Vec16 w1 = lds16(at + (2 * mt + 1) * kThreads * 16);
      if (!S::FP8) {
#pragma unroll
        for (int q = 0; q < 4; q += 2)
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
            for (int h = 0; h < S::kParts; ++h)
              mma_bf16(acc[mt][nt], w0.u[q], w1.u[q], w0.u[q + 1], w1.u[q + 1], b[nt][h][0].u[q],
                       b[nt][h][0].u[q + 1]);
      } else {
        const uint32_t sd = at - threadIdx.x * 16 + S::kSlots * kThreads * 16 +
                            (mt * kThreads + threadIdx.x) * 8;
        const float f0 = lds4(sd), f1 = lds4(sd + 4);
        float sum[S::NT][4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a0 = bf16x2_of_e4m3x2(w0.u[q]), a2 = bf16x2_of_e4m3x2(w0.u[q] >> 16);
          const uint32_t a1 = bf16x2_of_e4m3x2(w1.u[q]), a3 = bf16x2_of_e4m3x2(w1.u[q] >> 16);
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
            for (int h = 0; h < S::kParts; ++h)
              mma_bf16(sum[nt], a0, a1, a2, a3, b[nt][h][q / 2].u[q % 2 * 2],
                       b[nt][h][q / 2].u[q % 2 * 2 + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < S::NT; ++nt) {
          acc[mt][nt][0] = fmaf(f0, sum[nt][0], acc[mt][nt][0]);
          acc[mt][nt][1] = fmaf(f0, sum[nt][1], acc[mt][nt][1]);
          acc[mt][nt][2] = fmaf(f1, sum[nt][2], acc[mt][nt][2]);
          acc[mt][nt][3] = fmaf(f1, sum[nt][3], acc[mt][nt][3]);
        }
      }
    }
  }
};

__device__ __forceinline__ float act_value(float g, int act) {
  const float c = act == MOE_ACT_GELU
                      ? 1.5957691216057308f * g * (1.0f + 0.044715f * g * g) : g;
  return c < -80.0f ? g * 0.0f : g * __fdividef(1.0f, 1.0f + __expf(-c));
}

__device__ __forceinline__ void team_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}

template <typename S>
__global__ void __launch_bounds__(kThreads, S::MT * S::NT == 1 ? 2 : 1) layer_kernel(LayerArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  if (S::UP) {
    // what this grid reads of earlier ones is complete from here on; the down
    // grid starts behind this point, so it may read all but this grid's `a`
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  }
  float* red = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);
  Groups g;
  group_entries(a, g, smem + S::kStages * S::kStageBytes + S::kRedBytes);
  const Kernel<S> k(a, g, smem);
  const int lane = k.lane, warp = k.warp;
  const int KS = a.K + a.S;
  if (S::UP && blockIdx.x == 0) {
    for (int t = threadIdx.x; t < g.tokens; t += kThreads) {
      uint32_t kept = 0;
      for (int kk = 0; kk < KS; ++kk) kept |= (g.rank[t * KS + kk] != kNone ? 1u : 0u) << kk;
      a.kept[t] = kept;
    }
  }

  typename Kernel<S>::Cursor next = k.begin();
  {
    typename Kernel<S>::Cursor c = next;
#pragma unroll
    for (int s = 0; s < S::kStages; ++s) {
      k.copy_weights(c, s);
      if (k.valid(c.j)) k.advance(c);
    }
  }
  if (!S::UP) asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) {
    k.copy_tokens(next, s);
    copies_commit();
    if (k.valid(next.j)) k.advance(next);
  }

  int slot = 0;
  for (Job j = k.at(k.first_q); k.valid(j); j = k.next(j)) {
    float acc[S::MT][S::NT][4] = {};
    for (int st = k.part; st < k.stages; st += k.team) {
      copies_wait<S::kStages - 1>();
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) k.products(acc, slot, i);
      // the products have read the slot; its next contents
      k.copy_weights(next, slot);
      k.copy_tokens(next, slot);
      copies_commit();
      if (k.valid(next.j)) k.advance(next);
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
    }
    if (k.team > 1) {  // the team's partial sums, added in warp order
      const int id = warp / k.team;
      team_sync(id, k.team * 32);
#pragma unroll
      for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < S::NT; ++nt)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            red[((warp * S::MT * S::NT + mt * S::NT + nt) * 4 + r) * 32 + lane] = acc[mt][nt][r];
      team_sync(id, k.team * 32);
    }
    const int p = g.slot_expert[j.slot];
    const int cnt = g.cnt[p], at = g.start[p], r0 = j.tile * S::kRows;
#pragma unroll
    for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < S::NT; ++nt) {
        const int tile = mt * S::NT + nt;
        if (tile % k.team != k.part) continue;
        float v[4];
        if (k.team > 1) {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = 0.0f;
          for (int wv = warp - k.part; wv < warp - k.part + k.team; ++wv)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              v[r] += red[((wv * S::MT * S::NT + tile) * 4 + r) * 32 + lane];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[mt][nt][r];
        }
        const int n = j.c0 + nt * 8 + 2 * (lane & 3);
        const int row = r0 + mt * (S::UP ? 8 : 16) + (lane >> 2);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (n + c >= cnt) continue;
          const int entry = g.order[at + n + c];
          if (S::UP) {
            if (row >= a.I) continue;
            const float h = act_value(v[c], a.act) * v[2 + c];
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            const float rest = h - __bfloat162float(hi);
            __nv_bfloat16* dst = a.a + static_cast<int64_t>(entry) * a.I + row;
            dst[0] = hi;
            dst[static_cast<int64_t>(a.T) * KS * a.I] =
                __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
          } else {
            float* y = a.y + static_cast<int64_t>(entry) * a.H + row;
            if (row < a.H) y[0] = v[c];
            if (row + 8 < a.H) y[8] = v[2 + c];
          }
        }
      }
  }
}

// out[t] = round(sum over the token's entries of weight * y), in k order; a
// thread per 4 columns of a token.
__global__ void __launch_bounds__(kThreads) layer_combine_kernel(LayerArgs a) {
  grid_dependency_wait();
  const int KS = a.K + a.S;
  const int tokens = a.live ? min(max(__ldg(a.live), 0), a.T) : a.T;
  const int per = a.H / 4;
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int t = i / per, col = (i - t * per) * 4;
  if (t >= tokens) return;
  const uint32_t kept = __ldg(a.kept + t);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* y = a.y + static_cast<int64_t>(t) * KS * a.H + col;
#pragma unroll 4
  for (int k = 0; k < KS; ++k) {
    if (!((kept >> k) & 1u)) continue;
    const float w = k < a.K ? __ldg(a.w + t * a.K + k) : 1.0f;
    const float4 f = __ldg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(k) * a.H));
    v.x = fmaf(w, f.x, v.x);
    v.y = fmaf(w, f.y, v.y);
    v.z = fmaf(w, f.z, v.z);
    v.w = fmaf(w, f.w, v.w);
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 o;
  o.x = *reinterpret_cast<const uint32_t*>(&lo);
  o.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(t) * a.H + col) = o;
}

cudaError_t launch_combine_layer(const LayerArgs& a, cudaStream_t s) {
  const long long n = static_cast<long long>(a.T) * (a.H / 4);
  return launch_chained(layer_combine_kernel, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)),
                        dim3(kThreads), 0, s, false, a);
}

constexpr size_t kUpSmem = 116 * 1024;

template <typename S>
cudaError_t launch_shape(const moe_handle* h, const LayerArgs& a, cudaStream_t s) {
  auto k = layer_kernel<S>;
  // over half an SM's shared memory, so that every SM gets one block of the
  // up grid, whatever still runs there when the grid is scheduled
  const size_t smem = S::UP && S::smem(a) < kUpSmem ? kUpSmem : S::smem(a);
  // per device and cheap: no state to keep
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(h->num_sms), dim3(kThreads), smem, s, false, a);
}

}  // namespace

LayerPlan layer_plan(int T, int K, int S, int H, int I) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t entries = static_cast<size_t>(T) * (K + S);
  LayerPlan p;
  p.a = 0;
  p.y = up(2 * entries * I * sizeof(__nv_bfloat16));
  p.kept = p.y + up(entries * H * sizeof(float));
  p.total = p.kept + up(static_cast<size_t>(T) * sizeof(uint32_t));
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
  a.kept = reinterpret_cast<uint32_t*>(ws + p.kept);
  a.out = static_cast<__nv_bfloat16*>(q.d_out);
  a.T = T;
  a.K = K;
  a.S = q.num_shared;
  a.E = h->cfg.num_experts;
  a.H = q.H;
  a.I = q.I;
  a.act = q.act;
  a.flags = h->flags;
  const bool fp8 = q.weight_dtype == MOE_E4M3;
  const bool many = static_cast<int64_t>(T) * K > 6 * static_cast<int64_t>(a.E);
  cudaError_t e;
  if (many) {
    e = fp8 ? launch_shape<Shape<2, 4, 1, 3, true, true>>(h, a, s)
            : launch_shape<Shape<2, 4, 1, 5, false, true>>(h, a, s);
    if (e != cudaSuccess) return e;
    e = fp8 ? launch_shape<Shape<2, 4, 1, 2, true, false>>(h, a, s)
            : launch_shape<Shape<2, 4, 1, 3, false, false>>(h, a, s);
  } else {
    e = fp8 ? launch_shape<Shape<1, 1, 2, 3, true, true>>(h, a, s)
            : launch_shape<Shape<1, 1, 2, 4, false, true>>(h, a, s);
    if (e != cudaSuccess) return e;
    e = fp8 ? launch_shape<Shape<1, 1, 1, 4, true, false>>(h, a, s)
            : launch_shape<Shape<1, 1, 2, 3, false, false>>(h, a, s);
  }
  return e != cudaSuccess ? e : launch_combine_layer(a, s);
}

}  // namespace moe
