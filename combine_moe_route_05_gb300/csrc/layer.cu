// A whole MoE layer for a few tokens (sm_103a): after the routing, one kernel
// that streams the reached experts' weights once.
//
//   up:      a[t,k,i] = act(<w13_e[i], x_t>) * <w13_e[I + i], x_t>
//   down:    y[t,k,n] = <w2_e[n], a[t,k]>                            (fp32)
//   combine: out[t]   = round(sum_k w[t,k] y[t,k] + sum_j y[t, K + j])
//
// With at most 128 tokens an expert sees a handful of them, so the layer is
// bound by reading its weights.  The products run on mma.m16n8k16 with 16
// weight rows as the one operand and 8 of the expert's tokens as the other.
// The order of the k index is free as long as both operands agree, so a lane
// takes 16 contiguous bytes of its two weight rows as the operand registers
// of two (bf16) or four (e4m3) products, with its token's values at the same
// k beside them.  In the up products rows 0..7 of the 16 are gate rows and
// 8..15 the up rows of the same outputs: a lane's accumulators then hold gate
// and up of one output and the activation needs no exchange.
//
// Every lane copies what it will itself multiply into a queue of its own in
// shared memory (cp.async), several steps ahead and across the ends of jobs,
// so the stream of weights has no gaps and the queue needs no barrier.  A job
// is one expert and one tile of outputs; a team of 1, 2, 4 or 8 warps, as many
// as make the jobs fill the grid evenly, splits its k and adds its partial
// sums in warp order.  Jobs go round over the blocks, expert by expert, so
// that neighbouring blocks read neighbouring rows and the experts with many
// tokens spread over all blocks.
//
// The three parts are one cooperative kernel, with grid-wide barriers between
// them (bounded waits): the queue takes the first W2 rows before it waits for
// the up products.  Results do not depend on the order of blocks or warps.
//
// Precision: products and sums are fp32.  bf16 weights: x is taken as it is,
// and a as the sum of two bf16 numbers (16 bits), which costs a second
// product; one bf16 would add an error as large as the output's own rounding.
// e4m3 weights become fp16 exactly (one conversion for two weights, a bf16
// would take four); x becomes fp16 times a power of two that brings its
// token's largest value to [2^14, 2^15) (exact down to 2^-29 of that), and a
// likewise per entry (11 bits).
#include <cstdint>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxEntries = MOE_LAYER_MAX_TOKENS * (MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED);
constexpr int kMaxExperts = MOE_MAX_EXPERTS + MOE_LAYER_MAX_SHARED;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint16_t kNone = 0xffff;
constexpr int kSlotBytes = kThreads * 16;  // 16 bytes per lane
constexpr int kQueueBytes = 192 * 1024;

struct LayerArgs {
  const uint8_t* x;      // [T, H] bf16
  const int32_t* idx;    // [T, K]
  const float* w;        // [T, K]
  const int32_t* live;   // live tokens or NULL
  const uint8_t* w13;    // [E + S, 2I, H]
  const uint8_t* w2;     // [E + S, H, I]
  const float* s13;      // block scales of e4m3 weights
  const float* s2;
  __half* x16;           // [T, H] scaled x (e4m3)
  float* xscale;         // [T] 1 / its factor (e4m3)
  uint8_t* a;            // bf16 weights: bf16 [2][T (K + S), I], high and low part;
                         // e4m3: fp32 [T (K + S), I]
  uint32_t* amax;        // [T (K + S)] bits of the largest |a| of an entry (e4m3)
  float* y;              // [T (K + S), H]
  uint32_t* arrived;     // blocks that reached each grid barrier, zero at the start
  __nv_bfloat16* out;    // [T, H]
  int T, K, S, E, H, I;
  int act;
  unsigned long long wait_ns;
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
  return 2 * up16(2ull * T * KS) + up16(2ull * n_exp) + 2 * up16(4ull * n_exp) +
         up16(4ull * (kWarps + 1));
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
  constexpr int kMine = kMaxEntries / kThreads;
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
// grid-wide barriers

__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Waits until every block of the grid has come here; false, with the status
// bit set, after the handle's limit.
__device__ __forceinline__ bool grid_barrier(const LayerArgs& a, uint32_t* arrived, int* ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(arrived, 1u);
    const unsigned long long t0 = global_ns();
    bool done = true;
    for (;;) {
      uint32_t n;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(arrived) : "memory");
      if (n >= gridDim.x) break;
      if (global_ns() - t0 > a.wait_ns) {
        raise_flag(a.flags, MOE_DEVERR_TIMEOUT);
        done = false;
        break;
      }
    }
    __threadfence();
    *ok = done;
  }
  __syncthreads();
  return *ok != 0;
}

// ---------------------------------------------------------------------------
// copies and products

// Asynchronous copies of 16 bytes into shared memory; !valid writes zeros and
// reads nothing.  Weights pass by L1, tokens are kept in it.
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

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 values as two pairs of fp16 (exact; NaN stays NaN).
__device__ __forceinline__ void f16_of_e4m3(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two that brings a largest magnitude (its bits) to [2^14, 2^15);
// 1 for zero and for what is not finite.
__device__ __forceinline__ float f16_factor(uint32_t max_bits) {
  const int e = static_cast<int>(max_bits >> 23);
  if (max_bits == 0 || e >= 255) return 1.0f;
  return __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 + 127 - e, 1), 253)) << 23);
}

__device__ __forceinline__ float act_value(float g, int act) {
  const float c = act == MOE_ACT_GELU
                      ? 1.5957691216057308f * g * (1.0f + 0.044715f * g * g) : g;
  return c < -80.0f ? g * 0.0f : g * __fdividef(1.0f, 1.0f + __expf(-c));
}

// MT tiles of 16 weight rows by NT tiles of 8 tokens a job.
template <int MT_, int NT_, bool FP8_>
struct Shape {
  static constexpr int MT = MT_, NT = NT_;
  static constexpr bool FP8 = FP8_;
  // token vectors beside a weight vector: x, or a's two bf16 parts or fp32
  static constexpr int kVecUp = FP8 ? 2 : 1, kVecDown = FP8 ? 4 : 2;
  static constexpr int kSlotsUp = 2 * MT + NT * kVecUp, kSlotsDown = 2 * MT + NT * kVecDown;
  static constexpr int kStagesUp = kQueueBytes / (kSlotsUp * kSlotBytes);
  static constexpr int kStagesDown = kQueueBytes / (kSlotsDown * kSlotBytes);
  static constexpr size_t kRedBytes = static_cast<size_t>(kWarps) * MT * NT * 4 * 32 * 4;
  static constexpr size_t smem(int T, int KS, int n_exp) {
    return kQueueBytes + kRedBytes + groups_bytes(T, KS, n_exp) + (FP8 ? up16(4ull * T * KS) : 0);
  }
  static_assert(kStagesUp >= 2 && kStagesDown >= 2, "queue");
  static_assert(smem(MOE_LAYER_MAX_TOKENS, MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED, kMaxExperts) <=
                    227 * 1024, "shared memory budget");
};

// Tokens [c0, c0 + 8 NT) of the expert in slot `slot`, output tile `tile`;
// q = slot * tiles + tile.
struct Job {
  int q, slot, tile, c0;
};

// The products of one phase (up or down) for one thread.
template <typename S>
struct Phase {
  const LayerArgs& a;
  const Groups& g;
  bool up;
  uint32_t queue;   // shared-memory address of this lane's queue
  int tiles, kd, steps, nq;
  int rows;         // outputs a tile of 16 weight rows gives: 8 (up) or 16
  int limit;        // outputs in all
  int lane, warp, team, part, first_q, stride_q;
  int stage_bytes;
  int64_t half;     // bytes from a lane's first weight row to its second
  const uint8_t* weights;
  const float* scales;
  int scale_rows, scale_cols;
  static constexpr int kEb = S::FP8 ? 1 : 2;
  static constexpr int kStep = 64 / kEb;  // k of a step: 64 bytes of a weight row

  __device__ __forceinline__ Phase(const LayerArgs& args, const Groups& groups, uint8_t* smem,
                                   bool is_up)
      : a(args), g(groups), up(is_up), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    queue = smem_addr(smem) + threadIdx.x * 16;
    kd = up ? a.H : a.I;
    rows = up ? 8 : 16;
    limit = up ? a.I : a.H;
    tiles = (limit + rows * S::MT - 1) / (rows * S::MT);
    steps = (kd + kStep - 1) / kStep;
    nq = g.nslots * tiles;
    stage_bytes = (up ? S::kSlotsUp : S::kSlotsDown) * kSlotBytes;
    half = static_cast<int64_t>(up ? a.I : 8) * kd * kEb;
    weights = up ? a.w13 : a.w2;
    scales = up ? a.s13 : a.s2;
    scale_rows = ((up ? 2 * a.I : a.H) + 127) / 128;
    scale_cols = (kd + 127) / 128;
    // rounds of jobs over the grid, in units of a one-warp job
    team = 1;
    const int warps = kWarps * gridDim.x;
    float best = 0.0f;
#pragma unroll 1
    for (int n = 1; n <= 8 && n <= steps; n *= 2) {
      const float cost = static_cast<float>((nq * n + warps - 1) / warps) / n;
      if (n == 1 || cost < best) {
        best = cost;
        team = n;
      }
    }
    first_q = blockIdx.x + gridDim.x * (warp / team);
    stride_q = gridDim.x * (kWarps / team);
    part = warp % team;
  }

  __device__ __forceinline__ bool valid(const Job& j) const { return j.q < nq; }
  __device__ __forceinline__ Job at(int q) const {
    const int slot = q / tiles;
    return Job{q, slot, q - slot * tiles, 0};
  }
  __device__ __forceinline__ Job next(const Job& j) const {
    if (j.c0 + 8 * S::NT < g.cnt[g.slot_expert[j.slot]])
      return Job{j.q, j.slot, j.tile, j.c0 + 8 * S::NT};
    return at(j.q + stride_q);
  }

  // Where the next copies of this warp come from.
  struct Cursor {
    Job j;
    int step;
    const uint8_t* row;        // the lane's first weight row
    const uint8_t* col[S::NT]; // its token's values per token tile, NULL: none
  };

  __device__ __forceinline__ void open(Cursor& c) const {
    if (!valid(c.j)) return;
    const int p = g.slot_expert[c.j.slot];
    const int e = p < a.S ? a.E + p : p - a.S;
    c.row = weights + (static_cast<int64_t>(e) * (up ? 2 * a.I : a.H) + c.j.tile * rows * S::MT +
                       (lane >> 2)) * kd * kEb;
    const int cnt = g.cnt[p], at = g.start[p];
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) {
      const int n = c.j.c0 + nt * 8 + (lane >> 2);
      c.col[nt] = nullptr;
      if (n >= cnt) continue;
      const int entry = g.order[at + n];
      if (up)
        c.col[nt] = (S::FP8 ? reinterpret_cast<const uint8_t*>(a.x16) : a.x) +
                    static_cast<int64_t>(entry / (a.K + a.S)) * kd * 2;
      else
        c.col[nt] = a.a + static_cast<int64_t>(entry) * kd * (S::FP8 ? 4 : 2);
    }
  }
  __device__ __forceinline__ Cursor begin() const {
    Cursor c;
    c.j = at(first_q);
    c.step = part;
    open(c);
    return c;
  }
  __device__ __forceinline__ void advance(Cursor& c) const {
    if (!valid(c.j)) return;
    c.step += team;
    if (c.step < steps) return;
    c.step = part;
    c.j = next(c.j);
    open(c);
  }

  __device__ __forceinline__ void copy_weights(const Cursor& c, int stage) const {
    if (!valid(c.j)) return;
    const uint32_t dst = queue + stage * stage_bytes;
    const int o = c.step * 64 + (lane & 3) * 16;
    const bool in = o < kd * kEb;
#pragma unroll
    for (int mt = 0; mt < S::MT; ++mt) {
      const int r = (c.j.tile * S::MT + mt) * rows;  // outputs come in whole eights
      const uint8_t* p = c.row + static_cast<int64_t>(mt * rows) * kd * kEb + o;
      const bool ok0 = in && r < limit, ok1 = ok0 && (up || r + 8 < limit);
      copy16_stream(dst + (2 * mt) * kSlotBytes, ok0 ? p : c.row, ok0);
      copy16_stream(dst + (2 * mt + 1) * kSlotBytes, ok1 ? p + half : c.row, ok1);
    }
  }
  __device__ __forceinline__ void copy_tokens(const Cursor& c, int stage) const {
    if (!valid(c.j)) return;
    const uint32_t dst = queue + stage * stage_bytes + 2 * S::MT * kSlotBytes;
    const int k = c.step * kStep + (lane & 3) * (16 / kEb);
    const bool in = k < kd;
    const int bytes = k * (S::FP8 && !up ? 4 : 2);
    // the second vector: the next 16 bytes, or a's low part
    const int64_t second = S::FP8 ? 16 : static_cast<int64_t>(a.T) * (a.K + a.S) * kd * 2;
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) {
      const bool ok = in && c.col[nt];
      const uint8_t* p = ok ? c.col[nt] + bytes : weights;
      const uint32_t d = dst + nt * (up ? S::kVecUp : S::kVecDown) * kSlotBytes;
      copy16_keep(d, p, ok);
      if (S::FP8 || !up) copy16_keep(d + kSlotBytes, ok ? p + second : p, ok);
      if (S::FP8 && !up) {
        copy16_keep(d + 2 * kSlotBytes, ok ? p + 32 : p, ok);
        copy16_keep(d + 3 * kSlotBytes, ok ? p + 48 : p, ok);
      }
    }
  }

  // acc += the products of one step.  factor[nt]: what brings the lane's
  // entry to fp16; sc0 / sc1: block scales of the lane's accumulator rows.
  __device__ __forceinline__ void products(float (&acc)[S::MT][S::NT][4], int stage,
                                           const float (&factor)[S::NT],
                                           const float (&sc)[S::MT][2]) const {
    const uint32_t at = queue + stage * stage_bytes;
    constexpr int kWords = S::FP8 ? 8 : 4;  // operand words of the lane's token
    uint32_t b[S::NT][S::FP8 ? 1 : 2][kWords];
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) {
      const uint32_t d = at + (2 * S::MT + nt * (up ? S::kVecUp : S::kVecDown)) * kSlotBytes;
      if (!S::FP8) {
        const Vec16 hi = lds16(d);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[nt][0][i] = hi.u[i];
        if (!up) {
          const Vec16 lo = lds16(d + kSlotBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) b[nt][S::FP8 ? 0 : 1][i] = lo.u[i];
        }
      } else if (up) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const Vec16 x = lds16(d + v * kSlotBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) b[nt][0][(v * 4 + i) % kWords] = x.u[i];
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const Vec16 f = lds16(d + v * kSlotBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            b[nt][0][(v * 2 + i) % kWords] = f16x2(__uint_as_float(f.u[2 * i]) * factor[nt],
                                                   __uint_as_float(f.u[2 * i + 1]) * factor[nt]);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < S::MT; ++mt) {
      const Vec16 w0 = lds16(at + (2 * mt) * kSlotBytes);
      const Vec16 w1 = lds16(at + (2 * mt + 1) * kSlotBytes);
      if (!S::FP8) {
#pragma unroll
        for (int q = 0; q < 4; q += 2)
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt) {
            mma<false>(acc[mt][nt], w0.u[q], w1.u[q], w0.u[q + 1], w1.u[q + 1], b[nt][0][q],
                       b[nt][0][q + 1]);
            if (!up)
              mma<false>(acc[mt][nt], w0.u[q], w1.u[q], w0.u[q + 1], w1.u[q + 1],
                         b[nt][S::FP8 ? 0 : 1][q], b[nt][S::FP8 ? 0 : 1][q + 1]);
          }
      } else {
        float sum[S::NT][4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a0, a1, a2, a3;
          f16_of_e4m3(w0.u[q], a0, a2);
          f16_of_e4m3(w1.u[q], a1, a3);
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt)
            mma<true>(sum[nt], a0, a1, a2, a3, b[nt][0][(2 * q) % kWords],
                      b[nt][0][(2 * q + 1) % kWords]);
        }
#pragma unroll
        for (int nt = 0; nt < S::NT; ++nt) {
          acc[mt][nt][0] = fmaf(sc[mt][0], sum[nt][0], acc[mt][nt][0]);
          acc[mt][nt][1] = fmaf(sc[mt][0], sum[nt][1], acc[mt][nt][1]);
          acc[mt][nt][2] = fmaf(sc[mt][1], sum[nt][2], acc[mt][nt][2]);
          acc[mt][nt][3] = fmaf(sc[mt][1], sum[nt][3], acc[mt][nt][3]);
        }
      }
    }
  }

  // One result pair of entry `entry`: up: gate and up of output `row`; down:
  // outputs row and row + 8.
  __device__ __forceinline__ void store(int entry, int row, float v0, float v1,
                                        const float* inverse) const {
    if (row >= limit) return;
    const int KS = a.K + a.S;
    if (!up) {
      if (S::FP8) {
        v0 *= inverse[entry];
        v1 *= inverse[entry];
      }
      float* y = a.y + static_cast<int64_t>(entry) * a.H + row;
      y[0] = v0;
      if (row + 8 < limit) y[8] = v1;
      return;
    }
    if (S::FP8) {
      const float f = __ldcg(a.xscale + entry / KS);
      const float h = act_value(v0 * f, a.act) * (v1 * f);
      reinterpret_cast<float*>(a.a)[static_cast<int64_t>(entry) * a.I + row] = h;
      // a maximum does not depend on the order
      atomicMax(a.amax + entry, __float_as_uint(h) & 0x7fffffffu);
    } else {
      const float h = act_value(v0, a.act) * v1;
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      const float rest = h - __bfloat162float(hi);
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.a) + static_cast<int64_t>(entry) * a.I + row;
      dst[0] = hi;
      dst[static_cast<int64_t>(a.T) * KS * a.I] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
    }
  }
};

__device__ __forceinline__ void team_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}

// fp16 copies of x and their factors: a block per token.
__device__ void scale_tokens(const LayerArgs& a, int tokens, float* red) {
  for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
    const uint8_t* row = a.x + static_cast<int64_t>(t) * a.H * 2;
    uint32_t m = 0;  // the largest |x|, as bits of a bf16 in the high half
    for (int v = threadIdx.x; v < a.H / 8; v += kThreads) {
      const Vec16 x = ld_vec(row + v * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = max(m, max(x.u[i] & 0x7fff0000u, (x.u[i] << 16) & 0x7fff0000u));
    }
    m = __reduce_max_sync(kFull, m);
    if ((threadIdx.x & 31) == 0) reinterpret_cast<uint32_t*>(red)[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = max(m, reinterpret_cast<uint32_t*>(red)[i]);
    __syncthreads();
    const float f = f16_factor(m);
    uint8_t* dst = reinterpret_cast<uint8_t*>(a.x16) + static_cast<int64_t>(t) * a.H * 2;
    for (int v = threadIdx.x; v < a.H / 8; v += kThreads) {
      float e[8];
      VecTraits<__nv_bfloat16>::to_f32(ld_vec(row + v * 16), e);
      Vec16 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.u[i] = f16x2(e[2 * i] * f, e[2 * i + 1] * f);
      st_vec(dst + v * 16, o);
    }
    if (threadIdx.x == 0) a.xscale[t] = 1.0f / f;
    for (int k = threadIdx.x; k < a.K + a.S; k += kThreads) a.amax[t * (a.K + a.S) + k] = 0;
  }
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(LayerArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int ok;
  grid_dependency_wait();
  float* red = reinterpret_cast<float*>(smem + kQueueBytes);
  uint8_t* tables = smem + kQueueBytes + S::kRedBytes;
  float* inverse = reinterpret_cast<float*>(tables + groups_bytes(a.T, a.K + a.S, a.E + a.S));
  Groups g;
  group_entries(a, g, tables);
  const int KS = a.K + a.S;
  if (S::FP8) scale_tokens(a, g.tokens, red);

#pragma unroll 1
  for (int ph = 0; ph < 2; ++ph) {
    const Phase<S> k(a, g, smem, ph == 0);
    const int lane = k.lane, warp = k.warp;
    const int stages = k.up ? S::kStagesUp : S::kStagesDown;
    typename Phase<S>::Cursor next = k.begin();
    {
      typename Phase<S>::Cursor c = next;
#pragma unroll 1
      for (int s = 0; s < stages; ++s) {
        k.copy_weights(c, s);
        k.advance(c);
      }
    }
    // what the tokens' side reads was written by other blocks
    if ((S::FP8 || !k.up) && !grid_barrier(a, a.arrived + ph, &ok)) {
      copies_wait<0>();
      return;
    }
    if (S::FP8 && !k.up) {
      for (int i = threadIdx.x; i < g.tokens * KS; i += kThreads)
        inverse[i] = 1.0f / f16_factor(__ldcg(a.amax + i));
      __syncthreads();
    }
#pragma unroll 1
    for (int s = 0; s < stages; ++s) {
      k.copy_tokens(next, s);
      copies_commit();
      k.advance(next);
    }

    int stage = 0;
#pragma unroll 1
    for (Job j = k.at(k.first_q); k.valid(j); j = k.next(j)) {
      const int p = g.slot_expert[j.slot];
      const int cnt = g.cnt[p], at = g.start[p];
      float factor[S::NT] = {};
      const float* scale[S::MT][2] = {};
      float held[S::MT][2] = {}, sc[S::MT][2] = {};
      if (S::FP8) {
        const int e = p < a.S ? a.E + p : p - a.S;
        const float* base = k.scales + static_cast<int64_t>(e) * k.scale_rows * k.scale_cols;
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt) {
          const int r = min((j.tile * S::MT + mt) * k.rows, k.limit - 8);
          scale[mt][0] = base + static_cast<int64_t>(r / 128) * k.scale_cols;
          scale[mt][1] = k.up ? base + static_cast<int64_t>((a.I + r) / 128) * k.scale_cols : scale[mt][0];
        }
        if (!k.up) {
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt) {
            const int n = j.c0 + nt * 8 + (lane >> 2);
            factor[nt] = n < cnt ? 1.0f / inverse[g.order[at + n]] : 0.0f;
          }
        }
      }
      float acc[S::MT][S::NT][4] = {};
      int window = -1;  // the 32 k blocks whose scales the lanes hold
#pragma unroll 1
      for (int step = k.part; step < k.steps; step += k.team) {
        if (S::FP8) {
          const int block = step / 2;
          if (block / 32 != window) {
            window = block / 32;
            const int b = min(window * 32 + lane, k.scale_cols - 1);
#pragma unroll
            for (int mt = 0; mt < S::MT; ++mt) {
              held[mt][0] = __ldg(scale[mt][0] + b);
              held[mt][1] = __ldg(scale[mt][1] + b);
            }
          }
#pragma unroll
          for (int mt = 0; mt < S::MT; ++mt) {
            sc[mt][0] = __shfl_sync(kFull, held[mt][0], block % 32);
            sc[mt][1] = __shfl_sync(kFull, held[mt][1], block % 32);
          }
        }
        if (k.up) copies_wait<S::kStagesUp - 1>();
        else copies_wait<S::kStagesDown - 1>();
        k.products(acc, stage, factor, sc);
        // the products have read the stage; its next contents
        k.copy_weights(next, stage);
        k.copy_tokens(next, stage);
        copies_commit();
        k.advance(next);
        stage = stage + 1 == stages ? 0 : stage + 1;
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
#pragma unroll
      for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < S::NT; ++nt) {
          const int tile = mt * S::NT + nt;
          if (tile % k.team != k.part) continue;
          float (&v)[4] = acc[mt][nt];
          if (k.team > 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = 0.0f;
#pragma unroll 2
            for (int wv = warp - k.part; wv < warp - k.part + k.team; ++wv)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                v[r] += red[((wv * S::MT * S::NT + tile) * 4 + r) * 32 + lane];
          }
          const int n = j.c0 + nt * 8 + 2 * (lane & 3);
          const int row = (j.tile * S::MT + mt) * k.rows + (lane >> 2);
          if (n < cnt) k.store(g.order[at + n], row, v[0], v[2], inverse);
          if (n + 1 < cnt) k.store(g.order[at + n + 1], row, v[1], v[3], inverse);
        }
    }
    copies_wait<0>();
  }

  // the entries' rows summed per token, a thread per 4 columns
  if (!grid_barrier(a, a.arrived + 2, &ok)) return;
  const int per = a.H / 4;
  const int64_t n = static_cast<int64_t>(g.tokens) * per;
  for (int64_t i = (static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 + (threadIdx.x & 31);
       i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / per), col = static_cast<int>(i - static_cast<int64_t>(t) * per) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* y = a.y + static_cast<int64_t>(t) * KS * a.H + col;
#pragma unroll 4
    for (int kk = 0; kk < KS; ++kk) {
      if (g.rank[t * KS + kk] == kNone) continue;
      const float w = kk < a.K ? __ldg(a.w + t * a.K + kk) : 1.0f;
      const float4 f = __ldcg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(kk) * a.H));
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
}

// Zeroes the barrier counters where no routing kernel does.
__global__ void layer_start_kernel(uint32_t* arrived) {
  grid_dependency_wait();
  if (threadIdx.x < kLayerCounters) arrived[threadIdx.x] = 0;
}

template <typename S>
cudaError_t launch_shape(const moe_handle* h, const LayerArgs& a, cudaStream_t s) {
  auto k = layer_kernel<S>;
  const size_t smem = S::smem(a.T, a.K + a.S, a.E + a.S);
  // per device and cheap: no state to keep
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(h->num_sms), dim3(kThreads), smem, s, true, a);
}

}  // namespace

LayerPlan layer_plan(int T, int K, int S, int H, int I) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t entries = static_cast<size_t>(T) * (K + S);
  LayerPlan p;
  p.a = 0;
  p.y = up(entries * I * sizeof(float));
  p.x16 = p.y + up(entries * H * sizeof(float));
  p.xscale = p.x16 + up(static_cast<size_t>(T) * H * sizeof(__half));
  p.amax = p.xscale + up(static_cast<size_t>(T) * sizeof(float));
  p.arrived = p.amax + up(entries * sizeof(uint32_t));
  p.total = p.arrived + 256;
  return p;
}

cudaError_t launch_layer(const moe_handle* h, const moe_layer_args& q, int T, void* workspace,
                         cudaStream_t s) {
  const int K = h->cfg.top_k;
  if (T == 0) return cudaSuccess;
  const LayerPlan p = layer_plan(T, K, q.num_shared, q.H, q.I);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* arrived = reinterpret_cast<uint32_t*>(ws + p.arrived);
  const cudaError_t e =
      q.d_logits ? launch_route_topk(h, q.d_logits, q.d_bias, T, q.d_idx, q.d_w, s, q.d_live, arrived)
                 : launch_chained(layer_start_kernel, dim3(1), dim3(32), 0, s, false, arrived);
  if (e != cudaSuccess) return e;
  LayerArgs a{};
  a.x = static_cast<const uint8_t*>(q.d_x);
  a.idx = q.d_idx;
  a.w = q.d_w;
  a.live = q.d_live;
  a.w13 = static_cast<const uint8_t*>(q.d_w13);
  a.w2 = static_cast<const uint8_t*>(q.d_w2);
  a.s13 = q.d_s13;
  a.s2 = q.d_s2;
  a.x16 = reinterpret_cast<__half*>(ws + p.x16);
  a.xscale = reinterpret_cast<float*>(ws + p.xscale);
  a.a = ws + p.a;
  a.amax = reinterpret_cast<uint32_t*>(ws + p.amax);
  a.y = reinterpret_cast<float*>(ws + p.y);
  a.arrived = arrived;
  a.out = static_cast<__nv_bfloat16*>(q.d_out);
  a.T = T;
  a.K = K;
  a.S = q.num_shared;
  a.E = h->cfg.num_experts;
  a.H = q.H;
  a.I = q.I;
  a.act = q.act;
  a.wait_ns = h->wait_ns;
  a.flags = h->flags;
  return q.weight_dtype == MOE_E4M3 ? launch_shape<Shape<1, 1, true>>(h, a, s)
                                    : launch_shape<Shape<1, 1, false>>(h, a, s);
}

}  // namespace moe
