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
// A block has one or two groups: a producer warp that copies weight rows (and
// the expert's token rows beside them) into the group's ring in shared memory
// with bulk copies, and consumer warps that split each stage's k.  A job is one
// expert and one tile of outputs.  The producer runs several stages ahead and
// across the ends of jobs, so the stream of weights has no gaps; it takes its
// jobs from a counter, because the SMs do not all get the same share of the
// memory's rate (by up to a quarter on the largest layers), and a stage takes
// only the room that its tokens need.
//
// The three parts are one cooperative kernel, with grid-wide barriers between
// them (bounded waits): the ring takes the first W2 rows before it waits for
// the up products.  Results do not depend on which block takes which job.
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

constexpr int kMaxEntries = MOE_LAYER_MAX_TOKENS * (MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED);
constexpr int kMaxExperts = MOE_MAX_EXPERTS + MOE_LAYER_MAX_SHARED;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint16_t kNone = 0xffff;
constexpr int kBarriers = 4;  // grid barriers of a call

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
  uint8_t* a;            // bf16 [2][T (K + S), I], high and low part; e4m3: fp16, scaled
  float* a32;            // [T (K + S), I] (e4m3)
  uint32_t* amax;        // [T (K + S)] bits of the largest |a| of an entry (e4m3)
  float* y;              // [T (K + S), H]
  uint32_t* arrived;     // blocks that reached each grid barrier (kBarriers), then the
                         // jobs taken of each phase; zero at the start
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

constexpr int kMaxWarps = 20;

__host__ __device__ constexpr size_t groups_bytes(int T, int KS, int n_exp) {
  return 2 * up16(2ull * T * KS) + up16(2ull * n_exp) + 2 * up16(4ull * n_exp) +
         up16(4ull * (kMaxWarps + 1));
}

__device__ __forceinline__ int expert_of(const LayerArgs& a, int entry) {
  const int t = entry / (a.K + a.S), k = entry - t * (a.K + a.S);
  if (k >= a.K) return k - a.K;
  const int e = __ldcg(a.idx + t * a.K + k);
  return static_cast<unsigned>(e) < static_cast<unsigned>(a.E) ? e + a.S : e == -1 ? -1 : -2;
}

template <int kThreads>
__device__ __forceinline__ void group_entries(const LayerArgs& a, Groups& g, uint8_t* smem) {
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
  constexpr int kMine = (kMaxEntries + kThreads - 1) / kThreads;
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
  if (tid == kThreads - 1) g.head[kMaxWarps] = (base + sum) >> 16;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kThreads;
    if (i < n && g.rank[i] != kNone) g.order[g.start[mine[j]] + g.rank[i]] = static_cast<uint16_t>(i);
  }
  g.nslots = g.head[kMaxWarps];
  __syncthreads();
}

// ---------------------------------------------------------------------------
// grid-wide barriers

__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Waits until every block of the grid has arrived; false, with the status bit
// set, after the handle's limit.  One thread.
__device__ __forceinline__ bool grid_wait(const LayerArgs& a, const uint32_t* arrived) {
  const unsigned long long t0 = global_ns();
  for (;;) {
    uint32_t n;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(arrived) : "memory");
    if (n >= gridDim.x) break;
    if (global_ns() - t0 > a.wait_ns) {
      raise_flag(a.flags, MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
  __threadfence();
  return true;
}

// Waits for a phase of a shared-memory barrier; false, with the status bit
// set, after the handle's limit.
__device__ __forceinline__ bool ring_wait(const LayerArgs& a, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (global_ns() - t0 > a.wait_ns) {
      raise_flag(a.flags, MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------------------
// copies and products

// A bulk copy of `bytes` (16-byte aligned, a multiple of 16) into shared
// memory, reported to `bar`.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
// Orders what this thread has seen of global memory before its bulk copies.
__device__ __forceinline__ void fence_bulk() { asm volatile("fence.proxy.async;" ::: "memory"); }

// 16 bytes of shared memory, zeros where !valid.  Predicated: the lanes of a
// warp differ.
__device__ __forceinline__ Vec16 lds16_if(uint32_t p, bool valid) {
  Vec16 v{};
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
      "@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "+r"(v.u[0]), "+r"(v.u[1]), "+r"(v.u[2]), "+r"(v.u[3])
      : "r"(p), "r"(static_cast<int>(valid))
      : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
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

// GROUPS groups of a block; in each, WK x WM consumer warps: WK split the k of
// a stage, WM the MT WM tiles of 16 weight rows of a job, by NT tiles of 8
// tokens.  A stage holds STEPS steps of 64 bytes of a weight row per warp.
template <int GROUPS_, int COPIERS_, int WK_, int WM_, int MT_, int NT_, int STEPS_, bool FP8_>
struct Shape {
  static constexpr int kGroups = GROUPS_, kProducers = 1 + COPIERS_, WK = WK_, WM = WM_, MT = MT_, NT = NT_, kSteps = STEPS_;
  static constexpr bool FP8 = FP8_;
  static constexpr int kEb = FP8 ? 1 : 2;
  static constexpr int kTiles = WM * MT;                 // of 16 weight rows
  static constexpr int kConsumers = WK * WM;             // warps of a group
  static constexpr int kThreads = kGroups * (kConsumers + kProducers) * 32;
  static constexpr int kRowBytes = WK * kSteps * 64;     // of a weight row in a stage, at most
  static constexpr int kScales = FP8 ? kTiles * 2 * (kRowBytes / 128) : 0;
  static constexpr int kRed = kTiles * NT == 1 ? 2 : 1;  // buffers of partial sums
  static constexpr int kRedBytes = kRed * kConsumers * NT * 4 * 32 * 4;  // of a group
  static constexpr int kStages = 16;                     // at most in a ring
  static constexpr int kReducers = WM * NT;              // warps that add a buffer's sums
  static_assert(kRowBytes % 128 == 0 && kScales <= 32 && kGroups * kConsumers <= 16 && NT <= WK, "shape");
  // the largest stage: two of them have to fit the smallest ring
  static constexpr int kStageBytes =
      16 * kTiles * (kRowBytes + 64) + 8 * NT * 2 * (kRowBytes + 64);
};

struct Stage {
  int off;    // of the weight rows in the ring
  int slot, tile, c0;
  int bytes;  // of a weight row
  int tokens;
  int what;   // kLast, kHeld, and from bit 2 on the stage's place in its rows; -1: no more jobs
  int taken;  // bytes of the ring, with what a wrap skipped
};
constexpr int kLast = 1;  // the job's last stage
constexpr int kHeld = 2;  // its tokens come later

// A group's shared memory.
template <typename S>
struct Ring {
  uint32_t base;  // the ring itself
  int size;
  Stage* stage;
  uint64_t *full, *empty, *go;     // per stage
  uint64_t *red_full, *red_empty;  // per buffer of partial sums
  float* scales;  // [stage][tile][2][block] (e4m3)
  float* red;
};

template <typename S>
constexpr size_t group_bytes(int ring) {
  return static_cast<size_t>(ring) + S::kRedBytes + S::kStages * (sizeof(Stage) + 24 + 4 * S::kScales) + 32;
}
template <typename S>
constexpr int ring_bytes(int T, int KS, int n_exp) {
  const size_t rest = 1024 + groups_bytes(T, KS, n_exp) + S::kGroups * group_bytes<S>(0);
  return static_cast<int>((227 * 1024 - rest) / S::kGroups / 128 * 128);
}

// What the warps of a group have passed of its barriers, over both phases.
struct Progress {
  int stages = 0, sums = 0;
};

// One phase (up or down) of one group.
template <typename S, bool UP>
struct Phase {
  static constexpr int MT = S::MT, NT = S::NT, kEb = S::kEb;
  static constexpr bool FP8 = S::FP8;
  static constexpr int kVec = UP ? (FP8 ? 2 : 1) : 2;    // token vectors beside a weight vector
  static constexpr int kParts = FP8 || UP ? 1 : 2;       // rows of a token: x; a's two parts
  static constexpr int kRows = UP ? 8 : 16;              // outputs of 16 weight rows
  static constexpr int kBlocks = S::kRowBytes / 128;     // block scales along a stage's rows

  const LayerArgs& a;
  const Groups& g;
  const Ring<S>& ring;
  int kd, limit, tiles, stages, nq;
  int row_bytes;           // of a weight row in a stage
  int pitch, token_pitch;  // of rows in the ring, free of bank conflicts

  __device__ __forceinline__ Phase(const LayerArgs& args, const Groups& groups, const Ring<S>& r)
      : a(args), g(groups), ring(r) {
    kd = UP ? a.H : a.I;
    limit = UP ? a.I : a.H;
    tiles = (limit + kRows * S::kTiles - 1) / (kRows * S::kTiles);
    stages = (kd * kEb + S::kRowBytes - 1) / S::kRowBytes;
    row_bytes = ((kd * kEb + stages - 1) / stages + 127) / 128 * 128;
    pitch = row_bytes + 64;
    token_pitch = FP8 ? 2 * row_bytes + 16 : pitch;
    nq = g.nslots * tiles;
  }
  __device__ __forceinline__ int expert(int slot) const {
    const int p = g.slot_expert[slot];
    return p < a.S ? a.E + p : p - a.S;
  }

  // ------------------------------------------------------------- producer
  struct Place {
    int q, slot, tile, c0, st;
  };
  __device__ __forceinline__ Place at(int q) const {
    const int slot = q / tiles;
    return Place{q, slot, q - slot * tiles, 0, 0};
  }
  __device__ __forceinline__ bool valid(const Place& p) const { return p.q < nq; }

  // The block scales of a stage, one per lane.
  __device__ __forceinline__ float scale_of(const Place& p, int lane) const {
    if (!FP8 || !valid(p) || lane >= S::kScales) return 0.0f;
    const int cols = (kd + 127) / 128;
    const int block = min(p.st * (row_bytes / 128) + lane % kBlocks, cols - 1);
    const int h = lane / kBlocks % 2, mt = lane / kBlocks / 2;
    const int r = min((p.tile * S::kTiles + mt) * kRows, limit - 8) + (UP && h ? a.I : 0);
    return __ldg((UP ? a.s13 : a.s2) +
                 (static_cast<int64_t>(expert(p.slot)) * (((UP ? 2 * a.I : a.H) + 127) / 128) + r / 128) * cols +
                 block);
  }

  // This issuer's share of a stage's weight rows (of kProducers issuers: one
  // warp issues a copy in about 41 ns, which is 25 GB/s at 1 KB).
  __device__ __forceinline__ void copy_weights(const Place& p, int off, int bytes, uint64_t* bar, int issuer,
                                               int lane) const {
    const uint8_t* base = (UP ? a.w13 : a.w2) +
                          static_cast<int64_t>(expert(p.slot)) * (UP ? 2 * a.I : a.H) * kd * kEb +
                          static_cast<int64_t>(p.st) * row_bytes;
    for (int r = issuer + lane * S::kProducers; r < 16 * S::kTiles; r += 32 * S::kProducers) {
      const int out = (p.tile * S::kTiles + r / 16) * kRows + (UP ? r % 8 : r % 16);
      if (out >= limit) continue;
      const int row = UP && r % 16 >= 8 ? a.I + out : out;
      copy_bulk(ring.base + off + r * pitch, base + static_cast<int64_t>(row) * kd * kEb, bytes, bar);
    }
  }
  // The token rows `first`, first + step, ... of a stage.
  __device__ __forceinline__ void copy_tokens(const Place& p, int off, int bytes, int tokens, uint64_t* bar,
                                              int first, int step) const {
    const uint8_t* src = UP ? (FP8 ? reinterpret_cast<const uint8_t*>(a.x16) : a.x) : a.a;
    const int begin = g.start[g.slot_expert[p.slot]] + p.c0;
    for (int i = first; i < tokens * kParts; i += step) {
      const int n = kParts == 2 && i >= tokens ? i - tokens : i;
      const int entry = g.order[begin + n];
      const int64_t row = UP ? entry / (a.K + a.S) : entry + (i >= tokens ? static_cast<int64_t>(a.T) * (a.K + a.S) : 0);
      copy_bulk(ring.base + off + 16 * S::kTiles * pitch + i * token_pitch,
                src + row * kd * 2 + static_cast<int64_t>(p.st) * row_bytes * (2 / kEb), bytes * (2 / kEb), bar);
    }
  }

  // Issues every stage of this group's jobs.  `head` counts the stages of both
  // phases; the consumers release them in order.  barrier: the grid barrier
  // behind which the tokens' side is complete (NULL: it is).
  __device__ __forceinline__ bool produce(int& head, int& tail, int& off, int& used, uint32_t* taken, int first,
                                          const uint32_t* barrier, int lane) const {
    Place p = at(first);
    int ticket = 0;
    if (lane == 0) ticket = atomicAdd(taken, 1u);
    float scale = scale_of(p, lane);
    Place held = p;            // stages from here to p wait for their tokens
    const int held_head = head;
#pragma unroll 1
    while (valid(p)) {
      const int cnt = g.cnt[g.slot_expert[p.slot]];
      const int tokens = min(cnt - p.c0, 8 * NT);
      const int bytes = min(row_bytes, kd * kEb - p.st * row_bytes);
      const int size = 16 * S::kTiles * pitch + (tokens * kParts * token_pitch + 127) / 128 * 128;
      const bool wrap = off + size > ring.size;
      const int need = size + (wrap ? ring.size - off : 0);
      // the held stages' tokens, when their job ends or the ring has nothing
      // older to release
      if (barrier && (p.q != held.q || p.c0 != held.c0)) {
        if (!release(held, held_head, head, barrier, lane)) return false;
        barrier = nullptr;
      }
      while (used + need > ring.size || head - tail == S::kStages) {
        if (barrier && tail >= held_head) {
          if (!release(held, held_head, head, barrier, lane)) return false;
          barrier = nullptr;
        }
        if (!retire(tail, used)) return false;
      }
      if (wrap) off = 0;
      const int s = head % S::kStages;
      // the place behind this one, and its scales
      Place n = p;
      if (++n.st == stages) {
        n.st = 0;
        n.c0 += 8 * NT;
        if (n.c0 >= cnt) {
          n = at(static_cast<int>(gridDim.x) * S::kGroups + __shfl_sync(kFull, ticket, 0));
          if (lane == 0 && valid(n)) ticket = atomicAdd(taken, 1u);
        }
      }
      const float next_scale = scale_of(n, lane);
      if (FP8 && lane < S::kScales) ring.scales[s * S::kScales + lane] = scale;
      __syncwarp();
      int rows = 0;  // weight rows that are copied
#pragma unroll
      for (int mt = 0; mt < S::kTiles; ++mt) {
        const int left = min(max(limit - (p.tile * S::kTiles + mt) * kRows, 0), kRows);
        rows += UP ? 2 * left : left;
      }
      if (lane == 0) {
        ring.stage[s] = Stage{off, p.slot, p.tile, p.c0, bytes, tokens, p.st * 4 + (p.st + 1 == stages ? kLast : 0) + (barrier ? kHeld : 0), need};
        mbar_arrive_expect_tx(ring.full + s, rows * bytes + tokens * kParts * bytes * (2 / kEb));
        mbar_arrive(ring.go + s);
      }
      __syncwarp();
      copy_weights(p, off, bytes, ring.full + s, 0, lane);
      if (!barrier) copy_tokens(p, off, bytes, tokens, ring.full + s, lane * S::kProducers, 32 * S::kProducers);
      off += size;
      used += need;
      ++head;
      p = n;
      scale = next_scale;
    }
    if (barrier && head != held_head && !release(held, held_head, head, barrier, lane)) return false;
    // the end of this phase: a stage without copies
    while (head - tail == S::kStages)
      if (!retire(tail, used)) return false;
    if (lane == 0) {
      ring.stage[head % S::kStages] = Stage{0, 0, 0, 0, 0, 0, -1, 0};
      mbar_arrive(ring.full + head % S::kStages);
      mbar_arrive(ring.go + head % S::kStages);
    }
    __syncwarp();
    ++head;
    return true;
  }
  // Waits until the consumers have released the oldest stage.
  __device__ __forceinline__ bool retire(int& tail, int& used) const {
    const int s = tail % S::kStages;
    if (!__all_sync(kFull, ring_wait(a, ring.empty + s, (tail / S::kStages) & 1))) return false;
    used -= ring.stage[s].taken;
    ++tail;
    return true;
  }
  // The token rows of the stages held back since `p` (all of one job).
  __device__ __forceinline__ bool release(Place p, int from, int to, const uint32_t* barrier, int lane) const {
    bool ok = true;
    if (lane == 0) ok = grid_wait(a, barrier);
    if (!__all_sync(kFull, ok)) return false;
    fence_bulk();
    for (int h = from; h < to; ++h, ++p.st) {
      const Stage& st = ring.stage[h % S::kStages];
      copy_tokens(p, st.off, st.bytes, st.tokens, ring.full + h % S::kStages, lane, 32);
    }
    return true;
  }
  // A copier: its share of every stage that the producer announces.
  __device__ __forceinline__ bool assist(int& head, int issuer, int lane) const {
    bool fenced = false;
#pragma unroll 1
    for (;; ++head) {
      const int s = head % S::kStages;
      if (!__all_sync(kFull, ring_wait(a, ring.go + s, (head / S::kStages) & 1))) return false;
      const Stage st = ring.stage[s];
      if (st.what < 0) {
        ++head;
        return true;
      }
      const Place p{0, st.slot, st.tile, st.c0, st.what >> 2};
      copy_weights(p, st.off, st.bytes, ring.full + s, issuer, lane);
      if (st.what & kHeld) continue;
      if (!fenced) fence_bulk();  // behind the producer's grid barrier
      fenced = true;
      copy_tokens(p, st.off, st.bytes, st.tokens, ring.full + s, issuer + lane * S::kProducers, 32 * S::kProducers);
    }
  }

  // ------------------------------------------------------------- consumers

  // What undoes an entry's factor (e4m3).
  __device__ __forceinline__ float inverse(int entry) const {
    return UP ? __ldcg(a.xscale + entry / (a.K + a.S)) : 1.0f / f16_factor(__ldcg(a.amax + entry));
  }

  // One result pair of entry `entry`, f its inverse(): up: gate and up of
  // output `row`; down: outputs row and row + 8.
  __device__ __forceinline__ void store(int entry, int row, float v0, float v1, float f) const {
    if (row >= limit) return;
    const int KS = a.K + a.S;
    if (FP8) {
      v0 *= f;
      v1 *= f;
    }
    if (!UP) {
      float* y = a.y + static_cast<int64_t>(entry) * a.H + row;
      y[0] = v0;
      if (row + 8 < limit) y[8] = v1;
      return;
    }
    const float h = act_value(v0, a.act) * v1;
    if (FP8) {
      a.a32[static_cast<int64_t>(entry) * a.I + row] = h;
      // a maximum does not depend on the order
      atomicMax(a.amax + entry, __float_as_uint(h) & 0x7fffffffu);
    } else {
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      const float rest = h - __bfloat162float(hi);
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.a) + static_cast<int64_t>(entry) * a.I + row;
      dst[0] = hi;
      dst[static_cast<int64_t>(a.T) * KS * a.I] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
    }
  }

  // Sums that run beside each other, so that a product need not wait for the
  // one before it; added at the end of a job (bf16) or a stage (e4m3).
  static constexpr int kChains = MT * NT == 1 ? 4 : 1;

  // The group's stages until the phase ends.  warp: of the group's consumers.
  __device__ __forceinline__ bool consume(Progress& done, int warp, int lane) const {
    const int kp = warp % S::WK, mh = warp / S::WK;
    const uint32_t lane_row = (mh * MT * 16 + (lane >> 2)) * pitch + kp * S::kSteps * 64 + (lane & 3) * 16;
    const uint32_t lane_token = 16 * S::kTiles * pitch + (lane >> 2) * token_pitch +
                                (kp * S::kSteps * 64 + (lane & 3) * 16) * (2 / kEb);
    float acc[kChains][MT][NT][4] = {};
#pragma unroll 1
    for (;;) {
      const int i = done.stages % S::kStages;
      if (!__all_sync(kFull, ring_wait(a, ring.full + i, (done.stages / S::kStages) & 1))) return false;
      ++done.stages;
      const Stage st = ring.stage[i];
      if (st.what < 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty + i);
        return true;
      }
      Vec16 w[S::kSteps][MT][2], x[S::kSteps][NT][kVec];
      float sc[MT][2] = {};
#pragma unroll
      for (int e = 0; e < S::kSteps; ++e) {
        const bool in = (kp * S::kSteps + e) * 64 + (lane & 3) * 16 < st.bytes;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const bool any = in && nt * 8 + (lane >> 2) < st.tokens;
          const uint32_t from = ring.base + st.off + lane_token + nt * 8 * token_pitch + e * 64 * (2 / kEb);
#pragma unroll
          for (int v = 0; v < kVec; ++v)
            x[e][nt][v] = lds16_if(from + (kParts == 2 ? v * st.tokens * token_pitch : v * 16), any);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w[e][mt][h] = lds16_if(ring.base + st.off + lane_row + (mt * 16 + h * 8) * pitch + e * 64, in);
      }
      if (FP8) {
        const float* from = ring.scales + i * S::kScales + kp * S::kSteps / 2;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) sc[mt][h] = from[((mh * MT + mt) * 2 + h) * kBlocks];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty + i);
      multiply(acc, w, x, sc);
      if ((st.what & kLast) && !finish(acc, st, warp, lane, done.sums)) return false;
    }
  }

  // acc += the products of one stage.
  __device__ __forceinline__ void multiply(float (&acc)[kChains][MT][NT][4], const Vec16 (&w)[S::kSteps][MT][2],
                                           const Vec16 (&x)[S::kSteps][NT][kVec],
                                           const float (&sc)[MT][2]) const {
    float sum[FP8 ? kChains : 1][FP8 ? MT : 1][NT][4] = {};
#pragma unroll
    for (int e = 0; e < S::kSteps; ++e) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const Vec16& w0 = w[e][mt][0];
        const Vec16& w1 = w[e][mt][1];
        if (!FP8) {
#pragma unroll
          for (int q = 0; q < 4; q += 2)
#pragma unroll
            for (int v = 0; v < kVec; ++v)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<false>(acc[(q / 2 * kVec + v + e * (kVec == 1 ? 2 : 0)) % kChains][mt][nt], w0.u[q],
                           w1.u[q], w0.u[q + 1], w1.u[q + 1], x[e][nt][v].u[q], x[e][nt][v].u[q + 1]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t a0, a1, a2, a3;
            f16_of_e4m3(w0.u[q], a0, a2);
            f16_of_e4m3(w1.u[q], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<true>(sum[FP8 ? q % kChains : 0][FP8 ? mt : 0][nt], a0, a1, a2, a3,
                        x[e][nt][(q / 2) % kVec].u[q % 2 * 2], x[e][nt][(q / 2) % kVec].u[q % 2 * 2 + 1]);
          }
        }
      }
    }
    if (FP8) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float t = sum[0][FP8 ? mt : 0][nt][r];
#pragma unroll
            for (int c = 1; c < (FP8 ? kChains : 1); ++c) t += sum[c][FP8 ? mt : 0][nt][r];
            acc[0][mt][nt][r] = fmaf(sc[mt][r / 2], t, acc[0][mt][nt][r]);
          }
    }
  }

  // The end of a job: the WK warps' sums are added in warp order by one of
  // them (another one each time) and stored; acc is cleared.
  __device__ __forceinline__ bool finish(float (&acc)[kChains][MT][NT][4], const Stage& st, int warp, int lane,
                                         int& sums) const {
    const int kp = warp % S::WK, mh = warp / S::WK;
    const int begin = g.start[g.slot_expert[st.slot]] + st.c0;
    if (!FP8) {
#pragma unroll
      for (int c = 1; c < kChains; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[0][0][0][r] += acc[c][0][0][r];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt, ++sums) {
      const int buf = sums % S::kRed, use = sums / S::kRed;
      float* red = ring.red + buf * (S::kRedBytes / S::kRed / 4);
      if (use > 0 && !__all_sync(kFull, ring_wait(a, ring.red_empty + buf, (use - 1) & 1))) return false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[((warp * NT + nt) * 4 + r) * 32 + lane] = acc[0][mt][nt][r];
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.red_full + buf);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if ((nt + sums) % S::WK != kp) continue;
        if (!__all_sync(kFull, ring_wait(a, ring.red_full + buf, use & 1))) return false;
        const float* from = red + (mh * S::WK * NT + nt) * 4 * 32 + lane;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = from[r * 32];
#pragma unroll
        for (int i = 1; i < S::WK; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] += from[(i * NT * 4 + r) * 32];
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.red_empty + buf);
        const int n = nt * 8 + 2 * (lane & 3);
        const int row = (st.tile * S::kTiles + mh * MT + mt) * kRows + (lane >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (n + i < st.tokens) {
            const int entry = g.order[begin + n + i];
            store(entry, row, v[i], v[2 + i], FP8 ? inverse(entry) : 1.0f);
          }
      }
    }
#pragma unroll
    for (int c = 0; c < kChains; ++c)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[c][mt][nt][r] = 0.0f;
    return true;
  }
};

// fp16 copies of x and their factors: a block per token.
template <int kThreads>
__device__ __forceinline__ void scale_tokens(const LayerArgs& a, int tokens, uint32_t* red) {
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
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, red[i]);
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

// fp16 copies of the activations, their factors from the entries' maxima.
template <int kThreads>
__device__ __forceinline__ void scale_activations(const LayerArgs& a, const Groups& g) {
  const int per = a.I / 8;
  const int64_t n = static_cast<int64_t>(g.tokens) * (a.K + a.S) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int entry = static_cast<int>(i / per);
    if (g.rank[entry] == kNone) continue;
    const float f = f16_factor(__ldcg(a.amax + entry));
    const float4* src = reinterpret_cast<const float4*>(a.a32) + 2 * i;
    const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
    const Vec16 o{f16x2(lo.x * f, lo.y * f), f16x2(lo.z * f, lo.w * f), f16x2(hi.x * f, hi.y * f),
                  f16x2(hi.z * f, hi.w * f)};
    st_vec(a.a + i * 16, o);
  }
}

// A grid barrier for a block's consumers: all their writes before it, and the
// other blocks' after it, seen by every one of them.  A block in which a wait
// gave up does not arrive, so that no block goes on.
template <int kConsumerThreads>
__device__ __forceinline__ void consumers_arrive(uint32_t* arrived, const int* failed) {
  __threadfence();
  fence_bulk();
  named_sync(1, kConsumerThreads);
  if (threadIdx.x == 0 && !*failed) {
    __threadfence();
    atomicAdd(arrived, 1u);
  }
}
template <int kConsumerThreads>
__device__ __forceinline__ bool consumers_wait(const LayerArgs& a, const uint32_t* arrived, volatile int* failed) {
  if (threadIdx.x == 0 && !*failed && !grid_wait(a, arrived)) *failed = 1;
  named_sync(1, kConsumerThreads);
  const bool done = !*failed;
  named_sync(1, kConsumerThreads);
  return done;
}

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1) layer_kernel(LayerArgs a, int ring_size) {
  constexpr int kConsumerThreads = S::kGroups * S::kConsumers * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int failed;  // a wait of this block gave up
  const int KS = a.K + a.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool producer = warp >= S::kGroups * S::kConsumers;
  const int issuer = producer ? (warp - S::kGroups * S::kConsumers) % S::kProducers : 0;
  const int group = producer ? (warp - S::kGroups * S::kConsumers) / S::kProducers : warp / S::kConsumers;
  Ring<S> ring;
  {
    uint8_t* p = smem + group * static_cast<size_t>(ring_size);
    ring.base = smem_addr(p);
    ring.size = ring_size;
    p = smem + S::kGroups * static_cast<size_t>(ring_size) + group * group_bytes<S>(0);
    ring.red = reinterpret_cast<float*>(p);
    p += S::kRedBytes;
    ring.stage = reinterpret_cast<Stage*>(p);
    p += S::kStages * sizeof(Stage);
    ring.full = reinterpret_cast<uint64_t*>(p);
    ring.empty = ring.full + S::kStages;
    ring.go = ring.empty + S::kStages;
    ring.red_full = ring.go + S::kStages;
    ring.red_empty = ring.red_full + 2;
    ring.scales = reinterpret_cast<float*>(ring.red_empty + 2);
  }
  if (producer && issuer == 0) {
    if (lane < S::kStages) {
      mbar_init(ring.go + lane, 1);
      mbar_init(ring.full + lane, 1);
      mbar_init(ring.empty + lane, S::kConsumers);
    }
    if (lane < S::kRed) {
      mbar_init(ring.red_full + lane, S::kConsumers);
      mbar_init(ring.red_empty + lane, S::kReducers);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 0) failed = 0;
  grid_dependency_wait();
  Groups g;
  group_entries<S::kThreads>(a, g, smem + S::kGroups * group_bytes<S>(ring_size));

  // grid barriers: x16 (e4m3), a, a as fp16 (e4m3), y
  uint32_t* after_up = a.arrived + 1;
  uint32_t* after_scale = S::FP8 ? a.arrived + 2 : after_up;
  uint32_t* after_down = a.arrived + 3;
  uint32_t* taken = a.arrived + kBarriers;
  if (S::FP8) {
    scale_tokens<S::kThreads>(a, g.tokens, reinterpret_cast<uint32_t*>(smem + S::kGroups * static_cast<size_t>(ring_size)));
    __threadfence();
    fence_bulk();
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(a.arrived, 1u);
    }
  }
  const Phase<S, true> up(a, g, ring);
  const Phase<S, false> down(a, g, ring);
  if (producer) {
    const int first = blockIdx.x + gridDim.x * group;
    int head = 0, tail = 0, off = 0, used = 0;
    fence_bulk();
    if (issuer > 0) {
      if ((!up.assist(head, issuer, lane) || !down.assist(head, issuer, lane)) && lane == 0) failed = 1;
      return;
    }
    if (!up.produce(head, tail, off, used, taken, first, S::FP8 ? a.arrived : nullptr, lane) ||
        !down.produce(head, tail, off, used, taken + 1, first, after_scale, lane)) {
      // what is still in flight lands before the block may end
      if (lane == 0) failed = 1;
      for (; tail < head; ++tail) ring_wait(a, ring.full + tail % S::kStages, (tail / S::kStages) & 1);
    }
    return;
  }
  Progress done;
  bool ok = up.consume(done, warp % S::kConsumers, lane);
  if (!ok && lane == 0) failed = 1;
  consumers_arrive<kConsumerThreads>(after_up, &failed);
  if (S::FP8) {
    ok = consumers_wait<kConsumerThreads>(a, after_up, &failed);
    if (ok) scale_activations<kConsumerThreads>(a, g);
    consumers_arrive<kConsumerThreads>(after_scale, &failed);
  }
  ok = ok && down.consume(done, warp % S::kConsumers, lane);
  if (!ok && lane == 0) failed = 1;
  consumers_arrive<kConsumerThreads>(after_down, &failed);
  if (!consumers_wait<kConsumerThreads>(a, after_down, &failed)) return;

  // the entries' rows summed per token, a thread per 4 columns
  const int per = a.H / 4;
  const int64_t n = static_cast<int64_t>(g.tokens) * per;
  for (int64_t i = (static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 + (threadIdx.x & 31);
       i < n; i += static_cast<int64_t>(gridDim.x) * kConsumerThreads) {
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
  static_assert(2 * S::kStageBytes <= ring_bytes<S>(MOE_LAYER_MAX_TOKENS, MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED,
                                                    kMaxExperts),
                "ring");
  auto k = layer_kernel<S>;
  const int ring = ring_bytes<S>(a.T, a.K + a.S, a.E + a.S);
  const size_t smem = S::kGroups * group_bytes<S>(ring) + groups_bytes(a.T, a.K + a.S, a.E + a.S);
  // per device and cheap: no state to keep
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(h->num_sms), dim3(S::kThreads), smem, s, true, a, ring);
}

}  // namespace

LayerPlan layer_plan(int T, int K, int S, int H, int I) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t entries = static_cast<size_t>(T) * (K + S);
  LayerPlan p;
  p.a = 0;
  p.a32 = up(2 * entries * I * sizeof(__nv_bfloat16));
  p.y = p.a32 + up(entries * I * sizeof(float));
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
  a.a32 = reinterpret_cast<float*>(ws + p.a32);
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
  // few: 8 tokens an expert and less in the mean
  const bool many = static_cast<int64_t>(T) * K > 6 * static_cast<int64_t>(a.E);
  if (q.weight_dtype == MOE_E4M3)
    return many ? launch_shape<Shape<1, 3, 8, 1, 4, 2, 1, true>>(h, a, s)
                : launch_shape<Shape<2, 1, 8, 1, 1, 1, 2, true>>(h, a, s);
  return many ? launch_shape<Shape<1, 3, 8, 1, 4, 4, 1, false>>(h, a, s)
              : launch_shape<Shape<2, 1, 8, 1, 1, 1, 2, false>>(h, a, s);
}

}  // namespace moe
