// What the kernels of the few-token MoE layer share: entries grouped by expert,
// grid-wide barriers, fp16 copies of tokens and activations, the final sum.
#ifndef MOE_LAYER_CUH_
#define MOE_LAYER_CUH_

#include <cstdint>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "tensor.cuh"

namespace moe {

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
  // the next two by entry t (K + S) + k, for many tokens in the experts' order
  uint8_t* a;            // bf16 [2][T (K + S), I], high and low part; e4m3: fp16, scaled
  float* a32;            // [T (K + S), I] (e4m3)
  uint32_t* amax;        // [T (K + S)] bits of the largest |a| of an entry (e4m3); for many
                         // tokens a float, what undoes the entry's factor
  float* y;              // [T (K + S), H]; for many tokens first x in the experts' order
  uint32_t* arrived;     // blocks that reached each grid barrier (kBarriers), then the
                         // jobs given out in each phase; zero at the start
  __nv_bfloat16* out;    // [T, H]
  int T, K, S, E, H, I;
  int act;
  unsigned long long wait_ns;
  uint32_t* flags;
};

namespace {

constexpr int kMaxEntries = MOE_LAYER_MAX_TOKENS * (MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED);
constexpr int kMaxExperts = MOE_MAX_EXPERTS + MOE_LAYER_MAX_SHARED;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint16_t kNone = 0xffff;
static_assert(kMaxEntries < kNone && kMaxExperts < kNone, "16-bit tables");
constexpr int kMaskWords = 4;  // of 32 tokens, for each expert
static_assert(MOE_LAYER_MAX_TOKENS <= 32 * kMaskWords, "token masks");
constexpr int kBarriers = 4;  // grid barriers of a call, at most
constexpr int kTickets = 16;  // of a team's coming jobs

// ---------------------------------------------------------------------------
// entries (t, k) grouped by expert

// Shared-memory tables of a block.  Entry n = t (K + S) + k, the shared expert
// j as k = K + j; experts are numbered shared first, so that their many
// tokens do not come last.
struct Groups {
  uint16_t* order;        // entries, grouped
  uint16_t* rank;         // an entry's place within its expert (ordered: in `order`), kNone:
                          // dropped
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

constexpr size_t kMaxGroupsBytes =
    groups_bytes(MOE_LAYER_MAX_TOKENS, MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED, kMaxExperts);

// Lets a kernel have the shared memory of its largest call.  The limit belongs to
// the kernel and the device, so it is set once, at the handle's creation, and to
// a constant: set by each call to its own size it could go down between another
// thread's setting and launch.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, size_t fixed) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(fixed + kMaxGroupsBytes));
}

__device__ __forceinline__ int expert_of(const LayerArgs& a, int entry) {
  const int t = entry / (a.K + a.S), k = entry - t * (a.K + a.S);
  if (k >= a.K) return k - a.K;
  const int e = __ldcg(a.idx + t * a.K + k);
  return static_cast<unsigned>(e) < static_cast<unsigned>(a.E) ? e + a.S : e == -1 ? -1 : -2;
}

// The tables, in `smem`.  With `masks` (kMaskWords of scratch an expert) the
// entries of an expert come in the order of their tokens, so that all blocks
// agree on it.
template <int kThreads, bool kOrdered>
__device__ __forceinline__ void group_entries(const LayerArgs& a, Groups& g, uint8_t* smem,
                                              uint32_t* masks) {
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

  if (a.T * KS <= 32) {  // a warp's worth: without the tables of all experts
    g.tokens = a.live ? min(max(__ldcg(a.live), 0), a.T) : a.T;
    if (warp == 0) {
      const bool mine = lane < g.tokens * KS;
      int e = mine ? expert_of(a, lane) : -1;
      if (e == -2 && blockIdx.x == 0) raise_flag(a.flags, MOE_DEVERR_BAD_EXPERT);
      // the lanes of the same expert; a token's second one is dropped
      uint32_t same = __match_any_sync(kFull, e);
      const uint32_t token = ((1u << KS) - 1u) << (lane / KS * KS);
      const bool twice = e >= a.S && (same & token & lanemask_lt()) != 0;
      if (twice && blockIdx.x == 0) raise_flag(a.flags, MOE_DEVERR_DUP_EXPERT);
      const bool ok = e >= 0 && !twice;
      const uint32_t good = __ballot_sync(kFull, ok);
      same &= good;
      const int rank = __popc(same & lanemask_lt()), cnt = __popc(same);
      const bool first = ok && rank == 0;
      const uint32_t firsts = __ballot_sync(kFull, first);
      int start = first ? cnt : 0;  // of the experts in order of their first entry
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFull, start, off);
        if (lane >= off) start += v;
      }
      start = __shfl_sync(kFull, start - cnt, ok ? __ffs(same) - 1 : 0);
      if (mine) g.rank[lane] = ok ? static_cast<uint16_t>(kOrdered ? start + rank : rank) : kNone;
      if (ok) g.order[start + rank] = static_cast<uint16_t>(lane);
      if (first) {
        g.slot_expert[__popc(firsts & lanemask_lt())] = static_cast<uint16_t>(e);
        g.cnt[e] = cnt;
        g.start[e] = start;
      }
      if (lane == 0) g.head[kMaxWarps] = __popc(firsts);
    }
    __syncthreads();
    g.nslots = g.head[kMaxWarps];
    return;
  }
  if (kOrdered) {
    for (int i = tid; i < kMaskWords * n_exp; i += kThreads) masks[i] = 0;
  } else {
    for (int e = tid; e < n_exp; e += kThreads) g.cnt[e] = 0;
  }
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
    if (kOrdered) {
      const int t = i / KS;
      if (ok) atomicOr(&masks[kMaskWords * e + t / 32], 1u << (t % 32));
      g.rank[i] = ok ? 0 : kNone;
    } else {
      g.rank[i] = ok ? static_cast<uint16_t>(atomicAdd(&g.cnt[e], 1)) : kNone;
    }
  }
  __syncthreads();
  // exclusive scan of counts (low 16 bits) and of experts with entries (high)
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    int c = 0;
    if (e < n_exp) {
      if (kOrdered) {
        for (int i = 0; i < kMaskWords; ++i) c += __popc(masks[kMaskWords * e + i]);
        g.cnt[e] = c;
      } else {
        c = g.cnt[e];
      }
    }
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
    if (i < n && g.rank[i] != kNone) {
      int at = g.start[mine[j]] + g.rank[i];
      if (kOrdered) {  // rank: 0 so far
        const uint32_t* mask = masks + kMaskWords * mine[j];
        const int t = i / KS;
        at += __popc(mask[t / 32] & ((1u << (t % 32)) - 1u));
        for (int w = 0; w < t / 32; ++w) at += __popc(mask[w]);
        g.rank[i] = static_cast<uint16_t>(at);
      }
      g.order[at] = static_cast<uint16_t>(i);
    }
  }
  g.nslots = g.head[kMaxWarps];
  __syncthreads();
}

// ---------------------------------------------------------------------------
// grid-wide barriers

// This block is done with what the others wait for.  Release and acquire at the
// counter order the blocks' other accesses (the block's own threads by its
// barriers); full fences around it took 0.35 us more a barrier.
__device__ __forceinline__ void grid_arrive(uint32_t* arrived) {
  __syncthreads();
  if (threadIdx.x == 0)
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(arrived), "r"(1u) : "memory");
}

// Waits until every block of the grid has arrived; false, with the status bit
// set, after the handle's limit.
__device__ __forceinline__ bool grid_wait(const LayerArgs& a, uint32_t* arrived, int* ok) {
  if (threadIdx.x == 0) {
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
    *ok = done;
  }
  __syncthreads();
  return *ok != 0;
}

// ---------------------------------------------------------------------------
// copies and products

// Asynchronous copies of 16 bytes into shared memory; where !valid, zeros are
// written and nothing is read.  Weights pass by L1, tokens are kept in it.
__device__ __forceinline__ void copy16_stream(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
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

// The largest magnitude of a row of n bf16 values, as the bits of a float;
// `red` holds a word a warp.  All threads of the block.
template <int kThreads>
__device__ __forceinline__ uint32_t block_max_bits(const uint8_t* row, int n, uint32_t* red) {
  uint32_t m = 0;  // of a bf16 in the high half
  for (int v = threadIdx.x; v < n / 8; v += kThreads) {
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
  return m;
}

// 8 bf16 values times f, in fp16.
__device__ __forceinline__ Vec16 scaled_f16(const Vec16& x, float f) {
  float e[8];
  VecTraits<__nv_bfloat16>::to_f32(x, e);
  Vec16 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.u[i] = f16x2(e[2 * i] * f, e[2 * i + 1] * f);
  return o;
}

// Vector i (8 values) of the fp16 activations, of an entry whose largest one
// has the bits `max_bits`.
__device__ __forceinline__ void scale_activation(const LayerArgs& a, int64_t i, uint32_t max_bits) {
  const float f = f16_factor(max_bits);
  const float4* src = reinterpret_cast<const float4*>(a.a32) + 2 * i;
  const float4 lo = __ldcg(src), hi = __ldcg(src + 1);
  st_vec(a.a + i * 16, Vec16{f16x2(lo.x * f, lo.y * f), f16x2(lo.z * f, lo.w * f),
                             f16x2(hi.x * f, hi.y * f), f16x2(hi.z * f, hi.w * f)});
}

// The entries' rows summed per token, a thread per 4 columns.
template <int kThreads>
__device__ __forceinline__ void sum_entries(const LayerArgs& a, const Groups& g) {
  const int KS = a.K + a.S;
  const int per = a.H / 4;
  const int64_t n = static_cast<int64_t>(g.tokens) * per;
  for (int64_t i = (static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 +
                   (threadIdx.x & 31);
       i < n; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / per);
    const int col = static_cast<int>(i - static_cast<int64_t>(t) * per) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* y = a.y + static_cast<int64_t>(t) * KS * a.H + col;
    // 8 entries' loads on their way at a time, also of what is not added (one
    // after the other they took 3 us of a token's 29)
    for (int k0 = 0; k0 < KS; k0 += 8) {
      float4 f[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int kk = min(k0 + j, KS - 1);
        f[j] = __ldcg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(kk) * a.H));
        w[j] = __ldg(a.w + t * a.K + min(kk, a.K - 1));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int kk = k0 + j;
        if (kk >= KS || g.rank[t * KS + kk] == kNone) continue;
        const float s = kk < a.K ? w[j] : 1.0f;
        v.x = fmaf(s, f[j].x, v.x);
        v.y = fmaf(s, f[j].y, v.y);
        v.z = fmaf(s, f[j].z, v.z);
        v.w = fmaf(s, f[j].w, v.w);
      }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t*>(&lo);
    o.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(t) * a.H + col) = o;
  }
}

}  // namespace

// The kernel on the tensor memory, for many tokens an expert.
cudaError_t prepare_layer_many_kernels();
cudaError_t launch_layer_many(const moe_handle* h, const LayerArgs& a, bool e4m3, cudaStream_t s);

}  // namespace moe

#endif  // MOE_LAYER_CUH_
