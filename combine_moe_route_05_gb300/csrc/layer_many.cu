// The few-token MoE layer where an expert has many tokens (sm_103a): the same
// three parts as the kernel of layer.cu, the products on the tensor memory.
//
// With tens of tokens an expert the layer is still bound by reading its
// weights, but mma.sync no longer keeps up: each warp has to load every token's
// operand for the few weight rows it holds.  Here 128 weight rows are the A
// operand of tcgen05.mma and an expert's tokens (16 to 128 columns) the B
// operand, both read from shared memory by the tensor core itself.
//
//   warps 0..3, 16..19  epilogue: a thread per weight row (tensor-memory lane),
//                half the columns each
//   warp  4      issues the products
//   warps 5..7   fill the queue by tensor copies: 5 weights, 6 and 7 tokens
//                (a thread takes 80 ns for each copy it asks for)
//   warps 8..15  e4m3: turn the weights that have landed into fp16 (exact)
//
// For the tensor copies the tokens lie in the order of the experts: a first
// pass copies x so, and the up products store a so.  The first weights are on
// their way while the blocks wait for that pass.
//
// Up tiles hold 64 outputs: 8 gate rows and the 8 up rows of the same outputs
// in turn, so that the epilogue pairs gate and up with one exchange between
// lanes n and n + 8.
//
// bf16: x as it is; a as the sum of two bf16 numbers, the low parts as further
// columns, added at the end.  e4m3: x and a in fp16, scaled; the weights in tensor
// memory (in shared memory, written there by the converting warps, they took
// its bandwidth: 99 against 89 us); the block scale of a row and 128 columns
// multiplies the products of these columns, which the epilogue adds up in
// registers, half the columns a set of warps (every other column block a set,
// with the sums exchanged at the end, was slower: 90 against 83 us).
//
// A stage of the queue is 128 columns of the 128 weight rows and of the tokens;
// with 64 the waits on its barriers (some 100 cycles each, even on a stage that
// has landed) took as long as the products (97 against 91 us, bf16 shape below).
//
// Jobs (an expert and a tile) are handed out by a counter; every wait is
// bounded, and a wait that gives up ends the call with the status bit set.
// Results do not depend on which block computes what.
//
// Measured, routing included (GPU time of a replayed graph; in brackets: weights
// read once at the copy rate of 6.78 TB/s).  128 tokens, 8 experts, top 2, 4096
// x 2048: bf16 90-92 us (60), e4m3 80-81 (30); 128 tokens, 64 experts, top 8, 2048 x
// 1408, bf16: 192 us (163); 37 live of 64 tokens, 256 experts, top 8, 7168 x
// 2048, e4m3: 1174-1215 us (1156).  bf16: the up products read at 6.1, the down ones
// at 5.8 TB/s (DRAM reads 407 MB, the weights' 403); the rest is routing 5,
// grouping 3, sorting and its barrier 4, the other barriers and the first
// weights' latency 7, the sum 2 us.  e4m3: half the bytes and the same fixed
// parts; a stage takes some 900 cycles, which are its copies': 28 KB, 12 of them
// tokens, at 62 GB/s an SM (75 is the most that copies from L2 reached); without
// the products, the conversion or the epilogue it takes as long, within 4%.
// (It spills 36 bytes at its 96 registers, the most that 640 threads can have.)
#include "layer.cuh"

namespace moe {
namespace {

constexpr int kThreads = 640;
constexpr int kEpilogueWarps = 8, kSecondEpilogueWarp = 16;
constexpr int kMmaWarp = 4, kWeightWarp = 5, kTokenWarp = 6, kTokenWarps = 2;
constexpr int kLoadWarps = 1 + kTokenWarps;
constexpr int kFirstConvertWarp = 8, kConvertWarps = 8;
static_assert(kFirstConvertWarp + kConvertWarps == kSecondEpilogueWarp &&
                  (kSecondEpilogueWarp + 4) * 32 == kThreads, "roles");
constexpr int kTileRows = 128;
constexpr uint32_t kTileBytes = kTileRows * 128;  // 128 bytes of each row
// Tokens of a tensor copy, and the step in which products take columns (a copy of
// 32 fills more of the queue than most experts need: 1218 against 1199 us, 37 of
// 64 tokens below).
constexpr int kBoxTokens = 16;
constexpr uint32_t kBoxBytes = kBoxTokens * 128;
constexpr int kJobRing = 32;     // jobs on their way from the loading thread to the others
constexpr int kMaxRing = 10;     // stages of the queue
constexpr int kMaxAcc = 4;       // accumulators
constexpr size_t kQueueBytes = 208 * 1024 - 1024;
constexpr uint32_t kA16Columns = 64;  // of tensor memory: 128 fp16 columns of the weights
constexpr size_t kBarrierBytes = 1024;
constexpr size_t kFixedBytes = 1024 /* alignment */ + kQueueBytes + kBarrierBytes;
static_assert(kMaskWords * kMaxExperts * 4 <= kQueueBytes, "masks in the queue's place");
static_assert(kFixedBytes + kMaxGroupsBytes + 256 <= 227 * 1024, "shared memory budget");

struct Barriers {
  uint64_t landed[kMaxRing];  // a stage is there (an arrival per loading thread)
  uint64_t empty[kMaxRing];   // its products are done
  // e4m3: an accumulator's fp16 weights are there (an arrival per converting
  // warp), and it is free, which the converting warps have waited for
  uint64_t a16_full[kMaxAcc];
  uint64_t acc_full[kMaxAcc];   // an accumulator is complete
  uint64_t acc_empty[kMaxAcc];  // and read (an arrival per epilogue warp)
  uint64_t drained;           // after a wait that gave up: no product is under way
  int32_t issued[kLoadWarps]; // and the stages that each loading thread began
  unsigned long long jobs[kJobRing];  // number, counted from 1 << 32, plus q + 1 (0: the end)
  uint32_t tmem;
  int32_t max_tokens;         // of one expert
  int32_t rows;               // entries in all
};
static_assert(sizeof(Barriers) <= kBarrierBytes, "barriers");

// The call's tensor maps.
struct Maps {
  CUtensorMap w13, w2, x, a;
};

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// The same with A in tensor memory: lane = row, a 32-bit column two elements.
__device__ __forceinline__ void mma_f16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}

// One arrival on `bar` once every product this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int u, int v, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(smem_addr(bar))
      : "memory");
}

// What this thread wrote to or knows of in global memory, for tensor copies.
__device__ __forceinline__ void fence_copies() { asm volatile("fence.proxy.async;" ::: "memory"); }

// A place in a ring of n slots and the parity of its use.
struct Place {
  int slot;
  uint32_t parity;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Where each role stands in the rings: all run on from the up to the down
// products.
struct State {
  Place stage{0, 0};  // the next one to be filled or read
  int issued = 0;     // loading: stages asked for
  Place acc{0, 0};
  int job = 0;
};

template <bool FP8, bool UP>
struct ManyPhase {
  static constexpr int kTileOutputs = UP ? 64 : 128;
  static constexpr int kMaxN = FP8 ? 64 : 128;  // tokens of one pass over the weights
  static constexpr int kAcc = FP8 ? 4 : 2;      // accumulators
  static constexpr int kAccColumns = FP8 ? kMaxN : 2 * kMaxN;
  static constexpr bool kLow = !UP && !FP8;     // a's low parts follow as further columns
  // A stage: 128 columns of the weight rows, bf16 in two tiles, and of the
  // tokens' rows, in two slices (of which each has its low parts behind it).
  static constexpr uint32_t kWeightBytes = (FP8 ? 1 : 2) * kTileBytes;

  const LayerArgs& a;
  const Groups& g;
  Barriers& b;
  const CUtensorMap* weights;
  const CUtensorMap* tokens;
  uint32_t queue;
  int ring;               // stages
  uint32_t stage_bytes;
  int kd, limit, tiles, stages, nq;
  uint32_t* given;

  __device__ __forceinline__ ManyPhase(const LayerArgs& args, const Groups& groups, Barriers& bars,
                                       const Maps& maps, uint32_t smem)
      : a(args), g(groups), b(bars), weights(UP ? &maps.w13 : &maps.w2),
        tokens(UP ? &maps.x : &maps.a), queue(smem) {
    kd = UP ? a.H : a.I;
    limit = UP ? a.I : a.H;
    tiles = (limit + kTileOutputs - 1) / kTileOutputs;
    stages = (kd + 127) / 128;
    nq = g.nslots * tiles;
    given = a.arrived + kBarriers + (UP ? 0 : 1);
    // the same stages in both phases
    const int n = columns(min(b.max_tokens, kMaxN));
    stage_bytes = kWeightBytes + n * (FP8 ? 256 : 512);
    ring = min(static_cast<int>(kQueueBytes / stage_bytes), kMaxRing);
  }

  // Columns of the products, and rows that the tensor copies fill.
  static __device__ __forceinline__ int columns(int tokens) {
    return (tokens + kBoxTokens - 1) / kBoxTokens * kBoxTokens;
  }
  // Job number i, once the weights' thread has taken it: q, -1 at the end, -2
  // after the handle's limit.
  __device__ __forceinline__ int job(int i) const {
    const volatile unsigned long long* from = &b.jobs[i % kJobRing];
    unsigned long long v = *from;
    if (static_cast<int>(v >> 32) != i + 1) {
      const unsigned long long t0 = global_ns();
      while (static_cast<int>((v = *from) >> 32) != i + 1)
        if (global_ns() - t0 > a.wait_ns) return -2;
    }
    return static_cast<int>(v & 0xffffffffu) - 1;
  }
  __device__ __forceinline__ uint32_t stage(int slot) const { return queue + slot * stage_bytes; }
  __device__ __forceinline__ int expert(int slot) const {
    const int p = g.slot_expert[slot];
    return p < a.S ? a.E + p : p - a.S;
  }
  // The row of the expert's weights in row r of the tile, behind the last
  // output the last one's again.
  __device__ __forceinline__ int weight_row(int tile, int r) const {
    if (!UP) return min(tile * 128 + r, limit - 1);
    return min(tile * 64 + (r >> 4) * 8 + (r & 7), limit - 1) + (r & 8 ? a.I : 0);
  }

  // Every lane waits, and all leave together.
  __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(kFull, wait_phase(bar, parity, a.wait_ns));
  }

  // -- the loading threads

  // Asks for column block kb of the 128 weight rows of job q.  Behind the last
  // output and the last column zeros arrive.
  __device__ __forceinline__ void send_weights(State& s, int q, int kb) const {
    const int slot = q / tiles, tile = q - slot * tiles;
    uint64_t* bar = &b.landed[s.stage.slot];
    uint32_t to = stage(s.stage.slot);
    mbar_arrive_expect_tx(bar, kWeightBytes);
#pragma unroll
    for (int i = 0; i < (FP8 ? 1 : 2); ++i, to += kTileBytes) {
      if (UP) tma_load_5d(to, weights, kb * 128 + i * 64, 0, 0, tile * 8, expert(slot), bar);
      else tma_load_3d(to, weights, kb * 128 + i * 64, tile * 128, expert(slot), bar);
    }
    s.stage.step(ring);
    ++s.issued;
  }
  // Before the tokens are there: the weights of the first stages.
  __device__ __forceinline__ int send_ahead(State& s) const {
    const int q = blockIdx.x;
    if (q >= nq) return 0;
    const int n = min(ring, stages);
    for (int kb = 0; kb < n; ++kb) send_weights(s, q, kb);
    return n;
  }
  __device__ __forceinline__ bool load_weights(State& s, int ahead) const {
    int q = static_cast<int>(blockIdx.x) < nq ? static_cast<int>(blockIdx.x) : -1;
    for (;; ++s.job) {
      *const_cast<volatile unsigned long long*>(&b.jobs[s.job % kJobRing]) =
          (static_cast<unsigned long long>(s.job + 1) << 32) + static_cast<uint32_t>(q + 1);
      if (q < 0) break;
      const int ticket = static_cast<int>(atomicAdd(given, 1u));
      const int n = (g.cnt[g.slot_expert[q / tiles]] + kMaxN - 1) / kMaxN;
      for (int pass = 0; pass < n; ++pass, ahead = 0)
        for (int kb = ahead; kb < stages; ++kb) {
          if (!wait_phase(&b.empty[s.stage.slot], s.stage.parity ^ 1u, a.wait_ns)) return false;
          send_weights(s, q, kb);
        }
      q = ticket + static_cast<int>(gridDim.x);
      if (q >= nq) q = -1;
    }
    ++s.job;
    return true;
  }

  // Thread `i` of the tokens' threads: slice i.
  __device__ __forceinline__ bool load_tokens(State& s, int i) const {
    for (;; ++s.job) {
      const int q = job(s.job);
      if (q < 0) {
        ++s.job;
        return q == -1;
      }
      const int p = g.slot_expert[q / tiles];
      for (int c0 = 0; c0 < g.cnt[p]; c0 += kMaxN) {
        const int n = columns(min(g.cnt[p] - c0, kMaxN)), row = g.start[p] + c0;
        const uint32_t bytes = n * (kLow ? 256 : 128);
        for (int kb = 0; kb < stages; ++kb) {
          if (!wait_phase(&b.empty[s.stage.slot], s.stage.parity ^ 1u, a.wait_ns)) return false;
          uint64_t* bar = &b.landed[s.stage.slot];
          uint32_t to = stage(s.stage.slot) + kWeightBytes + i * bytes;
          mbar_arrive_expect_tx(bar, bytes);
          for (int low = 0; low < (kLow ? 2 : 1); ++low)
            for (int r = 0; r < n; r += kBoxTokens, to += kBoxBytes)
              tma_load_3d(to, tokens, kb * 128 + i * 64, row + r, low, bar);
          s.stage.step(ring);
          ++s.issued;
        }
      }
    }
  }

  // After a wait that gave up, by all threads: waits until what was asked for has
  // landed, a few microseconds (for certain after the default limit, whatever the
  // handle's).  The loading threads stand at different stages: those behind
  // arrive, without bytes, for the stages that another has begun, which would
  // not complete otherwise.  Whoever began a stage had seen the last use of its
  // place end, so these arrivals count for the stage and not for that use.
  __device__ __forceinline__ void drain(const State& s) const {
    const int i = static_cast<int>(threadIdx.x >> 5) - kWeightWarp;
    const bool loads = threadIdx.x % 32 == 0 && i >= 0 && i < kLoadWarps;
    if (loads) b.issued[i] = s.issued;
    __syncthreads();
    if (!loads) return;
    int last = 0;
#pragma unroll
    for (int j = 0; j < kLoadWarps; ++j) last = max(last, b.issued[j]);
    for (int n = s.issued; n < last; ++n) mbar_arrive(&b.landed[n % ring]);
    for (int n = max(last - ring, 0); n < last; ++n)
      if (!wait_phase(&b.landed[n % ring], (n / ring) & 1u, MOE_DEFAULT_WAIT_LIMIT_NS)) return;
  }

  // -- converting warps (e4m3)

  // Two warps a quarter of the rows, half the columns each; a thread has the
  // row of its tensor-memory lane.
  __device__ __forceinline__ bool convert(State& s, uint32_t tmem, int warp, int lane) const {
    const int row = warp % 4 * 32 + lane, half = warp / 4 % 2;
    const uint32_t mine = tmem + kAcc * kAccColumns + half * (kA16Columns / 2) +
                          (static_cast<uint32_t>(warp % 4 * 32) << 16);
    for (;; ++s.job) {
      const int q = __shfl_sync(kFull, job(s.job), 0);
      if (q < 0) {
        ++s.job;
        return q == -1;
      }
      const int p = g.slot_expert[q / tiles];
      for (int n = (g.cnt[p] + kMaxN - 1) / kMaxN * stages; n > 0; --n) {
        // the accumulator has been read, so the products of its last weights
        // are done, too
        if (!warp_wait(&b.landed[s.stage.slot], s.stage.parity) ||
            !warp_wait(&b.acc_empty[s.acc.slot], s.acc.parity ^ 1u))
          return false;
        tc_fence_after();
        const uint32_t from = stage(s.stage.slot) + row * 128;
        uint32_t h[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Vec16 v = lds16(from + (((half * 4 + i) ^ (row & 7)) << 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) f16_of_e4m3(v.u[j], h[i * 8 + j * 2], h[i * 8 + j * 2 + 1]);
        }
        tmem_st32(mine + s.acc.slot * kA16Columns, h);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.a16_full[s.acc.slot]);
        s.acc.step(kAcc);
        s.stage.step(ring);
      }
    }
  }

  // -- the issuing warp

  __device__ __forceinline__ bool products(State& s, uint32_t tmem) const {
    constexpr uint32_t kFormat = (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) |
                                 (static_cast<uint32_t>(kTileRows >> 4) << 24);
    // the whole warp goes along and one lane issues: the operands then stay in
    // uniform registers
    for (;; ++s.job) {
      const int q = __shfl_sync(kFull, job(s.job), 0);
      if (q < 0) {
        ++s.job;
        return q == -1;
      }
      const int p = g.slot_expert[q / tiles];
      const int all = __shfl_sync(kFull, g.cnt[p], 0);
      for (int c0 = 0; c0 < all; c0 += kMaxN) {
        const int cnt = min(all - c0, kMaxN);
        const int n = kLow ? 2 * columns(cnt) : columns(cnt);
        const uint32_t idesc = kFormat | (static_cast<uint32_t>(n >> 3) << 17);
        const uint32_t x_next = columns(cnt) * (kLow ? 16 : 8);
        for (int kb = 0; kb < stages; ++kb) {
          // e4m3: the converting warps have seen the stage land and the
          // accumulator free
          bool ok = FP8 ? wait_phase(&b.a16_full[s.acc.slot], s.acc.parity, a.wait_ns)
                        : wait_phase(&b.landed[s.stage.slot], s.stage.parity, a.wait_ns);
          if (!FP8 && kb == 0)
            ok = ok && wait_phase(&b.acc_empty[s.acc.slot], s.acc.parity ^ 1u, a.wait_ns);
          if (!__all_sync(kFull, ok)) return false;
          tc_fence_after();
          const uint32_t d = tmem + s.acc.slot * kAccColumns;
          const uint32_t at = stage(s.stage.slot);
          const uint64_t x = sw128_desc(at + kWeightBytes);
          const uint64_t w = sw128_desc(at);
          const uint32_t w16 = tmem + kAcc * kAccColumns + s.acc.slot * kA16Columns;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint64_t tokens = x + i * x_next + k * 2;
                if (FP8) mma_f16_tmem(d, w16 + (i * 4 + k) * 8, tokens, idesc, i + k > 0);
                else mma_f16(d, w + i * (kTileBytes / 16) + k * 2, tokens, idesc,
                             kb > 0 || i + k > 0);
              }
            mma_commit(&b.empty[s.stage.slot]);
            if (FP8 || kb == stages - 1) mma_commit(&b.acc_full[s.acc.slot]);
          }
          __syncwarp();
          s.stage.step(ring);
          if (FP8 || kb == stages - 1) s.acc.step(kAcc);
        }
      }
    }
  }

  // -- epilogue warps

  __device__ __forceinline__ bool acc_ready(const State& s) const {
    const bool got = warp_wait(&b.acc_full[s.acc.slot], s.acc.parity);
    tc_fence_after();
    return got;
  }
  __device__ __forceinline__ void acc_read(State& s, int lane) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b.acc_empty[s.acc.slot]);
    s.acc.step(kAcc);
  }

  // 16 columns (tokens n0 ..) of the warp's rows of the tile; lane n % 32 has
  // the inverse factor of token n (e4m3).
  __device__ __forceinline__ void store16(const float (&v)[16], int n0, int cnt, int begin, int tile,
                                          int quarter, int lane, float factors) const {
    if (UP) {
      const int o = tile * 64 + quarter * 16 + (lane >> 4) * 8 + (lane & 7);
      const bool upper = lane & 8;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        // lane l takes column j, lane l + 8 column j + 1
        const float other = __shfl_xor_sync(kFull, upper ? v[j] : v[j + 1], 8);
        float gate = upper ? other : v[j], up = upper ? v[j + 1] : other;
        const int n = n0 + j + (upper ? 1 : 0);
        if (FP8) {
          const float f = __shfl_sync(kFull, factors, n & 31);
          gate *= f;
          up *= f;
        }
        const float h = act_value(gate, a.act) * up;
        if (n >= cnt || o >= limit) continue;
        const int64_t at = static_cast<int64_t>(begin + n) * a.I + o;
        if (FP8) {
          a.a32[at] = h;
        } else {
          const __nv_bfloat16 hi = __float2bfloat16_rn(h);
          const float rest = h - __bfloat162float(hi);
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.a) + at;
          dst[0] = hi;
          dst[static_cast<int64_t>(a.T) * (a.K + a.S) * a.I] =
              __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
        }
      }
      return;
    }
    const int row = tile * 128 + quarter * 32 + lane;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float f = FP8 ? __shfl_sync(kFull, factors, (n0 + j) & 31) : 1.0f;
      if (n0 + j < cnt && row < limit)
        a.y[static_cast<int64_t>(g.order[begin + n0 + j]) * a.H + row] = FP8 ? v[j] * f : v[j];
    }
  }

  // Warp `quarter` of set `set`: the first or second half of the columns, in
  // steps of 16.
  __device__ __forceinline__ bool epilogue(State& s, uint32_t tmem, int set, int quarter,
                                           int lane) const {
    const uint32_t mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    for (;; ++s.job) {
      const int q = __shfl_sync(kFull, job(s.job), 0);
      if (q < 0) {
        ++s.job;
        return q == -1;
      }
      const int slot = q / tiles, tile = q - slot * tiles, p = g.slot_expert[slot];
      for (int c0 = 0; c0 < g.cnt[p]; c0 += kMaxN) {
        const int cnt = min(g.cnt[p] - c0, kMaxN), begin = g.start[p] + c0;
        const int half = (columns(cnt) / 16 + 1) / 2 * 16;
        const int first = set * half, last = min(first + half, cnt);
        if (FP8) {
          static_assert(!FP8 || kMaxN <= 64, "32 columns a set");
          const int r = weight_row(tile, quarter * 32 + lane);
          const int64_t row =
              static_cast<int64_t>(expert(slot)) * (((UP ? 2 * a.I : a.H) + 127) / 128) + r / 128;
          const float* scale = (UP ? a.s13 : a.s2) + row * stages;
          // what undoes the factor of column first + lane
          const int entry = g.order[begin + min(first + lane, cnt - 1)];
          const float factor = __ldcg((UP ? a.xscale + entry / (a.K + a.S)
                                          : reinterpret_cast<const float*>(a.amax) + entry));
          float sum[2][16] = {};
          float next = __ldg(scale);
          for (int kb = 0; kb < stages; ++kb) {
            const float f = next;
            if (kb + 1 < stages) next = __ldg(scale + kb + 1);
            if (!acc_ready(s)) return false;
            if (first < cnt && half == 16) {
              uint32_t v[16];
              tmem_ld16(mine + s.acc.slot * kAccColumns + first, v);
              acc_read(s, lane);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[0][j] = fmaf(f, __uint_as_float(v[j]), sum[0][j]);
            } else if (first < cnt) {
              uint32_t v[32];
              tmem_ld32(mine + s.acc.slot * kAccColumns + first, v);
              acc_read(s, lane);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                sum[j / 16][j % 16] = fmaf(f, __uint_as_float(v[j]), sum[j / 16][j % 16]);
            } else {
              acc_read(s, lane);
            }
          }
          // (a lane of the factors is a column modulo 32 from `first` on)
          const float turned = __shfl_sync(kFull, factor, (lane - first) & 31);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (first + c * 16 < last)
              store16(sum[c], first + c * 16, cnt, begin, tile, quarter, lane, turned);
        } else {
          if (!acc_ready(s)) return false;
#pragma unroll 1
          for (int n0 = first; n0 < last; n0 += 16) {
            uint32_t v[16], low[16];
            tmem_ld16(mine + s.acc.slot * kAccColumns + n0, v);
            if (kLow) tmem_ld16(mine + s.acc.slot * kAccColumns + columns(cnt) + n0, low);
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              f[j] = kLow ? __uint_as_float(v[j]) + __uint_as_float(low[j]) : __uint_as_float(v[j]);
            store16(f, n0, cnt, begin, tile, quarter, lane, 1.0f);
          }
          acc_read(s, lane);
        }
      }
    }
  }

  __device__ __forceinline__ bool run(State& s, int ahead, uint32_t tmem) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool ok = true;
    if (warp < 4 || warp >= kSecondEpilogueWarp) ok = epilogue(s, tmem, warp / 16, warp % 4, lane);
    else if (warp == kMmaWarp) ok = products(s, tmem);
    else if (warp == kWeightWarp) ok = lane != 0 || load_weights(s, ahead);
    else if (warp < kTokenWarp + kTokenWarps) ok = lane != 0 || load_tokens(s, warp - kTokenWarp);
    else if (FP8) ok = convert(s, tmem, warp, lane);
    if (!ok) raise_flag(a.flags, MOE_DEVERR_TIMEOUT);
    __syncwarp();
    return __syncthreads_and(ok) != 0;
  }
};

// The tokens in the order of the experts, a block per token: bf16 as they are;
// e4m3: fp16 times the token's factor.
template <bool FP8>
__device__ __forceinline__ void sort_tokens(const LayerArgs& a, const Groups& g, uint32_t* red) {
  const int KS = a.K + a.S;
  for (int t = blockIdx.x; t < g.tokens; t += gridDim.x) {
    const uint8_t* row = a.x + static_cast<int64_t>(t) * a.H * 2;
    const bool has = static_cast<int>(threadIdx.x) < a.H / 8;
    const Vec16 first = has ? ld_vec(row + threadIdx.x * 16) : Vec16{};
    float f = 1.0f;
    if (FP8) {
      f = f16_factor(block_max_bits<kThreads>(row, a.H, red));
      if (threadIdx.x == 0) a.xscale[t] = 1.0f / f;
    }
    for (int v = threadIdx.x; v < a.H / 8; v += kThreads) {
      Vec16 o = v < kThreads ? first : ld_vec(row + v * 16);
      if (FP8) o = scaled_f16(o, f);
      for (int k = 0; k < KS; ++k) {
        const int at = g.rank[t * KS + k];
        if (at != kNone)
          st_vec(reinterpret_cast<uint8_t*>(a.y) + static_cast<int64_t>(at) * a.H * 2 + v * 16,
                 o);
      }
    }
  }
}

// fp16 copies of the activations, a warp per row: its factor from its largest
// value, and what undoes it in place of the maximum.
__device__ __forceinline__ void scale_sorted(const LayerArgs& a, const Groups& g, int rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp * gridDim.x + blockIdx.x; r < rows; r += gridDim.x * (kThreads / 32)) {
    const int64_t at = static_cast<int64_t>(r) * (a.I / 8);
    const uint4* src = reinterpret_cast<const uint4*>(a.a32 + static_cast<int64_t>(r) * a.I);
    uint32_t m = 0;
#pragma unroll 4
    for (int v = lane; v < a.I / 4; v += 32) {
      const uint4 x = __ldcg(src + v);
      m = max(max(m, max(x.x & 0x7fffffffu, x.y & 0x7fffffffu)),
              max(x.z & 0x7fffffffu, x.w & 0x7fffffffu));
    }
    m = __reduce_max_sync(kFull, m);
#pragma unroll 2
    for (int v = lane; v < a.I / 8; v += 32) scale_activation(a, at + v, m);
    if (lane == 0) reinterpret_cast<float*>(a.amax)[g.order[r]] = 1.0f / f16_factor(m);
  }
}

template <bool FP8>
__device__ __forceinline__ bool layer_body(const LayerArgs& a, const Groups& g, Barriers& b,
                                           const Maps& maps, uint32_t queue, uint32_t tmem, int* ok,
                                           uint32_t* red) {
  const bool loads = threadIdx.x == kWeightWarp * 32;
  uint32_t* arrived = a.arrived;  // of the next barrier
  State s;
  const ManyPhase<FP8, true> up(a, g, b, maps, queue);
  const ManyPhase<FP8, false> down(a, g, b, maps, queue);
  int ahead = 0;
  // the weights behind the tokens, whose way to memory they would fill (91 us
  // so, 93 with the weights first: 128 tokens, 8 experts, 4096 x 2048)
  sort_tokens<FP8>(a, g, red);
  fence_copies();
  grid_arrive(arrived);
  if (loads) ahead = up.send_ahead(s);
  bool done = grid_wait(a, arrived++, ok);
  fence_copies();
  done = done && up.run(s, ahead, tmem);
  if (done) {
    fence_copies();
    grid_arrive(arrived);
    if (loads) ahead = down.send_ahead(s);
    done = grid_wait(a, arrived++, ok);
    fence_copies();
  }
  if (FP8 && done) {
    scale_sorted(a, g, b.rows);
    fence_copies();
    grid_arrive(arrived);
    done = grid_wait(a, arrived++, ok);
    fence_copies();
  }
  done = done && down.run(s, ahead, tmem);
  if (done) {
    grid_arrive(arrived);
    if (grid_wait(a, arrived, ok)) sum_entries<kThreads>(a, g);
    return true;
  }
  down.drain(s);
  return false;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) layer_many_kernel(
    const __grid_constant__ Maps maps, LayerArgs a) {
  constexpr uint32_t kColumns = 512;
  static_assert(ManyPhase<FP8, true>::kAcc * ManyPhase<FP8, true>::kAccColumns +
                    (FP8 ? ManyPhase<FP8, true>::kAcc * kA16Columns : 0) <= kColumns,
                "tensor memory budget");
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ int ok;
  __shared__ uint32_t red[kThreads / 32];
  grid_dependency_wait();
  // operands begin on the 1024 bytes after which the swizzle repeats
  uint8_t* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  Barriers& b = *reinterpret_cast<Barriers*>(smem + kQueueBytes);
  const int warp = threadIdx.x >> 5;
  Groups g;
  group_entries<kThreads, true>(a, g, smem + kQueueBytes + kBarrierBytes,
                                reinterpret_cast<uint32_t*>(smem));
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&b.landed[i], kLoadWarps);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < kMaxAcc; ++i) {
      mbar_init(&b.a16_full[i], kConvertWarps);
      mbar_init(&b.acc_full[i], 1);
      mbar_init(&b.acc_empty[i], kEpilogueWarps);
    }
    for (int i = 0; i < kJobRing; ++i) b.jobs[i] = 0;
    mbar_init(&b.drained, 1);
    fence_mbar_init();
    b.max_tokens = 0;
    b.rows = 0;
  }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&b.tmem)),
                 "r"(kColumns)
                 : "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int i = threadIdx.x; i < g.nslots; i += kThreads) {
    const int p = g.slot_expert[i];
    atomicMax(&b.max_tokens, g.cnt[p]);
    atomicMax(&b.rows, g.start[p] + g.cnt[p]);
  }
  // the queue was scratch memory of the grouping
  fence_copies();
  __syncthreads();
  const uint32_t tmem = b.tmem;
  if (!layer_body<FP8>(a, g, b, maps, smem_addr(smem), tmem, &ok, red)) {
    if (warp == kMmaWarp && elect_one()) {  // the lane that issued them
      mma_commit(&b.drained);
      wait_phase(&b.drained, 0, MOE_DEFAULT_WAIT_LIMIT_NS);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns)
                 : "memory");
}

// A tensor of 16-bit or 8-bit elements, innermost dimension first; boxes of 128
// bytes by box[1], box[2], ..., swizzled as the products read them.
bool encode(CUtensorMap* m, const void* base, bool bytes, int rank,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiled fn = encode_fn();
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_maps(Maps* m, const LayerArgs& a, bool e4m3) {
  const cuuint64_t n = a.E + a.S, H = a.H, I = a.I, rows = static_cast<cuuint64_t>(a.T) * (a.K + a.S);
  const cuuint64_t eb = e4m3 ? 1 : 2;
  const cuuint32_t k = static_cast<cuuint32_t>(128 / eb);
  // [expert][8 outputs][gate, up][output][column]: 8 gate rows and their 8 up
  // rows in turn
  const cuuint64_t d13[5] = {H, 8, 2, I / 8, n};
  const cuuint64_t s13[4] = {H * eb, I * H * eb, 8 * H * eb, 2 * I * H * eb};
  const cuuint32_t b13[5] = {k, 8, 2, 8, 1};
  const cuuint64_t d2[3] = {I, H, n};
  const cuuint64_t s2[2] = {I * eb, H * I * eb};
  const cuuint32_t b2[3] = {k, kTileRows, 1};
  // tokens: 16-bit either way
  const cuuint64_t dx[3] = {H, rows, 1};
  const cuuint64_t sx[2] = {H * 2, rows * H * 2};
  const cuuint64_t da[3] = {I, rows, e4m3 ? 1ull : 2ull};
  const cuuint64_t sa[2] = {I * 2, rows * I * 2};
  const cuuint32_t bt[3] = {64, kBoxTokens, 1};
  return encode(&m->w13, a.w13, e4m3, 5, d13, s13, b13) &&
         encode(&m->w2, a.w2, e4m3, 3, d2, s2, b2) &&
         encode(&m->x, a.y, false, 3, dx, sx, bt) &&
         encode(&m->a, a.a, false, 3, da, sa, bt);
}

template <bool FP8>
cudaError_t launch_one(const moe_handle* h, const LayerArgs& a, cudaStream_t s) {
  Maps maps;
  if (!encode_maps(&maps, a, FP8)) return cudaErrorInvalidValue;
  const size_t smem = kFixedBytes + groups_bytes(a.T, a.K + a.S, a.E + a.S);
  return launch_chained(layer_many_kernel<FP8>, dim3(h->num_sms), dim3(kThreads), smem, s, true, maps, a);
}

}  // namespace

cudaError_t prepare_layer_many_kernels() {
  const cudaError_t e = allow_shared(layer_many_kernel<false>, kFixedBytes);
  return e == cudaSuccess ? allow_shared(layer_many_kernel<true>, kFixedBytes) : e;
}

cudaError_t launch_layer_many(const moe_handle* h, const LayerArgs& a, bool e4m3, cudaStream_t s) {
  return e4m3 ? launch_one<true>(h, a, s) : launch_one<false>(h, a, s);
}

}  // namespace moe
