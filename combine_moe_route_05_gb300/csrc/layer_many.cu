// The few-token MoE layer where an expert has many tokens (sm_103a): the same
// three parts as the kernel of layer.cu, the products on the tensor memory.
//
// With tens of tokens an expert the layer is still bound by reading its
// weights, but mma.sync no longer keeps up: each warp has to load every token's
// operand for the few weight rows it holds.  Here 128 weight rows are the A
// operand of tcgen05.mma and an expert's tokens (16 to 128 columns) the B
// operand, both read from shared memory by the tensor core itself, so that a
// stage of the queue costs its copies and nothing else.
//
//   warps 0..3   epilogue: a thread per weight row (tensor-memory lane)
//   warp  4      issues the products
//   warps 8..15  fill the queue: weights by tensor copies (four threads, 32
//                rows each), tokens row by row, since they are gathered
//
// Up tiles hold 64 outputs: in each warp's quarter of the 128 rows 16 gate rows
// and the 16 up rows of the same outputs, so that the epilogue pairs gate and
// up with one exchange between lanes n and n + 16.
//
// bf16: x as it is; a as the sum of two bf16 numbers, the low parts as further
// products into the same accumulator.  e4m3: a copying thread turns the 16
// weights it copied into fp16 (exact) on their way from the queue to the A
// operand; the block scale of a row and 128 columns multiplies the products of
// these columns, which the epilogue adds up in registers.
//
// Jobs (an expert and a tile) are handed out by a counter; every wait is
// bounded, and a wait that gives up ends the call with the status bit set.
// Results do not depend on which block computes what.
#include "layer.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kEpilogueWarps = 4, kMmaWarp = 4, kFirstCopyWarp = 8, kCopyWarps = 8;
constexpr int kCopyThreads = 32 * kCopyWarps;
static_assert((kFirstCopyWarp + kCopyWarps) * 32 == kThreads, "roles");
constexpr int kTileRows = 128;
constexpr int kParts = 4;        // tensor copies of a stage's weights
constexpr uint32_t kWeightBytes = kTileRows * 128;  // of a stage: 128 bytes of each row
constexpr int kJobRing = 32;     // jobs on their way from the copying warps to the others
constexpr int kMaxRing = 10;     // stages of the queue
constexpr size_t kQueueBytes = 208 * 1024;
constexpr uint32_t kA16Bytes = 2 * kTileRows * 128;  // 128 columns in fp16
constexpr size_t kBarrierBytes = 512;
constexpr size_t kFixedBytes = 1024 /* alignment */ + kQueueBytes + kBarrierBytes;
static_assert(kFixedBytes + groups_bytes(MOE_LAYER_MAX_TOKENS, MOE_MAX_TOPK + MOE_LAYER_MAX_SHARED,
                                         kMaxExperts) + 64 <= 227 * 1024, "shared memory budget");

struct Barriers {
  uint64_t landed[kMaxRing];  // a stage's weights are there
  uint64_t full[kMaxRing];   // its tokens, too (an arrival per copying warp); e4m3: and
                             // its fp16 weights
  uint64_t empty[kMaxRing];  // its products are done
  uint64_t a16_empty[2];     // e4m3: the products of an fp16 slice are done
  uint64_t acc_full[2];      // an accumulator is complete (the commit, and the issuing thread)
  uint64_t acc_empty[2];     // and read (an arrival per epilogue warp)
  uint64_t drained;          // after a wait that gave up: no product is under way
  int32_t jobs[kJobRing];
  uint32_t tmem;
  int32_t max_tokens;        // of one expert
};
static_assert(sizeof(Barriers) <= kBarrierBytes, "barriers");

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// One arrival on `bar` once every product this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}

// What this thread wrote to shared memory, for the tensor core's reads.
__device__ __forceinline__ void fence_operands() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void sts16(uint32_t p, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
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

// All but the last `pending` groups of copies have landed.
__device__ __forceinline__ void copies_wait_for(int pending) {
  switch (pending) {
    case 1: copies_wait<1>(); break;
    case 2: copies_wait<2>(); break;
    case 3: copies_wait<3>(); break;
    case 4: copies_wait<4>(); break;
    case 5: copies_wait<5>(); break;
    case 6: copies_wait<6>(); break;
    case 7: copies_wait<7>(); break;
    case 8: copies_wait<8>(); break;
    default: copies_wait<0>(); break;
  }
}

// The copying warps' barrier, with the AND of `p` over them.
__device__ __forceinline__ bool copy_warps_and(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.and.pred po, 1, %2, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "n"(kCopyThreads)
      : "memory");
  return r != 0;
}

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

// Where each role stands in the queue and the accumulators: both run on from
// the up to the down products.
struct State {
  Place sent{0, 0};   // copying: the next stage whose weights are asked for
  int issued = 0;     // stages asked for
  Place fill{0, 0};   // copying: the next stage
  int landing = 0;    // copying: stages that are copied, not yet announced
  Place ready{0, 0};  // copying: the next to be announced; products: the next to be read
  Place a16{0, 0};
  Place acc{0, 0};
  int job = 0;
};

template <bool FP8, bool UP>
struct ManyPhase {
  static constexpr int kEb = FP8 ? 1 : 2;
  static constexpr int kTileOutputs = UP ? 64 : 128;
  static constexpr int kMaxN = FP8 ? 64 : 128;  // tokens of one pass over the weights
  static constexpr bool kLow = !UP && !FP8;     // a's low parts follow

  const LayerArgs& a;
  const Groups& g;
  Barriers& b;
  const CUtensorMap* map;
  uint32_t queue, a16;
  int ring, depth;        // stages, and how many of them are in flight
  uint32_t stage_bytes;
  int kd, limit, tiles, stages, nq;
  uint32_t* given;

  __device__ __forceinline__ ManyPhase(const LayerArgs& args, const Groups& groups, Barriers& bars,
                                       const CUtensorMap* weights, uint32_t smem)
      : a(args), g(groups), b(bars), map(weights), queue(smem) {
    kd = UP ? a.H : a.I;
    limit = UP ? a.I : a.H;
    tiles = (limit + kTileOutputs - 1) / kTileOutputs;
    stages = (kd * kEb + 127) / 128;
    nq = g.nslots * tiles;
    given = a.arrived + kBarriers + (UP ? 0 : 1);
    // the same stages in both phases
    const int n = columns(min(b.max_tokens, kMaxN));
    stage_bytes = kWeightBytes + n * 256;
    const int room = static_cast<int>(kQueueBytes - (FP8 ? 2 * kA16Bytes : 0));
    ring = min(room / static_cast<int>(stage_bytes), kMaxRing);
    depth = ring - 2;
    a16 = queue + static_cast<uint32_t>(kQueueBytes) - 2 * kA16Bytes;
  }

  static __device__ __forceinline__ int columns(int tokens) { return (tokens + 15) / 16 * 16; }
  __device__ __forceinline__ uint32_t stage(int slot) const { return queue + slot * stage_bytes; }
  __device__ __forceinline__ int expert(int slot) const {
    const int p = g.slot_expert[slot];
    return p < a.S ? a.E + p : p - a.S;
  }
  // The row of the expert's weights in row r of the tile, behind the last
  // output the last one's again.
  __device__ __forceinline__ int weight_row(int tile, int r) const {
    if (!UP) return min(tile * 128 + r, limit - 1);
    const int l = r & 31;
    return min(tile * 64 + (r >> 5) * 16 + (l & 15), limit - 1) + (l < 16 ? 0 : a.I);
  }

  // Every lane waits, and all leave together.
  __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(kFull, wait_phase(bar, parity, a.wait_ns));
  }

  // -- copying warps

  // Asks for 128 bytes (column block kb) of the 128 weight rows of job q: up,
  // for each quarter 16 gate rows and 16 up rows.  Behind the last output and
  // the last column zeros arrive.
  __device__ __forceinline__ void send_weights(State& s, int q, int kb, int tid) const {
    const int part = tid / 32;
    if (tid % 32 == 0 && part < kParts) {
      const int slot = q / tiles, tile = q - slot * tiles;
      uint64_t* bar = &b.landed[s.sent.slot];
      mbar_arrive_expect_tx(bar, kWeightBytes / kParts);
      tma_load_3d(stage(s.sent.slot) + part * (kWeightBytes / kParts), map, kb * (128 / kEb),
                  (tile * kParts + part) * (UP ? 16 : 32), expert(slot) * (UP ? 2 : 1), bar);
    }
    s.sent.step(ring);
    ++s.issued;
  }
  // Before the tokens are there: the weights of the first stages.
  __device__ __forceinline__ int send_ahead(State& s, int tid) const {
    const int q = blockIdx.x;
    if (q >= nq) return 0;
    const int n = min(depth, stages);
    for (int kb = 0; kb < n; ++kb) send_weights(s, q, kb, tid);
    return n;
  }
  // After a wait that gave up: the weights on their way have landed.
  __device__ __forceinline__ void drain(const State& s, int tid) const {
    if (tid % 32 != 0 || tid / 32 >= kParts) return;
    for (int i = max(s.issued - ring, 0); i < s.issued; ++i)
      wait_phase(&b.landed[i % ring], (i / ring) & 1u, MOE_DEFAULT_WAIT_LIMIT_NS);
  }

  // The oldest stage that was copied is complete: e4m3 weights to fp16, and the
  // news to the issuing warp.
  __device__ __forceinline__ bool announce(State& s, int tid) const {
    bool ok = true;
    if (FP8) {
      ok = warp_wait(&b.a16_empty[s.a16.slot], s.a16.parity ^ 1u);
      ok = warp_wait(&b.landed[s.ready.slot], s.ready.parity) && ok;
      const int row = tid / 8, c = tid % 8;
      const uint32_t from = stage(s.ready.slot) + tid * 16;
      const uint32_t to = a16 + s.a16.slot * kA16Bytes + (c >> 2) * (kTileRows * 128) + row * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Vec16 v = lds16(from + i * 4096);
        uint32_t h[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f16_of_e4m3(v.u[j], h[j / 2][j % 2 * 2], h[j / 2][j % 2 * 2 + 1]);
        // lanes of the second half write their units the other way round, so
        // that the 8 lanes of a row meet 8 different banks
        const int first = c >> 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int unit = (c & 3) * 2 + (j ^ first);
          const uint32_t v4[4] = {first ^ j ? h[1][0] : h[0][0], first ^ j ? h[1][1] : h[0][1],
                                  first ^ j ? h[1][2] : h[0][2], first ^ j ? h[1][3] : h[0][3]};
          if (ok) sts16(to + i * 4096 + ((unit ^ (row & 7)) << 4), v4);
        }
      }
      s.a16.step(2);
    }
    fence_operands();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&b.full[s.ready.slot]);
    s.ready.step(ring);
    --s.landing;
    return ok;
  }

  __device__ __forceinline__ bool copy(State& s, int ahead, int tid) const {
    bool ok = true;
    int q = static_cast<int>(blockIdx.x) < nq ? static_cast<int>(blockIdx.x) : -1;
    if (tid == 0) b.jobs[s.job % kJobRing] = q;
    while (q >= 0) {
      int ticket = 0;
      if (tid == 0) ticket = static_cast<int>(atomicAdd(given, 1u));
      const int p = g.slot_expert[q / tiles];
      const uint8_t* src = UP ? (FP8 ? reinterpret_cast<const uint8_t*>(a.x16) : a.x) : a.a;
      for (int c0 = 0; c0 < g.cnt[p] && ok; c0 += kMaxN) {
        const int cnt = min(g.cnt[p] - c0, kMaxN), begin = g.start[p] + c0;
        const int n = columns(cnt);
        // a row's units of 16 bytes: 8 in bf16, 16 (two slices) in fp16
        constexpr int kAcross = FP8 ? 16 : 8, kDown = kCopyThreads / kAcross, kMost = kMaxN / kDown;
        const int unit = tid % kAcross, row = tid / kAcross;
        uint32_t from[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
          const int r = row + j * kDown;
          const int entry = g.order[begin + min(r, cnt - 1)];
          from[j] = static_cast<uint32_t>(UP ? entry / (a.K + a.S) : entry) * (kd * 2u) + unit * 16;
        }
        const uint32_t to = kWeightBytes + (unit >> 3) * (n * 128) + row * 128 +
                            (((unit & 7) ^ (row & 7)) << 4);
        const int64_t low = static_cast<int64_t>(a.T) * (a.K + a.S) * kd * 2;
        for (int kb = 0; kb < stages; ++kb) {
          ok = warp_wait(&b.empty[s.fill.slot], s.fill.parity ^ 1u);
          if (!ok) break;
          const uint32_t at = stage(s.fill.slot);
          if (ahead > 0) --ahead;
          else send_weights(s, q, kb, tid);
          const bool in = kb * (kAcross * 16) + unit * 16 < kd * 2;
          const uint8_t* tokens = src + kb * (kAcross * 16);
#pragma unroll
          for (int j = 0; j < kMost; ++j)
            if (row + j * kDown < cnt) {
              copy16_stream(at + to + j * (kDown * 128), tokens + from[j], in);
              if (kLow) copy16_stream(at + to + n * 128 + j * (kDown * 128), tokens + low + from[j], in);
            }
          copies_commit();
          ++s.landing;
          s.fill.step(ring);
          if (s.landing > depth) {
            copies_wait_for(depth);
            ok = announce(s, tid);
            if (!ok) break;
          }
        }
      }
      ++s.job;
      if (tid == 0) {
        const int next = ticket + static_cast<int>(gridDim.x);
        b.jobs[s.job % kJobRing] = next < nq ? next : -1;
      }
      if (!copy_warps_and(ok)) {
        ok = false;
        break;
      }
      q = b.jobs[s.job % kJobRing];
    }
    copies_wait<0>();
    while (s.landing > 0 && ok) ok = announce(s, tid);
    // a stage of nothing carries the end (jobs: -1)
    if (ok) ok = warp_wait(&b.empty[s.fill.slot], s.fill.parity ^ 1u);
    if ((tid & 31) == 0) mbar_arrive(&b.full[s.fill.slot]);
    if (ok && tid % 32 == 0 && tid / 32 < kParts) mbar_arrive(&b.landed[s.fill.slot]);
    s.fill.step(ring);
    s.ready.step(ring);
    s.sent.step(ring);
    ++s.issued;
    ++s.job;
    return ok;
  }

  // -- the issuing thread

  __device__ __forceinline__ bool products(State& s, uint32_t tmem) const {
    constexpr uint32_t kFormat = (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) |
                                 (static_cast<uint32_t>(kTileRows >> 4) << 24);
    for (;; ++s.job) {
      if (!wait_phase(&b.full[s.ready.slot], s.ready.parity, a.wait_ns)) return false;
      const int q = b.jobs[s.job % kJobRing];
      if (q < 0) break;
      const int p = g.slot_expert[q / tiles];
      for (int c0 = 0; c0 < g.cnt[p]; c0 += kMaxN) {
        const int n = columns(min(g.cnt[p] - c0, kMaxN));
        const uint32_t idesc = kFormat | (static_cast<uint32_t>(n >> 3) << 17);
        for (int kb = 0; kb < stages; ++kb) {
          if (!wait_phase(&b.full[s.ready.slot], s.ready.parity, a.wait_ns)) return false;
          if (!FP8 && !wait_phase(&b.landed[s.ready.slot], s.ready.parity, a.wait_ns)) return false;
          if ((FP8 || kb == 0) && !wait_phase(&b.acc_empty[s.acc.slot], s.acc.parity ^ 1u, a.wait_ns))
            return false;
          tc_fence_after();
          const uint32_t d = tmem + s.acc.slot * kMaxN;
          const uint32_t at = stage(s.ready.slot);
          if (FP8) {
            const uint32_t w = a16 + s.a16.slot * kA16Bytes;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16(d, sw128_desc(w + k / 4 * (kTileRows * 128)) + k % 4 * 2,
                      sw128_desc(at + kWeightBytes + k / 4 * (n * 128)) + k % 4 * 2, idesc, k > 0);
            mma_commit(&b.a16_empty[s.a16.slot]);
            s.a16.step(2);
          } else {
            const uint64_t w = sw128_desc(at), x = sw128_desc(at + kWeightBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16(d, w + k * 2, x + k * 2, idesc, kb > 0 || k > 0);
            if (kLow) {
              const uint64_t lo = sw128_desc(at + kWeightBytes + n * 128);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_f16(d, w + k * 2, lo + k * 2, idesc, true);
            }
          }
          mma_commit(&b.empty[s.ready.slot]);
          s.ready.step(ring);
          if (FP8 || kb == stages - 1) {
            mma_commit(&b.acc_full[s.acc.slot]);
            mbar_arrive(&b.acc_full[s.acc.slot]);
            s.acc.step(2);
          }
        }
      }
    }
    // the end: passed on as an accumulator of nothing
    if (!wait_phase(&b.acc_empty[s.acc.slot], s.acc.parity ^ 1u, a.wait_ns)) return false;
    mma_commit(&b.empty[s.ready.slot]);
    mma_commit(&b.acc_full[s.acc.slot]);
    mbar_arrive(&b.acc_full[s.acc.slot]);
    s.ready.step(ring);
    s.acc.step(2);
    ++s.job;
    return true;
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
    s.acc.step(2);
  }

  // 16 columns (tokens n0 ..) of the warp's rows of the tile.
  __device__ __forceinline__ void store16(const float (&v)[16], int n0, int cnt, int begin, int tile,
                                          int warp, int lane) const {
    const int KS = a.K + a.S;
    if (UP) {
      const int o = tile * 64 + warp * 16 + (lane & 15);
      const bool upper = lane >= 16;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        if (n0 + j >= cnt) break;  // uniform
        // lane l takes column j, lane l + 16 column j + 1
        const float other = __shfl_xor_sync(kFull, upper ? v[j] : v[j + 1], 16);
        const float gate = upper ? other : v[j], up = upper ? v[j + 1] : other;
        const int n = n0 + j + (upper ? 1 : 0);
        const bool real = n < cnt && o < limit;
        const int entry = g.order[begin + min(n, cnt - 1)];
        if (FP8) {
          const float f = __ldcg(a.xscale + entry / KS);
          const float h = act_value(gate * f, a.act) * (up * f);
          if (real) a.a32[static_cast<int64_t>(entry) * a.I + o] = h;
          const uint32_t m = real ? __float_as_uint(h) & 0x7fffffffu : 0u;
          const uint32_t m0 = __reduce_max_sync(kFull, upper ? 0u : m);
          const uint32_t m1 = __reduce_max_sync(kFull, upper ? m : 0u);
          // a maximum does not depend on the order
          if ((lane & 15) == 0 && n < cnt) atomicMax(a.amax + entry, upper ? m1 : m0);
        } else if (real) {
          const float h = act_value(gate, a.act) * up;
          const __nv_bfloat16 hi = __float2bfloat16_rn(h);
          const float rest = h - __bfloat162float(hi);
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.a) + static_cast<int64_t>(entry) * a.I + o;
          dst[0] = hi;
          dst[static_cast<int64_t>(a.T) * KS * a.I] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.0f);
        }
      }
      return;
    }
    const int row = tile * 128 + warp * 32 + lane;
    if (row >= limit) return;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (n0 + j < cnt) {
        const int entry = g.order[begin + n0 + j];
        const float f = FP8 ? 1.0f / f16_factor(__ldcg(a.amax + entry)) : 1.0f;
        a.y[static_cast<int64_t>(entry) * a.H + row] = FP8 ? v[j] * f : v[j];
      }
  }

  __device__ __forceinline__ bool epilogue(State& s, uint32_t tmem, int warp, int lane) const {
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (;; ++s.job) {
      if (!acc_ready(s)) return false;
      const int q = b.jobs[s.job % kJobRing];
      if (q < 0) break;
      const int slot = q / tiles, tile = q - slot * tiles, p = g.slot_expert[slot];
      for (int c0 = 0; c0 < g.cnt[p]; c0 += kMaxN) {
        const int cnt = min(g.cnt[p] - c0, kMaxN), begin = g.start[p] + c0;
        if (FP8) {
          const int r = weight_row(tile, warp * 32 + lane);
          const int64_t row = static_cast<int64_t>(expert(slot)) * (((UP ? 2 * a.I : a.H) + 127) / 128) + r / 128;
          const float* scale = (UP ? a.s13 : a.s2) + row * stages;
          float sum[kMaxN / 16][16] = {};
          float next = __ldg(scale);
          for (int kb = 0; kb < stages; ++kb) {
            const float f = next;
            if (kb + 1 < stages) next = __ldg(scale + kb + 1);
            if (!acc_ready(s)) return false;
#pragma unroll
            for (int c = 0; c < kMaxN / 16; ++c)
              if (c * 16 < cnt) {
                uint32_t v[16];
                tmem_ld16(mine + s.acc.slot * kMaxN + c * 16, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[c][j] = fmaf(f, __uint_as_float(v[j]), sum[c][j]);
              }
            acc_read(s, lane);
          }
#pragma unroll
          for (int c = 0; c < kMaxN / 16; ++c)
            if (c * 16 < cnt) store16(sum[c], c * 16, cnt, begin, tile, warp, lane);
        } else {
          if (!acc_ready(s)) return false;
#pragma unroll 1
          for (int n0 = 0; n0 < cnt; n0 += 16) {
            uint32_t v[16];
            tmem_ld16(mine + s.acc.slot * kMaxN + n0, v);
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]);
            store16(f, n0, cnt, begin, tile, warp, lane);
          }
          acc_read(s, lane);
        }
      }
    }
    acc_read(s, lane);
    ++s.job;
    return true;
  }

  __device__ __forceinline__ bool run(State& s, int ahead, uint32_t tmem) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool ok = true;
    if (warp >= kFirstCopyWarp) ok = copy(s, ahead, threadIdx.x - kFirstCopyWarp * 32);
    else if (warp == kMmaWarp) ok = lane != 0 || products(s, tmem);
    else if (warp < kEpilogueWarps) ok = epilogue(s, tmem, warp, lane);
    if (!ok) raise_flag(a.flags, MOE_DEVERR_TIMEOUT);
    __syncwarp();
    return __syncthreads_and(ok) != 0;
  }
};

template <bool FP8>
__device__ __forceinline__ bool layer_body(const LayerArgs& a, const Groups& g, Barriers& b,
                                           const CUtensorMap* w13, const CUtensorMap* w2,
                                           uint32_t queue, uint32_t tmem, int* ok) {
  const int tid = static_cast<int>(threadIdx.x) - kFirstCopyWarp * 32;
  uint32_t* arrived = a.arrived;  // of the next barrier
  State s;
  const ManyPhase<FP8, true> up(a, g, b, w13, queue);
  const ManyPhase<FP8, false> down(a, g, b, w2, queue);
  int ahead = 0;
  bool done = true;
  if (FP8) {
    if (tid >= 0) ahead = up.send_ahead(s, tid);
    done = grid_wait(a, arrived++, ok);
  }
  done = done && up.run(s, ahead, tmem);
  if (done) {
    grid_arrive(arrived);
    ahead = tid >= 0 ? down.send_ahead(s, tid) : 0;
    done = grid_wait(a, arrived++, ok);
  }
  if (FP8 && done) {
    scale_activations<kThreads>(a, g);
    grid_arrive(arrived);
    done = grid_wait(a, arrived++, ok);
  }
  done = done && down.run(s, ahead, tmem);
  if (done) {
    grid_arrive(arrived);
    if (grid_wait(a, arrived, ok)) sum_entries<kThreads>(a, g);
    return true;
  }
  copies_wait<0>();
  if (tid >= 0) down.drain(s, tid);
  return false;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) layer_many_kernel(
    const __grid_constant__ CUtensorMap w13, const __grid_constant__ CUtensorMap w2, LayerArgs a) {
  constexpr uint32_t kColumns = 2 * ManyPhase<FP8, true>::kMaxN;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ int ok;
  grid_dependency_wait();
  // operands begin on the 1024 bytes after which the swizzle repeats
  uint8_t* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  Barriers& b = *reinterpret_cast<Barriers*>(smem + kQueueBytes);
  const int warp = threadIdx.x >> 5;
  Groups g;
  group_entries<kThreads>(a, g, smem + kQueueBytes + kBarrierBytes);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&b.landed[i], kParts);
      mbar_init(&b.full[i], kCopyWarps);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.a16_empty[i], 1);
      mbar_init(&b.acc_full[i], 2);
      mbar_init(&b.acc_empty[i], kEpilogueWarps);
    }
    mbar_init(&b.drained, 1);
    fence_mbar_init();
    b.max_tokens = 0;
  }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&b.tmem)),
                 "r"(kColumns)
                 : "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int i = threadIdx.x; i < g.nslots; i += kThreads) atomicMax(&b.max_tokens, g.cnt[g.slot_expert[i]]);
  if (FP8) {
    scale_tokens<kThreads>(a, g.tokens, reinterpret_cast<uint32_t*>(smem));
    grid_arrive(a.arrived);
  }
  __syncthreads();
  const uint32_t tmem = b.tmem;
  if (!layer_body<FP8>(a, g, b, &w13, &w2, smem_addr(smem), tmem, &ok)) {
    if (threadIdx.x == kMmaWarp * 32) {
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

// Weights as [matrices, rows, cols], boxes of 128 bytes of `box_rows` rows of
// `box_mats` matrices; bf16 swizzled as the products read them.
bool encode_weights(CUtensorMap* m, const void* base, bool e4m3, uint64_t cols, uint64_t rows,
                    uint64_t mats, uint32_t box_rows, uint32_t box_mats) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const uint64_t eb = e4m3 ? 1 : 2;
  const cuuint64_t dims[3] = {cols, rows, mats};
  const cuuint64_t strides[2] = {cols * eb, rows * cols * eb};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / eb), box_rows, box_mats};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8>
cudaError_t launch_one(const moe_handle* h, const LayerArgs& a, cudaStream_t s) {
  CUtensorMap w13, w2;
  const uint64_t n = a.E + a.S;
  if (!encode_weights(&w13, a.w13, FP8, a.H, a.I, 2 * n, 16, 2) ||
      !encode_weights(&w2, a.w2, FP8, a.I, a.H, n, 32, 1))
    return cudaErrorInvalidValue;
  auto k = layer_many_kernel<FP8>;
  const size_t smem = kFixedBytes + groups_bytes(a.T, a.K + a.S, a.E + a.S);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_chained(k, dim3(h->num_sms), dim3(kThreads), smem, s, true, w13, w2, a);
}

}  // namespace

cudaError_t launch_layer_many(const moe_handle* h, const LayerArgs& a, bool e4m3, cudaStream_t s) {
  return e4m3 ? launch_one<true>(h, a, s) : launch_one<false>(h, a, s);
}

}  // namespace moe
