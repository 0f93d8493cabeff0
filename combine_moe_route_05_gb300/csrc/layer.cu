// A whole MoE layer for a few tokens (sm_103a): after the routing, one kernel
// that streams the reached experts' weights from memory once.  This file: experts
// with a handful of tokens, and the call itself; layer_many.cu: more tokens an
// expert.
//
//   up:      a[t,k,i] = act(<w13_e[i], x_t>) * <w13_e[I + i], x_t>
//   down:    y[t,k,n] = <w2_e[n], a[t,k]>                            (fp32)
//   combine: out[t]   = round(sum_k w[t,k] y[t,k] + sum_j y[t, K + j])
//
// Bound by reading the weights: 2 operations a byte and token.  The products
// run on mma.m16n8k16 with 16 weight rows as the one operand and up to 8 of
// the expert's tokens as the other.  The order of the k index is free as long
// as both operands agree, so a lane takes 16 contiguous bytes of its two weight
// rows as the operand registers of two (bf16) or four (e4m3) products, with its
// token's values at the same k beside them.  In the up products rows 0..7 of
// the 16 are gate rows and 8..15 the up rows of the same outputs: a lane's
// accumulators then hold gate and up of one output and the activation needs no
// exchange.
//
// Every warp copies what it will itself multiply into a queue of its own in
// shared memory (cp.async), several stages ahead and across the ends of jobs,
// so the stream of weights has no gaps and the queue needs no barrier.  A job
// is one expert and one tile of outputs; a team of 1, 2, 4 or 8 warps splits
// its k and adds its partial sums in warp order.  A team's first jobs are dealt
// out beforehand, the others by a counter: the SMs differ in speed by a fifth
// (their way to memory), and jobs dealt out in turn all waited for the slowest.
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
//
// Measured, routing included (GPU time of a replayed graph; in brackets: weights
// read once at the copy rate of 6.78 TB/s; ranges: different boxes and routes, which
// reach more or fewer experts than the mean in brackets): 16 tokens,
// 128 experts, top 8, 2048 x 768, bf16: 127-136 us (115; DRAM reads 785 MB, the
// weights' 778 and the tokens); 4 tokens, 256 experts and a shared one, 7168 x
// 2048: 397-443 us (410); 1 token, 2048 x 768: 27-29 us (11): there the parts in
// front of and between the products bound it: routing 4.5, grouping 1, the
// first weights' latency 2, two grid barriers 3.5, the sum 2 us.  e4m3 weights: 4
// tokens of the second shape 252-257 us (205), 16 of the first 106 (57), 1 of it 29
// (6): the pass that scales the tokens, the one that scales the activations and a
// grid barrier behind each come on top.
#include "layer.cuh"

namespace moe {
namespace {

// Nothing at all where !any (predicated, since the lanes of a warp differ).
__device__ __forceinline__ void copy16_keep(uint32_t dst, const void* src, bool valid, bool any) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\t"
      "@p cp.async.ca.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(dst),
      "l"(src), "r"(valid ? 16 : 0), "r"(static_cast<int>(any))
      : "memory");
}
// 4 bytes of an asynchronous copy.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// 16 bytes of shared memory where `any`; else v keeps what it holds.
__device__ __forceinline__ void lds16_if(Vec16& v, uint32_t p, bool any) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\t"
      "@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "+r"(v.u[0]), "+r"(v.u[1]), "+r"(v.u[2]), "+r"(v.u[3])
      : "r"(p), "r"(static_cast<int>(any))
      : "memory");
}

__device__ __forceinline__ float lds4(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The products of one phase (up or down) for one thread.  PACKED: 4 tokens to a
// tile of 8, so that more of the queue holds weights.
constexpr int kWarps = 16, kThreads = 32 * kWarps;
static_assert(kWarps <= kMaxWarps, "warps");
constexpr int kMaxTeam = 8;
constexpr int kSteps = 2;  // of 64 bytes of a row, in a stage of the queue
constexpr int kQueueBytes = 192 * 1024;
constexpr int kMaxStages = 8;
// a team holds tickets for at most kMaxStages + 1 coming jobs (`fixed` below), and
// one warp may still read the last one's
static_assert(kMaxStages + 2 < kTickets, "tickets");
// behind the queue: two buffers of partial sums, tickets, block scales of the
// stages (e4m3)
constexpr int kSumFloats = kWarps * 4 * 32;
constexpr int kSumBytes = 2 * kSumFloats * 4;
constexpr int kTicketBytes = kWarps * kTickets * 4;
constexpr int kScaleBytes = kWarps * kMaxStages * 2 * 4;
constexpr size_t kFixedBytes = kQueueBytes + kSumBytes + kTicketBytes + kScaleBytes;
static_assert(kFixedBytes + kMaxGroupsBytes + 64 <= 227 * 1024, "shared memory budget");

// Tokens [c0, c0 + kTokens) of the expert in slot `slot`, output tile `tile`;
// q = slot * tiles + tile, i its place in the team's sequence.
struct Job {
  int i, q, slot, tile, c0;
};

template <bool FP8, bool PACKED, bool UP>
struct Phase {
  static_assert(PACKED || !FP8, "e4m3 comes packed");
  static constexpr int kEb = FP8 ? 1 : 2;
  static constexpr int kRowBytes = 64 * kSteps;  // of a weight row in a stage
  static constexpr int kRows = UP ? 8 : 16;      // outputs that 16 weight rows give
  // The low parts of a in bf16.  Packed: as rows (and columns) 4..7 of the tile,
  // one product for both, added at the end; else behind the tile.
  static constexpr bool kPacked = PACKED && (FP8 || !UP);
  static constexpr bool kLowColumns = kPacked && !FP8;
  static constexpr bool kLowRows = !UP && !PACKED;
  static constexpr int kTokens = kPacked ? 4 : 8;  // of a job
  static constexpr int kTokenRows = FP8 ? 4 : kLowRows ? 16 : 8;
  static constexpr int kTokenBytes = kRowBytes * 2 / kEb;  // of a token row in a stage
  static constexpr int kLoads = FP8 || kLowRows ? 2 : 1;   // 16-byte vectors of a lane and step
  // lanes along a row, and rows, of one copy instruction
  static constexpr int kAcross = kRowBytes / 16, kDown = 32 / kAcross;
  static constexpr int kTokenAcross = kTokenBytes / 16, kTokenDown = 32 / kTokenAcross;
  static constexpr int kTokenCopies = kTokenRows / kTokenDown;
  static constexpr int kWeightBytes = 16 * kRowBytes;  // of a warp's stage
  static constexpr int kWarpBytes = kWeightBytes + kTokenRows * kTokenBytes;
  static constexpr int kStageBytes = kWarps * kWarpBytes;
  static constexpr int kStages = kQueueBytes / kStageBytes < kMaxStages ? kQueueBytes / kStageBytes
                                                                        : kMaxStages;
  // an instruction's rows begin at an even one, and weights end on 128 bytes
  static_assert(kTokenRows % kTokenDown == 0 && 8 % kDown == 0 && kDown % 2 == 0 &&
                    kTokenDown % 2 == 0 && kWeightBytes % 128 == 0, "copies");
  static_assert(kStages >= 3, "queue");

  const LayerArgs& a;
  const Groups& g;
  uint32_t queue;   // shared-memory address of this warp's queue
  uint32_t scales;  // of the warp's block scales
  // this lane's places in a stage: where it copies to and loads from
  uint32_t copy_weight, copy_token, load_weight, load_token;
  int kd, tiles, limit, stages, nq;
  int lane, warp;
  int team, part, first_q, stride_q;  // warps that split a job's k
  int fixed;       // jobs of a team that are dealt out beforehand
  int* tickets;    // the team's others
  uint32_t* given;

  __device__ __forceinline__ Phase(const LayerArgs& args, const Groups& groups, uint8_t* smem)
      : a(args), g(groups), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    queue = smem_addr(smem) + warp * kWarpBytes;
    scales = smem_addr(smem) + kQueueBytes + kSumBytes + kTicketBytes + warp * kMaxStages * 2 * 4;
    {
      const int row = lane / kAcross, token = lane / kTokenAcross, odd = (lane >> 2) & 1;
      copy_weight = row * kRowBytes + ((lane % kAcross * 16) ^ (row % 2 * kTurn));
      copy_token = kWeightBytes + token * kTokenBytes +
                   ((lane % kTokenAcross * 16) ^ (token % 2 * kTokenTurn));
      load_weight = (lane >> 2) * kRowBytes + (((lane & 3) * 16) ^ (odd * kTurn));
      load_token = kWeightBytes + (lane >> 2) * kTokenBytes +
                   (((lane & 3) * (FP8 ? 32 : 16)) ^ (odd * kTokenTurn));
    }
    kd = UP ? a.H : a.I;
    limit = UP ? a.I : a.H;
    tiles = (limit + kRows - 1) / kRows;
    stages = (kd * kEb + kRowBytes - 1) / kRowBytes;
    nq = g.nslots * tiles;
    // Many jobs: a larger team makes them shorter, so that they even out at the
    // end what the SMs differ in speed, but has fewer stages between the
    // barriers at their ends.  A team grows while each of its warps keeps 8
    // stages and it has less than 64 jobs, or 4 stages and 20 jobs (37 of 64
    // tokens e4m3, DeepSeek-V3 shape: 1375 us with 4 stages and no count of
    // jobs, 1279 so; 16 tokens, Qwen3-30B shape: 139 us with 8 stages alone, 133
    // so).  Few: the team size with the fewest rounds over the grid, in rounds
    // of a job of one.
    const int warps = kWarps * gridDim.x;
    team = 1;
    if (nq >= warps / kMaxTeam * 6) {
      const auto grows = [&](int per_warp, int64_t jobs) {
        return 2 * per_warp * team <= stages && static_cast<int64_t>(nq) * team < jobs * warps;
      };
      while (team < kMaxTeam && (grows(8, 64) || grows(4, 20))) team *= 2;
    } else {
      float best = 0.0f;
#pragma unroll 1
      for (int n = 1; n <= kMaxTeam && n <= stages; n *= 2) {
        const float cost = static_cast<float>((nq * n + warps - 1) / warps) / n;
        if (n == 1 || cost < best) {
          best = cost;
          team = n;
        }
      }
    }
    first_q = blockIdx.x + gridDim.x * (warp / team);
    stride_q = gridDim.x * (kWarps / team);
    part = warp % team;
    // the copies of a warp run at most (per - 1 + kStages) / per jobs ahead,
    // and a ticket is there from the second job behind its request on
    const int per = stages / team;
    fixed = (per - 1 + kStages) / per + 1;
    tickets = reinterpret_cast<int*>(smem + kQueueBytes + kSumBytes) + warp / team * kTickets;
    given = a.arrived + kBarriers + (UP ? 0 : 1);
  }

  __device__ __forceinline__ bool valid(const Job& j) const { return j.q < nq; }
  __device__ __forceinline__ Job at(int i) const {
    const int q = i < fixed ? first_q + i * stride_q : tickets[i % kTickets];
    const int slot = q / tiles;
    return Job{i, q, slot, q - slot * tiles, 0};
  }
  __device__ __forceinline__ Job next(const Job& j) const {
    if (j.c0 + kTokens < g.cnt[g.slot_expert[j.slot]]) return Job{j.i, j.q, j.slot, j.tile, j.c0 + kTokens};
    return at(j.i + 1);
  }
  __device__ __forceinline__ int first_row(const Job& j) const { return j.tile * kRows; }
  // Odd rows have two halves of their 16-byte units changed over (bit 2 of a
  // unit's number, e4m3 tokens: bit 0), so that the 8 lanes of a shared-memory
  // access, 4 each of two rows, meet no bank twice.
  static constexpr int kTurn = 64, kTokenTurn = FP8 ? 16 : kTurn;

  // Where this warp's next copies come from.  A copy instruction takes kDown
  // rows of kRowBytes: whole 128-byte lines of few rows (16 rows by 64 bytes
  // an instruction took 49 GB/s an SM from L2, lines 75).
  struct Cursor {
    Job j;
    int o;                  // byte of the weight rows
    const uint8_t* row;     // this lane's place in the first kDown rows, from byte o on
    int64_t half;           // from rows 0..7 of a tile to rows 8..15
    const uint8_t* col[kTokenCopies];  // this lane's places in rows of x or a
    uint32_t have;          // bit i: there is a row in col[i]
    const float* scale;     // the block scales' row of lanes 0 and 1
  };

  __device__ __forceinline__ void open(Cursor& c) const {
    if (!valid(c.j)) return;
    const int p = g.slot_expert[c.j.slot];
    const int e = p < a.S ? a.E + p : p - a.S;
    const int r0 = first_row(c.j);
    const int64_t all_rows = UP ? 2 * a.I : a.H;
    c.o = part * kRowBytes;
    c.row = (UP ? a.w13 : a.w2) + (e * all_rows + r0 + lane / kAcross) * kd * kEb + c.o + lane % kAcross * 16;
    // the last tile of the down products may have no second half: it reads
    // the first again, and its results go nowhere
    c.half = static_cast<int64_t>(UP ? a.I : r0 + 8 >= limit ? 0 : 8) * kd * kEb;
    if (FP8 && lane < 2) {
      const int r = r0 + (UP && lane ? a.I : 0);
      c.scale = (UP ? a.s13 : a.s2) + (e * ((all_rows + 127) / 128) + r / 128) * ((kd + 127) / 128);
    }
    const int cnt = min(g.cnt[p] - c.j.c0, kTokens), begin = g.start[p] + c.j.c0;
    const uint8_t* src = UP ? (FP8 ? reinterpret_cast<const uint8_t*>(a.x16) : a.x) : a.a;
    src += c.o * (2 / kEb) + lane % kTokenAcross * 16;
    c.have = 0;
#pragma unroll
    for (int i = 0; i < kTokenCopies; ++i) {
      const int row = i * kTokenDown + lane / kTokenAcross;
      const bool low = kLowColumns ? row >= 4 : kLowRows && row >= 8;
      const int n = kLowColumns ? row & 3 : row & 7;
      c.col[i] = src;
      if (n < cnt) {
        const int entry = g.order[begin + n];
        c.col[i] += static_cast<int64_t>((UP ? entry / (a.K + a.S) : entry) +
                                         (low ? a.T * (a.K + a.S) : 0)) * kd * 2;
        c.have |= 1u << i;
      }
    }
  }
  __device__ __forceinline__ Cursor begin() const {
    Cursor c;
    c.j = at(0);
    open(c);
    return c;
  }
  __device__ __forceinline__ void advance(Cursor& c) const {
    const int step = team * kRowBytes;
    c.o += step;
    if (c.o < kd * kEb) {
      c.row += step;
#pragma unroll
      for (int i = 0; i < kTokenCopies; ++i) c.col[i] += step * (2 / kEb);
      return;
    }
    c.j = next(c.j);
    open(c);
  }

  __device__ __forceinline__ void copy_weights(const Cursor& c, uint32_t dst) const {
    const bool in = c.o + lane % kAcross * 16 < kd * kEb;
    const int64_t down = static_cast<int64_t>(kDown) * kd * kEb;
    dst += copy_weight;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8 / kDown; ++i)
        copy16_stream(dst + (h * 8 + i * kDown) * kRowBytes, c.row + (h ? c.half : 0) + i * down, in);
    if (FP8 && lane < 2)
      copy4(scales + ((dst - copy_weight - queue) / kStageBytes * 2 + lane) * 4, c.scale + c.o / 128);
  }
  __device__ __forceinline__ void copy_tokens(const Cursor& c, uint32_t dst) const {
    const bool in = c.o * (2 / kEb) + lane % kTokenAcross * 16 < kd * 2;
    dst += copy_token;
#pragma unroll
    for (int i = 0; i < kTokenCopies; ++i)
      copy16_keep(dst + i * kTokenDown * kTokenBytes, c.col[i], in, (c.have >> i) & 1u);
  }

  // The token (of the job) that this lane's operand holds.
  __device__ __forceinline__ int lane_token() const {
    return kLowColumns ? (lane >> 2) & 3 : lane >> 2;
  }

  // One stage's operands.
  struct Operands {
    Vec16 w[kSteps][2];
    Vec16 x[kSteps][kLoads];
    float sc[2];  // block scales of the lane's accumulator rows
  };

  // has: the lane has a token (without one its operand registers, and the
  // columns of its sums, mean nothing).
  __device__ __forceinline__ void load(Operands& v, uint32_t at, bool has) const {
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t from =
            FP8 ? (load_token ^ (i * kTokenTurn)) + st * 128 : load_token ^ (st * kTokenTurn);
        lds16_if(v.x[st][i], at + from + (kLowRows ? i * 8 : 0) * kTokenBytes, has);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v.w[st][h] = lds16(at + (load_weight ^ (st * kTurn)) + h * 8 * kRowBytes);
    }
    if (FP8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) v.sc[h] = lds4(scales + ((at - queue) / kStageBytes * 2 + h) * 4);
    }
  }

  // Sums that run beside each other, so that a product need not wait for the
  // one before it; added at the end of a job (bf16) or a stage (e4m3).
  static constexpr int kChains = FP8 ? 2 : 4;

  // acc += the products of one stage.
  __device__ __forceinline__ void multiply(float (&acc)[kChains][4], const Operands& v) const {
    float sum[kChains][4] = {};
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const Vec16& w0 = v.w[st][0];
      const Vec16& w1 = v.w[st][1];
      if (!FP8) {
#pragma unroll
        for (int q = 0; q < 4; q += 2)
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
            mma<false>(acc[(q / 2 + st * 2) % kChains], w0.u[q], w1.u[q], w0.u[q + 1], w1.u[q + 1],
                       v.x[st][i].u[q], v.x[st][i].u[q + 1]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a0, a1, a2, a3;
          f16_of_e4m3(w0.u[q], a0, a2);
          f16_of_e4m3(w1.u[q], a1, a3);
          mma<true>(sum[q % kChains], a0, a1, a2, a3, v.x[st][(q / 2) % kLoads].u[q % 2 * 2],
                    v.x[st][(q / 2) % kLoads].u[q % 2 * 2 + 1]);
        }
      }
    }
    if (FP8) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[0][r] = fmaf(v.sc[r / 2], sum[0][r] + sum[1][r], acc[0][r]);
    }
  }

  // What undoes an entry's factor (e4m3): loaded at a job's start, worked out
  // at its end.
  __device__ __forceinline__ uint32_t held_factor(int entry) const {
    return UP ? __ldcg(reinterpret_cast<const uint32_t*>(a.xscale) + entry / (a.K + a.S))
              : __ldcg(a.amax + entry);
  }
  static __device__ __forceinline__ float inverse(uint32_t held) {
    return UP ? __uint_as_float(held) : 1.0f / f16_factor(held);
  }

  // One result pair of entry `entry`, f its inverse(): up: gate and up of output
  // `row`; down: outputs row and row + 8.
  __device__ __forceinline__ void store(int entry, int row, float v0, float v1, float f) const {
    if (row >= limit) return;
    const int KS = a.K + a.S;
    if (!UP) {
      if (FP8) {
        v0 *= f;
        v1 *= f;
      }
      float* y = a.y + static_cast<int64_t>(entry) * a.H + row;
      y[0] = v0;
      if (row + 8 < limit) y[8] = v1;
      return;
    }
    if (FP8) {
      const float h = act_value(v0 * f, a.act) * (v1 * f);
      a.a32[static_cast<int64_t>(entry) * a.I + row] = h;
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

  __device__ __forceinline__ void sync_team() const {
    if (team == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(warp / team + 1), "r"(team * 32) : "memory");
  }

  // The first stages: all of them, or the weights alone while the tokens are
  // not there yet (c is then left where it was).
  template <bool WEIGHTS, bool TOKENS>
  __device__ __forceinline__ void start(Cursor& from) const {
    Cursor c = from;
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s) {
      if (valid(c.j)) {
        if (WEIGHTS) copy_weights(c, queue + s * kStageBytes);
        if (TOKENS) copy_tokens(c, queue + s * kStageBytes);
        advance(c);
      }
      if (TOKENS) copies_commit();
    }
    if (TOKENS) from = c;
  }

  // Everything else.
  __device__ __forceinline__ void run(Cursor& c, float* red) const {
    const bool leader = part == 0 && lane == 0;
    int ticket = 0, sums = 0;
    if (leader) ticket = static_cast<int>(atomicAdd(given, 1u));
    uint32_t from = queue, to = queue + (kStages - 1) * kStageBytes;
    Job j = at(0);
#pragma unroll 1
    while (valid(j)) {
      const int p = g.slot_expert[j.slot];
      const int cnt = min(g.cnt[p] - j.c0, kTokens), begin = g.start[p] + j.c0;
      uint32_t f[2] = {};
      if (FP8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * (lane & 3) + i;
          if (n < cnt) f[i] = held_factor(g.order[begin + n]);
        }
      }
      float acc[kChains][4] = {};
#pragma unroll 1
      for (int st = part; st < stages; st += team) {
        copies_wait<kStages - 2>();
        // the lanes' copies are there for one another, and no lane still
        // reads the slot that is filled next
        __syncwarp();
        Operands v;
        load(v, from, lane_token() < cnt);
        // the stage before this one has been multiplied: its slot is free
        if (valid(c.j)) {
          copy_weights(c, to);
          copy_tokens(c, to);
          advance(c);
        }
        copies_commit();
        multiply(acc, v);
        to = from;
        from = from + kStageBytes == queue + kStages * kStageBytes ? queue : from + kStageBytes;
      }
      float (&v)[4] = acc[0];
      if (!FP8) {
#pragma unroll
        for (int i = 1; i < kChains; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] += acc[i][r];
      }
      // the ticket that was asked for at the last job's end
      const bool ends = j.c0 + kTokens >= g.cnt[p];
      if (leader && ends) tickets[(fixed + j.i) % kTickets] = fixed * stride_q + ticket;
      // The team's partial sums, added in warp order by one of its warps.  With
      // two buffers, whoever writes one has passed the sync behind the reads
      // of its last contents.
      float* buf = red + sums % 2 * kSumFloats;
      if (team > 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) buf[(warp * 4 + r) * 32 + lane] = v[r];
      }
      sync_team();
      if (sums++ % team == part) {
        if (team > 1) {
          const float* at = buf + (warp - part) * 4 * 32 + lane;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = at[r * 32] + at[(4 + r) * 32];
#pragma unroll
          for (int u = 2; u < kMaxTeam; ++u)
            if (u < team) {
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] += at[(u * 4 + r) * 32];
            }
        }
        if (kLowColumns) {  // columns n and n + 4
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] += __shfl_xor_sync(kFull, v[r], 2);
        }
        const int n = 2 * (lane & 3);
        const int row = first_row(j) + (lane >> 2);
        if (n < cnt) store(g.order[begin + n], row, v[0], v[2], inverse(f[0]));
        if (n + 1 < cnt) store(g.order[begin + n + 1], row, v[1], v[3], inverse(f[1]));
      }
      if (leader && ends) ticket = static_cast<int>(atomicAdd(given, 1u));
      j = next(j);
    }
    copies_wait<0>();
  }
};

// fp16 copies of x and their factors: a block per token.
__device__ __forceinline__ void scale_tokens(const LayerArgs& a, int tokens, uint32_t* red) {
  for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
    const uint8_t* row = a.x + static_cast<int64_t>(t) * a.H * 2;
    const float f = f16_factor(block_max_bits<kThreads>(row, a.H, red));
    uint8_t* dst = reinterpret_cast<uint8_t*>(a.x16) + static_cast<int64_t>(t) * a.H * 2;
    for (int v = threadIdx.x; v < a.H / 8; v += kThreads)
      st_vec(dst + v * 16, scaled_f16(ld_vec(row + v * 16), f));
    if (threadIdx.x == 0) a.xscale[t] = 1.0f / f;
    for (int k = threadIdx.x; k < a.K + a.S; k += kThreads) a.amax[t * (a.K + a.S) + k] = 0;
  }
}

// fp16 copies of the activations, their factors from the entries' maxima.
__device__ __forceinline__ void scale_activations(const LayerArgs& a, const Groups& g) {
  const int per = a.I / 8;
  const int64_t n = static_cast<int64_t>(g.tokens) * (a.K + a.S) * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int entry = static_cast<int>(i / per);
    if (g.rank[entry] != kNone) scale_activation(a, i, __ldcg(a.amax + entry));
  }
}

template <bool FP8, bool PACKED>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(LayerArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int ok;
  grid_dependency_wait();
  float* red = reinterpret_cast<float*>(smem + kQueueBytes);
  Groups g;
  group_entries<kThreads, false>(a, g, smem + kFixedBytes, nullptr);
  uint32_t* arrived = a.arrived;  // of the next barrier
  if (FP8) {
    scale_tokens(a, g.tokens, reinterpret_cast<uint32_t*>(red));
    grid_arrive(arrived);
  }
  {
    const Phase<FP8, PACKED, true> up(a, g, smem);
    typename Phase<FP8, PACKED, true>::Cursor c = up.begin();
    if (FP8) {
      up.template start<true, false>(c);
      if (!grid_wait(a, arrived++, &ok)) {
        copies_wait<0>();
        return;
      }
      up.template start<false, true>(c);
    } else {
      up.template start<true, true>(c);
    }
    up.run(c, red);
  }
  grid_arrive(arrived);
  {
    const Phase<FP8, PACKED, false> down(a, g, smem);
    typename Phase<FP8, PACKED, false>::Cursor c = down.begin();
    down.template start<true, false>(c);
    bool done = grid_wait(a, arrived++, &ok);
    if (FP8 && done) {
      scale_activations(a, g);
      grid_arrive(arrived);
      done = grid_wait(a, arrived++, &ok);
    }
    if (!done) {
      copies_wait<0>();
      return;
    }
    down.template start<false, true>(c);
    down.run(c, red);
  }
  grid_arrive(arrived);
  if (!grid_wait(a, arrived, &ok)) return;

  sum_entries<kThreads>(a, g);
}

// Zeroes the barrier counters where no routing kernel does.
__global__ void layer_start_kernel(uint32_t* arrived) {
  grid_dependency_wait();
  if (threadIdx.x < kLayerCounters) arrived[threadIdx.x] = 0;
}

template <bool FP8, bool PACKED>
cudaError_t launch_few(const moe_handle* h, const LayerArgs& a, cudaStream_t s) {
  const size_t smem = kFixedBytes + groups_bytes(a.T, a.K + a.S, a.E + a.S);
  return launch_chained(layer_kernel<FP8, PACKED>, dim3(h->num_sms), dim3(kThreads), smem, s, true, a);
}

}  // namespace

cudaError_t prepare_layer_kernels() {
  cudaError_t e = allow_shared(layer_kernel<false, false>, kFixedBytes);
  if (e == cudaSuccess) e = allow_shared(layer_kernel<false, true>, kFixedBytes);
  if (e == cudaSuccess) e = allow_shared(layer_kernel<true, true>, kFixedBytes);
  return e == cudaSuccess ? prepare_layer_many_kernels() : e;
}

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
  // Tokens an expert in the mean from which on the kernel of layer_many.cu is the
  // faster one.  bf16: 3 to 7, the more the fewer weights there are (64 experts,
  // top 8, 2048 x 1408: 184 against 181 us at 4 tokens, 194 against 183 at 5;
  // 1024 x 512: 54 against 59 at 5, 65 against 59 at 8).  e4m3, whose weights
  // the kernel here converts again for every 4 tokens: 1, or some 48 entries in
  // all (16 experts, top 2, 4096 x 2048: 71 against 78 us at 16 entries, 93
  // against 89 at 24; 256 experts, top 8, 7168 x 2048: 234 against 250 at 32
  // entries, 426 against 408 at 64).  T counts, not the live tokens, which the
  // host does not know: 1 live of 128 tokens, 128 experts, top 8, 2048 x 768, takes
  // 34 us by this rule, 30 with the other kernel (8 experts, top 2, 4096 x 2048: 39
  // and 31).
  //
  // Packed up to 2 tokens: above it 4 tokens to a tile make second passes.  128
  // experts, top 8, 2048 x 768: packed 89.0 us, unpacked 89.9 at 0.5, 130.4 and
  // 131.1 at 1, 178.5 and 178.2 at 2, 196.1 and 193.0 at 3, 208.7 and 203.5 at 4;
  // 32 experts, top 4, 4096 x 1024: 66.3 and 67.1, 96.3 and 97.0, 117.7 and 117.2,
  // 132.1 and 128.2, 144.0 and 136.9.
  //
  // A shared expert has all T tokens, whose passes over a tile (8 or 4 tokens
  // each) one team makes in turn, and those of several run beside one another:
  // from T (S + 1) = 24 (16 experts) to 56 (128) on the other kernel is the faster
  // one with bf16 weights, from 16 on with e4m3 weights (64 experts, top 1, 2048 x
  // 1408: bf16 with 1 shared expert 86.6 against 86.6 us at 28 tokens, 211 against
  // 187 at 128, with 4 63 against 62 at 10, 341 against 197 at 128; e4m3 with 1
  // 43.5 against 46 at 8, 55 against 52 at 10, 132 against 89 at 48).  Over 130
  // random shapes with 1 to 4 shared experts the kernel taken is 0.6% above the
  // faster one in the mean, 13% at most; without this part 5% and 138%.
  const int64_t entries = static_cast<int64_t>(T) * K;
  const bool e4m3 = q.weight_dtype == MOE_E4M3;
  const int most_shared = e4m3 ? 16 : 16 + a.E / 2 < 56 ? 16 + a.E / 2 : 56;
  if (entries > (e4m3 ? (a.E < 48 ? a.E : 48) : 5 * a.E) ||
      (a.S > 0 && T * (a.S + 1) > most_shared))
    return launch_layer_many(h, a, e4m3, s);
  if (e4m3) return launch_few<true, true>(h, a, s);
  return entries > 2 * a.E ? launch_few<false, false>(h, a, s) : launch_few<false, true>(h, a, s);
}

}  // namespace moe
