// The persistent worker of the tiled GEMM (gfx950): main loop, tile schedulers and
// epilogue staging. gemm_kernel.hip instantiates it as the plain product, C (fp32) =
// A (bf16, M x K) . B (bf16, K x N), product_kernel.hip with other operand layouts,
// e4m3 operands and a fused epilogue; the operation's type (OP) says which.
//
// One workgroup = a 2 x 2 grid of wave64s. 256 x 256 tiles: one workgroup per
// CU, each wave owns 128 x 128 of the tile as 8 x 8 blocks of
// v_mfma_f32_16x16x32_bf16 (one wave per SIMD). 128 x 128 tiles: two
// workgroups per CU, each wave owns 64 x 64 as 2 x 2 blocks of
// v_mfma_f32_32x32x16_bf16. Accumulation is fp32 throughout. Operand tiles move
// global -> LDS with buffer_load_dwordx4 ... lds (16 bytes per lane, no VGPR
// round trip) into a ring of four 32-deep LDS stages, each load two to three
// k-steps ahead of its first reader.
//
// LDS layouts: the four B stages first, then the four A stages (so that reads
// of a stage known at compile time need no address arithmetic in the loop);
// 16-byte chunks, XOR-swizzled so fragment reads are bank-conflict free:
//   A stage: BM rows x 32 k, 64 B per row; logical chunk c of row r sits in slot
//            c ^ ((r >> 1) & 3) (16 x 16 blocks) or c ^ ((r >> 2) & 3) (32 x 32).
//            A fragments are read with ds_read_b128 (8 consecutive k of one row
//            per lane).
//   B stage: 32 k rows x BN n; logical chunk c of row k sits in slot
//            c ^ s(k), s(k) = (10 (k & 1) + 4 ((k >> 1) & 1)) ^ 2 ((k >> 3) & 1).
//            B fragments need 8 consecutive k of one column per lane;
//            ds_read_b64_tr_b16 delivers them from the row-major (n-contiguous)
//            tile: in each 16-lane group, lane L reads 4 n values of row L/4 and
//            lane i receives column i of the 4 x 16 block.
// An operand given the other way round takes the other one's layout: B as N x K
// rows (BT) is staged and read like A, A as K x M rows (AT) like B. e4m3 operands
// (E8, both K-contiguous) use A's layout byte for byte: the body counts K and the
// row strides in 16-bit units, a 64-byte stage row holds 64 e4m3 values, and a
// fragment becomes bf16 in registers (exact) on its way to the bf16 MFMAs. (The
// e4m3 MFMAs do not keep 32-bit sums: measured on gfx950, they add eight products
// at a time and drop what lies 2^-13 below the largest of the eight, so 2^14 -
// 2^14 + 1 gives 0, in the 32x32x64 and 16x16x128 f8f6f4 forms and in the older
// 32x32x16 and 16x16x32 ones alike.)
// The MFMA is issued with the B fragment as its first operand, so each group of
// four accumulators of a lane holds four consecutive n of one row m, which the
// epilogue writes as one 16-byte store.
//
// Work units. The schedulers hand out work units; a unit is one work item, or
// with claim groups g consecutive items that one worker runs back to back. An
// item is a whole tile, or with a split tail one K-chunk of a tile of the
// partial last wave: a chunk stores its fp32 partial tile to plan scratch and
// the workgroup that completes the tile's last chunk adds the partials in chunk
// order and writes C (no workgroup ever waits for another).
//
// Scheduling: see the header comment of ptg_gemm.h. The work loop is the
// persistent worker loop of the blog post "CUTLASS Cluster Launch Control
// dynamic persistent kernel" (section "cancelling the launch, receiving the
// work coordinate": compute the tile, fetch the next coordinate, stop on
// failure); the claim-ahead and its LDS ring of response records follow its
// section "following the CUTLASS source" (one elected producer thread, a
// depth-3 response pipeline, a throttle on how far ahead claims run, consumers
// check the success flag before the coordinate).
#pragma once

#include <type_traits>

#include "ptg_device.hpp"

namespace ptg {

// Tile shape, wave grid and MFMA shape. A workgroup has WAVES_M x WAVES_N
// wave64s; each wave owns a (BM/WAVES_M) x (BN/WAVES_N) block of the output
// tile, made of MB x MB MFMA blocks: MB = 32 uses v_mfma_f32_32x32x16_bf16 (two
// MFMAs per 32-deep stage), MB = 16 uses v_mfma_f32_16x16x32_bf16 (one).
template <int BM, int BN, int WAVES_M, int WAVES_N, int MB_, int STAGES = 4>
struct Cfg {
  static constexpr int BM_ = BM, BN_ = BN, WAVES_N_ = WAVES_N;
  static constexpr int NW = WAVES_M * WAVES_N;
  static constexpr int THREADS = 64 * NW;
  static constexpr int BK = 32, NSTAGE = STAGES;     // k per stage, LDS stages
  static constexpr int MB = MB_, KS = 512 / MB_;     // MFMA block edge, k per MFMA
  static constexpr int ACC_N = MB * MB / 64;         // accumulator floats per lane per block
  static constexpr int QUADS = ACC_N / 4;            // 16-byte groups of them
  static constexpr int A_ROW = BK * 2;              // bytes per row of the A stage
  static constexpr int A_ROW_CHUNKS = BK / 8;
  static constexpr int A_RPL = 1024 / A_ROW;         // A rows one wave-load (64 x 16 B) covers
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;  // wave tile
  static constexpr int MI = WM / MB, NI = WN / MB;            // MFMA blocks per wave
  static constexpr int A_LOADS = BM * (BK / 8) / THREADS;     // 16-byte loads per thread per stage
  static constexpr int B_LOADS = BK * (BN / 8) / THREADS;
  static constexpr int A_STAGE = BM * BK * 2;       // bytes
  static constexpr int B_STAGE = BK * BN * 2;
  static constexpr int B_ROW = BN * 2;              // bytes per k row of the B stage
  static constexpr int B_ROW_CHUNKS = BN / 8;
  static constexpr int STAGE = A_STAGE + B_STAGE;
  static constexpr int LDS = NSTAGE * STAGE;
  // LDS placement: the four B stages first, then the four A stages, so that
  // every fragment read of a stage known at compile time is a per-lane base
  // plus an offset that fits the 16-bit offset field of ds_read (the A base
  // carries the B region's size)
  static constexpr int B_REGION = NSTAGE * B_STAGE;
  static constexpr int a_off(int s) { return B_REGION + s * A_STAGE; }
  static constexpr int b_off(int s) { return s * B_STAGE; }
  static_assert(A_LOADS * THREADS == BM * (BK / 8) && B_LOADS * THREADS == BK * (BN / 8), "load split");
  static_assert(WM % MB == 0 && WN % MB == 0 && (MB == 16 || MB == 32), "wave tile");
};

// The wave grid used for each tile edge: 128 -> 2 x 2 waves of 64 x 64 in
// 32 x 32 blocks (two workgroups per CU, so two waves share each SIMD); 256 ->
// 2 x 2 waves of 128 x 128 in 16 x 16 blocks (one wave per SIMD, 256
// accumulator registers each). The large wave tile reads two thirds of the LDS
// bytes per flop that 128 x 64 wave tiles need, and the part is power-bound,
// so fewer LDS bytes buy clock.
template <int EDGE> struct TileCfg;
template <> struct TileCfg<128> { using type = Cfg<128, 128, 2, 2, 32>; };
template <> struct TileCfg<256> { using type = Cfg<256, 256, 2, 2, 16>; };

// A: the slot XOR for row r depends on the fragment read pattern. Measured with
// the LDS bank-conflict counter on gfx950 (ds_read_b128, 64 B rows): for 32 x 32
// blocks (32 rows x one chunk per half-wave) (r >> 2) & 3 is conflict-free and
// (r >> 1) & 3 is two-way; for 16 x 16 blocks (16 rows x four chunks) it is the
// other way round, and no XOR at all is two-way.
template <int MB>
__device__ __forceinline__ uint32_t swz_a(uint32_t row) { return MB == 32 ? (row >> 2) & 3u : (row >> 1) & 3u; }
__device__ __forceinline__ uint32_t swz_b(uint32_t k) {
  return (10u * (k & 1u) + 4u * ((k >> 1) & 1u)) ^ (2u * ((k >> 3) & 1u));
}

// Eight e4m3 values as bf16: 8 significant bits hold every one of them exactly.
__device__ __forceinline__ uint32_t bf16_pair(uint32_t four, bool high) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const bf16x2 v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)four, 1.0f, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)four, 1.0f, false);
  return __builtin_bit_cast(uint32_t, v);
}

// One record of the claim ring: the answer to one claim. `valid` is the success
// predicate; `tile` is meaningful only when valid. `seq` is the worker's tile
// ordinal the record answers (checked by the consumers).
struct RingRec {
  uint32_t tile, valid, seq, pad;
};

static constexpr int kRingDepth = 3;  // LDS slots; a run uses args.ring_depth (2 or 3) of them

// Record a device-side failure: in this run's control block (bit set of the
// run) and in the plan's status word, which only the host clears, so a failure
// of any run stays visible until the host has read it.
__device__ __forceinline__ void flag_error(const KernelArgs &a, uint32_t bit) {
  __hip_atomic_fetch_or(&a.ctrl->error, bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_fetch_or(a.status, bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Rotation of a unit's K order: the physical k-step its logical step kb + i
// reads is kb + ((i + rot) mod nsteps) (see the K order at the item set-up).
// `item` is the key the phase follows: the item id, or a grouped run's problem.
__device__ __forceinline__ int32_t k_rotation_of(const KernelArgs &a, uint32_t item, int32_t nsteps) {
  if (a.k_rotation == 0 || nsteps <= 1) return 0;
  uint32_t rot;
  if (a.k_rotation == 1 || a.k_rotation == 2) {
    // one phase per XCD region (item id mod 8; a plain launch sends item i to
    // XCD i mod 8): the workgroups of one XCD, which share operand panels
    // through its L2, keep walking K together. Or two phases per region (item
    // id mod 16), half the range apart.
    const uint32_t phases = a.k_rotation == 1 ? (uint32_t)kXcdRegions : 2u * kXcdRegions;
    rot = (item % phases) * (uint32_t)nsteps / phases;
  } else {
    // a phase per unit (multiplicative hash of the item id)
    rot = ((item * 2654435761u) >> 16) % (uint32_t)nsteps;
  }
  return (int32_t)wave_uniform(rot);
}

// Thread 0 of every workgroup, once, after its last use of the run's scheduler
// state, in runs that clean up after themselves (self_clean: launches captured
// into a graph, which replay on one state set): count the workgroup out; the
// last one of the grid resets the claim counters, the gate and the count
// itself, so the next replay starts from zero without a host-side reset. Other
// runs skip it: the plan's next run clears their set before it is used again
// (the count's two dependent atomics at the end of a launch cost 2-4 us).
// The count has two levels: a workgroup counts into its group (blockIdx mod
// kExitGroups, one cache line per group), and the workgroup that completes a
// group counts the group into exit_count; the one that completes the last
// group resets everything. (With one counter, the late launch slots of a
// dynamic run, thousands for small tiles, all hit one address at the end:
// 8192^3 with 128 x 128 tiles lost ~125 us to it.)
// Relaxed order is enough: a workgroup's claims are returning atomics whose
// answers it has waited for, so they are performed before its count goes out;
// the resetting workgroup resets only after its own counts have come back; and
// the next launch that reads this state starts after this kernel has ended,
// which orders everything before it. (An acquire-release count writes back and
// invalidates the XCD's whole L2 in every exiting workgroup, which the workers
// still running on that XCD then pay for: 8192^3 static 750 -> 741 us and
// dynamic 773 -> 755 us without it.)
__device__ __forceinline__ void leave_run(const KernelArgs &a) {
  const uint32_t g = blockIdx.x % (uint32_t)kExitGroups;
  const uint32_t in_group = (gridDim.x - g + (uint32_t)kExitGroups - 1u) / (uint32_t)kExitGroups;
  const uint32_t groups = min(gridDim.x, (uint32_t)kExitGroups);
  const uint32_t done =
      __hip_atomic_fetch_add(&a.ctrl->exit_group[g * kExitStride], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (done + 1u != in_group) return;
  const uint32_t groups_done = __hip_atomic_fetch_add(&a.ctrl->exit_count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (groups_done + 1u == groups) {
    __hip_atomic_store(&a.ctrl->counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&a.ctrl->gate, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&a.ctrl->error, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int x = 0; x < kXcdRegions; ++x)
      __hip_atomic_store(&a.ctrl->xcd_counter[(x) * kXcdStride], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int x = 0; x < kExitGroups; ++x)
      __hip_atomic_store(&a.ctrl->exit_group[x * kExitStride], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&a.ctrl->exit_count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// Ask the scheduler for an alternation of one MFMA and one LDS read in the
// current scheduling region (then the remaining MFMAs or reads).
template <int READS, int MFMAS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < MFMAS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                 // MFMA
    if (i < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
  }
  if constexpr (READS > MFMAS) __builtin_amdgcn_sched_group_barrier(0x100, READS - MFMAS, 0);
}

// One claim. Single-counter policy: the next value of the device-wide counter
// (plus the failure-forcing base); any value >= T is a failure. XCD-partitioned
// policies: region x (tiles 8i + x, or the x-th of eight consecutive runs of
// ids; see region_unit) is handed out by counter x; a worker claims
// from its own XCD's region first (the tiles its XCD's L2 already holds
// operands for) and, once that is exhausted, steals from another region. Each
// counter returns each index once, so every tile still has exactly one owner;
// the claim fails (returns T) only when every region is exhausted.
//
// A claim is split in two. claim_issue sends the first atomic (the global
// counter, or the counter of the worker's current region: its own XCD's to
// begin with) from lane 0 and returns its raw answer in lane 0's register,
// valid once the wave's memory operations have drained (vmcnt 0); the round
// trip hides under the MFMAs of the current tile. claim_resolve, called by a whole wave (all lanes active) once
// the answer is needed, broadcasts it and turns it into a tile id: every
// decision is wave-uniform and the scheduler state lives in scalar registers.
// Only when the current region is exhausted does it steal: it reads all eight
// counters at once (lanes 0-7), picks the first region after the worker's own
// that still has work, claims from it and makes it the current region, so the
// following claims are again a single hidden atomic. A claim that comes back
// out of range proves that region exhausted for good (counters only grow), so
// at most eight steal attempts are made.
// The claim atomic as one assembly statement that skips itself unless `now`
// (wave-uniform) is set: lane 0 alone adds 1 to *ctr (exec is narrowed inside
// the statement) and receives the old value in `ret`. The compiler does not see
// the atomic, so it never waits for it on its own (a claim the compiler could
// see, on any path into the main loop, made it drain every load at the loop
// head): readers of `ret` wait (vmcnt) explicitly. The 16 x 16 main loop sends
// its claims from this statement between two runs of the same loop body, so
// no k-step carries the claim's branch or EXEC write (either one inside the
// step cost 70-90 cycles per step, measured: it holds the wave until the MFMAs
// in flight drain) and no branch splits a step (the register allocator then
// copies accumulators around the split).
__device__ __forceinline__ void claim_issue_asm(uint32_t *ctr, bool now, uint32_t &ret) {
  uint64_t saved;
  asm volatile(
      "s_cmp_eq_u32 %[now], 0\n\t"
      "s_cbranch_scc1 1f\n\t"
      "s_mov_b64 %[saved], exec\n\t"
      "s_mov_b64 exec, 1\n\t"
      "global_atomic_add %[ret], %[off], %[one], %[ctr] sc0\n\t"
      "s_mov_b64 exec, %[saved]\n"
      "1:"
      : [ret] "+v"(ret), [saved] "=&s"(saved)
      : [now] "s"(__builtin_amdgcn_readfirstlane(now ? 1u : 0u)), [off] "v"(0u), [one] "v"(1u), [ctr] "s"(ctr)
      : "memory", "scc");
}
__device__ __forceinline__ uint32_t lane0_fetch_add(uint32_t *ctr, uint32_t lane) {
  uint32_t v = 0;
  if (lane == 0) v = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ uint32_t region_size(uint32_t T, uint32_t y) {
  return T > y ? (T - y + kXcdRegions - 1) / kXcdRegions : 0u;
}
// Id of the i-th unit of region y: interleaved regions (policy 1) hold the ids
// 8i + y; contiguous regions (policy 2) hold the y-th of eight consecutive runs
// of ids, of the same sizes (the first T mod 8 runs one longer).
__device__ __forceinline__ uint32_t region_unit(int policy, uint32_t T, uint32_t y, uint32_t i) {
  if (policy == 1) return i * (uint32_t)kXcdRegions + y;
  const uint32_t q = T / (uint32_t)kXcdRegions, r = T % (uint32_t)kXcdRegions;
  return y * q + (y < r ? y : r) + i;
}
__device__ __forceinline__ uint32_t claim_issue(const KernelArgs &a, uint32_t region) {
  uint32_t *ctr = a.claim_policy == 0 ? &a.ctrl->counter : &a.ctrl->xcd_counter[(region) * kXcdStride];
  uint32_t v = 0;
  claim_issue_asm(ctr, true, v);
  return v;
}
__device__ __forceinline__ uint32_t claim_resolve(const KernelArgs &a, uint32_t xcc, uint32_t lane, uint32_t raw,
                                                  uint32_t &region) {
  const uint32_t i0 = __builtin_amdgcn_readfirstlane(raw);
  if (a.claim_policy == 0) return i0 + a.counter_base;
  const uint32_t T = (uint32_t)a.T;
  if (i0 < region_size(T, region)) return region_unit(a.claim_policy, T, region, i0);
  // lane r < 8 watches region (xcc + r) mod 8
  const uint32_t my_y = (xcc + (lane & 7u)) % (uint32_t)kXcdRegions;
  for (int attempt = 0; attempt < kXcdRegions; ++attempt) {
    bool open = false;
    if (lane < (uint32_t)kXcdRegions) {
      const uint32_t seen = __hip_atomic_load(&a.ctrl->xcd_counter[(my_y) * kXcdStride], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      open = seen < region_size(T, my_y);
    }
    const uint64_t mask = __ballot(open);
    if (mask == 0) return T;
    const uint32_t r = (uint32_t)__builtin_ctzll(mask);
    const uint32_t y = (xcc + r) % (uint32_t)kXcdRegions;
    const uint32_t i = lane0_fetch_add(&a.ctrl->xcd_counter[(y) * kXcdStride], lane);
    if (i < region_size(T, y)) {
      region = y;
      return region_unit(a.claim_policy, T, y, i);
    }
  }
  return T;
}

__device__ __forceinline__ uint32_t claim_next(const KernelArgs &a, uint32_t xcc, uint32_t lane, uint32_t &region) {
  const uint32_t raw = claim_issue(a, region);
  wait_vmem_all();
  return claim_resolve(a, xcc, lane, raw, region);
}

// The plain product: fp32 C, row strides as long as the rows. BT: B is given as
// N x K row-major (C = A . B^T); its stage then holds BN rows x 32 k like A's, and
// its fragments are read like A's.
template <bool BT_>
struct PlainOp {
  struct Args {};
  static constexpr bool AT = false, BT = BT_, E8 = false, kPlain = true, kWide = false;
  template <int EDGE> using Tile = typename TileCfg<EDGE>::type;
  static __device__ __forceinline__ int32_t lda(const KernelProblem &pb, const Args &) { return pb.K; }
  static __device__ __forceinline__ int32_t ldb(const KernelProblem &pb, const Args &) { return BT_ ? pb.K : pb.N; }
};

template <int BM, int BN, int MODE, bool GROUPED, class OP>
__device__ __forceinline__ void gemm_body(const KernelArgs &args, const typename OP::Args &op) {
  using CF = typename OP::template Tile<BM>;
  constexpr bool AT = OP::AT, BT = OP::BT, E8 = OP::E8;
  // K-contiguous operands staged two k-steps (128 bytes of a row) at a time
  constexpr bool WA = OP::kWide && !AT, WB = OP::kWide && BT, WIDE = WA || WB;
  static_assert(!WIDE || CF::MB == 16, "wide stages are read in 16 x 16 blocks");
  static_assert(!E8 || (!AT && BT && CF::MB == 16), "e4m3 operands are both K-contiguous, in 16 x 16 blocks");
  static_assert(CF::BM_ == BM && CF::BN_ == BN, "config");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[CF::LDS];  // the stage ring
  __shared__ RingRec ring[kRingDepth];
  __shared__ uint32_t gate_ok;
  __shared__ uint32_t split_last;  // this workgroup finished the last K-chunk of a split tile

  const uint32_t tid = threadIdx.x;
  const uint32_t lane = tid & 63u;
  const uint32_t wave = wave_uniform(tid >> 6);
  const uint32_t wm = wave / (uint32_t)CF::WAVES_N_, wn = wave % (uint32_t)CF::WAVES_N_;
  const int32_t T = args.T;

  // ---- clear the next run's scheduler state (spread over the grid)
  if (blockIdx.x == 0 && tid == 0 && args.ctrl_next != nullptr) {
    args.ctrl_next->counter = 0u;
    args.ctrl_next->gate = 0u;
    args.ctrl_next->error = 0u;
    args.ctrl_next->exit_count = 0u;
    for (int x = 0; x < kXcdRegions; ++x) args.ctrl_next->xcd_counter[(x) * kXcdStride] = 0u;
    for (int x = 0; x < kExitGroups; ++x) args.ctrl_next->exit_group[x * kExitStride] = 0u;
  }
  if (args.clear_count > 0) {
    const uint32_t chunk = ((uint32_t)args.clear_count + gridDim.x - 1u) / gridDim.x;
    const uint32_t first = blockIdx.x * chunk;
    for (uint32_t i = tid; i < chunk; i += (uint32_t)CF::THREADS) {
      if (first + i < (uint32_t)args.clear_count) args.clear_next[first + i] = 0u;
    }
  }

  // ---- optional concurrency gate: at most max_concurrent workgroups compute at once
  if (args.max_concurrent > 0) {
    if (tid == 0) {
      // a bounded wait: at most gate_spin_limit polls (the host may preset
      // gate_base slots as taken, so that every wait runs out: failure forcing)
      uint32_t ok = 0;
      for (uint32_t it = 0; it < args.gate_spin_limit; ++it) {
        uint32_t cur = __hip_atomic_load(&args.ctrl->gate, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (cur + args.gate_base < (uint32_t)args.max_concurrent &&
            __hip_atomic_compare_exchange_strong(&args.ctrl->gate, &cur, cur + 1u, __ATOMIC_ACQUIRE,
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) {
          ok = 1;
          break;
        }
        __builtin_amdgcn_s_sleep(4);
      }
      // a workgroup that gives up computes nothing: its units are lost in the
      // static and non-persistent modes, so the failure is recorded for the host
      if (!ok) flag_error(args, 1u);
      gate_ok = ok;
    }
    __syncthreads();
    if (!gate_ok) {
      if (tid == 0 && args.self_clean) leave_run(args);
      return;
    }
  }

  // scalar reads, kept per wave (only wave 0's values are logged and used to claim)
  const uint32_t hwid = read_hw_id();
  const uint32_t xcc = read_xcc_id() % (uint32_t)kXcdRegions;

  // ---- first work unit (a whole tile, or one K-chunk of a split tile)
  uint32_t ord = 0;       // this worker's unit ordinal
  uint32_t unit = 0;
  bool valid = false;
  // producer state (wave 0, the elected producer, holds the meaningful copy)
  uint32_t next_ord = 1;  // next ordinal to claim
  bool failed = false;    // a claim has come back invalid
  uint32_t region = xcc;  // region the next claim is sent to (XCD-partitioned policy)
  if constexpr (MODE == kDynamic) {
    if (wave == 0) {
      // plain-load pre-check: a slot that starts after every tile was handed
      // out (counters only grow) exits without sending an atomic. Without it,
      // the thousands of late slots of a run with many small tiles sent their
      // atomics to the same counters as the last workers' final claims, whose
      // answers then came back many microseconds late (8192^3 with 128 x 128
      // tiles: 845 -> 955 TFLOP/s). The slots of the first wave (the ones
      // resident at launch) skip it: they start before any claim has gone out,
      // so the counters are open, and the load would only delay their first
      // claim by a round trip. (A first-wave slot that starts late claims
      // anyway, as every slot did before the pre-check.)
      bool open = false;
      if (blockIdx.x < (uint32_t)args.first_wave) {
        open = lane == 0;
      } else if (args.claim_policy != 0) {
        if (lane < (uint32_t)kXcdRegions)
          open = __hip_atomic_load(&args.ctrl->xcd_counter[(lane) * kXcdStride], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <
                 region_size((uint32_t)T, lane);
      } else if (lane == 0) {
        open = __hip_atomic_load(&args.ctrl->counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + args.counter_base <
               (uint32_t)T;
      }
      const uint32_t v = __ballot(open) != 0 ? claim_next(args, xcc, lane, region) : (uint32_t)T;
      const uint32_t ok = v < (uint32_t)T ? 1u : 0u;
      if (lane == 0) ring[0] = RingRec{v, ok, 0u, 0u};
      failed = !ok;
    }
    __syncthreads();
    unit = wave_uniform(ring[0].tile);
    valid = wave_uniform(ring[0].valid) != 0;
  } else {
    unit = blockIdx.x;
    valid = unit < (uint32_t)T;
  }

  uint32_t sub = 0;  // the current item's place in its unit (claim groups)
  while (valid) {
    // ---- the work item: unit u covers items [u g, u g + g) (g = claim_group, 1
    // unless claim groups are on); items below split_base are whole tiles (id =
    // tile id), item split_base + q*S + c is K-chunk c of tile split_base + q
    const uint32_t group = (uint32_t)args.claim_group;
    const uint32_t item = unit * group + sub;
    const bool last_sub = sub + 1 >= min(group, (uint32_t)args.items - unit * group);
    uint32_t tile = item;
    uint32_t chunk = 0;
    const bool split = !GROUPED && (int32_t)item >= args.split_base;
    if (split) {
      const uint32_t j = item - (uint32_t)args.split_base;
      tile = (uint32_t)args.split_base + j / (uint32_t)args.split_chunks;
      chunk = j % (uint32_t)args.split_chunks;
    }
    KernelProblem pb;
    int32_t local = (int32_t)tile;
    // what the K-order phase is keyed by: the item (single GEMMs), or the
    // problem (grouped runs: its tiles share its operand panels, so they walk
    // K in step, while different problems take different phases)
    uint32_t rot_key = item;
    if constexpr (GROUPED) {
      const int32_t prob = find_problem(args.groups, args.G, (int32_t)tile);
      rot_key = (uint32_t)prob;
      pb = args.groups[prob];
      // the descriptor is the same for the whole workgroup: keep it in SGPRs
      pb.A = uniform_ptr(pb.A);
      pb.B = uniform_ptr(pb.B);
      pb.C = uniform_ptr(pb.C);
      pb.M = (int32_t)wave_uniform((uint32_t)pb.M);
      pb.N = (int32_t)wave_uniform((uint32_t)pb.N);
      pb.K = (int32_t)wave_uniform((uint32_t)pb.K);
      pb.tiles_m = (int32_t)wave_uniform((uint32_t)pb.tiles_m);
      pb.tiles_n = (int32_t)wave_uniform((uint32_t)pb.tiles_n);
      pb.tile_start = (int32_t)wave_uniform((uint32_t)pb.tile_start);
      pb.unit_start = (int32_t)wave_uniform((uint32_t)pb.unit_start);
      local -= pb.unit_start;
      tile = (uint32_t)(pb.tile_start + local);  // the tile id in call-order numbering
    } else {
      pb = args.single;
    }
    int32_t m_t, n_t;
    decode_tile(local, pb.tiles_m, pb.tiles_n, args.raster_group, m_t, n_t);
    const int32_t m0 = m_t * BM, n0 = n_t * BN;
    const int32_t M = pb.M, N = pb.N, K = pb.K;

    const uint64_t t0 = clock_core();
    const uint64_t r0 = clock_wall();

    // ---- claim ahead (the throttle: at most claims_ahead beyond the current tile)
    uint32_t batch[2] = {0u, 0u};  // raw answers of the claims issued during this tile (lane 0)
    uint32_t batch_ord = 0, batch_n = 0;
    // reserve: the ordinals of the claims this unit sends (wave 0, scalar)
    auto reserve_claims = [&]() {
      if constexpr (MODE == kDynamic) {
        if (wave == 0 && !failed && args.claims_ahead >= 1) {
          batch_ord = next_ord;
          while (next_ord <= ord + (uint32_t)args.claims_ahead && batch_n < 2) {
            ++batch_n;
            ++next_ord;
          }
        }
      }
    };
    // reserve and send at once
    auto do_claims = [&]() {
      if constexpr (MODE == kDynamic) {
        reserve_claims();
        for (uint32_t b = 0; b < batch_n; ++b) {
          const uint32_t v = claim_issue(args, region);
          if (b == 0) batch[0] = v; else batch[1] = v;
        }
      }
    };

    // ---- per-thread load addressing for this tile. Load j of a wave moves a
    // 1 KiB block: A rows (j*NW+wave)*A_RPL .. +A_RPL (A_ROW_CHUNKS lanes per row),
    // B k rows (j*NW+wave)*kBRowsPerLoad .. (B_ROW_CHUNKS lanes per row). Each
    // lane fetches the global chunk whose swizzled slot is its own LDS position.
    // The A swizzle does not change between loads (they step by a multiple of 16
    // rows); the B swizzle flips its bit 1 when a load's k rows step by an odd
    // multiple of 8, so B has two per-lane bases. Each voffset is one of them
    // plus a wave-uniform step.
    constexpr uint32_t kBRowsPerLoad = 64u / CF::B_ROW_CHUNKS;  // k rows one wave-load covers
    constexpr uint32_t kBRowsPerJ = (uint32_t)CF::NW * kBRowsPerLoad;
    const uint32_t a_row0 = wave * (uint32_t)CF::A_RPL + lane / CF::A_ROW_CHUNKS;  // row of load j = a_row0 + RPL NW j
    const uint32_t a_c0 = (lane % CF::A_ROW_CHUNKS) ^ swz_a<CF::MB>(a_row0);
    const int32_t lda = OP::lda(pb, op), ldb = OP::ldb(pb, op);
    const uint32_t a_base = a_row0 * (uint32_t)lda * 2u;
    const uint32_t b_k0 = wave * kBRowsPerLoad + lane / CF::B_ROW_CHUNKS;  // k row of load j = b_k0 + kBRowsPerJ j
    const uint32_t b_c0 = (lane % CF::B_ROW_CHUNKS) ^ swz_b(b_k0);
    const uint32_t b_c1 = b_c0 ^ 2u;  // the chunk when k row bit 3 is flipped
    const uint32_t b_base0 = n0 + (int32_t)(b_c0 * 8u) < N ? (b_k0 * (uint32_t)ldb + b_c0 * 8u) * 2u : kBufOob;
    const uint32_t b_base1 = n0 + (int32_t)(b_c1 * 8u) < N ? (b_k0 * (uint32_t)ldb + b_c1 * 8u) * 2u : kBufOob;
    const int32_t m_left = M - m0;  // rows of A that exist in this tile
    const int32_t n_left = N - n0;  // rows of B^T that exist in this tile (BT)
    // AT: A's k rows like B's (BM == BN, so the same split of the loads)
    const uint32_t at_base0 = m0 + (int32_t)(b_c0 * 8u) < M ? (b_k0 * (uint32_t)lda + b_c0 * 8u) * 2u : kBufOob;
    const uint32_t at_base1 = m0 + (int32_t)(b_c1 * 8u) < M ? (b_k0 * (uint32_t)lda + b_c1 * 8u) * 2u : kBufOob;
    const uint16_t *a_tile = AT ? pb.A + m0 : pb.A + (size_t)m0 * (size_t)lda;
    if constexpr (!OP::kPlain) a_tile = uniform_ptr(a_tile);
    // the k-step enters through the resource base: + kt BK elements along a row
    // of A (and of B^T), + kt BK rows of B
    const uint16_t *b_tile = BT ? pb.B + (size_t)n0 * (size_t)ldb : pb.B + n0;
    if constexpr (!OP::kPlain) b_tile = uniform_ptr(b_tile);
    auto a_kstep = [&](int32_t kt) -> const uint16_t * {
      return AT ? a_tile + (size_t)(kt * CF::BK) * (size_t)lda : a_tile + kt * CF::BK;
    };
    auto b_kstep = [&](int32_t kt) -> const uint16_t * {
      return BT ? b_tile + kt * CF::BK : b_tile + (size_t)(kt * CF::BK) * (size_t)ldb;
    };
    const int32_t nk = (K + CF::BK - 1) / CF::BK;
    const int32_t full = K / CF::BK;  // k-steps with no K tail
    // k-steps [kb, ke) of this unit: all of them, or an even share for a K-chunk
    // (wide stages: an even k-step begins every range)
    const uint32_t nr = WIDE ? (uint32_t)(nk + 1) / 2u : (uint32_t)nk;
    const int32_t kb = split ? (int32_t)(nr * chunk / (uint32_t)args.split_chunks) * (WIDE ? 2 : 1) : 0;
    const int32_t ke = split ? min(nk, (int32_t)(nr * (chunk + 1u) / (uint32_t)args.split_chunks) * (WIDE ? 2 : 1)) : nk;
    // K order of the unit: logical k-step kt (kb <= kt < ke) reads physical k-step
    // kb + ((kt - kb + rot) mod (ke - kb)). When every workgroup walks K from the
    // same end, all concurrent operand reads of the machine share their low
    // address bits (the same 64-byte column of every row of A): measured on a
    // streaming probe of that pattern, 4.5 TB/s against 5.9 TB/s when each CU
    // starts at a different column. A rotation spreads them. It changes only the
    // order of the fp32 sum inside a tile (a function of the unit id alone, so
    // every scheduler still gives bitwise the same C). Off when K has a partial
    // k-step (the K-tail masking assumes that step comes last).
    const int32_t nsteps = ke - kb;
    // Wide stages rotate their whole pairs of k-steps; a pair that K ends in keeps
    // its place at the end.
    const int32_t npf = WIDE ? (min(ke, K / (2 * CF::BK) * 2) - kb) / 2 : 0;  // whole pairs
    const int32_t rot = WIDE ? (npf > 1 ? k_rotation_of(args, rot_key, npf) : 0)
                             : K % CF::BK == 0 ? k_rotation_of(args, rot_key, nsteps) : 0;
    // physical k-step of logical k-step kt (logical steps past ke read zeros
    // through a dead resource, whatever their base)
    auto phys = [&](int32_t kt) -> int32_t {
      if constexpr (WIDE) {
        // (selects, not branches: a branch holds the wave until its MFMAs drain)
        const int32_t i = kt - kb, p = i >> 1, t = p + rot, w = t - npf;
        const int32_t q = w >= 0 ? w : t, f = p < npf ? q : p;
        return kb + 2 * f + (i & 1);
      }
      return kt + rot >= ke ? kt + rot - nsteps : kt + rot;
    };

    // voffset of load j of a k-step with no partial K: chunks outside the matrix
    // (row / column edges) read as zero via kBufOob. The A swizzle of load j's
    // row differs from a_row0's by a compile-time XOR; B has two per-lane bases.
    auto load_chunk_a = [&](int j) -> uint32_t {
      return a_c0 ^ (swz_a<CF::MB>((uint32_t)(CF::A_RPL * CF::NW * j)) ^ swz_a<CF::MB>(0u));
    };
    auto load_voff_edge = [&](int j) -> uint32_t {
      if (AT && j < CF::A_LOADS) {
        const uint32_t ab = ((kBRowsPerJ * (uint32_t)j) & 8u) ? at_base1 : at_base0;
        return ab == kBufOob ? kBufOob : ab + (uint32_t)j * kBRowsPerJ * (uint32_t)lda * 2u;
      }
      if (j < CF::A_LOADS) {
        const uint32_t row = a_row0 + (uint32_t)(CF::A_RPL * CF::NW) * (uint32_t)j;
        const uint32_t vo = a_base + load_chunk_a(j) * 16u + (uint32_t)(CF::A_RPL * CF::NW * j) * (uint32_t)lda * 2u;
        return (int32_t)row >= m_left ? kBufOob : vo;
      }
      const int jb = j - CF::A_LOADS;
      if constexpr (BT) {
        // B^T rows like A rows (same row step per load, same swizzle)
        const uint32_t row = a_row0 + (uint32_t)(CF::A_RPL * CF::NW) * (uint32_t)jb;
        const uint32_t vo = a_row0 * (uint32_t)ldb * 2u + load_chunk_a(jb) * 16u +
                            (uint32_t)(CF::A_RPL * CF::NW * jb) * (uint32_t)ldb * 2u;
        return (int32_t)row >= n_left ? kBufOob : vo;
      }
      const uint32_t bb = ((kBRowsPerJ * (uint32_t)jb) & 8u) ? b_base1 : b_base0;
      return bb == kBufOob ? kBufOob : bb + (uint32_t)jb * kBRowsPerJ * (uint32_t)ldb * 2u;
    };
    // voffset of load j (A loads first, then B) for k-step kt: the same, and in
    // the partial k-step (K tail) chunks past K read as zero too. Every chunk of
    // a k-step past the unit's end reads as zero through its resource (record
    // count 0). The edge offsets do not depend on kt, so the 16 x 16 main loop
    // computes them once per tile and uses them in every trip with no partial
    // K: recomputing the masks every k-step cost about 220 cycles per step in
    // vector instructions interleaved with the MFMAs (measured: 406k -> 350k
    // cycles per 8192^3 tile).
    auto load_voff = [&](int j, int32_t kt) -> uint32_t {
      const uint32_t vo = load_voff_edge(j);
      if (kt < full) return vo;
      const int32_t k0 = kt * CF::BK;
      const int32_t kfirst = j < CF::A_LOADS ? (AT ? k0 + (int32_t)(b_k0 + kBRowsPerJ * (uint32_t)j)
                                                   : k0 + (int32_t)(load_chunk_a(j) * 8u))
                             : BT ? k0 + (int32_t)(load_chunk_a(j - CF::A_LOADS) * 8u)
                                  : k0 + (int32_t)(b_k0 + kBRowsPerJ * (uint32_t)(j - CF::A_LOADS));
      return kfirst >= K ? kBufOob : vo;
    };
    // LDS byte offset (from smem) of load j's 1 KiB block in stage st
    auto load_dst = [&](int j, int st) -> uint32_t {
      return j < CF::A_LOADS ? (uint32_t)CF::a_off(st) + (uint32_t)(j * CF::NW + (int)wave) * 1024u
                             : (uint32_t)CF::b_off(st) + (uint32_t)((j - CF::A_LOADS) * CF::NW + (int)wave) * 1024u;
    };
    // Wide loads: a wave-load moves eight rows of 128 bytes (whole cache lines, where
    // a k-step alone takes 64 bytes of 16 rows: from L2, 256 CUs at once, 103 ->
    // 133 GB/s a CU, and with rows that do not start on 64-byte lines 46 -> 99).
    // Chunk c of row r of a pair's 128-byte rows sits in slot c ^ ((r >> 1) & 7).
    // Of a pair's loads the first 2 A_LOADS are A's, the rest B's; rows step by 32 a
    // load, so a lane's chunk is the same for all.
    constexpr int kWideA = WA ? 2 * CF::A_LOADS : 0, kWideB = WB ? 2 * CF::B_LOADS : 0, kWide = kWideA + kWideB;
    // Rows past the matrix are out of the resource's range (its record count is the
    // bytes of the rows there are), so an offset is one per-lane base plus a
    // wave-uniform step; in the pair that K ends in, the bases of chunks past K are
    // out of range themselves.
    const uint32_t w_row0 = wave * 8u + (lane >> 3);
    const uint32_t w_chunk = (lane & 7u) ^ ((w_row0 >> 1) & 7u);
    const uint32_t w_base_a = w_row0 * (uint32_t)lda * 2u + w_chunk * 16u, w_base_b = w_row0 * (uint32_t)ldb * 2u + w_chunk * 16u;
    const uint32_t w_records_a = (uint32_t)min(m_left, BM) * (uint32_t)lda * 2u, w_records_b = (uint32_t)min(n_left, BN) * (uint32_t)ldb * 2u;
    auto wide_rsrc = [&](bool a, int32_t kt) -> i32x4 {  // of the pair that logical k-step kt begins
      i32x4 r = make_rsrc_words(a ? a_kstep(phys(kt)) : b_kstep(phys(kt)));
      r[2] = kt < ke ? (int32_t)(a ? w_records_a : w_records_b) : 0;
      return r;
    };
    auto wide_voff = [&](int j) -> uint32_t {
      return j < kWideA ? w_base_a + (uint32_t)(8 * CF::NW * j) * (uint32_t)lda * 2u
                        : w_base_b + (uint32_t)(8 * CF::NW * (j - kWideA)) * (uint32_t)ldb * 2u;
    };
    auto wide_voff_tail = [&](int j, int32_t pair_kt) -> uint32_t {
      return pair_kt * CF::BK + (int32_t)(w_chunk * 8u) >= K ? kBufOob : wide_voff(j);
    };
    auto wide_dst = [&](int j, int st) -> uint32_t {
      return j < kWideA ? (uint32_t)CF::a_off(st & ~1) + (uint32_t)(j * CF::NW + (int)wave) * 1024u
                        : (uint32_t)CF::b_off(st & ~1) + (uint32_t)((j - kWideA) * CF::NW + (int)wave) * 1024u;
    };
    // all loads of k-step kt into stage dst, back to back (prologue)
    auto issue_all = [&](int st, int32_t kt) {
      const i32x4 ra = make_rsrc_words(a_kstep(phys(kt)), kt < ke);
      const i32x4 rb = make_rsrc_words(b_kstep(phys(kt)), kt < ke);
      const uint32_t base = lds_addr(smem);
#pragma unroll
      for (int j = 0; j < CF::A_LOADS + CF::B_LOADS; ++j)
        if (!(j < CF::A_LOADS ? WA : WB)) load16_to_lds(j < CF::A_LOADS ? ra : rb, base + load_dst(j, st), load_voff(j, kt));
    };
    // the wide loads of the pair that begins at kt
    auto issue_pair = [&](int st, int32_t kt) {
      const i32x4 ra = wide_rsrc(true, kt), rb = wide_rsrc(false, kt);
      const uint32_t base = lds_addr(smem);
#pragma unroll
      for (int j = 0; j < kWide; ++j) load16_to_lds(j < kWideA ? ra : rb, base + wide_dst(j, st), wide_voff_tail(j, phys(kt)));
    };

    // fragment read offsets (bytes inside a stage). An MFMA operand is 8
    // consecutive k per lane: lanes l and l + MB hold the next 8 k of the same
    // row (A) or column (B).
    uint32_t off_a[CF::MI];
    uint32_t swa[CF::MI];
#pragma unroll
    for (int mi = 0; mi < CF::MI; ++mi) {
      const uint32_t row = wm * CF::WM + mi * CF::MB + (lane % CF::MB);
      off_a[mi] = row * (uint32_t)CF::A_ROW * (WA ? 2u : 1u);
      swa[mi] = (WA ? (row >> 1) & 7u : swz_a<CF::MB>(row)) ^ (lane / CF::MB);
    }
    if constexpr (AT) {  // A read like B below: transposing reads of its k rows
      const uint32_t q = lane >> 4, i = lane & 15u;
      const uint32_t kk = CF::MB == 32 ? 8u * (q >> 1) + (i >> 2) : 8u * q + (i >> 2);
#pragma unroll
      for (int mi = 0; mi < CF::MI; ++mi) {
        const uint32_t m = CF::MB == 32 ? wm * CF::WM + mi * 32 + 16u * (q & 1u) + 4u * (i & 3u)
                                        : wm * CF::WM + mi * 16 + 4u * (i & 3u);
        off_a[mi] = kk * CF::B_ROW + (((m >> 3) ^ swz_b(kk)) << 4) + ((m & 7u) << 1);
      }
    }
    uint32_t off_b[CF::NI];
    uint32_t swb[CF::NI];  // BT: the chunk XOR of each block's row, as swa
    if constexpr (BT) {
      // a B^T fragment is read like an A fragment: 8 consecutive k of one row n
#pragma unroll
      for (int ni = 0; ni < CF::NI; ++ni) {
        const uint32_t row = wn * CF::WN + ni * CF::MB + (lane % CF::MB);
        off_b[ni] = row * (uint32_t)CF::A_ROW * (WB ? 2u : 1u);
        swb[ni] = (WB ? (row >> 1) & 7u : swz_a<CF::MB>(row)) ^ (lane / CF::MB);
      }
    } else {
      // 32 x 32 blocks: lane group q = lane / 16 covers k half q / 2 and column
      // half q % 2; 16 x 16 blocks: k quarter q of all 16 columns
      const uint32_t q = lane >> 4, i = lane & 15u;
      const uint32_t kk = CF::MB == 32 ? 8u * (q >> 1) + (i >> 2) : 8u * q + (i >> 2);
#pragma unroll
      for (int ni = 0; ni < CF::NI; ++ni) {
        const uint32_t n = CF::MB == 32 ? wn * CF::WN + ni * 32 + 16u * (q & 1u) + 4u * (i & 3u)
                                        : wn * CF::WN + ni * 16 + 4u * (i & 3u);
        off_b[ni] = kk * CF::B_ROW + (((n >> 3) ^ swz_b(kk)) << 4) + ((n & 7u) << 1);
      }
    }

    // A fragment: 8 consecutive k of one row (ds_read_b128). B fragment: two
    // transposing reads of 4 k each (ds_read_b64_tr_b16) for one column. s
    // selects the MFMA's k slice of the stage. Optionally (the 32 x 32 main
    // loop), the loads of k-step kt_load into stage lst are placed in program
    // order between the reads, load j after read j; the reads alternate with
    // MFMAs, so the loads land between MFMAs instead of in one burst. (The
    // 16 x 16 main loop places its reads and loads itself.)
    constexpr int kReadsA = (AT ? 2 : 1) * CF::MI;
    constexpr int kReads = kReadsA + (BT ? 1 : 2) * CF::NI;
    typedef bf16x8 frag;
    typedef __attribute__((ext_vector_type(8))) short i16x8;
    auto join = [](const i16x4 &l, const i16x4 &h) -> bf16x8 {
      const i16x8 v = __builtin_shufflevector(l, h, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(bf16x8, v);
    };
    auto read_frags = [&](int st, int s, frag(&af)[CF::MI], frag(&bfr)[CF::NI], int lst, int32_t kt_load,
                          int count, const uint32_t *voff_fast = nullptr, int j0 = 0) {
      const unsigned char *sa = smem + CF::a_off(st);
      const unsigned char *sb = smem + CF::b_off(st);
      i32x4 ra = {0, 0, 0, 0}, rb = {0, 0, 0, 0};
      const uint32_t lbase = lds_addr(smem);
      if (count > 0) {
        ra = make_rsrc_words(a_kstep(phys(kt_load)), kt_load < ke);
        rb = make_rsrc_words(b_kstep(phys(kt_load)), kt_load < ke);
      }
      i16x4 alo[CF::MI], lo[CF::NI];
#pragma unroll
      for (int r = 0; r < kReads; ++r) {
        if (r < kReadsA) {
          if constexpr (AT) {
            const unsigned char *pa0 = sa + off_a[r >> 1] + (CF::KS * s) * CF::B_ROW;
            if ((r & 1) == 0) {
              alo[r >> 1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pa0));
            } else {
              af[r >> 1] = join(alo[r >> 1], __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pa0 + 4 * CF::B_ROW)));
            }
          } else {
            af[r] = *(const bf16x8 *)(sa + off_a[r] + ((((uint32_t)((CF::KS / 8) * s)) ^ swa[r]) << 4));
          }
        } else if constexpr (BT) {
          const int ni = r - kReadsA;
          bfr[ni] = *(const bf16x8 *)(sb + off_b[ni] + ((((uint32_t)((CF::KS / 8) * s)) ^ swb[ni]) << 4));
        } else {
          const int ni = (r - kReadsA) >> 1;
          const unsigned char *pb0 = sb + off_b[ni] + (CF::KS * s) * CF::B_ROW;
          if (((r - kReadsA) & 1) == 0) {
            lo[ni] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pb0));
          } else {
            bfr[ni] = join(lo[ni], __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pb0 + 4 * CF::B_ROW)));
          }
        }
#pragma unroll
        for (int j = 0; j < count; ++j)
          if (j == r)
            load16_to_lds(j0 + j < CF::A_LOADS ? ra : rb, lbase + load_dst(j0 + j, lst),
                          voff_fast ? voff_fast[j0 + j] : load_voff(j0 + j, kt_load));
      }
    };

    typedef float accv __attribute__((ext_vector_type(CF::ACC_N)));
    accv acc[CF::MI][CF::NI];
#pragma unroll
    for (int mi = 0; mi < CF::MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < CF::NI; ++ni)
#pragma unroll
        for (int e = 0; e < CF::ACC_N; ++e) acc[mi][ni][e] = 0.0f;

    // the MFMAs of one 16-deep k slice, 32 x 32 blocks (the 16 x 16 main loop
    // issues its own)
    auto mma = [&](const frag(&af)[CF::MI], const frag(&bfr)[CF::NI]) {
      if constexpr (CF::MB == 32) {
#pragma unroll
        for (int mi = 0; mi < CF::MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < CF::NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bfr[ni], af[mi], acc[mi][ni], 0, 0, 0);
      }
    };

    // the prefetch claim is issued claim_lead k-steps before the tile ends (the
    // throttle): late enough not to take work a not-yet-started slot would get,
    // early enough for the atomic's round trip to hide under the MFMAs
    // claims for the next unit go out during the unit's last item only
    const int32_t claim_at = !last_sub ? -1 : ke - kb > args.claim_lead ? ke - args.claim_lead : kb;
    if (ke == kb && last_sub) do_claims();

    constexpr int kLoads = CF::A_LOADS + CF::B_LOADS;
    constexpr int kMfma = CF::MI * CF::NI;
    constexpr int NST = CF::NSTAGE, kMask = NST - 1;
    static_assert((NST & kMask) == 0 && NST >= 4, "stage ring");
    if constexpr (CF::MB == 32) {
      if (ke > kb) {
        // four 32-deep stages (or eight): the loads of k-step kt+3 (kt+7) go out
        // during k-step kt into the stage k-step kt-1 just left, so a load has two
        // and a half to three (six and a half to seven) k-steps to land;
        // each k-step is two 16-deep MFMA slices, and the fragments of one slice
        // are read while the other's MFMAs run
        static_assert(kLoads == 4, "stage ring");
#pragma unroll
        for (int q = 0; q < NST - 1; ++q) issue_all(q, kb + q);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * kLoads) : "memory");
        wg_barrier();
        frag a0[CF::MI], b0[CF::NI], a1[CF::MI], b1[CF::NI];
        read_frags(0, 0, a0, b0, 0, 0, 0);
        // load offsets of a k-step with no partial K, once per tile (as in the
        // 16 x 16 loop); steps whose loads reach the partial k-step `full` use
        // the K-tail test
        uint32_t voff_fast[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) voff_fast[j] = load_voff_edge(j);
        const int32_t slow_from = (K % CF::BK != 0 && full < ke) ? max(kb, full - (NST - 1)) : ke;
        auto step = [&](int32_t kt, bool fast) {
          const int st = (kt - kb) & kMask;
          // two of the four loads of k-step kt+3 go out with each slice's reads
          // (spread over the step: 4096^3 dynamic 175 -> 152 us against all four
          // with the first slice)
          read_frags(st, 1, a1, b1, (st + NST - 1) & kMask, kt + NST - 1, kLoads / 2, fast ? voff_fast : nullptr);
          mma(a0, b0);
          interleave<kReads, kMfma>();
          // stage st fully read and stage st+1 landed (its loads went out during
          // step kt-2, or kt-6; the loads issued since, six or 22, may still be in flight)
          wait_lds_all();
          asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 3) * kLoads + kLoads / 2) : "memory");
          wg_barrier();
          read_frags((st + 1) & kMask, 0, a0, b0, (st + NST - 1) & kMask, kt + NST - 1, kLoads / 2, fast ? voff_fast : nullptr, kLoads / 2);
          mma(a1, b1);
          interleave<kReads, kMfma>();
        };
        int32_t kt = kb;
        auto steps = [&](int32_t end) {
          for (const int32_t fe = min(end, slow_from); kt < fe; ++kt) step(kt, true);
          for (; kt < end; ++kt) step(kt, false);
        };
        // the claims go out between two runs of the loop (no branch for them in a step)
        if constexpr (MODE == kDynamic) {
          steps(claim_at >= kb ? claim_at : ke);
          if (claim_at >= kb) do_claims();
        }
        steps(ke);
      }
    } else {
      if (ke > kb) {
        // four 32-deep stages, one 32-deep MFMA per block and k-step: the
        // fragments of k-step kt+1 are read from its stage while step kt's MFMAs
        // run on the fragments read during step kt-1. The loads of step kt+4 go
        // out during step kt into the stage step kt's fragments came from (every
        // wave finished reading it before the barrier that ended step kt-1), and
        // must have landed by the barrier that ends step kt+2: between two and
        // three k-steps in flight.
        // loads of a k-step that are not wide, and of a pair of k-steps
        constexpr int kNarrow = (WA ? 0 : CF::A_LOADS) + (WB ? 0 : CF::B_LOADS), kPair = kWide + 2 * kNarrow;
#pragma unroll
        for (int q = 0; q < NST; ++q) {
          if constexpr (WIDE) {
            if ((q & 1) == 0) issue_pair(q, kb + q);
          }
          issue_all(q, kb + q);
        }
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST / 2 - 1) * kPair) : "memory");  // stages 0 and 1 landed
        wg_barrier();
        frag a0[CF::MI], b0[CF::NI], a1[CF::MI], b1[CF::NI];
        // e4m3: the k-step's fragments as they lie in LDS, 16 values a lane: lane
        // group g = lane / 16 holds chunk g of its row. The first eight values of
        // every chunk are one 32-deep MFMA's operand, the last eight the next
        // one's (the same k in A and B, whatever its order). a0, b0 hold the first
        // half as bf16, a1, b1 the second.
        i32x4 raw[CF::MI + CF::NI];
        // odd: the stage is the second of its pair (chunks 4 to 7 of the wide rows)
        auto read_raw = [&](int st, bool odd, int q) {
          const int sp = WIDE ? st & ~1 : st;
          const unsigned char *row = q < CF::MI ? smem + CF::a_off(sp) + off_a[q < CF::MI ? q : 0]
                                                : smem + CF::b_off(sp) + off_b[q < CF::MI ? 0 : q - CF::MI];
          const uint32_t sw = q < CF::MI ? swa[q < CF::MI ? q : 0] : swb[q < CF::MI ? 0 : q - CF::MI];
          raw[q] = *(const i32x4 *)(row + ((sw ^ (WIDE && odd ? 4u : 0u)) << 4));
        };
        // two of the chunk's values (pair p of half h) to their fragment
        auto widen = [&](int q, int h, int p, frag(&af)[CF::MI], frag(&bfr)[CF::NI]) {
          const uint32_t v = bf16_pair((uint32_t)raw[q][2 * h + (p >> 1)], (p & 1) != 0);
          frag &f = q < CF::MI ? af[q < CF::MI ? q : 0] : bfr[q < CF::MI ? 0 : q - CF::MI];
          i32x4 w = __builtin_bit_cast(i32x4, f);
          w[p] = (int)v;
          f = __builtin_bit_cast(frag, w);
        };
        if constexpr (E8) {
#pragma unroll
          for (int q = 0; q < CF::MI + CF::NI; ++q) read_raw(0, false, q);
#pragma unroll
          for (int c = 0; c < 4 * (CF::MI + CF::NI); ++c) widen(c >> 2, 0, c & 3, a0, b0);
        } else {
          read_frags(0, 0, a0, b0, 0, 0, 0);
        }
        wait_lds_all();
        wg_barrier();  // stage 0 read by every wave before step kb's loads refill it
        // claims are reserved now and sent between the two loop runs below
        if (claim_at >= 0) reserve_claims();
        uint32_t *claim_ctr = args.claim_policy == 0 ? &args.ctrl->counter : &args.ctrl->xcd_counter[(region) * kXcdStride];
        // The MFMA as a statement of its own, accumulating in place: each of the
        // 64 accumulators keeps one AGPR quad for the whole loop (all 256 AGPRs
        // hold accumulators, and with the builtin the register allocator
        // rotated some through copies every trip). The statements are volatile
        // and clobber memory, so program order is issue order: MFMA i, then
        // fragment read i of the next k-step (24 reads), and the eight loads
        // of k-step kt + 4 after MFMAs 3, 10, ..., 52 (one every seven: spread
        // over the step, they hold the MFMA stream least; measured against one
        // after every third read, 302k against 317k cycles per 8192^3 tile and
        // 3-4% off the HBM-bound shapes; all eight together after the first
        // MFMA cost 392k). Hazards: within the loop the MFMA operands are
        // written only by LDS reads (waited for), and accumulators are written
        // only by MFMAs; the fences before and after the loop give the wait
        // states the compiler cannot see.
        auto mfma16 = [&](int mi, int ni, const frag &a, const frag &b) {
          asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[mi][ni]) : "v"(b), "v"(a) : "memory");
        };
        // per-lane load offsets of a k-step with no partial K (see load_voff_edge)
        uint32_t voff_fast[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) voff_fast[j] = load_voff_edge(j);
        // the loads that go out at place `at` of `places` in a k-step: the narrow ones
        // of step kt + NST, and in the second step of a pair, whose fragments have
        // all been read, the wide ones of the pair NST steps after it. Those must
        // have landed when the next even step but NST - 4 ends, but evenly spread over
        // their step they land soonest all the same: 8192^3 NT, one every four MFMAs
        // 728 us, every third 733, every second 770, each 794. Beside narrow loads
        // they take the first half of the step and those the second. (Waits below: all
        // loads up to that step's narrow ones, which follow its wide ones, may be in
        // flight.)
        auto step_loads = [&](auto fast, bool odd, int32_t kt, int st, int at, int places, const i32x4 &ra, const i32x4 &rb, const i32x4 &wa,
                              const i32x4 &wb, int32_t wide_kt) {
          const uint32_t lbase = lds_addr(smem);
          if constexpr (WIDE) {
            const int every = places / (kNarrow > 0 ? 2 * kWide : kWide), j = at / every;
            if (odd && at % every == 0 && j < kWide)
              load16_to_lds(j < kWideA ? wa : wb, lbase + wide_dst(j, st),
                            decltype(fast)::value ? wide_voff(j) : wide_voff_tail(j, wide_kt));
            if constexpr (kNarrow > 0) {
              const int gap = places / (2 * kNarrow), k = (at - places / 2) / gap + (WA ? CF::A_LOADS : 0);
              if (at >= places / 2 && (at - places / 2) % gap == 0)
                load16_to_lds(k < CF::A_LOADS ? ra : rb, lbase + load_dst(k, st), decltype(fast)::value ? voff_fast[k] : load_voff(k, kt + NST));
            }
          } else {
            // (a spacing of eight, which lines the loads up with the rows of the
            // accumulator grid, made the compiler give up unrolling the step)
            const int first = places >= 64 ? 3 : 1, every = places >= 64 ? 7 : places / kLoads, j = (at - first) / every;
            if (at >= first && (at - first) % every == 0 && j < kLoads)
              load16_to_lds(j < CF::A_LOADS ? ra : rb, lbase + load_dst(j, st), decltype(fast)::value ? voff_fast[j] : load_voff(j, kt + NST));
          }
        };
        // loads that may be in flight when a k-step ends. Wide: an even step s needs the
        // pair s + 2, whose loads went out in step s + 3 - NST, before that step's narrow ones
        auto step_wait = [&](bool odd) {
          if constexpr (!WIDE) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 2) * kLoads) : "memory");
          } else if (odd) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST / 2 - 1) * kPair) : "memory");
          } else {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST / 2 - 2) * kPair + 2 * kNarrow) : "memory");
          }
        };
        // FAST: the k-step's loads read whole 32-deep slices (or lie past the
        // unit and read zeros through the resource), so the offsets above serve;
        // otherwise they are computed with the K-tail test.
        // st: the stage step kt's fragments came from, (kt - kb) mod 4; a compile-time
        // constant in the four-step trips, so every LDS address of the step is a
        // per-lane base plus an immediate offset
        // odd: the second step of a pair (known at compile time)
        auto step = [&](auto fast, bool odd, int32_t kt, int st, const frag(&ac)[CF::MI], const frag(&bc)[CF::NI],
                        frag(&an)[CF::MI], frag(&bn)[CF::NI]) {
          const int rst = (st + 1) & kMask;
          const unsigned char *sa = smem + CF::a_off(WA ? rst & ~1 : rst);
          const unsigned char *sb = smem + CF::b_off(WB ? rst & ~1 : rst);
          const uint32_t xa = WA && !odd ? 4u : 0u, xb = WB && !odd ? 4u : 0u;  // the step read is the pair's second when this is its first
          const int32_t kt_load = kt + NST;
          const i32x4 ra = make_rsrc_words(a_kstep(phys(kt_load)), kt_load < ke);
          const i32x4 rb = make_rsrc_words(b_kstep(phys(kt_load)), kt_load < ke);
          // (st is its pair's second stage: the pair NST steps on begins at kt - 1 + NST)
          const int32_t pair_load = phys(kt + NST - 1);
          const i32x4 wa = WIDE && odd ? wide_rsrc(true, kt + NST - 1) : ra, wb = WIDE && odd ? wide_rsrc(false, kt + NST - 1) : rb;
          i16x4 alo[CF::MI], lo[CF::NI];
          auto read = [&](int r) {
            if (r < kReadsA) {
              if constexpr (AT) {
                const unsigned char *pa0 = sa + off_a[r >> 1];
                if ((r & 1) == 0) {
                  alo[r >> 1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pa0));
                } else {
                  an[r >> 1] = join(alo[r >> 1], __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pa0 + 4 * CF::B_ROW)));
                }
              } else {
                an[r] = *(const bf16x8 *)(sa + off_a[r] + ((swa[r] ^ xa) << 4));
              }
            } else if constexpr (BT) {
              bn[r - kReadsA] = *(const bf16x8 *)(sb + off_b[r - kReadsA] + ((swb[r - kReadsA] ^ xb) << 4));
            } else {
              const int ni = (r - kReadsA) >> 1;
              const unsigned char *pb0 = sb + off_b[ni];
              if (((r - kReadsA) & 1) == 0) {
                lo[ni] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pb0));
              } else {
                bn[ni] = join(lo[ni], __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(pb0 + 4 * CF::B_ROW)));
              }
            }
          };
          static_assert(kReads <= kMfma, "read placement");
#pragma unroll
          for (int i = 0; i < kMfma; ++i) {
            mfma16(i / CF::NI, i % CF::NI, ac[i / CF::NI], bc[i % CF::NI]);
            if (i < kReads) read(i);
            step_loads(fast, odd, kt, st, i, kMfma, ra, rb, wa, wb, pair_load);
          }
          if constexpr (OP::kPlain) wait_lds_all();
          else __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0), known to the compiler: no waits for these reads in the next step
          step_wait(odd);
          wg_barrier();
        };
        // The e4m3 k-step: the first half's MFMAs with the second half's widening
        // between them, then the second half's with the next k-step's reads and the
        // widening of their first half (64 conversions to 64 MFMAs in the 256 x 256
        // tile: they issue in the MFMAs' shadow). The conversions are pinned where
        // they stand; left free, they gather at the ends of the halves.
        auto step8 = [&](auto fast, bool odd, int32_t kt, int st) {
          const int rst = (st + 1) & kMask;
          const int32_t kt_load = kt + NST;
          const i32x4 ra = make_rsrc_words(a_kstep(phys(kt_load)), kt_load < ke);
          const i32x4 rb = make_rsrc_words(b_kstep(phys(kt_load)), kt_load < ke);
          const int32_t pair_load = phys(kt + NST - 1);
          const i32x4 wa = WIDE && odd ? wide_rsrc(true, kt + NST - 1) : ra, wb = WIDE && odd ? wide_rsrc(false, kt + NST - 1) : rb;
          constexpr int kChunks = CF::MI + CF::NI, kWiden = 4 * kChunks;
          // second half: reads first (kReadEach after each MFMA), conversions from kFrom on
          auto pair_of = [](int i, int c) { return i * (kWiden / kMfma) + c; };
          constexpr int kReadEach = kChunks / (kMfma / 4), kFrom = kMfma / 4 + kMfma / 8;
          static_assert(kReadEach * (kMfma / 4) == kChunks && kWiden % kMfma == 0 && 2 * (kMfma - kFrom) >= kWiden / (kWiden / kMfma), "step");
          auto half = [&](auto second) {
            constexpr bool h = decltype(second)::value;
#pragma unroll
            for (int i = 0; i < kMfma; ++i) {
              if (h) mfma16(i / CF::NI, i % CF::NI, a1[i / CF::NI], b1[i % CF::NI]);
              else mfma16(i / CF::NI, i % CF::NI, a0[i / CF::NI], b0[i % CF::NI]);
              __builtin_amdgcn_sched_barrier(0);
              if (!h) {
#pragma unroll
                for (int c = 0; c < kWiden / kMfma; ++c) widen(pair_of(i, c) >> 2, 1, pair_of(i, c) & 3, a1, b1);
              } else if (i < kMfma / 4) {
#pragma unroll
                for (int q = 0; q < kReadEach; ++q) read_raw(rst, !odd, i * kReadEach + q);
              } else if (i >= kFrom) {
#pragma unroll
                for (int c = 0; c < 2 * (kWiden / kMfma); ++c) {
                  const int next = 2 * pair_of(i - kFrom, 0) + c;
                  if (next < kWiden) widen(next >> 2, 0, next & 3, a0, b0);
                }
              }
              step_loads(fast, odd, kt, st, (h ? kMfma : 0) + i, 2 * kMfma, ra, rb, wa, wb, pair_load);
              __builtin_amdgcn_sched_barrier(0);
            }
          };
          half(std::false_type{});
          half(std::true_type{});
          __builtin_amdgcn_s_waitcnt(0xC07F);  // as in step
          step_wait(odd);
          wg_barrier();
        };
        // the zeroed accumulators in their registers, then 16 wait states, before
        // the first MFMA reads them
#pragma unroll
        for (int mi = 0; mi < CF::MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < CF::NI; ++ni) asm volatile("" : "+a"(acc[mi][ni]));
        asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");
        // two steps per trip, so the fragment buffers swap roles by name. An odd
        // count ends with one step past the unit: its stage was zero-filled, and
        // adding zero products leaves every accumulator bit for bit as it was.
        // The dynamic scheduler runs the loop in two parts and sends its claims
        // between them, at the trip boundary at or before claim_at.
        // Trips whose loads reach the partial k-step `full` (K not a multiple of
        // 32, and the unit ends after it) use the K-tail test: from the first trip
        // t (t - kb even) with t + 5 >= full on; the trips before it use the fast
        // offsets.
        const int32_t slow_from =
            (WIDE ? K % (2 * CF::BK) != 0 && ke == nk : K % CF::BK != 0 && full < ke)
                ? kb + ((max(full - (NST + 1) - kb, 0) + 1) / 2) * 2
                : ke + 2;
        // Fast trips of four steps while whole ones fit (constant stages), then
        // two-step trips with the stage computed at run time. A run starts with
        // kt - kb a multiple of 4.
        auto trips = [&](int32_t &kt, int32_t end) {
          const int32_t fast_end = min(end, slow_from);
          if constexpr (E8) {
            for (; kt + 4 <= fast_end; kt += 4) {
              const int st = NST == 4 ? 0 : (kt - kb) & kMask;
              step8(std::true_type{}, false, kt, st);
              step8(std::true_type{}, true, kt + 1, st + 1);
              step8(std::true_type{}, false, kt + 2, st + 2);
              step8(std::true_type{}, true, kt + 3, st + 3);
            }
            for (; kt < end; kt += 2) {
              const int st = (kt - kb) & kMask;
              step8(std::false_type{}, false, kt, st);
              step8(std::false_type{}, true, kt + 1, (st + 1) & kMask);
            }
            return;
          }
          for (; kt + 4 <= fast_end; kt += 4) {
            const int st = NST == 4 ? 0 : (kt - kb) & kMask;
            step(std::true_type{}, false, kt, st, a0, b0, a1, b1);
            step(std::true_type{}, true, kt + 1, st + 1, a1, b1, a0, b0);
            step(std::true_type{}, false, kt + 2, st + 2, a0, b0, a1, b1);
            step(std::true_type{}, true, kt + 3, st + 3, a1, b1, a0, b0);
          }
          for (; kt < fast_end; kt += 2) {
            const int st = (kt - kb) & kMask;
            step(std::true_type{}, false, kt, st, a0, b0, a1, b1);
            step(std::true_type{}, true, kt + 1, (st + 1) & kMask, a1, b1, a0, b0);
          }
          for (; kt < end; kt += 2) {
            const int st = (kt - kb) & kMask;
            step(std::false_type{}, false, kt, st, a0, b0, a1, b1);
            step(std::false_type{}, true, kt + 1, (st + 1) & kMask, a1, b1, a0, b0);
          }
        };
        int32_t kt = kb;
        if constexpr (MODE == kDynamic) {
          // the claims go out at the four-step boundary at or before claim_at
          const int32_t split_at = claim_at >= kb ? kb + ((claim_at - kb) & ~3) : ke;
          trips(kt, split_at);
          claim_issue_asm(claim_ctr, batch_n >= 1u, batch[0]);
          claim_issue_asm(claim_ctr, batch_n >= 2u, batch[1]);
        }
        trips(kt, ke);
        // 24 wait states after the last MFMA before anything reads an accumulator
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
        for (int mi = 0; mi < CF::MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < CF::NI; ++ni) asm volatile("" : "+a"(acc[mi][ni]));
      }
    }

    // ---- publish the claims issued during this unit (producer, wave 0): each
    // answer goes to its ring record. Prefetch claims are resolved here, before
    // the epilogue: reading an atomic's answer waits for every older memory
    // operation of the wave, and the C stores would otherwise be among them.
    auto publish_claims = [&]() {
      // the answers of claims sent from assembly. A full drain: a returning
      // atomic is not ordered with the loads issued after it, so only vmcnt 0
      // proves its answer (and the register it writes) has arrived
      wait_vmem_all();
      for (uint32_t b = 0; b < batch_n; ++b) {
        const uint32_t v = claim_resolve(args, xcc, lane, b == 0 ? batch[0] : batch[1], region);
        const uint32_t ok = v < (uint32_t)T ? 1u : 0u;
        if (!ok) failed = true;
        if (lane == 0) ring[(batch_ord + b) % (uint32_t)args.ring_depth] = RingRec{v, ok, batch_ord + b, 0u};
      }
    };
    // With claims sent during the unit, the next unit's record is read right
    // after they are published, so the end of the unit needs no barrier.
    RingRec next_rec = RingRec{0u, 0u, 0u, 0u};
    bool next_read = false;
    if constexpr (MODE == kDynamic) {
      if (args.claims_ahead >= 1) {
        if (wave == 0) publish_claims();
        if (last_sub) {
          __syncthreads();
          next_rec = ring[(ord + 1) % (uint32_t)args.ring_depth];
          next_read = true;
        }
      }
    }

    // ---- epilogue: fp32 accumulators -> C. Lane l holds, in each group of four
    // accumulators, 4 consecutive n of row m = l % MB of its block: n = 8 qd +
    // 4 (l / 32) for 32 x 32 blocks, 4 (l / 16) for 16 x 16 blocks; group g =
    // (mi NI + ni) QUADS + qd of a thread is its g-th group. C is written once
    // and never read by the kernel, so the stores are non-temporal: they do not
    // displace the A and B slices the XCD's other workgroups are still reading
    // from L2 (measured 1-3% faster across the modes).
    const bool interior = m0 + BM <= M && n0 + BN <= N;

    // Whole rows per store. Written straight from the accumulators, one store
    // covers 16 rows x 64 B (16 x 16 blocks) or 32 rows x 32 B (32 x 32
    // blocks), and a CU then writes a 256 KiB tile in about 7 us whether or not
    // other CUs store too (measured with a store-only kernel), while stores of
    // whole rows take about 2 us alone and reach about 8 TB/s when every CU
    // stores at once. So each wave passes its WM x WN results through its
    // quarter of the stage ring, RP rows (a pass) at a time, and reads them back
    // a row at a time: each store then writes RPR rows of WN contiguous floats.
    // 16-byte chunk c of row r sits in slot c ^ (r mod 16), which keeps the
    // block-shaped writes and the row-shaped reads free of bank conflicts.
    // epi_begin / epi_end bracket the use of the ring (every wave calls them);
    // stage writes a group of four results of pass p, flush stores pass p.
    constexpr int WAVE_LDS = CF::LDS / CF::NW;
    constexpr int ROW_B = CF::WN * 4;
    constexpr int RP = WAVE_LDS / ROW_B < CF::WM ? WAVE_LDS / ROW_B : CF::WM;
    constexpr int CHUNKS = ROW_B / 16;
    constexpr int RPR = 1024 / ROW_B;
    constexpr int MI_PASS = RP / CF::MB;
    constexpr int PASSES = CF::WM / RP;
    static_assert(CF::WM % RP == 0 && RP % CF::MB == 0 && CHUNKS * RPR == 64 && CHUNKS <= 32, "epilogue");
    unsigned char *wl = smem + wave * WAVE_LDS;
    // the staging addresses are computed here, not kept in registers over the main
    // loop (the e4m3 loop has none to spare)
    uint32_t elane = lane;
    if constexpr (!OP::kPlain) asm volatile("" : "+v"(elane));
    auto epi_begin = [&]() {
      // every wave's loads into the stages have landed and its fragment reads
      // are done before any wave overwrites the stages
      wait_vmem_all();
      wg_barrier();
    };
    auto stage = [&](int p, int mi, int ni, int qd, const f32x4 &v) {
      const uint32_t row = (uint32_t)((mi - p * MI_PASS) * CF::MB) + elane % CF::MB;
      const uint32_t c = (uint32_t)(ni * (CF::MB / 4) + 2 * qd) + elane / CF::MB;
      *(f32x4 *)(wl + row * ROW_B + ((c ^ (row & 15u)) << 4)) = v;
    };
    auto flush = [&](int p) {
      // the wave's own LDS writes complete before its reads of other lanes' data
      wait_lds_all();
      __builtin_amdgcn_wave_barrier();
      if constexpr (OP::kPlain) {
#pragma unroll 4
        for (int i = 0; i < RP / RPR; ++i) {
          const uint32_t row = (uint32_t)(i * RPR) + lane / CHUNKS;
          const uint32_t c = lane % CHUNKS;
          const f32x4 v = *(const f32x4 *)(wl + row * ROW_B + ((c ^ (row & 15u)) << 4));
          const int32_t m = m0 + (int32_t)(wm * CF::WM + p * RP + row);
          const int32_t n = n0 + (int32_t)(wn * CF::WN + 4 * c);
          if (interior || (m < M && n < N)) __builtin_nontemporal_store(v, (f32x4 *)(pb.C + (size_t)m * (size_t)N + n));
        }
      } else {
        // a K-chunk's rows go to its slot of the workspace as they are: a second
        // kernel adds the chunks and finishes the tile
        float *slot = split ? args.ws + (size_t)(item - (uint32_t)args.split_base) * (BM * BN) +
                                  (size_t)(wm * CF::WM + p * RP) * BN + wn * CF::WN
                            : nullptr;
        OP::template flush<RP, ROW_B, BN>(op, wl, lane, m0 + (int32_t)(wm * CF::WM) + p * RP, n0 + (int32_t)(wn * CF::WN), M, N, slot);
      }
      // the reads are done before the next pass (or the next unit's loads) writes the region
      wait_lds_all();
      __builtin_amdgcn_wave_barrier();
    };
    auto epi_end = [&]() { wg_barrier(); };

    if (!OP::kPlain || !split) {
      epi_begin();
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
#pragma unroll
        for (int mi = p * MI_PASS; mi < (p + 1) * MI_PASS; ++mi)
#pragma unroll
          for (int ni = 0; ni < CF::NI; ++ni)
#pragma unroll
            for (int qd = 0; qd < CF::QUADS; ++qd)
              stage(p, mi, ni, qd, f32x4{acc[mi][ni][4 * qd + 0], acc[mi][ni][4 * qd + 1], acc[mi][ni][4 * qd + 2],
                                         acc[mi][ni][4 * qd + 3]});
        flush(p);
      }
      epi_end();
    } else if constexpr (OP::kPlain) {
      // K-chunk of a split tile: publish the partial sum; the workgroup that
      // completes the tile's last chunk adds all partials in chunk order and
      // writes C. The order is fixed, so the result does not depend on who
      // finished last. Partial slots are thread-major per 16-byte group: fully
      // coalesced. The sum reads the other chunks' slots in batches of up to
      // 16 groups per thread, all of a chunk's loads of a batch in flight at once.
      // The partials are written and read with agent-scope cache policy
      // (store16_agent / load16_agent): the stores go through to memory and a
      // vmcnt(0) wait completes them before the arrival count goes out, so the
      // count itself can be relaxed. Release and acquire fences in their place
      // write back and invalidate the whole L2 of the XCD; with every tile of a
      // run split (fewer tiles than workers) they cost 2048 x 2048 x 8192 about
      // a third of its time.
      const uint32_t S = (uint32_t)args.split_chunks;
      const uint32_t q = tile - (uint32_t)args.split_base;
      const __amdgpu_buffer_rsrc_t wsr = make_rsrc(args.ws);
      const uint32_t slot_off = (item - (uint32_t)args.split_base) * (uint32_t)(BM * BN * 4);
#pragma unroll
      for (int mi = 0; mi < CF::MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < CF::NI; ++ni)
#pragma unroll
          for (int qd = 0; qd < CF::QUADS; ++qd) {
            const int g = (mi * CF::NI + ni) * CF::QUADS + qd;
            store16_agent(wsr, slot_off + (uint32_t)(g * CF::THREADS + (int)tid) * 16u,
                          f32x4{acc[mi][ni][4 * qd + 0], acc[mi][ni][4 * qd + 1], acc[mi][ni][4 * qd + 2],
                                acc[mi][ni][4 * qd + 3]});
          }
      wait_vmem_all();  // this thread's partial has reached memory
      __syncthreads();
      if (tid == 0) {
        const uint32_t prev = __hip_atomic_fetch_add(&args.arrivals[q], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        split_last = prev + 1u == S ? 1u : 0u;
        // every chunk has arrived: the count is done with for this run
        if (prev + 1u == S) __hip_atomic_store(&args.arrivals[q], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (wave_uniform(split_last) != 0) {
        // the sum in chunk order, staged straight into the ring a pass at a
        // time and stored in whole rows like a whole tile (the partial loads
        // go out after the count's answer, which every thread has waited for)
        const uint32_t base = q * S * (uint32_t)(BM * BN * 4) + tid * 16u;
        constexpr int kPassGroups = MI_PASS * CF::NI * CF::QUADS;  // groups g of pass p: p kPassGroups + [0, kPassGroups)
        constexpr int kBatch = kPassGroups < 16 ? kPassGroups : 16;
        static_assert(kPassGroups % kBatch == 0, "batches");
        epi_begin();
        for (int p = 0; p < PASSES; ++p) {
          for (int g0 = p * kPassGroups; g0 < (p + 1) * kPassGroups; g0 += kBatch) {
            f32x4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (uint32_t c = 0; c < S; ++c) {
              const uint32_t src = base + c * (uint32_t)(BM * BN * 4) + (uint32_t)(g0 * CF::THREADS) * 16u;
              f32x4 part[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) part[i] = load16_agent(wsr, src + (uint32_t)(i * CF::THREADS) * 16u);
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] += part[i][e];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int g = g0 + i;
              stage(p, g / (CF::NI * CF::QUADS), (g / CF::QUADS) % CF::NI, g % CF::QUADS, v[i]);
            }
          }
          flush(p);
        }
        epi_end();
      }
    }

    // ---- claims after the work (claims_ahead = 0): issue and publish
    if (wave == 0) {
      if constexpr (MODE == kDynamic) {
        if (args.claims_ahead == 0 && !failed && last_sub) {
          batch_ord = next_ord;
          batch[0] = claim_issue(args, region);
          batch_n = 1;
          ++next_ord;
          publish_claims();
        }
      }
    }
    // ---- log the tile
    if (tid == 0) {
      const uint64_t t1 = clock_core();
      const uint64_t r1 = clock_wall();
      if ((int32_t)item < args.log_cap) {
        TileRecDev rec;
        rec.tile = tile;
        rec.unit = unit;
        rec.pad = 0;
        rec.kb = (uint32_t)kb;
        rec.ke = (uint32_t)ke;
        rec.worker = blockIdx.x;
        rec.hw_id = hwid;
        rec.xcc_id = xcc;
        rec.t0 = t0;
        rec.t1 = t1;
        rec.r0 = r0;
        rec.r1 = r1;
        args.log[item] = rec;
        __hip_atomic_fetch_add(&args.visits[item], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }

    // ---- advance: the next item of this unit, else the next unit
    if (!last_sub) {
      ++sub;
      continue;
    }
    sub = 0;
    if constexpr (MODE == kDynamic) {
      if (!next_read) {
        __syncthreads();
        next_rec = ring[(ord + 1) % (uint32_t)args.ring_depth];
      }
      const RingRec rec = next_rec;
      const uint32_t seq = wave_uniform(rec.seq);
      valid = wave_uniform(rec.valid) != 0;
      unit = wave_uniform(rec.tile);
      if (seq != ord + 1) {
        // the ring protocol was violated: stop this worker and flag it
        if (tid == 0) flag_error(args, 2u);
        valid = false;
      }
    } else if constexpr (MODE == kStatic) {
      unit += (uint32_t)args.P;
      valid = unit < (uint32_t)T;
    } else {
      valid = false;
    }
    ++ord;
  }

  if (tid == 0) {
    if (args.max_concurrent > 0)
      __hip_atomic_fetch_sub(&args.ctrl->gate, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    if (args.self_clean) leave_run(args);
  }
}


}  // namespace ptg
