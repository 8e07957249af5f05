// The matrix-product core of the training kernels (grouped-product gradients
// and the Newton-Schulz products): D[m, n] = sum_k A[m, k] B[n, k] per tile,
// 16-bit operands, fp32 accumulation, tcgen05 + TMEM, operands staged by TMA.
//
// What the inference GEMMs do not have and these products need:
//  * either operand may be stored with its MN index along memory (the
//    transpose of what the forward reads): a row-major [k, mn] matrix is
//    loaded as 128-byte-swizzled boxes of 64 mn by 64 k and handed to the MMA
//    as an MN-major operand, so no transposed copy exists anywhere;
//  * the summed axis may be ragged (rows of one expert): the last k block of a
//    tile may end at any row. The rows past the end belong to the next expert
//    or lie outside the matrix, and may hold anything, NaN included, so they
//    are not multiplied: whole 16-row MMA steps past the end are not issued,
//    and a warp zeroes the up to 15 rows of both operands that share the last
//    step with valid rows, after the loads have landed and before the MMA;
//  * CTA pairs (CG = 2): a tile is 256 x BN over two SMs, each holding 128
//    rows of A and BN / 2 rows of B, so an SM streams 32 KB per k block instead
//    of 48 KB for the same MMA time;
//  * sums of any length in fp32: the MMA truncates its running sum at every
//    16-row step (measured: 1.9e-5 of the result's norm after 16397 rows, in
//    proportion to the steps), so an Op that asks for it (kChunk) has every
//    kChunk k blocks summed on their own and the partial sums added in
//    registers, rounded to nearest.
//
// Warp roles (384 threads): 0 TMA producer, 1 TMEM allocator + MMA issuer (the
// pair's leading CTA issues for both), 2 tail zeroing, 3 none, 4..11 epilogue
// (TMEM lane quarter warp % 4, half of the tile's columns (warp - 4) / 4). Two
// accumulator buffers let the epilogue of a tile or chunk overlap the next
// one's products. Persistent: CTA (pair) c takes tiles c, c + grid, ... Every
// wait is bounded (ptx::mbar_wait).
//
// An Op supplies the tiles and the epilogue:
//   kAMn, kBMn    operand stored with MN along memory
//   kBN           tile columns;  kFmt  1 bf16, 0 fp16
//   kTail         tiles may end inside a k block (both operands MN-major)
//   kVarN         a tile has Tile::n <= kBN columns, a multiple of 16: the MMA takes
//                 time in proportion down to about 128
//   kChunk        k blocks summed by the MMA at a time, 0: all
//   kStageWarp    bytes of staging per epilogue warp (a multiple of 1024)
//   kSharedInts   int32 words of shared memory for its tables
//   setup(sh)                 one warp fills the tables
//   total(sh)                 number of tiles
//   decode(sh, tile, Tile&)   coordinates and k range of a tile
//   prefetch(Tile, Warp&)     loads that do not need the accumulator
//   epilogue(Tile, Warp&, taddr) -> bool  (false: a wait ran out)  or, with kChunk,
//   store(Tile, Warp&, sum)
#pragma once

#include <atomic>

#include "gemm_common.cuh"
#include "ptx_pair.cuh"

namespace moe {
namespace mm {

constexpr int BM = 128;  // accumulator rows per CTA
constexpr int BK = 64;
constexpr int UK = 16;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kTileA = BM * BK * 2;         // 16 KB
constexpr int kSmemMax = 227 * 1024;
constexpr int kFew = 32;                    // kVarN: rows of the smaller box of b
constexpr int kBarBytes = 512;
constexpr int kSiteTail = 9;                // status word: the tail-zeroing wait,
constexpr int kSiteLoad = 10;               // an epilogue warp's wait for its own loads

struct Tile {
  int a_mn, a_k;  // A's coordinates of (row 0, k 0) of the pair's tile
  int b_mn, b_k;
  int nkb;        // k blocks; 0: the accumulator is zero and is not read
  int tail;       // valid k rows of the last block (1..64)
  int n;          // kVarN: columns
  int p[3];       // the Op's own
};

template <class Op, int CG>
struct Cfg {
  static constexpr int BN = Op::kBN;
  static constexpr int kBRows = BN / CG;  // B rows (or columns, MN-major) in one CTA
  static constexpr int kTileB = kBRows * BK * 2;
  static constexpr int kStage = kTileA + kTileB;
  // the operand ring takes what the staging, the barriers and the tables leave
  static constexpr int kStageOut = Op::kStageWarp * kEpiWarps;
  static constexpr int kRest = 1024 + kStageOut + kBarBytes + Op::kSharedInts * 4;
  static constexpr int STAGES = (kSmemMax - kRest) / kStage > 10 ? 10 : (kSmemMax - kRest) / kStage;
  static constexpr int kTmemCols = 2 * BN;  // two accumulators
  static constexpr uint32_t kIdesc = ptx::make_idesc(BM * CG, BN, Op::kFmt, Op::kFmt) |
                                     (Op::kAMn ? ptx::kIdescAMn : 0u) |
                                     (Op::kBMn ? ptx::kIdescBMn : 0u);
  static constexpr size_t kSmem = (size_t)STAGES * kStage + kRest;
  static_assert(kStage % 1024 == 0, "stages start on swizzle-atom boundaries");
  static_assert(kTileB % 1024 == 0, "B tiles are whole swizzle atoms");
  static_assert(!Op::kBMn || kBRows % 64 == 0, "MN-major boxes are 64 wide");
  static_assert(!Op::kTail || (Op::kAMn && Op::kBMn), "a ragged sum needs rows as k");
  static_assert(!Op::kVarN || (!Op::kBMn && !Op::kTail && Op::kChunk == 0 && kBRows >= kFew), "rows of a K-major b");
  static_assert(STAGES >= 2, "shared memory of one CTA");
};

// Loads MN rows [mn, mn + ROWS) by one k block of an operand into `dst`.
template <bool MN, int ROWS, int CG>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* tm, int mn, int k,
                                             uint32_t bar) {
  if constexpr (MN) {  // ROWS / 64 groups of 64 mn, one box of k rows each, by one instruction
    if constexpr (CG == 2) ptx::tma_load_3d_pair(dst, tm, 0, k, mn / 64, bar);
    else ptx::tma_load_3d(dst, tm, 0, k, mn / 64, bar);
  } else {
    static_assert(ROWS == 128 || ROWS == kFew, "one box of rows");
    if constexpr (CG == 2) ptx::tma_load_2d_pair(dst, tm, k, mn, bar);
    else ptx::tma_load_2d(dst, tm, k, mn, bar);
  }
}

// 32 accumulator columns of this thread's row.
__device__ __forceinline__ void load_acc32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();  // the load is one instruction of the whole warp
  ptx::tmem_ld32(taddr, r);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// A position in the operand ring.
template <int STAGES, int BYTES>
struct Ring {
  uint32_t stage;  // the stage's address
  uint32_t bar;    // its barriers' offset
  uint32_t parity = 0;
  bool wrapped = false;
  uint32_t base;
  __device__ __forceinline__ explicit Ring(uint32_t b) : stage(b), bar(0), base(b) {}
  __device__ __forceinline__ void step() {
    stage += BYTES;
    bar += 8;
    if (bar == STAGES * 8) {
      stage = base;
      bar = 0;
      parity ^= 1;
      wrapped = true;
    }
  }
};

struct Maps {
  CUtensorMap a, b;
  CUtensorMap b_few;  // kVarN: b in boxes of kFew rows
  CUtensorMap c[3];   // the epilogue's own
};

// An epilogue warp: which part of the tile it holds, and its staging, boxes of
// 32 rows (lane = row) of 64 or 128 bytes, swizzled as tiled copies read and
// write them. Staging is small on purpose: what it takes, the operand ring
// lacks.
struct Warp {
  const Maps* maps;
  int rank, q, half, lane;
  uint32_t base;     // staging, on a 1024-byte boundary
  uint32_t bar;      // two barriers of loads into the staging
  uint32_t parity;   // bit i: parity of barrier i's next phase
  uint32_t pending;  // bit i: a load is in flight on barrier i
  int32_t* status;
  float4 own;        // the Op's own, from prefetch to epilogue

  // first row of this warp in a tile that starts at row m
  __device__ __forceinline__ int row0(int m) const { return m + rank * BM + q * 32; }
  // every store so far has read its box
  __device__ __forceinline__ void free_boxes() const {
    if (lane == 0) ptx::bulk_wait_read0();
    __syncwarp();
  }
  // address of 16-byte piece j of row r: 64-byte rows (j < 4), 128-byte rows (j < 8)
  static __device__ __forceinline__ uint32_t at64(uint32_t box, int r, int j) {
    return box + r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
  }
  static __device__ __forceinline__ uint32_t at128(uint32_t box, int r, int j) {
    return box + r * 128 + ((j ^ (r & 7)) << 4);
  }
  static __device__ __forceinline__ void put(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  }
  static __device__ __forceinline__ uint4 get(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
  }
  // what every lane put is ready for tiled stores (by lane 0)
  __device__ __forceinline__ void publish() const {
    ptx::fence_proxy_async_smem();
    __syncwarp();
  }
  // box <- the tensor at {c0, c1, c2}; all lanes have done with the box
  __device__ __forceinline__ void load(int i, uint32_t box, const CUtensorMap* tm, int c0, int c1, int c2,
                                       uint32_t bytes) {
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(bar + 8 * i, bytes);
      ptx::tma_load_3d(box, tm, c0, c1, c2, bar + 8 * i);
    }
    pending |= 1u << i;
  }
  __device__ __forceinline__ bool wait(int i) {
    const bool ok = ptx::mbar_wait(bar + 8 * i, (parity >> i) & 1u, status, kSiteLoad);
    parity ^= 1u << i;
    pending &= ~(1u << i);
    return ok;
  }
};

template <class Op, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    mm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Op op, int32_t* status) {
  using C = Cfg<Op, CG>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* stage_out = smem + STAGES * C::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_out + C::kStageOut);
  // bars: full[STAGES], empty[STAGES], tail[STAGES], accf[2], acce[2], drain, load[8][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * STAGES + 5 + 2 * kEpiWarps);
  int32_t* sh = reinterpret_cast<int32_t*>(stage_out + C::kStageOut + kBarBytes);

  // (the same in every lane, and known to be: the roles' loops keep their state in
  // uniform registers, where the MMA takes its operands from)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)ptx::cluster_ctarank() : 0;
  const int unit0 = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;
  const uint32_t sbase = ptx::smem_addr(smem);
  const uint32_t full0 = ptx::smem_addr(bars), empty0 = full0 + STAGES * 8;
  const uint32_t tail0 = empty0 + STAGES * 8, accf0 = tail0 + STAGES * 8, acce0 = accf0 + 16, drain = acce0 + 16,
                 load0 = drain + 8;
  // the leading CTA's barriers (this CTA's own without pairs)
  const uint32_t lead_full0 = CG == 2 ? ptx::map_to_cta(full0, 0) : full0;
  const uint32_t lead_acce0 = CG == 2 ? ptx::map_to_cta(acce0, 0) : acce0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full0 + s * 8, CG);  // one arrival a CTA, with its bytes or after its zeroing
      ptx::mbar_init(empty0 + s * 8, 1);
      ptx::mbar_init(tail0 + s * 8, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(accf0 + a * 8, 1);
      ptx::mbar_init(acce0 + a * 8, kEpiWarps * CG);
    }
    ptx::mbar_init(drain, 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) ptx::mbar_init(load0 + i * 8, 1);
    ptx::fence_barrier_init();
    ptx::tma_prefetch_desc(&maps.a);
    ptx::tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), C::kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_addr(tmem_slot), C::kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  if (warp == 2) {
    ptx::wait_for_previous_grid();
    op.setup(sh);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) ptx::cluster_sync();  // both CTAs' barriers exist before anyone signals them
  ptx::tc_fence_after();
  ptx::let_next_grid_start();
  // Without tables to fill, the first tile's place needs nothing of the grid
  // ahead: found before the wait, it also brings the parameters into the caches.
  constexpr bool kEarly = Op::kSharedInts == 0;
  const uint32_t tmem_base = *tmem_slot;
  Tile t;  // each role's own, from here on
  int total;
  if constexpr (kEarly) {
    total = op.total(sh);
    if (unit0 < total) op.decode(sh, unit0, t);
  }
  ptx::wait_for_previous_grid();
  if constexpr (!kEarly) {
    total = op.total(sh);
    if (unit0 < total) op.decode(sh, unit0, t);
  }
  // the next tile of a role's loop
  auto next = [&](int tile) {
    tile += units;
    if (tile < total) op.decode(sh, tile, t);
    return tile;
  };
  // The producer's and the MMA issuer's loops run in one warp each, so a k block
  // costs them their instructions' latencies: positions in the ring are stepped,
  // not divided out (measured without loads: a loop with 64-bit quotients took 675
  // cycles a block, whatever the MMA's size, and 593 without them; 558 with the
  // whole warp in the loop; the MMAs themselves take 512).
  if (warp == 0) {
    // The whole warp walks the tiles and waits, one lane loads.
    const bool loader = ptx::elect_one();
    Ring<STAGES, C::kStage> at(sbase);
    bool ok = true;
    for (int tile = unit0; tile < total && ok; tile = next(tile)) {
      const int am = t.a_mn + rank * BM, bn = t.b_mn + rank * (Op::kVarN ? t.n / CG : C::kBRows);
      const bool few = Op::kVarN && t.n <= kFew * CG;  // of this CTA's rows of b
      int ka = t.a_k, kbb = t.b_k;
      for (int left = t.nkb; left > 0; --left, ka += BK, kbb += BK) {
        if (!ptx::mbar_wait(empty0 + at.bar, at.parity ^ 1, status, kSiteProducerEmpty)) {
          ok = false;
          break;
        }
        if (loader) {
          uint32_t bar;
          if (Op::kTail && left == 1 && (t.tail & (UK - 1))) {
            bar = tail0 + at.bar;  // this CTA's warp 2 waits for the bytes and arrives on `full` itself
            ptx::mbar_arrive_expect_tx(bar, C::kStage);
          } else {
            const uint32_t bytes = few ? kTileA + kFew * 128 : C::kStage;
            bar = lead_full0 + at.bar;
            if (CG == 2 && rank != 0) ptx::mbar_arrive_expect_tx_cluster(bar, bytes);
            else ptx::mbar_arrive_expect_tx(full0 + at.bar, bytes);
          }
          load_operand<Op::kAMn, BM, CG>(at.stage, &maps.a, am, ka, bar);
          load_operand<Op::kBMn, C::kBRows, CG>(at.stage + kTileA, few ? &maps.b_few : &maps.b, bn, kbb, bar);
        }
        at.step();
      }
    }
    // The leading CTA frees the other one's stages, too: all of it has come before that
    // one goes. (A stage that was never used is free.)
    if (CG == 2 && loader && rank != 0 && ok) {
      for (int i = 0; i < STAGES; ++i, at.step()) ptx::mbar_wait(empty0 + at.bar, at.parity ^ 1, status, kSiteDrain);
    }
    // every load of the ring has landed before this CTA (for a pair: both) goes
    if (loader && rank == 0) {
      for (uint32_t b = 0; b < STAGES * 8; b += 8) {
        const bool again = b < at.bar;  // used since the ring last began
        if (again || at.wrapped) ptx::mbar_wait(full0 + b, again ? at.parity : at.parity ^ 1, status, kSiteDrain);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // The whole warp walks the tiles and waits, one lane issues.
      const bool issuer = ptx::elect_one();
      Ring<STAGES, C::kStage> at(sbase);
      int acc = 0;
      uint32_t acc_ph = 0;
      bool ok = true;
      // descriptors of stage 0; a stage further, 16-byte units are added
      const uint64_t da0 = Op::kAMn ? ptx::sw128_mnmajor_desc(sbase, 8192) : ptx::sw128_kmajor_desc(sbase);
      const uint64_t db0 = Op::kBMn ? ptx::sw128_mnmajor_desc(sbase + kTileA, 8192)
                                    : ptx::sw128_kmajor_desc(sbase + kTileA);
      // 16 k further: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
      constexpr uint64_t stepA = Op::kAMn ? (UK * 128) >> 4 : (UK * 2) >> 4;
      constexpr uint64_t stepB = Op::kBMn ? (UK * 128) >> 4 : (UK * 2) >> 4;
      uint32_t idesc = C::kIdesc;
      auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t more) {
        if constexpr (CG == 2) ptx::mma_f16_pair(d, da, db, idesc, more);
        else ptx::mma_f16(d, da, db, idesc, more);
      };
      auto commit = [&](uint32_t bar) {
        if constexpr (CG == 2) ptx::mma_commit_pair(bar);
        else ptx::mma_commit(bar);
      };
      for (int tile = unit0; tile < total && ok; tile = next(tile)) {
        int left = t.nkb;
        if constexpr (Op::kVarN) idesc = (C::kIdesc & ~(63u << 17)) | (uint32_t)(t.n >> 3) << 17;
        do {  // once without chunks; an empty sum still hands over its (unread) accumulator
          if (!ptx::mbar_wait(acce0 + acc * 8, acc_ph ^ 1, status, kSiteMmaAccEmpty)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + acc * C::BN;
          uint32_t more = 0;
          for (int n = Op::kChunk ? min(left, Op::kChunk) : left; n > 0; --n, --left) {
            if (!ptx::mbar_wait(full0 + at.bar, at.parity, status, kSiteMmaFull)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t off = (at.stage - sbase) >> 4;
            const uint64_t da = da0 + off, db = db0 + off;
            if (issuer) {
              if (Op::kTail && left == 1) {  // no 16-row step past the last row
                for (int kk = 0; kk * UK < t.tail; ++kk) mma(d, da + kk * stepA, db + kk * stepB, kk ? 1 : more);
              } else {
                mma(d, da, db, more);
#pragma unroll
                for (int kk = 1; kk < BK / UK; ++kk) mma(d, da + kk * stepA, db + kk * stepB, 1);
              }
              commit(empty0 + at.bar);
            }
            more = 1;
            at.step();
          }
          if (!ok) break;
          if (issuer) commit(accf0 + acc * 8);
          acc ^= 1;
          if (acc == 0) acc_ph ^= 1;
        } while (left > 0);
      }
      // every MMA that was issued has completed once `drain` fires
      if (issuer) {
        commit(drain);
        ptx::mbar_wait(drain, 0, status, kSiteDrain);
      }
    }
  } else if (warp == 2) {
    if constexpr (Op::kTail) {
      int slot = 0;         // stage of the tile's first k block
      uint32_t phases = 0;  // bit s: parity of tail[s]'s next phase
      for (int tile = unit0; tile < total; tile = next(tile)) {
        const int s = (slot + t.nkb + STAGES - 1) % STAGES;  // of its last one
        slot = (slot + t.nkb) % STAGES;
        if (t.nkb == 0 || !(t.tail & (UK - 1))) continue;
        if (!ptx::mbar_wait(tail0 + s * 8, (phases >> s) & 1u, status, kSiteTail)) break;
        phases ^= 1u << s;
        // rows [tail, next multiple of 16) of every 64-wide group: whole
        // 128-byte rows, so the swizzle inside them does not matter. A lane
        // holds one of the eight 16-byte pieces of every fourth group.
        unsigned char* at = smem + s * C::kStage + (lane >> 3) * 8192 + (lane & 7) * 16;
        constexpr int GROUPS = (BM + C::kBRows) / 64;
        for (int r = t.tail; r & (UK - 1); ++r) {
#pragma unroll
          for (int g = 0; g < GROUPS; g += 4)
            if (g + (lane >> 3) < GROUPS)
              *reinterpret_cast<uint4*>(at + g * 8192 + r * 128) = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) ptx::mbar_arrive_cluster(lead_full0 + s * 8);
          else ptx::mbar_arrive(full0 + s * 8);
        }
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    Warp w{&maps, rank, q, half, lane, ptx::smem_addr(stage_out) + (warp - 4) * Op::kStageWarp,
           load0 + (warp - 4) * 16, 0, 0, status, {}};
    int acc = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    // waits for the next accumulator; release() gives it back
    auto take = [&]() {
      ok = ptx::mbar_wait(accf0 + acc * 8, acc_ph, status, kSiteEpiAccFull);
      ptx::tc_fence_after();
      return tmem_base + ((uint32_t)(q * 32) << 16) + acc * C::BN;
    };
    auto release = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) ptx::mbar_arrive_cluster(lead_acce0 + acc * 8);
        else ptx::mbar_arrive(acce0 + acc * 8);
      }
      acc ^= 1;
      if (acc == 0) acc_ph ^= 1;
    };
    for (int tile = unit0; tile < total && ok; tile = next(tile)) {
      if constexpr (Op::kChunk != 0) {
        // The first (often the only) partial sum is read straight into place,
        // all its loads in flight at once; later ones are added 16 columns at a time.
        constexpr int HALF = C::BN / 2;
        uint32_t sum[HALF];
        {
          const uint32_t taddr = take() + half * HALF;
          if (!ok) break;
          if (t.nkb != 0) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < HALF; c += 32)
              ptx::tmem_ld32(taddr + c, reinterpret_cast<uint32_t(&)[32]>(sum[c]));
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < HALF; ++i) sum[i] = 0u;
          }
          release();
        }
#pragma unroll 1
        for (int kb = Op::kChunk; kb < t.nkb; kb += Op::kChunk) {
          const uint32_t taddr = take() + half * HALF;
          if (!ok) break;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < HALF; c += 16) {
            uint32_t v[16];
            ptx::tmem_ld16(taddr + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              sum[c + i] = __float_as_uint(__uint_as_float(sum[c + i]) + __uint_as_float(v[i]));
          }
          release();
        }
        if (ok) op.store(t, w, sum);
      } else {
        op.prefetch(t, w);
        const uint32_t taddr = take();
        if (!ok) break;
        ok = op.epilogue(t, w, taddr);
        __syncwarp();
        release();
      }
    }
    // the staging outlives the copies in and out of it
    if (lane == 0) ptx::bulk_wait_all();
    for (int i = 0; i < 2; ++i)
      if (w.pending >> i & 1u) w.wait(i);
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the last commit reaches both CTAs: the one that issued it has waited for it
  if (CG == 2 && rank != 0 && warp == 1) ptx::mbar_wait(drain, 0, status, kSiteDrain);
  if constexpr (CG == 2) ptx::cluster_sync();  // no CTA leaves while the other may still signal or read it
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (CG == 2) ptx::tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// soff[0..E] = the experts' row offsets, clamped to [0, M_total]: an expert's
// rows are [soff[e], soff[e + 1]), none where that is empty. Warp-wide.
__device__ __forceinline__ void load_offsets(const int32_t* offsets, int E, int M_total, int32_t* soff) {
  for (int e = threadIdx.x & 31; e <= E; e += 32) soff[e] = min(max(offsets[e], 0), M_total);
  __syncwarp();
}

// tile_start[e] = number of tiles of the experts before e, tiles(e) each;
// tile_start[E] = their total. Warp-wide.
template <class F>
__device__ __forceinline__ void tile_starts(int E, int32_t* tile_start, F tiles) {
  const int lane = threadIdx.x & 31;
  int32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int32_t t = e < E ? tiles(e) : 0;
    int32_t incl = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (e < E) tile_start[e] = carry + incl - t;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) tile_start[E] = carry;
}

// ------------------------------------------------------------------ host
// A row-major [rows, cols] matrix of 16-bit elements (cols contiguous) as an
// operand of which a CTA holds `mn_rows` MN rows a stage: K-major (k = cols) in
// boxes of 64 k by mn_rows rows, or MN-major (mn = cols, a multiple of 64) as
// cols / 64 groups, in boxes of 64 mn by 64 k rows by mn_rows / 64 groups. Rows
// and columns past the matrix read as zeros.
inline bool make_operand(CUtensorMap* m, const void* base, bool bf16, int64_t rows, int64_t cols, bool mn_major,
                         int mn_rows) {
  const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!mn_major) return make_tmap(m, base, dt, 2, cols, rows, mn_rows);
  PFN_encodeTiled enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)(cols * 2), 128};
  cuuint32_t box[3] = {64, 64, (cuuint32_t)(mn_rows / 64)}, estr[3] = {1, 1, 1};
  return enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major [items, rows, cols] tensor for an epilogue warp's boxes: 32 rows by
// row_bytes (64 or 128) of one item. Copies read zeros and write nothing past an
// item's rows and columns.
inline bool make_boxes(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int elem_bytes, int64_t items,
                       int64_t rows, int64_t cols, int row_bytes) {
  PFN_encodeTiled enc = get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)items};
  cuuint64_t strides[2] = {(cuuint64_t)(cols * elem_bytes), (cuuint64_t)(rows * cols * elem_bytes)};
  cuuint32_t box[3] = {(cuuint32_t)(row_bytes / elem_bytes), 32u, 1u}, estr[3] = {1, 1, 1};
  return enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// set_smem once per device (a bit of `sized` each): a fifth of a launch's host time.
template <class K>
inline cudaError_t set_smem_once(std::atomic<uint64_t>& sized, K k, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (sized.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = set_smem(k, bytes);
  if (e == cudaSuccess) sized.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// overlap: the kernel may start (its set-up, up to wait_for_previous_grid)
// while the one ahead of it in the stream still runs.
// (static: were `sized` shared between two copies of this library in a process,
// only one of them would set its kernels' size)
template <class Op, int CG>
static cudaError_t launch(const Maps& maps, const Op& op, int64_t tiles, int32_t* status, cudaStream_t s,
                          bool overlap = false) {
  using C = Cfg<Op, CG>;
  auto k = mm_kernel<Op, CG>;
  static std::atomic<uint64_t> sized{0};
  cudaError_t e = set_smem_once(sized, k, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  cfg.attrs = at;
  if (CG == 2) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = CG;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (overlap) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const int64_t units = std::max<int64_t>(1, std::min<int64_t>(num_sms() / CG, tiles));
  cfg.gridDim = dim3((unsigned)(units * CG));
  e = cudaLaunchKernelEx(&cfg, k, maps, op, status);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

// A plain kernel that starts with wait_for_previous_grid, launched to overlap;
// its blocks in clusters of `cluster`.
template <typename... Par, typename... Arg>
inline cudaError_t launch_overlapped_smem(void (*k)(Par...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                                          unsigned cluster, Arg... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k, static_cast<Par>(args)...);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

template <typename... Par, typename... Arg>
inline cudaError_t launch_overlapped(void (*k)(Par...), dim3 grid, unsigned threads, cudaStream_t s, unsigned cluster,
                                     Arg... args) {
  return launch_overlapped_smem(k, grid, threads, 0, s, cluster, args...);
}

}  // namespace mm
}  // namespace moe
