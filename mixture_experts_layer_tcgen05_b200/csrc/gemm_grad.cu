// Gradients of the grouped GEMM (moe_grouped_gemm, bf16): with respect to its
// rows and with respect to the experts' weights. The forward computes, for the
// rows m of expert e, C[m, n] = sum_k A[m, k] B[e, n, k]; so
//   dA[m, k]    = sum_n dC[m, n] B[e, n, k]           (rows of e, summed over n)
//   dB[e, n, k] = sum_{m of e} dC[m, n] A[m, k]       (summed over the rows of e)
// Both read what the forward reads, as it is stored: in dA the weights enter
// with their k index (the product's columns) along memory, in dB both operands
// do, the rows being the summed axis (mm_core.cuh).
#include <cmath>

#include "mm_core.cuh"

namespace moe {
namespace mm {

// ------------------------------------------------------------- row gradient
// The gate's activation a(g) and its derivative.
//   silu: p = 1 / (1 + e^-g), a = g p, a' = p (1 + g (1 - p))
//   gelu: a = g Phi(g), a' = Phi(g) + g phi(g)
//   relu: a = max(g, 0), a' = [g > 0]; both NaN where g is
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float& a, float& da) {
  if constexpr (ACT == kActSilu) {
    const float p = __fdividef(1.0f, 1.0f + __expf(-g));
    a = g * p;
    da = p * (1.0f + g * (1.0f - p));
  } else if constexpr (ACT == kActGelu) {
    // erfc keeps Phi's relative accuracy for negative g, where 1 + erf cancels
    const float p = 0.5f * erfcf(-0.7071067811865476f * g);
    a = g * p;
    da = p + g * 0.3989422804014327f * __expf(-0.5f * g * g);
  } else {
    // (fmaxf would give 0 for a NaN, which the step would train on unseen)
    a = g > 0.0f || g != g ? g : 0.0f;
    da = g > 0.0f ? 1.0f : g != g ? g : 0.0f;
  }
}

// The product with the weights' columns (k, along memory) as the MMA's M and the
// expert's rows as its N, whose size is free: an expert with c rows takes
// ceil(c / kBN) tiles of as many rows each, rounded up to 16. The MMA's time goes
// with N (558 cycles a k block at N = 256, 418 at 192, 345 at 128 and below, where
// issuing it takes longest), so rows past an expert's end cost next to nothing.
// With the rows in M, tiles of 128 made the fine-grained case's MMAs a fifth
// longer. Tiles are 256 columns by up to 256 rows of a pair of SMs, or, for K =
// 128, 128 by up to 128 of one; by up to 64 rows of a pair where the call has at
// most 32 rows per expert on average: reading the weights is all there is to it
// then, and shorter tiles leave room for 8 to 10 stages of them instead of 4 to 6.
// Gated, 64 experts of 4096 x 14336 with 1024 rows: 1116 us so, 1241 with tiles of
// 256; with 4096 rows 1484 and 1400. Order: expert, band of row tiles, column tile, row
// tile, so that pairs that run together share the weights' columns.
// The accumulator's lanes are columns of the result and its columns rows: an
// epilogue warp takes 32 x 32 of it at a time, writes it transposed to a box and
// stores that where the expert has all 32 rows, else row by row. Gated, the fp32
// product is turned first, half of it at a time, so that g, u and what becomes of
// them are read and written 16 bytes a lane: 2 bytes a lane took 173 us for 1024 x
// 1024 and 16384 rows of 64 experts, this 70.
// ACT: the product is the gradient d of h = a(g) u; the epilogue writes
// dg = d u a'(g), du = d a(g) and, with h given, a(g) u.
template <int ACT, int CG, int BN>
struct RowGrad {
  static constexpr bool kAMn = true, kBMn = false, kTail = false, kVarN = true;
  static constexpr int kBN = BN, kCols = BM * CG, kFmt = 1, kChunk = 0;
  // Boxes of 32 x 32 are staged: the result; gated, the product while it is turned,
  // whose place h takes, and two of g and u each (the next ones on their way; tiles
  // of 64 rows have one only), which their gradients replace.
  static constexpr int kStageWarp = ACT == kActNone ? 2048 : 2048 + 4096 * (BN > 64 ? 2 : 1);
  static constexpr int kSharedInts = 2 * (gg::kMaxE + 1);
  static constexpr int kBand = 8;

  const int32_t* offsets;
  int E, M_total, N, K, NT;
  int parts;    // ranges of n that run as tiles of their own; above 1,
  float* part;  // their fp32 sums go here, [parts, M_total, K] (ACT none)
  __nv_bfloat16* dA;        // [M_total, K], with ACT [M_total, 2K]
  __nv_bfloat16* h;         // [M_total, K] or nullptr

  __device__ void setup(int32_t* sh) const {
    int32_t* soff = sh + gg::kMaxE + 1;
    load_offsets(offsets, E, M_total, soff);
    tile_starts(E, sh, [&](int e) { return (max(soff[e + 1] - soff[e], 0) + kBN - 1) / kBN * NT; });
  }
  __device__ int total(const int32_t* sh) const { return sh[E] * (ACT == kActNone ? parts : 1); }
  __device__ void decode(const int32_t* sh, int tile, Tile& t) const {
    const int32_t* soff = sh + gg::kMaxE + 1;
    t.nkb = N / BK;
    int kb0 = 0;
    if constexpr (ACT == kActNone) {
      const int p = tile % parts, nkb = t.nkb;
      tile /= parts;
      kb0 = (int)((int64_t)nkb * p / parts);
      t.nkb = (int)((int64_t)nkb * (p + 1) / parts) - kb0;
      t.p[1] = p;
    }
    const int e = gg::find_expert(sh, E, tile);
    const int local = tile - sh[e], c = soff[e + 1] - soff[e];
    const int mt = (c + kBN - 1) / kBN, each = ((c + mt - 1) / mt + 15) / 16 * 16;
    const int bsz = kBand * NT;
    const int b = local / bsz;
    const int rows = min(kBand, mt - b * kBand);
    const int l2 = local - b * bsz;
    const int n = l2 / rows, m = b * kBand + l2 % rows;
    t.a_mn = n * kCols;
    t.a_k = e * N + kb0 * BK;
    t.b_mn = soff[e] + m * each;
    t.b_k = kb0 * BK;
    t.n = each;
    t.tail = BK;
    t.p[0] = min(each, c - m * each);  // rows of the tile
  }
  // this warp's 32 columns, and its share of the tile's groups of 32 rows: every other one
  __device__ __forceinline__ int col0(const Tile& t, const Warp& w) const { return t.a_mn + w.rank * BM + w.q * 32; }
  __device__ __forceinline__ int steps(const Tile& t, const Warp& w) const {
    return col0(t, w) < K ? ((t.p[0] + 31) / 32 - w.half + 1) / 2 : 0;
  }
  __device__ __forceinline__ void load_gu(const Tile& t, Warp& w, int i) const {
    const int row = t.b_mn + 32 * (2 * i + w.half), col = col0(t, w);
    const uint32_t box = w.base + 2048 + (i & 1) * 4096, bar = w.bar + 8 * (i & 1);
    if (w.lane == 0) {
      ptx::mbar_arrive_expect_tx(bar, 4096);
      ptx::tma_load_3d(box, &w.maps->c[1], col, row, 0, bar);
      ptx::tma_load_3d(box + 2048, &w.maps->c[1], K + col, row, 0, bar);
    }
    w.pending |= 1u << (i & 1);
  }
  __device__ void prefetch(const Tile& t, Warp& w) const {
    if constexpr (ACT != kActNone) {
      if (steps(t, w) == 0) return;
      w.free_boxes();
      load_gu(t, w, 0);
    }
  }
  // element (row r, this lane's column) of a box
  static __device__ __forceinline__ uint32_t at(uint32_t box, int r, int lane) {
    return Warp::at64(box, r, lane >> 3) + (lane & 7) * 2;
  }
  static __device__ __forceinline__ void put(uint32_t addr, float v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(__float2bfloat16_rn(v))) : "memory");
  }
  // Gated, a lane holds columns 16 (lane & 1) .. + 15 of the rows lane / 2 and
  // 16 + lane / 2 of 32 x 32: pieces of 8 columns, p of the first row and p - 2 of the
  // second, which for eight lanes are spread over all banks.
  static __device__ __forceinline__ uint32_t piece(uint32_t box, int lane, int p) {
    return Warp::at64(box, lane / 2 + p / 2 * 16, (lane & 1) * 2 + p % 2);
  }
  static __device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ void put_half(uint32_t box, int lane, const float (&v)[32]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) Warp::put(piece(box, lane, p), pack8(v + 8 * p));
  }
  static __device__ __forceinline__ void get_half(uint32_t box, int lane, float (&v)[32]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint4 x = Warp::get(piece(box, lane, p));
      v[8 * p] = bf16lo_to_f32(x.x), v[8 * p + 1] = bf16hi_to_f32(x.x);
      v[8 * p + 2] = bf16lo_to_f32(x.y), v[8 * p + 3] = bf16hi_to_f32(x.y);
      v[8 * p + 4] = bf16lo_to_f32(x.z), v[8 * p + 5] = bf16hi_to_f32(x.z);
      v[8 * p + 6] = bf16lo_to_f32(x.w), v[8 * p + 7] = bf16hi_to_f32(x.w);
    }
  }
  // v[r] of the lane's column becomes what the lane holds of its two rows
  static __device__ __forceinline__ void turn(uint32_t box, int lane, float (&v)[32]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p) __syncwarp();
#pragma unroll
      for (int r = 0; r < 16; ++r)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(Warp::at128(box, r, lane >> 2) + (lane & 3) * 4),
                     "f"(v[16 * p + r])
                     : "memory");
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = Warp::get(Warp::at128(box, lane / 2, (lane & 1) * 4 + j));
        v[16 * p + 4 * j] = __uint_as_float(x.x), v[16 * p + 4 * j + 1] = __uint_as_float(x.y);
        v[16 * p + 4 * j + 2] = __uint_as_float(x.z), v[16 * p + 4 * j + 3] = __uint_as_float(x.w);
      }
    }
  }
  __device__ bool epilogue(const Tile& t, Warp& w, uint32_t taddr) const {
    const int n = steps(t, w), col = col0(t, w) + w.lane;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int r0 = 32 * (2 * i + w.half), row0 = t.b_mn + r0, rows = min(32, t.p[0] - r0);
      float d[32];
      if constexpr (ACT == kActNone) {
        load_acc32(taddr + r0, d);
        if (part) {
          float* dst = part + ((int64_t)t.p[1] * M_total + row0) * K + col;
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (r < rows) dst[(int64_t)r * K] = d[r];
        } else if (rows == 32) {
          w.free_boxes();
#pragma unroll
          for (int r = 0; r < 32; ++r) put(at(w.base, r, w.lane), d[r]);
          w.publish();
          if (w.lane == 0) {
            ptx::tma_store_3d(&w.maps->c[0], w.base, col, row0, 0);
            ptx::bulk_commit();
          }
        } else {
          __nv_bfloat16* dst = dA + (int64_t)row0 * K + col;
#pragma unroll
          for (int r = 0; r < 32; ++r)
            if (r < rows) dst[(int64_t)r * K] = __float2bfloat16_rn(d[r]);
        }
      } else {
        const uint32_t gbox = w.base + 2048 + (i & 1) * 4096, ubox = gbox + 2048;
        w.free_boxes();
        if (i + 1 < n) load_gu(t, w, i + 1);
        load_acc32(taddr + r0, d);
        turn(w.base, w.lane, d);
        float g[32], u[32];
        if (!w.wait(i & 1)) return false;
        get_half(gbox, w.lane, g);
        get_half(ubox, w.lane, u);
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          float a, da;
          act_grad<ACT>(g[q], a, da);
          g[q] = d[q] * u[q] * da;
          d[q] *= a;
          u[q] *= a;
        }
        const int c0 = col - w.lane;
        if (rows == 32) {
          __syncwarp();  // every lane has its part of d: h takes its place
          put_half(gbox, w.lane, g);
          put_half(ubox, w.lane, d);
          if (h) put_half(w.base, w.lane, u);
          w.publish();
          if (w.lane == 0) {
            ptx::tma_store_3d(&w.maps->c[0], gbox, c0, row0, 0);
            ptx::tma_store_3d(&w.maps->c[0], ubox, K + c0, row0, 0);
            if (h) ptx::tma_store_3d(&w.maps->c[2], w.base, c0, row0, 0);
            ptx::bulk_commit();
          }
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int r = w.lane / 2 + p / 2 * 16, c = c0 + (w.lane & 1) * 16 + p % 2 * 8;
            if (r >= rows) continue;
            __nv_bfloat16* dst = dA + (int64_t)(row0 + r) * 2 * K + c;
            *reinterpret_cast<uint4*>(dst) = pack8(g + 8 * p);
            *reinterpret_cast<uint4*>(dst + K) = pack8(d + 8 * p);
            if (h) *reinterpret_cast<uint4*>(h + (int64_t)(row0 + r) * K + c) = pack8(u + 8 * p);
          }
        }
      }
    }
    return true;
  }
};

// The row gradient from its parts, added in order: a warp per row, 256 columns a
// block step. Rows of no expert are left alone.
template <int ACT>
__global__ void __launch_bounds__(256)
    sum_rows_kernel(const float* __restrict__ part, int parts, const int32_t* __restrict__ offsets, int E, int M_total,
                    int K, const __nv_bfloat16* __restrict__ gu, __nv_bfloat16* __restrict__ dA,
                    __nv_bfloat16* __restrict__ h) {
  ptx::wait_for_previous_grid();
  const int row = (int)blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= M_total) return;
  bool mine = false;
  for (int e = lane; e < E; e += 32) mine |= __ldg(offsets + e) <= row && row < __ldg(offsets + e + 1);
  if (!__any_sync(0xffffffffu, mine)) return;
  const int64_t slice = (int64_t)M_total * K;
  for (int col = ((int)blockIdx.y * 32 + lane) * 8; col < K; col += (int)gridDim.y * 256) {
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = 0.0f;
    const float* src = part + (int64_t)row * K + col;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float4 lo = __ldg(reinterpret_cast<const float4*>(src + p * slice));
      const float4 hi = __ldg(reinterpret_cast<const float4*>(src + p * slice) + 1);
      d[0] += lo.x, d[1] += lo.y, d[2] += lo.z, d[3] += lo.w;
      d[4] += hi.x, d[5] += hi.y, d[6] += hi.z, d[7] += hi.w;
    }
    auto store = [](__nv_bfloat16* dst, const float (&v)[8]) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    };
    if constexpr (ACT == kActNone) {
      store(dA + (int64_t)row * K + col, d);
    } else {
      const int64_t at = (int64_t)row * 2 * K + col;
      const uint4 gv = __ldg(reinterpret_cast<const uint4*>(gu + at)), uv = __ldg(reinterpret_cast<const uint4*>(gu + at + K));
      const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w};
      float dg[8], hv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = i & 1 ? bf16hi_to_f32(gw[i / 2]) : bf16lo_to_f32(gw[i / 2]);
        const float u = i & 1 ? bf16hi_to_f32(uw[i / 2]) : bf16lo_to_f32(uw[i / 2]);
        float a, da;
        act_grad<ACT>(g, a, da);
        dg[i] = d[i] * u * da;
        d[i] *= a;
        hv[i] = a * u;
      }
      store(dA + at, dg);
      store(dA + at + K, d);
      if (h) store(h + (int64_t)row * K + col, hv);
    }
  }
}

// ----------------------------------------------------------- weight gradient
// Tiles of 128 CG by 256 of one expert's [N, K] gradient, summed over its rows.
// Experts without rows get zeros (or are left as they are when adding).
template <bool F32, bool ADD>
struct WeightGrad {
  static constexpr bool kAMn = true, kBMn = true, kTail = true, kVarN = false;
  static constexpr int kBN = 256, kFmt = 1, kChunk = F32 ? 12 : 64;
  static constexpr int kStageWarp = 2048, kSharedInts = gg::kMaxE + 1;

  const int32_t* offsets;
  int E, M_total, N, K, mt, nt, bm;
  int parts;  // ranges of rows that run as tiles of their own; above 1, their fp32 sums are items part * E + e

  __device__ void setup(int32_t* sh) const {
    load_offsets(offsets, E, M_total, sh);
  }
  static constexpr bool kParts = F32 && !ADD;
  __device__ int total(const int32_t*) const { return E * mt * nt * (kParts ? parts : 1); }
  __device__ void decode(const int32_t* sh, int tile, Tile& t) const {
    int p = 0;
    if constexpr (kParts) {
      p = tile % parts;
      tile /= parts;
    }
    const int e = tile / (mt * nt), l = tile - e * (mt * nt);
    const int lo = sh[e], rows = max(sh[e + 1] - lo, 0);
    t.a_mn = (l % mt) * bm;
    t.b_mn = (l / mt) * kBN;
    t.a_k = t.b_k = lo;
    t.nkb = (rows + BK - 1) / BK;
    t.tail = rows - (t.nkb - 1) * BK;
    t.p[0] = e;
    if (kParts && parts > 1) {
      const int kb0 = (int)((int64_t)t.nkb * p / parts), kb1 = (int)((int64_t)t.nkb * (p + 1) / parts);
      if (kb1 < t.nkb) t.tail = BK;
      t.a_k = t.b_k = lo + kb0 * BK;
      t.nkb = kb1 - kb0;
      t.p[0] = p * E + e;
    }
  }
  __device__ void store(const Tile& t, Warp& w, const uint32_t (&d)[kBN / 2]) const {
    const int n = w.row0(t.a_mn), col = t.b_mn + w.half * (kBN / 2);
    if (n >= N || col >= K || (ADD && t.nkb == 0)) return;  // all or none of the warp
    constexpr int PER = F32 ? 16 : 32;  // columns of a box
#pragma unroll
    for (int c = 0; c < kBN / 2; c += PER) {
      w.free_boxes();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          const uint32_t* v = d + c + 4 * j;
          Warp::put(Warp::at64(w.base, w.lane, j), make_uint4(v[0], v[1], v[2], v[3]));
        } else {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_bf16x2(__uint_as_float(d[c + 8 * j + 2 * i]), __uint_as_float(d[c + 8 * j + 2 * i + 1]));
          Warp::put(Warp::at64(w.base, w.lane, j), make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
      w.publish();
      if (w.lane == 0) {
        if constexpr (ADD) ptx::tma_add_3d(&w.maps->c[0], w.base, col + c, n, t.p[0]);
        else ptx::tma_store_3d(&w.maps->c[0], w.base, col + c, n, t.p[0]);
        ptx::bulk_commit();
      }
    }
  }
};

// The weight gradient from its parts, added in order (and to dB's values).
template <bool F32, bool ADD>
__global__ void __launch_bounds__(256) sum_weights_kernel(const float4* __restrict__ part, int parts, int64_t n4,
                                                          void* __restrict__ dB) {
  ptx::wait_for_previous_grid();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float4 v = __ldg(part + p * n4 + i);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  if constexpr (F32) {
    float4* dst = static_cast<float4*>(dB) + i;
    if constexpr (ADD) {
      const float4 o = *dst;
      s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
    }
    *dst = s;
  } else {
    static_cast<uint2*>(dB)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// Parts that a long sum of nkb k blocks is cut into where its tiles are fewer
// than the SMs (pairs): as many as there are SMs for, of at least 8 k blocks,
// and no more than the scratch holds; none below 32 k blocks, which the launch
// that adds them would not pay for (measured: 4 experts' 100 rows, gated, K =
// 512: N = 7168 in parts 26 us, without 49; N = 2048 25 and 25; one expert's
// 16384 rows to 512 x 1024 30 and 87).
inline int sum_parts(int64_t units, int64_t tiles, int64_t nkb, int64_t part_bytes, size_t scratch_bytes) {
  if (nkb < 32) return 1;
  const int64_t p = std::min({units / std::max<int64_t>(tiles, 1), nkb / 8, (int64_t)scratch_bytes / part_bytes});
  return (int)std::max<int64_t>(1, p);
}

}  // namespace mm

cudaError_t launch_grouped_dgrad(const void* dC, const void* B, const int32_t* offsets, int M_total,
                                 int E, int N, int K, int act, const void* gu, void* dA, void* h,
                                 int32_t* status, void* scratch, size_t scratch_bytes, cudaStream_t s,
                                 const char** why) {
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t out_cols = act == kActNone ? K : 2 * (int64_t)K;
  const int cg = K > 128 ? 2 : 1, cols = mm::BM * cg;
  const int bn = cg == 2 && M_total <= 32 * (int64_t)E ? 64 : 128 * cg;  // (RowGrad says why)
  const int64_t tiles = ((int64_t)M_total / bn + std::min(M_total, E)) * ceil_div(K, cols);  // at most
  const int parts = mm::sum_parts(num_sms() / cg, tiles, N / mm::BK, (int64_t)M_total * K * 4, scratch_bytes);
  mm::Maps maps = {};
  if (!mm::make_operand(&maps.a, B, true, (int64_t)E * N, K, true, mm::BM) ||
      !mm::make_operand(&maps.b, dC, true, M_total, N, false, bn / cg) ||
      !mm::make_operand(&maps.b_few, dC, true, M_total, N, false, mm::kFew) ||
      !mm::make_boxes(&maps.c[0], dA, bf16, 2, 1, M_total, out_cols, 64) ||
      (gu && !mm::make_boxes(&maps.c[1], gu, bf16, 2, 1, M_total, out_cols, 64)) ||
      (h && !mm::make_boxes(&maps.c[2], h, bf16, 2, 1, M_total, K, 64))) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  auto go = [&](auto op, auto cg_c) {
    constexpr int CG = decltype(cg_c)::value;
    op.offsets = offsets;
    op.E = E;
    op.M_total = M_total;
    op.N = N;
    op.K = K;
    op.NT = (int)ceil_div(K, op.kCols);
    op.parts = parts;
    op.part = parts > 1 ? static_cast<float*>(scratch) : nullptr;
    op.dA = static_cast<__nv_bfloat16*>(dA);
    op.h = static_cast<__nv_bfloat16*>(h);
    return mm::launch<decltype(op), CG>(maps, op, tiles * parts, status, s);
  };
  auto both = [&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    auto product = [&](auto a) {
      constexpr int A = decltype(a)::value;
      return bn == 64  ? go(mm::RowGrad<A, 2, 64>{}, Two{})
             : cg == 2 ? go(mm::RowGrad<A, 2, 256>{}, Two{})
                       : go(mm::RowGrad<A, 1, 128>{}, One{});
    };
    if (parts == 1) return product(act_c);
    cudaError_t e = product(std::integral_constant<int, kActNone>{});
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)ceil_div(M_total, 8), (unsigned)ceil_div(K, 1024));
    return mm::launch_overlapped(mm::sum_rows_kernel<ACT>, grid, 256, s, 1, static_cast<const float*>(scratch), parts,
                                 offsets, E, M_total, K, static_cast<const __nv_bfloat16*>(gu),
                                 static_cast<__nv_bfloat16*>(dA), static_cast<__nv_bfloat16*>(h));
  };
  switch (act) {
    case kActSilu: return both(std::integral_constant<int, kActSilu>{});
    case kActGelu: return both(std::integral_constant<int, kActGelu>{});
    case kActRelu: return both(std::integral_constant<int, kActRelu>{});
    default: return both(std::integral_constant<int, kActNone>{});
  }
}

cudaError_t launch_grouped_wgrad(const void* dC, const void* A, const int32_t* offsets, int M_total,
                                 int E, int N, int K, bool f32, bool add, void* dB, int32_t* status,
                                 void* scratch, size_t scratch_bytes, cudaStream_t s, const char** why) {
  mm::Maps maps = {};
  // A pair's tile is 256 rows of dB: with N = 128 half of it would be empty.
  const int pair = N > 128 ? 2 : 1;
  const int64_t tiles = (int64_t)E * ceil_div(N, mm::BM * pair) * ceil_div(K, 256), n = (int64_t)E * N * K;
  // (the rows an expert has are known on the device only: as if they were spread evenly)
  const int parts = mm::sum_parts(num_sms() / pair, tiles, M_total / mm::BK / E, n * 4, scratch_bytes);
  const bool wide = f32 || parts > 1;
  if (!mm::make_operand(&maps.a, dC, true, M_total, N, true, mm::BM) ||
      !mm::make_operand(&maps.b, A, true, M_total, K, true, 256 / pair) ||
      !mm::make_boxes(&maps.c[0], parts > 1 ? scratch : dB,
                      wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, wide ? 4 : 2,
                      (int64_t)parts * E, N, K, 64)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  auto go = [&](auto op, auto cg) {
    constexpr int CG = decltype(cg)::value;
    op.offsets = offsets;
    op.E = E;
    op.M_total = M_total;
    op.N = N;
    op.K = K;
    op.bm = mm::BM * CG;
    op.mt = (int)ceil_div(N, op.bm);
    op.nt = (int)ceil_div(K, op.kBN);
    op.parts = parts;
    return mm::launch<decltype(op), CG>(maps, op, tiles * parts, status, s);
  };
  auto any = [&](auto op) {
    return pair == 2 ? go(op, std::integral_constant<int, 2>{}) : go(op, std::integral_constant<int, 1>{});
  };
  if (parts > 1) {
    cudaError_t e = any(mm::WeightGrad<true, false>{});
    if (e != cudaSuccess) return e;
    auto sum = f32 ? add ? mm::sum_weights_kernel<true, true> : mm::sum_weights_kernel<true, false>
                   : mm::sum_weights_kernel<false, false>;
    return mm::launch_overlapped(sum, dim3((unsigned)ceil_div(n / 4, 256)), 256, s, 1,
                                 static_cast<const float4*>(scratch), parts, n / 4, dB);
  }
  return !f32 ? any(mm::WeightGrad<false, false>{})
              : add ? any(mm::WeightGrad<true, true>{}) : any(mm::WeightGrad<true, false>{});
}

}  // namespace moe
