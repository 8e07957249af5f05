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
//   relu: a = max(g, 0), a' = [g > 0]
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
    a = fmaxf(g, 0.0f);
    da = g > 0.0f ? 1.0f : 0.0f;
  }
}

__device__ __forceinline__ void load_row32(const __nv_bfloat16* src, float (&v)[32]) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 x = __ldg(s + q);
    v[8 * q + 0] = bf16lo_to_f32(x.x);
    v[8 * q + 1] = bf16hi_to_f32(x.x);
    v[8 * q + 2] = bf16lo_to_f32(x.y);
    v[8 * q + 3] = bf16hi_to_f32(x.y);
    v[8 * q + 4] = bf16lo_to_f32(x.z);
    v[8 * q + 5] = bf16hi_to_f32(x.z);
    v[8 * q + 6] = bf16lo_to_f32(x.w);
    v[8 * q + 7] = bf16hi_to_f32(x.w);
  }
}

// Tiles of one expert's rows by 256 columns, in the order of the forward's
// 128-row GEMM: expert, band of m-tiles, n-tile, m-tile. PAIR: 256 rows of a
// pair of SMs, else 128. A k block of a 128-row tile brings 48 KB for 512 cycles
// of MMA (the pair's 32 KB per SM), which at full rate is more than L2 delivers;
// but an expert's last 128 rows or fewer would leave half a pair's tile empty.
// So an expert's rows go to pairs as far as they fill more than half a tile, and
// a remainder of at most 128 rows to single SMs, in a second launch that starts
// as the first one's SMs run out of tiles.
// ACT: the product is the gradient d of h = a(g) u; the epilogue writes
// dg = d u a'(g), du = d a(g) and, with h given, a(g) u.
enum RowSet { kAllRows, kPairRows, kRestRows };

template <int ACT, bool PAIR, bool BOXED>
struct RowGrad {
  static_assert(BOXED || !PAIR, "a pair has the room");
  static constexpr bool kAMn = false, kBMn = true, kTail = false;
  static constexpr int kBN = 256, kFmt = 1, kChunk = 0;
  // BOXED: boxes of 32 x 32 are staged: the result; gated, g and u, which their
  // gradients replace, and h. A pair has room for g and u twice, the next ones on
  // their way; beside a single SM's wider stages there is room for one, and for
  // three stages instead of four. Not BOXED, lanes read and write rows of their
  // own, which touches 32 lines at once and takes as long as the products of about
  // 40 k blocks; so a single SM stages gated tiles where the sum is shorter (64
  // experts' 16384 rows, N = 2048, K = 7168: 822 us in boxes, 1249 without; 256
  // rows, N = K = 4096, bound by the weights: 353 and 327).
  static constexpr int kGu = ACT == kActNone || !BOXED ? 0 : PAIR ? 2 : 1;  // boxes of g and u
  static constexpr int kStageWarp = BOXED ? 2048 + kGu * 4096 : 0;
  static constexpr int kSharedInts = 2 * (gg::kMaxE + 1);
  static constexpr int kRows = PAIR ? 2 * BM : BM;

  const int32_t* offsets;
  int E, M_total, N, K, NT, band;
  RowSet set;
  int parts;    // ranges of n that run as tiles of their own; above 1, single SMs only, and
  float* part;  // their fp32 sums go here, [parts, M_total, K]
  const __nv_bfloat16* gu;  // [M_total, 2K]
  __nv_bfloat16* dA;        // [M_total, K], with ACT [M_total, 2K]
  __nv_bfloat16* h;         // [M_total, K] or nullptr

  // m-tiles of an expert with c rows, and its first row in them
  __device__ __forceinline__ int m_tiles(int c) const {
    if (PAIR) return c / 256 + (c % 256 > 128);
    if (set == kRestRows) return c % 256 >= 1 && c % 256 <= 128;
    return (c + BM - 1) / BM;
  }
  __device__ __forceinline__ int first_row(int c) const { return !PAIR && set == kRestRows ? c / 256 * 256 : 0; }

  __device__ void setup(int32_t* sh) const {
    int32_t* soff = sh + gg::kMaxE + 1;
    load_offsets(offsets, E, M_total, soff);
    tile_starts(E, sh, [&](int e) { return m_tiles(max(soff[e + 1] - soff[e], 0)) * NT; });
  }
  static constexpr bool kParts = !PAIR && ACT == kActNone;
  __device__ int total(const int32_t* sh) const { return sh[E] * (kParts ? parts : 1); }
  __device__ void decode(const int32_t* sh, int tile, Tile& t) const {
    const int32_t* soff = sh + gg::kMaxE + 1;
    t.nkb = N / BK;
    int kb0 = 0;
    if constexpr (kParts) {
      const int p = tile % parts, nkb = t.nkb;
      tile /= parts;
      kb0 = (int)((int64_t)nkb * p / parts);
      t.nkb = (int)((int64_t)nkb * (p + 1) / parts) - kb0;
      t.p[1] = p;
    }
    const int e = gg::find_expert(sh, E, tile);
    const int local = tile - sh[e], c = soff[e + 1] - soff[e];
    const int bsz = band * NT;
    const int b = local / bsz;
    const int rows = min(band, m_tiles(c) - b * band);
    const int l2 = local - b * bsz;
    const int n = l2 / rows, m = b * band + l2 % rows;
    t.a_mn = soff[e] + first_row(c) + m * kRows;
    t.a_k = kb0 * BK;
    t.b_mn = n * kBN;
    t.b_k = e * N + kb0 * BK;
    t.tail = BK;
    t.p[0] = soff[e + 1];
  }
  __device__ __forceinline__ int steps(const Tile& t, const Warp& w) const {
    if (w.row0(t.a_mn) >= t.p[0]) return 0;
    return max(0, min(kBN / 2, K - t.b_mn - w.half * (kBN / 2))) / 32;
  }
  __device__ __forceinline__ void load_gu(const Tile& t, Warp& w, int i) const {
    const int col = t.b_mn + w.half * (kBN / 2) + 32 * i, row0 = w.row0(t.a_mn), slot = kGu == 2 ? i & 1 : 0;
    const uint32_t box = w.base + 2048 + slot * 4096, bar = w.bar + 8 * slot;
    if (w.lane == 0) {
      ptx::mbar_arrive_expect_tx(bar, 4096);
      ptx::tma_load_3d(box, &w.maps->c[1], col, row0, 0, bar);
      ptx::tma_load_3d(box + 2048, &w.maps->c[1], K + col, row0, 0, bar);
    }
    w.pending |= 1u << slot;
  }
  __device__ void prefetch(const Tile& t, Warp& w) const {
    if constexpr (kGu != 0) {
      if (steps(t, w) == 0) return;
      w.free_boxes();
      load_gu(t, w, 0);
    }
  }
  static __device__ __forceinline__ void put_row(uint32_t box, int lane, const float (&v)[32]) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      Warp::put(Warp::at64(box, lane, u),
                make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                           pack_bf16x2(v[8 * u + 4], v[8 * u + 5]), pack_bf16x2(v[8 * u + 6], v[8 * u + 7])));
  }
  static __device__ __forceinline__ void get_row(uint32_t box, int lane, float (&v)[32]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 x = Warp::get(Warp::at64(box, lane, u));
      v[8 * u] = bf16lo_to_f32(x.x), v[8 * u + 1] = bf16hi_to_f32(x.x);
      v[8 * u + 2] = bf16lo_to_f32(x.y), v[8 * u + 3] = bf16hi_to_f32(x.y);
      v[8 * u + 4] = bf16lo_to_f32(x.z), v[8 * u + 5] = bf16hi_to_f32(x.z);
      v[8 * u + 6] = bf16lo_to_f32(x.w), v[8 * u + 7] = bf16hi_to_f32(x.w);
    }
  }
  __device__ bool epilogue(const Tile& t, Warp& w, uint32_t taddr) const {
    const int row0 = w.row0(t.a_mn), row = row0 + w.lane, n = steps(t, w);
    const bool valid = row < t.p[0];
    // a box reaches past the expert's rows: what is past them is not this
    // expert's to write, so each lane stores its own row
    const bool boxed = BOXED && row0 + 32 <= t.p[0];
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int c = w.half * (kBN / 2) + 32 * i, col = t.b_mn + c;
      float d[32];
      if constexpr (ACT == kActNone) {
        load_acc32(taddr + c, d);
        if (kParts && part) {
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(part + ((int64_t)t.p[1] * M_total + row) * K + col);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_float4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
          }
        } else if (boxed) {
          w.free_boxes();
          put_row(w.base, w.lane, d);
          w.publish();
          if (w.lane == 0) {
            ptx::tma_store_3d(&w.maps->c[0], w.base, col, row0, 0);
            ptx::bulk_commit();
          }
        } else if (valid) {
          gg::store_row32(dA + (int64_t)row * K + col, d);
        }
      } else {
        const int slot = kGu == 2 ? i & 1 : 0;
        const int64_t at = (int64_t)row * 2 * K + col;
        const uint32_t box = w.base + 2048 + slot * 4096;
        if constexpr (BOXED) {
          w.free_boxes();
          if (kGu == 2 ? i + 1 < n : i > 0) load_gu(t, w, kGu == 2 ? i + 1 : i);
        }
        load_acc32(taddr + c, d);
        float g[32], u[32];
        if constexpr (BOXED) {
          if (!w.wait(slot)) return false;
          get_row(box, w.lane, g);
          get_row(box + 2048, w.lane, u);
        } else if (valid) {
          load_row32(gu + at, g);
          load_row32(gu + at + K, u);
        }
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          float a, da;
          act_grad<ACT>(g[q], a, da);
          g[q] = d[q] * u[q] * da;
          d[q] *= a;
          u[q] *= a;
        }
        if (boxed) {
          put_row(box, w.lane, g);
          put_row(box + 2048, w.lane, d);
          if (h) put_row(w.base, w.lane, u);
          w.publish();
          if (w.lane == 0) {
            ptx::tma_store_3d(&w.maps->c[0], box, col, row0, 0);
            ptx::tma_store_3d(&w.maps->c[0], box + 2048, K + col, row0, 0);
            if (h) ptx::tma_store_3d(&w.maps->c[2], w.base, col, row0, 0);
            ptx::bulk_commit();
          }
        } else if (valid) {
          gg::store_row32(dA + at, g);
          gg::store_row32(dA + at + K, d);
          if (h) gg::store_row32(h + (int64_t)row * K + col, u);
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
  static constexpr bool kAMn = true, kBMn = true, kTail = true;
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
                                 int max_rows_per_expert, int32_t* status, void* scratch, size_t scratch_bytes,
                                 cudaStream_t s, const char** why) {
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t out_cols = act == kActNone ? K : 2 * (int64_t)K;
  // Pairs where they pay for their second launch, of the experts' last rows: 256
  // rows an expert over many waves of tiles, or 1024 over a few. (us, pairs and
  // singles: 16384 rows of 4 experts, N = K = 4096, 408 and 423; of 64, N = 2048,
  // K = 7168, 588 and 624; 8192 rows of 16, N = 7168, K = 2048, 4 waves, 241 and
  // 208; 4096 of 4, N = K = 4096, 125 and 112; 4096 of 64, 401 and 349.)
  const int most = max_rows_per_expert > 0 ? std::min(max_rows_per_expert, M_total) : M_total;
  const int64_t each = M_total / E, all = ((int64_t)M_total / mm::BM + E / 2) * ceil_div(K, 256);
  const bool many = most > mm::BM && each >= 256 &&
                    (all >= 16 * (int64_t)num_sms() || (each >= 1024 && M_total >= 8192 && all >= 4 * (int64_t)num_sms()));
  const int64_t tiles_ub = ((int64_t)M_total / mm::BM + std::min(M_total, E)) * ceil_div(K, 256);
  const int parts = mm::sum_parts(num_sms(), tiles_ub, N / mm::BK, (int64_t)M_total * K * 4, scratch_bytes);
  const bool pairs = many && parts == 1;
  // (in parts, the tiles' results go to the scratch, by plain stores)
  mm::Maps single = {}, pair = {};
  bool ok = mm::make_operand(&single.a, dC, true, M_total, N, false, mm::BM) &&
            mm::make_operand(&single.b, B, true, (int64_t)E * N, K, true, 256) &&
            mm::make_boxes(&single.c[0], dA, bf16, 2, 1, M_total, out_cols, 64) &&
            (!gu || mm::make_boxes(&single.c[1], gu, bf16, 2, 1, M_total, out_cols, 64)) &&
            (!h || mm::make_boxes(&single.c[2], h, bf16, 2, 1, M_total, K, 64));
  if (pairs) {
    pair = single;
    ok = ok && mm::make_operand(&pair.b, B, true, (int64_t)E * N, K, true, 128);
  }
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  auto go = [&](auto op, auto cg, mm::RowSet set) {
    constexpr int CG = decltype(cg)::value;
    op.offsets = offsets;
    op.E = E;
    op.M_total = M_total;
    op.N = N;
    op.K = K;
    op.NT = (int)ceil_div(K, op.kBN);
    op.band = 16 / CG;
    op.set = set;
    op.parts = parts;
    op.part = parts > 1 ? static_cast<float*>(scratch) : nullptr;
    op.gu = static_cast<const __nv_bfloat16*>(gu);
    op.dA = static_cast<__nv_bfloat16*>(dA);
    op.h = static_cast<__nv_bfloat16*>(h);
    const int64_t tiles = ((int64_t)M_total / op.kRows + std::min(M_total, E)) * op.NT * parts;
    return mm::launch<decltype(op), CG>(CG == 2 ? pair : single, op, tiles, status, s);
  };
  auto both = [&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (parts > 1) {
      cudaError_t e = go(mm::RowGrad<kActNone, false, true>{}, One{}, mm::kAllRows);
      if (e != cudaSuccess) return e;
      const dim3 grid((unsigned)ceil_div(M_total, 8), (unsigned)ceil_div(K, 1024));
      return mm::launch_overlapped(mm::sum_rows_kernel<ACT>, grid, 256, s, 1, static_cast<const float*>(scratch), parts,
                                   offsets, E, M_total, K, static_cast<const __nv_bfloat16*>(gu),
                                   static_cast<__nv_bfloat16*>(dA), static_cast<__nv_bfloat16*>(h));
    }
    if (pairs) {
      cudaError_t e = go(mm::RowGrad<ACT, true, true>{}, Two{}, mm::kPairRows);
      if (e != cudaSuccess) return e;
    }
    const mm::RowSet rows = pairs ? mm::kRestRows : mm::kAllRows;
    return ACT == kActNone || N < 4096 ? go(mm::RowGrad<ACT, false, true>{}, One{}, rows)
                                       : go(mm::RowGrad<ACT, false, ACT == kActNone>{}, One{}, rows);
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
