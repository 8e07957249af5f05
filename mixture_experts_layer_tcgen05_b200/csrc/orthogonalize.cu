// Orthogonalised update of a stack of matrices by Newton-Schulz products, as
// the Muon optimiser makes of a weight's momentum. For each matrix G [rows,
// cols], with p = min(rows, cols) and q = max(rows, cols):
//   X = G / (|G|_F + eps)
//   `steps` times:  A = X X^T,  B = b A + c A^2,  X <- a X + B X     (rows <= cols)
//                   A = X^T X,  B = b A + c A^2,  X <- a X + X B     (rows >  cols)
//   out = scale X
// (the right-sided form is the left-sided one of the transpose; it needs no
// transposed copy, since mm_core.cuh takes operands of either majorness).
//
// Numbers. A step multiplies a small singular value by up to a (3.4445 in
// Muon's polynomial), so five of them multiply a rounding of X that is not in
// X's own row and column space by almost 500. A bf16 or fp16 X loses matrices of
// low rank that way (measured with fp16 X on a rank-4 256 x 256 matrix: 7e-2 of
// the result's norm; bf16 X: 0.5). X is therefore held in 32 bits, as the sum of
// two fp16 halves (22 bits of it, so 500 roundings' worth stays below 1e-4),
// because the upper half is also what the products read: an fp32 X beside its
// fp16 copy moves 12 bytes an element and step, the halves 8 (measured: 32
// matrices of 7168 x 2048 16.9 ms, 18.3 with fp32). The products read the upper
// half alone: A and B multiply X from the side, and the X inside the products
// only meets B, so their roundings turn X's singular vectors by a rounding's
// size and are not multiplied up. fp16's 11 bits there cost 2e-4 to 2e-3 of the
// result's norm over spectra from white to rank 4 (bf16 operands: 3e-3 to
// 1.4e-2), at the same MMA rate. The largest part of that is the diagonal of
// b A + c A^2, which nears b + c while the rest of it nears 0: what its rounding
// takes is kept in fp32 and given back as a factor of X (a fifth to a third
// less). fp16's range holds because everything is stored times s = 2^floor(log2(q)
// / 2): |X|_2 and |A|_2 stay near 1, so entries of X reach from 1 / sqrt(p q) to 1,
// and those of A from 1 / (p sqrt(q)) to 1. Where eps is not small beside |G|_F, X
// starts below that, at rho = |G|_F / (|G|_F + eps) (an expert without rows has a
// momentum that decays past any eps); then 2^-t X is stored, which is near 1, and
// takes b 4^t and c 16^t (step_factors). The norm is summed in fp64.
//
// Three forms: p <= 8 on the FMA units (narrow_kernel), p <= 128 in one launch
// (orthogonalize_short.cuh), and this file's launches over MMA tiles.
//
// Work per step and matrix: p^2 q MACs for A and p^3 for A^2, each symmetric
// and computed for its upper tiles only (the epilogue stores a tile and its
// mirror image), and p^2 q for B X.
#include <cuda_fp16.h>

#include <cmath>

#include "mm_core.cuh"

namespace moe {
namespace mm {

// One stack in flight: nb matrices. The halves of s X (fp16 [nb, mp, np]; the
// upper ones in two buffers in turn), s A and s (b A + c A^2) (fp16 [nb, pp, pp])
// are padded to multiples of 64 in both directions with zeros, which stay zero
// through every step.
struct Stack {
  int nb, rows, cols;    // the caller's matrices
  int mp, np, pp;        // padded rows, cols and min(rows, cols)
  float s, inv_s;        // the operands' scale and its inverse
  float a;
  const void* g;         // [nb, rows, cols] fp32 or bf16
  const float2* inv;     // [nb] 2^-t / (|G|_F + eps) as a power of two and the rest
  const float4* factors; // [nb, steps] of each step (step_factors)
  int step, steps;
  float* rest;           // [nb, pp] what rounding took from the diagonal of b A + c A^2
  __nv_bfloat16* out;    // [nb, rows, cols]
  bool from_g, last;     // the step reads G as its state; it is the last one
  bool vec;              // cols % 8 == 0: rows of g and out in 16-byte units
};

// Two values of s X as pairs of halves: hi rounded to nearest, lo the rest times
// 2^11, which keeps it in fp16's normal range. join gives them back to 22 bits.
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn((x - f.x) * 2048.0f, (y - f.y) * 2048.0f);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ float2 join(uint32_t hi, uint32_t lo) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  return make_float2(fmaf(l.x, 1.0f / 2048.0f, h.x), fmaf(l.y, 1.0f / 2048.0f, h.y));
}

// A bf16 of G. cuda_bf16.h's __ldg is an asm without volatile, which the compiler may
// move ahead of the check that its address is inside. (It did: narrow_kernel's idle
// threads read past the end of a small G, which faults where nothing is mapped.)
__device__ __forceinline__ float ldg_bf16(const void* g, int64_t i) {
  return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(g) + i) << 16);
}

// The products of X with itself (kGram, kPart) or of A with itself (kPoly):
// symmetric results, tiles on and above the diagonal.
// kPart: a tile's sum over k is cut into `parts` ranges that run as tiles of
// their own and leave their fp32 sums in [part, matrix, pp, pp]; sum_parts_kernel
// adds them. One narrow matrix has too few tiles for the GPU otherwise (measured:
// 7168 x 256, two 128 x 128 tiles a side: the update takes 175 us, 127 in 14 parts).
enum SquareMode { kGram, kPart, kPoly };
template <bool MN, SquareMode MODE, int SIDE>
struct Square {
  static constexpr bool POLY = MODE == kPoly;
  static constexpr bool kAMn = MN, kBMn = MN, kTail = false, kVarN = false;
  static constexpr int kBN = SIDE, kFmt = 0, kChunk = 0;
  static constexpr int kStageWarp = POLY ? 8192 : 4096, kSharedInts = 0;

  Stack st;
  int k_rows;          // rows of one matrix in the operand's map
  int nkb, tiles;      // k blocks and tiles of one matrix
  int parts;           // kPart: ranges of k

  __device__ void setup(int32_t*) const {}
  __device__ int total(const int32_t*) const { return st.nb * tiles * (MODE == kPart ? parts : 1); }
  __device__ void decode(const int32_t*, int tile, Tile& t) const {
    int kb0 = 0, kb1 = nkb, part = 0;
    if constexpr (MODE == kPart) {
      part = tile % parts;
      tile /= parts;
      kb0 = (int)((int64_t)nkb * part / parts);
      kb1 = (int)((int64_t)nkb * (part + 1) / parts);
    }
    const int b = tile / tiles, l = tile - b * tiles;
    // column j of tiles holds j + 1 of them
    int j = (int)((sqrtf(1.0f + 8.0f * (float)l) - 1.0f) * 0.5f);
    while (j * (j + 1) / 2 > l) --j;
    while ((j + 1) * (j + 2) / 2 <= l) ++j;
    const int i = l - j * (j + 1) / 2;
    t.p[0] = MODE == kPart ? part * st.nb + b : b;  // the item written
    t.p[1] = i * SIDE;
    t.p[2] = j * SIDE;
    t.a_mn = i * SIDE + (MN ? 0 : b * k_rows);
    t.b_mn = j * SIDE + (MN ? 0 : b * k_rows);
    t.a_k = t.b_k = (MN ? b * k_rows : 0) + kb0 * BK;
    t.nkb = kb1 - kb0;
    t.tail = BK;
  }
  // The staging's boxes of 32 x 32: the tile as it is, its mirror image, and
  // (kPoly) two that s A arrives in; kPart: one box of 32 x 32 fp32.
  __device__ int steps(const Tile& t, const Warp& w) const {
    if (w.row0(t.p[1]) >= st.pp) return 0;
    const int left = st.pp - t.p[2] - w.half * (kBN / 2);  // columns of this half
    return max(0, min(kBN / 2, left)) / 32;
  }
  __device__ void load_gram(const Tile& t, Warp& w, int i) const {
    w.load(i & 1, w.base + 4096 + (i & 1) * 2048, &w.maps->c[1], t.p[2] + w.half * (kBN / 2) + 32 * i,
           w.row0(t.p[1]), t.p[0], 2048);
  }
  __device__ void prefetch(const Tile& t, Warp& w) const {
    if (!POLY || steps(t, w) == 0) return;
    load_gram(t, w, 0);
    w.own = st.factors[(int64_t)t.p[0] * st.steps + st.step];
  }
  __device__ bool epilogue(const Tile& t, Warp& w, uint32_t taddr) const {
    const int row0 = w.row0(t.p[1]), n = steps(t, w), col0 = t.p[2] + w.half * (kBN / 2);
    const bool mirror = t.p[1] != t.p[2];  // a tile on the diagonal holds both halves itself
    const float4 f = w.own;
    const float ci = f.y * st.inv_s;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int col = col0 + 32 * i;
      float v[32];
      if (POLY && i + 1 < n) load_gram(t, w, i + 1);  // its box's values were used two columns of boxes ago
      load_acc32(taddr + w.half * (kBN / 2) + 32 * i, v);
      if constexpr (POLY) {
        if (!w.wait(i & 1)) return false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = Warp::get(Warp::at64(w.base + 4096 + (i & 1) * 2048, w.lane, u));
          const uint32_t p[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&p[j]));
            v[8 * u + 2 * j] = fmaf(f.x, e.x, ci * v[8 * u + 2 * j]);
            v[8 * u + 2 * j + 1] = fmaf(f.x, e.y, ci * v[8 * u + 2 * j + 1]);
          }
        }
      } else if constexpr (MODE == kPart) {
        w.free_boxes();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          Warp::put(Warp::at128(w.base, w.lane, u),
                    make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]), __float_as_uint(v[4 * u + 2]),
                               __float_as_uint(v[4 * u + 3])));
        w.publish();
        if (w.lane == 0) {
          ptx::tma_store_3d(&w.maps->c[0], w.base, col, row0, t.p[0]);
          ptx::bulk_commit();
        }
        continue;
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= st.inv_s;
      }
      if (POLY && col == row0) {
        float d = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == w.lane) d = v[j];
        st.rest[(int64_t)t.p[0] * st.pp + row0 + w.lane] = (d - __half2float(__float2half_rn(d))) * st.inv_s;
      }
      w.free_boxes();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 h = __floats2half2_rn(v[8 * u + 2 * j], v[8 * u + 2 * j + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&h);
          if (mirror) {  // element (row, col + c) goes to (col + c, row): column `lane` of the box's row c
            const int c = 8 * u + 2 * j;
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(Warp::at64(w.base + 2048, c, w.lane >> 3) + (w.lane & 7) * 2),
                         "h"(__half_as_ushort(h.x))
                         : "memory");
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(Warp::at64(w.base + 2048, c + 1, w.lane >> 3) + (w.lane & 7) * 2),
                         "h"(__half_as_ushort(h.y))
                         : "memory");
          }
        }
        Warp::put(Warp::at64(w.base, w.lane, u), make_uint4(o[0], o[1], o[2], o[3]));
      }
      w.publish();
      if (w.lane == 0) {
        ptx::tma_store_3d(&w.maps->c[0], w.base, col, row0, t.p[0]);
        if (mirror) ptx::tma_store_3d(&w.maps->c[0], w.base + 2048, row0, col, t.p[0]);
        ptx::bulk_commit();
      }
    }
    return true;
  }
};

// X <- a X + B X (LEFT) or a X + X B.
template <bool LEFT, int SIDE>
struct Apply {
  static constexpr bool kAMn = false, kBMn = LEFT, kTail = false, kVarN = false;
  static constexpr int kBN = SIDE, kFmt = 0, kChunk = 0;
  static constexpr int kStageWarp = 8192, kSharedInts = 0;

  Stack st;
  int nkb, mt, nt;

  __device__ void setup(int32_t*) const {}
  __device__ int total(const int32_t*) const { return st.nb * mt * nt; }
  __device__ void decode(const int32_t*, int tile, Tile& t) const {
    const int b = tile / (mt * nt), l = tile - b * (mt * nt);
    // neighbours share X's tile (and all of B comes from L2): the right-sided
    // form walks B's columns first, the left-sided one its rows
    const int m = (LEFT ? l % mt : l / nt) * SIDE, n = (LEFT ? l / mt : l % nt) * SIDE;
    t.p[0] = b;
    t.p[1] = m;
    t.p[2] = n;
    t.a_mn = m + b * (LEFT ? st.pp : st.mp);
    t.a_k = 0;
    t.b_mn = n + (LEFT ? 0 : b * st.pp);
    t.b_k = LEFT ? b * st.mp : 0;
    t.nkb = nkb;
    t.tail = BK;
  }
  // The staging: two of 4 KB, each 32 x 32 of the old state (its two halves, or
  // an fp32 G), which the halves of the new one, or the result, replace.
  __device__ int steps(const Tile& t, const Warp& w) const {
    if (w.row0(t.p[1]) >= st.mp) return 0;
    const int left = st.np - t.p[2] - w.half * (kBN / 2);
    return max(0, min(kBN / 2, left)) / 32;
  }
  __device__ void load_state(const Tile& t, Warp& w, int i) const {
    const int col = t.p[2] + w.half * (kBN / 2) + 32 * i, row0 = w.row0(t.p[1]);
    const uint32_t box = w.base + (i & 1) * 4096, bar = w.bar + 8 * (i & 1);
    if (w.lane == 0) {
      ptx::mbar_arrive_expect_tx(bar, 4096);
      ptx::tma_load_3d(box, &w.maps->c[0], col, row0, t.p[0], bar);
      if (!st.from_g) ptx::tma_load_3d(box + 2048, &w.maps->c[1], col, row0, t.p[0], bar);
    }
    w.pending |= 1u << (i & 1);
  }
  __device__ void prefetch(const Tile& t, Warp& w) const {
    if (steps(t, w) == 0) return;
    w.free_boxes();
    load_state(t, w, 0);
    w.own = st.factors[(int64_t)t.p[0] * st.steps + st.step];
  }
  __device__ bool epilogue(const Tile& t, Warp& w, uint32_t taddr) const {
    const int row0 = w.row0(t.p[1]), row = row0 + w.lane, n = steps(t, w), col0 = t.p[2] + w.half * (kBN / 2);
    // v = s (a X + B X), times the step's change of t: the accumulator holds s^2 B X,
    // but for the rest of B's diagonal, which joins a: one of this row (LEFT), or one
    // of each column
    const float4 f = w.own;
    const float inv_s = f.z * st.inv_s;
    const float2 inv = st.from_g ? st.inv[t.p[0]] : make_float2(1.0f, 1.0f);
    const float* rest = st.rest + (int64_t)t.p[0] * st.pp;
    const float a_row = f.z * (LEFT && row < st.pp ? st.a + rest[row] : st.a);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int col = col0 + 32 * i;
      const uint32_t box = w.base + (i & 1) * 4096;
      w.free_boxes();
      if (i + 1 < n) load_state(t, w, i + 1);
      float v[32], x[32];
      load_acc32(taddr + w.half * (kBN / 2) + 32 * i, v);
      if (!w.wait(i & 1)) return false;
      if (st.from_g) {
        const float y = st.s * inv.y;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 g = Warp::get(Warp::at128(box, w.lane, j));
          x[4 * j] = inv.x * __uint_as_float(g.x) * y, x[4 * j + 1] = inv.x * __uint_as_float(g.y) * y;
          x[4 * j + 2] = inv.x * __uint_as_float(g.z) * y, x[4 * j + 3] = inv.x * __uint_as_float(g.w) * y;
        }
        __syncwarp();  // every lane has its row of G: the box may take the halves
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 h = Warp::get(Warp::at64(box, w.lane, u)), l = Warp::get(Warp::at64(box + 2048, w.lane, u));
          const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = join(hw[j], lw[j]);
            x[8 * u + 2 * j] = y.x, x[8 * u + 2 * j + 1] = y.y;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float4 d = make_float4(a_row, a_row, a_row, a_row);
        if constexpr (!LEFT) {
          const float4 r = __ldg(reinterpret_cast<const float4*>(rest + col) + j);
          d = make_float4(f.z * (st.a + r.x), f.z * (st.a + r.y), f.z * (st.a + r.z), f.z * (st.a + r.w));
        }
        v[4 * j] = fmaf(d.x, x[4 * j], inv_s * v[4 * j]);
        v[4 * j + 1] = fmaf(d.y, x[4 * j + 1], inv_s * v[4 * j + 1]);
        v[4 * j + 2] = fmaf(d.z, x[4 * j + 2], inv_s * v[4 * j + 2]);
        v[4 * j + 3] = fmaf(d.w, x[4 * j + 3], inv_s * v[4 * j + 3]);
      }
      if (st.last) {
        const float r = f.w * st.inv_s;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(r * v[8 * u + 2 * j], r * v[8 * u + 2 * j + 1]);
          Warp::put(Warp::at64(box, w.lane, u), make_uint4(o[0], o[1], o[2], o[3]));
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t o[4], l[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) split(v[8 * u + 2 * j], v[8 * u + 2 * j + 1], o[j], l[j]);
          Warp::put(Warp::at64(box, w.lane, u), make_uint4(o[0], o[1], o[2], o[3]));
          Warp::put(Warp::at64(box + 2048, w.lane, u), make_uint4(l[0], l[1], l[2], l[3]));
        }
      }
      if (st.last && !st.vec) {  // rows that a tiled store cannot address: row by row, lane = column
        __syncwarp();
        const int rows = min(32, st.rows - row0);
        __nv_bfloat16* dst = st.out + ((int64_t)t.p[0] * st.rows + row0) * st.cols + col + w.lane;
        if (col + w.lane < st.cols)
          for (int r = 0; r < rows; ++r) {
            unsigned short x;
            asm volatile("ld.shared.b16 %0, [%1];"
                         : "=h"(x)
                         : "r"(Warp::at64(box, r, w.lane >> 3) + (w.lane & 7) * 2)
                         : "memory");
            dst[(int64_t)r * st.cols] = __ushort_as_bfloat16(x);
          }
        __syncwarp();
        continue;
      }
      w.publish();
      if (w.lane == 0) {
        ptx::tma_store_3d(&w.maps->c[2], box, col, row0, t.p[0]);
        if (!st.last) ptx::tma_store_3d(&w.maps->c[1], box + 2048, col, row0, t.p[0]);
        ptx::bulk_commit();
      }
    }
    return true;
  }
};

constexpr int kNormThreads = 256;
constexpr int kNormChunk = 16384;  // elements of a matrix one block sums
constexpr int kNormMost = 512;     // most blocks per matrix

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kNormThreads / 32; ++i) v += part[i];
  return v;
}

// 1 / (|G|_F + eps), from the sum of squares, as x y 2^t. x is a power of two near 1
// / |G|_F: the norm of entries near fp32's largest has an inverse below fp32's
// smallest normal. rho = |G|_F / (|G|_F + eps), and 2^-t rho is in [1/2, 1]; t is
// 0 where that is so without it, and where rho is 0 or NaN.
struct Unit {
  float x, y;
  int t;
  double rho;
};
__device__ __forceinline__ Unit unit_norm(double sum, float eps) {
  const double norm = sqrt(sum);
  const double p2 = norm > 0.0 && isfinite(norm) ? ldexp(1.0, max(-140, min(126, -ilogb(norm)))) : 1.0;
  // (a zero matrix over an eps whose inverse leaves fp32: 0, not 0 times infinity)
  const double y = norm == 0.0 && eps > 0.0f ? 0.0 : 1.0 / (norm * p2 + (double)eps * p2);
  Unit u = {(float)p2, (float)y, 0, norm * p2 * y};
  if (u.rho > 0.0 && u.rho < 0.5) {
    u.t = ilogb(u.rho) + 1;
    u.y = (float)ldexp(y, -u.t);
  }
  return u;
}

constexpr int kMostSteps = 64;  // (of a call, as the entry checks)

// The factors of every step of a matrix that is stored as 2^-t X (and whose A is, so,
// as 4^-t A): b 4^t, c 16^t, 2^(t - t') for the t' of the next step, and scale 2^t,
// which the last one's result takes. t follows a bound of |X|_F up to 0 and no
// further: |X'| <= |a| |X| + |b| |X|^3 + |c| |X|^5. What fp16 loses of a small b A + c
// A^2 is below 2^-25 of X, beside a X. By the block's threads, `put` in any order.
template <class F>
__device__ __forceinline__ void step_factors(const Unit& u, float a, float b, float c, float scale, int steps, F put) {
  if (u.t == 0) {  // most matrices: t stays there
    for (int i = threadIdx.x; i < steps; i += blockDim.x) put(i, make_float4(b, c, 1.0f, scale));
    return;
  }
  if (threadIdx.x != 0) return;
  int t = u.t;
  double bound = u.rho;
  for (int i = 0; i < steps; ++i) {
    const double x2 = bound * bound;
    bound *= fabs((double)a) + x2 * (fabs((double)b) + x2 * fabs((double)c));
    const int next = i == steps - 1 ? t : bound < 0.5 ? max(t, ilogb(bound) + 1) : 0;
    put(i, make_float4((float)ldexp((double)b, 2 * t), (float)ldexp((double)c, 4 * t), (float)ldexp(1.0, t - next),
                       (float)ldexp((double)scale, t)));
    t = next;
  }
}

// part[b][chunk] = the sum of squares of a chunk of matrix b, in fp64 (squares
// of any fp32 value fit, and the sum has no rounding to speak of).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) sumsq_kernel(const T* __restrict__ g, int64_t n, int chunks,
                                                             double* __restrict__ part) {
  ptx::let_next_grid_start();
  ptx::wait_for_previous_grid();
  const int64_t b = blockIdx.y;
  const int64_t per = (n + chunks - 1) / chunks, lo = per * blockIdx.x, hi = min(lo + per, n);
  const T* src = g + b * n;
  double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
  int64_t i = lo + threadIdx.x;
  for (; i + 3 * kNormThreads < hi; i += 4 * kNormThreads) {
    const double v0 = (double)(float)src[i], v1 = (double)(float)src[i + kNormThreads],
                 v2 = (double)(float)src[i + 2 * kNormThreads], v3 = (double)(float)src[i + 3 * kNormThreads];
    s0 += v0 * v0;
    s1 += v1 * v1;
    s2 += v2 * v2;
    s3 += v3 * v3;
  }
  for (; i < hi; i += kNormThreads) {
    const double v = (double)(float)src[i];
    s0 += v * v;
  }
  const double s = block_sum((s0 + s1) + (s2 + s3));
  if (threadIdx.x == 0) part[b * chunks + blockIdx.x] = s;
}

// The upper half of s 2^-t G / (|G|_F + eps), zero in the padding; inv[b] kept for a
// first step that reads G as its state, else (xl given) the lower half too; and the
// steps' factors.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) normalize_kernel(Stack st, const double* __restrict__ part,
                                                                 int chunks, float b_coeff, float c_coeff, float scale,
                                                                 float eps, float2* __restrict__ inv,
                                                                 float4* __restrict__ factors,
                                                                 __half* __restrict__ xh, __half* __restrict__ xl) {
  ptx::let_next_grid_start();
  ptx::wait_for_previous_grid();
  const int64_t b = blockIdx.y;
  double v = 0.0;
  for (int i = threadIdx.x; i < chunks; i += kNormThreads) v += part[b * chunks + i];
  const Unit f = unit_norm(block_sum(v), eps);
  const float p = f.x, r = f.y;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) inv[b] = make_float2(p, r);
    step_factors(f, st.a, b_coeff, c_coeff, scale, st.steps,
                 [&](int i, float4 v) { factors[b * st.steps + i] = v; });
  }
  const T* src = static_cast<const T*>(st.g) + b * st.rows * st.cols;
  const int64_t base = b * st.mp * st.np;
  // odd rows: a warp takes 64 columns of a row at a time, lane = column (with the
  // result's stores likewise: 51 of 198 x 3553, one step, 241 us; eight columns a
  // lane and rows stored by their own lanes 560)
  if (!st.vec) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blocks = st.np / 64;
    for (int64_t u = (int64_t)blockIdx.x * (kNormThreads / 32) + warp; u < (int64_t)st.mp * blocks;
         u += (int64_t)gridDim.x * (kNormThreads / 32)) {
      const int row = (int)(u / blocks), col = (int)(u % blocks) * 64 + lane;
      float x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[j] = row < st.rows && col + 32 * j < st.cols ? p * (float)src[(int64_t)row * st.cols + col + 32 * j] * r * st.s
                                                        : 0.0f;
      uint32_t hi, lo;
      split(x[0], x[1], hi, lo);
      const int64_t at = base + (int64_t)row * st.np + col;
      xh[at] = __ushort_as_half((unsigned short)hi), xh[at + 32] = __ushort_as_half((unsigned short)(hi >> 16));
      if (xl) xl[at] = __ushort_as_half((unsigned short)lo), xl[at + 32] = __ushort_as_half((unsigned short)(lo >> 16));
    }
    return;
  }
  const int vpr = st.np / 8;
  const int64_t vecs = (int64_t)st.mp * vpr;
  for (int64_t i = (int64_t)blockIdx.x * kNormThreads + threadIdx.x; i < vecs;
       i += (int64_t)gridDim.x * kNormThreads) {
    const int row = (int)(i / vpr), col = (int)(i % vpr) * 8;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    if (row < st.rows && col < st.cols) {  // cols is a multiple of 8: all eight or none
      const T* at = src + (int64_t)row * st.cols + col;
      if constexpr (sizeof(T) == 4) {
        const float4 lo = __ldg(reinterpret_cast<const float4*>(at)), hi = __ldg(reinterpret_cast<const float4*>(at) + 1);
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
      } else {
        const uint4 o = __ldg(reinterpret_cast<const uint4*>(at));
        x[0] = bf16lo_to_f32(o.x), x[1] = bf16hi_to_f32(o.x), x[2] = bf16lo_to_f32(o.y), x[3] = bf16hi_to_f32(o.y);
        x[4] = bf16lo_to_f32(o.z), x[5] = bf16hi_to_f32(o.z), x[6] = bf16lo_to_f32(o.w), x[7] = bf16hi_to_f32(o.w);
      }
    }
    uint32_t o[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(p * x[2 * j] * r * st.s, p * x[2 * j + 1] * r * st.s, o[j], l[j]);
    const int64_t at = base + (int64_t)row * st.np + col;
    *reinterpret_cast<uint4*>(xh + at) = make_uint4(o[0], o[1], o[2], o[3]);
    if (xl) *reinterpret_cast<uint4*>(xl + at) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// s A from its parts, added in order: a block takes 32 x 32 elements of one
// matrix's upper tiles and writes them and, off the diagonal tiles, their mirror
// image.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts, int nb, int pp,
                                                        int side, float inv_s, __half* __restrict__ gram) {
  __shared__ float tile[32][33];
  ptx::let_next_grid_start();
  ptx::wait_for_previous_grid();
  const int nblk = pp / 32, r0 = (int)blockIdx.x / nblk * 32, c0 = (int)blockIdx.x % nblk * 32;
  if (c0 / side < r0 / side) return;  // stored by its mirror image
  const int b = (int)blockIdx.y, r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
  const int64_t one = (int64_t)pp * pp, at = b * one + (int64_t)(r0 + r) * pp + c0 + c;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int p = 0; p < parts; ++p) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(part + (int64_t)p * nb * one + at));
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  s.x *= inv_s, s.y *= inv_s, s.z *= inv_s, s.w *= inv_s;
  const __half2 lo = __floats2half2_rn(s.x, s.y), hi = __floats2half2_rn(s.z, s.w);
  *reinterpret_cast<uint2*>(gram + at) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (c0 / side == r0 / side) return;
  tile[r][c] = s.x, tile[r][c + 1] = s.y, tile[r][c + 2] = s.z, tile[r][c + 3] = s.w;
  __syncthreads();
  const __half2 tl = __floats2half2_rn(tile[c][r], tile[c + 1][r]), th = __floats2half2_rn(tile[c + 2][r], tile[c + 3][r]);
  *reinterpret_cast<uint2*>(gram + b * one + (int64_t)(c0 + r) * pp + r0 + c) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&tl), *reinterpret_cast<const uint32_t*>(&th));
}

// Tiles are 256 x 256 of a pair of SMs, or 128 x 128 of one where those are at
// most two for each SM in the largest product (a X + B X): then more SMs, an
// epilogue of half the columns and no pair to set up shorten each launch
// (measured: 7168 x 256 141 us, 178 with pairs; four 2048 x 512 178 and 200; two
// 2048 x 2048, 512 such tiles, 519 and 381).
constexpr int kSms = 148;
inline bool small_tiles(int64_t nb, int64_t mp, int64_t np) {
  return nb * ceil_div(mp, 128) * ceil_div(np, 128) <= 2 * kSms;
}
inline int64_t square_tiles(int64_t pp, int64_t side) { return ceil_div(pp, side) * (ceil_div(pp, side) + 1) / 2; }

// Parts that A's sum is cut into: as many as give every SM (pair) a tile, of at
// least eight k blocks each (7168 x 256: 128 us in 14 parts, 136 in 28), so none
// below 16, which the launch that adds the parts would not pay for, and no more than
// the parts' buffer (at most as large as the stack in fp32) holds. Measured, without
// parts and with: 7168 x 256 175 and 127 us, 2048 x 256 (four parts) 111 and 109.
inline int64_t units_of(int64_t pp, int64_t side) { return kSms / (side / 128) / square_tiles(pp, side); }
inline int64_t gram_parts(int64_t nb, int64_t mp, int64_t np, int64_t pp) {
  const int64_t nkb = std::max(mp, np) / BK;
  const int64_t units = small_tiles(nb, mp, np) ? units_of(pp, 128) : units_of(pp, 256);
  return std::max<int64_t>(1, std::min({units / nb, nkb / 8, mp * np / (pp * pp)}));
}

// Narrow matrices, p <= 8: every step in one launch and in fp32 on the FMA
// units. With so few rows a 64-wide MMA tile is mostly padding, the chain of
// launches is most of the time, and the roundings of A and B have too few
// elements to average out over (3 x 3, six steps: 4e-3 of the result's norm in
// fp16 operands, 1e-6 here). The matrix is q vectors of p numbers, x [q, P] in
// the workspace, P = p rounded up to a power of two, dealt to the threads of one
// block or a cluster of eight. A pass over them takes a step's y = a x + B x and
// sums y y^T, the next step's A; the cluster's blocks read each other's sums and
// add them in the same order. Bound by the latency of a pass's loads.
// Measured, against the MMA tiles: 4 x 4096 17 and 99 us, 16384 x 8 59 and 141,
// 300 of 400 x 8 64 and 262, 8 x 300000 678 and 631: one matrix has eight SMs here
// however long it is; one that long takes this form for its precision.
constexpr int kNarrow = 8, kNarrowThreads = 512, kNarrowCluster = 8;
inline bool narrow(int64_t rows, int64_t cols) { return std::min(rows, cols) <= kNarrow; }

template <int P>
__device__ __forceinline__ void load_vector(const float* src, float (&v)[P]) {
  if constexpr (P == 2) {
    const float2 x = *reinterpret_cast<const float2*>(src);
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < P / 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(src)[i];
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
}

template <int P, int CLUSTER>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    narrow_kernel(const void* __restrict__ g, bool g_f32, int p, int q, bool wide, int steps, float a, float b, float c,
                  float eps, float scale, float* xs, __nv_bfloat16* __restrict__ out) {
  constexpr int PAIRS = P * (P + 1) / 2, WARPS = kNarrowThreads / 32, THREADS = kNarrowThreads * CLUSTER;
  __shared__ double norms[WARPS], norm_of;
  __shared__ float part[WARPS][PAIRS], sum[PAIRS], A[P][P], B[P][P];
  ptx::let_next_grid_start();
  ptx::wait_for_previous_grid();
  const int item = (int)blockIdx.x / CLUSTER, rank = (int)blockIdx.x % CLUSTER;
  const int64_t at = (int64_t)item * p * q;
  const int64_t sp = wide ? q : 1, sq = wide ? 1 : p;  // strides of the short and the long axis
  float* x = xs + (int64_t)item * q * P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = rank * kNarrowThreads + threadIdx.x;
  auto load = [&](int r, int j) {
    const int64_t i = at + r * sp + j * sq;
    return g_f32 ? __ldg(static_cast<const float*>(g) + i) : ldg_bf16(g, i);
  };
  // another block's shared memory, read between two cluster barriers
  auto peer_f32 = [](const float* v, int r) {
    float o;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(ptx::map_to_cta(ptx::smem_addr(v), r)) : "memory");
    return o;
  };
  auto peer_f64 = [](const double* v, int r) {
    double o;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(o) : "r"(ptx::map_to_cta(ptx::smem_addr(v), r)) : "memory");
    return o;
  };
  auto sync = [] {
    if constexpr (CLUSTER > 1) ptx::cluster_sync();
    else __syncthreads();
  };
  double s = 0.0;
  for (int j = first; j < q; j += THREADS)
#pragma unroll
    for (int r = 0; r < P; ++r)
      if (r < p) {
        const double v = load(r, j);
        s += v * v;
      }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) norms[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int u = 0; u < WARPS; ++u) s += norms[u];
    norm_of = s;
  }
  sync();
  s = 0.0;
  for (int r = 0; r < CLUSTER; ++r) s += CLUSTER > 1 ? peer_f64(&norm_of, r) : norm_of;
  const Unit unit = unit_norm(s, eps);
  const float f = unit.x, inv = ldexpf(unit.y, unit.t);  // (fp32 has room for a small X)

  // step -1 takes G; step i < steps - 1 leaves A of the one after it
#pragma unroll 1
  for (int step = -1; step < steps; ++step) {
    float acc[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) acc[i] = 0.0f;
#pragma unroll 2
    for (int j = first; j < q; j += THREADS) {
      float y[P];
      if (step < 0) {
#pragma unroll
        for (int r = 0; r < P; ++r) y[r] = r < p ? f * load(r, j) * inv : 0.0f;
      } else {
        float v[P];
        load_vector<P>(x + (int64_t)j * P, v);
#pragma unroll
        for (int r = 0; r < P; ++r) {
          y[r] = a * v[r];
#pragma unroll
          for (int k = 0; k < P; ++k) y[r] = fmaf(B[r][k], v[k], y[r]);
        }
      }
      if (step == steps - 1) {
#pragma unroll
        for (int r = 0; r < P; ++r)
          if (r < p) out[at + r * sp + j * sq] = __float2bfloat16_rn(scale * y[r]);
      } else {
        int i = 0;
#pragma unroll
        for (int r = 0; r < P; ++r) {
          x[(int64_t)j * P + r] = y[r];
#pragma unroll
          for (int k = 0; k <= r; ++k) {
            acc[i] = fmaf(y[r], y[k], acc[i]);
            ++i;
          }
        }
      }
    }
    if (step == steps - 1) break;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (lane == 0) part[warp][i] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x < PAIRS) {
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < WARPS; ++u) v += part[u][threadIdx.x];
      sum[threadIdx.x] = v;
    }
    sync();
    if (threadIdx.x < P * P) {
      const int r = threadIdx.x / P, k = threadIdx.x % P, i = r >= k ? r * (r + 1) / 2 + k : k * (k + 1) / 2 + r;
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < CLUSTER; ++u) v += CLUSTER > 1 ? peer_f32(&sum[i], u) : sum[i];
      A[r][k] = v;
    }
    sync();  // (the others have read `sum` too)
    if (threadIdx.x < P * P) {
      const int r = threadIdx.x / P, k = threadIdx.x % P;
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < P; ++u) v = fmaf(A[r][u], A[u][k], v);
      B[r][k] = fmaf(b, A[r][k], c * v);
    }
    __syncthreads();
  }
  // (the last peer reads are behind a barrier of every step; with steps >= 1 there was one)
}

}  // namespace mm
}  // namespace moe

#include "orthogonalize_short.cuh"

namespace moe {
namespace mm {

struct OrthPlan {
  int64_t mp, np, pp, chunks;
  int64_t part, inv, factors, rest, xl, xh0, xh1, gram, poly, sums, total;  // byte offsets in the workspace
};

inline OrthPlan orth_plan(int64_t nb, int64_t rows, int64_t cols) {
  OrthPlan p;
  p.mp = align_up(rows, 64);
  p.np = align_up(cols, 64);
  p.pp = std::min(p.mp, p.np);
  p.chunks = std::min<int64_t>(kNormMost, ceil_div(rows * cols, kNormChunk));
  int64_t off = 256;  // the status word
  auto take = [&](int64_t bytes) {
    const int64_t o = off;
    off += align_up(bytes, 256);
    return o;
  };
  p.part = take(nb * p.chunks * 8);
  p.inv = take(nb * 8);
  p.factors = take(nb * kMostSteps * 16);
  p.rest = take(nb * p.pp * 4);
  p.xl = take(nb * p.mp * p.np * 2);
  p.xh0 = take(nb * p.mp * p.np * 2);
  p.xh1 = take(nb * p.mp * p.np * 2);
  p.gram = take(nb * p.pp * p.pp * 2);
  p.poly = take(nb * p.pp * p.pp * 2);
  // room for any batch's parts up to nb matrices
  p.sums = take(std::min(std::max(units_of(p.pp, 128), units_of(p.pp, 256)), nb * (p.mp * p.np / (p.pp * p.pp))) *
                p.pp * p.pp * 4);
  p.total = off;
  return p;
}

}  // namespace mm

int64_t orthogonalize_ws_bytes(int64_t nb, int64_t rows, int64_t cols) {
  return mm::orth_plan(nb, rows, cols).total;
}

// One batch (nb matrices) of the stack (`stack` matrices), as the workspace holds it at once.
static cudaError_t orthogonalize_batch(const void* g, int nb, int stack, int rows, int cols, bool g_f32, int steps,
                                       float a, float b, float c, float eps, float scale, void* out,
                                       char* ws, cudaStream_t s, const char** why) {
  using namespace mm;
  const OrthPlan P = orth_plan(nb, rows, cols);
  Stack st;
  st.nb = nb;
  st.rows = rows;
  st.cols = cols;
  st.mp = (int)P.mp;
  st.np = (int)P.np;
  st.pp = (int)P.pp;
  st.s = std::ldexp(1.0f, (int)std::floor(std::log2((double)std::max(rows, cols)) / 2));
  st.inv_s = 1.0f / st.s;
  st.a = a;
  st.steps = steps;
  st.g = g;
  st.vec = cols % 8 == 0;
  st.out = static_cast<__nv_bfloat16*>(out);
  __half* xl = reinterpret_cast<__half*>(ws + P.xl);
  void* gram = ws + P.gram;
  void* poly = ws + P.poly;
  float2* inv = reinterpret_cast<float2*>(ws + P.inv);
  st.inv = inv;
  float4* factors = reinterpret_cast<float4*>(ws + P.factors);
  st.factors = factors;
  st.rest = reinterpret_cast<float*>(ws + P.rest);
  double* part = reinterpret_cast<double*>(ws + P.part);
  __half* xh[2] = {reinterpret_cast<__half*>(ws + P.xh0), reinterpret_cast<__half*>(ws + P.xh1)};
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  // the first step reads an fp32 G whose rows tiled loads can address itself
  const bool g_state = g_f32 && cols % 4 == 0;
  __half* xl_init = g_state ? nullptr : xl;

  if (narrow(rows, cols)) {
    const int p = std::min(rows, cols), q = std::max(rows, cols);
    auto run = [&](auto pc, auto cc) {
      constexpr int PP = decltype(pc)::value, CLUSTER = decltype(cc)::value;
      return launch_overlapped(narrow_kernel<PP, CLUSTER>, dim3((unsigned)(nb * CLUSTER)), kNarrowThreads, s, CLUSTER, g,
                               g_f32, p, q, rows <= cols, steps, a, b, c, eps, scale,
                               reinterpret_cast<float*>(ws + P.xl), st.out);
    };
    auto sized = [&](auto pc) {
      return q >= 2 * kNarrowThreads ? run(pc, std::integral_constant<int, kNarrowCluster>{})
                                     : run(pc, std::integral_constant<int, 1>{});
    };
    if (p <= 2) return sized(std::integral_constant<int, 2>{});
    if (p <= 4) return sized(std::integral_constant<int, 4>{});
    return sized(std::integral_constant<int, 8>{});
  }
  if (is_short(stack, rows, cols)) {
    ShortArgs args;
    args.g = g;
    args.out = st.out;
    args.status = status;
    args.p = std::min(rows, cols);
    args.q = std::max(rows, cols);
    const int cluster = short_cluster(stack, args.q);
    args.slice = (int)align_up(ceil_div(args.q, cluster), 64);
    args.steps = steps;
    args.own = (int)align_up(ceil_div(args.p, cluster), 8);
    args.g_f32 = g_f32;
    args.wide = rows <= cols;
    args.s = st.s;
    args.inv_s = st.inv_s;
    args.a = a;
    args.b = b;
    args.c = c;
    args.eps = eps;
    args.scale = scale;
    switch (cluster) {
      case 1: return launch_short<1>(args, nb, s);
      case 2: return launch_short<2>(args, nb, s);
      case 4: return launch_short<4>(args, nb, s);
      case 8: return launch_short<8>(args, nb, s);
      default: return launch_short<16>(args, nb, s);
    }
  }
  const dim3 ngrid((unsigned)P.chunks, (unsigned)nb);
  const int64_t vecs = P.mp * P.np / 8;
  const dim3 cgrid((unsigned)std::min<int64_t>(1024, ceil_div(vecs, 4 * kNormThreads)), (unsigned)nb);
  const int64_t n = (int64_t)rows * cols;
  cudaError_t e = cudaSuccess;
  auto norms = [&](auto zero) {
    using T = decltype(zero);
    e = launch_overlapped(sumsq_kernel<T>, ngrid, kNormThreads, s, 1, static_cast<const T*>(g), n, (int)P.chunks, part);
    if (e == cudaSuccess)
      e = launch_overlapped(normalize_kernel<T>, cgrid, kNormThreads, s, 1, st, (const double*)part, (int)P.chunks, b, c,
                            scale, eps, inv, factors, xh[0], xl_init);
  };
  if (g_f32) norms(0.0f);
  else norms(__nv_bfloat16());
  if (e != cudaSuccess) return e;

  const bool left = rows <= cols;
  const CUtensorMapDataType f32t = CU_TENSOR_MAP_DATA_TYPE_FLOAT32, f16t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap xk[2], xmn[2], gk, pk;       // operands: X K-major and MN-major, A and B K-major
  CUtensorMap g_in, xl_io, xh_io[2], g_io, p_out, o_out = {};  // the epilogues' boxes
  // MN rows of an operand in one CTA are 128 either way
  bool ok = make_operand(&gk, gram, false, nb * P.pp, P.pp, false, 128) &&
            make_operand(&pk, poly, false, nb * P.pp, P.pp, false, 128) &&
            make_boxes(&xl_io, xl, f16t, 2, nb, P.mp, P.np, 64) && make_boxes(&g_io, gram, f16t, 2, nb, P.pp, P.pp, 64) &&
            make_boxes(&p_out, poly, f16t, 2, nb, P.pp, P.pp, 64);
  for (int i = 0; i < 2; ++i)
    ok = ok && make_operand(&xk[i], xh[i], false, nb * P.mp, P.np, false, 128) &&
         make_operand(&xmn[i], xh[i], false, nb * P.mp, P.np, true, 128) &&
         make_boxes(&xh_io[i], xh[i], f16t, 2, nb, P.mp, P.np, 64);
  if (g_state) ok = ok && make_boxes(&g_in, g, f32t, 4, nb, rows, cols, 128);
  if (st.vec) ok = ok && make_boxes(&o_out, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, nb, rows, cols, 64);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  const int parts = (int)gram_parts(stack, P.mp, P.np, P.pp);  // of the whole stack: the passes do not change the bits
  float* sums = reinterpret_cast<float*>(ws + P.sums);
  CUtensorMap sums_out = {};
  if (parts > 1 && !make_boxes(&sums_out, sums, f32t, 4, (int64_t)parts * nb, P.pp, P.pp, 128)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  auto run = [&](auto side, auto leftc) {
    constexpr int SIDE = decltype(side)::value, CG = SIDE / BM;
    constexpr bool LEFT = decltype(leftc)::value, MN = !LEFT;
    auto square = [&](auto op, const CUtensorMap& tm, int64_t k, int64_t k_rows, const CUtensorMap& result, int cuts) {
      op.st = st;
      op.k_rows = (int)k_rows;
      op.nkb = (int)(k / BK);
      op.parts = cuts;
      op.tiles = (int)square_tiles(P.pp, SIDE);
      const Maps maps = {tm, tm, tm, {result, g_io, g_io}};
      return launch<decltype(op), CG>(maps, op, (int64_t)nb * op.tiles * cuts, status, s, true);
    };
    for (int i = 0; i < steps; ++i) {
      const int in = i & 1;
      const CUtensorMap& x = LEFT ? xk[in] : xmn[in];
      const int64_t k = LEFT ? P.np : P.mp;
      st.from_g = i == 0 && g_state;
      st.last = i == steps - 1;
      st.step = i;
      cudaError_t e = parts == 1 ? square(Square<MN, kGram, SIDE>{}, x, k, P.mp, g_io, 1)
                                 : square(Square<MN, kPart, SIDE>{}, x, k, P.mp, sums_out, parts);
      if (e == cudaSuccess && parts > 1)
        e = launch_overlapped(sum_parts_kernel, dim3((unsigned)((P.pp / 32) * (P.pp / 32)), (unsigned)nb), 256, s, 1,
                              (const float*)sums, parts, nb, (int)P.pp, SIDE, st.inv_s, reinterpret_cast<__half*>(gram));
      if (e == cudaSuccess) e = square(Square<false, kPoly, SIDE>{}, gk, P.pp, P.pp, p_out, 1);
      if (e != cudaSuccess) return e;
      Apply<LEFT, SIDE> op;
      op.st = st;
      op.nkb = (int)(P.pp / BK);
      op.mt = (int)ceil_div(P.mp, SIDE);
      op.nt = (int)ceil_div(P.np, SIDE);
      const Maps maps = {LEFT ? pk : xk[in], LEFT ? xmn[in] : pk, pk,
                         {st.from_g ? g_in : xh_io[in], xl_io, st.last ? o_out : xh_io[in ^ 1]}};
      e = launch<decltype(op), CG>(maps, op, (int64_t)nb * op.mt * op.nt, status, s, true);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  };
  using Small = std::integral_constant<int, 128>;
  using Pair = std::integral_constant<int, 256>;
  if (small_tiles(stack, P.mp, P.np)) return left ? run(Small{}, std::true_type{}) : run(Small{}, std::false_type{});
  return left ? run(Pair{}, std::true_type{}) : run(Pair{}, std::false_type{});
}

cudaError_t launch_orthogonalize(const void* g, int nb, int rows, int cols, bool g_f32, int steps, float a,
                                 float b, float c, float eps, float scale, void* out, void* ws,
                                 size_t ws_bytes, cudaStream_t s, const char** why) {
  // as many matrices at once as the workspace holds (the caller has checked that one fits)
  int64_t at_once = nb;
  while (at_once > 1 && (size_t)orthogonalize_ws_bytes(at_once, rows, cols) > ws_bytes)
    at_once = std::min<int64_t>(at_once - 1, (int64_t)((double)at_once * ws_bytes / orthogonalize_ws_bytes(at_once, rows, cols)) + 1);
  at_once = std::max<int64_t>(1, std::min<int64_t>(at_once, 65535));
  const size_t in_bytes = (size_t)rows * cols * (g_f32 ? 4 : 2), out_bytes = (size_t)rows * cols * 2;
  for (int64_t i = 0; i < nb; i += at_once) {
    const int n = (int)std::min<int64_t>(at_once, nb - i);
    cudaError_t e = orthogonalize_batch(static_cast<const char*>(g) + i * in_bytes, n, nb, rows, cols, g_f32, steps, a, b,
                                        c, eps, scale, static_cast<char*>(out) + i * out_bytes,
                                        static_cast<char*>(ws), s, why);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
