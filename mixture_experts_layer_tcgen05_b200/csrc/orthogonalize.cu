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
// Numbers. X is held in fp32: a step multiplies a small singular value by up
// to a (3.4445 in Muon's polynomial), so five of them multiply a rounding of X
// that is not in X's own row and column space by almost 500. A bf16 or fp16 X
// loses matrices of low rank that way (measured with fp16 X on a rank-4 256 x
// 256 matrix: 7e-2 of the result's norm; bf16 X: 0.5). The operands of the
// products, though, may be rounded: A and B multiply X from the side, and the
// X inside the products only meets B, so their roundings turn X's singular
// vectors by a rounding's size and are not multiplied up. They are fp16, whose
// 11 bits cost 2e-4 to 2e-3 of the result's norm over spectra from white to
// rank 4 (bf16 operands: 3e-3 to 1.4e-2), at the same MMA rate. fp16's range
// holds because every operand is stored times s = 2^floor(log2(q) / 2): |X|_2
// and |A|_2 stay near 1, so entries of X reach from 1 / sqrt(p q) to 1, and
// those of A from 1 / (p sqrt(q)) to 1. The norm is summed in fp64.
//
// Work per step and matrix: p^2 q MACs for A and p^3 for A^2, each symmetric
// and computed for its upper tiles only (the epilogue stores a tile and its
// mirror image), and p^2 q for B X.
#include <cuda_fp16.h>

#include <cmath>

#include "mm_core.cuh"

namespace moe {
namespace mm {

// One stack in flight: nb matrices. Buffers are padded to multiples of 64 in
// both directions with zeros, which stay zero through every step.
struct Stack {
  int nb, rows, cols;    // the caller's matrices
  int mp, np, pp;        // padded rows, cols and min(rows, cols)
  float s, inv_s;        // the operands' scale and its inverse
  float a, b, c, scale;
  const void* g;         // [nb, rows, cols] fp32 or bf16
  const float* inv;      // [nb] 1 / (|G|_F + eps)
  float* x;              // [nb, mp, np] fp32, after the first step
  __half* xh_in;         // [nb, mp, np] s X
  __half* xh_out;
  __half* gram;          // [nb, pp, pp] s A
  __half* poly;          // [nb, pp, pp] s (b A + c A^2)
  __nv_bfloat16* out;    // [nb, rows, cols]
  bool first, last, g_f32, vec;  // vec: cols % 8 == 0, rows of g and out in 16-byte units
};

__device__ __forceinline__ void store_half32(__half* dst, const float (&v)[32]) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(v[8 * q + 2 * j], v[8 * q + 2 * j + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    d[q] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The products of X with itself (POLY: of A with itself): symmetric results,
// tiles on and above the diagonal.
template <bool MN, bool POLY>
struct Square {
  static constexpr bool kAMn = MN, kBMn = MN, kTail = false;
  static constexpr int kBN = 256, kFmt = 0, kChunk = 0;
  static constexpr int kSharedInts = 0;

  Stack st;
  int k_rows;      // rows of one matrix in the operand's map
  int nkb, bm, tiles;  // tiles of one matrix

  __device__ void setup(int32_t*) const {}
  __device__ int total(const int32_t*) const { return st.nb * tiles; }
  __device__ void decode(const int32_t*, int tile, Tile& t) const {
    const int b = tile / tiles, l = tile - b * tiles;
    // column j of tiles holds (j + 1) r of them, r = 256 / bm
    const int r = kBN / bm;
    int j = (int)((sqrtf(1.0f + 8.0f * (float)l / (float)r) - 1.0f) * 0.5f);
    while (r * j * (j + 1) / 2 > l) --j;
    while (r * (j + 1) * (j + 2) / 2 <= l) ++j;
    const int i = l - r * j * (j + 1) / 2;
    t.p[0] = b;
    t.p[1] = i * bm;
    t.p[2] = j * kBN;
    t.a_mn = i * bm + (MN ? 0 : b * k_rows);
    t.b_mn = j * kBN + (MN ? 0 : b * k_rows);
    t.a_k = t.b_k = MN ? b * k_rows : 0;
    t.nkb = nkb;
    t.tail = BK;
  }
  __device__ void epilogue(const int32_t*, const Tile& t, int rank, int q, int half, int lane, uint32_t taddr,
                           unsigned char*) const {
    const int row0 = t.p[1] + rank * BM + q * 32, row = row0 + lane;
    const int pp = st.pp;
    const int64_t base = (int64_t)t.p[0] * pp * pp;
    __half* dst = (POLY ? st.poly : st.gram) + base;
    const __half* gram = st.gram + base;
    if (row0 >= pp) return;
#pragma unroll 1
    for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2) && t.p[2] + c < pp; c += 32) {
      const int col = t.p[2] + c;
      if (col < row0) continue;  // below the diagonal: its mirror image is stored elsewhere
      float v[32];
      load_acc32(taddr + c, false, v);
      if constexpr (POLY) {
        const float ci = st.c * st.inv_s;
        const uint4* src = reinterpret_cast<const uint4*>(gram + (int64_t)row * pp + col);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = src[u];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[8 * u + 2 * j] = fmaf(st.b, f.x, ci * v[8 * u + 2 * j]);
            v[8 * u + 2 * j + 1] = fmaf(st.b, f.y, ci * v[8 * u + 2 * j + 1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= st.inv_s;
      }
      if (col > row0) {
        store_half32(dst + (int64_t)row * pp + col, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) dst[(int64_t)(col + i) * pp + row] = __float2half_rn(v[i]);
      } else {  // the diagonal block: each element of its upper half, both ways
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const __half h = __float2half_rn(v[i]);
          if (i >= lane) dst[(int64_t)row * pp + col + i] = h;
          if (i > lane) dst[(int64_t)(col + i) * pp + row] = h;
        }
      }
    }
  }
};

// X <- a X + B X (LEFT) or a X + X B.
template <bool LEFT>
struct Apply {
  static constexpr bool kAMn = false, kBMn = LEFT, kTail = false;
  static constexpr int kBN = 256, kFmt = 0, kChunk = 0;
  static constexpr int kSharedInts = 0;

  Stack st;
  int nkb, bm, mt, nt;

  __device__ void setup(int32_t*) const {}
  __device__ int total(const int32_t*) const { return st.nb * mt * nt; }
  __device__ void decode(const int32_t*, int tile, Tile& t) const {
    const int b = tile / (mt * nt), l = tile - b * (mt * nt);
    const int m = (l % mt) * bm, n = (l / mt) * kBN;
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
  __device__ void epilogue(const int32_t*, const Tile& t, int rank, int q, int half, int lane, uint32_t taddr,
                           unsigned char*) const {
    const int row = t.p[1] + rank * BM + q * 32 + lane;
    const bool in = row < st.mp, real = row < st.rows;
    const float f = st.inv_s * st.inv_s;
    const int64_t xrow = ((int64_t)t.p[0] * st.mp + row) * st.np;
    const int64_t grow = ((int64_t)t.p[0] * st.rows + row) * st.cols;
    const float inv = st.first ? st.inv[t.p[0]] : 0.0f;
#pragma unroll 1
    for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2) && t.p[2] + c < st.np; c += 32) {
      const int col = t.p[2] + c;
      float v[32];
      load_acc32(taddr + c, false, v);
      if (!in) continue;
      // x = the old state, 0 outside the matrix
      float x[32];
      if (!st.first) {
        const float4* src = reinterpret_cast<const float4*>(st.x + xrow + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 o = src[i];
          x[4 * i] = o.x, x[4 * i + 1] = o.y, x[4 * i + 2] = o.z, x[4 * i + 3] = o.w;
        }
      } else {
        load_g(grow, col, real, inv, x);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = fmaf(st.a, x[i], f * v[i]);
      if (!st.last) {
        float4* dst = reinterpret_cast<float4*>(st.x + xrow + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= st.s;
        store_half32(st.xh_out + xrow + col, v);
      } else if (real) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= st.scale;
        if (st.vec && col + 32 <= st.cols) {
          gg::store_row32(st.out + grow + col, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < st.cols) st.out[grow + col + i] = __float2bfloat16_rn(v[i]);
        }
      }
    }
  }
  __device__ __forceinline__ void load_g(int64_t grow, int col, bool real, float inv, float (&x)[32]) const {
    if (real && st.vec && col + 32 <= st.cols) {
      if (st.g_f32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(st.g) + grow + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 o = __ldg(src + i);
          x[4 * i] = inv * o.x, x[4 * i + 1] = inv * o.y, x[4 * i + 2] = inv * o.z, x[4 * i + 3] = inv * o.w;
        }
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(st.g) + grow + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 o = __ldg(src + i);
          const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = inv * bf16lo_to_f32(w[j]);
            x[8 * i + 2 * j + 1] = inv * bf16hi_to_f32(w[j]);
          }
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      x[i] = 0.0f;
      if (real && col + i < st.cols)
        x[i] = inv * (st.g_f32 ? static_cast<const float*>(st.g)[grow + col + i]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(st.g)[grow + col + i]));
    }
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

// part[b][chunk] = the sum of squares of a chunk of matrix b, in fp64 (squares
// of any fp32 value fit, and the sum has no rounding to speak of).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) sumsq_kernel(const T* __restrict__ g, int64_t n, int chunks,
                                                             double* __restrict__ part) {
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

// xh = s G / (|G|_F + eps) in fp16, zero in the padding; inv[b] kept for the
// first step. A block writes 32 padded rows by 64 columns... of one matrix.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) normalize_kernel(Stack st, const double* __restrict__ part,
                                                                 int chunks, float eps, float* __restrict__ inv) {
  const int64_t b = blockIdx.y;
  double v = 0.0;
  for (int i = threadIdx.x; i < chunks; i += kNormThreads) v += part[b * chunks + i];
  const float r = (float)(1.0 / (sqrt(block_sum(v)) + (double)eps));
  if (blockIdx.x == 0 && threadIdx.x == 0) inv[b] = r;
  const int vpr = st.np / 8;
  const int64_t vecs = (int64_t)st.mp * vpr;
  const T* src = static_cast<const T*>(st.g) + b * st.rows * st.cols;
  __half* dst = st.xh_in + b * st.mp * st.np;
  for (int64_t i = (int64_t)blockIdx.x * kNormThreads + threadIdx.x; i < vecs;
       i += (int64_t)gridDim.x * kNormThreads) {
    const int row = (int)(i / vpr), col = (int)(i % vpr) * 8;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    if (row < st.rows) {
      const T* p = src + (int64_t)row * st.cols + col;
      if (st.vec && col + 8 <= st.cols) {
        if constexpr (sizeof(T) == 4) {
          const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
          x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
        } else {
          const uint4 o = __ldg(reinterpret_cast<const uint4*>(p));
          x[0] = bf16lo_to_f32(o.x), x[1] = bf16hi_to_f32(o.x), x[2] = bf16lo_to_f32(o.y), x[3] = bf16hi_to_f32(o.y);
          x[4] = bf16lo_to_f32(o.z), x[5] = bf16hi_to_f32(o.z), x[6] = bf16lo_to_f32(o.w), x[7] = bf16hi_to_f32(o.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < st.cols) x[j] = (float)p[j];
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(x[2 * j] * r * st.s, x[2 * j + 1] * r * st.s);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(dst + (int64_t)row * st.np + col) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

struct OrthPlan {
  int64_t mp, np, pp, chunks;
  int64_t part, inv, x, xh0, xh1, gram, poly, total;  // byte offsets in the workspace
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
  p.inv = take(nb * 4);
  p.x = take(nb * p.mp * p.np * 4);
  p.xh0 = take(nb * p.mp * p.np * 2);
  p.xh1 = take(nb * p.mp * p.np * 2);
  p.gram = take(nb * p.pp * p.pp * 2);
  p.poly = take(nb * p.pp * p.pp * 2);
  p.total = off;
  return p;
}

}  // namespace mm

int64_t orthogonalize_ws_bytes(int64_t nb, int64_t rows, int64_t cols) {
  return mm::orth_plan(nb, rows, cols).total;
}

// One batch of the stack that the workspace holds at once.
static cudaError_t orthogonalize_batch(const void* g, int nb, int rows, int cols, bool g_f32, int steps,
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
  st.b = b;
  st.c = c;
  st.scale = scale;
  st.g = g;
  st.g_f32 = g_f32;
  st.vec = cols % 8 == 0;
  st.x = reinterpret_cast<float*>(ws + P.x);
  st.gram = reinterpret_cast<__half*>(ws + P.gram);
  st.poly = reinterpret_cast<__half*>(ws + P.poly);
  st.out = static_cast<__nv_bfloat16*>(out);
  float* inv = reinterpret_cast<float*>(ws + P.inv);
  st.inv = inv;
  double* part = reinterpret_cast<double*>(ws + P.part);
  __half* xh[2] = {reinterpret_cast<__half*>(ws + P.xh0), reinterpret_cast<__half*>(ws + P.xh1)};
  int32_t* status = reinterpret_cast<int32_t*>(ws);

  const dim3 ngrid((unsigned)P.chunks, (unsigned)nb);
  st.xh_in = xh[0];
  const int64_t vecs = P.mp * P.np / 8;
  const dim3 cgrid((unsigned)std::min<int64_t>(1024, ceil_div(vecs, 4 * kNormThreads)), (unsigned)nb);
  const int64_t n = (int64_t)rows * cols;
  if (g_f32) {
    sumsq_kernel<float><<<ngrid, kNormThreads, 0, s>>>(static_cast<const float*>(g), n, (int)P.chunks, part);
    normalize_kernel<float><<<cgrid, kNormThreads, 0, s>>>(st, part, (int)P.chunks, eps, inv);
  } else {
    sumsq_kernel<__nv_bfloat16><<<ngrid, kNormThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(g), n,
                                                               (int)P.chunks, part);
    normalize_kernel<__nv_bfloat16><<<cgrid, kNormThreads, 0, s>>>(st, part, (int)P.chunks, eps, inv);
  }
  note_launch();
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  const bool left = rows <= cols;
  CUtensorMap xk[2], xmn[2], gk, pk;  // X K-major (box 128 rows) and MN-major, A and B K-major
  bool ok = make_operand(&gk, st.gram, false, nb * P.pp, P.pp, 128) &&
            make_operand(&pk, st.poly, false, nb * P.pp, P.pp, 128);
  for (int i = 0; i < 2; ++i)
    ok = ok && make_operand(&xk[i], xh[i], false, nb * P.mp, P.np, 128) &&
         make_operand(&xmn[i], xh[i], false, nb * P.mp, P.np, 64);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  constexpr int CG = 1;
  auto square = [&](auto op, const CUtensorMap& tm, int64_t k, int64_t k_rows) {
    op.st = st;
    op.k_rows = (int)k_rows;
    op.nkb = (int)(k / BK);
    op.bm = BM * CG;
    const int64_t mt = ceil_div(P.pp, op.bm), nt = ceil_div(P.pp, op.kBN), r = op.kBN / op.bm;
    op.tiles = (int)(r * nt * (nt + 1) / 2 - (r * nt - mt));  // the last column may lack its last tile
    return launch<decltype(op), CG>(tm, tm, op, (int64_t)nb * op.tiles, status, s);
  };
  auto apply = [&](auto op, const CUtensorMap& ta, const CUtensorMap& tb) {
    op.st = st;
    op.nkb = (int)(P.pp / BK);
    op.bm = BM * CG;
    op.mt = (int)ceil_div(P.mp, op.bm);
    op.nt = (int)ceil_div(P.np, op.kBN);
    return launch<decltype(op), CG>(ta, tb, op, (int64_t)nb * op.mt * op.nt, status, s);
  };
  for (int i = 0; i < steps; ++i) {
    const int in = i & 1;
    st.xh_in = xh[in];
    st.xh_out = xh[in ^ 1];
    st.first = i == 0;
    st.last = i == steps - 1;
    e = left ? square(Square<false, false>{}, xk[in], P.np, P.mp) : square(Square<true, false>{}, xmn[in], P.mp, P.mp);
    if (e != cudaSuccess) return e;
    e = square(Square<false, true>{}, gk, P.pp, P.pp);
    if (e != cudaSuccess) return e;
    e = left ? apply(Apply<true>{}, pk, xmn[in]) : apply(Apply<false>{}, xk[in], pk);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
    cudaError_t e = orthogonalize_batch(static_cast<const char*>(g) + i * in_bytes, n, rows, cols, g_f32, steps, a, b,
                                        c, eps, scale, static_cast<char*>(out) + i * out_bytes,
                                        static_cast<char*>(ws), s, why);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
