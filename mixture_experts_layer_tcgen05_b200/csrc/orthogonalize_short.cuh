// Newton-Schulz products of matrices whose shorter side is at most 128, every
// step in one launch: a cluster of CTAs keeps a matrix on chip. (Numbers as in
// orthogonalize.cu: X times s in two fp16 halves, the upper one the products'.)
//
// The matrix is p <= 128 rows of q numbers (the transpose of one with more rows
// than columns), its columns dealt to the cluster, `slice` to a CTA. The upper
// halves are in shared memory, in blocks of 64 columns: 128 rows of 128 bytes,
// swizzled. Both products read that one copy, A = X X^T with the columns as k
// (K-major), B X with the rows as k (MN-major). The lower halves are in TMEM,
// two columns of X to a TMEM column. A step:
//   - the CTA's part of A by MMA, in fp32 to shared memory; cluster barrier;
//     each CTA adds 128 / C rows of the parts, in order, and writes them as fp16
//     into the A of every CTA; cluster barrier;
//   - A^2 by MMA and B = b A + c A^2 in every CTA alike, over its own part of A;
//   - B X by MMA, 128 columns at a time into two accumulators in turn, and
//     X <- a X + B X in place: a chunk's MMAs read that chunk's columns alone.
// Bound by latency: the MMAs are a tenth of the time, the rest waits for them, the
// barriers and the other CTAs' shared memory. @T
#pragma once

#include <cuda_fp16.h>

#include "mm_core.cuh"

namespace moe {
namespace mm {

constexpr int kShort = 128, kShortSlice = 512, kShortThreads = 256, kShortMost = 8;  // p, columns of a CTA, CTAs
constexpr size_t kShortSmem = 1024 + kShortSlice * 256 + 3 * 32768;  // X, A, and the part of A that B replaces
constexpr int kShortLow = 256;  // TMEM: two accumulators of 128 columns, then the lower halves

struct ShortArgs {
  const void* g;         // [nb, p, q], or [nb, q, p] where not wide; fp32 or bf16
  __nv_bfloat16* out;    // likewise
  int32_t* status;
  int p, q, slice, steps;
  bool g_f32, wide;
  float s, inv_s, a, b, c, eps, scale;
};

// byte of 16-byte piece j (8 columns) of row r, in blocks of 64 columns
__device__ __forceinline__ uint32_t short_at(uint32_t base, int r, int j) {
  return base + (j >> 3) * 16384 + r * 128 + (((j ^ r) & 7) << 4);
}
// byte of 16-byte piece j (4 columns) of row r of the part of A
__device__ __forceinline__ uint32_t short_part_at(uint32_t base, int r, int j) {
  return base + r * 512 + ((j ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 bytes at `addr` of CTA `rank`'s shared memory
template <int C>
__device__ __forceinline__ uint4 peer_get(uint32_t addr, int rank) {
  if constexpr (C == 1) return Warp::get(addr);
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(ptx::map_to_cta(addr, rank))
               : "memory");
  return v;
}
template <int C>
__device__ __forceinline__ void peer_put(uint32_t addr, int rank, uint4 v) {
  if constexpr (C == 1) return Warp::put(addr, v);
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ptx::map_to_cta(addr, rank)), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

template <int C>
__global__ void __launch_bounds__(kShortThreads, 1) short_kernel(ShortArgs o) {
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[2];
  __shared__ uint32_t tmem_of;
  __shared__ double norm_of;
  __shared__ float rest[kShort];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;
  const int rank = C > 1 ? (int)ptx::cluster_ctarank() : 0, item = (int)blockIdx.x / C;
  const uint32_t x_at = (ptx::smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t a_at = x_at + kShortSlice * 256, part_at = a_at + 32768, b_at = part_at;
  const uint32_t bar = ptx::smem_addr(bars);
  const bool used = (warp & 3) * 32 < o.p;  // the warp has rows of the matrix
  const int first = rank * o.slice, groups = o.slice / 32;
  const int64_t at = (int64_t)item * o.p * o.q;
  const int ksteps = (o.p + 15) / 16;  // of the products whose k is the rows

  ptx::let_next_grid_start();
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(bar + 8, 1);
    ptx::fence_barrier_init();
  }
  if (warp == 0) ptx::tmem_alloc(ptx::smem_addr(&tmem_of), 512);
  // what no one writes reads as zero: rows past p of X and of A
  for (int i = tid; i < (o.slice * 256 + 32768) / 16; i += kShortThreads)
    Warp::put(i < 2048 ? a_at + i * 16 : x_at + (i - 2048) * 16, make_uint4(0, 0, 0, 0));
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_of, lanes = (uint32_t)((warp & 3) * 32) << 16;
  if (warp == 0) ptx::tmem_relinquish();
  ptx::wait_for_previous_grid();

  // G at this lane's row and 32 columns from local column c0
  auto load_g = [&](int c0, float (&v)[32]) {
    const int col = first + c0;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    if (row >= o.p) return;
    if (o.wide && o.q % 8 == 0) {
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        if (col + j >= o.q) continue;
        const int64_t i = at + (int64_t)row * o.q + col + j;
        if (o.g_f32) {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(o.g) + i);
          const float4 lo = __ldg(src), hi = __ldg(src + 1);
          v[j] = lo.x, v[j + 1] = lo.y, v[j + 2] = lo.z, v[j + 3] = lo.w;
          v[j + 4] = hi.x, v[j + 5] = hi.y, v[j + 6] = hi.z, v[j + 7] = hi.w;
        } else {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(o.g) + i));
          v[j] = bf16lo_to_f32(x.x), v[j + 1] = bf16hi_to_f32(x.x);
          v[j + 2] = bf16lo_to_f32(x.y), v[j + 3] = bf16hi_to_f32(x.y);
          v[j + 4] = bf16lo_to_f32(x.z), v[j + 5] = bf16hi_to_f32(x.z);
          v[j + 6] = bf16lo_to_f32(x.w), v[j + 7] = bf16hi_to_f32(x.w);
        }
      }
      return;
    }
    const int64_t base = at + (o.wide ? (int64_t)row * o.q + col : (int64_t)col * o.p + row), step = o.wide ? 1 : o.p;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col + j < o.q)
        v[j] = o.g_f32 ? __ldg(static_cast<const float*>(o.g) + base + j * step)
                       : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(o.g) + base + j * step));
  };
  // 32 columns of the state from local column c0: two halves, 16 words each
  auto put_state = [&](int c0, const float (&v)[32]) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) split(v[2 * j], v[2 * j + 1], hi[j], lo[j]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      Warp::put(short_at(x_at, row, c0 / 8 + u), make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]));
    __syncwarp();
    ptx::tmem_st16(tmem + lanes + kShortLow + c0 / 2, lo);
  };

  double s0 = 0.0, s1 = 0.0;
  if (used)
#pragma unroll 1
    for (int i = half; i < groups; i += 2) {
      float v[32];
      load_g(32 * i, v);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        s0 += (double)v[j] * (double)v[j];
        s1 += (double)v[j + 1] * (double)v[j + 1];
      }
    }
  double sum = block_sum(s0 + s1);
  if constexpr (C > 1) {
    if (tid == 0) norm_of = sum;
    __syncwarp();
    ptx::cluster_sync();
    sum = 0.0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      double v;
      asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(ptx::map_to_cta(ptx::smem_addr(&norm_of), r)) : "memory");
      sum += v;
    }
  }
  {
    const float2 inv = inverse_norm(sum, o.eps);
    if (used)
#pragma unroll 1
      for (int i = half; i < groups; i += 2) {
        float v[32];
        load_g(32 * i, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = inv.x * v[j] * inv.y * o.s;
        put_state(32 * i, v);
      }
  }

  bool ok = true;
  uint32_t phase = 0;  // bit i: the parity that barrier i is waited on next
  auto wait = [&](int i) {
    if (ok) ok = ptx::mbar_wait(bar + 8 * i, (phase >> i) & 1u, o.status, kSiteEpiAccFull);
    phase ^= 1u << i;
    __syncwarp();
    ptx::tc_fence_after();
  };
  // what threads have written to shared memory, and TMEM that they have read, goes to the MMAs
  auto hand_over = [&] {
    __syncwarp();
    ptx::tmem_wait_st();
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  };
  constexpr uint32_t kSquare = ptx::make_idesc(128, 128, 0, 0);
  const int chunks = (o.slice + 127) / 128;
  auto issue_chunk = [&](int j) {
    const uint32_t d = ptx::make_idesc(128, o.slice - 128 * j >= 128 ? 128 : 64, 0, 0) | ptx::kIdescBMn;
#pragma unroll 1
    for (int k = 0; k < ksteps; ++k)
      ptx::mma_f16(tmem + (j & 1) * 128, ptx::sw128_kmajor_desc(b_at + (k >> 2) * 16384 + (k & 3) * 32),
                   ptx::sw128_mnmajor_desc(x_at + j * 32768 + k * 2048, 16384), d, k > 0);
    ptx::mma_commit(bar + 8 * (j & 1));
  };
  const float ci = o.c * o.inv_s;

#pragma unroll 1
  for (int step = 0; step < o.steps; ++step) {
    hand_over();
    if (tid == 0) {
#pragma unroll 1
      for (int k = 0; k < o.slice / 16; ++k) {
        const uint64_t d = ptx::sw128_kmajor_desc(x_at + (k >> 2) * 16384 + (k & 3) * 32);
        ptx::mma_f16(tmem, d, d, kSquare, k > 0);
      }
      ptx::mma_commit(bar);
    }
    __syncwarp();
    wait(0);
    if (used)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[32];
        load_acc32(tmem + lanes + 64 * half + 32 * i, v);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          Warp::put(short_part_at(part_at, row, 16 * half + 8 * i + u),
                    make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]), __float_as_uint(v[4 * u + 2]),
                               __float_as_uint(v[4 * u + 3])));
      }
    ptx::tc_fence_before();
    __syncwarp();
    if constexpr (C > 1) ptx::cluster_sync();
    else __syncthreads();
    // rows [128 / C rank, + 128 / C): pieces of 8 columns
#pragma unroll
    for (int i = 0; i < 8 / C; ++i) {
      const int r = rank * (kShort / C) + i * 16 + tid / 16, j = tid % 16;
      if (r >= o.p) continue;
      uint4 lo[C], hi[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        lo[k] = peer_get<C>(short_part_at(part_at, r, 2 * j), k);
        hi[k] = peer_get<C>(short_part_at(part_at, r, 2 * j + 1), k);
      }
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        v[0] += __uint_as_float(lo[k].x), v[1] += __uint_as_float(lo[k].y);
        v[2] += __uint_as_float(lo[k].z), v[3] += __uint_as_float(lo[k].w);
        v[4] += __uint_as_float(hi[k].x), v[5] += __uint_as_float(hi[k].y);
        v[6] += __uint_as_float(hi[k].z), v[7] += __uint_as_float(hi[k].w);
      }
      uint32_t h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) h[u] = pack_half2(v[2 * u] * o.inv_s, v[2 * u + 1] * o.inv_s);
#pragma unroll
      for (int k = 0; k < C; ++k) peer_put<C>(short_at(a_at, r, j), k, make_uint4(h[0], h[1], h[2], h[3]));
    }
    __syncwarp();
    if constexpr (C > 1) ptx::cluster_sync();
    hand_over();  // (each SM's own proxies: A came through the generic one, from wherever)
    if (tid == 0) {
#pragma unroll 1
      for (int k = 0; k < ksteps; ++k) {
        const uint64_t d = ptx::sw128_kmajor_desc(a_at + (k >> 2) * 16384 + (k & 3) * 32);
        ptx::mma_f16(tmem, d, d, kSquare, k > 0);
      }
      ptx::mma_commit(bar);
    }
    __syncwarp();
    wait(0);
    if (used)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c0 = 64 * half + 32 * i;
        float v[32];
        load_acc32(tmem + lanes + c0, v);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = Warp::get(short_at(a_at, row, c0 / 8 + u));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[8 * u + 2 * j] = fmaf(o.b, f.x, ci * v[8 * u + 2 * j]);
            v[8 * u + 2 * j + 1] = fmaf(o.b, f.y, ci * v[8 * u + 2 * j + 1]);
          }
        }
        if (c0 == (warp & 3) * 32) {
          float d = 0.0f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j == lane) d = v[j];
          rest[row] = (d - __half2float(__float2half_rn(d))) * o.inv_s;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          Warp::put(short_at(b_at, row, c0 / 8 + u),
                    make_uint4(pack_half2(v[8 * u], v[8 * u + 1]), pack_half2(v[8 * u + 2], v[8 * u + 3]),
                               pack_half2(v[8 * u + 4], v[8 * u + 5]), pack_half2(v[8 * u + 6], v[8 * u + 7])));
      }
    hand_over();
    if (tid == 0) {
      issue_chunk(0);
      if (chunks > 1) issue_chunk(1);
    }
    __syncwarp();
    const bool last = step == o.steps - 1;
    const float a_row = o.a + rest[row];
#pragma unroll 1
    for (int j = 0; j < chunks; ++j) {
      wait(j & 1);
      if (used)
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c0 = 128 * j + 64 * i + 32 * half, acc = (j & 1) * 128 + 64 * i + 32 * half;
          if (c0 >= o.slice) break;
          float v[32], x[32];
          uint32_t lo[16];
          __syncwarp();
          ptx::tmem_ld16(tmem + lanes + kShortLow + c0 / 2, lo);
          load_acc32(tmem + lanes + acc, v);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 h = Warp::get(short_at(x_at, row, c0 / 8 + u));
            const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = join(w[k], lo[4 * u + k]);
              x[8 * u + 2 * k] = y.x, x[8 * u + 2 * k + 1] = y.y;
            }
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = fmaf(a_row, x[k], o.inv_s * v[k]);
          if (!last) {
            put_state(c0, v);
            continue;
          }
          const float f = o.scale * o.inv_s;
          const int col = first + c0;
          if (row >= o.p) continue;
          if (o.wide && o.q % 8 == 0) {
            __nv_bfloat16* dst = o.out + at + (int64_t)row * o.q + col;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (col + 8 * u < o.q)
                *reinterpret_cast<uint4*>(dst + 8 * u) =
                    make_uint4(pack_bf16x2(f * v[8 * u], f * v[8 * u + 1]), pack_bf16x2(f * v[8 * u + 2], f * v[8 * u + 3]),
                               pack_bf16x2(f * v[8 * u + 4], f * v[8 * u + 5]),
                               pack_bf16x2(f * v[8 * u + 6], f * v[8 * u + 7]));
          } else {
            __nv_bfloat16* dst = o.out + at + (o.wide ? (int64_t)row * o.q + col : (int64_t)col * o.p + row);
            const int64_t next = o.wide ? 1 : o.p;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (col + k < o.q) dst[k * next] = __float2bfloat16_rn(f * v[k]);
          }
        }
      if (j + 2 < chunks) {
        hand_over();
        if (tid == 0) issue_chunk(j + 2);
        __syncwarp();
      }
    }
  }
  // (no CTA reads or writes another's memory past the last step's second barrier)
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

// The fewest CTAs that hold a matrix; more, down to slices of 128 columns, while
// they all find an SM.
inline int short_cluster(int64_t stack, int64_t q) {
  int c = 1;
  while (c * kShortSlice < q) c *= 2;
  while (c < kShortMost && c * 128 < q && stack * c * 2 <= kSms) c *= 2;
  return c;
}
inline bool is_short(int64_t rows, int64_t cols) {
  return std::min(rows, cols) <= kShort && std::max(rows, cols) <= kShortSlice * kShortMost;
}

template <int C>
static cudaError_t launch_short(const ShortArgs& args, int nb, cudaStream_t s) {
  static std::atomic<uint64_t> sized{0};
  cudaError_t e = set_smem_once(sized, short_kernel<C>, kShortSmem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(short_kernel<C>, dim3((unsigned)(nb * C)), kShortThreads, kShortSmem, s, C, args);
}

}  // namespace mm
}  // namespace moe
