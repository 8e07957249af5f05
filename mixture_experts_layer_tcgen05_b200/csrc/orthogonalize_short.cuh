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
//   - the CTA's part of A by MMA, in fp32 to shared memory; `own` rows of it to
//     each CTA by bulk copy; each adds what it got, in order, and copies its rows of
//     A, in fp16, to the others. The copies complete on barriers of the receiving
//     CTA, and each stage's data is only sent when all of the one before has come, so
//     nothing else keeps the buffers apart. (Loads of the other CTAs' memory, stores
//     to it and two cluster barriers took 10200 cycles a step instead of 6200.)
//   - A^2 by MMA and B = b A + c A^2 in every CTA alike, over its own part of A;
//   - B X by MMA, the first and the last 128 columns each into an accumulator, and
//     X <- a X + B X in place: a chunk's MMAs read that chunk's columns alone.
// Bound by latency. Of a step's 12700 cycles (128 x 128 to a CTA, four CTAs) the
// issue of the 24 MMAs takes 2500, the exchange of A 6200 (a third of it the copies'
// bytes, 48 KB each way) and the epilogues 3700; before the first step 10000 go to
// reading G and its norm. Measured, against the launches of the general form: eight
// 512 x 128 43 and 84 us, one 128 x 128 27 and 74, 16 x 512 25 and 67, 100 x 2000 55
// and 95, a thousand 128 x 128 199 and 648, 64 of 2048 x 128 312 and 339. A CTA's
// slice is at most the 256 columns that shared memory has room for beside the parts of
// A; the rest is the general form's.
#pragma once

#include <cuda_fp16.h>

#include "mm_core.cuh"

namespace moe {
namespace mm {

constexpr int kShort = 128, kShortSlice = 256, kShortThreads = 256, kShortMost = 8;  // p, columns of a CTA, CTAs
// of a cluster that every device grants
// X, A, the part of A (which B replaces), and the parts that others sent
constexpr size_t kShortSmem = 1024 + kShortSlice * 256 + 32768 + 2 * 65536;
constexpr int kShortLow = 256;  // TMEM: two accumulators of 128 columns, then the lower halves

struct ShortArgs {
  const void* g;         // [nb, p, q], or [nb, q, p] where not wide; fp32 or bf16
  __nv_bfloat16* out;    // likewise
  int32_t* status;
  int p, q, slice, steps;
  int own;               // rows of A that a CTA adds, a multiple of 8: CTA r those from r own, if below p
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

template <int C>
__global__ void __launch_bounds__(kShortThreads, 1) short_kernel(ShortArgs o) {
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[4];  // two accumulators, parts of A, rows of A
  __shared__ uint32_t tmem_of;
  __shared__ double norm_of;
  __shared__ float rest[kShort];
  __shared__ float4 factors[kMostSteps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;
  const int rank = C > 1 ? (int)ptx::cluster_ctarank() : 0, item = (int)blockIdx.x / C;
  const uint32_t x_at = (ptx::smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t a_at = x_at + kShortSlice * 256, part_at = a_at + 32768, got_at = part_at + 65536, b_at = part_at;
  const uint32_t bar = ptx::smem_addr(bars);
  const bool used = (warp & 3) * 32 < o.p;  // the warp has rows of the matrix
  const int first = rank * o.slice, groups = o.slice / 32;
  const int64_t at = (int64_t)item * o.p * o.q;
  const int ksteps = (o.p + 15) / 16;  // of the products whose k is the rows

  ptx::let_next_grid_start();
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) ptx::mbar_init(bar + 8 * i, 1);
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
    if (o.g_f32) {
      const float* src = static_cast<const float*>(o.g) + base;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j < o.q) v[j] = __ldg(src + j * step);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j < o.q) v[j] = ldg_bf16(o.g, base + j * step);
    }
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

  // Sum of squares: 32 at a time in fp32, times a power of two that keeps them in
  // its range, then in fp64. Up to 128 columns stay in registers meanwhile.
  float v0[32], v1[32];
  auto squares = [](const float(&v)[32]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(v[j]));
    const int e = min(126, max(-126, 127 - (int)(__float_as_uint(m) >> 23)));  // m 2^e is near 1
    const float f = __uint_as_float((uint32_t)(e + 127) << 23);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j & 3] = fmaf(v[j] * f, v[j] * f, s[j & 3]);
    return ldexp((double)((s[0] + s[1]) + (s[2] + s[3])), -2 * e);
  };
  double sum = 0.0;
  if (used) {
#pragma unroll 1
    for (int i = 4 + half; i < groups; i += 2) {
      load_g(32 * i, v0);
      sum += squares(v0);
    }
    load_g(32 * half, v0);
    if (groups > 2 + half) load_g(64 + 32 * half, v1);
    sum += squares(v0);
    if (groups > 2 + half) sum += squares(v1);
  }
  sum = block_sum(sum);
  if constexpr (C > 1) {
    if (tid == 0) norm_of = sum;
    __syncwarp();
    ptx::cluster_sync();
    sum = 0.0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      double v;
      asm volatile("ld.shared::cluster.f64 %0, [%1];"
                   : "=d"(v)
                   : "r"(ptx::map_to_cta(ptx::smem_addr(&norm_of), r))
                   : "memory");
      sum += v;
    }
  }
  {
    const Unit inv = unit_norm(sum, o.eps);
    step_factors(inv, o.a, o.b, o.c, o.scale, o.steps, [&](int i, float4 v) { factors[i] = v; });
    auto init = [&](int c0, float(&v)[32]) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = inv.x * v[j] * inv.y * o.s;
      put_state(c0, v);
    };
    if (used) {
      init(32 * half, v0);
      if (groups > 2 + half) init(64 + 32 * half, v1);
#pragma unroll 1
      for (int i = 4 + half; i < groups; i += 2) {
        load_g(32 * i, v0);
        init(32 * i, v0);
      }
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
  static_assert(kShortSlice == 2 * 128, "an accumulator of 128 columns for each chunk");
  const int chunks = (o.slice + 127) / 128;
  // The products, issued by thread 0. In the descriptors addresses count 16 bytes:
  // 16 k further is 2 along a K-major row, a block of 64 columns further 1024.
  auto issue_square = [&](uint32_t m, int n) {
    const uint64_t d0 = ptx::sw128_kmajor_desc(m);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const uint64_t d = d0 + (k >> 2) * 1024 + (k & 3) * 2;
      ptx::mma_f16(tmem, d, d, kSquare, k > 0);
    }
    ptx::mma_commit(bar);
  };
  auto issue_chunk = [&](int j) {
    const uint32_t i = ptx::make_idesc(128, o.slice - 128 * j >= 128 ? 128 : 64, 0, 0) | ptx::kIdescBMn;
    const uint64_t db = ptx::sw128_kmajor_desc(b_at), dx = ptx::sw128_mnmajor_desc(x_at + j * 32768, 16384);
#pragma unroll 4
    for (int k = 0; k < ksteps; ++k)
      ptx::mma_f16(tmem + j * 128, db + (k >> 2) * 1024 + (k & 3) * 2, dx + k * 128, i, k > 0);
    ptx::mma_commit(bar + 8 * j);
  };
#pragma unroll 1
  for (int step = 0; step < o.steps; ++step) {
    hand_over();
    if (tid == 0) issue_square(x_at, o.slice / 16);
    __syncwarp();
    const float4 f = factors[step];
    const float ci = f.y * o.inv_s, inv_s = f.z * o.inv_s;
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
    const int mine = rank * o.own;  // first of the rows of A that this CTA adds
    const bool adds = mine < o.p;
    hand_over();
    if (C > 1 && tid == 0) {
      if (adds) ptx::mbar_arrive_expect_tx(bar + 16, (C - 1) * o.own * 512);
      const int others = (o.p + o.own - 1) / o.own - adds;
      if (others) ptx::mbar_arrive_expect_tx(bar + 24, others * o.own * 256);
    }
    if (C > 1 && ok && warp == 0 && lane < C && lane != rank && lane * o.own < o.p)
      ptx::bulk_copy_to_cta(ptx::map_to_cta(got_at + rank * o.own * 512, lane), part_at + lane * o.own * 512,
                            o.own * 512, ptx::map_to_cta(bar + 16, lane));
    __syncwarp();
    if (adds) {
      if (C > 1) wait(2);
#pragma unroll 1
      for (int i = tid; i < o.own * 16; i += kShortThreads) {
        const int r = i / 16, j = i % 16;  // 8 columns of a row
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const uint32_t from = k == rank ? part_at + mine * 512 : got_at + k * o.own * 512;
          const uint4 lo = Warp::get(short_part_at(from, r, 2 * j)), hi = Warp::get(short_part_at(from, r, 2 * j + 1));
          v[0] += __uint_as_float(lo.x), v[1] += __uint_as_float(lo.y);
          v[2] += __uint_as_float(lo.z), v[3] += __uint_as_float(lo.w);
          v[4] += __uint_as_float(hi.x), v[5] += __uint_as_float(hi.y);
          v[6] += __uint_as_float(hi.z), v[7] += __uint_as_float(hi.w);
        }
        uint32_t h[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) h[u] = pack_half2(v[2 * u] * o.inv_s, v[2 * u + 1] * o.inv_s);
        Warp::put(short_at(a_at, mine + r, j), make_uint4(h[0], h[1], h[2], h[3]));
      }
    }
    if constexpr (C > 1) {
      hand_over();
      if (adds && ok && warp < 2 && lane < C && lane != rank) {  // a warp for each of A's blocks of 64 columns
        const uint32_t from = a_at + warp * 16384 + mine * 128;
        ptx::bulk_copy_to_cta(ptx::map_to_cta(from, lane), from, o.own * 128, ptx::map_to_cta(bar + 24, lane));
      }
      __syncwarp();
      if ((o.p + o.own - 1) / o.own > adds) wait(3);
      if (step == o.steps - 1) {  // all that was sent to this CTA has come
        __syncwarp();
        ptx::cluster_arrive_relaxed();
      }
    }
    hand_over();
    if (tid == 0) issue_square(a_at, ksteps);
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
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[8 * u + 2 * j] = fmaf(f.x, e.x, ci * v[8 * u + 2 * j]);
            v[8 * u + 2 * j + 1] = fmaf(f.x, e.y, ci * v[8 * u + 2 * j + 1]);
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
    const float a_row = f.z * (o.a + rest[row]);
#pragma unroll 1
    for (int j = 0; j < chunks; ++j) {
      wait(j);
      if (used)
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c0 = 128 * j + 64 * i + 32 * half;  // of X and of the accumulators
          if (c0 >= o.slice) break;
          float v[32], x[32];
          uint32_t lo[16];
          __syncwarp();
          ptx::tmem_ld16(tmem + lanes + kShortLow + c0 / 2, lo);
          load_acc32(tmem + lanes + c0, v);
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
          for (int k = 0; k < 32; ++k) v[k] = fmaf(a_row, x[k], inv_s * v[k]);
          if (!last) {
            put_state(c0, v);
            continue;
          }
          const float r = f.w * o.inv_s;
          const int col = first + c0;
          if (row >= o.p) continue;
          if (o.wide && o.q % 8 == 0) {
            __nv_bfloat16* dst = o.out + at + (int64_t)row * o.q + col;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (col + 8 * u < o.q)
                *reinterpret_cast<uint4*>(dst + 8 * u) =
                    make_uint4(pack_bf16x2(r * v[8 * u], r * v[8 * u + 1]),
                               pack_bf16x2(r * v[8 * u + 2], r * v[8 * u + 3]),
                               pack_bf16x2(r * v[8 * u + 4], r * v[8 * u + 5]),
                               pack_bf16x2(r * v[8 * u + 6], r * v[8 * u + 7]));
          } else {
            __nv_bfloat16* dst = o.out + at + (o.wide ? (int64_t)row * o.q + col : (int64_t)col * o.p + row);
            const int64_t next = o.wide ? 1 : o.p;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (col + k < o.q) dst[k * next] = __float2bfloat16_rn(r * v[k]);
          }
        }
    }
  }
  // a wait that gave up: time for what is still on its way here
  if (!ok)
    for (int i = 0; i < 100; ++i) __nanosleep(1000);
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (C > 1) ptx::cluster_wait();  // the others have what this CTA sent
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, 512);
}

template <int C>
static cudaError_t size_short() {
  static std::atomic<uint64_t> sized{0};
  if (C > kShortMost) {
    cudaError_t e = cudaFuncSetAttribute(short_kernel<C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return set_smem_once(sized, short_kernel<C>, kShortSmem);
}

// How many clusters of 16, a size that a device need not grant, the current one
// runs at a time.
static int clusters_of_16() {
  static std::atomic<int> known[64];  // that number and 1
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64) n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kShortThreads);
  cfg.dynamicSmemBytes = kShortSmem;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 16;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (size_short<16>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, short_kernel<16>, &cfg) != cudaSuccess) {
    cudaGetLastError();  // not this call's error
    n = 0;
  }
  if (dev < 64) known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

// The fewest CTAs that hold a matrix; more, down to slices of 128 columns, while
// they all find an SM (eight 512 x 128: 43 us with slices of 128, 54 with 256; sixteen
// 44 and 54, and 79 with slices of 64, whose clusters do not all run at once).
inline int short_cluster(int64_t stack, int64_t q) {
  int c = 1;
  while (c * kShortSlice < q) c *= 2;
  while (c < kShortMost && c * 128 < q && stack * c * 2 <= kSms) c *= 2;
  return c;
}
// Sides past eight slices take clusters of 16, of which few run at a time: only
// stacks that run at once (128 x 4096: one 63 us, 100 in the general form; 16 of them
// 192 and 240, but 64 of 64 x 4096 565 and 381, 128 of 128 x 2500 1989 and 808).
inline bool is_short(int64_t stack, int64_t rows, int64_t cols) {
  const int64_t q = std::max(rows, cols);
  return std::min(rows, cols) <= kShort &&
         (q <= kShortSlice * kShortMost || (q <= kShortSlice * 16 && stack <= clusters_of_16()));
}

template <int C>
static cudaError_t launch_short(const ShortArgs& args, int nb, cudaStream_t s) {
  cudaError_t e = size_short<C>();
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(short_kernel<C>, dim3((unsigned)(nb * C)), kShortThreads, kShortSmem, s, C, args);
}

}  // namespace mm
}  // namespace moe
