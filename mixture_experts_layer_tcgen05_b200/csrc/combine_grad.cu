// Gradient of the weighted combine out[t] = sum_j w[t, j] y[p(t, j)]:
//   dy[p(t, j)] = w[t, j] dout[t]          (one rounding to bf16)
//   dw[t, j]    = sum_h dout[t, h] y[p(t, j), h]   (fp32)
// Bound by memory: y is read and dy written once (2 R H 2 bytes), dout read
// once, since the thread that holds eight columns of dout[t] serves all k rows
// of the token. One block per token; the k sums of a block meet in shared
// memory in warp order, so the result does not depend on timing.
#include "common.cuh"

namespace moe {

constexpr int kCombineThreads = 128;

template <int KC>  // rows handled together: their loads are issued before any is used
__global__ void __launch_bounds__(kCombineThreads)
    combine_grad_kernel(const uint4* __restrict__ dout, const uint4* y, const float* __restrict__ w,
                        const int32_t* __restrict__ inv, int T, int vpr, int k, uint4* dy,
                        float* __restrict__ dw, int32_t* status) {
  __shared__ float part[kCombineThreads / 32][KC];
  const int t = (int)blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint4* d0 = dout + (int64_t)t * vpr;
  for (int j0 = 0; j0 < k; j0 += KC) {
    float wj[KC], acc[KC];
    int64_t row[KC];  // -1: no such slot, or an index outside the rows
#pragma unroll
    for (int u = 0; u < KC; ++u) {
      acc[u] = 0.0f;
      wj[u] = 0.0f;
      row[u] = -1;
      if (j0 + u < k) {
        const int p = __ldg(inv + (int64_t)t * k + j0 + u);
        wj[u] = __ldg(w + (int64_t)t * k + j0 + u);
        if ((unsigned)p < (unsigned)(T * k)) row[u] = (int64_t)p * vpr;
        else if (threadIdx.x == 0) record_bad_index(status);
      }
    }
    for (int v = threadIdx.x; v < vpr; v += kCombineThreads) {
      uint4 yv[KC];
#pragma unroll
      for (int u = 0; u < KC; ++u)
        if (row[u] >= 0) yv[u] = y[row[u] + v];
      const uint4 dv = __ldg(d0 + v);
      const float d[8] = {bf16lo_to_f32(dv.x), bf16hi_to_f32(dv.x), bf16lo_to_f32(dv.y), bf16hi_to_f32(dv.y),
                          bf16lo_to_f32(dv.z), bf16hi_to_f32(dv.z), bf16lo_to_f32(dv.w), bf16hi_to_f32(dv.w)};
#pragma unroll
      for (int u = 0; u < KC; ++u) {
        if (row[u] < 0) continue;
        const float f[8] = {bf16lo_to_f32(yv[u].x), bf16hi_to_f32(yv[u].x), bf16lo_to_f32(yv[u].y),
                            bf16hi_to_f32(yv[u].y), bf16lo_to_f32(yv[u].z), bf16hi_to_f32(yv[u].z),
                            bf16lo_to_f32(yv[u].w), bf16hi_to_f32(yv[u].w)};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u] = fmaf(d[i], f[i], acc[u]);
        uint4 o;
        o.x = pack_bf16x2(wj[u] * d[0], wj[u] * d[1]);
        o.y = pack_bf16x2(wj[u] * d[2], wj[u] * d[3]);
        o.z = pack_bf16x2(wj[u] * d[4], wj[u] * d[5]);
        o.w = pack_bf16x2(wj[u] * d[6], wj[u] * d[7]);
        dy[row[u] + v] = o;
      }
    }
#pragma unroll
    for (int u = 0; u < KC; ++u) {
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[u] += __shfl_down_sync(0xffffffffu, acc[u], o);
      if (lane == 0) part[warp][u] = acc[u];
    }
    __syncthreads();
    if (threadIdx.x < KC && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kCombineThreads / 32; ++i) s += part[i][threadIdx.x];
      dw[(int64_t)t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

cudaError_t launch_combine_backward(const void* dout, const void* y, const float* w, const int32_t* inv, int T,
                                    int H, int k, void* dy, float* dw, int32_t* status, cudaStream_t s) {
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)T, kCombineThreads, 0, s>>>(static_cast<const uint4*>(dout), static_cast<const uint4*>(y), w,
                                                   inv, T, H / 8, k, static_cast<uint4*>(dy), dw, status);
    note_launch();
    return cudaGetLastError();
  };
  return k <= 2 ? go(combine_grad_kernel<2>) : k <= 4 ? go(combine_grad_kernel<4>) : go(combine_grad_kernel<8>);
}

}  // namespace moe
