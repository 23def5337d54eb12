// Backward of the router product L = x W_g + b:
//   dW[i,e] = sum_t x[t,i] dL[t,e],  db[e] = sum_t dL[t,e],
//   dx[t,i] = sum_e dL[t,e] W[i,e].
#include "moe_kernels.cuh"

namespace moe {

namespace {

// One 64 x 64 tile of dW over the tokens of one part, 4 x 4 values a thread.
__global__ void __launch_bounds__(256) k_router_dw(const __nv_bfloat16* __restrict__ x,
                                                   const float* __restrict__ dl, int T, int d,
                                                   int E, int per_part, float* __restrict__ part) {
  __shared__ float xs[16][64], ds[16][64];
  pdl_trigger();
  pdl_wait();
  const int i0 = blockIdx.x * 64, e0 = blockIdx.y * 64;
  const int t0 = blockIdx.z * per_part, t1 = min(T, t0 + per_part);
  const int ti = threadIdx.x >> 4, te = threadIdx.x & 15;
  float acc[4][4] = {};
  for (int tb = t0; tb < t1; tb += 16) {
    for (int q = threadIdx.x; q < 16 * 64; q += 256) {
      const int t = tb + q / 64, c = q % 64;
      xs[q / 64][c] = t < t1 ? __bfloat162float(x[(size_t)t * d + i0 + c]) : 0.f;
      ds[q / 64][c] = t < t1 && e0 + c < E ? dl[(size_t)t * E + e0 + c] : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < 16; ++t)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[a][b] = fmaf(xs[t][ti * 4 + a], ds[t][te * 4 + b], acc[a][b]);
    __syncthreads();
  }
  float* out = part + (size_t)blockIdx.z * d * E;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (e0 + te * 4 + b < E) out[(size_t)(i0 + ti * 4 + a) * E + e0 + te * 4 + b] = acc[a][b];
}

// The parts' tiles added in order.
__global__ void __launch_bounds__(256) k_router_dw_sum(const float* __restrict__ part, int parts,
                                                       long long n, float* __restrict__ dw) {
  pdl_trigger();
  pdl_wait();
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += part[p * n + i];
    dw[i] = s;
  }
}

__global__ void __launch_bounds__(256) k_router_db(const float* __restrict__ dl, int T, int E,
                                                   float* __restrict__ db) {
  __shared__ double red[8][32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (e < E)
    for (int t = warp; t < T; t += 8) s += dl[(size_t)t * E + e];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && e < E) {
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += red[w][lane];
    db[e] = (float)s;
  }
}

// One 64 x 64 tile of dx.
__global__ void __launch_bounds__(256) k_router_dx(const float* __restrict__ dl,
                                                   const float* __restrict__ w_g, int T, int d,
                                                   int E, __nv_bfloat16* __restrict__ dx) {
  __shared__ float ds[64][17], ws[64][17];
  pdl_trigger();
  pdl_wait();
  const int t0 = blockIdx.x * 64, i0 = blockIdx.y * 64;
  const int tt = threadIdx.x >> 4, ti = threadIdx.x & 15;
  float acc[4][4] = {};
  for (int eb = 0; eb < E; eb += 16) {
    for (int q = threadIdx.x; q < 64 * 16; q += 256) {
      const int r = q / 16, c = q % 16;
      ds[r][c] = t0 + r < T && eb + c < E ? dl[(size_t)(t0 + r) * E + eb + c] : 0.f;
      ws[r][c] = eb + c < E ? w_g[(size_t)(i0 + r) * E + eb + c] : 0.f;
    }
    __syncthreads();
    for (int e = 0; e < 16; ++e)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[a][b] = fmaf(ds[tt + 16 * a][e], ws[ti + 16 * b][e], acc[a][b]);
    __syncthreads();
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (t0 + tt + 16 * a < T)
        dx[(size_t)(t0 + tt + 16 * a) * d + i0 + ti + 16 * b] = __float2bfloat16_rn(acc[a][b]);
}

}  // namespace

cudaError_t launch_router_bwd(const __nv_bfloat16* x, const float* w_g, const float* dl,
                              const moe_shape& s, float* dw, float* db, __nv_bfloat16* dx,
                              const BwdLayout& L, char* ws, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  float* part = reinterpret_cast<float*>(ws + L.dw_part);
  if (dw) {
    const int per = (s.T + L.dw_parts - 1) / L.dw_parts;
    e = launch_kernel(k_router_dw, dim3(s.d / 64, (s.E + 63) / 64, L.dw_parts), dim3(256), 0, st,
                      1, x, dl, s.T, s.d, s.E, per, part);
    if (e != cudaSuccess) return e;
    e = launch_kernel(k_router_dw_sum, dim3(592), dim3(256), 0, st, 1, part, L.dw_parts,
                      (long long)s.d * s.E, dw);
    if (e != cudaSuccess) return e;
  }
  if (db) {
    e = launch_kernel(k_router_db, dim3((s.E + 31) / 32), dim3(256), 0, st, 1, dl, s.T, s.E, db);
    if (e != cudaSuccess) return e;
  }
  if (dx)
    e = launch_kernel(k_router_dx, dim3((s.T + 63) / 64, s.d / 64), dim3(256), 0, st, 1, dl, w_g,
                      s.T, s.d, s.E, dx);
  return e;
}

}  // namespace moe
