// The global norm of a list of gradients and their clipping by it.
//
// The list goes to the kernels by value, as a launch parameter: nothing is
// uploaded, so the calls allocate nothing and can be captured.  Tensors are
// cut into chunks of equal length and the blocks stride over the chunks of all
// tensors, whatever the tensors' sizes.
#include "moe_kernels.cuh"

namespace moe {

namespace {

struct GradEntry {
  const void* in;
  void* out;
  long long n;
  int chunk0;   // the chunks of the tensors before this one
  int in_bf16;  // 0: fp32
  int out_bf16;
  int pad;
};

template <int N>
struct GradTable {
  GradEntry e[N];
  int count;   // entries
  int chunks;  // chunks of all entries
  int chunk;   // elements of a chunk, a multiple of 8
};

constexpr int kGradTable = 256;   // tensors of one launch
constexpr int kGradBlocks = 592;  // blocks of one launch (partial sums)

template <int N>
__device__ __forceinline__ const GradEntry& entry_of(const GradTable<N>& t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return t.e[lo];
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// 16 bytes of T as floats.
template <class T>
struct Vec16 {
  static constexpr int kN = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ void get(float (&f)[kN]) const {
    if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(raw.x), f[1] = __uint_as_float(raw.y);
      f[2] = __uint_as_float(raw.z), f[3] = __uint_as_float(raw.w);
    } else {
      const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
};

// Elements before the first 16-byte boundary.
template <class T>
__device__ __forceinline__ int head_of(const T* p, long long n) {
  const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return (int)min((long long)h, n);
}

// The sum of squares of n elements: products and sums in fp64, which neither
// overflow nor vanish for any fp32 value.
template <class T>
__device__ double sum_squares(const T* __restrict__ p, int n) {
  double s = 0.0;
  const int h = head_of(p, n);
  if ((int)threadIdx.x < h) {
    const double v = widen(p[threadIdx.x]);
    s += v * v;
  }
  constexpr int N = Vec16<T>::kN, U = 4;
  const int nv = (n - h) / N;
  const uint4* q = reinterpret_cast<const uint4*>(p + h);
  for (int i0 = threadIdx.x; i0 < nv; i0 += 256 * U) {
    Vec16<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u].raw = make_uint4(0, 0, 0, 0);
      if (i0 + 256 * u < nv) v[u].raw = __ldg(q + i0 + 256 * u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[N];
      v[u].get(f);
#pragma unroll
      for (int i = 0; i < N; ++i) s = fma((double)f[i], (double)f[i], s);
    }
  }
  const int at = h + nv * N + (int)threadIdx.x;
  if (at < n) {
    const double v = widen(p[at]);
    s += v * v;
  }
  return s;
}

// Block partials of this launch go to partial[first ...]; the last block of
// the list's last launch (done != nullptr) adds up all of them in order.
template <int N>
__global__ void __launch_bounds__(256) k_grad_sumsq(const __grid_constant__ GradTable<N> t,
                                                    double* __restrict__ partial, int first,
                                                    double* __restrict__ sumsq, int last_launch,
                                                    unsigned* __restrict__ ticket) {
  __shared__ double red[8];
  __shared__ int is_last;
  pdl_trigger();
  pdl_wait();
  double s = 0.0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const GradEntry& e = entry_of(t, c);
    const long long at = (long long)(c - e.chunk0) * t.chunk;
    const int n = (int)min((long long)t.chunk, e.n - at);
    s += e.in_bf16 ? sum_squares(static_cast<const __nv_bfloat16*>(e.in) + at, n)
                   : sum_squares(static_cast<const float*>(e.in) + at, n);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += red[w];
    partial[first + blockIdx.x] = s;
    __threadfence();
    is_last = last_launch && atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  s = 0.0;
  for (int i = threadIdx.x; i < first + (int)gridDim.x; i += 256) s += __ldcg(partial + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += red[w];
    *sumsq = s;
    *ticket = 0;
  }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int N>
__device__ __forceinline__ void put16(float* p, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    __stcs(reinterpret_cast<float4*>(p + i), make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]));
}
__device__ __forceinline__ void put16(__nv_bfloat16* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7])));
}

template <class TI, class TO>
__device__ void scale(const TI* in, TO* out, int n, float c) {
  constexpr int N = Vec16<TI>::kN, U = 4;
  const int h = head_of(in, n);
  if ((reinterpret_cast<uintptr_t>(out + h) & 15) != 0) {
    for (int i = threadIdx.x; i < n; i += 256) put(out + i, c * widen(in[i]));
    return;
  }
  if ((int)threadIdx.x < h) put(out + threadIdx.x, c * widen(in[threadIdx.x]));
  const int nv = (n - h) / N;
  const uint4* q = reinterpret_cast<const uint4*>(in + h);
  TO* o = out + h;
  for (int i0 = threadIdx.x; i0 < nv; i0 += 256 * U) {
    Vec16<TI> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 256 * u < nv) v[u].raw = __ldcs(q + i0 + 256 * u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + 256 * u >= nv) break;
      float f[N];
      v[u].get(f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] *= c;
      put16(o + (size_t)(i0 + 256 * u) * N, f);
    }
  }
  const int at = h + nv * N + (int)threadIdx.x;
  if (at < n) put(out + at, c * widen(in[at]));
}

template <int N>
__global__ void __launch_bounds__(256) k_grad_scale(const __grid_constant__ GradTable<N> t,
                                                    const double* __restrict__ sumsq,
                                                    float max_norm, float* __restrict__ norm) {
  pdl_trigger();
  pdl_wait();
  const double nrm = sqrt(__ldcg(sumsq));
  float c = 1.f;
  if (isfinite(nrm)) c = (float)fmin(1.0, (double)max_norm / (nrm + 1e-6));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = (float)nrm;
  // The last chunks first: the norm's pass read them last, so L2 still holds them.
  for (int r = blockIdx.x; r < t.chunks; r += gridDim.x) {
    const int q = t.chunks - 1 - r;
    const GradEntry& e = entry_of(t, q);
    if (c == 1.f && e.in == e.out) continue;
    const long long at = (long long)(q - e.chunk0) * t.chunk;
    const int n = (int)min((long long)t.chunk, e.n - at);
    if (!e.in_bf16)
      scale(static_cast<const float*>(e.in) + at, static_cast<float*>(e.out) + at, n, c);
    else if (e.out_bf16)
      scale(static_cast<const __nv_bfloat16*>(e.in) + at, static_cast<__nv_bfloat16*>(e.out) + at,
            n, c);
    else
      scale(static_cast<const __nv_bfloat16*>(e.in) + at, static_cast<float*>(e.out) + at, n, c);
  }
}

// Elements of a chunk: about eight chunks for each of 592 blocks, so that the
// blocks end together, between 2048 and 65536.
int chunk_elems(const moe_grad* g, int n) {
  long long total = 0;
  for (int i = 0; i < n; ++i) total += g[i].n;
  const long long c = (total / (8 * kGradBlocks) + 2047) / 2048 * 2048;
  return (int)std::max(2048LL, std::min(65536LL, c));
}

// Calls fn(table, grid, launch index, is the last) for each 256 tensors.
template <class F>
cudaError_t for_tables(const moe_grad* g, int n, F&& fn) {
  const int chunk = chunk_elems(g, n);
  const int launches = std::max(1, (n + kGradTable - 1) / kGradTable);
  for (int q = 0; q < launches; ++q) {
    GradTable<kGradTable> t;
    t.count = 0;
    t.chunk = chunk;
    long long chunks = 0;
    for (int i = q * kGradTable; i < std::min(n, (q + 1) * kGradTable); ++i) {
      if (g[i].n == 0) continue;
      t.e[t.count++] = GradEntry{g[i].data, g[i].out, g[i].n, (int)chunks,
                                 g[i].dtype == MOE_GRAD_BF16, g[i].out_dtype == MOE_GRAD_BF16, 0};
      chunks += (g[i].n + chunk - 1) / chunk;
    }
    if (chunks > INT_MAX / 2) return cudaErrorInvalidValue;
    t.chunks = (int)chunks;
    const int grid = (int)std::max(1LL, std::min<long long>(chunks, kGradBlocks));
    const cudaError_t e = fn(t, grid, q, q == launches - 1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grads_ws_bytes(int n) {
  const size_t launches = (size_t)std::max(1, (n + kGradTable - 1) / kGradTable);
  return 256 + 256 + align_up(launches * kGradBlocks * sizeof(double), 256);
}

double* grads_ws_sumsq(void* ws) {
  return reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
}

cudaError_t launch_grad_sumsq(const moe_grad* g, int n, double* sumsq, void* ws,
                              cudaStream_t st) {
  double* partial = reinterpret_cast<double*>(static_cast<char*>(ws) + 512);
  unsigned* ticket = static_cast<unsigned*>(ws) + kGradTicket;
  int first = 0;
  return for_tables(g, n, [&](const GradTable<kGradTable>& t, int grid, int, bool last) {
    const cudaError_t e = launch_kernel(k_grad_sumsq<kGradTable>, dim3(grid), dim3(256), 0, st, 1,
                                        t, partial, first, sumsq, (int)last, ticket);
    first += grid;
    return e;
  });
}

cudaError_t launch_grad_scale(const moe_grad* g, int n, const double* sumsq, float max_norm,
                              float* norm, cudaStream_t st) {
  return for_tables(g, n, [&](const GradTable<kGradTable>& t, int grid, int q, bool) {
    return launch_kernel(k_grad_scale<kGradTable>, dim3(grid), dim3(256), 0, st, 1, t, sumsq,
                         max_norm, q == 0 ? norm : nullptr);
  });
}

}  // namespace moe
