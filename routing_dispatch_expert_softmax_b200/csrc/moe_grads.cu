// The global norm of a list of gradients and their clipping by it.
//
// The list goes to the kernels by value, as a launch parameter: nothing is
// uploaded, so the calls allocate nothing and can be captured.  The tensors'
// elements count as one sequence in units of 2048 (a tensor's last unit may be
// shorter).  The sequence is cut into equal rounds, and every block takes an equal
// run of each: the blocks end together whatever the tensors' sizes, and those that
// run at the same time read neighbouring memory (one long run for each block took
// 15% longer where the scaling streams from and to HBM).
//
// Bound by HBM: 512 M bf16 in 8 tensors, into a flat buffer of odd-sized slices: 535
// us for three passes of 1.07 GB (6.0 TB/s).  96 fp32 gradients of 48 gates (50 MB):
// 29 us, the second read from L2; the two launches' starts and ends are a third of it.
#include "moe_kernels.cuh"

namespace moe {

namespace {

constexpr int kUnit = 2048;       // elements
constexpr int kPiece = 32;        // most units of a block's run in one round
// Tensors of one launch.  A table is copied with the launch, so a short list takes a
// small one (2.5 or 10 KB); the largest has 30 of the 32 KB of a launch's parameters.
constexpr int kTables[3] = {64, 256, 768};
constexpr int kGradBlocks = 592;  // blocks of one launch (partial sums), 4 for each SM

struct GradEntry {
  const void* in;
  void* out;
  long long n;
  long long unit0;  // the units of the tensors before this one
  int in_bf16;      // 0: fp32
  int out_bf16;
};

template <int N>
struct GradTable {
  long long units;  // of all entries
  int count;        // entries
  GradEntry e[N];
};

template <int N>
__device__ __forceinline__ const GradEntry& entry_of(const GradTable<N>& t, long long u) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].unit0 <= u) lo = mid;
    else hi = mid - 1;
  }
  return t.e[lo];
}

// Rounds of the sequence, and the units [first, last) of this block's run in one.
template <int N>
__device__ __forceinline__ long long rounds_of(const GradTable<N>& t) {
  return (t.units + (long long)gridDim.x * kPiece - 1) / ((long long)gridDim.x * kPiece);
}
template <int N>
__device__ __forceinline__ void run_of(const GradTable<N>& t, long long round, long long rounds,
                                       long long& first, long long& last) {
  const long long r0 = t.units * round / rounds, n = t.units * (round + 1) / rounds - r0;
  first = r0 + n * blockIdx.x / gridDim.x;
  last = r0 + n * (blockIdx.x + 1) / gridDim.x;
}

__device__ __forceinline__ long long units_of(const GradEntry& e) {
  return (e.n + kUnit - 1) / kUnit;
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

// The squares of a 16-byte vector (4 or 8 elements) are summed in fp32, off by at
// most 8 2^-24 of their sum, and added up in fp64: converting every element makes
// the pass three times as long (fp64 conversions bound it).  A vector whose sum is
// outside [1e-30, 1e38], where squares pass fp32's range or lose bits in it, is
// summed in fp64 after all, so no fp32 value overflows or vanishes.
template <class T>
__device__ __forceinline__ double vec_squares(const Vec16<T>& v) {
  constexpr int N = Vec16<T>::kN;
  float f[N];
  v.get(f);
  float s = f[0] * f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) s = fmaf(f[i], f[i], s);
  if (s >= 1e-30f && s <= 1e38f) return s;
  double d = 0.0;
  if ((v.raw.x | v.raw.y | v.raw.z | v.raw.w) != 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) d = fma((double)f[i], (double)f[i], d);
  }
  return d;
}

template <class T>
__device__ double sum_squares(const T* __restrict__ p, int n) {
  double s = 0.0;
  const int h = head_of(p, n);
  if ((int)threadIdx.x < h) {
    const double v = widen(p[threadIdx.x]);
    s += v * v;
  }
  constexpr int N = Vec16<T>::kN, U = 8;
  const int nv = (n - h) / N;
  const uint4* q = reinterpret_cast<const uint4*>(p + h);
  int i = threadIdx.x;
  for (; i + 256 * (U - 1) < nv; i += 256 * U) {
    Vec16<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u].raw = __ldg(q + i + 256 * u);
#pragma unroll
    for (int u = 0; u < U; ++u) s += vec_squares(v[u]);
  }
  if (i < nv) {
    Vec16<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u].raw = i + 256 * u < nv ? __ldg(q + i + 256 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) s += vec_squares(v[u]);
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
  const long long rounds = rounds_of(t);
  for (long long round = 0; round < rounds; ++round) {
    long long u, last;
    run_of(t, round, rounds, u, last);
    while (u < last) {
      const GradEntry& e = entry_of(t, u);
      const long long end = min(last, e.unit0 + units_of(e));
      const long long at = (u - e.unit0) * kUnit;
      const int n = (int)(min((end - e.unit0) * kUnit, e.n) - at);
      s += e.in_bf16 ? sum_squares(static_cast<const __nv_bfloat16*>(e.in) + at, n)
                     : sum_squares(static_cast<const float*>(e.in) + at, n);
      u = end;
    }
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

// 16 bytes from byte m (0 .. 14, even) of the 32 bytes lo, hi.
__device__ __forceinline__ uint4 window16(uint4 lo, uint4 hi, int m) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t t[6], u[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) u[i] = m & 4 ? t[i + 1] : t[i];
  const int sh = (m & 2) * 8;
  return make_uint4(__funnelshift_r(u[0], u[1], sh), __funnelshift_r(u[1], u[2], sh),
                    __funnelshift_r(u[2], u[3], sh), __funnelshift_r(u[3], u[4], sh));
}

// out[i] = c in[i] for a piece's n elements; [lo, hi) are the bytes of the whole
// tensor.  Stores are 16 bytes at 16-byte boundaries of out; where in lies
// otherwise, its elements come from two aligned loads that stay inside the tensor
// (a gradient of odd length shifts all that follow it in a flat buffer).
template <class TI, class TO>
__device__ void scale(const TI* in, TO* out, int n, float c, const char* lo, const char* hi) {
  constexpr int N = Vec16<TI>::kN, U = 4;
  int h = head_of(out, n);
  const int m = (int)(reinterpret_cast<uintptr_t>(in + h) & 15);
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(in + h) - m);
  int nv = (n - h) / N;
  if (m) {
    // the first and the last vectors whose loads would leave the tensor go one by one
    if (nv > 0 && reinterpret_cast<const char*>(q) < lo) h += N, ++q, --nv;
    if (nv > 0 && reinterpret_cast<const char*>(q + nv + 1) > hi) --nv;
  }
  TO* o = out + h;
  for (int i = threadIdx.x; i < h; i += 256) put(out + i, c * widen(in[i]));
  // all loads of a step before its first store
  auto store = [&](Vec16<TI> v, int i) {
    float f[N];
    v.get(f);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] *= c;
    put16(o + (size_t)i * N, f);
  };
  int i = threadIdx.x;
  if (m) {
    for (; i + 256 * (U - 1) < nv; i += 256 * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u] = __ldg(q + i + 256 * u), b[u] = __ldg(q + i + 256 * u + 1);
#pragma unroll
      for (int u = 0; u < U; ++u) store(Vec16<TI>{window16(a[u], b[u], m)}, i + 256 * u);
    }
    for (; i < nv; i += 256) store(Vec16<TI>{window16(__ldg(q + i), __ldg(q + i + 1), m)}, i);
  } else {
    for (; i + 256 * (U - 1) < nv; i += 256 * U) {
      uint4 a[U];
#pragma unroll
      for (int u = 0; u < U; ++u) a[u] = __ldcs(q + i + 256 * u);
#pragma unroll
      for (int u = 0; u < U; ++u) store(Vec16<TI>{a[u]}, i + 256 * u);
    }
    if (i < nv) {
      uint4 a[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        a[u] = i + 256 * u < nv ? __ldcs(q + i + 256 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 256 * u < nv) store(Vec16<TI>{a[u]}, i + 256 * u);
    }
  }
  for (int at = h + nv * N + (int)threadIdx.x; at < n; at += 256) put(out + at, c * widen(in[at]));
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
  // The last rounds first: the norm's pass read them last, so L2 still holds them.
  const long long rounds = rounds_of(t);
  for (long long round = rounds - 1; round >= 0; --round) {
    long long u, last;
    run_of(t, round, rounds, u, last);
    while (u < last) {
      const GradEntry& e = entry_of(t, u);
      const long long end = min(last, e.unit0 + units_of(e));
      const long long at = (u - e.unit0) * kUnit;
      const int n = (int)(min((end - e.unit0) * kUnit, e.n) - at);
      u = end;
      if (c == 1.f && e.in == e.out) continue;
      const char* lo = static_cast<const char*>(e.in);
      const char* hi = lo + e.n * (e.in_bf16 ? 2 : 4);
      const float* f32 = static_cast<const float*>(e.in) + at;
      const __nv_bfloat16* b16 = static_cast<const __nv_bfloat16*>(e.in) + at;
      if (!e.in_bf16)
        scale(f32, static_cast<float*>(e.out) + at, n, c, lo, hi);
      else if (e.out_bf16)
        scale(b16, static_cast<__nv_bfloat16*>(e.out) + at, n, c, lo, hi);
      else
        scale(b16, static_cast<float*>(e.out) + at, n, c, lo, hi);
    }
  }
}

// Calls fn(table, grid, launch index, is the last) for each N tensors.
template <int N, class F>
cudaError_t for_tables(const moe_grad* g, int n, F&& fn) {
  const int launches = std::max(1, (n + N - 1) / N);
  for (int q = 0; q < launches; ++q) {
    GradTable<N> t;
    t.count = 0;
    t.units = 0;
    for (int i = q * N; i < std::min(n, (q + 1) * N); ++i) {
      if (g[i].n == 0) continue;
      t.e[t.count++] = GradEntry{g[i].data, g[i].out, g[i].n, t.units,
                                 g[i].dtype == MOE_GRAD_BF16, g[i].out_dtype == MOE_GRAD_BF16};
      t.units += (g[i].n + kUnit - 1) / kUnit;
    }
    const int grid = (int)std::max(1LL, std::min<long long>(t.units, kGradBlocks));
    const cudaError_t e = fn(t, grid, q, q == launches - 1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t sumsq(const moe_grad* g, int n, double* out, void* ws, cudaStream_t st) {
  double* partial = reinterpret_cast<double*>(static_cast<char*>(ws) + 512);
  unsigned* ticket = static_cast<unsigned*>(ws) + kGradTicket;
  int first = 0;
  return for_tables<N>(g, n, [&](const GradTable<N>& t, int grid, int, bool last) {
    const cudaError_t e = launch_kernel(k_grad_sumsq<N>, dim3(grid), dim3(256), 0, st, 1, t,
                                        partial, first, out, (int)last, ticket);
    first += grid;
    return e;
  });
}

template <int N>
cudaError_t scale_all(const moe_grad* g, int n, const double* sumsq, float max_norm, float* norm,
                      cudaStream_t st) {
  return for_tables<N>(g, n, [&](const GradTable<N>& t, int grid, int q, bool) {
    return launch_kernel(k_grad_scale<N>, dim3(grid), dim3(256), 0, st, 1, t, sumsq, max_norm,
                         q == 0 ? norm : nullptr);
  });
}

}  // namespace

size_t grads_ws_bytes(int n) {
  const size_t launches = (size_t)std::max(1, (n + kTables[2] - 1) / kTables[2]);
  return 256 + 256 + align_up(launches * kGradBlocks * sizeof(double), 256);
}

double* grads_ws_sumsq(void* ws) {
  return reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
}

cudaError_t launch_grad_sumsq(const moe_grad* g, int n, double* out, void* ws, cudaStream_t st) {
  return n <= kTables[0]   ? sumsq<kTables[0]>(g, n, out, ws, st)
         : n <= kTables[1] ? sumsq<kTables[1]>(g, n, out, ws, st)
                           : sumsq<kTables[2]>(g, n, out, ws, st);
}

cudaError_t launch_grad_scale(const moe_grad* g, int n, const double* sumsq, float max_norm,
                              float* norm, cudaStream_t st) {
  return n <= kTables[0]   ? scale_all<kTables[0]>(g, n, sumsq, max_norm, norm, st)
         : n <= kTables[1] ? scale_all<kTables[1]>(g, n, sumsq, max_norm, norm, st)
                           : scale_all<kTables[2]>(g, n, sumsq, max_norm, norm, st);
}

}  // namespace moe
