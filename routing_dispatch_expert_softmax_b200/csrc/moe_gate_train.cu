// Training the gate: the balance loss with its per-expert counts, the
// gradient of the router logits, and the backward of the combine.
//
// The pages name the imbalance of the gate ("Serving MoE models with expert
// parallelism on 8xH200", section "Routing imbalance") but give no loss; the
// one here is the usual product of each expert's share of the selections and
// its mean probability, with the mean squared logsumexp beside it.
#include <type_traits>

#include "moe_kernels.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- row layout
// A group of LPR lanes owns one row of E fp32 logits, NV values a lane: in chunks
// of 4, chunk c of lane l the columns c * 4 * LPR + 4 l + (0..3), so that a group's
// 16-byte loads are contiguous; or, where rows are not 16-byte aligned, value i the
// column i * LPR + l, so that its 4-byte loads are (VEC = false).
//
// These kernels are bound by the instructions of a row that do not shrink with it
// (reductions, the k slots), so a lane holds 8 values up to 256 experts and a warp
// takes 32 / LPR rows at once: with 4 values (two rows of 64 experts a warp in place
// of four, one of 128 in place of two) the gate's gradient of 131072 rows took 29
// and 49 us in place of 21 and 36 (18 and 34 since).  Above 256 experts a warp has one
// row.  The next rows' loads are in flight meanwhile, up to 512 experts.
template <int LPR, int NV, bool VEC>
struct RowCfg {
  static constexpr int kLpr = LPR, kNv = NV;
  static constexpr bool kVec = VEC;
  static constexpr int kGroups = 32 / LPR;  // rows of a warp at once
  static constexpr int kCols = LPR * NV;    // columns a group can hold
  static constexpr bool kAhead = NV <= 16;
  // blocks of an SM: of the balance loss, of the gate's gradient
  static constexpr int kBlocks = NV <= 8 ? 4 : NV <= 16 ? 3 : 2;
  static constexpr int kGateBlocks = NV > 8 ? 2 : LPR == 1 || LPR == 32 ? 4 : 3;
};

template <int LPR, bool VEC>
__device__ __forceinline__ int col_of(int l, int i) {
  return VEC ? (i >> 2) * (4 * LPR) + 4 * l + (i & 3) : i * LPR + l;
}

// Element offsets below are 32-bit: T E <= 2^30.
//
// Two fp32 values as one 64-bit operand: the packed instructions of sm_100 do
// two adds, products or fmas each, with the roundings of the single ones.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

constexpr f32x2 kNone = 0xff800000ff800000ull;  // a pair of -inf

// A lane's NV values as pairs.  Columns at or past E read as -inf: their exp is
// 0 and they never are the maximum.
template <int LPR, int NV, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l,
                                         f32x2 (&v)[NV / 2]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < NV / 4; ++c) {
      const int e = c * 4 * LPR + 4 * l;
      // as 64-bit halves: a pair made of two floats would wait for the load here
      ulonglong2 q = make_ulonglong2(kNone, kNone);
      if (e < E) q = __ldcs(reinterpret_cast<const ulonglong2*>(row + e));
      v[2 * c] = q.x;
      v[2 * c + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      const int e = 2 * i * LPR + l;
      v[i] = pair(e < E ? __ldcs(row + e) : -INFINITY,
                  e + LPR < E ? __ldcs(row + e + LPR) : -INFINITY);
    }
  }
}

__device__ __forceinline__ float rcp_fast(float v) {  // 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// log v = log2 v times ln 2, for sums of exponentials in [1, 1024]: lg2.approx is off by
// 2^-22 up to 2 and by 2^-22 of itself above.
__device__ __forceinline__ float log_fast(float v) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r * 0.6931471805599453f;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// The maximum over each group of LPR lanes, NaN left aside.
template <int LPR>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (LPR == 32) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row's values become exp(v - max); returns the lane's sum of them and gives the
// row's maximum.  live: some value is not -inf (a NaN counts: it has to show in the
// result).  A row without a live value gives exp values of 0 and a sum of 0.
// exp is ex2.approx of the difference times log2 e: with a difference of size D
// off by at most (2.3 D + 4) 2^-24 of the value, and values below 2^-126 are 0.
// These kernels are bound by their instructions, of which expf takes four times as many.
template <int LPR, int NV>
__device__ __forceinline__ float row_exp(f32x2 (&v)[NV / 2], float& top, bool& live) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    const float2 q = unpair(v[i]);
    m = max3(m, q.x, q.y);
  }
  top = group_max<LPR>(m);
  live = top != -INFINITY;
  if (!__all_sync(0xffffffffu, live)) {  // nothing but -inf, and perhaps NaN
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      const float2 q = unpair(v[i]);
      nan |= q.x != q.x || q.y != q.y;
    }
    const unsigned votes = __ballot_sync(0xffffffffu, nan);
    const int g0 = (threadIdx.x & 31) / LPR * LPR;
    const unsigned mine = LPR == 32 ? votes : (votes >> g0) & ((1u << (LPR & 31)) - 1u);
    // with 0 in the maximum's place the -inf values keep giving 0
    if (!live) top = 0.f, live = mine != 0;
  }
  const f32x2 down = pair(-top, -top), log2e = pair(kLog2e, kLog2e);
  f32x2 t = 0;
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    const float2 q = unpair(mul2(add2(v[i], down), log2e));
    v[i] = pair(exp2_fast(q.x), exp2_fast(q.y));
    t = i ? add2(t, v[i]) : v[i];
  }
  const float2 q = unpair(t);
  return q.x + q.y;
}

// Three sums over each group of lanes; a whole warp does them in one chain, a
// quarter of it each, with 9 shuffles in place of 15.
template <int LPR>
__device__ __forceinline__ void sum3(float& a, float& b, float& c) {
  if constexpr (LPR == 32) {
    const bool hi = (threadIdx.x & 16) != 0, odd = (threadIdx.x & 8) != 0;
    float x = (hi ? c : a) + __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
    float y = b + __shfl_xor_sync(0xffffffffu, b, 16);
    x = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    a = __shfl_sync(0xffffffffu, x, 0);
    b = __shfl_sync(0xffffffffu, x, 8);
    c = __shfl_sync(0xffffffffu, x, 16);
  } else {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
  }
}

// The sequence s with off[s] <= t < off[s + 1] (the last such s, so an empty
// sequence owns nothing), or -1 before the first and S behind the last one.
// Offsets that do not ascend give some s in [-1, S]; nothing is read outside
// off[0 .. S].
__device__ __forceinline__ int find_seq(const int* __restrict__ off, int S, int t) {
  int lo = 0, hi = S + 1;  // the number of offsets <= t lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(off + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// ============================================================== balance loss
// Block b takes the tokens [b C, (b + 1) C).  Within them, each sequence's
// tokens are one run, whose probabilities are summed in registers (fp32, a
// few hundred rows at most), met in shared memory and stored as the partial
// of slot b + s: along the ascending (block, sequence) pairs that meet,
// b + s never repeats, so every partial has one writer and the sums have a
// fixed order.  Selections are counted in shared memory (integers: any order).
// 262144 x 256: 50 us (5.6 TB/s, 121 instructions a row and warp, issue slots 65%
// used; what is left is waiting for rows), and the whole call 54 us.
struct BalancePart {
  float* prob;  // [nblk + S][E]
  int* count;   // [nblk + S][E]
  float* z;     // [nblk + S]
  int* n;       // [nblk + S]
};

// The loss from the sums over all counted tokens (one thread): f = the sequences'
// sum of E / (k N^2) sum_e count prob_sum, z = the sum of lse^2.  A coefficient of
// 0 leaves its term out, whatever the term is.
__device__ __forceinline__ void write_loss(double f, double z, long long n, int live,
                                           float balance_coef, float z_coef, float* loss,
                                           int* totals) {
  const double lb = live > 0 && balance_coef != 0.f ? balance_coef * f / live : 0.0;
  const double lz = n > 0 && z_coef != 0.f ? z_coef * z / (double)n : 0.0;
  loss[0] = (float)(lb + lz);
  loss[1] = (float)lb;
  loss[2] = (float)lz;
  totals[0] = (int)n;
  totals[1] = live;
}

// The results of one sequence with few partials, which the block that finishes last
// (a ticket) adds up itself; loss == nullptr: k_balance_finish does.  A second launch
// costs the host 2.3 us and the device 2: 1024 x 128 in 8.8 us in place of 11.4; but
// one block adds no more than 8192 values (1024 x 1024: 15.3 us in place of 12.3).
constexpr int kWholeBlocks = 256, kWholeValues = 8192;
struct BalanceWhole {
  float balance_coef, z_coef;
  float* loss;
  int* counts;
  int* tokens;
  float* prob_mean;
};

// Called by all blocks after their partials are stored; the last one adds them up.
// A block alone (own: its sums and counts in shared memory, z and n of its warps) has
// stored nothing.
struct BalanceOwn {
  const float* prob;
  const int* count;
  const float* z;
  const int* n;
};
__device__ void finish_whole(const BalancePart& part, const BalanceOwn& own, int E, int k,
                             const BalanceWhole& out, int* ticket) {
  __shared__ int is_last;
  __shared__ double sums[256], fred[8];
  __shared__ int cnts[256];
  const int blocks = gridDim.x;
  if (blocks > 1) {
    if (threadIdx.x == 0) {
      __threadfence();
      is_last = atomicAdd(reinterpret_cast<unsigned*>(ticket), 1u) == blocks - 1u;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
  }
  // in every warp: z and n
  const int lane = threadIdx.x & 31;
  double z = 0.0, f = 0.0;
  int n = 0;
  if (blocks == 1) {
    if (lane < 8) z = own.z[lane], n = own.n[lane];
  } else {
    for (int q = lane; q < blocks; q += 32) z += __ldcg(part.z + q), n += __ldcg(part.n + q);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  // `span` experts at a time; the threads beyond them take the blocks in turn
  int span = 32;
  while (span < E && span < 256) span *= 2;
  const int groups = 256 / span, c = threadIdx.x % span, g = threadIdx.x / span;
  for (int e0 = 0; e0 < E; e0 += span) {
    const int e = e0 + c;
    double p = 0.0;
    int m = 0;
    if (blocks == 1) {
      if (e < E) p = own.prob[e], m = own.count[e];
    } else if (e < E) {
#pragma unroll 8
      for (int q = g; q < blocks; q += groups) {
        p += __ldcg(part.prob + (unsigned)(q * E + e));
        m += __ldcg(part.count + (unsigned)(q * E + e));
      }
    }
    if (groups > 1 && blocks > 1) {
      sums[threadIdx.x] = p, cnts[threadIdx.x] = m;
      __syncthreads();
      for (int i = 1; g == 0 && i < groups; ++i) p += sums[i * span + c], m += cnts[i * span + c];
    }
    if (g == 0 && e < E) {
      f += p * m;
      out.counts[e] = m;
      if (out.prob_mean) out.prob_mean[e] = n > 0 ? (float)(p / n) : 0.f;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
  if (lane == 0) fred[threadIdx.x / 32] = f;
  __syncthreads();
  if (threadIdx.x == 0) {
    f = 0.0;
    for (int w = 0; w < 8; ++w) f += fred[w];
    out.tokens[0] = n;
    write_loss(n > 0 ? f * E / ((double)k * n * n) : 0.0, z, n, n > 0, out.balance_coef,
               out.z_coef, out.loss, out.tokens + 1);
    if (blocks > 1) *ticket = 0;
  }
}

template <int LPR, int NV, bool VEC>
__global__ void __launch_bounds__(256, RowCfg<LPR, NV, VEC>::kBlocks) k_balance_rows(
    const float* __restrict__ logits, const int* __restrict__ idx,
    const uint8_t* __restrict__ mask, const int* __restrict__ off, int S, int T, int E, int k,
    int C, BalancePart part, int* err, const BalanceWhole whole) {
  using R = RowCfg<LPR, NV, VEC>;
  extern __shared__ float sm[];
  float* red = sm;                                        // [8][kCols]
  int* hist = reinterpret_cast<int*>(sm + 8 * R::kCols);  // [E]
  __shared__ float zred[8];
  __shared__ int nred[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, g = lane / LPR;
  const int t0 = blockIdx.x * C, t1 = min(T, t0 + C);
  for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  int s = off ? find_seq(off, S, t0) : 0;
  int t = t0;
  if (s < 0) {  // tokens before the first sequence
    s = 0;
    t = min(t1, max(t0, __ldg(off)));
  }
  bool bad_id = false;
  while (t < t1 && s < S) {
    const int end = off ? min(t1, __ldg(off + s + 1)) : t1;
    if (end <= t) {  // an empty sequence, perhaps the first of thousands (a step each: 7 ms)
      s = max(s + 1, find_seq(off, S, t));
      continue;
    }
    f32x2 acc[NV / 2];
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) acc[i] = 0;
    float zacc = 0.f;
    int nacc = 0;
    constexpr int kStep = 8 * R::kGroups;
    struct Row {
      f32x2 v[NV / 2];
      int id;  // the lane's first selection
      bool in;
    };
    auto load = [&](Row& q, int r) {
      q.in = r < end;
      if (r < end) {
        load_row<LPR, NV, VEC>(logits + (unsigned)(r * E), E, l, q.v);
        if (l < k) q.id = __ldg(idx + (unsigned)(r * k + l));
        if (mask) q.in = mask[r] != 0;
      }
    };
    auto count = [&](int e) {
      if ((unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
      else bad_id = true;
    };
    auto add_row = [&](Row& q, int r) {
      float top;
      bool live;
      const float sum = group_sum<LPR>(row_exp<LPR, NV>(q.v, top, live));
      if (!(q.in && live)) return;
      const float inv = rcp_fast(sum);
      const f32x2 inv2 = pair(inv, inv);
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) acc[i] = fma2(q.v[i], inv2, acc[i]);
      const float lse = top + log_fast(sum);  // every lane of the group the same
      zacc = fmaf(lse, lse, zacc);
      ++nacc;
      if (l < k) count(q.id);
      if (LPR < 32)
        for (int j = l + LPR; j < k; j += LPR) count(__ldg(idx + (unsigned)(r * k + j)));
    };
    // the group's rows are g, g + kStep, ...; a warp's groups stay together
    const int first = t + warp * R::kGroups;
    Row even = {}, odd = {};
    if constexpr (R::kAhead) {
      if (first < end) load(even, first + g);
      for (int r0 = first; r0 < end; r0 += 2 * kStep) {
        load(odd, r0 + kStep + g);  // past the end: nothing is read, nothing counts
        add_row(even, r0 + g);
        if (r0 + kStep >= end) break;
        load(even, r0 + 2 * kStep + g);
        add_row(odd, r0 + kStep + g);
      }
    } else {
      for (int r0 = first; r0 < end; r0 += kStep) {
        load(even, r0 + g);
        add_row(even, r0 + g);
      }
    }
    // groups of the warp, then the block's 8 warps
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < NV / 2; ++i)
        acc[i] = add2(acc[i], __shfl_xor_sync(0xffffffffu, acc[i], o));
      zacc += __shfl_xor_sync(0xffffffffu, zacc, o);
      nacc += __shfl_xor_sync(0xffffffffu, nacc, o);
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        const float2 q = unpair(acc[i]);
        red[warp * R::kCols + col_of<LPR, VEC>(l, 2 * i)] = q.x;
        red[warp * R::kCols + col_of<LPR, VEC>(l, 2 * i + 1)] = q.y;
      }
    }
    if (lane == 0) zred[warp] = zacc, nred[warp] = nacc;
    __syncthreads();
    const bool alone = whole.loss && gridDim.x == 1;
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += 256) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) p += red[w * R::kCols + e];
      if (alone) {
        red[e] = p;  // the first warp's sum of e, which only this thread reads
      } else {
        part.prob[slot * E + e] = p;
        part.count[slot * E + e] = hist[e];
        hist[e] = 0;
      }
    }
    if (threadIdx.x == 0 && !alone) {
      float z = 0.f;
      int n = 0;
      for (int w = 0; w < 8; ++w) z += zred[w], n += nred[w];
      part.z[slot] = z;
      part.n[slot] = n;
    }
    __syncthreads();
    t = end;
    ++s;
  }
  if (bad_id) record_error(err, MOE_ERR_DEVICE_CHECK, 40);
  if (whole.loss)
    finish_whole(part, BalanceOwn{red, hist, zred, nred}, E, k, whole, err + kBalanceTicket);
}

// Block (x, s): 32 experts of sequence s, summed over the slots of the token
// blocks that meet it; W warps take the slots in turn (many warps when a
// sequence has many slots: the sums are a chain of loads).  The last block to
// finish (a ticket) adds the sequences' terms up in order.
template <int W>
__global__ void __launch_bounds__(32 * W) k_balance_finish(
    BalancePart part, const int* __restrict__ off, int S, int T, int E, int k, int C,
    float balance_coef, float z_coef, double* __restrict__ term, double* __restrict__ zterm,
    float* __restrict__ loss, int* __restrict__ counts, int* __restrict__ tokens,
    float* __restrict__ prob_mean, int* err, int* ticket) {
  __shared__ double pred[W][32], zr[W];
  __shared__ int cred[W][32], nr[W], is_last;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntile = gridDim.x;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  const int a0 = off ? __ldg(off + s) : 0, b0 = off ? __ldg(off + s + 1) : T;
  const int a = max(0, min(T, a0)), b = max(0, min(T, b0));
  if (threadIdx.x == 0 && (a != a0 || b != b0 || b < a))
    record_error(err, MOE_ERR_DEVICE_CHECK, 41);
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  if (b > a) {
    const int blk0 = a / C, blk1 = (b - 1) / C;
    if (e < E) {
      for (int q0 = blk0 + warp; q0 <= blk1; q0 += 8 * W) {
        float v[8];  // 16 loads in flight
        int m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const size_t at = ((size_t)q0 + i * W + s) * E + e;
          const bool in = q0 + i * W <= blk1;
          v[i] = in ? __ldcg(part.prob + at) : 0.f;
          m[i] = in ? __ldcg(part.count + at) : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) p += v[i], c += m[i];
      }
    }
    for (int q = blk0 + (int)threadIdx.x; q <= blk1; q += 32 * W) {
      z += part.z[q + s];
      n += part.n[q + s];
    }
  }
  pred[warp][lane] = p;
  cred[warp][lane] = c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane == 0) zr[warp] = z, nr[warp] = n;
  __syncthreads();
  if (warp == 0) {
    p = 0.0, c = 0, z = 0.0, n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) p += pred[w][lane], c += cred[w][lane], z += zr[w], n += nr[w];
    if (e < E) {
      counts[(size_t)s * E + e] = c;
      if (prob_mean) prob_mean[(size_t)s * E + e] = n > 0 ? (float)(p / n) : 0.f;
    }
    double f = e < E ? p * c : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    if (lane == 0) {
      term[(size_t)s * ntile + blockIdx.x] = n > 0 ? f * E / ((double)k * n * n) : 0.0;
      if (blockIdx.x == 0) {
        tokens[s] = n;
        zterm[s] = z;
      }
      __threadfence();
      const unsigned all = gridDim.x * gridDim.y;
      is_last = atomicAdd(reinterpret_cast<unsigned*>(ticket), 1u) == all - 1;
    }
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  double f = 0.0;
  z = 0.0;
  long long tot = 0;
  int live = 0;
  for (long long i = threadIdx.x; i < (long long)S * ntile; i += 32 * W) f += __ldcg(term + i);
  for (int i = threadIdx.x; i < S; i += 32 * W) {
    const int m = __ldcg(tokens + i);
    z += __ldcg(zterm + i);
    tot += m;
    live += m > 0;
  }
  __shared__ double fr[W];
  __shared__ long long tr[W];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    f += __shfl_xor_sync(0xffffffffu, f, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
    live += __shfl_xor_sync(0xffffffffu, live, o);
  }
  if (lane == 0) fr[warp] = f, zr[warp] = z, tr[warp] = tot, nr[warp] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    f = 0.0, z = 0.0, tot = 0, live = 0;
    for (int w = 0; w < W; ++w) f += fr[w], z += zr[w], tot += tr[w], live += nr[w];
    write_loss(f, z, tot, live, balance_coef, z_coef, loss, tokens + S);
    *ticket = 0;
  }
}

// ============================================================== gate gradient
// dL[t,e] = sum_j 1[idx_j = e] w_j (dw_j - sum_i w_i dw_i)
//         + g p_e (f_e - sum_e' f_e' p_e' + zc lse),
//   f_e = a E c_e / (S' k N_s^2), zc = 2 b / N: one pass, a warp takes a run of
// consecutive rows so that its sequence (and f, in registers) rarely changes.
// The k gate terms of a row go to their columns through a row of shared
// memory that is zero between rows.
// 131072 x 256, k = 8: 55 us (5.1 TB/s; 261 instructions a row and warp, issue
// slots 61% used, waiting for shuffles and the shared row as much as for loads).
struct GateArgs {
  const float* logits;
  const int* idx;
  const float* w;
  const float* dw;
  const uint8_t* mask;
  const int* off;
  const int* counts;
  const int* tokens;
  const float* dloss;
  float* dlogits;
  float balance_coef, z_coef;
  int S, T, E, k, rows_per_warp;
  int* err;
};

template <int LPR, int NV, bool VEC>
__global__ void __launch_bounds__(256, RowCfg<LPR, NV, VEC>::kGateBlocks)
    k_gate_bwd(const GateArgs a) {
  using R = RowCfg<LPR, NV, VEC>;
  constexpr int kStep = R::kGroups;
  extern __shared__ float sm[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, g = lane / LPR;
  float* grow = sm + (size_t)(warp * R::kGroups + g) * R::kCols;
#pragma unroll
  for (int c = 0; c < NV / 4; ++c)
    *reinterpret_cast<float4*>(grow + c * 4 * LPR + 4 * l) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
  const bool aux = a.counts != nullptr;
  const long long gw = (long long)blockIdx.x * 8 + warp;
  const int first = (int)min((long long)a.T, gw * a.rows_per_warp);
  const int last = (int)min((long long)a.T, (gw + 1) * a.rows_per_warp);
  float cf = 0.f, zc = 0.f;
  int live_seqs = 1;
  if (aux) {
    const float up = a.dloss ? __ldg(a.dloss) : 1.f;
    const int tot = __ldg(a.tokens + a.S);
    live_seqs = max(1, __ldg(a.tokens + a.S + 1));
    zc = a.z_coef != 0.f ? 2.f * a.z_coef * up / (float)max(1, tot) : 0.f;
    cf = a.balance_coef * up;
  }
  f32x2 f[NV / 2];
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) f[i] = 0;
  int seq = -2, seq_end = -1;  // [.., seq_end) is the run whose f is loaded
  bool bad_id = false;
  struct Row {
    f32x2 v[NV / 2];
    float w, dw;  // the lane's first slot
    int id;
    bool in;
  };
  auto load = [&](Row& q, int t) {
    q.in = t < last;
    q.id = -1;
    q.w = q.dw = 0.f;
    if (t < last) {
      if (aux) {
        load_row<LPR, NV, VEC>(a.logits + (unsigned)(t * a.E), a.E, l, q.v);
        if (a.mask) q.in = a.mask[t] != 0;
      }
      if (a.dw && l < a.k) {
        const unsigned at = t * a.k + l;
        q.id = __ldg(a.idx + at);
        q.w = __ldg(a.w + at);
        q.dw = __ldg(a.dw + at);
      }
    }
  };
  auto grad_row = [&](Row& q, int t) {
    const bool in = t < last;
    float top = 0.f, sum = 0.f, dot = 0.f;
    bool live = false;
    if (aux) {
      sum = row_exp<LPR, NV>(q.v, top, live);
      if (in && t >= seq_end) {
        seq = a.off ? find_seq(a.off, a.S, t) : 0;
        const bool real = seq >= 0 && seq < a.S;
        seq_end = !a.off || seq >= a.S ? a.T : __ldg(a.off + seq + 1);
        if (real && cf != 0.f) {
          const int n = max(1, __ldg(a.tokens + seq));
          const float per =
              cf * (float)a.E / ((float)live_seqs * (float)a.k * (float)n * (float)n);
          const int* c = a.counts + (size_t)seq * a.E;
#pragma unroll
          for (int i = 0; i < NV / 2; ++i) {
            const int e = col_of<LPR, VEC>(l, 2 * i), e1 = col_of<LPR, VEC>(l, 2 * i + 1);
            f[i] = pair(e < a.E ? per * (float)__ldg(c + e) : 0.f,
                        e1 < a.E ? per * (float)__ldg(c + e1) : 0.f);
          }
        }
      }
      live = live && q.in && seq >= 0 && seq < a.S;
      f32x2 d = mul2(f[0], q.v[0]);
#pragma unroll
      for (int i = 1; i < NV / 2; ++i) d = fma2(f[i], q.v[i], d);
      const float2 h = unpair(d);
      dot = h.x + h.y;
    }
    float dotw = q.w * q.dw;
    if (LPR < 32 && a.dw && in)
      for (int j = l + LPR; j < a.k; j += LPR) {
        const unsigned at = t * a.k + j;
        dotw = fmaf(__ldg(a.w + at), __ldg(a.dw + at), dotw);
      }
    sum3<LPR>(sum, dot, dotw);
    if (live) {
      // v / sum (f + zc lse - dot / sum)
      const float inv = rcp_fast(sum);
      const float add = inv * ((zc != 0.f ? zc * (top + log_fast(sum)) : 0.f) - dot * inv);
      const f32x2 inv2 = pair(inv, inv), more = pair(add, add);
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) q.v[i] = mul2(q.v[i], fma2(f[i], inv2, more));
    } else {
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) q.v[i] = 0;
    }
    if (a.dw) {
      // A step adds the slots j0 .. j0 + LPR - 1.  Ids are distinct in a token;
      // should two slots of a step share one, the lower slot goes first.
      for (int j0 = 0; j0 < a.k; j0 += LPR) {
        int e = q.id;
        float wj = q.w, dwj = q.dw;
        if (LPR < 32 && j0 > 0) {
          e = -1;
          if (in && j0 + l < a.k) {
            const unsigned at = t * a.k + j0 + l;
            e = __ldg(a.idx + at), wj = __ldg(a.w + at), dwj = __ldg(a.dw + at);
          }
        }
        if (in && j0 + l < a.k && (unsigned)e >= (unsigned)a.E) bad_id = true;
        const bool has = (unsigned)e < (unsigned)a.E;
        const float term = wj * (dwj - dotw);
        const unsigned same = __match_any_sync(0xffffffffu, has ? g * a.E + e : -1 - lane);
        const int before = __popc(same & ((1u << lane) - 1u));
        if (has && before == 0) grow[e] = LPR < 32 ? grow[e] + term : term;
        __syncwarp();
        for (int turn = 1; __any_sync(0xffffffffu, before >= turn); ++turn) {
          if (has && before == turn) grow[e] += term;
          __syncwarp();
        }
      }
      if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < NV / 4; ++c) {
          float4* at = reinterpret_cast<float4*>(grow + c * 4 * LPR + 4 * l);
          const float4 more = *at;
          q.v[2 * c] = add2(q.v[2 * c], pair(more.x, more.y));
          q.v[2 * c + 1] = add2(q.v[2 * c + 1], pair(more.z, more.w));
          if (LPR < 32) *at = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
          float* at = grow + 2 * i * LPR + l;
          q.v[i] = add2(q.v[i], pair(at[0], at[LPR]));
          if (LPR < 32) at[0] = at[LPR] = 0.f;
        }
      }
      __syncwarp();
      if (LPR == 32) {  // k <= 32: one slot a lane
        if ((unsigned)q.id < (unsigned)a.E) grow[q.id] = 0.f;
        __syncwarp();
      }
    }
    if (in) {
      float* out = a.dlogits + (unsigned)(t * a.E);
      if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < NV / 4; ++c) {
          const int e = c * 4 * LPR + 4 * l;
          const float2 o0 = unpair(q.v[2 * c]), o1 = unpair(q.v[2 * c + 1]);
          if (e < a.E)
            __stcs(reinterpret_cast<float4*>(out + e), make_float4(o0.x, o0.y, o1.x, o1.y));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
          const int e = 2 * i * LPR + l;
          const float2 o = unpair(q.v[i]);
          if (e < a.E) __stcs(out + e, o.x);
          if (e + LPR < a.E) __stcs(out + e + LPR, o.y);
        }
      }
    }
  };
  Row even = {}, odd = {};
  if constexpr (R::kAhead) {
    if (first < last) load(even, first + g);
    for (int r0 = first; r0 < last; r0 += 2 * kStep) {
      load(odd, r0 + kStep + g);  // past the end: nothing is read or written
      grad_row(even, r0 + g);
      if (r0 + kStep >= last) break;
      load(even, r0 + 2 * kStep + g);
      grad_row(odd, r0 + kStep + g);
    }
  } else {
    for (int r0 = first; r0 < last; r0 += kStep) {
      load(even, r0 + g);
      grad_row(even, r0 + g);
    }
  }
  if (bad_id) record_error(a.err, MOE_ERR_DEVICE_CHECK, 42);
}

// ============================================================== combine backward
// dw[t,j] = sum_c dy[t,c] z[row_of[t,j],c]; dz[row_of[t,j],c] = w[t,j] dy[t,c].
// G lanes per (token, slot): 8 or 16 for rows of 64 or 128 columns, else a warp, or
// the block's eight warps (G = 256) when there are few rows.  The slots of a token
// are neighbours, so dy's row comes from L1 for all but the first of them.  A row
// index outside [0, T*k) gives dw = 0 and writes nothing.
// Bound by HBM: 8192 x 2048, k = 8, dw and dz: 96 us (6.0 TB/s); 10294 x 64, k = 13,
// dw alone: 38 us with a warp for each row of 128 bytes, 9 with 8 lanes.
template <int G, bool DW, bool DZ>
__global__ void __launch_bounds__(256) k_combine_bwd(
    const __nv_bfloat16* __restrict__ dy, const __nv_bfloat16* __restrict__ z,
    const int* __restrict__ row_of, const float* __restrict__ w, long long P, int d, int k,
    float* __restrict__ dw, __nv_bfloat16* __restrict__ dz) {
  __shared__ float red[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long p = (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
  float acc = 0.f;
  if (p < P) {
    const long long r = __ldg(row_of + p);
    if (r >= 0 && r < P) {
      const float wj = DZ ? __ldg(w + p) : 0.f;
      const uint4* yr = reinterpret_cast<const uint4*>(dy + (size_t)(p / k) * d);
      const uint4* zr = reinterpret_cast<const uint4*>(z + (size_t)r * d);
      uint4* gr = reinterpret_cast<uint4*>(dz + (size_t)r * d);
      const int nv = d / 8;
      constexpr int U = G < 32 ? 1 : 4;
      for (int c0 = threadIdx.x % G; c0 < nv; c0 += U * G) {
        uint4 yv[U], zv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * G;
          yv[u] = zv[u] = make_uint4(0, 0, 0, 0);
          if (c < nv) {
            yv[u] = __ldg(yr + c);
            if (DW) zv[u] = __ldcs(zr + c);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * G;
          const __nv_bfloat162* y2 = reinterpret_cast<const __nv_bfloat162*>(&yv[u]);
          const __nv_bfloat162* z2 = reinterpret_cast<const __nv_bfloat162*>(&zv[u]);
          uint4 o;
          uint32_t* o2 = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = __bfloat1622float2(y2[i]);
            if (DW) {
              const float2 q = __bfloat1622float2(z2[i]);
              acc = fmaf(y.x, q.x, acc);
              acc = fmaf(y.y, q.y, acc);
            }
            if (DZ) o2[i] = pack_bf16x2(wj * y.x, wj * y.y);
          }
          if (DZ && c < nv) __stcs(gr + c, o);
        }
      }
    }
  }
  if (!DW) return;
  constexpr int kLanes = G < 32 ? G : 32;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (G <= 32) {
    if (lane % kLanes == 0 && p < P) dw[p] = acc;
    return;
  }
  if (lane == 0) red[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0 && p < P) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i];
    dw[p] = s;
  }
}

// fn(RowCfg) for the layout that holds E experts.
template <bool VEC, class F>
cudaError_t with_columns(int E, F&& fn) {
  if (E <= 4) return fn(RowCfg<1, 4, VEC>{});
  if (E <= 8) return fn(RowCfg<1, 8, VEC>{});
  if (E <= 16) return fn(RowCfg<2, 8, VEC>{});
  if (E <= 32) return fn(RowCfg<4, 8, VEC>{});
  if (E <= 64) return fn(RowCfg<8, 8, VEC>{});
  if (E <= 128) return fn(RowCfg<16, 8, VEC>{});
  if (E <= 256) return fn(RowCfg<32, 8, VEC>{});
  if (E <= 512) return fn(RowCfg<32, 16, VEC>{});
  return fn(RowCfg<32, 32, VEC>{});
}
template <class F>
cudaError_t with_rows(int E, bool vec, F&& fn) {
  return vec ? with_columns<true>(E, fn) : with_columns<false>(E, fn);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

cudaError_t launch_balance_loss(const float* logits, const int* idx, const uint8_t* mask,
                                const int* off, int S, const moe_shape& s, float balance_coef,
                                float z_coef, float* loss, int* counts, int* tokens,
                                float* prob_mean, const BwdLayout& L, char* ws, cudaStream_t st) {
  BalancePart part{reinterpret_cast<float*>(ws + L.prob), reinterpret_cast<int*>(ws + L.count),
                   reinterpret_cast<float*>(ws + L.z), reinterpret_cast<int*>(ws + L.n)};
  int* err = reinterpret_cast<int*>(ws);
  const bool vec = s.E % 4 == 0 && aligned16(logits);
  const int C = L.chunk, nblk = (s.T + C - 1) / C;
  const bool one = !off && nblk <= kWholeBlocks && nblk * s.E <= kWholeValues;
  const BalanceWhole whole{balance_coef, z_coef, one ? loss : nullptr, counts, tokens, prob_mean};
  cudaError_t e = with_rows(s.E, vec, [&](auto cfg) {
    using R = decltype(cfg);
    const size_t smem = sizeof(float) * 8 * R::kCols + sizeof(int) * s.E;
    return launch_kernel(k_balance_rows<R::kLpr, R::kNv, R::kVec>, dim3(nblk), dim3(256), smem,
                         st, 1, logits, idx, mask, off, S, s.T, s.E, s.k, C, part, err, whole);
  });
  if (e != cudaSuccess || one) return e;
  const auto finish = [&](auto kern, int warps) {
    return launch_kernel(kern, dim3((s.E + 31) / 32, S), dim3(32 * warps), 0, st, 1, part, off, S,
                         s.T, s.E, s.k, C, balance_coef, z_coef,
                         reinterpret_cast<double*>(ws + L.term),
                         reinterpret_cast<double*>(ws + L.zterm), loss, counts, tokens, prob_mean,
                         err, err + kBalanceTicket);
  };
  // 4 warps for sequences of up to 16 blocks on average, else 32
  return nblk <= 16 * S ? finish(k_balance_finish<4>, 4) : finish(k_balance_finish<32>, 32);
}

cudaError_t launch_gate_bwd(const float* logits, const int* idx, const float* w, const float* dw,
                            const uint8_t* mask, const int* off, int S, const int* counts,
                            const int* tokens, const moe_shape& s, float balance_coef,
                            float z_coef, const float* dloss, float* dlogits, int* err, int sms,
                            cudaStream_t st) {
  const bool vec = s.E % 4 == 0 && (!counts || aligned16(logits)) && aligned16(dlogits);
  GateArgs a{logits, idx, w, dw, mask, off, counts, tokens, dloss, dlogits, balance_coef, z_coef,
             S, s.T, s.E, s.k, 1, err};
  return with_rows(s.E, vec, [&](auto cfg) {
    using R = decltype(cfg);
    // One run of whole groups for each warp that the SMs hold (two or four rounds of
    // shorter runs: 3% and 10% slower at 131072 x 256).
    const long long warps = 8LL * R::kGateBlocks * sms;
    long long rows = (s.T + warps - 1) / warps;
    rows = (rows + R::kGroups - 1) / R::kGroups * R::kGroups;
    a.rows_per_warp = (int)rows;
    const long long nw = (s.T + rows - 1) / rows;
    const size_t smem = sizeof(float) * 8 * R::kGroups * R::kCols;
    return launch_kernel(k_gate_bwd<R::kLpr, R::kNv, R::kVec>, dim3((unsigned)((nw + 7) / 8)),
                         dim3(256), smem, st, 1, a);
  });
}

cudaError_t launch_combine_bwd(const __nv_bfloat16* dy, const __nv_bfloat16* z, const int* row_of,
                               const float* w, const moe_shape& s, float* dw, __nv_bfloat16* dz,
                               int sms, cudaStream_t st) {
  const long long P = (long long)s.T * s.k;
  // Few rows of some length: eight warps a row, so that more loads are in flight.
  const bool wide = P < 16LL * sms && s.d > 256;
  const int lanes = wide ? 256 : s.d == 64 ? 8 : s.d == 128 ? 16 : 32;
  const unsigned blocks = (unsigned)((P * lanes + 255) / 256);
  auto go = [&](auto kern) {
    return launch_kernel(kern, dim3(blocks), dim3(256), 0, st, 1, dy, z, row_of, w, P, s.d, s.k,
                         dw, dz);
  };
  auto pick = [&](auto g) {
    constexpr int G = decltype(g)::value;
    return dw && dz ? go(k_combine_bwd<G, true, true>)
                    : dw ? go(k_combine_bwd<G, true, false>) : go(k_combine_bwd<G, false, true>);
  };
  switch (lanes) {
    case 8: return pick(std::integral_constant<int, 8>{});
    case 16: return pick(std::integral_constant<int, 16>{});
    case 32: return pick(std::integral_constant<int, 32>{});
    default: return pick(std::integral_constant<int, 256>{});
  }
}

}  // namespace moe
