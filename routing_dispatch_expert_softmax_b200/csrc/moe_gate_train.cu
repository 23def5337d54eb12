// Training the gate: the balance loss with its per-expert counts, the
// gradient of the router logits, and the backward of the combine.
//
// The pages name the imbalance of the gate ("Serving MoE models with expert
// parallelism on 8xH200", section "Routing imbalance") but give no loss; the
// one here is the usual product of each expert's share of the selections and
// its mean probability, with the mean squared logsumexp beside it.
#include "moe_kernels.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- row layout
// A group of LPR lanes owns one row of E fp32 logits, NV values a lane in
// chunks of 4: chunk v of lane l holds the columns v * 4 * LPR + 4 l + (0..3),
// so a group's 16-byte loads are contiguous.  Up to 128 experts a lane holds
// 4 values and a warp 32 / LPR rows at once; above, a whole warp takes one row.
template <int LPR, int NV>
struct RowCfg {
  static constexpr int kLpr = LPR, kNv = NV;
  static constexpr int kGroups = 32 / LPR;  // rows of a warp at once
  static constexpr int kCols = LPR * NV;    // columns a group can hold
};

template <int LPR, int NV>
__device__ __forceinline__ int col_of(int l, int i) {
  return (i >> 2) * (4 * LPR) + 4 * l + (i & 3);
}

// Columns at or past E read as -inf: their exp is 0 and they never are the
// maximum.  vec: rows are 16-byte aligned (E % 4 == 0 and the base is).
template <int LPR, int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, bool vec,
                                         float (&v)[NV]) {
#pragma unroll
  for (int c = 0; c < NV / 4; ++c) {
    const int e = c * 4 * LPR + 4 * l;
    if (vec) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) q = __ldcs(reinterpret_cast<const float4*>(row + e));
      v[4 * c] = q.x, v[4 * c + 1] = q.y, v[4 * c + 2] = q.z, v[4 * c + 3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * c + i] = e + i < E ? __ldcs(row + e + i) : -INFINITY;
    }
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int LPR>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The row's values become exp(v - max); returns their sum and the maximum.
// live: some value is not -inf (a NaN counts: it has to show in the result).
// A row without a live value gives exp values of 0 and a sum of 0.
template <int LPR, int NV>
__device__ __forceinline__ float row_exp(float (&v)[NV], float& top, bool& live) {
  float m = -INFINITY;
  bool some = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    m = fmaxf(m, v[i]);
    some |= v[i] != -INFINITY;
  }
  m = group_max<LPR>(m);
  unsigned votes = __ballot_sync(0xffffffffu, some);
  const int g0 = (threadIdx.x & 31) / LPR * LPR;
  live = LPR == 32 ? votes != 0 : ((votes >> g0) & ((1u << (LPR & 31)) - 1u)) != 0;
  // all -inf beside a NaN leaves m = -inf; 0 instead keeps the -inf columns at 0
  const float sub = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = expf(v[i] - sub);
    s += v[i];
  }
  top = sub;
  return group_sum<LPR>(s);
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
struct BalancePart {
  float* prob;  // [nblk + S][E]
  int* count;   // [nblk + S][E]
  float* z;     // [nblk + S]
  int* n;       // [nblk + S]
};

template <int LPR, int NV>
__global__ void __launch_bounds__(256) k_balance_rows(
    const float* __restrict__ logits, const int* __restrict__ idx,
    const uint8_t* __restrict__ mask, const int* __restrict__ off, int S, int T, int E, int k,
    int C, int vec, BalancePart part, int* err) {
  using R = RowCfg<LPR, NV>;
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
    if (end <= t) {  // an empty sequence
      ++s;
      continue;
    }
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    float zacc = 0.f;
    int nacc = 0;
    for (int r0 = t + warp * R::kGroups; r0 < end; r0 += 8 * R::kGroups) {
      const int r = r0 + g;
      const bool in = r < end && (!mask || mask[r]);
      float v[NV];
      if (in) {
        load_row<LPR, NV>(logits + (size_t)r * E, E, l, vec, v);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = -INFINITY;
      }
      float top;
      bool live;
      const float sum = row_exp<LPR, NV>(v, top, live);
      if (in && live) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += v[i] * inv;
        if (l == 0) {
          const float lse = top + logf(sum);
          zacc += lse * lse;
          ++nacc;
        }
        for (int j = l; j < k; j += LPR) {
          const int e = __ldg(idx + (size_t)r * k + j);
          if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
          else bad_id = true;
        }
      }
    }
    // groups of the warp, then the block's 8 warps
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      zacc += __shfl_xor_sync(0xffffffffu, zacc, o);
      nacc += __shfl_xor_sync(0xffffffffu, nacc, o);
    }
    if (g == 0) {
#pragma unroll
      for (int c = 0; c < NV / 4; ++c)
        *reinterpret_cast<float4*>(red + warp * R::kCols + c * 4 * LPR + 4 * l) =
            make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
    }
    if (lane == 0) zred[warp] = zacc, nred[warp] = nacc;
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += 256) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) p += red[w * R::kCols + e];
      part.prob[slot * E + e] = p;
      part.count[slot * E + e] = hist[e];
      hist[e] = 0;
    }
    if (threadIdx.x == 0) {
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
}

// Block (x, s): 32 experts of sequence s, summed over the slots of the token
// blocks that meet it; 8 warps take the slots in turn.  The last block to
// finish (a ticket) adds the sequences' terms up in order.
__global__ void __launch_bounds__(256) k_balance_finish(
    BalancePart part, const int* __restrict__ off, int S, int T, int E, int k, int C,
    float balance_coef, float z_coef, double* __restrict__ term, double* __restrict__ zterm,
    float* __restrict__ loss, int* __restrict__ counts, int* __restrict__ tokens,
    float* __restrict__ prob_mean, int* err, int* ticket) {
  __shared__ double pred[8][32], zr[8];
  __shared__ int cred[8][32], nr[8], is_last;
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
    for (int q = blk0 + warp; q <= blk1; q += 8) {
      const size_t slot = (size_t)q + s;
      if (e < E) {
        p += part.prob[slot * E + e];
        c += part.count[slot * E + e];
      }
    }
    for (int q = blk0 + (int)threadIdx.x; q <= blk1; q += 256) {
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
    for (int w = 0; w < 8; ++w) p += pred[w][lane], c += cred[w][lane], z += zr[w], n += nr[w];
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
  for (long long i = threadIdx.x; i < (long long)S * ntile; i += 256) f += __ldcg(term + i);
  for (int i = threadIdx.x; i < S; i += 256) {
    const int m = __ldcg(tokens + i);
    z += __ldcg(zterm + i);
    tot += m;
    live += m > 0;
  }
  __shared__ double fr[8];
  __shared__ long long tr[8];
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
    for (int w = 0; w < 8; ++w) f += fr[w], z += zr[w], tot += tr[w], live += nr[w];
    // a coefficient of 0 leaves its term out, whatever the term is
    const double lb = live > 0 && balance_coef != 0.f ? balance_coef * f / live : 0.0;
    const double lz = tot > 0 && z_coef != 0.f ? z_coef * z / (double)tot : 0.0;
    loss[0] = (float)(lb + lz);
    loss[1] = (float)lb;
    loss[2] = (float)lz;
    tokens[S] = (int)tot;
    tokens[S + 1] = live;
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
  int S, T, E, k, rows_per_warp, vec;
  int* err;
};

template <int LPR, int NV>
__global__ void __launch_bounds__(256) k_gate_bwd(const GateArgs a) {
  using R = RowCfg<LPR, NV>;
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
  const long long first = gw * a.rows_per_warp;
  const long long last = min((long long)a.T, first + a.rows_per_warp);
  float cf = 0.f, zc = 0.f;
  int live_seqs = 1;
  if (aux) {
    const float up = a.dloss ? __ldg(a.dloss) : 1.f;
    const int tot = __ldg(a.tokens + a.S);
    live_seqs = max(1, __ldg(a.tokens + a.S + 1));
    zc = a.z_coef != 0.f ? 2.f * a.z_coef * up / (float)max(1, tot) : 0.f;
    cf = a.balance_coef * up;
  }
  float f[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) f[i] = 0.f;
  int seq = -2, seq_end = -1;  // [.., seq_end) is the run whose f is loaded
  bool bad_id = false;
  for (long long r0 = first; r0 < last; r0 += R::kGroups) {
    const int t = (int)(r0 + g);
    const bool in = r0 + g < last;
    float v[NV], sum = 0.f, top = 0.f;
    bool live = false;
    if (aux) {
      bool use = in && (!a.mask || a.mask[t]);
      if (in && t >= seq_end) {
        seq = a.off ? find_seq(a.off, a.S, t) : 0;
        const bool real = seq >= 0 && seq < a.S;
        seq_end = !a.off || seq >= a.S ? a.T : __ldg(a.off + seq + 1);
        if (real && cf != 0.f) {
          const int n = max(1, __ldg(a.tokens + seq));
          const float per =
              cf * (float)a.E / ((float)live_seqs * (float)a.k * (float)n * (float)n);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = col_of<LPR, NV>(l, i);
            f[i] = e < a.E ? per * (float)__ldg(a.counts + (size_t)seq * a.E + e) : 0.f;
          }
        }
      }
      use = use && seq >= 0 && seq < a.S;
      if (use) {
        load_row<LPR, NV>(a.logits + (size_t)t * a.E, a.E, l, a.vec, v);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = -INFINITY;
      }
      sum = row_exp<LPR, NV>(v, top, live);
      live = live && use;
      float dot = 0.f;
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] *= inv;
        dot = fmaf(f[i], v[i], dot);
      }
      dot = group_sum<LPR>(dot);
      const float add = (zc != 0.f ? zc * (top + logf(sum)) : 0.f) - dot;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = live ? v[i] * (f[i] + add) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = 0.f;
    }
    if (a.dw) {
      float dotw = 0.f;
      if (in)
        for (int j = l; j < a.k; j += LPR)
          dotw = fmaf(__ldg(a.w + (size_t)t * a.k + j), __ldg(a.dw + (size_t)t * a.k + j), dotw);
      dotw = group_sum<LPR>(dotw);
      // A step adds the slots j0 .. j0 + LPR - 1.  Ids are distinct in a token;
      // should two slots of a step share one, the lower slot goes first.
      for (int j0 = 0; j0 < a.k; j0 += LPR) {
        const int j = j0 + l;
        int e = -1;
        float add = 0.f;
        if (in && j < a.k) {
          const size_t at = (size_t)t * a.k + j;
          e = __ldg(a.idx + at);
          if (e < 0 || e >= a.E) e = -1, bad_id = true;
          const float wj = __ldg(a.w + at);
          add = wj * (__ldg(a.dw + at) - dotw);
        }
        const unsigned same = __match_any_sync(0xffffffffu, e < 0 ? -1 - lane : g * a.E + e);
        const int before = __popc(same & ((1u << lane) - 1u));
        int most = before;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        for (int turn = 0; turn <= most; ++turn) {
          if (e >= 0 && before == turn) grow[e] += add;
          __syncwarp();
        }
      }
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) {
        float4* q = reinterpret_cast<float4*>(grow + c * 4 * LPR + 4 * l);
        const float4 add = *q;
        v[4 * c] += add.x, v[4 * c + 1] += add.y, v[4 * c + 2] += add.z, v[4 * c + 3] += add.w;
        *q = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      __syncwarp();
    }
    if (in) {
      float* out = a.dlogits + (size_t)t * a.E;
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) {
        const int e = c * 4 * LPR + 4 * l;
        if (a.vec) {
          if (e < a.E)
            __stcs(reinterpret_cast<float4*>(out + e),
                   make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < a.E) __stcs(out + e + i, v[4 * c + i]);
        }
      }
    }
  }
  if (bad_id) record_error(a.err, MOE_ERR_DEVICE_CHECK, 42);
}

// ============================================================== combine backward
// dw[t,j] = sum_c dy[t,c] z[row_of[t,j],c]; dz[row_of[t,j],c] = w[t,j] dy[t,c].
// WPR warps per (token, slot): the slots of a token are neighbours, so dy's
// row comes from L1 for all but the first of them.  A row index outside
// [0, T*k) gives dw = 0 and writes nothing.
template <int WPR, bool DW, bool DZ>
__global__ void __launch_bounds__(256) k_combine_bwd(
    const __nv_bfloat16* __restrict__ dy, const __nv_bfloat16* __restrict__ z,
    const int* __restrict__ row_of, const float* __restrict__ w, long long P, int d, int k,
    float* __restrict__ dw, __nv_bfloat16* __restrict__ dz) {
  __shared__ float red[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long p = (long long)blockIdx.x * (8 / WPR) + warp / WPR;
  float acc = 0.f;
  if (p < P) {
    const long long r = __ldg(row_of + p);
    if (r >= 0 && r < P) {
      const float wj = DZ ? __ldg(w + p) : 0.f;
      const uint4* yr = reinterpret_cast<const uint4*>(dy + (size_t)(p / k) * d);
      const uint4* zr = reinterpret_cast<const uint4*>(z + (size_t)r * d);
      uint4* gr = reinterpret_cast<uint4*>(dz + (size_t)r * d);
      const int nv = d / 8;
      constexpr int U = 4, kStep = 32 * WPR;
      for (int c0 = (warp % WPR) * 32 + lane; c0 < nv; c0 += U * kStep) {
        uint4 yv[U], zv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * kStep;
          yv[u] = zv[u] = make_uint4(0, 0, 0, 0);
          if (c < nv) {
            yv[u] = __ldg(yr + c);
            if (DW) zv[u] = __ldcs(zr + c);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * kStep;
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (WPR == 1) {
    if (lane == 0 && p < P) dw[p] = acc;
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
template <class F>
cudaError_t with_rows(int E, F&& fn) {
  if (E <= 4) return fn(RowCfg<1, 4>{});
  if (E <= 8) return fn(RowCfg<2, 4>{});
  if (E <= 16) return fn(RowCfg<4, 4>{});
  if (E <= 32) return fn(RowCfg<8, 4>{});
  if (E <= 64) return fn(RowCfg<16, 4>{});
  if (E <= 128) return fn(RowCfg<32, 4>{});
  if (E <= 256) return fn(RowCfg<32, 8>{});
  if (E <= 512) return fn(RowCfg<32, 16>{});
  return fn(RowCfg<32, 32>{});
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
  const int vec = s.E % 4 == 0 && aligned16(logits);
  const int C = L.chunk, nblk = (s.T + C - 1) / C;
  cudaError_t e = with_rows(s.E, [&](auto cfg) {
    using R = decltype(cfg);
    const size_t smem = sizeof(float) * 8 * R::kCols + sizeof(int) * s.E;
    return launch_kernel(k_balance_rows<R::kLpr, R::kNv>, dim3(nblk), dim3(256), smem, st, 1,
                         logits, idx, mask, off, S, s.T, s.E, s.k, C, vec, part, err);
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(k_balance_finish, dim3((s.E + 31) / 32, S), dim3(256), 0, st, 1, part, off,
                       S, s.T, s.E, s.k, C, balance_coef, z_coef,
                       reinterpret_cast<double*>(ws + L.term),
                       reinterpret_cast<double*>(ws + L.zterm), loss, counts, tokens, prob_mean,
                       err, err + kBalanceTicket);
}

cudaError_t launch_gate_bwd(const float* logits, const int* idx, const float* w, const float* dw,
                            const uint8_t* mask, const int* off, int S, const int* counts,
                            const int* tokens, const moe_shape& s, float balance_coef,
                            float z_coef, const float* dloss, float* dlogits, int* err, int sms,
                            cudaStream_t st) {
  const int vec = s.E % 4 == 0 && (!counts || aligned16(logits)) && aligned16(dlogits);
  GateArgs a{logits, idx, w, dw, mask, off, counts, tokens, dloss, dlogits, balance_coef, z_coef,
             S, s.T, s.E, s.k, 1, vec, err};
  return with_rows(s.E, [&](auto cfg) {
    using R = decltype(cfg);
    // Runs of rows: enough warps for 8 blocks an SM, whole groups of rows each.
    const long long warps = 64LL * sms;
    long long rows = (s.T + warps - 1) / warps;
    rows = (rows + R::kGroups - 1) / R::kGroups * R::kGroups;
    a.rows_per_warp = (int)rows;
    const long long nw = (s.T + rows - 1) / rows;
    const size_t smem = sizeof(float) * 8 * R::kGroups * R::kCols;
    return launch_kernel(k_gate_bwd<R::kLpr, R::kNv>, dim3((unsigned)((nw + 7) / 8)), dim3(256),
                         smem, st, 1, a);
  });
}

cudaError_t launch_combine_bwd(const __nv_bfloat16* dy, const __nv_bfloat16* z, const int* row_of,
                               const float* w, const moe_shape& s, float* dw, __nv_bfloat16* dz,
                               int sms, cudaStream_t st) {
  const long long P = (long long)s.T * s.k;
  // Few rows: eight warps a row, so that more loads are in flight.
  const bool wide = P < 16LL * sms;
  const unsigned blocks = (unsigned)(wide ? P : (P + 7) / 8);
  auto go = [&](auto kern) {
    return launch_kernel(kern, dim3(blocks), dim3(256), 0, st, 1, dy, z, row_of, w, P, s.d, s.k,
                         dw, dz);
  };
  if (wide)
    return dw && dz ? go(k_combine_bwd<8, true, true>)
                    : dw ? go(k_combine_bwd<8, true, false>) : go(k_combine_bwd<8, false, true>);
  return dw && dz ? go(k_combine_bwd<1, true, true>)
                  : dw ? go(k_combine_bwd<1, true, false>) : go(k_combine_bwd<1, false, true>);
}

}  // namespace moe
