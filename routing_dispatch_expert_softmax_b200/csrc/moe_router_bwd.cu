// Backward of the router product L = x W_g + b:
//   dW[i,e] = sum_t x[t,i] dL[t,e],  db[e] = sum_t dL[t,e],
//   dx[t,i] = sum_e dL[t,e] W[i,e]
// on the sm_100a tensor cores.  dL and W are fp32; the tensor cores take 16-bit
// operands.  A first kernel prepares them:
//   dW: dL splits into three bf16 planes of 8 bits each, hi + mid + lo = v.  x is
//       bf16, so the three products are exact and dW is as good as an fp32
//       product's;
//   dx: dL and W split into two fp16 parts of 11 bits each, of which lo lo, 2^-22 of
//       a product, is left out.  One part would be a third of the MMAs, but where terms
//       cancel (a softmax's gradients sum to zero over a row, and W's columns may
//       have much in common) its 2^-11 and not bf16's 2^-8 is the error that remains.
//       Each row is first scaled by an even power of two that brings its largest value
//       to [2^13, 2^15), so that no value overflows and only those below 2^-16 of the
//       row's largest lose bits (2^-38 of it at most); the epilogue scales back.
// One persistent kernel then runs the tiles of both products.  The tokens are
// the long axis of dW, so its tiles split over token ranges; a last kernel
// adds the ranges' partial tiles in order.  Few tokens take one kernel of their own.
//
// 16384 x 7168 x 256: 306 us (361 GFLOP of 16-bit products, dW's three and dx's three a
// term: 259 at the rate that the power limit leaves a library product), of which dW
// alone is 156 and dx alone 159, and 361 us back to back.  8192 x 2048 x 128: 38 us,
// dW alone 23 and dx alone 18 (the operands' kernel and the sum are 5 and 4 of it, an
// item's start and end 2).
#include <cuda_fp16.h>

#include <atomic>

#include "moe_kernels.cuh"

namespace moe {

namespace {

// ============================================================== planes
// Two values as pairs of bf16 (a in the low half): hi has the upper 8 bits of the
// mantissa as they stand, the rest v - hi is exact, mid has its upper 8 bits and lo the
// last 8: nothing is rounded.  11 instructions a pair; rounding each part to nearest,
// with its care for overflow, took four times as many (few tokens: 64 x
// 2048 x 128 6.0 us in place of 6.8; the three kernels 0.4 less).  inf leaves
// NaN in the rest, and a NaN as well.
struct Split3 {
  uint32_t hi, mid, lo;
};
__device__ __forceinline__ Split3 split3(float a, float b) {
  const auto upper = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); };
  const auto halves = [](float x, float y) {
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  };
  Split3 s;
  s.hi = halves(a, b);
  a -= upper(a), b -= upper(b);
  s.mid = halves(a, b);
  s.lo = halves(a - upper(a), b - upper(b));
  return s;
}

// The even power of two that brings |top| to [2^13, 2^15) (1 for 0, inf and NaN; at
// most 2^126, for rows below 2^-112), and the square root of its inverse.
__device__ __forceinline__ void half_scale(float top, float& scale, float& back) {
  const int e = (__float_as_int(top) >> 23) & 0xff;  // top >= 0; biased exponent
  const int h = e == 255 || top == 0.f ? 0 : min(63, (127 + 14 - e) >> 1);
  scale = __int_as_float((2 * h + 127) << 23);
  back = __int_as_float((127 - h) << 23);
}

// One [rows, cols] fp32 matrix a; every output is optional:
//   planes                its bf16 planes: plane p of row r at r * row + p * plane,
//                         `width` columns (zeros from cols on); with zero_plane a
//                         fourth of zeros
//   half [rows][2][cp], back [rows]  its rows scaled, in two fp16 parts (rounded, and
//                         the rounded rest), cp = cols rounded up to 64 with zeros,
//                         and the square roots of the factors that undo the scaling
//   sums [block][cols]    column sums of each block's rows, in fp32 (T / 592 + 32 rows
//                         at most, each thread a few of them; the blocks' go into fp64)
struct PlanesArgs {
  const float* a;
  __nv_bfloat16* planes;
  __half* half;
  __nv_bfloat16* back;
  float* sums;
  long long rows, row, plane;
  int cols, cp, width, zero_plane, rows_per_block, blocks, vec;
};

// G lanes take a row, 8 neighbouring columns of every 8 G-th.
template <int G, int NO>
__device__ void planes_block(const PlanesArgs& p, int block, float* red) {
  constexpr int kPar = 256 / G;
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  const long long first = (long long)block * p.rows_per_block;
  const long long last = min(p.rows, first + p.rows_per_block);
  float sum[NO][8];
#pragma unroll
  for (int n = 0; n < NO; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[n][i] = 0.f;
  for (long long r0 = first; r0 < last; r0 += kPar) {
    const long long r = r0 + g;
    float v[NO][8], top = 0.f;
#pragma unroll
    for (int n = 0; n < NO; ++n) {
      const int c0 = 8 * (l + n * G);
      const float* src = p.a + r * p.cols + c0;
      if (r < last && p.vec && c0 + 8 <= p.cols) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(src));
        const float4 y = __ldg(reinterpret_cast<const float4*>(src) + 1);
        v[n][0] = x.x, v[n][1] = x.y, v[n][2] = x.z, v[n][3] = x.w;
        v[n][4] = y.x, v[n][5] = y.y, v[n][6] = y.z, v[n][7] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[n][i] = r < last && c0 + i < p.cols ? __ldg(src + i) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[n][i] += v[n][i];
        top = fmaxf(top, fabsf(v[n][i]));
      }
    }
    float scale = 1.f, back = 1.f;
    if (p.half) {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      half_scale(top, scale, back);
      if (l == 0 && r < last) p.back[r] = __float2bfloat16_rn(back);
    }
#pragma unroll
    for (int n = 0; n < NO; ++n) {
      const int c0 = 8 * (l + n * G);
      if (r >= last || c0 >= p.cp) continue;
      if (p.planes && c0 < p.width) {
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Split3 q = split3(v[n][2 * i], v[n][2 * i + 1]);
          w[0][i] = q.hi, w[1][i] = q.mid, w[2][i] = q.lo;
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<uint4*>(p.planes + r * p.row + q * p.plane + c0) =
              make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        if (p.zero_plane)
          *reinterpret_cast<uint4*>(p.planes + r * p.row + 3 * p.plane + c0) =
              make_uint4(0, 0, 0, 0);
      }
      if (p.half) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = v[n][2 * i] * scale, b = v[n][2 * i + 1] * scale;
          const __half2 h = __floats2half2_rn(a, b);
          const float2 f = __half22float2(h);
          const __half2 rest = __floats2half2_rn(a - f.x, b - f.y);  // the differences are exact
          hi[i] = *reinterpret_cast<const uint32_t*>(&h);
          lo[i] = *reinterpret_cast<const uint32_t*>(&rest);
        }
        __half* to = p.half + (size_t)r * 2 * p.cp + c0;
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + p.cp) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int n = 0; n < NO; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * (l + n * G) + i;
      if (c < p.cp) red[g * p.cp + c] = sum[n][i];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    float s = 0.f;
#pragma unroll 8
    for (int r = 0; r < kPar; ++r) s += red[r * p.cp + c];
    p.sums[(size_t)block * p.cols + c] = s;
  }
}

// Blocks [0, dl.blocks) prepare dL, the others W.
template <int G, int NO>
__global__ void __launch_bounds__(256) k_router_planes(const PlanesArgs dl, const PlanesArgs w) {
  extern __shared__ float sm[];  // [256 / G][cp]
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < dl.blocks) planes_block<G, NO>(dl, blockIdx.x, sm);
  else planes_block<G, NO>(w, blockIdx.x - dl.blocks, sm);
}

// ============================================================== products
// One work item is a 128 x 256 tile of fp32 sums in TMEM:
//   dW: rows = 128 experts, columns = 256 of d, K = the tokens of one range;
//       A = dL planes and B = x, both with the non-K index contiguous
//       (MN-major): tiles of 64 tokens x 64 columns, 128 bytes a row;
//   dx: rows = 128 tokens, columns = 256 of d, K = experts; A = dL and B = W in two
//       fp16 parts each, all K-major: lo hi, hi lo and hi hi (the small ones first).
// dW takes the experts as rows so that a row of 256 columns of x serves the
// three planes, and a lane's accumulator row is one expert: the 32 lanes of a
// warp then store 32 neighbouring experts of dW[i, :].
// Shared memory: a ring of 16 KB A tiles and one of 32 KB B tiles (128-byte
// swizzle).  For each 64 of K, dW takes `sets` A (RouterPlanes) and 1 B tiles, dx two of
// each; with up to 128 experts a block keeps the W tiles of its 256 columns in the B
// ring while it goes down the tokens, so that a dx item loads 64 KB at most.
//
// The tensor cores cut, not round, when they add to an fp32 accumulator, so a
// sum is short by about 2^-25 of itself for every MMA in a row (measured: dW
// 2.4e-5 short over 3,000 tokens, 600 MMAs).  dW therefore leaves TMEM after
// every kChunk = 2 blocks of 64 tokens: the epilogue warps add the chunk's 128
// x 256 sums to registers, in fp32 to nearest, while the MMAs fill the other
// accumulator.  A block's small terms (lo, mid) go before its hi: 16 cuts of
// full size in a chunk at most.
//
// Order of work: a block has its dW items first, then a run of dx items long
// enough that all blocks end together (dx_first).
struct RouterGemmArgs {
  int T, d, E;
  int dw_items, dx_items;
  int ne, nd;            // expert and column tiles of dW
  int sets, parts;       // RouterPlanes
  int rb;                // tiles of the B ring
  int kblocks, kper;     // 64-token blocks in all, and of one range
  int mt;                // token tiles of dx
  int kx;                // 64-expert blocks of dx
  int light_dx;          // dx items of the blocks that have one dW item less
  const __nv_bfloat16* dl_back;  // [T], [d]: roots of the factors that undo the scaling
  const __nv_bfloat16* w_back;
  float* dw;             // [ranges][parts][d][E]
  int* err;
};

// The dx items [first, last) of block c of g: blocks [0, heavy) have one dW
// item more than the others; those others share the first light_dx items.
__device__ __forceinline__ void dx_run(const RouterGemmArgs& a, int c, int g, int& first,
                                       int& last) {
  const int heavy = a.dw_items % g;
  const bool is_heavy = c < heavy;
  const long long base = is_heavy ? a.light_dx : 0;
  const long long n = is_heavy ? a.dx_items - a.light_dx : a.light_dx;
  const long long j = is_heavy ? c : c - heavy, m = is_heavy ? heavy : g - heavy;
  first = (int)(base + n * j / m);
  last = (int)(base + n * (j + 1) / m);
}

constexpr int kChunk = 2;
constexpr int kRA = 4, kRB = 4;
constexpr int kATile = 128 * 64 * 2, kBTile = 256 * 64 * 2;
constexpr int kStageOut = 2 * 32 * 64;  // per epilogue warp: two times 32 rows x 32 bf16 of dx
constexpr int router_smem(int rb) {
  return kRA * kATile + rb * kBTile + 8 * kStageOut + 1024 + 256;
}
constexpr int kRouterThreads = 320;  // TMA, MMA and eight epilogue warps

// Descriptor of an MN-major operand tile with 128-byte swizzle: blocks of 64
// MN values (one 128-byte row per K index), 8 K rows in 1024 bytes (stride
// byte offset), 64 K rows to the next block of 64 MN values (leading byte
// offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFF) | (uint64_t)(8192 >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, uint64_t* bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, const void* src, int c0,
                                             int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::
          "l"(reinterpret_cast<uint64_t>(tm)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}

// 32 lanes x 16 columns (the registers beside 128 sums hold no more)
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, phase ^= 1u;
  }
};

__global__ void __launch_bounds__(kRouterThreads, 1) k_router_gemm(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dl_mn,
    const __grid_constant__ CUtensorMap tm_dl_k, const __grid_constant__ CUtensorMap tm_w,
    const __grid_constant__ CUtensorMap tm_dx, const RouterGemmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sa = smem;
  uint8_t* sb = smem + kRA * kATile;
  const int rb = args.rb;
  uint8_t* so = sb + rb * kBTile;
  uint64_t* a_full = reinterpret_cast<uint64_t*>(so + 8 * kStageOut);
  uint64_t* a_empty = a_full + kRA;
  uint64_t* b_full = a_empty + kRA;
  uint64_t* b_empty = b_full + kRB;
  uint64_t* tfull = b_empty + kRB;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRA; ++s) mbar_init(&a_full[s], 1), mbar_init(&a_empty[s], 1);
    for (int s = 0; s < kRB; ++s) mbar_init(&b_full[s], 1), mbar_init(&b_empty[s], 1);
    for (int a = 0; a < 2; ++a) mbar_init(&tfull[a], 1), mbar_init(&tempty[a], 256);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    if (args.dw_items) prefetch_tensormap(&tm_x), prefetch_tensormap(&tm_dl_mn);
    if (args.dx_items)
      prefetch_tensormap(&tm_dl_k), prefetch_tensormap(&tm_w), prefetch_tensormap(&tm_dx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();
  int dx0, dx1;
  dx_run(args, blockIdx.x, gridDim.x, dx0, dx1);

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producer
      const uint64_t policy = policy_evict_normal();
      Ring a, b;
      int a_fills[kRA], b_fills[kRB];
#pragma unroll
      for (int s = 0; s < kRA; ++s) a_fills[s] = 0;
#pragma unroll
      for (int s = 0; s < kRB; ++s) b_fills[s] = 0;
      bool ok = true;
      auto take_a = [&]() -> uint8_t* {
        if (!mbar_wait_bounded(&a_empty[a.slot], a.phase ^ 1u, abort_flag)) return nullptr;
        mbar_arrive_expect_tx(&a_full[a.slot], kATile);
        ++a_fills[a.slot];
        return sa + a.slot * kATile;
      };
      auto take_b = [&]() -> uint8_t* {
        if (!mbar_wait_bounded(&b_empty[b.slot], b.phase ^ 1u, abort_flag)) return nullptr;
        mbar_arrive_expect_tx(&b_full[b.slot], kBTile);
        ++b_fills[b.slot];
        return sb + b.slot * kBTile;
      };
      for (int w = blockIdx.x; w < args.dw_items && ok; w += gridDim.x) {
        const int et = w % args.ne, q = w / args.ne, dt = q % args.nd, range = q / args.nd;
        const int kb1 = min(args.kblocks, (range + 1) * args.kper);
        for (int kb = range * args.kper; kb < kb1 && ok; ++kb) {
          uint8_t* dst = take_b();
          if (!(ok = dst != nullptr)) break;
          tma_load_3d(dst, &tm_x, &b_full[b.slot], 0, kb * 64, dt * 4);
          b.next(rb);
          for (int p = args.sets - 1; p >= 0; --p) {
            dst = take_a();
            if (!(ok = dst != nullptr)) break;
            const bool apart = args.sets == 3;  // each plane for itself
            tma_load_4d(dst, &tm_dl_mn, &a_full[a.slot], 0, kb * 64, apart ? et * 2 : p * 2,
                        apart ? p : 0);
            a.next(kRA);
          }
        }
      }
      int nt = dx0 / args.mt, mt = dx0 - nt * args.mt;
      for (int w = dx0; w < dx1 && ok; ++w) {
        const bool load_b = 2 * args.kx > rb || w == dx0 || mt == 0;
        for (int i = 0; i < 2 * args.kx && ok; ++i) {  // W hi, dL lo; W lo, dL hi
          const int hi = (i >> 1) * 64, lo = hi + args.kx * 64;
          uint8_t* dst;
          if (load_b) {
            dst = take_b();
            if (!(ok = dst != nullptr)) break;
            tma_load_2d(dst, &tm_w, &b_full[b.slot], i & 1 ? lo : hi, nt * 256, policy);
            b.next(rb);
          }
          dst = take_a();
          if (!(ok = dst != nullptr)) break;
          tma_load_2d(dst, &tm_dl_k, &a_full[a.slot], i & 1 ? hi : lo, mt * 128, policy);
          a.next(kRA);
        }
        if (++mt == args.mt) mt = 0, ++nt;
      }
      if (*abort_flag) {
        // Let every copy already issued land before the CTA leaves.
        const unsigned long long t0 = globaltimer();
#pragma unroll
        for (int s = 0; s < kRA; ++s)
          while (a_fills[s] > 0 && !mbar_try_wait(&a_full[s], (a_fills[s] - 1) & 1) &&
                 globaltimer() - t0 < 100000000ull) {}
#pragma unroll
        for (int s = 0; s < kRB; ++s)
          while (b_fills[s] > 0 && !mbar_try_wait(&b_full[s], (b_fills[s] - 1) & 1) &&
                 globaltimer() - t0 < 100000000ull) {}
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------ MMA issuer
      // One thread's scalar work for a tile has to stay below its MMAs' 512
      // cycles: descriptors are a base plus a slot's offset, no divisions, and W's
      // tiles are waited for once (with all of that left out of this, a dx item
      // took 4,400 cycles, twice its MMAs).
      // bf16 A and B, both MN-major
      constexpr uint32_t kIdescMn = idesc_bf16_f32(128, 256) | 1u << 15 | 1u << 16;
      // fp16 A and B (format code 0 in bits [7, 10) and [10, 13)), K-major
      constexpr uint32_t kIdescK = idesc_bf16_f32(128, 256) & ~(1u << 7 | 1u << 10);
      constexpr uint64_t kA = kATile >> 4, kB = kBTile >> 4;  // descriptor units of a slot
      const uint64_t a_mn = sw128_mnmajor_desc(smem_u32(sa));
      const uint64_t b_mn = sw128_mnmajor_desc(smem_u32(sb));
      const uint64_t a_k = sw128_kmajor_desc(smem_u32(sa)), b_k = sw128_kmajor_desc(smem_u32(sb));
      Ring a, b;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return mbar_try_wait(bar, phase) || mbar_wait_bounded(bar, phase, abort_flag);
      };
      int it = 0;  // accumulators filled so far
      for (int w = blockIdx.x; w < args.dw_items && ok; w += gridDim.x) {
        const int range = w / args.ne / args.nd;
        const int kb1 = min(args.kblocks, (range + 1) * args.kper);
        for (int c0 = range * args.kper; c0 < kb1 && ok; c0 += kChunk, ++it) {
          const int ab = it & 1;
          if (!(ok = wait(&tempty[ab], ((it >> 1) & 1) ^ 1u))) break;
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(ab * 256);
          uint32_t acc = 0;
          for (int kb = c0; kb < min(kb1, c0 + kChunk) && ok; ++kb) {
            if (!(ok = wait(&b_full[b.slot], b.phase))) break;
            const uint64_t db = b_mn + b.slot * kB;
            for (int p = 0; p < args.sets; ++p) {
              if (!(ok = wait(&a_full[a.slot], a.phase))) break;
              const uint64_t da = a_mn + a.slot * kA;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {  // 16 K rows of 128 bytes each
                umma_bf16_ss(d, da + kk * (2048 >> 4), db + kk * (2048 >> 4), kIdescMn, acc);
                acc = 1;
              }
              umma_commit(&a_empty[a.slot]);
              a.next(kRA);
            }
            umma_commit(&b_empty[b.slot]);
            b.next(rb);
          }
          if (ok) umma_commit(&tfull[ab]);
        }
      }
      // W's tiles stay until the last item of a block of columns (or, with too
      // many experts for the ring, are new for each item).
      const bool keep = 2 * args.kx <= rb;
      Ring b0;
      int mt = dx0 < dx1 ? dx0 % args.mt : 0;
      for (int w = dx0; w < dx1 && ok; ++w, ++it) {
        const int ab = it & 1;
        if (!(ok = wait(&tempty[ab], ((it >> 1) & 1) ^ 1u))) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(ab * 256);
        const bool new_b = !keep || w == dx0 || mt == 0;
        if (++mt == args.mt) mt = 0;
        const bool free_b = !keep || w + 1 == dx1 || mt == 0;
        if (new_b) b0 = b;
        b = b0;
        auto products = [&](uint64_t da, uint64_t db, bool first) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 K columns of 2 bytes each
            umma_bf16_ss(d, da + kk * (32 >> 4), db + kk * (32 >> 4), kIdescK,
                         first && kk == 0 ? 0u : 1u);
        };
        for (int kb = 0; kb < args.kx; ++kb) {
          if (new_b && !(ok = wait(&b_full[b.slot], b.phase))) break;
          if (!(ok = wait(&a_full[a.slot], a.phase))) break;
          const int hi = b.slot;
          const uint64_t w_hi = b_k + hi * kB;
          products(a_k + a.slot * kA, w_hi, kb == 0);
          umma_commit(&a_empty[a.slot]);
          a.next(kRA);
          b.next(rb);
          if (new_b && !(ok = wait(&b_full[b.slot], b.phase))) break;
          if (!(ok = wait(&a_full[a.slot], a.phase))) break;
          const uint64_t dl_hi = a_k + a.slot * kA;
          products(dl_hi, b_k + b.slot * kB, false);
          if (free_b) umma_commit(&b_empty[b.slot]);
          products(dl_hi, w_hi, false);
          umma_commit(&a_empty[a.slot]);
          a.next(kRA);
          if (free_b) umma_commit(&b_empty[hi]);
          b.next(rb);
        }
        if (ok) umma_commit(&tfull[ab]);
      }
      if (*abort_flag) {
        umma_commit(drain);
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < 100000000ull) {}
      }
    }
  } else {
    // ------------------------------------------------ epilogue (warps 2..9)
    // Two warps for each quarter of the rows, 128 columns each.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t t_base = tmem_base + (uint32_t)(half * 128) + ((uint32_t)(q * 32) << 16);
    int it = 0;
    bool ok = true;
    auto full = [&]() {
      const bool got = mbar_wait_bounded(&tfull[it & 1], (it >> 1) & 1, abort_flag);
      tc_fence_after();
      return __all_sync(0xffffffffu, got) != 0;
    };
    auto release = [&]() {
      tc_fence_before();
      mbar_arrive(&tempty[it & 1]);
      ++it;
    };
    for (int w = blockIdx.x; w < args.dw_items && ok; w += gridDim.x) {
      const int et = w % args.ne, r = w / args.ne, dt = r % args.nd, range = r / args.nd;
      const int kb1 = min(args.kblocks, (range + 1) * args.kper);
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.f;
      for (int c0 = range * args.kper; c0 < kb1; c0 += kChunk) {
        if (!(ok = full())) break;
        const uint32_t t_addr = t_base + (uint32_t)((it & 1) * 256);
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(t_addr + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
        }
        release();
      }
      // the accumulator row's expert and part: planes side by side are 32 (hi, mid,
      // lo, zeros) or 64 rows (hi + lo, mid) apart
      const int part = args.sets == 3 ? 0 : args.sets == 2 ? q >> 1 : q;
      const int e = lane + (args.sets == 3 ? et * 128 + q * 32 : args.sets == 2 ? (q & 1) * 32 : 0);
      const int col = dt * 256 + half * 128;
      float* out = args.dw + ((size_t)(range * args.parts + part) * args.d + col) * args.E + e;
      if (ok && e < args.E && part < args.parts) {
        // d is a multiple of 64: 64 columns or none
#pragma unroll
        for (int c = 0; c < 128; c += 64)
          if (col + c < args.d) {
#pragma unroll
            for (int i = 0; i < 64; ++i) out[(size_t)(c + i) * args.E] = sum[c + i];
          }
      }
    }
    int nt = dx0 / args.mt, mt = dx0 - nt * args.mt;
    // The factors stay in registers: the columns' as long as the items go down one
    // block of them, the row's loaded an item ahead.
    auto row_back = [&](int m) {
      const int r = m * 128 + q * 32 + lane;
      return r < args.T ? args.dl_back[r] : __nv_bfloat16(0.f);
    };
    __nv_bfloat16 next_back = row_back(mt);
    uint4 f[16];
    for (int w = dx0; w < dx1 && ok; ++w) {
      if (w == dx0 || mt == 0) {
        const int col = nt * 256 + half * 128;
#pragma unroll
        for (int i = 0; i < 16; ++i)  // 64 columns or none
          f[i] = col + 8 * i < args.d
                     ? __ldg(reinterpret_cast<const uint4*>(args.w_back + col) + i)
                     : make_uint4(0, 0, 0, 0);
      }
      const int row = mt * 128 + q * 32;
      const __nv_bfloat162 back2 = __bfloat162bfloat162(next_back);
      next_back = row_back(mt + 1 == args.mt ? 0 : mt + 1);
      if (!(ok = full())) break;
      const uint32_t t_addr = t_base + (uint32_t)((it & 1) * 256);
      // The factors are powers of two, so they can follow the rounding to bf16, on pairs.
      // The row's and the column's may lie far on either side of 1 while their product
      // does not: their roots' product (2^-126 to 2^114) is multiplied with twice, so that
      // what lies between is between the sum and the result, and passes no range before
      // the result does.
      // A step of 32 columns loads the next one's sums before it packs its own.
      uint32_t v[2][32];
      tmem_ld_32x32b_x32(t_addr, v[0]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int col = nt * 256 + half * 128 + 32 * n;
        tmem_ld_wait();
        if (n < 3) tmem_ld_32x32b_x32(t_addr + 32 * (n + 1), v[(n + 1) & 1]);
        else release();
        // two staging buffers of 32 rows x 64 bytes: the copy before the last has read its one
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        uint8_t* stage = so + (warp - 2) * kStageOut + (n & 1) * (kStageOut / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 fi = f[4 * n + i];
          const uint32_t g[4] = {fi.x, fi.y, fi.z, fi.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t* u = v[n & 1] + 8 * i + 2 * j;
            __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(u[0]), __uint_as_float(u[1]));
            const __nv_bfloat162 m =
                __hmul2(back2, *reinterpret_cast<const __nv_bfloat162*>(&g[j]));
            y = __hmul2(__hmul2(y, m), m);
            o[j] = *reinterpret_cast<const uint32_t*>(&y);
          }
          // 64-byte swizzle: the 16-byte column of a row XOR bits 1 and 2 of the row
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (col < args.d && row < args.T) tma_store_2d(&tm_dx, stage, col, row);
          // a group for every step, stored or not: the waits above count steps
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
      if (++mt == args.mt) mt = 0, ++nt;
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) record_error(args.err, MOE_ERR_TIMEOUT, 43);
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// dw = the partials added in a fixed order (blocks [0, dw_blocks)): a block has 1024 / G
// values, which G groups of its threads sum over every G-th partial each.  db = the
// column sums of the dL blocks added in fp64 (8 experts a block, 32 threads each).
template <int G>
__global__ void __launch_bounds__(256) k_router_sum(const float* __restrict__ part, int partials,
                                                    long long n, float* __restrict__ dw,
                                                    int dw_blocks, const float* __restrict__ sums,
                                                    int sum_rows, int E, float* __restrict__ db) {
  __shared__ double red[32][8];
  __shared__ float4 meet[G > 1 ? 256 : 1];
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= dw_blocks) {
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int e = ((int)blockIdx.x - dw_blocks) * 8 + c;
    double s = 0.0;
    if (e < E) {
      for (int r = g; r < sum_rows; r += 256) {
        float v[8];  // eight loads in flight
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = r + 32 * i < sum_rows ? __ldg(sums + (size_t)(r + 32 * i) * E + e) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i];
      }
    }
    red[g][c] = s;
    __syncthreads();
    if (g == 0 && e < E) {
      s = 0.0;
#pragma unroll
      for (int i = 0; i < 32; ++i) s += red[i][c];
      db[e] = (float)s;
    }
    return;
  }
  // n is a multiple of 64 (d is); dw itself may be aligned to 4 bytes only
  constexpr int kSpan = 256 / G;
  const int c = threadIdx.x % kSpan, g = threadIdx.x / kSpan;
  const long long i = (long long)blockIdx.x * kSpan + c, n4 = n / 4;
  const float4* p4 = reinterpret_cast<const float4*>(part) + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < n4) {
#pragma unroll 8
    for (int p = g; p < partials; p += G) {
      const float4 v = __ldcs(p4 + p * n4);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  if (G > 1) {
    meet[threadIdx.x] = s;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 1; k < G; ++k) {
      const float4 v = meet[k * kSpan + c];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  if (i >= n4) return;
  if ((reinterpret_cast<uintptr_t>(dw) & 15) == 0) {
    reinterpret_cast<float4*>(dw)[i] = s;
  } else {
    dw[4 * i] = s.x, dw[4 * i + 1] = s.y, dw[4 * i + 2] = s.z, dw[4 * i + 3] = s.w;
  }
}

// ============================================================== few tokens
// Up to 192 tokens the products are small (64 x 2048 x 128: 134 MFLOP) and the time is
// launches, loads and stores, so all of it is one kernel and warp-wide MMAs on
// fragments made in registers: the tcgen05 tiles want their operands laid out by a
// kernel before.  A block takes 16 columns of d, with dL [T][E], its W [16][E] and its
// x [T][16] in shared memory.
//   dW: 16 columns x 8 experts a tile, K = tokens, x in bf16, dL in three bf16 planes
//       with a sum each, added last;
//   dx: 16 tokens x 8 columns a tile, K = experts, both in two tf32 parts (split2: 2^-21
//       of each value is lost), hi lo and lo hi with a sum of their own, added last.
// Rows lie ep = 4 (mod 32) words apart: the 8 x 4 lanes of a fragment hit 32 banks.
// 64 x 2048 x 128: 6.6 us, 3.7 with 16 tokens.  What bounds it is one latency after the
// other: the loads and the barrier behind them, new code's fetch, the MMAs, the stores
// (issue slots 36% used, L2 7%); 8 warps a block in place of 16 took 3 us more.
struct RouterSmallArgs {
  const __nv_bfloat16* x;
  const float* w;
  const float* dl;
  float* dw;
  float* db;
  __nv_bfloat16* dx;
  int T, d, E, ep, vec_dl, vec_w;
};
constexpr int kSmallT = 192, kSmallWarps = 16;
constexpr int kSmallXPitch = 24;  // bf16 of one token of x in shared memory

// rows x cols of src into rows of ep words, zeros up to rows_all x cols_all.
__device__ __forceinline__ void copy_rows(float* dst, const float* __restrict__ src, int rows,
                                          int cols, int rows_all, int cols_all, int ep, int vec) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < rows_all; r += kSmallWarps) {
    float* to = dst + r * ep;
    const float* from = src + (size_t)r * cols;
    const int n = r < rows ? cols : 0;
    if (vec) {
      for (int c = 4 * lane; c < n; c += 128)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + c)),
                     "l"(from + c)
                     : "memory");
    } else {
      for (int c = lane; c < n; c += 32)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + c)),
                     "l"(from + c)
                     : "memory");
    }
    for (int c = n + lane; c < cols_all; c += 32) to[c] = 0.f;
  }
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// v = hi + lo in tf32 (11 bits each): hi has the upper bits of the mantissa as they stand,
// so it cannot overflow, the rest is exact and is rounded.  A product of two such values
// leaves lo lo out (2^-20 of it at most); below 2^-114 lo nears tf32's lowest step, 2^-136.
// inf and NaN leave NaN in the rest.
struct Split2 {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split2 split2(float v) {
  Split2 s;
  s.hi = __float_as_uint(v) & 0xffffe000u;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(s.lo) : "f"(v - __uint_as_float(s.hi)));
  return s;
}
__device__ __forceinline__ uint32_t pair_of(__nv_bfloat16 lo, __nv_bfloat16 hi) {
  const __nv_bfloat162 v = __halves2bfloat162(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// KS: 16 tokens each, so that the steps of a tile are unrolled without a branch
// (64 x 2048 x 128: 6.8 us with them, 7.6 with one that leaves the loop early).
template <int KS>
__global__ void __launch_bounds__(32 * kSmallWarps, KS <= 4 ? 2 : 1)
    k_router_bwd_small(const RouterSmallArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int T16 = 16 * KS;
  const int E8 = (a.E + 7) / 8 * 8;
  float* sdl = sm;                       // [T16][ep]
  float* sw = sdl + (size_t)T16 * a.ep;  // [16][ep]
  float* meet = sw + 16 * a.ep;          // [warp][16][16]
  __nv_bfloat16* sx =                    // [T16][kSmallXPitch]
      reinterpret_cast<__nv_bfloat16*>(meet + 256 * kSmallWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;  // a fragment's row or column, and place in it
  pdl_trigger();
  pdl_wait();
  const int i0 = blockIdx.x * 16;
  copy_rows(sdl, a.dl, a.T, a.E, T16, E8, a.ep, a.vec_dl);
  if (a.dx) copy_rows(sw, a.w + (size_t)i0 * a.E, 16, a.E, 16, E8, a.ep, a.vec_w);
  if (a.dw)
    for (int q = threadIdx.x; q < 2 * T16; q += 32 * kSmallWarps) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (q < 2 * a.T)
        v = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)(q >> 1) * a.d + i0) + (q & 1));
      *reinterpret_cast<uint4*>(sx + (q >> 1) * kSmallXPitch + (q & 1) * 8) = v;
    }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  if (a.dw) {
    uint32_t xa[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const __nv_bfloat16* p = sx + (16 * ks + 2 * t4) * kSmallXPitch + g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows g, g + 8; tokens 2 t4, + 8
        const __nv_bfloat16* q = p + (i >> 1) * 8 * kSmallXPitch + (i & 1) * 8;
        xa[ks][i] = pair_of(q[0], q[kSmallXPitch]);
      }
    }
    const bool even = a.E % 2 == 0 && (reinterpret_cast<uintptr_t>(a.dw) & 7) == 0;
    for (int nt = warp; nt < E8 / 8; nt += kSmallWarps) {
      float c[4] = {}, cm[4] = {}, cl[4] = {};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const float* p = sdl + (16 * ks + 2 * t4) * a.ep + 8 * nt + g;
        const Split3 u = split3(p[0], p[a.ep]), v = split3(p[8 * a.ep], p[9 * a.ep]);
        mma_bf16(cl, xa[ks], u.lo, v.lo);
        mma_bf16(cm, xa[ks], u.mid, v.mid);
        mma_bf16(c, xa[ks], u.hi, v.hi);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] += cm[i] + cl[i];
      const int e = 8 * nt + 2 * t4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* out = a.dw + (size_t)(i0 + g + 8 * h) * a.E + e;
        if (even && e < a.E) {
          *reinterpret_cast<float2*>(out) = make_float2(c[2 * h], c[2 * h + 1]);
        } else {
          if (e < a.E) out[0] = c[2 * h];
          if (e + 1 < a.E) out[1] = c[2 * h + 1];
        }
      }
    }
  }
  if (a.dx) {
    // a warp takes 16 tokens, and with fewer than 8 such tiles a part of the experts
    constexpr int tiles = KS, parts = kSmallWarps / tiles;
    const int mt = warp % tiles, part = warp / tiles;
    float c[2][4] = {}, cs[2][4] = {};
    if (part < parts) {
      const int n8 = E8 / 8;
      const float* pa = sdl + (16 * mt + g) * a.ep + t4;
      const float* pb = sw + g * a.ep + t4;
#pragma unroll 4
      for (int k = part; k < n8; k += parts) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Split2 v = split2(pa[(i & 1) * 8 * a.ep + 8 * k + (i >> 1) * 4]);
          hi[i] = v.hi, lo[i] = v.lo;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float* q = pb + 8 * n * a.ep + 8 * k;
          const Split2 u = split2(q[0]), v = split2(q[4]);
          mma_tf32(cs[n], lo, u.hi, v.hi);
          mma_tf32(c[n], hi, u.hi, v.hi);
          mma_tf32(cs[n], hi, u.lo, v.lo);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        meet[warp * 256 + (g + (i >> 1) * 8) * 16 + 8 * n + 2 * t4 + (i & 1)] = c[n][i] + cs[n][i];
    __syncthreads();
    for (int q = threadIdx.x; q < 8 * a.T; q += 32 * kSmallWarps) {  // a pair of columns each
      const int t = q >> 3, i = 2 * (q & 7);
      float s0 = 0.f, s1 = 0.f;
      for (int p = 0; p < parts; ++p) {
        const float2 v = *reinterpret_cast<const float2*>(
            meet + (p * tiles + t / 16) * 256 + (t % 16) * 16 + i);
        s0 += v.x, s1 += v.y;
      }
      *reinterpret_cast<uint32_t*>(a.dx + (size_t)t * a.d + i0 + i) = pack_bf16x2(s0, s1);
    }
  }
  if (a.db)  // each block some experts; up to 192 values, 2^-24 an add
    for (int e = blockIdx.x * blockDim.x + threadIdx.x; e < a.E; e += gridDim.x * blockDim.x) {
      float s = 0.f;
#pragma unroll 8
      for (int r = 0; r < a.T; ++r) s += sdl[r * a.ep + e];
      a.db[e] = s;
    }
}

constexpr int kSmallSmem = 220 * 1024, kSmallSmem2 = 113 * 1024;  // one, two blocks an SM

// The KS that takes T tokens.
int router_small_steps(int T) {
  const int ks = (T + 15) / 16;
  return ks <= 4 ? ks : ks <= 6 ? 6 : ks <= 8 ? 8 : 12;
}
int router_small_ep(int E) { return ((E + 7) / 8 * 8 + 27) / 32 * 32 + 4; }
size_t router_small_smem(const moe_shape& s) {
  const size_t T16 = 16 * router_small_steps(s.T);
  return sizeof(float) * ((T16 + 16) * router_small_ep(s.E) + 256 * kSmallWarps) +
         2 * T16 * kSmallXPitch;
}
// Where the blocks of 16 columns fit the GPU at once (two an SM up to 64 tokens): E = 8
// to 256, d = 512 to 4096, 16 to 64 tokens took 2.7 to 11.9 us where the three kernels
// took 7.6 to 18.8, d = 512 and 2048, 96 to 192 tokens 4.9 to 11.5 in place of 10.3 to
// 14.0, less in each.  In a second wave each block loads dL again: up to 32 tokens still
// won (d = 7168: 5.2 to 12.0 against 8.2 to 18.3), 64 did at no E but 8 (16.0 against
// 14.2 with 256 experts, when dx took one product a term in both).
bool router_small(const moe_shape& s, int sms) {
  if (s.T > kSmallT || router_small_smem(s) > kSmallSmem) return false;
  const int resident = s.T <= 64 && router_small_smem(s) <= kSmallSmem2 ? 2 * sms : sms;
  return s.d / 16 <= (s.T <= 32 ? 2 * resident : resident);
}

// cuTensorMapEncodeTiled, looked up once; nullptr if the driver has none.
decltype(&cuTensorMapEncodeTiled) tensor_map_encoder() {
  static const auto fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found =
        cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(found ? p : nullptr);
  }();
  return fn;
}

// 16-bit tensor map of up to 4 dimensions, innermost first; strides in bytes of
// dimensions 1 and up.
bool make_map(CUtensorMap* tm, const void* base, int rank, const uint64_t* dims,
              const uint64_t* strides, const uint32_t* box,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = strides[i];
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Raises a kernel's dynamic shared memory limit once for each device (the attribute
// belongs to the device's copy of the kernel); `ready` has a bit for each.
typedef std::atomic<uint64_t> DeviceBits[2];
DeviceBits gemm_ready, small_ready[7];
template <class K>
cudaError_t allow_smem(K kern, int bytes, DeviceBits& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev < 128;
  if (known && (ready[dev / 64].load(std::memory_order_acquire) >> (dev % 64) & 1)) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known)
    ready[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_release);
  return e;
}

}  // namespace

cudaError_t launch_router_bwd(const __nv_bfloat16* x, const float* w_g, const float* dl,
                              const moe_shape& s, float* dw, float* db, __nv_bfloat16* dx,
                              const BwdLayout& L, char* ws, int sms, cudaStream_t st) {
  const int T = s.T, d = s.d, E = s.E, cp = L.cp;
  const auto vec = [&](const float* p) {
    return (int)(E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0);
  };
  const bool products = dw || dx;
  if (products && router_small(s, sms)) {
    const RouterSmallArgs a{x, w_g, dl, dw, db, dx, T, d, E, router_small_ep(E), vec(dl), vec(w_g)};
    const auto go = [&](auto kern, DeviceBits& ready) {
      const cudaError_t e = allow_smem(kern, kSmallSmem, ready);
      if (e != cudaSuccess) return e;
      return launch_kernel(kern, dim3(d / 16), dim3(32 * kSmallWarps), router_small_smem(s), st, 1,
                           a);
    };
    switch (router_small_steps(T)) {
      case 1: return go(k_router_bwd_small<1>, small_ready[0]);
      case 2: return go(k_router_bwd_small<2>, small_ready[1]);
      case 3: return go(k_router_bwd_small<3>, small_ready[2]);
      case 4: return go(k_router_bwd_small<4>, small_ready[3]);
      case 6: return go(k_router_bwd_small<6>, small_ready[4]);
      case 8: return go(k_router_bwd_small<8>, small_ready[5]);
      default: return go(k_router_bwd_small<12>, small_ready[6]);
    }
  }
  __nv_bfloat16* dlp = reinterpret_cast<__nv_bfloat16*>(ws + L.dl_planes);
  __half* dlh = reinterpret_cast<__half*>(ws + L.dl_half);
  __half* wh = reinterpret_cast<__half*>(ws + L.w_half);
  __nv_bfloat16* dl_back = reinterpret_cast<__nv_bfloat16*>(ws + L.dl_back);
  __nv_bfloat16* w_back = reinterpret_cast<__nv_bfloat16*>(ws + L.w_back);
  float* sums = reinterpret_cast<float*>(ws + L.db_part);
  float* part = reinterpret_cast<float*>(ws + L.dw_part);
  const RouterPlanes pl = router_planes(E, T);
  const bool apart = pl.sets == 3;  // each plane for itself, or side by side in a row of four
  const long long prow = apart ? pl.width : 4 * pl.width;
  const int sum_rows = (T + L.plane_rows - 1) / L.plane_rows;
  // one block's column sums are db itself
  const PlanesArgs pd{dl, dw ? dlp : nullptr, dx ? dlh : nullptr, dl_back,
                      !db ? nullptr : sum_rows == 1 ? db : sums, T, prow,
                      apart ? (long long)T * pl.width : pl.width, E, cp, pl.width, !apart,
                      L.plane_rows, sum_rows, vec(dl)};
  const PlanesArgs pw{w_g, nullptr, wh, w_back, nullptr, d, 0, 0, E, cp, 0, 0, 32,
                      dx ? (d + 31) / 32 : 0, vec(w_g)};
  const auto planes = [&](auto kern, int lanes) {
    return launch_kernel(kern, dim3(pd.blocks + pw.blocks), dim3(256),
                         sizeof(float) * (256 / lanes) * cp, st, 1, pd, pw);
  };
  cudaError_t e = cp <= 64    ? planes(k_router_planes<8, 1>, 8)
                  : cp <= 128 ? planes(k_router_planes<16, 1>, 16)
                  : cp <= 256 ? planes(k_router_planes<32, 1>, 32)
                  : cp <= 512 ? planes(k_router_planes<32, 2>, 32)
                              : planes(k_router_planes<32, 4>, 32);
  if (e != cudaSuccess) return e;

  const int kblocks = (T + 63) / 64, kper = router_range_blocks(s, dx != nullptr);
  const int ranges = (kblocks + kper - 1) / kper;
  const bool direct = ranges * pl.parts == 1;
  if (products) {
    RouterGemmArgs a{};
    a.T = T, a.d = d, a.E = E;
    a.sets = pl.sets, a.parts = pl.parts;
    a.rb = cp <= (dx ? 64 : 128) ? 3 : kRB;
    a.ne = apart ? (E + 127) / 128 : 1, a.nd = (d + 255) / 256;
    a.kblocks = kblocks, a.kper = kper;
    a.dw_items = dw ? a.ne * a.nd * ranges : 0;
    a.mt = (T + 127) / 128, a.kx = cp / 64;
    a.dl_back = dl_back, a.w_back = w_back;
    a.dx_items = dx ? a.mt * a.nd : 0;
    const int grid = std::min(a.dw_items + a.dx_items, sms);
    // Shares of dx: `heavy` blocks have one dW item more than the others, worth
    // `more` dx items; a level n of dx items for the heavy ones gives the others
    // n + more.
    const int heavy = a.dw_items % grid, light = grid - heavy;
    const double item_us = std::min(kper, kblocks) * router_dw_block_us(pl.sets) + kRouterItemUs;
    const double more = item_us / router_dx_tile_us(E);
    const double level = std::max(0.0, (a.dx_items - light * more) / grid);
    a.light_dx = heavy == 0 ? a.dx_items
                            : (int)std::min<double>(a.dx_items, light * (level + more) + 0.5);
    a.dw = direct ? dw : part, a.err = reinterpret_cast<int*>(ws);
    const uint64_t row = (uint64_t)cp * 4;
    CUtensorMap mx{}, mn{}, mk{}, mw{}, mdx{};
    const uint64_t xd[3] = {64, (uint64_t)T, (uint64_t)d / 64}, xs[2] = {(uint64_t)d * 2, 128};
    const uint64_t nd[4] = {64, (uint64_t)T, (uint64_t)prow / 64, apart ? 3u : 1u};
    const uint64_t ns[3] = {(uint64_t)prow * 2, 128, (uint64_t)prow * 2 * T};
    const uint64_t kd[2] = {2 * (uint64_t)cp, (uint64_t)T}, wd[2] = {2 * (uint64_t)cp, (uint64_t)d};
    const uint64_t od[2] = {(uint64_t)d, (uint64_t)T}, os[1] = {(uint64_t)d * 2};
    const uint32_t xb[3] = {64, 64, 4}, nb[4] = {64, 64, 2, 1}, kb[2] = {64, 128},
                   wb[2] = {64, 256}, ob[2] = {32, 32};
    // only the maps that the items use (another's bytes are never read)
    if (dw && (!make_map(&mx, x, 3, xd, xs, xb) || !make_map(&mn, dlp, 4, nd, ns, nb)))
      return cudaErrorInvalidValue;
    if (dx && (!make_map(&mk, dlh, 2, kd, &row, kb) || !make_map(&mw, wh, 2, wd, &row, wb) ||
               !make_map(&mdx, dx, 2, od, os, ob, CU_TENSOR_MAP_SWIZZLE_64B)))
      return cudaErrorInvalidValue;
    if ((e = allow_smem(k_router_gemm, router_smem(kRB), gemm_ready)) != cudaSuccess) return e;
    e = launch_kernel(k_router_gemm, dim3(grid), dim3(kRouterThreads), router_smem(a.rb), st, 1,
                      mx, mn, mk, mw, mdx, a);
    if (e != cudaSuccess) return e;
  }
  const long long n = (long long)d * E;
  const int partials = ranges * pl.parts, groups = partials >= 16 ? 8 : 1;
  const int span = 1024 / groups;  // values of one block
  const int dw_blocks = dw && !direct ? (int)((n + span - 1) / span) : 0;
  const int db_blocks = db && sum_rows > 1 ? (E + 7) / 8 : 0;
  if (dw_blocks + db_blocks == 0) return e;
  const auto sum = [&](auto kern) {
    return launch_kernel(kern, dim3(dw_blocks + db_blocks), dim3(256), 0, st, 1, part, partials, n,
                         dw, dw_blocks, sums, sum_rows, E, db);
  };
  return groups == 8 ? sum(k_router_sum<8>) : sum(k_router_sum<1>);
}

}  // namespace moe
