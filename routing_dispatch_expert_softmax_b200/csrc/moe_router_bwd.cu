// Backward of the router product L = x W_g + b:
//   dW[i,e] = sum_t x[t,i] dL[t,e],  db[e] = sum_t dL[t,e],
//   dx[t,i] = sum_e dL[t,e] W[i,e]
// on the sm_100a tensor cores.  dL and W are fp32; the tensor cores take
// bf16.  A first kernel splits them into bf16 planes, hi = bf16(v),
// mid = bf16(v - hi), lo = bf16(v - hi - mid), so hi + mid + lo = v to more
// than 24 bits:
//   dW = x (hi + mid + lo): x is bf16, so the three products are exact and the
//        result is an fp32 product's;
//   dx = dL_hi W_hi + dL_mid W_hi + dL_hi W_mid, what is left out is below
//        3 * 2^-18 of each product (dx itself is rounded to 2^-8).
// One persistent kernel then runs the tiles of both products.  The tokens are
// the long axis of dW, so its tiles split over token ranges; a last kernel
// adds the ranges' partial tiles in order.
#include "moe_kernels.cuh"

namespace moe {

namespace {

// ============================================================== planes
struct Split3 {
  __nv_bfloat16 hi, mid, lo;
};

// inf and NaN go to hi alone, so that a product shows them as an fp32 one would.
__device__ __forceinline__ Split3 split3(float v) {
  Split3 s;
  s.hi = __float2bfloat16_rn(v);
  if (__hisinf(s.hi)) s.hi = __float2bfloat16_rz(v);  // the largest fp32 values round to inf
  float r = v - __bfloat162float(s.hi);
  if (!(fabsf(v) <= 3.402823466e38f)) r = 0.f;
  s.mid = __float2bfloat16_rn(r);
  s.lo = __float2bfloat16_rn(r - __bfloat162float(s.mid));
  return s;
}

// planes[p][row][0 .. cp) of the [rows, cols] fp32 matrix a, cp = cols rounded
// up to 64 with zeros.  Each thread takes 8 columns of every (256 / (cp / 8))-th
// row of the block's; with sums != nullptr the block also stores its rows'
// column sums as sums[block][cols].
struct PlanesArgs {
  const float* a;
  __nv_bfloat16* planes;  // nullptr: only the sums
  float* sums;
  long long rows;
  int cols, cp, nplanes, rows_per_block, blocks, vec;
};

__device__ void planes_block(const PlanesArgs& p, int block, float* red) {
  const int oct = p.cp / 8, par = 256 / oct;
  const int o = threadIdx.x % oct, r0 = threadIdx.x / oct;
  const long long first = (long long)block * p.rows_per_block;
  const long long last = min(p.rows, first + p.rows_per_block);
  const int c0 = 8 * o;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  if (r0 < par) {
    for (long long r = first + r0; r < last; r += par) {
      const float* src = p.a + r * p.cols + c0;
      float v[8];
      if (p.vec && c0 + 8 <= p.cols) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(src));
        const float4 y = __ldg(reinterpret_cast<const float4*>(src) + 1);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i < p.cols ? __ldg(src + i) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
      if (p.planes) {
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Split3 a = split3(v[2 * i]), b = split3(v[2 * i + 1]);
          const __nv_bfloat162 h = __halves2bfloat162(a.hi, b.hi);
          const __nv_bfloat162 m = __halves2bfloat162(a.mid, b.mid);
          const __nv_bfloat162 l = __halves2bfloat162(a.lo, b.lo);
          w[0][i] = *reinterpret_cast<const uint32_t*>(&h);
          w[1][i] = *reinterpret_cast<const uint32_t*>(&m);
          w[2][i] = *reinterpret_cast<const uint32_t*>(&l);
        }
        for (int q = 0; q < p.nplanes; ++q)
          *reinterpret_cast<uint4*>(p.planes + ((size_t)q * p.rows + r) * p.cp + c0) =
              q == 0   ? make_uint4(w[0][0], w[0][1], w[0][2], w[0][3])
              : q == 1 ? make_uint4(w[1][0], w[1][1], w[1][2], w[1][3])
                       : make_uint4(w[2][0], w[2][1], w[2][2], w[2][3]);
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 < par) red[(size_t)r0 * p.cp + c0 + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    float s = 0.f;
    for (int r = 0; r < par; ++r) s += red[(size_t)r * p.cp + c];
    p.sums[(size_t)block * p.cols + c] = s;
  }
}

// Blocks [0, a.blocks) split dL, the others W.
__global__ void __launch_bounds__(256) k_router_planes(const PlanesArgs dl, const PlanesArgs w) {
  __shared__ float red[256 * 8];
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < dl.blocks) planes_block(dl, blockIdx.x, red);
  else planes_block(w, blockIdx.x - dl.blocks, red);
}

// ============================================================== products
// One work item is a 128 x 256 tile of fp32 sums in TMEM:
//   dW: rows = 128 experts, columns = 256 of d, K = the tokens of one range;
//       A = dL planes and B = x, both with the non-K index contiguous
//       (MN-major): tiles of 64 tokens x 64 columns, 128 bytes a row;
//   dx: rows = 128 tokens, columns = 256 of d, K = experts; A = dL planes and
//       B = W planes, both K-major.
// dW takes the experts as rows so that a row of 256 columns of x serves the
// three planes, and a lane's accumulator row is one expert: the 32 lanes of a
// warp then store 32 neighbouring experts of dW[i, :].
// Shared memory: a ring of 16 KB A tiles and one of 32 KB B tiles (128-byte
// swizzle).  For each 64 of K, dW takes 3 A and 1 B tiles, dx 2 and 2.
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
  int kblocks, kper;     // 64-token blocks in all, and of one range
  int xt;                // column tiles of dx
  int kx;                // 64-expert blocks of dx
  int light_dx;          // dx items of the blocks that have one dW item less
  float* dw;             // [ranges][d][E]
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
constexpr int kRA = 6, kRB = 3;
constexpr int kATile = 128 * 64 * 2, kBTile = 256 * 64 * 2;
constexpr int kStageOut = 32 * 128;  // per epilogue warp: 32 rows x 64 bf16 of dx
constexpr int kRouterSmem = kRA * kATile + kRB * kBTile + 8 * kStageOut + 1024 + 256;
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
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(tm)),
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
  uint8_t* so = sb + kRB * kBTile;
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
          b.next(kRB);
          for (int p = 2; p >= 0; --p) {
            dst = take_a();
            if (!(ok = dst != nullptr)) break;
            tma_load_4d(dst, &tm_dl_mn, &a_full[a.slot], 0, kb * 64, et * 2, p);
            a.next(kRA);
          }
        }
      }
      for (int w = dx0; w < dx1 && ok; ++w) {
        const int nt = w % args.xt, mt = w / args.xt;
        for (int kb = 0; kb < args.kx && ok; ++kb)
          for (int p = 0; p < 2; ++p) {
            uint8_t* dst = take_a();
            if (!(ok = dst != nullptr)) break;
            tma_load_3d(dst, &tm_dl_k, &a_full[a.slot], kb * 64, mt * 128, p);
            a.next(kRA);
            dst = take_b();
            if (!(ok = dst != nullptr)) break;
            tma_load_3d(dst, &tm_w, &b_full[b.slot], kb * 64, nt * 256, p);
            b.next(kRB);
          }
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
      constexpr uint32_t kIdescK = idesc_bf16_f32(128, 256);
      constexpr uint32_t kIdescMn = kIdescK | 1u << 15 | 1u << 16;  // A and B MN-major
      Ring a, b;
      bool ok = true;
      // four K = 16 steps of one pair of tiles
      auto mma_mn = [&](uint32_t d, int sa_slot, int sb_slot, uint32_t acc) {
        const uint32_t aa = smem_u32(sa + sa_slot * kATile), bb = smem_u32(sb + sb_slot * kBTile);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_ss(d, sw128_mnmajor_desc(aa + kk * 2048), sw128_mnmajor_desc(bb + kk * 2048),
                       kIdescMn, kk ? 1u : acc);
      };
      auto mma_k = [&](uint32_t d, int sa_slot, int sb_slot, uint32_t acc) {
        const uint32_t aa = smem_u32(sa + sa_slot * kATile), bb = smem_u32(sb + sb_slot * kBTile);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_ss(d, sw128_kmajor_desc(aa + kk * 32), sw128_kmajor_desc(bb + kk * 32),
                       kIdescK, kk ? 1u : acc);
      };
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        const bool got = mbar_wait_bounded(bar, phase, abort_flag);
        tc_fence_after();
        return got;
      };
      int it = 0;  // accumulators filled so far
      for (int w = blockIdx.x; w < args.dw_items && ok; w += gridDim.x) {
        const int range = w / args.ne / args.nd;
        const int kb1 = min(args.kblocks, (range + 1) * args.kper);
        for (int c0 = range * args.kper; c0 < kb1 && ok; c0 += kChunk, ++it) {
          const int ab = it & 1;
          if (!(ok = wait(&tempty[ab], ((it >> 1) & 1) ^ 1u))) break;
          const uint32_t d = tmem_base + (uint32_t)(ab * 256);
          for (int kb = c0; kb < min(kb1, c0 + kChunk) && ok; ++kb) {
            if (!(ok = wait(&b_full[b.slot], b.phase))) break;
            for (int p = 0; p < 3; ++p) {
              if (!(ok = wait(&a_full[a.slot], a.phase))) break;
              mma_mn(d, a.slot, b.slot, kb != c0 || p != 0);
              umma_commit(&a_empty[a.slot]);
              a.next(kRA);
            }
            umma_commit(&b_empty[b.slot]);
            b.next(kRB);
          }
          if (ok) umma_commit(&tfull[ab]);
        }
      }
      for (int w = dx0; w < dx1 && ok; ++w, ++it) {
        const int ab = it & 1;
        if (!wait(&tempty[ab], ((it >> 1) & 1) ^ 1u)) break;
        const uint32_t d = tmem_base + (uint32_t)(ab * 256);
        for (int kb = 0; kb < args.kx && ok; ++kb) {
          const Ring ahi = a;
          a.next(kRA);
          const Ring amid = a;
          a.next(kRA);
          const Ring bhi = b;
          b.next(kRB);
          const Ring bmid = b;
          b.next(kRB);
          if (!(ok = wait(&a_full[ahi.slot], ahi.phase) && wait(&b_full[bhi.slot], bhi.phase)))
            break;
          mma_k(d, ahi.slot, bhi.slot, kb != 0);
          if (!(ok = wait(&a_full[amid.slot], amid.phase))) break;
          mma_k(d, amid.slot, bhi.slot, 1);
          umma_commit(&a_empty[amid.slot]);
          umma_commit(&b_empty[bhi.slot]);
          if (!(ok = wait(&b_full[bmid.slot], bmid.phase))) break;
          mma_k(d, ahi.slot, bmid.slot, 1);
          umma_commit(&a_empty[ahi.slot]);
          umma_commit(&b_empty[bmid.slot]);
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
      const int e = et * 128 + q * 32 + lane, col = dt * 256 + half * 128;
      float* out = args.dw + ((size_t)range * args.d + col) * args.E + e;
      if (ok && e < args.E) {
        // d is a multiple of 64: 64 columns or none
#pragma unroll
        for (int c = 0; c < 128; c += 64)
          if (col + c < args.d) {
#pragma unroll
            for (int i = 0; i < 64; ++i) out[(size_t)(c + i) * args.E] = sum[c + i];
          }
      }
    }
    uint8_t* stage = so + (warp - 2) * kStageOut;
    for (int w = dx0; w < dx1 && ok; ++w) {
      const int nt = w % args.xt, mt = w / args.xt;
      if (!(ok = full())) break;
      const uint32_t t_addr = t_base + (uint32_t)((it & 1) * 256);
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        uint32_t v[64];
        tmem_ld_32x32b_x32(t_addr + c, v);
        tmem_ld_32x32b_x32(t_addr + c + 32, v + 32);
        tmem_ld_wait();
        if (c == 64) release();
        // the copy of the tile before has read the staging rows
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * j]),
                               __uint_as_float(v[8 * i + 2 * j + 1]));
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        const int col = nt * 256 + half * 128 + c, row = mt * 128 + q * 32;
        if (lane == 0 && col < args.d && row < args.T) tma_store_2d(&tm_dx, stage, col, row);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) record_error(args.err, MOE_ERR_TIMEOUT, 43);
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// dw = the ranges' tiles added in order (blocks [0, dw_blocks)); db = the
// plane blocks' column sums added in fp64 (32 experts a block).
__global__ void __launch_bounds__(256) k_router_sum(const float* __restrict__ part, int ranges,
                                                    long long n, float* __restrict__ dw,
                                                    int dw_blocks, const float* __restrict__ sums,
                                                    int sum_rows, int E, float* __restrict__ db) {
  __shared__ double red[8][32];
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < dw_blocks) {
    // n is a multiple of 64 (d is); dw itself may be aligned to 4 bytes only
    const bool vec = (reinterpret_cast<uintptr_t>(dw) & 15) == 0;
    const float4* p4 = reinterpret_cast<const float4*>(part);
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n / 4; i += dw_blocks * 256LL) {
      float4 s = __ldcs(p4 + i);
#pragma unroll 8
      for (int p = 1; p < ranges; ++p) {
        const float4 v = __ldcs(p4 + p * (n / 4) + i);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      if (vec) {
        reinterpret_cast<float4*>(dw)[i] = s;
      } else {
        dw[4 * i] = s.x, dw[4 * i + 1] = s.y, dw[4 * i + 2] = s.z, dw[4 * i + 3] = s.w;
      }
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = ((int)blockIdx.x - dw_blocks) * 32 + lane;
  double s = 0.0;
  if (e < E)
    for (int r = warp; r < sum_rows; r += 8) s += sums[(size_t)r * E + e];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && e < E) {
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += red[w][lane];
    db[e] = (float)s;
  }
}

// bf16 tensor map of up to 4 dimensions, innermost first, 128-byte swizzle;
// strides in bytes of dimensions 1 and up.
bool make_map(CUtensorMap* tm, const void* base, int rank, const uint64_t* dims,
              const uint64_t* strides, const uint32_t* box) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = strides[i];
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_router_bwd(const __nv_bfloat16* x, const float* w_g, const float* dl,
                              const moe_shape& s, float* dw, float* db, __nv_bfloat16* dx,
                              const BwdLayout& L, char* ws, int sms, cudaStream_t st) {
  const int T = s.T, d = s.d, E = s.E, cp = L.cp;
  __nv_bfloat16* dlp = reinterpret_cast<__nv_bfloat16*>(ws + L.dl_planes);
  __nv_bfloat16* wp = reinterpret_cast<__nv_bfloat16*>(ws + L.w_planes);
  float* sums = reinterpret_cast<float*>(ws + L.db_part);
  float* part = reinterpret_cast<float*>(ws + L.dw_part);
  const bool products = dw || dx;
  const auto vec = [&](const float* p) {
    return (int)(E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0);
  };
  const PlanesArgs pd{dl, products ? dlp : nullptr, db ? sums : nullptr, T, E, cp, dw ? 3 : 2,
                      L.plane_rows, (T + L.plane_rows - 1) / L.plane_rows, vec(dl)};
  const PlanesArgs pw{w_g, wp, nullptr, d, E, cp, 2, 32, dx ? (d + 31) / 32 : 0, vec(w_g)};
  cudaError_t e = launch_kernel(k_router_planes, dim3(pd.blocks + pw.blocks), dim3(256), 0, st, 1,
                                pd, pw);
  if (e != cudaSuccess) return e;

  const int kblocks = (T + 63) / 64, kper = router_range_blocks(s, dx != nullptr);
  const int ranges = (kblocks + kper - 1) / kper;
  const bool direct = ranges == 1;
  if (products) {
    RouterGemmArgs a{};
    a.T = T, a.d = d, a.E = E;
    a.ne = (E + 127) / 128, a.nd = (d + 255) / 256;
    a.kblocks = kblocks, a.kper = kper;
    a.dw_items = dw ? a.ne * a.nd * ranges : 0;
    a.xt = (d + 255) / 256, a.kx = cp / 64;
    a.dx_items = dx ? (T + 127) / 128 * a.xt : 0;
    const int grid = std::min(a.dw_items + a.dx_items, sms);
    // Shares of dx: `heavy` blocks have one dW item more than the others, worth
    // kper / kx dx items; a level n of dx items for the heavy ones gives the
    // others n + kper / kx.
    const int heavy = a.dw_items % grid, light = grid - heavy;
    const double more = (double)a.kper / a.kx;
    const double level = std::max(0.0, (a.dx_items - light * more) / grid);
    a.light_dx = heavy == 0 ? a.dx_items
                            : (int)std::min<double>(a.dx_items, light * (level + more) + 0.5);
    a.dw = direct ? dw : part, a.err = reinterpret_cast<int*>(ws);
    const uint64_t row = (uint64_t)cp * 2;
    CUtensorMap mx, mn, mk, mw, mdx;
    const uint64_t xd[3] = {64, (uint64_t)T, (uint64_t)d / 64}, xs[2] = {(uint64_t)d * 2, 128};
    const uint64_t nd[4] = {64, (uint64_t)T, (uint64_t)cp / 64, 3}, ns[3] = {row, 128, row * T};
    const uint64_t kd[3] = {(uint64_t)cp, (uint64_t)T, 3}, ks[2] = {row, row * T};
    const uint64_t wd[3] = {(uint64_t)cp, (uint64_t)d, 2}, wst[2] = {row, row * d};
    const uint64_t od[2] = {(uint64_t)d, (uint64_t)T}, os[1] = {(uint64_t)d * 2};
    const uint32_t xb[3] = {64, 64, 4}, nb[4] = {64, 64, 2, 1}, kb[3] = {64, 128, 1},
                   wb[3] = {64, 256, 1}, ob[2] = {64, 32};
    // without dW there may be no x, without dx no dx: a map of the planes, unused, stands in
    if (!make_map(&mx, dw ? (const void*)x : dlp, 3, dw ? xd : kd, dw ? xs : ks, dw ? xb : kb) ||
        !make_map(&mn, dlp, 4, nd, ns, nb) || !make_map(&mk, dlp, 3, kd, ks, kb) ||
        !make_map(&mw, wp, 3, wd, wst, wb) ||
        !make_map(&mdx, dx ? dx : dlp, dx ? 2 : 3, dx ? od : kd, dx ? os : ks, dx ? ob : kb))
      return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(k_router_gemm, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRouterSmem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(k_router_gemm, dim3(grid), dim3(kRouterThreads), kRouterSmem, st, 1, mx, mn,
                      mk, mw, mdx, a);
    if (e != cudaSuccess) return e;
  }
  const long long n = (long long)d * E;
  const int dw_blocks = dw && !direct ? (int)std::min<long long>((n / 4 + 255) / 256, 8LL * sms) : 0;
  const int db_blocks = db ? (E + 31) / 32 : 0;
  if (dw_blocks + db_blocks == 0) return e;
  return launch_kernel(k_router_sum, dim3(dw_blocks + db_blocks), dim3(256), 0, st, 1, part,
                       ranges, n, dw, dw_blocks, sums, pd.blocks, E, db);
}

}  // namespace moe
