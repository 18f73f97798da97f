// int8_side.cu -- the adapter's thin products on the tensor cores with all 24
// bits of the fp32 factors:
//   row products     U = X A^T, V = dY B          (A operand: tokens x columns)
//   column products  dA = s V^T X, dB = s dY^T U  (A operand: columns x tokens)
// D[m, n] = sum_k A[m, k] B[n, k], M = 128 rows of the large matrix a tile and
// N = 3 NP: the fp32 factor is split into three bf16 parts (each remainder is
// exact), so that bf16 products lose nothing of it, and the parts' sums are
// added at the end.  The large matrix is read once, by TMA, K-major for the row
// products and MN-major (from the same row-major bytes) for the column ones.
//
// The tensor core's own sums lose a little at every step, so a sum runs over
// 256 terms only (16 steps) in one of two accumulators in TMEM; the epilogue
// warps drain it into fp32 registers while the other one fills.  Measured error
// 2e-7 of the result where one running sum over 8192 tokens had 3e-6 to 9e-6.
//
// Matrices that TMA does not take as they are (fp32 values, or bf16 of a width that
// is no multiple of 8) are copied in bf16 parts first, where that pays: the parts'
// products meet in the same sums.  The backward of 8192 tokens of 4096 x 4096 in
// fp32 at rank 64: 465 us, by fp32 FMAs 3250.
//
// Each product's chunks, tile after tile, are dealt out in equal runs over the
// SMs; the partial sums of a tile that several CTAs share are added up in CTA
// order by a second, small launch.  (By the last CTA of a tile, that held up its
// own run: 73 us where this takes 50.)  The runs do not depend on what else is in
// the launch: a gradient has the same bits whichever others are wanted.  Bound
// by HBM on the large matrix: V of 8192 x 12288 at rank 32 in 42 us (201 MB, 4.8
// TB/s), dB of the same with dA of 8192 x 4096 in 48 (268 MB, 5.6 TB/s).
#include "common.cuh"
#include "int8.h"
#include "int8_dev.cuh"
#include "internal.h"

namespace qlora {
namespace {

using namespace int8;

constexpr int kStep = 64;   // terms per ring stage: one 128-byte swizzle row
constexpr int kChunk = 4;   // stages per accumulator
constexpr int kTileA = 128 * kStep * 2;
constexpr int kSideThreads = 192;  // producer, MMA issuer, four epilogue warps

__host__ __device__ constexpr int side_n(int NP) { return NP == 8 ? 32 : 3 * NP; }  // MMA N
__host__ __device__ constexpr int side_cols(int NP) {                              // TMEM columns of it
  return NP == 8 ? 32 : NP == 16 ? 64 : NP == 32 ? 128 : 256;
}

template <int NP>
struct SideCfg {
  static constexpr int kTileB = side_n(NP) * kStep * 2;
  static constexpr int kStage = kTileA + kTileB;
  static constexpr int kStages = NP == 64 ? 5 : NP == 32 ? 7 : 8;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA per SM");
};

struct SideOut {
  float* out;       // [M x r], or [r x M] (transposed)
  uint16_t* parts;  // nullable: the result's own three parts, [3][NP][ld]
  int64_t M, ld;
  int32_t chunks, steps;  // of a tile
  int32_t transposed;
  float s;
};
struct SideArgs {
  SideOut job[2];
  int64_t tiles[2];   // the second may be 0
  int64_t units[2];   // chunks of all the job's tiles
  int32_t r, ctas;
  float* part;        // [CTAs][2 jobs][2][NP][128]
  uint32_t* err;
  uint64_t wait_ns;
};

__device__ __forceinline__ int64_t side_lo(const SideArgs& p, int job, int64_t cta) {
  return p.units[job] * cta / p.ctas;
}

// The chunks of this CTA: its run of job 0, then its run of job 1.
struct SideWalk {
  int64_t left, tile;
  int32_t job, chunk;
  __device__ __forceinline__ explicit SideWalk(const SideArgs& p) {
    open(p, 0);
    if (left == 0) open(p, 1);
  }
  __device__ __forceinline__ void open(const SideArgs& p, int k) {
    job = k;
    const int64_t lo = side_lo(p, k, blockIdx.x);
    left = side_lo(p, k, (int64_t)blockIdx.x + 1) - lo;
    tile = left ? lo / p.job[k].chunks : 0;
    chunk = left ? (int32_t)(lo - tile * p.job[k].chunks) : 0;
  }
  __device__ __forceinline__ int steps(const SideArgs& p) const {
    const int n = p.job[job].steps - chunk * kChunk;
    return n < kChunk ? n : kChunk;
  }
  __device__ __forceinline__ void next(const SideArgs& p) {
    if (--left == 0) {
      if (job == 0) open(p, 1);
      return;
    }
    if (++chunk == p.job[job].chunks) {
      chunk = 0;
      ++tile;
    }
  }
};

// CTA whose run of the job holds unit u, and where that run begins.
__device__ __forceinline__ int64_t side_owner(const SideArgs& p, int job, int64_t u, int64_t& lo) {
  int64_t c = u * p.ctas / p.units[job];
  while (side_lo(p, job, c + 1) <= u) ++c;
  while ((lo = side_lo(p, job, c)) > u) --c;
  return c;
}

__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool a_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// Columns j0 .. j0 + J of row m of a product's result.
template <int NP, int J>
__device__ __forceinline__ void side_write(const SideOut& o, int r, int64_t m, int j0, const float (&acc)[J]) {
  if (m >= o.M) {
    // the parts' rows end with zeros: they meet zero rows of the large matrix
    if (o.parts && m < o.ld)
      for (int j = j0; j < min(r, j0 + J); ++j)
        for (int q = 0; q < 3; ++q) o.parts[((int64_t)q * NP + j) * o.ld + m] = 0;
    return;
  }
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int j = j0 + i;
    if (j < r) {
      const float v = o.s * acc[i];
      o.out[o.transposed ? (int64_t)j * o.M + m : m * r + j] = v;
      if (o.parts) {
        float rest = v;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const __nv_bfloat16 b = __float2bfloat16_rn(rest);
          o.parts[((int64_t)q * NP + j) * o.ld + m] = __bfloat16_as_ushort(b);
          rest -= __bfloat162float(b);
        }
      }
    }
  }
}

template <bool A_MN, int NP>
__global__ void __launch_bounds__(kSideThreads, 1)
    side_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap tb0,
                const __grid_constant__ CUtensorMap ta1, const __grid_constant__ CUtensorMap tb1,
                const SideArgs p) {
  using C = SideCfg<NP>;
  constexpr uint32_t kIdesc = idesc_bf16(side_n(NP), A_MN);
  constexpr int kCols = side_cols(NP);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(smem + C::kStages * C::kStage);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::kStages;
  uint64_t* acc_full = bars + 2 * C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  volatile uint32_t* tmem_slot = (volatile uint32_t*)(acc_empty + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    griddep_launch_dependents();  // the summing launch waits for this grid itself
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&ta0);
    prefetch_tensormap(&tb0);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)tmem_slot), 2 * kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (SideWalk w(p); w.left > 0 && ok; w.next(p)) {
      const CUtensorMap* ta = w.job ? &ta1 : &ta0;
      const CUtensorMap* tb = w.job ? &tb1 : &tb0;
      const int m0 = (int)w.tile * 128, steps = w.steps(p);
      for (int i = 0; i < steps; ++i) {
        if (__any_sync(0xffffffffu, *abort_flag != 0) ||
            !warp_wait(smem_u32(&empty[s]), ph ^ 1u, p.wait_ns, p.err, 0x801)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + s * C::kStage);
          const int k = (w.chunk * kChunk + i) * kStep;
          mbar_arrive_expect_tx(fb, C::kStage);
          if (A_MN) {
            tma_load_2d(dst, ta, fb, m0, k);
            tma_load_2d(dst + kTileA / 2, ta, fb, m0 + 64, k);
          } else {
            tma_load_2d(dst, ta, fb, k, m0);
          }
          tma_load_2d(dst + kTileA, tb, fb, k, 0);
        }
        __syncwarp();
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
    }
    if (!ok)  // copies in flight land before the CTA exits
      for (int i = 0; i < C::kStages; ++i) {
        warp_wait(smem_u32(&full[s]), ph ^ 1u, p.wait_ns, nullptr, 0);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
  } else if (warp == 1) {
    int s = 0, b = 0;
    uint32_t ph = 0, pa = 0;
    bool ok = true;
    for (SideWalk w(p); w.left > 0 && ok; w.next(p)) {
      const int steps = w.steps(p);
      if (!warp_wait(smem_u32(&acc_empty[b]), pa ^ 1u, p.wait_ns, p.err, 0x802)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(kCols * b);
      for (int i = 0; i < steps; ++i) {
        if (!warp_wait(smem_u32(&full[s]), ph, p.wait_ns, p.err, 0x803)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t base = smem_u32(smem + s * C::kStage);
          const uint64_t ad = A_MN ? sdesc(base, kTileA / 2, 1024) : sdesc(base, 16, 1024);
          const uint64_t bd = sdesc(base + kTileA, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)
            umma_bf16(d, ad + (A_MN ? 128 : 2) * kk, bd + 2 * kk, kIdesc, (i | kk) ? 1u : 0u);
          umma_commit(smem_u32(&empty[s]));
          if (i + 1 == steps) umma_commit(smem_u32(&acc_full[b]));
        }
        __syncwarp();
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      if (++b == 2) { b = 0; pa ^= 1u; }
    }
  } else {
    const int quad = warp & 3;
    int b = 0;
    uint32_t pa = 0;
    float acc[NP];
    int run = 0;  // chunks in acc
    int segment = 0;
    for (SideWalk w(p); w.left > 0;) {
      const int job = w.job, chunk = w.chunk;
      const int64_t tile = w.tile;
      if (run == 0) {
#pragma unroll
        for (int j = 0; j < NP; ++j) acc[j] = 0.0f;
      }
      // one answer for all four warps, which meet at barriers below
      if (!all_of<128>(mbar_wait(smem_u32(&acc_full[b]), pa, p.wait_ns, p.err, 0x804))) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(kCols * b);
#pragma unroll
      for (int j0 = 0; j0 < NP; j0 += 8) {
        uint32_t v[3][8];
#pragma unroll
        for (int q = 0; q < 3; ++q) tmem_ld_32x32b_x8(d + (uint32_t)(q * NP + j0), v[q]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[j0 + j] += (__uint_as_float(v[2][j]) + __uint_as_float(v[1][j])) + __uint_as_float(v[0][j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
      if (++b == 2) { b = 0; pa ^= 1u; }
      ++run;
      w.next(p);
      const SideOut& o = p.job[job];
      const bool run_ends = w.left == 0 || w.job != job;
      if (chunk + 1 < o.chunks && !run_ends) continue;
      // the segment of this CTA in the tile is done
      const int64_t m = tile * 128 + 32 * quad + lane;
      if (run == o.chunks) {
        side_write<NP, NP>(o, p.r, m, 0, acc);
      } else {
        float* mine = p.part + (((int64_t)blockIdx.x * 2 + job) * 2 + (segment ? 1 : 0)) * NP * 128 + 32 * quad + lane;
#pragma unroll
        for (int j = 0; j < NP; ++j) mine[j * 128] = acc[j];
      }
      run = 0;
      segment = run_ends ? 0 : segment + 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kCols);
  }
}

// The tiles that several CTAs shared: their partial sums in CTA order.  One CTA
// for eight columns of a tile, a thread an output row, four CTAs' sums on their
// way at once.  (All columns by one CTA: 22 us after the products of 8192 tokens
// at rank 64, where this takes 8.)
template <int NP>
__global__ void __launch_bounds__(128) side_sum_kernel(const SideArgs p) {
  constexpr int kGroups = NP / 8;
  const int64_t at = blockIdx.x / kGroups;
  const int j0 = 8 * (int)(blockIdx.x % kGroups);
  const int job = at >= p.tiles[0] ? 1 : 0;
  const SideOut& o = p.job[job];
  const int64_t tile = at - (job ? p.tiles[0] : 0), u0 = tile * o.chunks, u1 = u0 + o.chunks;
  int64_t lo;
  int64_t c = side_owner(p, job, u0, lo);
  griddep_wait();  // every CTA: this grid ends only after the one before it
  if (side_lo(p, job, c + 1) >= u1) return;  // one CTA had it all (and has written it)
  // walk on from CTA c by the quotient and remainder of units c / ctas
  const int64_t quo = p.units[job] / p.ctas, rest = p.units[job] % p.ctas;
  int64_t rem = p.units[job] * c - lo * p.ctas;
  int which = lo >= u0 ? 0 : 1;  // the first segment of its run, unless that began in a tile before
  auto next = [&](int64_t& from) {  // the next CTA with a run in the tile
    while (lo < u1) {
      int64_t hi = lo + quo;
      rem += rest;
      if (rem >= p.ctas) {
        rem -= p.ctas;
        ++hi;
      }
      const bool some = hi > lo;  // (more CTAs than chunks)
      lo = hi;
      from = ((c++ * 2 + job) * 2 + which) * NP * 128 + threadIdx.x;
      which = 0;
      if (some) return true;
    }
    return false;
  };
  float acc[8] = {};
  constexpr int kAhead = 4;
  for (bool more = true; more;) {
    float v[kAhead][8];
    bool have[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      int64_t from = 0;
      have[q] = more && next(from);
      more = have[q];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[q][j] = have[q] ? __ldcg(p.part + from + (j0 + j) * 128) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (have[q]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[q][j];
      }
  }
  side_write<NP, 8>(o, p.r, tile * 128 + threadIdx.x, j0, acc);
}

// The three bf16 parts of up to two fp32 factors, [3][NP][ld], zeros past a
// row's entries: F(k, j) = src[k r + j] (kr) or src[j n + k].
struct SplitJob {
  const float* src;
  uint16_t* dst;
  int64_t n, len, ld;
  uint32_t wrap, div;
  int32_t kr, blocks;
};
struct SplitArgs {
  SplitJob job[2];
  int32_t r, NP;
};
// A block takes 64 entries of 16 factor rows; a factor given as [n x r] is
// turned in shared memory, so that both sides are read and written in runs.
// (All rows of 64 entries in one block: 12 us at rank 64 over 4096 entries, where
// this takes 4.6.)
constexpr int kSplitRows = 16;
__global__ void __launch_bounds__(256) split_kernel(const SplitArgs a) {
  __shared__ float tile[kSplitRows][65];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int second = (int)blockIdx.x >= a.job[0].blocks ? 1 : 0;
  const SplitJob b = second ? a.job[1] : a.job[0];
  const int groups = (a.r + kSplitRows - 1) / kSplitRows;
  const int block = (int)blockIdx.x - (second ? a.job[0].blocks : 0);
  const int64_t k0 = (int64_t)(block / groups) * 64;
  const int j0 = block % groups * kSplitRows, rows = min(kSplitRows, a.r - j0);
#pragma unroll
  for (int i = threadIdx.x; i < 64 * kSplitRows; i += 256) {
    const int j = b.kr ? i % kSplitRows : i >> 6, k = b.kr ? i / kSplitRows : i & 63;
    const uint32_t e = (uint32_t)(k0 + k);
    const int64_t at = b.wrap ? e % b.wrap : e / b.div;
    float v = 0.0f;
    if (j < rows && k0 + k < b.len && at < b.n)
      v = __ldg(b.src + (b.kr ? at * a.r + j0 + j : (int64_t)(j0 + j) * b.n + at));
    tile[j][k] = v;
  }
  __syncthreads();
#pragma unroll
  for (int e = threadIdx.x; e < 64 * kSplitRows; e += 256) {
    const int j = e >> 6, k = e & 63;
    if (j >= rows || k0 + k >= b.ld) continue;
    float v = tile[j][k];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      b.dst[((int64_t)q * a.NP + j0 + j) * b.ld + k0 + k] = __bfloat16_as_ushort(h);
      v -= __bfloat162float(h);
    }
  }
}

// Copies of up to two matrices [R x N] in bf16 parts: a thread takes eight
// columns of a row.  Zeros past N.
struct CopyArgs {
  const void* src[2];
  uint4* dst[2];
  int64_t N[2], pitch[2];
  int64_t R;
};
template <typename T>
__global__ void __launch_bounds__(256) side_copy_kernel(const CopyArgs a) {
  constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
  const int job = blockIdx.y;
  const int64_t N = job ? a.N[1] : a.N[0], per = (job ? a.pitch[1] : a.pitch[0]) / 8, count = a.R * per;
  const T* src = (const T*)(job ? a.src[1] : a.src[0]);
  uint4* dst = job ? a.dst[1] : a.dst[0];
  const bool wide = sizeof(T) == 4 && N % 4 == 0 && (uintptr_t)src % 16 == 0;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < count; e += (int64_t)gridDim.x * 256) {
    const int64_t row = count <= UINT32_MAX ? (int64_t)((uint32_t)e / (uint32_t)per) : e / per, k = 8 * (e - row * per);
    const T* p = src + row * N + k;
    float v[8];
    if (wide && k + 8 <= N) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(p)), y = __ldcs(reinterpret_cast<const float4*>(p) + 1);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < N ? to_f32(p[i]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      uint32_t w[4] = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
        w[i / 2] |= (uint32_t)__bfloat16_as_ushort(h) << (16 * (i & 1));
        v[i] -= __bfloat162float(h);
      }
      dst[(row * kParts + q) * per + k / 8] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <bool A_MN, int NP>
cudaError_t side_go(const CUtensorMap* t, const SideArgs& a, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow_smem(side_kernel<A_MN, NP>, SideCfg<NP>::kSmem, done);
  if (e != cudaSuccess) return e;
  side_kernel<A_MN, NP><<<(unsigned)a.ctas, kSideThreads, SideCfg<NP>::kSmem, st>>>(t[0], t[1], t[2], t[3], a);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(side_sum_kernel<NP>, (int)(a.tiles[0] + a.tiles[1]) * (NP / 8), 128, 0, st, a);
  count_launch();
  return e;
}

template <bool A_MN>
cudaError_t side_rank(const CUtensorMap* t, const SideArgs& a, int NP, cudaStream_t st) {
  switch (NP) {
    case 8: return side_go<A_MN, 8>(t, a, st);
    case 16: return side_go<A_MN, 16>(t, a, st);
    case 32: return side_go<A_MN, 32>(t, a, st);
    default: return side_go<A_MN, 64>(t, a, st);
  }
}

}  // namespace

int side_np(int32_t r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64; }
int64_t side_ld(int64_t n) { return up(n, 8) * 8; }
size_t side_parts_bytes(int64_t len, int32_t r) {
  return align_up((size_t)3 * side_np(r) * (size_t)side_ld(len) * 2, 256);
}
size_t side_part_ws(int32_t r) { return (size_t)sm_count() * 4 * side_np(r) * 128 * 4; }
bool side_takes(const void* P, int64_t R, int64_t N) {
  return R > 0 && R <= INT32_MAX - 256 && N % 8 == 0 && (uintptr_t)P % 16 == 0;
}

// The copy costs its bytes (16 a value in fp32, with what the product reads, 6 in
// bf16), the fp32 kernels their products (eight columns of the factor at least).
// 8192 x 4096 in fp32 at rank 16 (2^29): U in 102 us with the copy, 141 by FMAs;
// at rank 8 100 and 70.  8191 x 4097 in bf16 at rank 8 (2^28): 48 and 110.
// A bf16 matrix of other N has no copy, also where its base is unaligned (8192 x
// 4096 x 4096, backward: 175 us aligned and 566 unaligned at rank 8, 212 and 4890 at
// rank 64): its room would be reserved for every aligned one.
bool side_copies(bool bf16, int64_t R, int64_t N, int32_t r) {
  if (R <= 256 || (bf16 && N % 8 == 0)) return false;
  return (double)R * (double)N * ((r + 7) / 8 * 8) >= (bf16 ? 134217728.0 : 536870912.0);
}
size_t side_copy_bytes(bool bf16, int64_t R, int64_t N) {
  return align_up((size_t)R * (bf16 ? 1 : 3) * (size_t)side_ld(N) * 2, 256);
}
SideMatrix side_matrix(const void* P, bool bf16, int64_t R, int64_t N, int32_t r, void* copy) {
  if (bf16 && side_takes(P, R, N)) return {P, N, N, 1};
  if (side_copies(bf16, R, N, r)) return {copy, N, side_ld(N), bf16 ? 1 : 3};
  return {P, N, N, 0};
}

cudaError_t launch_side_copy(const SideCopy* c, int count, bool bf16, int64_t R, cudaStream_t st) {
  if (count == 0) return cudaSuccess;
  CopyArgs a = {};
  a.R = R;
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    a.src[i] = c[i].src;
    a.dst[i] = (uint4*)c[i].m.P;
    a.N[i] = c[i].m.N;
    a.pitch[i] = c[i].m.pitch;
    const int64_t blocks = up(R * c[i].m.pitch / 8, 256);
    if (blocks > most) most = blocks;
  }
  const dim3 grid((unsigned)(most < sm_count() * 16 ? most : sm_count() * 16), (unsigned)count);
  if (bf16) side_copy_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  else side_copy_kernel<float><<<grid, 256, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_side_split(const SideFactor* f, int count, int32_t r, cudaStream_t st) {
  SplitArgs a = {};
  a.r = r;
  a.NP = side_np(r);
  int blocks = 0;
  for (int i = 0; i < count; ++i) {
    SplitJob& b = a.job[i];
    b.src = f[i].src;
    b.dst = f[i].parts;
    b.n = f[i].n;
    b.len = f[i].len;
    b.ld = side_ld(f[i].len);
    b.wrap = (uint32_t)f[i].wrap;
    b.div = (uint32_t)f[i].div;
    b.kr = f[i].kr ? 1 : 0;
    b.blocks = (int)(up(b.ld, 64) * up(r, kSplitRows));
    blocks += b.blocks;
  }
  if (blocks == 0) return cudaSuccess;
  split_kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_side(const SideProduct* f, int count, bool columns, int64_t R, int32_t r, void* part,
                        uint32_t* hdr, cudaStream_t st) {
  const int NP = side_np(r);
  CUtensorMap t[4];
  SideArgs a = {};
  for (int i = 0; i < count; ++i) {
    // P as [R x parts pitch] (rows: one output row each) or [parts R x pitch]
    const SideMatrix& m = f[i].m;
    const int64_t cols = columns ? m.pitch : m.parts * m.pitch, rows = columns ? m.parts * R : R;
    const int64_t K = columns ? rows : cols, M = columns ? m.N : R;
    SideOut& o = a.job[i];
    o.out = f[i].out;
    o.parts = f[i].parts;
    o.M = M;
    o.ld = side_ld(M);
    o.steps = (int32_t)up(K, kStep);
    o.chunks = (int32_t)up(o.steps, kChunk);
    o.transposed = f[i].transposed ? 1 : 0;
    o.s = f[i].s;
    a.tiles[i] = up(M, 128);
    a.units[i] = a.tiles[i] * o.chunks;
    const int64_t ld = side_ld(K);
    if (!make_map_2d(&t[2 * i], m.P, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)cols, (uint64_t)rows,
                     (uint64_t)cols * 2, 64, columns ? 64 : 128) ||
        !make_map_2d(&t[2 * i + 1], f[i].factor, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)ld,
                     (uint64_t)3 * NP, (uint64_t)ld * 2, 64, (uint32_t)side_n(NP)))
      return cudaErrorInvalidValue;
  }
  if (count == 1) {
    a.job[1].chunks = 1;
    t[2] = t[0];
    t[3] = t[1];
  }
  a.r = r;
  a.part = (float*)part;
  a.err = hdr;
  a.wait_ns = kWaitLimitNs;
  a.ctas = sm_count();
  return columns ? side_rank<true>(t, a, NP, st) : side_rank<false>(t, a, NP, st);
}

}  // namespace qlora
