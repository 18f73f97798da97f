// int8_tc.cu -- the integer product of the 8-bit base on the tensor cores
// (tcgen05.mma kind::i8: signed bytes in, exact 32-bit sums in TMEM).
//
// Two kernels share the operand layout: 128-byte K steps (one 128-byte
// swizzle row per operand row), loaded by TMA, zero-filled past the edges.
// The activations are K-major codes; the weight codes are K-major in the
// forward and, read from the same [O x I] bytes, MN-major in the input
// gradient (a 128 x 128 box with the rows along K), so one tensor map and no
// transposed copy serve both.
//
// pair_kernel   many tokens: a CTA pair takes 256 tokens x 256 outputs
//               (cta_group::2: each CTA loads its half of both operands, 32 KB
//               a step against the 48 KB that one CTA's 128 x 256 tile needs
//               for the same work; at the integer rate the latter asks L2 for
//               more bytes a cycle than an SM can take).  Persistent, two
//               accumulators in TMEM: the epilogue of one tile runs under the
//               next one's products.  16384 tokens, 17408 x 5120, rank 16: 916 us,
//               3.2 POP/s; the tensor pipes are busy for nearly all of a CTA's
//               time and the clock is what the power limit leaves (1.4 to 1.6 of
//               1.965 GHz).
// stream_kernel few tokens or few tiles: the weight tile is the MMA's M side
//               (128 outputs x 16..128 tokens), so few tokens cost no wasted
//               rows and the kernel runs at the weight's bandwidth; the K
//               steps of all tiles are dealt out evenly over the SMs, and
//               what several CTAs add to one tile meets in 32-bit integer
//               atomics, exact in any order.
//
// The adapter term s T L^T keeps fp32 accuracy in both.  The stream kernel adds
// it in its epilogue by fp32 FMAs: r an output against K integer products.  In
// the pair kernel that epilogue, whose factor comes out of shared memory at 16
// bytes for two FMAs, outlasted the products from rank 16 on (8192 tokens of 4096 x
// 4096: 86, 114, 186 and 341 us at ranks 8, 16, 32 and 64), so T and L are split
// into three bf16 parts and the term is one to six more K steps on the tensor
// cores (88, 90, 93 and 99 us).  It has no TMEM of its own: the epilogue warps
// take a tile's integer sums into registers, the adapter's product then fills the
// same columns from zero while the next tile's integer products run into the other
// half, and the warps add the two.
//
// Every wait is bounded; on expiry the kernel records QLORA_ERR_TIMEOUT,
// stops issuing, and still reaches its barriers and frees its TMEM.
#include "common.cuh"
#include "int8.h"
#include "int8_dev.cuh"
#include "internal.h"

namespace qlora {
namespace {

using namespace int8;

constexpr int kBK = 128;              // K bytes per step
constexpr int kHalf = 128 * kBK;      // bytes of a 128-row operand tile

struct Epi {
  int64_t R, N;
  const float* xs;   // [R] row scale
  const float* ws;   // [N] channel scale (forward), else null
  const float* T;    // [R x r] U or V
  const float* L;    // B [N x r] or A [r x N]
  int32_t r;
  float s;
  void* out;
  int32_t tma_out;   // pair
  int32_t bf16;      // stream
  uint32_t* err;
  uint64_t wait_ns;
};

// kind::i8 instruction descriptor: s8 x s8 -> s32.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N, bool a_mn, bool b_mn) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// kind::f16: bf16 x bf16 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int CTAS>
__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  if (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs of the pair once every
// prior MMA of the thread is complete.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
      "%1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// TMA load into this CTA, completing on a barrier that may be the peer's.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* tmap, uint32_t bar, int32_t x,
                                              int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// The same box into L2 only.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__host__ __device__ constexpr int rank_pad(int r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64; }

// ------------------------------------------------------------ pair kernel

constexpr int kPairStages = 5;
constexpr int kStage = 2 * kHalf;  // A and B half tiles of one CTA
constexpr int kEpiWarps = 8;       // two to a TMEM lane quarter, 64 columns in turn
constexpr int kOutBuf = 4096;      // staged output of a warp: 32 rows x 128 bytes
constexpr int kPairSmem = 1024 + kPairStages * kStage + kEpiWarps * kOutBuf + 2 * 1024 + 256;
static_assert(kPairSmem <= 227 * 1024, "one CTA per SM");
constexpr int kPairThreads = 128 + 32 * kEpiWarps;
// The epilogue warps hold 128 sums each and take registers from the other four:
// 128 kPairRegs + 256 kEpiRegs is no more than the 384 x 168 of the launch.
constexpr int kPairRegs = 72, kEpiRegs = 216;
static_assert(128 * kPairRegs + 32 * kEpiWarps * kEpiRegs <= kPairThreads * 168, "registers of the launch");

struct PairArgs {
  Epi e = {};
  int32_t KB, tiles_m, tiles_n;
  int32_t KA;   // K steps of the adapter's product
  int32_t at;   // the step of a tile before which the last tile's adapter product is issued
};

// Parts of T and of L that meet in the adapter's product, one pair of them after
// another along its K (see pack_kernel): the small ones first, so that the tensor
// core's own rounding, which goes with the sum so far, is small until the last.
__host__ __device__ constexpr int part_T(int c) { return c == 0 ? 2 : c == 1 || c == 3 ? 1 : 0; }
__host__ __device__ constexpr int part_L(int c) { return c == 2 ? 2 : c == 1 || c == 4 ? 1 : 0; }

// Tile t of the persistent order: groups of kGroup token tiles, every output
// tile of a group before the next, so that what runs at once shares its
// operands in L2.
__device__ __forceinline__ void pair_tile(int64_t t, int tiles_m, int tiles_n, int& m, int& n) {
  constexpr int kGroup = 8;
  const int64_t per = (int64_t)kGroup * tiles_n;
  const int first = (int)(t / per) * kGroup, in = (int)(t % per);
  const int size = min(tiles_m - first, kGroup);
  m = first + in % size;
  n = in / size;
}

template <bool DX, typename OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_l,
                const __grid_constant__ CUtensorMap tm_out, const PairArgs p) {
  constexpr uint32_t kIdesc = idesc_i8(256, 256, false, DX), kAdapter = idesc_bf16(256, 256);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* outbuf = smem + kPairStages * kStage;
  float* wscale = (float*)(outbuf + kEpiWarps * kOutBuf);  // [2][256]
  uint64_t* bars = (uint64_t*)(wscale + 512);
  uint64_t* full = bars;                      // leader: both CTAs' loads landed
  uint64_t* empty = bars + kPairStages;       // both: the step's products are done
  uint64_t* int_full = bars + 2 * kPairStages;  // both: the integer sums of a tile
  uint64_t* int_read = int_full + 2;          // leader: in the registers of both CTAs' epilogue warps
  uint64_t* acc_full = int_read + 2;          // both: the adapter's sums, in the same place
  uint64_t* acc_read = acc_full + 2;          // leader: read by the epilogue warps of both
  volatile uint32_t* tmem_slot = (volatile uint32_t*)(acc_read + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&int_full[b]), 1);
      mbar_init(smem_u32(&int_read[b]), 2 * kEpiWarps);
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_read[b]), 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_t);
    prefetch_tensormap(&tm_l);
    prefetch_tensormap(&tm_out);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32((const void*)tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegs));
    if (warp == 0) {
    // ---------------------------------------------------------- producer
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    // One step: a box of each operand, into this CTA's half of the stage.
    auto step = [&](const CUtensorMap* ma, int xa, int ya, const CUtensorMap* mb, int xb, int yb) {
      if (!ok) return;
      if (!warp_wait(smem_u32(&empty[s]), ph ^ 1u, p.e.wait_ns, p.e.err, 0x501)) {
        *abort_flag = 1;
        ok = false;
        return;
      }
      if (elect_one()) {
        const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + s * kStage);
        if (rank == 0) mbar_arrive_expect_tx(fb, 2 * kStage);
        const uint32_t lead = at_rank(fb, 0);
        tma_load_pair(dst, ma, lead, xa, ya);
        tma_load_pair(dst + kHalf, mb, lead, xb, yb);
      }
      __syncwarp();
      if (++s == kPairStages) { s = 0; ph ^= 1u; }
    };
    int m0 = 0, n0 = 0;
    bool last = false;  // a tile before this one, at m0, n0
    for (int64_t t = cluster; t < tiles && ok; t += clusters) {
      int tm, tn;
      pair_tile(t, p.tiles_m, p.tiles_n, tm, tn);
      const int m1 = tm * 256 + 128 * (int)rank, n1 = tn * 256 + 128 * (int)rank;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        ok = false;
        break;
      }
      for (int kb = 0; kb < p.KB; ++kb) {
        if (last && kb == p.at)
          for (int k = 0; k < p.KA; ++k) step(&tm_t, 64 * k, m0, &tm_l, 64 * k, n0);
        step(&tm_x, kb * kBK, m1, &tm_w, DX ? n1 : kb * kBK, DX ? kb * kBK : n1);
      }
      m0 = m1;
      n0 = n1;
      last = true;
    }
    if (last)
      for (int k = 0; k < p.KA; ++k) step(&tm_t, 64 * k, m0, &tm_l, 64 * k, n0);
    // every copy has landed and every commit to this CTA's barriers has
    // arrived before the pair may exit
    for (int i = 0; i < kPairStages; ++i) {
      warp_wait(smem_u32(&empty[s]), ph ^ 1u, p.e.wait_ns, ok ? p.e.err : nullptr, 0x502);
      if (++s == kPairStages) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    if (rank == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t where) {
        if (ok && !warp_wait(smem_u32(bar), parity, p.e.wait_ns, p.e.err, where)) {
          *abort_flag = 1;
          ok = false;
        }
        tc_fence_after();
        return ok;
      };
      // Tile i's adapter product, into the columns that its integer sums left.
      auto adapter = [&](int64_t i) {
        const int b = (int)(i & 1);
        if (!wait(&int_read[b], (uint32_t)(i >> 1) & 1u, 0x503)) return;
        const uint32_t d = tmem + 256u * (uint32_t)b;
        for (int k = 0; k < p.KA; ++k) {
          if (!wait(&full[s], ph, 0x504)) return;
          if (elect_one()) {
            const uint32_t base = smem_u32(smem + s * kStage);
            const uint64_t ad = sdesc(base, 16, 1024), bd = sdesc(base + kHalf, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_pair(d, ad + 2 * kk, bd + 2 * kk, kAdapter, (k | kk) ? 1u : 0u);
            umma_commit_pair(smem_u32(&empty[s]));
            if (k + 1 == p.KA) umma_commit_pair(smem_u32(&acc_full[b]));
          }
          __syncwarp();
          if (++s == kPairStages) { s = 0; ph ^= 1u; }
        }
      };
      int64_t i = 0;
      for (int64_t t = cluster; t < tiles && ok; t += clusters, ++i) {
        const int b = (int)(i & 1);
        if (!wait(&acc_read[b], ((uint32_t)(i >> 1) & 1u) ^ 1u, 0x505)) break;
        const uint32_t d = tmem + 256u * (uint32_t)b;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (i > 0 && kb == p.at) adapter(i - 1);
          if (!wait(&full[s], ph, 0x506)) break;
          if (elect_one()) {
            const uint32_t base = smem_u32(smem + s * kStage);
            const uint64_t ad = sdesc(base, 16, 1024);
            const uint64_t bd = DX ? sdesc(base + kHalf, kHalf, 1024) : sdesc(base + kHalf, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)
              umma_i8<2>(d, ad + 2 * kk, bd + (DX ? 256 : 2) * kk, kIdesc, (kb | kk) ? 1u : 0u);
            umma_commit_pair(smem_u32(&empty[s]));
            if (kb + 1 == p.KB) umma_commit_pair(smem_u32(&int_full[b]));
          }
          __syncwarp();
          if (++s == kPairStages) { s = 0; ph ^= 1u; }
        }
      }
      if (i > 0 && ok) adapter(i - 1);
    }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ---------------------------------------------------------- epilogue
    // Lane = token.  A warp takes 128 columns of its lane quarter: their integer
    // sums into registers, which frees the TMEM columns for the adapter's sums.
    const int ew = warp - 4, quad = warp & 3, half = ew >> 2;
    uint8_t* mine = outbuf + ew * kOutBuf;
    const uint32_t buf = smem_u32(mine);
    int b = 0;
    uint32_t pa = 0;
    bool ok = true;
    for (int64_t t = cluster; t < tiles; t += clusters) {
      int tm, tn;
      pair_tile(t, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t row0 = (int64_t)tm * 256 + 128 * (int)rank + 32 * quad, row = row0 + lane;
      const int64_t n0 = (int64_t)tn * 256;
      const float sx = row < p.e.R ? __ldcg(p.e.xs + row) : 0.0f;
      if (!DX) {
        const int64_t n = n0 + threadIdx.x - 128;
        wscale[256 * b + threadIdx.x - 128] = n < p.e.N ? __ldg(p.e.ws + n) : 0.0f;
      }
      // one answer for all warps, which also have the scales then
      ok = mbar_wait(smem_u32(&int_full[b]), pa, p.e.wait_ns, p.e.err, 0x507) && ok;
      if (!all_of<32 * kEpiWarps>(ok)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t cols = tmem + ((uint32_t)(quad * 32) << 16) + 256u * (uint32_t)b + 128u * (uint32_t)half;
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(cols + 32u * (uint32_t)c, v[c]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(at_rank(smem_u32(&int_read[b]), 0));
      const float4* sw = reinterpret_cast<const float4*>(wscale + 256 * b + 128 * half);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
          if (!DX) w = sw[(32 * c + j) / 4];
          v[c][j] = __float_as_uint(__fmul_rn(__fmul_rn((float)(int)v[c][j], sx), w.x));
          v[c][j + 1] = __float_as_uint(__fmul_rn(__fmul_rn((float)(int)v[c][j + 1], sx), w.y));
          v[c][j + 2] = __float_as_uint(__fmul_rn(__fmul_rn((float)(int)v[c][j + 2], sx), w.z));
          v[c][j + 3] = __float_as_uint(__fmul_rn(__fmul_rn((float)(int)v[c][j + 3], sx), w.w));
        }
      // (after an expired wait what follows is not right, and the call reports it)
      ok = mbar_wait(smem_u32(&acc_full[b]), pa, p.e.wait_ns, p.e.err, 0x508) && ok;
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t a[32];
        tmem_ld_32x32b_x32(cols + 32u * (uint32_t)c, a);
        tmem_ld_wait();
        if (c == 3) {  // the columns may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(at_rank(smem_u32(&acc_read[b]), 0));
        }
        const int64_t n = n0 + 128 * half + 32 * c;
        if (n >= p.e.N && (sizeof(OUT) == 4 || (c & 1) == 0)) continue;  // the same for the whole warp
        if (sizeof(OUT) == 2 && n - 32 * (c & 1) >= p.e.N) continue;
        if (sizeof(OUT) == 4 || (c & 1) == 0) {
          if (lane == 0)  // the buffer's last store has been read
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          a[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[c][j]), __uint_as_float(a[j])));
        const uint32_t line = buf + (uint32_t)lane * 128;
        if (sizeof(OUT) == 4) {  // 32 columns fill the buffer
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared_v4(line + (uint32_t)((q ^ (lane & 7)) << 4), a[4 * q], a[4 * q + 1], a[4 * q + 2],
                         a[4 * q + 3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(a[8 * q + 2 * i]), __uint_as_float(a[8 * q + 2 * i + 1]));
            st_shared_v4(line + (uint32_t)(((4 * (c & 1) + q) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
          if ((c & 1) == 0) continue;
        }
        const int64_t x = sizeof(OUT) == 4 ? n : n - 32;  // of the buffer's first column
        if (p.e.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row < p.e.R) tma_store_2d(&tm_out, buf, (int32_t)x, (int32_t)row);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {  // rows that TMA does not take: row after row, in runs
          __syncwarp();
          const int rows = (int)min((int64_t)32, p.e.R - row0);
          OUT* o = (OUT*)p.e.out + row0 * p.e.N + x;
#pragma unroll
          for (int e0 = 0; e0 < (int)(128 / sizeof(OUT)); e0 += 32) {
            const int e = e0 + lane, byte = e * (int)sizeof(OUT);
            if (x + e >= p.e.N) continue;
#pragma unroll 8
            for (int i = 0; i < rows; ++i)
              o[i * p.e.N + e] =
                  *reinterpret_cast<const OUT*>(mine + i * 128 + ((((byte >> 4) ^ (i & 7)) << 4) | (byte & 15)));
          }
          __syncwarp();
        }
      }
      if (++b == 2) { b = 0; pa ^= 1u; }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// T and s L as the pair kernel's adapter product reads them: an fp32 value is
// the sum of three bf16 parts (each remainder is exact), a row's six runs of RP
// hold the parts that part_T or part_L names, and the product over the whole row
// is s T L^T but for terms below 2^-24 of its summands.  Zeros past r.
struct PackJob {
  const float* src;  // [n x r] (kr), or [r x n]
  uint16_t* dst;     // [n x 6 RP]
  int64_t n;
  float s;
  int32_t kr, right, blocks;
};
struct PackArgs {
  PackJob job[2];
  int32_t r;
};
// Rows of a block: one or two pairs of values a thread.
__host__ __device__ constexpr int pack_rows(int RP) { return RP == 8 ? 64 : RP == 64 ? 16 : 32; }
template <int RP>
__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a) {
  constexpr int kRows = pack_rows(RP);
  __shared__ float tile[kRows][RP + 1];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int second = (int)blockIdx.x >= a.job[0].blocks ? 1 : 0;
  const PackJob b = second ? a.job[1] : a.job[0];
  const int64_t n0 = ((int64_t)blockIdx.x - (second ? a.job[0].blocks : 0)) * kRows;
  const int rows = (int)min((int64_t)kRows, b.n - n0);
  griddep_wait();  // T is there (and every CTA waits: the grid ends after the ones before it)
  // consecutive threads along the source's rows
#pragma unroll
  for (int e0 = 0; e0 < kRows * RP; e0 += 256) {
    const int e = e0 + threadIdx.x, k = b.kr ? e / RP : e % kRows, j = b.kr ? e % RP : e / kRows;
    tile[k][j] = k < rows && j < a.r ? b.s * __ldcg(b.src + (b.kr ? (n0 + k) * a.r + j : j * b.n + n0 + k)) : 0.0f;
  }
  __syncthreads();
#pragma unroll
  for (int e0 = 0; e0 < kRows * RP / 2; e0 += 256) {
    const int e = e0 + threadIdx.x, k = e / (RP / 2), j = 2 * (e % (RP / 2));
    if (k >= rows) continue;
    uint32_t part[3] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = tile[k][j + i];
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        part[q] |= (uint32_t)__bfloat16_as_ushort(h) << (16 * i);
        v -= __bfloat162float(h);
      }
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(b.dst + (n0 + k) * 6 * RP + j);
#pragma unroll
    for (int c = 0; c < 6; ++c) out[c * RP / 2] = b.right ? part[part_L(c)] : part[part_T(c)];
  }
}

// ---------------------------------------------------------- stream kernel

template <int BN, int RT>
struct StreamCfg {
  static constexpr int kTok = BN * kBK;
  static constexpr int kStage = kHalf + kTok;
  static constexpr int kStages = BN <= 16 ? 11 : BN <= 32 ? 10 : BN <= 64 ? (RT > 32 ? 7 : 8) : RT > 16 ? 5 : 6;
  static constexpr int kCols = BN < 32 ? 32 : BN;  // TMEM columns of one accumulator
  // the tokens' rows of T, their scales, and (up to 16 tokens) rows of U
  static constexpr int kSide = BN * (RT + 1) * 4 + (BN == 16 ? BN * RT * 4 : 0);
  static constexpr int kSmem = 1024 + kStages * kStage + kSide + 512;
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA per SM");
};
constexpr int kStreamEpi = 256;  // epilogue threads: two warps to a TMEM lane quarter
constexpr int kStreamThreads = 64 + kStreamEpi;  // after the producer and the MMA issuer

struct StreamArgs {
  Epi e = {};
  int32_t KB, tok_tiles;
  int32_t ctas;   // those with a run (the others have side sums only)
  int64_t tiles;  // one token tile after the other, then the next weight tile
  int32_t shared;       // deal out K steps (tiles may be shared by CTAs), else whole tiles
  int32_t* part;        // [tiles][BN][128] sums of tiles that several CTAs share (zeroed)
  uint32_t* tickets;    // [tiles] K steps added so far (zeroed)
  // input gradient of up to 16 tokens: the adapter gradients beside it
  const void* X;        // [R x I]
  const void* dY;       // [R x O]
  const float* U;       // [R x r]
  float* dA;            // [r x I], nullable
  float* dB;            // [O x r], nullable
  int64_t I, O;
};

// The backward's side sums over up to 16 tokens, by the epilogue warps while
// the products run: dA[j, i] = sum_t sV[t, j] X[t, i], dB[o, j] = sum_t
// sU[t, j] dY[t, o]; a thread takes a column of X or dY at a time.  The column
// does not depend on the launch before this one, sV and sU do ([16 x RT] in
// shared memory, s folded in): the first column is loaded ahead of the wait.
struct SideSums {
  int64_t e, total, nA;
  float x[16];
  __device__ __forceinline__ SideSums(const StreamArgs& p, int et) {
    nA = p.dA ? p.I : 0;
    total = nA + (p.dB ? p.O : 0);
    e = (int64_t)blockIdx.x * kStreamEpi + et;
    load(p);
  }
  __device__ __forceinline__ void load(const StreamArgs& p) {
    if (e >= total) return;
    const bool a = e < nA;
    const int64_t col = a ? e : e - nA, n = a ? p.I : p.O;
    const void* P = a ? p.X : p.dY;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      x[t] = 0.0f;
      if (t < (int)p.e.R)
        x[t] = p.e.bf16 ? __bfloat162float(((const __nv_bfloat16*)P)[t * n + col]) : ((const float*)P)[t * n + col];
    }
  }
  template <int RT>
  __device__ __forceinline__ void run(const StreamArgs& p, const float* sV, const float* sU) {
    const int R = (int)p.e.R, r = p.e.r;
    while (e < total) {
      const bool a = e < nA;
      const int64_t col = a ? e : e - nA, step = a ? p.I : 1;
      const float* f = a ? sV : sU;
      float* out = a ? p.dA + col : p.dB + col * r;
#pragma unroll 1
      for (int j = 0; j < r; j += 4) {
        float d[4] = {};
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          if (t < R) {  // rows past R of sV, sU are not filled
            const float4 v = *reinterpret_cast<const float4*>(f + t * RT + j);
            d[0] = fmaf(v.x, x[t], d[0]);
            d[1] = fmaf(v.y, x[t], d[1]);
            d[2] = fmaf(v.z, x[t], d[2]);
            d[3] = fmaf(v.w, x[t], d[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < r) out[(j + i) * step] = d[i];
      }
      e += (int64_t)gridDim.x * kStreamEpi;
      load(p);
    }
  }
};

// The K steps of this CTA, tile after tile: `steps` of them, from step kb of
// tile (weight tile mt, token tile tt) on.  Every role walks them with running
// counters: a 64-bit division is a hundred instructions of its one thread.
struct Walk {
  int64_t tile, steps;
  int32_t kb, mt, tt;
  __device__ __forceinline__ explicit Walk(const StreamArgs& p) {
    const int64_t n = p.shared ? p.tiles * p.KB : p.tiles;
    const int64_t c = (int)blockIdx.x < p.ctas ? (int)blockIdx.x : p.ctas;
    const int64_t lo = n * c / p.ctas, hi = (int)blockIdx.x < p.ctas ? n * (c + 1) / p.ctas : lo;
    tile = p.shared ? lo / p.KB : lo;
    kb = p.shared ? (int32_t)(lo - tile * p.KB) : 0;
    steps = p.shared ? hi - lo : (hi - lo) * p.KB;
    mt = (int32_t)(tile / p.tok_tiles);
    tt = (int32_t)(tile - (int64_t)mt * p.tok_tiles);
  }
  // steps left of the current tile
  __device__ __forceinline__ int run(const StreamArgs& p) const {
    return (int)(steps < p.KB - kb ? steps : p.KB - kb);
  }
  __device__ __forceinline__ void advance(const StreamArgs& p, int n) {  // within the tile
    steps -= n;
    kb += n;
    if (kb == p.KB) {
      kb = 0;
      ++tile;
      if (++tt == p.tok_tiles) { tt = 0; ++mt; }
    }
  }
};


template <bool DX, int BN, int RT>
__global__ void __launch_bounds__(kStreamThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const StreamArgs p) {
  using C = StreamCfg<BN, RT>;
  constexpr uint32_t kIdesc = idesc_i8(128, BN, DX, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* side = (float*)(smem + C::kStages * C::kStage);  // [BN][RT] T, then [BN] scales
  uint64_t* bars = (uint64_t*)((uint8_t*)side + C::kSide);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::kStages;
  uint64_t* acc_full = bars + 2 * C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  volatile uint32_t* tmem_slot = (volatile uint32_t*)(acc_empty + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* last_flag = tmem_slot + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), kStreamEpi / 32);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)tmem_slot), 2 * C::kCols);
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
    // The weight does not depend on the launch before this one, the codes of
    // the activations do: the first stages' weight tiles are on their way
    // while that launch still runs, and the next ones on their way into L2 (up
    // to 57 MB of its 126 on 148 SMs).
    Walk w(p);
    const int ahead = (int)min((int64_t)C::kStages, w.steps);
    auto load_w = [&](const Walk& at, int slot) {
      const uint32_t fb = smem_u32(&full[slot]);
      mbar_arrive_expect_tx(fb, C::kStage);
      tma_load_2d(smem_u32(smem + slot * C::kStage), &tm_w, fb, DX ? at.mt * 128 : at.kb * kBK,
                  DX ? at.kb * kBK : at.mt * 128);
    };
    auto load_x = [&](const Walk& at, int slot) {
      tma_load_2d(smem_u32(smem + slot * C::kStage + kHalf), &tm_x, smem_u32(&full[slot]), at.kb * kBK,
                  at.tt * BN);
    };
    Walk early = w;
    for (int i = 0; i < ahead; ++i, early.advance(p, 1)) {
      if (elect_one()) load_w(early, i);
      __syncwarp();
    }
    for (int i = 0; i < 24 && early.steps > 0; ++i, early.advance(p, 1)) {
      if (elect_one())
        tma_prefetch_2d(&tm_w, DX ? early.mt * 128 : early.kb * kBK, DX ? early.kb * kBK : early.mt * 128);
      __syncwarp();
    }
    griddep_wait();
    for (int i = 0; w.steps > 0; ++i, w.advance(p, 1)) {
      if (i >= ahead && (__any_sync(0xffffffffu, *abort_flag != 0) ||
                         !warp_wait(smem_u32(&empty[s]), ph ^ 1u, p.e.wait_ns, p.e.err, 0x601))) {
        *abort_flag = 1;
        ok = false;
        break;
      }
      if (elect_one()) {
        if (i >= ahead) load_w(w, s);
        load_x(w, s);
      }
      __syncwarp();
      if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
    // copies in flight land before the CTA exits (the MMA has waited for
    // them all unless something gave up)
    if (!ok) {
      for (int i = 0; i < C::kStages; ++i) {
        warp_wait(smem_u32(&full[s]), ph ^ 1u, p.e.wait_ns, nullptr, 0);
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    int s = 0, b = 0;
    uint32_t ph = 0, pa = 0;
    bool ok = true;
    for (Walk w(p); w.steps > 0 && ok;) {
      const int run = w.run(p);
      if (!warp_wait(smem_u32(&acc_empty[b]), pa ^ 1u, p.e.wait_ns, p.e.err, 0x602)) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(C::kCols * b);
      for (int i = 0; i < run; ++i) {
        if (!warp_wait(smem_u32(&full[s]), ph, p.e.wait_ns, p.e.err, 0x603)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t base = smem_u32(smem + s * C::kStage);
          const uint64_t ad = DX ? sdesc(base, kHalf, 1024) : sdesc(base, 16, 1024);
          const uint64_t bd = sdesc(base + kHalf, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            umma_i8<1>(d, ad + (DX ? 256 : 2) * kk, bd + 2 * kk, kIdesc, (i | kk) ? 1u : 0u);
          umma_commit(smem_u32(&empty[s]));
          if (i + 1 == run) umma_commit(smem_u32(&acc_full[b]));
        }
        __syncwarp();
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
      }
      if (++b == 2) { b = 0; pa ^= 1u; }
      w.advance(p, run);
    }
  } else {
    // epilogue: lane = output n, TMEM column = token
    // (two warps to a quarter take runs of eight tokens in turn)
    const int quad = warp & 3, et = (int)threadIdx.x - 64, c_first = 8 * ((warp - 2) >> 2);
    SideSums sums(p, et);
    griddep_wait();
    int b = 0;
    uint32_t pa = 0;
    int staged = -1;  // token tile whose T and scales are in shared memory
    auto stage_side = [&](int64_t t0, int toks) {
      for (int e = et; e < toks * RT; e += kStreamEpi) {
        const int t = e / RT, j = e % RT;
        side[e] = j < p.e.r ? p.e.s * __ldcg(p.e.T + (t0 + t) * p.e.r + j) : 0.0f;
      }
      for (int e = et; e < toks; e += kStreamEpi) side[BN * RT + e] = __ldcg(p.e.xs + t0 + e);
    };
    if constexpr (BN == 16 && DX) {
      if (p.dA || p.dB) {  // a single token tile
        float* su = side + BN * (RT + 1);
        stage_side(0, (int)p.e.R);
        if (p.dB)
          for (int e = et; e < (int)p.e.R * RT; e += kStreamEpi) {
            const int t = e / RT, j = e % RT;
            su[e] = j < p.e.r ? p.e.s * __ldcg(p.U + t * p.e.r + j) : 0.0f;
          }
        staged = 0;
        epi_sync<kStreamEpi>();
        sums.template run<RT>(p, side, su);
      }
    }
    Walk w(p);
    while (w.steps > 0) {
      const int64_t tile = w.tile;
      const int steps = w.run(p), tt = w.tt;
      const int64_t n = (int64_t)w.mt * 128 + 32 * quad + lane, t0 = (int64_t)tt * BN;
      w.advance(p, steps);
      const int toks = (int)min((int64_t)BN, p.e.R - t0);
      // this tile's side inputs, while its products run
      uint64_t l[RT / 2];
      const bool in = n < p.e.N;
      if (!DX && (p.e.r & 3) == 0 && ((uintptr_t)p.e.L & 15) == 0) {
#pragma unroll
        for (int j = 0; j < RT / 4; ++j) {
          const float4 v = in && 4 * j < p.e.r ? __ldg(reinterpret_cast<const float4*>(p.e.L + n * p.e.r) + j)
                                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          l[2 * j] = pack2(v.x, v.y);
          l[2 * j + 1] = pack2(v.z, v.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < RT / 2; ++j) {
          float v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int q = 2 * j + i;
            v[i] = in && q < p.e.r ? __ldg(p.e.L + (DX ? (int64_t)q * p.e.N + n : n * p.e.r + q)) : 0.0f;
          }
          l[j] = pack2(v[0], v[1]);
        }
      }
      const float sw = !DX && in ? __ldg(p.e.ws + n) : 1.0f;
      if (tt != staged) {
        epi_sync<kStreamEpi>();  // the last tile's are read
        stage_side(t0, toks);
        staged = tt;
      }
      // one answer for all warps, which meet at barriers below
      if (!all_of<kStreamEpi>(mbar_wait(smem_u32(&acc_full[b]), pa, p.e.wait_ns, p.e.err, 0x604))) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const bool whole = steps == p.KB;
      int32_t* part = p.part + (tile * BN) * 128 + 32 * quad + lane;
      const uint32_t acc0 = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(C::kCols * b);
      bool finish = whole;
      if (!whole) {
#pragma unroll 1
        for (int c0 = c_first; c0 < toks; c0 += 16) {
          uint32_t acc[8];
          tmem_ld_32x32b_x8(acc0 + (uint32_t)c0, acc);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + j < toks) atomicAdd(part + (c0 + j) * 128, (int)acc[j]);
        }
        __threadfence();
        epi_sync<kStreamEpi>();
        if (warp == 2 && lane == 0)
          *last_flag = atomicAdd(p.tickets + tile, (uint32_t)steps) + (uint32_t)steps == (uint32_t)p.KB;
        epi_sync<kStreamEpi>();
        finish = *last_flag != 0;
        __threadfence();
        epi_sync<kStreamEpi>();  // all have read the flag
      }
      if (finish) {
        // eight tokens at a time (columns past the last token hold sums of
        // zero-filled rows and are not stored)
#pragma unroll 1
        for (int c0 = c_first; c0 < toks; c0 += 16) {
          uint32_t acc[8];
          if (whole) {
            tmem_ld_32x32b_x8(acc0 + (uint32_t)c0, acc);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = (uint32_t)__ldcg(part + (c0 + j) * 128);
          }
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float* T = side + (c0 + j) * RT;
            uint64_t d = 0;
#pragma unroll
            for (int q = 0; q < RT / 4; ++q) {
              const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(T + 4 * q);
              d = fma2(l[2 * q], t.x, d);
              d = fma2(l[2 * q + 1], t.y, d);
            }
            v[j] = __fadd_rn(__fmul_rn(__fmul_rn((float)(int)acc[j], side[BN * RT + c0 + j]), sw), sum2(d));
          }
          const int64_t o = (t0 + c0) * p.e.N + n;
          if (in && p.e.bf16) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c0 + j < toks) ((__nv_bfloat16*)p.e.out)[o + j * p.e.N] = __float2bfloat16_rn(v[j]);
          } else if (in) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c0 + j < toks) ((float*)p.e.out)[o + j * p.e.N] = v[j];
          }
          __syncwarp();  // lanes past N beside lanes that store: the next load of TMEM is one of the whole warp
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
      if (++b == 2) { b = 0; pa ^= 1u; }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * C::kCols);
  }
}

// ------------------------------------------------------------------- host

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// K steps of the pair kernel's adapter product: 64 bf16 each of 6 RP.
int adapter_steps(int r) { return (6 * rank_pad(r) + 63) / 64; }

struct Plan {
  bool pair;
  int bn;          // stream: token tile
  int64_t tiles;   // stream: tiles;  pair: tiles of 256 x 256
  int ctas;
  bool shared;     // stream: some tile is shared between CTAs
};

// Pair or stream, and how the latter's work is dealt out, by cost in K steps
// of one SM (512 cycles: what the products of a 128 x 256 half tile take, and
// also what the 32 KB of a 128 x 128 stream step take from L2).  The pair
// kernel pays whole rounds of tiles over the CTA pairs, with the adapter's steps,
// the last tile's epilogue and the packing of its factors (8); the stream kernel
// pays whole rounds of tiles over the SMs and the last one's epilogue, or, with
// tiles shared, an equal run of steps and the meeting of the partial sums, which
// grows with the token tile.  A tile takes no less than its epilogue: about nine
// steps for the pair kernel's, and for the stream kernel's as many as its adapter
// term reads from shared memory (nine at 128 tokens and rank 8).  Whole forward
// calls on both sides of the choice, stream and pair: 200 tokens of 4096 x 1024 13.7
// and 16.2 us at rank 8, 25.8 and 19.4 at rank 32; of 4096 x 4096 23.5 and 26.1, 43.0
// and 37.6; 800 tokens of 4096 x 1024 24.4 and 19.4 at rank 8.
Plan plan_for(int64_t R, int64_t N, int64_t K, int r) {
  const int64_t sms = sm_count(), KB = up(K, kBK), RT = rank_pad(r);
  Plan p;
  p.bn = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128;
  const int64_t pair_tiles = up(R, 256) * up(N, 256), tiles = up(R, p.bn) * up(N, 128);
  const int64_t pairs = sms / 2 > 0 ? sms / 2 : 1;
  const int64_t pair_tile = KB + adapter_steps(r), pair_least = 9;
  const int64_t cost_pair = up(pair_tiles, pairs) * (pair_tile > pair_least ? pair_tile : pair_least) + 18;
  const int64_t least = (R < p.bn ? R : p.bn) * RT / 112;  // epilogue of a stream tile, in steps
  const int64_t cost_whole = up(tiles, sms) * (KB > least ? KB : least) + (KB > least ? least : KB) + 5;
  const int64_t run = up(tiles * KB, sms), ends = up(tiles, sms) * 2 * least;
  const int64_t cost_shared = (run > ends ? run : ends) + 4 + p.bn / 8;
  p.shared = cost_shared < cost_whole;
  p.pair = R > 64 && cost_pair < (p.shared ? cost_shared : cost_whole);
  if (p.pair) {
    p.tiles = pair_tiles;
    p.ctas = (int)(2 * (pair_tiles < pairs ? pair_tiles : pairs));
    p.shared = false;
    return p;
  }
  p.tiles = tiles;
  // shared: runs of at least four steps, so that a CTA's start is paid for
  int64_t ctas = p.shared ? (tiles * KB / 4 > tiles ? tiles * KB / 4 : tiles) : tiles;
  if (ctas > sms) ctas = sms;
  p.ctas = (int)ctas;
  return p;
}

size_t pack_bytes(int64_t n, int r) { return align_up((size_t)n * 12 * (size_t)rank_pad(r), 256); }
size_t stream_part_bytes(const Plan& p) { return !p.shared ? 0 : align_up((size_t)p.tiles * (size_t)p.bn * 128 * 4, 256); }
size_t stream_ticket_bytes(const Plan& p) { return !p.shared ? 0 : align_up((size_t)p.tiles * 4, 256); }

template <int RP>
cudaError_t go_pack(const PackArgs& a, cudaStream_t st) {
  const cudaError_t e = launch_after(pack_kernel<RP>, a.job[0].blocks + a.job[1].blocks, 256, 0, st, a);
  count_launch();
  return e;
}

template <bool DX, typename OUT>
cudaError_t go_pair(const Plan& pl, const Int8Call& c, const CUtensorMap& x, const CUtensorMap& w, Epi e,
                    int64_t K, void* ws, cudaStream_t st) {
  const int RP = rank_pad(e.r);
  uint16_t *t6 = (uint16_t*)ws, *l6 = (uint16_t*)((char*)ws + pack_bytes(e.R, e.r));
  PackArgs k = {};
  k.job[0] = {e.T, t6, e.R, 1.0f, 1, 0, (int32_t)up(e.R, pack_rows(RP))};
  k.job[1] = {e.L, l6, e.N, e.s, DX ? 0 : 1, 1, (int32_t)up(e.N, pack_rows(RP))};
  k.r = e.r;
  cudaError_t err = RP == 8 ? go_pack<8>(k, st) : RP == 16 ? go_pack<16>(k, st)
                                                : RP == 32 ? go_pack<32>(k, st) : go_pack<64>(k, st);
  if (err != cudaSuccess) return err;
  CUtensorMap mt, ml, mo;
  const uint64_t row = (uint64_t)6 * RP;
  if (!make_map_2d(&mt, t6, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, row, (uint64_t)e.R, 2 * row, 64, 128) ||
      !make_map_2d(&ml, l6, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, row, (uint64_t)e.N, 2 * row, 64, 128))
    return cudaErrorInvalidValue;
  e.tma_out = ((uintptr_t)c.out % 16 == 0 && (e.N * sizeof(OUT)) % 16 == 0) ? 1 : 0;
  if (e.tma_out &&
      !make_map_2d(&mo, c.out, sizeof(OUT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                (uint64_t)e.N, (uint64_t)c.R, (uint64_t)e.N * sizeof(OUT), 128 / sizeof(OUT), 32))
    return cudaErrorInvalidValue;
  if (!e.tma_out) mo = x;  // not used
  PairArgs a;
  a.e = e;
  a.KB = (int32_t)up(K, kBK);
  a.tiles_m = (int32_t)up(e.R, 256);
  a.tiles_n = (int32_t)up(e.N, 256);
  a.KA = adapter_steps(e.r);
  a.at = a.KB / 2 < 6 ? a.KB / 2 : 6;
  static std::atomic<bool> done[kMaxDevices];
  err = allow_smem(pair_kernel<DX, OUT>, kPairSmem, done);
  if (err != cudaSuccess) return err;
  // the epilogue warps' registers come out of the launch's own: a build with fewer
  // would wait for them
  static const bool fits = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, pair_kernel<DX, OUT>) == cudaSuccess &&
           f.numRegs * kPairThreads >= 128 * kPairRegs + 32 * kEpiWarps * kEpiRegs;
  }();
  if (!fits) return cudaErrorLaunchOutOfResources;
  err = launch_after(pair_kernel<DX, OUT>, pl.ctas, kPairThreads, kPairSmem, st, x, w, mt, ml, mo, a);
  count_launch();
  return err;
}

template <bool DX, int BN, int RT>
cudaError_t go_stream(const Plan& pl, const CUtensorMap& x, const CUtensorMap& w, const StreamArgs& a,
                      cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  auto kern = stream_kernel<DX, BN, RT>;
  cudaError_t e = allow_smem(kern, (StreamCfg<BN, RT>::kSmem), done);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, pl.ctas, kStreamThreads, StreamCfg<BN, RT>::kSmem, st, x, w, a);
  count_launch();
  return e;
}

template <bool DX, int RT>
cudaError_t go(const Plan& pl, const Int8Call& c, const CUtensorMap& mx, const CUtensorMap& mw, const Epi& e,
               const Int8Few* few, int64_t K, void* ws, cudaStream_t st) {
  StreamArgs a = {};
  a.e = e;
  a.KB = (int32_t)up(K, kBK);
  a.tok_tiles = (int32_t)up(c.R, pl.bn);
  a.tiles = pl.tiles;
  a.shared = pl.shared ? 1 : 0;
  Plan run = pl;
  a.ctas = pl.ctas;
  if (!c.out) a.tiles = 0;  // only the side sums
  if (DX && few && (few->dA || few->dB)) {
    const int64_t want = up(c.I + c.O, kStreamEpi), most = want < sm_count() ? want : sm_count();
    if (run.ctas < most) run.ctas = (int)most;
  }
  a.part = (int32_t*)ws;
  a.tickets = (uint32_t*)((char*)ws + stream_part_bytes(pl));
  if (few && DX) {
    a.X = few->X;
    a.dY = c.P;
    a.U = few->U;
    a.dA = few->dA;
    a.dB = few->dB;
    a.I = c.I;
    a.O = c.O;
  }
  switch (pl.bn) {
    case 16: return go_stream<DX, 16, RT>(run, mx, mw, a, st);
    case 32: return go_stream<DX, 32, RT>(run, mx, mw, a, st);
    case 64: return go_stream<DX, 64, RT>(run, mx, mw, a, st);
    default: return go_stream<DX, 128, RT>(run, mx, mw, a, st);
  }
}

template <bool DX>
cudaError_t go_rank(const Plan& pl, const Int8Call& c, const int8_t* xq, const Epi& e, const Int8Few* few,
                    void* ws, cudaStream_t st) {
  CUtensorMap mx, mw;
  const int64_t K = DX ? c.O : c.I, xp = int8_act_pitch(K), wp = int8_pitch(c.I);
  if (!make_map_2d(&mw, c.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)wp, (uint64_t)c.O, (uint64_t)wp, 128,
                128) ||
      !make_map_2d(&mx, xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)int8_pitch(K), (uint64_t)c.R, (uint64_t)xp, 128,
                pl.pair ? 128 : (uint32_t)pl.bn))
    return cudaErrorInvalidValue;
  if (pl.pair)
    return c.bf16 ? go_pair<DX, __nv_bfloat16>(pl, c, mx, mw, e, K, ws, st)
                  : go_pair<DX, float>(pl, c, mx, mw, e, K, ws, st);
  switch (rank_pad(c.r)) {
    case 8: return go<DX, 8>(pl, c, mx, mw, e, few, K, ws, st);
    case 16: return go<DX, 16>(pl, c, mx, mw, e, few, K, ws, st);
    case 32: return go<DX, 32>(pl, c, mx, mw, e, few, K, ws, st);
    default: return go<DX, 64>(pl, c, mx, mw, e, few, K, ws, st);
  }
}

}  // namespace

size_t int8_tc_ws(bool dx, int64_t R, int64_t O, int64_t I, int32_t r) {
  if (R == 0) return 0;
  const int64_t N = dx ? I : O;
  const Plan p = plan_for(R, N, dx ? O : I, r);
  return p.pair ? pack_bytes(R, r) + pack_bytes(N, r) : stream_part_bytes(p) + stream_ticket_bytes(p);
}

size_t int8_tc_zeroed(bool dx, int64_t R, int64_t O, int64_t I, int32_t r) {
  if (R == 0) return 0;
  const Plan p = plan_for(R, dx ? I : O, dx ? O : I, r);
  return p.pair ? 0 : stream_part_bytes(p) + stream_ticket_bytes(p);
}

cudaError_t launch_int8_tc(const Int8Call& c, const int8_t* xq, const float* xs, const Int8Few* few, void* ws,
                           uint32_t* hdr, cudaStream_t st) {
  const Plan pl = plan_for(c.R, c.dx ? c.I : c.O, c.dx ? c.O : c.I, c.r);
  Epi e = {};
  e.R = c.R;
  e.N = c.dx ? c.I : c.O;
  e.xs = xs;
  e.ws = c.dx ? nullptr : c.wscale;
  e.T = c.T;
  e.L = c.L;
  e.r = c.r;
  e.s = c.s;
  e.out = c.out;
  e.bf16 = c.bf16 ? 1 : 0;
  e.err = hdr;
  e.wait_ns = kWaitLimitNs;
  return c.dx ? go_rank<true>(pl, c, xq, e, few, ws, st) : go_rank<false>(pl, c, xq, e, few, ws, st);
}

}  // namespace qlora
