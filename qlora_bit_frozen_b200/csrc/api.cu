// api.cu -- the extern "C" entry points of libqlora (declared in qlora.h):
// host-side argument checks, workspace layout and kernel dispatch.
#include <math.h>
#include <string.h>

#include <mutex>
#include <vector>

#include "common.cuh"
#include "int8.h"
#include "internal.h"
#include "smallr.h"
#include "tc_gemm.h"

namespace qlora {

std::atomic<uint64_t> g_launches{0};

// ------------------------------------------------- kernel timing records
namespace {
struct TimingRec {
  cudaEvent_t a, b;
  int kind;
  double flops;
};
std::mutex g_tmu;
std::vector<TimingRec> g_trecs;
int g_tmax = 0;
}  // namespace

// Under stream capture an event record must be an external event node to
// record at every replay of the graph.
static void record_event(cudaEvent_t ev, cudaStream_t st) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusActive)
    cudaEventRecordWithFlags(ev, st, cudaEventRecordExternal);
  else
    cudaEventRecord(ev, st);
}

int timing_begin(cudaStream_t st, int kind, double flops) {
  std::lock_guard<std::mutex> lk(g_tmu);
  if ((int)g_trecs.size() >= g_tmax) return -1;
  TimingRec r;
  if (cudaEventCreate(&r.a) != cudaSuccess) return -1;
  if (cudaEventCreate(&r.b) != cudaSuccess) {
    cudaEventDestroy(r.a);
    return -1;
  }
  r.kind = kind;
  r.flops = flops;
  record_event(r.a, st);
  g_trecs.push_back(r);
  return (int)g_trecs.size() - 1;
}

bool timing_enabled() {
  std::lock_guard<std::mutex> lk(g_tmu);
  return g_tmax > 0;
}

void timing_end(int slot, cudaStream_t st) {
  if (slot < 0) return;
  std::lock_guard<std::mutex> lk(g_tmu);
  if (slot < (int)g_trecs.size()) record_event(g_trecs[slot].b, st);
}

static void timing_clear_locked() {
  for (auto& r : g_trecs) {
    cudaEventDestroy(r.a);
    cudaEventDestroy(r.b);
  }
  g_trecs.clear();
}

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
// Element alignment of fp32 arrays (null counts as aligned).
bool al4(const void* p) { return aligned(p, 4); }

qlora_status cuda_status(cudaError_t e) { return e == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA; }

qlora_status device_ready() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}

// Reads header words 0..2 of a workspace after synchronizing the stream.
qlora_status read_header(const void* ws, cudaStream_t st, uint32_t out[3]) {
  uint32_t h[4] = {0, 0, 0, 0};
  cudaError_t e = cudaMemcpyAsync(h, ws, sizeof(h), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return QLORA_ERR_CUDA;
  out[0] = h[0];
  out[1] = h[1];
  out[2] = h[2];
  return QLORA_OK;
}

// Flags in page-locked host memory that every device can write (one page,
// allocated once): one for each call that is waiting for its kernel.  Null
// where there is no such memory or all are taken.
constexpr int kHostFlags = 64;
std::mutex g_flag_mutex;
uint32_t* g_flags = nullptr;
bool g_flags_tried = false;
uint64_t g_flags_taken = 0;

volatile uint32_t* take_host_flag() {
  std::lock_guard<std::mutex> lk(g_flag_mutex);
  if (!g_flags_tried) {
    g_flags_tried = true;
    void* p = nullptr;
    if (cudaHostAlloc(&p, kHostFlags * 64, cudaHostAllocPortable | cudaHostAllocMapped) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    g_flags = (uint32_t*)p;
  }
  if (!g_flags || ~g_flags_taken == 0) return nullptr;
  const int i = __builtin_ctzll(~g_flags_taken);
  g_flags_taken |= 1ull << i;
  return g_flags + 16 * i;  // a cache line each
}
void give_host_flag(volatile uint32_t* flag) {
  std::lock_guard<std::mutex> lk(g_flag_mutex);
  g_flags_taken &= ~(1ull << (((uint32_t*)flag - g_flags) / 16));
}

int64_t nf4_blocks(int64_t N, int32_t B) { return (N + B - 1) / B; }

qlora_status check_weight(const qlora_weight* w, bool for_linear) {
  if (!w) return QLORA_ERR_INVALID_ARG;
  if (w->O < 0 || w->I < 0 || w->block < 1) return QLORA_ERR_SHAPE;
  if (!weight_count_ok(w->O, w->I)) return QLORA_ERR_SHAPE;
  const int64_t N = w->O * w->I;
  if (w->fmt == QLORA_FMT_NF4_DQ) {
    if (w->bits != 4 || w->group < 1) return QLORA_ERR_SHAPE;
    if (N > 0 && (!w->codes || !w->scale_codes || !w->group_absmax || !w->mean))
      return QLORA_ERR_INVALID_ARG;
    if (!al4(w->group_absmax) || !al4(w->mean)) return QLORA_ERR_ALIGNMENT;
  } else if (w->fmt == QLORA_FMT_NF4_FP32SCALE) {
    if (w->bits != 4) return QLORA_ERR_SHAPE;
    if (N > 0 && (!w->codes || !w->scale)) return QLORA_ERR_INVALID_ARG;
    if (!al4(w->scale)) return QLORA_ERR_ALIGNMENT;
  } else if (w->fmt == QLORA_FMT_AFFINE) {
    if (w->bits != 4 && w->bits != 8) return QLORA_ERR_SHAPE;
    if (N > 0 && (!w->codes || !w->scale || !w->bias)) return QLORA_ERR_INVALID_ARG;
    if (!al4(w->scale) || !al4(w->bias)) return QLORA_ERR_ALIGNMENT;
  } else if (w->fmt == QLORA_FMT_INT8) {
    if (w->bits != 8) return QLORA_ERR_SHAPE;
    if (N > 0 && (!w->codes || !w->scale)) return QLORA_ERR_INVALID_ARG;
    if (!al4(w->scale)) return QLORA_ERR_ALIGNMENT;
    if (for_linear) {
      if (w->O < 1 || w->I < 1) return QLORA_ERR_SHAPE;
      if (w->O > kInt8MaxK || w->I > kInt8MaxK) return QLORA_ERR_UNSUPPORTED;
      if (!aligned(w->codes, 16)) return QLORA_ERR_ALIGNMENT;
    }
    return QLORA_OK;
  } else {
    return QLORA_ERR_INVALID_ARG;
  }
  if (for_linear && w->I % w->block != 0) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

WView view_of(const qlora_weight* w) {
  WView v;
  v.fmt = w->fmt;
  v.O = w->O;
  v.I = w->I;
  v.block = w->block;
  v.group = w->group < 1 ? 1 : w->group;
  v.bits = w->bits;
  v.codes = w->codes;
  v.qcodes = w->scale_codes;
  v.t = w->group_absmax;
  v.mu = w->mean;
  v.scale = w->scale;
  v.bias = w->bias;
  return v;
}

// ---------------------------------------------------------------- layouts

// Every layout starts with the status header and the ticket counters, both
// zeroed by one memset at the start of the call.
constexpr size_t kWsZeroed = kWsHeader + kWsTickets;

struct FwdLayout {
  size_t u = 0, red = 0, split = 0, sr = 0, tc = 0, total = 0;
};
struct BwdLayout {
  size_t u = 0, v = 0, bt = 0, red = 0, red2 = 0, split = 0, split2 = 0, gemv = 0, sr = 0, tc = 0,
         total = 0;
};

FwdLayout fwd_layout(const qlora_weight* w, int64_t R, int32_t r, int32_t compute) {
  FwdLayout L;
  size_t off = kWsZeroed;
  L.u = off;
  off += align_up((size_t)R * r * 4, 256);
  L.red = off;  // split partials of U = X A^T
  off += rowdot_ws(R, w->I, r);
  L.split = off;  // bf16 hi / lo copy of A (above rank 8)
  off += adapter_split_ws(w->I, r);
  L.sr = off;  // split-K partials of the few-token path
  if (compute == QLORA_COMPUTE_BF16) off += smallr_ws(false, view_of(w), R);
  L.tc = off;
  if (compute == QLORA_COMPUTE_BF16) off += tc_fwd_ws(view_of(w), R);
  L.total = off;
  return L;
}

BwdLayout bwd_layout(const qlora_weight* w, int64_t R, int32_t r, int32_t compute) {
  BwdLayout L;
  size_t off = kWsZeroed;
  L.u = off;
  off += align_up((size_t)R * r * 4, 256);
  L.v = off;
  off += align_up((size_t)R * r * 4, 256);
  L.bt = off;  // B^T [r x O] for the pipelined V = dY B
  off += align_up((size_t)r * w->O * 4, 256);
  L.red = off;
  // partials of the four side products, used one after another
  size_t red = coldot_ws(R, w->I, r);
  const size_t more[3] = {coldot_ws(R, w->O, r), rowdot_ws(R, w->O, r), rowdot_ws(R, w->I, r)};
  for (size_t m : more)
    if (m > red) red = m;
  off += red;
  L.split = off;  // bf16 hi / lo copy of B, V, A or U (one at a time)
  size_t sp = adapter_split_ws(w->O, r);
  const size_t sps[2] = {adapter_split_ws(w->I, r), adapter_split_ws(R, r)};
  for (size_t m : sps)
    if (m > sp) sp = m;
  off += sp;
  L.red2 = off;  // dB partials when dA and dB share a launch
  off += coldot_ws(R, w->O, r);
  L.split2 = off;  // bf16 hi / lo copy of U for that launch
  off += adapter_split_ws(R, r);
  L.gemv = off;  // dX partials of the small-R affine path
  off += gemv_dx_ws(view_of(w), R);
  L.sr = off;  // split-K partials of the few-token path
  if (compute == QLORA_COMPUTE_BF16) off += smallr_ws(true, view_of(w), R);
  L.tc = off;
  if (compute == QLORA_COMPUTE_BF16) off += tc_dx_ws(view_of(w), R);
  L.total = off;
  return L;
}

// INT8 weights: the status header (cleared by the first kernel of a call), U and V,
// copies of X and dY that the tensor-core side products need, the parts of the
// factors and of U and V, the products' partial sums, the scratch of the fp32 ones
// (for activations that the others do not take), then the quantized rows and the
// product's own.
struct Int8Layout {
  size_t u = 0, v = 0, cX = 0, cY = 0, fA = 0, fB = 0, fU = 0, fV = 0, part = 0, red = 0, rows = 0, total = 0;
};

Int8Layout int8_layout(const qlora_weight* w, int64_t R, int32_t r, bool bwd, int32_t compute) {
  Int8Layout L;
  size_t off = kWsZeroed;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  L.u = take((size_t)R * r * 4);
  if (bwd) L.v = take((size_t)R * r * 4);
  const bool bf16 = compute == QLORA_COMPUTE_BF16;
  const bool copyX = side_copies(bf16, R, w->I, r), copyY = bwd && side_copies(bf16, R, w->O, r);
  const int parts = bf16 ? 1 : 3;
  if (copyX) L.cX = take(side_copy_bytes(bf16, R, w->I));
  if (copyY) L.cY = take(side_copy_bytes(bf16, R, w->O));
  if (bf16 || copyX) {
    L.fA = take(side_parts_bytes(copyX ? parts * side_ld(w->I) : w->I, r));
    if (bwd) L.fV = take(side_parts_bytes(copyX ? parts * R : R, r));
  }
  if (bwd && (bf16 || copyY)) {
    L.fB = take(side_parts_bytes(copyY ? parts * side_ld(w->O) : w->O, r));
    L.fU = take(side_parts_bytes(copyY ? parts * R : R, r));
  }
  if (bf16 || copyX || copyY) L.part = take(side_part_ws(r));
  if (bwd) {
    const size_t a = coldot_ws(R, w->I, r), b = coldot_ws(R, w->O, r);
    L.red = take(a > b ? a : b);
  }
  L.rows = take(int8_ws(bwd, R, w->O, w->I, r));
  L.total = off;
  return L;
}

Int8Call int8_call(const qlora_weight* w, bool dx, bool bf16, int64_t R, const void* P, const float* T,
                   const float* L, int32_t r, float s, void* out) {
  Int8Call c;
  c.dx = dx;
  c.bf16 = bf16;
  c.R = R;
  c.O = w->O;
  c.I = w->I;
  c.codes = (const int8_t*)w->codes;
  c.wscale = w->scale;
  c.P = P;
  c.T = T;
  c.L = L;
  c.r = r;
  c.s = s;
  c.out = out;
  return c;
}

cudaError_t int8_fwd(const qlora_weight* w, const void* X, int64_t R, const float* A, const float* B,
                     int32_t r, float sc, int32_t compute, void* Y, float* U_out, void* ws, cudaStream_t s) {
  const bool bf16 = compute == QLORA_COMPUTE_BF16;
  const Int8Layout L = int8_layout(w, R, r, false, compute);
  auto at = [&](size_t off) { return (char*)ws + off; };
  float* U = U_out ? U_out : (float*)at(L.u);
  const Int8Call c = int8_call(w, false, bf16, R, X, U, B, r, sc, Y);
  const Int8Clear header = {ws, kWsZeroed};
  cudaError_t e;
  if (int8_few_applies(R, w->I, r)) {
    Int8Few f = {};
    f.F = A;
    f.T = U;
    e = launch_int8_few(c, f, at(L.rows), header, s);
  } else {
    e = launch_int8_rows(c, at(L.rows), header, s);
    const SideMatrix m = side_matrix(X, bf16, R, w->I, r, at(L.cX));
    if (e == cudaSuccess && m.parts) {
      uint16_t* fA = (uint16_t*)at(L.fA);
      const SideFactor f = side_factor_of_columns(A, fA, false, m);
      const SideProduct p = {m, fA, U, nullptr, false, 1.0f};
      const SideCopy copy = {X, m};
      e = launch_side_copy(&copy, m.P != X, bf16, R, s);
      if (e == cudaSuccess) e = launch_side_split(&f, 1, r, s);
      if (e == cudaSuccess)
        e = launch_side(&p, 1, false, R, r, at(L.part), (uint32_t*)ws, s);
    } else if (e == cudaSuccess) {
      const Int8Dot d = {X, A, U, w->I, false};
      e = launch_int8_dots(&d, 1, bf16, R, r, s);
    }
  }
  if (e == cudaSuccess) e = launch_int8_product(c, at(L.rows), (uint32_t*)ws, nullptr, s);
  return e;
}

cudaError_t int8_bwd(const qlora_weight* w, const void* X, const void* dY, int64_t R, const float* A,
                     const float* B, int32_t r, float sc, const float* U_in, int32_t compute, void* dX,
                     float* dA, float* dB, void* ws, cudaStream_t s) {
  const bool bf16 = compute == QLORA_COMPUTE_BF16;
  const Int8Layout L = int8_layout(w, R, r, true, compute);
  auto at = [&](size_t off) { return (char*)ws + off; };
  float* V = (float*)at(L.v);
  float* Uw = (float*)at(L.u);
  const float* U = U_in ? U_in : Uw;
  uint16_t *fA = (uint16_t*)at(L.fA), *fB = (uint16_t*)at(L.fB), *fU = (uint16_t*)at(L.fU),
           *fV = (uint16_t*)at(L.fV);
  const Int8Clear header = {ws, kWsZeroed};
  const Int8Call c = int8_call(w, true, bf16, R, dY, V, A, r, sc, dX);
  const bool want_v = dX || dA, new_u = dB && !U_in;
  // what the tensor-core side products take (else the fp32 ones do)
  const SideMatrix mX = side_matrix(X, bf16, R, w->I, r, at(L.cX)), mY = side_matrix(dY, bf16, R, w->O, r, at(L.cY));
  const bool sX = mX.parts != 0, sY = mY.parts != 0;
  // dA = s V^T X, dB = s dY^T U: from the parts of V and U, or from V and U
  auto columns = [&]() {
    SideProduct p[2];
    int n = 0;
    if (dA && sX) p[n++] = {mX, fV, dA, nullptr, true, sc};
    if (dB && sY) p[n++] = {mY, fU, dB, nullptr, false, sc};
    cudaError_t e = cudaSuccess;
    if (n) e = launch_side(p, n, true, R, r, at(L.part), (uint32_t*)ws, s);
    if (e == cudaSuccess && dA && !sX) e = launch_coldot(X, bf16, R, w->I, V, r, sc, false, dA, at(L.red), s);
    if (e == cudaSuccess && dB && !sY) e = launch_coldot(dY, bf16, R, w->O, U, r, sc, true, dB, at(L.red), s);
    return e;
  };
  cudaError_t e;
  if (R == 0) {
    e = cudaMemsetAsync(ws, 0, kWsZeroed, s);
    return e != cudaSuccess ? e : columns();  // zeros
  }
  if (int8_few_applies(R, w->O, r) && int8_few_applies(R, w->I, r)) {
    // the rows, V and U in one launch; dA and dB beside the products, or, for
    // more tokens, by themselves (the same kernels whichever gradients are
    // wanted: each has the same bits)
    const bool beside = R <= kInt8Few;
    Int8Few f = {};
    f.F = B;
    f.T = want_v ? V : nullptr;
    f.X = X;
    f.A = A;
    f.U_new = new_u ? Uw : nullptr;
    f.U = U;
    if (beside) {
      f.dA = dA;
      f.dB = dB;
    } else {
      f.T_parts = dA && sX ? fV : nullptr;
      f.U_parts = dB && sY ? fU : nullptr;
      f.NP = side_np(r);
      f.ld = side_ld(R);
    }
    e = launch_int8_few(c, f, at(L.rows), header, s);
    if (e == cudaSuccess && !beside) e = columns();
    if (e == cudaSuccess && (dX || (beside && (dA || dB))))
      e = launch_int8_product(c, at(L.rows), (uint32_t*)ws, &f, s);
    return e;
  }
  e = dX ? launch_int8_rows(c, at(L.rows), header, s) : cudaMemsetAsync(ws, 0, kWsZeroed, s);
  // the copies, the parts of the factors, then V and U (with their own parts where
  // a tensor-core product makes them as they are wanted, else split after it)
  SideCopy copy[2];
  SideFactor f[2], late[2];
  SideProduct p[2];
  int nc = 0, nf = 0, np = 0, nlate = 0;
  const bool parts_v = dA && sX, parts_u = dB && sY;
  if (sX && mX.P != X && (dA || new_u)) copy[nc++] = {X, mX};
  if (sY && mY.P != dY && (dB || want_v)) copy[nc++] = {dY, mY};
  const bool own_v = parts_v && want_v && sY && mX.parts == 1, own_u = parts_u && new_u && sX && mY.parts == 1;
  if (want_v && sY) {
    f[nf++] = side_factor_of_columns(B, fB, true, mY);
    p[np++] = {mY, fB, V, own_v ? fV : nullptr, false, 1.0f};
  }
  if (parts_v && !own_v) late[nlate++] = side_factor_of_rows(V, fV, R, mX);
  if (new_u && sX) {
    f[nf++] = side_factor_of_columns(A, fA, false, mX);
    p[np++] = {mX, fA, Uw, own_u ? fU : nullptr, false, 1.0f};
  }
  if (parts_u && !own_u) {
    if (new_u || nf == 2) late[nlate++] = side_factor_of_rows(U, fU, R, mY);
    else f[nf++] = side_factor_of_rows(U, fU, R, mY);
  }
  if (e == cudaSuccess) e = launch_side_copy(copy, nc, bf16, R, s);
  if (e == cudaSuccess) e = launch_side_split(f, nf, r, s);
  if (e == cudaSuccess && np) e = launch_side(p, np, false, R, r, at(L.part), (uint32_t*)ws, s);
  Int8Dot d[2];
  int nd = 0;
  if (want_v && !sY) d[nd++] = {dY, B, V, w->O, true};
  if (new_u && !sX) d[nd++] = {X, A, Uw, w->I, false};
  if (e == cudaSuccess && nd) e = launch_int8_dots(d, nd, bf16, R, r, s);
  if (e == cudaSuccess) e = launch_side_split(late, nlate, r, s);
  if (e == cudaSuccess) e = columns();
  if (e == cudaSuccess && dX) e = launch_int8_product(c, at(L.rows), (uint32_t*)ws, nullptr, s);
  return e;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

const char* qlora_status_string(qlora_status st) {
  switch (st) {
    case QLORA_OK: return "ok";
    case QLORA_ERR_INVALID_ARG: return "invalid argument";
    case QLORA_ERR_SHAPE: return "inconsistent shape";
    case QLORA_ERR_ALIGNMENT: return "misaligned pointer or workspace";
    case QLORA_ERR_NONFINITE: return "non-finite weight";
    case QLORA_ERR_UNSUPPORTED: return "unsupported configuration";
    case QLORA_ERR_CUDA: return "CUDA runtime error";
    case QLORA_ERR_TIMEOUT: return "bounded device wait ran out";
    case QLORA_ERR_WORKSPACE: return "workspace too small";
  }
  return "unknown status";
}

qlora_status qlora_nf4_codebook(float out[16]) {
  if (!out) return QLORA_ERR_INVALID_ARG;
  memcpy(out, kNF4Host, sizeof(kNF4Host));
  return QLORA_OK;
}

size_t qlora_nf4_payload_bytes(int64_t N, int32_t B, int32_t C) {
  if (N < 0 || B < 1 || C < 1) return 0;
  const int64_t M = nf4_blocks(N, B);
  const int64_t S = (M + C - 1) / C;
  return (size_t)((N + 1) / 2 + M + 4 * S + 4);
}

size_t qlora_quantize_nf4_workspace_bytes(int64_t N, int32_t B, int32_t C) {
  if (N < 0 || N > kMaxWeights || B < 1 || C < 1) return 0;
  return nf4_quantize_ws(N, B, C);
}

qlora_status qlora_quantize_nf4(const float* W, int64_t O, int64_t I, int32_t B, int32_t C,
                                uint8_t* codes, uint8_t* scale_codes, float* t, float* mu,
                                void* ws, size_t ws_bytes, qlora_stream_t stream) {
  if (O < 0 || I < 0 || B < 1 || C < 1) return QLORA_ERR_SHAPE;
  if (!weight_count_ok(O, I)) return QLORA_ERR_SHAPE;
  const int64_t N = O * I;
  if (!mu || !ws) return QLORA_ERR_INVALID_ARG;
  if (N > 0 && (!W || !codes || !scale_codes || !t)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !al4(W) || !al4(t) || !al4(mu)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < nf4_quantize_ws(N, B, C)) return QLORA_ERR_WORKSPACE;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  st = cuda_status(launch_nf4_quantize(W, N, B, C, codes, scale_codes, t, mu, ws, s));
  if (st != QLORA_OK) return st;
  uint32_t h[3];
  st = read_header(ws, s, h);
  if (st != QLORA_OK) return st;
  if (h[2]) return QLORA_ERR_NONFINITE;
  return h[0] ? (qlora_status)h[0] : QLORA_OK;
}

size_t qlora_nf4_fp32scale_payload_bytes(int64_t N, int32_t B) {
  if (N < 0 || N > kMaxWeights || B < 1) return 0;
  return (size_t)((N + 1) / 2) + 4 * (size_t)((N + B - 1) / B);
}

size_t qlora_quantize_nf4_fp32scale_workspace_bytes(int64_t N, int32_t B) {
  if (N < 0 || N > kMaxWeights || B < 1) return 0;
  return kWsHeader;
}

qlora_status qlora_quantize_nf4_fp32scale(const float* W, int64_t O, int64_t I, int32_t B,
                                          uint8_t* codes, float* scale, void* ws, size_t ws_bytes,
                                          qlora_stream_t stream) {
  if (O < 0 || I < 0 || B < 1) return QLORA_ERR_SHAPE;
  if (!weight_count_ok(O, I)) return QLORA_ERR_SHAPE;
  const int64_t N = O * I;
  if (!ws) return QLORA_ERR_INVALID_ARG;
  if (N > 0 && (!W || !codes || !scale)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !al4(W) || !al4(scale)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < kWsHeader) return QLORA_ERR_WORKSPACE;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  st = cuda_status(launch_nf4_fp32scale_quantize(W, N, B, codes, scale, ws, s));
  if (st != QLORA_OK) return st;
  uint32_t h[3];
  st = read_header(ws, s, h);
  if (st != QLORA_OK) return st;
  if (h[2]) return QLORA_ERR_NONFINITE;
  return h[0] ? (qlora_status)h[0] : QLORA_OK;
}

size_t qlora_quantize_affine_workspace_bytes(int64_t N, int32_t bits, int32_t G) {
  (void)N;
  (void)bits;
  (void)G;
  return kWsHeader;
}

qlora_status qlora_quantize_affine(const float* W, int64_t O, int64_t I, int32_t bits, int32_t G,
                                   uint8_t* codes, float* scale, float* bias, void* ws,
                                   size_t ws_bytes, qlora_stream_t stream) {
  if (O < 0 || I < 0 || G < 1) return QLORA_ERR_SHAPE;
  if (bits != 4 && bits != 8) return QLORA_ERR_SHAPE;
  if (!weight_count_ok(O, I)) return QLORA_ERR_SHAPE;
  const int64_t N = O * I;
  if (!ws) return QLORA_ERR_INVALID_ARG;
  if (N > 0 && (!W || !codes || !scale || !bias)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !al4(W) || !al4(scale) || !al4(bias)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < kWsHeader) return QLORA_ERR_WORKSPACE;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  st = cuda_status(launch_affine_quantize(W, N, bits, G, codes, scale, bias, ws, s));
  if (st != QLORA_OK) return st;
  uint32_t h[3];
  st = read_header(ws, s, h);
  if (st != QLORA_OK) return st;
  if (h[2]) return QLORA_ERR_NONFINITE;
  return h[0] ? (qlora_status)h[0] : QLORA_OK;
}

int64_t qlora_int8_pitch(int64_t I) {
  return I < 0 || I > kMaxWeights ? 0 : int8_pitch(I);
}

size_t qlora_quantize_int8_workspace_bytes(int64_t O, int64_t I) {
  return weight_count_ok(O, I) ? kWsHeader : 0;
}

qlora_status qlora_quantize_int8(const float* W, int64_t O, int64_t I, int8_t* codes, float* scale,
                                 void* ws, size_t ws_bytes, qlora_stream_t stream) {
  if (O < 0 || I < 0 || O > 0x7fffffffLL) return QLORA_ERR_SHAPE;
  if (!weight_count_ok(O, I)) return QLORA_ERR_SHAPE;
  if (!ws) return QLORA_ERR_INVALID_ARG;
  if (O > 0 && (!scale || (I > 0 && (!W || !codes)))) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !al4(W) || !al4(scale)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < kWsHeader) return QLORA_ERR_WORKSPACE;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (volatile uint32_t* flag = take_host_flag()) {
    // the kernel writes the flag straight into host memory: no clearing and no
    // copy back around it
    *flag = 0;
    st = cuda_status(launch_int8_quantize(W, O, I, codes, scale, (uint32_t*)flag, s));
    // (also after an error: nothing may write to the flag once it is given back)
    if (cudaStreamSynchronize(s) != cudaSuccess) st = QLORA_ERR_CUDA;
    const bool bad = *flag != 0;
    give_host_flag(flag);
    return st != QLORA_OK ? st : bad ? QLORA_ERR_NONFINITE : QLORA_OK;
  }
  if (cudaMemsetAsync(ws, 0, kWsHeader, s) != cudaSuccess) return QLORA_ERR_CUDA;
  st = cuda_status(launch_int8_quantize(W, O, I, codes, scale, (uint32_t*)ws + 2, s));
  if (st != QLORA_OK) return st;
  uint32_t h[3];
  st = read_header(ws, s, h);
  if (st != QLORA_OK) return st;
  if (h[2]) return QLORA_ERR_NONFINITE;
  return h[0] ? (qlora_status)h[0] : QLORA_OK;
}

qlora_status qlora_dequantize(const qlora_weight* w, float* W_hat, qlora_stream_t stream) {
  qlora_status st = check_weight(w, false);
  if (st != QLORA_OK) return st;
  if (w->O * w->I > 0 && !W_hat) return QLORA_ERR_INVALID_ARG;
  if (!al4(W_hat)) return QLORA_ERR_ALIGNMENT;
  st = device_ready();
  if (st != QLORA_OK) return st;
  if (w->fmt == QLORA_FMT_INT8)
    return cuda_status(launch_int8_dequantize((const int8_t*)w->codes, w->scale, w->O, w->I, W_hat,
                                              (cudaStream_t)stream));
  return cuda_status(launch_dequantize(view_of(w), W_hat, (cudaStream_t)stream));
}

qlora_status qlora_merge(const qlora_weight* w, const float* A, const float* B, int32_t r,
                         float alpha, float* W_out, qlora_stream_t stream) {
  qlora_status st = check_weight(w, false);
  if (st != QLORA_OK) return st;
  if (r < 1) return QLORA_ERR_SHAPE;
  if (w->O * w->I > 0 && (!A || !B || !W_out)) return QLORA_ERR_INVALID_ARG;
  if (!al4(A) || !al4(B) || !al4(W_out)) return QLORA_ERR_ALIGNMENT;
  st = device_ready();
  if (st != QLORA_OK) return st;
  const float s = alpha / (float)r;
  return cuda_status(launch_merge(view_of(w), A, B, r, s, W_out, (cudaStream_t)stream));
}

qlora_status qlora_adam_step(float* params, const float* grads, float* m, float* v, int64_t n,
                             int64_t t, float lr, float beta1, float beta2, float eps,
                             int64_t page_elems, qlora_stream_t stream) {
  if (n < 0 || t < 1 || page_elems < 0) return QLORA_ERR_SHAPE;
  if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f))
    return QLORA_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps) || !isfinite(lr)) return QLORA_ERR_INVALID_ARG;
  if (n == 0) return QLORA_OK;
  if (!params || !grads || !m || !v) return QLORA_ERR_INVALID_ARG;
  if (!al4(params) || !al4(grads) || !al4(m) || !al4(v)) return QLORA_ERR_ALIGNMENT;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  return cuda_status(launch_adam(params, grads, m, v, n, t, lr, beta1, beta2, eps, page_elems,
                                 (cudaStream_t)stream));
}

// Shared checks of the many-tensor calls; `step`: the AdamW step's arrays too.
static qlora_status check_tensors(const qlora_tensor* t, int32_t count, bool step, int32_t bits) {
  if (count < 0) return QLORA_ERR_SHAPE;
  if (count > 0 && !t) return QLORA_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    const qlora_tensor& d = t[i];
    if (d.n < 0 || d.n > kMaxTensor) return QLORA_ERR_SHAPE;
    if (d.grad_type != QLORA_DTYPE_FP32 && d.grad_type != QLORA_DTYPE_BF16) return QLORA_ERR_INVALID_ARG;
    if (step && d.param_type != QLORA_DTYPE_FP32 && d.param_type != QLORA_DTYPE_BF16)
      return QLORA_ERR_INVALID_ARG;
    if (d.n == 0) continue;
    if (!d.grad || (step && (!d.param || !d.m || !d.v))) return QLORA_ERR_INVALID_ARG;
    if (step && bits == 8 && (!d.m_scale || !d.v_scale)) return QLORA_ERR_INVALID_ARG;
    if (!aligned(d.grad, d.grad_type == QLORA_DTYPE_BF16 ? 2 : 4)) return QLORA_ERR_ALIGNMENT;
    if (step && !aligned(d.param, d.param_type == QLORA_DTYPE_BF16 ? 2 : 4)) return QLORA_ERR_ALIGNMENT;
    if (step && bits == 32 && (!al4(d.m) || !al4(d.v))) return QLORA_ERR_ALIGNMENT;
    if (step && bits == 8 && (!al4(d.m_scale) || !al4(d.v_scale))) return QLORA_ERR_ALIGNMENT;
  }
  return QLORA_OK;
}

size_t qlora_grad_norm_workspace_bytes(const qlora_tensor* tensors, int32_t count) {
  if (check_tensors(tensors, count, false, 32) != QLORA_OK) return 0;
  return grad_norm_ws(tensors, count);
}

qlora_status qlora_grad_norm(const qlora_tensor* tensors, int32_t count, float max_norm,
                             qlora_step_control* control, void* ws, size_t ws_bytes,
                             qlora_stream_t stream) {
  qlora_status st = check_tensors(tensors, count, false, 32);
  if (st != QLORA_OK) return st;
  if (!isfinite(max_norm) || !control || !ws) return QLORA_ERR_INVALID_ARG;
  if (!al4(control) || !aligned(ws, 256)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < grad_norm_ws(tensors, count)) return QLORA_ERR_WORKSPACE;
  st = device_ready();
  if (st != QLORA_OK) return st;
  return cuda_status(launch_grad_norm(tensors, count, max_norm, control, ws, (cudaStream_t)stream));
}

qlora_status qlora_adamw_step(const qlora_tensor* tensors, int32_t count, int32_t state_bits, int64_t t,
                              float lr, float beta1, float beta2, float eps, float weight_decay,
                              const qlora_step_control* control, qlora_stream_t stream) {
  if (state_bits != 8 && state_bits != 32) return QLORA_ERR_INVALID_ARG;
  qlora_status st = check_tensors(tensors, count, true, state_bits);
  if (st != QLORA_OK) return st;
  if (!control && t < 1) return QLORA_ERR_SHAPE;
  if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f))
    return QLORA_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps) || !isfinite(lr)) return QLORA_ERR_INVALID_ARG;
  if (!(weight_decay >= 0.0f) || !isfinite(weight_decay)) return QLORA_ERR_INVALID_ARG;
  if (!al4(control)) return QLORA_ERR_ALIGNMENT;
  st = device_ready();
  if (st != QLORA_OK) return st;
  return cuda_status(launch_adamw(tensors, count, state_bits, t, lr, beta1, beta2, eps, weight_decay,
                                  control, (cudaStream_t)stream));
}

size_t qlora_linear_workspace_bytes(const qlora_weight* w, int64_t R, int32_t r, int32_t op,
                                    int32_t compute) {
  if (!w || R < 0 || r < 1 || r > 64) return 0;
  if (compute != QLORA_COMPUTE_FP32 && compute != QLORA_COMPUTE_BF16) return 0;
  if (w->fmt == QLORA_FMT_INT8) {
    if (w->O < 1 || w->I < 1 || w->O > kInt8MaxK || w->I > kInt8MaxK || R > kInt8MaxTokens) return 0;
    if (op != QLORA_OP_FWD && op != QLORA_OP_BWD) return 0;
    return int8_layout(w, R, r, op == QLORA_OP_BWD, compute).total;
  }
  if (op == QLORA_OP_FWD) return fwd_layout(w, R, r, compute).total;
  if (op == QLORA_OP_BWD) return bwd_layout(w, R, r, compute).total;
  return 0;
}

static qlora_status check_linear_common(const qlora_weight* w, int64_t R, const float* A,
                                        const float* B, int32_t r, int32_t compute, void* ws) {
  qlora_status st = check_weight(w, true);
  if (st != QLORA_OK) return st;
  if (R < 0) return QLORA_ERR_SHAPE;
  if (r < 1) return QLORA_ERR_SHAPE;
  if (r > 64) return QLORA_ERR_UNSUPPORTED;
  if (compute != QLORA_COMPUTE_FP32 && compute != QLORA_COMPUTE_BF16) return QLORA_ERR_INVALID_ARG;
  if (!A || !B || !ws) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !al4(A) || !al4(B)) return QLORA_ERR_ALIGNMENT;
  return QLORA_OK;
}

qlora_status qlora_linear_fwd(const qlora_weight* w, const void* X, int64_t R, const float* A,
                              const float* B, int32_t r, float alpha, int32_t compute, void* Y,
                              float* U_out, void* ws, size_t ws_bytes, qlora_stream_t stream) {
  qlora_status st = check_linear_common(w, R, A, B, r, compute, ws);
  if (st != QLORA_OK) return st;
  if (R > 0 && (!X || !Y)) return QLORA_ERR_INVALID_ARG;
  const size_t esz = compute == QLORA_COMPUTE_BF16 ? 2 : 4;
  if (!aligned(X, esz) || !aligned(Y, esz) || !al4(U_out)) return QLORA_ERR_ALIGNMENT;
  const bool int8 = w->fmt == QLORA_FMT_INT8;
  if (int8 && R > kInt8MaxTokens) return QLORA_ERR_SHAPE;
  const FwdLayout L = int8 ? FwdLayout() : fwd_layout(w, R, r, compute);
  if (ws_bytes < (int8 ? int8_layout(w, R, r, false, compute).total : L.total)) return QLORA_ERR_WORKSPACE;
  st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const float sc = alpha / (float)r;
  if (int8 && R > 0)
    return cuda_status(
        int8_fwd(w, X, R, A, B, r, sc, compute, Y, U_out, ws, s));
  cudaError_t e = cudaMemsetAsync(ws, 0, kWsZeroed, s);
  if (e != cudaSuccess) return QLORA_ERR_CUDA;
  if (R == 0) return QLORA_OK;
  unsigned* tickets = (unsigned*)((char*)ws + kWsHeader);
  float* red = (float*)((char*)ws + L.red);
  float* U = U_out ? U_out : (float*)((char*)ws + L.u);
  const WView v = view_of(w);
  const bool bf16 = compute == QLORA_COMPUTE_BF16;
  // bf16: the few-token kernels where they are measured faster (or the only
  // fast path), else the tensor-core kernel, else the SIMT tiles
  const bool fwd_tc = bf16 && tc_fwd_supported(v, X, Y, R);
  const bool fwd_sr = bf16 && smallr_supported(v, R, X, Y) && (!fwd_tc || smallr_preferred(false, v, R));
  if (fwd_sr) {
    // 1..16 tokens: U = X A^T, then the bandwidth-bound GEMV, which starts
    // its weight stream at once and waits for U only in its epilogue
    e = launch_rowdot(X, true, R, w->I, A, false, r, U, s, nullptr, nullptr, 0, 0, 1.0f, nullptr,
                      nullptr, red, tickets, (uint16_t*)((char*)ws + L.split));
    if (e == cudaSuccess)
      e = launch_smallr_fwd(v, X, R, U, B, r, sc, Y, (char*)ws + L.sr, (uint32_t*)ws, tickets, s);
  } else if (fwd_tc) {
    void* tcws = (char*)ws + L.tc;
    e = tc_prepare(false, v, R, tcws, s);
    if (e == cudaSuccess)
      e = launch_rowdot(X, true, R, w->I, A, false, r, U, s, tc_act_pad(tcws), B, w->O, 0, sc,
                      tc_w_pad(tcws, R), nullptr, red, tickets, (uint16_t*)((char*)ws + L.split));
    if (e == cudaSuccess) e = launch_tc_fwd(v, X, R, U, B, r, sc, Y, tcws, (uint32_t*)ws, s);
  } else {
    e = launch_simt_fwd(v, X, R, A, B, r, sc, bf16, Y, U, s);
  }
  return cuda_status(e);
}

qlora_status qlora_linear_bwd(const qlora_weight* w, const void* X, const void* dY, int64_t R,
                              const float* A, const float* B, int32_t r, float alpha,
                              const float* U_in, int32_t compute, void* dX, float* dA, float* dB,
                              void* ws, size_t ws_bytes, qlora_stream_t stream) {
  qlora_status st = check_linear_common(w, R, A, B, r, compute, ws);
  if (st != QLORA_OK) return st;
  if (R > 0 && !dY) return QLORA_ERR_INVALID_ARG;
  if (R > 0 && (dA || (dB && !U_in)) && !X) return QLORA_ERR_INVALID_ARG;
  const size_t esz = compute == QLORA_COMPUTE_BF16 ? 2 : 4;
  if (!aligned(X, esz) || !aligned(dY, esz) || !aligned(dX, esz) || !al4(U_in) || !al4(dA) ||
      !al4(dB))
    return QLORA_ERR_ALIGNMENT;
  const bool int8 = w->fmt == QLORA_FMT_INT8;
  if (int8 && R > kInt8MaxTokens) return QLORA_ERR_SHAPE;
  const BwdLayout L = int8 ? BwdLayout() : bwd_layout(w, R, r, compute);
  if (ws_bytes < (int8 ? int8_layout(w, R, r, true, compute).total : L.total)) return QLORA_ERR_WORKSPACE;
  st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf16 = compute == QLORA_COMPUTE_BF16;
  const float sc = alpha / (float)r;
  if (int8)
    return cuda_status(int8_bwd(w, X, dY, R, A, B, r, sc, U_in, compute, dX, dA, dB, ws, s));
  cudaError_t e = cudaMemsetAsync(ws, 0, kWsZeroed, s);
  if (e != cudaSuccess) return QLORA_ERR_CUDA;
  unsigned* tickets = (unsigned*)((char*)ws + kWsHeader);
  const WView v = view_of(w);
  float* V = (float*)((char*)ws + L.v);
  void* red = (char*)ws + L.red;
  // V = dY B  (B is [O x r]: L(k = o, j) = B[o*r + j]); its padded bf16 copy
  // feeds the tensor-core kernel's adapter step
  const bool dx_tc = dX && bf16 && tc_dx_supported(v, dY, dX, R);
  const bool sr = dX && bf16 && smallr_supported(v, R, dY, dX) && (!dx_tc || smallr_preferred(true, v, R));
  const bool tc = !sr && dx_tc;
  void* tcws = (char*)ws + L.tc;
  if (tc) e = tc_prepare(true, v, R, tcws, s);
  if (e == cudaSuccess && (dX || dA)) {
    float* bt = (float*)((char*)ws + L.bt);
    float* part = (float*)red;
    uint16_t* split = (uint16_t*)((char*)ws + L.split);
    if (tc)
      e = launch_rowdot(dY, bf16, R, w->O, B, true, r, V, s, tc_act_pad(tcws), A, w->I, 1, sc,
                        tc_w_pad(tcws, R), bt, part, tickets, split);
    else
      e = launch_rowdot(dY, bf16, R, w->O, B, true, r, V, s, nullptr, nullptr, 0, 0, 1.0f,
                        nullptr, bt, part, tickets, split);
  }
  // dA = s V^T X [r x I] and dB = s dY^T U [O x r]: one launch when both
  // are wanted (two independent side products), else one each.
  uint16_t* split = (uint16_t*)((char*)ws + L.split);
  const float* U = U_in;
  if (e == cudaSuccess && dB && !U) {
    float* Uw = (float*)((char*)ws + L.u);
    e = launch_rowdot(X, bf16, R, w->I, A, false, r, Uw, s, nullptr, nullptr, 0, 0, 1.0f,
                      nullptr, nullptr, (float*)red, tickets, split);
    U = Uw;
  }
  bool paired = false;
  if (e == cudaSuccess && dA && dB && bf16)
    e = launch_coldot_pair(X, w->I, V, false, dA, red, split, dY, w->O, U, true, dB,
                           (char*)ws + L.red2, (uint16_t*)((char*)ws + L.split2), R, r, sc, s,
                           tickets, &paired);
  if (e == cudaSuccess && dA && !paired)
    e = launch_coldot(X, bf16, R, w->I, V, r, sc, false, dA, red, s, tickets, split);
  if (e == cudaSuccess && dB && !paired)
    e = launch_coldot(dY, bf16, R, w->O, U, r, sc, true, dB, red, s, tickets, split);
  // dX last: the tensor-core kernel starts behind the side products
  // (programmatic dependent launch) and waits for them only before its
  // adapter step, which reads the padded V written above.
  if (e == cudaSuccess && dX) {
    if (sr)
      e = launch_smallr_dx(v, dY, R, V, A, r, sc, dX, (char*)ws + L.sr, (uint32_t*)ws, tickets, s);
    else if (tc)
      e = launch_tc_dx(v, dY, R, V, A, r, sc, dX, tcws, (uint32_t*)ws, s);
    else
      e = launch_simt_dx(v, dY, R, A, V, r, sc, bf16, dX, s, (float*)((char*)ws + L.gemv));
  }
  return cuda_status(e);
}

qlora_status qlora_workspace_status(const void* ws, qlora_stream_t stream) {
  if (!ws) return QLORA_ERR_INVALID_ARG;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  uint32_t h[3];
  st = read_header(ws, (cudaStream_t)stream, h);
  if (st != QLORA_OK) return st;
  return h[0] ? (qlora_status)h[0] : QLORA_OK;
}

qlora_status qlora_selftest_wait_timeout(void* ws, size_t ws_bytes, uint32_t limit_us,
                                         qlora_stream_t stream) {
  if (!ws) return QLORA_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return QLORA_ERR_ALIGNMENT;
  if (ws_bytes < kWsHeader) return QLORA_ERR_WORKSPACE;
  if (limit_us < 1 || limit_us > 1000000) return QLORA_ERR_INVALID_ARG;
  qlora_status st = device_ready();
  if (st != QLORA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (cudaMemsetAsync(ws, 0, kWsHeader, s) != cudaSuccess) return QLORA_ERR_CUDA;
  st = cuda_status(launch_wait_selftest((uint32_t*)ws, (uint64_t)limit_us * 1000ull, s));
  if (st != QLORA_OK) return st;
  return qlora_workspace_status(ws, stream);
}

uint64_t qlora_kernel_launch_count(void) { return g_launches.load(); }

qlora_status qlora_kernel_timing_enable(int32_t max_records) {
  if (max_records < 0) return QLORA_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lk(g_tmu);
  timing_clear_locked();
  g_tmax = max_records;
  return QLORA_OK;
}

int32_t qlora_kernel_timing_collect(float* ms, int32_t* kind, double* flops, int32_t max) {
  std::lock_guard<std::mutex> lk(g_tmu);
  int32_t n = 0;
  for (auto& r : g_trecs) {
    if (n >= max) break;
    if (cudaEventSynchronize(r.b) != cudaSuccess) return -1;
    float t = 0.0f;
    if (cudaEventElapsedTime(&t, r.a, r.b) != cudaSuccess) return -1;
    if (ms) ms[n] = t;
    if (kind) kind[n] = r.kind;
    if (flops) flops[n] = r.flops;
    ++n;
  }
  return n;
}

}  // extern "C"
