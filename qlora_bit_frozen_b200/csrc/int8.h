// int8.h -- host interface of the 8-bit integer linear kernels (int8.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qlora.h"

namespace qlora {

// Longest reduction whose 32-bit sum cannot overflow: 127^2 * 2^17 < 2^31.
constexpr int64_t kInt8MaxK = 131072;

// Most tokens of a call: counts of CTAs and token coordinates stay in 32 bits.
constexpr int64_t kInt8MaxTokens = 1 << 28;

constexpr int64_t int8_pitch(int64_t n) { return (n + 15) / 16 * 16; }
// Of the activations' codes, which only these kernels see: above 1024 columns
// the rows lie on 128 bytes, since a 128-byte box row that straddles two lines
// costs L2 two requests (9421 tokens of 2048 x 6992: 110 us, so 88).
constexpr int64_t int8_act_pitch(int64_t n) { return n > 1024 ? (n + 127) / 128 * 128 : int8_pitch(n); }

// codes [O x pitch], scale [O] of W [O x I]; *bad (device or mapped host
// memory) is set where W holds a NaN or Inf.
cudaError_t launch_int8_quantize(const float* W, int64_t O, int64_t I, int8_t* codes, float* scale,
                                 uint32_t* bad, cudaStream_t st);
cudaError_t launch_int8_dequantize(const int8_t* codes, const float* scale, int64_t O, int64_t I,
                                   float* out, cudaStream_t st);

// The base product of one call: `rows` activation rows over `K`, `N` outputs.
// Forward (dx false): K = I, N = O, row factor scale s_x, column factor
// scale_o, adapter rows L = B [N x r].  Input gradient: K = O, N = I, scale_o
// folded into the rows before they are quantized, adapter L = A [r x N].
struct Int8Call {
  bool dx;
  bool bf16;             // type of the activations and of the output
  int64_t R, O, I;
  const int8_t* codes;   // [O x int8_pitch(I)]
  const float* wscale;   // [O]
  const void* P;         // activations [R x K]
  const float* T;        // U or V [R x r]
  const float* L;        // B [O x r] or A [r x I]
  int32_t r;
  float s;
  void* out;             // [R x N], nullable in the input gradient: nothing is multiplied
};
size_t int8_ws(bool dx, int64_t R, int64_t O, int64_t I, int32_t r);

// Memory that the first kernel of a call clears for the ones after it.
struct Int8Clear {
  void* p;        // 16-byte aligned
  size_t bytes;   // a multiple of 16
};
// Quantizes the activation rows into the workspace ws (int8_ws bytes), clears
// `header` and what the product adds up in.
cudaError_t launch_int8_rows(const Int8Call& c, void* ws, Int8Clear header, cudaStream_t st);
// Few tokens: one launch does the same and takes T (and, in the backward, U)
// by fp32 dot products.
constexpr int64_t kInt8Few = 16;
bool int8_few_applies(int64_t R, int64_t K, int32_t r);
struct Int8Few {
  const float* F;      // factor of T: A [r x I] (forward) or B [O x r] (backward)
  float* T;            // [R x r] (null: not wanted)
  uint16_t* T_parts;   // nullable: T in three bf16 parts, [3][NP][ld]
  // backward only
  const void* X;       // [R x I]
  const float* A;      // where U is to be computed: its factor
  float* U_new;        // and its place (else null)
  const float* U;      // [R x r] for dB
  uint16_t* U_parts;   // nullable, as T_parts
  float* dA;           // [r x I]: what the product kernel adds up beside its
  float* dB;           // [O x r]  products, up to kInt8Few tokens (nullable)
  int32_t NP;
  int64_t ld;
};
cudaError_t launch_int8_few(const Int8Call& c, const Int8Few& f, void* ws, Int8Clear header, cudaStream_t st);
// Row products out[t, j] = sum_k P[t, k] L(k, j) by fp32 FMAs, for activations
// that the tensor-core ones do not take: L [r x K], or [K x r] (kr).
struct Int8Dot {
  const void* P;
  const float* L;
  float* out;
  int64_t K;
  bool kr;
};
cudaError_t launch_int8_dots(const Int8Dot* d, int count, bool bf16, int64_t R, int32_t r, cudaStream_t st);
// The product, over rows quantized before it, once T is computed; few:
// nullable, dA and dB.
cudaError_t launch_int8_product(const Int8Call& c, void* ws, uint32_t* hdr, const Int8Few* few,
                                cudaStream_t st);

// int8_tc.cu: the product over codes xq [R x int8_act_pitch(K)] with row scales
// xs; ws: int8_tc_ws bytes, of which the first int8_tc_zeroed are zero; few:
// the backward's side sums, nullable.
size_t int8_tc_ws(bool dx, int64_t R, int64_t O, int64_t I, int32_t r);
size_t int8_tc_zeroed(bool dx, int64_t R, int64_t O, int64_t I, int32_t r);
cudaError_t launch_int8_tc(const Int8Call& c, const int8_t* xq, const float* xs, const Int8Few* few, void* ws,
                           uint32_t* hdr, cudaStream_t st);

// int8_side.cu: the adapter's thin products over bf16 matrices: P [R x N] itself
// or a copy of it in bf16 parts (one of bf16 values whose N is no multiple of 8,
// three of fp32 values), a row's parts one after the other, `pitch` columns each.
// parts 0: the fp32 kernels take P (few rows, and bf16 of other N whose P does not
// start on 16 bytes: the workspace is sized without the pointers).
struct SideMatrix {
  const void* P;   // [R x parts * pitch]
  int64_t N, pitch;
  int parts;
};
bool side_takes(const void* P, int64_t R, int64_t N);
// Whether P [R x N], which side_takes refuses for its type or N, is worth a copy.
bool side_copies(bool bf16, int64_t R, int64_t N, int32_t r);
size_t side_copy_bytes(bool bf16, int64_t R, int64_t N);
SideMatrix side_matrix(const void* P, bool bf16, int64_t R, int64_t N, int32_t r, void* copy);
struct SideCopy {
  const void* src;
  SideMatrix m;  // m.P: the copy
};
cudaError_t launch_side_copy(const SideCopy* c, int count, bool bf16, int64_t R, cudaStream_t st);
// Parts: an fp32 factor [n x r] or [r x n] as three bf16 parts, [3][side_np(r)]
// rows of side_ld(len): entry e is the factor's entry e % wrap (row products: once
// for each part of the matrix's rows) or, with wrap 0, e / div (column products),
// zero past n.
int side_np(int32_t r);
int64_t side_ld(int64_t n);
size_t side_parts_bytes(int64_t len, int32_t r);
size_t side_part_ws(int32_t r);     // scratch of one launch
struct SideFactor {
  const float* src;
  uint16_t* parts;
  int64_t n;
  bool kr;  // [n x r]
  int64_t len, wrap;
  int div;
};
inline SideFactor side_factor_of_columns(const float* src, uint16_t* parts, bool kr, const SideMatrix& m) {
  return {src, parts, m.N, kr, m.parts * m.pitch, m.pitch, 1};
}
inline SideFactor side_factor_of_rows(const float* src, uint16_t* parts, int64_t R, const SideMatrix& m) {
  return {src, parts, R, true, m.parts * R, 0, m.parts};
}
cudaError_t launch_side_split(const SideFactor* f, int count, int32_t r, cudaStream_t st);
struct SideProduct {
  SideMatrix m;
  const uint16_t* factor;  // its parts over m's columns (row products) or rows (column products)
  float* out;              // s times the product: [R x r]; [N x r] or, transposed, [r x N]
  uint16_t* parts;         // nullable: its own parts (row products), [3][NP][side_ld(R)]
  bool transposed;
  float s;
};
// One or two products in one launch: P L^T (rows) or P^T T (columns).
cudaError_t launch_side(const SideProduct* f, int count, bool columns, int64_t R, int32_t r, void* part,
                        uint32_t* hdr, cudaStream_t st);

}  // namespace qlora
