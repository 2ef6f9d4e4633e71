// Attention inside the cells of a partition: argument bundle and helpers shared by the
// fp32 CUDA-core kernels (window_simt.cu) and the bf16 tensor-core kernels (window_mma.cu).
//
// MAPS = 1: window attention, optionally with a relative position bias.
// MAPS = 2: differential attention; an output head has two maps (heads 2h, 2h + 1 of q and k)
// and one value head of width 2 d (heads 2h, 2h + 1 of v side by side).  "Head" below is an
// output head: hq / MAPS of them read hkv / MAPS key heads, G = hq / hkv each.
//
// Scores are held in units of log2: s2 = (scale <q, k> + bias) log2(e), p = 2^(s2 - max) / sum.
// The backward keeps two numbers per row and map between its kernels: lse2 = max + log2(sum)
// (plus infinity for a row with nothing left, so that every p is 0) and D = sum_j p_j dP_j.  Where
// lse2 is so large that its rounding shows in the weights (kFarScore), what it rounded away is kept
// too; far from zero all of log2(sum) is lost in it, and the weights of a row would sum to its keys.
// D comes from the recomputed p and dP, not from the rounded output, so the fp32 gradients of
// the bias and of lambda do not carry a rounding to bf16; the forward has to leave nothing.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace ssa {
namespace win {

constexpr int kTile = SSA_WINDOW_TILE;  // rows of a work tile
constexpr int kDupFlag = 65536;         // tiles[].y: two tokens of the cell share a voxel
constexpr int kDupUnit = 131072;        // and from here on: the most tokens of one voxel, kDupTop at most
constexpr int kDupTop = 16383;
constexpr int kDupMost = 2048;  // up to here no cell's bias gradient goes to the 64-bit sums (bf16, kLone)

// Dynamic shared memory of a CTA at most, beside what kernels declare; and the bound that a kernel is
// given before its first launch above 48 KB.  The same for every call: the size of a launch depends on its
// plan, and a bound that follows it would be lowered by another host thread between this one's two calls.
constexpr size_t kSmemMost = 226 * 1024;
template <typename K>
cudaError_t need_smem(K kern, size_t smem) {
  return smem > 47 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost)
                          : cudaSuccess;
}

// Offsets of a window of edge m, and the number of the offset 0.
__host__ __device__ inline int offsets(int m) { return (2 * m - 1) * (2 * m - 1) * (2 * m - 1); }
// Floats from one head's table of offsets to the next in WinArgs::tab2.
__host__ __device__ inline int table_pitch(int m) { return (offsets(m) + 3) & ~3; }
__host__ __device__ inline int center(int m) { return (m - 1) * ((2 * m - 1) * (2 * m - 1) + (2 * m - 1) + 1); }

// The 64-bit sums of the bias gradient (WinArgs::sums): dS 2^s with 2^s <= 2^61 / (2 M N), M < 2^127 the
// largest |dP| of the head, as bits.
constexpr uint32_t kTopDp = 0x7f000000u;  // 2^127
__host__ __device__ inline int wide_bits(uint32_t amax, int64_t N) {
  int rb = 0;
  while (rb < 62 && (int64_t(1) << rb) <= N) ++rb;  // N < 2^rb
  return 61 - rb - 1 - ((int)(amax >> 23) - 126);
}

// 2^x (x <= 0 here, or minus infinity, or NaN).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kNegInf = -__builtin_inff();
constexpr float kPosInf = __builtin_inff();

// The maximum to subtract: 0 for a row with nothing left (every score minus infinity).
__device__ __forceinline__ float safe_max(float m) { return m == kNegInf ? 0.f : m; }
// The factor of sums taken against `old` when `now` (finite) is subtracted instead; 1 while nothing
// was summed (2^-now could be infinite, and its product with an empty sum NaN).
__device__ __forceinline__ float rescale(float old, float now) { return old == kNegInf ? 1.f : ex2(old - now); }
// 1 / sum, 0 for a row with nothing left; a NaN sum stays NaN.
__device__ __forceinline__ float safe_inv(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse2_of(float m, float l) { return l == 0.f ? kPosInf : m + log2f(l); }

// Rows whose |lse2| is at least this: rounding it is off by 2^-15 and more, and the rest goes to a.rest;
// *a.far (bf16) tells the kernels after it to look there.
constexpr float kFarScore = 1024.f;
__device__ __forceinline__ bool is_far(float lse2) { return fabsf(lse2) >= kFarScore && fabsf(lse2) < kPosInf; }
// Keeps lse2 of the row `at`: maximum m, sum l.
__device__ __forceinline__ void store_lse2(const WinArgs& a, size_t at, float m, float l) {
  const float lse2 = lse2_of(m, l);
  a.lse2[at] = lse2;
  if (is_far(lse2)) {
    a.rest[at] = log2f(l) - (lse2 - m);  // exact: |m| is the larger
    *a.far = 1;
  }
}
// What weights 2^(s - lse2) of the row `at` have to be multiplied by.
__device__ __forceinline__ float far_factor(const WinArgs& a, size_t at, float lse2) {
  return is_far(lse2) ? ex2(-a.rest[at]) : 1.f;
}

// exp(<a, b>) pair of one head: lambda = e1 - e2 + init, from lam [4, heads, d].  Called by
// whole warps.
template <int D>
__device__ __forceinline__ void lambda_terms(const float* __restrict__ lam, int heads, int h, float& e1, float& e2) {
  const int lane = threadIdx.x & 31;
  float s1 = 0.f, s2 = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = lane + 32 * i;
    const size_t st = (size_t)heads * D, at = (size_t)h * D + c;
    s1 = fmaf(lam[at], lam[st + at], s1);
    s2 = fmaf(lam[2 * st + at], lam[3 * st + at], s2);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    s2 += __shfl_xor_sync(0xffffffffu, s2, o);
  }
  e1 = expf(s1);
  e2 = expf(s2);
}

// Bias of offset `off` in units of log2; values at or below kBar bar as minus infinity does
// (in units of log2 the type's lowest would overflow).
constexpr float kBar = -1e38f;
__device__ __forceinline__ float bias2_at(const WinArgs& a, int h, int off) {
  const int b = a.bucket ? __ldg(a.bucket + off) : off;
  if ((unsigned)b >= (unsigned)a.nb) return 0.f;
  const float x = __ldg(a.table + (size_t)h * a.nb + b);
  return x <= kBar ? kNegInf : x * kLog2e;
}

// Whether the bias leaves the row with code `code` a key: looked at by `step` lanes from key lo + `at` on.
// For rows whose sum is 0: with a key left their scores are minus infinity by themselves (an infinity in
// q or k, or a product past fp32), and their softmax is NaN, not a row with nothing left.
__device__ __forceinline__ bool key_left(const WinArgs& a, int h, int code, int lo, int hi, int at, int step) {
  bool left = false;
#pragma unroll 1
  for (int j = lo + at; j < hi && !left; j += step)
    left = bias2_at(a, h, code - __ldg(&a.rows[j].y) + center(a.m)) > kNegInf;
  return left;
}

}  // namespace win
}  // namespace ssa
