// Attention inside the cells on the CUDA cores: fp32 products and sums from fp32 or 8-bit rows.  See
// window.cuh for the mathematics and the meaning of MAPS.
//
// One CTA (128 threads) takes tiles of 16 rows of a cell against the cell in chunks of 64.
// Thread (ty, tx), tid = 16 ty + tx, holds the scores of rows ty, ty + 8 against the chunk's
// rows tx + 16 j, and of the products with a chunk the columns tx * VEC (+ 64).  Cells of up
// to 64 tokens keep their one chunk's scores in registers; larger cells take two passes, one
// for the softmax statistics (and D), one for the products.  Products and sums are fp32: a weight is off
// by 2^-22 (the exponential) and 2^-24 ln 2 times its score in units of log2 for each rounding of the
// score, where operands of the tensor cores' formats would be off by 2^-11 (tf32) and more.  dbias sums
// its rows in fp32 one after another: a relative error of about 2^-23 sqrt(adds) / 6, adds those of an
// offset in a CTA.
// Bound by shared memory (59 to 79% of its wavefronts) and by the loads that fill a tile before its one
// or two chunks: 20011 tokens, 8/2 heads of 32, edge 6: forward 104 us, dq with dbias 177 us, dk/dv
// 137 us (7, 6 and 11 TFLOP/s of products); differential, 9001 tokens: 51, 73, 75.
// Loads of four rows ahead in `fill` cost registers and with them CTAs (dq 173 -> 238 us).
#include "window.cuh"

namespace ssa {
namespace {

using namespace win;

constexpr int kThreads = 128;
constexpr int kChunk = 64;
constexpr int kWStride = kChunk + 4;

template <typename E>
__device__ __forceinline__ float4 load4(const E* p, float s);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p, float) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<int8_t>(const int8_t* p, float s) {
  const int w = __ldg(reinterpret_cast<const int*>(p));
  return make_float4((float)(int8_t)w * s, (float)(int8_t)(w >> 8) * s, (float)(int8_t)(w >> 16) * s,
                     (float)(w >> 24) * s);
}

// dst[r][0 .. W): head `head` (W / D heads side by side) of the tokens rows[first + r], r < n;
// zeros for n <= r < total.
template <typename E, int D, int W>
__device__ __forceinline__ void fill(float* dst, const void* src, const float* scale, int heads, int head,
                                     const int2* __restrict__ rows, int first, int n, int total) {
  for (int i = threadIdx.x; i < total * (W / 4); i += kThreads) {
    const int r = i / (W / 4), c = i % (W / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n) {
      const size_t row = (size_t)__ldg(&rows[first + r].x) * heads + head;
      v = load4<E>(static_cast<const E*>(src) + row * D + c, scale ? __ldg(scale + row + c / D) : 1.f);
    }
    *reinterpret_cast<float4*>(dst + r * (W + 4) + c) = v;
  }
}

// s[i][j] = <A[ty + 8 i], B[tx + 16 j]> for j < NJ, 0 for the others
template <int W, int NJ>
__device__ __forceinline__ void dots_of(const float* A, const float* B, float s[2][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < W; c += 4) {
    float4 a[2], b[NJ];
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 8 * i) * (W + 4) + c);
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (W + 4) + c);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
      }
  }
}
// The rows of a chunk of n that are filled and multiplied: half a chunk, where that holds all (cells
// of the shells hold some 30 tokens at an edge of 6).
__device__ __forceinline__ int live(int n) { return n <= kChunk / 2 ? kChunk / 2 : kChunk; }
template <int W>
__device__ __forceinline__ void dots(const float* A, const float* B, int n, float s[2][4]) {
  if (live(n) < kChunk)
    dots_of<W, 2>(A, B, s);
  else
    dots_of<W, 4>(A, B, s);
}

// Columns of a product that a thread holds: VEC at tx * VEC + 16 * VEC * u, u < NU.
template <int W>
struct Cols {
  static constexpr int VEC = W >= 64 ? 4 : 2;
  static constexpr int NU = W / (16 * VEC);
  static constexpr int N = VEC * NU;
};

// acc[i][:] += sum_{j < n} P[ty + 8 i][j] B[j][cols], four j at a time: P and B are 0 from n on.
template <int W>
__device__ __forceinline__ void accum(const float* P, const float* B, int n, float (*acc)[Cols<W>::N]) {
  constexpr int VEC = Cols<W>::VEC, NU = Cols<W>::NU;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int j = 0; j < n; j += 4) {
    const float4 p0 = *reinterpret_cast<const float4*>(P + ty * kWStride + j);
    const float4 p1 = *reinterpret_cast<const float4*>(P + (ty + 8) * kWStride + j);
    const float q[2][4] = {{p0.x, p0.y, p0.z, p0.w}, {p1.x, p1.y, p1.z, p1.w}};
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
          const float b = B[(j + y) * (W + 4) + tx * VEC + 16 * VEC * u + x];
          acc[0][u * VEC + x] = fmaf(q[0][y], b, acc[0][u * VEC + x]);
          acc[1][u * VEC + x] = fmaf(q[1][y], b, acc[1][u * VEC + x]);
        }
  }
}

__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T, int D, int W>
__device__ __forceinline__ void store_rows(T* out, int heads, int head, const int2* rows, int first, int n,
                                           float (*acc)[Cols<W>::N], float mul) {
  constexpr int VEC = Cols<W>::VEC, NU = Cols<W>::NU;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = ty + 8 * i;
    if (r >= n) continue;
    T* p = out + ((size_t)rows[first + r].x * heads + head) * D;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int x = 0; x < VEC; ++x) p[tx * VEC + 16 * VEC * u + x] = Elem<T>::from_f(acc[i][u * VEC + x] * mul);
  }
}

// Shared memory (floats): query-side tiles A (MAPS of width D), key-side chunk B (MAPS of width
// D and one of width MAPS * D), dO (width MAPS * D), weights (MAPS).
template <int D, int MAPS>
struct Lay {
  static constexpr int DV = MAPS * D;
  static constexpr int A = 0;                                      // [MAPS][16][D + 4]
  static constexpr int O = A + MAPS * kTile * (D + 4);             // [16][DV + 4]
  static constexpr int B = O + kTile * (DV + 4);                   // [MAPS][64][D + 4]
  static constexpr int V = B + MAPS * kChunk * (D + 4);            // [64][DV + 4]
  static constexpr int P = V + kChunk * (DV + 4);                  // [MAPS][16][68]
  static constexpr int codes = P + MAPS * kTile * kWStride;        // int [64 + 16]
  static constexpr int stat = codes + kChunk + kTile;              // [2 MAPS][64]
  static constexpr int total = stat + 2 * MAPS * kChunk;
};

// Scores of the tile against one chunk in units of log2, bias included, minus infinity past
// the chunk's n rows; map u of MAPS.
template <int D, int MAPS>
__device__ __forceinline__ void scores(const WinArgs& a, int h, const float* sm, int u, int n, float mul,
                                       float s[2][4]) {
  using L = Lay<D, MAPS>;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  dots<D>(sm + L::A + u * kTile * (D + 4), sm + L::B + u * kChunk * (D + 4), n, s);
  const int* codes = reinterpret_cast<const int*>(sm + L::codes);
  const int c0 = a.table ? center(a.m) : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = s[i][j] * mul;
      if (a.table && tx + 16 * j < n) x += bias2_at(a, h, codes[kChunk + ty + 8 * i] - codes[tx + 16 * j] + c0);
      s[i][j] = tx + 16 * j < n ? x : kNegInf;
    }
}

// Sums of 0 are made NaN in rows that the bias leaves a key (key_left).  By whole warps, whose halves
// hold rows of their own.
template <int MAPS>
__device__ __forceinline__ void check_sums(const WinArgs& a, int h, const int* codes, int lo, int hi, float (*l)[2]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  bool none = false;
#pragma unroll
  for (int u = 0; u < MAPS; ++u) none |= l[u][0] == 0.f || l[u][1] == 0.f;
  if (!__any_sync(0xffffffffu, none)) return;
#pragma unroll
  for (int u = 0; u < MAPS; ++u)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bool left = l[u][i] == 0.f;
      if (a.table) left = left && key_left(a, h, codes[kChunk + ty + 8 * i], lo, hi, tx, 16);
      if (row_max(left ? 1.f : 0.f) > 0.f) l[u][i] = __uint_as_float(0x7fc00000u);
    }
}

template <typename E, typename T, int D, int MAPS>
__global__ void __launch_bounds__(kThreads) window_fwd_kernel(WinArgs a) {
  using L = Lay<D, MAPS>;
  constexpr int DV = L::DV;
  extern __shared__ float sm[];
  int* codes = reinterpret_cast<int*>(sm + L::codes);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int h = blockIdx.y, hk = h / (a.hq / a.hkv);
  const float mul = a.scale * kLog2e;
  float lam = 0.f;
  if constexpr (MAPS == 2) {
    float e1, e2;
    lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
    lam = e1 - e2 + a.lam_init;
  }
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int4 tile = a.tiles[t];
    const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
    if (nr == 0) continue;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MAPS; ++u)
      fill<E, D, D>(sm + L::A + u * kTile * (D + 4), a.q, nullptr, a.hq, MAPS * h + u, a.rows, first, nr, kTile);
    if (threadIdx.x < kTile) codes[kChunk + threadIdx.x] = threadIdx.x < nr ? a.rows[first + threadIdx.x].y : 0;
    const bool one = hi - lo <= kChunk;
    float m[MAPS][2], l[MAPS][2], s[MAPS][2][4];
    float acc[2][Cols<DV>::N];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int u = 0; u < MAPS; ++u) m[u][i] = kNegInf, l[u][i] = 0.f;
#pragma unroll
      for (int x = 0; x < Cols<DV>::N; ++x) acc[i][x] = 0.f;
    }
    for (int pass = one ? 1 : 0; pass < 2; ++pass)
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        const int n = hi - k0 < kChunk ? hi - k0 : kChunk;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          fill<E, D, D>(sm + L::B + u * kChunk * (D + 4), a.k, nullptr, a.hkv, MAPS * hk + u, a.rows, k0, n, live(n));
        if (pass == 1) fill<E, D, DV>(sm + L::V, a.v, nullptr, a.hkv, MAPS * hk, a.rows, k0, n, live(n));
        if (threadIdx.x < kChunk) codes[threadIdx.x] = threadIdx.x < n ? a.rows[k0 + threadIdx.x].y : 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u) scores<D, MAPS>(a, h, sm, u, n, mul, s[u]);
        if (pass == 0 || one) {
#pragma unroll
          for (int u = 0; u < MAPS; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mx = fmaxf(m[u][i], row_max(fmaxf(fmaxf(s[u][i][0], s[u][i][1]), fmaxf(s[u][i][2], s[u][i][3]))));
              const float ms = safe_max(mx);
              float e = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j) e += ex2(s[u][i][j] - ms);
              l[u][i] = l[u][i] * rescale(m[u][i], ms) + row_sum(e);
              m[u][i] = mx;
            }
        }
        if (pass == 0) continue;
        if (k0 == lo) check_sums<MAPS>(a, h, codes, lo, hi, l);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p = ex2(s[0][i][j] - safe_max(m[0][i])) * safe_inv(l[0][i]);
            if constexpr (MAPS == 2) p -= lam * (ex2(s[1][i][j] - safe_max(m[1][i])) * safe_inv(l[1][i]));
            sm[L::P + (ty + 8 * i) * kWStride + tx + 16 * j] = p;
          }
        __syncthreads();
        accum<DV>(sm + L::P, sm + L::V, n, acc);
      }
    store_rows<T, D, DV>(static_cast<T*>(a.out), a.hq, MAPS * h, a.rows, first, nr, acc, 1.f);
    if (MAPS == 1 && a.lse && tx == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (ty + 8 * i < nr) {
          const float x = lse2_of(m[0][i], l[0][i]);
          a.lse[(size_t)a.rows[first + ty + 8 * i].x * a.hq + h] = x == kPosInf ? kNegInf : x * kLn2;
        }
    }
  }
}

// dq, the row statistics for window_dkv_kernel, and the partial bias gradients.  Each CTA keeps
// one table of offsets; a row's keys have distinct offsets, so one warp adds a row's dS to it
// without atomics (keys of one voxel take turns), rows in order.
template <typename E, typename T, int D, int MAPS>
__global__ void __launch_bounds__(kThreads) window_dq_kernel(WinArgs a) {
  using L = Lay<D, MAPS>;
  constexpr int DV = L::DV;
  extern __shared__ float sm[];
  float* dtab = sm + L::total;
  int* codes = reinterpret_cast<int*>(sm + L::codes);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int h = blockIdx.y, hk = h / (a.hq / a.hkv);
  const float mul = a.scale * kLog2e;
  const int T3 = a.dbias ? offsets(a.m) : 0, c0 = a.table ? center(a.m) : 0;
  for (int i = threadIdx.x; i < T3; i += kThreads) dtab[i] = 0.f;
  float lam = 0.f;
  if constexpr (MAPS == 2) {
    float e1, e2;
    lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
    lam = e1 - e2 + a.lam_init;
  }
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int4 tile = a.tiles[t];
    const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
    if (nr == 0) continue;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MAPS; ++u)
      fill<E, D, D>(sm + L::A + u * kTile * (D + 4), a.q, a.sq, a.hq, MAPS * h + u, a.rows, first, nr, kTile);
    fill<T, D, DV>(sm + L::O, a.dout, nullptr, a.hq, MAPS * h, a.rows, first, nr, kTile);
    if (threadIdx.x < kTile) codes[kChunk + threadIdx.x] = threadIdx.x < nr ? a.rows[first + threadIdx.x].y : 0;
    const bool one = hi - lo <= kChunk;
    float m[MAPS][2], l[MAPS][2], dd[MAPS][2], s[MAPS][2][4], dp[2][4];
    float acc[MAPS][2][Cols<D>::N];
#pragma unroll
    for (int u = 0; u < MAPS; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[u][i] = kNegInf, l[u][i] = 0.f, dd[u][i] = 0.f;
#pragma unroll
        for (int x = 0; x < Cols<D>::N; ++x) acc[u][i][x] = 0.f;
      }
    for (int pass = one ? 1 : 0; pass < 2; ++pass)
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        const int n = hi - k0 < kChunk ? hi - k0 : kChunk;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          fill<E, D, D>(sm + L::B + u * kChunk * (D + 4), a.k, a.sk, a.hkv, MAPS * hk + u, a.rows, k0, n, live(n));
        fill<E, D, DV>(sm + L::V, a.v, a.sv, a.hkv, MAPS * hk, a.rows, k0, n, live(n));
        if (threadIdx.x < kChunk) codes[threadIdx.x] = threadIdx.x < n ? a.rows[k0 + threadIdx.x].y : 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u) scores<D, MAPS>(a, h, sm, u, n, mul, s[u]);
        dots<DV>(sm + L::O, sm + L::V, n, dp);
        if (pass == 0 || one) {
#pragma unroll
          for (int u = 0; u < MAPS; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mx = fmaxf(m[u][i], row_max(fmaxf(fmaxf(s[u][i][0], s[u][i][1]), fmaxf(s[u][i][2], s[u][i][3]))));
              const float ms = safe_max(mx), corr = rescale(m[u][i], ms);
              float e = 0.f, ed = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float p = ex2(s[u][i][j] - ms);
                e += p;
                if (tx + 16 * j < n) ed = fmaf(p, dp[i][j], ed);
              }
              l[u][i] = l[u][i] * corr + row_sum(e);
              dd[u][i] = dd[u][i] * corr + row_sum(ed);
              m[u][i] = mx;
            }
        }
        if (pass == 0) continue;
        if (k0 == lo) check_sums<MAPS>(a, h, codes, lo, hi, l);
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float inv = safe_inv(l[u][i]), ms = safe_max(m[u][i]), dm = dd[u][i] * inv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p = ex2(s[u][i][j] - ms) * inv;
              const float ds = tx + 16 * j < n ? p * (dp[i][j] - dm) : 0.f;
              sm[L::P + (u * kTile + ty + 8 * i) * kWStride + tx + 16 * j] = u ? -lam * ds : ds;
            }
          }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          accum<D>(sm + L::P + u * kTile * kWStride, sm + L::B + u * kChunk * (D + 4), n, acc[u]);
        if (T3 && threadIdx.x < 32) {
          // keys of one voxel take turns, by their rank among the lanes that hold the voxel
          const int lane = threadIdx.x, k0c = codes[lane], k1c = codes[32 + lane];
          const bool v0 = lane < n, v1 = lane + 32 < n;
          int r0 = 0, r1 = 0, most = 0;
          if (tile.y & kDupFlag) {
            const unsigned below = (1u << lane) - 1u;
            r0 = __popc(__match_any_sync(0xffffffffu, v0 ? k0c : -1 - lane) & below);
            r1 = __popc(__match_any_sync(0xffffffffu, v1 ? k1c : -1 - lane) & below);
            most = __reduce_max_sync(0xffffffffu, max(r0, r1));
          }
          if (!(tile.y & kDupFlag)) {  // a row's offsets are distinct: its two halves at once, dS read ahead
            float d0[kTile], d1[kTile];
#pragma unroll
            for (int r = 0; r < kTile; ++r) {
              d0[r] = sm[L::P + r * kWStride + lane];
              d1[r] = sm[L::P + r * kWStride + 32 + lane];
            }
#pragma unroll
            for (int r = 0; r < kTile; ++r) {
              if (r >= nr) break;
              float* at = dtab + codes[kChunk + r] + c0;
              float x0 = 0.f, x1 = 0.f;
              if (v0) x0 = at[-k0c];
              if (v1) x1 = at[-k1c];
              if (v0) at[-k0c] = x0 + d0[r];
              if (v1) at[-k1c] = x1 + d1[r];
              __syncwarp();
            }
          } else {
            for (int r = 0; r < nr; ++r) {
              const int cr = codes[kChunk + r] + c0;
              const float* ds = sm + L::P + r * kWStride;
              for (int i = 0; i <= most; ++i) {
                if (v0 && r0 == i) dtab[cr - k0c] += ds[lane];
                __syncwarp();
              }
              for (int i = 0; i <= most; ++i) {
                if (v1 && r1 == i) dtab[cr - k1c] += ds[32 + lane];
                __syncwarp();
              }
            }
          }
        }
      }
#pragma unroll
    for (int u = 0; u < MAPS; ++u) {
      store_rows<T, D, D>(static_cast<T*>(a.dq), a.hq, MAPS * h + u, a.rows, first, nr, acc[u], a.scale);
      if (tx == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (ty + 8 * i < nr) {
            const size_t at = (size_t)(MAPS * h + u) * a.N + first + ty + 8 * i;
            store_lse2(a, at, m[u][i], l[u][i]);
            a.D[at] = dd[u][i] * safe_inv(l[u][i]);
          }
    }
  }
  __syncthreads();
  float* part = a.part + ((size_t)h * a.parts + blockIdx.x) * T3;
  for (int i = threadIdx.x; i < T3; i += kThreads) part[i] = dtab[i];
}

// dk, dv of 16 keys (sums in registers, no atomics): the transposed scores of all query heads of the key head against the
// cell's rows in chunks of 64.
template <typename E, typename T, int D, int MAPS>
__global__ void __launch_bounds__(kThreads) window_dkv_kernel(WinArgs a) {
  using L = Lay<D, MAPS>;
  constexpr int DV = L::DV;
  extern __shared__ float sm[];
  int* codes = reinterpret_cast<int*>(sm + L::codes);
  float* stat = sm + L::stat;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int G = a.hq / a.hkv, hk = blockIdx.y;
  const float mul = a.scale * kLog2e;
  const int c0 = a.table ? center(a.m) : 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int4 tile = a.tiles[t];
    const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
    if (nr == 0) continue;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MAPS; ++u)
      fill<E, D, D>(sm + L::A + u * kTile * (D + 4), a.k, a.sk, a.hkv, MAPS * hk + u, a.rows, first, nr, kTile);
    fill<E, D, DV>(sm + L::O, a.v, a.sv, a.hkv, MAPS * hk, a.rows, first, nr, kTile);
    if (threadIdx.x < kTile) codes[kChunk + threadIdx.x] = threadIdx.x < nr ? a.rows[first + threadIdx.x].y : 0;
    float dk[MAPS][2][Cols<D>::N], dv[2][Cols<DV>::N];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int u = 0; u < MAPS; ++u)
#pragma unroll
        for (int x = 0; x < Cols<D>::N; ++x) dk[u][i][x] = 0.f;
#pragma unroll
      for (int x = 0; x < Cols<DV>::N; ++x) dv[i][x] = 0.f;
    }
    for (int h = hk * G; h < hk * G + G; ++h) {
      float lam = 0.f;
      if constexpr (MAPS == 2) {
        float e1, e2;
        lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
        lam = e1 - e2 + a.lam_init;
      }
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        const int n = hi - k0 < kChunk ? hi - k0 : kChunk;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          fill<E, D, D>(sm + L::B + u * kChunk * (D + 4), a.q, a.sq, a.hq, MAPS * h + u, a.rows, k0, n, live(n));
        fill<T, D, DV>(sm + L::V, a.dout, nullptr, a.hq, MAPS * h, a.rows, k0, n, live(n));
        bool any_far = false;
        if (threadIdx.x < kChunk) {
          codes[threadIdx.x] = threadIdx.x < n ? a.rows[k0 + threadIdx.x].y : 0;
#pragma unroll
          for (int u = 0; u < MAPS; ++u) {
            const size_t at = (size_t)(MAPS * h + u) * a.N + k0 + threadIdx.x;
            const float lse2 = threadIdx.x < n ? a.lse2[at] : kPosInf;
            any_far |= is_far(lse2);
            stat[2 * u * kChunk + threadIdx.x] = lse2;
            stat[(2 * u + 1) * kChunk + threadIdx.x] = threadIdx.x < n ? a.D[at] : 0.f;
          }
        }
        any_far = __syncthreads_or(any_far);
        float s[MAPS][2][4], dp[2][4];
        dots<DV>(sm + L::O, sm + L::V, n, dp);
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          dots<D>(sm + L::A + u * kTile * (D + 4), sm + L::B + u * kChunk * (D + 4), n, s[u]);
        float pv[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            pv[i][j] = 0.f;
#pragma unroll
            for (int u = 0; u < MAPS; ++u) {
              float x = s[u][i][j] * mul;
              if (a.table && c < n) x += bias2_at(a, h, codes[c] - codes[kChunk + ty + 8 * i] + c0);
              float p = c < n ? ex2(x - stat[2 * u * kChunk + c]) : 0.f;
              if (any_far && c < n) {
                const size_t at = (size_t)(MAPS * h + u) * a.N + k0 + c;
                p *= far_factor(a, at, stat[2 * u * kChunk + c]);
                if (p > 1.f) p = 1.f;  // a score may round to one side here, to the other where lse2 was taken
              }
              const float ds = c < n ? p * (dp[i][j] - stat[(2 * u + 1) * kChunk + c]) : 0.f;
              pv[i][j] += u ? -lam * p : p;
              s[u][i][j] = u ? -lam * ds : ds;
            }
          }
        // the MAPS weight buffers take dS first, then the first one P
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sm[L::P + (u * kTile + ty + 8 * i) * kWStride + tx + 16 * j] = s[u][i][j];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
          accum<D>(sm + L::P + u * kTile * kWStride, sm + L::B + u * kChunk * (D + 4), n, dk[u]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sm[L::P + (ty + 8 * i) * kWStride + tx + 16 * j] = pv[i][j];
        __syncthreads();
        accum<DV>(sm + L::P, sm + L::V, n, dv);
      }
    }
#pragma unroll
    for (int u = 0; u < MAPS; ++u)
      store_rows<T, D, D>(static_cast<T*>(a.dk), a.hkv, MAPS * hk + u, a.rows, first, nr, dk[u], a.scale);
    store_rows<T, D, DV>(static_cast<T*>(a.dv), a.hkv, MAPS * hk, a.rows, first, nr, dv, 1.f);
  }
}

template <typename K>
cudaError_t go(const char* name, K kern, dim3 grid, size_t smem, const WinArgs& a, cudaStream_t st) {
  const cudaError_t e = need_smem(kern, smem);
  if (e != cudaSuccess) return e;
  SSA_LAUNCH(name, kern, grid, kThreads, smem, st, a);
  return cudaGetLastError();
}

template <typename T, int D, int MAPS>
cudaError_t fwd(const WinArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * Lay<D, MAPS>::total;
  return go("window_fwd_kernel", window_fwd_kernel<T, T, D, MAPS>, dim3(a.T, a.hq / MAPS), smem, a, st);
}

template <typename E, typename T, int D, int MAPS>
cudaError_t bwd(const WinArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(float) * Lay<D, MAPS>::total;
  const size_t tab = a.dbias ? sizeof(float) * offsets(a.m) : 0;
  const int gx = a.dbias ? a.parts : a.T;
  cudaError_t e = go("window_dq_kernel", window_dq_kernel<E, T, D, MAPS>, dim3(gx, a.hq / MAPS), smem + tab, a, st);
  if (e != cudaSuccess) return e;
  return go("window_dkv_kernel", window_dkv_kernel<E, T, D, MAPS>, dim3(a.T, a.hkv / MAPS), smem, a, st);
}

template <typename E, typename T>
cudaError_t bwd_d(const WinArgs& a, cudaStream_t st) {
  if (a.maps == 2) return a.d == 32 ? bwd<E, T, 32, 2>(a, st) : bwd<E, T, 64, 2>(a, st);
  return a.d == 32 ? bwd<E, T, 32, 1>(a, st) : a.d == 64 ? bwd<E, T, 64, 1>(a, st) : bwd<E, T, 128, 1>(a, st);
}

template <typename T>
cudaError_t fwd_d(const WinArgs& a, cudaStream_t st) {
  if (a.maps == 2) return a.d == 32 ? fwd<T, 32, 2>(a, st) : fwd<T, 64, 2>(a, st);
  return a.d == 32 ? fwd<T, 32, 1>(a, st) : a.d == 64 ? fwd<T, 64, 1>(a, st) : fwd<T, 128, 1>(a, st);
}

}  // namespace

cudaError_t window_fwd_simt(const WinArgs& a, cudaStream_t st) { return fwd_d<float>(a, st); }

cudaError_t window_bwd_simt(const WinArgs& a, cudaStream_t st) {
  return a.act8 ? bwd_d<int8_t, float>(a, st) : bwd_d<float, float>(a, st);
}

// Up to six CTAs for every SM (three of the bf16 kernel, which takes two heads each): few enough for
// the sums of their tables, enough that the last ones to finish leave little idle; one or two while
// that gives a CTA fewer than 16 slots.
int window_parts(int hq, int64_t T) {
  const int64_t waves = max((int64_t)1, min((int64_t)3, hq * T / (32 * kSms)));
  return (int)max((int64_t)1, min(T, 2 * waves * kSms / hq));
}

}  // namespace ssa
