// Attention inside the cells on warp-level tensor-core MMAs (mma.sync m16n8k16, bf16 operands,
// fp32 sums).  See window.cuh for the mathematics and the meaning of MAPS.
//
// A warp works alone on 16 rows of a cell and one head.  All operands go from global memory
// (in practice L1: the warps of a CTA take neighbouring tiles, so they share a cell's keys)
// straight into MMA fragments, with 16-byte loads and without shared memory:
//   * a contraction over the head dim does not care about the order of the dim, as long as both
//     operands agree, so thread (g, t) of the fragment (g = lane / 4, t = lane % 4) takes dims
//     32 c + 8 t .. + 7 of its row as its elements of the steps 2c and 2c + 1;
//   * a contraction over keys wants two keys in one register.  The thread loads dims 8 g .. + 7 of
//     the keys 2t, 2t + 1, 2t + 8, 2t + 9 and pairs them with byte permutes; column g of the n-tile e
//     is then dim 8 g + e, and a thread's accumulators are 16 consecutive dims of its rows.
// A cell is walked in chunks of 64 keys whose scores stay in registers.  The cells of surface
// voxels hold some 60 tokens (windows of edge 8), so most have one chunk: nothing is recomputed
// or rescaled.  Tiles of 128 rows (tcgen05) would stand half empty on such cells and hand every
// score through TMEM; the warps here need no barrier at all.
#include "tc.cuh"
#include "window.cuh"

namespace ssa {
namespace {

using namespace win;
using bf16 = __nv_bfloat16;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kChunk = 64;
constexpr size_t kSmemMost = 226 * 1024;  // dynamic shared memory of a CTA, beside the barriers

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8-bit codes (as in an int) to bf16 values times s: the byte + 128 in the low mantissa bits
// of 2^23 is an exact float, so are the difference and the product with a power of two.
__device__ __forceinline__ uint2 codes4(uint32_t w, float s) {
  w ^= 0x80808080u;
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + i)) - 8388736.f) * s;
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// Rows of one tensor, [n, heads, D]; a row of W = MAPS * D values starts at head `head`.
template <typename E, int D>
struct Rows {
  const E* p;
  const float* s;  // row scales (8-bit rows)
  int heads, head;
  __device__ __forceinline__ size_t at(int tok) const { return (size_t)tok * heads + head; }
  // 8 (4) values from column `col` of row `r`
  __device__ __forceinline__ uint4 ld8(size_t r, int col) const {
    if constexpr (sizeof(E) == 2) {
      return __ldg(reinterpret_cast<const uint4*>(p + r * D + col));
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + r * D + col));
      const float f = __ldg(s + r + col / D);
      const uint2 a = codes4(w.x, f), b = codes4(w.y, f);
      return make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ uint2 ld4(size_t r, int col) const {
    if constexpr (sizeof(E) == 2) {
      return __ldg(reinterpret_cast<const uint2*>(p + r * D + col));
    } else {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p + r * D + col));
      return codes4(w, __ldg(s + r + col / D));
    }
  }
};

// A operand: 16 rows (tokens tg for row g, tg8 for row g + 8; zeros where the flag is off).
template <int W, typename R>
__device__ __forceinline__ void load_a(const R& src, int tg, bool vg, int tg8, bool vg8, uint32_t (*f)[4]) {
  const int t = threadIdx.x & 3;
  const size_t r0 = src.at(tg), r1 = src.at(tg8);
#pragma unroll
  for (int c = 0; c < W / 32; ++c) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    const uint4 x = vg ? src.ld8(r0, 32 * c + 8 * t) : z, y = vg8 ? src.ld8(r1, 32 * c + 8 * t) : z;
    f[2 * c][0] = x.x, f[2 * c][1] = y.x, f[2 * c][2] = x.y, f[2 * c][3] = y.y;
    f[2 * c + 1][0] = x.z, f[2 * c + 1][1] = y.z, f[2 * c + 1][2] = x.w, f[2 * c + 1][3] = y.w;
  }
}

// s[j] = A B^T for the n-tiles j < NT: column g of n-tile j is the row whose token lane 8 j + g of
// `tok` holds (32 rows per register).  Only 8-row tiles below n are computed, the others are 0.
template <int W, int NT, typename R>
__device__ __forceinline__ void contract_dim(const uint32_t (*a)[4], const R& src, const int* tok, int n,
                                             float (*s)[4]) {
  constexpr int B = W >= 128 ? 2 : 4;  // n-tiles in flight
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int j0 = 0; j0 < NT; j0 += B) {
#pragma unroll
    for (int j = j0; j < j0 + B; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
    if (8 * j0 < n) {
      uint4 b[B][W / 32];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const size_t r = src.at(__shfl_sync(kFull, tok[(j0 + j) / 4], (8 * (j0 + j) + g) & 31));
#pragma unroll
        for (int c = 0; c < W / 32; ++c) b[j][c] = src.ld8(r, 32 * c + 8 * t);
      }
#pragma unroll
      for (int c = 0; c < W / 32; ++c)
#pragma unroll
        for (int j = 0; j < B; ++j) {
          mma(s[j0 + j], a[2 * c], b[j][c].x, b[j][c].y);
          mma(s[j0 + j], a[2 * c + 1], b[j][c].z, b[j][c].w);
        }
    }
  }
}

// acc += P B, P as A fragments over NG groups of 16 rows of B; rows from n on count as zeros.
template <int W, int NG, typename R>
__device__ __forceinline__ void contract_rows(const uint32_t (*p)[4], const R& src, const int* tok, int n,
                                              float (*acc)[4]) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    if (16 * k < n) {
      size_t r[4];
      bool v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 16 * k + 2 * t + (i & 1) + 8 * (i >> 1);
        r[i] = src.at(__shfl_sync(kFull, tok[k / 2], key & 31));
        v[i] = key < n;
      }
      if constexpr (W == 32) {
        uint2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v[i] ? src.ld4(r[i], 4 * g) : make_uint2(0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
          mma(acc[e], p[k], __byte_perm(e < 2 ? x[0].x : x[0].y, e < 2 ? x[1].x : x[1].y, sel),
              __byte_perm(e < 2 ? x[2].x : x[2].y, e < 2 ? x[3].x : x[3].y, sel));
        }
      } else {
#pragma unroll
        for (int h = 0; h < W / 64; ++h) {
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = v[i] ? src.ld8(r[i], 64 * h + 8 * g) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4][4] = {{x[0].x, x[0].y, x[0].z, x[0].w},
                                    {x[1].x, x[1].y, x[1].z, x[1].w},
                                    {x[2].x, x[2].y, x[2].z, x[2].w},
                                    {x[3].x, x[3].y, x[3].z, x[3].w}};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
            mma(acc[8 * h + e], p[k], __byte_perm(w[0][e / 2], w[1][e / 2], sel),
                __byte_perm(w[2][e / 2], w[3][e / 2], sel));
          }
        }
      }
    }
  }
}

// Accumulators of contract_rows to rows (token tg / tg8 where the flags are on), times mul / mul8.
template <int D, int W>
__device__ __forceinline__ void store_acc(bf16* out, int heads, int head, int tg, bool vg, int tg8, bool vg8,
                                          float (*acc)[4], float mul, float mul8) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!(i ? vg8 : vg)) continue;
    const float f = i ? mul8 : mul;
    bf16* p = out + ((size_t)(i ? tg8 : tg) * heads + head) * D;
    if constexpr (W == 32) {
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = pack_bf16x2(acc[2 * (x & 1)][2 * i + x / 2] * f, acc[2 * (x & 1) + 1][2 * i + x / 2] * f);
      *reinterpret_cast<uint4*>(p + 8 * t) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int h = 0; h < W / 64; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = pack_bf16x2(acc[8 * h + 2 * x][2 * i + c] * f, acc[8 * h + 2 * x + 1][2 * i + c] * f);
          *reinterpret_cast<uint4*>(p + 64 * h + 16 * t + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
  }
}

// Scores of 8 n-tiles as A fragments of 4 groups of 16 (rounded to bf16).
template <int NT>
__device__ __forceinline__ void pack_a(float (*s)[4], uint32_t (*f)[4]) {
#pragma unroll
  for (int k = 0; k < NT / 2; ++k) {
    f[k][0] = pack_bf16x2(s[2 * k][0], s[2 * k][1]);
    f[k][1] = pack_bf16x2(s[2 * k][2], s[2 * k][3]);
    f[k][2] = pack_bf16x2(s[2 * k + 1][0], s[2 * k + 1][1]);
    f[k][3] = pack_bf16x2(s[2 * k + 1][2], s[2 * k + 1][3]);
  }
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
  return fmaxf(x, __shfl_xor_sync(kFull, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(kFull, x, 1);
  return x + __shfl_xor_sync(kFull, x, 2);
}

// The 64 keys of a chunk: lane l holds the tokens and codes of keys l and 32 + l (those past the
// end repeat the last one).
struct Keys {
  int tok[2], code[2], n;
  __device__ __forceinline__ void load(const int2* __restrict__ rows, int k0, int hi) {
    const int lane = threadIdx.x & 31;
    n = min(kChunk, hi - k0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int2 r = __ldg(&rows[k0 + min(32 * i + lane, n - 1)]);
      tok[i] = r.x;
      code[i] = r.y;
    }
  }
};

// s = s mul + bias in units of log2, minus infinity from key n on.  tab: the head's table by
// offset (shared or global memory); ci, ci8: codes of rows g, g + 8 plus the center.
template <bool BIAS>
__device__ __forceinline__ void finish_scores(float (*s)[4], const Keys& k, float mul, const float* tab, int ci,
                                              int ci8) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int key = 8 * j + 2 * t + x;
      float b0 = 0.f, b1 = 0.f;
      if constexpr (BIAS) {
        const int cj = __shfl_sync(kFull, k.code[j / 4], key & 31);
        b0 = tab[ci - cj];
        b1 = tab[ci8 - cj];
      }
      s[j][x] = key < k.n ? fmaf(s[j][x], mul, b0) : kNegInf;
      s[j][2 + x] = key < k.n ? fmaf(s[j][2 + x], mul, b1) : kNegInf;
    }
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int kFwdWarps = 8;

template <int D, int MAPS, bool BIAS>
__global__ void __launch_bounds__(32 * kFwdWarps, D == 128 || (MAPS == 2 && D == 64) ? 1 : 2)
    window_fwd_mma_kernel(WinArgs a) {
  constexpr int DV = MAPS * D;
  extern __shared__ float tab_s[];
  const int h = blockIdx.y, hk = h / (a.hq / a.hkv);
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, warp = threadIdx.x >> 5;
  const float mul = a.scale * kLog2e;
  const int c0 = BIAS ? center(a.m) : 0;
  if constexpr (BIAS) {
    for (int i = threadIdx.x; i < offsets(a.m); i += blockDim.x) tab_s[i] = bias2_at(a, h, i);
    __syncthreads();
  }
  float lam = 0.f;
  if constexpr (MAPS == 2) {
    float e1, e2;
    lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
    lam = e1 - e2 + a.lam_init;
  }
  const Rows<bf16, D> V = {static_cast<const bf16*>(a.v), nullptr, a.hkv, MAPS * hk};
  for (int t = blockIdx.x * kFwdWarps + warp; t < a.T; t += gridDim.x * kFwdWarps) {
    const int4 tile = __ldg(&a.tiles[t]);
    const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
    if (nr == 0) continue;
    const bool vg = g < nr, vg8 = g + 8 < nr;
    const int2 rg = __ldg(&a.rows[first + min(g, nr - 1)]), rg8 = __ldg(&a.rows[first + min(g + 8, nr - 1)]);
    uint32_t q[MAPS][D / 16][4];
#pragma unroll
    for (int u = 0; u < MAPS; ++u) {
      const Rows<bf16, D> Q = {static_cast<const bf16*>(a.q), nullptr, a.hq, MAPS * h + u};
      load_a<D>(Q, rg.x, vg, rg8.x, vg8, q[u]);
    }
    float m[MAPS][2], l[MAPS][2], acc[DV / 8][4];
#pragma unroll
    for (int u = 0; u < MAPS; ++u) m[u][0] = m[u][1] = kNegInf, l[u][0] = l[u][1] = 0.f;
#pragma unroll
    for (int e = 0; e < DV / 8; ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
    const bool one = hi - lo <= kChunk;
    Keys keys;
    float s[MAPS][8][4];
    auto scores = [&](int k0) {
      keys.load(a.rows, k0, hi);
#pragma unroll
      for (int u = 0; u < MAPS; ++u) {
        const Rows<bf16, D> K = {static_cast<const bf16*>(a.k), nullptr, a.hkv, MAPS * hk + u};
        contract_dim<D, 8>(q[u], K, keys.tok, keys.n, s[u]);
        finish_scores<BIAS>(s[u], keys, mul, tab_s, rg.y + c0, rg8.y + c0);
      }
    };
    // new maximum and sum of a row over the chunk; s becomes 2^(s - max); the old sum's factor comes back
    auto softmax = [&](int u, int i) {
      float mx = m[u][i];
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(s[u][j][2 * i], s[u][j][2 * i + 1]));
      mx = quad_max(mx);
      const float ms = safe_max(mx), old = ex2(safe_max(m[u][i]) - ms);
      float e = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[u][j][2 * i + x] = ex2(s[u][j][2 * i + x] - ms);
          e += s[u][j][2 * i + x];
        }
      l[u][i] = l[u][i] * old + quad_sum(e);
      m[u][i] = mx;
      return old;
    };
    uint32_t pf[4][4];
    if constexpr (MAPS == 1) {
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        scores(k0);
        const float f0 = softmax(0, 0), f1 = softmax(0, 1);
        pack_a<8>(s[0], pf);
        if (!one) {
#pragma unroll
          for (int e = 0; e < DV / 8; ++e) acc[e][0] *= f0, acc[e][1] *= f0, acc[e][2] *= f1, acc[e][3] *= f1;
        }
        contract_rows<DV, 4>(pf, V, keys.tok, keys.n, acc);
      }
      store_acc<D, DV>(static_cast<bf16*>(a.out), a.hq, MAPS * h, rg.x, vg, rg8.x, vg8, acc, safe_inv(l[0][0]),
                       safe_inv(l[0][1]));
      if (a.lse && t4 == 0) {
        if (vg) a.lse[(size_t)rg.x * a.hq + h] = l[0][0] == 0.f ? kNegInf : (m[0][0] + log2f(l[0][0])) * kLn2;
        if (vg8) a.lse[(size_t)rg8.x * a.hq + h] = l[0][1] == 0.f ? kNegInf : (m[0][1] + log2f(l[0][1])) * kLn2;
      }
    } else {
      // the maps are subtracted before the product with V, so both normalisers come first
      if (!one)
        for (int k0 = lo; k0 < hi; k0 += kChunk) {
          scores(k0);
#pragma unroll
          for (int u = 0; u < 2; ++u) softmax(u, 0), softmax(u, 1);
        }
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        scores(k0);
        float c[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (one) {
              softmax(u, i);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) s[u][j][2 * i + x] = ex2(s[u][j][2 * i + x] - safe_max(m[u][i]));
            }
            c[u][i] = safe_inv(l[u][i]) * (u ? -lam : 1.f);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[0][j][x] = fmaf(s[1][j][x], c[1][x >> 1], s[0][j][x] * c[0][x >> 1]);
        pack_a<8>(s[0], pf);
        contract_rows<DV, 4>(pf, V, keys.tok, keys.n, acc);
      }
      store_acc<D, DV>(static_cast<bf16*>(a.out), a.hq, MAPS * h, rg.x, vg, rg8.x, vg8, acc, 1.f, 1.f);
    }
  }
}

template <int D, int MAPS, bool BIAS>
cudaError_t fwd(const WinArgs& a, cudaStream_t st) {
  const size_t smem = BIAS ? sizeof(float) * offsets(a.m) : 0;
  auto kern = window_fwd_mma_kernel<D, MAPS, BIAS>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int heads = a.hq / MAPS, need = (a.T + kFwdWarps - 1) / kFwdWarps;
  int gx = (4 * 2 * 148 + heads - 1) / heads;
  gx = gx < need ? gx : need;
  SSA_LAUNCH("window_fwd_mma_kernel", kern, dim3(gx, heads), 32 * kFwdWarps, smem, st, a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// backward: dq, row statistics, partial bias gradients
// ---------------------------------------------------------------------------

// Eight warps.  With a bias gradient the last one is the CTA's collector: the others hand it their
// dS tiles (fp32, [16][64]) through a slot each, and it alone adds them to the CTA's table of
// offsets, in a fixed order.  A row's keys have distinct offsets, so a row is one read, add and
// write per lane without atomics (cells with two tokens in a voxel: lane by lane).
constexpr int kDqWarps = 8;
constexpr int kSlotStride = kChunk + 4;
constexpr int kSlot = kTile * kSlotStride;  // floats

// TAB: where the bias is read: 0 no bias, 1 shared memory, 2 global memory (the table beside the
// collector's does not fit: edge 16).
template <int D, int MAPS, int TAB, typename E>
__global__ void __launch_bounds__(32 * kDqWarps, D == 128 || (MAPS == 2 && D == 64) ? 1 : 2)
    window_dq_mma_kernel(WinArgs a) {
  constexpr int DV = MAPS * D;
  constexpr bool BIAS = TAB != 0;
  extern __shared__ float sm[];
  __shared__ uint64_t full[kDqWarps], empty[kDqWarps];
  const int h = blockIdx.y, hk = h / (a.hq / a.hkv);
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, warp = threadIdx.x >> 5;
  const float mul = a.scale * kLog2e;
  const bool collect = BIAS && a.dbias;
  const int T3 = BIAS ? offsets(a.m) : 0, c0 = BIAS ? center(a.m) : 0;
  const float* tab = TAB == 2 ? a.tab2 + (size_t)h * T3 : sm;
  float* dtab = sm + (TAB == 1 ? T3 : 0);
  float* slots = dtab + (T3 + 3) / 4 * 4 + (TAB == 1 ? (4 - T3 % 4) % 4 : 0);
  if constexpr (BIAS) {
    for (int i = threadIdx.x; i < T3; i += blockDim.x) {
      if (TAB == 1) sm[i] = bias2_at(a, h, i);
      if (collect) dtab[i] = 0.f;
    }
    if (threadIdx.x < kDqWarps) {
      tc::mbar_init(&full[threadIdx.x], 1);
      tc::mbar_init(&empty[threadIdx.x], 1);
    }
    tc::fence_mbar_init();
    __syncthreads();
  }
  const int nc = collect ? kDqWarps - 1 : kDqWarps;  // computing warps
  if (collect && warp == nc) {
    uint32_t phase = 0;
    bool ok = true;
    for (int base = blockIdx.x * nc; base < a.T && ok; base += gridDim.x * nc)
      for (int w = 0; w < nc && base + w < a.T && ok; ++w) {
        const int4 tile = __ldg(&a.tiles[base + w]);
        const int nr = tile.y & (kDupFlag - 1);
        if (nr == 0) continue;
        const bool dup = tile.y & kDupFlag;
        const int cr = __ldg(&a.rows[tile.x + min(lane, nr - 1)].y) + c0;
        for (int k0 = tile.z; k0 < tile.w; k0 += kChunk) {
          Keys k;
          k.load(a.rows, k0, tile.w);
          ok = tc::mbar_wait_warp(&full[w], (phase >> w) & 1);
          if (!ok) break;
          phase ^= 1u << w;
          const float* slot = slots + w * kSlot;
          if (!dup) {
            const bool v0 = lane < k.n, v1 = lane + 32 < k.n;
            float d0[kTile], d1[kTile];
#pragma unroll
            for (int r = 0; r < kTile; ++r) d0[r] = slot[r * kSlotStride + lane], d1[r] = slot[r * kSlotStride + 32 + lane];
#pragma unroll
            for (int r = 0; r < kTile; ++r) {
              const int c = __shfl_sync(kFull, cr, r);
              if (r < nr) {
                float* p0 = dtab + c - k.code[0];
                float* p1 = dtab + c - k.code[1];
                const float x0 = v0 ? *p0 : 0.f, x1 = v1 ? *p1 : 0.f;
                if (v0) *p0 = x0 + d0[r];
                if (v1) *p1 = x1 + d1[r];
              }
              __syncwarp();
            }
          } else {
            for (int r = 0; r < nr; ++r) {
              const int c = __shfl_sync(kFull, cr, r);
              for (int i = 0; i < k.n; ++i) {
                if (lane == (i & 31)) dtab[c - k.code[i >> 5]] += slot[r * kSlotStride + i];
                __syncwarp();
              }
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&empty[w]);
        }
      }
    __syncwarp();
    if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    float* part = a.part + ((size_t)h * a.parts + blockIdx.x) * T3;
    for (int i = lane; i < T3; i += 32) part[i] = dtab[i];
    return;
  }
  float lam = 0.f;
  if constexpr (MAPS == 2) {
    float e1, e2;
    lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
    lam = e1 - e2 + a.lam_init;
  }
  const Rows<bf16, D> O = {static_cast<const bf16*>(a.dout), nullptr, a.hq, MAPS * h};
  const Rows<E, D> V = {static_cast<const E*>(a.v), a.sv, a.hkv, MAPS * hk};
  uint32_t phase = 1;  // the first wait on `empty` passes
  for (int t = blockIdx.x * nc + warp; t < a.T; t += gridDim.x * nc) {
    const int4 tile = __ldg(&a.tiles[t]);
    const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
    if (nr == 0) continue;
    const bool vg = g < nr, vg8 = g + 8 < nr;
    const int2 rg = __ldg(&a.rows[first + min(g, nr - 1)]), rg8 = __ldg(&a.rows[first + min(g + 8, nr - 1)]);
    const bool one = hi - lo <= kChunk;
    float m[MAPS][2], l[MAPS][2], dd[MAPS][2], acc[MAPS][D / 8][4];
#pragma unroll
    for (int u = 0; u < MAPS; ++u) {
      m[u][0] = m[u][1] = kNegInf, l[u][0] = l[u][1] = dd[u][0] = dd[u][1] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) acc[u][e][0] = acc[u][e][1] = acc[u][e][2] = acc[u][e][3] = 0.f;
    }
    Keys keys;
    float s[MAPS][8][4], dp[8][4];
    auto products = [&](int k0) {
      keys.load(a.rows, k0, hi);
#pragma unroll
      for (int u = 0; u < MAPS; ++u) {
        const Rows<E, D> Q = {static_cast<const E*>(a.q), a.sq, a.hq, MAPS * h + u};
        const Rows<E, D> K = {static_cast<const E*>(a.k), a.sk, a.hkv, MAPS * hk + u};
        uint32_t q[D / 16][4];
        load_a<D>(Q, rg.x, vg, rg8.x, vg8, q);
        contract_dim<D, 8>(q, K, keys.tok, keys.n, s[u]);
        finish_scores<BIAS>(s[u], keys, mul, tab, rg.y + c0, rg8.y + c0);
      }
      uint32_t o[DV / 16][4];
      load_a<DV>(O, rg.x, vg, rg8.x, vg8, o);
      contract_dim<DV, 8>(o, V, keys.tok, keys.n, dp);
    };
    // maximum, sum and sum of p dP of a row over the chunk; s becomes 2^(s - max)
    auto stats = [&](int u, int i) {
      float mx = m[u][i];
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(s[u][j][2 * i], s[u][j][2 * i + 1]));
      mx = quad_max(mx);
      const float ms = safe_max(mx), old = ex2(safe_max(m[u][i]) - ms);
      float e = 0.f, ed = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p = ex2(s[u][j][2 * i + x] - ms);
          s[u][j][2 * i + x] = p;
          e += p;
          if (8 * j + 2 * t4 + x < keys.n) ed = fmaf(p, dp[j][2 * i + x], ed);
        }
      l[u][i] = l[u][i] * old + quad_sum(e);
      dd[u][i] = dd[u][i] * old + quad_sum(ed);
      m[u][i] = mx;
    };
    if (!one)
      for (int k0 = lo; k0 < hi; k0 += kChunk) {
        products(k0);
#pragma unroll
        for (int u = 0; u < MAPS; ++u) stats(u, 0), stats(u, 1);
      }
    bool ok = true;
    for (int k0 = lo; k0 < hi; k0 += kChunk) {
      products(k0);
#pragma unroll
      for (int u = 0; u < MAPS; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (one) {
            stats(u, i);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int x = 0; x < 2; ++x) s[u][j][2 * i + x] = ex2(s[u][j][2 * i + x] - safe_max(m[u][i]));
          }
          const float inv = safe_inv(l[u][i]), dm = dd[u][i] * inv, f = u ? -lam * inv : inv;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              s[u][j][2 * i + x] =
                  8 * j + 2 * t4 + x < keys.n ? s[u][j][2 * i + x] * f * (dp[j][2 * i + x] - dm) : 0.f;
        }
      if (collect) {
        ok = tc::mbar_wait_warp(&empty[warp], phase);
        if (!ok) break;
        phase ^= 1;
        float* slot = slots + warp * kSlot;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(slot + (g + 8 * i) * kSlotStride + 8 * j + 2 * t4) =
                make_float2(s[0][j][2 * i], s[0][j][2 * i + 1]);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full[warp]);
      }
#pragma unroll
      for (int u = 0; u < MAPS; ++u) {
        const Rows<E, D> K = {static_cast<const E*>(a.k), a.sk, a.hkv, MAPS * hk + u};
        uint32_t f[4][4];
        pack_a<8>(s[u], f);
        contract_rows<D, 4>(f, K, keys.tok, keys.n, acc[u]);
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.status, kStatusTimeout);
      break;
    }
#pragma unroll
    for (int u = 0; u < MAPS; ++u) {
      store_acc<D, D>(static_cast<bf16*>(a.dq), a.hq, MAPS * h + u, rg.x, vg, rg8.x, vg8, acc[u], a.scale, a.scale);
      if (t4 == 0) {
        const size_t at = (size_t)(MAPS * h + u) * a.N + first + g;
        if (vg) a.lse2[at] = lse2_of(m[u][0], l[u][0]), a.D[at] = dd[u][0] * safe_inv(l[u][0]);
        if (vg8) a.lse2[at + 8] = lse2_of(m[u][1], l[u][1]), a.D[at + 8] = dd[u][1] * safe_inv(l[u][1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward: dk, dv
// ---------------------------------------------------------------------------

// A warp takes 16 keys of a cell and one key head: the transposed scores of the cell's queries, 32
// at a time, of every query head that reads the key head.
constexpr int kDkvWarps = 4;

template <int D, int MAPS, bool BIAS, typename E>
__global__ void __launch_bounds__(32 * kDkvWarps, D == 128 || (MAPS == 2 && D == 64) ? 2 : 3)
    window_dkv_mma_kernel(WinArgs a) {
  constexpr int DV = MAPS * D;
  const int G = a.hq / a.hkv, hk = blockIdx.y;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, warp = threadIdx.x >> 5;
  const float mul = a.scale * kLog2e;
  const int c0 = BIAS ? center(a.m) : 0, T3 = BIAS ? offsets(a.m) : 0;
  const int t = blockIdx.x * kDkvWarps + warp;
  if (t >= a.T) return;
  const int4 tile = __ldg(&a.tiles[t]);
  const int first = tile.x, nr = tile.y & (kDupFlag - 1), lo = tile.z, hi = tile.w;
  if (nr == 0) return;
  const bool vg = g < nr, vg8 = g + 8 < nr;
  const int2 rg = __ldg(&a.rows[first + min(g, nr - 1)]), rg8 = __ldg(&a.rows[first + min(g + 8, nr - 1)]);
  const Rows<E, D> V = {static_cast<const E*>(a.v), a.sv, a.hkv, MAPS * hk};
  float dk[MAPS][D / 8][4], dv[DV / 8][4];
#pragma unroll
  for (int u = 0; u < MAPS; ++u)
#pragma unroll
    for (int e = 0; e < D / 8; ++e) dk[u][e][0] = dk[u][e][1] = dk[u][e][2] = dk[u][e][3] = 0.f;
#pragma unroll
  for (int e = 0; e < DV / 8; ++e) dv[e][0] = dv[e][1] = dv[e][2] = dv[e][3] = 0.f;
  for (int k0 = lo; k0 < hi; k0 += 32) {
    const int n = min(32, hi - k0);
    const int2 qr = __ldg(&a.rows[k0 + min(lane, n - 1)]);
    const int tok[1] = {qr.x};
    for (int h = hk * G; h < hk * G + G; ++h) {
      float lam = 0.f;
      if constexpr (MAPS == 2) {
        float e1, e2;
        lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
        lam = e1 - e2 + a.lam_init;
      }
      const Rows<bf16, D> O = {static_cast<const bf16*>(a.dout), nullptr, a.hq, MAPS * h};
      float dp[4][4], pv[4][4];
      {
        uint32_t f[DV / 16][4];
        load_a<DV>(V, rg.x, vg, rg8.x, vg8, f);
        contract_dim<DV, 4>(f, O, tok, n, dp);
      }
#pragma unroll
      for (int u = 0; u < MAPS; ++u) {
        const Rows<E, D> Q = {static_cast<const E*>(a.q), a.sq, a.hq, MAPS * h + u};
        const Rows<E, D> K = {static_cast<const E*>(a.k), a.sk, a.hkv, MAPS * hk + u};
        float s[4][4];
        {
          uint32_t f[D / 16][4];
          load_a<D>(K, rg.x, vg, rg8.x, vg8, f);
          contract_dim<D, 4>(f, Q, tok, n, s);
        }
        const size_t at = (size_t)(MAPS * h + u) * a.N + k0 + min(lane, n - 1);
        const float lse2 = lane < n ? a.lse2[at] : kPosInf, dd = a.D[at];
        const float* tab = BIAS ? a.tab2 + (size_t)h * T3 : nullptr;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int q = 8 * j + 2 * t4 + x;
            const float L = __shfl_sync(kFull, lse2, q), Dq = __shfl_sync(kFull, dd, q);
            float b0 = 0.f, b1 = 0.f;
            if constexpr (BIAS) {
              const int cq = __shfl_sync(kFull, qr.y, q) + c0;
              b0 = __ldg(tab + cq - rg.y);
              b1 = __ldg(tab + cq - rg8.y);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float p = q < n ? ex2(fmaf(s[j][2 * i + x], mul, i ? b1 : b0) - L) : 0.f;
              const float w = u ? -lam * p : p;
              pv[j][2 * i + x] = u ? pv[j][2 * i + x] + w : w;
              s[j][2 * i + x] = q < n ? w * (dp[j][2 * i + x] - Dq) : 0.f;
            }
          }
        uint32_t f[2][4];
        pack_a<4>(s, f);
        contract_rows<D, 2>(f, Q, tok, n, dk[u]);
      }
      uint32_t f[2][4];
      pack_a<4>(pv, f);
      contract_rows<DV, 2>(f, O, tok, n, dv);
    }
  }
#pragma unroll
  for (int u = 0; u < MAPS; ++u)
    store_acc<D, D>(static_cast<bf16*>(a.dk), a.hkv, MAPS * hk + u, rg.x, vg, rg8.x, vg8, dk[u], a.scale, a.scale);
  store_acc<D, DV>(static_cast<bf16*>(a.dv), a.hkv, MAPS * hk, rg.x, vg, rg8.x, vg8, dv, 1.f, 1.f);
}

// tab2[h][o]: the bias of every offset in units of log2.
__global__ void bias_expand_kernel(WinArgs a) {
  const int T3 = offsets(a.m), o = blockIdx.x * blockDim.x + threadIdx.x;
  if (o < T3) a.tab2[(size_t)blockIdx.y * T3 + o] = bias2_at(a, blockIdx.y, o);
}

template <int D, int MAPS, bool BIAS, typename E>
cudaError_t bwd(const WinArgs& a, cudaStream_t st) {
  const size_t T3 = BIAS ? offsets(a.m) : 0;
  const size_t collect = a.dbias ? sizeof(float) * (T3 + 8 + (kDqWarps - 1) * kSlot) : 0;
  size_t smem = sizeof(float) * T3 + collect;
  auto dq = window_dq_mma_kernel<D, MAPS, BIAS ? 1 : 0, E>;
  if (BIAS && smem > kSmemMost) {
    dq = window_dq_mma_kernel<D, MAPS, BIAS ? 2 : 0, E>;
    smem = collect;
  }
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int heads = a.hq / MAPS, nc = a.dbias ? kDqWarps - 1 : kDqWarps;
  const int need = (a.T + nc - 1) / nc;
  int gx = a.dbias ? a.parts : (4 * 2 * 148 + heads - 1) / heads;
  gx = !a.dbias && gx > need ? need : gx;
  if (BIAS)
    SSA_LAUNCH("bias_expand_kernel", bias_expand_kernel, dim3(((int)T3 + 255) / 256, a.hq), 256, 0, st, a);
  SSA_LAUNCH("window_dq_mma_kernel", dq, dim3(gx, heads), 32 * kDqWarps, smem, st, a);
  auto dkv = window_dkv_mma_kernel<D, MAPS, BIAS, E>;
  SSA_LAUNCH("window_dkv_mma_kernel", dkv, dim3((a.T + kDkvWarps - 1) / kDkvWarps, a.hkv / MAPS), 32 * kDkvWarps, 0,
             st, a);
  return cudaGetLastError();
}

template <typename E>
cudaError_t bwd_e(const WinArgs& a, cudaStream_t st) {
  if (a.maps == 2) return a.d == 32 ? bwd<32, 2, false, E>(a, st) : bwd<64, 2, false, E>(a, st);
  if (a.table)
    return a.d == 32   ? bwd<32, 1, true, E>(a, st)
           : a.d == 64 ? bwd<64, 1, true, E>(a, st)
                       : bwd<128, 1, true, E>(a, st);
  return a.d == 32   ? bwd<32, 1, false, E>(a, st)
         : a.d == 64 ? bwd<64, 1, false, E>(a, st)
                     : bwd<128, 1, false, E>(a, st);
}

}  // namespace

cudaError_t window_bwd_mma(const WinArgs& a, cudaStream_t st) {
  return a.act8 ? bwd_e<int8_t>(a, st) : bwd_e<bf16>(a, st);
}

cudaError_t window_fwd_mma(const WinArgs& a, cudaStream_t st) {
  if (a.maps == 2) return a.d == 32 ? fwd<32, 2, false>(a, st) : fwd<64, 2, false>(a, st);
  if (a.table)
    return a.d == 32 ? fwd<32, 1, true>(a, st) : a.d == 64 ? fwd<64, 1, true>(a, st) : fwd<128, 1, true>(a, st);
  return a.d == 32 ? fwd<32, 1, false>(a, st) : a.d == 64 ? fwd<64, 1, false>(a, st) : fwd<128, 1, false>(a, st);
}

}  // namespace ssa
