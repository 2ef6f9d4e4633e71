// Plan of the window operators, the sums of their parameter gradients, and 8-bit checkpoints.
#include "window.cuh"

namespace ssa {
namespace {

using namespace win;

// One thread per row (position in cell order): its token and offset code, and, from the first
// row of every 16 of a cell, the tile.  Tile slots need no scan: cell c takes the slots from
// ptr[c] / 16 + c on; floor(b / 16) - floor(a / 16) + 1 >= ceil((b - a) / 16) of them.  Made once per
// voxel set, so latency alone counts here.
__global__ void plan_rows_kernel(const int32_t* __restrict__ coords, int64_t N, int64_t W, int m,
                                 const int32_t* __restrict__ id, const int32_t* __restrict__ perm,
                                 const int32_t* __restrict__ ptr, int2* __restrict__ rows, int4* __restrict__ tiles,
                                 int* status) {
  for (int64_t pos = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; pos < N;
       pos += (int64_t)gridDim.x * blockDim.x) {
    const int tok = perm[pos];
    bool ok = (unsigned)tok < (unsigned)N;
    const int c = ok ? id[tok] : 0;
    ok = ok && (unsigned)c < (unsigned)W;
    const int a = ok ? ptr[c] : 0, b = ok ? ptr[c + 1] : 0;
    ok = ok && a >= 0 && a <= pos && pos < b && b <= N;
    if (!ok) {
      rows[pos] = make_int2(0, 0);
      atomicOr(status, kStatusSelection);
      continue;
    }
    int code = 0;
    if (coords) {
      const int e = 2 * m - 1;
      int x[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int r = coords[3 * (int64_t)tok + i] % m;
        x[i] = r < 0 ? r + m : r;
      }
      code = (x[0] * e + x[1]) * e + x[2];
    }
    rows[pos] = make_int2(tok, code);
    if ((pos - a) % kTile == 0) {
      const int n = (int)(b - pos < kTile ? b - pos : kTile);
      tiles[a / kTile + c + (pos - a) / kTile] = make_int4((int)pos, n, a, b);
    }
  }
}

// One warp per cell: the most tokens that one of its m^3 voxels holds (m <= 16, 16-bit counters,
// so no more than 65535; a larger count can only come from as many tokens in the cell, which is
// then taken instead).  Where it is above one the cell's tiles carry it; tiles[T].x: the maximum of
// all cells.
__global__ void plan_dup_kernel(int64_t N, int64_t W, int m, const int32_t* __restrict__ ptr,
                                const int2* __restrict__ rows, int4* __restrict__ tiles, int64_t T) {
  __shared__ uint32_t count[4][2048];  // two voxels to a word
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = 2 * m - 1, words = (m * m * m + 1) / 2;
  for (int64_t c = (int64_t)blockIdx.x * 4 + warp; c < W; c += (int64_t)gridDim.x * 4) {
    const int a = ptr[c], b = ptr[c + 1];
    if (a < 0 || b > N || b <= a) continue;  // reported by plan_rows_kernel
    int most = b - a;
    if (most > 1 && most <= 65535) {
      for (int i = lane; i < words; i += 32) count[warp][i] = 0;
      __syncwarp();
      most = 0;
      for (int i = a + lane; i < b; i += 32) {
        const int code = rows[i].y;
        const int v = (code / (e * e) * m + code / e % e) * m + code % e, sh = 16 * (v & 1);
        most = max(most, (int)((atomicAdd(&count[warp][v >> 1], 1u << sh) >> sh) & 65535u) + 1);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      __syncwarp();
    }
    if (lane == 0) atomicMax(&tiles[T].x, most);
    if (most > 1) {
      const int64_t slot = a / kTile + c, nt = (b - a + kTile - 1) / kTile;
      for (int64_t i = lane; i < nt; i += 32) tiles[slot + i].y |= kDupFlag + kDupUnit * min(most, kDupTop);
    }
  }
}

// dst[h][o] = sum over parts of part[h][i][o], in a fixed order, and of the 64-bit sums where cells or
// the whole gradient (a.wide) went there; NaN where the head's dP or softmax had no finite bound (the
// parts are NaN then).  dst may be part i = 0.  Reads the parts once out of L2, eight loads in flight:
// 11 us for 27 parts of 32 heads at an edge of 8 (11.7 MB), latency of the chain of adds.
__global__ void bias_parts_kernel(WinArgs a, float* dst, int pitch) {
  const int T3 = offsets(a.m), o = blockIdx.x * blockDim.x + threadIdx.x, h = blockIdx.y;
  if (o >= T3) return;
  const float* p = a.part + (size_t)h * a.parts * T3 + o;
  float s = 0.f;
  const int parts = a.wide ? 0 : a.parts;
  int i = 0;
  for (; i + 8 <= parts; i += 8) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[(size_t)(i + j) * T3];
#pragma unroll
    for (int j = 0; j < 8; ++j) s += x[j];
  }
  for (; i < parts; ++i) s += p[(size_t)i * T3];
  if (a.sums && (a.wide || __ldg(&a.tiles[a.T].x) > kDupMost)) {
    const uint32_t amax = a.amax[h];
    s += (float)ldexp((double)(long long)a.sums[(size_t)h * T3 + o], -wide_bits(amax, a.N));
    if (amax >= kTopDp) s = __uint_as_float(0x7fc00000u);
  }
  dst[(size_t)h * pitch + o] = s;
}

// dbias[h][b] = sum of the offsets o with bucket b, in a fixed order; one warp per bucket and head:
// it reads all offsets' buckets, so that no list of a bucket's offsets is needed: 18 us at an edge of 8,
// 343 buckets, 16 heads.  The reads grow with buckets times offsets: an explicit map with a bucket for
// every offset takes 99 us at an edge of 8 and 6.6 ms at 16 (32 heads); without a map there is no launch.
__global__ void bias_buckets_kernel(const float* __restrict__ sums, int pitch, int T, const int32_t* __restrict__ bucket,
                                    int nb, float* __restrict__ dbias) {
  const int b = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= nb) return;
  const float* p = sums + (size_t)blockIdx.y * pitch;
  float s = 0.f;
#pragma unroll 4
  for (int o = lane; o < T; o += 32)
    if (__ldg(bucket + o) == b) s += p[o];
#pragma unroll
  for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
  if (lane == 0) dbias[(size_t)blockIdx.y * nb + b] = s;
}

// dlambda of a head = -sum of D of its second map; then the chain rule through
// lambda = exp(<x0, x1>) - exp(<x2, x3>) + init.  One block per head, fixed order, fp64 sums
// (18 us for 16 pairs of 131072 rows: 8 MB read by 16 blocks, each bound by its own loads).
constexpr int kLamThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kLamThreads) lam_grad_kernel(const float* __restrict__ lam, const float* __restrict__ Drow, int64_t N, int heads,
                                float* __restrict__ dlam) {
  __shared__ double red[kLamThreads];
  const int h = blockIdx.x, t = threadIdx.x;
  const float* p = Drow + (size_t)(2 * h + 1) * N;
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = t; i < N; i += kLamThreads) s += (double)p[i];
  red[t] = s;
  __syncthreads();
  for (int o = kLamThreads / 2; o; o >>= 1) {
    if (t < o) red[t] += red[t + o];
    __syncthreads();
  }
  const float dl = (float)-red[0];
  float e1, e2;
  lambda_terms<D>(lam, heads, h, e1, e2);
  const size_t st = (size_t)heads * D, at = (size_t)h * D + t;
  if (t < D) {
    dlam[at] = dl * e1 * lam[st + at];
    dlam[st + at] = dl * e1 * lam[at];
    dlam[2 * st + at] = -dl * e2 * lam[3 * st + at];
    dlam[3 * st + at] = -dl * e2 * lam[2 * st + at];
  }
}

// ---------------------------------------------------------------------------
// 8-bit checkpoints
// ---------------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                            pack_bf16x2(x[6], x[7]));
}

// Packing: 2^sh = d / 16 lanes per row, 16 values each, two rounds in flight per thread; unpacking: d / 8
// lanes, 8 values, kGroups rounds.  Bound by HBM; with one round at a time a round's loads waited for the
// stores of the one before.  Q, K, V of 131072 tokens (32/2 heads of 64, 925 MB to move either way):
// 202 us packing (70% of the measured copy bandwidth; 234 us with 8 values a lane, whose codes are half
// a lane's widest store), 175 us unpacking (81%); 465 us together with one round of 8 values.  Packing
// takes the codes out of the low bits of a float sum, which costs fewer instructions than a conversion,
// a clamp and a shift for each (247 -> 234 us).
// The step is the smallest power of two s >= 2^-126 with top <= 127 s: with top = f 2^e, f in [1, 2),
// s = 2^(e - 6) while f <= 127 / 64, else 2^(e - 5).
constexpr int kGroups = 4;

template <typename T>
__global__ void act8_pack_kernel(const T* __restrict__ x, int64_t groups, int sh, int8_t* __restrict__ codes,
                                 float* __restrict__ scale) {
  constexpr int G = 2;  // rounds in flight, of 16 values a lane
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 - (threadIdx.x & 31) < groups;
       i0 += G * stride) {
    float v[G][16];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (i0 + g * stride < groups) {
        load8<T>(x + 16 * (i0 + g * stride), v[g]);
        load8<T>(x + 16 * (i0 + g * stride) + 8, v[g] + 8);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[g][j] = 0.f;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t i = i0 + g * stride;
      uint32_t top = 0;  // of the magnitudes' bits: NaN and infinity come out on top
#pragma unroll
      for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(v[g][j]) & 0x7fffffffu);
      for (int o = 1 << sh >> 1; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      int e = (int)(top >> 23);  // biased exponent; 0 for zero and subnormal rows
      e = e - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
      e = e < 1 ? 1 : e;
      const bool bad = top >= 0x7f800000u;
      const float s = bad ? __uint_as_float(0x7fc00000u) : top == 0 ? 1.f : __uint_as_float((uint32_t)e << 23);
      // codes above 63 with s = 2^122 would stand for an infinity
      const float limit = e == 249 ? 63.f * __uint_as_float(249u << 23) : __uint_as_float(0x7f7fffffu);
      const float r = bad || top == 0 ? 0.f : __uint_as_float((uint32_t)(254 - e) << 23);  // 1 / s
      if (i < groups) {
        // the nearest whole number is in the low bits of v / s + 1.5 2^23 (v / s is exact, so the sum
        // is rounded once, ties to even)
        uint32_t n[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          n[j] = bad ? 0u : __float_as_uint(fmaf(fminf(fmaxf(v[g][j], -limit), limit), r, 12582912.f));
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = __byte_perm(__byte_perm(n[4 * j], n[4 * j + 1], 0x0040), __byte_perm(n[4 * j + 2], n[4 * j + 3], 0x0040),
                             0x5410);
        reinterpret_cast<uint4*>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        if ((i & ((1 << sh) - 1)) == 0) scale[i >> sh] = s;
      }
    }
  }
}

template <typename T>
__global__ void act8_unpack_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scale, int64_t groups,
                                   int sh, T* __restrict__ x) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < groups; i0 += kGroups * stride) {
    uint2 w[kGroups];
    float s[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t i = min(i0 + g * stride, groups - 1);
      w[g] = __ldg(reinterpret_cast<const uint2*>(codes) + i);
      s[g] = __ldg(scale + (i >> sh));
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int64_t i = i0 + g * stride;
      if (i >= groups) break;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? w[g].x : w[g].y) >> (8 * (j & 3))) * s[g];
      store8(x + 8 * i, v);
    }
  }
}

int blocks_for(int64_t threads, int per_block) {
  const int64_t b = (threads + per_block - 1) / per_block;
  return (int)(b < 148 * 16 ? (b > 0 ? b : 1) : 148 * 16);
}

}  // namespace

cudaError_t window_plan(const int32_t* coords, int64_t N, int m, const ssa_partition* part, int2* rows, int4* tiles,
                        int* status, cudaStream_t st) {
  const int64_t T = N / kTile + part->count;
  cudaError_t e = cudaMemsetAsync(tiles, 0, sizeof(int4) * (T + 1), st);
  if (e != cudaSuccess) return e;
  SSA_LAUNCH("plan_rows_kernel", plan_rows_kernel, blocks_for(N, 256), 256, 0, st, coords, N, part->count, m, part->id,
             part->perm, part->ptr, rows, tiles, status);
  if (coords)
    SSA_LAUNCH("plan_dup_kernel", plan_dup_kernel, blocks_for(part->count, 4), 128, 0, st, N, part->count, m,
               part->ptr, rows, tiles, T);
  return cudaGetLastError();
}

cudaError_t window_param_grads(const WinArgs& a, cudaStream_t st) {
  if (a.dbias) {
    const int T = offsets(a.m);
    // every offset its own bucket: the sums are the gradient
    float* sums = a.bucket ? a.part : a.dbias;
    const int pitch = a.bucket ? a.parts * T : T;
    SSA_LAUNCH("bias_parts_kernel", bias_parts_kernel, dim3((T + 127) / 128, a.hq), 128, 0, st, a, sums, pitch);
    if (a.bucket)
      SSA_LAUNCH("bias_buckets_kernel", bias_buckets_kernel, dim3((a.nb + 7) / 8, a.hq), 256, 0, st, a.part, pitch, T,
                 a.bucket, a.nb, a.dbias);
  }
  if (a.dlam) {
    auto kern = a.d == 32 ? lam_grad_kernel<32> : lam_grad_kernel<64>;
    SSA_LAUNCH("lam_grad_kernel", kern, a.hq / 2, kLamThreads, 0, st, a.lam, a.D, a.N, a.hq / 2, a.dlam);
  }
  return cudaGetLastError();
}

cudaError_t act8_pack(int dtype, int64_t rows, int d, const void* x, int8_t* codes, float* scale, cudaStream_t st) {
  const int64_t g = rows * (d / 16);
  const int sh = d == 32 ? 1 : d == 64 ? 2 : 3;
  if (dtype == SSA_DTYPE_BF16)
    SSA_LAUNCH("act8_pack_kernel", act8_pack_kernel<__nv_bfloat16>, blocks_for((g + 1) / 2, 256), 256, 0, st,
               static_cast<const __nv_bfloat16*>(x), g, sh, codes, scale);
  else
    SSA_LAUNCH("act8_pack_kernel", act8_pack_kernel<float>, blocks_for((g + 1) / 2, 256), 256, 0, st,
               static_cast<const float*>(x), g, sh, codes, scale);
  return cudaGetLastError();
}

cudaError_t act8_unpack(int dtype, int64_t rows, int d, const int8_t* codes, const float* scale, void* x,
                        cudaStream_t st) {
  const int64_t g = rows * (d / 8);
  const int sh = d == 32 ? 2 : d == 64 ? 3 : 4;
  if (dtype == SSA_DTYPE_BF16)
    SSA_LAUNCH("act8_unpack_kernel", act8_unpack_kernel<__nv_bfloat16>, blocks_for((g + kGroups - 1) / kGroups, 256), 256, 0, st, codes, scale,
               g, sh, static_cast<__nv_bfloat16*>(x));
  else
    SSA_LAUNCH("act8_unpack_kernel", act8_unpack_kernel<float>, blocks_for((g + kGroups - 1) / kGroups, 256), 256, 0, st, codes, scale, g, sh,
               static_cast<float*>(x));
  return cudaGetLastError();
}

}  // namespace ssa
