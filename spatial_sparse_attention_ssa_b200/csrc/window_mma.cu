// Attention inside the cells on warp-level tensor-core MMAs (mma.sync m16n8k16, bf16 operands,
// fp32 sums).  See window.cuh for the mathematics and the meaning of MAPS.
//
// A CTA keeps one head, or two that share a key head (their bias tables lie in shared memory while they
// fit), and walks cells.  The keys of the cells, 64 at a time, go through a ring of stages in shared
// memory that two warps fill ahead (cp.async, completion on an mbarrier); the cell's rows, 16 at a time,
// go to the other warps in turn, so no warp waits for another but through the ring.  Scores never leave
// registers: a step is 16 rows by 32 keys.  Tiles of 128 rows on tcgen05 are not tried here.  Of one head
// and a cell of some 50 tokens they would stand half empty, but with rows of several heads that share a
// key head, as win_tc.cu packs them, or on cells of hundreds of tokens they would not; that kernel reaches
// 80 TFLOP/s of products on a shell of 131072 tokens (its hand-offs per item bind it), this forward 80.
//
// What bounds these kernels is instruction issue and its latencies: of some 330 instructions of a
// forward step 32 are products, the rest the bias, the mask, the exponential and the sums; and a tile
// of 16 rows costs some 500 before its first and after its last step, which cells of 47 tokens (1.9
// steps a tile) do not spread.  32768 tokens (32/2 heads of 64, edge 8; forward, statistics, dq,
// dk/dv): issue slots used 46, 48, 43, 39%, tensor pipe 19, 18, 20, 39%, shared memory 50, 43, 58,
// 59%, HBM below 20%.  Times at 131072 tokens, and the TFLOP/s of the products alone (31.3 GFLOP each):
// forward 787 us (80), statistics 808 us (77), dq with dbias 1325 us (71), dk/dv 887 us (141);
// differential 1171, 709, 1035, 963 us; full cube of 24576, 16/2 heads of 128: 390, 414, 656, 571 us.
#include "tc.cuh"
#include "window.cuh"

namespace ssa {
namespace {

using namespace win;
using bf16 = __nv_bfloat16;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kChunk = 64;
constexpr float kSlack = 8.f;

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same onto zeros
__device__ __forceinline__ void mma0(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// four 8x8 b16 matrices; lane l gives the address of row l % 8 of matrix l / 8
__device__ __forceinline__ void ldsm(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
// 16 bytes to shared memory, zeros where `on` is off
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// one arrival on the barrier when this thread's copies so far have landed
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// Waits for a phase, asleep between the looks: polling warps would take issue slots from the working
// ones.  Gives up after the time of tc::mbar_wait.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(kFull, tc::mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = tc::global_ns();
  for (uint32_t i = 1;; ++i) {
    __nanosleep(i < 4 ? 40 : 100);
    if (__all_sync(kFull, tc::mbar_try_wait(bar, parity))) return true;
    if ((i & 255u) == 0 && __any_sync(kFull, tc::global_ns() - t0 > tc::kWaitLimitNs)) return false;
  }
}
__device__ __forceinline__ void prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}

// Rows of a tensor [n, heads, D] from head `head` on.
struct Rows {
  const void* p;
  int heads, head;
};

// Shared-memory tiles of rows of W bf16 (16-byte units c): the unit's place is permuted by the row
// so that eight rows of one unit (ldmatrix) fall into different banks.
template <int W>
__device__ __forceinline__ uint32_t unit(int row, int c) {
  constexpr int U = W / 8;
  const int f = W == 32 ? (row >> 1) & 3 : row & 7;
  return 16u * (uint32_t)(row * U + (c ^ f));
}

// Address of unit e + c (e even, c 0 or 1) of a row of a staged tile: units that differ in e differ by
// an exclusive or, one instruction for the place of the first (tiles lie on multiples of 128 bytes,
// so up to eight units to a row its bits are those of the unit alone).
template <int W, bool XOR = true>
__device__ __forceinline__ uint32_t unit_pair(uint32_t tile, int row, int c, int e) {
  if (!XOR) return tile + unit<W>(row, e + c);
  const uint32_t first = unit<W>(row, c);
  return W <= 64 ? (tile + first) ^ (16u * e) : tile + (first ^ (16u * e));
}

// Rows first .. first + n - 1 (n <= ROWS) of the cell order to a staged tile of ROWS rows, zeros past
// n, by THREADS threads; one or two tensors of the same heads at once.  Unrolled: a unit costs its
// copy, its address and little else.
template <int D, int W, int ROWS, int THREADS, bool TWO>
__device__ __forceinline__ void stage(uint32_t dst, const Rows& src, uint32_t dst2, const Rows& src2,
                                      const int2* __restrict__ rows, int first, int n, int tid) {
  constexpr int U = W / 8, STEP = THREADS / U, IT = ROWS / STEP;
  static_assert(ROWS % STEP == 0, "whole steps");
  const int r = tid / U, c = tid % U;
  int tok[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) tok[i] = __ldg(&rows[first + min(i * STEP + r, n - 1)].x);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = i * STEP + r;
    const size_t at = ((size_t)tok[i] * src.heads + src.head) * D + 8 * c;
    cp16(dst + unit<W>(k, c), static_cast<const bf16*>(src.p) + at, k < n);
    if constexpr (TWO) cp16(dst2 + unit<W>(k, c), static_cast<const bf16*>(src2.p) + at, k < n);
  }
}

// A operand, k-step k, from a tile of 16 rows starting at row r0 of a staged tile.
template <int W, bool XOR = true>
__device__ __forceinline__ void load_a(uint32_t* f, uint32_t tile, int r0, int k) {
  const int lane = threadIdx.x & 31;
  ldsm(f, unit_pair<W, XOR>(tile + r0 * W * 2, lane & 15, lane >> 4, 2 * k));
}

// s[2 k], s[2 k + 1] = A B^T for the 16 rows 16 k .. of B, k < NK: W columns from unit u0 of a
// staged tile of PW columns; A as fragments, or (below) W columns from unit a0 of a staged tile of
// 16 rows, read for the occasion.
template <int PW, int W, int NK, bool XOR = true>
__device__ __forceinline__ void contract_step(const uint32_t* a, int d, uint32_t tile, int u0, float (*s)[4]) {
  const int lane = threadIdx.x & 31, row = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    uint32_t b[4];
    ldsm(b, unit_pair<PW, XOR>(tile, row, c, u0 + 2 * d) + k * 32 * PW);
    if (d == 0) {
      mma0(s[2 * k], a, b[0], b[1]);
      mma0(s[2 * k + 1], a, b[2], b[3]);
    } else {
      mma(s[2 * k], a, b[0], b[1]);
      mma(s[2 * k + 1], a, b[2], b[3]);
    }
  }
}
template <int PW, int W, int NK, bool XOR = true>
__device__ __forceinline__ void contract_dim(const uint32_t (*a)[4], uint32_t tile, int u0, float (*s)[4]) {
#pragma unroll
  for (int d = 0; d < W / 16; ++d) contract_step<PW, W, NK, XOR>(a[d], d, tile, u0, s);
}
template <int PW, int W, int NK>
__device__ __forceinline__ void contract_dim(uint32_t atile, int a0, uint32_t tile, int u0, float (*s)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 0; d < W / 16; ++d) {
    uint32_t a[4];
    ldsm(a, unit_pair<PW>(atile, lane & 15, lane >> 4, a0 + 2 * d));
    contract_step<PW, W, NK>(a, d, tile, u0, s);
  }
}

// acc_h += P_h B for h < NA, P_h as A fragments over NK groups of 16 rows of B (as above).
template <int PW, int W, int NK, int NA = 1, bool XOR = true>
__device__ __forceinline__ void contract_rows(const uint32_t (*p)[4], uint32_t tile, int u0, float (*acc)[4]) {
  const int lane = threadIdx.x & 31, row = lane & 15, c = lane >> 4;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
#pragma unroll
    for (int e = 0; e < W / 16; ++e) {
      uint32_t b[4];
      ldsm_t(b, unit_pair<PW, XOR>(tile, row, c, u0 + 2 * e) + k * 32 * PW);
#pragma unroll
      for (int h = 0; h < NA; ++h) {
        mma(acc[h * (W / 8) + 2 * e], p[h * NK + k], b[0], b[1]);
        mma(acc[h * (W / 8) + 2 * e + 1], p[h * NK + k], b[2], b[3]);
      }
    }
  }
}

// Accumulators (16 rows of W) times f (rows g) and f8 (rows g + 8), rounded to bf16, through the
// warp's scratch tile to rows first .. first + nr - 1.
template <int D, int W>
__device__ __forceinline__ void store_acc(uint32_t scratch, float (*acc)[4], float f, float f8, bf16* out, int heads,
                                          int head, const int2* __restrict__ rows, int first, int nr) {
  constexpr int U = W / 8;
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int e = 0; e < W / 16; ++e)
    stsm(scratch + unit<W>(lane & 15, 2 * e + (lane >> 4)), pack_bf16x2(acc[2 * e][0] * f, acc[2 * e][1] * f),
         pack_bf16x2(acc[2 * e][2] * f8, acc[2 * e][3] * f8), pack_bf16x2(acc[2 * e + 1][0] * f, acc[2 * e + 1][1] * f),
         pack_bf16x2(acc[2 * e + 1][2] * f8, acc[2 * e + 1][3] * f8));
  __syncwarp();
  const int r0 = lane / U, c = lane % U;
  int tok[U / 2];
#pragma unroll
  for (int i = 0; i < U / 2; ++i) tok[i] = __ldg(&rows[first + min(r0 + i * (32 / U), nr - 1)].x);
#pragma unroll
  for (int i = 0; i < U / 2; ++i) {
    const int r = r0 + i * (32 / U);
    if (r < nr)
      *reinterpret_cast<uint4*>(out + ((size_t)tok[i] * heads + head) * D + 8 * c) = lds16(scratch + unit<W>(r, c));
  }
}

// Scores of NT n-tiles as A fragments (rounded to bf16).
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

// A place in a head's table of offsets, in shared or in global memory; its neighbours by bytes.  The
// codes of a stage are held times four, so that a lookup costs one subtraction and the load.
template <bool SHARED>
struct Place {
  uint32_t p;
  __device__ __forceinline__ float at(int off) const {
    float v;
    asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p + off));
    return v;
  }
};
template <>
struct Place<false> {
  const char* p;
  __device__ __forceinline__ float at(int off) const { return __ldg(reinterpret_cast<const float*>(p + off)); }
};
__device__ __forceinline__ void red_shared(uint32_t at, int x) {
  asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(at), "r"(x));
}

// The bias gradient in fixed point.  A CTA keeps two whole numbers per offset: dS 2^s rounded, and
// what that rounding left times 2^k, rounded; both are added by native integer atomics in shared
// memory, whose order cannot change the sums.  Bounds: the |dS| of a row sum to at most 2 M, M the
// largest |dP| of the head (from the row statistics, a.amax), so 2^s <= 2^29 / (2 M rows) keeps the
// first (a rounding at most doubles a number that it does not make 0); each remainder is at most 1/2,
// so 2^k <= 2^31 / (adds per offset) keeps the second, adds = rows times the most tokens that a voxel
// of their cell holds.  Both stay below 2^13: before they pass it the CTA's sums go to its partial
// gradient and start again, so the unit is at most M 2^-33 however many rows a CTA has; a batch alone
// between two flushes counts its own (M 2^-41 for few rows).  An item of one crowded cell can pass the
// bound alone: below 2^19 adds (some thousand tokens in a voxel) its unit is M 2^-32, where dS is some
// M 2^-12; cells that are more crowded (kCrowd) take the 64-bit sums below (8/2 heads of 64: a voxel of
// 20000 tokens 43 -> 50 ms; from 2048 tokens on, four such voxels of 2500 in a cell took 36 ms, now 5).  A NaN or an infinity in dP or in a softmax makes
// the head's gradient NaN, and so does an M from 2^127 on (dP - D could overflow); below, 2^s and 2^-s are
// normal numbers.
constexpr int kAdds = 8191;      // at most between two flushes, but for a lone item
constexpr int kLone = 1 << 19;   // and for a lone item
constexpr int kCrowd = 1 << 16;  // items[].y: a cell for the 64-bit sums
struct Limbs {
  float s[2], k;         // 2^s for the rows g, g + 8 (times far_factor, see store_lse2), 2^k
  double unit, unit_lo;  // 2^-s, 2^-s-k
  __device__ __forceinline__ void set(const WinArgs& a, int h, int rows, int adds) {
    const uint32_t bits = __ldg(a.amax + h);
    const int rb = 32 - __clz(rows), ab = 32 - __clz(adds);  // rows < 2^rb, adds < 2^ab
    const int e = (int)(bits >> 23) - 126;                      // M < 2^e
    int sb = min(29 - rb - 1 - e, 20 - e);                      // |dS 2^s| < 2^22: see add()
    sb = max(-126, min(126, sb));
    const int kbits = max(0, min(21, 31 - ab));
    s[0] = s[1] = __uint_as_float(bits >= kTopDp ? 0x7fc00000u : (uint32_t)(sb + 127) << 23);
    k = (float)(1 << kbits);
    unit = (double)(1.f / s[0]);
    unit_lo = unit * (double)(1.f / k);
  }
  __device__ __forceinline__ float value(int hi, int lo) const {
    return (float)((double)hi * unit + (double)lo * unit_lo);
  }
  // x 2^s to the nearest whole number by adding 1.5 2^23 (|x 2^s| < 2^22), and the rest
  __device__ __forceinline__ void add(uint32_t hi, uint32_t lo, float x, int row) const {
    constexpr float kMagic = 12582912.f;
    const float a = fmaf(x, s[row], kMagic);
    const float r = fmaf(x, s[row], kMagic - a);
    const float b = fmaf(r, k, kMagic);
    red_shared(hi, __float_as_int(a) - __float_as_int(kMagic));
    red_shared(lo, __float_as_int(b) - __float_as_int(kMagic));
  }
};

// Edges whose two tables do not fit beside the ring, and cells with a crowded voxel: one 64-bit number
// per offset in global memory (wide_bits).
struct Wide {
  char* sums;  // of the head
  double s;
  float c[2];  // far_factor of the rows g, g + 8
  __device__ __forceinline__ void set(const WinArgs& a, int h) {
    c[0] = c[1] = 1.f;
    sums = reinterpret_cast<char*>(a.sums + (size_t)h * offsets(a.m));
    s = __longlong_as_double((long long)(wide_bits(__ldg(a.amax + h), a.N) + 1023) << 52);
  }
  __device__ __forceinline__ long long whole(float x, int row) const { return __double2ll_rn((double)(x * c[row]) * s); }
  // at: four times the offset
  __device__ __forceinline__ void add(int at, float x, int row) const { add_ll(at, whole(x, row)); }
  __device__ __forceinline__ void add_ll(int at, long long x) const {
    atomicAdd(reinterpret_cast<unsigned long long*>(sums + 2 * (int64_t)at), (unsigned long long)x);
  }
};

// add(4 (code of row - code of key), dS, 0 for the row g, 1 for g + 8) for a fragment tile of 16 rows and 32
// positions.  Rows and positions without a token have dS 0 and the codes of others.
template <typename F>
__device__ __forceinline__ void add_bias_grad(const F& add, float (*ds)[4], const int* codes, int ci, int ci8) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int2 cj = *reinterpret_cast<const int2*>(codes + 8 * j + 2 * t);
#pragma unroll
    for (int x = 0; x < 4; ++x) add((x & 2 ? ci8 : ci) - (x & 1 ? cj.y : cj.x), ds[j][x], x >> 1);
  }
}

// The same for a cell with a crowded voxel: a step whose rows and positions all lie in one voxel adds its
// 512 numbers up first, since their atomics would queue for one address.  Not inlined: it would stand in
// the way of the instructions of every step (dq of 131072 tokens: inlined 1536 us, called 1490).
__device__ __noinline__ void add_crowded(Wide wide, const float (*v)[4], const int* codes, int ci, int ci8) {
  float ds[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int x = 0; x < 4; ++x) ds[j][x] = v[j][x];
  const int lane = threadIdx.x & 31, code = codes[lane];
  const int code0 = __shfl_sync(kFull, code, 0), ci0 = __shfl_sync(kFull, ci, 0);  // by every lane
  if (__all_sync(kFull, code == code0 && ci == ci0 && ci8 == ci0)) {
    long long sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) sum += wide.whole(ds[j][x], x >> 1);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) wide.add_ll(ci - code, sum);
  } else {
    add_bias_grad([&](int at, float x, int row) { wide.add(at, x, row); }, ds, codes, ci, ci8);
  }
  __syncwarp();
}

// The keys of a chunk stand in shared memory in another order than in the cell: position
// 8 j + 2 t + x of 32 holds key 8 t + 2 j + x, so that the four lanes that share a row in a
// fragment (t) hold keys eight apart.  Neighbours in the cell are neighbours in the voxel grid, so
// without this such lanes would often hit one offset in one instruction (see add_bias_grad).
// (The map is its own inverse.)
__device__ __forceinline__ int key_at(int p) { return (p & 33) | (p & 6) << 2 | (p & 24) >> 2; }

// s = s mul + bias in units of log2 for the 32 positions of a half chunk, minus infinity where
// the key is not below `left`.  t0, t8: the head's table of offsets at the codes of rows g, g + 8
// (plus the center); codes: four times those of the positions (shared memory).
template <bool BIAS, typename P>
__device__ __forceinline__ void finish_scores(float (*s)[4], const int* codes, int left, float mul, const P& t0,
                                              const P& t8) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (BIAS) {
      const int2 cj = *reinterpret_cast<const int2*>(codes + 8 * j + 2 * t);
      b[0] = t0.at(-cj.x), b[1] = t0.at(-cj.y), b[2] = t8.at(-cj.x), b[3] = t8.at(-cj.y);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) s[j][x] = fmaf(s[j][x], mul, b[x]);
  }
  if (left < 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[j][x] = 8 * t + 2 * j + (x & 1) < left ? s[j][x] : kNegInf;
  }
}

// Number of tiles of the item (up to `size` row tiles of a cell, which take the cell's keys from one
// passage of the ring) that starts at a slot: 0 for empty slots and those inside an item.
__device__ __forceinline__ int item_tiles(const int4& tile, int size) {
  if ((tile.y & (kDupFlag - 1)) == 0) return 0;
  const int at = (unsigned)(tile.x - tile.z) / kTile, all = (unsigned)(tile.w - tile.z + kTile - 1) / kTile;
  return at % size == 0 ? min(size, all - at) : 0;
}

// What a walk over the rows does with the keys.
enum { kForward, kStats, kDq };

// Shared memory: a stage of the ring (keys, values, codes of a chunk of 64 or 32 tokens, the maps side
// by side), a warp's scratch tile of 16 rows (two in the backward, for dO), the list of items.
template <int D, int MAPS, int MODE>
struct Shape {
  static constexpr int DV = MAPS * D;
  static constexpr int row = DV * 2;          // bytes of a key or value
  static constexpr int token = 2 * row + 4;   // of a stage, per token
  static constexpr int scratch = kTile * row;
  static constexpr int warp = MODE == kForward ? scratch : 2 * scratch;
  static constexpr int items = 256;  // of a batch
  // Working warps of a CTA at most, beside the two that fill the ring; one CTA per SM, so that all
  // stages are one ring.  As many as leave a thread nearly the registers that its fragments need: spills
  // of fragments cost more than warps gain (dq of rows of 128, 131072 tokens, differential: ten warps
  // with 168 registers 1.68 ms, six with 255 1.04 ms; dq of rows of 64: fourteen with 128 1.69 ms, ten
  // 1.40 ms).  Eight of the instances still spill 4 to 76 bytes a thread.
  static constexpr int warps = DV == 128 ? (MODE == kDq || (MODE == kForward && MAPS == 2) ? 6 : 10)
                                         : MAPS == 2 || (MODE == kDq && DV == 64) ? 10 : 14;
  // Q and dO stay in registers as fragments, or are read again from the scratch tiles for every step
  // where that leaves registers for more warps (forward of rows of 128: six warps 452 us, ten 404 us;
  // differential, both maps' sums: 1259 -> 1155 us; its statistics 787 -> 705 us; dq of rows of 32,
  // 5003 tokens: ten warps 40.2 us, fourteen 38.3 us; but dq of rows of 64: 1324, 1386 us)
  static constexpr bool held = (MODE == kDq && DV >= 64) || (MODE == kStats && MAPS == 1);
};
constexpr int kStages = 8;  // of the ring at most

// One kernel body for the forward, the row statistics of the backward, and dq with the bias
// gradient: they share the walk over cells, keys and scores.  TAB: where the bias is read: 0 no
// bias, 1 shared memory, 2 global memory; 3 as 2, the bias gradient in global memory too.  NS: stages;
// chunk: keys of a stage; pairs: heads of the CTA (1, or 2 that share a key head), whose tiles are
// work of their own from the same stages.
template <int D, int MAPS, int TAB, int MODE>
__global__ void __launch_bounds__(32 * (Shape<D, MAPS, MODE>::warps + 2), 1)
    window_rows_kernel(WinArgs a, int NS, int chunk, int pairs) {
  using S = Shape<D, MAPS, MODE>;
  constexpr int DV = S::DV;
  constexpr bool BIAS = TAB != 0;
  extern __shared__ __align__(128) char sm[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ int n_slots, n_items;         // of the batch
  __shared__ int n_rows, n_adds, n_flush;  // since the last flush; whether the batch ends with one
  __shared__ int b_rows, b_adds;           // the bounds for Limbs
  const int NW = (int)blockDim.x / 32 - 2;  // working warps; two more fill the ring
  const uint32_t v_at = chunk * S::row, codes_at = 2 * v_at, stage_size = chunk * S::token;
  const int h0 = pairs * blockIdx.y, hk = h0 / (a.hq / a.hkv), item_size = NW / pairs;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, warp = threadIdx.x >> 5;
  const int T3 = BIAS ? offsets(a.m) : 0, c0 = BIAS ? center(a.m) : 0;
  const bool grad = MODE == kDq && BIAS && a.dbias;
  int4* items = reinterpret_cast<int4*>(sm + NS * stage_size + NW * S::warp);
  int* limbs = reinterpret_cast<int*>(items + S::items);  // [pairs][2][T3] with a bias gradient, not wide
  float* tab_s = reinterpret_cast<float*>(limbs + (grad && TAB != 3 ? pairs * 2 * T3 : 0));
  Place<TAB < 2> tab;
  if constexpr (TAB >= 2)
    tab.p = reinterpret_cast<const char*>(a.tab2 + (size_t)h0 * table_pitch(a.m));
  else
    tab.p = tc::smem_u32(tab_s);
  const int tab_pitch = TAB >= 2 ? table_pitch(a.m) : T3;
  const uint32_t ring = tc::smem_u32(sm);
  const uint32_t scratch = tc::smem_u32(sm + NS * stage_size + warp * S::warp), scratch2 = scratch + S::scratch;
  const float mul = a.scale * kLog2e;
  if constexpr (BIAS) {
    if (TAB == 1)
      for (int i = threadIdx.x; i < pairs * T3; i += blockDim.x)
        tab_s[i] = i < T3 ? bias2_at(a, h0, i) : bias2_at(a, h0 + 1, i - T3);
    if (grad && TAB != 3)
      for (int i = threadIdx.x; i < pairs * 2 * T3; i += blockDim.x) limbs[i] = 0;
  }
  if (threadIdx.x < NS) {
    tc::mbar_init(&full[threadIdx.x], 96);  // two filling warps' copies, and the stores of the codes
    tc::mbar_init(&empty[threadIdx.x], NW);
  }
  tc::fence_mbar_init();
  Limbs fx;
  Wide wide;
  float s2[2] = {0.f, 0.f};
  float lams[2] = {0.f, 0.f};
  if constexpr (MAPS == 2) {
    for (int i = 0; i < pairs; ++i) {
      float e1, e2;
      lambda_terms<D>(a.lam, a.hq / 2, h0 + i, e1, e2);
      (i ? lams[1] : lams[0]) = e1 - e2 + a.lam_init;
    }
  }
  uint32_t tops[2] = {0, 0};  // the largest |dP| of a head, as bits: NaN above all

  bool written = false;             // the CTA's partial gradient
  int rot = 0;                      // the warp that takes the next item's first tile
  int fs = 0, fphase = warp >= NW;  // stage and phase of the next fill (to make one never waits at first)
  bool ok = true;
  for (int64_t batch = blockIdx.x; batch < a.T && ok; batch += (int64_t)n_slots * gridDim.x) {
    // the batch's items, in the order of their slots
    __syncthreads();
    if (warp == NW) {
      int n = 0, i0 = 0, rows = 0, adds = 0;
      const bool fresh = batch == blockIdx.x || n_flush || n_adds == 0;
      if (grad && TAB != 3 && !fresh) rows = n_rows, adds = n_adds;
      bool more = true;
#pragma unroll 2
      while (more && i0 < S::items && batch + (int64_t)i0 * gridDim.x < a.T) {
        const int64_t t = batch + (int64_t)(i0 + lane) * gridDim.x;
        int4 x = t < a.T ? __ldg(&a.tiles[t]) : make_int4(0, 0, 0, 0);
        const int dup = max(1, x.y / kDupUnit);
        x.y = item_tiles(x, item_size);
        int take = 32;  // slots of these 32
        if (grad && TAB != 3) {
          const bool crowd = dup > kDupMost && item_size * kTile * dup >= kLone;
          const int r = x.y > 0 && !crowd ? min(item_size * kTile, x.w - x.x) : 0;
          const int all = __reduce_add_sync(kFull, r * dup);
          if (adds + all <= kAdds) {
            adds += all;
          } else {  // the first slot that passes the bound waits for a flush, but for a lone one
            int sum = r * dup;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(kFull, sum, o);
              if (lane >= o) sum += y;
            }
            sum += adds;
            const unsigned over = __ballot_sync(kFull, sum > kAdds && sum > r * dup);
            if (over) take = __ffs(over) - 1, more = false;
            if (take > 0) adds = __shfl_sync(kFull, sum, take - 1);
          }
          rows += __reduce_add_sync(kFull, lane < take ? r : 0);
          if (x.y > 0 && crowd) x.y |= kCrowd;
        }
        const bool mine = lane < take && x.y > 0;
        const unsigned some = __ballot_sync(kFull, mine);
        if (mine) items[n + __popc(some & ((1u << lane) - 1u))] = x;
        n += __popc(some);
        i0 += take;
      }
      if (lane == 0) {
        n_items = n, n_slots = i0, n_rows = rows, n_adds = adds;
        n_flush = !more || adds > kAdds || batch + (int64_t)i0 * gridDim.x >= a.T;
        const bool alone = fresh && n_flush;  // no adds of another batch since the last flush and to the next
        b_rows = alone ? rows : kAdds, b_adds = alone ? adds : kAdds;
      }
    }
    __syncthreads();
    const int count = n_items;
    if (grad && TAB != 3) {
      for (int i = pairs - 1; i >= 0; --i) {
        fx.set(a, h0 + i, b_rows, b_adds);
        (i ? s2[1] : s2[0]) = fx.s[0];
      }
    }
    if (warp >= NW) {
      // the filling warps, one for the keys and the codes, one for the values: lane l holds the places
      // (in units of 16 bytes) of the rows l and 32 + l of the coming chunk
      constexpr int U = DV / 8, STEP = 32 / U;
      const bool is_k = warp == NW;
      const int r = lane / U, c = lane % U;
      const uint4* src = static_cast<const uint4*>(is_k ? a.k : a.v) + c;
      const uint4* near = static_cast<const uint4*>(is_k ? a.q : a.dout);
      uint32_t at[2], qat[2];
      int code[2];
      auto entries = [&](int k0, int hi) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int2 e = __ldg(&a.rows[min(k0 + 32 * i + lane, hi - 1)]);
          at[i] = (uint32_t)(((size_t)e.x * a.hkv + MAPS * hk) * (D / 8));
          qat[i] = (uint32_t)(((size_t)e.x * a.hq + MAPS * h0) * (D / 8));
          // places without a key: codes that spread their (zero) shares of the bias gradient
          code[i] = k0 + 32 * i + lane < hi ? e.y : (32 * i + lane) * 17 % (c0 + 1);
        }
      };
      if (count > 0) entries(items[0].z, items[0].w);
      for (int ii = 0; ii < count && ok; ++ii) {
        const int lo = items[ii].z, hi = items[ii].w;
        for (int k0 = lo; k0 < hi; k0 += chunk) {
          const int n = min(chunk, hi - k0);
          ok = ring_wait(&empty[fs], fphase);
          if (!ok) break;
          const uint32_t dst = ring + fs * stage_size + (is_k ? 0 : v_at);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (32 * x < n) {
#pragma unroll
              for (int y = 0; y < 32; y += STEP) {
                const uint32_t u = __shfl_sync(kFull, at[x], (y + r) & 31);
                cp16(dst + unit<DV>(key_at(32 * x + y + r), c), src + u, 32 * x + y + r < n);
              }
              if (BIAS && is_k)
                *reinterpret_cast<int*>(sm + fs * stage_size + codes_at + 4 * key_at(32 * x + lane)) = 4 * code[x];
              // the item's queries are its keys: bring their rows (and dO's) near
              if (is_k || MODE != kForward) {
                prefetch(near + qat[x]);
                if (pairs == 2 && DV >= 64) prefetch(near + qat[x] + DV / 8);
              }
            }
          }
          cp_arrive(&full[fs]);
          if (is_k) tc::mbar_arrive(&full[fs]);
          if (++fs == NS) fs = 0, fphase ^= 1;
          if (k0 + chunk < hi)
            entries(k0 + chunk, hi);
          else if (ii + 1 < count)
            entries(items[ii + 1].z, items[ii + 1].w);
        }
      }
    }
    for (int ii = 0; ii < count && ok && warp < NW; ++ii) {
      int4 item = items[ii];
      const bool crowd = item.y & kCrowd, far = MODE == kDq && *a.far;
      item.y &= kCrowd - 1;
      const int lo = item.z, hi = item.w;
      int mine = warp - rot;
      if (mine < 0) mine += NW;
      const bool on = mine < pairs * item.y;
      rot += pairs * item.y;
      if (rot >= NW) rot -= NW;
      const int pair = mine >= item.y ? 1 : 0;  // the head among the CTA's
      const int first = item.x + kTile * (mine - pair * item.y), nr = min(kTile, hi - first);
      const int h = h0 + pair;
      const float lam = pair ? lams[1] : lams[0];
      uint32_t top = 0;
      constexpr int NACC = MODE == kStats ? 1 : MODE == kForward ? MAPS * DV / 8 : DV / 8;
      float m[MAPS][2], l[MAPS][2], dd[MAPS][2], acc[NACC][4];
      uint32_t q[S::held ? DV / 16 : 1][4], o[S::held ? DV / 16 : 1][4];
      Place<TAB < 2> t0 = tab, t8 = tab;
      int ci = 0, ci8 = 0;
      if (on) {
        __syncwarp();
        const Rows Q = {a.q, a.hq, MAPS * h}, O = {a.dout, a.hq, MAPS * h};
        stage<D, DV, kTile, 32, MODE != kForward>(scratch, Q, scratch2, O, a.rows, first, nr, lane);
        cp_commit();
        if (BIAS) {
          // rows without a token: codes that spread their (zero) shares of the bias gradient
          ci = 4 * (c0 + (g < nr ? __ldg(&a.rows[first + g].y) : g * 13 % (c0 + 1)));
          ci8 = 4 * (c0 + (g + 8 < nr ? __ldg(&a.rows[first + g + 8].y) : (g + 8) * 13 % (c0 + 1)));
          t0.p = tab.p + 4 * pair * tab_pitch + ci;
          t8.p = tab.p + 4 * pair * tab_pitch + ci8;
        }
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            m[u][i] = kNegInf;
            l[u][i] = dd[u][i] = 0.f;
            if constexpr (MODE == kDq) {  // rows without a token: every p is 0
              const size_t at = (size_t)(MAPS * h + u) * a.N + first + min(g + 8 * i, nr - 1);
              m[u][i] = g + 8 * i < nr ? a.lse2[at] : kPosInf;
              dd[u][i] = g + 8 * i < nr ? a.D[at] : 0.f;
            }
          }
        if (grad) {
          if (TAB == 3)
            wide.set(a, h);
          else
            fx.s[0] = fx.s[1] = pair ? s2[1] : s2[0];
          if (far) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float c = far_factor(a, (size_t)h * a.N + first + min(g + 8 * i, nr - 1), m[0][i]);
              wide.c[i] = c;
              fx.s[i] *= c;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < NACC; ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
      }
      bool fresh = true;
#pragma unroll 1
      for (int k0 = lo; k0 < hi; k0 += chunk) {
        const int n = min(chunk, hi - k0);
        ok = ok && ring_wait(&full[fs], fphase);
        if (!ok) break;
        const uint32_t kst = ring + fs * stage_size;
        const int* codes = reinterpret_cast<const int*>(sm + fs * stage_size + codes_at);
        uint64_t* done = &empty[fs];
        if (++fs == NS) fs = 0, fphase ^= 1;
        if (!on) {  // every warp passes every fill: none falls behind by a turn of the ring
          if (lane == 0) tc::mbar_arrive(done);
          continue;
        }
        if (fresh) {
          fresh = false;
          cp_wait<0>();
          __syncwarp();
          if constexpr (S::held) {
#pragma unroll
            for (int d = 0; d < DV / 16; ++d) {
              load_a<DV>(q[d], scratch, 0, d);
              load_a<DV>(o[d], scratch2, 0, d);
            }
          }
        }
#pragma unroll 1
        for (int half = 0; half < n; half += 32) {
          const uint32_t kt = kst + half * S::row, vt = kt + v_at;
          const int* hc = codes + half;
          float s[MAPS][4][4], dp[MODE == kForward ? 1 : 4][4];
#pragma unroll
          for (int u = 0; u < MAPS; ++u) {
            if constexpr (S::held)
              contract_dim<DV, D, 2>(q + u * D / 16, kt, u * D / 8, s[u]);
            else
              contract_dim<DV, D, 2>(scratch, u * D / 8, kt, u * D / 8, s[u]);
            finish_scores<BIAS>(s[u], hc, n - half, mul, t0, t8);
          }
          if constexpr (MODE != kForward) {
            if constexpr (S::held)
              contract_dim<DV, DV, 2>(o, vt, 0, dp);
            else
              contract_dim<DV, DV, 2>(scratch2, 0, vt, 0, dp);
          }
          if constexpr (MODE == kDq) {
            // p = 2^(s - lse2), dS = p (dP - D)
#pragma unroll
            for (int u = 0; u < MAPS; ++u) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float p = ex2(s[u][j][x] - m[u][x >> 1]);
                  s[u][j][x] = (u ? -lam * p : p) * (dp[j][x] - dd[u][x >> 1]);
                }
              if (BIAS) {
                if (grad) {
                  const uint32_t to = tc::smem_u32(limbs) + 8 * pair * T3;
                  if constexpr (TAB == 3) {
                    add_bias_grad([&](int at, float x, int row) { wide.add(at, x, row); }, s[0], hc, ci, ci8);
                  } else if (crowd) {
                    float ds[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                      for (int x = 0; x < 4; ++x) ds[j][x] = s[0][j][x];
                    wide.set(a, h);
                    const float one = pair ? s2[1] : s2[0];
                    wide.c[0] = fx.s[0] / one, wide.c[1] = fx.s[1] / one;
                    add_crowded(wide, ds, hc, ci, ci8);
                  } else {
                    add_bias_grad([&](int at, float x, int row) { fx.add(to + at, to + at + 4 * T3, x, row); }, s[0], hc,
                                  ci, ci8);
                  }
                }
              }
              uint32_t f[2][4];
              pack_a<4>(s[u], f);
              contract_rows<DV, D, 2>(f, kt, u * D / 8, acc + u * D / 8);
            }
          } else {
            // online maximum, sum (and sum of p dP) of a row; the sums stay per lane to the end.
            // The subtracted maximum follows the true one only once that has grown by a factor of
            // 2^kSlack; until then a step asks no neighbour for its maximum and rescales nothing
            bool grown = false;
            float mx[MAPS][2];
#pragma unroll
            for (int u = 0; u < MAPS; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                mx[u][i] = kNegInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) mx[u][i] = fmaxf(mx[u][i], fmaxf(s[u][j][2 * i], s[u][j][2 * i + 1]));
                grown |= mx[u][i] > m[u][i] + kSlack;
              }
            if (__any_sync(kFull, grown)) {
#pragma unroll
              for (int u = 0; u < MAPS; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float to = quad_max(mx[u][i]);
                  if (!(to > m[u][i] + kSlack)) to = m[u][i];
                  const float old = rescale(m[u][i], safe_max(to));
                  m[u][i] = to;
                  l[u][i] *= old;
                  if constexpr (MODE == kStats) dd[u][i] *= old;
                  if constexpr (MODE == kForward) {
                    if (half + k0 > lo) {
#pragma unroll
                      for (int e = 0; e < DV / 8; ++e) {
                        acc[u * (DV / 8) + e][2 * i] *= old;
                        acc[u * (DV / 8) + e][2 * i + 1] *= old;
                      }
                    }
                  }
                }
            }
#pragma unroll
            for (int u = 0; u < MAPS; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float ms = safe_max(m[u][i]);
                float e = 0.f, ed = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const float p = ex2(s[u][j][2 * i + x] - ms);
                    s[u][j][2 * i + x] = p;
                    e += p;
                    if constexpr (MODE == kStats) {
                      ed = fmaf(p, dp[j][2 * i + x], ed);
                      if (u == 0) top = max(top, __float_as_uint(dp[j][2 * i + x]) & 0x7fffffffu);
                    }
                  }
                l[u][i] += e;
                if constexpr (MODE == kStats) dd[u][i] += ed;
              }
            if constexpr (MODE == kForward) {
              // the maps of differential attention are rounded each on its own and subtracted as
              // fp32 outputs: subtracting first would need both normalisers first, that is every
              // score and exponential twice
              uint32_t p[2 * MAPS][4];
#pragma unroll
              for (int u = 0; u < MAPS; ++u) pack_a<4>(s[u], p + 2 * u);
              contract_rows<DV, DV, 2, MAPS>(p, vt, 0, acc);
            }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(done);
      }
      if (!on || !ok) continue;
      if constexpr (MODE != kDq) {
        bool none = false;
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[u][i] = quad_sum(l[u][i]);
            none |= l[u][i] == 0.f;
          }
        if (__any_sync(kFull, none)) {  // rows that sum to 0: NaN where the bias did not bar all keys
#pragma unroll
          for (int u = 0; u < MAPS; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              bool left = l[u][i] == 0.f;
              if constexpr (BIAS)
                left = left && key_left(a, h, (i ? ci8 : ci) / 4 - c0, lo, hi, t4, 4);
              if (quad_max(left ? 1.f : 0.f) > 0.f) l[u][i] = __uint_as_float(0x7fc00000u);
            }
        }
      }
      if constexpr (MODE == kForward) {
        float f[2] = {1.f, 1.f};
        if constexpr (MAPS == 1) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f[i] = safe_inv(l[0][i]);
            if (a.lse && t4 == 0 && g + 8 * i < nr)
              a.lse[(size_t)__ldg(&a.rows[first + g + 8 * i].x) * a.hq + h] =
                  l[0][i] == 0.f ? kNegInf : (m[0][i] + log2f(l[0][i])) * kLn2;
          }
        }
        if constexpr (MAPS == 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f0 = safe_inv(l[0][i]), f1 = lam * safe_inv(l[MAPS - 1][i]);
#pragma unroll
            for (int e = 0; e < DV / 8; ++e)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                acc[e][2 * i + x] = acc[e][2 * i + x] * f0 - acc[(MAPS - 1) * (DV / 8) + e][2 * i + x] * f1;
          }
        }
        store_acc<D, DV>(scratch, acc, f[0], f[1], static_cast<bf16*>(a.out), a.hq, MAPS * h, a.rows, first, nr);
      } else if constexpr (MODE == kStats) {
#pragma unroll
        for (int u = 0; u < MAPS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            dd[u][i] = quad_sum(dd[u][i]);
            if (t4 == 0 && g + 8 * i < nr) {
              const size_t at = (size_t)(MAPS * h + u) * a.N + first + g + 8 * i;
              store_lse2(a, at, m[u][i], l[u][i]);
              a.D[at] = dd[u][i] * safe_inv(l[u][i]);
              if (!(l[u][i] >= 0.f)) top = 0x7fffffffu;
            }
          }
        if (pair)
          tops[1] = max(tops[1], top);
        else
          tops[0] = max(tops[0], top);
      } else {
        if (far) {
#pragma unroll
          for (int u = 0; u < MAPS; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float c = far_factor(a, (size_t)(MAPS * h + u) * a.N + first + min(g + 8 * i, nr - 1), m[u][i]);
#pragma unroll
              for (int e = u * D / 8; e < (u + 1) * D / 8; ++e) acc[e][2 * i] *= c, acc[e][2 * i + 1] *= c;
            }
        }
        store_acc<D, DV>(scratch, acc, a.scale, a.scale, static_cast<bf16*>(a.dq), a.hq, MAPS * h, a.rows, first, nr);
      }
    }
    if (grad && TAB != 3 && n_flush) {
      // the sums since the last flush; each thread has offsets of its own
      __syncthreads();
      for (int p = 0; p < pairs; ++p) {
        fx.set(a, h0 + p, b_rows, b_adds);
        int* from = limbs + p * 2 * T3;
        float* part = a.part + ((size_t)(h0 + p) * a.parts + blockIdx.x) * T3;
        for (int i = threadIdx.x; i < T3; i += blockDim.x) {
          const float x = fx.value(from[i], from[T3 + i]);
          part[i] = written ? part[i] + x : x;
          from[i] = from[T3 + i] = 0;
        }
      }
      written = true;
    }
  }
  cp_commit();
  cp_wait<0>();
  if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
  if constexpr (MODE == kStats && BIAS) {
    for (int i = 0; i < pairs; ++i) {
      const uint32_t top = __reduce_max_sync(kFull, i ? tops[1] : tops[0]);
      if (lane == 0 && a.dbias) atomicMax(a.amax + h0 + i, top);
    }
  }
}

// CTAs along the slots for `heads` (pairs of) heads: up to six for every SM, so that the last ones to
// finish leave little idle, but no more than one while that gives a CTA fewer than 16 slots.
int grid_x(int64_t heads, int64_t T) {
  const int64_t waves = max((int64_t)1, min((int64_t)6, heads * T / (16 * kSms)));
  return (int)max((int64_t)1, min(T, waves * kSms / heads));
}

template <int D, int MAPS, bool BIAS, int MODE>
cudaError_t rows_pass(const char* name, const WinArgs& a, cudaStream_t st) {
  using S = Shape<D, MAPS, MODE>;
  constexpr int ON = BIAS ? 1 : 0;
  const bool grad = MODE == kDq && BIAS && a.dbias;
  const size_t T3 = BIAS ? offsets(a.m) : 0, list = sizeof(int4) * S::items;
  // Two heads to a CTA where they share a key head: the stages then serve twice the work.  Chunks of 64
  // keys: chunks of 32 cost 4 to 6% of a step of cells of 21 to 41 tokens (131072 tokens, edges 5 to 7:
  // 3638, 3234, 3560 us against 3776, 3423, 3680) and gain 1% at most where cells hold 4 to 16.  The bias
  // lies in shared memory where room is left beside it for eight warps and four stages (the forward always
  // has it there); then as many warps as may be, and as many stages as fit.  What does not fit takes one
  // head, then chunks of 32, then three stages.
  int chunk = 0, pairs = 0, NW = 0, NS = 0;
  bool in_smem = false;
  size_t smem = 0;
  for (int attempt = 0; attempt < 4 && !smem; ++attempt) {
    pairs = attempt == 0 && a.hq / a.hkv % 2 == 0 && S::warps >= 10 ? 2 : 1;
    chunk = attempt >= 2 ? 32 : kChunk;
    const size_t stage = (size_t)chunk * S::token, table = 4 * T3 * pairs, limbs = grad && !a.wide ? 8 * T3 * pairs : 0;
    const size_t least = list + limbs + min(8, S::warps) * S::warp + (attempt == 3 ? 3 : 4) * stage;
    in_smem = BIAS && !(grad && a.wide) && least + table <= kSmemMost;
    if (least > kSmemMost || (BIAS && !in_smem && (MODE == kForward || attempt == 0))) continue;
    const size_t fixed = list + limbs + (in_smem ? table : 0);
    NW = (int)min((size_t)S::warps, (kSmemMost - fixed - (attempt == 3 ? 3 : 4) * stage) / S::warp);
    NS = (int)min((size_t)kStages, (kSmemMost - fixed - NW * S::warp) / stage);
    smem = fixed + NW * S::warp + NS * stage;
  }
  if (!smem) return cudaErrorInvalidConfiguration;  // no edge that a bias can have comes here
  auto kern = window_rows_kernel<D, MAPS, ON, MODE>;
  if constexpr (MODE != kForward)
    if (!in_smem) kern = window_rows_kernel<D, MAPS, 2 * ON, MODE>;
  if constexpr (MODE == kDq)
    if (grad && a.wide) kern = window_rows_kernel<D, MAPS, 3 * ON, MODE>;
  const cudaError_t e = need_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const int heads = a.hq / MAPS / pairs;
  const int gx = grad && !a.wide ? a.parts : grid_x(heads, a.T);
  SSA_LAUNCH(name, kern, dim3(gx, heads), 32 * (NW + 2), smem, st, a, NS, chunk, pairs);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// backward: dk, dv
// ---------------------------------------------------------------------------

// A CTA of four warps takes 64 keys of a cell and one key head, 16 keys per warp: the transposed
// scores of the cell's queries, 64 at a time, of every query head that reads the key head.  Q, dO,
// the statistics and the head's bias table of the next step arrive while this one is computed.  Keys
// stay with a CTA so that dk and dv are sums in registers, with no atomics, rounded once.  Bound by
// issue and by the barriers of a step (cells of 47 tokens leave one warp in four without keys): 887 us
// at 131072 tokens, 32/2 heads of 64; one barrier a step instead of two, its copies begun after it, took
// 1% longer.
constexpr int kDkvWarps = 4;

// Number of key tiles of the CTA of a slot: four from every fourth tile of a cell.
__device__ __forceinline__ int dkv_tiles(const int4& tile) { return item_tiles(tile, kDkvWarps); }

template <int D, int MAPS>
struct DkvShape {
  static constexpr int DV = MAPS * D;
  // K and V as fragments in registers; wide rows leave no room for them
  static constexpr bool held = DV <= 64;
  static constexpr int KT = kChunk * DV * 2;               // one tile of 64 rows, bytes
  static constexpr int Q = held ? 0 : 2 * KT;              // two stages of Q, dO and the statistics
  static constexpr int stat = 2 * KT;                      // within a stage: lse2, D of MAPS maps
  static constexpr int stage = stat + 2 * MAPS * kChunk * 4;
  static constexpr int codes = Q + 2 * stage;              // codes of the queries, two stages
  static constexpr int tab = codes + 2 * kChunk * 4;       // two bias tables
};

// TAB: 0 no bias, 1 tables staged in shared memory, 2 read in global memory (the largest edges).
// FAR: weights of rows far from zero (kFarScore) are set right.  A body of its own, taken once per CTA,
// because tests inside the steps cost 9% (131072 tokens: 1001 -> 1088 us; differential 1044 -> 1176).
template <int D, int MAPS, int TAB, bool FAR>
__device__ __forceinline__ void dkv_body(const WinArgs& a) {
  using S = DkvShape<D, MAPS>;
  constexpr int DV = S::DV, NTH = 32 * kDkvWarps;
  constexpr bool BIAS = TAB != 0;
  // unit_pair's exclusive or holds the first unit's place in a register, which rows of 64 and two maps
  // have not left (rows of 64, 131072 tokens: 928 us without, 1064 with; d = 128, full cube: 576, 567)
  constexpr bool XOR = DV == 128 && MAPS == 1;
  extern __shared__ __align__(128) char sm[];
  const int G = a.hq / a.hkv, hk = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t4 = lane & 3, warp = tid >> 5;
  const float mul = a.scale * kLog2e;
  const int c0 = BIAS ? center(a.m) : 0, T3 = BIAS ? offsets(a.m) : 0, T3p = BIAS ? table_pitch(a.m) : 0;
  const int4 tile = __ldg(&a.tiles[blockIdx.x]);
  const int lo = tile.z, hi = tile.w, nt = dkv_tiles(tile);
  if (nt == 0) return;
  // K and V stay before the stages, or are in the second stage until it is needed
  const uint32_t base = tc::smem_u32(sm), kt = base + (S::held ? S::stage : 0), vt = kt + S::KT;
  const int keys0 = tile.x, nkeys = min(kTile * nt, hi - keys0);

  // a step: query head h, 64 queries from k0 on, into stage `st`; a head's first step brings its table.
  // The places of the queries' rows (in units of 16 bytes) and their codes stay while k0 does.
  constexpr int U = DV / 8, STEP = NTH / U, IT = kChunk / STEP;
  const int ur = tid / U, uc = tid % U;
  uint32_t place[IT];
  int k_now = -1, cst = 1;
  auto load = [&](int h, int k0, int st) {
    const int n = min(kChunk, hi - k0);
    if (k0 != k_now) {
      k_now = k0;
      cst ^= 1;
      int* codes = reinterpret_cast<int*>(sm + S::codes) + cst * kChunk;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int2 e = __ldg(&a.rows[k0 + min(i * STEP + ur, n - 1)]);
        place[i] = (uint32_t)((size_t)e.x * a.hq * (D / 8)) + uc;
        if (BIAS && uc == 0) codes[i * STEP + ur] = 4 * (e.y + c0);
      }
    }
    const uint32_t q = base + S::Q + st * S::stage;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = i * STEP + ur;
      if (i * STEP < ((n + 31) & ~31)) {
        const uint32_t at = place[i] + MAPS * h * (D / 8);
        cp16(q + unit<DV>(r, uc), static_cast<const uint4*>(a.q) + at, r < n);
        cp16(q + S::KT + unit<DV>(r, uc), static_cast<const uint4*>(a.dout) + at, r < n);
      }
    }
    const uint32_t stat = q + S::stat;
#pragma unroll
    for (int u = 0; u < MAPS; ++u) {  // 64 threads a row of lse2, 64 a row of D
      const int which = tid / kChunk, c = tid % kChunk;
      const uint32_t dst = stat + 4 * ((2 * u + which) * kChunk + c);
      if (c < n)
        cp4(dst, (which ? a.D : a.lse2) + (size_t)(MAPS * h + u) * a.N + k0 + c);
      else
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(which ? 0.f : kPosInf) : "memory");
    }
    if (TAB == 1 && k0 == lo) {
      const uint32_t dst = base + S::tab + (h & 1) * T3p * 4;
      const float* src = a.tab2 + (size_t)h * T3p;
      for (int i = tid; i < T3p / 4; i += NTH) cp16(dst + 16 * i, src + 4 * i, true);
    }
    cp_commit();
  };

  const Rows K = {a.k, a.hkv, MAPS * hk}, V = {a.v, a.hkv, MAPS * hk};
  stage<D, DV, kChunk, NTH, true>(kt, K, vt, V, a.rows, keys0, nkeys, tid);
  load(hk * G, lo, 0);
  const int r0 = kTile * warp, first = keys0 + r0, nr = min(kTile, hi - first);
  const bool on = warp < nt;
  int ck = 0, ck8 = 0;
  if (BIAS && on) {
    ck = __ldg(&a.rows[first + min(g, nr - 1)].y);
    ck8 = __ldg(&a.rows[first + min(g + 8, nr - 1)].y);
  }
  float dk[MAPS][D / 8][4], dv[DV / 8][4];
#pragma unroll
  for (int u = 0; u < MAPS; ++u)
#pragma unroll
    for (int e = 0; e < D / 8; ++e) dk[u][e][0] = dk[u][e][1] = dk[u][e][2] = dk[u][e][3] = 0.f;
#pragma unroll
  for (int e = 0; e < DV / 8; ++e) dv[e][0] = dv[e][1] = dv[e][2] = dv[e][3] = 0.f;

  uint32_t kf[S::held ? DV / 16 : 1][4], vf[S::held ? DV / 16 : 1][4];
  if constexpr (S::held) {
    cp_wait<0>();
    __syncthreads();
    if (on) {
#pragma unroll
      for (int d = 0; d < DV / 16; ++d) load_a<DV, XOR>(kf[d], kt, r0, d), load_a<DV, XOR>(vf[d], vt, r0, d);
    }
    __syncthreads();
  }

  int h = hk * G, k0 = lo, stg = 0, cnow = cst;
  while (true) {
    int h2 = h, k2 = k0 + kChunk;  // the step after this one
    if (k2 >= hi) k2 = lo, ++h2;
    const bool more = h2 < hk * G + G;
    if (more) {
      load(h2, k2, stg ^ 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    if (on) {
      const int n = min(kChunk, hi - k0);
      float lam = 0.f;
      if constexpr (MAPS == 2) {
        float e1, e2;
        lambda_terms<D>(a.lam, a.hq / 2, h, e1, e2);
        lam = e1 - e2 + a.lam_init;
      }
      const uint32_t qt = base + S::Q + stg * S::stage, ot = qt + S::KT;
      const float* stat = reinterpret_cast<const float*>(sm + S::Q + stg * S::stage + S::stat);
      const int* codes = reinterpret_cast<const int*>(sm + S::codes) + cnow * kChunk;
      Place<TAB != 2> tk, tk8;
      if constexpr (TAB == 2)
        tk.p = reinterpret_cast<const char*>(a.tab2 + (size_t)h * T3p);
      else
        tk.p = base + S::tab + 4 * (h & 1) * T3p;
      tk8.p = tk.p - 4 * ck8;
      tk.p -= 4 * ck;
#pragma unroll 1
      for (int q0 = 0; q0 < n; q0 += 32) {
        // rows q0 .. of the tiles: 32 rows on, the permutation of the units repeats
        const uint32_t qq = qt + q0 * DV * 2, oo = ot + q0 * DV * 2;
        float dp[4][4], pv[4][4];
        if constexpr (S::held) {
          contract_dim<DV, DV, 2, XOR>(vf, oo, 0, dp);
        } else {
          uint32_t f[DV / 16][4];
#pragma unroll
          for (int d = 0; d < DV / 16; ++d) load_a<DV, XOR>(f[d], vt, r0, d);
          contract_dim<DV, DV, 2, XOR>(f, oo, 0, dp);
        }
#pragma unroll
        for (int u = 0; u < MAPS; ++u) {
          float sc[4][4];
          if constexpr (S::held) {
            contract_dim<DV, D, 2, XOR>(kf + u * D / 16, qq, u * D / 8, sc);
          } else {
            uint32_t f[D / 16][4];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) load_a<DV, XOR>(f[d], kt, r0, u * D / 16 + d);
            contract_dim<DV, D, 2, XOR>(f, qq, u * D / 8, sc);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = q0 + 8 * j + 2 * t4;
            const float2 L = *reinterpret_cast<const float2*>(stat + 2 * u * kChunk + c);
            const float2 Dq = *reinterpret_cast<const float2*>(stat + (2 * u + 1) * kChunk + c);
            float b[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (BIAS) {
              const int2 cq = *reinterpret_cast<const int2*>(codes + c);
              b[0] = tk.at(cq.x), b[1] = tk.at(cq.y), b[2] = tk8.at(cq.x), b[3] = tk8.at(cq.y);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              // columns past the last query: lse2 is plus infinity, so p is 0, and their dO is 0
              float p = ex2(fmaf(sc[j][x], mul, b[x]) - (x & 1 ? L.y : L.x));
              if constexpr (FAR) {
                const size_t at = (size_t)(MAPS * h + u) * a.N + k0 + min(c + (x & 1), n - 1);
                p *= far_factor(a, at, x & 1 ? L.y : L.x);
                if (p > 1.f) p = 1.f;  // a score may round to one side here, to the other where lse2 was taken
              }
              const float w = u ? -lam * p : p;
              pv[j][x] = u ? pv[j][x] + w : w;
              sc[j][x] = w * (dp[j][x] - (x & 1 ? Dq.y : Dq.x));
            }
          }
          uint32_t f[2][4];
          pack_a<4>(sc, f);
          contract_rows<DV, D, 2, 1, XOR>(f, qq, u * D / 8, dk[u]);
        }
        uint32_t f[2][4];
        pack_a<4>(pv, f);
        contract_rows<DV, DV, 2, 1, XOR>(f, oo, 0, dv);
      }
    }
    __syncthreads();
    if (!more) break;
    h = h2;
    k0 = k2;
    stg ^= 1;
    cnow = cst;
  }
  if (!on) return;
  // the stages are free now; 16 rows of scratch per warp
  const uint32_t scratch = base + S::Q + warp * kTile * DV * 2;
#pragma unroll
  for (int u = 0; u < MAPS; ++u)
    store_acc<D, D>(scratch, dk[u], a.scale, a.scale, static_cast<bf16*>(a.dk), a.hkv, MAPS * hk + u, a.rows, first, nr);
  store_acc<D, DV>(scratch, dv, 1.f, 1.f, static_cast<bf16*>(a.dv), a.hkv, MAPS * hk, a.rows, first, nr);
}

template <int D, int MAPS, int TAB>
__global__ void __launch_bounds__(32 * kDkvWarps, D* MAPS == 128 ? 2 : 3) window_dkv_mma_kernel(WinArgs a) {
  if (*a.far) return dkv_body<D, MAPS, TAB, true>(a);
  dkv_body<D, MAPS, TAB, false>(a);
}

// tab2[h][o]: the bias of every offset in units of log2, rows of a multiple of 4; clears amax, far and,
// where something will be added to them, the 64-bit sums.
__global__ void bias_expand_kernel(WinArgs a) {
  const int T3 = offsets(a.m), T3p = table_pitch(a.m), o = blockIdx.x * blockDim.x + threadIdx.x;
  if (o == 0) a.amax[blockIdx.y] = 0;
  if (o == 0 && blockIdx.y == 0) *a.far = 0;
  if ((a.wide || __ldg(&a.tiles[a.T].x) > kDupMost) && o < T3) a.sums[(size_t)blockIdx.y * T3 + o] = 0;
  if (o < T3p) a.tab2[(size_t)blockIdx.y * T3p + o] = o < T3 ? bias2_at(a, blockIdx.y, o) : 0.f;
}

template <int D, int MAPS, bool BIAS>
cudaError_t bwd(const WinArgs& a, cudaStream_t st) {
  constexpr int ON = BIAS ? 1 : 0;
  const size_t T3p = BIAS ? table_pitch(a.m) : 0;
  if (!BIAS) {
    const cudaError_t e = cudaMemsetAsync(a.far, 0, sizeof(int), st);
    if (e != cudaSuccess) return e;
  }
  if (BIAS)
    SSA_LAUNCH("bias_expand_kernel", bias_expand_kernel, dim3(((int)T3p + 255) / 256, a.hq), 256, 0, st, a);
  cudaError_t r = rows_pass<D, MAPS, BIAS, kStats>("window_stats_kernel", a, st);
  if (r == cudaSuccess) r = rows_pass<D, MAPS, BIAS, kDq>("window_dq_kernel", a, st);
  if (r != cudaSuccess) return r;
  {
    using K = DkvShape<D, MAPS>;
    // three CTAs per SM (two for wide rows) while the tables fit beside them
    const bool in_smem = K::tab + 2 * sizeof(float) * T3p <= (D * MAPS == 128 ? 113 : 75) * 1024;
    const size_t smem = K::tab + (in_smem ? 2 * sizeof(float) * T3p : 0);
    auto kern = in_smem ? window_dkv_mma_kernel<D, MAPS, ON> : window_dkv_mma_kernel<D, MAPS, 2 * ON>;
    const cudaError_t e = need_smem(kern, smem);
    if (e != cudaSuccess) return e;
    SSA_LAUNCH("window_dkv_mma_kernel", kern, dim3(a.T, a.hkv / MAPS), 32 * kDkvWarps, smem, st, a);
  }
  return cudaGetLastError();
}

cudaError_t bwd_any(const WinArgs& a, cudaStream_t st) {
  if (a.maps == 2) return a.d == 32 ? bwd<32, 2, false>(a, st) : bwd<64, 2, false>(a, st);
  if (a.table)
    return a.d == 32   ? bwd<32, 1, true>(a, st)
           : a.d == 64 ? bwd<64, 1, true>(a, st)
                       : bwd<128, 1, true>(a, st);
  return a.d == 32   ? bwd<32, 1, false>(a, st)
         : a.d == 64 ? bwd<64, 1, false>(a, st)
                     : bwd<128, 1, false>(a, st);
}

}  // namespace

cudaError_t window_fwd_mma(const WinArgs& a, cudaStream_t st) {
  const char* name = "window_fwd_kernel";
  if (a.maps == 2)
    return a.d == 32 ? rows_pass<32, 2, false, kForward>(name, a, st)
                     : rows_pass<64, 2, false, kForward>(name, a, st);
  if (a.table)
    return a.d == 32   ? rows_pass<32, 1, true, kForward>(name, a, st)
           : a.d == 64 ? rows_pass<64, 1, true, kForward>(name, a, st)
                       : rows_pass<128, 1, true, kForward>(name, a, st);
  return a.d == 32   ? rows_pass<32, 1, false, kForward>(name, a, st)
         : a.d == 64 ? rows_pass<64, 1, false, kForward>(name, a, st)
                     : rows_pass<128, 1, false, kForward>(name, a, st);
}

cudaError_t window_bwd_mma(const WinArgs& a, cudaStream_t st) {
  return bwd_any(a, st);
}

}  // namespace ssa
