// Row-wise operators of a language model's token step, next to the denoiser:
//   rms_norm     the residual's addition and RMS norm, bf16 and / or e4m3 rows
//   quantize_w4  4-bit weights with a scale for each group along K
//   gemv_w4      products of up to 16 vectors with such weights
// with their entry points of the C ABI.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "capi_util.h"
#include "mmdit.h"
#include "mmdit_internal.h"
#include "token.cuh"

namespace mmdit {

namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ------------------------------------------------------------------ RMS norm
// h = x + delta; y = h / sqrt(mean(h^2) + eps) * gain.  The row stays in
// registers as fp32 between the sum of squares, the maximum of |y| (e4m3
// rows) and the stores, so every input is read once and every output written
// once.  The norm is taken of the unrounded sum: x_out rounds it once to the
// residual's type.  e4m3 rows are rounded from the fp32 values, with
// s = max|y| / 448 (1 for a zero row, never below 2^-126): a bf16 value in
// between would round twice.
//
// Bound: HBM for many rows.  16381 bf16 rows of 4096 with e4m3 output move
// 470 MB in 75.5 us, 6.2 TB/s (0.92 of the copy bandwidth); 512 fp32 rows take
// 5.1 us, 0.67 of it, with a launch's fill and drain; one row 2.1 us, launch and
// two reductions.
struct RmsArgs {
  const void* x;
  const void* delta;
  const float* gain;
  void* x_out;
  uint16_t* y;
  uint8_t* q;
  float* s;
  long long rows, x_ld, delta_ld;
  int nv;  // D / 8
  float eps;
};

// Eight elements as they lie in memory.
template <bool F32>
struct Raw8 {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, long long i) {
    const uint4* a = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
    u[0] = a[0];
    if (F32) u[F32 ? 1 : 0] = a[1];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) u[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    if (F32) {
      const uint4 t = u[F32 ? 1 : 0];
      const uint32_t z[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(w[k]), v[4 + k] = __uint_as_float(z[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(w[k]), v[2 * k + 1] = bf16_hi(w[k]);
    }
  }
};
template <bool F32>
__device__ __forceinline__ void store8(void* p, long long i, const float* v) {
  if (F32) {
    float4* a = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    a[0] = make_float4(v[0], v[1], v[2], v[3]);
    a[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// DM: 0 no delta, 1 bf16, 2 fp32.  V vectors of 8 elements per thread;
// blockDim = (threads of a row, rows).  A row of 32 threads reduces with
// shuffles alone, a longer one through shared memory (one row per block).
// Every load of x and delta is issued before the first store: x_out may be x.
template <bool XF32, int DM, int V>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const RmsArgs a) {
  __shared__ float red[2][32];
  const int T = blockDim.x, tid = threadIdx.x;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  grid_wait();
  grid_release();
  if (row >= a.rows) return;  // whole warps: T is a multiple of 32, and blocks of several rows use no barrier
  Raw8<XF32> xr[V];
  Raw8<DM == 2> dr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * T;
    if (v < a.nv) {
      xr[i].load(a.x, row * a.x_ld + 8ll * v);
      if (DM) dr[i].load(a.delta, row * a.delta_ld + 8ll * v);
    } else {
      xr[i].zero();
      dr[i].zero();
    }
  }
  float h[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    xr[i].get(h[i]);
    if (DM) {
      float t[8];
      dr[i].get(t);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] += t[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(h[i][k], h[i][k], ss);
  }
  if (DM && a.x_out) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * T < a.nv) store8<XF32>(a.x_out, row * a.x_ld + 8ll * (tid + i * T), h[i]);
  }
  ss = warp_sum(ss);
  const int lane = tid & 31, warp = tid >> 5, nw = T >> 5;
  if (nw > 1) {
    if (lane == 0) red[0][warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < nw ? red[0][lane] : 0.f);
  }
  const float r = rsqrtf(ss / (8.0f * (float)a.nv) + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * T;
    if (v >= a.nv) break;
    const float4 g0 = reinterpret_cast<const float4*>(a.gain)[2 * v];
    const float4 g1 = reinterpret_cast<const float4*>(a.gain)[2 * v + 1];
    const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[i][k] = h[i][k] * r * g[k];
      amax = fmaxf(amax, fabsf(h[i][k]));
    }
    if (a.y) store8<false>(a.y, row * 8ll * a.nv + 8ll * v, h[i]);
  }
  if (!a.q) return;
  amax = warp_max(amax);
  if (nw > 1) {
    if (lane == 0) red[1][warp] = amax;
    __syncthreads();
    amax = warp_max(lane < nw ? red[1][lane] : 0.f);
  }
  const float sq = amax == 0.f ? 1.0f : fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f);
  if (tid == 0) a.s[row] = sq;
  // The quotient y / s as a product with the reciprocal, corrected once by its
  // remainder, which a fused multiply-add gives exactly (Markstein, IBM J. Res.
  // Dev. 34, 1990): with the rounded reciprocal that is the rounded quotient,
  // so the codes are those of the division.  16381 rows of 4096 take 75.6 us
  // (the product alone 74, divisions 95).  A maximum below 2^-100, whose
  // reciprocal or remainders could leave the range, is brought up first
  // (exactly).
  const float up = amax < 7.8886e-31f ? 1.2676506e30f : 1.0f;  // 2^-100, 2^100
  const float su = sq * up, inv = __fdiv_rn(1.0f, su);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * T;
    if (v >= a.nv) break;
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float t = h[i][k] * up, q0 = t * inv;
      q[k] = fmaf(fmaf(-q0, su, t), inv, q0);
    }
    *reinterpret_cast<uint2*>(a.q + row * 8ll * a.nv + 8ll * v) =
        make_uint2((uint32_t)f8x2_e4m3(q[0], q[1]) | ((uint32_t)f8x2_e4m3(q[2], q[3]) << 16),
                   (uint32_t)f8x2_e4m3(q[4], q[5]) | ((uint32_t)f8x2_e4m3(q[6], q[7]) << 16));
  }
}

template <bool XF32, int DM>
cudaError_t launch_rms_dm(const RmsArgs& a, cudaStream_t st) {
  // Few rows: one vector per thread, the row spread over as many threads as
  // it has vectors (up to 1024); many rows: two per thread, so that a warp has
  // four loads in flight and a block half the warps to wait for; four where a
  // row has more than 2048.  bf16 rows of 4096 with e4m3 output, one and two per
  // thread: 1 row 2.17 and 2.35 us, 128 rows 2.40 and 2.56, 304 rows 2.91 and
  // 2.93, 320 rows 4.10 and 3.26, 4096 rows 24.4 and 21.5.
  const bool few = a.rows <= 2ll * num_sms();
  const int per = a.nv > 2048 ? 4 : few && a.nv <= 1024 ? 1 : 2;
  const int T = ((a.nv + per - 1) / per + 31) / 32 * 32;
  const int R = T == 32 ? 4 : 1;
  const long long grid = (a.rows + R - 1) / R;
  const dim3 block(T, R);
  launch_begin(KID_RMS_NORM, st);
  const cudaError_t e = launch_after(per == 1   ? rms_norm_kernel<XF32, DM, 1>
                                     : per == 2 ? rms_norm_kernel<XF32, DM, 2>
                                                : rms_norm_kernel<XF32, DM, 4>,
                                     dim3((unsigned)grid), block, 0, 1, st, a);
  launch_end(st);
  return e;
}

cudaError_t launch_rms_norm(const RmsArgs& a, bool x_f32, int dm, cudaStream_t st) {
  if (x_f32) return dm == 0 ? launch_rms_dm<true, 0>(a, st) : dm == 1 ? launch_rms_dm<true, 1>(a, st)
                                                                     : launch_rms_dm<true, 2>(a, st);
  return dm == 0 ? launch_rms_dm<false, 0>(a, st) : dm == 1 ? launch_rms_dm<false, 1>(a, st)
                                                           : launch_rms_dm<false, 2>(a, st);
}

// ------------------------------------------------------------------ 4-bit weights
// Rows are stored in chunks of 128 elements (64 bytes), the last one filled
// up with code 8 (a zero).  Word 4 c + i of a chunk (c, i in 0..3) holds the
// elements m + {0, 2, 4, 6, 1, 3, 5, 7}, m = 32 i + 8 c, from its lowest four
// bits up, as q + 8.  So the 16 bytes that lane c of a row reads hold, word by
// word, its 8 elements of each 32-element group, and the two halves of a word
// hold neighbours.  Scales: bf16, 128 / group per chunk.

// One warp per row and chunk, four elements per lane.
template <bool F32>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const void* __restrict__ w, int N, int K, int C, int group,
                                                          uint32_t* __restrict__ q, uint16_t* __restrict__ scale) {
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= (long long)N * C) return;
  const int n = (int)(unit / C), ch = (int)(unit - (long long)n * C);
  const int k0 = ch * 128 + lane * 4;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (k0 < K) {  // K is a multiple of 32: four elements at once
    if (F32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + (long long)n * K + k0);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + (long long)n * K + k0);
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    }
  }
  float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
  for (int o = 1; o < group / 4; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const uint16_t sb = (uint16_t)(pack_bf16x2(__fdiv_rn(amax, 7.0f), 0.f) & 0xFFFFu);
  float s = bf16_lo(sb);
  if (s == 0.f) s = 1.0f;
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -7.0f), 7.0f);
    const int el = (lane & 1) * 4 + e;  // element of the 8-element word
    word |= (uint32_t)((int)t + 8) << (4 * ((el & 1) * 4 + (el >> 1)));
  }
  word |= __shfl_xor_sync(0xffffffffu, word, 1);
  const int L = lane >> 1;  // elements 8 L .. 8 L + 7 of the chunk
  if (!(lane & 1)) q[unit * 16 + 4 * (L & 3) + (L >> 2)] = word;
  if (lane * 4 % group == 0)
    scale[unit * (128 / group) + lane * 4 / group] = k0 < K ? (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu) : (uint16_t)0;
}

// y[b, n] = sum over groups of s[n, group] * (sum_k q[n, k] x[b, k]) + bias.
//
// Both operands of the matrix instruction (m16n8k16, 16 rows of W) are bf16 and
// exact: x as it is given, and the codes as q 2^-6.  A code n = q + 8 (0 .. 15)
// in the low bits of a 16-bit half, read as bf16, is the subnormal n 2^-133, and
// four bits further up n 2^-129 (the first normal numbers go on where the
// subnormal ones end), so a mask and one fused multiply-add for two codes,
//   n 2^-133 2^127 - 2^-3 = n 2^-129 2^123 - 2^-3 = q 2^-6,
// make them; a word of eight takes four of each and a shift.  The sums of a
// group are fp32 (the matrix unit cuts off where an addition would round) and
// are scaled and added up in fp32; what is summed is q x itself, so a term whose
// code is 0 takes nothing from the others, however large its x, and an infinity
// gives what the definition does.  (Codes left at n, with 8 sum x taken off
// again, saved the multiply-adds, but cost the results the bits of 8 sum |x|.
// The e4m3 instruction would take a mask per four codes, but it runs as
// conversions and f16 products here: 40 instructions for one.)
//
// The bound is the read of the codes, then instruction issue: an item of 16
// rows and 4 chunks (4 KB) is due every 180 cycles of an SM at full bandwidth,
// and takes some 540 instructions with up to 8 vectors, besides 150 cycles of
// the L1 data path (the operands from shared memory, and 8 cycles for a load of
// 8 rows).  So each warp streams its own items straight into registers, each
// chunk's loads for the next item issued as soon as the chunk has been
// multiplied, across tiles, with no barrier in between; x stays in shared
// memory for all tiles of a block, one block of 16 warps per SM, since staging
// it costs every block the same reads of L2.  The warps of a block form teams:
// a team takes a tile of 16 rows (SwiGLU: 8 gate rows and their 8 up rows), its
// warps split the tile's items, leave their parts in shared memory, and one of
// them in turn adds the parts up a tile later, so no warp waits for the slowest
// at every tile.  Rings in shared memory, filled by bulk or tensor copies, had
// as many bytes in flight, but cost a warp 300 instructions per item.  Where
// the vectors do not fit (large B K) or their staging outweighs the products, a
// cluster of blocks splits K and adds the parts up through distributed shared
// memory.
//
// Measured: 131071 rows of 4096, groups of 64, three vectors 52.0 us (286 MB,
// 5.5 TB/s, 0.81 of the copy bandwidth; 61 % of the issue slots, 62 % of the L1
// data path); 24576 rows (SwiGLU), one vector 14.7 us (3.5 TB/s: 4 us of it are
// launch, staging and the last tiles; 49 % of the issue slots); 4096 x 4096, one
// vector 5.1 us; 4096 x 12288, groups of 32, 13 vectors 14.2 us (43 % of the
// issue slots).  Two accumulators per group, for the even and odd words, are no
// faster: 53.2, 15.2, 5.9 and 14.9 us where one had 52.3, 15.1, 5.8 and 14.5.
struct W4Args {
  const uint8_t* w;
  const uint16_t* scale;
  const float* bias;
  const uint16_t* x;
  void* y;
  int B, N, K;
  int nch;     // chunks of a row
  int segc;    // chunks of a row per block of the cluster, a multiple of 4
  int units;   // tiles
  int n_out;   // columns of y
  int team;    // warps of a team, a power of two
  int team_log, cluster_log;
  int slots;   // tiles whose parts wait for one cluster exchange
  int swiglu;
  int f32_out;
  unsigned* status;
};

constexpr int kW4Warps = 16;
constexpr int kW4WarpsLog = 4;
constexpr int kW4Slots = 16;  // most tiles whose parts wait for one cluster exchange
constexpr int kW4Chunks = 4;  // chunks of an item
constexpr int kW4Pitch = 20;  // floats between the columns of a warp's part: conflict-free fragment stores

// d = a b + c.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
      "%12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// The codes in the lowest four bits of w's halves, and those four bits further
// up, as pairs of bf16 q 2^-6.
constexpr uint32_t kBf2m3 = 0xBE00BE00u;  // -2^-3, twice
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return fma_bf16x2(w & 0x000F000Fu, 0x7F007F00u, kBf2m3); }  // 2^127
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return fma_bf16x2(w & 0x00F000F0u, 0x7D007D00u, kBf2m3); }  // 2^123
// The scales of a row's item: lane c of the row's four holds the 128 / G of
// chunk c, so that one load fetches an item's (a load of 8 rows costs the L1
// data path 8 cycles, whatever it fetches of each; with each lane loading
// every chunk's the logits took 56.4 us).
template <int G>
struct W4Scales {
  static constexpr int W = G == 32 ? 2 : 1;
  uint32_t v[W];
  // volatile: asked for where the code says
  __device__ __forceinline__ void load(const uint16_t* p) {
    if (G == 32) {
      asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[W - 1]) : "l"(p));
    } else if (G == 64) {
      asm volatile("ld.global.u32 %0, [%1];" : "=r"(v[0]) : "l"(p));
    } else {
      asm volatile("ld.global.u16 %0, [%1];" : "=r"(v[0]) : "l"(p));
    }
  }
  // those of chunk ci, to all lanes of the row
  __device__ __forceinline__ W4Scales of(int ci) const {
    W4Scales s;
#pragma unroll
    for (int i = 0; i < W; ++i) s.v[i] = __shfl_sync(0xffffffffu, v[i], ci, 4);
    return s;
  }
  __device__ __forceinline__ float get(int group) const {
    return (group & 1) ? bf16_hi(v[group / 2]) : bf16_lo(v[group / 2]);
  }
};

// Shared memory: the warps' parts of two tiles [2][8][8 NT vectors][20],
// (cluster) finished parts [slots][teams][8 NT][16], then the vectors in their
// order, 64 bytes between them so that two neighbours lie in different halves of
// the banks.  Columns that no vector has take the last vector: a column's sums
// depend on that column alone, and theirs are read by nobody.
template <int NT>
struct W4Smem {
  static constexpr int part = NT * 8 * kW4Pitch;  // floats of a warp's part
  static constexpr int red = 2 * kW4Warps * part * 4;
  static constexpr int res = NT * 128 * 4;  // of a slot
};
__host__ __device__ constexpr int w4_pitch(int segc) { return segc * 256 + 64; }

__device__ __forceinline__ void w4_store(const W4Args& a, int n, int col, float v) {
  if (a.f32_out)
    static_cast<float*>(a.y)[(long long)col * a.n_out + n] = v;
  else
    static_cast<uint16_t*>(a.y)[(long long)col * a.n_out + n] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
}

// Copies the block's part of the vectors, 16 bytes at a time, zeros beyond K
// (a multiple of 32: no piece is cut).  Asynchronous, every piece in flight at
// once, and through L1 (4096 x 4096, one vector 5.1 us; past it 5.8); the caller
// waits for its own with stage_wait and for the others' with a barrier.
__device__ __forceinline__ void w4_stage(const W4Args& a, int c0, uint8_t* xs) {
  const int per = a.segc * 16, pitch = w4_pitch(a.segc);  // pieces of a vector
  const int db = kW4Warps * 32 / per, dj = kW4Warps * 32 - db * per;
  int b = threadIdx.x / per, j = threadIdx.x - b * per;
  const uint32_t dst = smem_u32(xs);
  while (b < a.B) {
    const int k = c0 * 128 + 8 * j;
    const uint16_t* src = a.x + (long long)b * a.K + min(k, a.K - 8);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst + b * pitch + 16 * j), "l"(src),
                 "r"(k < a.K ? 16 : 0)
                 : "memory");
    b += db, j += dj;
    if (j >= per) j -= per, ++b;
  }
}
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Codes are read once: not kept in L1.  An item's 256 bytes of a row come to L2
// with the first of its four loads (logits 54.1 to 51.7 us).
__device__ __forceinline__ uint4 ld_stream16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int G, int NT, bool CL>
__global__ void __launch_bounds__(kW4Warps * 32, 1) gemv_w4_kernel(const W4Args a) {
  using SM = W4Smem<NT>;
  constexpr int CW = kW4Chunks;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kW4Warps * 4];
  __shared__ int sh_abort;
  float* red = reinterpret_cast<float*>(smem);
  float* res = red + SM::red / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int team = warp >> a.team_log, wt = warp & (a.team - 1), teams = kW4Warps >> a.team_log;
  uint8_t* xs = reinterpret_cast<uint8_t*>(res + (CL ? a.slots * teams * (SM::res / 4) : 0));
  volatile int* abort_flag = &sh_abort;
  const uint32_t part_full0 = smem_u32(bars + 4 * team), part_free0 = part_full0 + 16;  // [2] per buffer of parts
  const int csize = CL ? 1 << a.cluster_log : 1, rank = CL ? (int)cluster_ctarank() : 0;
  // the team's tiles
  const int first = (CL ? blockIdx.x >> a.cluster_log : blockIdx.x) * teams + team;
  const int stride = (CL ? gridDim.x >> a.cluster_log : gridDim.x) * teams;
  const int c0 = rank * a.segc;  // this block's chunks [c0, c0 + nc)
  const int nc = max(0, min(a.segc, a.nch - c0));
  const int groups = (nc + CW - 1) / CW;
  const int items = groups > wt ? (groups - wt + a.team - 1) >> a.team_log : 0;  // of this warp per tile
  const int n_tiles = first < a.units ? (a.units - first + stride - 1) / stride : 0;
  // of the block's first team: the others have as many, or one less
  const int most_tiles = first - team < a.units ? (a.units - first + team + stride - 1) / stride : 0;

  // The lane's two rows of a tile, g and g + 8 (SwiGLU: gate row g, up row g),
  // as one pointer each to codes and scales; both move by a constant from tile
  // to tile.  Rows past the end are not loaded, and their sums not stored.
  const int rpt = a.swiglu ? 8 : 16;  // output rows of a tile
  int left[2];                        // rows from the lane's row to the last one
  const uint8_t* wp[2];
  const uint16_t* sp[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = first * rpt + g + (a.swiglu ? 0 : 8 * hh);
    const long long at = (long long)(a.swiglu && hh ? a.n_out + r : r) * a.nch + c0 + wt * CW;
    left[hh] = a.n_out - r;
    wp[hh] = a.w + at * 64 + 16 * c;
    sp[hh] = a.scale + at * (128 / G);
  }
  const long long step = (long long)stride * rpt * a.nch;  // chunks
  uint4 wv[CW][2];
  W4Scales<G> sv[2] = {}, sn[2] = {};
#pragma unroll
  for (int hh = 0; hh < 2; ++hh)
#pragma unroll
    for (int ci = 0; ci < CW; ++ci) wv[ci][hh] = make_uint4(0, 0, 0, 0);
  // chunk ci of item i of the tile that the pointers stand at
  auto load_chunk = [&](int i, int ci) {
    const int j = (wt + i * a.team) * CW + ci;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      if (left[hh] > 0 && j < nc) wv[ci][hh] = ld_stream16(wp[hh] + (i * a.team * CW + ci) * 64);
  };
  auto load_scales = [&](int i) {
    const int j = (wt + i * a.team) * CW + c;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      if (left[hh] > 0 && j < nc) sn[hh].load(sp[hh] + (i * a.team * CW + c) * (128 / G));
  };
  grid_wait();
  grid_release();
  if (n_tiles > 0 && items > 0) {
    load_scales(0);
#pragma unroll
    for (int ci = 0; ci < CW; ++ci) load_chunk(0, ci);
  }
  w4_stage(a, c0, xs);

  if (lane == 0) {
    if (wt == 0)
      for (int i = 0; i < 2; ++i) mbar_init(part_full0 + 8 * i, a.team), mbar_init(part_free0 + 8 * i, 1);
    if (warp == 0) sh_abort = 0;
    fence_barrier_init();
  }
  stage_wait();
  __syncthreads();

  float y[NT][4];  // rows g and g + 8, vectors 8 nt + 2 c and + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 4; ++k) y[nt][k] = 0.f;
  const uint8_t* xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xrow[nt] = xs + min(nt * 8 + g, a.B - 1) * w4_pitch(a.segc) + c * 16;

  // row of the tile in the matrix, for the bias; past the end: the last row
  auto bias_of = [&](int u, int r) -> float {
    if (!a.bias) return 0.f;
    const int n = min(u * rpt + (a.swiglu ? r & 7 : r), a.n_out - 1);
    return a.bias[a.swiglu && r >= 8 ? a.n_out + n : n];
  };
  // Row r of tile u and vector col, with the sums v (and for SwiGLU the up
  // row's, v2).
  auto store = [&](int u, int r, int col, float v, float v2) {
    const int n = u * rpt + r;
    if (n < a.n_out) w4_store(a, n, col, a.swiglu ? silu_f(v) * v2 : v);
  };
  // Adds up the team's parts of its k-th tile and finishes the outputs.
  auto finish = [&](int k) {
    const int u = first + k * stride, r = lane & 15;  // lanes 0 .. 15 and 16 .. 31 hold one vector's rows each
    const float* buf = red + (k & 1) * (SM::red / 8) + team * a.team * SM::part + (lane >> 4) * kW4Pitch + r;
    const float b0 = CL ? 0.f : bias_of(u, r);
    mbar_wait_warp(part_full0 + 8 * (k & 1), (k >> 1) & 1, abort_flag, a.status, ST_TIMEOUT_EPILOGUE);
    float v[4 * NT];  // vectors 2 i and 2 i + 1; behind the last one nothing that is stored
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) v[i] = buf[2 * i * kW4Pitch];
#pragma unroll 1
    for (int w = 1; w < a.team; ++w) {
      buf += SM::part;
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) v[i] += buf[2 * i * kW4Pitch];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(part_free0 + 8 * (k & 1));
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) {
      if (2 * i >= a.B) break;
      const int col = 2 * i + (lane >> 4);
      v[i] *= 64.0f;  // out of the units of 2^-6
      if (CL) {
        if (col < a.B) res[(((k % a.slots) << (kW4WarpsLog - a.team_log)) + team) * NT * 128 + col * 16 + r] = v[i];
      } else {
        v[i] += b0;
        const float v2 = __shfl_xor_sync(0xffffffffu, v[i], 8);  // SwiGLU: the up row
        if (col < a.B && (!a.swiglu || r < 8)) store(u, r, col, v[i], v2);
      }
    }
  };

  int finished = 0;  // tiles
#pragma unroll 1
  for (int k = 0; k < (CL ? most_tiles : n_tiles); ++k) {
    if (!CL || k < n_tiles) {
#pragma unroll 1
      for (int i = 0; i < items; ++i) {
        const int j0 = (wt + i * a.team) * CW;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) sv[hh] = sn[hh];
        int ni = i + 1;
        bool more = true;
        if (ni == items) {
          ni = 0, more = k + 1 < n_tiles;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) wp[hh] += step * 64, sp[hh] += step * (128 / G), left[hh] -= stride * rpt;
        }
        if (more) load_scales(ni);
        // Chunks beyond K meet zeros: x is zero there, up to whole items, and the
        // registers hold some codes and some finite scales.
        const uint8_t* xj[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xj[nt] = xrow[nt] + j0 * 256;
#pragma unroll
        for (int ci = 0; ci < CW; ++ci) {
          const W4Scales<G> sg = sv[0].of(ci), sh = sv[1].of(ci);
          float acc[NT][4];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            if (32 * i4 % G == 0) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
            }
            const uint4 &lo = wv[ci][0], &hi = wv[ci][1];
            const uint32_t wg = i4 == 0 ? lo.x : i4 == 1 ? lo.y : i4 == 2 ? lo.z : lo.w;
            const uint32_t wh = i4 == 0 ? hi.x : i4 == 1 ? hi.y : i4 == 2 ? hi.z : hi.w;
            const uint32_t vg = wg >> 8, vh = wh >> 8;
            const uint32_t q0 = codes_lo(wg), q1 = codes_lo(wh), q2 = codes_hi(wg), q3 = codes_hi(wh);
            const uint32_t q4 = codes_lo(vg), q5 = codes_lo(vh), q6 = codes_hi(vg), q7 = codes_hi(vh);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 xb = *reinterpret_cast<const uint4*>(xj[nt] + ci * 256 + i4 * 64);
              float(&q)[4] = acc[nt];
              mma_bf16(q, q0, q1, q2, q3, xb.x, xb.y, q[0], q[1], q[2], q[3]);
              mma_bf16(q, q4, q5, q6, q7, xb.z, xb.w, q[0], q[1], q[2], q[3]);
            }
            if (32 * (i4 + 1) % G == 0) {
              const float s0 = sg.get(32 * i4 / G), s1 = sh.get(32 * i4 / G);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                y[nt][0] = fmaf(s0, acc[nt][0], y[nt][0]);
                y[nt][1] = fmaf(s0, acc[nt][1], y[nt][1]);
                y[nt][2] = fmaf(s1, acc[nt][2], y[nt][2]);
                y[nt][3] = fmaf(s1, acc[nt][3], y[nt][3]);
              }
            }
          }
          if (more) load_chunk(ni, ci);
        }
      }
      // the warp's part of the tile goes to one of two buffers
      if (k >= 2)
        mbar_wait_warp(part_free0 + 8 * (k & 1), ((k >> 1) & 1) ^ 1, abort_flag, a.status, ST_TIMEOUT_EPILOGUE);
      float* mine = red + (k & 1) * (SM::red / 8) + warp * SM::part;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* p = mine + (nt * 8 + 2 * c) * kW4Pitch + g;
        p[0] = y[nt][0], p[kW4Pitch] = y[nt][1], p[8] = y[nt][2], p[kW4Pitch + 8] = y[nt][3];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[nt][q] = 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(part_full0 + 8 * (k & 1));
    }
    const int done = k + 1;
    const bool flush = done == (CL ? most_tiles : n_tiles) || (CL && done % a.slots == 0);
    for (const int upto = min(flush ? done : k, n_tiles); finished < upto; ++finished)
      if (finished % a.team == wt) finish(finished);
    if (CL && flush) {
      // The teams of one place in the blocks of a cluster have the same tiles:
      // exchange the parts of the last ones, each block finishing a share of
      // the outputs.  (A team without a tile in the last round leaves no part:
      // that tile is past the end and nothing of it is stored.)
      const int slots = (done - 1) % a.slots + 1, t0 = done - slots;
      // A half warp takes the 16 rows (SwiGLU: its first lanes the 8 outputs)
      // of one vector of one tile.  The first ones' biases are on their way while
      // the blocks wait for each other.
      constexpr int H = kW4Warps * 2;
      const int n = slots * teams * a.B, r = threadIdx.x & 15;
      auto tile_of = [&](int sl) {
        return first - team + (sl & (teams - 1)) + (t0 + (sl >> (kW4WarpsLog - a.team_log))) * stride;
      };
      float bias[2];
      auto load_bias = [&](int e) {
        const int u = tile_of(e / a.B);
        bias[0] = bias_of(u, r), bias[1] = a.swiglu ? bias_of(u, r | 8) : 0.f;
      };
      const int e0 = rank * H + (int)(threadIdx.x / 16);
      load_bias(e0);
      __syncwarp();
      cluster_sync();
      for (int e = e0; e < n; e += csize * H) {
        const int sl = e / a.B, col = e - sl * a.B;
        if (r >= rpt) continue;
        if (e != e0) load_bias(e);
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          if (hh && !a.swiglu) break;
          const uint32_t at = smem_u32(res + sl * NT * 128 + col * 16 + r + 8 * hh);
          float t[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            t[q] = 0.f;
            if (q < csize) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(t[q]) : "r"(mapa_shared(at, q)));
          }
          v[hh] = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7])) + bias[hh];
        }
        store(tile_of(sl), r, col, v[0], v[1]);
      }
      __syncwarp();
      cluster_sync();
    }
  }
}

// dynamic shared memory of a block (227 KB, some of it static)
constexpr int kW4Room = 226 * 1024;

// Chunks of a block of a cluster: whole items.
int w4_segment(int nch, int csize) { return ((nch + csize - 1) / csize + kW4Chunks - 1) / kW4Chunks * kW4Chunks; }

template <int G, int NT>
int w4_least(int B, int segc, bool cl) {
  return W4Smem<NT>::red + (cl ? W4Smem<NT>::res : 0) + B * w4_pitch(segc);
}

// Tiles of a team between two exchanges of a cluster, with `left` bytes beside
// the first part's.
template <int NT>
int w4_slots(int left, int team, int rounds) {
  const int teams = kW4Warps / team;
  return std::max(1, std::min({left / W4Smem<NT>::res + 1, kW4Slots, rounds * teams}) / teams);
}

// How a product is cut: clusters of csize blocks along K, teams along N.
struct W4Plan {
  int csize, segc, team, rounds;
};

// A team's warps split the items of a tile.  A large team fills the SMs with
// few tiles, a small one has more items per tile to set against the tile's own
// cost (leaving the parts, adding them up), about half an item's.  A cluster
// divides the vectors to be staged by its blocks, at the cost of exchanges.
// In cycles of an SM, as measured: 17 for a chunk of a vector (every SM reads
// the same lines of L2, at 15 bytes a cycle), 3000 for an item of each of 16
// warps (4000 with more than 8 vectors), 10000 for an exchange with the wait
// for the slowest block.  13 vectors, 4096 rows: K = 12288 took 14.9 us in
// clusters of 4, 17.4 of 2, 24.9 of 8; K = 4096 took 8.4 us without, 8.4 in
// clusters of 4, 8.6 of 2; the cut chosen was within 3 % of the fastest one for
// ten shapes of 1 to 16 vectors.
template <int G, int NT>
W4Plan w4_plan(const W4Args& a, int csize, int most, double& cost) {
  W4Plan p = {csize, w4_segment(a.nch, csize), 0, 0};
  const int left = kW4Room - w4_least<G, NT>(a.B, p.segc, csize > 1);
  const int groups = p.segc / kW4Chunks;
  for (int team = kW4Warps; left >= 0 && team >= 1; team /= 2) {
    if (csize > 1 && (kW4Warps / team - 1) * W4Smem<NT>::res > left) break;  // no room for a part of each team's tile
    if (team > 1 && team / 2 >= groups) continue;                            // warps without an item
    const int need = (a.units + kW4Warps / team - 1) / (kW4Warps / team);
    const int r = (need + most - 1) / most;
    const int slots = w4_slots<NT>(left, team, r);
    const double c = 17.0 * a.B * p.segc + r * ((groups + team - 1) / team + 0.5) * (NT == 1 ? 3000 : 4000) +
                     (csize > 1 ? 10000.0 * ((r + slots - 1) / slots) : 0.0);
    if (p.team == 0 || c < cost) cost = c, p.team = team, p.rounds = r;
  }
  return p;
}

template <int G, int NT, bool CL>
cudaError_t launch_w4(const W4Args& a_in, const W4Plan& p, cudaStream_t st) {
  using SM = W4Smem<NT>;
  W4Args a = a_in;
  a.segc = p.segc, a.team = p.team;
  a.status = device_status_ptr();
  while ((1 << a.team_log) < a.team) ++a.team_log;
  while ((1 << a.cluster_log) < p.csize) ++a.cluster_log;
  // evened out over the rounds
  const int teams = kW4Warps / a.team, need = (a.units + teams - 1) / teams;
  const int ncl = (need + p.rounds - 1) / p.rounds;
  // parts of all teams' tiles between two exchanges of a cluster
  const int least = w4_least<G, NT>(a.B, a.segc, CL);
  a.slots = CL ? w4_slots<NT>(kW4Room - least, a.team, p.rounds) : 0;
  const int smem = least + (CL ? (a.slots * teams - 1) * SM::res : 0);
  launch_begin(KID_GEMV_W4, st);
  const cudaError_t e =
      launch_after(gemv_w4_kernel<G, NT, CL>, dim3(ncl * p.csize), dim3(kW4Warps * 32), smem, p.csize, st, a);
  launch_end(st);
  return e;
}

template <int G, int NT>
cudaError_t launch_w4_n(const W4Args& a, cudaStream_t st) {
  // Clusters that run at once.  Blocks that fill an SM each leave SMs of a
  // graphics processing cluster over (GB300: 36 clusters of 4, not 38); one
  // more than fit costs a second wave.
  struct Setup {
    std::once_flag once;
    cudaError_t err;
    int most[4];
  };
  static Setup setup[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Setup& s = setup[dev];
  std::call_once(s.once, [&] {
    s.err = cudaFuncSetAttribute(gemv_w4_kernel<G, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Room);
    if (s.err == cudaSuccess)
      s.err = cudaFuncSetAttribute(gemv_w4_kernel<G, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Room);
    s.most[0] = num_sms();
    for (int i = 1; i < 4 && s.err == cudaSuccess; ++i) {
      cudaLaunchConfig_t q = {};
      q.gridDim = dim3(1 << i), q.blockDim = dim3(kW4Warps * 32), q.dynamicSmemBytes = kW4Room;
      cudaLaunchAttribute qa[1];
      qa[0].id = cudaLaunchAttributeClusterDimension;
      qa[0].val.clusterDim.x = 1 << i, qa[0].val.clusterDim.y = 1, qa[0].val.clusterDim.z = 1;
      q.attrs = qa, q.numAttrs = 1;
      s.err = cudaOccupancyMaxActiveClusters(&s.most[i], gemv_w4_kernel<G, NT, true>, &q);
      s.most[i] = std::max(1, s.most[i]);
    }
  });
  if (s.err != cudaSuccess) return s.err;
  // 8 blocks hold every shape
  W4Plan best = {};
  double least = 0;
  for (int i = 0; i < 4; ++i) {
    double cost = 0;
    const W4Plan p = w4_plan<G, NT>(a, 1 << i, s.most[i], cost);
    if (p.team && (!best.team || cost < least)) best = p, least = cost;
  }
  if (!best.team) return cudaErrorInvalidConfiguration;
  return best.csize > 1 ? launch_w4<G, NT, true>(a, best, st) : launch_w4<G, NT, false>(a, best, st);
}

template <int G>
cudaError_t launch_w4_g(W4Args a, cudaStream_t st) {
  a.units = a.swiglu ? (a.n_out + 7) / 8 : (a.n_out + 15) / 16;
  return a.B <= 8 ? launch_w4_n<G, 1>(a, st) : launch_w4_n<G, 2>(a, st);
}

bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

constexpr int kW4MaxK = 32768;

}  // namespace

}  // namespace mmdit

using namespace mmdit;

extern "C" {

int mmdit_rms_norm(const void* x, int x_dtype, const void* delta, int delta_dtype, int64_t rows, int D, int64_t x_ld,
                   int64_t delta_ld, const float* gain, float eps, void* x_out, void* y, uint8_t* q, float* s,
                   void* stream) {
  if (rows < 0) return MMDIT_ERR_ARG;
  if (rows > 0 && (!x || !gain || (!y && !q) || (q != nullptr) != (s != nullptr))) return MMDIT_ERR_ARG;
  if (x_dtype != MMDIT_F32 && x_dtype != MMDIT_BF16) return MMDIT_ERR_ARG;
  if (delta && delta_dtype != MMDIT_F32 && delta_dtype != MMDIT_BF16) return MMDIT_ERR_ARG;
  if (rows > 0 && !delta && x_out) return MMDIT_ERR_ARG;
  if (D < 8 || D % 8 || D > 32768 || rows > (1ll << 31) - 1) return MMDIT_ERR_SHAPE;
  if (x_ld < D || x_ld % 8 || (delta && (delta_ld < D || delta_ld % 8))) return MMDIT_ERR_SHAPE;
  if (!al16(x) || !al16(gain) || (delta && !al16(delta)) || (x_out && !al16(x_out)) || (y && !al16(y)) ||
      (q && !al16(q)) || (s && (reinterpret_cast<uintptr_t>(s) & 3u)))
    return MMDIT_ERR_ALIGN;
  if (rows == 0) return MMDIT_OK;
  MMDIT_TRY(device_check());
  RmsArgs a;
  a.x = x, a.delta = delta, a.gain = gain, a.x_out = x_out, a.y = static_cast<uint16_t*>(y), a.q = q, a.s = s;
  a.rows = rows, a.x_ld = x_ld, a.delta_ld = delta_ld, a.nv = D / 8, a.eps = eps;
  return cuda_status(launch_rms_norm(a, x_dtype == MMDIT_F32, !delta ? 0 : delta_dtype == MMDIT_F32 ? 2 : 1, S(stream)));
}

int mmdit_quantize_w4(const void* w, int w_dtype, int N, int K, int group, uint8_t* q, void* scale, void* stream) {
  if (!w || !q || !scale) return MMDIT_ERR_ARG;
  if (w_dtype != MMDIT_F32 && w_dtype != MMDIT_BF16) return MMDIT_ERR_ARG;
  if (N < 1 || !group_ok(group) || K < group || K % group || K > kW4MaxK) return MMDIT_ERR_SHAPE;
  if (!al16(w) || !al16(q) || !al16(scale)) return MMDIT_ERR_ALIGN;
  MMDIT_TRY(device_check());
  const int C = (K + 127) / 128;
  const long long units = (long long)N * C, grid = (units + 7) / 8;
  if (grid > (1ll << 31) - 1) return MMDIT_ERR_SHAPE;
  cudaStream_t st = S(stream);
  launch_begin(KID_QUANTIZE_W4, st);
  if (w_dtype == MMDIT_F32)
    quantize_w4_kernel<true><<<(unsigned)grid, 256, 0, st>>>(w, N, K, C, group, reinterpret_cast<uint32_t*>(q),
                                                             static_cast<uint16_t*>(scale));
  else
    quantize_w4_kernel<false><<<(unsigned)grid, 256, 0, st>>>(w, N, K, C, group, reinterpret_cast<uint32_t*>(q),
                                                              static_cast<uint16_t*>(scale));
  launch_end(st);
  return cuda_status(cudaGetLastError());
}

int mmdit_gemv_w4(const mmdit_linear_w4_t* lin, int B, int N, int K, const void* x, int epilogue, void* y,
                  void* stream) {
  if (!lin || !lin->w || !lin->scale || !x || !y) return MMDIT_ERR_ARG;
  if (epilogue != MMDIT_EPI_BF16 && epilogue != MMDIT_EPI_F32 && epilogue != MMDIT_EPI_SWIGLU) return MMDIT_ERR_ARG;
  if (B < 1 || B > 16 || N < 1 || N > (1 << 30) || !group_ok(lin->group) || K < lin->group || K % lin->group ||
      K > kW4MaxK)
    return MMDIT_ERR_SHAPE;
  if (epilogue == MMDIT_EPI_SWIGLU && N % 2) return MMDIT_ERR_SHAPE;
  if (!al16(lin->w) || !al16(lin->scale) || (lin->b && !al16(lin->b)) || !al16(x) || !al16(y)) return MMDIT_ERR_ALIGN;
  MMDIT_TRY(device_check());
  W4Args a = {};
  a.w = static_cast<const uint8_t*>(lin->w);
  a.scale = static_cast<const uint16_t*>(lin->scale);
  a.bias = lin->b;
  a.x = static_cast<const uint16_t*>(x);
  a.y = y;
  a.B = B, a.N = N, a.K = K, a.nch = (K + 127) / 128;
  a.swiglu = epilogue == MMDIT_EPI_SWIGLU;
  a.f32_out = epilogue == MMDIT_EPI_F32;
  a.n_out = a.swiglu ? N / 2 : N;
  cudaStream_t st = S(stream);
  return cuda_status(lin->group == 32 ? launch_w4_g<32>(a, st) : lin->group == 64 ? launch_w4_g<64>(a, st)
                                                                                      : launch_w4_g<128>(a, st));
}

}  // extern "C"
