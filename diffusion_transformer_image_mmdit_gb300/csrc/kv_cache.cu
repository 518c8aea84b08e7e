// The paged key/value cache of a language model's token step: the append with
// the rotation of queries and keys, and attention over the cache, with their
// entry points of the C ABI.
//
// The cache holds e4m3 codes in blocks of 64 tokens with one power-of-two
// scale per block, kv head and tensor:
//   k [n_blocks][H_kv][64][d], v [n_blocks][H_kv][d][64]
// so a block's keys of one head, and its values, are contiguous (4 or 8 KB):
// one bulk copy each.  v is kept transposed because the tokens of a channel
// are neighbours along the axis that P V sums over.  Powers of two: when a
// later token of a block needs a larger scale, the codes that are there move
// down by whole exponents, exactly but for those that fall below the smallest
// normal code; a code's relative precision does not depend on the scale.
#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda_fp16.h>

#include "capi_util.h"
#include "mmdit.h"
#include "mmdit_internal.h"
#include "token.cuh"

namespace mmdit {

namespace {

constexpr int kBlk = MMDIT_KV_BLOCK;

// Two e4m3 codes (the low half of v) to f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
  return d;
}

struct KvDims {
  int B, H, Hkv, G;
  int n_blocks, table_ld, n_new, max_new, max_len;
};

struct KvPtrs {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;
  const int32_t* len;
  const int32_t* start;
  unsigned* status;
};

// First row, first row of the next sequence, and length of sequence b, as the
// arrays have them; and whether they lie within the cache and the rows.
__device__ __forceinline__ int3 kv_seq_raw(const KvPtrs& p, int b) {
  int3 r;  // volatile: asked for where the code says, which is ahead of use
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.x) : "l"(p.start + b));
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.y) : "l"(p.start + b + 1));
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.z) : "l"(p.len + b));
  return r;
}
__device__ __forceinline__ bool kv_seq_ok(const KvDims& d, int3 r) {
  return r.x >= 0 && r.y >= r.x && r.y <= d.n_new && r.y - r.x <= d.max_new && r.z >= 0 && r.z <= d.max_len;
}

// ------------------------------------------------------------------ append
constexpr int kQueryHeads = 4;  // of a block that rotates queries

struct AppendArgs {
  KvDims d;
  KvPtrs p;
  const uint16_t* qkv;
  long long qkv_ld;
  const float* gq;
  const float* gk;
  const float* cs;
  const float* sn;
  uint16_t* q_out;
  int heads;  // blocks for the kv heads' keys, and for their values
  int roles;  // blocks of one cache block: `heads` for keys, `heads` for values, then one per kQueryHeads heads
  float eps;
};

// A head's row is held by VH = d / 8 lanes, 8 channels each: 8 v .. 8 v + 7, or,
// where channels i and i + d / 2 turn together, 4 v .. 4 v + 3 and the four
// d / 2 behind them, so that a lane holds both of each pair.
template <bool HALVES>
__device__ __forceinline__ uint4 load_head(const uint16_t* first, int second) {
  if (!HALVES) return *reinterpret_cast<const uint4*>(first);
  const uint2 a = *reinterpret_cast<const uint2*>(first), b = *reinterpret_cast<const uint2*>(first + second);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Cosines and sines of one position for a lane's four pairs.
struct Turn {
  float c[4], s[4];
  __device__ __forceinline__ void load(int v, int half, long long pos, const float* cs, const float* sn) {
    const float4 a = *reinterpret_cast<const float4*>(cs + pos * half + 4 * v);
    const float4 b = *reinterpret_cast<const float4*>(sn + pos * half + 4 * v);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
    s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
  }
};

// Each product is rounded by itself (no fused multiply-add), so the result is
// the one of an elementwise rotation with these tables, bit for bit.
template <int ROPE>
__device__ __forceinline__ void rotate8(float* x, const Turn& t) {
  if (ROPE == MMDIT_ROPE_NONE) return;
  constexpr int P = ROPE == MMDIT_ROPE_PAIRS ? 2 : 1, Q = ROPE == MMDIT_ROPE_PAIRS ? 1 : 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[P * i], b = x[P * i + Q];
    x[P * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
    x[P * i + Q] = __fadd_rn(__fmul_rn(a, t.s[i]), __fmul_rn(b, t.c[i]));
  }
}

// RMS norm over a head with gain g.
template <int VH, bool HALVES>
__device__ __forceinline__ void head_norm8(float* x, int v, const float* g, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int o = VH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(ss * (1.0f / (VH * 8)) + eps);
  const float4 a = *reinterpret_cast<const float4*>(g + (HALVES ? 4 : 8) * v);
  const float4 b = *reinterpret_cast<const float4*>(g + (HALVES ? VH * 4 + 4 * v : 8 * v + 4));
  const float gg[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * gg[i];
}

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
}

// |x| for the block's maximum: an infinity does not set the scale (its code
// saturates at 448), and fmaxf drops NaN (whose code is NaN).
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a == INFINITY ? 0.f : a;
}

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), at least -100.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127;
  const int e = (u & 0x7FFFFFu) <= 0x600000u ? k - 8 : k - 7;
  return max(e, -100);
}
__device__ __forceinline__ int scale_exponent(float s) {
  return max(-100, min(120, (int)((__float_as_uint(s) >> 23) & 255) - 127));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 .. 127

// Four codes (one word) at 2^shift of their values, shift <= 0.
__device__ __forceinline__ uint32_t move_codes(uint32_t w, float factor) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t f = e4m3x2_f16x2((uint16_t)(w >> (16 * h)));
    const __half2 v = *reinterpret_cast<const __half2*>(&f);
    out |= (uint32_t)f8x2_e4m3(__low2float(v) * factor, __high2float(v) * factor) << (16 * h);
  }
  return out;
}

// Blocks of 256 threads, of three kinds, per touched cache block and sequence;
// all kinds of one cache block lie side by side in the grid (24 prompts 94.9 us,
// one token 3.5; one kind after the other 93.9 and 3.6).
//   keys of NH kv heads: rotates them, finds their maxima, sets the scales
//     (moving the codes that are there if a scale grows) and writes the codes;
//   values of NH kv heads: the same without a rotation, transposed through
//     shared memory, so that whole words of a channel are written;
//   queries of kQueryHeads heads: rotates them, the next heads' loads in flight
//     while one batch is turned, on one position's cosines and sines (2 or 8
//     heads per block take 108 us for 95).
// Keys and values wait in registers as they came between the maximum and the
// codes.  Bound by the read of the rows and the write of queries and codes, and
// by having enough loads in flight: 64 registers leave four blocks on an SM
// (three blocks of 80: 104 us).  24 prompts of 77 to 2048 tokens (32 query, 8 kv
// heads of 128) move 575 MB in 95 us, 6.1 TB/s, 0.89 of the copy bandwidth; one
// token of one sequence takes 3.5 us, three loads one behind the other.
template <int HD, int NH, int ROPE>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const AppendArgs a) {
  constexpr int NTH = 256;
  constexpr int VH = HD / 8;      // lanes of a head
  constexpr bool HALVES = ROPE == MMDIT_ROPE_HALVES;
  constexpr int TP = NTH / VH;    // tokens per pass
  constexpr int P = kBlk / TP;    // passes
  constexpr int PITCH = kBlk + 4;
  __shared__ __align__(16) uint8_t sv[HD * PITCH];
  __shared__ uint32_t red[NH][NTH / 32];
  const KvDims& d = a.d;
  const int b = blockIdx.y, jblk = blockIdx.x / a.roles, h = blockIdx.x - jblk * a.roles, tid = threadIdx.x;
  grid_wait();
  grid_release();
  const int3 seq = kv_seq_raw(a.p, b);
  const int s0 = seq.x, T = seq.y - seq.x, len = seq.z;
  if (!kv_seq_ok(d, seq) || len < T) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(a.p.status, kStatusBadIndex);
    return;
  }
  const int first = len - T, blk = first / kBlk + jblk, p0 = blk * kBlk;
  if (T == 0 || p0 >= len) return;
  const int lo = max(first - p0, 0), hi = min(len - p0, kBlk);
  const int v = tid % VH, tt = tid / VH;
  const long long row0 = s0 + p0 - first;  // row of the block's slot 0 (may lie before the sequence's rows)

  if (h >= 2 * a.heads) {  // queries
    const int h0 = (h - 2 * a.heads) * kQueryHeads, nh = min(kQueryHeads, d.H - h0);
    // The heads of one pass, the next pass's loads in flight while they are
    // turned.  A lane whose slot gets no token repeats the nearest one that does,
    // and stores nothing.
    uint4 u[kQueryHeads], un[kQueryHeads];
    auto slot_of = [&](int p) { return min(max(p * TP + tt, lo), hi - 1); };
    auto load_q = [&](int p) {
      const uint16_t* src = a.qkv + (row0 + slot_of(p)) * a.qkv_ld + (long long)h0 * HD + (HALVES ? 4 : 8) * v;
#pragma unroll
      for (int k = 0; k < kQueryHeads; ++k)
        if (k < nh) un[k] = load_head<HALVES>(src + k * HD, HD / 2);
    };
    const int last = (hi - 1) / TP;
    load_q(lo / TP);
#pragma unroll 1
    for (int p = lo / TP; p <= last; ++p) {
      const int slot = slot_of(p);
      Turn turn;
      if (ROPE != MMDIT_ROPE_NONE) turn.load(v, HD / 2, p0 + slot, a.cs, a.sn);
#pragma unroll
      for (int k = 0; k < kQueryHeads; ++k) u[k] = un[k];
      if (p < last) load_q(p + 1);
      const bool live = slot == p * TP + tt;
      uint16_t* dst = a.q_out + (row0 + slot) * ((long long)d.H * HD) + (long long)h0 * HD;
#pragma unroll
      for (int k = 0; k < kQueryHeads; ++k) {
        if (k >= nh) break;
        float x[8];
        unpack8(u[k], x);
        if (a.gq) head_norm8<VH, HALVES>(x, v, a.gq, a.eps);
        rotate8<ROPE>(x, turn);
        if (!live) continue;
        const uint2 lo4 = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        const uint2 hi4 = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        if (HALVES) {
          *reinterpret_cast<uint2*>(dst + k * HD + 4 * v) = lo4;
          *reinterpret_cast<uint2*>(dst + k * HD + HD / 2 + 4 * v) = hi4;
        } else {
          *reinterpret_cast<uint4*>(dst + k * HD + 8 * v) = make_uint4(lo4.x, lo4.y, hi4.x, hi4.y);
        }
      }
    }
    return;
  }

  // keys (h < heads) or values of NH kv heads from h0 on
  const bool vals = h >= a.heads;
  const int h0 = NH * (vals ? h - a.heads : h), nh = min(NH, d.Hkv - h0);
  const int at = HALVES && !vals ? 4 * v : 8 * v, second = HALVES && !vals ? HD / 2 : 4;
  uint4 u[NH][P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int slot = p * TP + tt;
    const uint16_t* r = a.qkv + (row0 + slot) * a.qkv_ld + (long long)(d.H + (vals ? d.Hkv : 0) + h0) * HD + at;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      u[n][p] = make_uint4(0, 0, 0, 0);
      if (slot >= lo && slot < hi && n < nh) u[n][p] = load_head<HALVES>(r + n * HD, second);
    }
  }
  const int id = a.p.table[(long long)b * d.table_ld + blk];
  if (id < 0 || id >= d.n_blocks) {
    if (tid == 0 && h == 0) atomicOr(a.p.status, kStatusBadIndex);
    return;
  }
  float* sp = (vals ? a.p.vs : a.p.ks) + (long long)id * d.Hkv + h0;
  float s_old[NH] = {};  // the block's scales so far, where it holds older tokens
#pragma unroll
  for (int n = 0; n < NH; ++n)
    if (lo > 0 && n < nh) s_old[n] = sp[n];

  // the keys of pass p, rotated: once for the maximum and once more for the
  // codes, so that only their 16 bytes wait in registers in between
  auto turn_of = [&](int p, Turn& turn) {
    if (ROPE != MMDIT_ROPE_NONE) turn.load(v, HD / 2, p0 + min(max(p * TP + tt, lo), hi - 1), a.cs, a.sn);
  };
  auto key = [&](uint4 raw, const Turn& turn, float* x) {
    unpack8(raw, x);
    if (a.gk) head_norm8<VH, HALVES>(x, v, a.gk, a.eps);
    rotate8<ROPE>(x, turn);
  };
  // The maxima over the block's new tokens, as bits; an infinity, which sets no
  // scale, is rare enough for a second look at everything without it.  A NaN is
  // dropped by fmaxf (keys) and stands above infinity as a pattern (values).
  uint32_t top[NH];
  auto maxima = [&](bool finite) {
    float m[NH] = {};
    uint32_t mb[NH] = {};  // |v|: two bf16 patterns at a time, which order as integers
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (p * TP + TP <= lo || p * TP >= hi) continue;  // the same for the whole block
      Turn turn;
      if (!vals) turn_of(p, turn);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (vals && !finite) {
          mb[n] = __vmaxu2(mb[n], __vmaxu2(__vmaxu2(u[n][p].x & 0x7FFF7FFFu, u[n][p].y & 0x7FFF7FFFu),
                                           __vmaxu2(u[n][p].z & 0x7FFF7FFFu, u[n][p].w & 0x7FFF7FFFu)));
        } else {
          float x[8];
          if (vals)
            unpack8(u[n][p], x);
          else
            key(u[n][p], turn, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) m[n] = fmaxf(m[n], finite ? finite_abs(x[i]) : fabsf(x[i]));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const uint32_t w =
          __reduce_max_sync(0xffffffffu, max(__float_as_uint(m[n]), max(mb[n] << 16, mb[n] & 0xFFFF0000u)));
      if ((tid & 31) == 0) red[n][tid >> 5] = w;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      top[n] = 0;
#pragma unroll
      for (int i = 0; i < NTH / 32; ++i) top[n] = max(top[n], red[n][i]);
    }
  };
  maxima(false);
  if (max(top[0], top[NH - 1]) >= 0x7F800000u) {  // the same for the whole block
    __syncthreads();
    maxima(true);
  }
  int e_old[NH], e_new[NH];
#pragma unroll
  for (int n = 0; n < NH; ++n) {
    e_old[n] = lo > 0 ? scale_exponent(s_old[n]) : -100;
    e_new[n] = max(block_exponent(__uint_as_float(top[n])), e_old[n]);
    if (tid == 0 && n < nh) sp[n] = exp2_int(e_new[n]);
  }
  uint8_t* codes = (vals ? a.p.v : a.p.k) + ((long long)id * d.Hkv + h0) * (kBlk * HD);
  if (!vals) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (p * TP + TP <= lo || p * TP >= hi) continue;
      const int slot = p * TP + tt;
      Turn turn;
      turn_of(p, turn);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        float x[8];
        key(u[n][p], turn, x);
        if (slot < lo || slot >= hi || n >= nh) continue;
        const float inv = exp2_int(-e_new[n]);
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = (uint32_t)f8x2_e4m3(x[4 * j] * inv, x[4 * j + 1] * inv) |
                 ((uint32_t)f8x2_e4m3(x[4 * j + 2] * inv, x[4 * j + 3] * inv) << 16);
        uint8_t* to = codes + n * (kBlk * HD) + slot * HD + at;
        if (HALVES) {
          *reinterpret_cast<uint32_t*>(to) = w[0];
          *reinterpret_cast<uint32_t*>(to + HD / 2) = w[1];
        } else {
          *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      if (n >= nh || lo == 0 || e_new[n] == e_old[n]) continue;
      const float down = exp2f((float)(e_old[n] - e_new[n]));
      uint32_t* w = reinterpret_cast<uint32_t*>(codes + n * (kBlk * HD));
      for (int i = tid; i < lo * HD / 4; i += NTH) w[i] = move_codes(w[i], down);
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < NH; ++n) {
    if (n >= nh) break;
    if (n) __syncthreads();  // the first head's values have been read
    const float inv = exp2_int(-e_new[n]);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int slot = p * TP + tt;
      if (slot < lo || slot >= hi) continue;
      float x[8];
      unpack8(u[n][p], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t c2 = f8x2_e4m3(x[2 * j] * inv, x[2 * j + 1] * inv);
        sv[(8 * v + 2 * j) * PITCH + slot] = (uint8_t)c2;
        sv[(8 * v + 2 * j + 1) * PITCH + slot] = (uint8_t)(c2 >> 8);
      }
    }
    __syncthreads();
    uint32_t* w = reinterpret_cast<uint32_t*>(codes + n * (kBlk * HD));
    if (lo == 0 && hi == kBlk) {  // a whole block
#pragma unroll
      for (int i = tid; i < HD * (kBlk / 4); i += NTH)
        w[i] = *reinterpret_cast<const uint32_t*>(sv + i / (kBlk / 4) * PITCH + i % (kBlk / 4) * 4);
      continue;
    }
    const bool move = lo > 0 && e_new[n] > e_old[n];
    const float down = exp2f((float)(e_old[n] - e_new[n]));
    // words w0 .. w1 - 1 of each channel hold a slot that is written
    const int w0 = move ? 0 : lo / 4, w1 = (hi + 3) / 4;
    for (int i = tid; i < HD * (kBlk / 4); i += NTH) {
      const int ch = i / (kBlk / 4), k = i % (kBlk / 4);
      if (k < w0 || k >= w1) continue;
      const int n0 = max(lo - 4 * k, 0), n1 = min(hi - 4 * k, 4);  // new bytes [n0, n1) of the word
      uint32_t val = *reinterpret_cast<const uint32_t*>(sv + ch * PITCH + 4 * k);
      uint32_t* at = w + ch * (kBlk / 4) + k;
      if (n0 <= 0 && n1 >= 4) {
        *at = val;
      } else if (!move) {  // some bytes of the word, without reading it
        for (int e = n0; e < n1; ++e) reinterpret_cast<uint8_t*>(at)[e] = (uint8_t)(val >> (8 * e));
      } else {
        // bytes below n0: older tokens; from n1 on: no token yet, left as they are
        const uint32_t old = *at;
        const uint32_t below = n0 >= 4 ? 0xFFFFFFFFu : (1u << (8 * n0)) - 1u;
        const uint32_t upto = n1 >= 4 ? 0xFFFFFFFFu : (1u << (8 * n1)) - 1u;
        *at = (move_codes(old, down) & below) | (val & ~below & upto) | (old & ~upto & ~below);
      }
    }
  }
}

// ------------------------------------------------------------------ attention
// Row (token t of T, query head h G + g) of sequence b sees the keys below
// len - T + t + 1.  The rows of one kv head are taken 8 or 16 at a time (a
// row tile); a unit is a row tile of one (sequence, kv head) over the
// sequence's blocks.
//
// S^T = K Q^T and O^T = V^T P^T: the keys, then the channels, are the 16-row
// operand of m16n8k16 and the query rows its 8-column operand, so up to 8
// rows (one token of a group of up to 8 heads) waste nothing.  The codes
// become f16 (exact); q is f16 after a power of two per row has brought its
// largest element to [2^14, 2^15) (an element of 2^-31 of that stays exact);
// P is f16, so that both products have 11-bit operands and fp32 sums, and
// the block's key scale goes to the exponent's argument, its value scale to
// the fp32 sum of the blocks.  P's reference lies 14 below the maximum
// (p_reference): a p stays normal, off by 2^-11 of itself at most, down to
// 2^-28 of the largest, and by 2^-39 of the largest below, so that a token
// which stands far above 2^28 others does not drop what they give together.
//
// Bound: the read of the codes, 2 d bytes per token and kv head.  Every warp
// has its own ring of slots of one block of keys or of values, filled by bulk
// copies that one lane issues as soon as a slot has been read, and its own
// running maximum, sum and output, so warps wait for nothing but their own
// copies; the warps of a block merge once per piece.  The blocks of all units
// are numbered through and cut into equal ranges, one per thread block: a
// long sequence is read by as many SMs as a batch of short ones.  A unit that
// is cut goes to fp32 parts in the workspace, which a second kernel adds up
// in a fixed order.
//
// Two blocks per SM: the outputs of 16 rows and 128 channels, the queries and
// the scores fill 255 registers (three blocks of 168 registers and rings of two
// slots were slower: 48 sequences 73.5 us for 70.5, one long 59.7 for 55.0).
// Measured with 32 query and 8 kv heads of 128: one token of 48 sequences of 33
// to 8192 70 us (405 MB, 5.8 TB/s, 0.85 of the copy bandwidth), three tokens of
// one sequence of 131069 51.9 us (5.2 TB/s, 0.76: of twice the length the second
// half takes 40 us, the copy bandwidth; 12 us are the way to the first block, the
// SMs that are slower than others, and the merge), one token behind 511 6.7 us in
// one launch of 8 blocks: six loads one behind the other, then two items of keys
// and of values per warp, and the merge of the warps.
//
// Prompts are right but not fast here: every 16 rows of a kv head read and widen
// the cache anew, and every such tile is a unit with its fixed cost (one prompt of
// 512 43.6 us, of 2048 330; 24 of 77 to 2048 2.85 ms).
constexpr int kKvMaxCtas = 320;
constexpr int kKvWarps = 4;
constexpr int kKvRing = 24576;      // bytes of a warp's ring
constexpr int kKvCtaMinBlocks = 4;  // least blocks per thread block when units are cut
// Units of up to so many blocks are not cut (no workspace, one launch).  One token
// each of 1, 4 and 16 sequences, us, whole and cut: of 512 tokens 6.6, 6.9, 7.2 and
// 6.9, 7.8, 10.0; of 1024 tokens 9.3, 9.6, 10.4 and 6.9, 8.0, 12.3; of 2048 tokens
// 14.9, 15.2, 16.6 and 7.0, 11.1, 19.0.
constexpr int kKvWholeBlocks = 8;
// What a unit costs beside its blocks (queries, merge), in blocks.  With 0, 4, 10
// and 16, us: 48 sequences of 33 to 8192 tokens 88.7, 73.7, 70.3, 70.9; 16 of 2000
// to 6000 30.2, 29.5, 28.5, 29.2; 200 of 100 to 1500 98.8, 71.4, 64.2, 65.7; one of
// 60000 and 40 of 300 48.9, 39.2, 32.3, 32.4.
constexpr int kKvUnitCost = 10;

struct KvAttnArgs {
  KvDims d;
  KvPtrs p;
  const uint16_t* q;
  uint16_t* out;
  float* part;  // [grid][2][R][HD], then stats [grid][2][R][2]
  float scale_log2;
  int split;
};

// Units and their sizes of sequence b: rt row tiles, the length of a unit in the
// numbering (1 where units are not cut; else kKvUnitCost places that stand for
// no block, then one per block), and the total for all kv heads.
struct KvSeq {
  int s0, T, len, rt, nb;
  long long w;
};
template <int R>
__device__ __forceinline__ KvSeq kv_units(const KvAttnArgs& a, int3 raw) {  // {start[b], start[b + 1], len[b]}
  KvSeq s;
  const bool ok = kv_seq_ok(a.d, raw);
  s.s0 = raw.x, s.T = ok ? raw.y - raw.x : 0, s.len = ok ? raw.z : 0;
  s.rt = (s.T * a.d.G + R - 1) / R;
  s.nb = a.split ? max(1, (s.len + kBlk - 1) / kBlk) + kKvUnitCost : 1;
  s.w = (long long)s.rt * a.d.Hkv * s.nb;
  return s;
}

// Sum of v over a block of W warps, and the sum over the threads before this one.
template <int W>
__device__ __forceinline__ long long block_scan(long long v, long long& before, long long (&sh)[W]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  long long pre = 0, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) pre += sh[w];
    all += sh[w];
  }
  before = pre + inc - v;
  return all;
}

// n / d for n >= 0, d > 0, in 32 bits where both fit (nearly always: a block
// begins with three of these one behind the other).
__device__ __forceinline__ long long div_pos(long long n, long long d) {
  if (((n | d) >> 32) == 0) return (long long)((uint32_t)n / (uint32_t)d);
  return n / d;
}

__device__ __forceinline__ int kv_ctas(long long total, int grid, int split) {
  const long long most = split ? (total + kKvCtaMinBlocks - 1) / kKvCtaMinBlocks : total;
  return (int)max(1ll, min((long long)grid, most));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t word_of(const uint4& u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// The reference that p = 2^(score - reference) is taken against, from a maximum:
// p reaches kPTop = 2^14, of f16's 65504.  Where the fp32 steps of the scores
// are so coarse that 14 could round to more, the maximum itself; any reference
// serves, since a row's sum l and its output go by the same one.  The output is
// kept in units of kPTop (kPUnit rides on the blocks' value scales), so that it
// has the range of the values.
constexpr float kPTop = 16384.0f, kPUnit = 1.0f / 16384.0f;
__device__ __forceinline__ float p_reference(float m) { return fabsf(m) < 1048576.0f ? m - 14.0f : m; }

template <int HD, int NT>
__global__ void __launch_bounds__(128, 2) kv_attention_kernel(const KvAttnArgs a) {
  constexpr int R = 8 * NT;
  constexpr uint32_t ITEM = kBlk * HD;         // bytes of a block's keys, or values, of one head
  constexpr int NS = kKvRing / ITEM;           // slots: 3 (d 128) or 6 (d 64)
  constexpr int OP = HD + 4;                   // floats between rows of a warp's merged output
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kKvWarps * NS];
  __shared__ long long sh_scan[4];
  __shared__ long long sh_at[2];
  __shared__ int3 sh_raw;
  __shared__ float sh_m[kKvWarps][R], sh_l[kKvWarps][R];
  __shared__ int sh_abort, sh_nan[kKvWarps][HD];
  const KvDims& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  for (int i = lane; i < HD; i += 32) sh_nan[warp][i] = INT_MAX;
  uint8_t* ring = smem + warp * kKvRing;
  const uint32_t ring_u = smem_u32(ring), bar_u = smem_u32(bars + warp * NS);
  volatile int* abort_flag = &sh_abort;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(bar_u + 8 * i, 1);
    if (warp == 0) sh_abort = 0;
    fence_barrier_init();
  }
  grid_wait();

  // this block's range of the numbering, and the sequence that it begins in
  long long total = 0, w = 0, before = 0;
  int3 raw = make_int3(0, 0, 0);
  for (int b0 = 0; b0 < d.B; b0 += 128) {
    w = 0;
    if (b0 + tid < d.B) {
      raw = kv_seq_raw(a.p, b0 + tid);
      if (blockIdx.x == 0 && !kv_seq_ok(d, raw)) atomicOr(a.p.status, kStatusBadIndex);
      w = kv_units<R>(a, raw).w;
    }
    total += block_scan(w, before, sh_scan);
  }
  const int ctas = kv_ctas(total, gridDim.x, a.split);
  grid_release();  // kv_combine_kernel starts, and waits for this grid's end
  if ((int)blockIdx.x >= ctas || total == 0) return;
  const long long x0 = div_pos(total * blockIdx.x, ctas), x1 = div_pos(total * (blockIdx.x + 1), ctas);
  if (x0 >= x1) return;
  {
    long long at = 0;
    for (int b0 = 0; b0 < d.B; b0 += 128) {
      long long all = total;
      if (d.B > 128) {  // else the scan above was the only one
        if (b0 + tid < d.B) raw = kv_seq_raw(a.p, b0 + tid);
        w = b0 + tid < d.B ? kv_units<R>(a, raw).w : 0;
        all = block_scan(w, before, sh_scan);
      }
      if (w > 0 && at + before <= x0 && x0 < at + before + w)
        sh_at[0] = b0 + tid, sh_at[1] = at + before, sh_raw = raw;
      at += all;
    }
    __syncthreads();
  }
  int b = (int)sh_at[0];
  long long x = x0, base = sh_at[1];
  KvSeq sq = kv_units<R>(a, sh_raw);
  int3 next = kv_seq_raw(a.p, min(b + 1, d.B - 1));  // of sequence b + 1, asked for ahead
  int ahead = -1, ahead_b = -1;                      // a lane's block number of the next piece, and its sequence
  uint32_t slot_in = 0, ph_out = 0, slot_out = 0;  // ring positions of the next copy and of the next item to read
  uint32_t copies = 0, reads = 0;                  // copies issued and waited for
  bool ok = true;

  while (x < x1) {
    if (x - base >= sq.w) {
      base += sq.w;
      sq = kv_units<R>(a, next);
      ++b;
      next = kv_seq_raw(a.p, min(b + 1, d.B - 1));
      continue;
    }
    const long long off = x - base;
    const long long unit = div_pos(off, sq.nb);
    const int h = sq.rt == 1 ? (int)unit : (int)div_pos(unit, sq.rt), r0 = (int)(unit - (long long)h * sq.rt) * R;
    const int nbk = (sq.len + kBlk - 1) / kBlk;  // the sequence's blocks
    int j0 = 0, j1 = nbk;
    long long took = 1;
    if (a.split) {
      const int v0 = (int)(off - unit * sq.nb);
      took = min((long long)(sq.nb - v0), x1 - x);
      if (v0 + took <= kKvUnitCost) {  // none of the unit's blocks
        x += took;
        continue;
      }
      j0 = max(0, v0 - kKvUnitCost);
      j1 = min(nbk, v0 + (int)took - kKvUnitCost);
    }
    const bool whole = !a.split || (j0 == 0 && off - unit * sq.nb + took == sq.nb);
    const int first = sq.len - sq.T;  // position of new token 0
    const int rows = min(R, sq.T * d.G - r0);
    // the last row sees the most keys, the first one the fewest
    const int lim_lo = max(0, min(sq.len, first + r0 / d.G + 1));
    const int lim_hi = max(0, min(sq.len, first + (r0 + rows - 1) / d.G + 1));
    const int j_end = min(j1, (lim_hi + kBlk - 1) / kBlk);
    const int n_w = j_end - j0 - warp > 0 ? (j_end - j0 - warp + kKvWarps - 1) / kKvWarps : 0;  // this warp's blocks

    // the first 32 of this warp's blocks: lane l asks for the l-th's number
    int t_first = -1;
    {
      const int j = j0 + warp + kKvWarps * lane;
      if (j < j_end) t_first = j0 == 0 && ahead_b == b ? ahead : a.p.table[(long long)b * d.table_ld + j];
    }

    // the lane's part of the queries (channels 16 c .. 16 c + 15 of each 64 of
    // row g of each 8 rows), asked for before the blocks' numbers are waited for
    uint4 qr[NT][HD / 32];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = r0 + nt * 8 + g, t = rr / d.G, hq = rr - t * d.G;
      const uint16_t* qp = a.q + ((long long)(sq.s0 + t) * d.H + (long long)h * d.G + hq) * HD + 16 * c;
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) {
        qr[nt][i] = make_uint4(0, 0, 0, 0);
        if (nt * 8 + g < rows) qr[nt][i] = *reinterpret_cast<const uint4*>(qp + 64 * (i >> 1) + 8 * (i & 1));
      }
    }

    // 32 of this warp's blocks at a time: lane l holds block number, scales of the l-th
    int id_n = 0;
    float ks_n = 0.f, vs_n = 0.f;
    auto window = [&](int i) {
      const int j = j0 + warp + kKvWarps * (i + lane);
      id_n = 0, ks_n = 0.f, vs_n = 0.f;
      if (j < j_end) {
        const int t = i == 0 ? t_first : a.p.table[(long long)b * d.table_ld + j];
        if (t >= 0 && t < d.n_blocks) {
          id_n = t;
          ks_n = a.p.ks[(long long)t * d.Hkv + h];
          vs_n = a.p.vs[(long long)t * d.Hkv + h];
        } else {
          id_n = -1, ks_n = 1.f;  // left out: its keys are masked
          atomicOr(a.p.status, kStatusBadIndex);
        }
      }
    };
    int m_in = 0;  // items (block's keys, then its values) issued for this piece
    auto issue = [&]() {
      const int i = m_in >> 1;
      if (i >= n_w) return;
      if ((m_in & 1) == 0 && (i & 31) == 0) window(i);
      const int id = max(0, __shfl_sync(0xffffffffu, id_n, i & 31));
      const uint8_t* src = ((m_in & 1) ? a.p.v : a.p.k) + ((long long)id * d.Hkv + h) * ITEM;
      __syncwarp();
      if (lane == 0) {
        mbar_expect_tx(bar_u + 8 * slot_in, ITEM);
        bulk_load(ring_u + slot_in * ITEM, src, ITEM, bar_u + 8 * slot_in);
      }
      ++m_in, ++copies;
      if (++slot_in == NS) slot_in = 0;
    };
    auto wait_item = [&]() -> const uint8_t* {
      const uint8_t* at = ring + slot_out * ITEM;
      ok = mbar_wait_warp(bar_u + 8 * slot_out, ph_out, abort_flag, a.p.status, ST_TIMEOUT_SOFTMAX) && ok;
      ++reads;
      if (++slot_out == NS) slot_out = 0, ph_out ^= 1;
      return at;
    };
    if (ok)
      for (int i = 0; i < NS; ++i) issue();
    // the block numbers that the next piece begins with: of this sequence or,
    // behind its last unit, of the next one
    {
      const bool same = x + took - base < sq.w;
      ahead_b = same ? b : b + 1;
      const int j = warp + kKvWarps * lane;
      const int n = same ? sq.len : b + 1 < d.B && kv_seq_ok(d, next) ? next.z : 0;
      ahead = -1;
      if (x + took < x1 && j < (n + kBlk - 1) / kBlk)
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(ahead) : "l"(a.p.table + (long long)ahead_b * d.table_ld + j));
    }

    // Q^T operand
    uint32_t qf[NT][HD / 16][2];
    float sc[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x8[HD / 4];
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) unpack8(qr[nt][i], x8 + 8 * i);
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) mx = fmaxf(mx, finite_abs(x8[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = mx > 0.f ? max(-112, min(127, (int)(__float_as_uint(mx) >> 23) - 127)) - 14 : 0;
      const float down = exp2_int(-e);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        qf[nt][i][0] = pack_f16x2(x8[4 * i] * down, x8[4 * i + 1] * down);
        qf[nt][i][1] = pack_f16x2(x8[4 * i + 2] * down, x8[4 * i + 3] * down);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // columns 2 c + k of the accumulators
        const int ec = __shfl_sync(0xffffffffu, e, (2 * c + k) * 4);
        sc[nt][k] = a.scale_log2 * exp2_int(ec);
        const int row = nt * 8 + 2 * c + k;
        lim[nt][k] = row < rows ? max(0, min(sq.len, first + (r0 + row) / d.G + 1)) : sq.len;
      }
    }

    float o[HD / 16][NT][4];
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) m_run[nt][k] = -INFINITY, l_run[nt][k] = 0.f;
#pragma unroll
    for (int dt = 0; dt < HD / 16; ++dt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[dt][nt][k] = 0.f;

    int id_w = 0;
    float ks_w = 0.f, vs_w = 0.f;
#pragma unroll 1
    for (int i = 0; i < n_w && ok; ++i) {
      if ((i & 31) == 0) id_w = id_n, ks_w = ks_n, vs_w = vs_n;  // copies run at most 3 blocks ahead
      const int j = j0 + warp + kKvWarps * i;
      const bool lost = __shfl_sync(0xffffffffu, id_w, i & 31) < 0;
      const float ks = __shfl_sync(0xffffffffu, ks_w, i & 31);
      const float vs = __shfl_sync(0xffffffffu, vs_w, i & 31) * kPUnit;
      const bool edge = j * kBlk + kBlk > lim_lo || lost;  // some row does not see all of the block's keys

      const uint8_t* kt = wait_item();
      if (!ok) break;
      // scores: accumulator rows g and g + 8 of tile mt are the keys
      // 16 (g / 2) + 4 mt + g % 2 and that + 2, so that P V finds the 4 mt-th
      // word of a lane's 16 value bytes beside them
      float s[4][NT][4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.f;
        const int key = 16 * (g >> 1) + 4 * mt + (g & 1);
#pragma unroll
        for (int hc = 0; hc < HD / 64; ++hc) {
          const uint4 ka = *reinterpret_cast<const uint4*>(kt + key * HD + hc * 64 + 16 * c);
          const uint4 kb = *reinterpret_cast<const uint4*>(kt + (key + 2) * HD + hc * 64 + 16 * c);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t wa = word_of(ka, t), wb = word_of(kb, t);
            const uint32_t a0 = e4m3x2_f16x2((uint16_t)wa), a2 = e4m3x2_f16x2((uint16_t)(wa >> 16));
            const uint32_t a1 = e4m3x2_f16x2((uint16_t)wb), a3 = e4m3x2_f16x2((uint16_t)(wb >> 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(s[mt][nt], a0, a1, a2, a3, qf[nt][hc * 4 + t][0], qf[nt][hc * 4 + t][1]);
          }
        }
      }
      issue();

      if (edge) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = j * kBlk + 16 * (g >> 1) + 4 * mt + (g & 1) + 2 * (k >> 1);
              if (lost || key >= lim[nt][k & 1]) s[mt][nt][k] = -INFINITY;
            }
      }
      float alpha[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // Neither 0 nor so large that a product with a sum (below 2^32) leaves
          // the range: a masked score, -infinity, stays one, a score of 0 stays
          // 0, and no other becomes infinite.  Every score is rounded by
          // itself, as the maximum is: with the exact product in its place the
          // largest one's distance from the maximum would be that rounding,
          // 2^5 and more for scores of 2^29.
          const float f = fminf(fmaxf(sc[nt][k] * ks, 1.17549435e-38f), 3.9614081e28f);  // 2^-126, 2^95
          float mx = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) mx = fmaxf(mx, s[mt][nt][2 * e + k]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(m_run[nt][k], p_reference(__fmul_rn(mx, f)));
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: every p is 0
          alpha[nt][k] = ex2_approx(m_run[nt][k] - ref);
          m_run[nt][k] = m_new;
          float l = 0.f;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = ex2_approx(__fmul_rn(s[mt][nt][2 * e + k], f) - ref);
              s[mt][nt][2 * e + k] = p;
              l += p;
            }
          l_run[nt][k] = l_run[nt][k] * alpha[nt][k] + l;
        }
      }
      // a maximum that stays, which is the rule behind the first blocks, leaves
      // the output as it is
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) grew = grew || alpha[nt][0] != 1.f || alpha[nt][1] != 1.f;
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int dt = 0; dt < HD / 16; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[dt][nt][k] *= alpha[nt][k & 1];
      }
      uint32_t pb[4][NT][2];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pb[mt][nt][e] = transpose8x8(pack_f16x2(s[mt][nt][2 * e], s[mt][nt][2 * e + 1]));

      uint8_t* vt = const_cast<uint8_t*>(wait_item());
      if (!ok) break;
      // Values behind the sequence are masked out of the product (0 * NaN):
      // word t of a lane's 16 bytes holds the keys 16 c + 4 t .. + 3.
      uint32_t keep[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
      bool nan_found = false;
      if (edge) {
        const int end = lost ? 0 : min(sq.len - j * kBlk, kBlk), lo = lost ? 0 : max(lim_lo - j * kBlk, 0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int n = end - (16 * c + 4 * t);
          keep[t] = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        }
        if (lo < end) {
          // A NaN (code 0x7F or 0xFF) that not every row sees is taken out of
          // the tile too; rows that do see it get it below.
          uint32_t any = 0;
          for (int i = lane; i < HD * 4; i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + 16 * i);
            any |= ((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u) |
                   ((v.z & 0x7F7F7F7Fu) + 0x01010101u) | ((v.w & 0x7F7F7F7Fu) + 0x01010101u);
          }
          if (__any_sync(0xffffffffu, (any & 0x80808080u) != 0)) {
#pragma unroll 1
            for (int i = lane; i < HD * kBlk; i += 32) {
              const int key = i % kBlk;
              if (key >= lo && key < end && (vt[i] & 0x7F) == 0x7F) {
                vt[i] = 0;
                nan_found = true;
                atomicMin(&sh_nan[warp][i / kBlk], j * kBlk + key);
              }
            }
            nan_found = __any_sync(0xffffffffu, nan_found);
            fence_proxy_async_smem();  // the slot's next copy comes after these stores
            __syncwarp();
          }
        }
      }
#pragma unroll
      for (int dt = 0; dt < HD / 16; ++dt) {
        uint4 va = *reinterpret_cast<const uint4*>(vt + (16 * dt + g) * kBlk + 16 * c);
        uint4 vb = *reinterpret_cast<const uint4*>(vt + (16 * dt + g + 8) * kBlk + 16 * c);
        if (edge) {
          va.x &= keep[0], va.y &= keep[1], va.z &= keep[2], va.w &= keep[3];
          vb.x &= keep[0], vb.y &= keep[1], vb.z &= keep[2], vb.w &= keep[3];
        }
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t wa = word_of(va, t), wb = word_of(vb, t);
          const uint32_t a0 = e4m3x2_f16x2((uint16_t)wa), a2 = e4m3x2_f16x2((uint16_t)(wa >> 16));
          const uint32_t a1 = e4m3x2_f16x2((uint16_t)wb), a3 = e4m3x2_f16x2((uint16_t)(wb >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, pb[t][nt][0], pb[t][nt][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[dt][nt][k] = fmaf(vs, acc[nt][k], o[dt][nt][k]);
      }
      issue();
      if (nan_found) {  // channel ch is NaN for the rows that see key sh_nan[ch]
#pragma unroll
        for (int dt = 0; dt < HD / 16; ++dt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (lim[nt][k & 1] > sh_nan[warp][16 * dt + g + 8 * (k >> 1)]) o[dt][nt][k] = NAN;
        __syncwarp();
        for (int i = lane; i < HD; i += 32) sh_nan[warp][i] = INT_MAX;
        __syncwarp();
      }
    }

    // ---- merge the warps: each writes its rows and statistics; its ring is
    // free (every copy of the piece has been read)
    const bool all_ok = __syncthreads_and(ok);
    if (!all_ok) {
      ok = false;
      break;
    }
    float* om = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = l_run[nt][k];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) sh_m[warp][nt * 8 + 2 * c + k] = m_run[nt][k], sh_l[warp][nt * 8 + 2 * c + k] = l;
      }
#pragma unroll
      for (int dt = 0; dt < HD / 16; ++dt)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          om[(nt * 8 + 2 * c + (k & 1)) * OP + 16 * dt + g + 8 * (k >> 1)] = o[dt][nt][k];
    }
    __syncthreads();
    const int slot = blockIdx.x * 2 + (x == x0 ? 0 : 1);
    for (int e = tid; e < rows * (HD / 2); e += 128) {
      const int row = e / (HD / 2), ch = 2 * (e - row * (HD / 2));
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) m = fmaxf(m, sh_m[w][row]);
      const float ref = m == -INFINITY ? 0.f : m;
      float l = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) {
        const float f = ex2_approx(sh_m[w][row] - ref);
        const float2 t = *reinterpret_cast<const float2*>(smem + w * kKvRing + (row * OP + ch) * 4);
        l = fmaf(f, sh_l[w][row], l), v0 = fmaf(f, t.x, v0), v1 = fmaf(f, t.y, v1);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : kPTop / l;  // a row that sees no key: zeros
        const int t = (r0 + row) / d.G, hq = r0 + row - t * d.G;
        *reinterpret_cast<uint32_t*>(a.out + ((long long)(sq.s0 + t) * d.H + (long long)h * d.G + hq) * HD + ch) =
            pack_bf16x2(v0 * inv, v1 * inv);
      } else {
        *reinterpret_cast<float2*>(a.part + ((long long)slot * R + row) * HD + ch) = make_float2(v0, v1);
        if (ch == 0)
          *reinterpret_cast<float2*>(a.part + (long long)gridDim.x * 2 * R * HD + ((long long)slot * R + row) * 2) =
              make_float2(m, l);
      }
    }
    fence_proxy_async_smem();  // the next piece's copies overwrite what was read here
    __syncthreads();
    x += took;
  }
  if (!ok) {
    // a wait was given up: wait (bounded) for the copies still in flight into
    // this block's shared memory before it is released
    while (reads < copies) {
      mbar_wait(bar_u + 8 * slot_out, ph_out, nullptr, nullptr, 0, 100000000ull);
      ++reads;
      if (++slot_out == NS) slot_out = 0, ph_out ^= 1;
    }
  }
}

// Adds up the parts of the units that were cut, one block per unit and row, its
// W warps taking every W-th part (a long sequence alone is cut into as many
// parts as its kv head has thread blocks), then merged in a fixed order.  The
// grid's x dimension goes over the units or, where fewer (as with many tokens,
// or bounds above the lengths: units are numbered by the shape's bounds), over
// the boundaries between the attention's blocks: a unit that is cut is merged by
// the first boundary inside it.  Few registers (48 per thread; 40 with 16
// warps): blocks come on an SM beside one of the attention's, and find their
// unit while others still read.
template <int HD, int NT, int W>
__global__ void __launch_bounds__(W * 32) kv_combine_kernel(const KvAttnArgs a, int grid, int rt_max, int by_unit) {
  constexpr int R = 8 * NT;
  constexpr int CL = HD / 32;  // channels of a lane
  __shared__ long long sh_scan[W];
  __shared__ long long sh_base;
  __shared__ int sh_b;
  __shared__ float sh_o[W][HD];
  __shared__ float2 sh_ml[W];
  // This grid starts while the attention's last blocks run: everything up to
  // grid_wait reads the arguments alone, which were there before the attention
  // released it.  Every block waits for the attention to have finished, also
  // those with nothing to do: what follows in the stream counts on both.
  const KvDims& d = a.d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = blockIdx.y;
  auto nothing = [] { grid_wait(), grid_release(); };
  int b = by_unit ? blockIdx.x / rt_max / d.Hkv : 0;
  KvSeq sq;
  if (by_unit) {
    sq = kv_units<R>(a, kv_seq_raw(a.p, b));
    const int r = blockIdx.x % rt_max;
    if (r >= sq.rt || row >= sq.T * d.G - r * R) return nothing();  // the same for the whole block
  }
  long long total = 0, w = 0, before = 0;
  for (int b0 = 0; b0 < d.B; b0 += W * 32) {
    w = b0 + tid < d.B ? kv_units<R>(a, kv_seq_raw(a.p, b0 + tid)).w : 0;
    const long long all = block_scan(w, before, sh_scan);
    if (by_unit && b0 + tid == b) sh_base = total + before;
    total += all;
  }
  const int ctas = kv_ctas(total, grid, 1), cut = blockIdx.x + 1;  // boundary: block `cut` begins at x
  long long x = 0;
  if (!by_unit) {
    if (cut >= ctas || total == 0) return nothing();
    x = div_pos(total * cut, ctas);
    long long at = 0;
    for (int b0 = 0; b0 < d.B; b0 += W * 32) {  // the sequence that x lies in
      long long all = total;
      if (d.B > W * 32) {  // else the scan above was the only one
        w = b0 + tid < d.B ? kv_units<R>(a, kv_seq_raw(a.p, b0 + tid)).w : 0;
        all = block_scan(w, before, sh_scan);
      }
      if (w > 0 && at + before <= x && x < at + before + w) sh_b = b0 + tid, sh_base = at + before;
      at += all;
    }
  }
  __syncthreads();
  const long long base = sh_base;
  int h = (blockIdx.x / rt_max) % d.Hkv, r = blockIdx.x % rt_max;
  if (!by_unit) {
    b = sh_b;
    sq = kv_units<R>(a, kv_seq_raw(a.p, b));
    const long long unit = div_pos(x - base, sq.nb);
    h = (int)div_pos(unit, sq.rt), r = (int)(unit - (long long)h * sq.rt);
    if (row >= sq.T * d.G - r * R) return nothing();
  }
  const long long u0 = base + ((long long)h * sq.rt + r) * sq.nb, u1 = u0 + sq.nb - 1;
  // the block with the largest number c such that total c / ctas <= u, for the
  // unit's first and last block
  const int c0 = (int)(((u0 + kKvUnitCost + 1) * ctas + total - 1) / total) - 1, c1 = (int)(((u1 + 1) * ctas + total - 1) / total) - 1;
  if (c0 == c1 || (!by_unit && c0 != cut - 1)) return nothing();  // not cut, or not here first
  grid_wait();
  grid_release();
  const float* stat = a.part + (long long)grid * 2 * R * HD;
  const bool first = total * c0 / ctas >= u0;  // block c0 begins with this unit
  float m = -INFINITY, l = 0.f, o[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) o[i] = 0.f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += W) {
    const long long slot = 2ll * c + (c > c0 || first ? 0 : 1);
    const float2 ml = *reinterpret_cast<const float2*>(stat + (slot * R + row) * 2);
    const float* p = a.part + (slot * R + row) * HD + lane * CL;
    float t[CL];
    if (CL == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      t[0] = v.x, t[1] = v.y, t[2 % CL] = v.z, t[3 % CL] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      t[0] = v.x, t[1] = v.y;
    }
    const float m_new = fmaxf(m, ml.x), ref = m_new == -INFINITY ? 0.f : m_new;
    const float f0 = ex2_approx(m - ref), f1 = ex2_approx(ml.x - ref);
    l = l * f0 + ml.y * f1;
#pragma unroll
    for (int i = 0; i < CL; ++i) o[i] = o[i] * f0 + t[i] * f1;
    m = m_new;
  }
#pragma unroll
  for (int i = 0; i < CL; ++i) sh_o[warp][lane * CL + i] = o[i];
  if (lane == 0) sh_ml[warp] = make_float2(m, l);
  __syncthreads();
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) mm = fmaxf(mm, sh_ml[w].x);
  const float ref = mm == -INFINITY ? 0.f : mm;
  const int rr = r * R + row, q = rr / d.G, hq = rr - q * d.G;
  uint16_t* out = a.out + ((long long)(sq.s0 + q) * d.H + (long long)h * d.G + hq) * HD;
  for (int ch = 2 * tid; ch < HD; ch += 2 * W * 32) {
    float ll = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2_approx(sh_ml[w].x - ref);
      ll = fmaf(f, sh_ml[w].y, ll), v0 = fmaf(f, sh_o[w][ch], v0), v1 = fmaf(f, sh_o[w][ch + 1], v1);
    }
    const float inv = ll == 0.f ? 0.f : kPTop / ll;
    *reinterpret_cast<uint32_t*>(out + ch) = pack_bf16x2(v0 * inv, v1 * inv);
  }
}

int kv_row_tile(const KvDims& d) { return (long long)d.max_new * d.G <= 8 ? 8 : 16; }
bool kv_split(const KvDims& d) { return (d.max_len + kBlk - 1) / kBlk > kKvWholeBlocks; }
size_t kv_part_floats(const KvDims& d, int HD) {
  return kv_split(d) ? (size_t)kKvMaxCtas * 2 * kv_row_tile(d) * (HD + 2) : 0;
}

template <int HD, int NT>
cudaError_t launch_kv_attention(KvAttnArgs a, cudaStream_t st) {
  static std::once_flag once[64];
  static cudaError_t setup_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    setup_err[dev] = cudaFuncSetAttribute(kv_attention_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          kKvWarps * kKvRing);
  });
  if (setup_err[dev] != cudaSuccess) return setup_err[dev];
  const int R = 8 * NT;
  const long long rt = ((long long)std::min(a.d.max_new, a.d.n_new) * a.d.G + R - 1) / R;
  const long long units = rt * a.d.B * a.d.Hkv;
  a.split = kv_split(a.d) ? 1 : 0;
  const long long blocks = a.split ? units * ((a.d.max_len + kBlk - 1) / kBlk) : units;
  const int grid = (int)std::min<long long>(std::min(2 * num_sms(), kKvMaxCtas), blocks);
  launch_begin(KID_KV_ATTENTION, st);
  cudaError_t e = launch_after(kv_attention_kernel<HD, NT>, dim3(grid), dim3(kKvWarps * 32), kKvWarps * kKvRing, 1, st, a);
  launch_end(st);
  if (e != cudaSuccess || !a.split) return e;
  launch_begin(KID_KV_COMBINE, st);
  const int by_unit = units < grid;
  const dim3 rows((unsigned)(by_unit ? units : std::max(1, grid - 1)),
                  (unsigned)std::min<long long>(R, (long long)a.d.max_new * a.d.G));
  // Few rows to merge have many parts each.  One sequence of 131069 took 51.4
  // us with 16 warps a row, 53 with 8, 54.3 with 4, 57.4 with 2; 48 sequences
  // 81.8, 73.1, 70.0 and 70.1; 8 sequences 28.5 with 16, 28.8 with 4.
  const bool few = (long long)rows.x * rows.y <= 2 * num_sms();
  e = launch_after(few ? kv_combine_kernel<HD, NT, 16> : kv_combine_kernel<HD, NT, 4>, rows, dim3(few ? 512 : 128), 0, 1, st,
                   a, grid, (int)rt, by_unit);
  launch_end(st);
  return e;
}

template <int HD, int NH>
cudaError_t launch_kv_append_n(AppendArgs a, int rope, cudaStream_t st) {
  a.heads = (a.d.Hkv + NH - 1) / NH;
  a.roles = 2 * a.heads + (a.q_out ? (a.d.H + kQueryHeads - 1) / kQueryHeads : 0);
  // a sequence's new tokens touch at most so many blocks
  const dim3 grid(((std::min(a.d.max_new, a.d.n_new) + kBlk - 2) / kBlk + 1) * a.roles, a.d.B);
  launch_begin(KID_KV_APPEND, st);
  const cudaError_t e = launch_after(rope == MMDIT_ROPE_NONE    ? kv_append_kernel<HD, NH, MMDIT_ROPE_NONE>
                                     : rope == MMDIT_ROPE_PAIRS ? kv_append_kernel<HD, NH, MMDIT_ROPE_PAIRS>
                                                                : kv_append_kernel<HD, NH, MMDIT_ROPE_HALVES>,
                                     grid, dim3(256), 0, 1, st, a);
  launch_end(st);
  return e;
}

// Two kv heads per block share a position's cosines and sines and have twice the
// loads in flight, one per block is done sooner.  Heads of 128, 32 query and 8
// kv: 24 prompts of 77 to 2048 tokens take 95.7 us with two, 106 with one; 8
// prompts of 64 5.9 and 6.5; 48 sequences of one new token 8.8 and 7.6, one
// sequence of one 4.9 and 3.5.
template <int HD>
cudaError_t launch_kv_append(const AppendArgs& a, int rope, cudaStream_t st) {
  return a.d.n_new >= 32ll * a.d.B ? launch_kv_append_n<HD, 2>(a, rope, st) : launch_kv_append_n<HD, 1>(a, rope, st);
}

int kv_check_shape(const mmdit_kv_shape_t* s, KvDims* d) {
  if (!s) return MMDIT_ERR_ARG;
  if (s->rope != MMDIT_ROPE_NONE && s->rope != MMDIT_ROPE_PAIRS && s->rope != MMDIT_ROPE_HALVES) return MMDIT_ERR_ARG;
  if (s->B < 1 || s->B > 65535 || s->H_kv < 1 || s->H_kv > 32767 || s->H < s->H_kv || s->H % s->H_kv || s->H > 65536)
    return MMDIT_ERR_SHAPE;
  if (s->d_head != 64 && s->d_head != 128) return MMDIT_ERR_SHAPE;
  if (s->n_blocks < 1 || s->n_new < 0 || s->max_new < 1 || s->max_len < 1 || s->max_len > (1 << 28) ||
      s->max_new > s->max_len || s->n_new > (1 << 28))
    return MMDIT_ERR_SHAPE;
  if ((long long)s->table_ld * kBlk < s->max_len) return MMDIT_ERR_SHAPE;
  if (!(s->scale >= 0.f) || std::isinf(s->scale)) return MMDIT_ERR_ARG;
  d->B = s->B, d->H = s->H, d->Hkv = s->H_kv, d->G = s->H / s->H_kv;
  d->n_blocks = s->n_blocks, d->table_ld = s->table_ld, d->n_new = s->n_new;
  d->max_new = s->max_new, d->max_len = s->max_len;
  // the query rows of one kv head, and the row tiles of one launch, are
  // numbered with 32 bits
  const long long rows = (long long)d->max_new * d->G, rt = (rows + 7) / 8;
  if (rows > (1ll << 30) || rt * d->B > (1ll << 30) || rt * d->B * d->Hkv > (1ll << 30)) return MMDIT_ERR_SHAPE;
  return MMDIT_OK;
}

int kv_check_cache(const mmdit_kv_cache_t* c, KvPtrs* p) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->len || !c->start) return MMDIT_ERR_ARG;
  if (!al16(c->k) || !al16(c->v) || !al16(c->k_scale) || !al16(c->v_scale) || !al16(c->table) || !al16(c->len) ||
      !al16(c->start))
    return MMDIT_ERR_ALIGN;
  p->k = c->k, p->v = c->v, p->ks = c->k_scale, p->vs = c->v_scale;
  p->table = c->table, p->len = c->len, p->start = c->start;
  p->status = nullptr;
  return MMDIT_OK;
}

}  // namespace

}  // namespace mmdit

using namespace mmdit;

extern "C" {

int mmdit_kv_append(const mmdit_kv_shape_t* shape, const mmdit_kv_cache_t* cache, const void* qkv, int64_t qkv_ld,
                    const float* q_norm, const float* k_norm, const float* cos_, const float* sin_, void* q_out,
                    void* stream) {
  AppendArgs a = {};
  MMDIT_TRY(kv_check_shape(shape, &a.d));
  MMDIT_TRY(kv_check_cache(cache, &a.p));
  if (a.d.n_new == 0) return MMDIT_OK;
  if (!qkv) return MMDIT_ERR_ARG;
  if ((cos_ == nullptr) != (shape->rope == MMDIT_ROPE_NONE) || (sin_ == nullptr) != (shape->rope == MMDIT_ROPE_NONE))
    return MMDIT_ERR_ARG;
  if ((q_norm == nullptr) != (k_norm == nullptr)) return MMDIT_ERR_ARG;
  if (qkv_ld < (long long)(a.d.H + 2 * a.d.Hkv) * shape->d_head || qkv_ld % 8) return MMDIT_ERR_SHAPE;
  if (!al16(qkv) || (q_out && !al16(q_out)) || (cos_ && (!al16(cos_) || !al16(sin_))) ||
      (q_norm && (!al16(q_norm) || !al16(k_norm))))
    return MMDIT_ERR_ALIGN;
  MMDIT_TRY(device_check());
  a.p.status = device_status_ptr();
  a.qkv = static_cast<const uint16_t*>(qkv), a.qkv_ld = qkv_ld;
  a.gq = q_norm, a.gk = k_norm, a.cs = cos_, a.sn = sin_;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.eps = shape->eps_rms;
  return cuda_status(shape->d_head == 128 ? launch_kv_append<128>(a, shape->rope, S(stream))
                                          : launch_kv_append<64>(a, shape->rope, S(stream)));
}

int mmdit_kv_workspace_size(const mmdit_kv_shape_t* shape, size_t* bytes) {
  if (!bytes) return MMDIT_ERR_ARG;
  KvDims d;
  MMDIT_TRY(kv_check_shape(shape, &d));
  *bytes = kv_part_floats(d, shape->d_head) * sizeof(float) + 256;
  return MMDIT_OK;
}

int mmdit_kv_attention(const mmdit_kv_shape_t* shape, const mmdit_kv_cache_t* cache, const void* q, void* out, void* ws,
                       size_t ws_bytes, void* stream) {
  KvAttnArgs a = {};
  MMDIT_TRY(kv_check_shape(shape, &a.d));
  MMDIT_TRY(kv_check_cache(cache, &a.p));
  if (a.d.n_new == 0) return MMDIT_OK;
  if (!q || !out || !ws) return MMDIT_ERR_ARG;
  if (!al16(q) || !al16(out) || !al16(ws)) return MMDIT_ERR_ALIGN;
  size_t need = 0;
  MMDIT_TRY(mmdit_kv_workspace_size(shape, &need));
  if (ws_bytes < need) return MMDIT_ERR_WORKSPACE;
  MMDIT_TRY(device_check());
  a.p.status = device_status_ptr();
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out);
  a.part = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
  const double sc = shape->scale > 0.f ? (double)shape->scale : 1.0 / std::sqrt((double)shape->d_head);
  a.scale_log2 = (float)(1.4426950408889634 * sc);
  cudaStream_t st = S(stream);
  const bool small = kv_row_tile(a.d) == 8;
  if (shape->d_head == 128)
    return cuda_status(small ? launch_kv_attention<128, 1>(a, st) : launch_kv_attention<128, 2>(a, st));
  return cuda_status(small ? launch_kv_attention<64, 1>(a, st) : launch_kv_attention<64, 2>(a, st));
}

}  // extern "C"
