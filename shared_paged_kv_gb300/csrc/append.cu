// New tokens into the pool: rotary positions on one to three axes, the
// rotated append into bf16 and 4-bit pools, and the read-back of rows.
//
// All three move rows of head_dim values once from one place to another, so
// HBM bounds them (large calls) or the chain of dependent loads that finds a
// token's place: its sequence (a search of tok_off), the sequence's length,
// the block table's entry (single-token calls).  Measured in CUDA-graph replays:
// 11,600 prompt tokens, 32 KV and 32 query heads: 88 us, 6.4 TB/s; 16,384 rows of
// 40 heads on three axes: 51 us, 6.6 TB/s; 32 single tokens: 3.5 us (as a call
// from Python 8 to 10, the host's time).  Into a 4-bit pool the codes'
// arithmetic is the limit, 60 % of the issue slots (7,900 tokens, 8 KV and 32
// query heads: 38.5 us, 4.4 TB/s; at five CTAs per SM, 48 registers, a thread of
// this kernel spills 64 bytes); read back from it, 11.7 us.  Into a microscaled pool
// (6,535 tokens, 8 / 32 heads, rotated): 30 us, 4.6 TB/s, half of the issue slots, and
// read back 13 us; twelve single tokens and their read-back 6.7 us, two launches.
//
// Split: a CTA takes 1 or 4 tokens.  Its first step finds each token's place
// and computes cos / sin once for all heads of a token (head_dim / 2 angles,
// one per thread, into shared memory).  Then a row (one head of K, V or Q) is
// taken by head_dim / 16 lanes; a lane holds elements [8v, 8v + 8) and their
// partners [d/2 + 8v, d/2 + 8v + 8), so that a rotation needs no exchange and
// every access is 16 bytes wide.
//
// Angles: turns per position f = w / 2 pi as a 64-bit fixed-point fraction F;
// pos * F modulo 2^64 is the exact phase of the rounded frequency for every
// int32 position (error below 2^-53 * f * |pos| turns), its top 32 bits the
// reduced angle of sincospif.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace kvs {

namespace {

constexpr int kApThreads = 256;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApTokens = 4;   // tokens of a CTA in large calls (two warps each)
// Rows a lane loads before it stores any, and CTAs per SM.  Measured for 7,900
// tokens into a 4-bit pool (8 KV heads, 32 query heads) / 11,600 tokens of 32
// KV and 32 query heads into a bf16 pool: 8 tokens, 4 rows 50 / 90.5 us; 4
// tokens, 4 rows 48 / 87.6; 4 tokens, 2 rows, 5 CTAs 42.7 / 88.6; 2 tokens or
// 6 CTAs slower on both.
constexpr int kApBatch = 2, kGaBatch = 2;
constexpr int kApCtas = 5;

struct Place {
  int phys, at, pos, ok;   // physical block (-1: none), row inside it, logical position; ok: the row belongs to a sequence
};

struct RowPlaces {
  const int32_t* tok_off;
  const int32_t* seq_len;
  const int32_t* table;
  uint32_t* status;
  int n_tokens, n_seq, max_blocks, capacity, block_tokens;
};

// The sequence of packed row t: the number of i in [1, n_seq] with
// tok_off[i] <= t.  Whole warp: every round 32 lanes probe the range, so up
// to 32 sequences take one trip to memory and 1,024 take two.  Whatever
// tok_off holds, the result lies in [0, n_seq].
__device__ __forceinline__ int find_seq(const int32_t* tok_off, int n_seq, int t, int lane) {
  int lo = 0, n = n_seq;
  while (n > 32) {
    const int step = (n + 31) / 32, i = (lane + 1) * step;
    const bool le = i <= n && __ldg(tok_off + lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  const bool le = lane < n && __ldg(tok_off + lo + lane + 1) <= t;
  return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// Whole warp: the place of row t in the pool.
__device__ __forceinline__ Place find_place(const RowPlaces& p, int t, int lane) {
  Place r{-1, 0, 0, 0};
  if (t >= p.n_tokens) return r;
  const int a = find_seq(p.tok_off, p.n_seq, t, lane);
  if (a >= p.n_seq) return r;
  const int t0 = __ldg(p.tok_off + a), t1 = __ldg(p.tok_off + a + 1);
  const long long pos = (long long)__ldg(p.seq_len + a) - t1 + t;
  if (t < t0 || t >= t1) return r;
  r.ok = 1;
  r.pos = (int)pos;
  if (pos < 0 || pos >= (long long)p.max_blocks * p.block_tokens) {
    if (lane == 0) set_err(p.status, KVS_DEVERR_SEQ_LEN);
    return r;
  }
  const int b = r.pos / p.block_tokens;
  const int phys = __ldg(p.table + (size_t)a * p.max_blocks + b);
  if (phys < 0 || phys >= p.capacity) {
    if (lane == 0) set_err(p.status, KVS_DEVERR_BLOCK_ID);
    return r;
  }
  r.phys = phys;
  r.at = r.pos - b * p.block_tokens;
  return r;
}

struct AppendParams {
  const uint16_t *k, *v, *q;      // rows of new tokens
  uint16_t* q_out;
  long long ks, vs, qs, qos;      // elements between two tokens' rows
  RowPlaces at;
  const int32_t* pos;             // [axes][n_tokens] or nullptr: the logical position
  uint8_t *kslab, *vslab;
  __half *ksb, *vsb;
  int hkv, hq, rotate, inverse, s0, s1;   // pairs below s0 turn with axis 0, below s1 with axis 1
  unsigned long long turn[64];    // turns per position, 64-bit fraction
};

// 4-bit codes of one 64-element group held by 8 consecutive lanes, 8 values
// each as bf16 pairs: bit for bit those of kvs_quantize_q4, rint of the
// rounded quotient (x - b) / s.
//  * The extremes are found on the bf16 values (exact): minimum and negated
//    maximum side by side in one register, so that one exchange serves both.
//  * 15 times (x - b) * (1 / (15 s)), clamped on the way, is within 2^-18 of
//    the clamped quotient, so its rint is the same unless it lies within 1e-4
//    of a half; then the quotients are taken.  Rint by the addition of
//    1.5 * 2^23, whose last place is 1.
// With a division per value and scalar extremes the call was bound by its
// instructions (7,900 tokens, 8 KV and 32 query heads: 57 us).
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t q4_codes(const uint32_t* w, __half2& sb) {
  constexpr uint32_t kNeg = 0x80008000u;
  const uint32_t lo = min_bf16x2(min_bf16x2(w[0], w[1]), min_bf16x2(w[2], w[3]));
  const uint32_t hi = min_bf16x2(min_bf16x2(w[0] ^ kNeg, w[1] ^ kNeg), min_bf16x2(w[2] ^ kNeg, w[3] ^ kNeg));
  uint32_t ext = min_bf16x2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));   // {min, -max}
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ext = min_bf16x2(ext, __shfl_xor_sync(0xffffffffu, ext, o));
  const float mn = bf16_lo(ext), mx = -bf16_hi(ext);
  const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
  const __half b16 = __float2half_rn(mn);
  const float s = __half2float(s16), b = __half2float(b16);
  sb = __halves2half2(s16, b16);
  if (s == 0.f) return 0u;
  const float inv = __frcp_rn(s) * (1.f / 15.f), magic = 12582912.f;
  const float2 b2 = make_float2(-b, -b), m2 = make_float2(magic, magic), k2 = make_float2(15.f, 15.f);
  const float2 n2 = make_float2(-magic, -magic);
  float n[8];
  bool clear = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 d = __fadd2_rn(make_float2(bf16_lo(w[e]), bf16_hi(w[e])), b2);
    const float2 y = make_float2(__saturatef(d.x * inv), __saturatef(d.y * inv));
    const float2 r = __fadd2_rn(__ffma2_rn(y, k2, m2), n2);
    const float2 off = __ffma2_rn(y, k2, make_float2(-r.x, -r.y));
    clear &= fabsf(off.x) < 0.4999f;
    clear &= fabsf(off.y) < 0.4999f;
    n[2 * e] = r.x;
    n[2 * e + 1] = r.y;
  }
  if (!clear) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[2 * e] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(bf16_lo(w[e]), b), s)), 0.f), 15.f);
      n[2 * e + 1] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(bf16_hi(w[e]), b), s)), 0.f), 15.f);
    }
  }
  // four codes as one whole number below 2^16 each, exact in float32
  const float a = fmaf(4096.f, n[3], fmaf(256.f, n[2], fmaf(16.f, n[1], n[0]))) + magic;
  const float c = fmaf(4096.f, n[7], fmaf(256.f, n[6], fmaf(16.f, n[5], n[4]))) + magic;
  return __byte_perm(__float_as_uint(a), __float_as_uint(c), 0x5410);
}

// Microscaled codes of one 32-element group held by 4 consecutive lanes, 8
// values each as bf16 pairs.  The largest magnitude is found on the bf16 bits;
// its exponent field less 2 is the scale byte, so that the largest value lies in
// [4, 8) of the scale, and the products with 2^(127 - e) are exact.
__device__ __forceinline__ uint32_t mx4_codes(const uint32_t* w, uint32_t& scale) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t top = __vmaxu2(__vmaxu2(w[0] & kAbs, w[1] & kAbs), __vmaxu2(w[2] & kAbs, w[3] & kAbs));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t e = max(top & 0xffffu, top >> 16) >> 7;
  scale = e > 2u ? min(e, 254u) - 2u : 0u;   // infinities and NaN as the largest finite exponent
  const float up = __uint_as_float((254u - scale) << 23);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]) * up;
    x[2 * i + 1] = bf16_hi(w[i]) * up;
  }
  return mx_codes(x);
}

enum { kApBf16 = 0, kApQ4 = 1, kApRows = 2, kApMx = 3 };   // pool type, or rows only (kvs_rope_apply)

template <int D, int MODE>
__global__ void __launch_bounds__(kApThreads, kApCtas) append_kernel(const __grid_constant__ AppendParams p, int tokens_per_cta) {
  constexpr int NV = D / 16;         // lanes per row
  constexpr int RPW = 32 / NV;       // rows of a warp step
  constexpr int H = D / 2;
  __shared__ __align__(16) float2 cs[kApTokens][H];
  __shared__ Place where[kApTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t_cta = blockIdx.x * tokens_per_cta;
  const int wpt = kApWarps / tokens_per_cta;    // warps that share a token
  const int slot = warp / wpt, t = t_cta + slot;
  const int v = lane % NV;
  const int rows = MODE == kApRows ? p.hq : 2 * p.hkv + p.hq;
  const int r0 = (warp % wpt) * RPW + lane / NV, rstep = wpt * RPW;

  uint4 lo[kApBatch], hi[kApBatch];
  auto load = [&](int rb) {
#pragma unroll
    for (int i = 0; i < kApBatch; ++i) {
      const int r = rb + i * rstep;
      if (r < rows && t < p.at.n_tokens) {
        const uint16_t* src;
        if (MODE == kApRows || r >= 2 * p.hkv)
          src = p.q + t * p.qs + (size_t)(MODE == kApRows ? r : r - 2 * p.hkv) * D;
        else
          src = r < p.hkv ? p.k + t * p.ks + (size_t)r * D : p.v + t * p.vs + (size_t)(r - p.hkv) * D;
        lo[i] = *reinterpret_cast<const uint4*>(src + v * 8);
        hi[i] = *reinterpret_cast<const uint4*>(src + H + v * 8);
      } else {
        lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  load(r0);   // in flight while the places are looked up

  if constexpr (MODE == kApRows) {
    if (threadIdx.x < tokens_per_cta) where[threadIdx.x] = Place{-1, 0, 0, t_cta + (int)threadIdx.x < p.at.n_tokens};
  } else if (warp < tokens_per_cta) {
    const Place w = find_place(p.at, t_cta + warp, lane);
    if (lane == 0) where[warp] = w;
  }
  if (MODE != kApRows) __syncthreads();
  if (p.rotate) {
    const int i = threadIdx.x % H;      // kApThreads is a multiple of H: one pair per thread
    const unsigned long long f = p.turn[i];
    const int axis = (i >= p.s0) + (i >= p.s1);
    for (int s = threadIdx.x / H; s < tokens_per_cta; s += kApThreads / H) {
      const int tt = t_cta + s;
      if (tt >= p.at.n_tokens) break;
      const int pos = p.pos ? __ldg(p.pos + (size_t)axis * p.at.n_tokens + tt) : where[s].pos;
      const unsigned long long ph = (unsigned long long)(long long)pos * f;
      float sn, c;
      const int top = static_cast<int>(ph >> 32);
      const float half_turns = static_cast<float>(top) * 0x1p-31f;
      sincospif(half_turns, &sn, &c);
      if constexpr (MODE == kApMx) {
        // what the conversion cut off, up to 2^-25 half turns: a key near the border of
        // two codes falls on the wrong side less often
        const float rest = (static_cast<float>(top - static_cast<long long>(static_cast<float>(top))) + static_cast<float>(static_cast<uint32_t>(ph)) * 0x1p-32f) *
                           (0x1p-31f * 3.14159265f);
        const float s1 = fmaf(c, rest, sn);
        c = fmaf(-sn, rest, c);
        sn = s1;
      }
      cs[s][i] = make_float2(c, p.inverse ? -sn : sn);
    }
  }
  __syncthreads();
  const Place w = where[slot];
  if (!w.ok) return;
  float c[8], s[8];
  if (p.rotate) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 x = *reinterpret_cast<const float4*>(&cs[slot][v * 8 + e]);
      c[e] = x.x;
      s[e] = x.y;
      c[e + 1] = x.z;
      s[e + 1] = x.w;
    }
  }
  for (int rb = r0; rb - lane / NV < rows; rb += kApBatch * rstep) {   // uniform over the warp
    if (rb != r0) load(rb);
#pragma unroll
    for (int i = 0; i < kApBatch; ++i) {
      const int r = rb + i * rstep;
      const bool is_q = MODE == kApRows || r >= 2 * p.hkv, is_v = !is_q && r >= p.hkv;
      if (p.rotate && !is_v) {
        const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
        const uint32_t hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
        uint32_t ol[4], oh[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = bf16_lo(lw[e]), a1 = bf16_hi(lw[e]), b0 = bf16_lo(hw[e]), b1 = bf16_hi(hw[e]);
          ol[e] = pack_bf16(a0 * c[2 * e] - b0 * s[2 * e], a1 * c[2 * e + 1] - b1 * s[2 * e + 1]);
          oh[e] = pack_bf16(b0 * c[2 * e] + a0 * s[2 * e], b1 * c[2 * e + 1] + a1 * s[2 * e + 1]);
        }
        lo[i] = make_uint4(ol[0], ol[1], ol[2], ol[3]);
        hi[i] = make_uint4(oh[0], oh[1], oh[2], oh[3]);
      }
      if (MODE == kApQ4) {
        // groups of 64: the low halves of a row's 8 lanes and the high ones
        const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
        const uint32_t hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
        if (__any_sync(0xffffffffu, r < 2 * p.hkv)) {
          __half2 sl, sh;
          const uint32_t cl = q4_codes(lw, sl), ch = q4_codes(hw, sh);
          if (r < 2 * p.hkv && w.phys >= 0) {
            const size_t row = ((size_t)w.phys * p.hkv + (is_v ? r - p.hkv : r)) * p.at.block_tokens + w.at;
            uint8_t* code = (is_v ? p.vslab : p.kslab) + row * (D / 2);
            *reinterpret_cast<uint32_t*>(code + v * 4) = cl;
            *reinterpret_cast<uint32_t*>(code + D / 4 + v * 4) = ch;
            if (v < 2) reinterpret_cast<__half2*>(is_v ? p.vsb : p.ksb)[row * 2 + v] = v ? sh : sl;
          }
        }
      }
      if (MODE == kApMx) {
        // groups of 32: four lanes of the low half of a row, four of the high half
        const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
        const uint32_t hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
        if (__any_sync(0xffffffffu, r < 2 * p.hkv)) {
          uint32_t sl, sh;
          const uint32_t cl = mx4_codes(lw, sl), ch = mx4_codes(hw, sh);
          const uint32_t mine = sl | (sh << 16), other = __shfl_down_sync(0xffffffffu, mine, 4);
          if (r < 2 * p.hkv && w.phys >= 0) {
            const size_t row = ((size_t)w.phys * p.hkv + (is_v ? r - p.hkv : r)) * p.at.block_tokens + w.at;
            uint8_t* code = (is_v ? p.vslab : p.kslab) + row * (D / 2);
            *reinterpret_cast<uint32_t*>(code + v * 4) = cl;
            *reinterpret_cast<uint32_t*>(code + D / 4 + v * 4) = ch;
            if (v == 0) reinterpret_cast<uint32_t*>(is_v ? p.vsb : p.ksb)[row] = mine | (other << 8);
          }
        }
      }
      if (r >= rows || ((MODE == kApQ4 || MODE == kApMx) && !is_q)) continue;
      uint16_t* dst;
      if (is_q) {
        dst = p.q_out + t * p.qos + (size_t)(MODE == kApRows ? r : r - 2 * p.hkv) * D;
      } else {
        if (w.phys < 0) continue;
        const size_t row = ((size_t)w.phys * p.hkv + (is_v ? r - p.hkv : r)) * p.at.block_tokens + w.at;
        dst = reinterpret_cast<uint16_t*>(is_v ? p.vslab : p.kslab) + row * D;
      }
      *reinterpret_cast<uint4*>(dst + v * 8) = lo[i];
      *reinterpret_cast<uint4*>(dst + H + v * 8) = hi[i];
    }
  }
}

struct GatherParams {
  RowPlaces at;
  const uint8_t *kslab, *vslab;
  const __half *ksb, *vsb;
  uint16_t *k, *v;
  int hkv;
};

// D / 16 lanes take a row, 16 elements (32 bytes of output) each.
template <int D, int MODE>
__global__ void __launch_bounds__(kApThreads) gather_kernel(const __grid_constant__ GatherParams p, int tokens_per_cta) {
  constexpr int NV = D / 16, RPW = 32 / NV;
  __shared__ Place where[kApTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t_cta = blockIdx.x * tokens_per_cta;
  if (warp < tokens_per_cta) {
    const Place w = find_place(p.at, t_cta + warp, lane);
    if (lane == 0) where[warp] = w;
  }
  __syncthreads();
  const int wpt = kApWarps / tokens_per_cta, slot = warp / wpt, t = t_cta + slot;
  const Place w = where[slot];
  if (w.phys < 0) return;
  const int v = lane % NV, rows = 2 * p.hkv, rstep = wpt * RPW;
  for (int rb = (warp % wpt) * RPW + lane / NV; rb < rows; rb += kGaBatch * rstep) {
    uint4 x[kGaBatch][2];
    uint2 code[kGaBatch];
    float2 sb[kGaBatch];
#pragma unroll
    for (int i = 0; i < kGaBatch; ++i) {
      const int r = rb + i * rstep;
      if (r >= rows) continue;
      const bool is_v = r >= p.hkv;
      const size_t row = ((size_t)w.phys * p.hkv + (is_v ? r - p.hkv : r)) * p.at.block_tokens + w.at;
      if constexpr (MODE == kApMx) {
        code[i] = __ldg(reinterpret_cast<const uint2*>((is_v ? p.vslab : p.kslab) + row * (D / 2)) + v);
        const uint32_t e = __ldg(reinterpret_cast<const uint8_t*>(is_v ? p.vsb : p.ksb) + row * (D / 32) + v / 2);
        sb[i].x = __uint_as_float(e ? e << 23 : 0x00400000u);   // 2^(e - 127)
      } else if constexpr (MODE == kApQ4) {
        code[i] = __ldg(reinterpret_cast<const uint2*>((is_v ? p.vslab : p.kslab) + row * (D / 2)) + v);
        sb[i] = __half22float2(__ldg(reinterpret_cast<const __half2*>(is_v ? p.vsb : p.ksb) + row * 2 + v / 4));
      } else {
        const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.vslab : p.kslab) + row * (2 * D)) + 2 * v;
        x[i][0] = __ldg(src);
        x[i][1] = __ldg(src + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kGaBatch; ++i) {
      const int r = rb + i * rstep;
      if (r >= rows) continue;
      const bool is_v = r >= p.hkv;
      if constexpr (MODE == kApMx) {
        uint32_t h[8], o[8];
        mx_pairs(code[i].x, h);
        mx_pairs(code[i].y, h + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
          o[e] = pack_bf16(f.x * sb[i].x, f.y * sb[i].x);
        }
        x[i][0] = make_uint4(o[0], o[1], o[2], o[3]);
        x[i][1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else if constexpr (MODE == kApQ4) {   // code * scale is exact in float32, so this is one rounding of the sum
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = (e < 4 ? code[i].x : code[i].y) >> (8 * (e & 3));
          o[e] = pack_bf16(fmaf(static_cast<float>(c & 15u), sb[i].x, sb[i].y),
                           fmaf(static_cast<float>((c >> 4) & 15u), sb[i].x, sb[i].y));
        }
        x[i][0] = make_uint4(o[0], o[1], o[2], o[3]);
        x[i][1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + ((size_t)t * p.hkv + (is_v ? r - p.hkv : r)) * D) + 2 * v;
      dst[0] = x[i][0];
      dst[1] = x[i][1];
    }
  }
}

// Single-token steps spread a token over a CTA's eight warps, so that its
// rows are loaded at once; once the grid fills the device twice over, tokens
// share a CTA's look-ups and angles.
int append_tokens_per_cta(int n_tokens, int num_sms) { return n_tokens <= 2 * num_sms ? 1 : kApTokens; }

// "" or what is wrong with the description
const char* axes_error(const kvs_rope_axes* a, int head_dim) {
  if (!(a->theta > 0.f) || !std::isfinite(a->theta)) return "theta must be positive and finite";
  if (a->n_axes < 1 || a->n_axes > 3) return "1 to 3 position axes";
  if (a->own_spectrum != 0 && a->own_spectrum != 1) return "own_spectrum is 0 or 1";
  long long sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (a->section[i] < 0 || (i >= a->n_axes && a->section[i] != 0)) return "bad axis section";
    sum += a->section[i];
  }
  return sum == head_dim / 2 ? "" : "the axis sections must sum to head_dim / 2";
}

// The frequency table is a function of the description alone: a thread keeps
// the last one (64 powers take longer than the rest of a call).
void axes_turns(const kvs_rope_axes* a, int head_dim, AppendParams& p) {
  struct Last {
    kvs_rope_axes axes;
    int head_dim = 0;
    unsigned long long turn[64];
  };
  static thread_local Last last;
  p.rotate = 1;
  p.s0 = a->section[0];
  p.s1 = a->section[0] + a->section[1];
  if (last.head_dim == head_dim && std::memcmp(&last.axes, a, sizeof *a) == 0) {
    std::memcpy(p.turn, last.turn, sizeof p.turn);
    return;
  }
  const double two_pi = 6.283185307179586476925286766559;
  int axis = 0, j = 0;
  for (int i = 0; i < head_dim / 2; ++i, ++j) {
    while (j >= a->section[axis]) {
      ++axis;
      j = 0;
    }
    const double e = a->own_spectrum ? -(double)j / a->section[axis] : -2.0 * i / head_dim;
    const double f = std::pow((double)a->theta, e) / two_pi;
    p.turn[i] = static_cast<unsigned long long>(std::ldexp(f - std::floor(f), 64));
  }
  last.axes = *a;
  last.head_dim = head_dim;
  std::memcpy(last.turn, p.turn, sizeof p.turn);
}

bool bad_stride(long long stride, long long row) { return stride < row || (stride & 7); }

}  // namespace

kvs_status check_pool_device(const kvs_pool* pool, const char* what) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(KVS_ERR_CUDA, std::string(what) + ": cannot query the current device");
  if (dev != pool->device) return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": the pool belongs to another device than the current one");
  return KVS_OK;
}

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_rope_apply(const void* x_dev, int64_t x_stride, const int32_t* pos_dev,
                                     const kvs_rope_axes* axes, int32_t inverse, void* out_dev, int64_t out_stride,
                                     int32_t n_tokens, int32_t n_heads, int32_t head_dim, cudaStream_t stream) {
  if (head_dim != 64 && head_dim != 128) return fail(KVS_ERR_UNSUPPORTED, "rope_apply: head_dim must be 64 or 128");
  if (n_tokens < 0 || n_heads < 1) return fail(KVS_ERR_INVALID_ARG, "rope_apply: bad sizes");
  if (!axes) return fail(KVS_ERR_INVALID_ARG, "rope_apply: null axes");
  if (const char* e = axes_error(axes, head_dim); *e) return fail(KVS_ERR_INVALID_ARG, std::string("rope_apply: ") + e);
  const long long row = (long long)n_heads * head_dim;
  if (bad_stride(x_stride, row) || bad_stride(out_stride, row))
    return fail(KVS_ERR_INVALID_ARG, "rope_apply: a stride must hold n_heads * head_dim elements and be a multiple of 8");
  if (n_tokens == 0) return KVS_OK;
  if (!x_dev || !pos_dev || !out_dev) return fail(KVS_ERR_INVALID_ARG, "rope_apply: null pointer");
  if (!aligned16(x_dev) || !aligned16(out_dev)) return fail(KVS_ERR_INVALID_ARG, "rope_apply: x and out must be 16-byte aligned");
  if (x_dev == out_dev && x_stride != out_stride) return fail(KVS_ERR_INVALID_ARG, "rope_apply: in place needs equal strides");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(KVS_ERR_CUDA, "rope_apply: cannot query the current device");
  AppendParams p{};
  p.q = static_cast<const uint16_t*>(x_dev);
  p.q_out = static_cast<uint16_t*>(out_dev);
  p.qs = x_stride;
  p.qos = out_stride;
  p.pos = pos_dev;
  p.at.n_tokens = n_tokens;
  p.hq = n_heads;
  p.inverse = inverse != 0;
  axes_turns(axes, head_dim, p);
  const int tpc = append_tokens_per_cta(n_tokens, sms);
  const unsigned grid = (unsigned)((n_tokens + tpc - 1) / tpc);
  if (head_dim == 128)
    append_kernel<128, kApRows><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else
    append_kernel<64, kApRows><<<grid, kApThreads, 0, stream>>>(p, tpc);
  count_launch();
  return check_launch("rope_apply");
}

extern "C" kvs_status kvs_append(kvs_pool* pool, int32_t layer, const void* k_dev, int64_t k_stride, const void* v_dev,
                                 int64_t v_stride, const void* q_dev, int64_t q_stride, int32_t n_q_heads,
                                 void* q_out_dev, const int32_t* tok_off_dev, int32_t n_tokens, const int32_t* pos_dev,
                                 const kvs_rope_axes* axes, const int32_t* block_table_dev, int32_t max_blocks,
                                 const int32_t* seq_len_dev, int32_t n_seq, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "append: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (layer < 0 || layer >= d.num_layers) return fail(KVS_ERR_INVALID_ARG, "append: layer out of range");
  if (n_tokens < 0 || n_seq < 0 || max_blocks < 1 || n_q_heads < 0) return fail(KVS_ERR_INVALID_ARG, "append: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "append: n_seq exceeds the pool's max_seqs");
  if (axes)
    if (const char* e = axes_error(axes, d.head_dim); *e) return fail(KVS_ERR_INVALID_ARG, std::string("append: ") + e);
  const long long krow = (long long)d.num_kv_heads * d.head_dim, qrow = (long long)n_q_heads * d.head_dim;
  if (bad_stride(k_stride, krow) || bad_stride(v_stride, krow) || (q_dev && bad_stride(q_stride, qrow)))
    return fail(KVS_ERR_INVALID_ARG, "append: a stride must hold heads * head_dim elements and be a multiple of 8");
  if (n_tokens == 0 || n_seq == 0) return KVS_OK;
  if (!q_dev != !q_out_dev || (q_dev != nullptr) != (n_q_heads > 0))
    return fail(KVS_ERR_INVALID_ARG, "append: q, q_out and n_q_heads go together");
  if (axes && !pos_dev && axes->n_axes != 1) return fail(KVS_ERR_INVALID_ARG, "append: several axes need positions");
  if (!k_dev || !v_dev || !tok_off_dev || !block_table_dev || !seq_len_dev)
    return fail(KVS_ERR_INVALID_ARG, "append: null pointer");
  if (!aligned16(k_dev) || !aligned16(v_dev) || !aligned16(q_dev) || !aligned16(q_out_dev))
    return fail(KVS_ERR_INVALID_ARG, "append: k, v, q and q_out must be 16-byte aligned");
  if (q_dev && q_dev == q_out_dev && q_stride != qrow)
    return fail(KVS_ERR_INVALID_ARG, "append: queries are rotated in place only where their rows have no gaps");
  if (kvs_status st = check_pool_device(pool, "append"); st != KVS_OK) return st;
  AppendParams p{};
  p.k = static_cast<const uint16_t*>(k_dev);
  p.v = static_cast<const uint16_t*>(v_dev);
  p.q = static_cast<const uint16_t*>(q_dev);
  p.q_out = static_cast<uint16_t*>(q_out_dev);
  p.ks = k_stride;
  p.vs = v_stride;
  p.qs = q_stride;
  p.qos = qrow;
  p.at = RowPlaces{tok_off_dev, seq_len_dev, block_table_dev, pool->status, n_tokens, n_seq, max_blocks,
                   d.capacity_blocks, d.block_tokens};
  p.pos = pos_dev;
  p.kslab = static_cast<uint8_t*>(pool->k[layer]);
  p.vslab = static_cast<uint8_t*>(pool->v[layer]);
  const bool q4 = d.dtype == KVS_DTYPE_Q4G64, mx = d.dtype == KVS_DTYPE_MX4;
  if (q4 || mx) {
    p.ksb = static_cast<__half*>(pool->ksb[layer]);
    p.vsb = static_cast<__half*>(pool->vsb[layer]);
  }
  p.hkv = d.num_kv_heads;
  p.hq = n_q_heads;
  if (axes) axes_turns(axes, d.head_dim, p);
  const int tpc = append_tokens_per_cta(n_tokens, pool->num_sms);
  const unsigned grid = (unsigned)((n_tokens + tpc - 1) / tpc);
  if (mx)
    append_kernel<128, kApMx><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else if (q4)
    append_kernel<128, kApQ4><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else if (d.head_dim == 128)
    append_kernel<128, kApBf16><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else
    append_kernel<64, kApBf16><<<grid, kApThreads, 0, stream>>>(p, tpc);
  count_launch();
  return check_launch("append");
}

extern "C" kvs_status kvs_gather(kvs_pool* pool, int32_t layer, const int32_t* tok_off_dev, int32_t n_tokens,
                                 const int32_t* block_table_dev, int32_t max_blocks, const int32_t* seq_len_dev,
                                 int32_t n_seq, void* k_out_dev, void* v_out_dev, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "gather: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (layer < 0 || layer >= d.num_layers) return fail(KVS_ERR_INVALID_ARG, "gather: layer out of range");
  if (n_tokens < 0 || n_seq < 0 || max_blocks < 1) return fail(KVS_ERR_INVALID_ARG, "gather: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "gather: n_seq exceeds the pool's max_seqs");
  if (n_tokens == 0 || n_seq == 0) return KVS_OK;
  if (!tok_off_dev || !block_table_dev || !seq_len_dev || !k_out_dev || !v_out_dev)
    return fail(KVS_ERR_INVALID_ARG, "gather: null pointer");
  if (!aligned16(k_out_dev) || !aligned16(v_out_dev)) return fail(KVS_ERR_INVALID_ARG, "gather: k_out and v_out must be 16-byte aligned");
  if (kvs_status st = check_pool_device(pool, "gather"); st != KVS_OK) return st;
  GatherParams p{};
  p.at = RowPlaces{tok_off_dev, seq_len_dev, block_table_dev, pool->status, n_tokens, n_seq, max_blocks,
                   d.capacity_blocks, d.block_tokens};
  p.kslab = static_cast<const uint8_t*>(pool->k[layer]);
  p.vslab = static_cast<const uint8_t*>(pool->v[layer]);
  const bool q4 = d.dtype == KVS_DTYPE_Q4G64, mx = d.dtype == KVS_DTYPE_MX4;
  if (q4 || mx) {
    p.ksb = static_cast<const __half*>(pool->ksb[layer]);
    p.vsb = static_cast<const __half*>(pool->vsb[layer]);
  }
  p.k = static_cast<uint16_t*>(k_out_dev);
  p.v = static_cast<uint16_t*>(v_out_dev);
  p.hkv = d.num_kv_heads;
  const int tpc = append_tokens_per_cta(n_tokens, pool->num_sms);
  const unsigned grid = (unsigned)((n_tokens + tpc - 1) / tpc);
  if (mx)
    gather_kernel<128, kApMx><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else if (q4)
    gather_kernel<128, kApQ4><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else if (d.head_dim == 128)
    gather_kernel<128, kApBf16><<<grid, kApThreads, 0, stream>>>(p, tpc);
  else
    gather_kernel<64, kApBf16><<<grid, kApThreads, 0, stream>>>(p, tpc);
  count_launch();
  return check_launch("gather");
}
