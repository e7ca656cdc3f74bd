// Decode attention that also adds up each stored token's attention weight, over
// bf16 pools and pools of microscaled 4-bit values.
//
//   w_h(t) = e^(scale q_h.K_t) / sum_t' e^(scale q_h.K_t'),  out_h = sum_t w_h(t) V_t,
//   mass[t] = carry * mass_in[t] + sum_h w_h(t)
//
// in one pass over keys and values: the weights need the whole sum, so the first
// kernel leaves its scores (4 bytes per token and head, against 512 / G bytes of
// keys and values) and the second turns them into weights with the final
// maximum and sum.
//
// Work: the units of all sequences, KV head by KV head, form one line that the CTAs
// of one wave share evenly, whatever the lengths; a CTA's stretch may cover the
// ends of several (sequence, KV head) pairs, and a pair several CTAs, whose parts
// the last one to arrive joins in their order.  A warp takes every W-th unit of
// its CTA's stretch and brings it with its own ring of TMA copies, which run on
// across the pairs' borders.  Up to 64 sequences are placed by every warp for
// itself; there, where all pairs fit, each begins a CTA.
//
// Tokens are the 16 rows of the products, query heads the 8 (or twice 8)
// columns: S^T = K q^T, O^T += V^T P^T.  P^T is the transposed accumulator of S^T
// (movmatrix) in three bf16 parts, which hold a weight's 24 bits (in two, 2e-6 of
// the result were lost, in three 3e-7, at 1 us of 26), or in two fp16 parts.  The
// reference of the exponentials moves only when a score exceeds it by more than
// 2^4, so that a unit needs no exchange between lanes.
//
// bf16: a unit is a block of 16 tokens; operands by ldmatrix.
// Microscaled: a unit is 32 tokens.  A byte holds two e2m1 values, which one
// conversion turns into an fp16 pair.  Keys: the products of a group of 32
// channels are scaled by the group's power of two in fp32, exactly.  Values: a
// token's scale multiplies the fp16 pairs, relative to the largest one that this
// warp has met in the group (E): 2^(e - E + 13), exact for e >= E - 27 and zero
// below.  E goes by the scales alone: next to weights of one size a value lost is
// 2^-27 of a sum that fp32 holds to 2^-24, but a token of a huge scale hides the others
// even where its own weight is small.  Weights are two fp16 parts at 2^11 and more of the
// largest one met, so 2^-36 of that is the least that they hold.  The
// accumulators follow E when it grows.  Row r of a product is token
// r ^ (r >> 1 & 1) of its 16, with which all shared loads (64-byte swizzle) are
// free of bank conflicts.
//
// Measured, graph replays with the masses (without for *): eight sequences of
// 9,830 to 16,384 tokens, 32 heads of their own: 262 us, 6.4 TB/s, bound by HBM; 32
// that share 4,096 of 5,400, 16 / 2 heads: 27 us, every sequence reads the common
// part from L2 (6.5 TB/s), bound by a unit's chain of products and exponentials;
// four of 350, 8 / 2 of 64 channels: 8.7 us, start, four units, arrival, join and the
// second kernel, each a trip to memory.  In 4 bits: twelve of 4,000 to 8,191, 32 / 8
// (*): 29 us; eight of 16,384 to 32,768: 72 us, 3.1 TB/s.  There three warps a scheduler
// (168 registers) wait for one another's results: of 5.3 cycles a warp takes for an
// instruction, 1.8 are the latency of the one before, 0.4 a busy pipe, 0.7 memory and
// shared memory; 52 % of the issue slots are used.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kvs {

namespace {

enum { kFmtBf16x64, kFmtBf16x128, kFmtMx };

constexpr int kDmMaxGroup = 16, kDmMaxStages = 4, kDmMaxCtas = 3, kDmJoin = 8;

template <int FMT, int NT>
struct Dm {   // what a format and the number of 8-column tiles fix
  static constexpr bool mx = FMT == kFmtMx;
  static constexpr int D = FMT == kFmtBf16x64 ? 64 : 128;
  static constexpr int UT = mx ? 32 : 16;                 // tokens of a unit
  static constexpr int kBlockTokens = mx ? 64 : 16;
  static constexpr int W = !mx && NT == 2 ? 8 : 4;        // warps of a CTA
  static constexpr int kCtas = mx ? (NT == 1 ? 3 : 2) : NT == 1 ? 2 : 1;   // per SM (kDmMaxCtas at most)
  static constexpr int kCodes = mx ? UT * D / 2 : UT * D * 2;   // bytes of a unit's K or V
  static constexpr int kScales = mx ? UT * 4 : 0;
  static constexpr int kStage = 2 * kCodes + (mx ? 512 : 0);    // scales in the last 512 bytes
  static constexpr int ST = FMT == kFmtBf16x64 && NT == 1 ? 4 : 2;   // three or four of 128 channels were slower (below)
  static constexpr int kHead = W == 4 ? 1024 : 2048;      // barriers and the warps' sums, in front of the ring
  // Measured for bf16, one n-tile, 128 channels (8 x 13,000 tokens of 32 / 32 heads,
  // 16 x 8,000 of 32 / 8, us): four warps, two CTAs an SM, two stages 266, 94; three
  // stages 281, 99; five or six warps 272, 96; three CTAs 274, 98; two warps and
  // four CTAs 337, 125.  Microscaled (8 x 24,000 of 32 / 8, 64 x 4,000 of 32 / 8):
  // four warps, three CTAs 69.8, 78.9; two CTAs of eight warps, with 128 registers a
  // thread, 77.3, 83.9; two of four 74.2, 83.7; four of three 74.4, 78.8.
  static constexpr int kPrep = mx ? UT * 16 + 4 * UT * 2 : 0;   // a warp's prepared scales
  static constexpr int kSmem = kHead + W * (ST * kStage + NT * 8 * D * 4 + kPrep);
  static constexpr float kBias = mx ? 11.f : 0.f;         // weights reach 2^(kBias + kLag)
};
constexpr float kLag = 4.f;

template <int W>
struct DmShared {
  uint64_t full[W][kDmMaxStages];
  float2 ml[W][kDmMaxGroup];
  int warp_sums[32];
  int a, b, cuts;
  long long per, first;         // places of a CTA on the line, that of the first unit of the pair at work
  int gap;                      // places between two pairs
  struct Cut {                  // a pair that other CTAs share: this CTA's first and last
    int seq, head, parts, last;
    size_t slot;                // of its first part
  } cut[2];
};

struct DmParams {
  const uint16_t* q;            // bf16 [n_seq][hq][D]
  const int32_t *table, *seq_len;
  const uint8_t *ksc, *vsc;     // scale bytes of this layer
  float* out;
  float* part;                  // [CTAs + pairs][g][D]
  float* part_ml;               // [CTAs + pairs][g][2]
  float2* fin;                  // [pairs][g] {reference, 1 / sum}
  float* scores;                // [pair][max tokens][g], or nullptr
  int32_t* tickets;
  uint32_t* status;
  int n_seq, max_blocks, hkv, g, hq, capacity, most;   // most: tokens of a table row
  float scale_log2;
};

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(x, y);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack_f16(x - f.x, y - f.y);
}
__device__ __forceinline__ int mx_token(int r) { return r ^ ((r >> 1) & 1); }   // of row r of 16

struct DmSpan {   // a sequence's length and units
  int len, units;
};
template <int UT>
__device__ __forceinline__ DmSpan dm_span(const DmParams& p, int a) {
  const int len = min(max(__ldg(p.seq_len + a), 0), p.most);
  return DmSpan{len, (len + UT - 1) / UT};
}

// a / b; 64-bit division takes some hundred instructions
__device__ __forceinline__ int quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? (int)(a / b) : (int)((unsigned)a / (unsigned)b);
}

// A place on the line of units.
struct DmAt {
  int h, a, b, units;   // KV head, sequence, unit in it, its units
};
template <int UT>
__device__ __forceinline__ void dm_advance(const DmParams& p, DmAt& at, int by) {
  at.b += by;
  while (at.h < p.hkv && at.b >= at.units) {
    at.b -= at.units;
    if (++at.a == p.n_seq) {
      at.a = 0;
      ++at.h;
    }
    at.units = dm_span<UT>(p, at.a).units;
  }
}

template <int FMT, int NT>
__global__ void __launch_bounds__(Dm<FMT, NT>::W * 32, Dm<FMT, NT>::kCtas)
decode_mass_kernel(const __grid_constant__ DmParams p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using F = Dm<FMT, NT>;
  constexpr int D = F::D, W = F::W, UT = F::UT, ST = F::ST, MT = UT / 16, T = W * 32;
  static_assert(sizeof(DmShared<W>) <= F::kHead && ST <= kDmMaxStages, "the ring begins behind the head");
  extern __shared__ __align__(1024) uint8_t smem_raw[];   // no static shared memory: it begins on 1,024 bytes
  DmShared<W>& sh = *reinterpret_cast<DmShared<W>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem_raw + F::kHead + warp * ST * F::kStage;
  float* s_acc = reinterpret_cast<float*>(smem_raw + F::kHead + W * ST * F::kStage);   // [W][g][D]
  uint8_t* prep = smem_raw + F::kSmem - W * F::kPrep + warp * F::kPrep;   // microscaled: a unit's scales, prepared
  if (tid == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    sh.cuts = 0;
  }
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&sh.full[warp][s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto empty_sequences = [&]() {
    for (int a = blockIdx.x; a < p.n_seq; a += gridDim.x) {
      const int raw = p.seq_len[a];
      if (tid == 0 && (raw < 0 || raw > p.most)) set_err(p.status, KVS_DEVERR_SEQ_LEN);
      if (raw <= 0)
        for (int i = tid; i < p.hq * D; i += T) p.out[(size_t)a * p.hq * D + i] = 0.f;
    }
  };

  // ---- this CTA's stretch of the line
  long long per, first;
  int n_mine, gap = 0;   // units of this CTA
  DmAt seg;
  // units of a CTA: an even share, but no more parts of a pair than are worth their
  // joining (a sequence of 32,000 tokens, eight heads on one KV head: 45 us evenly,
  // 23 with fewer CTAs; in 4 bits 39 and 26)
  auto share = [&](int total) {
    const int least = (int)sqrtf((F::mx ? 0.03f : 0.06f) * (float)p.g * (float)total / (float)p.n_seq);
    return (long long)max(max(W, least), quotient((long long)total * p.hkv + gridDim.x - 1, gridDim.x));
  };
  if (p.n_seq <= 64) {
    // every warp for itself, a lane two sequences (64 of 500 tokens, 16 / 2 heads: 13.8 us,
    // 16.1 by the whole CTA)
    const int a0 = 2 * lane;
    const int real0 = a0 < p.n_seq ? dm_span<UT>(p, a0).units : 0, real1 = a0 + 1 < p.n_seq ? dm_span<UT>(p, a0 + 1).units : 0;
    per = share(__reduce_add_sync(0xffffffffu, real0 + real1));
    // Where they fit, every pair begins a CTA (its units are rounded up to whole
    // CTAs): a second pair costs a CTA more than a unit or two of every warp (four
    // sequences of 300 tokens, 8 / 2 heads of 64 channels, with the masses: 8.4 us,
    // 10.1 evenly).
    const int whole = (int)((per + W - 1) / W) * W;
    int n0 = real0, n1 = real1;
    bool rounded = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int m = whole + k * W, up0 = (real0 + m - 1) / m, up1 = (real1 + m - 1) / m;
      if ((long long)__reduce_add_sync(0xffffffffu, up0 + up1) * p.hkv <= gridDim.x) {
        n0 = up0 * m;
        n1 = up1 * m;
        per = m;
        rounded = true;
        break;
      }
    }
    // Elsewhere a gap in front of every pair stands for what beginning it costs (32
    // sequences that share 4,096 of 5,400 tokens, 16 / 2 heads: 26.2 us, 28.1 without).
    if (!rounded) {
      gap = 4 * W;
      n0 = real0 ? real0 + gap : 0;
      n1 = real1 ? real1 + gap : 0;
    }
    int end = n0 + n1, units = real0 + real1;   // places and units up to this lane's sequences, both among them
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o), y = __shfl_up_sync(0xffffffffu, units, o);
      end += lane >= o ? x : 0;
      units += lane >= o ? y : 0;
    }
    const int per_head = __shfl_sync(0xffffffffu, end, 31), units_head = __shfl_sync(0xffffffffu, units, 31);
    const long long places = (long long)per_head * p.hkv;
    if (!rounded) per = max(per, (long long)quotient(places + gridDim.x - 1, gridDim.x));
    // the pair of a place, and the units before the place
    auto locate = [&](long long u, DmAt& at, int& place) {
      at.h = quotient(u, per_head);
      const int r = (int)(u - (long long)at.h * per_head);
      const int l = __popc(__ballot_sync(0xffffffffu, end <= r)) & 31;
      const int from = __shfl_sync(0xffffffffu, end - n0 - n1, l), size = __shfl_sync(0xffffffffu, n0, l);
      const int u_0 = __shfl_sync(0xffffffffu, real0, l), u_1 = __shfl_sync(0xffffffffu, real1, l);
      const bool second = r >= from + size;
      at.a = 2 * l + second;
      place = r - from - (second ? size : 0) - gap;
      at.units = second ? u_1 : u_0;
      at.b = min(max(place, 0), at.units);
      return (long long)at.h * units_head + __shfl_sync(0xffffffffu, units - real0 - real1, l) + (second ? u_0 : 0) + at.b;
    };
    const long long u0 = per * blockIdx.x, u1 = min(places, u0 + per);
    if (u0 < u1) {
      int place, unused;
      DmAt behind;
      const long long before = locate(u0, seg, place);
      n_mine = (int)((u1 < places ? locate(u1, behind, unused) : (long long)units_head * p.hkv) - before);
      first = u0 - place;
    }
    if (u0 >= u1 || n_mine == 0) {
      empty_sequences();
      return;
    }
  } else {
    int per_head = 0, mine = 0, mine_before = 0;   // of the sequences tid, tid + T, ...: the first one's units, and those before it
    for (int a0 = 0; a0 < p.n_seq; a0 += T) {
      const int a = a0 + tid;
      const int n = a < p.n_seq ? dm_span<UT>(p, a).units : 0;
      int total;
      const int before = block_exclusive_scan(n, sh.warp_sums, total);
      if (a0 == 0) {
        mine = n;
        mine_before = before;
      }
      per_head += total;
    }
    per = share(per_head);
    const long long u0 = per * blockIdx.x, u1 = min((long long)per_head * p.hkv, u0 + per);
    if (u0 >= u1) {
      empty_sequences();
      return;
    }
    seg.h = quotient(u0, per_head);
    const int r0 = (int)(u0 - (long long)seg.h * per_head);
    if (mine_before <= r0 && r0 < mine_before + mine) {
      sh.a = tid;
      sh.b = r0 - mine_before;
    }
    int carry = 0;
    for (int a0 = 0; p.n_seq > T && a0 < p.n_seq; a0 += T) {   // more sequences than threads: once more
      const int a = a0 + tid, n = a < p.n_seq ? dm_span<UT>(p, a).units : 0;
      int total;
      const int before = carry + block_exclusive_scan(n, sh.warp_sums, total);
      if (before <= r0 && r0 < before + n) {
        sh.a = a;
        sh.b = r0 - before;
      }
      carry += total;
    }
    __syncthreads();
    seg.a = sh.a;
    seg.b = sh.b;
    seg.units = dm_span<UT>(p, sh.a).units;
    n_mine = (int)(u1 - u0);
    first = u0 - seg.b;
  }

  if (tid == 0) {
    sh.per = per;
    sh.first = first;
    sh.gap = gap;
  }

  // ---- copies of this warp's units k = warp, warp + W, ...
  DmAt ahead = seg;
  dm_advance<UT>(p, ahead, warp);
  int k_ahead = warp, stage_ahead = 0;
  uint32_t there = 0;      // bit s: the block of the unit in stage s lies in the pool
  auto look_up = [&]() {   // physical block of the unit ahead
    if (k_ahead >= n_mine) return -1;
    return __ldg(p.table + (size_t)ahead.a * p.max_blocks + ahead.b * UT / F::kBlockTokens);
  };
  int id_ahead = look_up();
  auto issue = [&]() {     // whole warp; lane 0 copies
    if (k_ahead >= n_mine) return;
    const int s = stage_ahead;
    if (++stage_ahead == ST) stage_ahead = 0;
    const bool ok = id_ahead >= 0 && id_ahead < p.capacity;
    there = (there & ~(1u << s)) | ((ok ? 1u : 0u) << s);
    if (lane == 0) {
      uint64_t* bar = &sh.full[warp][s];
      if (!ok) {
        set_err(p.status, KVS_DEVERR_BLOCK_ID);
        mbar_arrive(bar);
      } else {
        mbar_arrive_expect_tx(bar, 2 * (F::kCodes + F::kScales));
        uint8_t* st = ring + s * F::kStage;
        const int row = (id_ahead * p.hkv + ahead.h) * F::kBlockTokens + ahead.b * UT % F::kBlockTokens;
        if constexpr (F::mx) {
          tma_load_2d(st, &tk, 0, row, bar);
          tma_load_2d(st + F::kCodes, &tv, 0, row, bar);
          bulk_load(st + 2 * F::kCodes, p.ksc + (size_t)row * 4, F::kScales, bar);
          bulk_load(st + 2 * F::kCodes + F::kScales, p.vsc + (size_t)row * 4, F::kScales, bar);
        } else {
          tma_load_kv_tile<D>(st, &tk, row, bar);
          tma_load_kv_tile<D>(st + F::kCodes, &tv, row, bar);
        }
      }
    }
    k_ahead += W;
    ahead.b += W;
    if (ahead.b >= ahead.units && k_ahead < n_mine) dm_advance<UT>(p, ahead, 0);
    id_ahead = look_up();
  };
  for (int i = 0; i < ST; ++i) issue();
  empty_sequences();

  int k = warp;                    // this warp's next unit, relative to u0
  int stage = 0, uses = 0;
  uint32_t phase = 0;
  bool dead = false;
  int got0 = 0, got1 = 0;   // thread 0: arrivals
  for (int done = 0; done < n_mine;) {
    // ---- one (sequence, KV head): units [seg.b, seg.units) as far as the stretch goes
    const int n_seg = min(seg.units - seg.b, n_mine - done);
    const int len = dm_span<UT>(p, seg.a).len;
    const uint16_t* qp = p.q + ((size_t)seg.a * p.hq + seg.h * p.g) * D;
    // queries as the B operand: column g of n-tile nt, in the order of the
    // channels in which K's fragments come
    uint32_t qb[NT][D / 16][2];
    float cs[NT][2];   // scale of the scores of columns 2c and 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g;
      const bool ok = row < p.g;
      cs[nt][0] = cs[nt][1] = p.scale_log2;
      if constexpr (F::mx) {
        uint4 w[4];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = ok ? __ldg(reinterpret_cast<const uint4*>(qp + (size_t)row * D + 32 * j + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[e])), fabsf(bf16_hi(x[e]))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // a power of two brings the row's largest value to [2^10, 2^11): products
        // with codes up to 6 stay far inside fp32, and values down to 2^-24 of
        // the largest keep all their bits
        const int be = (int)((__float_as_uint(top) >> 23) & 255u);
        int e = be > 0 && be < 255 ? be - 127 - 10 : 0;
        e = min(max(e, -100), 113);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) qb[nt][2 * j + i / 2][i & 1] = pack_f16(bf16_lo(x[i]) * down, bf16_hi(x[i]) * down);
        }
        cs[nt][0] *= __shfl_sync(0xffffffffu, up, 8 * c);
        cs[nt][1] *= __shfl_sync(0xffffffffu, up, 8 * c + 4);
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[nt][j][i] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qp + (size_t)row * D + 16 * j + 8 * i + 2 * c)) : 0u;
      }
    }
    // ref: reference of the exponentials; thr: scores above it move ref (both in
    // the units in which the products come, cs times which is log2)
    float ref[NT][2], thr[NT][2], l[NT][2], acc[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = thr[nt][0] = thr[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.f;
    }
    uint32_t top_e = 0, top01 = 0, top23 = 0;   // microscaled: the largest scale byte met of each group of channels; two to a word
    const int row0 = F::mx ? mx_token(g) : g;   // token of this lane's first row
    const bool even = (p.g & 1) == 0;
    float* sc_out = p.scores ? p.scores + (((size_t)seg.a * p.hkv + seg.h) * p.most + row0) * p.g + 2 * c : nullptr;

    for (; k < done + n_seg; k += W) {
      const int t_unit = (seg.b + k - done) * UT, nv = len - t_unit;   // nv: tokens of the sequence from here on
      if (!dead && !__all_sync(0xffffffffu, mbar_wait_bounded(&sh.full[warp][stage], phase, p.status))) dead = true;
      const uint8_t* kc = ring + stage * F::kStage;
      const uint8_t* vc = kc + F::kCodes;
      if (((there >> stage) & 1u) && !dead) {
        float s[MT][NT][4];
        // ---- S^T
        if constexpr (F::mx) {
          // every lane turns the scales of one token into what the products take:
          // keys' powers of two (the byte becomes the exponent), row by row; values'
          // relative to the largest so far, 2^(e - E + 13) as fp16, group by group
          constexpr uint32_t kLeast = 0x00400000u;   // 2^-127, of byte 0
          const uint32_t ke = *reinterpret_cast<const uint32_t*>(kc + 2 * F::kCodes + lane * 4);
          const uint32_t ve = *reinterpret_cast<const uint32_t*>(kc + 2 * F::kCodes + F::kScales + lane * 4);
          const int at = (lane & 16) | mx_token(lane & 15);   // the row of token `lane` (the map is its own inverse)
          *reinterpret_cast<float4*>(prep + at * 16) =
              make_float4(__uint_as_float(max((ke << 23) & 0x7f800000u, kLeast)), __uint_as_float(max((ke << 15) & 0x7f800000u, kLeast)),
                          __uint_as_float(max((ke << 7) & 0x7f800000u, kLeast)), __uint_as_float(max((ke >> 1) & 0x7f800000u, kLeast)));
          const uint32_t mine = lane < nv ? ve : 0u;
          const uint32_t v01 = __byte_perm(mine, 0u, 0x4140), v23 = __byte_perm(mine, 0u, 0x4342);
          const uint32_t m01 = __vmaxu2(v01, top01), m23 = __vmaxu2(v23, top23);
          if (__any_sync(0xffffffffu, m01 != top01 || m23 != top23)) {
            uint32_t n01 = m01, n23 = m23;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
              n01 = __vmaxu2(n01, __shfl_xor_sync(0xffffffffu, n01, o));
              n23 = __vmaxu2(n23, __shfl_xor_sync(0xffffffffu, n23, o));
            }
            const uint32_t next = __byte_perm(n01, n23, 0x6420);
            const int up = (int)((next >> (8 * (g >> 1))) & 255u) - (int)((top_e >> (8 * (g >> 1))) & 255u);
            const float f = up > 126 ? 0.f : __uint_as_float((uint32_t)(127 - up) << 23);
            top_e = next;
            top01 = n01;
            top23 = n23;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][j][e] *= f;
          }
          // 28 less the distance to the largest, none beyond 28: exponent bits of fp16
          const uint32_t x01 = (0x001c001cu - __vminu2(top01 - v01, 0x001c001cu)) << 10;
          const uint32_t x23 = (0x001c001cu - __vminu2(top23 - v23, 0x001c001cu)) << 10;
          uint16_t* vf = reinterpret_cast<uint16_t*>(prep + 512) + at;
          vf[0] = (uint16_t)x01;
          vf[32] = (uint16_t)(x01 >> 16);
          vf[64] = (uint16_t)x23;
          vf[96] = (uint16_t)(x23 >> 16);
          __syncwarp();
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int t0 = mt * 16 + row0;
            const float4 e0 = *reinterpret_cast<const float4*>(prep + (mt * 16 + g) * 16);
            const float4 e1 = *reinterpret_cast<const float4*>(prep + (mt * 16 + g + 8) * 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t x0[4], x1[4];
              const uint8_t* kr = kc + swz64(t0 * 64 + 16 * j + 4 * c);   // rows 8 apart have the same swizzle
              mx_pairs(*reinterpret_cast<const uint32_t*>(kr), x0);
              mx_pairs(*reinterpret_cast<const uint32_t*>(kr + 512), x1);
              const float f0 = j == 0 ? e0.x : j == 1 ? e0.y : j == 2 ? e0.z : e0.w;
              const float f1 = j == 0 ? e1.x : j == 1 ? e1.y : j == 2 ? e1.z : e1.w;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(y, x0[0], x1[0], x0[1], x1[1], qb[nt][2 * j][0], qb[nt][2 * j][1]);
                mma_f16(y, x0[2], x1[2], x0[3], x1[3], qb[nt][2 * j + 1][0], qb[nt][2 * j + 1][1]);
                s[mt][nt][0] = fmaf(y[0], f0, s[mt][nt][0]);
                s[mt][nt][1] = fmaf(y[1], f0, s[mt][nt][1]);
                s[mt][nt][2] = fmaf(y[2], f1, s[mt][nt][2]);
                s[mt][nt][3] = fmaf(y[3], f1, s[mt][nt][3]);
              }
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[0][nt][0] = s[0][nt][1] = s[0][nt][2] = s[0][nt][3] = 0.f;
          // two chains of products, so that a warp waits half as long for its scores
          float s2[NT][4] = {};
          const uint32_t ka = smem_u32(kc);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t x[4];
            ldsm_x4(ka + kv_tile_off<D>(lane & 15, j * 16 + (lane >> 4) * 8), x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(j & 1 ? s2[nt] : s[0][nt], x, qb[nt][j][0], qb[nt][j][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[0][nt][e] += s2[nt][e];
        }
        if (nv < UT) {   // the sequence ends here
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (mt * 16 + row0 + 8 * (e >> 1) >= nv) s[mt][nt][e] = -INFINITY;
        }
        if (sc_out) {
          // rows 8 apart are 8 g apart; lanes whose columns are no heads store nothing
          float* o = sc_out + (size_t)t_unit * p.g;
          const int left = nv - row0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int cols = p.g - nt * 8 - 2 * c;   // heads from this lane's first column on
            if (cols <= 0) continue;
            float* q = o + nt * 8;
#pragma unroll
            for (int hr = 0; hr < 2 * MT; ++hr, q += 8 * p.g) {
              if (8 * hr >= left) break;
              const float y0 = s[hr / 2][nt][2 * (hr & 1)] * cs[nt][0], y1 = s[hr / 2][nt][2 * (hr & 1) + 1] * cs[nt][1];
              if (even) {
                *reinterpret_cast<float2*>(q) = make_float2(y0, y1);
              } else {
                q[0] = y0;
                if (cols > 1) q[1] = y1;
              }
            }
          }
        }
        bool above = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            top[nt][i] = fmaxf(s[0][nt][i], s[0][nt][2 + i]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) top[nt][i] = fmaxf(top[nt][i], fmaxf(s[mt][nt][i], s[mt][nt][2 + i]));
            above |= top[nt][i] > thr[nt][i];
          }
        if (__any_sync(0xffffffffu, above)) {
          // some column's reference moves to its maximum so far
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = top[nt][i];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const bool move = mx > thr[nt][i];
              const float next = move ? mx * cs[nt][i] : ref[nt][i];
              f[i] = move ? fast_exp2(ref[nt][i] - next) : 1.f;
              ref[nt][i] = next;
              if (move) thr[nt][i] = mx + kLag / cs[nt][i];
              l[nt][i] *= f[i];
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              acc[nt][j][0] *= f[0]; acc[nt][j][1] *= f[1];
              acc[nt][j][2] *= f[0]; acc[nt][j][3] *= f[1];
            }
          }
        }
        // ---- weights, transposed into the B operand
        uint32_t ph[MT][NT][2], pl[MT][NT][2], pm[MT][NT][2];   // pm: bf16, between the two
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = fast_exp2(fmaf(s[mt][nt][e], cs[nt][e & 1], F::kBias - ref[nt][e & 1]));
            l[nt][0] += w[0] + w[2];
            l[nt][1] += w[1] + w[3];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t hi, lo;
              if constexpr (F::mx) {
                split_f16(w[2 * i], w[2 * i + 1], hi, lo);
              } else {
                hi = pack_bf16(w[2 * i], w[2 * i + 1]);
                uint32_t mid;
                split_bf16(w[2 * i] - bf16_lo(hi), w[2 * i + 1] - bf16_hi(hi), mid, lo);
                pm[mt][nt][i] = movm_t(mid);
              }
              ph[mt][nt][i] = movm_t(hi);
              pl[mt][nt][i] = movm_t(lo);
            }
          }
        // ---- O^T += V^T P^T.  Each unit's products are added in plain fp32: the
        // tensor cores cut their sums, which over a long context is a bias (16,384
        // tokens: 5.5e-6 of the result, added here 2.2e-6, with weights of two parts; in
        // 4 bits 1.3e-6 and 2.6e-7).
        auto values = [&](int nt, int j, const uint32_t* x, int mt) {
          float y[4] = {0.f, 0.f, 0.f, 0.f};
          if constexpr (F::mx) {
            mma_f16(y, x[0], x[1], x[2], x[3], ph[mt][nt][0], ph[mt][nt][1]);
            mma_f16(y, x[0], x[1], x[2], x[3], pl[mt][nt][0], pl[mt][nt][1]);
          } else {
            mma_bf16(y, x, pl[mt][nt][0], pl[mt][nt][1]);
            mma_bf16(y, x, pm[mt][nt][0], pm[mt][nt][1]);
            mma_bf16(y, x, ph[mt][nt][0], ph[mt][nt][1]);
          }
          float* a = acc[nt][j];
          const float2 u = __fadd2_rn(make_float2(a[0], a[1]), make_float2(y[0], y[1]));
          const float2 v = __fadd2_rn(make_float2(a[2], a[3]), make_float2(y[2], y[3]));
          a[0] = u.x; a[1] = u.y; a[2] = v.x; a[3] = v.y;
        };
        if constexpr (F::mx) {
          const uint8_t* vf = prep + 512 + (g >> 1) * 64 + 4 * c;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // tokens of the four rows 2c, 2c + 1, 2c + 8, 2c + 9; channels 16 g .. 16 g + 15
            uint2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = mt * 16 + mx_token(2 * c + (i & 1));
              v[i] = *reinterpret_cast<const uint2*>(vc + swz64(t * 64 + 16 * (g >> 1)) + 8 * (g & 1) + 512 * (i >> 1));
            }
            const uint32_t s01 = *reinterpret_cast<const uint32_t*>(vf + mt * 32), s89 = *reinterpret_cast<const uint32_t*>(vf + mt * 32 + 16);
#pragma unroll
            for (int word = 0; word < 2; ++word) {
              const uint32_t w0 = word ? v[0].y : v[0].x, w1 = word ? v[1].y : v[1].x;
              const uint32_t w8 = word ? v[2].y : v[2].x, w9 = word ? v[3].y : v[3].x;
              constexpr uint32_t kLow = 0x0f0f0f0fu;
              uint32_t a0[4], a1[4], a2[4], a3[4];   // even channels, odd ones; tokens 2c, 2c + 1 and 2c + 8, 2c + 9
              mx_pairs((w0 & kLow) | ((w1 << 4) & ~kLow), a0);
              mx_pairs(((w0 >> 4) & kLow) | (w1 & ~kLow), a1);
              mx_pairs((w8 & kLow) | ((w9 << 4) & ~kLow), a2);
              mx_pairs(((w8 >> 4) & kLow) | (w9 & ~kLow), a3);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t x[4] = {mul_f16x2(a0[j], s01), mul_f16x2(a1[j], s01), mul_f16x2(a2[j], s89), mul_f16x2(a3[j], s89)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) values(nt, word * 4 + j, x, mt);
              }
            }
          }
        } else {
          if (nv < UT) {
            // rows behind the end hold anything, and 0 * NaN is not 0
            for (int i = lane; i < (UT - nv) * (D / 8); i += 32)
              *reinterpret_cast<uint4*>(const_cast<uint8_t*>(vc) + kv_tile_off<D>(nv + i / (D / 8), (i % (D / 8)) * 8)) = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
          }
          const uint32_t va = smem_u32(vc);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t x[4];
            ldsm_x4_t(va + kv_tile_off<D>((lane & 7) + (lane >> 4) * 8, j * 16 + ((lane >> 3) & 1) * 8), x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) values(nt, j, x, 0);
          }
          if (nv < UT) fence_proxy_async_smem();   // the zeros are written before a copy overwrites them
        }
      } else if (p.scores) {
        float* o = p.scores + (((size_t)seg.a * p.hkv + seg.h) * p.most + t_unit) * p.g;
        for (int i = lane; i < min(nv, UT) * p.g; i += 32) o[i] = -INFINITY;
      }
      __syncwarp();
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
      if (!dead) {
        ++uses;
        issue();
      }
    }

    // ---- the warps' states become one
    // microscaled: times 2^(E - 127 - 13 - kBias), as two factors that float32 holds; kBias
    // goes out of the sums here, so that those of large values stay finite as over bf16 pools.
    // What the weights were taken against is ref - kBias as float32 rounds it; adding kBias to
    // that is exact
    constexpr float kUnbias = F::mx ? 0x1p-11f : 1.f;
    static_assert(F::kBias == (F::mx ? 11.f : 0.f), "kUnbias is 2^-kBias");
    const int e_up = (int)((top_e >> (8 * (g >> 1))) & 255u) - 151;
    const float up1 = __uint_as_float((uint32_t)(127 + e_up / 2) << 23), up2 = __uint_as_float((uint32_t)(127 + e_up - e_up / 2) << 23);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], o);
        const int row = nt * 8 + 2 * c + i;
        if (row >= p.g) continue;
        if (g == 0) sh.ml[warp][row] = make_float2(__fadd_rn(__fsub_rn(ref[nt][i], F::kBias), F::kBias), l[nt][i] * kUnbias);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          float* o = s_acc + ((size_t)warp * p.g + row) * D;
          if constexpr (F::mx) {
            *reinterpret_cast<float2*>(o + 16 * g + 2 * j) = make_float2(acc[nt][j][i] * up1 * up2, acc[nt][j][2 + i] * up1 * up2);
          } else {
            o[16 * j + g] = acc[nt][j][i];
            o[16 * j + g + 8] = acc[nt][j][2 + i];
          }
        }
      }
    __syncthreads();
    const int cta0 = quotient(sh.first, sh.per), n_parts = quotient(sh.first + seg.units - 1, sh.per) - cta0 + 1;
    const int order = seg.h * p.n_seq + seg.a, pair = seg.a * p.hkv + seg.h;
    const size_t slot = (size_t)blockIdx.x + order;
    for (int i = tid; i < p.g * (D / 4); i += T) {
      const int row = i / (D / 4), col = (i - row * (D / 4)) * 4;
      float M = -INFINITY, L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (sh.ml[w][row].y > 0.f) M = fmaxf(M, sh.ml[w][row].x);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 ml = sh.ml[w][row];
        const float f = ml.y > 0.f ? fast_exp2(ml.x - M) : 0.f;
        const float4 x = *reinterpret_cast<const float4*>(s_acc + ((size_t)w * p.g + row) * D + col);
        L += f * ml.y;
        o.x += f * x.x; o.y += f * x.y; o.z += f * x.z; o.w += f * x.w;
      }
      if (n_parts == 1) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<float4*>(p.out + ((size_t)seg.a * p.hq + seg.h * p.g + row) * D + col) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (col == 0 && p.scores) p.fin[(size_t)pair * p.g + row] = make_float2(L > 0.f ? M : 0.f, inv);
      } else {
        __stcg(reinterpret_cast<float4*>(p.part + (slot * p.g + row) * D + col), o);
        if (col == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + (slot * p.g + row) * 2), make_float2(M, L));
      }
    }
    if (n_parts > 1) __threadfence();
    __syncthreads();   // the states are read: the next pair's may be written
    if (tid == 0) {
      sh.first += seg.units + sh.gap;
      if (n_parts > 1) {
        // the parts are there; whether they were the last ones is looked at when
        // this CTA has nothing else to do
        sh.cut[sh.cuts] = {seg.a, seg.h, n_parts, 0, (size_t)cta0 + order};
        if (sh.cuts++ == 0) got0 = atomicAdd(p.tickets + pair, 1);
        else got1 = atomicAdd(p.tickets + pair, 1);
      }
    }
    done += n_seg;
    if (done < n_mine) dm_advance<UT>(p, seg, n_seg);
  }
  // Only a stretch's first and last pair can have parts of other CTAs; the last CTA
  // of a pair joins its parts in their order.
  if (tid == 0)
    for (int k = 0; k < sh.cuts; ++k) {
      const bool last = (k ? got1 : got0) == sh.cut[k].parts - 1;
      if (last) p.tickets[(size_t)sh.cut[k].seq * p.hkv + sh.cut[k].head] = 0;
      sh.cut[k].last = last;
    }
  __syncthreads();
  const int cuts = sh.cuts;
  if (cuts > 0) {
    for (int k = 0; k < cuts; ++k) {
      const auto cut = sh.cut[k];
      if (!cut.last) continue;
      __threadfence();
      // four channels of a row a thread; where these are fewer than the threads,
      // several groups of them share the parts
      struct State {
        float M, L;
        float4 o;
        __device__ void add(const float2* m, const float4* x) {   // kDmJoin states
          float top = M;
#pragma unroll
          for (int u = 0; u < kDmJoin; ++u)
            if (m[u].y > 0.f) top = fmaxf(top, m[u].x);
          const float f = top > M ? fast_exp2(M - top) : 1.f;
          M = top;
          L *= f;
          o.x *= f; o.y *= f; o.z *= f; o.w *= f;
#pragma unroll
          for (int u = 0; u < kDmJoin; ++u) {
            const float w = m[u].y > 0.f ? fast_exp2(m[u].x - M) : 0.f;
            L += w * m[u].y;
            o.x += w * x[u].x; o.y += w * x[u].y; o.z += w * x[u].z; o.w += w * x[u].w;
          }
        }
      };
      const int items = p.g * (D / 4), groups = min(kDmJoin, max(1, T / items)), group = tid / items;
      float2 m[kDmJoin];
      float4 x[kDmJoin];
      auto join = [&](int i, int first) {   // parts first, first + groups, ...; kDmJoin of them under way
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + cut.slot * p.g + i / (D / 4);
        const float4* part = reinterpret_cast<const float4*>(p.part + cut.slot * p.g * D) + i;
        State st{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int s0 = first; s0 < cut.parts; s0 += kDmJoin * groups) {
#pragma unroll
          for (int u = 0; u < kDmJoin; ++u) {
            const int s = s0 + u * groups, at = min(s, cut.parts - 1);
            m[u] = __ldcg(ml + (size_t)at * p.g);
            x[u] = __ldcg(part + (size_t)at * items);
            if (s >= cut.parts) m[u].y = 0.f;
          }
          st.add(m, x);
        }
        return st;
      };
      auto finish = [&](int i, const State& st) {
        const float inv = st.L > 0.f ? 1.f / st.L : 0.f;
        reinterpret_cast<float4*>(p.out + ((size_t)cut.seq * p.hq + cut.head * p.g) * D)[i] =
            make_float4(st.o.x * inv, st.o.y * inv, st.o.z * inv, st.o.w * inv);
        if (i % (D / 4) == 0 && p.scores)
          p.fin[((size_t)cut.seq * p.hkv + cut.head) * p.g + i / (D / 4)] = make_float2(st.L > 0.f ? st.M : 0.f, inv);
      };
      if (groups == 1) {
        for (int i = tid; i < items; i += T) finish(i, join(i, 0));
        continue;
      }
      float4* s_o = reinterpret_cast<float4*>(s_acc);
      float2* s_ml = reinterpret_cast<float2*>(s_acc + T * 4);
      if (group < groups) {
        const State st = join(tid - group * items, group);
        s_o[tid] = st.o;
        s_ml[tid] = make_float2(st.M, st.L);
      }
      __syncthreads();
      if (group == 0) {
        State st{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int u = 0; u < kDmJoin; ++u) {
          m[u] = u < groups ? s_ml[u * items + tid] : make_float2(0.f, 0.f);
          x[u] = u < groups ? s_o[u * items + tid] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        st.add(m, x);
        finish(tid, st);
      }
      __syncthreads();   // s_acc may be written again
    }
  }
  // Only now may the next kernel's CTAs come: sooner, they would crowd where this
  // grid's first CTAs end (eight sequences of 16,384 to 32,768 tokens in 4 bits: 85 us
  // with the call at the start, 73 here).
  asm volatile("griddepcontrol.launch_dependents;");
  if (dead)   // copies in flight land before the shared memory goes away
    for (int i = 0; i < ST; ++i) {
      const int use = uses + i;
      if (warp + use * W < k_ahead) mbar_drain(&sh.full[warp][use % ST], (use / ST) & 1);
    }
}

// ------------------------------------------------------------------- mass ---
struct AddMassParams {
  const float* scores;
  const float2* fin;
  const int32_t* seq_len;
  const float* mass_in;
  float* mass;
  int n_seq, hkv, g, most;
  float carry;
};

constexpr int kMassThreads = 128;

// A thread takes a token; the heads in their order, so the sum is the same in
// every call.  G: query heads of a KV head (0: any), as many scores side by side.
// The scores were just written and lie in L2 for the most part; sixteen loads are
// in flight a thread.
template <int G>
__global__ void __launch_bounds__(kMassThreads) add_mass_kernel(const __grid_constant__ AddMassParams p) {
  extern __shared__ float2 s_fin[];   // [hkv * g]
  const int a = blockIdx.y, g = G ? G : p.g;
  pdl_enter();
  const int len = min(max(__ldg(p.seq_len + a), 0), p.most);
  const int t = blockIdx.x * kMassThreads + threadIdx.x;
  if ((int)blockIdx.x * kMassThreads >= len) return;
  for (int i = threadIdx.x; i < p.hkv * g; i += kMassThreads) s_fin[i] = p.fin[(size_t)a * p.hkv * g + i];
  __syncthreads();
  if (t >= len) return;
  float sum = 0.f;
  const size_t step = (size_t)p.most * g;
  const float* s = p.scores + (size_t)a * p.hkv * step + (size_t)t * g;
  auto add = [&](float x, int i) {
    const float2 f = s_fin[i];
    sum += fast_exp2(x - f.x) * f.y;
  };
  if constexpr (G == 0) {
    for (int h = 0; h < p.hkv; ++h, s += step)
      for (int i = 0; i < g; ++i) add(__ldcs(s + i), h * g + i);
  } else {
    constexpr int V = G % 4 == 0 ? 4 : G % 2 == 0 ? 2 : 1, U = G >= 16 ? 1 : 16 / G;   // values a load, KV heads at a time
    int h = 0;
    for (; h + U <= p.hkv; h += U, s += U * step) {
      float x[U][G];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < G; i += V) {
          const float* q = s + u * step + i;
          if constexpr (V == 4) {
            const float4 y = __ldcs(reinterpret_cast<const float4*>(q));
            x[u][i] = y.x; x[u][i + 1] = y.y; x[u][i + 2] = y.z; x[u][i + 3] = y.w;
          } else if constexpr (V == 2) {
            const float2 y = __ldcs(reinterpret_cast<const float2*>(q));
            x[u][i] = y.x; x[u][i + 1] = y.y;
          } else {
            x[u][i] = __ldcs(q);
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < G; ++i) add(x[u][i], (h + u) * G + i);
    }
    for (; h < p.hkv; ++h, s += step)
#pragma unroll
      for (int i = 0; i < G; ++i) add(__ldcs(s + i), h * G + i);
  }
  const size_t o = (size_t)a * p.most + t;
  p.mass[o] = p.mass_in ? fmaf(p.carry, p.mass_in[o], sum) : sum;
}

struct DmLayout {
  size_t part, ml, fin, scores, total;
  size_t bytes(bool masses) const { return masses ? total : scores; }   // the scores are for the masses alone
};
DmLayout dm_layout(const kvs_pool* pool, int n_seq, int max_blocks, int g) {
  const kvs_pool_desc& d = pool->desc;
  DmLayout l{};
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t{255};
    return at;
  };
  const size_t pairs = (size_t)n_seq * d.num_kv_heads, parts = (size_t)pool->num_sms * kDmMaxCtas + pairs;
  l.part = take(parts * g * d.head_dim * 4);
  l.ml = take(parts * g * 8);
  l.fin = take(pairs * g * 8);
  l.scores = take(pairs * g * (size_t)max_blocks * d.block_tokens * 4);
  l.total = o;
  return l;
}

template <int FMT, int NT>
bool launch_dm(const DmParams& p, const kvs_pool* pool, int layer, cudaStream_t stream) {
  constexpr int smem = Dm<FMT, NT>::kSmem;
  if (!smem_limit_once<decode_mass_kernel<FMT, NT>>(smem, pool->device)) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pool->num_sms * Dm<FMT, NT>::kCtas));
  cfg.blockDim = dim3(Dm<FMT, NT>::W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_mass_kernel<FMT, NT>, p, pool->tk[layer], pool->tv[layer]) == cudaSuccess;
}

kvs_status decode_mass(kvs_pool* pool, int32_t layer, const void* q, int32_t n_q_heads, const int32_t* table, int32_t max_blocks,
                       const int32_t* seq_len, int32_t n_seq, float scale, float* out, const float* mass_in, float carry,
                       float* mass, void* ws, size_t ws_bytes, cudaStream_t stream, const std::string& what) {
  const kvs_pool_desc& d = pool->desc;
  if (layer < 0 || layer >= d.num_layers) return fail(KVS_ERR_INVALID_ARG, what + ": layer out of range");
  if (n_seq < 0 || max_blocks < 1) return fail(KVS_ERR_INVALID_ARG, what + ": bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, what + ": n_seq exceeds the pool's max_seqs");
  if (n_q_heads < 1 || n_q_heads % d.num_kv_heads) return fail(KVS_ERR_INVALID_ARG, what + ": n_q_heads must be a multiple of num_kv_heads");
  const int g = n_q_heads / d.num_kv_heads;
  if (g > kDmMaxGroup) return fail(KVS_ERR_UNSUPPORTED, what + ": more than 16 query heads per KV head");
  if (n_q_heads > 6144) return fail(KVS_ERR_UNSUPPORTED, what + ": more than 6,144 query heads");
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !std::isfinite(scale_log2)) return fail(KVS_ERR_INVALID_ARG, what + ": scale must be positive and finite");
  if (!std::isfinite(carry)) return fail(KVS_ERR_INVALID_ARG, what + ": carry must be finite");
  if (!mass && mass_in) return fail(KVS_ERR_INVALID_ARG, what + ": mass_in without mass");
  if (n_seq > 65535) return fail(KVS_ERR_UNSUPPORTED, what + ": more than 65,535 sequences");
  const long long most = (long long)max_blocks * d.block_tokens;
  if (most > 0x40000000ll || most * n_seq > 0x7fffffffll * 8) return fail(KVS_ERR_CAPACITY, what + ": too many tokens in the tables");
  if (n_seq == 0) return KVS_OK;
  if (!q || !table || !seq_len || !out || !ws) return fail(KVS_ERR_INVALID_ARG, what + ": null pointer");
  if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return fail(KVS_ERR_INVALID_ARG, what + ": q, out and ws must be 16-byte aligned");
  const DmLayout l = dm_layout(pool, n_seq, max_blocks, g);
  if (ws_bytes < l.bytes(mass != nullptr)) return fail(KVS_ERR_CAPACITY, what + ": workspace too small");
  if (kvs_status st = check_pool_device(pool, what.c_str()); st != KVS_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DmParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.table = table;
  p.seq_len = seq_len;
  const bool mx = d.dtype == KVS_DTYPE_MX4;
  if (mx) {
    p.ksc = static_cast<const uint8_t*>(pool->ksb[layer]);
    p.vsc = static_cast<const uint8_t*>(pool->vsb[layer]);
  }
  p.out = out;
  p.part = reinterpret_cast<float*>(w + l.part);
  p.part_ml = reinterpret_cast<float*>(w + l.ml);
  p.fin = reinterpret_cast<float2*>(w + l.fin);
  p.scores = mass ? reinterpret_cast<float*>(w + l.scores) : nullptr;
  p.tickets = pool->tickets;
  p.status = pool->status;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.hkv = d.num_kv_heads;
  p.g = g;
  p.hq = n_q_heads;
  p.capacity = d.capacity_blocks;
  p.most = (int)most;
  p.scale_log2 = scale_log2;
  bool ok;
  if (mx)
    ok = g <= 8 ? launch_dm<kFmtMx, 1>(p, pool, layer, stream) : launch_dm<kFmtMx, 2>(p, pool, layer, stream);
  else if (d.head_dim == 128)
    ok = g <= 8 ? launch_dm<kFmtBf16x128, 1>(p, pool, layer, stream) : launch_dm<kFmtBf16x128, 2>(p, pool, layer, stream);
  else
    ok = g <= 8 ? launch_dm<kFmtBf16x64, 1>(p, pool, layer, stream) : launch_dm<kFmtBf16x64, 2>(p, pool, layer, stream);
  if (ok) count_launch();
  if (ok && mass) {
    AddMassParams m{p.scores, p.fin, seq_len, mass_in, mass, n_seq, p.hkv, g, p.most, carry};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((most + kMassThreads - 1) / kMassThreads), (unsigned)n_seq);
    cfg.blockDim = dim3(kMassThreads);
    cfg.dynamicSmemBytes = (size_t)n_q_heads * sizeof(float2);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = g == 1 ? add_mass_kernel<1> : g == 2 ? add_mass_kernel<2> : g == 4 ? add_mass_kernel<4> : g == 8 ? add_mass_kernel<8>
                : g == 5 ? add_mass_kernel<5> : g == 16 ? add_mass_kernel<16> : add_mass_kernel<0>;
    ok = cudaLaunchKernelEx(&cfg, kern, m) == cudaSuccess;
    if (ok) count_launch();
  }
  return check_launch(what.c_str());
}

}  // namespace

size_t decode_mass_workspace_bytes(const kvs_pool* pool, int n_seq, int max_blocks, int g, bool masses) {
  return dm_layout(pool, n_seq, max_blocks, g).bytes(masses);
}

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_decode_attn_mass(kvs_pool* pool, int32_t layer, const void* q_dev, int32_t n_q_heads,
                                           const int32_t* block_table_dev, int32_t max_blocks, const int32_t* seq_len_dev,
                                           int32_t n_seq, float scale, float* out_dev, const float* mass_in_dev, float carry,
                                           float* mass_dev, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "decode_attn_mass: null pool");
  if (pool->desc.dtype != KVS_DTYPE_BF16) return fail(KVS_ERR_INVALID_ARG, "decode_attn_mass: pool is not BF16");
  if (!mass_dev && n_seq != 0) return fail(KVS_ERR_INVALID_ARG, "decode_attn_mass: null mass");
  return decode_mass(pool, layer, q_dev, n_q_heads, block_table_dev, max_blocks, seq_len_dev, n_seq, scale, out_dev, mass_in_dev,
                     carry, mass_dev, ws, ws_bytes, stream, "decode_attn_mass");
}

extern "C" kvs_status kvs_decode_attn_mx4(kvs_pool* pool, int32_t layer, const void* q_dev, int32_t n_q_heads,
                                          const int32_t* block_table_dev, int32_t max_blocks, const int32_t* seq_len_dev,
                                          int32_t n_seq, float scale, float* out_dev, const float* mass_in_dev, float carry,
                                          float* mass_dev, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "decode_attn_mx4: null pool");
  if (pool->desc.dtype != KVS_DTYPE_MX4) return fail(KVS_ERR_INVALID_ARG, "decode_attn_mx4: pool is not MX4");
  return decode_mass(pool, layer, q_dev, n_q_heads, block_table_dev, max_blocks, seq_len_dev, n_seq, scale, out_dev, mass_in_dev,
                     carry, mass_dev, ws, ws_bytes, stream, "decode_attn_mx4");
}
