// The attention weights of query chunks, added up by stored token:
//
//   mass[t] = carry * mass_in[t] + sum over rows r and heads h of e^(x_rht) / sum_t' e^(x_rht'),
//   x_rht = scale <q_rh, K_t>, t' and t below the row's limit
//
// Values are not read.  A weight needs its row's whole sum, and the scores of a
// prompt do not fit anywhere (8,192 rows of 32 heads: 4 GB), so the products are
// taken twice on the fifth-generation tensor cores, each time with the sum along
// a thread's own accumulator row, so that nothing is exchanged between threads:
//  pass 1  S = Q K^T: a thread has half a row of 128 scores of a query row, and keeps
//          that row's reference and sum;
//  pass 2  S^T = K Q^T: a thread has a key and adds up 2^(s - lse) over its half of
//          the columns, 128 (token, head) rows at a time, whose lse = log2 of the sum
//          lies in shared memory.
// Both are em_pass_kernel: two tiles of 128 rows (X) go to tensor memory, tiles of the
// other operand (Y) stream through a TMA ring past both, and four warpgroups turn S,
// in tensor memory too, into sums.  Scores and sums are float32.  Where a sequence has
// a tile of rows at most, pass 2 is em_keys_kernel: the rows stay and the keys stream;
// short calls of that kind are one kernel (em_whole_kernel).
//
// Items (a pair of X tiles, a range of Y tiles) are claimed in order, the longest
// first; with few rows and many keys, every CTA takes an even stretch of key tiles
// instead.  Calls with few of them cut the Y ranges: pass 1 leaves (reference, sum) of
// each cut, which em_join_kernel joins; pass 2 leaves a sum for each cut and KV head,
// which the last kernel adds in a fixed order.  A plan kernel counts the units of
// every sequence; up to 32 sequences are counted by a warp of pass 1.
//
// Measured, graph replays: 8,192 rows of 32 heads over themselves (8 KV heads of 128
// channels) 450 us, 217 and 226 for the passes: 1,270 and 1,220 TFLOP/s, 0.66 and 0.64
// of what cuBLAS reaches.  A pair of tiles takes 1,024 cycles of
// products and 1,024 of exponentials (8 lanes a cycle and scheduler); without any
// exponentials the passes take 172 and 150.  Eight times 32 rows after 3,500 to 8,192
// tokens 47 us: the keys are read twice at 5.8 TB/s (15 us each), the rest is starts (3
// us until the first copy of each pass) and the two small kernels.
#include <algorithm>
#include <cmath>

#include "tcgen05.cuh"
#include "internal.h"

namespace kvs {

namespace {

// Four warpgroups of sums, two for each X tile: one takes columns 0 to 63 of a
// product, one the others, so that a scheduler has four warps to choose from.
// Behind them a warp for each X tile that issues its products, one for the copies,
// and one that has the columns of pass 2 and in pass 1 half of the copies: a key
// tile is sixteen, which a warp issues in about 1,300 cycles.
constexpr int kEmSumWarps = 16, kEmThreads = (kEmSumWarps + 4) * 32;
constexpr int kEmMma = kEmSumWarps, kEmTma = kEmSumWarps + 2;   // and one more
constexpr int kEmTile = 128;
constexpr int kEmMaxCuts = 16;
constexpr int kEmEven = 10;   // tiles a CTA from which on stretches are even
constexpr uint32_t kEmCols = 512, kEmX = 384;   // scores in three buffers of 128 columns, behind them the X tiles

template <int D>
__host__ __device__ constexpr int em_tile_bytes() { return kEmTile * D * 2; }
template <int D>
__host__ __device__ constexpr int em_stages() { return D == 128 ? 4 : 8; }
template <int D>
__host__ __device__ constexpr int em_smem() { return 1024 + em_tile_bytes<D>() * (2 + em_stages<D>()); }

enum { kMClaim1, kMClaim2, kMBad, kMCuts1, kMCuts2, kMPer, kMTotal = 16 };

struct EmParams {
  const int32_t *table, *tok_off, *seq_len;
  uint32_t* status;
  int* hdr;
  int4* seq;          // [n_seq] {first row, rows, keys}
  int *off1, *off2;   // [n_seq + 1] units before each sequence: pairs of row tiles, pairs of key tiles
  float2* parts;      // pass 1: [cut][column half][n_tokens][hq] {reference, sum}
  float* nlse;        // [hkv][n_tokens][g] -log2 of the rows' sums
  float* sums;        // pass 2: [cut][column half][hkv][n_seq][most], few rows: [row tile][column half][hkv][most]
  int n_tokens, n_seq, max_blocks, capacity, g, hkv, hq, causal, slab_rows, most, cuts1, cuts2, sms, few, whole;   // cuts: the most there is room for; few: em_keys_kernel is pass 2; whole: CTAs of em_whole_kernel
  float scale_log2;
  int* tickets;       // calls without a plan: the claims of pass 1, zero between calls
};

// Cuts of every unit's Y tiles (1 to `most`, a lane each).  Items of about one
// length go in rounds over the SMs, others fill them evenly but for the last one's
// half; an item costs its tiles and about two more.
__device__ __forceinline__ int em_cuts(float units, float tiles, float longest, int most, float sms, int lane) {
  const float c = (float)(lane + 1), mean = tiles / fmaxf(units, 1.f), rounds = ceilf(units * c / sms);
  const bool even = mean > 0.9f * longest;
  float cost = (even ? rounds * mean / c : fmaxf(longest / c, tiles / sms + 0.5f * longest / c)) + 2.f * rounds;
  if (lane >= most || (lane > 0 && longest < c)) cost = INFINITY;
  int best = lane;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float cost2 = __shfl_xor_sync(0xffffffffu, cost, o);
    const int best2 = __shfl_xor_sync(0xffffffffu, best, o);
    if (cost2 < cost || (cost2 == cost && best2 < best)) {
      cost = cost2;
      best = best2;
    }
  }
  return best + 1;
}

// What a sequence brings.
struct EmCount {
  int t0, rows, keys, units1, units2, longest1, longest2, bad;
  unsigned long long tiles1, tiles2;   // twice the Y tiles of all units
};
__device__ __forceinline__ EmCount em_count(const EmParams& p, int a) {
  const int tt = kEmTile / p.g, tu = 2 * tt;
  const int t0 = __ldg(p.tok_off + a), t1 = __ldg(p.tok_off + a + 1), raw = __ldg(p.seq_len + a);
  if (raw < 0 || raw > p.most) set_err(p.status, KVS_DEVERR_SEQ_LEN);
  EmCount c{};
  c.bad = t0 < 0 || t1 < t0 || t1 > p.n_tokens;
  c.t0 = t0;
  c.rows = t1 - t0;
  c.keys = min(max(raw, 0), p.most);
  if (c.bad || c.rows == 0) return c;
  const int k = (c.keys + kEmTile - 1) / kEmTile, t = (c.rows - 1) / tt + 1;   // key tiles, row tiles
  c.units1 = (c.rows - 1) / tu + 1;
  c.units2 = p.few ? t : (c.keys + 2 * kEmTile - 1) / (2 * kEmTile);
  // causal: the new tokens' share of either range is half full on the mean
  c.tiles1 = (unsigned long long)c.units1 * (2 * k - (p.causal ? min(k, c.rows / kEmTile) : 0));
  c.tiles2 = p.few ? (unsigned long long)c.units2 * (2 * k) : (unsigned long long)t * (2 * c.units2 - (p.causal ? min(c.units2, c.rows / (2 * kEmTile)) : 0));
  c.longest1 = k;
  c.longest2 = p.few ? k : t;
  return c;
}

__global__ void __launch_bounds__(1024) em_plan_kernel(const __grid_constant__ EmParams p) {
  __shared__ int warp_sums[32];
  __shared__ unsigned long long s_tiles[2];
  __shared__ int s_longest[2];
  const int tid = threadIdx.x;
  if (tid < 2) {
    s_tiles[tid] = 0;
    s_longest[tid] = 0;
  }
  pdl_enter();
  int n1 = 0, n2 = 0, bad = 0;
  unsigned long long tiles1 = 0, tiles2 = 0;
  int longest1 = 0, longest2 = 0;
  for (int a0 = 0; a0 < p.n_seq; a0 += 1024) {
    const int a = a0 + tid;
    EmCount c{};
    if (a < p.n_seq) {
      c = em_count(p, a);
      p.seq[a] = make_int4(c.t0, c.rows, c.keys, 0);
    }
    bad |= c.bad;
    tiles1 += c.tiles1;
    tiles2 += c.tiles2;
    longest1 = max(longest1, c.longest1);
    longest2 = max(longest2, c.longest2);
    int total;
    const int b1 = block_exclusive_scan(c.units1, warp_sums, total);
    if (a < p.n_seq) p.off1[a] = n1 + b1;
    n1 += total;
    const int b2 = block_exclusive_scan(c.units2, warp_sums, total);
    if (a < p.n_seq) p.off2[a] = n2 + b2;
    n2 += total;
  }
  if (longest1) {
    atomicAdd(&s_tiles[0], tiles1);
    atomicAdd(&s_tiles[1], tiles2);
    atomicMax(&s_longest[0], longest1);
    atomicMax(&s_longest[1], longest2);
  }
  bad = __syncthreads_or(bad);
  if (tid >= 32) return;
  const float h = (float)p.hkv, sms = (float)p.sms;
  const int cuts1 = em_cuts((float)n1 * h, 0.5f * (float)s_tiles[0] * h, (float)s_longest[0], p.cuts1, sms, tid);
  const int cuts2 = em_cuts((float)n2 * h, 0.5f * (float)s_tiles[1] * h, (float)s_longest[1], p.cuts2, sms, tid);
  if (tid == 0) {
    p.hdr[kMCuts1] = cuts1;
    p.hdr[kMCuts2] = cuts2;
    if (bad) set_err(p.status, KVS_DEVERR_JOB);
    p.off1[p.n_seq] = bad ? 0 : n1;
    p.off2[p.n_seq] = bad ? 0 : n2;
    p.hdr[kMClaim1] = p.hdr[kMClaim2] = p.hdr[kMPer] = 0;
    p.hdr[kMBad] = bad;
  }
}

struct __align__(16) EmItem {
  int seq, head, cut, done;
  int t0, rows, keys, x0;       // of the sequence; x0: first token (pass 1) or key (pass 2) of the X tiles
  int y0, y1, behind, pad;      // Y tiles of the item; cuts behind this one that are empty
  int xs[2], xe[2];             // of them, those that X tile 0 / 1 takes
};

struct EmBars {
  uint64_t full[8], empty[8];
  uint64_t x_full, x_empty, x_there;     // X tiles in shared memory, read from there, in tensor memory
  uint64_t s_full[2][2], s_empty[2][2];  // scores of X tile 0 in buffers 0 and 1, of X tile 1 in buffer 2
  uint64_t it_full[2], it_empty[2];
  uint64_t fin[2];
};

struct EmCols {   // pass 2: of the 128 columns of a Y tile
  float nlse[kEmTile];
  int lim[kEmTile];
  int least;      // smallest limit
  int pad[3];
};

// Whole warp: the number of i in [1, n] with off[i] <= v (off ascends).
__device__ __forceinline__ int em_find(const int* off, int n, int v, int lane) {
  int lo = 0;
  while (n > 32) {
    const int step = (n + 31) / 32, i = (lane + 1) * step;
    const bool le = i <= n && __ldg(off + lo + i) <= v;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  const bool le = lane < n && __ldg(off + lo + lane + 1) <= v;
  return lo + __popc(__ballot_sync(0xffffffffu, le));
}

// Key tiles that row tile i of a sequence sees.
__device__ __forceinline__ int ek_tiles(const EmParams& p, int rows, int keys, int i, int tt) {
  const int lim = p.causal ? min(max(keys - rows + min(rows, (i + 1) * tt), 0), keys) : keys;
  return (lim + kEmTile - 1) / kEmTile;
}

// At most 32 sequences, a lane each.
struct EmLine {
  int t0, rows, keys, units;   // of this lane's sequence
  int end;                     // units up to it, its own among them
  int all, cuts;
  // Even stretches: where every sequence has one row tile at most, the key tiles of all
  // of them, KV head by KV head, form a line of which each CTA takes `per` (0: items
  // are claimed).  Eight times 32 rows after 3,500 to 8,192 tokens, 18 tiles a CTA: 47
  // us, 54 with claimed items; but 16 x 4 after 1,000, 40 / 8 heads, 7 tiles: 29.6
  // and 27.7, 4 x 16 after 500, 2 tiles: 21 and 16.5 (a second pair costs its start).
  int tiles, tiles_end, line, per;   // of this lane's sequence, up to it, of a KV head
};
// Whole warp: the lanes' tiles on the line.
__device__ __forceinline__ void em_even_line(const EmParams& p, EmLine& r, int lane) {
  r.tiles = r.rows > 0 ? ek_tiles(p, r.rows, r.keys, 0, kEmTile / p.g) : 0;
  r.tiles_end = r.tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, r.tiles_end, o);
    r.tiles_end += lane >= o ? x : 0;
  }
  r.line = __shfl_sync(0xffffffffu, r.tiles_end, 31);
}
// Whole warp: what the stretch [place, stop) has of the pair at `place`.
struct EmStretch {
  int seq, head, y0, y1, cut, behind;   // behind: cuts that the pair does not have
};
__device__ __forceinline__ EmStretch em_stretch(const EmParams& p, const EmLine& r, int place, int stop, int lane) {
  constexpr unsigned kAll = 0xffffffffu;
  EmStretch e;
  e.head = place / r.line;
  const int at = place - e.head * r.line;
  e.seq = __popc(__ballot_sync(kAll, lane < p.n_seq && r.tiles_end <= at));
  const int tiles = __shfl_sync(kAll, r.tiles, e.seq);
  e.y0 = at - (__shfl_sync(kAll, r.tiles_end, e.seq) - tiles);
  e.y1 = min(tiles, e.y0 + stop - place);
  e.cut = (int)blockIdx.x - (place - e.y0) / r.per;
  e.behind = e.y1 == tiles ? r.cuts - 1 - e.cut : 0;
  return e;
}
// Whole warp, pass 1: what the plan kernel finds otherwise; the first CTA leaves what
// the kernels behind it need.
__device__ __forceinline__ EmLine em_line1(const EmParams& p, int lane) {
  constexpr unsigned kAll = 0xffffffffu;
  EmCount c{};
  if (lane < p.n_seq) c = em_count(p, lane);
  const bool bad = __any_sync(kAll, c.bad);
  auto scan = [&](int end, float tiles, int longest, int most, int& last, int& cuts) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kAll, end, o);
      end += lane >= o ? x : 0;
      tiles += __shfl_xor_sync(kAll, tiles, o);
    }
    last = __shfl_sync(kAll, end, 31);
    cuts = em_cuts((float)last * (float)p.hkv, 0.5f * tiles * (float)p.hkv, (float)__reduce_max_sync(kAll, longest), most, (float)p.sms, lane);
    return end;
  };
  EmLine r{c.t0, c.rows, c.keys, c.units1};
  r.end = scan(c.units1, (float)c.tiles1, c.longest1, p.cuts1, r.all, r.cuts);
  if (p.few && p.cuts1 > 1 && !bad) {
    em_even_line(p, r, lane);
    const long long line = (long long)r.line * p.hkv;
    if (!__any_sync(kAll, r.rows > kEmTile / p.g || (r.rows > 0 && r.tiles == 0)) && line >= kEmEven * p.sms && line <= 0x3fffffff) {
      const int longest = __reduce_max_sync(kAll, r.tiles), most = p.cuts1 - 1;
      r.per = max(((int)line + p.sms - 1) / p.sms, (longest + most - 1) / most);
      r.cuts = (longest + r.per - 2) / r.per + 1;
    }
  }
  if (blockIdx.x == 0) {
    int n2, cuts2;
    const int end2 = scan(c.units2, (float)c.tiles2, c.longest2, p.cuts2, n2, cuts2);
    if (lane < p.n_seq) {
      p.seq[lane] = make_int4(c.t0, c.rows, c.keys, 0);
      p.off2[lane] = end2 - c.units2;
    }
    if (lane == 0) {
      if (bad) set_err(p.status, KVS_DEVERR_JOB);
      p.off2[p.n_seq] = bad ? 0 : n2;
      p.hdr[kMCuts1] = r.cuts;
      p.hdr[kMCuts2] = cuts2;
      p.hdr[kMClaim2] = 0;
      p.hdr[kMPer] = r.per;
      p.hdr[kMBad] = bad;
    }
  }
  if (bad) r.all = 0;
  return r;
}
// Pass 2: what that CTA or the plan kernel left.
__device__ __forceinline__ EmLine em_line2(const EmParams& p, int lane) {
  EmLine r{};
  r.cuts = __ldg(p.hdr + kMCuts2);
  r.all = __ldg(p.off2 + p.n_seq);
  if (lane < p.n_seq) {
    const int4 s = __ldg(p.seq + lane);
    const int first = __ldg(p.off2 + lane);
    r.t0 = s.x;
    r.rows = s.y;
    r.keys = s.z;
    r.end = __ldg(p.off2 + lane + 1);
    r.units = r.end - first;
  }
  r.per = p.n_seq <= 32 ? __ldg(p.hdr + kMPer) : 0;
  if (r.per) em_even_line(p, r, lane);
  return r;
}

// Whole warp: the sequence of a unit, with its rows and units.
struct EmPlace {
  int seq, t0, rows, keys, first, count;
};
__device__ __forceinline__ EmPlace em_place(const EmParams& p, const EmLine& line, const int* off, int unit, int lane) {
  constexpr unsigned kAll = 0xffffffffu;
  EmPlace r;
  if (p.n_seq <= 32) {
    r.seq = __popc(__ballot_sync(kAll, lane < p.n_seq && line.end <= unit));
    r.t0 = __shfl_sync(kAll, line.t0, r.seq);
    r.rows = __shfl_sync(kAll, line.rows, r.seq);
    r.keys = __shfl_sync(kAll, line.keys, r.seq);
    r.count = __shfl_sync(kAll, line.units, r.seq);
    r.first = __shfl_sync(kAll, line.end, r.seq) - r.count;
  } else {
    r.seq = em_find(off, p.n_seq, unit, lane);
    const int4 s = __ldg(p.seq + r.seq);
    r.t0 = s.x;
    r.rows = s.y;
    r.keys = s.z;
    r.first = __ldg(off + r.seq);
    r.count = __ldg(off + r.seq + 1) - r.first;
  }
  return r;
}

// Blocks of key tiles j .. j + 3 of sequence a, eight lanes a tile; -1 where there is none.
__device__ __forceinline__ int em_blocks(const EmParams& p, int a, int j, int keys, int lane) {
  const int b = j * 8 + lane;
  int id = -1;
  if (b < (keys + 15) / 16) {
    id = __ldg(p.table + (size_t)a * p.max_blocks + b);
    if (id < 0 || id >= p.capacity) {
      set_err(p.status, KVS_DEVERR_BLOCK_ID);
      id = -1;
    }
  }
  return id;
}

// Lanes [from, to): block `lane` of a key tile; one without an id arrives as zeros.
template <int HF>
__device__ __forceinline__ void em_copy_keys(const EmParams& p, const CUtensorMap& tk, uint8_t* dst, int id, int head, uint64_t* bar,
                                             int lane, int from, int to) {
  if (lane >= from && lane < to) {
    const int row = id >= 0 ? (id * p.hkv + head) * 16 : p.slab_rows;
#pragma unroll
    for (int hf = 0; hf < HF; ++hf) tma_load_3d(dst + hf * kEmTile * 128 + lane * 2048, &tk, 0, row, hf, bar);
  }
  __syncwarp();
}

// sum over 64 columns of 2^(scale v + by); by(i): what is added to columns i and i + 1.
template <typename F>
__device__ __forceinline__ float em_sum_up(const uint32_t* v, float2 scale, F by) {
  float2 sum[4] = {};
#pragma unroll
  for (int i = 0; i < 64; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = __ffma2_rn(make_float2(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1])), scale, by(i + 2 * k));
      sum[k] = __fadd2_rn(sum[k], make_float2(fast_exp2(a.x), fast_exp2(a.y)));
    }
  const float2 t = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
  return t.x + t.y;
}

template <int D, int PASS>
__global__ void __launch_bounds__(kEmThreads, 1)
em_pass_kernel(const __grid_constant__ EmParams p, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk) {
  constexpr int HF = D / 64;
  constexpr int ST = em_stages<D>();
  constexpr int kTile = em_tile_bytes<D>();
  constexpr int kHalf = kEmTile * 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ EmBars bars;
  __shared__ EmItem work[2];
  __shared__ __align__(16) EmCols cols[PASS == 2 ? ST : 1];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.full[i], PASS == 2 ? 2 : 1);     // the copies; pass 2: the column warp
      mbar_init(&bars.empty[i], PASS == 2 ? 2 + kEmSumWarps : 2);   // both X tiles' products; pass 2: the columns are read
    }
    mbar_init(&bars.x_full, 1);
    mbar_init(&bars.x_empty, kEmSumWarps);
    mbar_init(&bars.x_there, kEmSumWarps);
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[x][b], 1);
        mbar_init(&bars.s_empty[x][b], kEmSumWarps / 2);
      }
      mbar_init(&bars.it_full[x], 1);
      mbar_init(&bars.it_empty[x], kEmSumWarps + 3);
    }
    mbar_init(&bars.fin[0], 1);
    mbar_init(&bars.fin[1], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, kEmCols);
    tmem_relinquish();
  }
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto sX = [&](int x) { return base + kTile * x; };
  auto ring = [&](int i) { return base + kTile * (2 + i); };
  // Rows of a query tile behind its last whole token are never copied to; what they
  // hold stays in their own rows (pass 1) or columns (pass 2, masked) of S.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tt = kEmTile / p.g;
  auto stop = [&]() { return __any_sync(0xffffffffu, s_abort != 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, p.status);
    return __all_sync(0xffffffffu, ok);
  };

  auto key_blocks = [&](int a, int j, int keys) { return em_blocks(p, a, j, keys, lane); };
  auto copy_keys = [&](uint8_t* dst, int id, int head, uint64_t* bar, int from, int to) {
    em_copy_keys<HF>(p, tk, dst, id, head, bar, lane, from, to);
  };

  if (warp >= kEmSumWarps) {
    if (warp == kEmTma) {
      // --------------------------------------------- claims and TMA copies
      const int* off = PASS == 1 ? p.off1 : p.off2;
      int* counter = PASS == 1 && p.tickets ? p.tickets : p.hdr + (PASS == 1 ? kMClaim1 : kMClaim2);
      int n = 0, nx = 0, ni = 0, armed = -1;
      bool ok = true;
      // a claim is under way while other loads are
      int claimed = 0;
      auto claim_next = [&]() {
        if (lane == 0) claimed = atomicAdd(counter, 1);
      };
      auto claim_there = [&]() { return (unsigned)__shfl_sync(0xffffffffu, claimed, 0); };
      claim_next();
      EmLine line{};
      if (PASS == 2) {
        line = em_line2(p, lane);
      } else if (p.tickets) {   // no plan: this warp counts for itself
        line = em_line1(p, lane);
      } else {
        line.cuts = __ldg(p.hdr + kMCuts1);
        line.all = __ldg(off + p.n_seq);
      }
      const int cuts = line.cuts;
      const bool even = PASS == 1 && line.per;
      const unsigned claims = even ? 0u : (unsigned)line.all * p.hkv * cuts;
      unsigned claim = claim_there();
      int place = (int)blockIdx.x * line.per;   // even stretches
      const int stop_at = min(line.line * p.hkv, place + line.per);
      auto copy_rows = [&](uint8_t* dst, int tok, int head, uint64_t* bar) {  // one lane
        for (int hf = 0; hf < HF; ++hf) tma_load_5d(dst + hf * kHalf, &tq, 0, 0, tok, head, hf, bar);
      };
      const uint32_t row_bytes = (uint32_t)(HF * tt * p.g * 128);
      for (;; claim = claim_there()) {
        if (stop()) { ok = false; break; }
        const int slot = ni & 1;
        if (ni >= 2 && !wait(&bars.it_empty[slot], ((ni - 2) >> 1) & 1)) { ok = false; break; }
        EmItem it{};
        it.done = even ? place >= stop_at : claim >= claims;
        int nt_x[2] = {0, 0};
        if (even && !it.done) {
          const EmStretch e = em_stretch(p, line, place, stop_at, lane);
          it.seq = e.seq;
          it.head = e.head;
          it.cut = e.cut;
          it.behind = e.behind;
          it.t0 = __shfl_sync(0xffffffffu, line.t0, e.seq);
          it.rows = __shfl_sync(0xffffffffu, line.rows, e.seq);
          it.keys = __shfl_sync(0xffffffffu, line.keys, e.seq);
          it.y0 = it.xs[0] = it.xs[1] = e.y0;
          it.y1 = it.xe[0] = e.y1;   // rows of the second X tile: none
          place += e.y1 - e.y0;
        } else if (!it.done) {
          const unsigned u = claim / (unsigned)cuts, unit = u / (unsigned)p.hkv;
          it.cut = (int)(claim - u * cuts);
          it.head = (int)(u - unit * p.hkv);
          const EmPlace at = em_place(p, line, off, (int)unit, lane);
          it.seq = at.seq;
          it.t0 = at.t0;
          it.rows = at.rows;
          it.keys = at.keys;
          const int first = at.first, count = at.count;
          const int before = it.keys - it.rows;   // row j sees keys up to before + j (causal)
          if constexpr (PASS == 1) {
            it.x0 = (count - 1 - ((int)unit - first)) * 2 * tt;   // the last rows, which see most, first
            for (int x = 0; x < 2; ++x) {
              const int j0 = it.x0 + x * tt, j1 = min(it.rows, j0 + tt);
              const int lim = p.causal ? min(max(before + j1, 0), it.keys) : it.keys;
              nt_x[x] = j0 < it.rows ? (lim + kEmTile - 1) / kEmTile : 0;
            }
            const int nt = max(nt_x[0], nt_x[1]);
            it.y0 = nt * it.cut / cuts;
            it.y1 = nt * (it.cut + 1) / cuts;
            for (int x = 0; x < 2; ++x) {
              it.xs[x] = it.y0;
              it.xe[x] = min(it.y1, nt_x[x]);
            }
          } else {
            it.x0 = ((int)unit - first) * 2 * kEmTile;
            const int tiles = (it.rows + tt - 1) / tt;
            for (int x = 0; x < 2; ++x) {
              const int key = it.x0 + x * kEmTile;
              nt_x[x] = key < it.keys ? min(tiles, p.causal ? max(0, key - before) / tt : 0) : tiles;   // first tile that sees the key
            }
            const int n_y = tiles - nt_x[0];
            it.y0 = nt_x[0] + n_y * it.cut / cuts;
            it.y1 = nt_x[0] + n_y * (it.cut + 1) / cuts;
            for (int x = 0; x < 2; ++x) {
              it.xs[x] = max(it.y0, nt_x[x]);
              it.xe[x] = it.y1;
            }
          }
        }
        if (lane == 0) {
          work[slot] = it;
          mbar_arrive(&bars.it_full[slot]);
        }
        __syncwarp();
        ++ni;
        if (it.done) break;
        if (!even) claim_next();
        if (it.y0 >= it.y1) continue;
        int ids = PASS == 1 ? key_blocks(it.seq, it.y0, it.keys) : key_blocks(it.seq, it.x0 / kEmTile, it.keys);
        int ids_next = PASS == 1 ? key_blocks(it.seq, it.y0 + 4, it.keys) : 0;
        // X tiles, once those of the item before are in tensor memory
        if (nx >= 1 && !wait(&bars.x_empty, (nx - 1) & 1)) { ok = false; break; }
        const bool two = PASS == 1 ? it.x0 + tt < it.rows : it.x0 + kEmTile < it.keys;
        if (lane == 0) mbar_arrive_expect_tx(&bars.x_full, (two ? 2u : 1u) * (PASS == 1 ? row_bytes : (uint32_t)kTile));
        __syncwarp();
        for (int x = 0; x < (two ? 2 : 1); ++x) {
          if constexpr (PASS == 1) {
            if (lane == 0) copy_rows(sX(x), it.t0 + it.x0 + x * tt, it.head, &bars.x_full);
            __syncwarp();
          } else {
            copy_keys(sX(x), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * x), it.head, &bars.x_full, 0, 8);
          }
        }
        ++nx;
        for (int j = it.y0; j < it.y1; ++j) {
          const int turn = (j - it.y0) & 3;
          if (PASS == 1 && turn == 0 && j > it.y0) {
            ids = ids_next;
            ids_next = key_blocks(it.seq, j + 4, it.keys);
          }
          const int s = n % ST;
          if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bars.full[s], PASS == 1 ? (uint32_t)kTile : row_bytes);
          __syncwarp();
          if constexpr (PASS == 1) {
            copy_keys(ring(s), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * turn), it.head, &bars.full[s], 0, 4);
          } else {
            if (lane == 0) copy_rows(ring(s), it.t0 + j * tt, it.head, &bars.full[s]);
            __syncwarp();
          }
          armed = n++;
        }
        if (!ok) break;
      }
      if (!ok) {
        s_abort = 1;
        // copies in flight land before the shared memory goes away
        for (int m = max(0, armed - ST + 1); m <= armed; ++m) mbar_drain(&bars.full[m % ST], (m / ST) & 1);
        if (nx) mbar_drain(&bars.x_full, (nx - 1) & 1);
      }
      if (PASS == 1 && p.tickets) {
        // every CTA claims once in vain; who does so last leaves the counter at zero
        for (claim = claim_there(); claim < claims; claim = claim_there()) claim_next();
        if (lane == 0 && claim == claims + gridDim.x - 1) *reinterpret_cast<volatile int*>(p.tickets) = 0;
      }
    } else if (warp < kEmTma) {
      // ------------------------------------------- products of one X tile
      const int x = warp - kEmMma;
      constexpr uint32_t idS = umma_idesc_bf16(128, 128, false, false);
      constexpr uint32_t kHi = ex_desc_hi(1024);
      const uint32_t y_lo = ex_desc_lo(smem_u32(ring(0)), 16), tX = tmem + kEmX + (uint32_t)(D / 2) * x;
      int nx = 0, b = 0, s = 0;
      uint32_t full_par = 0, free_par = 1;   // a fresh buffer counts as handed back
      bool ok = true;
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      for (int ni = 0;; ++ni) {
        const int slot = ni & 1;
        if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
        const int y0 = work[slot].y0, y1 = work[slot].y1, xs = work[slot].xs[x], xe = work[slot].xe[x], done = work[slot].done;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
        if (done) break;
        if (y0 >= y1) continue;
        if (!wait(&bars.x_there, nx & 1)) { ok = false; break; }
        ++nx;
        for (int j = y0; j < y1; ++j) {
          if (!wait(&bars.full[s], full_par)) { ok = false; break; }
          if (j >= xs && j < xe) {
            if (!wait(&bars.s_empty[x][b], free_par)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ya = y_lo + s * (kTile / 16), d = tmem + 128u * (2 * x + b);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                ex_mma_ts(d, tX + 8u * kk, ya + ((kk >> 2) * kHalf + (kk & 3) * 32) / 16, kHi, idS, kk > 0);
              umma_commit(&bars.s_full[x][b]);
              umma_commit(&bars.empty[s]);
            }
            __syncwarp();
            if (x == 1 || b == 1) free_par ^= 1u;
            if (x == 0) b ^= 1;
          } else {
            commit(&bars.empty[s]);
          }
          if (++s == ST) {
            s = 0;
            full_par ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (!ok) s_abort = 1;
      // every product issued has completed before the tensor memory is released
      commit(&bars.fin[x]);
      mbar_wait_bounded(&bars.fin[x], 0, p.status);
    } else if (PASS == 1) {
      // ---------------------------------- the other half of every key tile
      int n = 0;
      bool ok = true;
      for (int ni = 0;; ++ni) {
        const int slot = ni & 1;
        if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
        const int seq = work[slot].seq, head = work[slot].head, keys = work[slot].keys, y0 = work[slot].y0, y1 = work[slot].y1;
        const int done = work[slot].done, behind = work[slot].behind, cut = work[slot].cut, t0 = work[slot].t0, rows = work[slot].rows;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
        if (done) break;
        for (int i = lane; behind > 0 && i < rows * p.g; i += 32) {   // even stretches: one row tile
          const size_t at = (size_t)(t0 + i / p.g) * p.hq + head * p.g + i % p.g;
          for (int k = 2 * (cut + 1); k < 2 * (cut + 1 + behind); ++k) p.parts[(size_t)k * p.n_tokens * p.hq + at] = make_float2(0.f, 0.f);
        }
        if (y0 >= y1) continue;
        int ids = key_blocks(seq, y0, keys), ids_next = key_blocks(seq, y0 + 4, keys);
        for (int j = y0; j < y1; ++j) {
          const int turn = (j - y0) & 3, s = n % ST;
          if (turn == 0 && j > y0) {
            ids = ids_next;
            ids_next = key_blocks(seq, j + 4, keys);
          }
          if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
          // counted by the barrier that the other warp arms, before or after this
          copy_keys(ring(s), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * turn), head, &bars.full[s], 4, 8);
          ++n;
        }
        if (!ok) break;
      }
      if (!ok) {
        s_abort = 1;
        // copies in flight land before the shared memory goes away
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 24)) {
        }
      }
    } else {
      // ------------------------------------- columns: limits and sums of the rows
      int n = 0;
      bool ok = true;
      for (int ni = 0;; ++ni) {
        const int slot = ni & 1;
        if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
        const EmItem it = work[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
        if (it.done) break;
        // column c of tile j is row (j tt g + c) of the sequence and KV head
        const float* rows = p.nlse + ((size_t)it.head * p.n_tokens + it.t0) * p.g;
        const int n_rows = it.rows * p.g, per = tt * p.g;
        float next[4];
        auto load = [&](int j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = i * 32 + lane, row = j * per + c;
            next[i] = c < per && row < n_rows ? rows[row] : -INFINITY;
          }
        };
        if (it.y0 < it.y1) load(it.y0);
        for (int j = it.y0; j < it.y1; ++j) {
          float v[4];
          int lim[4], least = 0x7fffffff;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = next[i];
            const int c = i * 32 + lane, tok = j * tt + c / p.g;
            lim[i] = v[i] == -INFINITY ? 0 : p.causal ? max(it.keys - it.rows + tok + 1, 0) : it.keys;
            least = min(least, lim[i]);
          }
          if (j + 1 < it.y1) load(j + 1);
          least = __reduce_min_sync(0xffffffffu, least);
          const int s = n % ST;
          if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cols[s].nlse[i * 32 + lane] = v[i];
            cols[s].lim[i * 32 + lane] = lim[i];
          }
          if (lane == 0) cols[s].least = least;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.full[s]);
          ++n;
        }
        if (!ok) break;
      }
      if (!ok) s_abort = 1;
    }
  } else {
    // ------------------------------------------------------------ sums
    const int x = (warp >> 2) & 1, half = warp >> 3, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, tS = tmem + lanes + 256u * x + 64u * half;
    const int rt = r / p.g, rg = r - rt * p.g;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    int n = 0, nx = 0, b = 0;   // Y tiles, items with any, score buffer
    uint32_t s_par = 0;
    bool ok = true;
    for (int ni = 0;; ++ni) {
      const int slot = ni & 1;
      if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
      const EmItem it = work[slot];
      const int xs = work[slot].xs[x], xe = work[slot].xe[x];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
      if (it.done) break;
      const int tok = it.x0 + x * tt + rt;               // pass 1: this row's token
      const int key = it.x0 + x * kEmTile + r;           // pass 2: this row's key
      const bool live = PASS == 1 ? rt < tt && tok < it.rows : key < it.keys;
      const int lim = p.causal ? min(it.keys - it.rows + tok + 1, it.keys) : it.keys;   // pass 1: keys that the row sees
      float m = 0.f, l = 0.f;
      if (it.y0 < it.y1) {
        // X goes to tensor memory (a product that takes it from there reads half
        // as much of shared memory, which bounds it otherwise): every thread half
        // of its row.  The products of the item before are complete: this
        // thread has seen its X tile's last ones.
        if (!wait(&bars.x_full, nx & 1)) { ok = false; break; }
        ++nx;
        uint32_t w[D / 4];
        const uint8_t* row = sX(x) + (D == 128 ? half * kHalf : 0);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + swz128((uint32_t)r * 128 + 16 * (i + (D == 128 ? 0 : 4 * half))));
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
        const uint32_t tX = tmem + lanes + kEmX + (uint32_t)(D / 2) * x + (uint32_t)(D / 4) * half;
        if constexpr (D == 128) tmem_st32(tX, w);
        else tmem_st16(tX, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.x_empty);
          mbar_arrive(&bars.x_there);
        }
      }
      // Pass 1: keys below `whole` are visible to every live row of the warp.
      // Pass 2: this warp's last key.
      const bool any_live = __any_sync(0xffffffffu, live);
      const int whole = PASS == 1 ? __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff) : 0;
      const int last_key = it.x0 + x * kEmTile + (warp & 3) * 32 + 31;
      uint32_t v[64];
      for (int j = it.y0; j < it.y1; ++j) {
        const int s = n % ST;
        // also where this X tile passes the Y tile by: a stage is handed back once a turn
        if (PASS == 2 && !wait(&bars.full[s], (n / ST) & 1)) { ok = false; break; }
        if (j >= xs && j < xe) {
          if (!wait(&bars.s_full[x][b], s_par)) { ok = false; break; }
          tc_fence_after();
          tmem_ld32_issue(tS + 128u * b, v);
          tmem_ld32_issue(tS + 128u * b + 32, v + 32);
          tmem_ld32x2_wait(v, v + 32);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.s_empty[x][b]);
          if (x == 1 || b == 1) s_par ^= 1u;
          if (x == 0) b ^= 1;
          if (!any_live) {
            // no row of this warp belongs to the sequence
          } else if constexpr (PASS == 1) {
            const int key0 = j * kEmTile + 64 * half;
            if (key0 + 64 > whole) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (key0 + i >= lim) v[i] = 0xff800000u;
            }
            // The reference is the maximum of the first columns (a row that sees
            // later ones sees all of these) and moves only where a sum gets out of
            // hand: any reference within 2^60 of the maximum serves float32 as well.
            const bool fresh = j == xs;
            float sum = fresh ? INFINITY : em_sum_up(v, sc2, [&](int) { return make_float2(-m, -m); });
            if (__any_sync(0xffffffffu, !(sum < 0x1p60f))) {
              float top = __uint_as_float(v[0]);
#pragma unroll
              for (int i = 1; i < 64; ++i) top = fmaxf(top, __uint_as_float(v[i]));
              top *= p.scale_log2;
              if (!(sum < 0x1p60f)) {
                if (!fresh) l *= fast_exp2(m - top);
                m = top == -INFINITY ? 0.f : top;
              }
              sum = em_sum_up(v, sc2, [&](int) { return make_float2(-m, -m); });
            }
            l += sum;
          } else {
            const EmCols& cl = cols[s];
            if (last_key >= cl.least) {
#pragma unroll
              for (int i = 0; i < 64; i += 4) {
                const int4 u = *reinterpret_cast<const int4*>(cl.lim + 64 * half + i);
                if (key >= u.x) v[i] = 0xff800000u;
                if (key >= u.y) v[i + 1] = 0xff800000u;
                if (key >= u.z) v[i + 2] = 0xff800000u;
                if (key >= u.w) v[i + 3] = 0xff800000u;
              }
            }
            l += em_sum_up(v, sc2, [&](int i) { return *reinterpret_cast<const float2*>(cl.nlse + 64 * half + i); });
          }
        }
        if (PASS == 2) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.empty[s]);
        }
        ++n;
      }
      if (!ok) break;
      if (!live) continue;
      const size_t cut = 2 * it.cut + half;
      if constexpr (PASS == 1)
        p.parts[(cut * p.n_tokens + it.t0 + tok) * p.hq + it.head * p.g + rg] = make_float2(m, l);
      else
        p.sums[((cut * p.hkv + it.head) * p.n_seq + it.seq) * p.most + key] = l;
    }
    if (!ok) s_abort = 1;
  }
  asm volatile("griddepcontrol.launch_dependents;");   // not sooner: small CTAs would crowd where this grid's first ones end
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kEmCols);
  }
}

// ------------------------------------------------- few rows: keys stream past
// Pass 2 for calls whose rows are few tiles: a pair of key tiles would wait for
// its copies, its items and its tensor memory to see one tile of rows.  Here a row
// tile stays in shared memory and the keys stream past it, as in pass 1: S^T =
// K Q^T of one key tile after the other, alternating between two groups of warps,
// whose threads write the sum of a key's 64 columns for each half.  A key's sums
// of all row tiles, halves and KV heads are added by the last kernel.
struct EkBars {
  uint64_t full[8], empty[8];
  uint64_t x_full[2], x_empty[2], c_full[2], c_empty[2];
  uint64_t s_full[2][2], s_empty[2][2];
  uint64_t it_full[2], it_empty[2];
  uint64_t fin[2];
};

struct EkItem {
  int seq, head, tile, done;    // tile: row tile of the sequence
  int t0, rows, keys, unit;     // unit: row tile of the call
  int y0, y1, pad[2];           // key tiles
};

template <int D>
__global__ void __launch_bounds__(kEmThreads, 1)
em_keys_kernel(const __grid_constant__ EmParams p, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk) {
  constexpr int HF = D / 64, ST = em_stages<D>(), kTile = em_tile_bytes<D>(), kHalf = kEmTile * 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ EkBars bars;
  __shared__ EkItem work[2];
  __shared__ __align__(16) EmCols cols[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 2);      // both product warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.x_full[i], 1);
      mbar_init(&bars.x_empty[i], 2);
      mbar_init(&bars.c_full[i], 1);
      mbar_init(&bars.c_empty[i], kEmSumWarps);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[i][b], 1);
        mbar_init(&bars.s_empty[i][b], kEmSumWarps / 2);
      }
      mbar_init(&bars.it_full[i], 1);
      mbar_init(&bars.it_empty[i], kEmSumWarps + 3);
      mbar_init(&bars.fin[i], 1);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, kEmCols);
    tmem_relinquish();
  }
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto ring = [&](int i) { return base + kTile * (2 + i); };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tt = kEmTile / p.g;
  auto stop = [&]() { return __any_sync(0xffffffffu, s_abort != 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, p.status);
    return __all_sync(0xffffffffu, ok);
  };
  auto key_blocks = [&](int a, int j, int keys) { return em_blocks(p, a, j, keys, lane); };
  auto copy_keys = [&](uint8_t* dst, int id, int head, uint64_t* bar, int from, int to) {
    em_copy_keys<HF>(p, tk, dst, id, head, bar, lane, from, to);
  };

  if (warp >= kEmSumWarps) {
    bool ok = true;
    if (warp == kEmTma) {
      // ----------------------------------- claims, rows, half of every key tile
      int claimed = 0;
      auto claim_next = [&]() {
        if (lane == 0) claimed = atomicAdd(p.hdr + kMClaim2, 1);
      };
      auto claim_there = [&]() { return (unsigned)__shfl_sync(0xffffffffu, claimed, 0); };
      claim_next();
      const EmLine line = em_line2(p, lane);
      const int cuts = line.cuts;
      const bool even = line.per != 0;
      const unsigned claims = (unsigned)line.all * p.hkv * cuts;
      unsigned claim = claim_there();
      int place = (int)blockIdx.x * line.per;
      const int stop_at = min(line.line * p.hkv, place + line.per);
      int n = 0, nx = 0, armed = -1;
      for (int ni = 0;; ++ni, claim = claim_there()) {
        if (stop()) { ok = false; break; }
        const int slot = ni & 1;
        if (ni >= 2 && !wait(&bars.it_empty[slot], ((ni - 2) >> 1) & 1)) { ok = false; break; }
        EkItem it{};
        it.done = even ? place >= stop_at : claim >= claims;
        if (even && !it.done) {
          const EmStretch e = em_stretch(p, line, place, stop_at, lane);
          it.seq = e.seq;
          it.head = e.head;
          it.unit = __shfl_sync(0xffffffffu, line.end - line.units, e.seq);
          it.t0 = __shfl_sync(0xffffffffu, line.t0, e.seq);
          it.rows = __shfl_sync(0xffffffffu, line.rows, e.seq);
          it.keys = __shfl_sync(0xffffffffu, line.keys, e.seq);
          it.y0 = e.y0;
          it.y1 = e.y1;
          place += e.y1 - e.y0;
        } else if (!it.done) {
          const unsigned u = claim / (unsigned)cuts, unit = u / (unsigned)p.hkv;
          const int cut = (int)(claim - u * cuts);
          it.head = (int)(u - unit * p.hkv);
          const EmPlace at = em_place(p, line, p.off2, (int)unit, lane);
          it.seq = at.seq;
          it.unit = (int)unit;
          it.tile = it.unit - at.first;
          it.t0 = at.t0;
          it.rows = at.rows;
          it.keys = at.keys;
          const int nt = ek_tiles(p, it.rows, it.keys, it.tile, tt);
          it.y0 = nt * cut / cuts;
          it.y1 = nt * (cut + 1) / cuts;
        }
        if (lane == 0) {
          work[slot] = it;
          mbar_arrive(&bars.it_full[slot]);
        }
        __syncwarp();
        if (it.done) break;
        if (!even) claim_next();
        if (it.y0 >= it.y1) continue;
        int ids = key_blocks(it.seq, it.y0, it.keys), ids_next = key_blocks(it.seq, it.y0 + 4, it.keys);
        const int xs = nx & 1;
        if (nx >= 2 && !wait(&bars.x_empty[xs], ((nx - 2) >> 1) & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.x_full[xs], (uint32_t)(HF * tt * p.g * 128));
          for (int hf = 0; hf < HF; ++hf)
            tma_load_5d(base + xs * kTile + hf * kHalf, &tq, 0, 0, it.t0 + it.tile * tt, it.head, hf, &bars.x_full[xs]);
        }
        __syncwarp();
        ++nx;
        for (int j = it.y0; j < it.y1; ++j) {
          const int turn = (j - it.y0) & 3, s = n % ST;
          if (turn == 0 && j > it.y0) {
            ids = ids_next;
            ids_next = key_blocks(it.seq, j + 4, it.keys);
          }
          if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&bars.full[s], kTile);
          __syncwarp();
          copy_keys(ring(s), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * turn), it.head, &bars.full[s], 0, 4);
          armed = n++;
        }
        if (!ok) break;
      }
      if (!ok) {
        for (int m = max(0, armed - ST + 1); m <= armed; ++m) mbar_drain(&bars.full[m % ST], (m / ST) & 1);
        for (int m = max(0, nx - 2); m < nx; ++m) mbar_drain(&bars.x_full[m & 1], (m >> 1) & 1);
      }
    } else if (warp < kEmTma) {
      // ------------------------------- products of every other key tile
      const int x = warp - kEmMma;
      constexpr uint32_t idS = umma_idesc_bf16(128, 128, false, false);
      constexpr uint32_t kHi = ex_desc_hi(1024);
      const uint32_t x_lo = ex_desc_lo(smem_u32(base), 16), y_lo = ex_desc_lo(smem_u32(ring(0)), 16);
      int nx = 0, b = 0, s = 0;
      uint32_t full_par = 0, free_par = 1;
      for (int ni = 0;; ++ni) {
        const int slot = ni & 1;
        if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
        const int y0 = work[slot].y0, y1 = work[slot].y1, done = work[slot].done;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
        if (done) break;
        if (y0 >= y1) continue;
        const int xs = nx & 1;
        if (!wait(&bars.x_full[xs], (nx >> 1) & 1)) { ok = false; break; }
        ++nx;
        for (int j = y0; j < y1; ++j) {
          if (!wait(&bars.full[s], full_par)) { ok = false; break; }
          if (((j - y0) & 1) == x) {
            if (!wait(&bars.s_empty[x][b], free_par)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ya = y_lo + s * (kTile / 16), xa = x_lo + xs * (kTile / 16), d = tmem + 128u * (2 * x + b);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) / 16;
                ex_mma_ss(d, ya + o, xa + o, kHi, idS, kk > 0);
              }
              umma_commit(&bars.s_full[x][b]);
              umma_commit(&bars.empty[s]);
            }
            __syncwarp();
            if (b) free_par ^= 1u;
            b ^= 1;
          } else {
            if (lane == 0) mbar_arrive(&bars.empty[s]);
            __syncwarp();
          }
          if (++s == ST) {
            s = 0;
            full_par ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit(&bars.x_empty[xs]);
        __syncwarp();
      }
      // every product issued has completed before the tensor memory is released
      if (elect_one()) umma_commit(&bars.fin[x]);
      __syncwarp();
      mbar_wait_bounded(&bars.fin[x], 0, p.status);
    } else {
      // ------------------------- the rows' columns, the other half of the keys
      int n = 0, nx = 0;
      for (int ni = 0;; ++ni) {
        const int slot = ni & 1;
        if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
        const EkItem it = work[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
        if (it.done) break;
        if (it.y0 >= it.y1) continue;
        int ids = key_blocks(it.seq, it.y0, it.keys), ids_next = key_blocks(it.seq, it.y0 + 4, it.keys);
        const int per = tt * p.g, xs = nx & 1;
        const float* rows = p.nlse + ((size_t)it.head * p.n_tokens + it.t0) * p.g;
        float v[4];
        int lim[4], least = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = i * 32 + lane, row = it.tile * per + c;
          v[i] = c < per && row < it.rows * p.g ? rows[row] : -INFINITY;
          lim[i] = v[i] == -INFINITY ? 0 : p.causal ? max(it.keys - it.rows + row / p.g + 1, 0) : it.keys;
          least = min(least, lim[i]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        if (nx >= 2 && !wait(&bars.c_empty[xs], ((nx - 2) >> 1) & 1)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cols[xs].nlse[i * 32 + lane] = v[i];
          cols[xs].lim[i * 32 + lane] = lim[i];
        }
        if (lane == 0) cols[xs].least = least;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.c_full[xs]);
        ++nx;
        for (int j = it.y0; j < it.y1; ++j) {
          const int turn = (j - it.y0) & 3, s = n % ST;
          if (turn == 0 && j > it.y0) {
            ids = ids_next;
            ids_next = key_blocks(it.seq, j + 4, it.keys);
          }
          if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
          // counted by the barrier that the other warp arms, before or after this
          copy_keys(ring(s), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * turn), it.head, &bars.full[s], 4, 8);
          ++n;
        }
        if (!ok) break;
      }
      if (!ok) {   // copies in flight land before the shared memory goes away
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 24)) {
        }
      }
    }
    if (!ok) s_abort = 1;
  } else {
    // ------------------------------------------------------------ sums
    const int x = (warp >> 2) & 1, half = warp >> 3, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * x + 64u * half;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    int nx = 0, b = 0;
    uint32_t s_par = 0;
    bool ok = true;
    for (int ni = 0;; ++ni) {
      const int slot = ni & 1;
      if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
      const EkItem it = work[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
      if (it.done) break;
      if (it.y0 >= it.y1) continue;
      const int xs = nx & 1;
      if (!wait(&bars.c_full[xs], (nx >> 1) & 1)) { ok = false; break; }
      ++nx;
      const EmCols& cl = cols[xs];
      // columns behind the tile's last row hold nothing: whole halves are passed by
      const bool any = 64 * half < min(tt, it.rows - it.tile * tt) * p.g;
      float* out = p.sums + ((size_t)(2 * it.unit + half) * p.hkv + it.head) * p.most;
      for (int j = it.y0 + x; j < it.y1; j += 2) {
        if (!wait(&bars.s_full[x][b], s_par)) { ok = false; break; }
        tc_fence_after();
        uint32_t v[64];
        if (any) {
          tmem_ld32_issue(tS + 128u * b, v);
          tmem_ld32_issue(tS + 128u * b + 32, v + 32);
          tmem_ld32x2_wait(v, v + 32);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_empty[x][b]);
        if (b) s_par ^= 1u;
        b ^= 1;
        const int key = j * kEmTile + r;
        float l = 0.f;
        if (any) {
          if (j * kEmTile + (warp & 3) * 32 + 31 >= cl.least) {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const int4 u = *reinterpret_cast<const int4*>(cl.lim + 64 * half + i);
              if (key >= u.x) v[i] = 0xff800000u;
              if (key >= u.y) v[i + 1] = 0xff800000u;
              if (key >= u.z) v[i + 2] = 0xff800000u;
              if (key >= u.w) v[i + 3] = 0xff800000u;
            }
          }
          l = em_sum_up(v, sc2, [&](int i) { return *reinterpret_cast<const float2*>(cl.nlse + 64 * half + i); });
        }
        if (key < it.keys) out[key] = l;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.c_empty[xs]);
    }
    if (!ok) s_abort = 1;
  }
  asm volatile("griddepcontrol.launch_dependents;");   // not sooner: small CTAs would crowd where this grid's first ones end
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kEmCols);
  }
}

// --------------------------------------------------- short calls: one kernel
// A row tile of one KV head a CTA, for both passes: S = Q K^T over the key tiles, the
// row sums of two halves and of every other tile joined in shared memory, then S^T =
// K Q^T over the same key tiles again, whose key sums the last kernel adds up.
struct EwBars {
  uint64_t full[8], empty[8], x_full;
  uint64_t s_full[2][2], s_empty[2][2];
  uint64_t fin[2];
};

template <int D>
__global__ void __launch_bounds__(kEmThreads, 1)
em_whole_kernel(const __grid_constant__ EmParams p, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk) {
  constexpr int HF = D / 64, ST = em_stages<D>(), kTile = em_tile_bytes<D>(), kHalf = kEmTile * 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ EwBars bars;
  __shared__ EkItem work;
  __shared__ float2 states[4][kEmTile];
  __shared__ __align__(16) EmCols cl;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 2);      // both product warps
    }
    mbar_init(&bars.x_full, 1);
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[i][b], 1);
        mbar_init(&bars.s_empty[i][b], kEmSumWarps / 2);
      }
      mbar_init(&bars.fin[i], 1);
    }
    s_abort = 0;
    cl.least = 0x7fffffff;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, kEmCols);
    tmem_relinquish();
  }
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto ring = [&](int i) { return base + kTile * (2 + i); };
  tc_fence_before();
  const int tt = kEmTile / p.g;
  if (warp == 1) {
    // this CTA's row tile, a lane two sequences
    constexpr unsigned kAll = 0xffffffffu;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int a = 2 * lane;
    EmCount c0{}, c1{};
    if (a < p.n_seq) c0 = em_count(p, a);
    if (a + 1 < p.n_seq) c1 = em_count(p, a + 1);
    const bool bad = __any_sync(kAll, c0.bad | c1.bad);
    int end = c0.units2 + c1.units2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kAll, end, o);
      end += lane >= o ? x : 0;
    }
    const int begin = end - c0.units2 - c1.units2, middle = begin + c0.units2;   // units before these sequences, before the second
    const int units = __shfl_sync(kAll, end, 31), unit = (int)blockIdx.x / p.hkv;
    const int l = __popc(__ballot_sync(kAll, end <= unit)) & 31;
    const bool second = unit >= __shfl_sync(kAll, middle, l);
    auto of = [&](int x0, int x1) {   // of the unit's sequence
      x0 = __shfl_sync(kAll, x0, l);
      x1 = __shfl_sync(kAll, x1, l);
      return second ? x1 : x0;
    };
    EkItem it{};
    it.seq = 2 * l + second;
    it.head = (int)blockIdx.x - unit * p.hkv;
    it.unit = unit;
    it.tile = unit - of(begin, middle);
    it.t0 = of(c0.t0, c1.t0);
    it.rows = of(c0.rows, c1.rows);
    it.keys = of(c0.keys, c1.keys);
    it.y1 = bad || unit >= units ? 0 : ek_tiles(p, it.rows, it.keys, it.tile, tt);
    if (lane == 0) work = it;
    if (blockIdx.x == 0) {
      if (a < p.n_seq) {
        p.seq[a] = make_int4(c0.t0, c0.rows, c0.keys, 0);
        p.off2[a] = begin;
      }
      if (a + 1 < p.n_seq) {
        p.seq[a + 1] = make_int4(c1.t0, c1.rows, c1.keys, 0);
        p.off2[a + 1] = middle;
      }
      if (lane == 0) {
        if (bad) set_err(p.status, KVS_DEVERR_JOB);
        p.hdr[kMBad] = bad;
        p.hdr[kMCuts2] = 1;
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = s_tmem;
  const EkItem it = work;
  const int nt = it.y1;
  auto stop = [&]() { return __any_sync(0xffffffffu, s_abort != 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, p.status);
    return __all_sync(0xffffffffu, ok);
  };

  if (nt == 0) {
    // nothing to do
  } else if (warp >= kEmSumWarps) {
    bool ok = true;
    if (warp == kEmTma || warp == kEmTma + 1) {
      // ----------------------------- the rows, and half of every key tile each
      const bool first = warp == kEmTma;
      int armed = -1;
      if (first && lane == 0) {
        mbar_arrive_expect_tx(&bars.x_full, (uint32_t)(HF * tt * p.g * 128));
        for (int hf = 0; hf < HF; ++hf) tma_load_5d(base + hf * kHalf, &tq, 0, 0, it.t0 + it.tile * tt, it.head, hf, &bars.x_full);
      }
      __syncwarp();
      int ids = 0;
      for (int n = 0; n < 2 * nt; ++n) {
        const int j = n < nt ? n : n - nt, s = n % ST;
        if ((j & 3) == 0) ids = em_blocks(p, it.seq, j, it.keys, lane);
        if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) { ok = false; break; }
        if (first && lane == 0) mbar_arrive_expect_tx(&bars.full[s], kTile);
        __syncwarp();
        // (the barrier counts the copies of both warps, before or after it is armed)
        em_copy_keys<HF>(p, tk, ring(s), __shfl_sync(0xffffffffu, ids, (lane & 7) + 8 * (j & 3)), it.head, &bars.full[s], lane, first ? 0 : 4,
                         first ? 4 : 8);
        armed = n;
      }
      if (!ok) {   // copies in flight land before the shared memory goes away
        if (first) {
          for (int m = max(0, armed - ST + 1); m <= armed; ++m) mbar_drain(&bars.full[m % ST], (m / ST) & 1);
          mbar_drain(&bars.x_full, 0);
        } else {
          const long long t0 = clock64();
          while (clock64() - t0 < (1ll << 24)) {
          }
        }
      }
    } else {
      // ------------------------------- products of every other tile
      const int x = warp - kEmMma;
      constexpr uint32_t idS = umma_idesc_bf16(128, 128, false, false);
      constexpr uint32_t kHi = ex_desc_hi(1024);
      const uint32_t xa = ex_desc_lo(smem_u32(base), 16), y_lo = ex_desc_lo(smem_u32(ring(0)), 16);
      int b = 0, s = 0;
      uint32_t full_par = 0, free_par = 1;   // a fresh buffer counts as handed back
      ok = wait(&bars.x_full, 0);
      for (int n = 0; ok && n < 2 * nt; ++n) {
        if (stop() || !wait(&bars.full[s], full_par)) { ok = false; break; }
        if ((n & 1) == x) {
          if (!wait(&bars.s_empty[x][b], free_par)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ya = y_lo + s * (kTile / 16), d = tmem + 128u * (2 * x + b);
            const uint32_t ra = n < nt ? xa : ya, rb = n < nt ? ya : xa;   // rows and columns of the product
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) / 16;
              ex_mma_ss(d, ra + o, rb + o, kHi, idS, kk > 0);
            }
            umma_commit(&bars.s_full[x][b]);
            umma_commit(&bars.empty[s]);
          }
          __syncwarp();
          if (b) free_par ^= 1u;
          b ^= 1;
        } else {
          if (lane == 0) mbar_arrive(&bars.empty[s]);
          __syncwarp();
        }
        if (++s == ST) {
          s = 0;
          full_par ^= 1u;
        }
      }
      // every product issued has completed before the tensor memory is released
      if (elect_one()) umma_commit(&bars.fin[x]);
      __syncwarp();
      mbar_wait_bounded(&bars.fin[x], 0, p.status);
    }
    if (!ok) s_abort = 1;
  } else {
    // ------------------------------------------------------------ sums
    const int x = (warp >> 2) & 1, half = warp >> 3, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * x + 64u * half;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    int b = 0;
    uint32_t s_par = 0;
    uint32_t v[64];
    auto scores = [&](bool wanted) {
      if (stop() || !wait(&bars.s_full[x][b], s_par)) return false;
      tc_fence_after();
      if (wanted) {
        tmem_ld32_issue(tS + 128u * b, v);
        tmem_ld32_issue(tS + 128u * b + 32, v + 32);
        tmem_ld32x2_wait(v, v + 32);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_empty[x][b]);
      if (b) s_par ^= 1u;
      b ^= 1;
      return true;
    };
    const int tok = it.tile * tt + r / p.g;               // this row's token
    const bool live = r / p.g < tt && tok < it.rows;
    const int lim = !live ? 0 : p.causal ? min(it.keys - it.rows + tok + 1, it.keys) : it.keys;   // keys that it sees
    const bool any_live = __any_sync(0xffffffffu, live);
    bool ok = true;
    float m = 0.f, l = 0.f;
    for (int n = x; n < nt; n += 2) {
      if (!scores(any_live)) { ok = false; break; }
      if (!any_live) continue;
      const int key0 = n * kEmTile + 64 * half;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (key0 + i >= lim) v[i] = 0xff800000u;
      const bool fresh = n == x;
      float sum = fresh ? INFINITY : em_sum_up(v, sc2, [&](int) { return make_float2(-m, -m); });
      if (__any_sync(0xffffffffu, !(sum < 0x1p60f))) {   // as in em_pass_kernel
        float top = __uint_as_float(v[0]);
#pragma unroll
        for (int i = 1; i < 64; ++i) top = fmaxf(top, __uint_as_float(v[i]));
        top *= p.scale_log2;
        if (!(sum < 0x1p60f)) {
          if (!fresh) l *= fast_exp2(m - top);
          m = top == -INFINITY ? 0.f : top;
        }
        sum = em_sum_up(v, sc2, [&](int) { return make_float2(-m, -m); });
      }
      l += sum;
    }
    states[2 * x + half][r] = make_float2(m, l);
    asm volatile("bar.sync 1, %0;" ::"n"(kEmSumWarps * 32) : "memory");
    if (warp < 4) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (states[i][r].y > 0.f) top = fmaxf(top, states[i][r].x);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (states[i][r].y > 0.f) sum += states[i][r].y * fast_exp2(states[i][r].x - top);
      const bool seen = live && sum > 0.f;
      cl.nlse[r] = seen ? -(top + log2f(sum)) : -INFINITY;
      const int to = seen ? max(lim, 0) : 0, least = __reduce_min_sync(0xffffffffu, to);
      cl.lim[r] = to;
      if (lane == 0) atomicMin(&cl.least, least);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kEmSumWarps * 32) : "memory");
    // columns behind the tile's last row hold nothing: whole halves are passed by
    const bool any = 64 * half < min(tt, it.rows - it.tile * tt) * p.g;
    float* out = p.sums + ((size_t)(2 * it.unit + half) * p.hkv + it.head) * p.most;
    for (int n = nt + ((nt ^ x) & 1); ok && n < 2 * nt; n += 2) {
      if (!scores(any)) { ok = false; break; }
      const int key = (n - nt) * kEmTile + r;
      float sum = 0.f;
      if (any) {
        if ((n - nt) * kEmTile + (warp & 3) * 32 + 31 >= cl.least) {
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const int4 u = *reinterpret_cast<const int4*>(cl.lim + 64 * half + i);
            if (key >= u.x) v[i] = 0xff800000u;
            if (key >= u.y) v[i + 1] = 0xff800000u;
            if (key >= u.z) v[i + 2] = 0xff800000u;
            if (key >= u.w) v[i + 3] = 0xff800000u;
          }
        }
        sum = em_sum_up(v, sc2, [&](int i) { return *reinterpret_cast<const float2*>(cl.nlse + 64 * half + i); });
      }
      if (key < it.keys) out[key] = sum;
    }
    if (!ok) s_abort = 1;
  }
  asm volatile("griddepcontrol.launch_dependents;");
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kEmCols);
  }
}

// Joins the parts of every row: -log2 of its whole sum, -inf where it has none.
__global__ void __launch_bounds__(256) em_join_kernel(const __grid_constant__ EmParams p) {
  pdl_enter();
  const int bad = p.hdr[kMBad], n = 2 * p.hdr[kMCuts1], t0 = p.tok_off[0], t1 = p.tok_off[p.n_seq];
  const size_t rows = (size_t)p.n_tokens * p.hq;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i / p.hq), h = (int)(i - (size_t)t * p.hq);
  if (bad || i >= rows || t < t0 || t >= t1) return;   // rows of no sequence have no parts
  constexpr int U = 16;
  float m = -INFINITY, l = 0.f;
  for (int k0 = 0; k0 < n; k0 += U) {   // as many loads under way
    float2 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = k0 + k < n ? p.parts[(k0 + k) * rows + i] : make_float2(0.f, 0.f);
    float top = m;
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (v[k].y > 0.f) top = fmaxf(top, v[k].x);
    if (top > m) {
      l *= fast_exp2(m - top);
      m = top;
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (v[k].y > 0.f) l += v[k].y * fast_exp2(v[k].x - m);
  }
  p.nlse[((size_t)(h / p.g) * p.n_tokens + t) * p.g + h % p.g] = l > 0.f ? -(m + log2f(l)) : -INFINITY;
}

// Adds the cuts' and heads' sums in their order.
__global__ void __launch_bounds__(256) em_add_kernel(const __grid_constant__ EmParams p, const float* mass_in, float carry, float* mass) {
  pdl_enter();
  const int a = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
  const int bad = p.hdr[kMBad], cuts = p.hdr[kMCuts2], first = p.off2[a];
  const int4 s = p.seq[a];
  if (bad || t >= s.z) return;
  float sum = 0.f;
  const float* v = p.sums + (size_t)a * p.most + t;
  const size_t step = (size_t)p.n_seq * p.most;
  const size_t o = (size_t)a * p.most + t;
  const float before = mass_in ? mass_in[o] : 0.f;
  if (s.y > 0 && p.few) {
    // of every row tile that sees the key, and of its halves that hold rows
    const int tt = kEmTile / p.g;
    v = p.sums + (size_t)first * 2 * p.hkv * p.most + t;
    for (int i = 0; i * tt < s.y; ++i) {
      if (t / kEmTile >= ek_tiles(p, s.y, s.z, i, tt)) continue;
      const int n = (min(tt, s.y - i * tt) * p.g > 64 ? 2 : 1) * p.hkv;
      const float* w = v + (size_t)2 * i * p.hkv * p.most;
      if (n % 16 == 0) {   // as many loads under way as divide their number
#pragma unroll 16
        for (int k = 0; k < n; ++k) sum += w[(size_t)k * p.most];
      } else if (n % 4 == 0) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) sum += w[(size_t)k * p.most];
      } else {
#pragma unroll 2
        for (int k = 0; k < n; ++k) sum += w[(size_t)k * p.most];
      }
    }
  } else if (s.y > 0) {
    const int n = 2 * cuts * p.hkv;
#pragma unroll 16
    for (int i = 0; i < n; ++i) sum += v[i * step];
  }
  mass[o] = mass_in ? fmaf(carry, before, sum) : sum;
}

struct EmLayout {
  size_t hdr, seq, off1, off2, parts, nlse, sums, total;
  int cuts1, cuts2, few;
};
EmLayout em_layout(const kvs_pool* pool, int n_tokens, int n_seq, int max_blocks, int hq) {
  const kvs_pool_desc& d = pool->desc;
  const int hkv = d.num_kv_heads, g = hq / hkv, tt = kEmTile / g;
  EmLayout l{};
  // room for cuts: as many as bring four items to every SM where the units are
  // few; the plan, which knows the lengths, takes no more
  const long long sms4 = 4ll * pool->num_sms, key_tiles = ((long long)max_blocks * 16 + kEmTile - 1) / kEmTile;
  const long long u1 = ((long long)n_tokens / (2 * tt) + 1) * hkv, u2 = ((key_tiles + 1) / 2) * hkv;   // of one sequence
  const long long row_tiles = ((long long)n_tokens + tt - 1) / tt;
  auto cuts = [&](long long units, long long tiles) {
    return (int)std::clamp<long long>((sms4 + units - 1) / std::max(1ll, units), 1, std::clamp<long long>(tiles, 1, kEmMaxCuts));
  };
  l.cuts1 = cuts(u1, key_tiles);
  // On the mean at most one row tile a sequence: the keys stream past them
  // (em_keys_kernel; 8 x 32 rows after 6,000 tokens, 32 / 8 heads: 60 us, else 75;
  // 64 x 4 after 8,000, 40 / 8: 375 and 573).  With more, each would read the keys
  // again (1 x 128 rows after 6,000, 32 / 8: 48 and 42; 1 x 512 after 4,096, 16 / 2:
  // 77 and 42).
  l.few = row_tiles <= n_seq;
  l.cuts2 = l.few ? cuts(hkv, key_tiles) : cuts(u2, row_tiles);
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t{255};
    return at;
  };
  l.hdr = take(kMTotal * 4);
  l.seq = take((size_t)n_seq * 16);
  l.off1 = take((size_t)(n_seq + 1) * 4);
  l.off2 = take((size_t)(n_seq + 1) * 4);
  // Fewer rows or keys may take more cuts, so the two buffers of cuts are given
  // what any smaller call takes: cuts <= sms4 / units + 1, units > n_tokens / (2 tt)
  // hkv and units >= max_blocks * 16 / 256 hkv.
  const long long most = (long long)max_blocks * 16;
  const long long rows1 = std::min(std::clamp<long long>(key_tiles, 1, kEmMaxCuts) * n_tokens, 2 * tt * (sms4 / hkv + 1) + n_tokens);
  const long long keys2 = std::min(std::clamp<long long>(row_tiles, 1, kEmMaxCuts) * most, 256 * (sms4 / hkv + 1) + most);
  l.parts = take((size_t)2 * rows1 * hq * 8);
  l.nlse = take((size_t)n_tokens * hq * 4);
  // sums by row tile: few rows, and short calls of some more (em_whole)
  const long long by_rows = (std::min<long long>(row_tiles, n_seq) + n_seq) * most;
  const long long by_rows_whole = (std::min<long long>(row_tiles, 2ll * n_seq + 6) + n_seq) * std::min<long long>(most, 8 * kEmTile);
  l.sums = take((size_t)2 * std::max({n_seq * keys2, by_rows, by_rows_whole}) * hkv * 4);
  l.total = o;
  return l;
}

template <typename... KArgs, typename... Args>
cudaError_t em_launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D>
kvs_status em_run(const kvs_pool* pool, int layer, const EmParams& p, const CUtensorMap& tq, const float* mass_in, float carry,
                  float* mass, cudaStream_t stream) {
  if (!smem_limit_once<em_pass_kernel<D, 1>>(em_smem<D>(), pool->device) ||
      !smem_limit_once<em_pass_kernel<D, 2>>(em_smem<D>(), pool->device) ||
      !smem_limit_once<em_keys_kernel<D>>(em_smem<D>(), pool->device) ||
      !smem_limit_once<em_whole_kernel<D>>(em_smem<D>(), pool->device))
    return fail(KVS_ERR_CUDA, "extend_mass: cannot raise the shared-memory limit");
  const CUtensorMap& tk = D == 128 ? pool->tk1[layer] : pool->tk[layer];
  const dim3 grid((unsigned)pool->num_sms);
  bool ok = true;
  if (p.whole)
    ok = em_launch(em_whole_kernel<D>, dim3((unsigned)p.whole), dim3(kEmThreads), em_smem<D>(), stream, p, tq, tk) == cudaSuccess;
  else if (p.n_tokens > 0)
    ok = em_launch(em_pass_kernel<D, 1>, grid, dim3(kEmThreads), em_smem<D>(), stream, p, tq, tk) == cudaSuccess &&
         em_launch(em_join_kernel, dim3((unsigned)(((long long)p.n_tokens * p.hq + 255) / 256)), dim3(256), 0, stream, p) == cudaSuccess &&
         em_launch(p.few ? em_keys_kernel<D> : em_pass_kernel<D, 2>, grid, dim3(kEmThreads), em_smem<D>(), stream, p, tq, tk) == cudaSuccess;
  if (ok && p.n_tokens > 0) count_launch(p.whole ? 1 : 3);
  if (ok && em_launch(em_add_kernel, dim3((unsigned)((p.most + 255) / 256), (unsigned)p.n_seq), dim3(256), 0, stream, p, mass_in, carry,
                      mass) == cudaSuccess)
    count_launch();
  return check_launch("extend_mass");
}

}  // namespace

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_extend_mass_workspace_size(const kvs_pool* pool, int32_t n_tokens, int32_t n_seq, int32_t max_blocks,
                                                     int32_t n_q_heads, size_t* bytes) {
  if (!bytes) return fail(KVS_ERR_INVALID_ARG, "extend_mass_workspace_size: null pointer");
  if (kvs_status st = ex_check(pool, "extend_mass_workspace_size", n_tokens, n_seq, max_blocks, n_q_heads); st != KVS_OK) return st;
  *bytes = em_layout(pool, n_tokens, n_seq, max_blocks, n_q_heads).total;
  return KVS_OK;
}

extern "C" kvs_status kvs_extend_mass(kvs_pool* pool, int32_t layer, const void* q_dev, int64_t q_stride, const int32_t* tok_off_dev,
                                      int32_t n_tokens, int32_t n_q_heads, const int32_t* block_table_dev, int32_t max_blocks,
                                      const int32_t* seq_len_dev, int32_t n_seq, int32_t causal, float scale,
                                      const float* mass_in_dev, float carry, float* mass_dev, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  if (kvs_status st = ex_check(pool, "extend_mass", n_tokens, n_seq, max_blocks, n_q_heads); st != KVS_OK) return st;
  const kvs_pool_desc& d = pool->desc;
  if (layer < 0 || layer >= d.num_layers) return fail(KVS_ERR_INVALID_ARG, "extend_mass: layer out of range");
  if (causal != 0 && causal != 1) return fail(KVS_ERR_INVALID_ARG, "extend_mass: causal is 0 or 1");
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.f) || !std::isfinite(scale_log2))
    return fail(KVS_ERR_INVALID_ARG, "extend_mass: scale must be positive, and scale * log2(e) finite");
  if (!std::isfinite(carry)) return fail(KVS_ERR_INVALID_ARG, "extend_mass: carry must be finite");
  const long long row = (long long)n_q_heads * d.head_dim;
  if (q_stride < row || (q_stride & 7)) return fail(KVS_ERR_INVALID_ARG, "extend_mass: q_stride must hold n_q_heads * head_dim elements and be a multiple of 8");
  if (n_seq > 65535) return fail(KVS_ERR_UNSUPPORTED, "extend_mass: more than 65,535 sequences");
  if (n_seq == 0) return KVS_OK;
  if ((n_tokens > 0 && !q_dev) || !tok_off_dev || !block_table_dev || !seq_len_dev || !mass_dev || !ws)
    return fail(KVS_ERR_INVALID_ARG, "extend_mass: null pointer");
  if (!aligned16(q_dev) || !aligned16(ws)) return fail(KVS_ERR_INVALID_ARG, "extend_mass: q and ws must be 16-byte aligned");
  const EmLayout l = em_layout(pool, n_tokens, n_seq, max_blocks, n_q_heads);
  if (ws_bytes < l.total) return fail(KVS_ERR_CAPACITY, "extend_mass: workspace too small");
  if (kvs_status st = check_pool_device(pool, "extend_mass"); st != KVS_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  EmParams p{};
  p.table = block_table_dev;
  p.tok_off = tok_off_dev;
  p.seq_len = seq_len_dev;
  p.status = pool->status;
  p.hdr = reinterpret_cast<int*>(w + l.hdr);
  p.seq = reinterpret_cast<int4*>(w + l.seq);
  p.off1 = reinterpret_cast<int*>(w + l.off1);
  p.off2 = reinterpret_cast<int*>(w + l.off2);
  p.parts = reinterpret_cast<float2*>(w + l.parts);
  p.nlse = reinterpret_cast<float*>(w + l.nlse);
  p.sums = reinterpret_cast<float*>(w + l.sums);
  p.n_tokens = n_tokens;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.capacity = d.capacity_blocks;
  p.hkv = d.num_kv_heads;
  p.g = n_q_heads / d.num_kv_heads;
  p.hq = n_q_heads;
  p.causal = causal;
  p.slab_rows = d.capacity_blocks * d.num_kv_heads * d.block_tokens;
  p.most = max_blocks * 16;
  p.cuts1 = l.cuts1;
  p.cuts2 = l.cuts2;
  p.sms = pool->num_sms;
  p.few = l.few;
  p.scale_log2 = scale_log2;
  CUtensorMap tq{};
  if (n_tokens > 0 && !ex_query_map(&tq, q_dev, n_tokens, p.g, p.hkv, d.head_dim, q_stride))
    return fail(KVS_ERR_CUDA, "extend_mass: cuTensorMapEncodeTiled failed for q");
  // a warp of pass 1 counts up to 32 sequences for itself (1 row after 1,000 tokens
  // 19.0 us with a plan, 17.1 without; 16 x 4 after 1,000, 40 / 8 heads: 31.9, 27.3)
  // One kernel for both passes where keys are few, or rows and heads enough for as many
  // CTAs as make up for them (us, whole and in two passes: 16 x 4 rows after 1,000
  // tokens, 40 / 8 heads, 17.2 and 28.1; 4 x 16 after 500, 16 / 2, 12.3 and 17.9; 16 x 4
  // after 4,000, 40 / 8, 52.8 and 62.9; but 4 x 16 after 2,000, 32 / 8 of 64 channels,
  // 25.2 and 21.9; after 4,000 of 128 channels 45 and 28).
  // Over tables of eight key tiles also where sequences have a few row tiles (1 x 64
  // rows after 300, 8 / 2: 10.1 and 17.3; 8 x 64 after 300, 32 / 8: 12.5 and 21.1; 1 x 256
  // after 200: 18.9 and 21.7; but after 700: 24.1 and 22.2).
  const int tt = kEmTile / p.g;
  const long long ctas = ((long long)n_tokens / tt + n_seq) * p.hkv, tiles = (p.most + kEmTile - 1) / kEmTile;
  if (n_tokens > 0 && n_seq <= 64 && ctas <= 4ll * p.sms &&
      (tiles <= 8 ? p.few || ((long long)n_tokens + tt - 1) / tt <= 2ll * n_seq + (tiles <= 4 ? 6 : 2) : p.few && tiles <= 32 && ctas >= 4 * tiles)) {
    p.few = 1;
    p.whole = (int)ctas;
  } else if (n_seq <= 32 && n_tokens > 0) {
    p.tickets = pool->tickets;
  } else {
    if (launch_pdl(em_plan_kernel, dim3(1), dim3(1024), stream, p) != cudaSuccess) return check_launch("extend_mass");
    count_launch();
  }
  return d.head_dim == 128 ? em_run<128>(pool, layer, p, tq, mass_in_dev, carry, mass_dev, stream)
                           : em_run<64>(pool, layer, p, tq, mass_in_dev, carry, mass_dev, stream);
}
