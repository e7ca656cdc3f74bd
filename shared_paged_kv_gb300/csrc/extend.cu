// Attention of query chunks over the paged pool (prompt chunks, drafted
// tokens, cross attention) on the fifth-generation tensor cores.
//
//   out_r = sum_p e^(x_rp) V_p / sum_p e^(x_rp),  x_rp = scale <q_r, K_p>,  p < lim_r
//
// in one pass over the keys: with a reference point m (a running maximum that
// moves only when it is exceeded by more than 2^8), l = sum_p 2^(s_p - m) and
// O = sum_p 2^(s_p - m) V_p in fp32, s = x log2 e; moving m rescales l and O.
//
// GB300 layout of the work:
//  * Rows are (token, query head of a KV head): 128 / G whole tokens make the
//    M = 128 rows of a tile.  A CTA holds two tiles, A and B, of consecutive
//    tokens, and streams the keys in tiles of 128 through both: each K / V tile
//    that TMA brings (block by block through the block table, 128-byte
//    swizzle) feeds six 128 x 128 x head_dim products.
//  * S = Q K^T lands in tensor memory; two warpgroups (one per tile, one row
//    per thread, so the softmax needs no shuffles) turn it into P = 2^(s - m)
//    in the same columns, and O += P V takes P from tensor memory.
//    While one tile's softmax runs, the tensor cores work for the other tile.
//  * P is held as two bf16 parts, as decode attention holds it: the upper 16 bits
//    of the float32 weight and the remainder, rounded (2^-15 of a weight is
//    lost), so that O += P V is two products; the parts fill the columns that S
//    took.  With one rounded part the result was 2.0e-3 to 2.3e-3 (relative L2)
//    from 64 bits, beyond the 2e-3 that every attention here keeps; with two it
//    is the 1.7e-3 of the bf16 output.  It costs a third of the rate of long
//    chunks (8,192 rows after 8,192 tokens, 32 heads: 1,160 us with one part),
//    a sixth in calls of few rows.  l sums the whole weights; O, m, l are fp32.
//  * Warp 8 issues the MMAs, warp 9 the TMA copies and the work claims.
//
// The plan lists the work as items (row tile pair, block table, key range).
// Long key ranges are split into pieces so that the items fill the SMs evenly;
// runs of sequences whose tables begin with the same blocks put their rows,
// which lie side by side in the packed batch, into common tiles over the
// common part ("shared" items) and go on alone behind it.  Rows with more than
// one part leave (m, l, O) in fp32, and a merge kernel joins them in a fixed
// order.  CTAs claim items (longest first) from a counter in the plan.  Calls with
// nothing to split or share go without a plan, in one launch (ex_direct).
//
// What bounds it: in long chunks the products, and the chain S, softmax, P V of a
// row tile.  The six products of a tile pair take 3,072 cycles of the tensor
// cores (2,048 of them P V's two parts), and two chains share the SM: a pair
// takes about 4,600, the tensor pipe is busy 76 % of the time on the busiest SM.
// Times of CUDA-graph replays / of public calls one by one: 8,192 rows after
// 8,192 tokens, 32 heads of 128: 1.55 to 1.59 / 1.61 ms, 1,040 to 1,065 / 1,026
// TFLOP/s of the formula's operations; 16 chunks over one document of 8,192
// states: 450 / 471 us.  Few rows over long contexts are bound by the items'
// chains, starts and ends (64 sequences of 3 to 8 rows over 8,192 shared and
// 1,000 to 6,100 own tokens: 260 / 264 us, 3.8 TB/s), calls without a plan by one
// chain of key tiles (12 rows over 1,300 states: 25 / 26 us).
#include <algorithm>
#include <cmath>

#include <cudaTypedefs.h>

#include "tcgen05.cuh"
#include "internal.h"

namespace kvs {

namespace {

// Two softmax warpgroups; MMA warp, TMA warp and two idle ones that complete
// their warpgroup.  384 threads start with 168 registers each (64,512 in all);
// the softmax threads, which hold a row's 128 scores, take 216 (with 208 they
// spill) and the others 72: 256 * 216 + 128 * 72 = 64,512.
constexpr int kExThreads = 384;
constexpr int kExRegsSoftmax = 216, kExRegsOther = 72;
constexpr int kExTile = 128;             // keys of a tile, rows of a row tile
constexpr int kExBlocks = kExTile / 16;  // pool blocks of a key tile
constexpr int kExMagic = 0x45585431;
// above this many (token, query head) rows a call fills the device without
// splits or shared parts (2,048 row-tile pairs and more), and none are made:
// the workspace's part buffers stay below about a gigabyte
constexpr long long kExPartRows = 1ll << 19;
constexpr int kExMergeRows = 2;          // rows a warp of the merge joins at a time
constexpr int kExItemsPerSm = 4;         // pieces aimed at per SM
// Writing 256 rows of a part (133 KB) and reading them again, in key tiles of
// a row tile pair at a 152nd of the L2's rate
constexpr float kExPartCost = 5.f;
constexpr int kExMinPiece = 2;           // key tiles of the shortest piece
// Calls that run without a plan: up to this many blocks a sequence, and rounds
// of units over the SMs (see ex_direct).
constexpr int kExDirectBlocks = 96, kExDirectShort = 256;
constexpr int kExDirectRounds = 4;

template <int D>
__host__ __device__ constexpr int ex_tile_bytes() { return kExTile * D * 2; }
template <int D>
__host__ __device__ constexpr int ex_stages() { return D == 128 ? 5 : 8; }
template <int D>
__host__ __device__ constexpr int ex_smem() { return 1024 + ex_tile_bytes<D>() * (2 + ex_stages<D>()); }
constexpr uint32_t kExCols = 512;        // S/P of A and B at 0 and 128, O at 256 and 256 + D

// Plan header (int indices)
enum { kHMagic, kHSeq, kHBlocks, kHGroup, kHKv, kHCausal, kHTokens, kHItems, kHCounter, kHUnits, kHParts, kHTotal = 16 };

// One item: a row-tile pair over a range of key tiles of one block table.
struct __align__(16) ExItem {
  int t0, n_tok;      // packed rows t0 .. t0 + n_tok
  int seq;            // row of the block table
  int kv0, kv1;       // key tiles
  int lim0, step;     // keys visible to token k of the item: min(lim0 + step * k, kv_end)
  int kv_end;         // keys of the sequence (or of the shared part)
  int part;           // first part row, -1: the output itself
  int pad[3];
};
static_assert(sizeof(ExItem) == 48, "three 16-byte loads");

// One row-tile pair of the plan, as the merge reads it.
struct __align__(16) ExUnit {
  int t0, n_tok;
  int part, pieces;   // first part row and pieces of its own range (part -1: written directly)
  int sh_t0, sh_unit; // shared range: first token of the run, its first unit (-1: none)
  int pad[2];
};
static_assert(sizeof(ExUnit) == 32, "two 16-byte loads");

struct ExWorkspace {
  int* hdr;
  int4* seq;        // [n_seq] {first row, rows, keys, shareable tiles}
  int* lcp;         // [n_seq] common leading key tiles with the next sequence
  int4* run;        // [n_seq] by run index: {shared tiles, first sequence, sequences, rows}
  int2* seg;        // [n_seq] by sequence: {run, first unit}
  int2* runseg;     // [n_seq] by run: {first shared unit, shared units}
  ExItem* items;
  ExUnit* units;
  float* part;      // [rows][hkv][D]
  float2* ml;       // [rows][hkv]
  int max_items, max_units;
  long long part_rows;
  size_t bytes;
};

int ex_tokens_per_unit(int g) { return 2 * (kExTile / g); }

ExWorkspace ex_layout(const kvs_pool* pool, int n_tokens, int n_seq, int max_blocks, int g, void* base) {
  const int hkv = pool->desc.num_kv_heads, D = pool->desc.head_dim;
  const int tu = ex_tokens_per_unit(g);
  ExWorkspace w{};
  const long long own = n_tokens / tu + n_seq;
  w.max_units = (int)(2 * own);
  // sum of pieces <= (all key tiles of all units) / piece + units, and the
  // piece is at least the total over kExItemsPerSm * SMs / heads (calls with
  // many units: over 2 * SMs / heads, so that at most 2 * SMs / heads units are cut)
  const long long extra = (long long)kExItemsPerSm * pool->num_sms / hkv + 1;
  w.max_items = (int)(w.max_units + extra);
  // Rows of a unit x its pieces: every row of its own and of a shared range
  // once, and 2 * 128 rows for each piece beyond the first.  One sequence shares
  // nothing; at most 4 * SMs / heads units of it are split (the plan's rules).
  // Calls above kExPartRows make no parts; they keep the room of those below, so
  // that a workspace serves every call of no more tokens, sequences and blocks.
  const long long with_parts = std::min<long long>(n_tokens, kExPartRows / ((long long)g * hkv));
  const long long few = (long long)((4 * pool->num_sms - 1) / hkv) * tu;
  w.part_rows = (n_seq > 1 ? 2 * with_parts : std::min(with_parts, few)) * g + extra * 2 * kExTile;
  const long long tiles = ((long long)max_blocks + kExBlocks - 1) / kExBlocks + 1;
  w.part_rows = std::min(w.part_rows, with_parts * g * (tiles + 1));   // at most a piece per key tile
  char* p = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t{255};
    return p + at;
  };
  w.hdr = reinterpret_cast<int*>(take(kHTotal * 4));
  w.seq = reinterpret_cast<int4*>(take((size_t)n_seq * 16));
  w.lcp = reinterpret_cast<int*>(take((size_t)n_seq * 4));
  w.run = reinterpret_cast<int4*>(take((size_t)n_seq * 16));
  w.seg = reinterpret_cast<int2*>(take((size_t)n_seq * 8));
  w.runseg = reinterpret_cast<int2*>(take((size_t)n_seq * 8));
  w.items = reinterpret_cast<ExItem*>(take((size_t)w.max_items * sizeof(ExItem)));
  w.units = reinterpret_cast<ExUnit*>(take((size_t)w.max_units * sizeof(ExUnit)));
  w.part = reinterpret_cast<float*>(take((size_t)w.part_rows * hkv * D * 4));
  w.ml = reinterpret_cast<float2*>(take((size_t)w.part_rows * hkv * 8));
  w.bytes = o;
  return w;
}

// ------------------------------------------------------------------- plan ---
struct ExPlanParams {
  ExWorkspace w;
  const int32_t *tok_off, *seq_len, *table;
  uint32_t* status;
  int n_tokens, n_seq, max_blocks, capacity, g, hkv, causal, sms;
  int share;      // 1: look for common parts, 0: one sequence, -1: neither shared parts nor splits
  int lcp_here;   // the plan kernel finds the common parts itself
};

// {first row, rows (-1: bad offsets), keys, key tiles that every row of the
// sequence sees whole}
__device__ __forceinline__ int4 ex_seq(const ExPlanParams& p, int a, bool report) {
  const int t0 = __ldg(p.tok_off + a), t1 = __ldg(p.tok_off + a + 1);
  if (t0 < 0 || t1 < t0 || t1 > p.n_tokens) return make_int4(0, -1, 0, 0);
  const long long most = (long long)p.max_blocks * 16;
  long long n = __ldg(p.seq_len + a);
  if (n < 0 || n > most) {
    if (report) set_err(p.status, KVS_DEVERR_SEQ_LEN);
    n = n < 0 ? 0 : most;
  }
  const int rows = t1 - t0;
  const long long seen = p.causal ? max(n - rows + 1, 0ll) : n;
  return make_int4(t0, rows, (int)n, rows > 0 ? (int)(min(seen, n) / kExTile) : 0);
}

// Leading key tiles that sequence a's table has in common with the next
// one's (blocks of valid ids, equal one by one), among those every row sees.
__global__ void __launch_bounds__(256) extend_lcp_kernel(const __grid_constant__ ExPlanParams p) {
  pdl_enter();
  const int a = blockIdx.x;
  const int tiles = min(ex_seq(p, a, false).w, ex_seq(p, a + 1, false).w);
  const int n = tiles * kExBlocks;
  const int32_t* x = p.table + (size_t)a * p.max_blocks;
  const int32_t* y = x + p.max_blocks;
  __shared__ int first;
  if (threadIdx.x == 0) first = n;
  __syncthreads();
  constexpr int U = 8;   // loads in flight per thread and row
  for (int b0 = 0; b0 < n; b0 += 256 * U) {
    int xv[U], yv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * 256 + threadIdx.x;
      xv[u] = b < n ? __ldg(x + b) : 0;
      yv[u] = b < n ? __ldg(y + b) : 0;
    }
    int bad = n;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * 256 + threadIdx.x;
      if (b < n && (xv[u] != yv[u] || xv[u] < 0 || xv[u] >= p.capacity)) bad = min(bad, b);
    }
    if (bad < n) atomicMin(&first, bad);
    __syncthreads();
    if (first < n) break;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.w.lcp[a] = first / kExBlocks;
}

constexpr int kPlanThreads = 256;
constexpr int kPlanSeqs = 512;     // up to this many sequences the plan's arrays stay in shared memory
constexpr int kPlanUnits = 640;    // more units than calls that are split have (4 per SM)
constexpr int kPlanCands = 16;     // piece lengths that are tried
constexpr long long kPlanTable = 8192;   // table entries up to which the plan kernel compares neighbours itself

// Exclusive scan over the CTA plus a running total, one barrier per call:
// calls alternate between two rows of warp sums.
struct ExScan {
  int (*sums)[kPlanThreads / 32];
  int carry = 0, turn = 0;
  __device__ __forceinline__ int operator()(int x) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sums[turn][warp] = incl;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const int v = sums[turn][w];
      before += w < warp ? v : 0;
      carry += v;
    }
    turn ^= 1;
    return before + incl - x;
  }
};

// Key tiles of unit i of a sequence's own range, behind `skip` shared tiles.
__device__ __forceinline__ int ex_own_tiles(const int4& s, int i, int tu, int causal, int skip) {
  const int last = min(s.y, (i + 1) * tu) - 1;    // the unit's last row sees most
  const int lim = causal ? min(max(s.z - s.y + last + 1, 0), s.z) : s.z;
  return max(0, (lim + kExTile - 1) / kExTile - skip);
}

__device__ __forceinline__ int ex_pieces(int tiles, int piece) { return max(1, (tiles + piece - 1) / piece); }

// Candidate i of kPlanCands for the piece length: the longest unit in 1.41^i
// pieces (1 to 181).
__device__ __forceinline__ int ex_candidate(int most, int least, int i) {
  return max(least, (int)ceilf((float)most * exp2f(-0.5f * (float)i)));
}

// One CTA: runs of sequences, units, piece length, items sorted by cost.  A
// chain of short dependent steps bounds it: 4.4 us for one sequence, 8 to 9 us
// with the search for common parts of 32 or 64 long tables (1,024 threads and a
// piece per loop step: 7 and 12 us).
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const __grid_constant__ ExPlanParams p) {
  __shared__ int sums[2][kPlanThreads / 32];
  __shared__ int hist[256];
  __shared__ float cost[kPlanCands];
  __shared__ int s_parts, s_most;
  __shared__ unsigned long long s_sum;
  __shared__ int tiles_of[kPlanUnits];
  __shared__ float part_of[kPlanUnits];   // what a part of the unit costs, in key tiles
  __shared__ int2 src_of[kPlanUnits];   // {sequence, or ~run, index in it}
  __shared__ int4 sm_seq[kPlanSeqs], sm_run[kPlanSeqs];
  __shared__ int2 sm_seg[kPlanSeqs], sm_runseg[kPlanSeqs];
  __shared__ int sm_lcp[kPlanSeqs];
  const bool small = p.n_seq <= kPlanSeqs;
  int4* const seq = small ? sm_seq : p.w.seq;          // {first row, rows, keys, shareable tiles}
  int4* const run = small ? sm_run : p.w.run;          // {shared tiles, first sequence, sequences, rows}
  int2* const seg = small ? sm_seg : p.w.seg;          // {run, first unit} of a sequence
  int2* const runseg = small ? sm_runseg : p.w.runseg; // {first shared unit, shared units} of a run
  int* const lcp = small ? sm_lcp : p.w.lcp;           // key tiles in common with the next sequence
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tu = 2 * (kExTile / p.g), tt = kExTile / p.g;
  int* hdr = p.w.hdr;
  hist[tid] = 0;
  if (tid == 0) {
    s_parts = 0;
    s_sum = 0;
    s_most = 1;
  }
  pdl_enter();
  int bad = 0;
  for (int a = tid; a < p.n_seq; a += kPlanThreads) {
    if (small && p.share > 0 && !p.lcp_here) sm_lcp[a] = a + 1 < p.n_seq ? p.w.lcp[a] : 0;
    const int4 s = ex_seq(p, a, true);
    bad |= s.y < 0;
    seq[a] = s;
  }
  // offsets that do not ascend within [0, n_tokens] give an empty plan: rows
  // of sequences are disjoint and side by side in everything below
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      set_err(p.status, KVS_DEVERR_JOB);
      hdr[kHMagic] = 0;
      hdr[kHItems] = hdr[kHUnits] = hdr[kHCounter] = 0;
    }
    return;
  }
  if (p.lcp_here) {   // short tables: a warp per pair of neighbours
    for (int a = warp; a + 1 < p.n_seq; a += kPlanThreads / 32) {
      const int n = min(seq[a].w, seq[a + 1].w) * kExBlocks;
      const int32_t* x = p.table + (size_t)a * p.max_blocks;
      const int32_t* y = x + p.max_blocks;
      int first = n;
      constexpr int U = 4;   // loads in flight per lane and row
      for (int b0 = 0; b0 < first; b0 += 32 * U) {
        int xv[U], yv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int b = b0 + u * 32 + lane;
          xv[u] = b < n ? __ldg(x + b) : 0;
          yv[u] = b < n ? __ldg(y + b) : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int b = b0 + u * 32 + lane;
          if (b < n && (xv[u] != yv[u] || xv[u] < 0 || xv[u] >= p.capacity)) first = min(first, b);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      }
      if (lane == 0) lcp[a] = first / kExBlocks;
    }
    __syncthreads();
  }
  // runs: a sequence starts a new one unless its common part with the one
  // before it is at least half of the neighbouring common parts (so that a
  // short common part does not cut down two families of long ones); in the
  // same pass every sequence's own units
  auto link = [&](int a) {   // between a and a + 1
    if (p.share <= 0 || a < 0 || a + 1 >= p.n_seq) return 0;
    return min(lcp[a], min(seq[a].w, seq[a + 1].w));
  };
  ExScan runs{sums}, units{sums};
  for (int a0 = 0; a0 < p.n_seq; a0 += kPlanThreads) {
    const int a = a0 + tid;
    int head = 0, n = 0;
    if (a < p.n_seq) {
      const int l = link(a - 1);
      head = a == 0 || l == 0 || 2 * l < max(link(a - 2), link(a));
      n = (seq[a].y + tu - 1) / tu;
    }
    const int r = runs(head) + head - 1;
    units.turn = runs.turn;
    const int at = units(n);
    runs.turn = units.turn;
    if (a < p.n_seq) {
      seg[a] = make_int2(r, at);
      if (head) run[r] = make_int4(0, a, 0, 0);
    }
  }
  const int n_runs = runs.carry, own_units = units.carry;
  int n_units = own_units;
  __syncthreads();
  if (p.share > 0) {
    // a run shares when its rows fill at most three quarters of the row tiles
    // that its sequences would fill one by one; its units follow the others.
    // A warp takes a run; runs of one sequence share nothing.
    for (int r = warp; r < n_runs; r += kPlanThreads / 32) {
      const int first = run[r].y, count = (r + 1 < n_runs ? run[r + 1].y : p.n_seq) - first;
      int sh = 0, rows = seq[first].y;
      if (count > 1) {
        int sep = 0;
        sh = 0x7fffffff;
        rows = 0;
        for (int a = first + lane; a < first + count; a += 32) {
          rows += seq[a].y;
          sep += (seq[a].y + tt - 1) / tt;
          if (a > first) sh = min(sh, link(a - 1));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          rows += __shfl_xor_sync(0xffffffffu, rows, o);
          sep += __shfl_xor_sync(0xffffffffu, sep, o);
          sh = min(sh, __shfl_xor_sync(0xffffffffu, sh, o));
        }
        if (4 * ((rows + tt - 1) / tt) > 3 * sep) sh = 0;
      }
      __syncwarp();
      if (lane == 0) {
        run[r].x = sh;
        run[r].z = count;
        run[r].w = rows;
      }
    }
    __syncthreads();
    for (int r0 = 0; r0 < n_runs; r0 += kPlanThreads) {
      const int r = r0 + tid;
      const int n = r < n_runs && run[r].x > 0 ? (run[r].w + tu - 1) / tu : 0;
      const int at = units(n);
      if (r < n_runs) runseg[r] = make_int2(at, n);
    }
    n_units = units.carry;
  } else {
    for (int r = tid; r < n_runs; r += kPlanThreads) runseg[r] = make_int2(0, 0);   // one sequence each
  }
  __syncthreads();
  // visits every unit: f(unit, tiles, {sequence or ~run, index}, shared tiles
  // in front of it); units of a sequence or run go over a warp's lanes
  const bool split = p.share >= 0 && (long long)n_units * p.hkv < 4ll * p.sms && n_units <= kPlanUnits;
  auto walk = [&](auto f) {
    for (int a = warp; a < p.n_seq; a += kPlanThreads / 32) {
      const int4 s = seq[a];
      const int2 sg = seg[a];
      const int skip = run[sg.x].x, n = (s.y + tu - 1) / tu;
      for (int i = lane; i < n; i += 32) f(sg.y + i, ex_own_tiles(s, i, tu, p.causal, skip), make_int2(a, i), skip);
    }
    for (int r = warp; r < n_runs; r += kPlanThreads / 32) {
      const int2 rs = runseg[r];
      const int sh = run[r].x;
      for (int i = lane; i < rs.y; i += 32) f(rs.x + i, sh, make_int2(~r, i), 0);
    }
  };
  // whether a unit fills more than one row tile
  auto two_tiles = [&](int2 src) { return (src.x >= 0 ? seq[src.x].y : run[~src.x].w) - src.y * tu > tt; };
  {
    int most = 1;
    unsigned long long sum = 0;
    if (split) {   // few units: a thread each, its sequence or run found by bisection
      for (int u = tid; u < n_units; u += kPlanThreads) {
        const bool own = u < own_units;
        const int2* first = own ? seg : runseg;   // .y of a sequence, .x of a run: its first unit
        int lo = 0, n = own ? p.n_seq : n_runs;
        while (n > 1) {   // the last one whose first unit is at most u
          const int h = n >> 1;
          const int f = own ? first[lo + h].y : first[lo + h].x;
          lo = f <= u ? lo + h : lo;
          n = f <= u ? n - h : h;
        }
        int2 src;
        int tiles;
        if (own) {
          src = make_int2(lo, u - seg[lo].y);
          tiles = ex_own_tiles(seq[lo], src.y, tu, p.causal, run[seg[lo].x].x);
        } else {
          src = make_int2(~lo, u - runseg[lo].x);
          tiles = run[lo].x;
        }
        most = max(most, tiles);
        sum += tiles;
        tiles_of[u] = tiles | (two_tiles(src) ? 1 << 30 : 0);
        part_of[u] = kExPartCost * (float)(min(tu, (own ? seq[lo].y : run[lo].w) - src.y * tu) * p.g) / (2.f * kExTile);
        src_of[u] = src;
      }
    } else {
      walk([&](int, int tiles, int2, int) {
        most = max(most, tiles);
        sum += tiles;
      });
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
      atomicMax(&s_most, most);
      atomicAdd(&s_sum, sum);
    }
    __syncthreads();
  }
  const int most = s_most;
  int piece = most;
  // piece length: of 16 candidates the one with the least estimated time (the
  // mean load of an SM, or the rounds that the larger half of the pieces
  // takes; a piece costs its tiles, 0.8 of them with one row tile, 1.5 more,
  // and what writing and joining its part takes).  Sixteen lanes work on a
  // candidate.  Calls with at least four units per SM fill the device unsplit,
  // and only units longer than an SM's mean load are cut, into halves of it
  // (128 single rows, 127 of them after 1,000 tokens and one after 60,000, 32 / 8
  // heads: 821 us uncut, 189 cut).  Calls too large for part buffers are not cut.
  if (split) {
    const float heads = (float)p.hkv, sms = (float)p.sms;
    const int least = max(kExMinPiece, (int)ceilf((float)s_sum * heads / (kExItemsPerSm * sms)));
    const int c = tid >> 4, cand = ex_candidate(most, least, c);
    const float inv = __frcp_rn((float)cand);
    auto piece_cost = [&](int u, float& np) {
      const float tiles = (float)(tiles_of[u] & ~(1 << 30));
      np = fmaxf(1.f, ceilf(tiles * inv - 1e-4f));
      return (tiles_of[u] >> 30 ? 1.f : 0.8f) * __fdividef(tiles, np) + 1.5f + (np > 1.f ? part_of[u] : 0.f);
    };
    float load = 0.f, big = 0.f, n_big = 0.f, top = 0.f, np;
    for (int u = tid & 15; u < n_units; u += 16) top = fmaxf(top, piece_cost(u, np));
#pragma unroll
    for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int u = tid & 15; u < n_units; u += 16) {
      const float one = piece_cost(u, np);
      load += one * np;
      if (2.f * one > top) {
        big += one * np;
        n_big += np;
      }
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      load += __shfl_xor_sync(0xffffffffu, load, o);
      big += __shfl_xor_sync(0xffffffffu, big, o);
      n_big += __shfl_xor_sync(0xffffffffu, n_big, o);
    }
    if ((tid & 15) == 0) cost[c] = fmaxf(load * heads / sms, ceilf(n_big * heads / sms) * big / fmaxf(n_big, 1.f));
    __syncthreads();
    float low = cost[tid & 15];   // the longest piece on a tie
    int best = tid & 15;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
      const float low2 = __shfl_xor_sync(0xffffffffu, low, o);
      const int best2 = __shfl_xor_sync(0xffffffffu, best, o);
      if (low2 < low || (low2 == low && best2 < best)) {
        low = low2;
        best = best2;
      }
    }
    piece = ex_candidate(most, least, best);
  } else if (p.share >= 0) {
    const unsigned long long even = (s_sum * p.hkv + p.sms - 1) / p.sms;
    if ((unsigned long long)most > even) piece = max(kExMinPiece, (int)((even + 1) / 2));
  }
  // items by cost (key tiles x row tiles), largest first: 256 classes; the
  // order inside a class changes no result.  The pieces of a unit are equal
  // to one tile, so they fall into two classes.
  auto pieces_of = [&](int tiles, int skip) { return tiles == 0 && skip > 0 ? 0 : ex_pieces(tiles, piece); };
  const float per_class = 255.f / (float)(2 * most);
  auto klass = [&](int len, bool two) { return 255 - (int)((float)(two ? 2 * len : len) * per_class); };
  auto skip_of = [&](int2 src) { return src.x >= 0 ? run[seg[src.x].x].x : 0; };
  auto count = [&](int, int tiles, int2 src, int skip) {
    const int np = pieces_of(tiles, skip);
    if (np == 0) return;
    const int len = tiles / np, longer = tiles - len * np;
    const bool two = two_tiles(src);
    atomicAdd(&hist[klass(len, two)], np - longer);
    if (longer) atomicAdd(&hist[klass(len + 1, two)], longer);
  };
  if (split) {
    for (int u = tid; u < n_units; u += kPlanThreads) count(u, tiles_of[u] & ~(1 << 30), src_of[u], skip_of(src_of[u]));
  } else {
    walk(count);
  }
  __syncthreads();
  ExScan items{sums};
  items.turn = units.turn;
  hist[tid] = items(hist[tid]);
  const int n_items = items.carry;
  __syncthreads();
  // writes a unit and the items k = k0, k0 + step, ... of it; with step 16
  // the sixteen lanes of a group share the unit, the first one reserves
  auto emit = [&](int unit, int tiles, int2 src, int skip, int k0, int step, bool valid) {
    const int np = valid ? pieces_of(tiles, skip) : 0;
    const bool own = src.x >= 0, parts = !own || np > 1 || skip > 0;
    const int i = src.y;
    ExUnit u{};
    ExItem it{};
    if (own) {
      const int4 s = seq[src.x];
      const int r = seg[src.x].x;
      u.t0 = s.x + i * tu;
      u.n_tok = min(tu, s.y - i * tu);
      u.sh_unit = skip > 0 ? runseg[r].x : -1;
      u.sh_t0 = seq[run[r].y].x;
      it.seq = src.x;
      it.lim0 = p.causal ? s.z - s.y + i * tu + 1 : s.z;
      it.step = p.causal;
      it.kv_end = s.z;
    } else {
      const int4 v = run[~src.x];
      u.t0 = seq[v.y].x + i * tu;
      u.n_tok = min(tu, v.w - i * tu);
      u.sh_unit = -1;
      it.seq = v.y;
      it.lim0 = it.kv_end = v.x * kExTile;
    }
    const int len = np ? tiles / np : 0, longer = np ? tiles - len * np : 0;
    const bool two = two_tiles(src);
    u.pieces = np;
    u.part = -1;
    int at = 0, at_longer = 0;
    if (k0 == 0 && np > 0) {
      if (parts) u.part = atomicAdd(&s_parts, u.n_tok * p.g * np);
      at = atomicAdd(&hist[klass(len, two)], np - longer);
      if (longer) at_longer = atomicAdd(&hist[klass(len + 1, two)], longer);
    }
    if (step > 1) {
      u.part = __shfl_sync(0xffffffffu, u.part, 0, 16);
      at = __shfl_sync(0xffffffffu, at, 0, 16);
      at_longer = __shfl_sync(0xffffffffu, at_longer, 0, 16);
    }
    if (u.part >= 0 && (long long)u.part + u.n_tok * p.g * np > p.w.part_rows) {   // the sizes exclude it: drop the rows
      set_err(p.status, KVS_DEVERR_PLAN);
      u.part = 0;
      u.n_tok = 0;
    }
    if (valid && k0 == 0 && unit < p.w.max_units) p.w.units[unit] = u;
    it.t0 = u.t0;
    it.n_tok = u.n_tok;
    for (int k = k0; k < np; k += step) {
      it.kv0 = skip + k * len + min(k, longer);
      it.kv1 = it.kv0 + len + (k < longer ? 1 : 0);
      it.part = u.part < 0 ? -1 : u.part + k * u.n_tok * p.g;
      const int slot = k < longer ? at_longer + k : at + k - longer;
      if (slot < p.w.max_items) p.w.items[slot] = it;
    }
  };
  if (split && n_items <= 4 * n_units) {   // few pieces each: a thread per unit
    for (int u = tid; u < n_units; u += kPlanThreads)
      emit(u, tiles_of[u] & ~(1 << 30), src_of[u], skip_of(src_of[u]), 0, 1, true);
  } else if (split) {
    for (int u0 = 0; u0 < n_units; u0 += kPlanThreads / 16) {   // whole warps take part in the exchanges
      const int u = u0 + (tid >> 4), at = min(u, n_units - 1);
      emit(u, tiles_of[at] & ~(1 << 30), src_of[at], skip_of(src_of[at]), tid & 15, 16, u < n_units);
    }
  } else {
    walk([&](int unit, int tiles, int2 src, int skip) { emit(unit, tiles, src, skip, 0, 1, true); });
  }
  __syncthreads();
  if (tid == 0) {
    hdr[kHSeq] = p.n_seq;
    hdr[kHBlocks] = p.max_blocks;
    hdr[kHGroup] = p.g;
    hdr[kHKv] = p.hkv;
    hdr[kHCausal] = p.causal;
    hdr[kHTokens] = p.n_tokens;
    hdr[kHItems] = min(n_items, p.w.max_items);
    hdr[kHCounter] = 0;
    hdr[kHParts] = s_parts;
    hdr[kHUnits] = min(own_units, p.w.max_units);
    hdr[kHMagic] = kExMagic;
  }
}

// -------------------------------------------------------------- attention ---
struct ExParams {
  ExWorkspace w;
  const int32_t *table, *tok_off, *seq_len;
  uint16_t* out;
  uint32_t* status;
  int n_tokens, n_seq, max_blocks, capacity, g, hkv, hq, causal, slab_rows;
  float scale_log2;
};

__device__ __forceinline__ bool ex_plan_ok(const int* hdr, int n_seq, int max_blocks, int g, int hkv, int causal, int n_tokens) {
  const int4* h4 = reinterpret_cast<const int4*>(hdr);
  const int4 a = h4[0], b = h4[1];
  return (a.x == kExMagic) & (a.y == n_seq) & (a.z == max_blocks) & (a.w == g) & (b.x == hkv) & (b.y == causal) & (b.z == n_tokens);
}

struct ExBars {
  uint64_t full[8], empty[8];            // K / V ring
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2];
  uint64_t it_full[2], it_empty[2];      // item slots
  uint64_t fin;
};

// The item as the CTA's roles see it, with the key tiles of each row tile.
struct ExWork {
  ExItem it;
  int head;
  int done;
};

// Key tiles that tile x (0: A, 1: B) of an item takes.
__device__ __forceinline__ int ex_tiles(const ExItem& it, int x, int tt) {
  const int first = x * tt;
  if (first >= it.n_tok) return 0;
  const int last = min(it.n_tok, first + tt) - 1;
  const int lim = min(it.lim0 + it.step * last, it.kv_end);
  return max(0, min((lim + kExTile - 1) / kExTile, it.kv1) - it.kv0);
}

// A 32-byte store: a thread's columns of a row fill whole sectors.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// DIRECT (at most 32 sequences): no plan; the TMA warp makes each item from
// the offsets and lengths, a unit over its whole key range, the CTAs take the
// items in turn and write the result without parts.
template <int D, bool DIRECT>
__global__ void __launch_bounds__(kExThreads, 1)
extend_attn_kernel(const __grid_constant__ ExParams p, const __grid_constant__ CUtensorMap tq,
                   const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  constexpr int HF = D / 64;                  // 64-column halves
  constexpr int ST = ex_stages<D>();
  constexpr int kTile = ex_tile_bytes<D>();
  constexpr int kHalf = kExTile * 128;        // one [128][64] bf16 half, bytes
  constexpr int kBlock = 16 * D * 2;          // one block of a KV head
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExBars bars;
  __shared__ __align__(16) ExWork work[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    mbar_init(&bars.q_full, 1);
    mbar_init(&bars.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_half[i], 4);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.pv_done[i], 1);
      mbar_init(&bars.it_full[i], 1);
      mbar_init(&bars.it_empty[i], 9);   // eight softmax warps and the MMA thread
    }
    mbar_init(&bars.fin, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, kExCols);
    tmem_relinquish();
  }
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto sQ = [&](int x) { return base + kTile * x; };
  auto ring = [&](int i) { return base + kTile * (2 + i); };
  // rows of a query tile behind its last whole token are never copied to
  for (int i = threadIdx.x; i < 2 * kTile / 16; i += kExThreads) reinterpret_cast<uint4*>(base)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tt = kExTile / p.g;
  auto stop = [&]() { return __any_sync(0xffffffffu, s_abort != 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, p.status);
    return __all_sync(0xffffffffu, ok);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kExRegsOther));
  if (warp == 9) {
    // ------------------------------------------- claims and TMA copies
    int n = 0, nq = 0, ni = 0;      // ring uses, query loads, items
    int armed = -1, q_armed = 0;
    int claim = blockIdx.x;
    bool ok = true;
    int n_claims = 0;
    int4 seq{};          // DIRECT: lane a holds sequence a ({first row, rows, keys}) and the units up to its last
    int upto = 0;
    const int tu = 2 * tt;
    if constexpr (DIRECT) {
      bool bad = false;
      if (lane < p.n_seq) {
        const int t0 = __ldg(p.tok_off + lane), t1 = __ldg(p.tok_off + lane + 1), n = __ldg(p.seq_len + lane);
        bad = t0 < 0 || t1 < t0 || t1 > p.n_tokens;
        const int most = p.max_blocks * 16;
        if ((n < 0 || n > most) && blockIdx.x == 0) set_err(p.status, KVS_DEVERR_SEQ_LEN);
        seq = make_int4(t0, t1 - t0, min(max(n, 0), most), 0);
        upto = (seq.y + tu - 1) / tu;
      }
      if (__any_sync(0xffffffffu, bad)) {   // as in the plan: nothing is written
        if (lane == 0 && blockIdx.x == 0) set_err(p.status, KVS_DEVERR_JOB);
        upto = 0;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      n_claims = __shfl_sync(0xffffffffu, upto, 31) * p.hkv;
    } else {
      const bool plan_ok = ex_plan_ok(p.w.hdr, p.n_seq, p.max_blocks, p.g, p.hkv, p.causal, p.n_tokens);
      if (!plan_ok && lane == 0) set_err(p.status, KVS_DEVERR_PLAN);
      n_claims = plan_ok ? min(p.w.hdr[kHItems], p.w.max_items) * p.hkv : 0;
    }
    auto copy = [&](const CUtensorMap* map, bool is_v, int id, int head) {
      // stage n: lanes k < 8 copy block k of the tile; a block without an id
      // lies behind the slab's last row and arrives as zeros
      const int s = n % ST;
      if (n >= ST && !wait(&bars.empty[s], ((n - ST) / ST) & 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&bars.full[s], kTile);
      __syncwarp();
      if (lane < kExBlocks) {
        const int row = id >= 0 ? (id * p.hkv + head) * 16 : p.slab_rows;
        if (is_v) {   // V: the whole block, [block][half][16 tokens][64]
          tma_load_3d(ring(s) + lane * kBlock, map, 0, row, 0, &bars.full[s]);
        } else {      // K: [half][128 tokens][64]
#pragma unroll
          for (int hf = 0; hf < HF; ++hf) tma_load_3d(ring(s) + hf * kHalf + lane * 2048, map, 0, row, hf, &bars.full[s]);
        }
      }
      __syncwarp();
      armed = n++;
      return true;
    };
    while (ok) {
      if (stop()) { ok = false; break; }
      const int slot = ni & 1;
      if (ni >= 2 && !wait(&bars.it_empty[slot], ((ni - 2) >> 1) & 1)) { ok = false; break; }
      const bool end = claim >= n_claims;
      ExItem it{};
      int head = 0, next = 0;
      if (!end) {
        const int item = claim / p.hkv;
        head = claim - item * p.hkv;
        if constexpr (DIRECT) {
          const int a = __ffs(__ballot_sync(0xffffffffu, upto > item)) - 1;   // the first sequence with a unit behind it
          const int t0 = __shfl_sync(0xffffffffu, seq.x, a), rows = __shfl_sync(0xffffffffu, seq.y, a);
          const int keys = __shfl_sync(0xffffffffu, seq.z, a), end = __shfl_sync(0xffffffffu, upto, a);
          const int i = end - 1 - item;   // the last unit, which sees most, first
          it.t0 = t0 + i * tu;
          it.n_tok = min(tu, rows - i * tu);
          it.seq = a;
          it.kv1 = ex_own_tiles(make_int4(t0, rows, keys, 0), i, tu, p.causal, 0);
          it.lim0 = p.causal ? keys - rows + i * tu + 1 : keys;
          it.step = p.causal;
          it.kv_end = keys;
          it.part = -1;
          // rounds over the CTAs in alternating order, so that whoever had a
          // long item takes a short one (a causal chunk's units get shorter)
          next = claim + (ni & 1 ? 2 * (int)blockIdx.x + 1 : 2 * (int)(gridDim.x - blockIdx.x) - 1);
        } else {
          const int4* src = reinterpret_cast<const int4*>(p.w.items + item);
          int4* dst = reinterpret_cast<int4*>(&it);
          dst[0] = __ldg(src);
          dst[1] = __ldg(src + 1);
          dst[2] = __ldg(src + 2);
          if (lane == 0) next = (int)gridDim.x + atomicAdd(p.w.hdr + kHCounter, 1);
        }
      }
      if (lane == 0) {
        work[slot].it = it;
        work[slot].head = head;
        work[slot].done = end;
        mbar_arrive(&bars.it_full[slot]);
      }
      __syncwarp();
      ++ni;
      if (end) break;
      const int na = ex_tiles(it, 0, tt), nb = ex_tiles(it, 1, tt), nt = max(na, nb);
      const int32_t* row = p.table + (size_t)it.seq * p.max_blocks;
      const int nblk = (it.kv_end + 15) / 16;
      auto block = [&](int j) {
        const int b = (it.kv0 + j) * kExBlocks + lane;
        int id = -1;
        if (lane < kExBlocks && j < nt && b < nblk) {
          id = __ldg(row + b);
          if (id < 0 || id >= p.capacity) {
            set_err(p.status, KVS_DEVERR_BLOCK_ID);
            id = -1;
          }
        }
        return id;
      };
      int id = block(0);
      for (int j = 0; j < nt; ++j) {
        const int id_next = block(j + 1);
        if (!copy(&tk, false, id, head)) { ok = false; break; }
        if (j == 0) {
          // the query tiles, once the last S of the item before has read them
          if (nq >= 1 && !wait(&bars.q_empty, (nq - 1) & 1)) { ok = false; break; }
          if (lane == 0) {
            const int tiles = nb > 0 ? 2 : 1;
            mbar_arrive_expect_tx(&bars.q_full, (uint32_t)(tiles * HF * tt * p.g * 128));
            for (int x = 0; x < tiles; ++x)
              for (int hf = 0; hf < HF; ++hf)
                tma_load_5d(sQ(x) + hf * kHalf, &tq, 0, 0, it.t0 + x * tt, head, hf, &bars.q_full);
          }
          __syncwarp();
          q_armed = ++nq;
        }
        if (!copy(&tv, true, id, head)) { ok = false; break; }
        id = id_next;
      }
      claim = __shfl_sync(0xffffffffu, next, 0);
    }
    if (!ok) {
      s_abort = 1;
      // copies in flight land before the shared memory goes away
      for (int m = max(0, armed - ST + 1); m <= armed; ++m) mbar_drain(&bars.full[m % ST], (m / ST) & 1);
      if (q_armed) mbar_drain(&bars.q_full, (q_armed - 1) & 1);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------- MMA issue
    constexpr uint32_t idS = umma_idesc_bf16(128, 128, false, false);
    constexpr uint32_t idO = umma_idesc_bf16(128, D, false, true);
    constexpr uint32_t kHi = ex_desc_hi(1024);
    const uint32_t q_lo = ex_desc_lo(smem_u32(base), 16);
    const uint32_t k_lo = ex_desc_lo(smem_u32(ring(0)), 16), v_lo = ex_desc_lo(smem_u32(ring(0)), 2048);
    struct Pos {   // a use of the ring
      int s;
      uint32_t par;
      __device__ __forceinline__ void next() {
        if (++s == ST) {
          s = 0;
          par ^= 1u;
        }
      }
    };
    Pos at{0, 0};                         // K of the tile to come
    uint32_t q_par = 0, np[2] = {0, 0};   // query loads, P uses
    bool ok = true;
    auto issue_s = [&](int x, const Pos& k) {    // S_x = Q_x K^T
      if (elect_one()) {
        const uint32_t a = q_lo + x * (kTile / 16), b = k_lo + k.s * (kTile / 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) / 16;
          ex_mma_ss(tmem + 128u * x, a + o, b + o, kHi, idS, kk > 0);
        }
        umma_commit(&bars.s_full[x]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, const Pos& v, int k0, bool acc) {   // O_x (+)= P_x V over keys 16 k0 .. 16 k0 + 63
      if (elect_one()) {
        const uint32_t b = v_lo + v.s * (kTile / 16);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)   // per 32 keys 16 columns of first parts, then 16 of second ones
          ex_mma_ts(tmem + 256u + (uint32_t)D * x, tmem + 128u * x + 16u * k0 + 32u * (kk >> 2) + 8u * (kk >> 1 & 1) + 16u * (kk & 1),
                    b + (k0 + (kk >> 1)) * (kBlock / 16), kHi, idO, acc || kk > 0);
        if (k0) umma_commit(&bars.pv_done[x]);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    for (int ni = 0;; ++ni) {
      const int slot = ni & 1;
      if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
      const int na = __shfl_sync(0xffffffffu, ex_tiles(work[slot].it, 0, tt), 0);
      const int nb = __shfl_sync(0xffffffffu, ex_tiles(work[slot].it, 1, tt), 0);
      const int done = __shfl_sync(0xffffffffu, work[slot].done, 0);
      if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
      __syncwarp();
      if (done) break;
      const int nt = max(na, nb), last_x = nb > 0 ? 1 : 0;
      if (nt == 0) continue;
      Pos kj = at;
      if (!wait(&bars.full[at.s], at.par) || !wait(&bars.q_full, q_par)) { ok = false; break; }
      q_par ^= 1u;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if ((x ? nb : na) == 0) continue;
        // P of the item before has been read (its last P V is complete)
        if (np[x] > 0 && !wait(&bars.pv_done[x], (np[x] - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        issue_s(x, at);
      }
      if (!ok) break;
      if (nt == 1) commit(&bars.q_empty);
      at.next();
      for (int j = 0; j < nt; ++j) {
        const Pos v = at;
        at.next();
        const Pos k = at;     // K(j + 1)
        const bool more = j + 1 < nt;
        if (more) at.next();
        if (!wait(&bars.full[v.s], v.par)) { ok = false; break; }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nx = x ? nb : na;
          if (j >= nx) continue;
          const uint32_t par = np[x] & 1;
          ++np[x];
          if (!wait(&bars.p_half[x], par)) { ok = false; break; }
          tc_fence_after();
          issue_pv(x, v, 0, j > 0);
          // weights of the last row tile: its S, the last to read this K, is
          // complete.  Stages are handed back by plain arrivals where a wait
          // has shown them free: a commit costs the MMA pipe more (1.5 % of a
          // long chunk for two of six).
          if (x == last_x && lane == 0) mbar_arrive(&bars.empty[kj.s]);
          if (!wait(&bars.p_full[x], par)) { ok = false; break; }
          tc_fence_after();
          issue_pv(x, v, 4, true);
          if (j + 1 < nx) {
            if (!wait(&bars.full[k.s], k.par) || !wait(&bars.pv_done[x], par)) { ok = false; break; }   // S goes where P was
            tc_fence_after();
            issue_s(x, k);
            if (x == last_x && lane == 0) mbar_arrive(&bars.empty[v.s]);
          } else if (x == last_x) {
            commit(&bars.empty[v.s]);
          }
        }
        if (!ok) break;
        kj = k;
        if (j + 2 == nt) commit(&bars.q_empty);
      }
      if (!ok) break;
    }
    if (!ok) s_abort = 1;
    // every MMA issued has completed before the tensor memory is released
    commit(&bars.fin);
    mbar_wait_bounded(&bars.fin, 0, p.status);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kExRegsSoftmax));
    // ---------------------------------------------------------- softmax
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;   // row tile, row = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128u * x, tO = tmem + lanes + 256u + (uint32_t)D * x;
    const int rt = r / p.g, rg = r - rt * p.g;             // token and head of the row
    const float sl2 = p.scale_log2;
    int ns = 0, n = 0;      // S uses of this tile, ring position
    bool ok = true;
    for (int ni = 0;; ++ni) {
      const int slot = ni & 1;
      if (stop() || !wait(&bars.it_full[slot], (ni >> 1) & 1)) { ok = false; break; }
      const ExItem it = work[slot].it;
      const int head = work[slot].head, done = work[slot].done;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.it_empty[slot]);
      if (done) break;
      const int nt = ex_tiles(it, x, tt), nt_other = ex_tiles(it, x ^ 1, tt), nt_all = max(nt, nt_other);
      const int tok = x * tt + rt;
      const bool live = rt < tt && tok < it.n_tok;
      const int lim = min(it.lim0 + it.step * tok, it.kv_end);   // keys this row sees
      // rows of the last V tile behind the sequence's end hold anything: the
      // first tile that takes it zeroes them up to the block's end (P is zero
      // there, but 0 * NaN is not)
      const int tail = it.kv_end - (it.kv0 + nt_all - 1) * kExTile;
      const bool fix_tail = nt == nt_all && (x == 0 || nt_other < nt_all) && tail < kExTile && (tail & 15);
      float m = -INFINITY, l = 0.f;   // reference point of l and O, sum of the weights
      const float2 sc2 = make_float2(sl2, sl2);
      float2 sum0, sum1;
      // p[0..15] and p[16..31] = the two bf16 parts of 2^(s - ref) of 32 scores
      auto weigh = [&](const uint32_t* s, uint32_t* p, float ref) {
        const float2 rf2 = make_float2(-ref, -ref), neg = make_float2(-1.f, -1.f);
        auto split = [&](float2 w, uint32_t& h, uint32_t& rest) {   // the remainder is exact
          const uint32_t x = __float_as_uint(w.x), y = __float_as_uint(w.y);
          h = __byte_perm(x, y, 0x7632);
          const float2 r = __ffma2_rn(make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u)), neg, w);
          rest = pack_bf16(r.x, r.y);
        };
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float2 a = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          float2 b = make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
          a = __ffma2_rn(a, sc2, rf2);
          b = __ffma2_rn(b, sc2, rf2);
          a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
          b = make_float2(fast_exp2(b.x), fast_exp2(b.y));
          sum0 = __fadd2_rn(sum0, a);
          sum1 = __fadd2_rn(sum1, b);
          split(a, p[i / 2], p[16 + i / 2]);
          split(b, p[i / 2 + 1], p[17 + i / 2]);
        }
      };
      auto most = [&](const uint32_t* s) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          a = fmaxf(a, fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
          b = fmaxf(b, fmaxf(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])));
        }
        return fmaxf(a, b);
      };
      for (int j = 0; j < nt; ++j) {
        if (!wait(&bars.s_full[x], ns & 1)) { ok = false; break; }
        tc_fence_after();
        uint32_t sa[32], sb[32], sc[32], sd[32], pa[32];
        tmem_ld32_issue(tS, sa);
        tmem_ld32_issue(tS + 32, sb);
        tmem_ld32x2_wait(sa, sb);
        tmem_ld32_issue(tS + 64, sc);
        tmem_ld32_issue(tS + 96, sd);
        const int rem = lim - (it.kv0 + j) * kExTile;   // visible keys of this tile
        const bool masked = __any_sync(0xffffffffu, rem < kExTile && live);
        auto mask = [&](uint32_t* v, int first) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i + first >= rem) v[i] = 0xff800000u;
        };
        if (masked) {
          mask(sa, 0);
          mask(sb, 32);
        }
        float mx = fmaxf(most(sa), most(sb));
        tmem_ld32x2_wait(sc, sd);
        if (masked) {
          mask(sc, 64);
          mask(sd, 96);
        }
        mx = fmaxf(mx, fmaxf(most(sc), most(sd))) * sl2;
        const float next = mx > m + 8.f ? mx : m;
        const float ref = next == -INFINITY ? 0.f : next;   // nothing visible yet: 2^(-inf - 0) = 0
        sum0 = sum1 = make_float2(0.f, 0.f);
        weigh(sa, pa, ref);
        tmem_st32(tS, pa);
        weigh(sb, pa, ref);
        tmem_st32(tS + 32, pa);
        // a row whose reference moved rescales its O once the P V before is done
        const bool move = m != -INFINITY && next > m;
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? fast_exp2(m - next) : 1.f;
          if (!wait(&bars.pv_done[x], (ns - 1) & 1)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t v[16];
            tmem_ld16(tO + 16 * q, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_st16(tO + 16 * q, v);
          }
          l *= f;
        }
        m = next;
        if (j == nt - 1 && fix_tail) {
          const int mv = n + 2 * j + 1;
          if (!wait(&bars.full[mv % ST], (mv / ST) & 1)) { ok = false; break; }
          const int rows = ((tail + 15) & ~15) - tail;
          for (int i = threadIdx.x & 127; i < rows * HF * 8; i += 128) {
            const int c = i & 7, hf = (i >> 3) % HF, rr = tail + (i >> 3) / HF;
            *reinterpret_cast<uint4*>(ring(mv % ST) + (rr >> 4) * kBlock + hf * 2048 + (rr & 15) * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_half[x]);
        weigh(sc, pa, ref);
        tmem_st32(tS + 64, pa);
        weigh(sd, pa, ref);
        tmem_st32(tS + 96, pa);
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[x]);
        ++ns;
      }
      n += 2 * nt_all;
      if (!ok) break;
      // the rows' results
      if (nt > 0) {
        if (!wait(&bars.pv_done[x], (ns - 1) & 1)) { ok = false; break; }
        tc_fence_after();
      }
      const bool some = live && !(l == 0.f);
      const size_t prow = ((size_t)(it.part + tok * p.g + rg)) * p.hkv + head;
      const float inv = some ? 1.f / l : 0.f;
      if (x == 1 && it.n_tok <= tt) continue;   // no tile B
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t v[32];
        if (nt > 0) tmem_ld32(tO + 32 * q, v);
        if (live && it.part >= 0) {
          float* dst = p.w.part + prow * D + 32 * q;
          if (!some) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) st_global_v8(dst + 8 * e, v + 8 * e);
        } else if (live) {
          uint16_t* dst = p.out + ((size_t)(it.t0 + tok) * p.hq + head * p.g + rg) * D + 32 * q;
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = some ? pack_bf16(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv) : 0u;
          st_global_v8(dst, o);
          st_global_v8(dst + 16, o + 8);
        }
        __syncwarp();
      }
      if (live && it.part >= 0) p.w.ml[prow] = make_float2(some ? m : -INFINITY, some ? l : 0.f);
    }
    if (!ok) s_abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kExCols);
  }
}

// ------------------------------------------------------------------ merge ---
// Joins the parts of the rows that have several, in the order shared range,
// own range, each by its pieces.  A CTA takes one unit and KV head and every
// gridDim.z-th sixteen rows of it, a warp two rows at a time.  The parts lie
// in L2 and the chain of loads bounds it: up to four parts of both rows are
// loaded at once; with more, 32 lanes take the factors of 32 parts and four
// parts are in flight.  2,800 rows of 16 heads with two to four parts: 18 us
// alone (71 us with a row per warp, parts one by one).
template <int D>
__global__ void __launch_bounds__(256) extend_merge_kernel(const __grid_constant__ ExParams p) {
  pdl_enter();
  constexpr int E = D / 32;   // elements per lane
  constexpr int U = 4, R = kExMergeRows;
  const bool plan_ok = ex_plan_ok(p.w.hdr, p.n_seq, p.max_blocks, p.g, p.hkv, p.causal, p.n_tokens);
  if (!plan_ok) return;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) p.w.hdr[kHCounter] = 0;   // for the next layer
  const int n_units = p.w.hdr[kHUnits], head = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tu = 2 * (kExTile / p.g);
  struct Vec {
    float v[E];
  };
  auto load = [&](size_t row) {
    Vec x;
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p.w.part + row * D + lane * 4);
      x.v[0] = y.x; x.v[1] = y.y; x.v[2] = y.z; x.v[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(p.w.part + row * D + lane * 2);
      x.v[0] = y.x; x.v[1] = y.y;
    }
    return x;
  };
  if (p.w.hdr[kHParts] == 0) return;   // every row has been written by the attention
  for (int i = blockIdx.x; i < n_units; i += gridDim.x) {
    const ExUnit u = p.w.units[i];
    if (u.part < 0 && u.sh_unit < 0) continue;   // written by the attention itself
    const int rows = u.n_tok * p.g, n_own = u.part >= 0 ? u.pieces : 0;
    for (int r0 = (blockIdx.z * 8 + warp) * R; r0 < rows; r0 += 8 * R * gridDim.z) {
      // a row's parts: n_sh of the shared range from sh_at on, sh_step rows
      // apart (every unit of a shared range has as many), then its own
      int row[R], sh_at[R], sh_step[R], n_sh = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        row[j] = min(r0 + j, rows - 1);
        sh_at[j] = sh_step[j] = 0;
        if (u.sh_unit >= 0) {
          const int t = u.t0 + row[j] / p.g;
          const ExUnit sh = p.w.units[u.sh_unit + (t - u.sh_t0) / tu];
          n_sh = sh.pieces;
          sh_step[j] = sh.n_tok * p.g;
          sh_at[j] = sh.part + (t - sh.t0) * p.g + row[j] % p.g;
        }
      }
      const int n = n_sh + n_own;
      auto at = [&](int j, int k) {
        const int r = k < n_sh ? sh_at[j] + k * sh_step[j] : u.part + (k - n_sh) * rows + row[j];
        return (size_t)r * p.hkv + head;
      };
      Vec acc[R];
      float l[R];
      if (n <= U) {
        float2 ml[R][U];
        Vec x[R][U];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int k = 0; k < U; ++k) {
            ml[j][k] = make_float2(-INFINITY, 0.f);
            x[j][k] = Vec{};
            if (k < n) {
              ml[j][k] = p.w.ml[at(j, k)];
              x[j][k] = load(at(j, k));
            }
          }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const float mx = fmaxf(fmaxf(ml[j][0].x, ml[j][1].x), fmaxf(ml[j][2].x, ml[j][3].x));
          const float ref = mx == -INFINITY ? 0.f : mx;   // no part saw a key: factors 0
          acc[j] = Vec{};
          l[j] = 0.f;
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const float f = fast_exp2(ml[j][k].x - ref);
            l[j] += f * ml[j][k].y;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[j].v[e] += f * x[j][k].v[e];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < R; ++j) {
          float mx = -INFINITY, lj = 0.f;
          Vec a{};
          for (int k = lane; k < n; k += 32) mx = fmaxf(mx, p.w.ml[at(j, k)].x);
#pragma unroll
          for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float ref = mx == -INFINITY ? 0.f : mx;
          for (int k0 = 0; k0 < n; k0 += 32) {
            float f = 0.f;
            if (k0 + lane < n) {
              const float2 ml = p.w.ml[at(j, k0 + lane)];
              f = fast_exp2(ml.x - ref);
              lj += f * ml.y;
            }
            const int m = min(32, n - k0);
            for (int k = 0; k < m; k += U) {
              Vec x[U];
#pragma unroll
              for (int q = 0; q < U; ++q) x[q] = k + q < m ? load(at(j, k0 + k + q)) : Vec{};
#pragma unroll
              for (int q = 0; q < U; ++q) {
                const float fq = __shfl_sync(0xffffffffu, f, min(k + q, 31));
#pragma unroll
                for (int e = 0; e < E; ++e) a.v[e] += fq * x[q].v[e];
              }
            }
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) lj += __shfl_xor_sync(0xffffffffu, lj, o);
          acc[j] = a;
          l[j] = lj;
        }
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (r0 + j >= rows) break;
        const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            p.out + ((size_t)(u.t0 + row[j] / p.g) * p.hq + head * p.g + row[j] % p.g) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[j].v[e] * inv, acc[j].v[e + 1] * inv);
      }
    }
  }
}

// ------------------------------------------------------------------- host ---
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 ex_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

// Queries [tokens][hkv][G][D] as {64 elements, G heads, tokens, KV heads, D/64
// halves}: a box {64, G, 128/G, 1, 1} is one half of a row tile, row = token *
// G + head.  Tokens behind the last one arrive as zeros.
bool ex_query_map(CUtensorMap* m, const void* q, int n_tokens, int g, int hkv, int d, long long stride) {
  auto enc = ex_encoder();
  if (!enc) return false;
  cuuint64_t dims[5] = {64, (cuuint64_t)g, (cuuint64_t)n_tokens, (cuuint64_t)hkv, (cuuint64_t)(d / 64)};
  cuuint64_t strides[4] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2, (cuuint64_t)g * d * 2, 128};
  cuuint32_t box[5] = {64, (cuuint32_t)g, (cuuint32_t)(kExTile / g), 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(q), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

kvs_status ex_check(const kvs_pool* pool, const char* what, int n_tokens, int n_seq, int max_blocks, int n_q_heads) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": null pool");
  const kvs_pool_desc& d = pool->desc;
  if (d.dtype != KVS_DTYPE_BF16) return fail(KVS_ERR_UNSUPPORTED, std::string(what) + ": bf16 pools only");
  if (n_tokens < 0 || n_seq < 0 || max_blocks < 1) return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, std::string(what) + ": n_seq exceeds the pool's max_seqs");
  if (n_q_heads < 1 || n_q_heads % d.num_kv_heads)
    return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": n_q_heads must be a multiple of num_kv_heads");
  if (n_q_heads / d.num_kv_heads > 16) return fail(KVS_ERR_UNSUPPORTED, std::string(what) + ": more than 16 query heads per KV head");
  // key tiles, part rows and claims (units x KV heads) are counted in 32
  // bits, KV heads are a grid dimension
  const long long rows = (long long)n_tokens * n_q_heads, units = 4ll * n_seq * d.num_kv_heads;
  if ((long long)max_blocks * 16 > (1ll << 30) || rows > (1ll << 30) || units > (1ll << 30) || d.num_kv_heads > 65535)
    return fail(KVS_ERR_CAPACITY, std::string(what) + ": too many tokens, sequences or KV heads");
  return KVS_OK;
}

namespace {

constexpr float kExLog2e = 1.4426950408889634f;   // scores are taken to base 2
bool ex_scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * kExLog2e); }

kvs_status ex_check_ws(const ExWorkspace& w, const void* ws, size_t ws_bytes, const char* what) {
  if (!ws) return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": null workspace");
  if (!aligned32(ws)) return fail(KVS_ERR_INVALID_ARG, std::string(what) + ": ws must be 32-byte aligned");
  if (ws_bytes < w.bytes) return fail(KVS_ERR_CAPACITY, std::string(what) + ": workspace too small");
  return KVS_OK;
}

template <typename... KArgs, typename... Args>
cudaError_t ex_launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
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

// Whether the whole attention goes in one launch (DIRECT), with nothing split
// or shared; the rule goes by what the host knows.  Times below are of CUDA-graph
// replays, planned and in one launch.
//  * Short tables and at most two rounds of units: a plan and a merge mostly take
//    longer than they save (16 x 4 rows after 1,000 tokens, 40 / 8 heads: 30 and
//    19 us; 8 x 128 rows after 1,000, 32 / 8: 36 and 27; 2 x 64 rows after 300,
//    8 / 2: 21 and 13).  The bound is crude: few rows near it would gain from
//    splits (1 row after 1,500, 32 / 8: 20 and 25), and calls behind it that
//    fill the device once would do without (16 x 4 after 2,000, 40 / 8: 49 and 33).
//  * Chunks of at least a unit on the mean that fill the SMs without splits (8 x
//    256 rows after 1,800 tokens, 32 / 8 heads: 93 and 81 us; 1 x 2,048 rows after
//    2,048, 32 / 32: 128 and 112).  The host knows the longest table, not
//    whose it is: with several sequences a single row may own it, so the tables
//    must be short enough that this row's chain of key tiles costs no more than
//    the plan (2,048 rows and 1 row after 4,000: 72 and 90 us; 1 row after 8,000:
//    72 and 141, after 60,000: 116 and 800; 2 x 1,024 rows after 8,000, which
//    are planned for that reason: 311 and 304).  One sequence's units are about
//    equally long; its last round must not be mostly empty where they are long.
//    Beyond kExDirectRounds rounds the plan's order by length is worth more than
//    its time.
bool ex_direct(const kvs_pool* pool, int n_tokens, int n_seq, int max_blocks, int g) {
  if (pool->test_flags & KVS_TEST_EXTEND_PLANNED) return false;
  const long long tu = ex_tokens_per_unit(g), whole = n_tokens / tu, hkv = pool->desc.num_kv_heads, sms = pool->num_sms;
  if (n_seq > 32) return false;
  const bool small = max_blocks <= kExDirectBlocks && (whole + n_seq) * hkv <= 2 * sms;
  const long long likely = (2 * whole + n_seq) * hkv / 2, rounds = (likely + sms - 1) / sms;   // half a unit left per sequence
  const bool even = max_blocks <= kExDirectShort || (n_seq == 1 && 4 * likely >= 3 * rounds * sms);
  const bool full = n_tokens >= n_seq * tu && whole * hkv >= sms && rounds <= kExDirectRounds && even;
  return small || full;
}

template <int D>
kvs_status ex_direct_run(kvs_pool* pool, int layer, const ExParams& p, const CUtensorMap& tq, long long max_claims, cudaStream_t stream) {
  if (!smem_limit_once<extend_attn_kernel<D, true>>(ex_smem<D>(), pool->device))
    return fail(KVS_ERR_CUDA, "extend_attn: cannot raise the shared-memory limit");
  const unsigned grid = (unsigned)std::min<long long>(pool->num_sms, max_claims);
  const CUtensorMap& tk = D == 128 ? pool->tk1[layer] : pool->tk[layer];
  if (ex_launch(extend_attn_kernel<D, true>, dim3(grid), dim3(kExThreads), ex_smem<D>(), stream, p, tq, tk, pool->tv[layer]) != cudaSuccess)
    return fail(KVS_ERR_CUDA, std::string("extend_attn: ") + cudaGetErrorString(cudaGetLastError()));
  count_launch();
  return check_launch("extend_attn");
}

template <int D>
kvs_status ex_run(kvs_pool* pool, int layer, const ExParams& p, const CUtensorMap& tq, long long max_claims, cudaStream_t stream) {
  if (!smem_limit_once<extend_attn_kernel<D, false>>(ex_smem<D>(), pool->device))
    return fail(KVS_ERR_CUDA, "extend_attn: cannot raise the shared-memory limit");
  const unsigned grid = (unsigned)std::min<long long>(pool->num_sms, max_claims);
  const CUtensorMap& tk = D == 128 ? pool->tk1[layer] : pool->tk[layer];
  const CUtensorMap& tv = pool->tv[layer];
  if (ex_launch(extend_attn_kernel<D, false>, dim3(grid), dim3(kExThreads), ex_smem<D>(), stream, p, tq, tk, tv) != cudaSuccess)
    return fail(KVS_ERR_CUDA, std::string("extend_attn: ") + cudaGetErrorString(cudaGetLastError()));
  count_launch();
  // about 8 CTAs per SM over units, heads and blocks of sixteen rows
  const unsigned units = (unsigned)std::min(p.w.max_units / 2, 4096);
  const long long most = std::min<long long>(32 / kExMergeRows, ((long long)p.n_tokens * p.g + 8 * kExMergeRows - 1) / (8 * kExMergeRows));
  const unsigned z = (unsigned)std::clamp<long long>(8ll * pool->num_sms / ((long long)units * p.hkv), 1, most);
  if (ex_launch(extend_merge_kernel<D>, dim3(units, (unsigned)p.hkv, z), dim3(256), 0, stream, p) != cudaSuccess)
    return fail(KVS_ERR_CUDA, std::string("extend_attn merge: ") + cudaGetErrorString(cudaGetLastError()));
  count_launch();
  return check_launch("extend_attn");
}

}  // namespace

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_extend_workspace_size(const kvs_pool* pool, int32_t n_tokens, int32_t n_seq, int32_t max_blocks,
                                                int32_t n_q_heads, size_t* bytes) {
  if (!bytes) return fail(KVS_ERR_INVALID_ARG, "extend_workspace_size: null pointer");
  if (kvs_status st = ex_check(pool, "extend_workspace_size", n_tokens, n_seq, max_blocks, n_q_heads); st != KVS_OK) return st;
  *bytes = ex_layout(pool, n_tokens, n_seq, max_blocks, n_q_heads / pool->desc.num_kv_heads, nullptr).bytes;
  return KVS_OK;
}

extern "C" kvs_status kvs_extend_plan(kvs_pool* pool, const int32_t* tok_off_dev, int32_t n_tokens, int32_t n_q_heads,
                                      const int32_t* block_table_dev, int32_t max_blocks, const int32_t* seq_len_dev,
                                      int32_t n_seq, int32_t causal, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (kvs_status st = ex_check(pool, "extend_plan", n_tokens, n_seq, max_blocks, n_q_heads); st != KVS_OK) return st;
  if (causal != 0 && causal != 1) return fail(KVS_ERR_INVALID_ARG, "extend_plan: causal is 0 or 1");
  if (n_tokens == 0 || n_seq == 0) return KVS_OK;
  if (!tok_off_dev || !block_table_dev || !seq_len_dev) return fail(KVS_ERR_INVALID_ARG, "extend_plan: null pointer");
  const int hkv = pool->desc.num_kv_heads, g = n_q_heads / hkv;
  if (kvs_status st = check_pool_device(pool, "extend_plan"); st != KVS_OK) return st;
  if (ex_direct(pool, n_tokens, n_seq, max_blocks, g)) return KVS_OK;
  ExPlanParams p{};
  p.w = ex_layout(pool, n_tokens, n_seq, max_blocks, g, ws);
  if (kvs_status st = ex_check_ws(p.w, ws, ws_bytes, "extend_plan"); st != KVS_OK) return st;
  p.tok_off = tok_off_dev;
  p.seq_len = seq_len_dev;
  p.table = block_table_dev;
  p.status = pool->status;
  p.n_tokens = n_tokens;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.capacity = pool->desc.capacity_blocks;
  p.g = g;
  p.hkv = hkv;
  p.causal = causal;
  p.sms = pool->num_sms;
  const bool parts = (long long)n_tokens * n_q_heads <= kExPartRows;
  p.share = !parts ? -1 : n_seq > 1 ? 1 : 0;
  // Short tables are compared by the plan's one CTA (12 sequences of 94 blocks:
  // 7.4 -> 6.2 us for the plan), long ones by a CTA per pair before it (64
  // sequences of 900 blocks: 11.0 us, 22.2 in the one CTA).
  p.lcp_here = p.share == 1 && (long long)n_seq * max_blocks <= kPlanTable;
  if (p.share == 1 && !p.lcp_here) {
    if (launch_pdl(extend_lcp_kernel, dim3((unsigned)(n_seq - 1)), dim3(256), stream, p) != cudaSuccess)
      return fail(KVS_ERR_CUDA, std::string("extend_plan: ") + cudaGetErrorString(cudaGetLastError()));
    count_launch();
  }
  if (launch_pdl(extend_plan_kernel, dim3(1), dim3(kPlanThreads), stream, p) != cudaSuccess)
    return fail(KVS_ERR_CUDA, std::string("extend_plan: ") + cudaGetErrorString(cudaGetLastError()));
  count_launch();
  return check_launch("extend_plan");
}

extern "C" kvs_status kvs_extend_attn_planned(kvs_pool* pool, int32_t layer, const void* q_dev, int64_t q_stride,
                                              const int32_t* tok_off_dev, int32_t n_tokens, int32_t n_q_heads,
                                              const int32_t* block_table_dev, int32_t max_blocks,
                                              const int32_t* seq_len_dev, int32_t n_seq, int32_t causal, float scale,
                                              void* out_dev, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (kvs_status st = ex_check(pool, "extend_attn", n_tokens, n_seq, max_blocks, n_q_heads); st != KVS_OK) return st;
  const kvs_pool_desc& d = pool->desc;
  if (layer < 0 || layer >= d.num_layers) return fail(KVS_ERR_INVALID_ARG, "extend_attn: layer out of range");
  if (causal != 0 && causal != 1) return fail(KVS_ERR_INVALID_ARG, "extend_attn: causal is 0 or 1");
  if (!ex_scale_ok(scale)) return fail(KVS_ERR_INVALID_ARG, "extend_attn: scale must be positive, and scale * log2(e) finite");
  const long long row = (long long)n_q_heads * d.head_dim;
  if (q_stride < row || (q_stride & 7)) return fail(KVS_ERR_INVALID_ARG, "extend_attn: q_stride must hold n_q_heads * head_dim elements and be a multiple of 8");
  if (n_tokens == 0 || n_seq == 0) return KVS_OK;
  if (!q_dev || !tok_off_dev || !block_table_dev || !seq_len_dev || !out_dev)
    return fail(KVS_ERR_INVALID_ARG, "extend_attn: null pointer");
  if (!aligned16(q_dev) || !aligned32(out_dev))
    return fail(KVS_ERR_INVALID_ARG, "extend_attn: q must be 16-byte, out 32-byte aligned");
  const int g = n_q_heads / d.num_kv_heads;
  const bool direct = ex_direct(pool, n_tokens, n_seq, max_blocks, g);
  ExParams p{};
  if (!direct) {
    p.w = ex_layout(pool, n_tokens, n_seq, max_blocks, g, ws);
    if (kvs_status st = ex_check_ws(p.w, ws, ws_bytes, "extend_attn"); st != KVS_OK) return st;
  }
  if (kvs_status st = check_pool_device(pool, "extend_attn"); st != KVS_OK) return st;
  p.table = block_table_dev;
  p.tok_off = tok_off_dev;
  p.seq_len = seq_len_dev;
  p.out = static_cast<uint16_t*>(out_dev);
  p.status = pool->status;
  p.n_tokens = n_tokens;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.capacity = d.capacity_blocks;
  p.g = g;
  p.hkv = d.num_kv_heads;
  p.hq = n_q_heads;
  p.causal = causal;
  p.slab_rows = d.capacity_blocks * d.num_kv_heads * d.block_tokens;
  p.scale_log2 = scale * kExLog2e;
  CUtensorMap tq;
  if (!ex_query_map(&tq, q_dev, n_tokens, g, d.num_kv_heads, d.head_dim, q_stride))
    return fail(KVS_ERR_CUDA, "extend_attn: cuTensorMapEncodeTiled failed for q");
  if (direct) {
    const long long claims = (n_tokens / ex_tokens_per_unit(g) + n_seq) * (long long)d.num_kv_heads;
    return d.head_dim == 128 ? ex_direct_run<128>(pool, layer, p, tq, claims, stream)
                             : ex_direct_run<64>(pool, layer, p, tq, claims, stream);
  }
  const long long max_claims = (long long)p.w.max_items * d.num_kv_heads;
  return d.head_dim == 128 ? ex_run<128>(pool, layer, p, tq, max_claims, stream)
                           : ex_run<64>(pool, layer, p, tq, max_claims, stream);
}

extern "C" kvs_status kvs_extend_attn(kvs_pool* pool, int32_t layer, const void* q_dev, int64_t q_stride,
                                      const int32_t* tok_off_dev, int32_t n_tokens, int32_t n_q_heads,
                                      const int32_t* block_table_dev, int32_t max_blocks, const int32_t* seq_len_dev,
                                      int32_t n_seq, int32_t causal, float scale, void* out_dev, void* ws,
                                      size_t ws_bytes, cudaStream_t stream) {
  // the layer's own arguments are checked before the plan is enqueued
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "extend_attn: null pool");
  if (layer < 0 || layer >= pool->desc.num_layers) return fail(KVS_ERR_INVALID_ARG, "extend_attn: layer out of range");
  if (!ex_scale_ok(scale)) return fail(KVS_ERR_INVALID_ARG, "extend_attn: scale must be positive, and scale * log2(e) finite");
  if (n_tokens > 0 && n_seq > 0 && (!q_dev || !out_dev || !aligned16(q_dev) || !aligned32(out_dev)))
    return fail(KVS_ERR_INVALID_ARG, "extend_attn: q must be set and 16-byte, out set and 32-byte aligned");
  if (q_stride < (long long)n_q_heads * pool->desc.head_dim || (q_stride & 7))
    return fail(KVS_ERR_INVALID_ARG, "extend_attn: q_stride must hold n_q_heads * head_dim elements and be a multiple of 8");
  kvs_status st = kvs_extend_plan(pool, tok_off_dev, n_tokens, n_q_heads, block_table_dev, max_blocks, seq_len_dev, n_seq,
                                  causal, ws, ws_bytes, stream);
  if (st != KVS_OK) return st;
  return kvs_extend_attn_planned(pool, layer, q_dev, q_stride, tok_off_dev, n_tokens, n_q_heads, block_table_dev,
                                 max_blocks, seq_len_dev, n_seq, causal, scale, out_dev, ws, ws_bytes, stream);
}
