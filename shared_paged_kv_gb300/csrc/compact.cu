// Eviction by accumulated attention weight: the choice of the tokens worth
// keeping and the compaction of the blocks that hold them.
//
// kvs_keep_heavy: of the tokens behind the first n_first and before the last
// n_recent of a sequence, those with the largest mass (ties: the lower index).
// A cluster of CTAs takes a sequence; the threshold is found by a radix select
// over the order-preserving bits of the masses, three digits of 11, 11 and 10
// bits, each CTA with the histogram of its own slice, added up through
// distributed shared memory.  Sixteen masses a thread stay in registers, so a
// sequence is read once (up to 131,072 tokens on eight CTAs).
//
// kvs_compact: row i of a sequence's kept tokens moves from place idx[i] to
// place i, in every layer's slabs.  Places only fall (idx[i] >= i), blocks in
// front of the first change stay, and a block that others reference is replaced
// by a free one.  Four launches:
//  cp_check  a CTA per sequence: the list's order, the first change, which
//            blocks have to be replaced;
//  cp_apply  a CTA per sequence: tables, counts, lengths, masses;
//  cp_move   the rows.  An item is 16 KB of one slab and head; its rows are all
//            in registers before any is written.  A row may be written in place
//            where another item still has to read: items publish that they have
//            read, and an item that writes in place waits for the (at most few)
//            items of lower places whose sources lie in its range.  Items are
//            claimed in order, so the awaited ones are running or done;
//  cp_push   one CTA: blocks that nobody references any more go back.
#include <algorithm>
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace kvs {

namespace {

// ------------------------------------------------------------ keep heavy ---
constexpr int kKhThreads = 1024;
constexpr int kKhKeys = 16;                     // masses a thread holds
constexpr int kKhTile = kKhThreads * kKhKeys;
constexpr int kKhBins = 2048;

struct KeepParams {
  const float* mass;
  const int32_t* seq_len;
  const int32_t* budget;
  int32_t* idx;
  int64_t* idx_off;
  uint32_t* status;
  int n_seq, most, n_first, n_recent;   // most: tokens a table row holds
};

struct KeepRange {
  int len, lo, hi, take;   // candidates [lo, hi), how many of them are kept
  __device__ int kept() const { return len - (hi - lo) + take; }
};

__device__ __forceinline__ KeepRange keep_range(const KeepParams& p, int a) {
  KeepRange r;
  r.len = min(max(__ldg(p.seq_len + a), 0), p.most);
  r.lo = min(p.n_first, r.len);
  r.hi = max(r.lo, r.len - p.n_recent);
  const int must = r.len - (r.hi - r.lo);
  r.take = min(max(__ldg(p.budget + a) - must, 0), r.hi - r.lo);
  return r;
}

// Unsigned keys in the order of the masses; -0 equals 0, NaN is below all.
__device__ __forceinline__ unsigned mass_key(float x) {
  x += 0.f;
  const unsigned b = __float_as_uint(x);
  return x != x ? 0u : (b >> 31 ? ~b : b | 0x80000000u);
}

__global__ void __launch_bounds__(kKhThreads) keep_heavy_kernel(const __grid_constant__ KeepParams p) {
  __shared__ unsigned hist[kKhBins];
  __shared__ int wsum[32];
  __shared__ long long wlong[32];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  __shared__ int2 s_count;                        // {above the threshold, equal to it} in this CTA's slice
  __shared__ int s_pair[kKhKeys * 32];            // per (round, warp) of a tile: taken tokens before it
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int a = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_enter();
  const KeepRange r = keep_range(p, a);
  // the kept tokens of the sequences before this one
  long long part = 0;
  for (int c = tid; c < a; c += kKhThreads) part += keep_range(p, c).kept();
#pragma unroll
  for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) wlong[warp] = part;
  __syncthreads();
  long long out0 = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) out0 += wlong[w];
  if (rank == 0 && tid == 0) {
    const int raw = p.seq_len[a];
    if (raw < 0 || raw > p.most) set_err(p.status, KVS_DEVERR_SEQ_LEN);
    p.idx_off[a] = out0;
    if (a == p.n_seq - 1) p.idx_off[p.n_seq] = out0 + r.kept();
  }
  int32_t* out = p.idx + out0;
  const int who = rank * kKhThreads + tid, all = ranks * kKhThreads;
  for (int t = who; t < r.lo; t += all) out[t] = t;
  for (int t = r.hi + who; t < r.len; t += all) out[r.lo + r.take + t - r.hi] = t;
  const int n = r.hi - r.lo;
  if (r.take == 0) return;                        // the same for the whole cluster
  if (r.take == n) {
    for (int t = who; t < n; t += all) out[r.lo + t] = r.lo + t;
    return;
  }
  const float* m = p.mass + (size_t)a * p.most + r.lo;
  // this CTA's slice of the candidates: whole rounds of the CTA's threads
  const int slice = ((n + ranks - 1) / ranks + kKhThreads - 1) / kKhThreads * kKhThreads;
  const int s0 = min(n, rank * slice), s1 = min(n, s0 + slice);
  unsigned key[kKhKeys];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kKhKeys; ++i) {
      const int t = t0 + i * kKhThreads + tid;
      key[i] = t < s1 ? mass_key(m[t]) : 0u;
    }
  };
  load(s0);
  unsigned prefix = 0, mask = 0;
  int left = r.take;
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bins = digit == 2 ? 1024 : 2048;
    for (int i = tid; i < bins; i += kKhThreads) hist[i] = 0;
    __syncthreads();
    for (int t0 = s0; t0 < s1; t0 += kKhTile) {
      if (t0 != s0 || (digit && s1 - s0 > kKhTile)) load(t0);
#pragma unroll
      for (int i = 0; i < kKhKeys; ++i)
        if (t0 + i * kKhThreads + tid < s1 && (key[i] & mask) == prefix) atomicAdd(&hist[(key[i] >> shift) & (bins - 1)], 1u);
    }
    cluster.sync();
    // the bin that holds the left-th largest: thread t takes the t-th largest
    // two bins (digit 2: one) of all CTAs' histograms
    const int per = bins / kKhThreads;
    unsigned c[2] = {0u, 0u};
    for (int q = 0; q < ranks; ++q) {
      const unsigned* h = cluster.map_shared_rank(hist, q);
      for (int j = 0; j < per; ++j) c[j] += h[bins - 1 - tid * per - j];
    }
    int total;
    const int mine = (int)(c[0] + c[1]);
    const int before = block_exclusive_scan(mine, wsum, total);
    if (before < left && left <= before + mine) {
      const int second = left > before + (int)c[0];
      s_prefix = prefix | ((unsigned)(bins - 1 - tid * per - second) << shift);
      s_left = left - before - (second ? (int)c[0] : 0);
    }
    cluster.sync();   // every CTA has read the histograms; s_prefix is there
    prefix = s_prefix;
    left = s_left;
    mask |= (unsigned)(bins - 1) << shift;
  }
  // left of the tokens equal to the threshold are kept, in order
  int gt = 0, eq = 0;
  for (int t0 = s0; t0 < s1; t0 += kKhTile) {
    if (t0 != s0 || s1 - s0 > kKhTile) load(t0);
#pragma unroll
    for (int i = 0; i < kKhKeys; ++i) {
      const bool in = t0 + i * kKhThreads + tid < s1;
      gt += in && key[i] > prefix;
      eq += in && key[i] == prefix;
    }
  }
  int gt_all, eq_all;
  block_exclusive_scan(gt, wsum, gt_all);
  block_exclusive_scan(eq, wsum, eq_all);
  if (tid == 0) s_count = make_int2(gt_all, eq_all);
  cluster.sync();
  int base = 0, eq_seen = 0;   // of the slices before this one
  for (int q = 0; q < rank; ++q) {
    const int2 v = *cluster.map_shared_rank(&s_count, q);
    base += v.x;
    eq_seen += v.y;
  }
  base += min(eq_seen, left);
  for (int t0 = s0; t0 < s1; t0 += kKhTile) {
    if (s1 - s0 > kKhTile) load(t0);
    // packed counts of a (round, warp): equal ones in the high half
#pragma unroll
    for (int i = 0; i < kKhKeys; ++i) {
      const bool in = t0 + i * kKhThreads + tid < s1;
      const unsigned g = __ballot_sync(0xffffffffu, in && key[i] > prefix), e = __ballot_sync(0xffffffffu, in && key[i] == prefix);
      if (lane == 0) s_pair[i * 32 + warp] = __popc(g) | (__popc(e) << 16);
    }
    __syncthreads();
    // a tile holds up to 16,384 of either: the two sums are scanned apart
    const int v = tid < kKhKeys * 32 ? s_pair[tid] : 0;
    int g_all, e_all;
    const int g_before = block_exclusive_scan(v & 0xffff, wsum, g_all);
    const int e_before = block_exclusive_scan(v >> 16, wsum, e_all);
    if (tid < kKhKeys * 32) s_pair[tid] = g_before | (e_before << 16);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKhKeys; ++i) {
      const int t = t0 + i * kKhThreads + tid;
      const bool in = t < s1;
      const unsigned g = __ballot_sync(0xffffffffu, in && key[i] > prefix), e = __ballot_sync(0xffffffffu, in && key[i] == prefix);
      const unsigned under = (1u << lane) - 1u;
      const int at = s_pair[i * 32 + warp];
      const int e_here = eq_seen + (at >> 16) + __popc(e & under);   // equal ones before this token
      const int g_here = (at & 0xffff) + __popc(g & under);
      // base counts the tokens taken before this tile
      const int pos = base + g_here + min(e_here, left) - min(eq_seen, left);
      if (in && (key[i] > prefix || (key[i] == prefix && e_here < left))) out[r.lo + pos] = r.lo + t;
    }
    base += g_all + min(eq_seen + e_all, left) - min(eq_seen, left);
    eq_seen += e_all;
    __syncthreads();
  }
  cluster.sync();   // s_count of this CTA has been read
}

// ---------------------------------------------------------------- compact ---
constexpr int kCpThreads = 128;
constexpr int kCpVecs = 8;                                  // 16-byte pieces a thread holds
constexpr int kCpCtas = 4;                                  // per SM
constexpr int kCpItem = kCpThreads * kCpVecs * 16;          // bytes of an item
constexpr int kCpMaxRows = 256;
constexpr int kCpSeqThreads = 1024;

struct __align__(16) CpSeq {
  int len, kept, start, need;   // start: first place that is written; need: blocks to take (-1: the sequence is left alone)
};

enum { kCpTicket, kCpSegs, kCpTaken, kCpHdr = 16 };

struct CompactParams {
  int32_t *table, *seq_len;
  const int32_t* idx;
  const int64_t* idx_off;
  float* mass;
  int32_t *refcount, *free_ids, *n_free;
  uint32_t* status;
  int* hdr;
  CpSeq* seq;
  int* segoff;             // [n_seq + 1] items' first segment of each sequence
  int32_t *old_tab, *new_tab;   // [n_seq][max_blocks]
  unsigned* freed;         // bitmap [capacity]
  uint8_t* flags;          // [segment][chain] 1: read
  void** slabs;
  long long max_flags;
  int n_seq, max_blocks, B, hkv, capacity, n_slabs, per_layer, row_bytes, sb_bytes, rows;   // rows: tokens of an item
};

struct CpLayout {
  size_t hdr, seq, segoff, old_tab, new_tab, freed, flags, total;
  long long max_flags;
};

int cp_rows(const kvs_pool_desc& d) {
  const int row = d.dtype == KVS_DTYPE_BF16 ? d.head_dim * 2 : d.head_dim / 2;
  return kCpItem / row;
}

CpLayout cp_layout(const kvs_pool* pool, int n_seq, int max_blocks) {
  const kvs_pool_desc& d = pool->desc;
  CpLayout l{};
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t{255};
    return at;
  };
  l.hdr = take(kCpHdr * 4);
  l.seq = take((size_t)n_seq * sizeof(CpSeq));
  l.segoff = take((size_t)(n_seq + 1) * 4);
  l.old_tab = take((size_t)n_seq * max_blocks * 4);
  l.new_tab = take((size_t)n_seq * max_blocks * 4);
  l.freed = take(((size_t)d.capacity_blocks + 31) / 32 * 4 + 16);
  // moved rows are written to blocks of one sequence each, so they fit the pool
  const long long rows = cp_rows(d);
  const long long by_pool = (long long)d.capacity_blocks * d.block_tokens / rows + n_seq;
  const long long by_table = (long long)n_seq * (((long long)max_blocks * d.block_tokens + rows - 1) / rows);
  l.max_flags = std::min(by_pool, by_table) * pool->n_blk_slabs * d.num_kv_heads;
  l.flags = take((size_t)l.max_flags);
  l.total = o;
  return l;
}

// A CTA per sequence.
__global__ void __launch_bounds__(kCpSeqThreads) cp_check(const __grid_constant__ CompactParams p) {
  __shared__ int s_same, s_bad;
  const int a = blockIdx.x, tid = threadIdx.x;
  pdl_enter();
  for (long long w = (long long)a * kCpSeqThreads + tid; w < (p.capacity + 31) / 32; w += (long long)p.n_seq * kCpSeqThreads)
    p.freed[w] = 0;
  const long long o0 = p.idx_off[a], o1 = p.idx_off[a + 1];
  const int len = p.seq_len[a];
  const bool ok = len >= 0 && len <= p.max_blocks * p.B && o0 >= 0 && o1 >= o0 && o1 - o0 <= len;
  const int kept = ok ? (int)(o1 - o0) : 0;
  if (tid == 0) {
    s_same = kept;
    s_bad = ok ? 0 : 1;
    if (!ok) set_err(p.status, len < 0 || len > p.max_blocks * p.B ? KVS_DEVERR_SEQ_LEN : KVS_DEVERR_JOB);
  }
  __syncthreads();
  const int32_t* idx = p.idx + o0;
  constexpr int U = 8;
  int same = kept;
  bool bad = false;
  for (int i0 = 0; i0 < kept; i0 += U * kCpSeqThreads) {
    int v[U], before[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kCpSeqThreads + tid;
      v[u] = i < kept ? idx[i] : i;
      before[u] = i < kept && i > 0 ? idx[i - 1] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kCpSeqThreads + tid;
      if (i >= kept) continue;
      bad |= v[u] <= before[u] || v[u] >= len;
      if (v[u] != i) same = min(same, i);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) same = min(same, __shfl_xor_sync(0xffffffffu, same, o));
  if ((tid & 31) == 0 && same < kept) atomicMin(&s_same, same);
  if (bad) s_bad = 1;
  __syncthreads();
  same = s_same;
  if (s_bad) {
    if (tid == 0) {
      if (ok) set_err(p.status, KVS_DEVERR_JOB);
      p.seq[a] = CpSeq{0, 0, 0, -1};
    }
    return;
  }
  const int nb_old = (len + p.B - 1) / p.B, nb_new = (kept + p.B - 1) / p.B;
  const int first = same < kept ? same / p.B : nb_new;   // first block that is written
  const size_t row = (size_t)a * p.max_blocks;
  int need = 0, start = same;
  bool wrong = false;
  for (int b = tid; b < nb_old; b += kCpSeqThreads) {
    const int id = p.table[row + b];
    const bool in = id >= 0 && id < p.capacity;
    wrong |= !in;
    const bool fresh = in && b >= first && b < nb_new && p.refcount[id] > 1;
    need += fresh;
    if (fresh && b == first) start = first * p.B;        // its unchanged rows move too
    p.old_tab[row + b] = id;
    p.new_tab[row + b] = b >= nb_new ? -1 : fresh ? -2 : id;
  }
  need = __reduce_add_sync(0xffffffffu, need);
  start = __reduce_min_sync(0xffffffffu, start);
  const int any_wrong = __syncthreads_or(wrong);
  if (tid == 0) {
    s_same = same;
    s_bad = 0;
  }
  __syncthreads();
  if ((tid & 31) == 0) {
    if (need) atomicAdd(&s_bad, need);
    atomicMin(&s_same, start);
  }
  __syncthreads();
  if (tid == 0) {
    if (any_wrong) set_err(p.status, KVS_DEVERR_BLOCK_ID);
    p.seq[a] = any_wrong ? CpSeq{0, 0, 0, -1} : CpSeq{len, kept, s_same, s_bad};
  }
}

__device__ __forceinline__ int cp_segments(const CompactParams& p, const CpSeq& s) {
  return s.need < 0 ? 0 : (s.kept - s.start + p.rows - 1) / p.rows;
}

// A CTA per sequence: every CTA adds up what the sequences before it take.
__global__ void __launch_bounds__(kCpSeqThreads) cp_apply(const __grid_constant__ CompactParams p) {
  __shared__ int warp_sums[32];
  __shared__ int s_base, s_seg, s_drop, s_taken;
  const int a = blockIdx.x, tid = threadIdx.x;
  pdl_enter();
  const CpSeq s = p.seq[a];
  const int avail = min(max(*p.n_free, 0), p.capacity);
  const int chains = p.n_slabs * p.hkv;
  {
    long long need = 0;
    int before = 0, segs = 0, bad = 0;
    for (int c = tid; c < p.n_seq; c += kCpSeqThreads) {
      const CpSeq q = p.seq[c];
      need += max(q.need, 0);
      if (c < a) {
        before += max(q.need, 0);
        segs += cp_segments(p, q);
      }
    }
    bad = __syncthreads_or(need > avail);   // one thread's sum alone
    int total, b0, g0;
    block_exclusive_scan((int)min(need, (long long)avail + 1), warp_sums, total);
    block_exclusive_scan(before, warp_sums, b0);
    block_exclusive_scan(segs, warp_sums, g0);
    if (tid == 0) {
      s_drop = s.need < 0;
      s_base = b0;
      s_seg = g0;
      s_taken = b0 + max(s.need, 0);
      if (bad || total > avail || total < 0) {
        // the stack is short: a sequence gets its blocks if those before it left enough
        int left = avail, seg = 0;
        for (int c = 0; c <= a; ++c) {
          const CpSeq q = p.seq[c];
          s_base = avail - left;
          s_seg = seg;
          if (c == a) s_drop = q.need < 0 || q.need > left;
          if (q.need >= 0 && q.need <= left) {
            left -= q.need;
            seg += cp_segments(p, q);
          }
        }
        s_taken = avail - left;
        if (s_drop && s.need >= 0) set_err(p.status, KVS_DEVERR_CAPACITY);
      }
    }
  }
  __syncthreads();
  const int base = s_base, seg0 = s_seg;
  const int segs = s_drop ? 0 : cp_segments(p, s);
  const bool fits = (long long)(seg0 + segs) * chains <= p.max_flags;   // counts that belong to no real pool
  if (tid == 0) {
    if (!fits) set_err(p.status, KVS_DEVERR_REFCOUNT);
    p.segoff[a] = seg0;
    if (a == p.n_seq - 1) {
      p.segoff[p.n_seq] = seg0 + segs;
      p.hdr[kCpSegs] = (int)min((long long)(seg0 + segs), p.max_flags / chains);
      p.hdr[kCpTaken] = s_taken;
      p.hdr[kCpTicket] = 0;
    }
  }
  if (s_drop) return;
  if (fits)
    for (long long i = (long long)seg0 * chains + tid; i < (long long)(seg0 + segs) * chains; i += kCpSeqThreads) p.flags[i] = 0;
  const int nb_old = (s.len + p.B - 1) / p.B;
  const size_t row = (size_t)a * p.max_blocks;
  int carry = base;
  for (int b0 = 0; b0 < nb_old; b0 += kCpSeqThreads) {
    const int b = b0 + tid;
    const int was = b < nb_old ? p.old_tab[row + b] : 0;
    int to = b < nb_old ? p.new_tab[row + b] : 0;
    int total;
    const int k = carry + block_exclusive_scan(to == -2, warp_sums, total);
    carry += total;
    if (b >= nb_old) continue;
    const bool fresh = to == -2;
    if (fresh) {
      to = p.free_ids[avail - 1 - k];
      if (to < 0 || to >= p.capacity) {   // a stack that holds no block: the row moves nowhere
        set_err(p.status, KVS_DEVERR_BLOCK_ID);
        to = -1;
      } else {
        p.refcount[to] = 1;
      }
      p.new_tab[row + b] = to;
    }
    if (to != was) {
      p.table[row + b] = to;
      const int before = atomicSub(p.refcount + was, 1);
      if (before == 1) atomicOr(p.freed + was / 32, 1u << (was % 32));
      if (before <= 0) set_err(p.status, KVS_DEVERR_REFCOUNT);
    }
  }
  if (tid == 0) p.seq_len[a] = s.kept;
  if (!p.mass) return;
  // masses: whole tiles are read before they are written (sources lie at or behind their places)
  float* m = p.mass + row * p.B;
  const int32_t* idx = p.idx + p.idx_off[a];
  constexpr int U = 8;
  for (int i0 = 0; i0 < s.kept; i0 += U * kCpSeqThreads) {
    int src[U];
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kCpSeqThreads + tid;
      src[u] = i < s.kept ? idx[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = src[u] >= 0 ? m[src[u]] : 0.f;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0) m[i0 + u * kCpSeqThreads + tid] = v[u];
  }
  __syncthreads();
  for (int i = s.kept + tid; i < s.len; i += kCpSeqThreads) m[i] = 0.f;
}

__device__ __forceinline__ int lower_bound(const int32_t* x, int n, int v) {   // first i with x[i] >= v
  int lo = 0;
  while (n > 0) {
    const int h = n >> 1;
    if (__ldg(x + lo + h) < v) {
      lo += h + 1;
      n -= h + 1;
    } else {
      n = h;
    }
  }
  return lo;
}

template <int VECS>   // VECS: 16-byte pieces of a row, 0: 4-byte words
__device__ __forceinline__ void cp_rows_move(const CompactParams& p, uint8_t* slab, int row_bytes, int n, const int* src, const int* dst,
                                             bool in_place, volatile uint8_t* flag, int wait0, int wait1, long long wait_at,
                                             int chains) {
  uint4 x[kCpVecs];
  if constexpr (VECS > 0) {
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / VECS;
      if (r < n && src[r] >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(slab + (size_t)src[r] * row_bytes) + v % VECS);
    }
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(x);
    const int words = row_bytes / 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / words;
      if (r < n && src[r] >= 0) w[k] = *(reinterpret_cast<const uint32_t*>(slab + (size_t)src[r] * row_bytes) + v % words);
    }
  }
  // every row of the item is read: said once the loads of all threads are done
  if (in_place) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) *flag = 1;
  }
  if (wait1 > wait0) {
    for (int s = wait0 + (int)threadIdx.x; s < wait1; s += kCpThreads) {
      volatile uint8_t* f = p.flags + wait_at + (long long)s * chains;
      const long long t0 = clock64();
      while (!*f) {
        if (clock64() - t0 > (1ll << 31)) {
          set_err(p.status, KVS_DEVERR_WAIT_TIMEOUT);
          break;
        }
      }
    }
    __threadfence();
    __syncthreads();
  }
  if constexpr (VECS > 0) {
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / VECS;
      if (r < n && dst[r] >= 0) *(reinterpret_cast<uint4*>(slab + (size_t)dst[r] * row_bytes) + v % VECS) = x[k];
    }
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
    const int words = row_bytes / 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / words;
      if (r < n && dst[r] >= 0) *(reinterpret_cast<uint32_t*>(slab + (size_t)dst[r] * row_bytes) + v % words) = w[k];
    }
  }
}

__global__ void __launch_bounds__(kCpThreads, kCpCtas) cp_move(const __grid_constant__ CompactParams p) {
  __shared__ int s_item, s_wait[2];
  __shared__ int s_src[kCpMaxRows], s_dst[kCpMaxRows];
  pdl_enter();
  const int chains = p.n_slabs * p.hkv, tid = threadIdx.x;
  const long long items = (long long)p.hdr[kCpSegs] * chains;
  while (true) {
    if (tid == 0) {
      s_item = atomicAdd(p.hdr + kCpTicket, 1);
      s_wait[0] = s_wait[1] = 0;
    }
    __syncthreads();
    const long long item = (unsigned)s_item;
    if (item >= items) return;
    const int sg = (int)(item / chains), chain = (int)(item - (long long)sg * chains);
    // the sequence: the last one whose first segment is at most sg
    int lo = 0, n = p.n_seq;
    while (n > 1) {
      const int h = n >> 1;
      if (p.segoff[lo + h] <= sg) {
        lo += h;
        n -= h;
      } else {
        n = h;
      }
    }
    const int a = lo, seg = sg - p.segoff[a];
    const CpSeq s = p.seq[a];
    const int32_t* idx = p.idx + p.idx_off[a];
    const size_t row = (size_t)a * p.max_blocks;
    const int i0 = s.start + seg * p.rows, m = min(p.rows, s.kept - i0);
    const int slab = chain / p.hkv, head = chain - slab * p.hkv;
    // nothing of a sequence is written in place where all its written blocks are new
    const bool in_place = s.need < (s.kept + p.B - 1) / p.B - s.start / p.B;
    for (int r = tid; r < m; r += kCpThreads) {
      const int from = __ldg(idx + i0 + r), to = i0 + r;
      const int sb = p.old_tab[row + from / p.B], db = p.new_tab[row + to / p.B];
      s_src[r] = (sb * p.hkv + head) * p.B + from % p.B;
      s_dst[r] = db >= 0 ? (db * p.hkv + head) * p.B + to % p.B : -1;
    }
    // rows of lower places whose sources this item overwrites
    __syncthreads();
    if (in_place && seg > 0) {
      if (tid < 2) s_wait[tid] = lower_bound(idx + s.start, i0 - s.start, tid ? i0 + m : i0);
      __syncthreads();
    }
    const int w0 = s_wait[0], w1 = s_wait[1];
    const int wait0 = w0 / p.rows, wait1 = w1 > w0 ? (w1 - 1) / p.rows + 1 : wait0;
    const long long wait_at = (long long)p.segoff[a] * chains + chain;
    uint8_t* base = static_cast<uint8_t*>(p.slabs[slab]);
    volatile uint8_t* flag = p.flags + item;
    if (slab % p.per_layer >= 2)
      cp_rows_move<0>(p, base, p.sb_bytes, m, s_src, s_dst, in_place, flag, wait0, wait1, wait_at, chains);
    else if (p.row_bytes == 256)
      cp_rows_move<16>(p, base, p.row_bytes, m, s_src, s_dst, in_place, flag, wait0, wait1, wait_at, chains);
    else if (p.row_bytes == 128)
      cp_rows_move<8>(p, base, p.row_bytes, m, s_src, s_dst, in_place, flag, wait0, wait1, wait_at, chains);
    else
      cp_rows_move<4>(p, base, p.row_bytes, m, s_src, s_dst, in_place, flag, wait0, wait1, wait_at, chains);
    __syncthreads();
  }
}

// One CTA: the blocks whose count reached zero go onto the stack, the smallest
// id on top.
__global__ void __launch_bounds__(kCpSeqThreads) cp_push(const __grid_constant__ CompactParams p) {
  __shared__ int warp_sums[32];
  pdl_enter();
  const int words = (p.capacity + 31) / 32, tid = threadIdx.x;
  const int per = (words + kCpSeqThreads - 1) / kCpSeqThreads;
  const int left = min(max(*p.n_free, 0), p.capacity) - p.hdr[kCpTaken];
  const int w1 = words - tid * per, w0 = max(0, w1 - per);   // this thread's words, from the highest down
  int n = 0, total;
#pragma unroll 4
  for (int w = w1 - 1; w >= w0; --w) n += __popc(p.freed[w]);
  int at = left + block_exclusive_scan(n, warp_sums, total);
  if (n)
    for (int w = w1 - 1; w >= w0; --w)
      for (unsigned bits = p.freed[w]; bits; ) {
        const int b = 31 - __clz(bits);
        bits &= ~(1u << b);
        if (at < p.capacity) p.free_ids[at] = w * 32 + b;
        else set_err(p.status, KVS_DEVERR_CAPACITY);
        ++at;
      }
  __syncthreads();
  if (tid == 0) *p.n_free = min(left + total, p.capacity);
}

}  // namespace

size_t compact_workspace_bytes(const kvs_pool* pool, int n_seq, int max_blocks) {
  return cp_layout(pool, n_seq, max_blocks).total;
}

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_keep_heavy(kvs_pool* pool, const float* mass_dev, const int32_t* seq_len_dev, int32_t n_seq,
                                     int32_t max_blocks, const int32_t* budget_dev, int32_t n_first, int32_t n_recent,
                                     int32_t* idx_out_dev, int64_t* idx_off_dev, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "keep_heavy: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (n_seq < 0 || max_blocks < 1 || n_first < 0 || n_recent < 0) return fail(KVS_ERR_INVALID_ARG, "keep_heavy: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "keep_heavy: n_seq exceeds the pool's max_seqs");
  const long long most = (long long)max_blocks * d.block_tokens;
  if (most > 0x40000000ll) return fail(KVS_ERR_CAPACITY, "keep_heavy: more than 2^30 tokens in a table row");
  if (n_seq == 0) return KVS_OK;
  if (!mass_dev || !seq_len_dev || !budget_dev || !idx_out_dev || !idx_off_dev)
    return fail(KVS_ERR_INVALID_ARG, "keep_heavy: null pointer");
  if (kvs_status st = check_pool_device(pool, "keep_heavy"); st != KVS_OK) return st;
  KeepParams p{mass_dev, seq_len_dev, budget_dev, idx_out_dev, idx_off_dev, pool->status, n_seq, (int)most, n_first, n_recent};
  // a CTA for every 4,096 tokens of the table row, eight at most
  int ranks = 1;
  while (ranks < 8 && most > 4096ll * ranks) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_seq * ranks);
  cfg.blockDim = dim3(kKhThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, keep_heavy_kernel, p) != cudaSuccess) return check_launch("keep_heavy");
  count_launch();
  return check_launch("keep_heavy");
}

extern "C" kvs_status kvs_compact(kvs_pool* pool, int32_t* block_table_dev, int32_t max_blocks, int32_t* seq_len_dev,
                                  int32_t n_seq, const int32_t* idx_dev, const int64_t* idx_off_dev, float* mass_dev,
                                  int32_t* refcount_dev, int32_t* free_ids_dev, int32_t* n_free_dev, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "compact: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (n_seq < 0 || max_blocks < 1) return fail(KVS_ERR_INVALID_ARG, "compact: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "compact: n_seq exceeds the pool's max_seqs");
  if ((long long)max_blocks * d.block_tokens > 0x40000000ll)
    return fail(KVS_ERR_CAPACITY, "compact: more than 2^30 tokens in a table row");
  if (n_seq == 0) return KVS_OK;
  if (!block_table_dev || !seq_len_dev || !idx_dev || !idx_off_dev || !refcount_dev || !free_ids_dev || !n_free_dev || !ws)
    return fail(KVS_ERR_INVALID_ARG, "compact: null pointer");
  if (!aligned16(ws)) return fail(KVS_ERR_INVALID_ARG, "compact: ws must be 16-byte aligned");
  const CpLayout l = cp_layout(pool, n_seq, max_blocks);
  if (ws_bytes < l.total) return fail(KVS_ERR_CAPACITY, "compact: workspace too small");
  if (kvs_status st = check_pool_device(pool, "compact"); st != KVS_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  CompactParams p{};
  p.table = block_table_dev;
  p.seq_len = seq_len_dev;
  p.idx = idx_dev;
  p.idx_off = idx_off_dev;
  p.mass = mass_dev;
  p.refcount = refcount_dev;
  p.free_ids = free_ids_dev;
  p.n_free = n_free_dev;
  p.status = pool->status;
  p.hdr = reinterpret_cast<int*>(w + l.hdr);
  p.seq = reinterpret_cast<CpSeq*>(w + l.seq);
  p.segoff = reinterpret_cast<int*>(w + l.segoff);
  p.old_tab = reinterpret_cast<int32_t*>(w + l.old_tab);
  p.new_tab = reinterpret_cast<int32_t*>(w + l.new_tab);
  p.freed = reinterpret_cast<unsigned*>(w + l.freed);
  p.flags = w + l.flags;
  p.slabs = pool->blk_slabs;
  p.max_flags = l.max_flags;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.B = d.block_tokens;
  p.hkv = d.num_kv_heads;
  p.capacity = d.capacity_blocks;
  p.n_slabs = pool->n_blk_slabs;
  p.per_layer = p.n_slabs / d.num_layers;
  p.row_bytes = d.dtype == KVS_DTYPE_BF16 ? d.head_dim * 2 : d.head_dim / 2;
  p.sb_bytes = d.dtype == KVS_DTYPE_Q4G64 ? d.head_dim / 16 : d.head_dim / 32;
  p.rows = cp_rows(d);
  const long long chains = (long long)p.n_slabs * p.hkv;
  if (chains > 0x7fffffffll / 2) return fail(KVS_ERR_UNSUPPORTED, "compact: too many layers and heads");
  const unsigned grid = (unsigned)std::max(1ll, std::min(p.max_flags, (long long)pool->num_sms * 8));
  const bool ok = launch_pdl(cp_check, dim3(n_seq), dim3(kCpSeqThreads), stream, p) == cudaSuccess &&
                  launch_pdl(cp_apply, dim3(n_seq), dim3(kCpSeqThreads), stream, p) == cudaSuccess &&
                  launch_pdl(cp_move, dim3(grid), dim3(kCpThreads), stream, p) == cudaSuccess &&
                  launch_pdl(cp_push, dim3(1), dim3(kCpSeqThreads), stream, p) == cudaSuccess;
  if (ok) count_launch(4);
  return check_launch("compact");
}
