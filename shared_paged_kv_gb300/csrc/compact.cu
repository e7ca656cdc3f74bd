// Eviction by accumulated attention weight: the choice of the tokens worth
// keeping and the compaction of the blocks that hold them.
//
// kvs_keep_heavy: of the tokens behind the first n_first and before the last
// n_recent of a sequence, those with the largest mass (ties: the lower index).
// A cluster of CTAs takes a sequence; the threshold is found by a radix select
// over the order-preserving bits of the masses, three digits of 11, 11 and 10
// bits, each CTA with the histogram of its own slice, added up through
// distributed shared memory.  A thread's masses stay in registers, so a sequence is
// read once (up to 131,072 tokens on eight CTAs).  131,072 tokens: 25 us, a chain of
// loads (5), for each digit a histogram, an exchange and a scan, and the writing in
// order (6); 32 sequences of 6,144 tokens: 9 us.
//
// kvs_compact: row i of a sequence's kept tokens moves from place idx[i] to
// place i, in every layer's slabs.  Places only fall (idx[i] >= i), blocks in
// front of the first change stay, and a block that others reference is replaced
// by a free one.  Three launches (two for few short sequences):
//  cp_check  a CTA per sequence: the list's order, the first change, which
//            blocks have to be replaced;
//  cp_apply  a CTA per sequence: tables, counts, lengths, masses;
//  cp_move   the rows.  An item is the next 16 KB of places of a sequence, looked
//            up once, in some chains (a layer's K or V of one head) one after the
//            other; a chain's rows are all in registers before any is written,
//            and the next chain's are under way meanwhile.  A row may be written
//            in place where another item still has to read: items publish
//            that they have read, and an item that writes in place waits for
//            the (at most few) items of lower places whose sources lie in its
//            range.  Items are claimed in order, so the awaited ones are running
//            or done.  The last CTA puts the blocks that nobody references any
//            more onto the free stack.
// Bound by HBM where rows are long (32 sequences, 4 layers of 256-byte rows: 473 MB in
// 88 us, 5.4 TB/s), by a chain's two trips to memory and its barriers where they
// are 64 bytes and lie apart (one sequence of 131,072 tokens in 4 bits, 8 layers: 581
// MB in 124 us); small calls by the three launches' chains (4 sequences of some hundred
// tokens: 14 us with the choice).  These are copies into new blocks; in place the flags
// and waits come on top (32 sequences, the whole eviction: 253 us instead of 114).
#include <algorithm>
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace kvs {

namespace {

// ------------------------------------------------------------ keep heavy ---
constexpr int kKhThreads = 1024;
constexpr int kKhBins = 2048;
// Masses gather in few of the first digit's bins: four histograms, a lane in one
// of them, eight banks apart.
constexpr int kKhCopies = 4, kKhStride = kKhBins + 8;

struct KeepParams {
  const float* mass;
  const int32_t* seq_len;
  const int32_t* budget;
  int32_t* idx;
  int64_t* idx_off;
  uint32_t* status;
  long long cap;                        // entries of idx
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

// RANKS CTAs take a sequence, a thread holds KEYS masses at a time.
template <int RANKS, int KEYS>
__global__ void __launch_bounds__(kKhThreads) keep_heavy_kernel(const __grid_constant__ KeepParams p) {
  __shared__ unsigned hist4[kKhCopies * kKhStride];
  __shared__ __align__(8) unsigned hist[kKhBins];
  __shared__ int wsum[32];
  __shared__ long long wlong[32];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  __shared__ int2 s_count;                        // {above the threshold, equal to it} in this CTA's slice
  __shared__ int s_pair[KEYS * 32];            // per (round, warp) of a tile: taken tokens before it
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int ranks = RANKS, kKhKeys = KEYS, kKhTile = kKhThreads * KEYS;
  const int rank = RANKS > 1 ? (int)cluster.block_rank() : 0;
  auto sync_all = [&]() {
    if constexpr (RANKS > 1) cluster.sync();
    else __syncthreads();
  };
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
    if (out0 + r.kept() > p.cap) set_err(p.status, KVS_DEVERR_CAPACITY);
  }
  if (out0 + r.kept() > p.cap) return;            // the same for the whole cluster
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
    for (int i = tid; i < kKhCopies * kKhStride; i += kKhThreads) hist4[i] = 0;
    __syncthreads();
    unsigned* mine4 = hist4 + (tid % kKhCopies) * kKhStride;
    for (int t0 = s0; t0 < s1; t0 += kKhTile) {
      if (t0 != s0 || (digit && s1 - s0 > kKhTile)) load(t0);
#pragma unroll
      for (int i = 0; i < kKhKeys; ++i)
        if (t0 + i * kKhThreads + tid < s1 && (key[i] & mask) == prefix) atomicAdd(&mine4[(key[i] >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    for (int i = tid; i < bins; i += kKhThreads) {
      unsigned n = 0;
#pragma unroll
      for (int c = 0; c < kKhCopies; ++c) n += hist4[c * kKhStride + i];
      hist[i] = n;
    }
    sync_all();
    // the bin that holds the left-th largest: thread t takes the t-th largest
    // two bins (digit 2: one) of all CTAs' histograms
    const int per = bins / kKhThreads;
    unsigned c[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < ranks; ++q) {
      const unsigned* h = RANKS > 1 ? cluster.map_shared_rank(hist, q) : hist;
      if (per > 1) {   // a pair as one load: distributed shared memory takes its time by the load
        const uint2 v = reinterpret_cast<const uint2*>(h)[bins / 2 - 1 - tid];
        c[0] += v.y;
        c[1] += v.x;
      } else {
        c[0] += h[bins - 1 - tid];
      }
    }
    int total;
    const int mine = (int)(c[0] + c[1]);
    const int before = block_exclusive_scan(mine, wsum, total);
    if (before < left && left <= before + mine) {
      const int second = left > before + (int)c[0];
      s_prefix = prefix | ((unsigned)(bins - 1 - tid * per - second) << shift);
      s_left = left - before - (second ? (int)c[0] : 0);
    }
    sync_all();   // every CTA has read the histograms; s_prefix is there
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
  int base = 0, eq_seen = 0;   // of the slices before this one
  if constexpr (RANKS > 1) {
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (tid == 0) s_count = make_int2(0, 0);
    __syncthreads();
    if (lane == 0) {
      if (gt) atomicAdd(&s_count.x, gt);
      if (eq) atomicAdd(&s_count.y, eq);
    }
    cluster.sync();
    for (int q = 0; q < rank; ++q) {
      const int2 v = *cluster.map_shared_rank(&s_count, q);
      base += v.x;
      eq_seen += v.y;
    }
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
    // a tile holds up to 16,384 of either, so both sums fit half a word
    int all;
    const int before = block_exclusive_scan(tid < kKhKeys * 32 ? s_pair[tid] : 0, wsum, all);
    const int g_all = all & 0xffff, e_all = all >> 16;
    if (tid < kKhKeys * 32) s_pair[tid] = before;
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
  if constexpr (RANKS > 1) cluster.sync();   // s_count of this CTA has been read
}

// ---------------------------------------------------------------- compact ---
constexpr int kCpThreads = 128;
constexpr int kCpVecs = 8;                                  // 16-byte pieces a thread holds
constexpr int kCpCtas = 5;                                  // per SM
constexpr int kCpItemsPerSm = 16, kCpMaxGroup = 16;
constexpr int kCpItem = kCpThreads * kCpVecs * 16;          // bytes of an item
constexpr int kCpMaxRows = 256;
constexpr int kCpSeqThreads = 1024;

struct __align__(16) CpSeq {
  int len, kept, start, need;   // start: first place that is written; need: blocks to take (-1: the sequence is left alone)
};

// A segment: the next `rows` places of a sequence, as the moving kernel reads it.
struct __align__(16) CpSeg {
  int seq, i0, n, start;   // places i0 .. i0 + n; start: the sequence's first (-1 - start: all its written blocks are new)
  long long idx0;          // where its list begins
  int first, pad;          // the sequence's first segment
};

enum { kCpTicket, kCpSegs, kCpTaken, kCpDone, kCpGroup, kCpHdr = 16 };

struct CompactParams {
  int32_t *table, *seq_len;
  const int32_t* idx;
  const int64_t* idx_off;
  long long idx_cap;       // entries of idx
  float* mass;
  int32_t *refcount, *free_ids, *n_free;
  uint32_t* status;
  int* hdr;
  CpSeq* seq;
  CpSeg* segs;
  float* mass_was;         // [n_seq][max_blocks * B] masses before the call
  int32_t *old_tab, *new_tab;   // [n_seq][max_blocks]
  unsigned* freed;         // bitmap [capacity]
  uint8_t* flags;          // [segment][chain] 1: read
  void** slabs;
  long long max_segs;
  int n_seq, max_blocks, B, hkv, capacity, chains, per_layer, row_bytes, sb_bytes, rows;   // chain: a layer's K or V of one head
  int sms;
  int stall_first;         // test-only (KVS_TEST_STALL_COMPACT): the first item does not say that it has read its first chain
};

struct CpLayout {
  size_t hdr, seq, segs, mass, old_tab, new_tab, freed, flags, total;
  long long max_segs;
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
  l.mass = take((size_t)n_seq * max_blocks * d.block_tokens * 4);
  l.old_tab = take((size_t)n_seq * max_blocks * 4);
  l.new_tab = take((size_t)n_seq * max_blocks * 4);
  l.freed = take(((size_t)d.capacity_blocks + 31) / 32 * 4 + 16);
  // moved rows are written to blocks of one sequence each, so they fit the pool
  const long long rows = cp_rows(d);
  const long long by_pool = (long long)d.capacity_blocks * d.block_tokens / rows + n_seq;
  const long long by_table = (long long)n_seq * (((long long)max_blocks * d.block_tokens + rows - 1) / rows);
  l.max_segs = std::min(by_pool, by_table);
  l.segs = take((size_t)l.max_segs * sizeof(CpSeg));
  l.flags = take((size_t)l.max_segs * 2 * d.num_layers * d.num_kv_heads);
  l.total = o;
  return l;
}

// gridDim.y CTAs take the masses of a sequence, each its share of [0, n).
__device__ __forceinline__ int2 cp_share(int n) {
  const int per = ((n + (int)gridDim.y - 1) / (int)gridDim.y + 3) & ~3;
  return make_int2(min(n, (int)blockIdx.y * per), min(n, ((int)blockIdx.y + 1) * per));
}

// A CTA per sequence, and some more to copy long rows of masses.
__device__ __forceinline__ void check_sequence(const CompactParams& p) {
  __shared__ int s_same, s_bad;
  const int a = blockIdx.x, tid = threadIdx.x;
  for (long long w = (long long)(blockIdx.y * p.n_seq + a) * kCpSeqThreads + tid; w < (p.capacity + 31) / 32;
       w += (long long)p.n_seq * gridDim.y * kCpSeqThreads)
    p.freed[w] = 0;
  if (p.mass) {
    const int2 mine = cp_share(min(max(p.seq_len[a], 0), p.max_blocks * p.B));
    const float* from = p.mass + (size_t)a * p.max_blocks * p.B;
    float* to = p.mass_was + (size_t)a * p.max_blocks * p.B;
#pragma unroll 8
    for (int i = mine.x + tid; i < mine.y; i += kCpSeqThreads) to[i] = from[i];
  }
  if (blockIdx.y > 0) return;
  const long long o0 = p.idx_off[a], o1 = p.idx_off[a + 1];
  const int len = p.seq_len[a];
  const bool ok = len >= 0 && len <= p.max_blocks * p.B && o0 >= 0 && o1 >= o0 && o1 - o0 <= len && o1 <= p.idx_cap;
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

__device__ __forceinline__ int cp_moved(const CpSeq& s) { return s.need < 0 ? 0 : s.kept - s.start; }   // rows
__device__ __forceinline__ int cp_segments(const CompactParams& p, const CpSeq& s) { return (cp_moved(s) + p.rows - 1) / p.rows; }

// The sum over the CTA's threads, in 64 bits; *total is 0 before and read after it.
__device__ __forceinline__ void cp_add_up(long long x, unsigned long long* total) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0 && x) atomicAdd(total, (unsigned long long)x);
}

// A CTA per sequence (and some more for long rows of masses): every CTA adds up
// what the sequences before it take.
__device__ __forceinline__ void apply_sequence(const CompactParams& p) {
  __shared__ int warp_sums[32];
  __shared__ unsigned long long s_need, s_moved;
  __shared__ int s_base, s_seg, s_drop, s_taken;
  const int a = blockIdx.x, tid = threadIdx.x;
  const CpSeq s = p.seq[a];
  const int avail = min(max(*p.n_free, 0), p.capacity);
  if (tid == 0) s_need = s_moved = 0;
  __syncthreads();
  {
    long long need = 0, moved = 0;
    int before = 0, segs = 0;
    for (int c = tid; c < p.n_seq; c += kCpSeqThreads) {
      const CpSeq q = p.seq[c];
      need += max(q.need, 0);
      moved += cp_moved(q);
      if (c < a) {
        before += max(q.need, 0);
        segs += cp_segments(p, q);
      }
    }
    cp_add_up(need, &s_need);
    cp_add_up(moved, &s_moved);
    int b0, g0;
    block_exclusive_scan(before, warp_sums, b0);
    block_exclusive_scan(segs, warp_sums, g0);
    if (tid == 0) {
      s_drop = s.need < 0;
      s_base = b0;
      s_seg = g0;
      s_taken = b0 + max(s.need, 0);
      const long long room = (long long)p.capacity * p.B;   // what a pool holds, and the segments are laid out for
      if (s_need > (unsigned long long)avail || s_moved > (unsigned long long)room) {
        // The stack is short, or more rows are to be written than there are (a block of two
        // sequences that is counted once): a sequence is served if those before it left
        // enough of both.
        int left = avail, seg = 0;
        long long rows = room;
        for (int c = 0; c <= a; ++c) {
          const CpSeq q = p.seq[c];
          const bool blocks = q.need <= left, fits = blocks && cp_moved(q) <= rows;
          if (c == a) {
            s_base = avail - left;
            s_seg = seg;
            s_drop = q.need < 0 || !fits;
            if (q.need >= 0 && !fits) set_err(p.status, blocks ? KVS_DEVERR_REFCOUNT : KVS_DEVERR_CAPACITY);
          }
          if (q.need >= 0 && fits) {
            left -= q.need;
            rows -= cp_moved(q);
            seg += cp_segments(p, q);
          }
        }
        s_taken = avail - left;
      }
    }
  }
  __syncthreads();
  const int base = s_base, seg0 = s_seg;
  const int segs = s_drop ? 0 : cp_segments(p, s);
  if (tid == 0 && blockIdx.y == 0 && a == p.n_seq - 1) {
    const int total = seg0 + segs;   // all of them are written below
    p.hdr[kCpSegs] = total;
    p.hdr[kCpTaken] = s_taken;
    p.hdr[kCpTicket] = p.hdr[kCpDone] = 0;
    // chains that an item takes one after the other: its places are looked up
    // once; as many as leave sixteen items to an SM
    const long long items = (long long)total * p.chains;
    p.hdr[kCpGroup] = (int)min(max(items / (kCpItemsPerSm * (long long)p.sms), 1ll), (long long)kCpMaxGroup);
  }
  if (s_drop) return;
  const size_t row = (size_t)a * p.max_blocks;
  if (p.mass) {   // list and lengths are those that cp_check read
    const int32_t* idx = p.idx + p.idx_off[a];
    const float* from = p.mass_was + row * p.B;
    float* to = p.mass + row * p.B;
    const int2 mine = cp_share(s.len);
#pragma unroll 8
    for (int i = mine.x + tid; i < mine.y; i += kCpSeqThreads) to[i] = i < s.kept ? from[idx[i]] : 0.f;
  }
  if (blockIdx.y > 0) return;
  const long long idx0 = p.idx_off[a];
  const int all_new = s.need == (s.kept + p.B - 1) / p.B - s.start / p.B;
  for (int i = tid; i < segs; i += kCpSeqThreads) {
    const int i0 = s.start + i * p.rows;
    p.segs[seg0 + i] = CpSeg{a, i0, min(p.rows, s.kept - i0), all_new ? -1 - s.start : s.start, idx0, seg0, 0};
  }
  if (!all_new)
    for (long long i = (long long)seg0 * p.chains + tid; i < (long long)(seg0 + segs) * p.chains; i += kCpSeqThreads) p.flags[i] = 0;
  const int nb_old = (s.len + p.B - 1) / p.B;
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
}

__global__ void __launch_bounds__(kCpSeqThreads) cp_check(const __grid_constant__ CompactParams p) {
  pdl_enter();
  check_sequence(p);
}

__global__ void __launch_bounds__(kCpSeqThreads) cp_apply(const __grid_constant__ CompactParams p) {
  pdl_enter();
  apply_sequence(p);
}

// Both, by one cluster: up to eight sequences with short rows of masses (four of some
// hundred tokens: the choice and this call take the host 18 us, 21.5 with two
// launches; in a graph they take the same).
constexpr int kCpCluster = 8;
__global__ void __cluster_dims__(kCpCluster) __launch_bounds__(kCpSeqThreads) cp_both(const __grid_constant__ CompactParams p) {
  pdl_enter();
  const bool there = (int)blockIdx.x < p.n_seq;
  if (there) check_sequence(p);
  __threadfence();
  cg::this_cluster().sync();
  if (there) apply_sequence(p);
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

// Kept rows lie apart, and 4-bit ones are 64 bytes: L2 fetches no more than that
// (one sequence of 131,072 tokens, 32,768 kept: 336 MB read instead of 519, the whole
// eviction 193 -> 177 us then).
__device__ __forceinline__ uint4 load_row(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_row(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.L2::64B.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ bool flag_set(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v != 0;
}

// 16-byte pieces of an item's rows: thread v of the k-th hundred and twenty-eight
// has piece v % VECS of row v / VECS.
template <int VECS>
struct CpRows {
  uint4 x[kCpVecs];
  __device__ __forceinline__ void load(const uint8_t* slab, int n, const int* src, int at) {
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / VECS;
      x[k] = r < n ? load_row(reinterpret_cast<const uint4*>(slab + (size_t)(src[r] + at) * (VECS * 16)) + v % VECS) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ uint32_t any() const {
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) a |= x[k].x | x[k].y | x[k].z | x[k].w;
    return a;
  }
  __device__ __forceinline__ void store(uint8_t* slab, int n, const int* dst, int at) const {
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) {
      const int v = k * kCpThreads + threadIdx.x, r = v / VECS;
      if (r < n && dst[r] >= 0) *(reinterpret_cast<uint4*>(slab + (size_t)(dst[r] + at) * (VECS * 16)) + v % VECS) = x[k];
    }
  }
};

// The free stack of the call's end (by one CTA): the blocks whose count reached
// zero go onto it, the smallest id on top.
__device__ __forceinline__ void cp_push(const CompactParams& p, int* warp_sums) {
  const int words = (p.capacity + 31) / 32, tid = threadIdx.x;
  const int per = (words + kCpThreads - 1) / kCpThreads;
  const int left = min(max(*p.n_free, 0), p.capacity) - p.hdr[kCpTaken];
  const int w1 = words - tid * per, w0 = max(0, w1 - per);   // this thread's words, from the highest down
  int n = 0, total;
#pragma unroll 8
  for (int w = w1 - 1; w >= w0; --w) n += __popc(__ldcg(p.freed + w));
  int at = left + block_exclusive_scan(n, warp_sums, total);
  if (n)
    for (int w = w1 - 1; w >= w0; --w)
      for (unsigned bits = __ldcg(p.freed + w); bits; ) {
        const int b = 31 - __clz(bits);
        bits &= ~(1u << b);
        if (at < p.capacity) p.free_ids[at] = w * 32 + b;
        else set_err(p.status, KVS_DEVERR_CAPACITY);
        ++at;
      }
  __syncthreads();
  if (tid == 0) *p.n_free = min(left + total, p.capacity);
}

template <int VECS>
__global__ void __launch_bounds__(kCpThreads, kCpCtas) cp_move(const __grid_constant__ CompactParams p) {
  __shared__ int s_item, s_wait[2], s_last;
  __shared__ int warp_sums[32];
  __shared__ int s_src[kCpMaxRows], s_dst[kCpMaxRows];
  const int tid = threadIdx.x;
  pdl_enter();
  const int group = p.hdr[kCpGroup], n_groups = (p.chains + group - 1) / group;
  const long long items = (long long)p.hdr[kCpSegs] * n_groups;
  long long item = 0;
  int ticket = 0;
  if (tid == 0) ticket = atomicAdd(p.hdr + kCpTicket, 1);
  while (true) {
    if (tid == 0) s_item = ticket;
    __syncthreads();
    item = (unsigned)s_item;
    if (item >= items) break;
    if (tid == 0) ticket = atomicAdd(p.hdr + kCpTicket, 1);   // the next one, known when this one is done
    const int sg = (int)(item / n_groups), c0 = (int)(item - (long long)sg * n_groups) * group;
    const CpSeg s = p.segs[sg];
    const int32_t* idx = p.idx + s.idx0;
    const size_t row = (size_t)s.seq * p.max_blocks;
    const bool in_place = s.start >= 0;
    for (int r = tid; r < s.n; r += kCpThreads) {
      const int from = __ldg(idx + s.i0 + r), to = s.i0 + r;
      const int sb = p.old_tab[row + from / p.B], db = p.new_tab[row + to / p.B];
      s_src[r] = sb * p.hkv * p.B + from % p.B;
      s_dst[r] = db >= 0 ? db * p.hkv * p.B + to % p.B : -p.hkv * p.B;
    }
    // rows of lower places whose sources this item overwrites
    int wait0 = 0, wait1 = 0;
    if (in_place && s.i0 > s.start) {
      if (tid < 2) s_wait[tid] = lower_bound(idx + s.start, s.i0 - s.start, tid ? s.i0 + s.n : s.i0);
      __syncthreads();
      wait0 = s_wait[0] / p.rows;
      wait1 = s_wait[1] > s_wait[0] ? (s_wait[1] - 1) / p.rows + 1 : wait0;
    }
    __syncthreads();
    const int c1 = min(p.chains, c0 + group);
    auto slab_of = [&](int c, int more) {
      const int kv = c / p.hkv;
      return static_cast<uint8_t*>(p.slabs[(kv >> 1) * p.per_layer + (kv & 1) + more]);
    };
    // chain c, whose rows are under way into x; those of the next one go into y
    auto step = [&](CpRows<VECS>& x, CpRows<VECS>& y, int c) {
      const int at = c % p.hkv * p.B;
      // a 4-bit row's scales go along, as words
      uint32_t w[4] = {};
      const int words = p.sb_bytes / 4;   // 0, 1 or 2
      if (VECS == 4) {
        const uint8_t* slab = slab_of(c, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int v = k * kCpThreads + tid, r = v / words;
          if (r < s.n) w[k] = load_row(reinterpret_cast<const uint32_t*>(slab + (size_t)(s_src[r] + at) * p.sb_bytes) + v % words);
        }
      }
      auto next = [&]() {
        if (c + 1 < c1) y.load(slab_of(c + 1, 0), s.n, s_src, (c + 1) % p.hkv * p.B);
      };
      int n = s.n;
      if (in_place) {
        // Every row of this chain is read: said once the loads of all threads have
        // returned, which the barrier's predicate needs.
        uint32_t any = x.any();
        if (VECS == 4) any |= w[0] | w[1] | w[2] | w[3];
        __syncthreads_or(any == 1u);
        if (tid == 0 && !(p.stall_first && sg == 0 && c == 0)) {
          __threadfence();
          *const_cast<volatile uint8_t*>(p.flags + (size_t)sg * p.chains + c) = 1;
        }
        next();   // on their way while this chain waits and is written
        bool late = false;
        for (int q = wait0 + tid; q < wait1; q += kCpThreads) {
          const uint8_t* f = p.flags + (size_t)(s.first + q) * p.chains + c;
          const long long t0 = clock64();
          while (!flag_set(f)) {
            if (clock64() - t0 > (1ll << 31)) {
              set_err(p.status, KVS_DEVERR_WAIT_TIMEOUT);
              late = true;
              break;
            }
          }
        }
        if (__syncthreads_or(late)) n = 0;   // rows that others still have to read are not written over
      } else {
        next();
      }
      x.store(slab_of(c, 0), n, s_dst, at);
      if (VECS == 4) {
        uint8_t* slab = slab_of(c, 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int v = k * kCpThreads + tid, r = v / words;
          if (r < n && s_dst[r] >= 0) *(reinterpret_cast<uint32_t*>(slab + (size_t)(s_dst[r] + at) * p.sb_bytes) + v % words) = w[k];
        }
      }
    };
    CpRows<VECS> x, y;
    x.load(slab_of(c0, 0), s.n, s_src, c0 % p.hkv * p.B);
    for (int c = c0; c < c1; c += 2) {
      step(x, y, c);
      if (c + 1 < c1) step(y, x, c + 1);
    }
    __syncthreads();
  }
  // the last CTA to find nothing left brings the free stack up to date: blocks
  // that are given up are read by now
  __threadfence();
  if (tid == 0) s_last = atomicAdd(p.hdr + kCpDone, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (s_last) cp_push(p, warp_sums);
}

}  // namespace

size_t compact_workspace_bytes(const kvs_pool* pool, int n_seq, int max_blocks) {
  return cp_layout(pool, n_seq, max_blocks).total;
}

}  // namespace kvs

using namespace kvs;

extern "C" kvs_status kvs_keep_heavy_bounded(kvs_pool* pool, const float* mass_dev, const int32_t* seq_len_dev, int32_t n_seq,
                                             int32_t max_blocks, const int32_t* budget_dev, int32_t n_first, int32_t n_recent,
                                             int32_t* idx_out_dev, int64_t idx_capacity, int64_t* idx_off_dev, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "keep_heavy: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (n_seq < 0 || max_blocks < 1 || n_first < 0 || n_recent < 0 || idx_capacity < 0)
    return fail(KVS_ERR_INVALID_ARG, "keep_heavy: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "keep_heavy: n_seq exceeds the pool's max_seqs");
  const long long most = (long long)max_blocks * d.block_tokens;
  if (most > 0x40000000ll) return fail(KVS_ERR_CAPACITY, "keep_heavy: more than 2^30 tokens in a table row");
  if (n_seq == 0) return KVS_OK;
  if (!mass_dev || !seq_len_dev || !budget_dev || (!idx_out_dev && idx_capacity > 0) || !idx_off_dev)
    return fail(KVS_ERR_INVALID_ARG, "keep_heavy: null pointer");
  if (kvs_status st = check_pool_device(pool, "keep_heavy"); st != KVS_OK) return st;
  KeepParams p{mass_dev, seq_len_dev, budget_dev, idx_out_dev, idx_off_dev, pool->status, idx_capacity, n_seq, (int)most, n_first, n_recent};
  // Few CTAs with their masses in registers: exchanges between CTAs cost more than
  // longer slices.  (32 sequences of 6,144 tokens: one CTA 9.4 us, two 11.1; 16 of
  // 32,000: four 15.9, eight, which no longer are resident together, 44; one of 65,000:
  // four with sixteen masses a thread 20.2, eight 23.2; but one of 16,000: two 13.5,
  // four 12.7.)
  const int ranks = most <= 8192 ? 1 : most <= 16384 ? 2 : most <= 65536 ? 4 : 8;
  auto kern = most <= 4096    ? keep_heavy_kernel<1, 4>
              : most <= 8192  ? keep_heavy_kernel<1, 8>
              : most <= 16384 ? keep_heavy_kernel<2, 8>
              : most <= 32768 ? keep_heavy_kernel<4, 8>
              : most <= 65536 ? keep_heavy_kernel<4, 16>
                              : keep_heavy_kernel<8, 16>;
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
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return check_launch("keep_heavy");
  count_launch();
  return check_launch("keep_heavy");
}

extern "C" kvs_status kvs_keep_heavy(kvs_pool* pool, const float* mass_dev, const int32_t* seq_len_dev, int32_t n_seq,
                                     int32_t max_blocks, const int32_t* budget_dev, int32_t n_first, int32_t n_recent,
                                     int32_t* idx_out_dev, int64_t* idx_off_dev, cudaStream_t stream) {
  return kvs_keep_heavy_bounded(pool, mass_dev, seq_len_dev, n_seq, max_blocks, budget_dev, n_first, n_recent, idx_out_dev,
                                INT64_MAX, idx_off_dev, stream);
}

extern "C" kvs_status kvs_compact_bounded(kvs_pool* pool, int32_t* block_table_dev, int32_t max_blocks, int32_t* seq_len_dev,
                                          int32_t n_seq, const int32_t* idx_dev, int64_t idx_capacity, const int64_t* idx_off_dev,
                                          float* mass_dev, int32_t* refcount_dev, int32_t* free_ids_dev, int32_t* n_free_dev,
                                          void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!pool) return fail(KVS_ERR_INVALID_ARG, "compact: null pool");
  const kvs_pool_desc& d = pool->desc;
  if (n_seq < 0 || max_blocks < 1 || idx_capacity < 0) return fail(KVS_ERR_INVALID_ARG, "compact: bad sizes");
  if (n_seq > d.max_seqs) return fail(KVS_ERR_CAPACITY, "compact: n_seq exceeds the pool's max_seqs");
  if ((long long)max_blocks * d.block_tokens > 0x40000000ll)
    return fail(KVS_ERR_CAPACITY, "compact: more than 2^30 tokens in a table row");
  if (n_seq == 0) return KVS_OK;
  if (!block_table_dev || !seq_len_dev || (!idx_dev && idx_capacity > 0) || !idx_off_dev || !refcount_dev || !free_ids_dev ||
      !n_free_dev || !ws)
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
  p.idx_cap = idx_capacity;
  p.mass = mass_dev;
  p.refcount = refcount_dev;
  p.free_ids = free_ids_dev;
  p.n_free = n_free_dev;
  p.status = pool->status;
  p.hdr = reinterpret_cast<int*>(w + l.hdr);
  p.seq = reinterpret_cast<CpSeq*>(w + l.seq);
  p.segs = reinterpret_cast<CpSeg*>(w + l.segs);
  p.mass_was = reinterpret_cast<float*>(w + l.mass);
  p.old_tab = reinterpret_cast<int32_t*>(w + l.old_tab);
  p.new_tab = reinterpret_cast<int32_t*>(w + l.new_tab);
  p.freed = reinterpret_cast<unsigned*>(w + l.freed);
  p.flags = w + l.flags;
  p.slabs = pool->blk_slabs;
  p.max_segs = l.max_segs;
  p.n_seq = n_seq;
  p.max_blocks = max_blocks;
  p.B = d.block_tokens;
  p.hkv = d.num_kv_heads;
  p.capacity = d.capacity_blocks;
  p.chains = 2 * d.num_layers * d.num_kv_heads;
  p.per_layer = pool->n_blk_slabs / d.num_layers;
  p.row_bytes = d.dtype == KVS_DTYPE_BF16 ? d.head_dim * 2 : d.head_dim / 2;
  p.sb_bytes = d.dtype == KVS_DTYPE_BF16 ? 0 : d.dtype == KVS_DTYPE_Q4G64 ? d.head_dim / 16 : d.head_dim / 32;
  p.rows = cp_rows(d);
  p.sms = pool->num_sms;
  p.stall_first = (pool->test_flags & KVS_TEST_STALL_COMPACT) ? 1 : 0;
  pool->test_flags &= ~KVS_TEST_STALL_COMPACT;   // one launch only
  // more CTAs for the masses of a sequence whose table holds more than 8,192
  const long long most = (long long)max_blocks * d.block_tokens;
  const dim3 per_seq((unsigned)n_seq, (unsigned)(mass_dev ? std::clamp<long long>(most / 8192, 1, 16) : 1));
  const unsigned grid = (unsigned)std::max(1ll, std::min(p.max_segs * p.chains, (long long)pool->num_sms * kCpCtas));
  auto move = p.row_bytes == 256 ? cp_move<16> : p.row_bytes == 128 ? cp_move<8> : cp_move<4>;
  const bool both = n_seq <= kCpCluster && per_seq.y == 1;
  const bool ok = (both ? launch_pdl(cp_both, dim3(kCpCluster), dim3(kCpSeqThreads), stream, p) == cudaSuccess
                        : launch_pdl(cp_check, per_seq, dim3(kCpSeqThreads), stream, p) == cudaSuccess &&
                              launch_pdl(cp_apply, per_seq, dim3(kCpSeqThreads), stream, p) == cudaSuccess) &&
                  launch_pdl(move, dim3(grid), dim3(kCpThreads), stream, p) == cudaSuccess;
  if (ok) count_launch(both ? 2 : 3);
  return check_launch("compact");
}

extern "C" kvs_status kvs_compact(kvs_pool* pool, int32_t* block_table_dev, int32_t max_blocks, int32_t* seq_len_dev,
                                  int32_t n_seq, const int32_t* idx_dev, const int64_t* idx_off_dev, float* mass_dev,
                                  int32_t* refcount_dev, int32_t* free_ids_dev, int32_t* n_free_dev, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  return kvs_compact_bounded(pool, block_table_dev, max_blocks, seq_len_dev, n_seq, idx_dev, INT64_MAX, idx_off_dev, mass_dev,
                             refcount_dev, free_ids_dev, n_free_dev, ws, ws_bytes, stream);
}
