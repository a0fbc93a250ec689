// pa_pages.cu -- the block pool's bookkeeping on the device: blocks freed, reserved, forked
// and compacted by reference counts, and the copy of the blocks that those calls list.
//
// A block is free while no table entry refers to it (ref_counts[b] == 0).  Every call has
// one answer whatever the order of its threads: free blocks are taken in ascending order by
// the entries that want one in (sequence, logical block) order.  Both orders are ranks, and
// a rank is a prefix sum: each warp counts its contiguous part, the warps' totals are
// summed over the thread block and over the cluster, and the warp walks its part again with
// its rank at hand.
//
// Bound by latency: a pool of 131,072 blocks has 512 KiB of counts.  One cluster of 8
// thread blocks of 32 warps walks it, so the sums over all warps cost a cluster barrier
// instead of a kernel boundary; with 256 warps a warp's part of such a pool is 512 counts,
// four 16-byte loads a lane, which stay in registers between the two walks.  (16 thread
// blocks: no faster there, 3 us slower for small pools.  64-bit index arithmetic and the
// tables' entries read twice: 31 us against 18 for 256 sequences in such a pool.)
#include <algorithm>

#include "../../include/pagedattn.h"
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace pa {
namespace {

// All threads of the cluster of C thread blocks (a warp arrives as one).
template <int C>
__device__ __forceinline__ void sync_all() {
  if constexpr (C == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    cluster_sync_all();
  }
}

constexpr int kWarpsPerCta = 32;
constexpr int kMaxCluster = 8;

// A contiguous part of [0, n) for each of the cluster's warps, in whole steps of 128.
// (n < 2^30: check_pool)
struct Part {
  int lo, hi;
};
template <int C>
__device__ __forceinline__ Part part_of(int n, int gw) {
  constexpr int kAllWarps = C * kWarpsPerCta;
  const int per = (n + 128 * kAllWarps - 1) / (128 * kAllWarps);
  Part p;
  p.lo = min(n, gw * per * 128);
  p.hi = min(n, p.lo + per * 128);
  return p;
}

// Four counts (or entries) at i .. i + 3 of an array of n; `fill` past its end.  Read
// through L2: these arrays are written by the calls before and by this one.
__device__ __forceinline__ int4 load4(const int32_t *p, int i, int n, int fill) {
  if (i + 4 <= n) return __ldcg(reinterpret_cast<const int4 *>(p + i));
  int4 v = make_int4(fill, fill, fill, fill);
  if (i < n) v.x = __ldcg(p + i);
  if (i + 1 < n) v.y = __ldcg(p + i + 1);
  if (i + 2 < n) v.z = __ldcg(p + i + 2);
  return v;
}

__device__ __forceinline__ int warp_sum(int v) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)v); }
// Sum over the lanes before this one.
__device__ __forceinline__ int warp_before(int v) {
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) >= o) s += u;
  }
  return s - v;
}

// The totals of the cluster's warps, [which][warp]: each warp leaves its own in its thread
// block, and after a cluster barrier reads those of the warps before it.
struct Totals {
  int of[2][kWarpsPerCta];
};
// Sum of totals `which` over the warps before gw (before) and over all (all).
template <int C>
__device__ __forceinline__ void ranks(Totals &t, int which, int gw, int &before, int &all) {
  const int lane = threadIdx.x & 31;
  before = all = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int v = C == 1 ? t.of[which][lane] : dsmem_ld_s32(dsmem_map(smem_u32(&t.of[which][lane]), c));
    all += v;
    if (c * kWarpsPerCta + lane < gw) before += v;
  }
  before = warp_sum(before);
  all = warp_sum(all);
}

// Four of a warp's steps at once: lane l holds the counts lo + 128 u + 4 l .. + 3 of step u,
// `fill` past the part's end.  A part of no more than that stays in registers between the
// counting and the walk with ranks.
constexpr int kSteps = 4;
struct Counts {
  int4 v[kSteps];
  __device__ __forceinline__ void load(const int32_t *refs, int lo, int hi, int fill) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) v[u] = load4(refs, lo + 128 * u + 4 * lane, hi, fill);
  }
  __device__ __forceinline__ int zeros() const {
    int n = 0;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) n += (v[u].x == 0) + (v[u].y == 0) + (v[u].z == 0) + (v[u].w == 0);
    return n;
  }
};

// Free blocks of this warp's part of the counts; c: its last steps.
__device__ __forceinline__ int count_free(const int32_t *refs, Part p, Counts &c) {
  int n = 0;
  for (int lo = p.lo; lo < p.hi; lo += 128 * kSteps) {
    c.load(refs, lo, p.hi, 1);
    n += c.zeros();
  }
  return warp_sum(n);
}

// The first `want` free blocks, ascending, to list (rank of this warp's first: before).
__device__ __forceinline__ void list_free(const int32_t *refs, Part p, Counts &c, int before, int want,
                                          int32_t *list) {
  const int lane = threadIdx.x & 31;
  const bool kept = p.hi - p.lo <= 128 * kSteps;
  int at = before;
  for (int lo = p.lo; lo < p.hi && at < want; lo += 128 * kSteps) {
    if (!kept) c.load(refs, lo, p.hi, 1);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int4 v = c.v[u];
      const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
      const int mine = f[0] + f[1] + f[2] + f[3];
      int r = at + warp_before(mine);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (f[k]) {
          if (r < want) list[r] = lo + 128 * u + 4 * lane + k;
          ++r;
        }
      at += warp_sum(mine);
    }
  }
}

struct PoolArgs {
  int32_t *tables, *refs;
  const int32_t *lens;  // reserve: tokens wanted; free: tokens kept
  int32_t *missing, *list;
  int num_seqs, width, num_blocks, shift;  // blocks of 2^shift tokens
  unsigned *err;
};

__device__ __forceinline__ unsigned blocks_of(int len, int shift) {
  return len > 0 ? ((unsigned)len + (1u << shift) - 1u) >> shift : 0u;
}

// ---- free ------------------------------------------------------------------------
__global__ void __launch_bounds__(256) free_blocks_kernel(const PoolArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = a.num_seqs * a.width;
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int4 v = load4(a.tables, i, n, -1);
  const int id[4] = {v.x, v.y, v.z, v.w};
  int row = i / a.width;
  int col = i - row * a.width;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (id[k] >= 0 && (unsigned)col >= blocks_of(__ldg(a.lens + row), a.shift)) {
      bool bad = id[k] >= a.num_blocks;
      if (!bad && atomicSub(a.refs + id[k], 1) <= 0) {  // was not counted: leave the count
        atomicAdd(a.refs + id[k], 1);
        bad = true;
      }
      if (bad) record_error(a.err, kErrCheck);
      a.tables[i + k] = -1;
    }
    if (++col == a.width) {
      col = 0;
      ++row;
    }
  }
}

// ---- reserve ---------------------------------------------------------------------
// The blocks that the rows of a thread block's part need, from its first row on, in shared
// memory: read once, with the first loads under way (a part of more rows reads on).
constexpr int kNeeds = 1024;
__device__ __forceinline__ unsigned need_of(const PoolArgs &a, const unsigned *needs, int row0, int row) {
  return row - row0 < kNeeds ? needs[row - row0] : blocks_of(__ldg(a.lens + row), a.shift);
}

// Of entries v at i .. i + 3 of the tables, those that want a block, as four bits.
// (i is column col of row `row`.)
__device__ __forceinline__ int wants4(const PoolArgs &a, const unsigned *needs, int row0, int4 v, int i, int hi,
                                      int row, int col) {
  if ((v.x | v.y | v.z | v.w) >= 0) return 0;  // (no negative one; past hi they are 0)
  const int id[4] = {v.x, v.y, v.z, v.w};
  unsigned need = need_of(a, needs, row0, row);
  int f = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (id[k] < 0 && (unsigned)col < need) f |= 1 << k;
    if (++col == a.width && k < 3 && i + k + 1 < hi) {
      col = 0;
      need = need_of(a, needs, row0, ++row);
    }
  }
  return f;
}

template <int C>
__global__ void __launch_bounds__(1024, 1) reserve_blocks_kernel(const PoolArgs a) {
  __shared__ Totals tot;
  __shared__ unsigned needs[kNeeds];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gw = (C == 1 ? 0 : (int)cluster_ctarank()) * kWarpsPerCta + warp;
  const Part pe = part_of<C>(a.num_seqs * a.width, gw), pb = part_of<C>(a.num_blocks, gw);
  const int row0 = part_of<C>(a.num_seqs * a.width, gw - warp).lo / a.width;
  const int len = row0 + (int)threadIdx.x < a.num_seqs ? __ldg(a.lens + row0 + threadIdx.x) : 0;
  Counts c, e;
  e.load(a.tables, pe.lo, pe.hi, 0);  // (all three loads under way before the first wait)
  const int free = count_free(a.refs, pb, c);
  needs[threadIdx.x] = blocks_of(len, a.shift);
  __syncthreads();
  // the entries that want one; of the first steps the flags are kept, four bits a step
  constexpr int kFlagged = 8;
  unsigned flags = 0u;
  int wanted = 0, row = (pe.lo + 4 * lane) / a.width, col = pe.lo + 4 * lane - row * a.width;
  for (int lo = pe.lo; lo < pe.hi; lo += 128 * kSteps) {
    if (lo > pe.lo) e.load(a.tables, lo, pe.hi, 0);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const unsigned f = wants4(a, needs, row0, e.v[u], lo + 128 * u + 4 * lane, pe.hi, row, col);
      for (col += 128; col >= a.width; col -= a.width) ++row;
      const int step = (lo - pe.lo) / 128 + u;
      if (step < kFlagged) flags |= f << (4 * step);
      wanted += __popc(f);
    }
  }
  wanted = warp_sum(wanted);
  if (lane == 0) {
    tot.of[0][warp] = wanted;
    tot.of[1][warp] = free;
  }
  sync_all<C>();
  int want0, wants, free0, frees;
  ranks<C>(tot, 0, gw, want0, wants);
  ranks<C>(tot, 1, gw, free0, frees);
  list_free(a.refs, pb, c, free0, wants, a.list);
  sync_all<C>();  // the list is written, every count read
  int at = want0;
  if (wanted > 0) {
    for (int i0 = pe.lo; i0 < pe.hi; i0 += 128) {
      const int i = i0 + 4 * lane, step = (i0 - pe.lo) / 128;
      const unsigned f = step < kFlagged ? flags >> (4 * step) & 15u
                                         : wants4(a, needs, row0, load4(a.tables, i, pe.hi, 0), i, pe.hi,
                                                  i / a.width, i % a.width);
      const int mine = __popc(f);
      if (!__any_sync(0xffffffffu, mine > 0)) continue;
      int r = at + warp_before(mine);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (f >> k & 1u) {
          if (r < frees) {
            const int id = __ldcg(a.list + r);
            a.tables[i + k] = id;
            a.refs[id] = 1;
          }
          ++r;
        }
      at += warp_sum(mine);
    }
  }
  if (gw == 0 && lane == 0) *a.missing = max(0, wants - frees);
  // rows longer than the table, among those at hand and (parts of very many rows) the rest
  const int rows_hi = part_of<C>(a.num_seqs * a.width, gw - warp + kWarpsPerCta).lo / a.width;
  bool over = needs[threadIdx.x] > (unsigned)a.width;
  for (int i = row0 + kNeeds + (int)threadIdx.x; i <= min(rows_hi, a.num_seqs - 1); i += 1024)
    over |= blocks_of(__ldg(a.lens + i), a.shift) > (unsigned)a.width;
  if (over) record_error(a.err, kErrCheck);
}

// ---- fork ------------------------------------------------------------------------
struct ForkArgs {
  int32_t *tables, *lens, *refs;
  const int32_t *src, *dst;
  int32_t *src_blocks, *dst_blocks, *counts, *list, *tail_of;
  int num_forks, num_seqs, width, num_blocks, shift;
  unsigned *err;
};

// Fork f's parent and child; false: an id outside the batch, or a parent its own child.
__device__ __forceinline__ bool fork_pair(const ForkArgs &a, int f, int &s, int &d) {
  s = __ldg(a.src + f);
  d = __ldg(a.dst + f);
  return s >= 0 && s < a.num_seqs && d >= 0 && d < a.num_seqs && s != d;
}

// The partial block at the end of fork f's parent (-1: none, or the fork is skipped).
__device__ __forceinline__ int parent_tail(const ForkArgs &a, int f, bool rec) {
  int s, d, id = -1;
  bool bad = !fork_pair(a, f, s, d);
  if (!bad) {
    const int len = max(0, __ldcg(a.lens + s));
    bad = blocks_of(len, a.shift) > (unsigned)a.width;
    if (!bad && (len & ((1 << a.shift) - 1)) != 0) {
      id = __ldcg(a.tables + s * a.width + (len >> a.shift));
      bad = id < 0 || id >= a.num_blocks;
    }
  }
  if (bad && rec) record_error(a.err, kErrCheck);
  return bad ? -1 : id;
}

template <int C>
__global__ void __launch_bounds__(1024, 1) fork_blocks_kernel(const ForkArgs a) {
  constexpr int kAllWarps = C * kWarpsPerCta;
  __shared__ Totals tot;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gw = (C == 1 ? 0 : (int)cluster_ctarank()) * kWarpsPerCta + warp;
  const Part pb = part_of<C>(a.num_blocks, gw);
  // forks in parts of whole warps: f = lo + lane, lo + lane + 32, ..
  const int per = (a.num_forks + kAllWarps * 32 - 1) / (kAllWarps * 32) * 32;
  const int lo = min(a.num_forks, gw * per), hi = min(a.num_forks, lo + per);
  Counts c;
  const int free = count_free(a.refs, pb, c);
  int tail = -1, tails = 0;  // (tail: of the lane's last fork; of its only one where a part is a warp)
  for (int f = lo + lane; f < hi; f += 32) {
    tail = parent_tail(a, f, true);
    tails += tail >= 0;
  }
  __syncwarp();
  tails = warp_sum(tails);
  if (lane == 0) {
    tot.of[0][warp] = tails;
    tot.of[1][warp] = free;
  }
  sync_all<C>();
  int tail0, all, free0, frees;
  ranks<C>(tot, 0, gw, tail0, all);
  ranks<C>(tot, 1, gw, free0, frees);
  list_free(a.refs, pb, c, free0, all, a.list);
  sync_all<C>();  // the list is written, every count read
  int at = tail0;
  for (int f0 = lo; f0 < hi; f0 += 32) {
    const int f = f0 + lane;
    const int t = f >= hi ? -1 : per == 32 ? tail : parent_tail(a, f, false);
    const int r = at + warp_before(t >= 0);
    at += warp_sum(t >= 0);
    if (f < hi) {
      int id = -1;
      if (t >= 0 && r < frees) {
        id = __ldcg(a.list + r);
        a.refs[id] = 1;
        a.src_blocks[r] = t;
        a.dst_blocks[r] = id;
      }
      a.tail_of[f] = id;
    }
  }
  if (gw == 0 && lane == 0) {
    a.counts[0] = min(all, frees);
    a.counts[1] = max(0, all - frees);
  }
  // the children's rows: so many warps a fork that every warp has one, each the same share of
  // the row.  What they read of a fork is on its way while the cluster meets.
  const int share = max(1, kAllWarps / a.num_forks), part = gw % share;
  int f = gw / share, s = 0, d = 0, len = 0;
  bool ok = f < a.num_forks && fork_pair(a, f, s, d);
  if (ok) len = max(0, __ldcg(a.lens + s));
  sync_all<C>();  // the tails' new blocks
  while (f < a.num_forks) {
    if (ok) {
      const int full = min(len >> a.shift, a.width), fresh = __ldcg(a.tail_of + f);
      const int32_t *from = a.tables + s * a.width;
      int32_t *to = a.tables + d * a.width;
#pragma unroll 4
      for (int j = part * 32 + lane; j < a.width; j += share * 32) {
        int id = j < full ? __ldcg(from + j) : j == full ? fresh : -1;
        if (j < full) {
          if (id < 0 || id >= a.num_blocks) {
            record_error(a.err, kErrCheck);
            id = -1;
          } else {
            atomicAdd(a.refs + id, 1);
          }
        }
        to[j] = id;
      }
      // (no parent is a child: its length is read by no one else)
      if (part == 0 && lane == 0) a.lens[d] = fresh >= 0 ? len : full << a.shift;
    }
    f += max(1, kAllWarps / share);
    ok = f < a.num_forks && fork_pair(a, f, s, d);
    if (ok) len = max(0, __ldcg(a.lens + s));
  }
}

// ---- compact ---------------------------------------------------------------------
struct CompactArgs {
  int32_t *tables_out, *refs_out;
  const int32_t *tables, *refs;
  int32_t *src_blocks, *dst_blocks, *counts;
  int32_t *name;   // [num_blocks]: new id of a block that moves, -1 for a free one
  int32_t *moved;  // [num_blocks / 2]: reference counts of the moving blocks
  int num_seqs, width, num_blocks;
  unsigned *err;
};

template <int C>
__global__ void __launch_bounds__(1024, 1) compact_blocks_kernel(const CompactArgs a) {
  constexpr int kAllWarps = C * kWarpsPerCta;
  __shared__ Totals tot;
  __shared__ int s_below;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gw = (C == 1 ? 0 : (int)cluster_ctarank()) * kWarpsPerCta + warp;
  const Part p = part_of<C>(a.num_blocks, gw);
  if (threadIdx.x == 0) s_below = 0;
  Counts c;
  const int used = p.hi - p.lo - count_free(a.refs, p, c);
  const bool kept = p.hi - p.lo <= 128 * kSteps;
  if (lane == 0) tot.of[0][warp] = used;
  sync_all<C>();
  int used0, live;
  ranks<C>(tot, 0, gw, used0, live);
  // used blocks below `live`: the warp whose part holds that border counts them
  if (p.lo < live && live <= p.hi) {
    int below = 0;
    for (int i = p.lo + lane; i < live; i += 32) below += __ldcg(a.refs + i) != 0;
    below = warp_sum(below);
    if (lane == 0) s_below = used0 + below;
  }
  sync_all<C>();
  int below = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) below += C == 1 ? s_below : dsmem_ld_s32(dsmem_map(smem_u32(&s_below), c));
  // the k-th used block at or past `live` goes to the k-th free one before it
  int at = used0;
  for (int lo = p.lo; lo < p.hi; lo += 128 * kSteps) {
    if (!kept) c.load(a.refs, lo, p.hi, 0);  // (kept ones are 1 past the part's end)
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int i = lo + 128 * t + 4 * lane;
      const int ref[4] = {c.v[t].x, c.v[t].y, c.v[t].z, c.v[t].w};
      int mine = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine += i + k < p.hi && ref[k] != 0;
      int u = at + warp_before(mine);  // used blocks before i + k
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = i + k;
        if (b < p.hi) {
          if (b < live) {
            if (ref[k] == 0)
              a.dst_blocks[b - u] = b;
            else
              a.refs_out[b] = ref[k];
          } else {
            if (ref[k] != 0) {
              a.src_blocks[u - below] = b;
              a.moved[u - below] = ref[k];
            }
            a.name[b] = -1;
            a.refs_out[b] = 0;
          }
          u += ref[k] != 0;
        }
      }
      at += warp_sum(mine);
    }
  }
  const int moves = live - below;
  if (gw == 0 && lane == 0) {
    a.counts[0] = moves;
    a.counts[1] = live;
  }
  sync_all<C>();
  for (int k = gw * 32 + lane; k < moves; k += kAllWarps * 32) {
    const int to = __ldcg(a.dst_blocks + k);
    a.name[__ldcg(a.src_blocks + k)] = to;
    a.refs_out[to] = __ldcg(a.moved + k);
  }
  sync_all<C>();
  const int n = a.num_seqs * a.width;
#pragma unroll 4
  for (int i = (gw * 32 + lane) * 4; i < n; i += kAllWarps * 128) {
    const int4 v = load4(a.tables, i, n, -1);
    int id[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k >= n) continue;
      if (id[k] >= live) {
        id[k] = id[k] < a.num_blocks ? __ldcg(a.name + id[k]) : -1;
        if (id[k] < 0) record_error(a.err, kErrCheck);  // outside the pool, or counted as free
      }
      a.tables_out[i + k] = id[k];
    }
  }
}

// ---- copy ------------------------------------------------------------------------
// x: a 16 KiB piece of the block's K or V; y: the pairs (further pairs loop).  A pair's scales
// go with its first piece of K.
constexpr int kPieceThreads = 256, kPieceLoads = 4;
constexpr int kPiece = kPieceThreads * kPieceLoads;  // 16-byte chunks

struct CopyArgs {
  uint4 *cache[2];
  float *kv_scales;
  const int32_t *src, *dst, *counts;
  int64_t chunks;  // 16-byte chunks of a block in one cache
  int max_pairs, num_blocks, pieces, scales_per_block;
  unsigned *err;
};

__global__ void __launch_bounds__(kPieceThreads) copy_pages_kernel(const CopyArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int pairs = min(max(0, __ldcg(a.counts)), a.max_pairs);
  const int piece = blockIdx.x >> 1, kv = blockIdx.x & 1;
  for (int pair = blockIdx.y; pair < pairs; pair += gridDim.y) {
    const int s = __ldcg(a.src + pair), d = __ldcg(a.dst + pair);
    if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks) {
      if (piece == 0 && kv == 0 && threadIdx.x == 0) record_error(a.err, kErrCheck);
      continue;
    }
    const uint4 *from = a.cache[kv] + s * a.chunks;
    uint4 *to = a.cache[kv] + d * a.chunks;
    const int64_t c0 = (int64_t)piece * kPiece + threadIdx.x;
    if (c0 + (kPieceLoads - 1) * kPieceThreads < a.chunks) {  // all loads before the first store
      uint4 v[kPieceLoads];
#pragma unroll
      for (int u = 0; u < kPieceLoads; ++u) v[u] = __ldcs(from + c0 + u * kPieceThreads);
#pragma unroll
      for (int u = 0; u < kPieceLoads; ++u) __stcs(to + c0 + u * kPieceThreads, v[u]);
    } else {
      for (int64_t c = c0; c < a.chunks; c += kPieceThreads) __stcs(to + c, __ldcs(from + c));
    }
    if (a.kv_scales != nullptr && piece == 0 && kv == 0)
      for (int i = threadIdx.x; i < a.scales_per_block; i += kPieceThreads)
        a.kv_scales[(int64_t)d * a.scales_per_block + i] = __ldcg(a.kv_scales + (int64_t)s * a.scales_per_block + i);
  }
}

// One cluster of C thread blocks, as a dependent of the work before it.
template <int C, typename A>
cudaError_t launch_cluster(void (*kern)(A), cudaStream_t st, const A &args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kWarpsPerCta * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args);
}

// Whether one thread block alone is faster, whose barriers cost nothing.  Reserving in a
// pool of 2048 blocks took it 7.1 us and the cluster 9.1, of 16,384 blocks both 9.7, of 65,536
// 31 and 12; a fork in 8192 blocks 17 and 11, a compaction of 16,384 25 and 13.
bool one_block(int num_blocks, int64_t entries) { return num_blocks <= 4096 && entries <= 4096; }

// Sizes that the bookkeeping calls share.
pa_status check_pool(int num_seqs, int max_blocks_per_seq, int num_blocks, int block_size) {
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0) return PA_ERR_INVALID_ARG;
  if (!supported_block(block_size)) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * max_blocks_per_seq >= (int64_t)1 << 30 || num_blocks >= 1 << 30 ||
      (int64_t)max_blocks_per_seq * block_size >= (int64_t)1 << 31)
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// (8, 16 or 32)
int shift_of(int block_size) { return block_size == 8 ? 3 : block_size == 16 ? 4 : 5; }

size_t ints(int64_t n) { return (size_t)n * 4; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

PA_API size_t pa_pages_workspace_size(int num_blocks, int num_forks) {
  if (num_blocks <= 0 || num_forks < 0) return 0;
  return ((size_t)num_blocks + (size_t)std::max(num_forks, num_blocks / 2) + 4) * 4;
}

PA_API pa_status pa_free_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *keep_lens,
                                int num_seqs, int max_blocks_per_seq, int num_blocks, int block_size,
                                void *stream) {
  if (!block_tables || !ref_counts || !keep_lens) return PA_ERR_INVALID_ARG;
  const pa_status st = check_pool(num_seqs, max_blocks_per_seq, num_blocks, block_size);
  if (st != PA_OK) return st;
  if (!aligned16(block_tables) || !aligned16(ref_counts) || !aligned4(keep_lens)) return PA_ERR_INVALID_ARG;
  const size_t table = ints((int64_t)num_seqs * max_blocks_per_seq), refs = ints(num_blocks), lens = ints(num_seqs);
  if (overlap(block_tables, table, ref_counts, refs) || overlap(block_tables, table, keep_lens, lens) ||
      overlap(ref_counts, refs, keep_lens, lens))
    return PA_ERR_INVALID_ARG;
  PoolArgs a = {};
  a.tables = block_tables;
  a.refs = ref_counts;
  a.lens = keep_lens;
  a.num_seqs = num_seqs;
  a.width = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.shift = shift_of(block_size);
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  const unsigned ctas = (unsigned)(((int64_t)num_seqs * max_blocks_per_seq + 1023) / 1024);
  return launch_dependent(free_blocks_kernel, ctas, 256, static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

PA_API pa_status pa_reserve_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *lens,
                                   int32_t *missing, int num_seqs, int max_blocks_per_seq, int num_blocks,
                                   int block_size, void *workspace, size_t workspace_bytes, void *stream) {
  if (!block_tables || !ref_counts || !lens || !missing || !workspace) return PA_ERR_INVALID_ARG;
  const pa_status st = check_pool(num_seqs, max_blocks_per_seq, num_blocks, block_size);
  if (st != PA_OK) return st;
  if (!aligned16(block_tables) || !aligned16(ref_counts) || !aligned16(workspace) || !aligned4(lens) ||
      !aligned4(missing))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < pa_pages_workspace_size(num_blocks, 0)) return PA_ERR_INVALID_ARG;
  struct {
    const void *p;
    size_t n;
  } buf[] = {{block_tables, ints((int64_t)num_seqs * max_blocks_per_seq)}, {ref_counts, ints(num_blocks)},
             {lens, ints(num_seqs)}, {missing, 4}, {workspace, pa_pages_workspace_size(num_blocks, 0)}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n)) return PA_ERR_INVALID_ARG;
  PoolArgs a = {};
  a.tables = block_tables;
  a.refs = ref_counts;
  a.lens = lens;
  a.missing = missing;
  a.list = static_cast<int32_t *>(workspace);
  a.num_seqs = num_seqs;
  a.width = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.shift = shift_of(block_size);
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = one_block(num_blocks, (int64_t)num_seqs * max_blocks_per_seq)
                            ? launch_cluster<1>(reserve_blocks_kernel<1>, s, a)
                            : launch_cluster<kMaxCluster>(reserve_blocks_kernel<kMaxCluster>, s, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_API pa_status pa_fork_blocks(int32_t *block_tables, int32_t *context_lens, int32_t *ref_counts,
                                const int32_t *src_seqs, const int32_t *dst_seqs, int32_t *src_blocks,
                                int32_t *dst_blocks, int32_t *counts, int num_forks, int num_seqs,
                                int max_blocks_per_seq, int num_blocks, int block_size, void *workspace,
                                size_t workspace_bytes, void *stream) {
  if (!block_tables || !context_lens || !ref_counts || !counts || !workspace) return PA_ERR_INVALID_ARG;
  const pa_status st = check_pool(num_seqs, max_blocks_per_seq, num_blocks, block_size);
  if (st != PA_OK) return st;
  if (num_forks < 0 || num_forks > num_seqs) return PA_ERR_INVALID_ARG;
  if (num_forks > 0 && (!src_seqs || !dst_seqs || !src_blocks || !dst_blocks)) return PA_ERR_INVALID_ARG;
  if (!aligned16(ref_counts) || !aligned16(workspace)) return PA_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(block_tables), static_cast<const void *>(context_lens),
                        static_cast<const void *>(src_seqs), static_cast<const void *>(dst_seqs),
                        static_cast<const void *>(src_blocks), static_cast<const void *>(dst_blocks),
                        static_cast<const void *>(counts)})
    if (!aligned4(p)) return PA_ERR_INVALID_ARG;
  const size_t room = pa_pages_workspace_size(num_blocks, num_forks);
  if (workspace_bytes < room) return PA_ERR_INVALID_ARG;
  struct {
    const void *p;
    size_t n;
  } buf[] = {{block_tables, ints((int64_t)num_seqs * max_blocks_per_seq)}, {context_lens, ints(num_seqs)},
             {ref_counts, ints(num_blocks)}, {src_blocks, ints(num_forks)}, {dst_blocks, ints(num_forks)},
             {counts, 8}, {workspace, room}, {src_seqs, ints(num_forks)}, {dst_seqs, ints(num_forks)}};
  for (int i = 0; i < 7; ++i)  // (the inputs, 7 and 8, may be one array)
    for (int j = i + 1; j < 9; ++j)
      if (overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n)) return PA_ERR_INVALID_ARG;
  if (num_forks == 0)
    return cudaMemsetAsync(counts, 0, 8, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  ForkArgs a = {};
  a.tables = block_tables;
  a.lens = context_lens;
  a.refs = ref_counts;
  a.src = src_seqs;
  a.dst = dst_seqs;
  a.src_blocks = src_blocks;
  a.dst_blocks = dst_blocks;
  a.counts = counts;
  a.list = static_cast<int32_t *>(workspace);
  a.tail_of = a.list + num_blocks;
  a.num_forks = num_forks;
  a.num_seqs = num_seqs;
  a.width = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.shift = shift_of(block_size);
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = one_block(num_blocks, (int64_t)num_forks * max_blocks_per_seq)
                            ? launch_cluster<1>(fork_blocks_kernel<1>, s, a)
                            : launch_cluster<kMaxCluster>(fork_blocks_kernel<kMaxCluster>, s, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_API pa_status pa_compact_blocks(int32_t *block_tables_out, int32_t *ref_counts_out,
                                   const int32_t *block_tables, const int32_t *ref_counts, int32_t *src_blocks,
                                   int32_t *dst_blocks, int32_t *counts, int num_seqs, int max_blocks_per_seq,
                                   int num_blocks, void *workspace, size_t workspace_bytes, void *stream) {
  if (!block_tables_out || !ref_counts_out || !block_tables || !ref_counts || !counts || !workspace)
    return PA_ERR_INVALID_ARG;
  if (num_blocks > 1 && (!src_blocks || !dst_blocks)) return PA_ERR_INVALID_ARG;
  const pa_status st = check_pool(num_seqs, max_blocks_per_seq, num_blocks, 16);
  if (st != PA_OK) return st;
  if (!aligned16(block_tables) || !aligned16(ref_counts) || !aligned16(workspace) || !aligned4(block_tables_out) ||
      !aligned4(ref_counts_out) || !aligned4(src_blocks) || !aligned4(dst_blocks) || !aligned4(counts))
    return PA_ERR_INVALID_ARG;
  const size_t room = pa_pages_workspace_size(num_blocks, 0);
  if (workspace_bytes < room) return PA_ERR_INVALID_ARG;
  const size_t table = ints((int64_t)num_seqs * max_blocks_per_seq), refs = ints(num_blocks);
  struct {
    const void *p;
    size_t n;
  } buf[] = {{block_tables_out, table}, {ref_counts_out, refs}, {src_blocks, ints(num_blocks / 2)},
             {dst_blocks, ints(num_blocks / 2)}, {counts, 8}, {workspace, room}, {block_tables, table},
             {ref_counts, refs}};
  for (int i = 0; i < 8; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (!((i == 0 && j == 6 && block_tables_out == block_tables) ||
            (i == 1 && j == 7 && ref_counts_out == ref_counts)) &&
          overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n))
        return PA_ERR_INVALID_ARG;
  CompactArgs a = {};
  a.tables_out = block_tables_out;
  a.refs_out = ref_counts_out;
  a.tables = block_tables;
  a.refs = ref_counts;
  a.src_blocks = src_blocks;
  a.dst_blocks = dst_blocks;
  a.counts = counts;
  a.name = static_cast<int32_t *>(workspace);
  a.moved = a.name + num_blocks;
  a.num_seqs = num_seqs;
  a.width = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = one_block(num_blocks, (int64_t)num_seqs * max_blocks_per_seq)
                            ? launch_cluster<1>(compact_blocks_kernel<1>, s, a)
                            : launch_cluster<kMaxCluster>(compact_blocks_kernel<kMaxCluster>, s, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_API pa_status pa_copy_pages(void *k_cache, void *v_cache, float *kv_scales, const int32_t *src_blocks,
                               const int32_t *dst_blocks, const int32_t *counts, int max_pairs, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, int element_bytes, void *stream) {
  if (!k_cache || !v_cache || !src_blocks || !dst_blocks || !counts) return PA_ERR_INVALID_ARG;
  if (max_pairs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(src_blocks) || !aligned4(dst_blocks) ||
      !aligned4(counts) || !aligned4(kv_scales))
    return PA_ERR_INVALID_ARG;
  if (element_bytes != 1 && element_bytes != 2) return PA_ERR_UNSUPPORTED;
  if (!supported_block(block_size)) return PA_ERR_UNSUPPORTED;
  if (head_dim != 128 && !(head_dim == 64 && element_bytes == 2)) return PA_ERR_UNSUPPORTED;
  if (kv_scales && element_bytes != 1) return PA_ERR_INVALID_ARG;
  if ((int64_t)num_blocks * num_kv_heads * 2 >= (int64_t)1 << 31) return PA_ERR_INVALID_ARG;
  if (max_pairs == 0) return PA_OK;
  // the caches and their scales apart from one another and from the lists (which may be one array)
  const size_t cache = (size_t)num_blocks * num_kv_heads * block_size * head_dim * element_bytes;
  const size_t scales = kv_scales ? (size_t)num_blocks * num_kv_heads * 8 : 0;
  struct {
    const void *p;
    size_t n;
  } buf[] = {{k_cache, cache}, {v_cache, cache}, {kv_scales, scales}, {src_blocks, ints(max_pairs)},
             {dst_blocks, ints(max_pairs)}, {counts, 8}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 6; ++j)
      if (buf[i].n && buf[j].n && overlap(buf[i].p, buf[i].n, buf[j].p, buf[j].n)) return PA_ERR_INVALID_ARG;
  CopyArgs a = {};
  a.cache[0] = static_cast<uint4 *>(k_cache);
  a.cache[1] = static_cast<uint4 *>(v_cache);
  a.kv_scales = kv_scales;
  a.src = src_blocks;
  a.dst = dst_blocks;
  a.counts = counts;
  a.chunks = (int64_t)num_kv_heads * block_size * head_dim * element_bytes / 16;
  a.max_pairs = max_pairs;
  a.num_blocks = num_blocks;
  a.pieces = (int)((a.chunks + kPiece - 1) / kPiece);
  a.scales_per_block = 2 * num_kv_heads;
  a.err = error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  // how many pairs there are is known on the device alone: at most a wave of thread blocks
  const int x = 2 * a.pieces;
  const int y = std::min(std::min(max_pairs, 65535), std::max(1, sms * 8 / x));
  const cudaError_t e = launch_dependent(copy_pages_kernel, dim3((unsigned)x, (unsigned)y, 1), kPieceThreads,
                                         static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
