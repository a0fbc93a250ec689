// pa_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// For each sequence whose context is longer than `budget` rows, every KV head keeps
// `budget` of its rows: those of the `sinks` first and the `recent` last positions,
// and of the others the ones with the highest scores (ties: the lowest row).  A KV
// head's choice is its own: a block-table entry names a block for all KV heads, but
// each head's rows of it are separate memory, so heads may hold different positions
// in the same row.  ("LLM推理与服务：面试问题与推荐回答" Q4: drop the tokens that draw
// little attention.)
//
// Keys.  A row's score as an unsigned integer whose order is the floats' order; NaN
// below every number; a protected position above all.  Kept = the `budget` largest
// (key, then lower row).  Two ways to find them, by how many rows are over budget:
//   * up to kFew (a serving step appends one row, or a few with drafts): that many
//     times the smallest (key, then higher row) that is larger than the last one found;
//   * more: the budget-th largest key by a radix select, eight bits at a time, then the
//     rows in order.
// 64 sequences x 8 heads, 1, 4, 6 and 8 rows over 1024: 5.3, 9.8, 12.8 and 15.9 us by the
// first, 12.7, 13.2, 13.7 and 14.1 by the second; 2 x 8 heads, 1, 4 and 8 over 32768:
// 7.0, 13.7 and 22.8 against 30.1 to 30.4.  Keys are held in shared memory.
//
// Moves.  Attention does not depend on the order of cached rows (K rows carry their
// rotation), so nothing is shifted: with m rows evicted below `budget`, exactly m kept
// rows lie at or past it, and the i-th of these is copied into the i-th hole.  Sources
// are never written and holes never read, so the copies need no order, and repeating
// the call repeats the same copies.  They are latency-bound one by one (302 us for 128
// heads of 1800 rows): a warp works out 32 pairs at once, one per lane, and keeps eight
// rows' loads in flight.
//
// A (sequence, KV head) is one thread block, or a cluster of them that shares its rows
// when there are fewer than the GPU holds: counts and sums then meet through distributed
// shared memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_launch.h"

namespace {

constexpr int kKeyCap = 44 * 1024;  // keys a CTA can hold in shared memory (176 KiB)
constexpr uint32_t kProtected = 0xffffffffu;
constexpr int kFew = 8;
constexpr int kListCap = 512;  // moves a single CTA lists in shared memory
constexpr int kMaxCluster = 8;

struct EvictArgs {
  uint8_t *k_cache, *v_cache;
  const float *scores;
  const int32_t *row_pos;
  float *scores_out;
  int32_t *row_pos_out, *new_lens;
  const int32_t *block_tables, *context_lens, *seq_lens;
  int2 *moves;  // workspace: (hole, source) pairs, `budget` per (sequence, head)
  int num_kv_heads, block_shift, max_blocks_per_seq, num_blocks, max_rows;
  int budget, sinks, recent, key_cap;
  int row_chunks;  // 16-byte chunks of a cached row: 8 or 16
  unsigned *err;
};

__device__ __forceinline__ uint32_t key_of(float score, int pos, int sinks, int64_t recent_from) {
  if (pos < sinks || pos >= recent_from) return kProtected;
  if (score != score) return 0u;
  const uint32_t b = __float_as_uint(score + 0.f);  // (-0 counts as 0)
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint64_t warp_min(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ uint64_t dsmem_ld_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// All threads of the cluster (or of the CTA that is one).
__device__ __forceinline__ void group_sync(int csize) {
  if (csize > 1)
    pa::cluster_sync_all();
  else
    __syncthreads();
}

// Rows of a contiguous range: above the border key and equal to it, below the budget and
// from it on.
struct Counts {
  int gt_lo, gt_hi, eq_lo, eq_hi, n_lo;
  // with `t` equal rows before the range, of which `left` stay in all: holes and sources
  __device__ __forceinline__ int kept_lo(int t, int left) const {
    return gt_lo + min(eq_lo, max(0, left - t));
  }
  __device__ __forceinline__ int holes(int t, int left) const { return n_lo - kept_lo(t, left); }
  __device__ __forceinline__ int sources(int t, int left) const {
    return gt_hi + min(eq_hi, max(0, left - t - eq_lo));
  }
};

// Copy the cached rows of cnt <= 32 pairs: lane l holds pair l's row indices (in rows of
// the pool; rt < 0: nothing to copy).
__device__ __forceinline__ void copy_rows(const EvictArgs &a, int64_t rt, int64_t rf, int cnt) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.row_chunks;             // chunks of a pair, K then V
  const int side = 32 / per;                    // pairs per step of the warp: 1 or 2
  const int sub = lane / per, c = lane % per;
  uint4 *cache = reinterpret_cast<uint4 *>(c < a.row_chunks ? a.k_cache : a.v_cache);
  const int cc = c < a.row_chunks ? c : c - a.row_chunks;
  constexpr int kUnroll = 8;
  for (int j0 = 0; j0 < cnt; j0 += kUnroll * side) {
    uint4 x[kUnroll];
    int64_t to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * side + sub;
      const int64_t from = __shfl_sync(0xffffffffu, rf, j & 31);
      to[u] = __shfl_sync(0xffffffffu, rt, j & 31);
      if (j >= cnt) to[u] = -1;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (to[u] >= 0) x[u] = cache[from * a.row_chunks + cc];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (to[u] >= 0) cache[to[u] * a.row_chunks + cc] = x[u];
  }
}

// (64 registers a thread: 32 warps per SM)
template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_kernel(const EvictArgs a) {
  constexpr int NW = NT / 32;
  constexpr int kUnroll = 3;
  extern __shared__ uint32_t s_keys[];
  __shared__ int hist[4][256];
  __shared__ Counts s_cnt[NW];        // by warp
  __shared__ Counts s_pub;            // of this CTA, read by its peers
  __shared__ uint64_t s_min[kFew][NW];
  __shared__ uint64_t s_cta_min[kFew];
  __shared__ int2 s_moves[kListCap];
  __shared__ int s_digit, s_left;
  pa::griddep_wait();
  pa::griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = (int)pa::cluster_nctarank(), crank = (int)pa::cluster_ctarank();
  const int unit = blockIdx.x / csize;
  const int seq = unit / a.num_kv_heads, head = unit % a.num_kv_heads;
  int L = max(0, __ldg(a.context_lens + seq));
  const int64_t recent_from = (int64_t)__ldg(a.seq_lens + seq) - a.recent;
  if (L > a.max_rows) {  // context longer than its table
    if (tid == 0 && head == 0 && crank == 0) pa::record_error(a.err, pa::kErrCheck);
    L = a.max_rows;
  }
  if (tid == 0 && head == 0 && crank == 0) a.new_lens[seq] = min(L, a.budget);
  const int64_t led = (int64_t)unit * a.max_rows;
  const float *scores = a.scores + led;
  const int32_t *row_pos = a.row_pos + led;
  float *scores_out = a.scores_out + led;
  int32_t *row_pos_out = a.row_pos_out + led;
  const bool apart = a.scores != a.scores_out;
  const int over = L - a.budget;  // rows to evict
  if (over <= 0 && !apart) return;  // (all CTAs of the cluster)

  // this CTA's rows [lo, hi), of which each warp takes a contiguous range [w0, w1).  Keys
  // into shared memory; with ledgers apart, the rows below the budget are copied as they
  // are (every evicted one of them is written again below).
  const int slice = ((L + csize - 1) / csize + 31) & ~31;
  const int lo = min(L, crank * slice), hi = min(L, lo + slice);
  const int held = min(hi - lo, a.key_cap);
  const int per = ((hi - lo + NW - 1) / NW + 31) & ~31;
  const int w0 = min(hi, lo + warp * per), w1 = min(hi, w0 + per);
  uint64_t least = ~0ull;
  auto rank_of = [](uint32_t key, int r) -> uint64_t {  // smallest: evicted first
    return ((uint64_t)key << 32) | (uint32_t)~r;
  };
  for (int i = tid; i < 4 * 256; i += NT) (&hist[0][0])[i] = 0;
  // four rows a thread and load (ranges begin at multiples of 32 rows, and a table holds a
  // multiple of 8)
  for (int r0 = w0 + 4 * lane; r0 < w1; r0 += 128 * kUnroll) {
    float4 sc[kUnroll];
    int4 ps[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + 128 * u < w1 ? r0 + 128 * u : r0;
      sc[u] = __ldcg(reinterpret_cast<const float4 *>(scores + r));
      ps[u] = __ldcg(reinterpret_cast<const int4 *>(row_pos + r));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + 128 * u;
      if (r >= w1) break;
      const int n = min(4, w1 - r);
      if (apart && r + 3 < min(a.budget, w1)) {
        *reinterpret_cast<float4 *>(scores_out + r) = sc[u];
        *reinterpret_cast<int4 *>(row_pos_out + r) = ps[u];
      } else if (apart) {
        const float f[4] = {sc[u].x, sc[u].y, sc[u].z, sc[u].w};
        const int p[4] = {ps[u].x, ps[u].y, ps[u].z, ps[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < n && r + i < a.budget) {
            scores_out[r + i] = f[i];
            row_pos_out[r + i] = p[i];
          }
      }
      const uint4 k = make_uint4(key_of(sc[u].x, ps[u].x, a.sinks, recent_from),
                                 key_of(sc[u].y, ps[u].y, a.sinks, recent_from),
                                 key_of(sc[u].z, ps[u].z, a.sinks, recent_from),
                                 key_of(sc[u].w, ps[u].w, a.sinks, recent_from));
      // (held is a multiple of 4 wherever it is less than the slice, and the rows of a
      // slice are padded to 32 in shared memory)
      if (r - lo < held) *reinterpret_cast<uint4 *>(s_keys + (r - lo)) = k;
      least = min(least, rank_of(k.x, r));
      if (n > 1) least = min(least, rank_of(k.y, r + 1));
      if (n > 2) least = min(least, rank_of(k.z, r + 2));
      if (n > 3) least = min(least, rank_of(k.w, r + 3));
    }
  }
  __syncwarp();  // (a warp's later passes read its rows' keys in another order)
  if (over <= 0) return;
  auto key = [&](int r) {
    return r - lo < held ? s_keys[r - lo]
                         : key_of(__ldcg(scores + r), __ldcg(row_pos + r), a.sinks, recent_from);
  };
  // f(key, row) for every row of this warp, four at a time
  auto each_row = [&](auto f) {
#pragma unroll 2
    for (int r = w0 + 4 * lane; r < w1; r += 128) {
      uint32_t k[4];
      if (r - lo < held) {
        const uint4 x = *reinterpret_cast<const uint4 *>(s_keys + (r - lo));
        k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = key(min(r + i, w1 - 1));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < w1) f(k[i], r + i);
    }
  };
  const unsigned below = (1u << lane) - 1u;
  const int32_t *table = a.block_tables + (int64_t)seq * a.max_blocks_per_seq;
  // move pair p: the ledgers here, and the row indices of its copy (-1: a block outside the
  // pool, and the hole's row and ledger entries stay as they are)
  auto start_move = [&](int2 p, int64_t &rt, int64_t &rf) {
    const float score = __ldcg(scores + p.y);
    const int pos = __ldcg(row_pos + p.y);
    const int sh = a.block_shift, mask = (1 << sh) - 1;
    const int bt = __ldg(table + (p.x >> sh)), bf = __ldg(table + (p.y >> sh));
    rt = rf = -1;
    if (bt < 0 || bt >= a.num_blocks || bf < 0 || bf >= a.num_blocks) {
      pa::record_error(a.err, pa::kErrCheck);
      return;
    }
    scores_out[p.x] = score;
    row_pos_out[p.x] = pos;
    rt = (((int64_t)bt * a.num_kv_heads + head) << sh) + (p.x & mask);
    rf = (((int64_t)bf * a.num_kv_heads + head) << sh) + (p.y & mask);
  };

  if (over <= kFew) {
    // the `over` smallest, one at a time; every warp ends up with all of them
    int evicted = -1;  // lane i < over: the i-th
    uint64_t last = 0ull;
    for (int e = 0; e < over; ++e) {
      if (e > 0) {
        least = ~0ull;
        each_row([&](uint32_t k, int r) {
          const uint64_t x = rank_of(k, r);
          if (x > last) least = min(least, x);
        });
      }
      const uint64_t w = warp_min(least);
      if (lane == 0) s_min[e][warp] = w;
      __syncthreads();
      uint64_t m = warp_min(lane < NW ? s_min[e][lane] : ~0ull);
      if (csize > 1) {
        if (tid == 0) s_cta_min[e] = m;
        pa::cluster_sync_all();
        m = warp_min(lane < csize ? dsmem_ld_u64(pa::dsmem_map(pa::smem_u32(&s_cta_min[e]), lane)) : ~0ull);
      }
      last = m;
      if (lane == e) evicted = (int)~(uint32_t)m;
    }
    // no CTA leaves, and no copied ledger row is written again, before all are done
    group_sync(csize);
    if (crank != 0 || warp != 0) return;
    // holes: evicted rows below the budget, in order; sources: rows past it that stay
    const bool is_hole = lane < over && evicted < a.budget;
    int hole_rank = 0;
    bool gone = false;  // row budget + lane is evicted
    for (int e = 0; e < over; ++e) {
      const int x = __shfl_sync(0xffffffffu, evicted, e);
      hole_rank += x < evicted;
      gone |= x == a.budget + lane;
    }
    const bool is_src = lane < over && !gone;
    const unsigned srcs = __ballot_sync(0xffffffffu, is_src);
    if (is_hole) s_moves[hole_rank].x = evicted;
    if (is_src) s_moves[__popc(srcs & below)].y = a.budget + lane;
    __syncwarp();
    const int m = __popc(srcs);
    int64_t rt = -1, rf = -1;
    if (lane < m) start_move(s_moves[lane], rt, rf);
    copy_rows(a, rt, rf, m);
    return;
  }

  // radix select of the budget-th largest key, from the top byte down: `prefix` holds
  // the bytes known so far, `left` how many rows with that prefix are still to keep
  uint32_t prefix = 0;
  int left = a.budget;
  __syncthreads();  // zeroed counts
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t mask = pass == 0 ? 0u : ~0u << (shift + 8);
    each_row([&](uint32_t k, int) {
      if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> shift) & 255u], 1);
    });
    group_sync(csize);
    if (warp == 0) {
      // lane l takes digits 255 - 8 l .. 248 - 8 l, highest first
      int cnt[8], part = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = 255 - 8 * lane - i;
        cnt[i] = hist[pass][d];
      }
      if (csize > 1) {
        for (int c = 1; c < csize; ++c) {
          const int peer = crank + c < csize ? crank + c : crank + c - csize;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cnt[i] += pa::dsmem_ld_s32(pa::dsmem_map(pa::smem_u32(&hist[pass][255 - 8 * lane - i]), peer));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) part += cnt[i];
      int incl = part;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      int run = incl - part;
      if (run < left && incl >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (run < left && run + cnt[i] >= left) {
            s_digit = 255 - 8 * lane - i;
            s_left = left - run;
          }
          run += cnt[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    left = s_left;
    __syncthreads();
  }
  const uint32_t border = prefix;  // rows above it are kept, and the first `left` equal to it

  // how many rows of each kind every warp holds; from those, where its holes (evicted rows
  // below the budget) and sources (kept rows from there on) stand in the lists
  Counts mine = {0, 0, 0, 0, 0};
  each_row([&](uint32_t k, int r) {
    const bool low = r < a.budget;
    mine.gt_lo += k > border && low;
    mine.gt_hi += k > border && !low;
    mine.eq_lo += k == border && low;
    mine.eq_hi += k == border && !low;
  });
  mine.gt_lo = __reduce_add_sync(0xffffffffu, mine.gt_lo);
  mine.gt_hi = __reduce_add_sync(0xffffffffu, mine.gt_hi);
  mine.eq_lo = __reduce_add_sync(0xffffffffu, mine.eq_lo);
  mine.eq_hi = __reduce_add_sync(0xffffffffu, mine.eq_hi);
  mine.n_lo = max(0, min(w1, a.budget) - w0);
  if (lane == 0) s_cnt[warp] = mine;
  __syncthreads();
  if (csize > 1 && tid == 0) {
    Counts all = {0, 0, 0, 0, 0};
    for (int w = 0; w < NW; ++w) {
      all.gt_lo += s_cnt[w].gt_lo;
      all.gt_hi += s_cnt[w].gt_hi;
      all.eq_lo += s_cnt[w].eq_lo;
      all.eq_hi += s_cnt[w].eq_hi;
      all.n_lo += s_cnt[w].n_lo;
    }
    s_pub = all;
  }
  if (csize > 1) pa::cluster_sync_all();
  int t = 0, nh = 0, ns = 0, m = 0;  // equal rows, holes, sources before this warp; sources in all
  {
    int tt = 0;
    for (int c = 0; c < csize; ++c) {
      if (c == crank) {
        t = tt;
        for (int w = 0; w < NW; ++w) {
          const Counts x = s_cnt[w];
          if (w < warp) {
            nh += x.holes(tt, left);
            ns += x.sources(tt, left);
            t += x.eq_lo + x.eq_hi;
          }
          m += x.sources(tt, left);
          tt += x.eq_lo + x.eq_hi;
        }
      } else {
        Counts x;
        const uint32_t at = pa::dsmem_map(pa::smem_u32(&s_pub), c);
        x.gt_lo = pa::dsmem_ld_s32(at);
        x.gt_hi = pa::dsmem_ld_s32(at + 4);
        x.eq_lo = pa::dsmem_ld_s32(at + 8);
        x.eq_hi = pa::dsmem_ld_s32(at + 12);
        x.n_lo = pa::dsmem_ld_s32(at + 16);
        if (c < crank) {
          nh += x.holes(tt, left);
          ns += x.sources(tt, left);
        }
        m += x.sources(tt, left);
        tt += x.eq_lo + x.eq_hi;
      }
    }
  }
  int2 *moves = csize == 1 && m <= kListCap ? s_moves : a.moves + (int64_t)unit * a.budget;
  for (int r0 = w0; r0 < w1; r0 += 32) {
    const int r = r0 + lane;
    const uint32_t k = r < w1 ? key(r) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, r < w1 && k == border);
    const bool kept = r < w1 && (k > border || (k == border && t + __popc(eq & below) < left));
    t += __popc(eq);
    const unsigned hb = __ballot_sync(0xffffffffu, r < w1 && !kept && r < a.budget);
    const unsigned sb = __ballot_sync(0xffffffffu, kept && r >= a.budget);
    if ((hb >> lane) & 1u) moves[nh + __popc(hb & below)].x = r;
    if ((sb >> lane) & 1u) moves[ns + __popc(sb & below)].y = r;
    nh += __popc(hb);
    ns += __popc(sb);
  }
  group_sync(csize);  // the whole list, and every read of the old ledgers, before the moves

  const int warps = csize * NW;
  const int batch = min(32, (m + warps - 1) / warps);
  for (int i0 = (crank * NW + warp) * batch; i0 < m; i0 += warps * batch) {
    const int cnt = min(batch, m - i0);
    int64_t rt = -1, rf = -1;
    if (lane < cnt) start_move(moves[i0 + lane], rt, rf);
    copy_rows(a, rt, rf, cnt);
  }
  // (distributed shared memory was last read before the barrier above)
}

// Tables of at most so many rows: CTAs of 256 threads, one per head; longer ones: 512, and
// clusters of them.  Half the rows kept of 1024, 4096 and 8192, 64 x 8 heads: 42, 129 and
// 257 us the first way, 46, 137 and 252 the second; 16 x 8 heads: 17.5, 62 and 134 against
// 19.4, 48 and 78; one row over 1023, 4095 and 8191, 64 x 8 heads: 5.0, 7.3 and 10.6
// against 8.5, 10.2 and 13.5.  (The table's width stands for the contexts, whose lengths
// the host does not know: 1025 rows of 64 x 8 heads in tables of 1040 or 4096 rows 5.3 us,
// 8192 8.1, 32768 12.7.)
constexpr int kSmallRows = 4096;

template <int NT>
cudaError_t launch_evict(const EvictArgs &a, unsigned units, int cluster, int smem, cudaStream_t s) {
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kKeyCap * (int)sizeof(uint32_t));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster, 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<NT>, a);
}

}  // namespace

extern "C" PA_API size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int budget) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || budget <= 0) return 0;
  return (size_t)num_seqs * num_kv_heads * budget * 2 * sizeof(int32_t);
}

extern "C" PA_API pa_status pa_evict(
    void *k_cache, void *v_cache, float *scores_out, int32_t *row_pos_out, int32_t *new_lens,
    const float *scores, const int32_t *row_pos, const int32_t *block_tables,
    const int32_t *context_lens, const int32_t *seq_lens, int num_seqs, int num_kv_heads,
    int head_dim, int block_size, int max_blocks_per_seq, int num_blocks, int budget, int sinks,
    int recent, int element_bytes, void *workspace, size_t workspace_bytes, void *stream) {
  if (!k_cache || !v_cache || !scores_out || !row_pos_out || !new_lens || !scores || !row_pos ||
      !block_tables || !context_lens || !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  if (num_seqs <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (budget <= 0 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return PA_ERR_INVALID_ARG;
  // the ledgers are both updated in place or both written elsewhere
  if ((scores == scores_out) != (row_pos == row_pos_out)) return PA_ERR_INVALID_ARG;
  const void *ptrs[7] = {k_cache, v_cache, workspace, scores, row_pos, scores_out, row_pos_out};
  for (const void *p : ptrs)
    if (!pa::aligned16(p)) return PA_ERR_INVALID_ARG;
  if (element_bytes != 1 && element_bytes != 2) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (element_bytes == 1 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!pa::supported_block(block_size)) return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size >= (int64_t)1 << 30) return PA_ERR_INVALID_ARG;
  if ((int64_t)num_seqs * num_kv_heads >= (int64_t)1 << 31) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < pa_evict_workspace_size(num_seqs, num_kv_heads, budget))
    return PA_ERR_INVALID_ARG;
  // every KV head reads the old lengths while one writes the new; ledgers are updated in
  // place or quite apart
  const size_t lens = (size_t)num_seqs * sizeof(int32_t);
  const size_t ledger = (size_t)num_seqs * num_kv_heads * max_blocks_per_seq * block_size * 4;
  if (pa::overlap(new_lens, lens, context_lens, lens) || pa::overlap(new_lens, lens, seq_lens, lens))
    return PA_ERR_INVALID_ARG;
  if (scores != scores_out &&
      (pa::overlap(scores_out, ledger, scores, ledger) || pa::overlap(row_pos_out, ledger, row_pos, ledger) ||
       pa::overlap(scores_out, ledger, row_pos, ledger) || pa::overlap(row_pos_out, ledger, scores, ledger)))
    return PA_ERR_INVALID_ARG;
  EvictArgs a;
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.scores = scores;
  a.row_pos = row_pos;
  a.scores_out = scores_out;
  a.row_pos_out = row_pos_out;
  a.new_lens = new_lens;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.seq_lens = seq_lens;
  a.moves = static_cast<int2 *>(workspace);
  a.num_kv_heads = num_kv_heads;
  a.block_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.max_rows = max_blocks_per_seq * block_size;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.row_chunks = head_dim * element_bytes / 16;
  a.err = pa::error_word();
  if (a.err == nullptr) return PA_ERR_CUDA;
  // few units: a cluster each, while the clusters' CTAs fill at most about two per SM
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  const long long units = (long long)num_seqs * num_kv_heads;
  int cluster = 1;
  if (a.max_rows > kSmallRows)
    while (cluster < kMaxCluster && units * cluster * 2 <= 2LL * sms) cluster *= 2;
  if (units * cluster >= 1LL << 31) return PA_ERR_INVALID_ARG;
  const int slice = ((a.max_rows + cluster - 1) / cluster + 31) & ~31;
  a.key_cap = std::min(slice, kKeyCap);
  const int smem = a.key_cap * (int)sizeof(uint32_t);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.max_rows > kSmallRows ? launch_evict<512>(a, (unsigned)units, cluster, smem, s)
                                                : launch_evict<256>(a, (unsigned)units, cluster, smem, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
