// pa_mass_tc.cuh -- the attention weight that each cached row draws from many query
// rows, on the 5th-generation tensor cores: the second look of scored attention at its
// scores when they are too many to keep.
//
// For cached row t of KV head h:  share(t) = sum_r 2^(c s_rt - m_r - log2 l_r)  over the
// head's query rows r that see t, with s = q . k, c = scale * log2(e) (times the K scale
// of an FP8 cache) and -(m_r + log2 l_r) from the attention pass.
//
// S^T is computed with the cached rows as the MMA's M, so that a thread of the epilogue
// owns one cached row (a TMEM lane) and adds up its columns alone: no reduction across
// threads, one order of summation.  The K rows are the MMA's A operand in tensor memory:
// the thread that owns a row gathers it through the block table (any block size; bad
// blocks read as zeros; e4m3 codes widened on the way, exact in fp16 and bf16) and stores
// it once per unit.  Only Q passes through shared memory, 128 rows at a time by TMA, and
// each of its tiles serves two chunks of 128 cached rows: 32 KiB of L2 reads for two
// 128 x 128 x 128 products.
//   warp 0      TMA producer of the Q blocks (ring of NQ stages)
//   warp 1      owns tensor memory, issues the MMAs
//   warp 2      the Q block's row statistics and causal limits into a ring
//   warps 4-19  epilogue: four warps (the TMEM lane quarters) for each chunk of the unit
//               and each half of a tile's 128 columns; the two halves of a cached row's
//               sum meet at the unit's end
// A unit is 256 cached rows of one KV head.  CTAs are persistent, one per SM; rings,
// buffers and barrier phases run on from unit to unit.  Every wait is bounded.
//
// Order of the units: those that every query token sees first (equal work), then the
// ones among the new rows by how far they lie behind the first of them (less and less
// work); CTA c takes c, 2G - 1 - c, 2G + c, ...  On 4 x 1024 query tokens over contexts
// of 2259..8167 (32/8 heads) the busiest of 152 CTAs has 136 blocks' work against 133 on
// average, 165 in the plain order.
#pragma once

#include "pa_prefill_tc.cuh"
#include "pa_scored.h"

namespace pa {

constexpr int kMassChunk = 128;                // cached rows per MMA (M)
constexpr int kMassUnit = 2 * kMassChunk;      // per unit
constexpr int kMassCols = 128;                 // query rows per MMA (N)
constexpr int kMassCtl = 4, kMassEpi = 16;
constexpr int kMassThreads = 32 * (kMassCtl + kMassEpi);
constexpr int kMassStats = 4;                  // ring of row statistics
constexpr int kMassBufs = 3;                   // accumulators in flight
constexpr int kMassMaxSeqs = 4096;             // per launch (their units' prefix sums)

template <int D>
struct MassLayout {
  static constexpr int kNQ = 4;
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = kHalves * kMassCols * 128;  // [half][128 rows][128 B]
  static constexpr int smem_bytes(int num_seqs) {
    return kNQ * kQBytes + 1024 + (2 * num_seqs + 1) * (int)sizeof(int);
  }
  static constexpr int kColD = 128;  // accumulators after the A operand (2 x D/2 columns)
};

struct MassUnitInfo {
  int valid, seq, kvh, t0, Lc, L, u0, nblk;
};

// heads and tokens of a Q block (hb * tb <= 128 rows), blocks that cover a head group
struct MassGeo {
  int hb, tb, nhb;
};
__host__ __device__ __forceinline__ MassGeo mass_geo(int group) {
  MassGeo g;
  g.hb = group < kMassCols ? group : kMassCols;
  g.tb = kMassCols / g.hb;
  g.nhb = (group + g.hb - 1) / g.hb;
  return g;
}

// The unit list, in shared memory: start[i] = full units (seen by every query token) of
// the sequences before i; partial[i] = sequence i's units that only some query tokens see;
// level[j] = units of the list before the j-th partial units of all sequences.
constexpr int kMassLevels = 4096 / kMassUnit + 2;  // (q_len is at most 4096)
struct MassList {
  const int *start, *partial, *level;
};

// The k-th unit of this CTA (all lanes of a warp call it).
__device__ __forceinline__ MassUnitInfo mass_unit(const LedgerArgs &a, const MassGeo &geo,
                                                  const MassList &list, int k) {
  MassUnitInfo t;
  const int G = gridDim.x;
  const long long id = (long long)k * G + ((k & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
  t.valid = id < list.level[kMassLevels];
  if (!t.valid) return t;
  int chunk;
  if (id < list.level[0]) {
    int lo = 0, hi = a.num_seqs;  // start[lo] <= id < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (list.start[mid] <= id) lo = mid; else hi = mid;
    }
    t.seq = lo;
    const int rem = (int)id - list.start[lo];
    chunk = rem / a.num_kv_heads;
    t.kvh = rem % a.num_kv_heads;
  } else {
    int j = 0;
    while (list.level[j + 1] <= id) ++j;
    const int rem = (int)id - list.level[j], want = rem / a.num_kv_heads;
    t.kvh = rem % a.num_kv_heads;
    // the sequence that is number `want` of those with more than j partial units
    const int lane = threadIdx.x & 31;
    int seen = 0;
    t.seq = 0;
    for (int i0 = 0; i0 < a.num_seqs; i0 += 32) {
      const unsigned has = __ballot_sync(0xffffffffu, i0 + lane < a.num_seqs && list.partial[i0 + lane] > j);
      const int n = __popc(has);
      if (want < seen + n) {
        t.seq = i0 + (int)__fns(has, 0, want - seen + 1);
        break;
      }
      seen += n;
    }
    chunk = (list.start[t.seq + 1] - list.start[t.seq]) / a.num_kv_heads + j;
  }
  t.t0 = chunk * kMassUnit;
  t.Lc = max(0, __ldg(a.context_lens + t.seq));
  t.L = min(t.Lc, a.max_rows);
  t.u0 = max(0, t.t0 - (t.Lc - a.q_len));  // earlier query tokens see none of these rows
  t.nblk = (a.q_len - t.u0 + geo.tb - 1) / geo.tb * geo.nhb;
  return t;
}

template <typename T, int D, bool KV8>
__global__ void __launch_bounds__(kMassThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap qmap, const LedgerArgs a) {
  using Lay = MassLayout<D>;
  constexpr int NQ = Lay::kNQ, H = Lay::kHalves;
  constexpr bool kBf16 = Elt<T>::kMantBits < 10;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[NQ], q_empty[NQ];
  // accumulator i (2 per Q block) uses buffer i % 3; its "full" barrier is i % 6, so that
  // each is waited on by one epilogue group at every phase (a group sees every other i)
  __shared__ __align__(8) uint64_t d_full[2 * kMassBufs], d_empty[kMassBufs];
  __shared__ __align__(8) uint64_t st_full[kMassStats], st_empty[kMassStats];
  __shared__ __align__(8) uint64_t a_full, a_free, mma_fin;
  __shared__ __align__(8) uint64_t h_full[8], h_free[8];  // per chunk and lane quarter
  __shared__ __align__(16) float s_nlse[kMassStats][kMassCols];
  __shared__ __align__(16) int s_lim[kMassStats][kMassCols];
  __shared__ float s_half[kMassUnit];            // the second column half's sums
  __shared__ int s_level[kMassLevels + 1];
  __shared__ int s_failed;
  __shared__ uint32_t s_tmem;

  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  int *s_start = reinterpret_cast<int *>(smem_raw + (base - smem_u32(smem_raw)) + NQ * Lay::kQBytes);
  int *s_partial = s_start + a.num_seqs + 1;
  const MassList list = {s_start, s_partial, s_level};

  // the unit list
  if (warp == 0) {
    int run = 0;
    int at_least = 0;  // lane j: sequences with more than j partial units
    for (int i0 = 0; i0 < a.num_seqs; i0 += 32) {
      const int i = i0 + lane;
      int n = 0, part = 0;
      if (i < a.num_seqs) {
        const int Lc = max(0, __ldg(a.context_lens + i)), L = min(Lc, a.max_rows);
        const int all = (L + kMassUnit - 1) / kMassUnit;
        // unit c is full while its first row c * 256 <= Lc - q_len
        const int full = Lc >= a.q_len ? min(all, (Lc - a.q_len) / kMassUnit + 1) : 0;
        n = full * a.num_kv_heads;
        part = all - full;
        s_partial[i] = part;
      }
#pragma unroll 1
      for (int j = 0; j < kMassLevels; ++j) {
        const int cnt = __popc(__ballot_sync(0xffffffffu, part > j));
        if (lane == j) at_least += cnt;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (i < a.num_seqs) s_start[i] = run + incl - n;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_start[a.num_seqs] = run;
    int incl = at_least * a.num_kv_heads;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 0) s_level[0] = run;
    if (lane < kMassLevels) s_level[lane + 1] = run + incl;
  }
  // Q rows that no TMA box writes (a head group that does not divide 128) stay zero
  for (int i = threadIdx.x; i < NQ * Lay::kQBytes / 16; i += kMassThreads) sts128_zero(base + 16 * i);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    s_failed = 0;
    for (int s = 0; s < NQ; ++s) {
      mbar_init(smem_u32(&q_full[s]), 1);
      mbar_init(smem_u32(&q_empty[s]), 1);
    }
    for (int s = 0; s < kMassBufs; ++s) {
      mbar_init(smem_u32(&d_full[2 * s]), 1);
      mbar_init(smem_u32(&d_full[2 * s + 1]), 1);
      mbar_init(smem_u32(&d_empty[s]), kMassEpi / 2);  // a chunk's warps
    }
    for (int s = 0; s < kMassStats; ++s) {
      mbar_init(smem_u32(&st_full[s]), 1);
      mbar_init(smem_u32(&st_empty[s]), kMassEpi);
    }
    for (int s = 0; s < 8; ++s) {
      mbar_init(smem_u32(&h_full[s]), 1);
      mbar_init(smem_u32(&h_free[s]), 1);
    }
    mbar_init(smem_u32(&a_full), kMassEpi);
    mbar_init(smem_u32(&a_free), 1);
    mbar_init(smem_u32(&mma_fin), 1);
    fence_mbar_init();
    prefetch_tensormap(&qmap);
  }
  if (warp == 1) {
    tc::alloc(smem_u32(&s_tmem), 512);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  volatile int *failed = &s_failed;
  const MassGeo geo = mass_geo(a.group);
  bool ok = true;
  auto wait = [&](uint64_t *bar, int parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
    const bool w = mbar_wait_bounded(smem_u32(bar), parity);
    ok = __all_sync(0xffffffffu, w) && !*failed;
    return ok;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ Q blocks
    int g = 0;  // blocks of this CTA so far
    for (int k = 0; ok; ++k) {
      const MassUnitInfo t = mass_unit(a, geo, list, k);
      if (!t.valid) break;
      for (int b = 0; b < t.nblk; ++b, ++g) {
        const int s = g % NQ;
        if (!wait(&q_empty[s], ((g / NQ) & 1) ^ 1)) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&q_full[s]);
          mbar_arrive_expect_tx(bar, (uint32_t)(H * geo.hb * geo.tb * 128));
          const int tok = t.seq * a.q_len + t.u0 + b / geo.nhb * geo.tb;
          const int head = t.kvh * a.group + b % geo.nhb * geo.hb;
#pragma unroll
          for (int hh = 0; hh < H; ++hh)
            tma_load_3d(base + s * Lay::kQBytes + hh * (kMassCols * 128), &qmap, hh * 64, head, tok, bar);
        }
        __syncwarp();
      }
    }
    // the last loads have landed before the CTA may exit
    for (int i = max(0, g - NQ); i < g; ++i)
      (void)mbar_wait_bounded(smem_u32(&q_full[i % NQ]), (i / NQ) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    constexpr uint32_t kId = tc::idesc_f16(kMassChunk, kMassCols, kBf16, false);
    const uint64_t dQ = tc::sdesc_sw128(base, 16, 1024);
    int g = 0;
    for (int k = 0; ok; ++k) {
      const MassUnitInfo t = mass_unit(a, geo, list, k);
      if (!t.valid) break;
      if (!wait(&a_full, k & 1)) break;
      for (int b = 0; ok && b < t.nblk; ++b, ++g) {
        const int s = g % NQ;
        if (!wait(&q_full[s], (g / NQ) & 1)) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int i = 2 * g + c, buf = i % kMassBufs;
          if (!wait(&d_empty[buf], ((i / kMassBufs) & 1) ^ 1)) break;
          tc::fence_after();
          if (lane == 0) {
            const uint64_t qd = dQ + (uint64_t)((s * Lay::kQBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_f16_ts(tmem + Lay::kColD + kMassCols * buf, tmem + c * (D / 2) + kk * 8,
                             qd + (uint64_t)(((kk >> 2) * (kMassCols * 128) + (kk & 3) * 32) >> 4), kId,
                             kk > 0 ? 1u : 0u);
            tc::commit(smem_u32(&d_full[i % (2 * kMassBufs)]));
            if (c == 1) tc::commit(smem_u32(&q_empty[s]));
            if (c == 1 && b == t.nblk - 1) tc::commit(smem_u32(&a_free));
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) tc::commit(smem_u32(&mma_fin));
    __syncwarp();
    (void)mbar_wait_bounded(smem_u32(&mma_fin), 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------ row statistics
    // The columns of a block are the same (token, head) offsets in every block: worked
    // out once.  The next block's statistics are loaded before the wait for a free slot
    // of the ring: with the load's latency in every block, this warp bounded the kernel
    // (399 us for 4 x 1024 query tokens, 32/8 heads, contexts of 2048..8192).
    constexpr int kPer = kMassCols / 32;
    int du[kPer], dh[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int col = lane + 32 * i;
      du[i] = col < geo.hb * geo.tb ? col / geo.hb : a.q_len;  // past every token: no row
      dh[i] = col % geo.hb;
    }
    int g = 0;
    for (int k = 0; ok; ++k) {
      const MassUnitInfo t = mass_unit(a, geo, list, k);
      if (!t.valid) break;
      const float *stat = a.row_nlse + ((size_t)t.seq * a.num_kv_heads + t.kvh) * a.rows;
      float nlse[kPer], next[kPer];
      int lim[kPer], lim_next[kPer];
      // lim: the last cached row that the query row sees (-1: no query row)
      auto load = [&](int b, float (&n)[kPer], int (&m)[kPer]) {
        const int u0 = t.u0 + b / geo.nhb * geo.tb, h0 = b % geo.nhb * geo.hb;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int u = u0 + du[i], h = h0 + dh[i];
          const bool in = b < t.nblk && u < a.q_len && h < a.group;
          n[i] = in ? __ldg(stat + (size_t)u * a.group + h) : 0.f;
          m[i] = in ? t.Lc - a.q_len + u : -1;
        }
      };
      load(0, nlse, lim);
      for (int b = 0; b < t.nblk; ++b, ++g) {
        const int s = g % kMassStats;
        load(b + 1, next, lim_next);
        if (!wait(&st_empty[s], ((g / kMassStats) & 1) ^ 1)) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          s_nlse[s][lane + 32 * i] = nlse[i];
          s_lim[s][lane + 32 * i] = lim[i];
          nlse[i] = next[i];
          lim[i] = lim_next[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&st_full[s]));
      }
    }
  } else if (warp >= kMassCtl) {
    // ------------------------------------------------------------ epilogue
    const int c = ((warp - kMassCtl) >> 2) & 1, half = (warp - kMassCtl) >> 3;
    const int quarter = warp & 3;  // TMEM lanes this warp may touch
    const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
    int g = 0;
    for (int k = 0; ok; ++k) {
      const MassUnitInfo t = mass_unit(a, geo, list, k);
      if (!t.valid) break;
      const int t_first = t.t0 + c * kMassChunk;
      const int pos = t_first + 32 * quarter + lane;
      // this thread's cached row (its half of head_dim): the A operand's lane
      {
        constexpr int kHalfBytes = D / 2 * (KV8 ? 1 : 2), kWords = D / 4;
        const uint8_t *row = nullptr;
        if (pos < t.L) {
          const int id = __ldg(a.block_tables + (size_t)t.seq * a.max_blocks_per_seq + pos / a.block_size);
          if (id >= 0 && id < a.num_blocks)  // (the attention pass has reported a bad one)
            row = static_cast<const uint8_t *>(a.k_cache) +
                  (((size_t)id * a.num_kv_heads + t.kvh) * a.block_size + pos % a.block_size) *
                      (2 * kHalfBytes) +
                  half * kHalfBytes;
        }
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kHalfBytes / 16; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row) v = __ldg(reinterpret_cast<const uint4 *>(row) + i);
          if constexpr (KV8) {
            float f[16];
            e4m3x16_to_f32(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[8 * i + e] = Elt<T>::from_f2(f[2 * e], f[2 * e + 1]);
          } else {
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
          }
        }
        if (k > 0 && !wait(&a_free, (k - 1) & 1)) break;
        tc::fence_after();
        const uint32_t dst = trow + c * (D / 2) + half * kWords;
        if constexpr (kWords == 32) {
          tc::st32u(dst, w);
        } else {
#pragma unroll
          for (int j = 0; j < kWords / 8; ++j) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = w[8 * j + i];
            tc::st8u(dst + 8 * j, x);
          }
        }
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&a_full));
      }
      const float cs = a.scale_log2 * (KV8 ? __ldg(a.k_scale + t.kvh) : 1.f);
      const uint64_t cs2 = tc::f2pack(cs, cs);
      float share = 0.f;
      for (int b = 0; b < t.nblk; ++b, ++g) {
        const int s = g % kMassStats, i = 2 * g + c, buf = i % kMassBufs;
        if (!wait(&d_full[i % (2 * kMassBufs)], (i / (2 * kMassBufs)) & 1)) break;
        tc::fence_after();
        // this warp's 64 columns to registers, and the accumulator is free again
        float sv[64];
        tc::ld64(trow + Lay::kColD + kMassCols * buf + 64 * half, sv);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&d_empty[buf]));
        if (!wait(&st_full[s], (g / kMassStats) & 1)) break;
        const int u0 = t.u0 + b / geo.nhb * geo.tb, h0 = b % geo.nhb * geo.hb;
        // every column a query row that sees the whole chunk?
        const bool plain = geo.hb * geo.tb == kMassCols && u0 + geo.tb <= a.q_len &&
                           h0 + geo.hb <= a.group && t.Lc - a.q_len + u0 >= t_first + kMassChunk - 1;
        const float *nl = &s_nlse[s][64 * half];
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
        if (plain) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 n = *reinterpret_cast<const float4 *>(nl + e);
            float x0, x1, x2, x3;
            tc::f2unpack(tc::ffma2(tc::f2pack(sv[e], sv[e + 1]), cs2, tc::f2pack(n.x, n.y)), x0, x1);
            tc::f2unpack(tc::ffma2(tc::f2pack(sv[e + 2], sv[e + 3]), cs2, tc::f2pack(n.z, n.w)), x2, x3);
            sum[(e >> 1) & 3] = tc::fadd2(sum[(e >> 1) & 3], tc::f2pack(ex2_ftz(x0), ex2_ftz(x1)));
            sum[((e >> 1) + 1) & 3] =
                tc::fadd2(sum[((e >> 1) + 1) & 3], tc::f2pack(ex2_ftz(x2), ex2_ftz(x3)));
          }
        } else {
          const int *lm = &s_lim[s][64 * half];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const float2 n = *reinterpret_cast<const float2 *>(nl + e);
            const int2 lim = *reinterpret_cast<const int2 *>(lm + e);
            const float p0 = pos <= lim.x ? ex2_ftz(fmaf(sv[e], cs, n.x)) : 0.f;
            const float p1 = pos <= lim.y ? ex2_ftz(fmaf(sv[e + 1], cs, n.y)) : 0.f;
            sum[(e >> 1) & 3] = tc::fadd2(sum[(e >> 1) & 3], tc::f2pack(p0, p1));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&st_empty[s]));
        float x, y;
        tc::f2unpack(tc::fadd2(tc::fadd2(sum[0], sum[1]), tc::fadd2(sum[2], sum[3])), x, y);
        share += x + y;
      }
      // the halves of a row's columns meet: the second half's sum through shared memory
      const int pair = 4 * c + quarter, slot = kMassChunk * c + 32 * quarter + lane;
      if (!ok) break;
      if (half == 1) {
        if (k > 0 && !wait(&h_free[pair], (k - 1) & 1)) break;
        s_half[slot] = share;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&h_full[pair]));
      } else {
        if (!wait(&h_full[pair], k & 1)) break;
        share += s_half[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&h_free[pair]));
        if (pos < t.L) {
          const int64_t at = ((int64_t)t.seq * a.num_kv_heads + t.kvh) * a.max_rows + pos;
          ledger_write(a.scores, a.row_pos, a.seq_lens, t.seq, at, pos, t.Lc, a.q_len, a.scores[at], share);
        }
      }
    }
  }
  if (!ok && lane == 0) {
    record_error(a.err, kErrTimeout);
    atomicExch(&s_failed, 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

}  // namespace pa
