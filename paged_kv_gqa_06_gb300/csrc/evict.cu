// Choosing among cached tokens by weight: adding a decode's attention weights
// to running totals, selecting the tokens to keep, and moving kept tokens
// together in the paged cache.
#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace forge {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// All of these kernels start while the grid before them may still run, so what
// that grid can have written (totals, lists, lengths, tables) is read with
// ordinary loads after the wait, never with non-coherent ones, whose data must
// not change while a kernel lives.

// Length of sequence b, clamped to [0, most]; a length outside is recorded.
// AHEAD: read before the wait, past L1.
template <bool AHEAD = false>
__device__ __forceinline__ int length_of(const int32_t* lens, int b, int most, int* err, bool report) {
  int L = AHEAD ? __ldcg(lens + b) : lens[b];
  if (L < 0 || L > most) {
    if (report) record_error(err, kDevErrLength);
    L = L < 0 ? 0 : most;
  }
  return L;
}

// ------------------------------------------------------------------ totals
// weights[b, g, t] += sum_h 2^(logit - max_h) / sum_h over the G heads of
// group g, from the logits the decode left.  One thread per 4 tokens; the sum
// runs over the heads in order, so it repeats bit for bit.  The decode's CTAs
// let this grid start once they have all seen the previous grid complete:
// lengths and old totals are read while the decode still runs, and only the
// logits and norms (in L2 by then) after it.
// A warp reads 32 tokens' G floats with each load: with four neighbouring
// tokens a thread, a load touched 16 lines and the kernel was bound by L1.
// What it adds to the decode: 5.7 us alone for 32 sequences of 512-8192 tokens
// (18 MB of logits from L2, 9 MB of totals).
constexpr int kAccThreads = 256;
constexpr int kAccEach = 4;  // tokens of a thread, kAccThreads apart
constexpr int kAccTokens = kAccEach * kAccThreads;

template <int G>
__global__ void __launch_bounds__(kAccThreads, G <= 4 ? 8 : 5) accumulate_weights_kernel(const WeightsParams p) {
  griddep_launch_dependents();
  const int g = blockIdx.y, b = blockIdx.z;
  int L = length_of<true>(p.context_lens, b, p.MB * kBlockSize, nullptr, false);  // recorded by the decode
  if (L > p.S) {
    if (g == 0 && blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, kDevErrLength);
    L = p.S;
  }
  const int t0 = blockIdx.x * kAccTokens + threadIdx.x;
  if (t0 >= L) {
    // before the wait: blocks past the sequence hold no place on the SMs.  Its
    // first block waits all the same, so that this grid is never complete
    // before the decode, whatever the lengths: what follows waits for this
    // grid alone.
    if (blockIdx.x == 0) griddep_wait();
    return;
  }
  float* dst = p.weights + b * p.w_sb + g * p.w_sh + t0;
  float w[kAccEach];
#pragma unroll
  for (int e = 0; e < kAccEach; ++e) w[e] = t0 + e * kAccThreads < L ? __ldcg(dst + e * kAccThreads) : 0.f;
  griddep_wait();  // the decode that writes the logits is complete
  float2 nm[G];
#pragma unroll
  for (int h = 0; h < G; ++h) nm[h] = __ldcg(p.norm + (static_cast<int64_t>(b) * p.Hkv + g) * G + h);
  const float* src =
      p.logits + ((static_cast<int64_t>(b) * p.Hkv + g) * (static_cast<int64_t>(p.MB) * kBlockSize) + t0) * G;
  float x[kAccEach][G];
#pragma unroll
  for (int e = 0; e < kAccEach; ++e) {
    if (t0 + e * kAccThreads >= L) continue;
    const float* at = src + e * kAccThreads * G;
    if constexpr (G == 1) {
      x[e][0] = __ldcg(at);
    } else if constexpr (G == 2) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(at));
      x[e][0] = v.x;
      x[e][1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < G; i += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(at + i));
        x[e][i] = v.x;
        x[e][i + 1] = v.y;
        x[e][i + 2] = v.z;
        x[e][i + 3] = v.w;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kAccEach; ++e) {
    if (t0 + e * kAccThreads >= L) continue;
    float add = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) add = fmaf(fast_exp2(x[e][h] - nm[h].x), nm[h].y, add);
    dst[e * kAccThreads] = w[e] + add;
  }
}

// --------------------------------------------------------------- selection
// An ordinary load that the compiler leaves where it is.  (Merged with the
// shared-memory side of the choice it is used in, it took the kernel past 32
// registers a thread and one CTA off each SM: 256 lists 13.6 -> 14.9 us.)
__device__ __forceinline__ float ld_here(const float* ptr) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(ptr) : "memory");
  return v;
}

// Weights as unsigned keys of the same order: NaN as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// One cluster per (sequence, KV head); each CTA takes an equal run of the
// middle's positions and holds their keys in shared memory (a run longer than
// that is read again from L2).  Radix selection from the top, 11 + 11 + 10
// bits: a pass counts the digits of the keys that match the digits found so
// far, the cluster's CTAs add their counts up through distributed shared
// memory, and every CTA finds the digit that holds the last token kept.  When
// all keys of that digit are kept the threshold is known: two passes for most
// lists (22 bits tell their keys apart), three for lists of equal totals.
// Kept are the keys above the threshold and the first `need` that match it;
// each thread counts both over a run of its own, a scan over threads and CTAs
// ranks them, and the positions go out in order.
//
// What bounds it: the latency of these steps and the instructions of their
// scans; a list is tens of KB.  Wide digits and one CTA for lists of up to
// 8192 keep the steps few.  256 lists of 512 to 8192 tokens: 13.7 us (24.8 us
// with four 8-bit passes over clusters of two CTAs of 512 threads; 16.5 us
// with 512 threads here); one of 32768 for each of 8 heads: 16.7 us over
// clusters of 8 (34 us while every CTA read all of the others' 2048 counters
// and not the groups' sums first).
constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCap = 8192;   // keys a CTA holds
constexpr int kSelAhead = 8;    // loads of a thread under way

struct SelectShared {
  int hist[2][kSelBins];  // this CTA's counts, by pass parity: read by the cluster
  int coarse[2][64];      // and their sums over 32 digits
  int sums[64], digits[32];  // the cluster's sums
  int tail[64];           // scan scratch
  int counts[2];          // this CTA's keys above and at the threshold: read by the cluster
};

// Exclusive scan over the block of two counters; `total` of both.
__device__ __forceinline__ int2 block_scan2(int a, int b, int* scratch, int lane, int warp, int2& total) {
  static_assert(kSelThreads == 1024, "a warp sum per lane");
  int x = a, y = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(kFull, x, off), v = __shfl_up_sync(kFull, y, off);
    if (lane >= off) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    scratch[warp] = x;
    scratch[32 + warp] = y;
  }
  __syncthreads();
  int p = scratch[lane], q = scratch[32 + lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(kFull, p, off), v = __shfl_up_sync(kFull, q, off);
    if (lane >= off) {
      p += u;
      q += v;
    }
  }
  total = make_int2(__shfl_sync(kFull, p, 31), __shfl_sync(kFull, q, 31));
  const int before = warp > 0 ? warp - 1 : 0;
  const int bx = __shfl_sync(kFull, p, before), by = __shfl_sync(kFull, q, before);
  return make_int2((warp > 0 ? bx : 0) + x - a, (warp > 0 ? by : 0) + y - b);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p, int cluster) {
  extern __shared__ uint32_t keys[];
  __shared__ SelectShared sh;
  const int rank = static_cast<int>(cluster_rank());
  const int g = blockIdx.x / cluster, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  for (int i = tid; i < 2 * kSelBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
  griddep_wait();
  const int L = length_of(p.context_lens, b, p.S, p.err, g == 0 && rank == 0 && tid == 0);
  int32_t* out = p.kept + b * p.k_sb + g * p.k_sh;
  const int first = rank * kSelThreads + tid, step = cluster * kSelThreads;
  if (g == 0 && rank == 0 && tid == 0) p.kept_lens[b] = min(L, p.budget);
  if (L <= p.budget) {
    for (int64_t t = first; t < L; t += step) out[t] = static_cast<int32_t>(t);
    return;
  }
  const float* w = p.weights + b * p.w_sb + g * p.w_sh;
  const int lo = p.sink, hi = L - p.recent;      // the middle
  const int want = p.budget - p.sink - p.recent; // of hi - lo > want
  // this CTA's run of the middle
  const int share = static_cast<int>((static_cast<int64_t>(hi) - lo + cluster - 1) / cluster);
  const int run0 = lo + static_cast<int>(min(static_cast<int64_t>(rank) * share, static_cast<int64_t>(hi) - lo));
  const int run = min(share, hi - run0);
  const bool held = run <= kSelCap;
  auto key = [&](int i) { return held ? keys[i] : weight_key(ld_here(w + run0 + i)); };
  // counts `digit` (negative: none); a warp of equal digits (totals that are
  // all alike) counts once, not 32 times in turn
  auto count_digit = [&](int* hist, int digit) {
    if (__all_sync(kFull, digit == __shfl_sync(kFull, digit, 0))) {
      if (digit >= 0 && lane == 0) atomicAdd(hist + digit, 32);
    } else if (digit >= 0) {
      atomicAdd(hist + digit, 1);
    }
  };
  auto ends = [&] {  // the tokens that always stay
    for (int64_t t = first; t < p.sink; t += step) out[t] = static_cast<int32_t>(t);
    for (int64_t t = first; t < p.recent; t += step) out[p.budget - p.recent + t] = static_cast<int32_t>(hi + t);
  };
  if (want == 0) {
    ends();
    return;
  }
  __syncthreads();  // the cleared counters
  {
    // the keys, and their first digits; a thread's loads are all under way
    // before the first is counted
    for (int i0 = 0; i0 < run; i0 += kSelAhead * kSelThreads) {
      float x[kSelAhead];
#pragma unroll
      for (int e = 0; e < kSelAhead; ++e) {
        const int i = i0 + e * kSelThreads + tid;
        x[e] = i < run ? w[run0 + i] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kSelAhead; ++e) {
        const int i = i0 + e * kSelThreads + tid;
        if (i0 + e * kSelThreads >= run) break;
        const uint32_t k = weight_key(x[e]);
        if (held && i < run) keys[i] = k;
        count_digit(sh.hist[0], i < run ? static_cast<int>(k >> 21) : -1);
      }
    }
  }
  uint32_t prefix = 0, known = 0;
  int need = want;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    int* hist = sh.hist[pass & 1];
    if (pass > 0) {
      for (int i0 = 0; i0 < run; i0 += kSelThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < run ? key(i) : 0u;
        const bool on = i < run && (k & known) == prefix;
        if (__any_sync(kFull, on))  // few keys share the first digits
          count_digit(hist, on ? static_cast<int>((k >> shift) & (pass == 1 ? 2047u : 1023u)) : -1);
      }
    }
    __syncthreads();
    {
      const int s0 = __reduce_add_sync(kFull, hist[64 * warp + lane]);
      const int s1 = __reduce_add_sync(kFull, hist[64 * warp + 32 + lane]);
      if (lane == 0) {
        sh.coarse[pass & 1][2 * warp] = s0;
        sh.coarse[pass & 1][2 * warp + 1] = s1;
      }
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_shared();
    // the cluster's counts of the groups, and once the group is known of its
    // digits: a warp adds them up for all
    const int* coarse = sh.coarse[pass & 1];
    if (cluster > 1) {
      if (warp < 2) sh.sums[tid] = cluster_sum_int(coarse + tid, cluster);
      __syncthreads();
      coarse = sh.sums;
    }
    // from the highest digit: the group that holds the last token kept (a
    // lane has two), then its digit; every warp finds them for itself
    auto scan = [&](int v) {
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(kFull, v, off);
        if (lane >= off) v += u;
      }
      return v;
    };
    const int c0 = coarse[63 - 2 * lane], c1 = coarse[62 - 2 * lane];
    const int groups = scan(c0 + c1);
    const int src = __ffs(__ballot_sync(kFull, groups >= need)) - 1;
    const bool low = groups - c1 < need;  // in the lane's lower group
    const int over = __shfl_sync(kFull, groups - c1 - (low ? 0 : c0), src);
    const int group = 63 - 2 * src - __shfl_sync(kFull, low ? 1 : 0, src);
    const int* fine = hist + 32 * group;
    if (cluster > 1) {
      if (warp == 0) sh.digits[lane] = cluster_sum_int(fine + lane, cluster);
      __syncthreads();
      fine = sh.digits;
    }
    const int c = fine[31 - lane];
    const int digits = over + scan(c);
    const int at = __ffs(__ballot_sync(kFull, digits >= need)) - 1;
    prefix |= static_cast<uint32_t>(32 * group + 31 - at) << shift;
    known |= (pass == 2 ? 1023u : 2047u) << shift;
    const int there = __shfl_sync(kFull, c, at);
    need -= __shfl_sync(kFull, digits, at) - there;
    if (need == there) break;  // all keys of the digit stay
    if (pass == 1) {
      // pass 2 counts in pass 0's counters, which no CTA reads after the
      // cluster's barrier of pass 1
      for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[0][i] = 0;
      __syncthreads();
    }
  }
  // keys above the threshold, and the first `need` of those that match it; a
  // thread's run has an odd length, so that lanes read different banks
  const int each = ((run + kSelThreads - 1) / kSelThreads) | 1;
  const int i0 = static_cast<int>(min(static_cast<int64_t>(tid) * each, static_cast<int64_t>(run)));
  const int i1 = min(run - i0, each) + i0;
  int above = 0, equal = 0;
  uint32_t above_bits = 0, equal_bits = 0;  // of the run's first 32 keys
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i) & known;
    above += k > prefix;
    equal += k == prefix;
    if (i - i0 < 32) {
      above_bits |= static_cast<uint32_t>(k > prefix) << (i - i0);
      equal_bits |= static_cast<uint32_t>(k == prefix) << (i - i0);
    }
  }
  int2 total;
  int2 before = block_scan2(above, equal, sh.tail, lane, warp, total);
  if (cluster > 1) {
    if (tid == 0) {
      sh.counts[0] = total.x;
      sh.counts[1] = total.y;
    }
    __syncthreads();
    cluster_sync_shared();
    for (int r = 0; r < rank; ++r) {
      before.x += cluster_read_int(&sh.counts[0], r);
      before.y += cluster_read_int(&sh.counts[1], r);
    }
    cluster_arrive();  // this thread's reads of the others' shared memory are done
  }
  auto keep = [&](int i, bool is_above) {
    if (is_above) {
      out[p.sink + before.x + min(before.y, need)] = run0 + i;
      ++before.x;
    } else {
      if (before.y < need) out[p.sink + before.x + before.y] = run0 + i;
      ++before.y;
    }
  };
  for (uint32_t bits = above_bits | equal_bits; bits; bits &= bits - 1) {
    const int e = __ffs(bits) - 1;
    keep(i0 + e, (above_bits >> e) & 1u);
  }
  for (int i = i0 + 32; i < i1; ++i) {  // (only runs that are read from L2 are this long)
    const uint32_t k = key(i) & known;
    if (k >= prefix) keep(i, k > prefix);
  }
  ends();
  if (cluster > 1) {  // no CTA leaves while another reads its shared memory
    __syncwarp();
    cluster_wait();
  }
}

// -------------------------------------------------------------- compaction
// One cluster per (sequence, KV head, plane): K rows, V rows, or the totals.
// A list is ascending with kept[i] >= d + i, so position x is only ever the
// source of an entry at or before the one that writes x.  The entries are
// moved in rounds over the cluster; a round's writes wait (cluster barrier)
// until all of its reads are done, and can then overwrite no row that is
// still to be read.  Reads of a later round never meet writes of an earlier
// one, so the next rounds' rows are on their way while one is written.
//
// What bounds it: HBM, one read and one write of each kept row (256 bytes at
// D = 128, scattered by the list).  A row's address takes two dependent loads
// (list, table) before its own: addresses are translated kMoveBlock rows at a
// time into shared memory, and rows go through a ring of kMoveStages rounds
// with asynchronous 16-byte copies, which hold no registers.  (With rows and
// addresses in registers, 170 a thread let one CTA onto an SM: 248 us on 32
// sequences of 512-8192 tokens cut to 1024, 114 us with one round at a time;
// now 44.4 us, 6.0 TB/s.)  The barrier's arrival is relaxed: the asynchronous
// copies of the round are complete, their values lie in shared memory, and no
// write can change what they read; an arrival that releases would also wait
// for the last round's own writes to reach L2.  That batch / one list of 16383
// among short ones: 44.4 / 28.9 us; released 48.0 / 37.3; released a round
// ahead, with a fourth stage, 53.7 / 37.0.  The ring's sizes: 512 threads, 3
// rounds of 1024 chunks 44.2 / 28.5 us; 2048 chunks, 2 or 3 rounds 45.9 / 28.8
// and 46.6 / 32.9; 256 threads 45.8 / 28.7.
constexpr int kMoveThreads = 512;
constexpr int kMoveStages = 3;
constexpr int kMoveChunks = 1024;   // 16-byte chunks of a round and CTA, at most
constexpr int kMoveRows = 128;      // rows of a round and CTA, at most
constexpr int kMoveBlock = 512;     // rows translated at a time
constexpr int kMoveRing = 1024;     // translated rows held
constexpr int kMoveTotals = 4;      // totals a thread moves per round
constexpr uint32_t kNoMove = 0xffffffffu;
// A fast thread translates for round r + kMoveStages while a slow one still
// writes the rows of round r: kMoveStages + 1 rounds, and what a block adds.
static_assert(kMoveRing >= kMoveBlock - 1 + (kMoveStages + 1) * kMoveRows, "rows in flight keep their addresses");

template <int CHUNKS>               // 16-byte chunks of a row; 0: p.D / 8
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const CompactParams p, int cluster) {
  extern __shared__ uint4 rows[];   // [kMoveStages][kMoveChunks]
  __shared__ uint32_t ring_src[kMoveRing], ring_dst[kMoveRing];  // block * 16 + slot
  griddep_launch_dependents();
  griddep_wait();
  const int rank = static_cast<int>(cluster_rank()), tid = threadIdx.x;
  const int g = blockIdx.x / cluster, b = blockIdx.y, plane = blockIdx.z;
  const bool first = g == 0 && plane == 0 && rank == 0 && tid == 0;
  const int L = p.context_lens[b];
  const int n = p.kept_lens[b];
  const int d = p.dst_start ? p.dst_start[b] : 0;
  if (L < 0 || L > p.MB * kBlockSize) {
    if (first) record_error(p.err, kDevErrLength);
    return;
  }
  if (n < 0 || n > p.K || d < 0 || d > L - n) {
    if (first) record_error(p.err, kDevErrKept);
    return;
  }
  const int32_t* list = p.kept + b * p.k_sb + g * p.k_sh;
  auto wait = [&] {
    if (cluster > 1)
      cluster_wait();
    else
      __syncthreads();
  };
  // source of entry i, -1 when it breaks the rules
  auto entry = [&](int i) -> int {
    const int s = list[i];
    const int before = i > 0 ? list[i - 1] : -1;
    if (s >= d + i && s < L && s > before) return s;
    record_error(p.err, kDevErrKept);
    return -1;
  };

  if (plane == 2) {  // the running totals, and zeros behind the new end
    float* w = p.weights + b * p.w_sb + g * p.w_sh;
    if (L > p.S && g == 0 && rank == 0 && tid == 0) record_error(p.err, kDevErrLength);
    const int round = cluster * kMoveThreads * kMoveTotals;
    for (int64_t i0 = 0; i0 < n; i0 += round) {
      float x[kMoveTotals];
      unsigned ok = 0;
#pragma unroll
      for (int u = 0; u < kMoveTotals; ++u) {
        const int64_t i = i0 + (u * cluster + rank) * kMoveThreads + tid;
        const int s = i < n ? entry(static_cast<int>(i)) : -1;
        if (s >= 0 && s < p.S && s != d + i) {
          x[u] = w[s];
          ok |= 1u << u;
        }
      }
      if (cluster > 1) cluster_arrive();
      wait();
#pragma unroll
      for (int u = 0; u < kMoveTotals; ++u)
        if ((ok >> u) & 1u) w[d + i0 + (u * cluster + rank) * kMoveThreads + tid] = x[u];
    }
    // every read of the cluster is done
    for (int64_t t = static_cast<int64_t>(d) + n + rank * kMoveThreads + tid; t < min(L, p.S); t += cluster * kMoveThreads)
      w[t] = 0.f;
    return;
  }

  const int32_t* table = p.block_tables + b * p.bt_sb;
  __nv_bfloat16* cache = (plane ? p.v_cache : p.k_cache) + g * (plane ? p.vc_sh : p.kc_sh);
  const int64_t sblk = plane ? p.vc_sblk : p.kc_sblk;
  const int chunks = CHUNKS ? CHUNKS : p.D / 8;
  const int per = min(kMoveRows, kMoveChunks / chunks);  // rows of a round and CTA
  const int rounds = (n + cluster * per - 1) / (cluster * per);
  auto slot_of = [&](int t) -> uint32_t {
    const int blk = table[t / kBlockSize];
    if (static_cast<unsigned>(blk) < static_cast<unsigned>(p.NB))
      return static_cast<uint32_t>(blk) * kBlockSize + t % kBlockSize;
    record_error(p.err, kDevErrBlockId);
    return kNoMove;
  };
  // this CTA's rows in order: row q is row q % per of round q / per
  int translated = 0;
  auto translate = [&] {
#pragma unroll
    for (int u = 0; u < kMoveBlock / kMoveThreads; ++u) {
      const int q = translated + u * kMoveThreads + tid;
      const int64_t i = (static_cast<int64_t>(q / per) * cluster + rank) * per + q % per;
      uint32_t from = kNoMove, to = kNoMove;
      if (i < n) {
        const int s = entry(static_cast<int>(i));
        if (s >= 0 && s != d + i) {
          from = slot_of(s);
          to = slot_of(static_cast<int>(d + i));
          if (to == kNoMove) from = kNoMove;
        }
      }
      ring_src[q % kMoveRing] = from;
      ring_dst[q % kMoveRing] = to;
    }
    translated += kMoveBlock;
    __syncthreads();
  };
  auto at = [&](uint32_t slot, int c) -> uint4* {
    return reinterpret_cast<uint4*>(cache + (slot / kBlockSize) * sblk + (slot % kBlockSize) * (chunks * 8) + c * 8);
  };
  // A thread reads and writes the same chunks of a round, so the copies need
  // be complete for itself alone.
  auto read = [&](int r) {
    if (r < rounds) {
      while (translated < (r + 1) * per) translate();
      uint4* stage = rows + (r % kMoveStages) * kMoveChunks;
#pragma unroll
      for (int u = 0; u < kMoveChunks / kMoveThreads; ++u) {
        const int idx = u * kMoveThreads + tid, w = idx / chunks, c = idx % chunks;
        if (w < per) {
          const uint32_t from = ring_src[(r * per + w) % kMoveRing];
          if (from != kNoMove) cp_async16(stage + idx, at(from, c));
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int r = 0; r < kMoveStages - 1; ++r) read(r);
  for (int r = 0; r < rounds; ++r) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kMoveStages - 2) : "memory");
    if (cluster > 1) cluster_arrive_relaxed();  // this CTA's reads of round r are done: their rows have landed
    read(r + kMoveStages - 1);
    wait();
    const uint4* stage = rows + (r % kMoveStages) * kMoveChunks;
#pragma unroll
    for (int u = 0; u < kMoveChunks / kMoveThreads; ++u) {
      const int idx = u * kMoveThreads + tid, w = idx / chunks, c = idx % chunks;
      if (w < per && ring_src[(r * per + w) % kMoveRing] != kNoMove)
        *at(ring_dst[(r * per + w) % kMoveRing], c) = stage[idx];
    }
  }
}

template <int G>
cudaError_t launch_acc(const WeightsParams& p, cudaStream_t stream) {
  const int64_t span = std::min<int64_t>(p.S, static_cast<int64_t>(p.MB) * kBlockSize);
  // (one block where the totals have no columns: it records longer sequences)
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (span + kAccTokens - 1) / kAccTokens)),
                  static_cast<unsigned>(p.Hkv), static_cast<unsigned>(p.B));
  return launch_pdl(accumulate_weights_kernel<G>, grid, dim3(kAccThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_accumulate_weights(const WeightsParams& p, int G, cudaStream_t stream) {
  if (p.B == 0 || p.MB == 0) return cudaSuccess;
  switch (G) {
    case 1: return launch_acc<1>(p, stream);
    case 2: return launch_acc<2>(p, stream);
    case 4: return launch_acc<4>(p, stream);
    case 8: return launch_acc<8>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

// Allows a kernel clusters of up to 16 CTAs (above 8 it has to be asked for)
// and `smem` bytes of dynamic shared memory, set once per device.
static cudaError_t prepare_kernel(const void* kernel, int smem, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) dev = 63;
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done[dev].store(1);
  return e;
}

// CTAs per list: until each can hold its keys, and down to 2048 keys each
// while all lists' CTAs fit onto the SMs at once (two each).
cudaError_t launch_evict_select(const SelectParams& p, int num_sms, cudaStream_t stream) {
  int cluster = 1;
  while (cluster < 16 && (p.S > cluster * kSelCap || (p.S > cluster * 2048 && 2ll * p.B * p.Hkv * cluster <= 2ll * num_sms)))
    cluster *= 2;
  static std::atomic<int> done[64];
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(evict_select_kernel), kSelCap * 4, done);
  if (e != cudaSuccess) return e;
  const int held = std::min(kSelCap, (p.S + cluster - 1) / cluster);
  return launch_pdl_cluster(evict_select_kernel,
                            dim3(static_cast<unsigned>(p.Hkv) * cluster, static_cast<unsigned>(p.B)), cluster,
                            dim3(kSelThreads), static_cast<size_t>(held) * 4, stream, p, cluster);
}

template <int CHUNKS>
static cudaError_t launch_move(const CompactParams& p, int cluster, cudaStream_t stream) {
  constexpr int kSmem = kMoveStages * kMoveChunks * 16;
  auto kernel = kv_compact_kernel<CHUNKS>;
  static std::atomic<int> done[64];
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kernel), kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel,
                            dim3(static_cast<unsigned>(p.Hkv) * cluster, static_cast<unsigned>(p.B), p.totals ? 3u : 2u),
                            cluster, dim3(kMoveThreads), kSmem, stream, p, cluster);
}

// CTAs per list and plane: as many as leave each about eight rounds of the
// longest list; doubled while K's and V's CTAs are fewer than 8 to an SM (which
// holds 4), so up to 16.
// Measured with 1 / 2 / 4 / 8 / 16: 32 sequences cut to 1024 tokens 49.1 /
// 45.7 / 47.0 / 57.4 / 95.6 us, one list of 16383 221 / 113 / 70 / 40 / 28 us.
cudaError_t launch_kv_compact(const CompactParams& p, int num_sms, cudaStream_t stream) {
  int cluster = 1;
  const int64_t chunks = static_cast<int64_t>(p.K) * (p.D / 8);
  while (cluster < 16 && chunks > static_cast<int64_t>(cluster) * kMoveChunks * 8 &&
         static_cast<int64_t>(p.B) * p.Hkv * 2 * cluster < 8ll * num_sms)
    cluster *= 2;
  switch (p.D) {
    case 64: return launch_move<8>(p, cluster, stream);
    case 128: return launch_move<16>(p, cluster, stream);
    default: return launch_move<0>(p, cluster, stream);
  }
}

}  // namespace forge
