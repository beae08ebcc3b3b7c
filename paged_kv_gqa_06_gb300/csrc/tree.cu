// Attention of a tree of drafted tokens per sequence over its paged cache, on
// the 5th-generation tensor cores.
//
// Node i of sequence b (query row r = query_start[b] + i, n_b nodes, at the
// last n_b of its L_b cached positions) sees the positions before
// P = L_b - n_b and the nodes whose bit its mask has set:
//   out[r, h, :] = sum_{t seen} softmax_t(scale * q[r, h, :] . K[t, h/G, :]) V[t, h/G, :]
// A row that sees nothing gives zeros.
//
// What bounds it: a tree has tens of nodes, so a KV head serves n_b G rows,
// 16 to 256, and each K/V byte read from HBM feeds 2 n_b G products: the
// stream of K and V bounds the call up to about 128 rows, the tensor cores
// beyond.  One tile is M = 128 rows (128 / G nodes x the G heads of a KV
// head; rows past the tree are computed and not stored, since an MMA takes
// its time whatever M holds).  Measured on GB300 (152 SMs, copy peak 6766
// GB/s): 32 sequences of 512-8192 tokens, trees of 5-24 nodes, 32 / 8 heads,
// D 128: 113 to 117 us from GPU to GPU, 5.4 TB/s; 8 sequences of 512-4096, 64
// nodes: 38 us, 508 TFLOP/s of Q K^T and P V (the MMAs issued are half as many again); one of
// 32768 among three short ones, 13 nodes, fp32 out: 42 us, 3.4 TB/s.
//
// Work split.  An item is (sequence, KV head, group of rows); its length is
// its sequence's stages of 64 tokens.  All items laid end to end, the grid's
// CTAs take equal shares of the line, cut at any stage: every CTA streams the
// same number of bytes whatever the lengths, and an item is cut into few
// pieces.  A share is a run of segments (item, first stage, end stage).  A
// segment that is its whole item writes `out`; the pieces of a cut item leave
// unnormalised (O, max, sum) rows in the workspace, at most two per CTA, and a
// second, short kernel merges them, over all SMs (the last CTA of an item to
// finish would have to read all its pieces alone).  The CTAs derive the line
// from the lengths, so the host knows only the sizes.  (Counting an item's
// stages alone, the CTA with 13 one-stage items took twice as long as the
// others: an item costs item_cost stages more.)
//
// In a CTA: softmax warps (a row per thread), a producer warp and two MMA
// warps, on rings of K and V stages:
//   * S = Q K^T (M 128, N 64, K = D) alternates between two TMEM buffers, so
//     the next stage's S is ready when a stage's weights are done;
//   * the weights go over the S they came from as bf16 parts, and O += P V
//     (M 128, N = D, K 64) reads them from TMEM.  bf16 out takes two parts
//     (about 16 bits: a weight rounded to bf16 once could move the result by
//     as much as its own rounding), fp32 out three (24 bits);
//   * the running maximum moves only when it grows by more than 8 in log2
//     units, so O is rescaled rarely.
// MMAs back to back take 49 cycles (Q K^T: M 128, N 64, K 16; its operands
// are 6 KB, which shared memory gives at 128 B a cycle) and 65 cycles (P V: N
// 128, A in TMEM), whatever M holds.  Two tiles at two parts are 1824 cycles a
// stage, and the kernel takes 2500 for it; one tile is 912, where HBM takes
// 1400.  So MMAs are saved where rows are few: see Mode.
// Two CTAs share an SM in the one-tile modes (256 TMEM columns each), so one
// CTA's softmax overlaps the other's MMAs.
//
// Each addition of an MMA to O drops bits of the sum so far, in one direction,
// so the error of one accumulation grows with its length: less than 2^-23 of a
// sum that grows evenly, 2^-24 of the result for each.  Over a share of 16384
// tokens (weights just above 0.5, V of one sign) it was 7.6e-4 on results near
// 7.5, and bf16 out was off by 0.0164.  So a segment's O starts anew after
// sum_stages() stages; what it held goes to a side sum in the scratch (the slot
// that the segment's piece takes when it is cut), added in fp32 with the
// maxima's factors.  The bound is 3.1e-4 of |out| < 8 for bf16 out, whose own
// rounding is 1.56e-2, and 1.8e-4 for fp32 out; measured 0.0159 and 1.5e-4, at any
// length.  Segments that long are those of large batches; 32 sequences of 16384
// tokens, 12 / 24 nodes, 8 KV heads of 4: 336 / 349 us with bf16 out (334 / 347 in
// one sum), 381 / 531 us with fp32 out (376 / 530).
//
// Masked positions: only the stages that reach past P take the masked path.
// There the V rows of nodes may hold infinities or NaN that some rows do not
// see, and 0 * inf is NaN: such elements are set to zero in shared memory and
// added, for the rows that see them, to O at the end.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace forge {
namespace {

constexpr unsigned kFullMask = 0xffffffffu;
constexpr int kRows = 128;             // rows of a tile (MMA M)
constexpr int kTok = 64;               // tokens of a stage
constexpr int kStageBlks = kTok / kBlockSize;
constexpr float kRescaleSlack = 8.0f;  // log2 units: weights stay <= 2^8
constexpr int kAddRow = 36;            // floats of a row of 32 dims in shared memory
constexpr int kMergeThreads = 256;
constexpr int kMaxShares = 640;        // CTAs of a launch, at most (their tasks fit the merge kernel's shared memory)

// ------------------------------------------------------------ configuration
// How a launch lays out an item's rows:
//   kOneTile   bf16 out, one tile; an item of at most 64 rows puts the weights'
//              high parts into rows 0-63 and the low parts into rows 64-127
//              (Q twice in the tile, so both halves compute the same scores),
//              and one MMA does what two do otherwise; the halves of O are
//              added at the end;
//   kTwoTiles  bf16 out, two tiles that share a stream of K and V;
//   kFull32    fp32 out, one tile, three parts of each weight (24 bits);
//   kHalf32    fp32 out, 64 rows, high and low parts in the tile's halves and
//              the third part in a second MMA.
enum Mode { kOneTile, kTwoTiles, kFull32, kHalf32 };

template <int D, int MODE>
struct Cfg {
  static constexpr int TILES = MODE == kTwoTiles ? 2 : 1;
  static constexpr int kItemRows = MODE == kHalf32 ? 64 : TILES * kRows;
  static constexpr bool kPair = MODE == kOneTile || MODE == kHalf32;  // two CTAs share an SM
  using Out = std::conditional_t<(MODE >= kFull32), float, __nv_bfloat16>;
  static constexpr int kSoftmaxWarps = 4 * TILES;
  static constexpr int kProducer = kSoftmaxWarps, kQk = kSoftmaxWarps + 1, kPv = kSoftmaxWarps + 2;
  static constexpr int kThreads = (kSoftmaxWarps + 3) * 32;
  static constexpr int kBoxes = D / 64;
  static constexpr int kQTile = kBoxes * kRows * 128;
  static constexpr int kStage = kBoxes * kTok * 128;       // K or V of a stage
  static constexpr int kRing = kPair && D == 128 ? 2 : 4;  // stages of the K ring, and of the V ring
  // Stages of one accumulation of O, at most: 640 products of 16 tokens for
  // bf16 out, 384 for fp32 out, of a weight's parts 2 and 3 (in the halves of a
  // tile 1 and 2).
  __host__ __device__ static constexpr int sum_stages(bool half) {
    return MODE >= kFull32 ? (half ? 48 : 32) : (half ? 160 : 80);
  }
  static constexpr int kSWidth = MODE == kFull32 ? 96 : 64;  // TMEM columns of an S buffer
  static constexpr int kTmem = kPair ? 256 : 512;
  __host__ __device__ static constexpr int o_col(int t) { return 128 * t; }
  __host__ __device__ static constexpr int s_col(int t, int buf) { return 128 * TILES + (2 * t + buf) * kSWidth; }
  static_assert(128 * TILES + 2 * TILES * kSWidth <= kTmem, "TMEM columns");
  // shared memory, from a 1024-byte boundary: Q | K ring | V ring | halves of
  // O on their way to be added | barriers
  static constexpr int kQ = 0;
  static constexpr int kK = TILES * kQTile;
  static constexpr int kV = kK + kRing * kStage;
  static constexpr int kAdd = kV + kRing * kStage;
  static constexpr int kBars = kAdd + (kPair ? 64 * kAddRow * 4 : 0);
  // barrier slots
  static constexpr int kQFull = 0, kQEmpty = 1;
  static constexpr int kKFull = 2, kKEmpty = kKFull + kRing, kVFull = kKEmpty + kRing, kVEmpty = kVFull + kRing;
  static constexpr int kSFull = kVEmpty + kRing;         // [tile][buffer]
  static constexpr int kPFull = kSFull + 2 * TILES;      // [tile][buffer], one arrival per softmax warp
  static constexpr int kPvDone = kPFull + 2 * TILES;     // [tile][buffer]
  static constexpr int kDrain = kPvDone + 2 * TILES;     // [QK, PV]
  static constexpr int kWords = kDrain + 2;              // 32-bit words behind the barriers
  static constexpr int kSmem = kBars + kWords * 8 + 64 + 1024;
};

// ------------------------------------------------------------ the work line
// An item costs its stages and item_cost more (its Q, its first scores, its
// rows' stores); a stage of two tiles takes twice as long as one of one.
// Measured at 2 / 4 / 6 / 8: one-tile modes, 32 sequences 116.3 / 114 / 116.6
// / 118.3 us, one long sequence 46.2 / 41.8 / 41.7 / 41.5 us; two tiles 37.6 /
// 38.8 / 40.0 / 40.3 us.
__host__ __device__ constexpr int item_cost(int item_rows) { return item_rows > kRows ? 2 : 4; }

// A sequence's part of the line.
struct Seq {
  int q0, n, L;   // first query row, nodes, cached tokens
  int stages;     // stages of each of its items
  int groups;     // row-tile groups (items per KV head); 0: nothing to do
  int item;       // line length of each of its items
  __device__ __forceinline__ int64_t cost(int Hkv) const { return static_cast<int64_t>(item) * groups * Hkv; }
};

template <int G, int IR>  // IR: rows of an item
__device__ __forceinline__ Seq seq_of(const TreeParams& p, int b) {
  Seq s;
  s.q0 = p.query_start[b];
  const int64_t n = static_cast<int64_t>(p.query_start[b + 1]) - s.q0;
  s.L = p.context_lens[b];
  const bool ok = n > 0 && s.q0 >= 0 && s.q0 + n <= p.T && s.L <= p.MB * kBlockSize && n <= s.L && n <= 64ll * p.W;
  s.n = ok ? static_cast<int>(n) : 0;
  s.stages = ok ? (s.L + kTok - 1) / kTok : 0;
  constexpr int kNodes = IR / G;
  s.groups = ok ? (s.n + kNodes - 1) / kNodes : 0;
  s.item = s.stages + item_cost(IR);
  return s;
}

// A share of the line: where it starts (item (b, group, g), whose own start is
// line position item0; order: sequence, group, KV head), positions [w0, w1),
// and the line's length and number of shares.
struct Share {
  int b, group, g, count;
  int64_t item0, w0, w1, len;
};

// A quotient of non-negative numbers; 32 bits where they do (a 64-bit division
// takes some hundred cycles).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Shares of a line of `len`, and the line position where share c starts.
__device__ __forceinline__ int sharers(int64_t len, int most, int least) {
  const int64_t c = quotient(len, least);
  return c < 1 ? 1 : c > most ? most : static_cast<int>(c);
}
__device__ __forceinline__ int64_t share_start(int64_t len, int count, int c) { return quotient(len * c, count); }

// Share c of `most` or fewer (all lanes of a warp).
template <int G, int IR>
__device__ __forceinline__ Share share_of(const TreeParams& p, int c, int most, int lane) {
  Share r{0, 0, 0, 0, 0, 0, 0, 0};
  // the line's length; the first 32 sequences and their scan stay in registers
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t u = __shfl_up_sync(kFullMask, v, off);
      if (lane >= off) v += u;
    }
    return v;
  };
  Seq mine{0, 0, 0, 0, 0, 1};
  if (lane < p.B) mine = seq_of<G, IR>(p, lane);
  int64_t cost = mine.cost(p.Hkv), incl = scan(cost);
  int64_t sum = __shfl_sync(kFullMask, incl, 31);
  if (p.B > 32) {
    int64_t rest = 0;
    for (int b = lane + 32; b < p.B; b += 32) rest += seq_of<G, IR>(p, b).cost(p.Hkv);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(kFullMask, rest, off);
    sum += rest;
  }
  r.len = sum;
  r.count = sharers(sum, most, p.min_share);
  if (c >= r.count || sum == 0) return r;
  r.w0 = share_start(sum, r.count, c);
  r.w1 = share_start(sum, r.count, c + 1);
  int64_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (b0 > 0) {
      mine = Seq{0, 0, 0, 0, 0, 1};
      if (b0 + lane < p.B) mine = seq_of<G, IR>(p, b0 + lane);
      cost = mine.cost(p.Hkv);
      incl = scan(cost);
    }
    const unsigned who = __ballot_sync(kFullMask, r.w0 < base + incl);
    if (who) {
      const int src = __ffs(who) - 1;
      const int64_t first = base + __shfl_sync(kFullMask, incl - cost, src);
      const int64_t one = __shfl_sync(kFullMask, mine.item, src);
      const int64_t item = quotient(r.w0 - first, one);
      r.b = b0 + src;
      r.group = static_cast<int>(quotient(item, p.Hkv));
      r.g = static_cast<int>(item - static_cast<int64_t>(r.group) * p.Hkv);
      r.item0 = first + item * one;
      break;
    }
    base += __shfl_sync(kFullMask, incl, 31);
  }
  return r;
}

// A share's segments, one after the other; every warp walks the same list.
// With p.split a segment is the part of its item inside the share, without it
// the whole item, for the items that start in the share.
template <int G, int IR>
struct Walk {
  int b, group, g;
  int st0, st1;        // this segment's stages of the item
  int64_t item0, w0, w1;
  Seq s;
  // to the first segment; false if the share has none
  __device__ __forceinline__ bool start(const TreeParams& p, const Share& sh) {
    b = sh.b;
    group = sh.group;
    g = sh.g;
    w0 = sh.w0;
    w1 = sh.w1;
    item0 = sh.item0;
    if (w1 <= w0) return false;
    s = seq_of<G, IR>(p, b);
    if (!p.split && item0 < w0) return next(p);
    span(p);
    return st1 > st0 || next(p);
  }
  // stages before line position w
  __device__ __forceinline__ int stages_to(int64_t w) const {
    const int64_t x = w - item0 - item_cost(IR);
    return x <= 0 ? 0 : x < s.stages ? static_cast<int>(x) : s.stages;
  }
  __device__ __forceinline__ void span(const TreeParams& p) {
    st0 = p.split ? stages_to(w0) : 0;
    st1 = p.split ? stages_to(w1) : s.stages;
  }
  __device__ __forceinline__ bool whole() const { return st0 == 0 && st1 == s.stages; }
  __device__ __forceinline__ int rows() const { return s.n * G - group * IR; }  // of this item (IR at most)
  __device__ __forceinline__ int tiles() const { return IR <= kRows || rows() <= kRows ? 1 : 2; }
  // on to the next segment; false at the end of the share
  __device__ __forceinline__ bool next(const TreeParams& p) {
    do {
      item0 += s.item;
      if (item0 >= w1) return false;
      if (++g == p.Hkv) {
        g = 0;
        if (++group == s.groups) {
          group = 0;
          do {
            if (++b >= p.B) return false;  // not reached: the share ends inside the line
            s = seq_of<G, IR>(p, b);
          } while (s.groups == 0);
        }
      }
      span(p);
    } while (st1 == st0);  // the share ends before the item's first stage
    return true;
  }
};

// What the merge kernel has to do after share c: the item that starts in the
// share and ends in a later one (pieces = 0: there is none).
struct MergeTask {
  int pieces, slot0;   // pieces: of this share in slot0, of the next ones in slots 2 (c + k)
  int q0, n, group, g;
  int pad[2];
};

__device__ __forceinline__ void store_row32(float* dst, const uint32_t (&v)[32], float inv) {
#pragma unroll
  for (int c = 0; c < 32; c += 4)
    *reinterpret_cast<float4*>(dst + c) = make_float4(__uint_as_float(v[c]) * inv, __uint_as_float(v[c + 1]) * inv,
                                                      __uint_as_float(v[c + 2]) * inv, __uint_as_float(v[c + 3]) * inv);
}
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&v)[32], float inv) {
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__uint_as_float(v[c + 2 * e]) * inv, __uint_as_float(v[c + 2 * e + 1]) * inv);
    *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 32 mask bits of a row for positions t .. t + 31 of its sequence: ones below
// P, the node's bits from P, zeros from L.
// `first` is the row's first mask word, read ahead.
__device__ __forceinline__ uint32_t seen_bits(uint64_t first, const int64_t* mask, int words, int t, int P, int L) {
  auto word = [&](int w) { return w == 0 ? first : static_cast<uint64_t>(mask[w]); };
  const int j = t - P;  // node index of position t
  uint32_t bits;
  if (j <= -32) {
    bits = 0xffffffffu;
  } else if (j < 0) {
    bits = ((1u << -j) - 1u) | (static_cast<uint32_t>(first) << -j);
  } else {
    const int w = j >> 6, sh = j & 63;
    uint64_t x = w < words ? word(w) >> sh : 0ull;
    if (sh > 32 && w + 1 < words) x |= word(w + 1) << (64 - sh);
    bits = static_cast<uint32_t>(x);
  }
  const int left = L - t;
  if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
  return bits;
}

// bf16 pairs: all-ones mask in each half whose exponent is all ones.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); }

// 32 columns of a row's O.  Where the weights' parts lie in the tile's halves
// (`half`, all of the tile's threads call this), the low parts' O is added in
// the thread with the high parts', over `add` in shared memory.
template <bool PAIR>
__device__ __forceinline__ void read_o(uint32_t taddr, bool half, bool upper, float4* add, uint32_t (&v)[32]) {
  tc::ld_32x32b_x32(taddr, v);
  tc::wait_ld();
  if constexpr (PAIR) {
    if (half) {
      if (upper) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          add[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                               __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
      }
      named_barrier(1, kRows);
      if (!upper) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 x = add[e];
          v[4 * e] = __float_as_uint(__uint_as_float(v[4 * e]) + x.x);
          v[4 * e + 1] = __float_as_uint(__uint_as_float(v[4 * e + 1]) + x.y);
          v[4 * e + 2] = __float_as_uint(__uint_as_float(v[4 * e + 2]) + x.z);
          v[4 * e + 3] = __float_as_uint(__uint_as_float(v[4 * e + 3]) + x.w);
        }
      }
      named_barrier(1, kRows);
    }
  }
}
// A row of a piece or of a side sum lies as [4-dim group][row], so that a
// warp's 32 rows store together.
template <int ITEM_ROWS>
__device__ __forceinline__ void store_piece(float4* po, int c4, const uint32_t (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    po[(8 * c4 + e) * ITEM_ROWS] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                               __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
}
template <int ITEM_ROWS>
__device__ __forceinline__ void add_piece(const float4* po, int c4, float f, uint32_t (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 x = po[(8 * c4 + e) * ITEM_ROWS];
    v[4 * e] = __float_as_uint(fmaf(x.x, f, __uint_as_float(v[4 * e])));
    v[4 * e + 1] = __float_as_uint(fmaf(x.y, f, __uint_as_float(v[4 * e + 1])));
    v[4 * e + 2] = __float_as_uint(fmaf(x.z, f, __uint_as_float(v[4 * e + 2])));
    v[4 * e + 3] = __float_as_uint(fmaf(x.w, f, __uint_as_float(v[4 * e + 3])));
  }
}
// What a side sum against `from` is worth against `to` (-inf: nothing seen).
__device__ __forceinline__ float side_factor(float from, float to) {
  return fast_exp2(from - (to == -INFINITY ? 0.f : to));
}
// O into the side sum at `po` (whose maximum is kept in `ml`), before the next
// products start it anew.  `mine`: this thread keeps the row.  (Not inlined:
// rarely called, its registers would be spilled in the loop over the stages.)
template <int D, int ITEM_ROWS, bool PAIR>
__device__ __noinline__ void sum_aside(uint32_t tcol, bool half, bool upper, bool mine, bool first, float m,
                                       float4* add, float4* po, float2* ml) {
  tc::fence_after_sync();
  const float f = mine && !first ? side_factor(ml->x, m) : 0.f;
#pragma unroll 1
  for (int c4 = 0; c4 < D / 32; ++c4) {
    uint32_t v[32];
    read_o<PAIR>(tcol + 32 * c4, half, upper, add, v);
    if (mine) {
      if (!first) add_piece<ITEM_ROWS>(po, c4, f, v);
      store_piece<ITEM_ROWS>(po, c4, v);
    }
    __syncwarp();
  }
  if (mine) ml->x = m;
}

// ------------------------------------------------------------ main kernel
template <int D, int G, int MODE>
__global__ void __launch_bounds__(Cfg<D, MODE>::kThreads, Cfg<D, MODE>::kPair ? 2 : 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv, const TreeParams p) {
  using C = Cfg<D, MODE>;
  using OutT = typename C::Out;
  constexpr int TILES = C::TILES;
  constexpr int QT = kRows / G;           // nodes of a tile
  constexpr int kNodes = C::kItemRows / G;  // nodes of an item
  constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(kRows, kTok, false);
  constexpr uint32_t IDESC_O = tc::idesc_bf16_f32(kRows, D, true);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
  const uint32_t sm_s = smem_addr(sm);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kWords);
  volatile int* bad_v = reinterpret_cast<volatile int*>(tmem_slot + 1);  // a node's V holds infinities or NaN
  Share* share = reinterpret_cast<Share*>(tmem_slot + 4);
  static_assert(sizeof(Share) <= 48, "words behind the barriers");

  if (threadIdx.x == 0) {
    mbar_init(bars + C::kQFull, 1);
    mbar_init(bars + C::kQEmpty, 1);
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(bars + C::kKFull + i, 1);
      mbar_init(bars + C::kKEmpty + i, 1);
      mbar_init(bars + C::kVFull + i, 1);
      mbar_init(bars + C::kVEmpty + i, 1);
    }
    for (int i = 0; i < 2 * TILES; ++i) {
      mbar_init(bars + C::kSFull + i, 1);
      mbar_init(bars + C::kPFull + i, 4);
      mbar_init(bars + C::kPvDone + i, 1);
    }
    mbar_init(bars + C::kDrain, 1);
    mbar_init(bars + C::kDrain + 1, 1);
    fence_barrier_init();
    *bad_v = 0;
  }
  if (warp == C::kPv) {
    tc::tmem_alloc(smem_addr(tmem_slot), C::kTmem);
    tc::tmem_relinquish();
    // The merge kernel's CTAs may take their places as this grid's leave.  Not
    // before this CTA has its TMEM: one of a following grid that took it first
    // would hold it until this grid is complete.
    griddep_launch_dependents();
  }
  // The lengths, tables, masks, q and cache below are the previous grid's
  // results: read after the wait, with ordinary loads (that grid may have run
  // beside this one, and a non-coherent load wants unchanging data).
  griddep_wait();
  if (warp == 0) {
    const Share sh = share_of<G, C::kItemRows>(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), lane);
    if (lane == 0) *share = sh;
  } else if (warp == 1 && blockIdx.x == 0) {  // the rules for every sequence, checked once
    int code = 0;
    for (int b = lane; b < p.B; b += 32) {
      const int s0 = p.query_start[b], s1 = p.query_start[b + 1], L = p.context_lens[b];
      const int64_t n = static_cast<int64_t>(s1) - s0;
      if (n < 0 || s1 > p.T || (b == 0 && s0 != 0)) code = kDevErrQuery;
      if (n > 0 && (L < 0 || L > p.MB * kBlockSize))
        code = kDevErrLength;
      else if (n > L || n > 64ll * p.W)
        code = n > 0 ? kDevErrQuery : code;
    }
    if (code) record_error(p.err, code);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walk<G, C::kItemRows> k;
  const bool any = k.start(p, *share);

  if (!any) {
    // an empty share
  } else if (warp == C::kProducer) {
    // ------------------------------------------------------------ producer
    int ring = 0, seg = 0;  // stages and segments so far
    const uint64_t once = l2_read_once();
    auto load_q = [&] {
      if (lane == 0) {
        const int nt = k.tiles();
        const bool half = MODE == kHalf32 || (MODE == kOneTile && k.rows() <= 64);
        mbar_arrive_expect_tx(bars + C::kQFull, nt * C::kQTile);
        for (int t = 0; t < nt; ++t)
#pragma unroll
          for (int x = 0; x < 2 * C::kBoxes; ++x) {  // 64 rows of 64 dims
            const int upper = x & 1, c64 = x >> 1;
            tma_load_3d(sm + C::kQ + t * C::kQTile + (2 * c64 + upper) * 64 * 128, &tmq, c64 * 64, k.g * G,
                        k.s.q0 + k.group * kNodes + t * QT + (upper && !half ? QT / 2 : 0), bars + C::kQFull);
          }
      }
      __syncwarp();
    };
    do {
      const int32_t* row = p.block_tables + static_cast<int64_t>(k.b) * p.bt_sb;
      // block ids of 8 stages: lane l holds block l % 4 of stage l / 4
      auto table_group = [&](int st) -> int {
        const int jb = kStageBlks * st + lane;
        return jb * kBlockSize < k.s.L ? row[jb] : -1;
      };
      int ids = table_group(k.st0), ahead = k.st1 - k.st0 > 8 ? table_group(k.st0 + 8) : -1;
      if (seg == 0) load_q();  // while the block ids are on their way
      for (int st = k.st0; st < k.st1; ++st, ++ring) {
        const int in = st - k.st0;
        if (in > 0 && in % 8 == 0) {
          ids = ahead;
          if (st + 8 < k.st1) ahead = table_group(st + 8);
        }
        // lane u + 4 c copies box c of block u
        const int u = lane & 3, c = lane >> 2;
        int e = __shfl_sync(kFullMask, ids, (in % 8) * 4 + u);
        const bool used = (kStageBlks * st + u) * kBlockSize < k.s.L;
        const bool bad = used && static_cast<unsigned>(e) >= static_cast<unsigned>(p.NB);
        if (bad && c == 0) record_error(p.err, kDevErrBlockId);
        const bool mine = c < C::kBoxes && used && !bad;
        const uint32_t bytes = __popc(__ballot_sync(kFullMask, mine)) * kBoxBytes;
        const int slot = ring % C::kRing, use = ring / C::kRing;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint64_t* full = bars + (v ? C::kVFull : C::kKFull) + slot;
          if (use > 0) mbar_wait(bars + (v ? C::kVEmpty : C::kKEmpty) + slot, (use - 1) & 1, p.err);
          if (lane == 0) {
            if (bytes)
              mbar_arrive_expect_tx(full, bytes);
            else
              mbar_arrive(full);  // nothing to copy (a bad id is recorded above)
          }
          __syncwarp();
          if (mine) {
            unsigned char* dst = sm + (v ? C::kV : C::kK) + slot * C::kStage + c * kTok * 128 + u * kBlockSize * 128;
            // K and V that one item alone reads make way in L2 for the pieces'
            // rows (the batch above: 121.8 -> 116.2 us)
            if (k.s.groups == 1)
              tma_load_4d(dst, v ? &tmv : &tmk, c * 64, 0, k.g, e, full, once);
            else
              tma_load_4d(dst, v ? &tmv : &tmk, c * 64, 0, k.g, e, full);
          }
        }
        // Q of a later segment: once the last one's products are done with it;
        // the first stage's K and V are under way by then
        if (in == 0 && seg > 0) {
          mbar_wait(bars + C::kQEmpty, (seg - 1) & 1, p.err);
          load_q();
        }
      }
      ++seg;
    } while (k.next(p));
  } else if (warp == C::kQk) {
    // ------------------------------------------------------- S = Q K^T issue
    // S(i) goes into the buffer that P(i-2) leaves.  The warp waits together;
    // one elected lane issues.  Q K^T and P V are issued by a warp each: an
    // issuing warp is held until the tensor pipe takes its MMAs, and with one
    // warp for both the pipe stood idle while that warp waited for barriers.
    const uint64_t dq0 = tc::smem_desc_sw128(sm_s + C::kQ, 0, 1024);
    const uint64_t dk0 = tc::smem_desc_sw128(sm_s + C::kK, 0, 1024);
    int ring = 0, seg = 0;
    int done[TILES];  // stages of each tile so far
#pragma unroll
    for (int t = 0; t < TILES; ++t) done[t] = 0;
    bool ok = true;
    do {
      const int ns = k.st1 - k.st0, nt = k.tiles();
      ok = ok && mbar_wait(bars + C::kQFull, seg & 1, p.err);
      for (int i = 0; ok && i < ns; ++i, ++ring) {
        ok = ok && mbar_wait(bars + C::kKFull + ring % C::kRing, (ring / C::kRing) & 1, p.err);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (t >= nt) break;
          const int at = done[t];
          if (at > 1) ok = ok && mbar_wait(bars + C::kPvDone + 2 * t + (at & 1), ((at - 2) >> 1) & 1, p.err);
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t dq = tc::desc_at(dq0, t * C::kQTile), dk = tc::desc_at(dk0, (ring % C::kRing) * C::kStage);
          const uint32_t ds = tmem + C::s_col(t, at & 1);
          if (tc::elect_one()) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              tc::mma_bf16_ss(ds, tc::desc_at(dq, (s >> 2) * kRows * 128 + (s & 3) * 32),
                              tc::desc_at(dk, (s >> 2) * kTok * 128 + (s & 3) * 32), IDESC_S, s > 0);
            tc::commit(smem_addr(bars + C::kSFull + 2 * t + (at & 1)));
            if (t == nt - 1) {
              tc::commit(smem_addr(bars + C::kKEmpty + ring % C::kRing));
              if (i == ns - 1) tc::commit(smem_addr(bars + C::kQEmpty));
            }
          }
          __syncwarp();
          ++done[t];
        }
      }
      ++seg;
    } while (ok && k.next(p));
    // every MMA of this warp done before TMEM is freed, whatever happened above
    if (tc::elect_one()) tc::commit(smem_addr(bars + C::kDrain));
    __syncwarp();
    mbar_wait(bars + C::kDrain, 0, p.err);
  } else if (warp == C::kPv) {
    // ----------------------------------------------------------- O += P V issue
    const uint64_t dv0 = tc::smem_desc_sw128(sm_s + C::kV, kTok * 128, 1024);
    int ring = 0;
    int done[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) done[t] = 0;
    bool ok = true;
    do {
      const int ns = k.st1 - k.st0, nt = k.tiles();
      const bool half = MODE == kHalf32 || (MODE == kOneTile && k.rows() <= 64);
      int fresh = 0;  // the next stage that starts O anew
      for (int i = 0; ok && i < ns; ++i, ++ring) {
        const bool add = i != fresh;
        if (!add) fresh += C::sum_stages(half);
        ok = ok && mbar_wait(bars + C::kVFull + ring % C::kRing, (ring / C::kRing) & 1, p.err);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (t >= nt) break;
          const int at = done[t];
          ok = ok && mbar_wait(bars + C::kPFull + 2 * t + (at & 1), (at >> 1) & 1, p.err);
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t pc = tmem + C::s_col(t, at & 1), dout = tmem + C::o_col(t);
          const uint64_t dv = tc::desc_at(dv0, (ring % C::kRing) * C::kStage);
          if (tc::elect_one()) {
#pragma unroll
            for (int s = 0; s < kTok / 16; ++s) {
              const uint64_t bd = tc::desc_at(dv, s * 16 * 128);  // 16 tokens
              if (half) {
                // 8 columns hold high (rows 0-63) and low parts (64-127); the
                // third parts follow behind 32 columns
                tc::mma_bf16_ts(dout, pc + 8 * s, bd, IDESC_O, add || s > 0);
                if constexpr (MODE == kHalf32) tc::mma_bf16_ts(dout, pc + 32 + 8 * s, bd, IDESC_O, true);
              } else {
                // high parts in 8 columns of their chunk of 32, low parts 16
                // columns on, third parts behind the 64 columns
                const uint32_t hi = pc + 32 * (s >> 1) + 8 * (s & 1);
                tc::mma_bf16_ts(dout, hi, bd, IDESC_O, add || s > 0);
                tc::mma_bf16_ts(dout, hi + 16, bd, IDESC_O, true);
                if constexpr (MODE == kFull32) tc::mma_bf16_ts(dout, pc + 64 + 8 * s, bd, IDESC_O, true);
              }
            }
            tc::commit(smem_addr(bars + C::kPvDone + 2 * t + (at & 1)));
            if (t == nt - 1) tc::commit(smem_addr(bars + C::kVEmpty + ring % C::kRing));
          }
          __syncwarp();
          ++done[t];
        }
      }
    } while (ok && k.next(p));
    if (tc::elect_one()) tc::commit(smem_addr(bars + C::kDrain + 1));
    __syncwarp();
    mbar_wait(bars + C::kDrain + 1, 0, p.err);
  } else {
    // ---------------------------------------------------------- softmax rows
    // (Two threads a row, each with half of a stage's tokens, made the 64-node
    // batch slower, 42.4 us for 38.6.)
    const int t = warp / 4;                // this warpgroup's tile
    const int r = threadIdx.x - 128 * t;   // this thread's row (TMEM lane)
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const float scale = p.qk_scale_log2;
    int ring = 0, at = 0, seg = 0;
    bool task = false;
    do {
      const int ns = k.st1 - k.st0;
      if (t < k.tiles()) {
        const bool half = MODE == kHalf32 || (MODE == kOneTile && k.rows() <= 64);
        const bool upper = half && r >= 64;       // of two threads with the same row, the one with the low parts
        const int rr = half ? r & 63 : r;
        const int node = k.group * kNodes + t * QT + rr / G, head = k.g * G + rr % G;
        const bool ok = node < k.s.n;
        const bool live = __any_sync(kFullMask, ok);  // a warp past the tree's rows only keeps step
        const int P = k.s.L - k.s.n;
        const int64_t* mask = p.mask + static_cast<int64_t>(k.s.q0 + (ok ? node : 0)) * p.m_st;
        const uint64_t first_word = static_cast<uint64_t>(*mask);
        float m_used = -INFINITY, l = 0.f;  // max the weights are taken against; row sum
        // this row of the piece, and of the side sum until then, and its (max,
        // sum); this thread alone writes and reads them here
        auto piece = [&] {
          const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (seg > 0);
          return reinterpret_cast<float4*>(p.ws_o) + slot * (C::kItemRows * (D / 4)) + t * kRows + rr;
        };
        auto piece_ml = [&] {
          const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (seg > 0);
          return reinterpret_cast<float2*>(p.ws_ml) + slot * C::kItemRows + t * kRows + rr;
        };
        auto add_at = [&] { return reinterpret_cast<float4*>(sm + C::kAdd) + (r & 63) * (kAddRow / 4); };
        for (int i0 = 0, i1; i0 < ns; i0 = i1) {  // runs of one accumulation of O
          i1 = min(ns, i0 + C::sum_stages(half));
          if (i0 > 0 && (live || half)) {
            mbar_wait(bars + C::kPvDone + 2 * t + ((at - 1) & 1), ((at - 1) >> 1) & 1, p.err);
            sum_aside<D, C::kItemRows, C::kPair>(trow + C::o_col(t), half, upper, ok && !upper,
                                                 i0 == C::sum_stages(half), m_used, add_at(), piece(), piece_ml());
          }
          for (int i = i0; i < i1; ++i, ++at) {
            const int buf = at & 1;
            mbar_wait(bars + C::kSFull + 2 * t + buf, (at >> 1) & 1, p.err);
            tc::fence_after_sync();
            const int t0 = (k.st0 + i) * kTok;
            const bool edge = t0 + kTok > P;  // the stage reaches the nodes (or the end)
            if (live) {
              const uint32_t sc = trow + C::s_col(t, buf);
              uint32_t v[kTok];
              tc::ld_32x32b_x32(sc, *reinterpret_cast<uint32_t(*)[32]>(v));
              tc::ld_32x32b_x32(sc + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
              tc::wait_ld();
              float mx;
              float mul = scale;
              if (edge || scale < 0.f) {
                // scaled and masked here; a negative scale also turns the maximum
                mul = 1.f;
                mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t bits = edge ? seen_bits(first_word, mask, p.W, t0 + 32 * h, P, k.s.L) : 0xffffffffu;
#pragma unroll
                  for (int c = 0; c < 32; ++c) {
                    const float x = (bits >> c) & 1u ? __uint_as_float(v[32 * h + c]) * scale : -INFINITY;
                    v[32 * h + c] = __float_as_uint(x);
                    mx = fmaxf(mx, x);
                  }
                }
              } else {
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < kTok; c += 8) {
                  m0 = fmax3(m0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                  m1 = fmax3(m1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                  m2 = fmax3(m2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
                  m3 = fmax3(m3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
                }
                mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * scale;
              }
              const float m_new = fmaxf(m_used, mx);
              const bool need = ok && m_new > m_used + kRescaleSlack;
              const float alpha = need ? fast_exp2(m_used - m_new) : 1.f;  // 0 at the row's first seen token
              if (need) {
                l *= alpha;
                m_used = m_new;
              }
              if (i > i0 && __any_sync(kFullMask, need)) {
                mbar_wait(bars + C::kPvDone + 2 * t + ((at - 1) & 1), ((at - 1) >> 1) & 1, p.err);  // O stands still
                tc::fence_after_sync();
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                  uint32_t o[32];
                  tc::ld_32x32b_x32(trow + C::o_col(t) + 32 * c4, o);
                  tc::wait_ld();
#pragma unroll
                  for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                  tc::st_32x32b_x32(trow + C::o_col(t) + 32 * c4, o);
                }
              }
              const float m_ref = m_used == -INFINITY ? 0.f : m_used;  // nothing seen yet: every weight is 2^-inf
              const float2 mul2 = make_float2(mul, mul), nm2 = make_float2(-m_ref, -m_ref);
              float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t hi[16], lo[16], lo2[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 y = ffma2(make_float2(__uint_as_float(v[32 * h + 2 * e]), __uint_as_float(v[32 * h + 2 * e + 1])),
                                         mul2, nm2);
                  const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                  l2[e & 1] = fadd2(l2[e & 1], w);
                  split_bf16x2(w.x, w.y, hi[e], lo[e]);
                  if constexpr (MODE >= kFull32) {
                    const float r0 = w.x - bf16lo(hi[e]) - bf16lo(lo[e]), r1 = w.y - bf16hi(hi[e]) - bf16hi(lo[e]);
                    lo2[e] = pack_bf16x2(r0, r1);
                  }
                }
                if (half) {
                  if constexpr (MODE == kHalf32) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) lo2[e] = upper ? 0u : lo2[e];
                    tc::st_32x32b_x16(sc + 32 + 16 * h, lo2);
                  }
#pragma unroll
                  for (int e = 0; e < 16; ++e) hi[e] = upper ? lo[e] : hi[e];
                  tc::st_32x32b_x16(sc + 16 * h, hi);
                } else {
                  tc::st_32x32b_x16(sc + 32 * h, hi);
                  tc::st_32x32b_x16(sc + 32 * h + 16, lo);
                  if constexpr (MODE == kFull32) tc::st_32x32b_x16(sc + 64 + 16 * h, lo2);
                }
              }
              l += (l2[0].x + l2[1].x) + (l2[0].y + l2[1].y);
              tc::wait_st();
            }
            if (edge && t == 0) {
              // V rows of the nodes without their infinities and NaN, zeros
              // past the end (the slots there may hold anything)
              const int slot = (ring + i) % C::kRing;
              mbar_wait(bars + C::kVFull + slot, ((ring + i) / C::kRing) & 1, p.err);
              unsigned char* vst = sm + C::kV + slot * C::kStage;
              const int z0 = max(P - t0, 0);
              for (int idx = r; idx < (kTok - z0) * C::kBoxes * 8; idx += kRows) {
                const int vr = z0 + idx / (C::kBoxes * 8), rest = idx % (C::kBoxes * 8);
                uint4* at4 = reinterpret_cast<uint4*>(vst + (rest >> 3) * kTok * 128 + vr * 128 + (rest & 7) * 16);
                if (t0 + vr >= k.s.L) {
                  *at4 = make_uint4(0u, 0u, 0u, 0u);
                } else {
                  uint4 x = *at4;
                  const uint32_t b0 = nonfinite2(x.x), b1 = nonfinite2(x.y), b2 = nonfinite2(x.z), b3 = nonfinite2(x.w);
                  if (b0 | b1 | b2 | b3) {
                    *at4 = make_uint4(x.x & ~b0, x.y & ~b1, x.z & ~b2, x.w & ~b3);
                    *bad_v = 1;
                  }
                }
              }
              fence_proxy_async_smem();  // before the tensor cores read it
            }
            // (every warp sees every phase of a barrier, in order: a parity tells
            // a phase only from its neighbours)
            if (i > 0) mbar_wait(bars + C::kPvDone + 2 * t + ((at - 1) & 1), ((at - 1) >> 1) & 1, p.err);
            tc::fence_before_sync();  // P in TMEM before the arrival
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + C::kPFull + 2 * t + buf);
          }
        }

        // ---- this segment's rows, after its last P V
        mbar_wait(bars + C::kPvDone + 2 * t + ((at - 1) & 1), ((at - 1) >> 1) & 1, p.err);
        tc::fence_after_sync();
        const bool fix = *bad_v != 0;  // written before the arrivals that this P V followed
        const bool whole = k.whole();
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that saw nothing gives zeros
        OutT* dst = reinterpret_cast<OutT*>(p.out) + static_cast<int64_t>(k.s.q0 + node) * p.o_st +
                    static_cast<int64_t>(head) * p.o_sh;
        if (live || half) {
#pragma unroll 1
          for (int c4 = 0; c4 < D / 32; ++c4) {
            uint32_t v[32];
            read_o<C::kPair>(trow + C::o_col(t) + 32 * c4, half, upper, add_at(), v);
            if (upper) continue;
            if (ok && ns > C::sum_stages(half))
              add_piece<C::kItemRows>(piece(), c4, side_factor(piece_ml()->x, m_used), v);
            if (fix && ok) {
              // the infinities and NaN of the nodes this row sees
              const int a = max(P, k.st0 * kTok), z = min(k.s.L, k.st1 * kTok);
              for (int x = a; x < z; ++x) {
                const int j = x - P;
                if (!((mask[j >> 6] >> (j & 63)) & 1)) continue;
                const int blk = p.block_tables[static_cast<int64_t>(k.b) * p.bt_sb + x / kBlockSize];
                if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.NB)) continue;
                const __nv_bfloat16* vr =
                    p.v_cache + blk * p.vc_sblk + k.g * p.vc_sh + (x % kBlockSize) * D + 32 * c4;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  const float y = __bfloat162float(vr[c]);
                  if (!(fabsf(y) < INFINITY)) v[c] = __float_as_uint(__uint_as_float(v[c]) + y);
                }
              }
            }
            if (ok) {
              if (whole)
                store_row32(dst + 32 * c4, v, inv);
              else
                store_piece<C::kItemRows>(piece(), c4, v);
            }
          }
          if (ok && !whole && !upper) *piece_ml() = make_float2(m_used, l);
        }
        tc::fence_before_sync();  // O read before the next segment's first P V
        if (!whole && k.st0 == 0 && threadIdx.x == 0) {
          // the shares that hold the rest end with the one that holds line
          // position end - 1: the last c with floor(len c / count) < end
          const int64_t end = k.item0 + k.s.item;
          const int last = static_cast<int>(quotient(end * share->count + share->len - 1, share->len)) - 1;
          MergeTask m{last - static_cast<int>(blockIdx.x) + 1, 2 * static_cast<int>(blockIdx.x) + (seg > 0), k.s.q0,
                      k.s.n, k.group, k.g, {0, 0}};
          reinterpret_cast<MergeTask*>(p.ws_task)[blockIdx.x] = m;
          task = true;
        }
      }
      ring += ns;
      ++seg;
    } while (k.next(p));
    if (p.split && threadIdx.x == 0 && !task) reinterpret_cast<MergeTask*>(p.ws_task)[blockIdx.x].pieces = 0;
  }
  if (!any && p.split && threadIdx.x == 0) reinterpret_cast<MergeTask*>(p.ws_task)[blockIdx.x].pieces = 0;

  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kPv) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmem);
  }
}

// ------------------------------------------------------------ merge kernel
// Rows first .. first + 31 (a row per lane) of task `m` (of share c): with M =
// max of the pieces' maxima, out = sum 2^(m - M) O / sum 2^(m - M) l, for the
// 32 PER / SPLIT dims from d0: a warp takes 4 PER dims of one of SPLIT runs of
// the pieces, and the runs are joined in order at the end.  8 pieces' 4-dim
// groups are read at once: a round trip to L2 takes 1 to 2 us here.
template <int D, int G, typename OutT, int ITEM_ROWS, int PER, int SPLIT>
__device__ __forceinline__ void merge_rows(const TreeParams& p, const MergeTask& m, int c, int first, int d0,
                                           float (&stage)[32][D + 4], float2 (&joined)[32][9], int warp, int lane) {
  constexpr int kAhead = PER == 4 ? 2 : 8 / PER;
  constexpr int kAcross = kMergeThreads / 32 / SPLIT;  // warps that share the dims
  static_assert(SPLIT == 1 || PER == 1, "runs are joined for one 4-dim group a warp");
  const int part = warp / kAcross, across = warp % kAcross;
  const int k0 = m.pieces * part / SPLIT, k1 = m.pieces * (part + 1) / SPLIT;
  const int row = first + lane;
  const bool ok = m.group * ITEM_ROWS + row < m.n * G;
  auto slot = [&](int k) -> int64_t { return k == 0 ? m.slot0 : 2 * (c + k); };
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row;
  const float4* po = reinterpret_cast<const float4*>(p.ws_o) + row + (d0 / 4 + across * PER) * ITEM_ROWS;
  float M = -INFINITY, den = 0.f;
  float4 acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto scale = [&](float f) {
    den *= f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = make_float4(acc[e].x * f, acc[e].y * f, acc[e].z * f, acc[e].w * f);
  };
  for (int kk = k0; kk < k1; kk += kAhead) {
    float2 x[kAhead];
    float4 f[kAhead][PER];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool on = ok && kk + k < k1;
      x[k] = on ? __ldcg(ml + slot(kk + k) * ITEM_ROWS) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < PER; ++e)
        f[k][e] = on ? __ldcg(po + slot(kk + k) * (ITEM_ROWS * (D / 4)) + e * ITEM_ROWS)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) top = fmaxf(top, x[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    scale(fast_exp2(M - ref));
    M = top;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float w = fast_exp2(x[k].x - ref);
      den = fmaf(w, x[k].y, den);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        acc[e].x = fmaf(w, f[k][e].x, acc[e].x);
        acc[e].y = fmaf(w, f[k][e].y, acc[e].y);
        acc[e].z = fmaf(w, f[k][e].z, acc[e].z);
        acc[e].w = fmaf(w, f[k][e].w, acc[e].w);
      }
    }
  }
  if constexpr (SPLIT > 1) {
    joined[lane][warp] = make_float2(M, den);
    *reinterpret_cast<float4*>(&stage[lane][4 * warp]) = acc[0];
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int s = 1; s < SPLIT; ++s) {
        const float2 o = joined[lane][s * kAcross + across];
        const float4 x = *reinterpret_cast<const float4*>(&stage[lane][4 * (s * kAcross + across)]);
        const float top = fmaxf(M, o.x), ref = top == -INFINITY ? 0.f : top;
        scale(fast_exp2(M - ref));
        M = top;
        const float w = fast_exp2(o.x - ref);
        den = fmaf(w, o.y, den);
        acc[0].x = fmaf(w, x.x, acc[0].x);
        acc[0].y = fmaf(w, x.y, acc[0].y);
        acc[0].z = fmaf(w, x.z, acc[0].z);
        acc[0].w = fmaf(w, x.w, acc[0].w);
      }
    }
    __syncthreads();
  }
  if (part == 0) {
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int e = 0; e < PER; ++e)
      *reinterpret_cast<float4*>(&stage[lane][4 * (across * PER + e)]) =
          make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
  }
  __syncthreads();
  // out: kLanes lanes store a row's dims
  constexpr int kLanes = kAcross * PER;
#pragma unroll
  for (int i = threadIdx.x; i < 32 * kLanes; i += kMergeThreads) {
    const int r = i / kLanes, d = 4 * (i % kLanes), at = m.group * ITEM_ROWS + first + r;
    if (at < m.n * G) {
      OutT* dst = reinterpret_cast<OutT*>(p.out) + static_cast<int64_t>(m.q0 + at / G) * p.o_st +
                  static_cast<int64_t>(m.g * G + at % G) * p.o_sh + d0 + d;
      const float4 x = *reinterpret_cast<const float4*>(&stage[r][d]);
      if constexpr (sizeof(OutT) == 4)
        *reinterpret_cast<float4*>(dst) = x;
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
  }
  __syncthreads();
}

// Every block reads the shares' tasks, lists the groups of 32 rows that they
// make and takes its part.  A unit of work is a group, or where there are
// few (one long sequence's items) a slice of its dims.
template <int D, int G, int MODE>
__global__ void __launch_bounds__(kMergeThreads, 4) tree_merge_kernel(const TreeParams p, int shares) {
  constexpr int kWarps = kMergeThreads / 32, kMost = D / (4 * kWarps);  // slices of 32 dims
  constexpr int kItemRows = Cfg<D, MODE>::kItemRows;
  using OutT = typename Cfg<D, MODE>::Out;
  extern __shared__ int4 merge_smem[];       // the tasks, then the inclusive sums of their row groups
  MergeTask* tasks = reinterpret_cast<MergeTask*>(merge_smem);
  int* groups_to = reinterpret_cast<int*>(tasks + shares);
  __shared__ int warp_sum[kWarps];
  __shared__ float stage[32][D + 4];
  __shared__ float2 joined[32][9];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int sum = 0;
  for (int c0 = 0; c0 < shares; c0 += kMergeThreads) {
    const int c = c0 + tid;
    int groups = 0;
    if (c < shares) {
      const int4* src = reinterpret_cast<const int4*>(reinterpret_cast<const MergeTask*>(p.ws_task) + c);
      const int4 t0 = __ldcg(src), t1 = __ldcg(src + 1);
      merge_smem[2 * c] = t0;
      merge_smem[2 * c + 1] = t1;
      // (a task that this call cannot have left, from a call that wrongly
      // shared the scratch, is not followed: its rows could lie anywhere)
      const bool own = t0.x > 0 && c + t0.x <= shares && (t0.y >> 1) == c && t0.z >= 0 && t0.w > 0 &&
                       static_cast<int64_t>(t0.z) + t0.w <= p.T && t1.x >= 0 &&
                       static_cast<int64_t>(t1.x) * kItemRows < static_cast<int64_t>(t0.w) * G &&
                       static_cast<unsigned>(t1.y) < static_cast<unsigned>(p.Hkv);
      if (own) groups = (min(t0.w * G - t1.x * kItemRows, kItemRows) + 31) / 32;
    }
    int incl = groups;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFullMask, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += warp_sum[w];
      all += warp_sum[w];
    }
    if (c < shares) groups_to[c] = sum + incl;
    sum += all;
    __syncthreads();
  }
  const int blocks = static_cast<int>(gridDim.x);
  const int slices = sum * 4 * kMost <= blocks ? 4 * kMost : kMost == 4 && sum * 4 <= blocks ? 4 : sum * 2 <= blocks ? 2 : 1;
  for (int u = blockIdx.x; u < sum * slices; u += blocks) {
    const int rg = u / slices, d0 = (u % slices) * (D / slices);
    int lo = 0, hi = shares - 1;  // the first task with groups_to > rg
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (groups_to[mid] > rg)
        hi = mid;
      else
        lo = mid + 1;
    }
    const MergeTask m = tasks[lo];
    const int first = (rg - (lo > 0 ? groups_to[lo - 1] : 0)) * 32;  // of the item's rows
    if (slices == 4 * kMost) {  // few rows: the warps share the pieces too
      merge_rows<D, G, OutT, kItemRows, 1, 4>(p, m, lo, first, d0, stage, joined, warp, lane);
    } else if (slices == 1) {
      merge_rows<D, G, OutT, kItemRows, kMost, 1>(p, m, lo, first, d0, stage, joined, warp, lane);
    } else if (kMost == 2 || slices == 4) {
      merge_rows<D, G, OutT, kItemRows, 1, 1>(p, m, lo, first, d0, stage, joined, warp, lane);
    } else {
      merge_rows<D, G, OutT, kItemRows, 2, 1>(p, m, lo, first, d0, stage, joined, warp, lane);
    }
  }
}

// ------------------------------------------------------------ launch
template <int D, int G, int MODE>
cudaError_t launch_mode(const TreeParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        const TreePlan& plan, cudaStream_t stream) {
  using C = Cfg<D, MODE>;
  auto kernel = tree_kernel<D, G, MODE>;
  static std::atomic<int> smem_set[64];  // one record per instantiation
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) dev = 63;
  if (!smem_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    smem_set[dev].store(1);
  }
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(plan.grid)), dim3(C::kThreads), C::kSmem, stream, tmq, tmk, tmv, p);
  if (e != cudaSuccess || !p.split) return e;
  return launch_pdl(tree_merge_kernel<D, G, MODE>, dim3(static_cast<unsigned>(plan.merge_grid)), dim3(kMergeThreads),
                    static_cast<size_t>(plan.grid) * (sizeof(MergeTask) + 4), stream, p, plan.grid);
}

template <int D, int G>
cudaError_t launch_plan(const TreeParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        const TreePlan& plan, cudaStream_t stream) {
  switch (plan.mode) {
    case kOneTile: return launch_mode<D, G, kOneTile>(p, tmq, tmk, tmv, plan, stream);
    case kTwoTiles: return launch_mode<D, G, kTwoTiles>(p, tmq, tmk, tmv, plan, stream);
    case kFull32: return launch_mode<D, G, kFull32>(p, tmq, tmk, tmv, plan, stream);
    case kHalf32: return launch_mode<D, G, kHalf32>(p, tmq, tmk, tmv, plan, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <int D>
cudaError_t launch_g(const TreeParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int G,
                     const TreePlan& plan, cudaStream_t stream) {
  switch (G) {
    case 1: return launch_plan<D, 1>(p, tmq, tmk, tmv, plan, stream);
    case 2: return launch_plan<D, 2>(p, tmq, tmk, tmv, plan, stream);
    case 4: return launch_plan<D, 4>(p, tmq, tmk, tmv, plan, stream);
    case 8: return launch_plan<D, 8>(p, tmq, tmk, tmv, plan, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// bf16 out: two tiles per item when the sequences' rows fill more than one on
// average (then both share one stream of K and V).  fp32 out: 64 rows per item
// while the rows fit on average, else 128.  CTAs: what is resident at once,
// fewer when the table's span has no min_share for each: one stage and an
// item's start (above item_cost, so that no share inside an item is without a
// stage).  One sequence of 2000 tokens with 16 nodes, 8 KV heads of 4: 18.3 us
// at 5, 18.8, 20.7, 24.5 and 28.0 at 6, 8, 12 and 16.  Items of up to
// kWholeStages stages are not cut, as the merge kernel costs more than the
// stages of one item do: 400 tokens 15.5 us whole, 17.4 us cut.
TreePlan plan_tree(int64_t T, int64_t B, int64_t Hkv, int64_t MB, int G, int D, bool out_bf16, int num_sms) {
  constexpr int kWholeStages = 8;
  TreePlan r;
  r.mode = out_bf16 ? (T * G > B * kRows ? kTwoTiles : kOneTile) : (T * G > B * 64 ? kFull32 : kHalf32);
  const int64_t rows = r.mode == kTwoTiles ? 2 * kRows : r.mode == kHalf32 ? 64 : kRows;  // of an item
  const int64_t nodes = rows / G;
  const int64_t stages = (MB * kBlockSize + kTok - 1) / kTok;      // of the longest item
  const int64_t items = ((T + nodes - 1) / nodes + B) * Hkv;       // at least as many as there are
  const int64_t resident = static_cast<int64_t>(num_sms) * (r.mode == kOneTile || r.mode == kHalf32 ? 2 : 1);
  r.split = stages > kWholeStages;
  r.min_share = r.split ? 5 : 1;
  const int64_t most = r.split ? items * (stages + item_cost(static_cast<int>(rows))) / r.min_share : items;
  r.grid = static_cast<int>(most < 1 ? 1 : most > resident ? resident : most);
  r.grid = r.grid > kMaxShares ? kMaxShares : r.grid;
  r.merge_grid = 4 * num_sms;
  const int64_t pieces = 2ll * r.grid;                             // two a CTA
  r.o_bytes = static_cast<size_t>(pieces * rows) * D * 4;
  r.ml_bytes = static_cast<size_t>(pieces * rows) * 2 * 4;
  r.task_bytes = static_cast<size_t>(r.grid) * sizeof(MergeTask);
  return r;
}

cudaError_t launch_tree(const TreeParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                        int D, int G, const TreePlan& plan, cudaStream_t stream) {
  if (D == 128) return launch_g<128>(p, tmq, tmk, tmv, G, plan, stream);
  if (D == 64) return launch_g<64>(p, tmq, tmk, tmv, G, plan, stream);
  return cudaErrorInvalidValue;
}

}  // namespace forge
