// Attention of a call's new tokens over the paged cache (dspark_block_attention), on the
// fifth-generation tensor cores (tcgen05).
//
// Mathematics. For one new token and query head, out = sum_t e^(z_t) v_t / sum_t e^(z_t),
// z_t = scale q . k_t over the seen positions t. One pass over the keys with the running
// maximum m and sum l of the softmax: a tile of 128 positions adds p_t = 2^(c z_t - c m) to l and
// p_t v_t to O (c = log2 e); when a new maximum exceeds m by more than 8 binary orders, l and O
// are scaled by 2^(c m - c m'). Smaller excesses leave m as it is: p then reaches at most 2^8,
// which costs float32 and the 16-bit weights no precision, and the rescaling of O is rare. f16
// weights (and with them l and O) are made 2^12 times larger and may exceed that by 3 orders, up to
// 2^15: unscaled, the small weights of a long context, each below 2^-25, would vanish while l
// counts them. Now a weight is off by at most 2^-37 of the largest (f16's subnormal half step)
// beside its relative 2^-11: 2^-17 of the result for 2^20 of them.
//
// What bounds it. The keys and values of a cache head are read once for all G query heads that
// share it and all new tokens of the sequence: with few tokens 2 head_dim 2 bytes of HBM per
// position are the cost, with a prompt's chunk the 4 head_dim operations (and one exponential)
// per (row, position).
//
// Rows and items. The n G rows (new token, query head) of a sequence and cache head are cut into
// items of at most 128 rows when there are so few, else 256: an item's rows all read the same
// keys. A unit is a tile of 128 positions of one item (or the like of a tile's time, for an
// item's own cost: without it 64 decode tokens over 256 to 4096 positions took 84 us instead of
// 70). The call's units, in the order (sequence, cache head, item, tile), are dealt in equal
// contiguous runs to one CTA per SM, so sequences of any lengths balance; an item that a run's
// border cuts is finished by attention_join_kernel from float32 partial results (at most two per
// CTA).
//
// One CTA, 12 warps:
//  - warps 0-3 and 4-7, softmax groups 0 and 1: thread = row = TMEM lane. Group s reads its scores
//    S_s from tensor memory, keeps m and l, writes the weights P_s (16 bits, over S_s) back, and
//    at the end O_s to global memory. An item of 256 rows gives each group 128 rows and every
//    tile; an item of up to 128 rows gives both groups the same rows and every other tile, and
//    the group of the first tile (they take turns at that) joins the two results at the end.
//  - warps 8 and 10: look up pages and issue the TMA copies of the K and the V tiles (boxes of up
//    to 128 slots x 64 elements, 128-byte swizzle) into a ring of stages; warp 8 also deals the
//    units and announces the items.
//  - warp 11: zeroes values that must not count (see below).
//  - warp 9: per tile S_s = Q_s K^T (both from shared memory), then O_s += P_s V (P_s
//    from tensor memory). Q_s, written by the group, stays in shared memory for the item.
// Tensor memory: S_0, S_1 (128 columns each, P_s over S_s), O_0, O_1 (128 columns each).
//
// Measured (one B200, back to back in a graph): blocks of up to 8 tokens of 64 sequences over 1024
// to 16384 positions, 32 / 8 heads of 128, 1.47 GB: 232 us, 6.3 TB/s, 98% of the measured copy
// rate; in seconds-long loops, where the power limit sets the clock, 248 us, 92%. A 4096-token chunk
// at 12288: 589 us, 1.17 PFLOP/s, 71% of cuBLAS's bf16 rate in a burst; 671 us in such loops
// (cuBLAS itself then makes 86% of its burst rate). There a group's chain (scores, weights, both products) takes some 3600 clocks a
// tile against 2048 of the tensor cores' own; a one-tile item costs 12 us beside its launch.
//
// Sums. Tensor memory holds O of at most 64 tiles of a group (bf16: 256); then the group moves it
// to a float32 sum in the workspace, by ordinary rounded additions. Without that equal weights over
// 131072 positions gave values 4.6e-4 too small, over 524288 2.8e-3, and a sum of ones stopped at
// 2^26.
//
// Waits. Every mbarrier wait is bounded (2^31 clocks, about a second; the zeroing warp's, which can
// take as long as an item, 32 times that); one that runs out sets an
// abort flag that ends every role's loop, is counted (dspark_pipeline_timeouts) and noted for the
// kernel that joins pieces, which reports it (DSPARK_SEQ_TIMEOUT) and gives NaN for the items that
// lack a piece; the CTA lets the copies and products in flight finish (again bounded) and frees the
// tensor memory.
//
// Unseen places. Scores outside a row's range become -inf whatever they are. A weight of 0 times
// a non-finite value would be NaN, so in a tile that some row of the item does not see in full
// the values outside the item's range, and any with a non-finite element, are zeroed in shared
// memory first; a row that sees a value so zeroed, or a page whose id is out of range (its TMA
// box is filled with zeros), gives NaN.
#pragma once

#include <type_traits>

#include "markov_mma.cuh"
#include "rotary.cuh"
#include "stream.cuh"

namespace dspark {

constexpr int kAtThreads = 384;    // three warpgroups: two of softmax, one of the other roles
// Registers a thread: the launch gives 168; the softmax groups keep a tile's 128 scores in
// registers and take what the third warpgroup gives up (216 + 216 + 72 = 3 x 168).
constexpr int kAtGroupRegs = 216, kAtOtherRegs = 72;
constexpr int kAtTile = 128;        // positions per tile (and rows per softmax group)
constexpr int kAtItemRows = 256;    // rows of an item, at most
constexpr int kAtItemUnits = 3;     // what an item costs beside its tiles, in tiles
constexpr int kAtDescs = 4;         // items announced ahead
constexpr int kAtBadRing = 16;      // tiles whose bad-page masks are kept
constexpr int kAtFixRing = 8;       // tiles whose masks of zeroed values are kept
// |c m| from which scores are reduced to z - m before the product with c: below it the rounding of
// c m is at most 2^-17, relative to a weight a 64th of f16's half step. (Always reducing them: 683
// us instead of 623 for a 4096-token chunk at 12288; the instructions lie on a warp's chain.)
constexpr float kAtLargeScore = 128.f;

// Binary orders by which the weights (and l and O) are enlarged.
template <typename T>
__host__ __device__ constexpr float at_shift() {
  return std::is_same<T, __half>::value ? 12.f : 0.f;
}
// Binary orders that a new maximum may exceed the kept one by.
template <typename T>
__host__ __device__ constexpr float at_rescale() {
  return std::is_same<T, __half>::value ? 3.f : 8.f;
}
// Tiles of a group after which its O moves from tensor memory to a sum in the workspace (a power of
// two). The tensor cores cut each product off 25 places below the sum that it joins, a bias of up
// to 128 x 2^-25 of O per tile: 2.4e-4 for 64 and 9.8e-4 for 256, half and a quarter of the half
// step of f16 and bf16. (With 64 for bf16 too, a 4096-token chunk at 12288, where an item then
// moves its sum once, took 665 us instead of 646.)
template <typename T>
__host__ __device__ constexpr int at_sum_tiles() {
  return std::is_same<T, __half>::value ? 64 : 256;
}
__host__ __device__ constexpr int at_stage_bytes(int dp) { return kAtTile * dp * 2; }
__host__ __device__ constexpr int at_stages(int dp) { return dp == 128 ? 5 : 10; }

struct AttnParams {
  dspark_heads_t q, out;
  dspark_kv_cache_t cache;
  dspark_rows_t rows;
  float* lse;
  int32_t* status;
  int Hq, causal, window;
  FastDiv by_group;  // division by the query heads of a cache head
  float scale_log2;  // scale log2(e)
  int box, box_log2; // slots per TMA box: min(page_size, 128)
  int page_log2;
  int part_rows;     // rows of a partial result's slot
  int which_k, which_v;  // last coordinate of keys and of values in their tensor maps
  int withhold;      // (tests of the timeout path) each CTA's first K copy is not issued
  float* part_o;     // [2 CTAs][part_rows][DP]
  float2* part_ml;   // [2 CTAs][part_rows]: (m; l)
  struct AttnJoin* join;  // [CTAs]
  float* sums;       // [CTAs][2 groups][DP][sum_rows]: O of an item's earlier tiles (at_sum_tiles)
  int sum_rows;
};

// An item cut by a border: its first piece is in slot 2 cta + 1 of the CTA it begins in, the
// others in slots 2 (cta + 1), 2 (cta + 2), ...; pieces == 0: nothing to join. Every CTA writes its
// record at its start, and at its end whether it gave up on a wait.
struct AttnJoin {
  int h, row0, rows, first, pieces, gave_up;
};

// What a CTA does with one item (or its piece of it).
struct AttnItem {
  int b, h, row0, rows;  // the rows row0 .. row0 + rows - 1 of (sequence b, cache head h)
  int L, n, first;       // the sequence's SeqRows
  int t0, nt;            // tiles t0 .. t0 + nt - 1
  int slot;              // partial result's slot; -1: the item is whole
  int load0;             // loads (two per tile) that the CTA made before this item
  int lo, hi;            // positions that some row of the item sees
  int full0, full1;      // tiles [full0, full1) are seen in full by every row
  int fix0;              // tiles not seen in full that the CTA met before this item

  __device__ __forceinline__ bool partial(int t) const { return t < full0 || t >= full1; }
  // tiles of the piece before t that are not seen in full
  __device__ __forceinline__ int partials_before(int t) const {
    return t - t0 - max(0, min(t, full1) - max(t0, full0));
  }
};

// The positions [lo, hi) that new token i (of n, in a cache of L tokens) sees.
__device__ __forceinline__ void seen_range(int L, int n, int i, int causal, int window, int& lo,
                                           int& hi) {
  const int pos = L - n + i;
  hi = causal ? min(L, pos + 1) : L;
  lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  if (hi < lo) hi = lo;
}

// ------------------------------------------------------------------------ PTX helpers

// One box of a tile: each lane of a loader issues its own. (One elected lane issuing them all: 374
// us instead of 275 for the serving blocks in pages of 8, 367 instead of 295 for 128 of them with
// heads of 64 in pages of 16; no difference from pages of 32 on.)
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, int v, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
      : "memory");
}
// The MMA issuer is a whole warp that follows one path, so that addresses and descriptors stay in
// uniform registers; one elected lane issues each product and commit. (Issued from inside a
// one-lane branch, a 4096-token chunk at 12288 took 736 us instead of 609.)
// A value known to be the same in every lane, as such.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// D = A B (first) or D += A B, both operands in shared memory.
__device__ __forceinline__ void at_mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A (128 x 16 of 16-bit values) in tensor memory.
__device__ __forceinline__ void at_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void at_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
          "r"(bar)
      : "memory");
}

// 32 consecutive 32-bit columns of this warp's 32 TMEM lanes (one row per lane).
#define DSPARK_R32(X)                                                                       \
  X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13),   \
      X(14), X(15), X(16), X(17), X(18), X(19), X(20), X(21), X(22), X(23), X(24), X(25),   \
      X(26), X(27), X(28), X(29), X(30), X(31)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
#define DSPARK_OUT(i) "=f"(v[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : DSPARK_R32(DSPARK_OUT)
      : "r"(taddr)
      : "memory");
#undef DSPARK_OUT
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
#define DSPARK_IN(i) "r"(v[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::DSPARK_R32(DSPARK_IN),
      "r"(taddr)
      : "memory");
#undef DSPARK_IN
}
#undef DSPARK_R32
// 16 bytes from global to shared memory; the last 16 - bytes of them are zeros.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// mbar_wait with little code (it is inlined often, and the kernel's code should stay in the
// instruction cache): a wait that expires (2^31 clocks, and 2^30 more for every further
// round) sets the abort flag, which the CTA counts once at its end.
template <int kRounds = 1>
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  uint32_t t0 = static_cast<uint32_t>(clock());
  int round = 1;
  do {
    if (mbar_try(bar, parity)) return true;
    if (round < kRounds && static_cast<uint32_t>(clock()) - t0 >= (1u << 30)) {
      t0 += 1u << 30;
      ++round;
    }
  } while (!*abort && static_cast<uint32_t>(clock()) - t0 < (1u << 31));
  *abort = 1;
  return false;
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of V as the B operand of P V: element (position k, dim n) with
// the dims contiguous (MN-major), 128-byte swizzle: atoms of 8 positions x 64 dims (1024 bytes),
// the next 8 positions 1024 bytes on, the next 64 dims a tile's half (128 x 128 bytes) on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((kAtTile * 128) >> 4) << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// Instruction descriptor: kind::f16, A and B bf16 (bf) or f16, D float32, M = 128, N = n; B
// K-major, or MN-major (mn).
__host__ __device__ constexpr uint32_t at_idesc(int n, bool bf, bool mn) {
  return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// A mean of finite f16 values lies within their range, but weights that were rounded up (by 2^-11)
// can carry one next to the end over it, where f16 rounds to infinity. What is not finite stays.
constexpr float kF16Max = 65504.f;
__device__ __forceinline__ float f16_range(float x) {
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -kF16Max), kF16Max) : x;
}

// O of a row (t_o: its warp's lanes and columns) plus f times the sum kept at `sum` (load), to
// there (store) or back to tensor memory. Element d of the row is at sum[d * stride], so that a
// warp's accesses are whole lines (16-byte accesses by row: 695 us for the chunk above with 64).
// Not inlined: cold code between the hot costs instruction fetches.
template <int DP>
__device__ __noinline__ void at_move_sum(uint32_t t_o, float* sum, int stride, float f, bool load,
                                         bool store, bool to_tmem) {
#pragma unroll 1
  for (int q = 0; q < DP; q += 32) {
    float o[32];
    tmem_ld32(t_o + q, o);
    float a[32];
#pragma unroll
    for (int y = 0; y < 32; ++y) a[y] = load ? sum[(q + y) * stride] : 0.f;
    __syncwarp();
    tmem_ld_wait();
#pragma unroll
    for (int y = 0; y < 32; ++y) o[y] += a[y] * f;
    if (store) {
#pragma unroll
      for (int y = 0; y < 32; ++y) sum[(q + y) * stride] = o[y];
    }
    __syncwarp();
    if (to_tmem) {
      uint32_t ow[32];
#pragma unroll
      for (int y = 0; y < 32; ++y) ow[y] = __float_as_uint(o[y]);
      tmem_st32(t_o + q, ow);
    }
  }
  if (to_tmem) tmem_st_wait();
}

// ------------------------------------------------------------------------ units and items

// Items of a (sequence, cache head) with R rows, and the tiles of an item.
__device__ __forceinline__ int item_count(int R) {
  return R <= kAtTile ? (R > 0) : (R + kAtItemRows - 1) / kAtItemRows;
}
// The positions that the first and the last token of an item see: the item needs [lo, hi), and
// every row of it sees [flo, fhi).
struct ItemRange {
  int lo, hi, flo, fhi;
};
__device__ __forceinline__ ItemRange item_range(const AttnParams& p, int L, int n, int row0,
                                                int rows) {
  ItemRange r;
  seen_range(L, n, p.by_group.div(row0), p.causal, p.window, r.lo, r.fhi);
  seen_range(L, n, p.by_group.div(row0 + rows - 1), p.causal, p.window, r.flo, r.hi);
  return r;
}
__device__ __forceinline__ int first_tile(const ItemRange& r) { return r.lo / kAtTile; }
__device__ __forceinline__ int tile_count(const ItemRange& r) {
  return r.hi > r.lo ? (r.hi + kAtTile - 1) / kAtTile - r.lo / kAtTile : 0;
}
// Units of one cache head of a sequence: its items' tiles, and kAtItemUnits before each item's
// first for what an item costs beside its tiles.
__device__ __forceinline__ long long head_units(const AttnParams& p, int L, int n, int G) {
  const int R = n * G, items = item_count(R);
  long long u = 0;
#pragma unroll 1
  for (int i = 0; i < items; ++i)
    u += kAtItemUnits + tile_count(item_range(p, L, n, i * kAtItemRows,
                                              min(kAtItemRows, R - i * kAtItemRows)));
  return u;
}
// Element offset of token i of sequence b.
__device__ __forceinline__ int64_t token_offset(const dspark_heads_t& t, const AttnParams& p,
                                                int b, int first, int i) {
  return p.rows.q_start ? static_cast<int64_t>(first + i) * t.token_stride
                        : b * t.seq_stride + static_cast<int64_t>(i) * t.token_stride;
}

// a / b for non-negative values: a 32-bit division where both fit (a call waits for it).
__device__ __forceinline__ long long quick_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Loads of an item of nt tiles, in ring order: the first `look` K tiles, then V_j and K_{j+look}
// in turn. The index of K_j and of V_j among them.
__device__ __forceinline__ int load_of_k(int j, int look) {
  return j < look ? j : 2 * j - look + 1;
}
__device__ __forceinline__ int load_of_v(int j, int look, int nt) {
  return look + j + min(j, nt - look);
}
// K tiles loaded ahead of the first V: one when both groups take every tile, two when they
// alternate.
__device__ __forceinline__ int look_ahead(int rows, int nt) {
  return rows > kAtTile ? 1 : min(2, nt);
}

template <int DP>
struct AttnSmem {
  static constexpr int kStages = at_stages(DP);
  static constexpr int kStage = at_stage_bytes(DP);
  static constexpr int kQ = 0;                                // [2][kStage]
  static constexpr int kKv = 2 * kStage;                      // [kStages][kStage]
  static constexpr int kBars = kKv + kStages * kStage;        // 64 mbarriers
  static constexpr int kItems = kBars + 512;                  // [kAtDescs] AttnItem
  static constexpr int kBad = kItems + kAtDescs * 64;         // [kAtBadRing][4] masks
  static constexpr int kNf = kBad + kAtBadRing * 16;          // [kAtFixRing][4] masks
  static constexpr int kMl = kNf + kAtFixRing * 16;                       // [128] float2
  static constexpr int kMisc = kMl + 1024;                    // tensor memory's base, abort flag
  static constexpr int kTotal = kMisc + 128;
};
static_assert(sizeof(AttnItem) == 64, "item descriptor");
static_assert(AttnSmem<128>::kTotal <= 232448 && AttnSmem<64>::kTotal <= 232448, "shared memory");

// Barriers of the CTA (indices into the 64 at kBars), and the arrivals each takes.
enum AttnBar {
  kBarFull = 0,       // [10] a stage's copy has landed (1, expect_tx)
  kBarEmpty = 10,     // [10] a stage's products are done (1, commit)
  kBarS = 20,         // [2] S_s is ready (1, commit)
  kBarO = 22,         // [2] the item's O_s is done (1, commit)
  kBarItem = 24,      // [4] an item is announced (1)
  kBarFix = 28,       // [8] a tile's unseen values are zeroed (1)
  kBarToFix = 36,     // [8] the copy of such a tile is on its way (1)
  kBarDrain = 44,     // the MMAs in flight at an abort (1, commit)
  kBarP = 45,         // [2] P_s is written (4 warps)
  kBarQ = 47,         // [2] Q_s is written (4 warps)
  kBarMl = 49,        // the other group's m and l are written (4 warps)
  kBarJoined = 50,    // and its O is read (4 warps)
  kBarItemFree = 51,  // [4] an item is read by the warps of all roles but the dealer (11)
  kBarCount = 55
};

template <typename T, int DP>
__global__ void __launch_bounds__(kAtThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ AttnParams p) {
  using Sm = AttnSmem<DP>;
  constexpr bool kBf = sizeof(T) == 2 && !std::is_same<T, __half>::value;
  constexpr float kShift = at_shift<T>(), kRescale = at_rescale<T>();
  constexpr int kSumTiles = at_sum_tiles<T>();
  constexpr int kStages = Sm::kStages;
  constexpr int kHalves = DP / 64;
  extern __shared__ __align__(1024) uint8_t at_smem[];
  uint8_t* sm = at_smem;
  const uint32_t sb = smem_u32(sm);
  auto bar = [&](int i) { return sb + Sm::kBars + 8 * i; };
  // a wait of the whole warp, with one outcome for all its lanes
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + Sm::kMisc + 4);
  auto wait_rounds = [&](auto rounds, int i, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      at_wait<decltype(rounds)::value>(bar(i), parity & 1, s_abort)) != 0;
  };
  constexpr std::integral_constant<int, 1> kOnce{};
  auto wait = [&](int i, uint32_t parity) { return wait_rounds(kOnce, i, parity); };
  AttnItem* s_items = reinterpret_cast<AttnItem*>(sm + Sm::kItems);
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(sm + Sm::kBad);
  uint32_t* s_nf = reinterpret_cast<uint32_t*>(sm + Sm::kNf);
  float2* s_ml = reinterpret_cast<float2*>(sm + Sm::kMl);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + Sm::kMisc);

  const int tid = threadIdx.x, wi = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const dspark_kv_cache_t& c = p.cache;
  const int Hk = c.n_heads, G = p.Hq / Hk, D = c.head_dim;
  const int64_t cap = static_cast<int64_t>(c.max_pages) << p.page_log2;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kBarCount; ++i)
      mbar_init(bar(i), i < kBarP ? 1 : i < kBarItemFree ? 4 : 11);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  if (wi == 9) tmem_alloc_all(s_tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *s_tmem, 0);
  grid_dependency_wait();  // lengths, queries and the cache come from the kernels before
  grid_dependents_launch();

  // the next announced item (rows == 0: the end); false on an abort
  int items = 0;
  auto fetch_rounds = [&](auto rounds, AttnItem& to) {
    const int d = items % kAtDescs;
    if (!wait_rounds(rounds, kBarItem + d, items / kAtDescs)) return false;
    to = s_items[d];
    ++items;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemFree + d));
    return true;
  };
  auto fetch = [&](AttnItem& to) { return fetch_rounds(kOnce, to); };

  if (wi >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtOtherRegs));
  if (wi == 8 || wi == 10) {
    // ------------------------------------------------------------------ loaders
    // Warp 8 deals the items and loads K, warp 10 loads V.
    const bool is_k = wi == 8;
    const CUtensorMap* map = is_k ? &kmap : &vmap;
    const int which = is_k ? p.which_k : p.which_v;
    const int boxes = kAtTile >> p.box_log2;
    bool live = true;
    int last = -1;  // lane i: the last load into stage i by this warp
    // The lanes hold the page ids of a window of 32 boxes; the next window's, and those of the
    // next item's first window, are on their way.
    auto fetch_ids = [&](const AttnItem& it, int w) {
      const int x0 = (32 * w + lane) << p.box_log2;
      return x0 < it.hi ? __ldg(c.page_table + it.b * c.ld_table + (x0 >> p.page_log2)) : -1;
    };
    auto first_window = [&](const AttnItem& it) { return (it.t0 << (7 - p.box_log2)) >> 5; };
    // the tiles of an item (piece)
    auto load_item = [&](const AttnItem& it, int ids) {
      const int look = look_ahead(it.rows, it.nt);
      int window = first_window(it);
      int ids_next = fetch_ids(it, window + 1);
#pragma unroll 1
      for (int j = 0; j < it.nt; ++j) {
        const int t = it.t0 + j, box0 = t << (7 - p.box_log2);
        if ((box0 >> 5) != window) {
          window = box0 >> 5;
          ids = ids_next;
          ids_next = fetch_ids(it, window + 1);
        }
        // the boxes that overlap [lo, hi); a page id out of range becomes n_pages, whose boxes
        // are filled with zeros, and with K the mask of its positions is kept
        int page = __shfl_sync(0xffffffffu, ids, (box0 + lane) & 31);
        const int x0 = t * kAtTile + (lane << p.box_log2);
        const bool need = lane < boxes && x0 < it.hi && x0 + p.box > it.lo;
        const bool out = page < 0 || page >= c.n_pages;
        const uint32_t all = __ballot_sync(0xffffffffu, need);
        const uint32_t bad = __ballot_sync(0xffffffffu, need && out);
        if (out) page = c.n_pages;
        const int g = it.load0 + (is_k ? load_of_k(j, look) : load_of_v(j, look, it.nt));
        const int st = g % kStages;
        if (is_k && lane < 4) {
          uint32_t m = 0;
          if (bad) {
#pragma unroll 1
            for (int k = 0; k < 32; ++k)
              if ((bad >> ((32 * lane + k) >> p.box_log2)) & 1) m |= 1u << k;
          }
          s_bad[((it.load0 / 2 + j) % kAtBadRing) * 4 + lane] = m;
        }
        __syncwarp();  // (lane 0's arrive below releases all four words)
        if (!wait(kBarEmpty + st, (g / kStages) ^ 1)) return false;
        if (p.withhold && g == 0 && is_k) continue;
        if (lane == 0)
          mbar_arrive_tx(bar(kBarFull + st),
                         static_cast<uint32_t>(__popc(all)) * p.box * 128 * kHalves);
        if (lane == st) last = g;
        if (!is_k && lane == 0 && it.partial(t))
          mbar_arrive(bar(kBarToFix + (it.fix0 + it.partials_before(t)) % kAtFixRing));
        __syncwarp();
        if (need) {
          const uint32_t dst = sb + Sm::kKv + st * Sm::kStage + (lane << p.box_log2) * 128;
          const int y = p.box < kAtTile ? 0 : (t * kAtTile) & (c.page_size - 1);
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf)
            tma_load_5d(dst + hf * (kAtTile * 128), map, 64 * hf, y, it.h, page, which,
                        bar(kBarFull + st));
        }
        __syncwarp();
      }
      return true;
    };

    // The dealer's state: the sequence, its rows and items per head, the next item among its heads,
    // the units to skip before the first item and those left of this CTA's run.
    const int B = p.rows.B;
    int b = B, R = 0, count = 0, x = 0, loads = 0, fixes = 0;
    long long off = 0, left = 0, quota = 1;
    int win = -64;  // the lanes hold the rows of 32 sequences
    SeqRows ws{}, sq{};
    if (is_k) {
      // this CTA's run: a scan of the sequences' units, `per` neighbouring sequences a lane
      const int per = (B + 31) / 32, b_lo = min(B, lane * per), b_hi = min(B, b_lo + per);
      long long mine = 0;
#pragma unroll 4
      for (int i = b_lo; i < b_hi; ++i) {
        seq_rows(p.rows, c.kv_len, cap, i, ws);
        mine += Hk * head_units(p, ws.L, ws.n, G);
      }
      if (per == 1) win = 0;  // (one sequence a lane: ws holds it)
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const long long total = __shfl_sync(0xffffffffu, upto, 31);
      // two units a CTA at least: the two softmax groups take one each, in the time of one
      quota = max(2ll, quick_div(total + gridDim.x - 1, gridDim.x));
      const long long u0 = quota * blockIdx.x;
      left = min(quota, total - u0);
      if (left > 0) {
        const int at = __popc(__ballot_sync(0xffffffffu, upto <= u0));  // the lane of unit u0
        off = u0 - __shfl_sync(0xffffffffu, upto - mine, at);
        b = at * per - 1;  // (the walk steps to the next sequence first)
      }
      if (lane == 0) p.join[blockIdx.x] = AttnJoin{};
    }
    // the next item of the run (rows == 0: the end)
    auto deal = [&](AttnItem& it) {
      it.rows = 0;
      while (left > 0) {
        if (x >= Hk * count) {  // the next sequence with rows
          if (++b >= B) return;
          if (b >= win + 32) {
            win = b;
            ws = SeqRows{};
            if (b + lane < B) seq_rows(p.rows, c.kv_len, cap, b + lane, ws);
          }
          sq.L = __shfl_sync(0xffffffffu, ws.L, b - win);
          sq.n = __shfl_sync(0xffffffffu, ws.n, b - win);
          sq.first = __shfl_sync(0xffffffffu, ws.first, b - win);
          R = sq.n * G;
          count = item_count(R);
          x = 0;
          if (off > 0 && count > 0) {  // (only until the first item is located)
            const long long hu = head_units(p, sq.L, sq.n, G);
            x = static_cast<int>(min(quick_div(off, hu), static_cast<long long>(Hk))) * count;
            off -= x / count * hu;
          }
          continue;
        }
        const int h = x / count, row0 = (x - h * count) * kAtItemRows;
        ++x;
        const int rows = min(kAtItemRows, R - row0);
        const ItemRange rg = item_range(p, sq.L, sq.n, row0, rows);
        const int nt = tile_count(rg), u = kAtItemUnits + nt;
        if (off >= u) {  // (only while the first item is being located)
          off -= u;
          continue;
        }
        // this run's units of the item, and the tiles among them
        const int o = static_cast<int>(off);
        const int take = static_cast<int>(min(static_cast<long long>(u - o), left));
        off = 0;
        left -= take;
        const int t_lo = max(0, o - kAtItemUnits), t_hi = max(0, o + take - kAtItemUnits);
        if (nt > 0 ? t_hi <= t_lo : o > 0) continue;
        it.b = b;
        it.h = h;
        it.row0 = row0;
        it.rows = rows;
        it.L = sq.L;
        it.n = sq.n;
        it.first = sq.first;
        it.t0 = first_tile(rg) + t_lo;
        it.nt = t_hi - t_lo;
        it.slot = t_lo == 0 && t_hi == nt ? -1 : 2 * static_cast<int>(blockIdx.x) + (t_lo == 0);
        it.load0 = loads;
        it.lo = rg.lo;
        it.hi = rg.hi;
        it.full0 = (rg.flo + kAtTile - 1) / kAtTile;
        it.full1 = max(it.full0, rg.fhi / kAtTile);
        it.fix0 = fixes;
        loads += 2 * it.nt;
        fixes += it.partials_before(it.t0 + it.nt);
        if (lane == 0 && t_lo == 0 && t_hi < nt)
          p.join[blockIdx.x] =
              AttnJoin{h, row0, rows, sq.first,
                       1 + static_cast<int>(quick_div(nt - t_hi + quota - 1, quota)), 0};
        return;
      }
    };
    auto announce = [&](const AttnItem& it) {
      const int d = items % kAtDescs;
      if (!wait(kBarItemFree + d, (items / kAtDescs) ^ 1)) return false;
      if (lane == 0) {
        s_items[d] = it;
        mbar_arrive(bar(kBarItem + d));
      }
      ++items;
      return true;
    };
    AttnItem now, it;
    now.rows = 0;
    int ids_now = -1;
    while (true) {
      if (is_k) {
        deal(it);
        live = announce(it);
      } else {
        live = fetch(it);
      }
      if (!live) break;
      const int ids = it.rows > 0 ? fetch_ids(it, first_window(it)) : -1;
      if (now.rows > 0) live = load_item(now, ids_now);
      if (!live || it.rows == 0) break;
      now = it;
      ids_now = ids;
    }
    if (*s_abort && last >= 0)  // let the copies in flight land
      drain_wait(bar(kBarFull + lane), (last / kStages) & 1);
  } else if (wi == 11) {
    // ------------------------------------------------------------------ unseen values
    // In a tile that some row of the item does not see in full: the values outside the item's
    // range become zeros, and so do those that only some rows see and that have an element that
    // is not finite; the latter are noted. Such tiles are an item's first and last, so this warp
    // waits while all the others pass: 2^23 tiles of some 4000 clocks at most (kv_len <= 2^30),
    // 2^35 clocks. (A pipeline that stalls ends it sooner, through the other warps' flag.)
    constexpr std::integral_constant<int, 64> kItemLong{};
    AttnItem it;
    bool live = true;
    while (live && fetch_rounds(kItemLong, it) && it.rows > 0) {
      const int look = look_ahead(it.rows, it.nt);
      const ItemRange rg = item_range(p, it.L, it.n, it.row0, it.rows);
      int fix = it.fix0;
      for (int j = 0; j < it.nt && live; ++j) {
        if (!it.partial(it.t0 + j)) continue;
        const int g = it.load0 + load_of_v(j, look, it.nt);
        // (first that the copy was issued: before that the stage may still hold an earlier load,
        // whose phase a wait by parity could take for this one's)
        live = wait_rounds(kItemLong, kBarToFix + fix % kAtFixRing, fix / kAtFixRing) &&
               wait(kBarFull + g % kStages, g / kStages);
        if (!live) break;
#pragma unroll 1
        for (int y = 0; y < 4; ++y) {
          const int r = 32 * y + lane, x = (it.t0 + j) * kAtTile + r;
          uint8_t* v = sm + Sm::kKv + (g % kStages) * Sm::kStage + r * 128;
          const bool outside = x < it.lo || x >= it.hi;
          uint32_t odd = 0;
          if (!outside && (x < rg.flo || x >= rg.fhi)) {
#pragma unroll
            for (int q = 0; q < DP / 8; ++q) {
              const uint4 e = *reinterpret_cast<const uint4*>(
                  v + (q >> 3) * (kAtTile * 128) + (((q & 7) ^ (r & 7)) << 4));
              const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
              // an element is not finite when its exponent is all ones: adding one to the
              // exponent's last place then carries into the cleared sign bit
              constexpr uint32_t kMag = 0x7fff7fffu, kOne = kBf ? 0x00800080u : 0x04000400u;
#pragma unroll
              for (int z = 0; z < 4; ++z) odd |= ((ew[z] & kMag) + kOne) & 0x80008000u;
            }
          }
          if (outside || odd) {
#pragma unroll
            for (int q = 0; q < DP / 8; ++q)
              *reinterpret_cast<uint4*>(v + (q >> 3) * (kAtTile * 128) + ((q & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          const uint32_t word = __ballot_sync(0xffffffffu, odd != 0);
          if (lane == 0) s_nf[(fix % kAtFixRing) * 4 + y] = word;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarFix + fix % kAtFixRing));
        ++fix;
      }
    }
  } else if (wi == 9) {
    // ------------------------------------------------------------------ MMA issuer
    {
      constexpr uint32_t qk_desc = at_idesc(kAtTile, kBf, false);
      constexpr uint32_t pv_desc = at_idesc(DP, kBf, true);
      uint32_t nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;  // phases used of kBarQ, kBarP
      int loads = 0;
      bool live = true;
      AttnItem it;
      while (live && fetch(it)) {
        // (a shuffle from lane 0: known to be the same for all lanes)
        const int rows = __shfl_sync(0xffffffffu, it.rows, 0);
        const int nt = __shfl_sync(0xffffffffu, it.nt, 0);
        const int load0 = loads;
        loads += 2 * nt;
        if (rows == 0) break;
        if (nt == 0) continue;
        const bool dual = rows > kAtTile;
        const int flip = (items - 1) & 1;  // the group that takes tile 0 (see the groups)
        const int look = look_ahead(rows, nt);
        auto stage = [&](int idx) { return (load0 + idx) % kStages; };
        auto landed = [&](int idx) {
          return wait(kBarFull + stage(idx), (load0 + idx) / kStages);
        };
        // S_s = Q_s K_j^T
        auto qk = [&](int s, int j) {
          // (a descriptor's start address counts 16 bytes: a step of 16 dims is 2, the next 64
          // dims a tile's half on)
          const uint32_t t_s = uniform(tbase + s * 128);
          const uint64_t q0 = sw128_desc(uniform(sb + Sm::kQ + s * Sm::kStage));
          const uint64_t k0 =
              sw128_desc(uniform(sb + Sm::kKv + stage(load_of_k(j, look)) * Sm::kStage));
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const int at = (k >> 2) * (kAtTile * 8) + 2 * (k & 3);
            at_mma_ss(t_s, q0 + at, k0 + at, qk_desc, k != 0);
          }
          at_commit(bar(kBarS + s));
        };
        // O_s += P_s V_j
        auto pv = [&](int s, int j, bool first) {
          const uint32_t t_o = uniform(tbase + 256 + s * 128), t_p = uniform(tbase + s * 128);
          const uint64_t v0 =
              sw128_mn_desc(uniform(sb + Sm::kKv + stage(load_of_v(j, look, nt)) * Sm::kStage));
#pragma unroll
          for (int k = 0; k < kAtTile / 16; ++k)
            at_mma_ts(t_o, t_p + 8 * k,
                       v0 + 128 * k, pv_desc, !(first && k == 0));
        };
        auto free_stage = [&](int idx) { at_commit(bar(kBarEmpty + stage(idx))); };
        auto wait_q = [&](int s) {
          const uint32_t phase = s ? nq1++ : nq0++;
          return wait(kBarQ + s, phase);
        };
#pragma unroll 1
        for (int x = 0; x < (dual ? 2 : min(2, nt)) && live; ++x) {
          const int s = dual ? x : x ^ flip, j = dual ? 0 : x;
          live = wait_q(s) && landed(load_of_k(j, look));
          if (!live) break;
          tc_fence_after();
          qk(s, j);
          if (!dual || x == 1) free_stage(load_of_k(j, look));
        }
        for (int j = 0; j < nt && live; ++j) {
          live = landed(load_of_v(j, look, nt));
          if (live && it.partial(it.t0 + j)) {
            const int fix = it.fix0 + it.partials_before(it.t0 + j);
            live = wait(kBarFix + fix % kAtFixRing, fix / kAtFixRing);
          }
#pragma unroll 1
          for (int x = dual ? 0 : 1; x < 2 && live; ++x) {
            const int s = dual ? x : (j & 1) ^ flip;
            const uint32_t phase = s ? np1++ : np0++;
            live = wait(kBarP + s, phase);
            if (!live) break;
            tc_fence_after();
            pv(s, j, (dual ? j : j >> 1) % kSumTiles == 0);
            if (x == 1) free_stage(load_of_v(j, look, nt));
            const int jn = j + (dual ? 1 : 2);
            if (jn < nt) {
              live = landed(load_of_k(jn, look));
              if (!live) break;
              tc_fence_after();
              qk(s, jn);
              if (x == 1) free_stage(load_of_k(jn, look));
            } else {
              at_commit(bar(kBarO + s));
            }
          }
        }
      }
      if (*s_abort) {  // let the MMAs in flight finish
        at_commit(bar(kBarDrain));
        drain_wait(bar(kBarDrain), 0);
      }
    }
  } else if (wi < 8) {
    // ------------------------------------------------------------------ softmax groups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtGroupRegs));
    const int s = wi >> 2, w = wi & 3, r = 32 * w + lane;  // group, TMEM quarter, lane = row
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const uint32_t t_s = tbase + lanes + s * 128, t_o = tbase + lanes + 256 + s * 128;
    const uint32_t t_other = tbase + lanes + 256 + (s ^ 1) * 128;
    const float cl = p.scale_log2;
    uint32_t n_s = 0, n_o = 0, n_pair = 0;
    bool owed = false;        // the other group may still be reading this group's O
    uint32_t owed_phase = 0;
    AttnItem it, next;
    int rel = 0, rel_next = 0;  // items of up to 128 rows: this group takes tiles rel, rel + 2, ..

    auto my_tiles = [&](const AttnItem& a, int first) {
      return a.rows > kAtTile ? a.nt : (a.nt - first + 1) / 2;
    };
    auto my_rows = [&](const AttnItem& a) {
      return a.rows > kAtTile ? (s ? a.rows - kAtTile : kAtTile) : a.rows;
    };
    auto my_row0 = [&](const AttnItem& a) {
      return a.row0 + (a.rows > kAtTile ? s * kAtTile : 0);
    };
    // Q_s of an item into shared memory (128-byte swizzle, K-major); elements past head_dim and
    // rows past the item's are zeros: their scores are never used, but the tensor cores' products
    // of zeros draw less power, which sets the clock of a long run of calls
    int q_rows = kAtTile;  // rows of Q_s that may hold something (at first whatever was there)
    auto load_q = [&](const AttnItem& a) {
      if (my_tiles(a, rel_next) == 0) return;
      constexpr int kCh = DP / 8;
      const int rows = my_rows(a), row0 = my_row0(a);
      uint8_t* dst = sm + Sm::kQ + s * Sm::kStage;
      const T* q = static_cast<const T*>(p.q.p);
      const int ch = r % kCh, bytes = 8 * ch < D ? 16 : 0;
#pragma unroll 4
      for (int row = r / kCh; row < rows; row += kAtTile / kCh) {
        const int i = p.by_group.div(row0 + row), h = a.h * G + row0 + row - i * G;
        const T* src = q + token_offset(p.q, p, a.b, a.first, i) + h * p.q.head_stride +
                       (bytes ? 8 * ch : 0);
        copy16_async(smem_u32(dst) + (ch >> 3) * (kAtTile * 128) + row * 128 +
                         (((ch & 7) ^ (row & 7)) << 4),
                     src, bytes);
      }
      for (int row = rows + r / kCh; row < q_rows; row += kAtTile / kCh)
        *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kAtTile * 128) + row * 128 +
                                  ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
      q_rows = rows;
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQ + s));
    };

    // Per turn: the next item's queries, the results of the item before it (whose last products
    // ran meanwhile), then the next item's tiles.
    bool live = true, dual = false, active = false, real = false;
    int cnt = 0, row0 = 0, token = 0, head = 0;
    float m = -INFINITY, l = 0.f;
    float m_sum = -INFINITY;  // the maximum that the sum of earlier tiles is relative to
    it.rows = 0;
    // The row's O joins the sum of earlier tiles (first: there is none yet), which goes back to
    // tensor memory (to_tmem) or to the workspace.
    auto move_sum = [&](bool to_tmem, bool first) {
      const float f = m_sum == -INFINITY ? 0.f : ex2((m_sum - m) * cl);
      at_move_sum<DP>(t_o,
                      p.sums + (2 * static_cast<int64_t>(blockIdx.x) + s) * DP * p.sum_rows + r,
                      p.sum_rows, f, real && !first, real && !to_tmem, to_tmem);
      m_sum = m;
    };
    while (true) {
      live = fetch(next);
      if (!live) break;
      rel_next = s ^ ((items - 1) & 1);  // short items alternate between the groups
      if (next.rows > 0) load_q(next);
      if (it.rows > 0) {
        if (cnt > 0) {
          live = wait(kBarO + s, n_o);
          if (!live) break;
          ++n_o;
          tc_fence_after();
          if (cnt > kSumTiles && active) {  // O of all tiles
            move_sum(true, false);
            tc_fence_before();
          }
        }
        // both groups hold the same rows: the one of tile 0 takes the other's part in
        const bool pair = !dual && it.nt > 1;
        float a0 = 1.f, a1 = 0.f;
        if (pair) {
          if (rel == 1) {
            s_ml[r] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarMl));
          } else {
            live = wait(kBarMl, n_pair);
            if (!live) break;
            tc_fence_after();
            const float2 o = s_ml[r];
            const float mm = fmaxf(m, o.x);
            a0 = m == -INFINITY ? 0.f : ex2((m - mm) * cl);
            a1 = o.x == -INFINITY ? 0.f : ex2((o.x - mm) * cl);
            l = l * a0 + o.y * a1;
            m = mm;
          }
        }
        if (active && (dual || rel == 0)) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int row = it.first + token;
          T* out = static_cast<T*>(p.out.p) + token_offset(p.out, p, it.b, it.first, token) +
                   head * p.out.head_stride;
          const int64_t pr = static_cast<int64_t>(it.slot) * p.part_rows + (row0 - it.row0) + r;
          // (rolled: code that runs once an item should not push the tile's out of the
          // instruction cache)
#pragma unroll 1
          for (int q = 0; q < DP; q += 32) {
            float o[32];
            if (cnt > 0) {
              tmem_ld32(t_o + q, o);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = 0.f;
            }
            if (pair) {
              float o1[32];
              tmem_ld32(t_other + q, o1);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = o[y] * a0 + o1[y] * a1;
            }
            if (!real) {
              // (no row of the item: the loads above still need the whole warp)
            } else if (it.slot >= 0) {
#pragma unroll
              for (int y = 0; y < 32; y += 4)
                *reinterpret_cast<float4*>(p.part_o + pr * DP + q + y) =
                    make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
            } else {
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] *= inv;
              if (!kBf) {
                float top = 0.f;
#pragma unroll
                for (int y = 0; y < 32; ++y) top = fmaxf(top, fabsf(o[y]));
                if (top > kF16Max) {
#pragma unroll
                  for (int y = 0; y < 32; ++y) o[y] = f16_range(o[y]);
                }
              }
#pragma unroll
              for (int y = 0; y < 32; y += 8) {
                if (q + y < D) {
                  uint4 v;
                  v.x = Half16<T>::down(o[y], o[y + 1]);
                  v.y = Half16<T>::down(o[y + 2], o[y + 3]);
                  v.z = Half16<T>::down(o[y + 4], o[y + 5]);
                  v.w = Half16<T>::down(o[y + 6], o[y + 7]);
                  *reinterpret_cast<uint4*>(out + q + y) = v;
                }
              }
            }
          }
          if (real) {
            if (it.slot >= 0)
              p.part_ml[pr] = make_float2(m, l);
            else if (p.lse)
              p.lse[static_cast<int64_t>(row) * p.Hq + head] =
                  l == 0.f ? -INFINITY : (m * cl - kShift + log2f(l)) * 0.69314718055994531f;
          }
        }
        if (pair) {
          if (rel == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarJoined));
          } else {
            owed = true;
            owed_phase = n_pair;
          }
          ++n_pair;
        }
      }
      if (next.rows == 0) break;
      it = next;
      rel = rel_next;
      dual = it.rows > kAtTile;
      cnt = my_tiles(it, rel);
      row0 = my_row0(it);
      const int rows = my_rows(it);
      active = 32 * w < rows;  // some row of this warp is real
      real = r < rows;
      const int mine_row = row0 + min(r, rows - 1);
      token = p.by_group.div(mine_row);
      head = it.h * G + mine_row - token * G;
      int lo, hi;
      seen_range(it.L, it.n, token, p.causal, p.window, lo, hi);
      m = m_sum = -INFINITY;
      l = 0.f;
      bool poison = false, large = false;

#pragma unroll 1
      for (int k0 = 0; k0 < cnt && live; k0 += kSumTiles) {
        if (k0 > 0) {  // (scores that are ready: the products before them are done)
          live = wait(kBarS + s, n_s);
          if (!live) break;
          tc_fence_after();
          if (active) move_sum(false, k0 == kSumTiles);
        }
        const int k1 = min(cnt, k0 + kSumTiles);
        for (int k = k0; k < k1 && live; ++k) {
          const int j = dual ? k : 2 * k + rel;
          const int x0 = (it.t0 + j) * kAtTile;
          const bool partial = it.partial(it.t0 + j);
          live = wait(kBarS + s, n_s);
          if (!live) break;
          ++n_s;
          tc_fence_after();
          if (active) {
            float z[kAtTile];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, z + 32 * q);
            tmem_ld_wait();
            if (partial) {
              // the row's seen positions as bits, 32 at a time
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int at = x0 + 32 * y;
                const int a = min(max(lo - at, 0), 32), e = min(max(hi - at, 0), 32);
                const uint32_t seen = static_cast<uint32_t>((1ull << e) - (1ull << min(a, e)));
#pragma unroll
                for (int q = 0; q < 32; ++q)
                  if (!((seen >> q) & 1)) z[32 * y + q] = -INFINITY;
              }
            }
            float mx[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) mx[y] = max_nan(z[2 * y], z[2 * y + 1]);
#pragma unroll
            for (int q = 8; q < kAtTile; q += 8) {
#pragma unroll
              for (int y = 0; y < 4; ++y) mx[y] = max3_nan(mx[y], z[q + 2 * y], z[q + 2 * y + 1]);
            }
            const float mt = max_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3]);
            if (!(mt < INFINITY)) poison = true;  // a NaN or an infinity among the seen scores
            // the kept maximum moves when the tile's exceeds it by kRescale binary orders
            const bool move = real && mt > m && !((mt - m) * cl <= kRescale);
            if (__any_sync(0xffffffffu, move)) {
              const float mn = move ? mt : m;
              const float f = move ? ex2((m - mn) * cl) : 1.f;  // m == -inf: 0
              l *= f;
              m = mn;
              large = __any_sync(0xffffffffu, real && m != -INFINITY &&
                                                  fabsf(m) * cl > kAtLargeScore);
              if (k > k0) {
#pragma unroll 1
                for (int q = 0; q < DP; q += 32) {
                  float o[32];
                  tmem_ld32(t_o + q, o);
                  tmem_ld_wait();
                  uint32_t ow[32];
#pragma unroll
                  for (int y = 0; y < 32; ++y) ow[y] = __float_as_uint(o[y] * f);
                  tmem_st32(t_o + q, ow);
                }
              }
            }
            // p = 2^(c z - c m), two at a time; 0 in rows past the item's. The rounding of c m puts
            // all of a row's weights off by half a place of c m (for scores of 10^8, by up to four
            // binary orders), so large scores are reduced to z - m first.
            const bool seen_any = m != -INFINITY;
            if (large) {
              const float minus_m = seen_any ? -m : 0.f;
              const uint64_t m2 = pk2(minus_m, minus_m);
#pragma unroll
              for (int q = 0; q < kAtTile; q += 2)
                upk2(add2(pk2(z[q], z[q + 1]), m2), z[q], z[q + 1]);
            }
            const float base = !real ? -INFINITY : large || !seen_any ? kShift : kShift - m * cl;
            const float factor = real ? cl : 0.f;
            const uint64_t c2 = pk2(factor, factor), base2 = pk2(base, base);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < kAtTile; q += 64) {
              uint32_t pw[32];
#pragma unroll
              for (int y = 0; y < 32; ++y) {
                float e0, e1;
                upk2(fma2(pk2(z[q + 2 * y], z[q + 2 * y + 1]), c2, base2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum[y & 3] = add2(sum[y & 3], pk2(e0, e1));
                pw[y] = Half16<T>::down(e0, e1);
              }
              tmem_st32(t_s + q / 2, pw);
            }
            {
              float s0, s1;
              upk2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
              l += s0 + s1;
            }
            tmem_st_wait();
          }
          if (owed) {  // before this group's O may be written again
            live = wait(kBarJoined, owed_phase);
            if (!live) break;
            owed = false;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarP + s));
          // positions in a page out of range, or whose value was not finite and is now zero
          uint4 hit = *reinterpret_cast<const uint4*>(
              s_bad + ((it.load0 / 2 + j) % kAtBadRing) * 4);
          if (partial) {
            const int fix = it.fix0 + it.partials_before(it.t0 + j);
            live = wait(kBarFix + fix % kAtFixRing, fix / kAtFixRing);
            if (!live) break;
            const uint4 nf = *reinterpret_cast<const uint4*>(s_nf + (fix % kAtFixRing) * 4);
            hit.x |= nf.x;
            hit.y |= nf.y;
            hit.z |= nf.z;
            hit.w |= nf.w;
          }
          if (hit.x | hit.y | hit.z | hit.w) {
#pragma unroll 1
            for (int q = max(lo - x0, 0); q < min(hi - x0, kAtTile); ++q) {
              const uint32_t word = q < 64 ? (q < 32 ? hit.x : hit.y) : (q < 96 ? hit.z : hit.w);
              if ((word >> (q & 31)) & 1) poison = true;
            }
          }
        }
      }
      if (!live) break;
      if (poison) l = NAN;

    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    const int gave_up = *s_abort;
    p.join[blockIdx.x].gave_up = gave_up;
    if (gave_up) atomicAdd(&g_pipeline_timeouts, 1ull);
  }
  if (wi == 9) tmem_free_all(*s_tmem);
}

// ------------------------------------------------------------------------ joining pieces

// The items that a border cut, and the sequences' status. CTA (x, y): item of CTA x of the
// attention kernel, a warp per row. With m_i, l_i and O_i of the pieces and M = max m_i:
// out = sum 2^(c (m_i - M)) O_i / sum 2^(c (m_i - M)) l_i.
constexpr int kJoinWarps = 8;
template <typename T, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_kernel(const AttnParams p) {
  constexpr int kPer = DP / 32;
  constexpr float kShift = at_shift<T>();
  const float cl = p.scale_log2;
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const dspark_kv_cache_t& c = p.cache;
  const int G = p.Hq / c.n_heads;
  const int b0 = (blockIdx.y * gridDim.x + blockIdx.x) * kJoinWarps + warp;
  if (p.status && b0 < p.rows.B) {
    const int warps = gridDim.x * gridDim.y * kJoinWarps;
    const int64_t cap = static_cast<int64_t>(c.max_pages) << p.page_log2;
    int gave_up = 0;  // a CTA that gave up leaves any sequence's rows incomplete
#pragma unroll 4
    for (int x = lane; x < gridDim.x; x += 32) gave_up |= p.join[x].gave_up;
    gave_up = __any_sync(0xffffffffu, gave_up) ? DSPARK_SEQ_TIMEOUT : 0;
    for (int b = b0; b < p.rows.B; b += warps) {
      SeqRows s;
      const bool ok = seq_rows(p.rows, c.kv_len, cap, b, s);
      bool bad = false;
      if (ok && s.n > 0) {
        int lo, hi, x;
        seen_range(s.L, s.n, 0, p.causal, p.window, lo, x);
        seen_range(s.L, s.n, s.n - 1, p.causal, p.window, x, hi);
        if (hi > lo)
          for (int g = (lo >> p.page_log2) + lane; g <= (hi - 1) >> p.page_log2; g += 32) {
            const int page = c.page_table[b * c.ld_table + g];
            bad |= page < 0 || page >= c.n_pages;
          }
      }
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0)
        p.status[b] = gave_up | (!ok ? DSPARK_SEQ_BAD_PARAM : bad ? DSPARK_SEQ_BAD_PAGE : 0);
    }
  }
  const AttnJoin jn = p.join[blockIdx.x];
  if (jn.pieces == 0) return;
  const int x = blockIdx.x;
  for (int r = blockIdx.y * kJoinWarps + warp; r < jn.rows; r += gridDim.y * kJoinWarps) {
    float m = -INFINITY;
    int gave_up = 0;
    for (int i = lane; i < jn.pieces; i += 32) {
      const int slot = i == 0 ? 2 * x + 1 : 2 * (x + i);
      m = fmaxf(m, p.part_ml[static_cast<int64_t>(slot) * p.part_rows + r].x);
      gave_up |= p.join[x + i].gave_up;
    }
    m = warp_max_nan(m);
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < jn.pieces; ++i) {
      const int slot = i == 0 ? 2 * x + 1 : 2 * (x + i);
      const int64_t pr = static_cast<int64_t>(slot) * p.part_rows + r;
      const float2 ml = p.part_ml[pr];
      const float a = ex2((ml.x - mu) * cl);  // -inf: 0
      l += ml.y * a;
#pragma unroll
      for (int k = 0; k < kPer; ++k) o[k] += p.part_o[pr * DP + lane * kPer + k] * a;
    }
    if (__any_sync(0xffffffffu, gave_up)) l = NAN;  // a piece is missing
    const int token = (jn.row0 + r) / G, g = jn.row0 + r - token * G, row = jn.first + token;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(p.out.p) + row_offset(p.out, p.rows, row) +
             (jn.h * G + g) * p.out.head_stride;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      o[k] *= inv;
      if (std::is_same<T, __half>::value) o[k] = f16_range(o[k]);
    }
    if (lane * kPer < c.head_dim) {
      if (kPer == 4)
        *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(
            Half16<T>::down(o[0], o[1]), Half16<T>::down(o[kPer - 2], o[kPer - 1]));
      else
        *reinterpret_cast<uint32_t*>(out + 2 * lane) = Half16<T>::down(o[0], o[1]);
    }
    if (p.lse && lane == 0)
      p.lse[static_cast<int64_t>(row) * p.Hq + jn.h * G + g] =
          l == 0.f ? -INFINITY : (mu * cl - kShift + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace dspark
