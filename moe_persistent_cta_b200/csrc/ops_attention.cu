// ops_attention.cu -- attention of one query token per batch entry over the
// paged cache, with the pages of a prefix that a group of entries shares read
// once for as many of them as two tiles of rows hold.
//
// For entry b and query head h, with seen = positions[b] + 1:
//   o = sum_t exp(s_t - lse) v_t,  s_t = scale q . k_t,  t < seen,
// the sum taken over tiles of 128 tokens with a running reference m and sum l:
//   P = 2^(s log2(e) - m), O = O 2^(m_old - m) + P V, l likewise.
// Any m not far below the largest score serves, so O is only rescaled when a
// row's largest score has grown by more than 8 (a factor of 256).
//
// Work.  Query rows are (entry, query head of one KV head).  Prefix units: one
// KV head's rows of up to 2 x MB entries of a group (MB = floor(128 / G), G
// query heads per KV head) against the group's prefix.  Own units: one entry's
// rows against its own tokens; the entries of a chunk (MB consecutive ones)
// share one tile of query rows, and one after another meet their tokens with
// the other entries' rows masked, so that a block works through many short
// remainders without a break.  The tiles of all units form one line, and every
// block takes an equal stretch of it, so a long prefix is split over many blocks.
// (A tile costs about the same whatever its rows: of 256 entries on 32768 tokens,
// 5300 cycles with two tiles of rows and 5000 with one entry's.)  Each block finds
// its stretch from the device arrays: the host needs no lengths, and a captured
// graph replays with new ones.  A block's share of a unit leaves partial results
// (O, m, l); a second launch adds them up.  A group of more than 2 x MB entries is
// several units, and its prefix is read as often.
//
// One block: a TMA warp streams K and V tiles, two warps issue tcgen05 MMAs,
// and two groups of four warps hold a softmax row per thread.  S = Q K^T and O
// live in tensor memory, two of each ("streams"), each with an MMA warp of its
// own.  A tile's tokens go in two halves: while the softmax has one half of S, the
// other's P (which goes back to tensor memory over S and is the A operand of P V)
// is multiplied and replaced by S of the stream's next tile.  With more than 128
// rows the streams are the two tiles of rows, and each K and V tile serves both;
// with fewer they are alternate tiles of tokens of the same rows, two partial
// results.
//
// Sums, maxima and O are 32-bit.  P alone is rounded to the cache's type, since
// both operands of an MMA are of one 16-bit type and V is the cache's: each weight
// is off by at most half a step, a row by at most half a step of its weighted |v|
// (against 64 bits, bf16: 0.0023 of the result's norm, with P in 32 bits 0.0017, of
// which the output's own rounding is 0.0017).  P in two parts would double P V.
//
// What bounds it: 256 entries on 32768 shared and up to 300 own tokens each (16
// query heads of 128, 4 KV heads, bf16) take 128 us (124 to 132, by the clocks), 0.54
// PFLOP/s, the tensor pipe a third busy.  The MMAs alone, without the softmax, take
// about nine tenths of that (119 of 132): with 64 columns of S each Q K^T reads
// three times its share from shared memory (Q has no room in tensor memory beside S
// and O), and with 128 S cannot be replaced by halves (135).  One MMA warp that also
// passed over the other stream's tiles: 138.  Few rows: 8 entries on 8192 tokens
// 17.7 us, of which 5 find the block's share of the work and 5 add up the partial
// results.
//
// Values that are no numbers.  A masked weight is 0, and 0 x infinity is NaN:
// V's rows outside a unit's tokens are cleared in shared memory, but a row can
// also meet tokens that only other rows of its tile see.  A row whose sum is
// not finite is therefore computed once more, from its own tokens alone.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "ops_common.cuh"
#include "ops_step.h"

namespace mk {
namespace ops {
namespace {

constexpr int kRows = 128;           // query rows of a stream
constexpr int kTile = 128;           // tokens of a K or V tile
constexpr int kGroupThreads = 128;   // a softmax group: one row per thread
constexpr int kTmaWarp = 8, kMmaWarp = 9;   // one MMA warp per stream
constexpr int kThreads = 352;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxItems = 32;        // of one pass of a block over its stretch; a power of two
constexpr int kMaxBatch = 4096;
constexpr int kMaxGroup = 64;        // query heads per KV head
constexpr float kRescale = 8.0f;     // log2 of the growth that O may lag behind
constexpr uint32_t kFull = 0xffffffffu;
// Limit of a wait: about half a second at any clock.  (As an argument of the
// launch it cost 1 % of a long call, by the compiler's order of things alone.)
constexpr int kWaitCycles = 1 << 30;

// What the joining launch needs of an entry, written by the last block: the places
// in the line of its unit's first prefix tile and of its first own tile for KV
// head 0, how far the next head's are, and how many tiles there are.
struct __align__(16) Entry {
  int prefix_at, prefix_tiles;
  int dual;                          // two tiles of rows meet each prefix tile
  int own_at, own_tiles, own_stride;
  int lead;                          // first entry of its prefix unit; -1: the entry is in no group
  int group;
};
struct Line {                        // the line of tiles and how blocks share it
  int total, blocks, each, extra;    // block i has `each` tiles, the first `extra` blocks one more
  __device__ __forceinline__ Line(int all, int grid) {
    total = all;
    blocks = max(1, min(grid, all));
    each = all / blocks;
    extra = all - each * blocks;
  }
  __device__ __forceinline__ int start(int i) const { return i * each + min(i, extra); }
  __device__ __forceinline__ int block_of(int x) const {
    const int cut = extra * (each + 1);
    return x < cut ? x / (each + 1) : extra + (x - cut) / each;
  }
};

struct AttnParams {
  int B, n_groups, max_pages, n_pages, Hq, Hkv, G, MB;   // MB: entries of a stream's rows
  int grid;
  float c;                           // scale x log2(e)
  const int32_t *page_table, *positions, *group_start, *prefix_lens;
  // partial results: [slot][stream][row] of split units, [kind][stream][b][hq]
  // of whole ones (prefix, then own tokens)
  float* part;
  float2* part_ml;
  Entry* entries;                    // [B]
  int* line_total;                   // the line's length
  int* gave_up;                      // [block]: a wait ran out, and its shares are not complete
  int stall;                         // block whose tiles never arrive (the self-test), or -1
  int n_slots, slot_rows;            // split shares, and the rows that one can hold
  const void *q, *k_pool, *v_pool;   // for rows computed alone
  long long q_stride;
  void* out;
  float* lse;
  StepSink sink;
  int32_t* status;
};

// Row of `part` that holds a share of a whole unit.
__device__ __forceinline__ size_t whole_row(const AttnParams& p, int kind, int stream, int b, int hq) {
  return (size_t)p.n_slots * 2 * p.slot_rows + (((size_t)kind * 2 + stream) * p.B + b) * p.Hq + hq;
}

// A block's share of a unit.  Consecutive items whose rows share O make a run.
struct Item {
  int head;           // KV head
  int b0, nmem;       // entries b0 .. b0 + nmem - 1 hold the rows
  int row;            // page-table row of the keys; with `own`, the one entry that meets them
  int lo, hi;         // tokens lo .. hi - 1 belong to the unit; its first tile starts at lo's page
  int t0, t1;         // tiles
  int j0, steps;      // steps of the run before the item, and of the whole run
  short slot;         // partial: split slot, or -1 whole
  bool dual;          // both streams share each tile
  bool own;
};

template <int HD>
struct Layout {
  static constexpr int kChunks = HD / 64;
  static constexpr int kTileBytes = kTile * HD * 2;
  static constexpr int kStages = HD == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kDyn = kRing + kStages * kTileBytes;
};

// ------------------------------------------------------------------- PTX --
__device__ __forceinline__ uint32_t saddr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const void* map, int x, int y, int z,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const void* map, int x, int y, int z, int w,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Pairs of floats in one 64-bit register: one instruction for two.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest of three; NaN if any is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The following are run by a whole warp and issued by one elected lane: in
// code that only one lane reaches, the operands would have to be moved to
// uniform registers before each instruction (measured: 85 cycles an MMA).
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem], four steps of 16 along K: 32 bytes of a row each
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], four steps of 16 along K: 8 columns of A, 16
// rows of 128 bytes of B each
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
#define MK_R4(r, i) "=r"((r)[i]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3])
#define MK_I4(r, i) "r"((r)[i]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3])
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MK_R4(r, 0), MK_R4(r, 4), MK_R4(r, 8), MK_R4(r, 12), MK_R4(r, 16), MK_R4(r, 20),
        MK_R4(r, 24), MK_R4(r, 28)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::MK_I4(r, 0),
      MK_I4(r, 4), MK_I4(r, 8), MK_I4(r, 12), MK_I4(r, 16), MK_I4(r, 20), MK_I4(r, 24),
      MK_I4(r, 28), "r"(addr)
      : "memory");
}
// 16 columns
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::MK_I4(r, 0), MK_I4(r, 4), MK_I4(r, 8), MK_I4(r, 12), "r"(addr)
      : "memory");
}
#undef MK_R4
#undef MK_I4
#define MK_W4(r, i) "+r"((r)[i]), "+r"((r)[(i) + 1]), "+r"((r)[(i) + 2]), "+r"((r)[(i) + 3])
#define MK_W16(r, i) MK_W4(r, i), MK_W4(r, (i) + 4), MK_W4(r, (i) + 8), MK_W4(r, (i) + 12)
// Waits for loads; tied to their registers, so that no use of these moves up.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : MK_W16(r, 0), MK_W16(r, 16)::"memory");
}
__device__ __forceinline__ void tmem_wait_ld64(uint32_t* r) {
  tmem_wait_ld32(r);
  asm volatile("" : MK_W16(r, 32), MK_W16(r, 48)::"memory");
}
#undef MK_W4
#undef MK_W16
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand descriptors, 128-byte swizzle.  Along K (Q and K
// tiles: rows of 64 columns): groups of 8 rows 1024 bytes apart.  Along N (V
// tiles: tokens are K, 64 columns of N per row): groups of 8 tokens 1024 bytes
// apart, the next 64 columns a chunk apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t lead_bytes) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead_bytes >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[4], p_ready[4];    // per stream, of the two halves of a tile's tokens
  uint64_t pv_done[2];               // P V of the first half of a stream's last step
  uint64_t o_full[2], o_free[2];
};

struct Block {
  Bars bars;
  Item items[kMaxItems];             // unit u in place u mod kMaxItems
  int scan[kWarps][4];
  unsigned first, last;              // units of the block's stretch
  int win_lo, win_hi;                // stretch of this pass
  int n_steps;
  uint32_t tmem;
  int abort;
};

// With the tiles at 1024-byte alignment, all of a block's shared memory.
static_assert(((sizeof(Block) + 1023) & ~size_t(1023)) + Layout<128>::kDyn <= 227 * 1024 &&
                  ((sizeof(Block) + 1023) & ~size_t(1023)) + Layout<64>::kDyn <= 227 * 1024,
              "a block's shared memory does not fit");

// Bounded wait: false once any wait of the block has run out.
__device__ __forceinline__ bool wait(Block& s, uint32_t bar, uint32_t parity, const AttnParams& p) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*(volatile int*)&s.abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *(volatile int*)&s.abort = 1;
      report(p.status, MK_ERR_TIMEOUT, MK_OP_PREFIX_ATTENTION, (int)blockIdx.x, 0, 0);
      return false;
    }
  }
  return true;
}

// ----------------------------------------------------------------- steps --
// The block's steps, in order: one S tile each.  Step n belongs to stream
// n & 1.  An item with two tiles of rows has two steps per tile.  Tiles are
// loaded in the order the MMA warp first needs them: K of steps 0 and 1, then
// for each n V of step n and K of step n + 2.
struct Walk {
  const Item* items;
  int n, base;                       // items, unit of the first
  int i = 0, j = 0, run = 0;         // item, step of it, run
  int count = 0, j0 = 0, total = 0;  // the item's steps, those of the run before it and in all
  int tile = 0, tile1 = -1, tile2 = -1;   // number of the step's tile, of those one and two steps before
  bool dual = false;
  __device__ __forceinline__ Walk(const Item* it, int n_items, int first) : items(it), n(n_items), base(first) {
    enter();
  }
  __device__ __forceinline__ void enter() {
    if (i >= n) return;
    const Item& q = at();
    dual = q.dual;
    count = (q.t1 - q.t0) << (dual ? 1 : 0);
    j0 = q.j0;
    total = q.steps;
  }
  __device__ __forceinline__ const Item& at() const { return items[(base + i) % kMaxItems]; }
  __device__ __forceinline__ bool done() const { return i >= n; }
  // Places in the ring of a step that loads: K lies behind the V tiles of the
  // steps up to the last but one, V behind the K tiles up to the next step's.
  __device__ __forceinline__ uint32_t k_place() const { return tile + tile2 + 1; }
  __device__ __forceinline__ uint32_t v_place(bool another) const { return 2 * tile + 1 + (!dual && another ? 1 : 0); }
  __device__ __forceinline__ bool loads() const { return !(dual && (j & 1)); }   // a new tile
  __device__ __forceinline__ bool first() const { return j0 + j == 0; }          // of the run
  __device__ __forceinline__ bool last() const { return j0 + j == total - 1; }
  __device__ __forceinline__ bool first_of_stream() const { return j0 + j < 2; }
  __device__ __forceinline__ bool last_of_stream() const { return j0 + j >= total - 2; }
  __device__ __forceinline__ int q_slot(int stream) const { return dual ? stream : (run & 1); }
  __device__ __forceinline__ void next() {
    if (last()) ++run;
    tile2 = tile1;
    tile1 = tile;
    if (++j == count) {
      j = 0;
      ++i;
      enter();
      ++tile;
    } else if (loads()) {
      ++tile;
    }
  }
};

// ------------------------------------------------------------------ list --
// Sums of four numbers over lower threads; *total gets those of all.
__device__ void scan4(Block& s, const int* v, int* below, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    inc[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kFull, inc[i], o);
      if (lane >= o) inc[i] += up;
    }
  }
  if (lane == 31) *reinterpret_cast<int4*>(s.scan[warp]) = make_int4(inc[0], inc[1], inc[2], inc[3]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) total[i] = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int4 t = *reinterpret_cast<const int4*>(s.scan[w]);
    if (w == warp) {
#pragma unroll
      for (int i = 0; i < 4; ++i) below[i] = total[i] + inc[i] - v[i];
    }
    total[0] += t.x;
    total[1] += t.y;
    total[2] += t.z;
    total[3] += t.w;
  }
}

// Words of shared memory that list_items needs.
__host__ __device__ constexpr int list_words(int batch, int groups) {
  return 2 * (groups + 1) + 6 * batch + 2;
}
static_assert(list_words(kMaxBatch, kMaxBatch) * 4 <= Layout<128>::kDyn - Layout<128>::kRing &&
                  list_words(kMaxBatch, kMaxBatch) * 4 <= Layout<64>::kDyn - Layout<64>::kRing,
              "the list's scratch does not fit the ring");

// Fills s.items with items [skip, skip + kMaxItems) of this block's stretch;
// returns how many there are in all, and the unit of the pass's first.  `tmp` is list_words of shared memory,
// idle now.
__device__ int list_items(Block& s, const AttnParams& p, int32_t* tmp, int skip, int* first) {
  const int n = p.n_groups, B = p.B;
  int32_t* gs = tmp;                               // [n + 1]
  int32_t* pl = gs + n + 1;                        // [n]
  int32_t* seen = pl + n + 1;                      // [B]
  int32_t* group = seen + B;                       // [B]; -1: none
  int32_t* most = group + B;                       // [B]: prefix tokens that a leader's unit sees
  int32_t* ppre = most + B;                        // [B]: tiles of the prefix units led below
  int32_t* pre = ppre + B;                         // [B + 1]: own tiles of lower entries
  int32_t* cnt = pre + B + 1;                      // [B + 1]: lower entries that have any
  const int limit = p.max_pages * kPageTokens;
  const bool teller = blockIdx.x == gridDim.x - 1 && skip == 0;
  bool bad = false;                  // group bounds out of order: nothing is in a group
  for (int i = threadIdx.x; i <= n; i += kThreads) {
    const int from = __ldg(p.group_start + i);
    gs[i] = from;
    if (i < n) {
      const int to = __ldg(p.group_start + i + 1);
      if (from < 0 || from > to || to > B) {
        bad = true;
        if (teller) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, i, to, B);
      }
      const int len = __ldg(p.prefix_lens + i), fit = min(max(len, 0), limit);
      pl[i] = fit;
      if (teller && len != fit) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, i, len, limit);
    }
  }
  for (int b = threadIdx.x; b < B; b += kThreads) {
    const int pos = __ldg(p.positions + b);
    const bool fits = pos >= -1 && pos < limit;
    if (teller && !fits) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, b, pos, limit);
    seen[b] = fits ? pos + 1 : 0;
    most[b] = 0;
  }
  if (threadIdx.x == 0) {
    s.first = INT32_MAX;
    s.last = 0;
    s.n_steps = 0;
  }
  bad = __syncthreads_or(bad);
  const int span = 2 * p.MB;                       // entries of a prefix unit
  auto lead_of = [&](int b, int g) { return b - (b - gs[g]) % span; };
  for (int b = threadIdx.x; b < B; b += kThreads) {
    int lo = 0, hi = n;                            // last group that starts at or before b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gs[mid] <= b) lo = mid;
      else hi = mid;
    }
    const int g = !bad && gs[lo] <= b && b < gs[lo + 1] ? lo : -1;
    group[b] = g;
    if (g >= 0) atomicMax(&most[lead_of(b, g)], min(seen[b], pl[g]));
  }
  __syncthreads();
  // this thread's entries: places of their tiles in the line
  const int per = (B + kThreads - 1) / kThreads;
  const int e0 = min(B, (int)threadIdx.x * per), e1 = min(B, e0 + per);
  auto members = [&](int b) { return min(min(span, gs[group[b] + 1] - b), B - b); };
  auto prefix_tiles = [&](int b) { return (most[b] + kTile - 1) / kTile; };
  auto own_tiles = [&](int b) {
    const int g = group[b];
    if (g < 0 || seen[b] <= pl[g]) return 0;
    return (seen[b] - pl[g] / kPageTokens * kPageTokens + kTile - 1) / kTile;
  };
  int v[4] = {0, 0, 0, 0}, below[4], total[4];     // prefix tiles, prefix units, own tiles, own units
  for (int b = e0; b < e1; ++b) {
    const int np = prefix_tiles(b), no = own_tiles(b);
    v[0] += np;
    v[1] += np > 0;
    v[2] += no;
    v[3] += no > 0;
  }
  scan4(s, v, below, total);
  {
    int shared = below[0], tiles = below[2], units = below[3];
    for (int b = e0; b < e1; ++b) {
      ppre[b] = shared;
      pre[b] = tiles;
      cnt[b] = units;
      const int np = prefix_tiles(b), no = own_tiles(b);
      shared += np;
      tiles += no;
      units += no > 0;
    }
    if (threadIdx.x == 0) {
      pre[B] = total[2];
      cnt[B] = total[3];
    }
  }
  __syncthreads();
  const int own0 = p.Hkv * total[0];               // place of the first own tile
  const Line line(own0 + p.Hkv * total[2], p.grid);
  auto chunk_of = [&](int b) { return b / p.MB * p.MB; };
  if (teller) {
    if (threadIdx.x == 0) *p.line_total = line.total;
    for (int b = threadIdx.x; b < B; b += kThreads) {
      const int g = group[b], cf = chunk_of(b), ce = min(B, cf + p.MB);
      Entry e{};
      e.lead = -1;
      if (g >= 0) {
        e.lead = lead_of(b, g);
        e.group = g;
        e.prefix_tiles = prefix_tiles(e.lead);
        if (e.prefix_tiles) {
          e.dual = members(e.lead) > p.MB;
          e.prefix_at = p.Hkv * ppre[e.lead];
        }
        e.own_tiles = own_tiles(b);
        e.own_stride = pre[ce] - pre[cf];
        e.own_at = own0 + (p.Hkv - 1) * pre[cf] + pre[b];
      }
      p.entries[b] = e;
    }
  }
  int r0 = 0, r1 = 0;
  if (line.total > 0 && (int)blockIdx.x < line.blocks) {
    r0 = line.start(blockIdx.x);
    r1 = line.start(blockIdx.x + 1);
  }
  // this thread's units that fall to the stretch: (prefix, entry, head, place
  // in the line, tiles of the unit, share t0 .. t1 - 1, number of the unit)
  auto visit = [&](auto&& emit) {
    int units = p.Hkv * below[1];
    for (int b = e0; b < e1; ++b) {
      const int nt = prefix_tiles(b);
      if (nt == 0) continue;
      const int at = p.Hkv * ppre[b];
      if (at < r1 && at + p.Hkv * nt > r0) {
        for (int h = max(0, (r0 - at) / nt); h < p.Hkv; ++h) {
          const int us = at + h * nt;
          if (us >= r1) break;
          const int t0 = max(0, r0 - us), t1 = min(nt, r1 - us);
          if (t1 > t0) emit(true, b, h, us, nt, t0, t1, units + h);
        }
      }
      units += p.Hkv;
    }
    units = p.Hkv * total[1];
    for (int b = e0; b < e1; ++b) {
      const int nt = own_tiles(b);
      if (nt == 0) continue;
      const int cf = chunk_of(b), ce = min(B, cf + p.MB), stride = pre[ce] - pre[cf];
      const int at = own0 + (p.Hkv - 1) * pre[cf] + pre[b];
      if (at >= r1 || at + (p.Hkv - 1) * stride + nt <= r0) continue;
      for (int h = max(0, (r0 - at - nt) / stride); h < p.Hkv; ++h) {
        const int us = at + h * stride;
        if (us >= r1) break;
        const int t0 = max(0, r0 - us), t1 = min(nt, r1 - us);
        if (t1 > t0)
          emit(false, b, h, us, nt, t0, t1,
               units + (p.Hkv - 1) * cnt[cf] + h * (cnt[ce] - cnt[cf]) + cnt[b]);
      }
    }
  };
  // `keep` says which units to write; their place needs no count of those before
  auto write = [&](auto&& keep) { visit([&](bool prefix, int b, int h, int us, int nt, int t0, int t1, int unit) {
    if (!keep(unit)) return;
    const int g = group[b];
    Item& q = s.items[unit % kMaxItems];
    q.head = h;
    q.t0 = t0;
    q.t1 = t1;
    q.own = !prefix;
    if (prefix) {
      q.b0 = b;
      q.nmem = members(b);
      q.row = gs[g];
      q.lo = 0;
      q.hi = most[b];
      q.dual = q.nmem > p.MB;
      q.j0 = 0;
      q.steps = (t1 - t0) << (q.dual ? 1 : 0);
      atomicAdd(&s.n_steps, q.steps);
    } else {
      q.b0 = chunk_of(b);
      q.nmem = min(p.MB, B - q.b0);
      q.row = b;
      q.lo = pl[g];
      q.hi = seen[b];
      q.dual = false;
      // the run: the chunk's own tiles of this head, as far as they are here
      const int stride = pre[q.b0 + q.nmem] - pre[q.b0];
      const int hs = us - (pre[b] - pre[q.b0]);
      const int from = max(r0, hs), to = min(r1, hs + stride);
      q.j0 = us + t0 - from;
      q.steps = to - from;
      atomicAdd(&s.n_steps, t1 - t0);
    }
    const bool whole = t0 == 0 && t1 == nt;
    q.slot = (short)(whole ? -1 : 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0));
  }); };
  write([&](int unit) {
    atomicMin(&s.first, (unsigned)unit);
    atomicMax(&s.last, (unsigned)unit + 1u);
    return true;
  });
  __syncthreads();
  *first = (int)s.first + skip;
  const int n_items = s.last == 0 ? 0 : (int)(s.last - s.first);
  if (n_items > kMaxItems) {         // more than one pass: the runs end with a pass
    const int from = *first;
    if (threadIdx.x == 0) {
      s.win_lo = r0;
      s.win_hi = r1;
      s.n_steps = 0;
    }
    __syncthreads();
    visit([&](bool, int, int, int us, int, int t0, int, int unit) {
      if (unit == from) s.win_lo = us + t0;
      if (unit == from + kMaxItems) s.win_hi = us;
    });
    __syncthreads();
    r0 = max(r0, s.win_lo);
    r1 = min(r1, s.win_hi);
    write([&](int unit) { return unit >= from && unit < from + kMaxItems; });
    __syncthreads();
  }
  return n_items;
}

__device__ __forceinline__ int first_token(const Item& q, int tile) {
  return q.lo / kPageTokens * kPageTokens + tile * kTile;
}

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static constexpr float kShift = 0.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Half<__half> {
  static constexpr uint32_t kFormat = 0;
  // P is 2^7 larger than the softmax's, its largest 2^15 with the lag of the
  // reference: fp16 then keeps weights down to 2^-31 of the largest, where
  // 2^-24 would lose the tail of a long context.
  static constexpr float kShift = 7.0f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap qmap_one) {
  using L = Layout<HD>;
  extern __shared__ __align__(1024) uint8_t base[];
  __shared__ Block s;
  const uint32_t sb = saddr(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b_full = saddr(s.bars.full), b_empty = saddr(s.bars.empty);
  const uint32_t b_qfull = saddr(s.bars.q_full), b_qempty = saddr(s.bars.q_empty);
  const uint32_t b_sfull = saddr(s.bars.s_full), b_pready = saddr(s.bars.p_ready);
  const uint32_t b_pv = saddr(s.bars.pv_done);
  const uint32_t b_ofull = saddr(s.bars.o_full), b_ofree = saddr(s.bars.o_free);

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, 2);
      mbar_init(b_sfull + 16 * i, 1);
      mbar_init(b_sfull + 16 * i + 8, 1);
      mbar_init(b_pready + 16 * i, kGroupThreads);
      mbar_init(b_pready + 16 * i + 8, kGroupThreads);
      mbar_init(b_pv + 8 * i, 1);
      mbar_init(b_ofull + 8 * i, 1);
      mbar_init(b_ofree + 8 * i, kGroupThreads);
    }
    s.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    prefetch_map(&qmap);
    prefetch_map(&qmap_one);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     saddr(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // Nothing of the call's memory is touched before the kernels ahead are done.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // Barrier use counts, carried from pass to pass by every role that needs them.
  // (No arrays: one whose index is not known when compiling would lie in memory,
  // and next to this much shared memory there is no L1 cache for it.)
  uint32_t ring = 0;                 // tiles loaded so far
  uint32_t q0_uses = 0, q1_uses = 0; // of the query slots
  uint32_t sn = 0, on = 0;           // steps and runs of the warp's stream
  uint32_t passes = 0;               // that had a step of it
  bool ok = true;
  uint32_t tm = 0;

  for (int skip = 0;; skip += kMaxItems) {
    int first;
    const int n_all = list_items(s, p, reinterpret_cast<int32_t*>(base + L::kRing), skip, &first);
    const int n_items = min(kMaxItems, n_all - skip), n_steps = s.n_steps;
    // the list's scratch is the ring: later writes there go through TMA
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_before();
    __syncthreads();
    tc_after();
    tm = s.tmem;
    const int st = warp < kTmaWarp ? warp >> 2 : warp - kMmaWarp;   // the warp's stream
    const uint32_t tm_s = tm + 128 * st, tm_o = tm + 256 + 128 * st;
    auto q_uses = [&](int slot) { return slot ? q1_uses : q0_uses; };
    auto use_q = [&](int slot) {
      q0_uses += slot == 0;
      q1_uses += slot == 1;
    };

    if (warp == kTmaWarp) {
      // -------------------------------------------------------- loads -----
      // Lane i holds where the two pages of tile from + i begin in the pools'
      // rows, of 32 tiles at a time and of the 32 before.
      int from = -32, y0 = 0, y1 = 0, y0_was = 0, y1_was = 0;
      auto look_up = [&]() {
        from += 32;
        y0_was = y0;
        y1_was = y1;
        int x = from + lane, i = 0;
        for (; i < n_items; ++i) {
          const Item& q = s.items[(first + i) % kMaxItems];
          const int nt = q.t1 - q.t0;
          if (x < nt) break;
          x -= nt;
        }
        int id[2] = {p.n_pages, p.n_pages}, head = 0;    // beyond the pool: loads as zeros
        if (i < n_items) {
          const Item& q = s.items[(first + i) % kMaxItems];
          head = q.head;
          const int page = first_token(q, q.t0 + x) / kPageTokens;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int lp = page + k;
            if (lp < p.max_pages && lp * kPageTokens < q.hi)
              id[k] = __ldg(p.page_table + (size_t)q.row * p.max_pages + lp);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (id[k] < 0 || id[k] > p.n_pages ||
                (id[k] == p.n_pages && page + k < p.max_pages && (page + k) * kPageTokens < q.hi)) {
              report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, q.row, id[k], p.n_pages);
              id[k] = p.n_pages;
            }
        }
        y0 = (id[0] * p.Hkv + head) * kPageTokens;
        y1 = (id[1] * p.Hkv + head) * kPageTokens;
      };
      // A tile that one stream alone uses is released here for the other, so that
      // an MMA warp need not look at what is not its stream's.
      auto load_tile = [&](int tile, const void* map, bool both) {
        if (tile >= from + 32) look_up();
        const bool now = tile >= from;
        const int src = now ? tile - from : tile - from + 32;
        const int a = __shfl_sync(kFull, now ? y0 : y0_was, src);
        const int b = __shfl_sync(kFull, now ? y1 : y1_was, src);
        const uint32_t st = ring % L::kStages, bar = b_full + 8 * st;
        if (ring >= L::kStages) ok = ok && wait(s, b_empty + 8 * st, (ring / L::kStages - 1) & 1, p);
        ok = __all_sync(kFull, ok);
        if (ok && lane == 0 && (int)blockIdx.x != p.stall) {
          if (!both) mbar_arrive(b_empty + 8 * st);
          mbar_expect(bar, L::kTileBytes);
          const uint32_t dst = sb + L::kRing + st * L::kTileBytes;
#pragma unroll
          for (int c2 = 0; c2 < L::kChunks; ++c2) {
            tma_3d(dst + c2 * kTile * 128, map, 0, a, c2, bar);
            tma_3d(dst + c2 * kTile * 128 + kPageTokens * 128, map, 0, b, c2, bar);
          }
        }
        __syncwarp();
        ++ring;
      };
      auto load_q = [&](const Walk& w) {
        const Item& q = w.at();
        for (int h = 0; h < (q.dual ? 2 : 1); ++h) {
          const int sl = w.q_slot(h);
          if (q_uses(sl) > 0) ok = ok && wait(s, b_qempty + 8 * sl, (q_uses(sl) - 1) & 1, p);
          ok = __all_sync(kFull, ok);
          if (ok && lane == 0) {
            const bool one = q.nmem == 1;
            const int rows = one ? p.G : p.G * p.MB;
            if (w.dual || w.total == 1) mbar_arrive(b_qempty + 8 * sl);   // for the stream without it
            mbar_expect(b_qfull + 8 * sl, (uint32_t)rows * HD * 2);
            const uint32_t dst = sb + L::kQ + sl * L::kTileBytes;
#pragma unroll
            for (int c2 = 0; c2 < L::kChunks; ++c2)
              tma_4d(dst + c2 * kRows * 128, one ? &qmap_one : &qmap, 0, q.head * p.G,
                     q.b0 + h * p.MB, c2, b_qfull + 8 * sl);
          }
          __syncwarp();
          use_q(sl);
        }
      };
      Walk k(s.items, n_items, first), v(s.items, n_items, first);
      int kt = 0, vt = 0;
      auto do_k = [&]() {
        if (k.first()) load_q(k);
        if (k.loads()) load_tile(kt++, &kmap, k.dual);
        k.next();
      };
      for (int i = 0; i < 2 && i < n_steps && ok; ++i) do_k();
      for (int n = 0; n < n_steps && ok; ++n) {
        if (v.loads()) load_tile(vt++, &vmap, v.dual);
        v.next();
        if (ok && n + 2 < n_steps) do_k();
      }
    } else if (warp >= kMmaWarp) {
      // --------------------------------------------------------- MMAs -----
      // Every lane keeps count, one issues.  The warp goes through its stream's
      // steps, K two of them ahead of V: S of a half takes the place of P while
      // the softmax has the other half.
      const uint32_t fmt = (1u << 4) | (Half<T>::kFormat << 7) | (Half<T>::kFormat << 10) |
                           ((uint32_t)(kRows >> 4) << 24);
      const uint32_t id_qk = fmt | ((uint32_t)(kTile / 2 >> 3) << 17);
      const uint32_t id_pv = fmt | (1u << 16) | ((uint32_t)(HD >> 3) << 17);
      Walk k(s.items, n_items, first), v(s.items, n_items, first);
      uint32_t k_at = 0, v_at = 0;     // places in the ring
      const uint32_t bar_s = b_sfull + 16 * st, bar_p = b_pready + 16 * st;
      // a wait whose outcome is the same in every lane
      auto hold = [&](uint32_t bar, uint32_t parity) { ok = __all_sync(kFull, ok && wait(s, bar, parity, p)); };
      auto hold_tile = [&](uint32_t at) { hold(b_full + 8 * (at % L::kStages), (at / L::kStages) & 1); };
      auto see_k = [&]() {
        if (k.loads()) k_at = ring + k.k_place();
      };
      auto leave_k = [&]() {           // to the next step, its stream's or the other's
        if (k.done()) return;
        if (k.last()) {
          const int sl = k.q_slot(0);
          use_q(sl);
          if (k.dual) use_q(1);
        }
        k.next();
        see_k();
      };
      auto qk = [&](int half) {
        const uint32_t stage = k_at % L::kStages;
        const int sl = k.q_slot(st);
        if (half == 0) {
          hold_tile(k_at);
          if (k.first_of_stream()) hold(b_qfull + 8 * sl, q_uses(sl) & 1);
          if (!ok) return;
        }
        tc_after();
        const uint32_t qa = sb + L::kQ + sl * L::kTileBytes;
        const uint32_t ka = sb + L::kRing + stage * L::kTileBytes + half * (kTile / 2) * 128;
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
          mma_ss4(tm_s + half * (kTile / 2), desc_of(qa + c * kRows * 128, 16), desc_of(ka + c * kTile * 128, 16),
                  id_qk, c > 0);
        tc_commit(bar_s + 8 * half);
        if (half == 1) {
          tc_commit(b_empty + 8 * stage);
          if (k.last_of_stream()) tc_commit(b_qempty + 8 * sl);   // the run's last use of a slot
        }
      };
      see_k();
      if (st == 1 && n_steps > 1) {
        leave_k();
        v.next();
      }
      if (st < n_steps) {
        qk(0);
        if (ok) qk(1);
        leave_k();
        leave_k();
      }
      for (int n = st; n < n_steps && ok; n += 2) {
        if (v.loads()) v_at = ring + v.v_place(n + 1 < n_steps);
        else v_at = ring + v.v_place(false);           // of the step before, which shares it
        const bool more = n + 2 < n_steps;
        const uint32_t stage = v_at % L::kStages;
        const uint32_t va = sb + L::kRing + stage * L::kTileBytes;
        hold_tile(v_at);
        if (v.first_of_stream() && on > 0) hold(b_ofree + 8 * st, (on - 1) & 1);
        hold(bar_p, sn & 1);
        if (!ok) break;
        tc_after();
        mma_ts4(tm_o, tm_s, desc_of(va, kTile * 128), id_pv, !v.first_of_stream());
        if (more) qk(0);
        else tc_commit(b_pv + 8 * st);
        hold(bar_p + 8, sn & 1);
        if (!ok) break;
        tc_after();
        mma_ts4(tm_o, tm_s + kTile / 2, desc_of(va + (kTile / 2) * 128, kTile * 128), id_pv, 1);
        tc_commit(b_empty + 8 * stage);
        if (v.last_of_stream()) {
          tc_commit(b_ofull + 8 * st);
          on += 1;
        }
        sn += 1;
        if (more) {
          qk(1);
          leave_k();
          leave_k();
          v.next();
          v.next();
        }
      }
      while (!k.done()) leave_k();
      ring += 2 * k.tile;
    } else {
      // ------------------------------------------------------ softmax -----
      // A wait that runs out ends no loop here: once one has, all return at once.
      const int r = threadIdx.x & (kGroupThreads - 1); // row
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 lanes
      const uint32_t ts = tm_s + lanes;
      const int j = r / p.G;                           // entry among the rows, less b0
      float m = -INFINITY, l = 0.0f;
      int slot = -2;                                   // the row's partial result; -2: none
      int n0 = 0, tiles = 0;                           // steps and tiles of the items before
      for (int i = 0; i < n_items; ++i) {
        const Item& q = s.items[(first + i) % kMaxItems];
        const bool dual = q.dual, own = q.own;
        const int nt = q.t1 - q.t0, steps = dual ? 2 * nt : nt;
        const int lo = q.lo, hi = q.hi;
        const int a0 = first_token(q, q.t0);
        if (q.j0 == 0) {
          m = -INFINITY;
          l = 0.0f;
          slot = -2;
        }
        // this thread's row of the item
        const int e = (dual ? st * p.MB : 0) + j;
        const bool real = j < p.MB && (own ? q.b0 + e == q.row : e < q.nmem);
        const bool busy = __any_sync(kFull, real);
        int lim = 0;                                   // tokens that the row sees
        if (real) {
          slot = q.slot;
          lim = hi;
          if (!own) {
            const int pos = __ldg(p.positions + q.b0 + e);
            lim = min(pos < 0 || pos >= p.max_pages * kPageTokens ? 0 : pos + 1, hi);
          }
        }
        const int all_see = __reduce_min_sync(kFull, lim);
        for (int u = (st ^ n0) & 1; u < steps; u += 2) {
          const int tile = dual ? u >> 1 : u;
          for (int half = 0; half < 2; ++half) {
            const uint32_t th = ts + half * (kTile / 2);
            const int a = a0 + tile * kTile + half * 64;   // the half's first token
            const bool masked = a < lo || a + 64 > all_see;
            wait(s, b_sfull + 16 * st + 8 * half, sn & 1, p);
            __syncwarp();
            uint32_t x[64];                              // the row's scores
            float ref = 0.0f;
            if (busy) {
              tc_after();
              tmem_ld32(th, x);
              tmem_ld32(th + 32, x + 32);
              tmem_wait_ld64(x);
              if (masked) {                              // tokens that are not the row's
                auto bits = [](int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; };
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                  const uint32_t keep = bits(lim - a - c) & ~bits(lo - a - c);
#pragma unroll
                  for (int k = 0; k < 32; ++k)
                    if (!((keep >> k) & 1u)) x[c + k] = 0xff800000u;
                }
              }
              float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
              for (int k = 2; k < 62; k += 4) {
                t0 = max3(t0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                t1 = max3(t1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
              }
              t0 = max3(t0, __uint_as_float(x[62]), __uint_as_float(x[63]));
              const float top = max3(t0, t1, t1) * p.c;
              // a score that is no number, or +infinity, makes the sum NaN
              if (top != -INFINITY) l += top - top;
              const bool grow = top > m + kRescale;      // also the first score of a row
              const bool some = grow && m != -INFINITY;
              float f_old = 1.0f;
              if (grow) {
                f_old = ex2(m - top);                    // 0 for the first
                l *= f_old;
                m = top;
              }
              // O of a row without a score so far is 0 already
              if (__any_sync(kFull, some)) {
                // O is at rest behind P V of the stream's half before this one, which
                // the S that took that half's place was committed after; behind the
                // last step's first half P V has its own commit
                if (half == 0) wait(s, b_sfull + 16 * st + 8, sn & 1, p);
                else if (n0 + u + 2 < n_steps) wait(s, b_sfull + 16 * st, (sn + 1) & 1, p);
                else wait(s, b_pv + 8 * st, passes & 1, p);
                __syncwarp();
                tc_after();
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(tm_o + lanes + c, o);
                  tmem_wait_ld32(o);
#pragma unroll
                  for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f_old);
                  tmem_st32(tm_o + lanes + c, o);
                }
              }
              ref = (m == -INFINITY ? 0.0f : m) - Half<T>::kShift;
            }
            const int before = lo - a, behind = hi - a;
            if (before > 0 || (behind > 0 && behind < 64)) {
              // Clear V's rows of tokens inside the half's page that are not the
              // unit's: what lies there is not the sequence's, and 0 x infinity would
              // spoil the row.  The tile's place in the ring is behind the V tiles
              // before and the K tiles of the steps up to the one after that which
              // loaded it.
              const uint32_t at = ring + 2 * (tiles + tile) + 1 + (!dual && n0 + u + 1 < n_steps ? 1 : 0);
              const uint32_t vs = at % L::kStages;
              if (wait(s, b_full + 8 * vs, (at / L::kStages) & 1, p)) {
                const uint32_t va = sb + L::kRing + vs * L::kTileBytes + half * 64 * 128;
                auto clear = [&](int tok0, int tok1) {
                  for (int k = tok0 * 8 + r; k < tok1 * 8; k += kGroupThreads)
#pragma unroll
                    for (int c = 0; c < L::kChunks; ++c)
                      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                       va + c * kTile * 128 + k * 16),
                                   "r"(0)
                                   : "memory");
                };
                clear(0, min(max(before, 0), 64));
                clear(behind > 0 ? min(behind, 64) : 64, 64);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              }
              __syncwarp();
            }
            if (busy) {
              const uint64_t c2 = pair(p.c, p.c), r2 = pair(-ref, -ref);
              uint64_t sum[2] = {0, 0};
#pragma unroll
              for (int c = 0; c < 64; c += 32) {
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  uint64_t w = fma2(pair(__uint_as_float(x[c + 2 * k]), __uint_as_float(x[c + 2 * k + 1])), c2, r2);
                  float wa, wb;
                  unpair(w, wa, wb);
                  wa = ex2(wa);
                  wb = ex2(wb);
                  sum[k & 1] = add2(sum[k & 1], pair(wa, wb));
                  o[k] = Half<T>::pack(wa, wb);
                }
                tmem_st16(th + c / 2, o);        // over scores that have been read
              }
              tmem_wait_st();
              tc_before();
              mbar_arrive(b_pready + 16 * st + 8 * half);
              float s0, s1, s2, s3;
              unpair(sum[0], s0, s1);
              unpair(sum[1], s2, s3);
              l += (s0 + s1) + (s2 + s3);
            } else {
              if (own) {                 // other entries' tokens: no weight
                tc_after();
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = 0;
                tmem_st32(th, x);
                tmem_wait_st();
                tc_before();
              }
              mbar_arrive(b_pready + 16 * st + 8 * half);
            }
          }
          sn += 1;
        }
        n0 += steps;
        tiles += nt;
        if (q.j0 + steps == q.steps) {
          // ----------------------------------------------- the run's end --
          const int last = (n0 - 1) & 1;                     // stream of its last step
          const bool took = q.steps >= 2 || last == st;      // this stream took part
          if (took) {
            wait(s, b_ofull + 8 * st, on & 1, p);
            on += 1;
            __syncwarp();
          }
          if (__any_sync(kFull, slot != -2)) {
            float* dst = nullptr;
            if (slot != -2) {
              const int hq = q.head * p.G + r % p.G;
              const size_t row = slot >= 0 ? ((size_t)slot * 2 + st) * p.slot_rows + r
                                           : whole_row(p, own ? 1 : 0, dual ? 0 : st, q.b0 + e, hq);
              dst = p.part + row * HD;
              // without a step of its own the stream has seen nothing, and O is not its
              p.part_ml[row] = make_float2((m == -INFINITY ? 0.0f : m) - Half<T>::kShift, took ? l : 0.0f);
            }
            if (took) {
              tc_after();
#pragma unroll 1
              for (int c = 0; c < HD; c += 32) {
                uint32_t o[32];
                tmem_ld32(tm_o + lanes + c, o);
                tmem_wait_ld32(o);
                if (slot != -2) {
#pragma unroll
                  for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<uint4*>(dst + c + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
              }
              tc_before();
            }
          }
          if (took) mbar_arrive(b_ofree + 8 * st);
        }
      }
      ring += 2 * tiles;               // the other roles' ring count
      passes += n_steps > st;
    }
    __syncthreads();
    ok = ok && *(volatile int*)&s.abort == 0;
    if (!ok || skip + kMaxItems >= n_all) break;
    __syncthreads();
  }

  // A wait that ran out may have left copies and MMAs in flight: give them time.
  // The block's shares are then not looked at.
  const bool gave_up = *(volatile int*)&s.abort != 0;
  if (threadIdx.x == 0) p.gave_up[blockIdx.x] = gave_up;
  if (gave_up) {
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000) {
    }
  }
  tc_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
  }
}

// Row (b, hq) from its own tokens alone, one warp, HD / 32 columns per lane:
// what the tiles gave is not finite.  Slow, and right whatever the memory of
// other entries holds.  `acc` is kept as the weighted mean of the values so far,
// which stays in range where their sum would not (bf16 values near 3e38).
template <typename T, int HD>
__device__ __noinline__ void row_alone(const AttnParams& p, int b, int hq, int group, float* acc, float* m_out,
                                       float* l_out) {
  constexpr int C = HD / 32;
  const int lane = threadIdx.x & 31, h = hq / p.G;
  const int limit = p.max_pages * kPageTokens;
  const int lead = __ldg(p.group_start + group), pos = __ldg(p.positions + b);
  const int prefix = min(max(__ldg(p.prefix_lens + group), 0), limit);
  const int seen = pos < 0 || pos >= limit ? 0 : pos + 1;
  const T* q = static_cast<const T*>(p.q) + (size_t)b * p.q_stride + (size_t)hq * HD + lane * C;
  float qv[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    qv[i] = to_float(q[i]);
    acc[i] = 0.0f;
  }
  for (int t = 0; t < seen; ++t) {
    const int row = t < prefix ? lead : b;
    const int id = __ldg(p.page_table + (size_t)row * p.max_pages + t / kPageTokens);
    const bool there = id >= 0 && id < p.n_pages;
    const size_t at = (((size_t)(there ? id : 0) * p.Hkv + h) * kPageTokens + t % kPageTokens) * HD + lane * C;
    const T* k = static_cast<const T*>(p.k_pool) + at;
    const T* v = static_cast<const T*>(p.v_pool) + at;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) dot = fmaf(qv[i], there ? to_float(k[i]) : 0.0f, dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    const float s = dot * p.c;
    const float mn = fmaxf(m, s);
    const float f = m == mn ? 1.0f : ex2(m - mn), w = s == -INFINITY ? 0.0f : ex2(s - mn);
    m = mn;
    const float before = l * f;
    l = before + w;                      // 1 or more behind the first score
    if (l != 0.0f) {
      const float fo = before / l, fw = w / l;
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] = fmaf(fw, there ? to_float(v[i]) : 0.0f, acc[i] * fo);
    }
  }
  *m_out = m;
  *l_out = l;
}

// Adds up a row's partial results: prefix shares, then shares of its own
// tokens, in a fixed order.  W warps per (entry, query head), HD / 32 columns
// per lane.
// A row's result as the decode step's next operation reads it.
template <int HD>
__device__ __forceinline__ void to_step(const AttnParams& p, int b, int hq, const float* o) {
  constexpr int C = HD / 32;
  const int lane = threadIdx.x & 31;
  float* a = p.sink.out + ((size_t)b * p.Hq + hq) * HD + lane * C;
  float* f = reinterpret_cast<float*>(p.sink.frag + (size_t)(hq / p.G) * p.sink.frag_bytes) +
             (size_t)b * p.sink.frag_stride + hq % p.G * HD + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) a[i] = f[i] = o[i];
}

template <int W>
constexpr int kJoinWarps = W > 4 ? W : 4;   // of a block

template <typename T, int HD, int W>
__global__ void __launch_bounds__(32 * kJoinWarps<W>, W > 1 ? 1 : 8) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int C = HD / 32;
  // Many rows: few shares each, and room for more warps matters more (8000 rows:
  // 2 us less than with 8).
  constexpr int kAhead = W > 1 ? 8 : 4;
  __shared__ float s_acc[W > 1 ? W : 1][HD];
  __shared__ float2 s_ml[W > 1 ? W : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % W;
  const int row = (int)blockIdx.x * (kJoinWarps<W> / W) + warp / W;
  const int b = row / p.Hq, hq = row % p.Hq, h = hq / p.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= p.B * p.Hq) return;
  const Entry e = p.entries[b];
  if (e.lead < 0) {                  // of no group: left as it was, but a step needs all rows
    if (p.sink.out && sub == 0) {
      if (lane == 0) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, b, -1, p.n_groups);
      float zero[C] = {};
      to_step<HD>(p, b, hq, zero);
    }
    return;
  }
  const Line line(*p.line_total, p.grid);
  float acc[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) acc[i] = 0.0f;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const int nt = kind == 0 ? e.prefix_tiles : e.own_tiles;
    if (nt == 0) continue;
    const bool dual = kind == 0 && e.dual;
    const int at = kind == 0 ? e.prefix_at + h * nt : e.own_at + h * e.own_stride;
    const int c0 = line.block_of(at), c1 = line.block_of(at + nt - 1);
    const bool whole = c0 == c1;
    // the row's place among its unit's rows
    const int j = kind == 0 ? b - e.lead : b;
    const int half = dual ? j / p.MB : 0, r = (j % p.MB) * p.G + hq % p.G;
    const int n = (c1 - c0 + 1) * (dual ? 1 : 2);
    for (int i0 = sub; i0 < n; i0 += 32 * W) {
      // lane i looks at share i0 + W i: of a block, and of one of its streams
      const int x = i0 + W * lane;
      const int c = c0 + (dual ? x : x >> 1), stream = dual ? half : x & 1;
      size_t at_row = 0;
      float2 ml = make_float2(0.0f, 0.0f);
      if (x < n) {
        at_row = whole ? whole_row(p, kind, dual ? 0 : stream, b, hq)
                       : ((size_t)(2 * c + (c == c0 ? 1 : 0)) * 2 + stream) * p.slot_rows + r;
        ml = p.part_ml[at_row];
        // unfinished: the row's sum is no number, and it is computed alone
        if (p.gave_up[c]) ml = make_float2(0.0f, __int_as_float(0x7fffffff));
      }
      // a share that saw nothing has no weight, and its O is not looked at
      float top = ml.y == 0.0f ? -INFINITY : ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float mn = fmaxf(m, top);
      const float fo = m == mn ? 1.0f : ex2(m - mn);
      const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - mn);
      m = mn;
      l *= fo;
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] *= fo;
      const int shares = min(32, (n - i0 + W - 1) / W);
      // kAhead shares' rows on their way at once
      for (int i1 = 0; i1 < shares; i1 += kAhead) {
        float fi[kAhead], v[kAhead][C];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          fi[u] = __shfl_sync(kFull, f, i1 + u);
          const float li = __shfl_sync(kFull, ml.y, i1 + u);   // 0 behind the last
          const float* src = p.part + __shfl_sync(kFull, (unsigned long long)at_row, i1 + u) * HD + lane * C;
#pragma unroll
          for (int k = 0; k < C; ++k) v[u][k] = 0.0f;
          // Any share that saw something counts, however small its weight: NaN and
          // infinities stay what they are when the weight's exponential is 0.
          if (li != 0.0f) {
            l = fmaf(li, fi[u], l);
            if constexpr (C == 4) {
              const float4 t = *reinterpret_cast<const float4*>(src);
              v[u][0] = t.x;
              v[u][1] = t.y;
              v[u][2] = t.z;
              v[u][3] = t.w;
            } else {
              const float2 t = *reinterpret_cast<const float2*>(src);
              v[u][0] = t.x;
              v[u][1] = t.y;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
          for (int k = 0; k < C; ++k) acc[k] = fmaf(v[u][k], fi[u], acc[k]);
      }
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < C; ++i) s_acc[warp][lane * C + i] = acc[i];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float mn = m;
#pragma unroll
    for (int k = 1; k < W; ++k) mn = fmaxf(mn, s_ml[warp + k].x);
    const float f0 = m == mn ? 1.0f : ex2(m - mn);
    l *= f0;
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] *= f0;
#pragma unroll
    for (int k = 1; k < W; ++k) {
      const float2 ml = s_ml[warp + k];
      const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - mn);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] = fmaf(s_acc[warp + k][lane * C + i], f, acc[i]);
    }
    m = mn;
  }
  float size = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) size += fabsf(acc[i]);
  const bool alone = __any_sync(kFull, !(size < INFINITY) || !(l < INFINITY));
  if (alone) row_alone<T, HD>(p, b, hq, e.group, acc, &m, &l);
  const float inv = alone ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) acc[i] *= inv;
  if (p.sink.out) {
    to_step<HD>(p, b, hq, acc);
    return;
  }
  uint32_t o[C / 2];
#pragma unroll
  for (int i = 0; i < C; i += 2) o[i / 2] = Half<T>::pack(acc[i], acc[i + 1]);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + (size_t)row * HD + lane * C);
#pragma unroll
  for (int i = 0; i < C / 2; ++i) out[i] = o[i];
  if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* ptr, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = encoder();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn && fn(m, type, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Streaming multiprocessors of a device (looked up once per device).
int sm_count(int device) {
  static std::once_flag once[kMaxDevices];
  static int count[kMaxDevices];
  if (device < 0 || device >= kMaxDevices) return 0;
  std::call_once(once[device], [&] {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) == cudaSuccess) count[device] = n;
  });
  return count[device];
}

// Rows up to which eight warps join one.  Two such blocks run on a multiprocessor,
// 296 in all.  Up to there eight warps were faster in every case measured (heads of
// 64 and 128; 128 rows on 8192 tokens 17.8 us, with one warp 27.7; 288 rows on 1000
// tokens 16.7 and 17.2), from 640 rows on slower in every one (8192: 35.7 and 30.6;
// 1000: 28.4 and 20.9).  Between, rows of many shares gain (448 rows on 8192: 30.0
// and 34.2, on 32768: 35.3 and 40.8) and rows of few lose (on 1000: 23.8 and 20.2, in
// 4 groups on 4999: 30.8 and 28.5).  The host does not know the lengths: this is
// where the two even out.
constexpr unsigned kWideJoin = 448;

constexpr int kMaxBlocks = 160;      // at least the device's multiprocessors

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// Rows of a split share: a stream's, or as many as the whole batch has.
int slot_rows(const mk_prefix_attention_args* a) {
  return std::min(kRows, a->batch * (a->n_q_heads / a->n_kv_heads));
}

// Split shares: two per block and stream; whole units: two kinds and streams.
size_t part_rows(const mk_prefix_attention_args* a) {
  return (size_t)2 * kMaxBlocks * 2 * slot_rows(a) + (size_t)4 * a->batch * a->n_q_heads;
}

mk_status validate(const mk_prefix_attention_args* a) {
  if (!a) return MK_ERR_INVALID;
  if (a->batch < 0 || a->n_groups < 0 || a->max_pages < 1 || a->n_pages < 1) return MK_ERR_INVALID;
  if (a->n_kv_heads < 1 || a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads) return MK_ERR_INVALID;
  if (a->head_dim != 64 && a->head_dim != 128) return MK_ERR_INVALID;
  if (a->type != MK_BF16 && a->type != MK_FP16) return MK_ERR_INVALID;
  if (!(a->scale > 0.0f) || !(a->scale < 1e30f)) return MK_ERR_INVALID;
  if (a->batch > kMaxBatch || a->n_groups > kMaxBatch) return MK_ERR_CAPACITY;
  if (a->n_q_heads / a->n_kv_heads > kMaxGroup || a->n_q_heads > (1 << 16)) return MK_ERR_CAPACITY;
  if (a->max_pages > (INT32_MAX - kTile) / kPageTokens) return MK_ERR_CAPACITY;
  // places in the line of tiles are 32-bit, and so are row numbers of the pools' tensor maps
  if ((long long)a->batch * a->n_kv_heads * ((long long)a->max_pages + 4) > INT32_MAX) return MK_ERR_CAPACITY;
  if (((long long)a->n_pages + 1) * a->n_kv_heads * kPageTokens > INT32_MAX) return MK_ERR_CAPACITY;
  return MK_OK;
}

// Both launches may begin while the one ahead is finishing: they wait for it
// before they touch memory.  Neither lets the one behind begin earlier than its
// own blocks end: that one's blocks would take the room that the join's are
// waiting for (256 entries on 32768 tokens: 149 us, not 135).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t st,
                   const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The kernel's right to its shared memory, asked for once per device.
template <typename T, int HD>
cudaError_t allow_shared(int device) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t result[kMaxDevices];
  std::call_once(once[device], [&] {
    result[device] = cudaFuncSetAttribute(attention_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          Layout<HD>::kDyn);
  });
  return result[device];
}

template <typename T, int HD>
cudaError_t launch_attention(const AttnParams& p, const CUtensorMap* maps, int device, cudaStream_t st) {
  cudaError_t e = allow_shared<T, HD>(device);
  if (e != cudaSuccess) return e;
  e = launch(attention_kernel<T, HD>, (unsigned)p.grid, kThreads, Layout<HD>::kDyn, st, p, maps[0], maps[1],
             maps[2], maps[3]);
  if (e != cudaSuccess) return e;
  const unsigned rows = (unsigned)(p.B * p.Hq);
  if (rows <= kWideJoin) return launch(join_kernel<T, HD, 8>, rows, 256, 0, st, p);
  return launch(join_kernel<T, HD, 1>, (rows + 3) / 4, 128, 0, st, p);
}

size_t workspace_size(const mk_prefix_attention_args* a) {
  if (validate(a) != MK_OK) return 0;
  const size_t rows = part_rows(a);
  return round256(rows * a->head_dim * sizeof(float)) + round256(rows * sizeof(float2)) +
         round256(sizeof(Entry) * (size_t)a->batch + sizeof(int) * (1 + kMaxBlocks));
}

mk_status run(const mk_prefix_attention_args* a, const StepSink& sink, cudaStream_t st, int stall) {
  mk_status s = validate(a);
  if (s != MK_OK) return s;
  if (a->batch == 0 || a->n_groups == 0) return MK_OK;
  if (!a->q || !a->k_pool || !a->v_pool || !a->page_table || !a->positions || !a->group_start ||
      !a->prefix_lens || !(a->out || sink.out) || !a->workspace)
    return MK_ERR_INVALID;
  const long long row = (long long)a->n_q_heads * a->head_dim;
  if (a->q_token_stride % 8 || (a->batch > 1 && a->q_token_stride < row)) return MK_ERR_INVALID;
  if (!aligned(a->q, 16) || !aligned(a->k_pool, 16) || !aligned(a->v_pool, 16) ||
      !aligned(a->out, 16) || !aligned(a->workspace, 256))
    return MK_ERR_INVALID;
  if (a->workspace_bytes < workspace_size(a)) return MK_ERR_CAPACITY;
  DeviceGuard guard(a->device);
  if (guard.status() != MK_OK) return guard.status();
  const int sms = sm_count(a->device);
  if (sms < 1) return MK_ERR_CUDA;
  const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;

  AttnParams p{};
  p.B = a->batch;
  p.n_groups = a->n_groups;
  p.max_pages = a->max_pages;
  p.n_pages = a->n_pages;
  p.Hq = a->n_q_heads;
  p.Hkv = a->n_kv_heads;
  p.G = a->n_q_heads / a->n_kv_heads;
  p.MB = kRows / p.G;
  p.c = a->scale * 1.4426950408889634f;
  p.page_table = a->page_table;
  p.positions = a->positions;
  p.group_start = a->group_start;
  p.prefix_lens = a->prefix_lens;
  const size_t rows = part_rows(a);
  uint8_t* w = static_cast<uint8_t*>(a->workspace);
  p.part = reinterpret_cast<float*>(w);
  w += round256(rows * a->head_dim * sizeof(float));
  p.part_ml = reinterpret_cast<float2*>(w);
  w += round256(rows * sizeof(float2));
  p.entries = reinterpret_cast<Entry*>(w);
  p.line_total = reinterpret_cast<int*>(p.entries + a->batch);
  p.gave_up = p.line_total + 1;
  p.stall = stall;
  p.grid = blocks;
  p.q = a->q;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.q_stride = a->batch > 1 ? a->q_token_stride : row;
  p.n_slots = 2 * kMaxBlocks;
  p.slot_rows = slot_rows(a);
  p.out = a->out;
  p.lse = a->lse;
  p.sink = sink;
  p.status = a->status;

  const auto type = a->type == MK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t hd = (cuuint64_t)a->head_dim;
  CUtensorMap maps[4];
  {
    // {64 columns, tokens of all pages and heads, 64-column chunks}
    const cuuint64_t dims[3] = {64, (cuuint64_t)a->n_pages * a->n_kv_heads * kPageTokens, hd / 64};
    const cuuint64_t strides[2] = {hd * 2, 128};
    const cuuint32_t box[3] = {64, kPageTokens, 1};
    if (!encode(&maps[0], type, 3, a->k_pool, dims, strides, box) ||
        !encode(&maps[1], type, 3, a->v_pool, dims, strides, box))
      return MK_ERR_INVALID;
  }
  {
    // {64 columns, query heads, entries, chunks}: the heads of one KV head of
    // as many entries as a stream's rows hold, and of one
    const cuuint64_t dims[4] = {64, (cuuint64_t)a->n_q_heads, (cuuint64_t)a->batch, hd / 64};
    const cuuint64_t strides[3] = {hd * 2, (cuuint64_t)p.q_stride * 2, 128};
    cuuint32_t box[4] = {64, (cuuint32_t)p.G, (cuuint32_t)p.MB, 1};
    if (!encode(&maps[2], type, 4, a->q, dims, strides, box)) return MK_ERR_INVALID;
    box[2] = 1;
    if (!encode(&maps[3], type, 4, a->q, dims, strides, box)) return MK_ERR_INVALID;
  }
  cudaError_t e;
  if (a->type == MK_BF16)
    e = a->head_dim == 128 ? launch_attention<__nv_bfloat16, 128>(p, maps, a->device, st)
                           : launch_attention<__nv_bfloat16, 64>(p, maps, a->device, st);
  else
    e = a->head_dim == 128 ? launch_attention<__half, 128>(p, maps, a->device, st)
                           : launch_attention<__half, 64>(p, maps, a->device, st);
  return from_cuda(e);
}

}  // namespace

mk_status prefix_attention(const mk_prefix_attention_args* a, const StepSink& sink, cudaStream_t st) {
  return run(a, sink, st, -1);
}

}  // namespace ops
}  // namespace mk

extern "C" size_t mk_prefix_attention_workspace(const mk_prefix_attention_args* args) {
  return mk::ops::workspace_size(args);
}

extern "C" mk_status mk_prefix_attention_selftest(const mk_prefix_attention_args* args, void* stream) {
  if (!args || !args->status) return MK_ERR_INVALID;
  return mk::ops::run(args, mk::ops::StepSink{}, static_cast<cudaStream_t>(stream), 0);
}

extern "C" mk_status mk_prefix_attention(const mk_prefix_attention_args* args, void* stream) {
  return mk::ops::prefix_attention(args, mk::ops::StepSink{}, static_cast<cudaStream_t>(stream));
}
