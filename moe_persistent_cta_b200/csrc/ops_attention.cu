// ops_attention.cu -- attention of one query token per batch entry over the
// paged cache, with the pages of a prefix that a group of entries shares read
// once for the whole group.
//
// For entry b and query head h, with seen = positions[b] + 1:
//   o = sum_t exp(s_t - lse) v_t,  s_t = scale q . k_t,  t < seen,
// the sum taken over tiles of 128 tokens with a running reference m and sum l:
//   P = 2^(s log2(e) - m), O = O 2^(m_old - m) + P V, l likewise.
// Any m not far below the largest score serves, so O is only rescaled when a
// row's largest score has grown by more than 8 (a factor of 256).
//
// Work.  A unit is one KV head's query rows against one token range: the
// prefix of up to 2 x floor(128 / G) entries of a group (G query heads per KV
// head), or one entry's own tokens.  Units are cut into tiles; the tiles of
// all units form one line, and every block takes an equal stretch of it, so a
// long prefix is split over many blocks and short remainders share one.  Each
// block finds its stretch from the device arrays: the host needs no lengths,
// and a captured graph replays with new ones.  A block's share of a unit
// leaves a partial result (O, m, l); a second launch adds them up.
//
// One block: a TMA warp streams K and V tiles, a warp issues tcgen05 MMAs,
// and two groups of four warps hold a softmax row per thread.  S = Q K^T and O
// live in tensor memory, two of each ("streams"), so that one stream's softmax
// runs under the other's MMAs.  With more than 128 rows the streams are the
// two halves of the rows, and each K and V tile serves both; with fewer they
// are alternate tiles of the same rows, joined at the end.  P goes back to
// tensor memory over S and is the A operand of P V.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "ops_common.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kRows = 128;           // query rows of a stream
constexpr int kTile = 128;           // tokens of a K or V tile
constexpr int kGroupThreads = 128;   // a softmax group: one row per thread
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSegments = 24;     // of one pass of a block over its stretch
constexpr int kMaxBatch = 4096;
constexpr int kMaxGroup = 64;        // query heads per KV head
constexpr float kRescale = 8.0f;     // log2 of the growth that O may lag behind
constexpr uint32_t kFull = 0xffffffffu;
// Tiles of one unit cost alike, whatever their rows, while memory is the bound.
constexpr int kWaitCycles = 1 << 30; // about half a second at any clock

struct AttnParams {
  int B, n_groups, max_pages, n_pages, Hq, Hkv, G, MB;   // MB: entries of a stream's rows
  float c;                           // scale x log2(e)
  const int32_t *page_table, *positions, *group_start, *prefix_lens;
  // partial results: [slot][stream][row] of split units, [stream][b][hq] of
  // whole ones (prefix, then own tokens)
  float* part;
  float2* part_ml;
  long long* tab;                    // see Table
  int n_slots;
  void* out;
  float* lse;
  int32_t* status;
};

// What the joining launch needs of the line of tiles, written by block 0:
// tab[0] its length, tab[1] the blocks that share it, then per entry the place
// of its first prefix tile (entries that lead a unit), of its first own tile,
// the number of both, and its unit's leader (-1: the entry is in no group).
struct Table {
  long long* t;
  int B;
  __device__ long long& total() const { return t[0]; }
  __device__ long long& blocks() const { return t[1]; }
  __device__ long long& prefix_at(int b) const { return t[2 + b]; }
  __device__ long long& own_at(int b) const { return t[2 + B + b]; }
  __device__ int& prefix_tiles(int b) const { return reinterpret_cast<int*>(t + 2 + 2 * B)[b]; }
  __device__ int& own_tiles(int b) const { return reinterpret_cast<int*>(t + 2 + 2 * B)[B + b]; }
  __device__ int& leader(int b) const { return reinterpret_cast<int*>(t + 2 + 2 * B)[2 * B + b]; }
};
__host__ __device__ inline size_t table_bytes(int B) { return 8 * (2 + 2 * (size_t)B) + 12 * (size_t)B; }

// The line's block that tile x (its place in the line) falls to, and the first
// place of block i's stretch.
__device__ __forceinline__ int block_of(long long x, long long total, long long blocks) {
  return (int)(((x + 1) * blocks - 1) / total);
}
__device__ __forceinline__ long long stretch(long long i, long long total, long long blocks) {
  return i * total / blocks;
}

struct Segment {      // a block's share of a unit
  int head;           // KV head
  int b0, nmem;       // entries b0 .. b0 + nmem - 1
  int row;            // page-table row of the keys
  int tok0;           // first token of the unit's first tile (a page start)
  int lo, hi;         // tokens lo .. hi - 1 belong to the unit
  int limit;          // entry b sees tokens below min(seen(b), limit)
  int t0, t1;         // tiles
  int dual;           // both streams share each tile
  int slot;           // partial: split slot, or -1 prefix / -2 own for whole units
};

template <int HD>
struct Layout {
  static constexpr int kChunks = HD / 64;
  static constexpr int kTileBytes = kTile * HD * 2;
  static constexpr int kStages = HD == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kEnd = kRing + kStages * kTileBytes;
  static constexpr int kDyn = kEnd;
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
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
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
#undef MK_R4
#undef MK_I4
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
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
  uint64_t s_full[2], p_ready[2];
  uint64_t o_full[2], o_free[2], ml_full[2];
};

struct Block {
  Bars bars;
  Segment seg[kMaxSegments];
  float2 ml[kRows];                  // a stream's (m, l), handed to the other
  long long scan[kWarps][4];
  int n_seg;                         // segments of this pass
  int total_seg;
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
// n & 1.  A segment with both halves of the rows has two steps per tile.  Tiles
// are loaded in the order the MMA warp first needs them: K of steps 0 and 1,
// then for each n V of step n and K of step n + 2.
struct Walk {
  const Segment* seg;
  int n_seg;
  int i = 0, j = 0;                  // segment, step of it
  __device__ __forceinline__ Walk(const Segment* s, int n) : seg(s), n_seg(n) {}
  __device__ __forceinline__ bool done() const { return i >= n_seg; }
  __device__ __forceinline__ const Segment& at() const { return seg[i]; }
  __device__ __forceinline__ int steps() const {
    return (seg[i].t1 - seg[i].t0) << (seg[i].dual ? 1 : 0);
  }
  __device__ __forceinline__ int tile() const { return seg[i].t0 + (seg[i].dual ? j >> 1 : j); }
  __device__ __forceinline__ bool loads() const { return !(seg[i].dual && (j & 1)); }   // a new tile
  __device__ __forceinline__ bool frees() const { return !seg[i].dual || (j & 1); }     // its last use
  __device__ __forceinline__ bool first() const { return j == 0; }
  __device__ __forceinline__ bool last() const { return j == steps() - 1; }
  __device__ __forceinline__ bool first_of_stream() const { return j < 2; }
  __device__ __forceinline__ bool last_of_stream() const { return j >= steps() - 2; }
  __device__ __forceinline__ void next() {
    if (++j == steps()) {
      j = 0;
      ++i;
    }
  }
};

// Where a segment's query rows lie: half s in slot s, or, when one tile of rows
// serves both streams, slot (segment & 1).
__device__ __forceinline__ int q_slot(const Walk& w, int stream) {
  return w.at().dual ? stream : (w.i & 1);
}

// ------------------------------------------------------------------ list --
// Sums of up to four numbers over lower threads; *total gets those of all.
__device__ void scan4(Block& s, const long long* v, long long* below, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    inc[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(kFull, inc[i], o);
      if (lane >= o) inc[i] += up;
    }
  }
  __syncthreads();
  if (lane == 31)
    for (int i = 0; i < 4; ++i) s.scan[warp][i] = inc[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    long long base = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) base = all;
      all += s.scan[w][i];
    }
    below[i] = base + inc[i] - v[i];
    total[i] = all;
  }
}

// Fills s.seg with segments [skip, skip + kMaxSegments) of this block's
// stretch.  `tmp` is shared memory of 3 B + 2 (n_groups + 1) words, idle now.
__device__ void list_segments(Block& s, const AttnParams& p, int32_t* tmp, int skip) {
  int32_t* gs = tmp;                               // [n_groups + 1]
  int32_t* pl = gs + p.n_groups + 1;               // [n_groups]
  int32_t* seen = pl + p.n_groups + 1;             // [B]
  int32_t* group = seen + p.B;                     // [B]; -1: none
  int32_t* most = group + p.B;                     // [B]: prefix tokens that a leader's unit sees
  const int limit = p.max_pages * kPageTokens;
  for (int i = threadIdx.x; i <= p.n_groups; i += kThreads) {
    gs[i] = __ldg(p.group_start + i);
    if (i < p.n_groups) pl[i] = min(max(__ldg(p.prefix_lens + i), 0), limit);
  }
  __syncthreads();
  const bool teller = blockIdx.x == 0 && skip == 0;
  if (teller) {
    for (int i = threadIdx.x; i < p.n_groups; i += kThreads) {
      if (gs[i] < 0 || gs[i] > gs[i + 1] || gs[i + 1] > p.B)
        report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, i, gs[i + 1], p.B);
      const int len = __ldg(p.prefix_lens + i);
      if (len != pl[i]) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, i, len, limit);
    }
  }
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int pos = __ldg(p.positions + b);
    int n = pos + 1;
    if (pos < 0) n = 0;
    if (pos < -1 || pos >= limit) {
      if (teller) report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, b, pos, limit);
      n = 0;
    }
    int g = -1;
    if (p.n_groups > 0) {
      int lo = 0, hi = p.n_groups;                 // last group that starts at or before b
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (gs[mid] <= b) lo = mid;
        else hi = mid;
      }
      if (gs[lo] >= 0 && gs[lo] <= b && b < gs[lo + 1]) g = lo;
    }
    seen[b] = n;
    group[b] = g;
    most[b] = 0;
  }
  __syncthreads();
  const int span = 2 * p.MB;                       // entries of a prefix unit
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const int g = group[b];
    if (g >= 0) {
      const int lead = b - (b - gs[g]) % span;
      if (group[lead] == g) atomicMax(&most[lead], min(seen[b], pl[g]));
    }
  }
  __syncthreads();
  // this thread's entries: places of their tiles in the line
  const int per = (p.B + kThreads - 1) / kThreads;
  const int e0 = min(p.B, (int)threadIdx.x * per), e1 = min(p.B, e0 + per);
  auto prefix_tiles = [&](int b) { return (most[b] + kTile - 1) / kTile; };
  auto own_first = [&](int b) { return pl[group[b]] / kPageTokens * kPageTokens; };
  auto own_tiles = [&](int b) {
    const int g = group[b];
    if (g < 0 || seen[b] <= pl[g]) return 0;
    return (seen[b] - own_first(b) + kTile - 1) / kTile;
  };
  long long v[4] = {0, 0, 0, 0}, below[4], total[4];
  for (int b = e0; b < e1; ++b) {
    v[0] += (long long)prefix_tiles(b) * p.Hkv;
    v[1] += (long long)own_tiles(b) * p.Hkv;
  }
  scan4(s, v, below, total);
  const long long all = total[0] + total[1];
  const long long blocks = max(1ll, min((long long)gridDim.x, all));
  if (teller) {
    const Table tab{p.tab, p.B};
    if (threadIdx.x == 0) {
      tab.total() = all;
      tab.blocks() = blocks;
    }
    long long pa = below[0], oa = total[0] + below[1];
    for (int b = e0; b < e1; ++b) {
      const int g = group[b];
      const int np = prefix_tiles(b), no = own_tiles(b);
      tab.prefix_at(b) = pa;
      tab.own_at(b) = oa;
      tab.prefix_tiles(b) = np;
      tab.own_tiles(b) = no;
      tab.leader(b) = g < 0 ? -1 : b - (b - gs[g]) % span;
      pa += (long long)np * p.Hkv;
      oa += (long long)no * p.Hkv;
    }
  }
  long long r0 = 0, r1 = 0;
  if (all > 0 && (long long)blockIdx.x < blocks) {
    r0 = stretch(blockIdx.x, all, blocks);
    r1 = stretch(blockIdx.x + 1, all, blocks);
  }
  // count this thread's segments, then write them at their places
  auto visit = [&](auto&& emit) {
    long long at = below[0];
    for (int b = e0; b < e1; ++b) {
      const int nt = prefix_tiles(b);
      const long long end = at + (long long)nt * p.Hkv;
      if (nt > 0 && end > r0 && at < r1) {
        for (int h = (int)max(0ll, (r0 - at) / nt); h < p.Hkv; ++h) {
          const long long us = at + (long long)h * nt;
          if (us >= r1) break;
          const int t0 = (int)max(0ll, r0 - us), t1 = (int)min((long long)nt, r1 - us);
          if (t1 > t0) emit(true, b, h, nt, t0, t1);
        }
      }
      at = end;
    }
    at = total[0] + below[1];
    for (int b = e0; b < e1; ++b) {
      const int nt = own_tiles(b);
      const long long end = at + (long long)nt * p.Hkv;
      if (nt > 0 && end > r0 && at < r1) {
        for (int h = (int)max(0ll, (r0 - at) / nt); h < p.Hkv; ++h) {
          const long long us = at + (long long)h * nt;
          if (us >= r1) break;
          const int t0 = (int)max(0ll, r0 - us), t1 = (int)min((long long)nt, r1 - us);
          if (t1 > t0) emit(false, b, h, nt, t0, t1);
        }
      }
      at = end;
    }
  };
  long long n[4] = {0, 0, 0, 0}, nb[4], nt_all[4];
  visit([&](bool prefix, int, int, int, int, int) { n[prefix ? 0 : 1] += 1; });
  scan4(s, n, nb, nt_all);
  long long place[2] = {nb[0], nt_all[0] + nb[1]};
  const int total_seg = (int)(nt_all[0] + nt_all[1]);
  if (threadIdx.x == 0) {
    s.total_seg = total_seg;
    s.n_seg = min(kMaxSegments, total_seg - skip);
  }
  visit([&](bool prefix, int b, int h, int nt, int t0, int t1) {
    const long long at = place[prefix ? 0 : 1]++ - skip;
    if (at < 0 || at >= kMaxSegments) return;
    const int g = group[b];
    Segment& q = s.seg[at];
    q.head = h;
    q.b0 = b;
    q.t0 = t0;
    q.t1 = t1;
    if (prefix) {
      q.nmem = min(min(span, gs[g + 1] - b), p.B - b);
      q.row = gs[g];
      q.tok0 = 0;
      q.lo = 0;
      q.hi = most[b];
      q.limit = pl[g];
    } else {
      q.nmem = 1;
      q.row = b;
      q.tok0 = own_first(b);
      q.lo = pl[g];
      q.hi = seen[b];
      q.limit = seen[b];
    }
    q.dual = q.nmem > p.MB;
    const bool whole = t0 == 0 && t1 == nt;
    q.slot = whole ? (prefix ? -1 : -2) : 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
  });
  __syncthreads();
  if (threadIdx.x == 0) {
    int steps = 0;
    for (int i = 0; i < s.n_seg; ++i) steps += (s.seg[i].t1 - s.seg[i].t0) << (s.seg[i].dual ? 1 : 0);
    s.n_steps = steps;
  }
  __syncthreads();
}

// Whether a tile has tokens inside its loaded pages that nobody may see: what
// lies there is not the sequence's, and 0 x infinity would spoil the row.
__device__ __forceinline__ bool ragged(const Segment& q, int tile) {
  const int a = q.tok0 + tile * kTile;
  return a < q.lo || a + kTile > q.hi;
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
  if (sb & 1023) {                   // the swizzled tiles would not line up
    report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, -1, (int)sb, 1024);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b_full = saddr(s.bars.full), b_empty = saddr(s.bars.empty);
  const uint32_t b_qfull = saddr(s.bars.q_full), b_qempty = saddr(s.bars.q_empty);
  const uint32_t b_sfull = saddr(s.bars.s_full), b_pready = saddr(s.bars.p_ready);
  const uint32_t b_ofull = saddr(s.bars.o_full), b_ofree = saddr(s.bars.o_free);
  const uint32_t b_ml = saddr(s.bars.ml_full);

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_qfull + 8 * i, 1);
      mbar_init(b_qempty + 8 * i, 1);
      mbar_init(b_sfull + 8 * i, 1);
      mbar_init(b_pready + 8 * i, kGroupThreads);
      mbar_init(b_ofull + 8 * i, 1);
      mbar_init(b_ofree + 8 * i, kGroupThreads);
      mbar_init(b_ml + 8 * i, kGroupThreads);
    }
    s.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     saddr(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = s.tmem;
  const uint32_t tm_s[2] = {tm, tm + 128}, tm_o[2] = {tm + 256, tm + 384};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Barrier use counts, carried from pass to pass by every role that needs them.
  uint32_t ring = 0;                 // tiles loaded so far
  uint32_t qn[2] = {0, 0};           // uses of each query slot
  uint32_t sn[2] = {0, 0};           // steps of each stream
  uint32_t on[2] = {0, 0};           // segments of each stream
  uint32_t mln[2] = {0, 0};          // hand-overs of each stream
  bool ok = true;

  for (int skip = 0;; skip += kMaxSegments) {
    list_segments(s, p, reinterpret_cast<int32_t*>(base + L::kRing), skip);
    const int n_seg = s.n_seg, n_steps = s.n_steps;
    // the list's scratch is the ring: later writes there go through TMA
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();

    if (warp == kTmaWarp) {
      // -------------------------------------------------------- loads -----
      // lane i of `kp` holds the physical page of the segment's page i + base
      struct Pages {
        int seg = -1, first = 0, id = 0;
      } kc, vc;
      auto page = [&](Pages& c, const Walk& w, int index) {
        const Segment& q = w.at();
        if (c.seg != w.i || index < c.first || index >= c.first + 32) {
          c.seg = w.i;
          c.first = index;
          const int lp = index + lane;
          int id = p.n_pages;                     // beyond the pool: loads as zeros
          if (lp < p.max_pages && lp * kPageTokens < q.hi) {
            id = __ldg(p.page_table + (size_t)q.row * p.max_pages + lp);
            if (id < 0 || id >= p.n_pages) {
              report(p.status, MK_ERR_DEVICE, MK_OP_PREFIX_ATTENTION, q.row, id, p.n_pages);
              id = p.n_pages;
            }
          }
          c.id = id;
        }
        return __shfl_sync(kFull, c.id, index - c.first);
      };
      auto load_tile = [&](Pages& c, const Walk& w, const void* map) {
        const Segment& q = w.at();
        const int first = (q.tok0 + w.tile() * kTile) / kPageTokens;
        const int id0 = page(c, w, first), id1 = page(c, w, first + 1);
        const uint32_t st = ring % L::kStages, bar = b_full + 8 * st;
        if (ring >= L::kStages) ok = ok && wait(s, b_empty + 8 * st, (ring / L::kStages - 1) & 1, p);
        ok = __all_sync(kFull, ok);
        if (ok && lane == 0) {
          mbar_expect(bar, L::kTileBytes);
          const uint32_t dst = sb + L::kRing + st * L::kTileBytes;
          const int y0 = (id0 * p.Hkv + q.head) * kPageTokens;
          const int y1 = (id1 * p.Hkv + q.head) * kPageTokens;
#pragma unroll
          for (int c2 = 0; c2 < L::kChunks; ++c2) {
            tma_3d(dst + c2 * kTile * 128, map, 0, y0, c2, bar);
            tma_3d(dst + c2 * kTile * 128 + kPageTokens * 128, map, 0, y1, c2, bar);
          }
        }
        __syncwarp();
        ++ring;
      };
      auto load_q = [&](const Walk& w) {
        const Segment& q = w.at();
        for (int h = 0; h < (q.dual ? 2 : 1); ++h) {
          const int sl = q_slot(w, h);
          if (qn[sl] > 0) ok = ok && wait(s, b_qempty + 8 * sl, (qn[sl] - 1) & 1, p);
          ok = __all_sync(kFull, ok);
          if (ok && lane == 0) {
            const bool one = q.nmem == 1;
            const int rows = one ? p.G : p.G * p.MB;
            mbar_expect(b_qfull + 8 * sl, (uint32_t)rows * HD * 2);
            const uint32_t dst = sb + L::kQ + sl * L::kTileBytes;
#pragma unroll
            for (int c2 = 0; c2 < L::kChunks; ++c2)
              tma_4d(dst + c2 * kRows * 128, one ? &qmap_one : &qmap, 0, q.head * p.G,
                     q.b0 + h * p.MB, c2, b_qfull + 8 * sl);
          }
          __syncwarp();
          qn[sl] += 1;
        }
      };
      Walk k(s.seg, n_seg), v(s.seg, n_seg);
      auto do_k = [&]() {
        if (k.first()) load_q(k);
        if (k.loads()) load_tile(kc, k, &kmap);
        k.next();
      };
      for (int i = 0; i < 2 && i < n_steps && ok; ++i) do_k();
      for (int n = 0; n < n_steps && ok; ++n) {
        if (v.loads()) load_tile(vc, v, &vmap);
        v.next();
        if (ok && n + 2 < n_steps) do_k();
      }
    } else if (warp == kMmaWarp) {
      // --------------------------------------------------------- MMAs -----
      if (lane == 0) {
        const uint32_t fmt = (1u << 4) | (Half<T>::kFormat << 7) | (Half<T>::kFormat << 10) |
                             ((uint32_t)(kRows >> 4) << 24);
        const uint32_t id_qk = fmt | ((uint32_t)(kTile >> 3) << 17);
        const uint32_t id_pv = fmt | (1u << 16) | ((uint32_t)(HD >> 3) << 17);
        Walk k(s.seg, n_seg), v(s.seg, n_seg);
        uint32_t k_st = 0, v_st = 0;
        int kstep = 0;
        auto do_k = [&]() {
          const int st = kstep & 1;
          const int sl = q_slot(k, st);
          if (k.loads()) {
            k_st = ring % L::kStages;
            ok = ok && wait(s, b_full + 8 * k_st, (ring / L::kStages) & 1, p);
            ++ring;
          }
          if (k.first()) {
            const int n = k.at().dual ? 2 : 1;
            for (int h = 0; h < n; ++h) {
              const int s2 = q_slot(k, h);
              ok = ok && wait(s, b_qfull + 8 * s2, qn[s2] & 1, p);
              qn[s2] += 1;
            }
          }
          if (!ok) return;
          tc_after();
          const uint32_t qa = sb + L::kQ + sl * L::kTileBytes;
          const uint32_t ka = sb + L::kRing + k_st * L::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kRows * 128 + (kk & 3) * 32;
            mma_ss(tm_s[st], desc_of(qa + off, 16), desc_of(ka + off, 16), id_qk, kk > 0);
          }
          tc_commit(b_sfull + 8 * st);
          if (k.frees()) tc_commit(b_empty + 8 * k_st);
          // the segment's last use of a slot
          if (k.at().dual ? k.last_of_stream() : k.last()) tc_commit(b_qempty + 8 * sl);
          k.next();
          ++kstep;
        };
        for (int i = 0; i < 2 && i < n_steps && ok; ++i) do_k();
        for (int n = 0; n < n_steps && ok; ++n) {
          const int st = n & 1;
          if (v.loads()) {
            v_st = ring % L::kStages;
            ok = ok && wait(s, b_full + 8 * v_st, (ring / L::kStages) & 1, p);
            ++ring;
          }
          if (v.first_of_stream() && on[st] > 0) ok = ok && wait(s, b_ofree + 8 * st, (on[st] - 1) & 1, p);
          ok = ok && wait(s, b_pready + 8 * st, sn[st] & 1, p);
          if (!ok) break;
          sn[st] += 1;
          tc_after();
          const uint32_t va = sb + L::kRing + v_st * L::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(tm_o[st], tm_s[st] + kk * 8, desc_of(va + kk * 16 * 128, kTile * 128), id_pv,
                   !(v.first_of_stream() && kk == 0));
          if (v.frees()) tc_commit(b_empty + 8 * v_st);
          if (v.last_of_stream()) {
            tc_commit(b_ofull + 8 * st);
            on[st] += 1;
          }
          v.next();
          if (n + 2 < n_steps) do_k();
        }
      }
      ok = __all_sync(kFull, ok);
    } else {
      // ------------------------------------------------------ softmax -----
      const int st = warp >> 2;                        // stream
      const int r = threadIdx.x & (kGroupThreads - 1); // row
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 lanes
      const uint32_t ts = tm_s[st] + lanes;
      Walk w(s.seg, n_seg);
      uint32_t kloads = 0, vloads = 0;                 // among the steps so far
      float m = -INFINITY, l = 0.0f;
      bool real = false, busy = false;
      int lim = 0;
      for (int n = 0; n < n_steps && ok; ++n) {
        const Segment& q = w.at();
        if (w.loads()) {
          ++kloads;
          ++vloads;
        }
        if (w.first()) {
          // this thread's row of the segment
          const int j = r / p.G, e = (q.dual ? st * p.MB : 0) + j;
          real = j < p.MB && e < q.nmem;
          busy = __any_sync(kFull, real);
          lim = INT32_MAX;
          if (real) {
            const int pos = __ldg(p.positions + q.b0 + e);
            lim = min(pos < 0 || pos >= p.max_pages * kPageTokens ? 0 : pos + 1, q.limit);
          }
        }
        if ((n & 1) != st) {
          if (!w.last()) {
            w.next();
            continue;
          }
        }
        if ((n & 1) == st) {
          if (w.first_of_stream()) {
            m = -INFINITY;
            l = 0.0f;
          }
          const int a = q.tok0 + w.tile() * kTile;
          if (ragged(q, w.tile())) {
            // clear V's rows of tokens that are not the unit's.  The tile's
            // place in the ring: behind the V tiles so far and the K tiles of
            // the steps up to the one after that which loaded it.
            Walk nx = w;
            nx.next();
            const uint32_t ahead = w.loads() && !nx.done() && nx.loads() ? 1 : 0;
            const uint32_t at = ring + kloads + ahead + vloads - 1;
            const uint32_t vs = at % L::kStages;
            ok = wait(s, b_full + 8 * vs, (at / L::kStages) & 1, p);
            if (ok) {
              const uint32_t va = sb + L::kRing + vs * L::kTileBytes;
              for (int i = r; i < kTile * L::kChunks * 8; i += kGroupThreads) {
                const int tok = a + ((i >> 3) & (kTile - 1));
                if (tok < q.lo || tok >= q.hi)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(va + i * 16), "r"(0)
                               : "memory");
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
          }
          ok = ok && wait(s, b_sfull + 8 * st, sn[st] & 1, p);
          if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
          }
          sn[st] += 1;
          if (busy) {
            tc_after();
            uint32_t x[kTile];
#pragma unroll
            for (int i = 0; i < kTile; i += 32) tmem_ld32(ts + i, x + i);
            tmem_wait_ld();
            float* f = reinterpret_cast<float*>(x);
            if (__any_sync(kFull, a < q.lo || a + kTile > lim)) {
              const int from = q.lo - a, to = lim - a;
#pragma unroll
              for (int i = 0; i < kTile; ++i)
                if (i < from || i >= to) f[i] = -INFINITY;
            }
            float mx[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
            for (int i = 4; i < kTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], f[i]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
            const bool grow = top > m + kRescale;      // also the first score of a row
            if (__any_sync(kFull, grow)) {
              const float m_new = grow ? top : m;
              const float f_old = m == m_new ? 1.0f : ex2(m - m_new);
              l *= f_old;
              m = m_new;
              if (!w.first_of_stream()) {
                // S of this step was committed after P V of the stream's last
                // one, so O is at rest
                const uint32_t to = tm_o[st] + lanes;
#pragma unroll 1
                for (int i = 0; i < HD; i += 32) {
                  uint32_t o[32];
                  tmem_ld32(to + i, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int k2 = 0; k2 < 32; ++k2)
                    o[k2] = __float_as_uint(__uint_as_float(o[k2]) * f_old);
                  tmem_st32(to + i, o);
                }
              }
            }
            const float ref = (m == -INFINITY ? 0.0f : m) - Half<T>::kShift;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kTile; i += 2) {
              const float pa = ex2(fmaf(f[i], p.c, -ref)), pb = ex2(fmaf(f[i + 1], p.c, -ref));
              sum[i & 2] += pa;
              sum[(i & 2) + 1] += pb;
              x[i >> 1] = Half<T>::pack(pa, pb);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st32(ts, x);
            tmem_st32(ts + 32, x + 32);
            tmem_wait_st();
            tc_before();
          }
          mbar_arrive(b_pready + 8 * st);
        }
        if (w.last()) {
          // ------------------------------------------- the segment's end --
          const int steps = w.steps();
          const bool mine = q.dual || steps >= 2 || (n & 1) == st;   // this stream took part
          const bool both = !q.dual && steps >= 2;
          const bool owner = q.dual || (n & 1) == st;
          float m2 = -INFINITY, l2 = 0.0f;
          if (mine && !owner) {
            // hand (m, l) over; the other group reads O.  Its reading of the
            // last hand-over is behind the o_free of that segment.
            if (on[st] > 0) ok = wait(s, b_ofree + 8 * st, (on[st] - 1) & 1, p);
            if (!__all_sync(kFull, ok)) {
              ok = false;
              break;
            }
            s.ml[r] = make_float2(m, l);
            mbar_arrive(b_ml + 8 * st);
          }
          if (owner) {
            ok = ok && wait(s, b_ofull + 8 * st, on[st] & 1, p);
            if (both) {
              ok = ok && wait(s, b_ofull + 8 * (st ^ 1), on[st ^ 1] & 1, p);
              ok = ok && wait(s, b_ml + 8 * (st ^ 1), mln[st ^ 1] & 1, p);
              if (ok) {
                const float2 t = s.ml[r];
                m2 = t.x;
                l2 = t.y;
              }
            }
            if (!__all_sync(kFull, ok)) {
              ok = false;
              break;
            }
            if (busy) {
              tc_after();
              const float mm = fmaxf(m, m2);
              const float f1 = m == mm ? 1.0f : ex2(m - mm), f2 = m2 == -INFINITY ? 0.0f : ex2(m2 - mm);
              float* dst = nullptr;
              if (real) {
                const int j = r / p.G, e = (q.dual ? st * p.MB : 0) + j;
                const int b = q.b0 + e, hq = q.head * p.G + r % p.G;
                const size_t row = q.slot >= 0
                                       ? ((size_t)q.slot * 2 + (q.dual ? st : 0)) * kRows + r
                                       : (size_t)p.n_slots * 2 * kRows +
                                             ((size_t)(-1 - q.slot) * p.B + b) * p.Hq + hq;
                dst = p.part + row * HD;
                p.part_ml[row] = make_float2((mm == -INFINITY ? 0.0f : mm) - Half<T>::kShift,
                                             l * f1 + l2 * f2);
              }
#pragma unroll 1
              for (int i = 0; i < HD; i += 32) {
                uint32_t o[32];
                tmem_ld32(tm_o[st] + lanes + i, o);
                tmem_wait_ld();
                float* of = reinterpret_cast<float*>(o);
#pragma unroll
                for (int k2 = 0; k2 < 32; ++k2) of[k2] *= f1;
                if (both) {
                  uint32_t o2[32];
                  tmem_ld32(tm_o[st ^ 1] + lanes + i, o2);
                  tmem_wait_ld();
#pragma unroll
                  for (int k2 = 0; k2 < 32; ++k2) of[k2] = fmaf(__uint_as_float(o2[k2]), f2, of[k2]);
                }
                if (real) {
#pragma unroll
                  for (int k2 = 0; k2 < 32; k2 += 4)
                    *reinterpret_cast<float4*>(dst + i + k2) =
                        make_float4(of[k2], of[k2 + 1], of[k2 + 2], of[k2 + 3]);
                }
              }
              tc_before();
            }
            mbar_arrive(b_ofree + 8 * st);
            if (both) mbar_arrive(b_ofree + 8 * (st ^ 1));
          }
          // both groups keep both streams' counts
          for (int t = 0; t < 2; ++t) {
            const bool took = q.dual || steps >= 2 || (n & 1) == t;
            if (took) on[t] += 1;
            if (both && (n & 1) != t) mln[t] += 1;
          }
        }
        w.next();
      }
      // the other roles' ring count
      ring += kloads + vloads;
    }
    __syncthreads();
    ok = ok && *(volatile int*)&s.abort == 0;
    if (!ok || skip + kMaxSegments >= s.total_seg) break;
    __syncthreads();
  }

  // A wait that ran out may have left copies and MMAs in flight: give them time.
  if (*(volatile int*)&s.abort) {
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

// Adds up a row's partial results: prefix shares, then shares of its own
// tokens, in the order of their blocks.  One warp per (entry, query head),
// HD / 32 columns per lane.
template <typename T, int HD>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int C = HD / 32;
  const int row = (int)((blockIdx.x * 128u + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= p.B * p.Hq) return;
  const int b = row / p.Hq, hq = row % p.Hq, h = hq / p.G;
  const Table tab{p.tab, p.B};
  const int lead = tab.leader(b);
  if (lead < 0) return;
  const long long total = tab.total(), blocks = tab.blocks();
  float acc[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) acc[i] = 0.0f;
  for (int kind = 0; kind < 2; ++kind) {
    const int nt = kind == 0 ? tab.prefix_tiles(lead) : tab.own_tiles(b);
    if (nt == 0) continue;
    const long long at = (kind == 0 ? tab.prefix_at(lead) : tab.own_at(b)) + (long long)h * nt;
    const int c0 = block_of(at, total, blocks), c1 = block_of(at + nt - 1, total, blocks);
    // the row's place among its unit's rows
    const int j = kind == 0 ? b - lead : 0;
    const int stream = j / p.MB, r = (j % p.MB) * p.G + hq % p.G;
    for (int c = c0; c <= c1; c += 32) {
      // lane i looks at block c + i's share
      const int n = min(32, c1 - c + 1), mine = c + min(lane, n - 1);
      const size_t at_row =
          c0 == c1 ? (size_t)p.n_slots * 2 * kRows + ((size_t)kind * p.B + b) * p.Hq + hq
                   : ((size_t)(2 * mine + (mine == c0 ? 1 : 0)) * 2 + stream) * kRows + r;
      const float2 ml = p.part_ml[at_row];
      // a share that saw nothing has l = 0 (and O = 0): no weight
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
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const float fi = __shfl_sync(kFull, f, i);
        l = fmaf(__shfl_sync(kFull, ml.y, i), fi, l);
        const float* src = p.part + __shfl_sync(kFull, (unsigned long long)at_row, i) * HD + lane * C;
        if constexpr (C == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          acc[0] = fmaf(v.x, fi, acc[0]);
          acc[1] = fmaf(v.y, fi, acc[1]);
          acc[2] = fmaf(v.z, fi, acc[2]);
          acc[3] = fmaf(v.w, fi, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          acc[0] = fmaf(v.x, fi, acc[0]);
          acc[1] = fmaf(v.y, fi, acc[1]);
        }
      }
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // NaN stays
  uint32_t o[C / 2];
#pragma unroll
  for (int i = 0; i < C; i += 2) o[i / 2] = Half<T>::pack(acc[i] * inv, acc[i + 1] * inv);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + (size_t)row * HD + lane * C);
#pragma unroll
  for (int i = 0; i < C / 2; ++i) out[i] = o[i];
  if (p.lse && lane == 0) {
    p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
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

// Streaming multiprocessors of a device (looked up once per device).
int sm_count(int device) {
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static int count[kMaxDevices];
  if (device < 0 || device >= kMaxDevices) return 0;
  std::call_once(once[device], [&] {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) == cudaSuccess) count[device] = n;
  });
  return count[device];
}

constexpr int kMaxBlocks = 160;      // at least the device's multiprocessors

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

size_t part_rows(const mk_prefix_attention_args* a) {
  return (size_t)2 * kMaxBlocks * 2 * kRows + (size_t)2 * a->batch * a->n_q_heads;
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
  // row numbers of the pools' tensor maps are 32-bit
  if (((long long)a->n_pages + 1) * a->n_kv_heads * kPageTokens > INT32_MAX) return MK_ERR_CAPACITY;
  return MK_OK;
}

template <typename T, int HD>
cudaError_t launch_attention(const AttnParams& p, const CUtensorMap* maps, int blocks, cudaStream_t st) {
  using L = Layout<HD>;
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<T, HD>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kDyn);
  if (e != cudaSuccess) return e;
  attention_kernel<T, HD><<<blocks, kThreads, L::kDyn, st>>>(p, maps[0], maps[1], maps[2], maps[3]);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.B * p.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, HD>, p);
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" size_t mk_prefix_attention_workspace(const mk_prefix_attention_args* a) {
  using namespace mk::ops;
  if (validate(a) != MK_OK) return 0;
  const size_t rows = part_rows(a);
  return round256(rows * a->head_dim * sizeof(float)) + round256(rows * sizeof(float2)) +
         round256(table_bytes(a->batch));
}

extern "C" mk_status mk_prefix_attention(const mk_prefix_attention_args* a, void* stream) {
  using namespace mk::ops;
  mk_status s = validate(a);
  if (s != MK_OK) return s;
  if (a->batch == 0 || a->n_groups == 0) return MK_OK;
  if (!a->q || !a->k_pool || !a->v_pool || !a->page_table || !a->positions || !a->group_start ||
      !a->prefix_lens || !a->out || !a->workspace)
    return MK_ERR_INVALID;
  const long long row = (long long)a->n_q_heads * a->head_dim;
  if (a->q_token_stride % 8 || (a->batch > 1 && a->q_token_stride < row)) return MK_ERR_INVALID;
  if (!aligned(a->q, 16) || !aligned(a->k_pool, 16) || !aligned(a->v_pool, 16) ||
      !aligned(a->out, 16) || !aligned(a->workspace, 256))
    return MK_ERR_INVALID;
  if (a->workspace_bytes < mk_prefix_attention_workspace(a)) return MK_ERR_CAPACITY;
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
  p.tab = reinterpret_cast<long long*>(w);
  p.n_slots = 2 * kMaxBlocks;
  p.out = a->out;
  p.lse = a->lse;
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
    const long long ts = a->batch > 1 ? a->q_token_stride : row;
    const cuuint64_t dims[4] = {64, (cuuint64_t)a->n_q_heads, (cuuint64_t)a->batch, hd / 64};
    const cuuint64_t strides[3] = {hd * 2, (cuuint64_t)ts * 2, 128};
    cuuint32_t box[4] = {64, (cuuint32_t)p.G, (cuuint32_t)p.MB, 1};
    if (!encode(&maps[2], type, 4, a->q, dims, strides, box)) return MK_ERR_INVALID;
    box[2] = 1;
    if (!encode(&maps[3], type, 4, a->q, dims, strides, box)) return MK_ERR_INVALID;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->type == MK_BF16)
    e = a->head_dim == 128 ? launch_attention<__nv_bfloat16, 128>(p, maps, blocks, st)
                           : launch_attention<__nv_bfloat16, 64>(p, maps, blocks, st);
  else
    e = a->head_dim == 128 ? launch_attention<__half, 128>(p, maps, blocks, st)
                           : launch_attention<__half, 64>(p, maps, blocks, st);
  return from_cuda(e);
}
