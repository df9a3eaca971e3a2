// ops_append.cu -- keys rotated and written, with their values, into the
// paged cache that the decode step reads; queries rotated on the way.
//
// For token t at position P with rotary_dim = 2 R, pair i < R of a query or
// key head turns by the angle P * inv_freq[i]:
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
// where the pair is columns (i, R + i), or (2 i, 2 i + 1) when interleaved;
// columns from rotary_dim on are copied.  The angle is formed and brought
// into [-pi, pi] in 64 bits, since at position 2^18 one 32-bit rounding step
// of the angle is already 2^-6; the sine and cosine are then 32-bit.
//
// Bound: each row is read and written once, without reuse, so memory is the floor.
// What it is bound by now is the chain of a warp: its loads, its look-ups, its
// stores, with 24 warps on a multiprocessor (80 registers a thread).  A warp takes a token, or some heads of
// one: it asks for all its rows first (16 columns a lane and head, two 16-byte
// loads of 16-bit rows); while they are on their way it looks up the token's
// place and forms its sines and cosines, two a lane, which a lane then holds in
// registers for all its heads.  No warp waits for another.  8192 tokens of 24
// heads of 128 in bf16 take 21.3 us (4.7 TB/s; memory is 31 % busy, as most of what
// is written stays in the L2 cache, and the multiprocessors 44 %), 16381 in fp16 with
// half of each head rotated 37.1 us (5.4 TB/s, 84 % of a plain copy), 8192 in fp32 27.0
// us (5.6 TB/s); single tokens are bound by the launch.
#include "ops_common.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

struct AppendParams {
  int T, rows, max_pages, n_pages, Hq, Hkv, R;
  int splits, rounds;        // warps of a token, and how many times each turns the heads it can at once
  int blocks;
  float magnitude;
  const void *q, *k, *v;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;   // strides in elements
  void *q_out, *k_pool, *v_pool;
  const double* inv_freq;
  const int32_t *positions, *seq, *page_table;
  int32_t* status;
};

// cos and sin of position * f, times magnitude: the angle in turns, less the
// nearest whole number, in 64 bits.
__device__ __forceinline__ float2 turn(int position, double f, float magnitude) {
  const double a = (double)position * f * 0.15915494309189535;   // 1 / (2 pi)
  float s, c;
  sincospif((float)(2.0 * (a - rint(a))), &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

// Rounds whose rows a lane holds at once: 8 registers each of 16-bit rows, 16
// of 32-bit ones.  (8192 tokens of 24 heads of 128: 21.5 us with 6 rounds, 21.4
// with 4, 21.1 with 2; a block of 256 threads that kept its tokens' sines in
// shared memory for all heads took 27.1, with the next tokens' rows under way 27.6.)
template <typename S>
constexpr int kMostRounds = sizeof(S) == 4 ? 2 : 4;
// Up to so many single rounds (32 warps on each of 148 multiprocessors) every
// warp takes one: there is room for them, and the chain of a warp is shortest.
constexpr long long kFewWarps = 148 * 32;

// 16 elements as they lie in memory: two groups of 8.
template <typename S>
struct Raw {
  uint4 w[sizeof(S)];
};

template <typename S, bool WIDE>
__device__ __forceinline__ void load8(const S* p, uint4* w) {
  if constexpr (WIDE) {              // the address is 16-byte aligned
#pragma unroll
    for (int i = 0; i < (int)sizeof(S) / 2; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  } else {
    S* e = reinterpret_cast<S*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
}
template <typename S>
__device__ __forceinline__ void unpack16(const Raw<S>& r, float* x) {
  if constexpr (sizeof(S) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(r.w[i].x);
      x[4 * i + 1] = __uint_as_float(r.w[i].y);
      x[4 * i + 2] = __uint_as_float(r.w[i].z);
      x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
  } else {
    Vec8<S>::unpack(r.w[0], x);
    Vec8<S>::unpack(r.w[1], x + 8);
  }
}

// MODE 0: half layout, R a multiple of 8: the lane's two groups of 8 columns
// are the two halves of its 8 pairs.  MODE 1: interleaved: 16 consecutive
// columns.  MODE 2: half layout, any R: 16 consecutive columns whose partners,
// held by other lanes, are exchanged through shared memory, whose banks the 16
// columns of a lane share with other lanes': 8192 tokens with 100 of 128 columns
// rotated take 87 us, with 36 of them 53, where mode 0 takes 21.
template <typename S, typename D, int HD, int MODE, bool WIDE>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int PER_HEAD = HD / 16;          // lanes of a head
  constexpr int kHeads = 32 / PER_HEAD;      // heads that a warp turns at once
  constexpr int kAhead = kMostRounds<S>;
  // cos and sin of pair i; for MODE 0 and 1 the two of pairs 8 j + k, k even and
  // odd, at place (k / 2) PER_HEAD + j, so that lanes j read without bank conflicts
  __shared__ __align__(16) float2 s_tab[kWarps][HD / 2];
  __shared__ float s_rows[kWarps][MODE == 2 ? 512 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.R, heads = p.Hq + 2 * p.Hkv;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(unit / p.splits), part = (int)(unit - (long long)t * p.splits);
  const int j = lane % PER_HEAD, h0 = part * p.rounds * kHeads + lane / PER_HEAD;
  // where the lane's two groups of 8 columns start
  auto columns = [&](int head, int* c0, int* c1) {
    const bool paired = MODE == 0 && head < p.Hq + p.Hkv && 8 * j < R;
    *c0 = paired ? 8 * j : 16 * j;
    *c1 = paired ? R + 8 * j : 16 * j + 8;
  };
  // Nothing of the call's memory is touched before the kernels ahead are done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t >= p.T) return;
  const int pos = __ldg(p.positions + t), seq = p.seq ? __ldg(p.seq + t) : t;
  Raw<S> raw[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const int head = h0 + a * kHeads;
    if (a < p.rounds && head < heads) {
      const S* src = head < p.Hq ? static_cast<const S*>(p.q) + t * p.q_ts + head * p.q_hs
                     : head < p.Hq + p.Hkv
                         ? static_cast<const S*>(p.k) + t * p.k_ts + (head - p.Hq) * p.k_hs
                         : static_cast<const S*>(p.v) + t * p.v_ts + (head - p.Hq - p.Hkv) * p.v_hs;
      int c0, c1;
      columns(head, &c0, &c1);
      load8<S, WIDE>(src + c0, raw[a].w);
      load8<S, WIDE>(src + c1, raw[a].w + sizeof(S) / 2);
    }
  }
  // the token's place: a negative sequence is padding
  int page = -1;
  if (seq >= p.rows) {
    if (lane == 0) report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, seq, p.rows);
  } else if (seq >= 0) {
    if (pos < 0 || pos / kPageTokens >= p.max_pages) {
      if (lane == 0) report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, pos, p.max_pages * kPageTokens);
    } else {
      page = __ldg(p.page_table + (size_t)seq * p.max_pages + pos / kPageTokens);
      if (page < 0 || page >= p.n_pages) {
        if (lane == 0) report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, page, p.n_pages);
        page = -1;
      }
    }
  }
  if (page < 0) return;                      // the whole warp
#pragma unroll
  for (int i = lane; i < HD / 2; i += 32)
    if (i < R) s_tab[warp][MODE == 2 ? i : (i % 8 / 2 * PER_HEAD + i / 8) * 2 + i % 2] = turn(pos, __ldg(p.inv_freq + i), p.magnitude);
  __syncwarp();
  float2 cs[MODE == 2 ? 1 : 8];
  if constexpr (MODE != 2) {
    if (8 * j < R) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 two = reinterpret_cast<const float4*>(s_tab[warp])[k / 2 * PER_HEAD + j];
        cs[k] = make_float2(two.x, two.y);
        cs[k + 1] = make_float2(two.z, two.w);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const int head = h0 + a * kHeads;
    if (a >= p.rounds) break;                // the whole warp
    const bool in = head < heads, is_v = head >= p.Hq + p.Hkv;
    float x[16];
    unpack16(raw[a], x);
    if constexpr (MODE == 2) {
      __syncwarp();                          // the previous rows have been read
      float* row = s_rows[warp] + lane * 16;
#pragma unroll
      for (int k = 0; k < 16; ++k) row[k] = x[k];
      __syncwarp();
    }
    if (!in) continue;
    int c0, c1;
    columns(head, &c0, &c1);
    if (!is_v) {
      if constexpr (MODE == 2) {
        const float* row = s_rows[warp] + (lane - j) * 16;   // the head's
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int c = 16 * j + k;
          if (c < R) {
            const float2 w = s_tab[warp][c];
            x[k] = x[k] * w.x - row[c + R] * w.y;
          } else if (c < 2 * R) {
            const float2 w = s_tab[warp][c - R];
            x[k] = x[k] * w.x + row[c - R] * w.y;
          }
        }
      } else if (8 * j < R) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float& lo = MODE == 0 ? x[k] : x[2 * k];
          float& hi = MODE == 0 ? x[8 + k] : x[2 * k + 1];
          if (MODE == 0 || 8 * j + k < R) {
            const float a0 = lo, b0 = hi;
            lo = a0 * cs[k].x - b0 * cs[k].y;
            hi = b0 * cs[k].x + a0 * cs[k].y;
          }
        }
      }
    }
    D* dst;
    if (head < p.Hq) {
      dst = static_cast<D*>(p.q_out) + ((size_t)t * p.Hq + head) * HD;
    } else {
      const int h = is_v ? head - p.Hq - p.Hkv : head - p.Hq;
      dst = static_cast<D*>(is_v ? p.v_pool : p.k_pool) +
            (((size_t)page * p.Hkv + h) * kPageTokens + (pos & (kPageTokens - 1))) * HD;
    }
    *reinterpret_cast<uint4*>(dst + c0) = Vec8<D>::pack(x);
    *reinterpret_cast<uint4*>(dst + c1) = Vec8<D>::pack(x + 8);
  }
}

// A warp takes all heads of a token, as far as its registers hold them; while
// that gives the device fewer warps than it can run, as few as it turns at once.
// Returns the number of blocks.
long long share_out(AppendParams* p, int hd, bool wide_rows) {
  const int at_once = 32 / (hd / 16), most = wide_rows ? kMostRounds<float> : kMostRounds<__half>;
  const int rounds = (p->Hq + 2 * p->Hkv + at_once - 1) / at_once;
  p->splits = (long long)p->T * rounds <= kFewWarps ? rounds : (rounds + most - 1) / most;
  p->rounds = (rounds + p->splits - 1) / p->splits;
  return ((long long)p->T * p->splits + kWarps - 1) / kWarps;
}

template <typename S, typename D, int HD, int MODE, bool WIDE>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<S, D, HD, MODE, WIDE>, p);
}

template <typename S, typename D, int HD, int MODE>
cudaError_t pick_wide(const AppendParams& p, bool wide, cudaStream_t st) {
  return wide ? launch<S, D, HD, MODE, true>(p, st) : launch<S, D, HD, MODE, false>(p, st);
}

template <typename S, typename D, int HD>
cudaError_t pick_mode(const AppendParams& p, bool interleaved, bool wide, cudaStream_t st) {
  if (interleaved) return pick_wide<S, D, HD, 1>(p, wide, st);
  return p.R % 8 == 0 ? pick_wide<S, D, HD, 0>(p, wide, st) : pick_wide<S, D, HD, 2>(p, wide, st);
}

template <typename S, typename D>
cudaError_t pick_hd(const AppendParams& p, int hd, bool il, bool wide, cudaStream_t st) {
  return hd == 128 ? pick_mode<S, D, 128>(p, il, wide, st) : pick_mode<S, D, 64>(p, il, wide, st);
}

template <typename S>
cudaError_t pick_dst(const AppendParams& p, int dst, int hd, bool il, bool wide, cudaStream_t st) {
  return dst == MK_BF16 ? pick_hd<S, __nv_bfloat16>(p, hd, il, wide, st)
                        : pick_hd<S, __half>(p, hd, il, wide, st);
}

}  // namespace
}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_rope_append(const mk_rope_append_args* a, void* stream) {
  using namespace mk::ops;
  if (!a) return MK_ERR_INVALID;
  if (a->n_tokens < 0 || a->n_rows < 0 || a->max_pages < 1 || a->n_pages < 1) return MK_ERR_INVALID;
  if (a->n_q_heads < 0 || a->n_kv_heads < 1) return MK_ERR_INVALID;
  if (a->n_q_heads > 1024 || a->n_kv_heads > 1024) return MK_ERR_CAPACITY;
  if (a->max_pages > INT32_MAX / kPageTokens) return MK_ERR_CAPACITY;
  if (a->head_dim != 64 && a->head_dim != 128) return MK_ERR_INVALID;
  if (a->rotary_dim < 0 || a->rotary_dim > a->head_dim || a->rotary_dim % 2) return MK_ERR_INVALID;
  if (a->src_type != MK_BF16 && a->src_type != MK_FP16 && a->src_type != MK_FP32)
    return MK_ERR_INVALID;
  if (a->dst_type != MK_BF16 && a->dst_type != MK_FP16) return MK_ERR_INVALID;
  const bool with_q = a->n_q_heads > 0;
  if (!a->k || !a->v || !a->k_pool || !a->v_pool || !a->positions || !a->page_table)
    return MK_ERR_INVALID;
  if (with_q && (!a->q || !a->q_out)) return MK_ERR_INVALID;
  if (a->rotary_dim > 0 && !a->inv_freq) return MK_ERR_INVALID;
  if (!a->seq && a->n_tokens > a->n_rows) return MK_ERR_INVALID;
  if (!aligned(a->k_pool, 16) || !aligned(a->v_pool, 16) || (with_q && !aligned(a->q_out, 16)))
    return MK_ERR_INVALID;
  const size_t es = a->src_type == MK_FP32 ? 4 : 2;
  if (!aligned(a->k, es) || !aligned(a->v, es) || (with_q && !aligned(a->q, es)))
    return MK_ERR_INVALID;
  AppendParams p{};
  p.T = a->n_tokens;
  p.rows = a->n_rows;
  p.max_pages = a->max_pages;
  p.n_pages = a->n_pages;
  p.Hq = a->n_q_heads;
  p.Hkv = a->n_kv_heads;
  p.R = a->rotary_dim / 2;
  const long long blocks = share_out(&p, a->head_dim, es == 4);
  if (blocks > INT32_MAX) return MK_ERR_CAPACITY;   // of a grid
  p.blocks = (int)blocks;
  DeviceGuard guard(a->device);
  if (guard.status() != MK_OK) return guard.status();
  if (a->n_tokens == 0) return MK_OK;
  p.magnitude = a->magnitude;
  p.q = a->q; p.k = a->k; p.v = a->v;
  p.q_ts = a->q_token_stride; p.q_hs = a->q_head_stride;
  p.k_ts = a->k_token_stride; p.k_hs = a->k_head_stride;
  p.v_ts = a->v_token_stride; p.v_hs = a->v_head_stride;
  p.q_out = a->q_out; p.k_pool = a->k_pool; p.v_pool = a->v_pool;
  p.inv_freq = a->inv_freq;
  p.positions = a->positions; p.seq = a->seq; p.page_table = a->page_table;
  p.status = a->status;
  // 16-byte loads need every row start on a 16-byte boundary
  const long long unit = 16 / (long long)es;
  bool wide = aligned(a->k, 16) && aligned(a->v, 16);
  for (long long s : {p.k_ts, p.k_hs, p.v_ts, p.v_hs}) wide = wide && s % unit == 0;
  if (with_q) wide = wide && aligned(a->q, 16) && p.q_ts % unit == 0 && p.q_hs % unit == 0;
  const bool il = a->interleaved != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->src_type == MK_BF16)
    e = pick_dst<__nv_bfloat16>(p, a->dst_type, a->head_dim, il, wide, st);
  else if (a->src_type == MK_FP16)
    e = pick_dst<__half>(p, a->dst_type, a->head_dim, il, wide, st);
  else
    e = pick_dst<float>(p, a->dst_type, a->head_dim, il, wide, st);
  return from_cuda(e);
}
