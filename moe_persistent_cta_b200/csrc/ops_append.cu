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
// Bound: memory (each row is read and written once, no reuse).  A block takes
// kTokens tokens, forms their sines and cosines once for all heads in shared
// memory, and each thread turns 16 columns of a head: two 16-byte loads and
// two 16-byte stores for 16-bit rows, issued before the block waits for the
// table.
#include "ops_common.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  int T, rows, max_pages, n_pages, Hq, Hkv, R;
  int stage_q;               // query heads present (0: none)
  float magnitude;
  const void *q, *k, *v;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;   // strides in elements
  void *q_out, *k_pool, *v_pool;
  const double* inv_freq;
  const int32_t *positions, *seq, *page_table;
  int32_t* status;
};

// cos and sin of position * f: the angle less the nearest multiple of 2 pi,
// the multiple subtracted in two parts (2 pi as a sum of two doubles).
__device__ __forceinline__ float2 turn(int position, double f, float magnitude) {
  constexpr double kTwoPiHi = 6.283185307179586;         // 2 pi rounded to 53 bits
  constexpr double kTwoPiLo = 2.4492935982947064e-16;    // 2 pi - kTwoPiHi
  const double a = (double)position * f;
  const double n = rint(a * 0.15915494309189535);        // 1 / (2 pi)
  const float r = (float)fma(-n, kTwoPiLo, fma(-n, kTwoPiHi, a));
  float s, c;
  sincosf(r, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

// 8 consecutive elements as floats; WIDE: the address is 16-byte aligned.
template <typename S, bool WIDE>
__device__ __forceinline__ void load8(const S* p, float* f) {
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_float(p[i]);
  } else if constexpr (sizeof(S) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    Vec8<S>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), f);
  }
}

// MODE 0: half layout, R a multiple of 8: the thread's two groups of 8 columns
// are the two halves of its 8 pairs.  MODE 1: interleaved: 16 consecutive
// columns.  MODE 2: half layout, any R: 16 consecutive columns whose partners
// are read back from the row staged in shared memory.
template <typename S, typename D, int HD, int MODE, bool WIDE>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const AppendParams p, int tokens) {
  extern __shared__ float2 s_tab[];          // [tokens][R], then MODE 2's rows
  constexpr int PER_HEAD = HD / 16;
  const int R = p.R;
  const int heads = p.stage_q + 2 * p.Hkv;
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, p.T - t0);
  const int items = nt * heads * PER_HEAD;
  float* rows = reinterpret_cast<float*>(s_tab + (size_t)tokens * R);

  for (int i = threadIdx.x; i < nt * R; i += kThreads) {
    const int t = i / R;
    s_tab[i] = turn(__ldg(p.positions + t0 + t), __ldg(p.inv_freq + (i - t * R)), p.magnitude);
  }
  for (int base = 0; base < items; base += kThreads) {
    const int it = base + threadIdx.x;
    const int j = it % PER_HEAD, hh = (it / PER_HEAD) % heads, t = t0 + it / (PER_HEAD * heads);
    const bool in = it < items;
    const bool is_v = hh >= p.stage_q + p.Hkv;
    const bool is_q = hh < p.stage_q;
    // where this thread's two groups of 8 columns start
    const bool paired = MODE == 0 && !is_v && 8 * j < R;
    const int c0 = paired ? 8 * j : 16 * j;
    const int c1 = paired ? R + 8 * j : 16 * j + 8;
    float x[16];
    if (in) {
      const S* src = is_q   ? static_cast<const S*>(p.q) + t * p.q_ts + hh * p.q_hs
                     : is_v ? static_cast<const S*>(p.v) + t * p.v_ts + (hh - p.stage_q - p.Hkv) * p.v_hs
                            : static_cast<const S*>(p.k) + t * p.k_ts + (hh - p.stage_q) * p.k_hs;
      load8<S, WIDE>(src + c0, x);
      load8<S, WIDE>(src + c1, x + 8);
    }
    // the token's place: a negative sequence is padding, skipped
    int page = -1, pos = 0, seq = -1;
    if (in) {
      pos = __ldg(p.positions + t);
      seq = p.seq ? __ldg(p.seq + t) : t;
      if (seq >= 0) {
        if (seq >= p.rows) {
          report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, seq, p.rows);
        } else if (pos < 0 || pos / kPageTokens >= p.max_pages) {
          report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, pos, p.max_pages * kPageTokens);
        } else {
          page = __ldg(p.page_table + (size_t)seq * p.max_pages + pos / kPageTokens);
          if (page < 0 || page >= p.n_pages) {
            report(p.status, MK_ERR_DEVICE, MK_OP_ROPE_APPEND, t, page, p.n_pages);
            page = -1;
          }
        }
      }
    }
    if constexpr (MODE == 2) {
      if (base) __syncthreads();             // the previous rows have been read
      if (in && !is_v) {
        float* row = rows + threadIdx.x * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) row[i] = x[i];
      }
    }
    if (base == 0 || MODE == 2) __syncthreads();   // the table (and the staged rows) are written
    if (page < 0) continue;
    if (!is_v) {
      const float2* tab = s_tab + (t - t0) * R;
      if constexpr (MODE == 0) {
        if (paired) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = tab[8 * j + i];
            const float a = x[i], b = x[8 + i];
            x[i] = a * cs.x - b * cs.y;
            x[8 + i] = b * cs.x + a * cs.y;
          }
        }
      } else if constexpr (MODE == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (8 * j + i < R) {
            const float2 cs = tab[8 * j + i];
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cs.x - b * cs.y;
            x[2 * i + 1] = b * cs.x + a * cs.y;
          }
        }
      } else {
        // a head's items are consecutive threads of one block, HD / 16 a
        // power of two, so the head's row starts at this thread less j
        const float* row = rows + (threadIdx.x - j) * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 16 * j + i;
          if (c < R) {
            const float2 cs = tab[c];
            x[i] = x[i] * cs.x - row[c + R] * cs.y;
          } else if (c < 2 * R) {
            const float2 cs = tab[c - R];
            x[i] = x[i] * cs.x + row[c - R] * cs.y;
          }
        }
      }
    }
    D* dst;
    if (is_q) {
      dst = static_cast<D*>(p.q_out) + ((size_t)t * p.Hq + hh) * HD;
    } else {
      const int h = is_v ? hh - p.stage_q - p.Hkv : hh - p.stage_q;
      dst = static_cast<D*>(is_v ? p.v_pool : p.k_pool) +
            (((size_t)page * p.Hkv + h) * kPageTokens + pos % kPageTokens) * HD;
    }
    *reinterpret_cast<uint4*>(dst + c0) = Vec8<D>::pack(x);
    *reinterpret_cast<uint4*>(dst + c1) = Vec8<D>::pack(x + 8);
  }
}

template <typename S, typename D, int HD, int MODE, bool WIDE>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  const int tokens = 1;
  const size_t smem = (size_t)tokens * p.R * sizeof(float2) +
                      (MODE == 2 ? (size_t)kThreads * 16 * sizeof(float) : 0);
  rope_append_kernel<S, D, HD, MODE, WIDE>
      <<<(p.T + tokens - 1) / tokens, kThreads, smem, stream>>>(p, tokens);
  return cudaGetLastError();
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
  DeviceGuard guard(a->device);
  if (guard.status() != MK_OK) return guard.status();
  if (a->n_tokens == 0) return MK_OK;

  AppendParams p{};
  p.T = a->n_tokens;
  p.rows = a->n_rows;
  p.max_pages = a->max_pages;
  p.n_pages = a->n_pages;
  p.Hq = a->n_q_heads;
  p.Hkv = a->n_kv_heads;
  p.R = a->rotary_dim / 2;
  p.stage_q = a->n_q_heads;
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
