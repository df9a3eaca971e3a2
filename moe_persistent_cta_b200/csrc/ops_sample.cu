// ops_sample.cu -- one token per row of logits, from a given uniform number.
//
// With w_i = exp((x_i - max) / T), the kept tokens are a prefix of the tokens
// in descending order of (logit, -id): the first k, of those the shortest
// prefix whose sum reaches p of the k tokens' sum, of those the ones with
// w >= m.  A prefix is one cut (key, id): token i is kept if its logit's
// order-preserving key is larger, or equal with i <= id.  The draw then runs
// over the kept tokens in id order: the first at which the running sum passes
// u Z.
//
// Weights and sums are 64-bit: among 1.5e5 tokens a 32-bit sum would draw a
// neighbour of the defined token in a few per cent of the rows.  All sums are
// taken in a fixed order, so a call gives the same tokens every time.
//
// Bound: one read of the logits.  A cluster of up to 8 blocks holds a row in
// its shared memory, so the passes below touch memory once.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace mk {
namespace ops {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kFull = 0xffffffffu;

struct SampleParams {
  int B, V;
  int per;             // consecutive tokens of a thread
  long long stride;    // elements between rows
  const void* logits;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* tokens;
  float* logprobs;
  int32_t* status;
  // a decode loop's state, advanced by the drawn token (null otherwise)
  int32_t *next_token, *position, *seq_len;
};

// Order-preserving bits of a logit (never NaN, never -0): larger is larger.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyMinusInf = 0x007fffffu;   // key_of(-infinity)

// NaN counts as -infinity; -0 becomes +0.
__device__ __forceinline__ float clean(float x) {
  return isnan(x) ? -INFINITY : x + 0.0f;
}

template <typename T>
__device__ __forceinline__ T store_clean(T x);
template <>
__device__ __forceinline__ float store_clean<float>(float x) { return clean(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 store_clean<__nv_bfloat16>(__nv_bfloat16 x) {
  return __float2bfloat16_rn(clean(__bfloat162float(x)));
}
template <>
__device__ __forceinline__ __half store_clean<__half>(__half x) {
  return __float2half_rn(clean(__half2float(x)));
}

struct Exchange {
  double val[2][kMaxCluster][3];
  unsigned long long key[2][kMaxCluster];
};

struct Shared {
  double warp_val[kWarps][3];
  unsigned long long warp_key[kWarps];
  Exchange ex;
  double total[3];
  unsigned long long key;
  unsigned int first;        // first thread past the target
};

// A row's state, the same in every thread of the cluster.
template <typename T>
struct Row {
  const T* vals;         // this block's tokens
  int n;                 // how many of them
  int id0;               // id of the first
  int lo, hi;            // this thread's range of them
  float mx;
  double inv_t;
  bool inf;              // the largest logit is +infinity

  __device__ __forceinline__ double weight(float x) const {
    if (inf) return x == INFINITY ? 1.0 : 0.0;
    return exp(((double)x - (double)mx) * inv_t);
  }
};

class Cluster {
 public:
  __device__ Cluster(Shared* s, int rank, int size) : s_(s), rank_(rank), size_(size) {}

  // Sums three numbers over the cluster in a fixed order; every thread gets
  // them.  `mine`, where not null, receives the sums over lower-ranked blocks.
  __device__ void sum3(double a, double b, double c, double* out, double* below = nullptr) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(kFull, a, o);
      b += __shfl_xor_sync(kFull, b, o);
      c += __shfl_xor_sync(kFull, c, o);
    }
    if (lane == 0) {
      s_->warp_val[warp][0] = a;
      s_->warp_val[warp][1] = b;
      s_->warp_val[warp][2] = c;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
      double t = 0.0;
      for (int w = 0; w < kWarps; ++w) t += s_->warp_val[w][threadIdx.x];
      for (int r = 0; r < size_; ++r)
        *remote(&s_->ex.val[turn_][rank_][threadIdx.x], r) = t;
    }
    sync();
    for (int i = 0; i < 3; ++i) {
      double t = 0.0, under = 0.0;
      for (int r = 0; r < size_; ++r) {
        if (r == rank_) under = t;
        t += s_->ex.val[turn_][r][i];
      }
      out[i] = t;
      if (below) below[i] = under;
    }
    turn_ ^= 1;
  }

  // The largest key over the cluster.
  __device__ unsigned long long max_key(unsigned long long k) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(kFull, k, o);
      k = other > k ? other : k;
    }
    if (lane == 0) s_->warp_key[warp] = k;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) k = s_->warp_key[w] > k ? s_->warp_key[w] : k;
      for (int r = 0; r < size_; ++r) *remote(&s_->ex.key[turn_][rank_], r) = k;
    }
    sync();
    unsigned long long best = 0;
    for (int r = 0; r < size_; ++r) best = s_->ex.key[turn_][r] > best ? s_->ex.key[turn_][r] : best;
    turn_ ^= 1;
    return best;
  }

  __device__ void sync() {
    if (size_ == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  }

 private:
  template <typename U>
  __device__ U* remote(U* p, int r) {
    return size_ == 1 ? p : cg::this_cluster().map_shared_rank(p, r);
  }

  Shared* s_;
  int rank_, size_;
  int turn_ = 0;
};

// Largest key c such that the tokens with keys >= c add up to `target` or
// more: their number (COUNT) or their weights, each round splitting the range
// of keys in four.  *above receives the sum over keys > c, *at the sum over
// keys == c.  If all tokens together fall short, c is the lowest key in use.
template <bool COUNT, typename T>
__device__ uint32_t find_cut(Cluster& cl, const Row<T>& row, uint32_t floor_key, double target,
                             double* above, double* at) {
  unsigned long long lo = floor_key, hi = (unsigned long long)key_of(row.mx) + 1;
  double over = 0.0, in = 0.0;
  while (true) {
    const unsigned long long d = hi - lo;
    const unsigned long long m1 = lo + d / 4, m2 = lo + d / 2, m3 = lo + d - d / 4;
    double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
    for (int i = row.lo; i < row.hi; ++i) {
      const float x = to_float(row.vals[i]);
      const unsigned long long k = key_of(x);
      if (k < lo || k >= hi) continue;
      const double w = COUNT ? 1.0 : row.weight(x);
      if (k >= m3) s3 += w;
      else if (k >= m2) s2 += w;
      else if (k >= m1) s1 += w;
      else s0 += w;
    }
    double t[3];
    if (d == 1) {                    // m1 == m2 == lo and m3 == hi: all in s2
      cl.sum3(s2, 0.0, 0.0, t);
      in = t[0];
      break;
    }
    cl.sum3(s3, s2, s1, t);
    if (m3 < hi && over + t[0] >= target) {
      lo = m3;
    } else if (over + t[0] + t[1] >= target) {
      over += t[0];
      lo = m2;
      hi = m3;
    } else if (m1 == lo || over + t[0] + t[1] + t[2] >= target) {   // m1 == lo: nothing is lower
      over += t[0] + t[1];
      lo = m1;
      hi = m2;
    } else {
      over += t[0] + t[1] + t[2];
      hi = m1;
    }
  }
  *above = over;
  *at = in;
  return (uint32_t)lo;
}

// Sum of `v` over the block's lower threads.
__device__ double below_in_block(Shared* s, double v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += up;
  }
  const double exc = __shfl_up_sync(kFull, inc, 1);
  __syncthreads();
  if (lane == 31) s->warp_val[warp][0] = inc;
  __syncthreads();
  double base = 0.0;
  for (int w = 0; w < warp; ++w) base += s->warp_val[w][0];
  __syncthreads();
  return lane == 0 ? base : base + exc;
}

// Id of the rank-th (from 1) token, in id order, whose key is `key`.
template <typename T>
__device__ uint32_t nth_equal(Cluster& cl, Shared* s, const Row<T>& row, uint32_t key, double rank) {
  double mine = 0.0;
  for (int i = row.lo; i < row.hi; ++i) mine += key_of(to_float(row.vals[i])) == key ? 1.0 : 0.0;
  double t[3], under[3];
  cl.sum3(mine, 0.0, 0.0, t, under);
  double at = under[0] + below_in_block(s, mine);
  unsigned long long found = 0;      // 1 + the id, in the one thread that holds it
  if (at < rank && at + mine >= rank) {
    for (int i = row.lo; i < row.hi; ++i)
      if (key_of(to_float(row.vals[i])) == key && (at += 1.0) == rank) found = 1ull + row.id0 + i;
  }
  return (uint32_t)(cl.max_key(found) - 1ull);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, int cluster) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ Shared s;
  const int rank = cluster == 1 ? 0 : (int)cg::this_cluster().block_rank();
  const int b = blockIdx.x / cluster;
  Cluster cl(&s, rank, cluster);
  T* vals = reinterpret_cast<T*>(s_raw);

  Row<T> row;
  row.vals = vals;
  row.id0 = rank * kThreads * p.per;
  row.n = max(0, min(p.V - row.id0, kThreads * p.per));
  row.lo = min(row.n, (int)threadIdx.x * p.per);
  row.hi = min(row.n, row.lo + p.per);

  const float temp = p.temperature ? __ldg(p.temperature + b) : 1.0f;
  const float u = __ldg(p.u + b);
  const int k = p.top_k ? __ldg(p.top_k + b) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + b) : 1.0f;
  const float min_p = p.min_p ? __ldg(p.min_p + b) : 0.0f;

  // the row's part into shared memory; the largest logit, at its lowest id
  const T* src = static_cast<const T*>(p.logits) + (size_t)b * p.stride + row.id0;
  unsigned long long best = 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < row.n; i += kThreads) {
    const T x = store_clean<T>(src[i]);
    vals[i] = x;
    const unsigned long long c =
        ((unsigned long long)key_of(to_float(x)) << 32) | (uint32_t)~(uint32_t)(row.id0 + i);
    best = c > best ? c : best;
  }
  best = cl.max_key(best);           // also: every block's part is written
  const uint32_t max_k = (uint32_t)(best >> 32);
  const int max_id = (int)~(uint32_t)best;

  const bool bad = !(temp >= 0.0f) || isinf(temp) || !(u >= 0.0f && u < 1.0f) || isnan(top_p) ||
                   isnan(min_p);
  int token = -1;
  float logprob = -INFINITY;
  bool writer = rank == 0 && threadIdx.x == 0;
  if (bad) {
    if (writer)
      report(p.status, MK_ERR_DEVICE, MK_OP_SAMPLE, b, __float_as_int(!(u >= 0.0f && u < 1.0f) ? u : temp), 0);
  } else if (max_k <= kKeyMinusInf) {
    // nothing to draw
  } else if (temp == 0.0f) {
    token = max_id;
    logprob = 0.0f;
  } else {
    const uint32_t mb = (max_k & 0x80000000u) ? (max_k & 0x7fffffffu) : ~max_k;
    row.mx = __uint_as_float(mb);
    row.inf = row.mx == INFINITY;
    row.inv_t = 1.0 / (double)temp;
    const uint32_t floor_key = row.inf ? max_k : kKeyMinusInf + 1;
    // the cut: tokens with a larger key, or an equal one and id <= cut_id
    uint32_t cut = floor_key, cut_id = 0xffffffffu;
    double whole = -1.0;             // the first top_k tokens' sum, where needed
    double t[3];
    if (k > 0 && k < p.V) {
      double above, at;
      cut = find_cut<true>(cl, row, floor_key, (double)k, &above, &at);
      if (above + at > (double)k) cut_id = nth_equal(cl, &s, row, cut, (double)k - above);
    }
    auto kept = [&](float x, int id) {
      const uint32_t key = key_of(x);
      return key > cut || (key == cut && (uint32_t)id <= cut_id);
    };
    if (top_p < 1.0f) {
      double sum = 0.0;
      for (int i = row.lo; i < row.hi; ++i) {
        const float x = to_float(vals[i]);
        if (kept(x, row.id0 + i)) sum += row.weight(x);
      }
      cl.sum3(sum, 0.0, 0.0, t);
      whole = t[0];
      const double target = (double)top_p * whole;
      double above, at;
      const uint32_t c = find_cut<false>(cl, row, cut, target, &above, &at);
      if (c > cut || (c == cut && above < target)) {
        // of the equal tokens at the cut, as many as reach the target
        const uint32_t cb = (c & 0x80000000u) ? (c & 0x7fffffffu) : ~c;
        const double w = row.weight(__uint_as_float(cb));
        double need = w > 0.0 ? ceil((target - above) / w) : 1.0;
        if (need < 1.0) need = 1.0;
        const double have = w > 0.0 ? rint(at / w) : 1.0;
        if (need < have) {
          const uint32_t id = nth_equal(cl, &s, row, c, need);
          cut_id = c == cut ? min(cut_id, id) : id;
        } else if (c > cut) {
          cut_id = 0xffffffffu;
        }
        cut = c;
      }
    }
    // the draw, in id order
    double mine = 0.0;
    int last = -1;
    for (int i = row.lo; i < row.hi; ++i) {
      const float x = to_float(vals[i]);
      if (!kept(x, row.id0 + i)) continue;
      const double w = row.weight(x);
      if (w < (double)min_p || w == 0.0) continue;
      mine += w;
      last = i;
    }
    double under[3];
    cl.sum3(mine, 0.0, 0.0, t, under);
    const double z = t[0], target = (double)u * z;
    const double before = under[0] + below_in_block(&s, mine);
    // the first thread that holds kept tokens and passes the target; by
    // rounding there may be none, then the last that holds any
    const uint32_t place = (uint32_t)(rank * kThreads + threadIdx.x);
    unsigned long long c = 0;
    if (last >= 0)
      c = before + mine > target ? (1ull << 62) - place : 1ull + place;
    const unsigned long long won = cl.max_key(c);
    writer = last >= 0 && c == won;
    if (writer) {
      double acc = before, w = 0.0;
      int pick = last;
      for (int i = row.lo; i <= last; ++i) {
        const float x = to_float(vals[i]);
        if (!kept(x, row.id0 + i)) continue;
        w = row.weight(x);
        if (w < (double)min_p || w == 0.0) continue;
        acc += w;
        if (acc > target) {
          pick = i;
          break;
        }
      }
      token = row.id0 + pick;
      logprob = (float)log(row.weight(to_float(vals[pick])) / z);
    }
  }
  if (writer) {
    p.tokens[b] = token;
    if (p.logprobs) p.logprobs[b] = logprob;
    if (p.next_token) {
      p.next_token[b] = token < 0 ? 0 : token;   // the step's embedding needs a token id
      const int pos = p.position[b];
      p.position[b] = pos + 1;
      if (p.seq_len != p.position) p.seq_len[b] += 1;
    }
  }
  cl.sync();                         // no block leaves while another may write to it
}

// Blocks a row is spread over and consecutive tokens of a thread.  The part a
// thread walks is an odd number of elements, so that the 32 threads of a warp
// read 32 banks.
int cluster_for(int vocab) {
  int c = 1;
  while (c < kMaxCluster && vocab > c * kThreads * 4) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_sample(const SampleParams& p0, cudaStream_t stream) {
  SampleParams p = p0;
  const int c = cluster_for(p.V);
  p.per = ((p.V + c * kThreads - 1) / (c * kThreads)) | 1;
  const size_t smem = (size_t)p.per * kThreads * sizeof(T);
  static_assert((MK_SAMPLE_MAX_VOCAB / (kMaxCluster * kThreads) + 1) * kThreads * 4 +
                        sizeof(Shared) <= 227 * 1024,
                "the largest vocabulary does not fit the cluster's shared memory");
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.B * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, (const SampleParams)p, c);
}

}  // namespace

mk_status sample(const mk_sample_args* a, int32_t* next_token, int32_t* position, int32_t* seq_len,
                 cudaStream_t stream) {
  if (!a) return MK_ERR_INVALID;
  if (a->batch < 0 || a->vocab < 1) return MK_ERR_INVALID;
  if (a->vocab > MK_SAMPLE_MAX_VOCAB || a->batch > (1 << 24)) return MK_ERR_CAPACITY;
  if (a->type != MK_FP32 && a->type != MK_BF16 && a->type != MK_FP16) return MK_ERR_INVALID;
  if (a->batch == 0) return MK_OK;
  if (!a->logits || !a->u || !a->tokens) return MK_ERR_INVALID;
  if (!aligned(a->logits, a->type == MK_FP32 ? 4 : 2)) return MK_ERR_INVALID;
  DeviceGuard guard(a->device);
  if (guard.status() != MK_OK) return guard.status();
  SampleParams p{};
  p.B = a->batch;
  p.V = a->vocab;
  p.stride = a->row_stride;
  p.logits = a->logits;
  p.u = a->u;
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.tokens = a->tokens;
  p.logprobs = a->logprobs;
  p.status = a->status;
  p.next_token = next_token;
  p.position = position;
  p.seq_len = seq_len;
  if (a->type == MK_FP32) return from_cuda(launch_sample<float>(p, stream));
  if (a->type == MK_BF16) return from_cuda(launch_sample<__nv_bfloat16>(p, stream));
  return from_cuda(launch_sample<__half>(p, stream));
}

}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_sample(const mk_sample_args* args, void* stream) {
  return mk::ops::sample(args, nullptr, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}
