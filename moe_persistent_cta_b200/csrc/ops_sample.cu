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
// Bound: one read of the logits.  A cluster of up to 8 (few rows: 16) blocks holds a row in
// its shared memory, so the passes below touch memory once.  The cut is found
// by one of three ways:
//  * top_k up to 512: the k-th largest of the maxima of 512 groups of tokens is a
//    logit that at least k tokens reach, and hardly more than k; those are
//    gathered in one block and ordered, which settles everything.
//  * top_p alone: the range of logits is narrowed by a factor of 16 at a time by
//    32-bit sums of the weights, until few tokens are left about the cut; they are
//    gathered and ordered, and 64-bit sums say which is the last, or that it is
//    not among them.
//  * otherwise (large top_k, very many equal logits): the range of keys is
//    split in four, again and again, by exact sums.
// Few tokens are ordered by counting, for each, the larger ones: all threads read
// the same word at a time, and there is no chain of barriers (1024 tokens: 7.9 us
// by a bitonic sort, 1.6 by counting).
//
// What bounds it: the passes over shared memory, about 2 us each for 151552 tokens
// over 8 blocks, and for the passes that weigh every token 14 64-bit operations a
// token (5 us).  256 rows of 151552 with mixed rules take 215 us (0.72 TB/s of
// logits); calls for one row of 1024, one behind another, 8.5 to 10 us each.
#include <cooperative_groups.h>

#include <mutex>

#include "ops_common.cuh"
#include "ops_step.h"

namespace cg = cooperative_groups;

namespace mk {
namespace ops {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;          // blocks of a row, at most ...
constexpr int kMaxCluster = 16;      // ... and where so many clusters run at once anyway
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kList = 2 * kThreads;  // tokens that can be gathered and ordered
constexpr int kBins = kWarps;        // parts of a range of logits, one per warp

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
  float bin[2][kMaxCluster][kBins];
};

struct Shared {
  union {
    struct {
      unsigned long long list[kList];      // gathered tokens, (key << 32) | ~id
      unsigned long long sorted[kList];    // in descending order
      struct {
        double w[kThreads];
        int id[kThreads], by_id[kThreads];
      } draw;                              // the draw among sorted tokens
      uint32_t group_max[kThreads];
    };
    float bins[kBins][kThreads];           // sums of weights, each thread its own
  };
  double exp2_tab[256];              // 2^(j / 256)
  double warp_val[kWarps][3];
  unsigned long long warp_key[kWarps];
  Exchange ex;
  uint32_t cut, cut_id;              // handed round by the ordering block
  int n_list, kept, picked;
};

// exp(z) for z = d / T <= 0, d = x - max: with y = d (256 / ln 2) / T = n + r,
// |r| <= 1/2, it is 2^(n / 256) exp(r ln 2 / 256): a table of 256 values and a
// polynomial of degree 4, whose remainder is below 2^-54 (Tang's table-driven
// method).  10 64-bit operations; the library's exp takes about twice as many
// and bounded the passes over a row.
struct Weight {
  const double* tab;
  double mx, k;                      // largest logit, (256 / ln 2) / T
  __device__ __forceinline__ double operator()(float x) const {
    constexpr double kMagic = 6755399441055744.0;          // 1.5 x 2^52: rounds to an integer
    constexpr double c1 = 0.0027076061740622863;           // ln 2 / 256
    constexpr double c2 = c1 * c1 / 2, c3 = c1 * c1 * c1 / 6, c4 = c1 * c1 * c1 * c1 / 24;
    const double y = fmax(((double)x - mx) * k, -300000.0);
    const double t = y + kMagic;
    const int n = __double2loint(t);
    const double r = y - (t - kMagic);
    const double v = tab[n & 255];
    const double w = fma(v * r, fma(r, fma(r, fma(r, c4, c3), c2), c1), v);
    const int e = n >> 8;
    return e < -1021 ? 0.0 : __hiloint2double(__double2hiint(w) + (e << 20), __double2loint(w));
  }
};

// A row's state, the same in every thread of the cluster.
template <typename T>
struct Row {
  const T* vals;         // this block's tokens
  int n;                 // how many of them
  int id0;               // id of the first
  int lo, hi;            // this thread's range of them
  float mx;
  Weight exp_of;
  bool inf;              // the largest logit is +infinity

  __device__ __forceinline__ double weight(float x) const {
    if (inf) return x == INFINITY ? 1.0 : 0.0;
    return exp_of(x);
  }
};

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

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

  // Sums a number over the cluster as above; says whether this is the block at
  // which the running sum over blocks passes u of the whole, or, if by rounding
  // none does, the last that adds anything.
  __device__ bool sum_drawn(double a, float u, double* out, double* below) {
    const int turn = turn_;
    sum3(a, 0.0, 0.0, out, below);
    double upto = 0.0;
    int at = -1, some = -1;
    for (int r = 0; r < size_; ++r) {
      const double v = s_->ex.val[turn][r][0];
      upto += v;
      if (v > 0.0) {
        some = r;
        if (at < 0 && upto > (double)u * out[0]) at = r;
      }
    }
    return (at >= 0 ? at : some) == rank_;
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

  // Sums a block's parts (one per warp, in its lane 0) over the cluster in a
  // fixed order; lane i of every warp gets part i.
  __device__ float sum_bins(float mine) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < size_) *remote(&s_->ex.bin[turn_][rank_][warp], lane) = mine;
    sync();
    float t = 0.0f;
    if (lane < kBins)
      for (int r = 0; r < size_; ++r) t += s_->ex.bin[turn_][r][lane];
    turn_ ^= 1;
    return t;
  }

  __device__ void sync() {
    if (size_ == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  }

  template <typename U>
  __device__ U* remote(U* p, int r) {
    return size_ == 1 ? p : cg::this_cluster().map_shared_rank(p, r);
  }
  // A barrier in two parts; what a block has read of another's memory before
  // the first is read before the other block gets past the second.
  __device__ void arrive() {
    __syncwarp();
    if (size_ > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  __device__ void wait() {
    __syncwarp();
    if (size_ > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __device__ int size() const { return size_; }
  __device__ int rank() const { return rank_; }

 private:
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

// Sum of `v` over the block's lower threads; *all: over all of them.
__device__ double below_in_block(Shared* s, double v, double* all = nullptr) {
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
  double base = 0.0, sum = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) base = sum;
    sum += s->warp_val[w][0];
  }
  __syncthreads();
  if (all) *all = sum;
  return lane == 0 ? base : base + exc;
}

// f(logit, place) for this thread's tokens in order, eight loads ahead.
template <typename T, typename F>
__device__ __forceinline__ void each(const Row<T>& row, F f) {
  for (int i = row.lo; i < row.hi; i += 8) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = i + e < row.hi ? to_float(row.vals[i + e]) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < row.hi) f(x[e], i + e);
  }
}

// Weights of the tokens of this thread that `want` picks (0 for the
// others), four at a time so that their chains overlap: take(i, weight) in order.
template <typename T, typename F, typename G>
__device__ __forceinline__ void weigh(const Row<T>& row, F want, G take) {
  for (int i = row.lo; i < row.hi; i += 4) {
    float x[4];
    bool in[4], any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      in[e] = i + e < row.hi;
      x[e] = in[e] ? to_float(row.vals[i + e]) : row.mx;
      in[e] = in[e] && want(x[e], row.id0 + i + e);
      any |= in[e];
    }
    if (!any) continue;
    double w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = row.weight(x[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (in[e]) take(i + e, w[e]);
  }
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

// s->sorted: s->list[0 .. n) in descending order (n <= kList, no two alike);
// ends with a barrier.
__device__ void order_list(Shared* s, int n) {
  if (threadIdx.x == 0 && n < kList) s->list[n] = 0;
  __syncthreads();
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(s->list);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = s->list[i];
    int larger = 0;
#pragma unroll 8
    for (int k = 0; k < (n + 1) / 2; ++k) {
      const ulonglong2 v = two[k];
      larger += (v.x > mine) + (v.y > mine);
    }
    s->sorted[larger] = mine;
  }
  __syncthreads();
}

// Gathers the row's tokens that `want` picks in block 0 of the cluster, kList at
// most, and orders them there.  Returns how many there are (if more than kList,
// nothing is ordered); n_list has been 0 in block 0 since an earlier cluster
// barrier.  Ends behind a cluster barrier that block 0 alone has to wait for
// (cl.wait(), before it touches n_list or leaves).
template <typename T, typename F>
__device__ int gather(Cluster& cl, Shared* s, const Row<T>& row, F want) {
  int* count = cl.remote(&s->n_list, 0);
  unsigned long long* list = cl.remote(s->list, 0);
  each(row, [&](float x, int i) {
    if (want(x)) {
      const int at = atomicAdd(count, 1);
      if (at < kList) list[at] = ((unsigned long long)key_of(x) << 32) | (uint32_t)~(uint32_t)(row.id0 + i);
    }
  });
  cl.sync();
  const int n = *count;
  cl.arrive();
  if (n <= kList && cl.rank() == 0) order_list(s, n);
  return n;
}

// Ordered tokens of a thread: consecutive ones.
constexpr int kEach = kList / kThreads;

// Block 0, with the list ordered: how many of the first n tokens are kept by
// a limit on the sum before each, starting from `above`: `target`, or top_p of
// the n tokens' sum where target is negative.  *all: the sum behind them.
template <typename T>
__device__ int keep_sorted(Shared* s, const Row<T>& row, int n, float top_p, double above, double target,
                           double* all) {
  double w[kEach], mine = 0.0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = kEach * (int)threadIdx.x + e;
    w[e] = i < n ? row.weight(value_of((uint32_t)(s->sorted[i] >> 32))) : 0.0;
    mine += w[e];
  }
  if (threadIdx.x == 0) s->kept = 0;         // behind the scan's barriers
  double before = above + below_in_block(s, mine, all);
  *all += above;
  if (target < 0.0) target = (double)top_p * *all;
  int keep = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = kEach * (int)threadIdx.x + e;
    keep += i < n && (top_p >= 1.0f || before < target);
    before += w[e];
  }
  // what is kept is a prefix, so the number says which
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) keep += __shfl_xor_sync(kFull, keep, o);
  if ((threadIdx.x & 31) == 0 && keep) atomicAdd(&s->kept, keep);
  __syncthreads();
  return s->kept;
}

// The draw among the first `keep` (1 .. kThreads) of the ordered tokens, one per
// thread: put in the order of their ids, their running sums say which.  True in
// the thread that holds the drawn token.
template <typename T>
__device__ bool draw_sorted(Shared* s, const Row<T>& row, int keep, float min_p, float u, int* token,
                            float* logprob) {
  const int i = threadIdx.x;
  double w = 0.0;
  int id = 0x7fffffff;
  if (i < keep) {
    const unsigned long long e = s->sorted[i];
    w = row.weight(value_of((uint32_t)(e >> 32)));
    if (i > 0 && w < (double)min_p) w = 0.0;
    id = (int)~(uint32_t)e;
  }
  s->draw.id[i] = id;
  if (i == 0) s->picked = 0x7fffffff;
  __syncthreads();
  if (i < keep) {
    int lower = 0;
    const int4* four = reinterpret_cast<const int4*>(s->draw.id);
#pragma unroll 4
    for (int k = 0; k < (keep + 3) / 4; ++k) {
      const int4 v = four[k];
      lower += (v.x < id) + (v.y < id) + (v.z < id) + (v.w < id);
    }
    s->draw.w[lower] = w;
    s->draw.by_id[lower] = id;
  }
  __syncthreads();
  w = i < keep ? s->draw.w[i] : 0.0;
  double z;
  const double upto = below_in_block(s, w, &z) + w;
  if (w > 0.0 && upto > (double)u * z) atomicMin(&s->picked, i);
  __syncthreads();
  if (s->picked == 0x7fffffff) {     // by rounding: the last one, then
    __syncthreads();
    if (i == 0) s->picked = -1;
    __syncthreads();
    if (w > 0.0) atomicMax(&s->picked, i);
    __syncthreads();
  }
  if (i != s->picked) return false;
  *token = s->draw.by_id[i];
  *logprob = (float)log(w / z);
  return true;
}

// The cut of top_p over all tokens, by narrowing; also this thread's sum of the
// tokens nearer to the largest than *from, all of which are kept.  False if it has to be found
// another way (the same in every thread of the cluster).
template <typename T>
__device__ bool narrow_cut(Cluster& cl, Shared* s, const Row<T>& row, int V, float top_p, float temp,
                           uint32_t* cut, uint32_t* cut_id, float* from_out, double* above_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double sum = 0.0, t[3];
  weigh(row, [](float, int) { return true; }, [&](int, double w) { sum += w; });
  cl.sum3(sum, 0.0, 0.0, t);
  const double target = (double)top_p * t[0];
  // Tokens further than `reach` below the largest (in exponents) weigh less than
  // V exp(-reach) = (1 - top_p) / e of it together: the cut is not among them.
  const float reach = logf((float)V / (1.0f - top_p)) + 1.0f, rate = 1.4426950f / temp;
  float lo = 0.0f, width = reach * temp;     // the range: distances to the largest
  float over = 0.0f;                         // weight before it
  for (int level = 0;; ++level) {
    const float scale = (float)kBins / width;
#pragma unroll
    for (int b = 0; b < kBins; ++b) s->bins[b][threadIdx.x] = 0.0f;
    each(row, [&](float x, int) {
      const float d = row.mx - x, place = (d - lo) * scale;
      if (place >= 0.0f && place < (float)kBins) s->bins[(int)place][threadIdx.x] += exp2f(-d * rate);
    });
    __syncthreads();
    float part = 0.0f;                       // each warp adds up one bin
#pragma unroll
    for (int k = 0; k < kThreads; k += 32) part += s->bins[warp][k + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kFull, part, o);
    const float bin = cl.sum_bins(part);
    float upto = bin;
#pragma unroll
    for (int o = 1; o < kBins; o <<= 1) {
      const float up = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += up;
    }
    // 32-bit weights and their sums are good to 1e-5
    const float reached = over + upto, want = (float)target;
    const uint32_t maybe = __ballot_sync(kFull, lane < kBins && reached * (1.0f + 1e-5f) >= want);
    const uint32_t surely = __ballot_sync(kFull, lane < kBins && reached * (1.0f - 1e-5f) >= want);
    if (surely == 0) return false;
    const int first = __ffs(maybe) - 1, last = __ffs(surely) - 1;
    const float here = __shfl_sync(kFull, upto, last) - (first ? __shfl_sync(kFull, upto, max(first - 1, 0)) : 0.0f);
    if (first) over += __shfl_sync(kFull, upto, first - 1);
    lo += (float)first / scale;
    width = (float)(last - first + 1) / scale;
    // every token of the range weighs at least 2^(-rate (lo + width))
    // (ordering n tokens takes n^2: 1000 as long as three more rounds)
    if (here * exp2f(rate * (lo + width)) < 256.0f || level == 5) break;
  }
  // a little wider, by more than the places' rounding
  const float slack = 1e-6f * (fabsf(row.mx) + lo + width);
  const float from = lo - slack, to = lo + width + slack;
  double above = 0.0;
  weigh(row, [&](float x, int) { return row.mx - x < from; }, [&](int, double w) { above += w; });
  cl.sum3(above, 0.0, 0.0, t);
  const int n = gather(cl, s, row, [&](float x) {
    const float d = row.mx - x;
    return d >= from && d < to;
  });
  cl.wait();
  if (n > kList) return false;
  if (cl.rank() == 0) {
    double all;
    const int keep = keep_sorted(s, row, n, top_p, t[0], target, &all);
    if ((int)threadIdx.x < cl.size()) {
      // the cut has to lie among these tokens
      const bool found = keep > 0 && (keep < n || all >= target);
      const unsigned long long e = found ? s->sorted[keep - 1] : 0ull;
      *cl.remote(&s->cut, threadIdx.x) = (uint32_t)(e >> 32);
      *cl.remote(&s->cut_id, threadIdx.x) = (uint32_t)~(uint32_t)e;
    }
  }
  cl.sync();
  if (s->cut == 0) return false;
  *cut = s->cut;
  *cut_id = s->cut_id;
  *from_out = from;
  *above_out = above;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cluster) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ Shared s;
  const int rank = cluster == 1 ? 0 : (int)cg::this_cluster().block_rank();
  const int b = blockIdx.x / cluster;
  Cluster cl(&s, rank, cluster);
  cl.arrive();
  // Nothing of the call's memory is touched before the kernels ahead are done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (No early word to the kernel behind: its blocks would take room from this
  // one's: 33 rows of 151541, 29 us and not 24.)

  Row<T> row;
  row.id0 = rank * kThreads * p.per;
  row.n = max(0, min(p.V - row.id0, kThreads * p.per));
  row.lo = min(row.n, (int)threadIdx.x * p.per);
  row.hi = min(row.n, row.lo + p.per);

  const float temp = p.temperature ? __ldg(p.temperature + b) : 1.0f;
  const float u = __ldg(p.u + b);
  const int k = p.top_k ? __ldg(p.top_k + b) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + b) : 1.0f;
  const float min_p = p.min_p ? __ldg(p.min_p + b) : 0.0f;

  // the row's part into shared memory, at the same place within 16 bytes as in
  // global memory; the largest logit, at its lowest id
  const T* src = static_cast<const T*>(p.logits) + (size_t)b * p.stride + row.id0;
  const int shift = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  T* vals = reinterpret_cast<T*>(s_raw + shift);
  row.vals = vals;
  uint32_t top = 0;                  // this thread's largest key and its id
  int top_id = 0;
  auto take = [&](T v, int i) {
    const T x = store_clean<T>(v);
    const uint32_t key = key_of(to_float(x));
    if (key > top) {                 // ids ascend: the first of equal ones stays
      top = key;
      top_id = row.id0 + i;
    }
    return x;
  };
  constexpr int VE = 16 / sizeof(T);
  const int lead = min(row.n, ((16 - shift) & 15) / (int)sizeof(T));
  const int vecs = (row.n - lead) / VE;
  if ((int)threadIdx.x < lead) vals[threadIdx.x] = take(src[threadIdx.x], threadIdx.x);
  {
    const uint4* from = reinterpret_cast<const uint4*>(src + lead);
    uint4* to = reinterpret_cast<uint4*>(vals + lead);
    constexpr int kAhead = 8;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kAhead * kThreads) {
      uint4 v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (i0 + a * kThreads < vecs) v[a] = __ldcs(from + i0 + a * kThreads);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * kThreads;
        if (i < vecs) {
          T* e = reinterpret_cast<T*>(&v[a]);
#pragma unroll
          for (int c = 0; c < VE; ++c) e[c] = take(e[c], lead + i * VE + c);
          to[i] = v[a];
        }
      }
    }
  }
  for (int i = lead + vecs * VE + threadIdx.x; i < row.n; i += kThreads) vals[i] = take(src[i], i);
  if (threadIdx.x == 0) s.n_list = 0;
  if (threadIdx.x < 256) s.exp2_tab[threadIdx.x] = exp2((double)threadIdx.x / 256.0);
  {
    uint32_t g = top;
    if (vecs < kThreads) {           // some threads have loaded nothing: go by the tokens they walk
      __syncthreads();
      g = 0;
      for (int i = row.lo; i < row.hi; ++i) g = max(g, key_of(to_float(vals[i])));
    }
#pragma unroll
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
      const uint32_t other = __shfl_xor_sync(kFull, g, o);
      if (o < cluster) g = max(g, other);
    }
    cl.wait();                       // every block runs: its memory may be written
    if ((threadIdx.x & (cluster - 1)) == 0)
      for (int r = 0; r < cluster; ++r)
        *cl.remote(&s.group_max[(rank * kThreads + threadIdx.x) / cluster], r) = g;
  }
  // also: every block's part, table and maxima are written
  const unsigned long long best =
      cl.max_key(((unsigned long long)top << 32) | (uint32_t)~(uint32_t)top_id);
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
  } else if (temp == 0.0f || top_p <= 0.0f || k == 1 || min_p > 1.0f) {
    token = max_id;                  // nothing else is kept
    logprob = 0.0f;
  } else {
    row.mx = value_of(max_k);
    row.inf = row.mx == INFINITY;
    row.exp_of = Weight{s.exp2_tab, (double)row.mx, 369.32993046757463 / (double)temp};
    const uint32_t floor_key = row.inf ? max_k : kKeyMinusInf + 1;
    // the cut: tokens with a larger key, or an equal one and id <= cut_id
    uint32_t cut = floor_key, cut_id = 0xffffffffu;
    bool settled = false;            // block 0 has drawn among the gathered tokens
    double t[3];
    float from = -INFINITY;          // this thread's tokens nearer than this are in `summed`
    double summed = 0.0;
    const bool limited = k > 0 && k < p.V;
    if (limited && k <= kThreads) {
      // the k-th largest of the groups' maxima to 20 bits, rounded down: k
      // tokens or more reach it
      uint32_t t0 = 0;
      const uint32_t mine = s.group_max[threadIdx.x];
      for (int bit = 31; bit >= 12; --bit) {
        const uint32_t c = t0 | (1u << bit);
        if (__syncthreads_count(mine >= c) >= k) t0 = c;
      }
      t0 = max(t0, floor_key);
      const int n = gather(cl, &s, row, [&](float x) { return key_of(x) >= t0; });
      if (n <= kList) {
        settled = true;
        writer = false;
        if (rank == 0) {
          double all;
          const int keep = keep_sorted(&s, row, min(n, k), top_p, 0.0, -1.0, &all);
          writer = draw_sorted(&s, row, max(keep, 1), min_p, u, &token, &logprob);
        }
      }
      cl.wait();
    }
    if (limited && !settled) {
      double above, at;
      cut = find_cut<true>(cl, row, floor_key, (double)k, &above, &at);
      if (above + at > (double)k) cut_id = nth_equal(cl, &s, row, cut, (double)k - above);
    }
    if (!settled) {
      auto kept = [&](float x, int id) {
        const uint32_t key = key_of(x);
        return key > cut || (key == cut && (uint32_t)id <= cut_id);
      };
      if (top_p < 1.0f && (limited || row.inf || !narrow_cut(cl, &s, row, p.V, top_p, temp, &cut, &cut_id, &from, &summed))) {
        double sum = 0.0;
        weigh(row, kept, [&](int, double w) { sum += w; });
        cl.sum3(sum, 0.0, 0.0, t);
        const double target = (double)top_p * t[0];
        double above, at;
        const uint32_t c = find_cut<false>(cl, row, cut, target, &above, &at);
        if (c > cut || (c == cut && above < target)) {
          // of the equal tokens at the cut, as many as reach the target
          const double w = row.weight(value_of(c));
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
      if (min_p > 0.0f && !row.inf) {
        // what is surely below min_p needs no weight: min_p's logit, lowered by
        // more than its rounding
        const double x = (double)row.mx + (double)temp * log((double)min_p);
        const double low = x - 1e-6 * (fabs(x) + fabs((double)row.mx));
        if (low > -3e38) {
          const uint32_t c = key_of((float)low + 0.0f);
          if (c > cut) {
            cut = c;
            cut_id = 0xffffffffu;
          }
        }
      }
      // the draw, in id order
      double mine = 0.0;
      int last = -1;
      if (min_p > 0.0f) from = -INFINITY;    // not all of those are kept
      if (from > -INFINITY) {
        mine = summed;
        each(row, [&](float x, int i) {
          if (row.mx - x < from) last = i;
        });
      }
      weigh(row, [&](float x, int id) { return !(row.mx - x < from) && kept(x, id); }, [&](int i, double w) {
        if (w < (double)min_p || w == 0.0) return;
        mine += w;
        last = max(last, i);
      });
      double under[3];
      const bool here = cl.sum_drawn(mine, u, t, under);
      const double z = t[0], target = (double)u * z;
      // in the one block whose tokens pass the target: the first thread that holds
      // kept tokens and passes it; by rounding there may be none, then the last
      // that holds any
      int won = -1;
      double before = 0.0;
      if (here) {
        before = under[0] + below_in_block(&s, mine);
        if (threadIdx.x == 0) s.picked = 0x7fffffff;
        __syncthreads();
        if (last >= 0) atomicMin(&s.picked, before + mine > target ? (int)threadIdx.x : 2 * kThreads - (int)threadIdx.x);
        __syncthreads();
        won = s.picked < kThreads ? s.picked : 2 * kThreads - s.picked;
      }
      // that thread's warp goes through its tokens together
      const int lane = threadIdx.x & 31;
      const uint32_t winner = __ballot_sync(kFull, (int)threadIdx.x == won);
      writer = false;
      if (winner) {
        const int src = __ffs(winner) - 1;
        const int end = __shfl_sync(kFull, last, src) + 1;
        double acc = __shfl_sync(kFull, before, src);
        int pick = end - 1;
        for (int i0 = __shfl_sync(kFull, row.lo, src); i0 < end; i0 += 32) {
          const int i = i0 + lane;
          const float x = i < end ? to_float(vals[i]) : 0.0f;
          double w = i < end && kept(x, row.id0 + i) ? row.weight(x) : 0.0;
          if (w < (double)min_p) w = 0.0;
          double upto = w;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += up;
          }
          const uint32_t passed = __ballot_sync(kFull, w > 0.0 && acc + upto > target);
          if (passed) {
            pick = i0 + __ffs(passed) - 1;
            break;
          }
          acc += __shfl_sync(kFull, upto, 31);
        }
        writer = lane == src;
        token = row.id0 + pick;
        logprob = (float)log(row.weight(to_float(vals[pick])) / z);
      }
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
  // No barrier: behind the last one no block touches another's memory.
}

constexpr size_t smem_for(int per, size_t size) { return (size_t)per * kThreads * size + 16; }
// Consecutive tokens of a thread: an odd number, so that the 32 threads of a
// warp read 32 banks.
constexpr int per_thread(int vocab, int cluster) {
  return ((vocab + cluster * kThreads - 1) / (cluster * kThreads)) | 1;
}
static_assert(smem_for(per_thread(MK_SAMPLE_MAX_VOCAB, kCluster), 4) + sizeof(Shared) <= 227 * 1024,
              "the largest vocabulary does not fit the cluster's shared memory");

// What a device allows the kernel, asked once: shared memory, clusters of 16
// blocks, and how many of those run at the same time, with one block on a
// multiprocessor and with two.
struct Allowed {
  std::once_flag once;
  cudaError_t error = cudaSuccess;
  int wide[2] = {0, 0};
};
constexpr size_t kHalfDevice = 113 * 1024;   // shared memory of a block, where two run
constexpr int kMaxDevices = 64;

template <typename T>
const Allowed& allowed(int device) {
  static Allowed all[kMaxDevices];
  Allowed& a = all[device];
  std::call_once(a.once, [&] {
    auto kernel = sample_kernel<T>;
    constexpr int most = (int)smem_for(per_thread(MK_SAMPLE_MAX_VOCAB, kCluster), sizeof(T));
    a.error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (a.error != cudaSuccess) return;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      (void)cudaGetLastError();
      return;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kThreads);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kMaxCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    for (int two = 0; two < 2; ++two) {
      cfg.dynamicSmemBytes = two ? kHalfDevice - sizeof(Shared) : (size_t)most;
      if (cudaOccupancyMaxActiveClusters(&a.wide[two], kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        a.wide[two] = 0;
      }
    }
  });
  return a;
}

template <typename T>
cudaError_t launch_sample(const SampleParams& p0, int device, cudaStream_t stream) {
  if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  const Allowed& a = allowed<T>(device);
  if (a.error != cudaSuccess) return a.error;
  SampleParams p = p0;
  // Blocks of a row: four tokens a thread at least; 16 where all rows then still
  // run at once (7 on B200; 4 rows of 151552 with top_p: 30.6 us, with 8 blocks
  // 39.8; with 8 rows one would wait for the others).
  int c = 1;
  while (c < kCluster && p.V > c * kThreads * 4) c *= 2;
  if (c == kCluster && p.V > c * kThreads * 4) {
    const size_t block = smem_for(per_thread(p.V, kMaxCluster), sizeof(T)) + sizeof(Shared);
    if (p.B <= a.wide[block <= kHalfDevice]) c = kMaxCluster;
  }
  p.per = per_thread(p.V, c);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.B * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_for(p.per, sizeof(T));
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
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
  if (a->type == MK_FP32) return from_cuda(launch_sample<float>(p, a->device, stream));
  if (a->type == MK_BF16) return from_cuda(launch_sample<__nv_bfloat16>(p, a->device, stream));
  return from_cuda(launch_sample<__half>(p, a->device, stream));
}

}  // namespace ops
}  // namespace mk

extern "C" mk_status mk_sample(const mk_sample_args* args, void* stream) {
  return mk::ops::sample(args, nullptr, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}
