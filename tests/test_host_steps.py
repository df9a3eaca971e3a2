"""The host side of the decode loop's steps (host-compiled, no GPU): what a step
does when a launch fails part-way, or when its stream is being captured.

mk_host.cpp and mk_plan.cpp are compiled with g++ and linked against a fake of
the few CUDA runtime calls that they make (device memory is host memory) and of
the kernels' launch functions, which count and fail when told to.  Counters are
kept as the kernels would leave them: every launch of the interpreter or of the
attention adds to a tally that a reset clears.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_persistent_cta_b200", "csrc")
CUDA = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
             if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)

FAKE = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include "mk.h"
#include "mk_internal.h"
#include "ops_step.h"

// ---- the runtime: host memory, no streams ----
static cudaStreamCaptureStatus g_capture = cudaStreamCaptureStatusNone;
static int g_allocs = 0;
extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) { ++g_allocs; *p = std::calloc(n + 256, 1); return cudaSuccess; }
cudaError_t cudaFree(void* p) { std::free(p); return cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { std::memcpy(d, s, n); return cudaSuccess; }
cudaError_t cudaMemset(void* d, int v, size_t n) { std::memset(d, v, n); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { std::memset(d, v, n); return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDeviceCount(int* n) { *n = 1; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 148; return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = g_capture; return cudaSuccess; }
static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPoint(const char*, void** f, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}

// ---- the kernels: counted, failing when told to ----
static int g_interp = 0, g_append = 0, g_attend = 0, g_sample = 0, g_added = 0, g_checked = 0;
static int g_fail_interp = -1, g_fail_append = -1, g_fail_attend = -1, g_fail_sample = -1;
static uint32_t g_epoch = 0;
static uint32_t* g_counters = nullptr;
static std::vector<int> g_touched;   // counters that a shared step adds to ahead of its launches
static void clear_tally() { g_interp = g_append = g_attend = g_sample = g_added = 0; }
namespace mk {
cudaError_t launch_interp(const Params& p, int, cudaStream_t) {
  g_epoch = p.epoch;
  return g_interp++ == g_fail_interp ? cudaErrorLaunchOutOfResources : cudaSuccess;
}
cudaError_t max_coresident(int, int* n) { *n = 1; return cudaSuccess; }
mk_status static_scratch_setup(int) { return MK_OK; }
namespace ops {
mk_status prefix_attention(const mk_prefix_attention_args*, const StepSink&, cudaStream_t) {
  return g_attend++ == g_fail_attend ? MK_ERR_CUDA : MK_OK;
}
mk_status sample(const mk_sample_args*, int32_t*, int32_t*, int32_t*, cudaStream_t) {
  return g_sample++ == g_fail_sample ? MK_ERR_CUDA : MK_OK;
}
cudaError_t check_equal(const int32_t*, const int32_t*, int, int32_t*, cudaStream_t) {
  ++g_checked;
  return cudaSuccess;
}
cudaError_t add_to_counters(uint32_t* c, const int32_t* pairs, int n, cudaStream_t) {
  ++g_added;
  g_counters = c;
  g_touched.clear();
  for (int i = 0; i < n; ++i) {
    c[pairs[2 * i]] += (uint32_t)pairs[2 * i + 1];
    g_touched.push_back(pairs[2 * i]);
  }
  return cudaSuccess;
}
}  // namespace ops
}  // namespace mk
extern "C" mk_status mk_rope_append(const mk_rope_append_args*, void*) {
  return g_append++ == g_fail_append ? MK_ERR_CUDA : MK_OK;
}
extern "C" size_t mk_prefix_attention_workspace(const mk_prefix_attention_args*) { return 4096; }

// ---- a context of the tiny shape ----
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
constexpr int L = 2, B = 3, V = 64, STEPS = 4;
alignas(16) static char g_mem[1024];
static const void* g_ptrs[L] = {g_mem, g_mem};
static void* g_pools[L] = {g_mem, g_mem};
static int32_t tokens[B], positions[B], table[B * 8], lens[B], out[STEPS * B], starts[2] = {0, B}, prefix[1] = {0};
static float logits[B * V], u[STEPS * B];
static mk_ctx* make() {
  mk_config c{L, 256, 4, 2, 64, 8, 2, 512, V, 64, 8, 32, 1e4f, 1e-5f};
  mk_tensors t{};
  t.embed = t.lm_head = t.final_norm = g_mem;
  t.attn_norm = t.w_qkv = t.w_o = t.w_router = t.w_gate = t.w_up = t.w_down = g_ptrs;
  t.k_pool = t.v_pool = g_pools;
  mk_ctx* ctx = nullptr;
  if (mk_create(&c, &t, 0, &ctx) != MK_OK) return nullptr;
  int32_t n[B] = {0, 10, 100};
  if (mk_build_schedule(ctx, B, n, nullptr, 8) != MK_OK) return nullptr;
  return ctx;
}
static mk_status step(mk_ctx* c) { return mk_decode_step(c, tokens, positions, table, lens, logits, nullptr); }
static mk_status shared(mk_ctx* c) {
  return mk_decode_step_shared(c, tokens, positions, table, lens, 1, starts, prefix, logits, nullptr);
}
static mk_status sampled(mk_ctx* c, int n_groups, int n = STEPS) {
  mk_sampling how{};
  how.u = u;
  how.group_start = starts;
  how.prefix_lens = prefix;
  how.n_groups = n_groups;
  return mk_decode_sample(c, n, tokens, positions, table, lens, logits, out, &how, nullptr);
}
"""

CASES = {
    "ordinary": r"""
  CHECK(shared(c) == MK_OK && g_interp == L + 1 && g_append == L && g_attend == L && g_added == 1 && g_epoch == 1);
  CHECK(step(c) == MK_OK && g_epoch == 2 && mk_check(c, nullptr, nullptr) == MK_OK);
  clear_tally();
  CHECK(sampled(c, 1) == MK_OK && g_checked == 1 && g_sample == STEPS && g_attend == STEPS * L && g_epoch == 2 + STEPS);
  CHECK(sampled(c, 0) == MK_OK && g_sample == 2 * STEPS && g_epoch == 2 + 2 * STEPS);
""",
    "captured": r"""
  // the epoch is an argument of the launches: a replayed step would wait for counts long passed
  CHECK(shared(c) == MK_OK && g_epoch == 1);
  clear_tally();
  g_capture = cudaStreamCaptureStatusActive;
  const int allocs = g_allocs;
  CHECK(shared(c) == MK_ERR_STATE && sampled(c, 1) == MK_ERR_STATE && sampled(c, 0) == MK_ERR_STATE);
  CHECK(sampled(c, 1, 0) == MK_OK);       // no step: nothing to launch
  CHECK(g_interp == 0 && g_added == 0 && g_sample == 0 && g_checked == 0 && g_allocs == allocs);
  g_capture = cudaStreamCaptureStatusNone;
  CHECK(shared(c) == MK_OK && g_epoch == 2);
""",
    "refused": r"""
  // group counts that are no counts, and group arrays that are not there
  CHECK(sampled(c, -1) == MK_ERR_INVALID && sampled(c, B + 1) == MK_ERR_INVALID && sampled(c, -1, 0) == MK_ERR_INVALID);
  mk_sampling how{};
  how.u = u;
  how.n_groups = 1;
  CHECK(mk_decode_sample(c, 1, tokens, positions, table, lens, logits, out, &how, nullptr) == MK_ERR_INVALID);
  CHECK(mk_decode_step_shared(c, tokens, positions, table, lens, 0, starts, prefix, logits, nullptr) == MK_ERR_INVALID);
  CHECK(mk_decode_step_shared(c, tokens, positions, table, lens, 1, starts, nullptr, logits, nullptr) == MK_ERR_INVALID);
  CHECK(g_interp == 0 && g_added == 0 && g_sample == 0 && shared(c) == MK_OK);
""",
    "cut_short": r"""
  // whichever launch of a shared step fails: nothing runs on the counters that it left short
  // until mk_check, or a new schedule, has cleared them
  CHECK(shared(c) == MK_OK);
  for (int which = 0; which < 8; ++which) {
    clear_tally();
    int* fail = which < 3 ? &g_fail_interp : which < 5 ? &g_fail_append : &g_fail_attend;
    if (which == 7) fail = &g_fail_sample;
    *fail = which < 3 ? which : which < 5 ? which - 3 : which < 7 ? which - 5 : 0;
    CHECK(sampled(c, 1) == MK_ERR_CUDA);
    *fail = -1;
    const int ran = g_interp + g_append + g_attend + g_added;
    if (which == 7) {                     // between two steps: both can go on
      CHECK(step(c) == MK_OK && shared(c) == MK_OK && mk_check(c, nullptr, nullptr) == MK_OK);
      continue;
    }
    CHECK(shared(c) == MK_ERR_STATE && step(c) == MK_ERR_STATE && sampled(c, 0) == MK_ERR_STATE);
    CHECK(mk_decode_greedy(c, 1, tokens, positions, table, lens, logits, out, nullptr) == MK_ERR_STATE);
    CHECK(g_interp + g_append + g_attend + g_added == ran && g_sample == 0);
    if (which % 2) {
      CHECK(mk_check(c, nullptr, nullptr) == MK_OK);
    } else {
      int32_t n[B] = {0, 10, 100};
      CHECK(mk_build_schedule(c, B, n, nullptr, 8) == MK_OK);
    }
    CHECK(!g_touched.empty());
    for (int i : g_touched) CHECK(g_counters[i] == 0);
    CHECK((which % 2 ? shared(c) : step(c)) == MK_OK && g_epoch == 1);
    CHECK(step(c) == MK_OK && g_epoch == 2);
  }
""",
}


def run(tmp_path, body):
    src, exe = str(tmp_path / "steps.cpp"), str(tmp_path / "steps")
    with open(src, "w") as f:
        f.write(FAKE + "int main() {\n  mk_ctx* c = make();\n  CHECK(c);\n" + body
                + "\n  mk_destroy(c);\n  return 0;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(CUDA, "include"), src, os.path.join(CSRC, "mk_host.cpp"),
                    os.path.join(CSRC, "mk_plan.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr


@pytest.mark.skipif(shutil.which("g++") is None or CUDA is None, reason="needs a host C++ compiler and CUDA's headers")
@pytest.mark.parametrize("name", sorted(CASES))
def test_steps_on_the_host(tmp_path, name):
    run(tmp_path, CASES[name])
