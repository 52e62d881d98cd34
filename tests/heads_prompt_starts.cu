// Where each CTA of attend_heads' kernel for prompts begins its run of key tiles, for tests/test_gpu_heads_runs.py: the search alone, so that
// calls of any length can be looked at without their tensors.
#include "heads_prompt.cu"

namespace hs {
void count_launch(int) {}

namespace {
__global__ void __launch_bounds__(kThreads) starts_kernel(const HeadsAttendParams p, int limit, Start* out) {
  __shared__ Scratch scratch;
  if (threadIdx.x == 0) scratch.start = Start{};
  __syncthreads();
  find_start(p, limit, &scratch);
  if (threadIdx.x == 0) out[blockIdx.x] = scratch.start;
}
}  // namespace
}  // namespace hs

// out: a Start for each of `grid` CTAs; header: {tiles of a run, tiles of the call}.  All pointers are of the device.
extern "C" int heads_prompt_starts(int kv_heads, int group, int causal, int limit, int R, int max_pages, int64_t n, const int32_t* ctx_len,
                                   const int32_t* cu, int grid, void* out, void* header) {
  static_assert(sizeof(hs::Start) == 32 && sizeof(hs::heads::RunHeader) == 16, "what the test reads");
  hs::HeadsAttendParams p{};
  p.a.R = R, p.a.n = n, p.a.max_pages = max_pages, p.a.causal = causal, p.a.ctx_len = ctx_len, p.a.q_heads = kv_heads * group;
  p.pages.kv_heads = kv_heads, p.pages.max_pages = max_pages;
  p.ragged = hs::Ragged{cu, R, cu ? 0 : (int32_t)(n / R), n};
  p.group = group;
  p.workspace = static_cast<float*>(header);
  hs::starts_kernel<<<grid, hs::kThreads>>>(p, limit, static_cast<hs::Start*>(out));
  return cudaDeviceSynchronize();
}
