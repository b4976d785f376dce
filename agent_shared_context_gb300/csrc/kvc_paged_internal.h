// kvc_paged_internal.h -- launch interface between the host layer of the paged
// cache (kvc_paged.cu) and its kernels.  Not part of the public ABI.
#pragma once

#include <utility>

#include "kvc_internal.h"

namespace kvc {

// The kernels of the paged cache follow one another on a stream many times a step, and
// most of them run for a few microseconds: each is launched while the one before it
// ends, prepares itself and then waits for its results (grid_wait).
template <typename... P, typename... A>
cudaError_t launch_early(void (*fn)(P...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...);
}

#ifdef __CUDACC__
// Nothing that an earlier kernel may have written is read before this, and what is
// read after it is read by ordinary loads: it was not constant since the launch.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

// Requests of one kvc_page_plan call: their scans live in shared memory.
constexpr int kMaxPlanRequests = 4096;

struct PlanArgs {
  const int32_t* new_lens;
  const int32_t* kv_in;
  int32_t* kv_out;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* n_free_in;
  int32_t* n_free_out;
  int32_t* q_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* status;
  int32_t R, P, B, width, max_tokens;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream);

struct WriteArgs {
  View src[2], pool[2];       // src [Rs, nl, H, T, d]; pool [P, L, H, B, d]
  const int64_t* slots;       // [Rs * T]
  int64_t rows;               // Rs * T
  int64_t n_slots;            // P * B
  int32_t T, B, L0, nl, H;
  int32_t vec_row;            // 16-byte vectors per row
  int32_t elem;               // bytes per element
};
cudaError_t launch_page_write(const WriteArgs& a, cudaStream_t stream);

// Paged attention.  q and out are [N, Hq, d] with element strides.
struct AttnArgs {
  const void* q;
  void* out;
  float* lse;                 // [N, Hq] or nullptr
  int64_t q_tok, q_head, o_tok, o_head;
  View pool[2];               // [P, L, H, B, d]
  const int32_t* table;       // [R, width]
  const int32_t* q_start;     // [R + 1]
  const int32_t* kv_lens;     // [R]
  int32_t R, N, H, G, d, P, L, B, width, layer, causal, window;
  float scale_log2;           // scale * log2(e)
  void* workspace;
  int32_t* dev_status;
};

// Bytes of the workspace: arrival counters (zero between calls), then the
// partial rows of divided items.
constexpr size_t kAttnCounterBytes = 8192;
size_t attn_f32_workspace_bytes(int d);   // f32
cudaError_t launch_attn_f32(const AttnArgs& a, cudaStream_t stream);
size_t attn_tc_workspace_bytes(int d);     // bf16, d = 64 or 128
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream);
// bf16, decoding; its workspace is part of the one above.
bool attn_decode_fits(const AttnArgs& a);
cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream);

}  // namespace kvc
