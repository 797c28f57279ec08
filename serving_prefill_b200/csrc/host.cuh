// Host-side helpers shared by the units that implement the C ABI: launch
// accounting, tensor maps and argument checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rag_prefill.h"
#include "common.cuh"

namespace rag {

// kernel kinds of the per-kernel timing (rag_profile_collect)
enum Kind { kKindPoolWrite = 0, kKindAttn, kKindCombine, kKindImpact, kKindTopk, kKindSimtAttn, kKindSimtImpact,
            kKindRcPlan, kKindRcCopy, kKindRcGemm, kKindRope, kKindKvDecode, kKindDecAttn,
            kKindKvAppend, kKindKv8Append, kKindRopeTable, kKindKv8Attn, kKindKv8Combine, kKindKv8SplitQ, kKindKv8Decode, kKindRopeQ, kNumKinds };

// Counts one launch and, while profiling is on, brackets it with events.
struct LaunchScope {
  int kind;
  cudaStream_t stream;
  cudaEvent_t start = nullptr, stop = nullptr;
  LaunchScope(int k, cudaStream_t s);
  void done(cudaError_t e);
};

// Tensor map of a bf16 (or, with bytes, 8-bit) tensor with rank (<= 3) dims
// (innermost first), 128B swizzle, zero fill.
bool make_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
              const uint32_t* box, bool bytes = false);

int num_sms();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether two ranges of bytes share one.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + uintptr_t(b_bytes) && y < x + uintptr_t(a_bytes);
}
inline int cdiv(int64_t a, int64_t b) { return int((a + b - 1) / b); }

rag_status check_pool(const rag_kv_pool* pool);
rag_status check_batch(const rag_batch* b);
BatchDev to_dev(const rag_batch& b);

}  // namespace rag
