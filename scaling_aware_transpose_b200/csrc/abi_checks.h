// abi_checks.h — small host-side helpers of the extern "C" entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8q.h"

namespace fp8q {

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t to_stream(fp8q_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
constexpr int64_t kMaxInt32 = 0x7FFFFFFFll;  // grid sizes, group offsets and row ids are int32

}  // namespace fp8q
