// api_util.hpp -- what the files of the C ABI share: the calling thread's error
// message, the checks of pointers, and device facts looked up once.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mx_api {

int fail(int code, const char* fmt, ...);   // records the message, returns code
int ok();                                   // clears it, returns MXFP8_OK
int hip_status(hipError_t e, const char* what);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_fmt(int f);
inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
// CUs of the device that `st` runs on (0 if unknown)
int device_cus(hipStream_t st);
// An expert weight operand at least this large (8x one XCD's 4 MB L2) is shared
// by all XCDs through the infinity cache: its GEMM hands tiles out round robin
// (moe_tiles.hpp).
constexpr int64_t kRoundRobinWeightBytes = int64_t(32) << 20;

}  // namespace mx_api
