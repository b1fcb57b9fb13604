// Status codes, error messages and argument checks shared by the C ABI sources
// (defined in qmoe_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"

#define REQUIRE(cond, code, ...)                         \
  do {                                                   \
    if (!(cond)) return qmoe::fail((code), __VA_ARGS__); \
  } while (0)

namespace qmoe {

int fail(int code, const char *fmt, ...);              // records the message, returns code
int ok();                                              // clears it, returns MOE_OK
int hip_status(hipError_t e, const char *what);        // MOE_OK or MOE_EHIP

int check_routing_sizes(int M, int E, int top_k, const char *fn);
long long max_padded_ll(int M, int E, int top_k, int block_m);

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool valid_block_m(int b) {
  return b == 16 || b == 32 || b == 64 || b == 128 || b == 256;
}

}  // namespace qmoe
