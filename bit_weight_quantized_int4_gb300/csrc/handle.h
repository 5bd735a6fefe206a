// The handle behind the C ABI and what its entry points share (q4lin.cpp, operators.cpp):
// the device guard, checked size arithmetic and the launch context.
#pragma once

#include "../../include/q4lin.h"

#include <cuda_runtime.h>
#include <stdint.h>

#include "q4lin_internal.h"

struct q4lin_handle {
    int device = 0;
    int sm_count = 0;
    int max_smem_optin = 0;
    int force_path = Q4LIN_PATH_AUTO;
    int even_high = 0;
    int pdl = 0;
    int64_t wait_limit = 0;  // ns; 0: default
    int tc_skip_first_copy = 0;
    int tc_f16 = 0;
    int tc_small_operands = 0;
    int64_t attention_split_rows = 0;  // 0: the measured rule
    int* d_status = nullptr;
    float* d_ws = nullptr;     // split-K partial sums
    int* d_tickets = nullptr;  // split-K row-block counters (zero between launches)
};

namespace q4lin {

constexpr int64_t kDefaultWaitLimit = 2000000000LL;  // 2 s of GPU global time
// Scratch of a handle: partial sums of split-K launches and their row-block counters.
constexpr int64_t kWsFloats = 1 << 24;   // 64 MiB (split-K partials; the fp16 copy of x)
constexpr int64_t kTickets = 1 << 14;    // 64 KiB

class DeviceGuard {
   public:
    explicit DeviceGuard(int device) {
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        if (prev_ != device) ok_ = cudaSetDevice(device) == cudaSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev_) cudaSetDevice(prev_);
    }
    bool ok() const { return ok_; }

   private:
    int prev_ = -1;
    bool ok_ = true;
};

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

inline LaunchCtx make_ctx(q4lin_handle_t h, cudaStream_t stream) {
    LaunchCtx c;
    c.stream = stream;
    c.sm_count = h->sm_count;
    c.max_smem_optin = h->max_smem_optin;
    c.pdl = h->pdl;
    c.status_word = h->d_status;
    c.wait_limit_ns = h->wait_limit > 0 ? h->wait_limit : kDefaultWaitLimit;
    c.tc_skip_first_copy = h->tc_skip_first_copy;
    c.tc_f16 = h->tc_f16;
    c.tc_small_operands = h->tc_small_operands;
    c.ws = h->d_ws;
    c.ws_floats = kWsFloats;
    c.tickets = h->d_tickets;
    c.ticket_count = kTickets;
    return c;
}

}  // namespace q4lin
