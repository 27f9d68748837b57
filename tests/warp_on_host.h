// warp_on_host.h -- a warp's device code run on the host: 32 fibres that take turns between the operations that exchange
// values.  Every lane has to reach each of these operations.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#include <cuda_runtime.h>

struct HostIndex {
    unsigned x;
};
static HostIndex threadIdx, blockIdx, gridDim;
using std::max;
using std::min;

namespace host_warp {

struct Warp {
    ucontext_t home, at[32];
    std::vector<char> stacks;
    bool done[32];
    int lane, turn[32];
    uint32_t slot[2][32];
    void (*body)(void*);
    void* arg;
};
static Warp w;

static void lane_main() {
    w.body(w.arg);
    w.done[w.lane] = true;
    swapcontext(&w.at[w.lane], &w.home);
}
// Every lane's value; back when all have given theirs.
static const uint32_t* exchange(uint32_t x) {
    const int lane = w.lane;
    uint32_t* slot = w.slot[w.turn[lane]++ & 1];
    slot[lane] = x;
    swapcontext(&w.at[lane], &w.home);
    return slot;
}
static void run(unsigned block, unsigned first_thread, void (*body)(void*), void* arg) {
    constexpr size_t kStack = 128 << 10;
    w.stacks.resize(32 * kStack);
    w.body = body, w.arg = arg;
    blockIdx.x = block;
    for (int i = 0; i < 32; ++i) {
        getcontext(&w.at[i]);
        w.at[i].uc_stack.ss_sp = w.stacks.data() + i * kStack;
        w.at[i].uc_stack.ss_size = kStack;
        w.at[i].uc_link = nullptr;
        makecontext(&w.at[i], lane_main, 0);
        w.done[i] = false, w.turn[i] = 0;
    }
    for (bool left = true; left;) {
        left = false;
        for (int i = 0; i < 32; ++i) {
            if (w.done[i]) continue;
            w.lane = i;
            threadIdx.x = first_thread + i;
            swapcontext(&w.home, &w.at[i]);
            left = left || !w.done[i];
        }
    }
}

}  // namespace host_warp

template <class T>
static T __ldg(const T* p) { return *p; }
static int __shfl_sync(unsigned, int x, int lane) { return static_cast<int>(host_warp::exchange(x)[lane & 31]); }
static int __shfl_up_sync(unsigned, int x, int by) {
    const int from = host_warp::w.lane - by;
    const uint32_t* all = host_warp::exchange(x);
    return from >= 0 ? static_cast<int>(all[from]) : x;
}
static unsigned __ballot_sync(unsigned, bool x) {
    const uint32_t* all = host_warp::exchange(x);
    unsigned bits = 0;
    for (int i = 0; i < 32; ++i) bits |= (all[i] ? 1u : 0u) << i;
    return bits;
}
static bool __all_sync(unsigned mask, bool x) { return __ballot_sync(mask, x) == 0xffffffffu; }
static int __ffs(int x) { return __builtin_ffs(x); }
static int __popc(unsigned x) { return __builtin_popcount(x); }
