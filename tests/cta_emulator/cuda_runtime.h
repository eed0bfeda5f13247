// Runs kernels on the host, a CTA at a time, to test what the order of a CTA's
// threads must not change.  A C++ compiler that finds this header in the place
// of CUDA's own compiles a kernel's source as it is: every CUDA thread is a
// fiber that runs until it has to wait (__syncthreads, __syncwarp, a shuffle or
// a vote), and the next one is picked in an order that the test sets.  Nothing
// keeps the lanes of a warp together but what the kernel itself asks for.
//
// Only what the page operations use is here.  Memory is sequentially
// consistent, launches run at once, copies and stream waits too.
#pragma once
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <memory>
#include <utility>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __shared__ static
#define __grid_constant__
#define __launch_bounds__(...)
#define asm
#define volatile(...) ((void)0)  // (only inline PTX opens a parenthesis there)

using std::max;
using std::min;

struct dim3 {
    unsigned x, y, z;
    dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};
struct int4 { int x, y, z, w; };
struct alignas(16) uint4 { unsigned x, y, z, w; };
inline int4 make_int4(int x, int y, int z, int w) { return {x, y, z, w}; }

enum cudaError_t { cudaSuccess = 0, cudaErrorUnknown = 999 };
typedef struct CUstream_st* cudaStream_t;
enum cudaMemcpyKind { cudaMemcpyDeviceToHost = 2 };
enum cudaLaunchAttributeID { cudaLaunchAttributeProgrammaticStreamSerialization = 6 };
struct cudaLaunchAttribute {
    int id;
    struct { int programmaticStreamSerializationAllowed; } val;
};
struct cudaLaunchConfig_t {
    dim3 gridDim, blockDim;
    size_t dynamicSmemBytes;
    cudaStream_t stream;
    cudaLaunchAttribute* attrs;
    unsigned numAttrs;
};

inline dim3 threadIdx, blockIdx, blockDim, gridDim;

namespace emu {

enum Order { kAscending, kDescending, kRandom };
inline int order = kAscending;
inline uint64_t rng = 1;
inline void (*at_stream_wait)() = nullptr;  // what other streams do while the host waits
inline uint64_t draw() {
    rng ^= rng << 13;
    rng ^= rng >> 7;
    rng ^= rng << 17;
    return rng;
}

constexpr size_t kStack = 64 << 10;
enum State { kReady, kBarrier, kWarp, kDone };
struct Fiber {
    ucontext_t ctx;
    std::unique_ptr<char[]> stack;
    State state;
    unsigned mask;        // of the collective it waits in
    uint64_t gave;        // its value there
    uint64_t got[32];     // every lane's value
};
inline std::vector<Fiber> fibers;
inline ucontext_t scheduler;
inline int current;
inline std::function<void()> body;

inline void entry() {
    body();
    fibers[current].state = kDone;
    swapcontext(&fibers[current].ctx, &scheduler);
}
inline void yield(State s) {
    Fiber& f = fibers[current];
    f.state = s;
    swapcontext(&f.ctx, &scheduler);
}
inline const uint64_t* collective(unsigned mask, uint64_t value) {
    Fiber& f = fibers[current];
    f.mask = mask;
    f.gave = value;
    yield(kWarp);
    return fibers[current].got;
}
[[noreturn]] inline void fail(const char* what) {
    std::fprintf(stderr, "cta emulator: %s\n", what);
    std::abort();
}

// Lets those go whose collective, or barrier, is complete.
inline bool release(int n) {
    bool any = false;
    for (int w = 0; w < n; w += 32)
        for (int lane = 0; lane < 32 && w + lane < n; ++lane) {
            if (fibers[w + lane].state != kWarp) continue;
            const unsigned mask = fibers[w + lane].mask;
            bool all = true;
            for (int i = 0; i < 32; ++i)
                if ((mask >> i) & 1)
                    all &= w + i < n && fibers[w + i].state == kWarp && fibers[w + i].mask == mask;
            if (!all) continue;
            for (int i = 0; i < 32; ++i) {
                if (!((mask >> i) & 1)) continue;
                for (int k = 0; k < 32; ++k)
                    fibers[w + i].got[k] = (mask >> k) & 1 ? fibers[w + k].gave : 0;
            }
            for (int i = 0; i < 32; ++i)
                if ((mask >> i) & 1) fibers[w + i].state = kReady;
            any = true;
        }
    if (any) return true;
    bool all = true, some = false;
    for (int i = 0; i < n; ++i) {
        all &= fibers[i].state == kBarrier || fibers[i].state == kDone;
        some |= fibers[i].state == kBarrier;
    }
    if (!all || !some) return false;
    for (int i = 0; i < n; ++i)
        if (fibers[i].state == kBarrier) fibers[i].state = kReady;
    return true;
}

inline void run_cta(int n) {
    if ((int)fibers.size() < n) fibers.resize(n);
    for (int i = 0; i < n; ++i) {
        Fiber& f = fibers[i];
        if (!f.stack) f.stack.reset(new char[kStack]);
        getcontext(&f.ctx);
        f.ctx.uc_stack.ss_sp = f.stack.get();
        f.ctx.uc_stack.ss_size = kStack;
        f.ctx.uc_link = nullptr;
        makecontext(&f.ctx, entry, 0);
        f.state = kReady;
    }
    std::vector<int> ready;
    for (;;) {
        ready.clear();
        for (int i = 0; i < n; ++i)
            if (fibers[i].state == kReady) ready.push_back(i);
        if (order == kDescending) std::reverse(ready.begin(), ready.end());
        if (order == kRandom)
            for (size_t i = ready.size(); i > 1; --i) std::swap(ready[i - 1], ready[draw() % i]);
        for (int i : ready) {
            current = i;
            threadIdx = dim3(i);
            swapcontext(&scheduler, &fibers[i].ctx);
        }
        if (ready.empty() && !release(n)) break;
    }
    for (int i = 0; i < n; ++i)
        if (fibers[i].state != kDone) fail("threads wait for others that never come");
}

inline uint64_t bits_of(const void* p, size_t n) {
    uint64_t x = 0;
    std::memcpy(&x, p, n);
    return x;
}
template <typename T>
T value_of(uint64_t x) {
    T t;
    std::memcpy(&t, &x, sizeof(T));
    return t;
}

}  // namespace emu

template <typename... K, typename... A>
cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t* cfg, void (*kern)(K...), A&&... args) {
    gridDim = cfg->gridDim;
    blockDim = cfg->blockDim;
    const unsigned n = gridDim.x * gridDim.y;
    const unsigned first = emu::order == emu::kRandom ? (unsigned)(emu::draw() % n) : 0;
    emu::body = [&] { kern(K(args)...); };
    for (unsigned i = 0; i < n; ++i) {  // CTAs from any one on, or backwards
        unsigned c = (first + i) % n;
        if (emu::order == emu::kDescending) c = n - 1 - c;
        blockIdx = dim3(c % gridDim.x, c / gridDim.x);
        emu::run_cta((int)blockDim.x);
    }
    return cudaSuccess;
}
inline cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
    std::memcpy(d, s, n);
    return cudaSuccess;
}
inline cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) {
    std::memset(d, v, n);
    return cudaSuccess;
}
inline cudaError_t cudaStreamSynchronize(cudaStream_t) {
    if (emu::at_stream_wait) emu::at_stream_wait();
    return cudaSuccess;
}

inline void __syncthreads() { emu::yield(emu::kBarrier); }
inline void __syncwarp(unsigned mask = 0xffffffffu) { emu::collective(mask, 0); }
inline unsigned __ballot_sync(unsigned mask, bool x) {
    const uint64_t* got = emu::collective(mask, x);
    unsigned out = 0;
    for (int i = 0; i < 32; ++i) out |= (unsigned)(got[i] & 1) << i;
    return out;
}
template <typename T>
T __shfl_sync(unsigned mask, T v, int src, int width = 32) {
    const int lane = emu::current & 31;
    const uint64_t* got = emu::collective(mask, emu::bits_of(&v, sizeof(T)));
    return emu::value_of<T>(got[(lane & ~(width - 1)) | (src & (width - 1))]);
}
template <typename T>
T __shfl_up_sync(unsigned mask, T v, unsigned by) {
    const int lane = emu::current & 31;
    const uint64_t* got = emu::collective(mask, emu::bits_of(&v, sizeof(T)));
    return lane >= (int)by ? emu::value_of<T>(got[lane - by]) : v;
}
inline int __popc(unsigned x) { return __builtin_popcount(x); }
inline uint4 __ldcs(const uint4* p) { return *p; }
inline void __stcs(uint4* p, uint4 v) { *p = v; }
inline int atomicCAS(int* p, int expect, int v) {
    const int old = *p;
    if (old == expect) *p = v;
    return old;
}
inline int atomicOr(int* p, int v) { const int old = *p; *p |= v; return old; }
inline int atomicAnd(int* p, int v) { const int old = *p; *p &= v; return old; }
inline int atomicAdd(int* p, int v) { const int old = *p; *p += v; return old; }
inline int atomicSub(int* p, int v) { const int old = *p; *p -= v; return old; }
inline int atomicExch(int* p, int v) { const int old = *p; *p = v; return old; }

extern "C" inline void emu_order(int order, unsigned long long seed) {
    emu::order = order;
    emu::rng = seed * 2 + 1;
}
extern "C" inline void emu_at_stream_wait(void (*f)()) { emu::at_stream_wait = f; }
