// The eviction's source as the host runs it, beside the page operations' (cache.cpp).
#include "cuda_runtime.h"

inline int __ffs(int x) { return __builtin_ffs(x); }
inline int __reduce_add_sync(unsigned mask, int v) {
    const uint64_t* got = emu::collective(mask, emu::bits_of(&v, sizeof(v)));
    int sum = 0;
    for (int i = 0; i < 32; ++i)
        if ((mask >> i) & 1) sum += emu::value_of<int>(got[i]);
    return sum;
}
enum { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
template <typename K>
cudaError_t cudaFuncSetAttribute(K, int, int) { return cudaSuccess; }

// Keys in shared memory: fewer than on the device where a test says so.
#define FA_DYNAMIC_SHARED(type, name) static type name[FA_MOST_KEYS]
#include "../../bwd_tiled_attention_gb300/csrc/evict.cu"
