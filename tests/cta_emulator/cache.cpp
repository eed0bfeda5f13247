// The page operations' source as the host runs it.
#include "cuda_runtime.h"

#include "../../bwd_tiled_attention_gb300/csrc/cache.cu"

extern "C" void order_threads(int order, unsigned long long seed) { emu_order(order, seed); }
extern "C" void at_stream_wait(void (*f)()) { emu_at_stream_wait(f); }
