// bwd_window.cu -- the backward of bwd.cu for a sliding window with sinks: the same
// kernels with the window's units and mask, and the sum of the sinks' partials,
// compiled as a unit of their own.
#define FA_WINDOW 1
#include "bwd.cu"
