// fwd_window.cu -- the forward of fwd.cu for a sliding window with sinks: the same
// kernels with the window's tiles and mask, compiled as a unit of their own (both
// take as long as the longest of the others).
#define FA_WINDOW 1
#include "fwd.cu"
