// tree_window.cu -- the attention over the cache of tree.cu for a sliding window with
// sinks: the same kernels with the window's tiles and mask, compiled as a unit of
// their own.
#define FA_WINDOW 1
#include "tree.cu"
