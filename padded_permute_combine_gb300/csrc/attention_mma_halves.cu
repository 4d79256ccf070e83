// Decode attention of bf16 caches: rows off 4 bytes.
#include "attend_mma.h"

int moe::attend_mma_2(AttendArgs& a, cudaStream_t s) { return launch_mma_dim<2>(a, s); }
