// Decode attention of bf16 caches: rows of 16-byte pieces.
#include "attend_mma.h"

int moe::attend_mma_16(AttendArgs& a, cudaStream_t s) { return launch_mma_dim<16>(a, s); }
