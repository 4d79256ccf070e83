// Decode attention of bf16 caches: rows of 4-byte words.
#include "attend_mma.h"

int moe::attend_mma_4(AttendArgs& a, cudaStream_t s) { return launch_mma_dim<4>(a, s); }
