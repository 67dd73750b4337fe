// Functions that a kernel and a program on the host compile alike.
#pragma once

#ifdef __HIP__
#include <hip/hip_runtime.h>
#define MX_BOTH_SIDES __host__ __device__ __forceinline__
#else
#define MX_BOTH_SIDES inline
#endif
