// Arithmetic that kernels share with the host, where it is built with undefined-behaviour checks.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define NVFP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define NVFP4_HOST_DEVICE inline
#endif
