// Shared by the library's source files; nothing here is exported.
#ifndef SGEMV_INTERNAL_H
#define SGEMV_INTERNAL_H

#include "sgemv.h"

// Keep a failed HIP call's hipError_t for sgemv_last_hip_error.
__attribute__((visibility("hidden"))) int sgemv_hip_failed(int hip_error);

// SGEMV_OK when *d is a description that the q4 packer makes.
__attribute__((visibility("hidden"))) int sgemv_q4_check_desc(const sgemv_q4_desc* d);

#endif
