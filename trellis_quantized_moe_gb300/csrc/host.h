// Host-side checks that every entry point makes before it launches (api.cpp).
#pragma once
#include <cuda_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace exl3 {

// Device of the stream (must be the current one) and its SM count; sets the
// kernels' attributes on the first call per device.  Notes whether the stream
// is capturing, which on_device then takes into account.
int setup_device(cudaStream_t s, int *dev_out, int *sms_out);
bool on_device(const void *p, int dev);
bool aligned(const void *p, size_t a);

inline bool is_act_dtype(int d) { return d == 0 || d == 1; }             // f16, bf16
inline bool is_float_dtype(int d) { return d >= 0 && d <= 2; }           // f16, bf16, f32
inline size_t float_size(int d) { return d == 2 ? 4 : 2; }

}  // namespace exl3
