// The linear layer: arguments shared by the C ABI and the passes (linear.hip, linear_rows.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/externd.h"

namespace externd {

struct LinearArgs {
  const void *x, *w, *bias, *residual;
  int64_t tokens, cols, rows;
  int64_t ldx, ldw, ldr;
  int dtype, act;
  void* y;
  float* z;               // forward: x W^T + bias, kept, or null; backward: read where there is an activation
  const void* dy;
  int64_t lddy;
  void *dx, *dw, *db;     // backward outputs, each may be null
  int cus;
};

// x and W start on 16 bytes, their row strides and the columns are multiples of 8 entries
bool linear_is_aligned(const LinearArgs& a);
// whether the backward products read dy itself
bool linear_reads_dy(const LinearArgs& a);
size_t linear_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus);
hipError_t run_linear_forward(const LinearArgs& a, void* ws, hipStream_t s);
// reads_dy: as linear_reads_dy gives it
size_t linear_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int act, bool aligned, bool reads_dy, int cus);
hipError_t run_linear_backward(const LinearArgs& a, void* ws, hipStream_t s);
hipError_t run_linear_rows(const LinearArgs& a, hipStream_t s);

}  // namespace externd
