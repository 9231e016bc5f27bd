// The AdamW step: arguments shared by the C ABI and the kernels (adamw.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/externd.h"

namespace externd {

constexpr int kAdamBlock = EXTERND_ADAMW_BLOCK;   // entries that share an exponent
constexpr int kAdamTensors = 48;                  // tensors of a launch: they travel in its 4 KB of arguments

struct AdamTensor {
  void* p;
  const void* g;
  float* master;
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  int64_t n;
  uint32_t first;   // its first chunk
  float decay;
};

struct AdamArgs {
  AdamTensor t[kAdamTensors];
  int count;
  uint32_t chunks;
  double lr, b1, b2, eps;
  const float *lr_device, *scale_device;   // or null
  float scale;
  int advance;      // whether this launch counts the step
  double* step;     // steps taken, their powers of the betas, workgroups that have arrived
};
static_assert(sizeof(AdamArgs) <= 4096, "a launch's arguments");

hipError_t run_adamw(const externd_adamw_tensor* tensors, int64_t count, const externd_adamw_opts& o, int cus, hipStream_t s);
hipError_t run_adamw_moments(const uint8_t* m, const uint8_t* m_exp, const uint8_t* v, const uint8_t* v_exp, int64_t blocks,
                             float* m_out, float* v_out, int cus, hipStream_t s);

}  // namespace externd
