// Internal interface between the C ABI of the operators around the layer
// (ops_api.cpp) and their gfx950 kernels.  Launchers validate nothing: the ABI
// layer has checked every argument before calling.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace moe {

// ---- norm.hip
struct NormArgs {
  const void* x;      // bf16, ldx elements from row to row
  int64_t ldx;
  const void* res;    // residual [M, H], or nullptr
  void* zout;         // [M, H] of the residual's type, or nullptr
  const void* w;      // bf16 [H]
  float eps;
  void* out;          // bf16, or e4m3fn codes when scale != nullptr
  float* scale;
  float* rstd;        // or nullptr
  int64_t M;
  int H;
};
hipError_t launch_norm(const NormArgs& a, bool res_f32, hipStream_t s);

struct NormBackwardArgs {
  const void* dy;
  const void* z;
  const void* w;
  const float* rstd;
  const void* dz;     // or nullptr
  void* dx;
  float* part;        // partial columns' sums, one row per workgroup; set at launch
  int64_t M;
  int H;
};
size_t norm_backward_workspace(int64_t M, int H);
hipError_t launch_norm_backward(const NormBackwardArgs& a, bool z_f32, float* dw, float* ws, hipStream_t s);

// ---- permute.hip
struct PermuteArgs {
  const void* x;        // rows of row_bytes
  const float* x_scale; // [M, scales] or nullptr
  const int32_t* perm;  // [M * top_k]
  void* out;
  float* out_scale;
  int64_t M, rows;
  int top_k, row_bytes, scales;
};
hipError_t launch_permute(const PermuteArgs& a, hipStream_t s);

struct UnpermuteArgs {
  const uint16_t* y;    // bf16 [rows, H]
  const int32_t* perm;
  const float* w;       // [M, top_k] or nullptr (all 1)
  uint16_t* out;        // bf16 [M, H]
  int64_t M, rows;
  int top_k, H;
};
hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s);

struct UnpermuteBackwardArgs {
  const uint16_t* dout;
  const uint16_t* y;
  const int32_t* perm;
  const float* w;
  uint16_t* dy;
  float* dw;            // [M, top_k]
  int64_t M, rows;
  int top_k, H;
};
hipError_t launch_unpermute_backward(const UnpermuteBackwardArgs& a, hipStream_t s);

// ---- linear.hip: the experts' products over sorted rows
struct LinearArgs {
  const int32_t* offsets;  // nullptr: one expert that holds every row
  const int32_t* counts;
  int rows, E;
  // forward: Q = x rows [rows, K], P = weights [E, N, K]; K is the depth
  // backward x: Q = dz rows [rows, parts * N], P = weights [E, N, K] by depth rows; N is the depth
  // backward w: Q = dz, P = x, both by depth rows; an expert's rows are the depth
  int N, K;
  const void* x;           // forward: x; backward w: x
  const float* x_scale;
  const void* dz;
  const void* w[2];        // weights (gate), up
  const float* ws[2];      // their 128x128 block scales
  const uint16_t* bias[2];
  const uint16_t* residual;
  void* y;                 // forward: y (bf16 or e4m3fn codes); backward x: dx
  float* y_scale;          // non-nullptr: y is 8-bit
  uint16_t* preact;
  int act;                 // moe_act
  int parts;               // 2: gated, two weights
  void* dw[2];
  int dw_f32;
  float* db[2];            // nullptr: no bias gradient
  float* part;             // backward w: partial sums of the row splits (splits > 1)
  int splits;
};
hipError_t launch_linear(const LinearArgs& a, bool fp8, hipStream_t s);
hipError_t launch_linear_backward_x(const LinearArgs& a, hipStream_t s);
// Row splits of the weight gradient and the floats of workspace they take.
int backward_w_splits(int64_t rows, int E, int N, int K, int parts);
hipError_t launch_linear_backward_w(const LinearArgs& a, hipStream_t s);
hipError_t launch_act_backward(const LinearArgs& a, const uint16_t* dy, const uint16_t* pre, uint16_t* dz, hipStream_t s);

// ---- linear_mx.hip: the same products on MXFP4 weights
struct MxLinearArgs : LinearArgs {
  const uint8_t* xs;       // scale bytes of MXFP4 rows x, or nullptr: bf16 rows
  const uint8_t* wsb[2];   // the weights' scale bytes
  uint8_t* ysb;            // non-nullptr: y is MXFP4 rows
};
hipError_t launch_linear_mx(const MxLinearArgs& a, hipStream_t s);
hipError_t launch_linear_mx_backward_x(const MxLinearArgs& a, hipStream_t s);

// ---- mx.hip
struct MxQuantizeArgs {
  const void* x;        // bf16 or float32, ldx elements from row to row
  int64_t ldx;
  const int32_t* perm;  // [M * top_k] rows the tokens go to, or nullptr: row t to row t
  int top_k;
  int64_t M, rows;
  int H;
  uint8_t* codes;       // [rows, H / 2]
  uint8_t* scales;      // [rows, H / 32]
};
hipError_t launch_mx_quantize(const MxQuantizeArgs& a, bool f32, hipStream_t s);

struct MxDequantizeArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;            // bf16 or float32
  int64_t pieces;       // of 8 values
};
hipError_t launch_mx_dequantize(const MxDequantizeArgs& a, bool f32, hipStream_t s);

// ---- gradnorm.hip
struct GradTensor {
  const void* g;
  void* out;
  int64_t n;            // elements
  bool f32;             // float32, else bf16
};
size_t grad_norm_workspace(int64_t count);
// Whether every launch's chunks can be counted in 32 bits.
bool grad_sizes_ok(const GradTensor* list, int64_t count);
// Sums of squares into `part`, *parts of them.
hipError_t launch_grad_squares(const GradTensor* list, int64_t count, double* part, int* parts, hipStream_t s);
hipError_t launch_grad_norm(const double* part, int parts, float* norm, hipStream_t s);
// With `part` the norm is formed from the sums and written, else read.
hipError_t launch_grad_clip(const GradTensor* list, int64_t count, const double* part, int parts, float* norm, float max_norm,
                            bool in_place, hipStream_t s);

}  // namespace moe
