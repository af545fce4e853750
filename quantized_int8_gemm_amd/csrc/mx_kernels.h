// Argument blocks and launchers of the norm, MX quantiser and MX product.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qgemm_mx.h"

namespace qg {

struct RmsNormArgs {
    int64_t M; int n;
    const void* x; int64_t ldx;
    const void* res; int64_t ldr;            // NULL: none
    const void* weight; float eps;
    void* h; int64_t ldh;
    void* out; int64_t ldo;                  // elements; bytes for MXFP4
    uint8_t* block_scale; int64_t lds;
    float* row_scale;
};
hipError_t launch_rms_norm(const RmsNormArgs& a, qg_dtype type, bool weight_f32, qg_dtype format, hipStream_t s,
                           const char** name);

struct RmsNormGradArgs {
    int64_t M; int n;
    const void* dy; int64_t ldy;
    const void* h; int64_t ldh;
    const void* weight; const float* rstd;
    const void* dh; int64_t lddh;            // NULL: none
    void* dx; int64_t ldx; void* dweight;
    float* part; int parts;                  // [parts, n] partial sums of dweight
};
// Partial rows that fill the machine.  Growing a shape (M, n or both) may lower their
// number, but not below the smaller one of GRAD_PARTS_KEPT and what it was.
constexpr int GRAD_PARTS_KEPT = 256;
int rms_norm_grad_parts(int64_t M, int64_t n);
hipError_t launch_rms_norm_grad(const RmsNormGradArgs& a, qg_dtype type, bool weight_f32, hipStream_t s,
                                const char** name);

struct MxCodecArgs {
    int64_t M; int64_t n;
    const void* x; int64_t ldx;              // quantise: values in; dequantise: values out through `out`
    void* out; int64_t ldo;
    uint8_t* codes; int64_t ldc;             // bytes
    uint8_t* scale; int64_t lds;             // bytes
};
hipError_t launch_mx_quantize(const MxCodecArgs& a, qg_dtype type, qg_dtype format, hipStream_t s, const char** name);
hipError_t launch_mx_dequantize(const MxCodecArgs& a, qg_dtype type, qg_dtype format, hipStream_t s, const char** name);

struct MxMatmulArgs {
    int M, N, K;
    const uint8_t* A; int64_t lda;           // bytes
    const uint8_t* as; int64_t ldas;
    const uint8_t* W; int64_t ldw;
    const uint8_t* ws; int64_t ldws;
    const float* act_scale;                  // NULL: 1
    void* out; int64_t ldo; int out_type;    // qg_dtype
};
// Reads bytes: any strides, any alignment.
hipError_t launch_mx_bytes(const MxMatmulArgs& a, bool a8, hipStream_t s, const char** name);

// Tiled kernels: code rows 16-byte aligned, scale rows 4-byte aligned and
// readable to the end of their last word.
constexpr int MX_ROUND = 256;   // compute units: workgroups that run at once if each fills one
hipError_t launch_mx_256x256(const MxMatmulArgs& a, bool a8, hipStream_t s);
hipError_t launch_mx_128x128(const MxMatmulArgs& a, bool a8, hipStream_t s);
hipError_t launch_mx_64x128(const MxMatmulArgs& a, bool a8, hipStream_t s);
hipError_t launch_mx_64x64(const MxMatmulArgs& a, bool a8, hipStream_t s);
hipError_t launch_mx_64x32(const MxMatmulArgs& a, bool a8, hipStream_t s);
hipError_t launch_mx_32x32(const MxMatmulArgs& a, bool a8, hipStream_t s);

// At most 8 rows: W streamed once, 16 columns per workgroup; operands laid out as
// for the tiled kernels.
constexpr int MX_DECODE_MAX_M = 8;
hipError_t launch_mx_decode(const MxMatmulArgs& a, bool a8, hipStream_t s);

// Names the kernel for qgemm_last_kernel().
void record_kernel(const char* name);

}  // namespace qg
