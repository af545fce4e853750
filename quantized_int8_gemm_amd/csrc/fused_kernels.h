// Argument blocks and launchers of the fused A8W8 products, their gradients and
// the int8 quantiser.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qgemm_fused.h"

namespace qg {

constexpr int INT8_BLOCK = 32;   // columns of a checkpoint's block

// What follows a product: out [M,N], of one product or of a gated pair.
struct Epilogue {
    int M, N;
    const float* act_scale; int as_stride;
    const float* w_scale[2]; int ws_stride[2];
    const float* bias;                        // NULL: none
    int activation;
    const void* res; int64_t ldr;             // NULL: none
    void* out; int64_t ldo; int out_type;
    int8_t* ckpt[2]; int64_t ld_ckpt;         // NULL: none
    float* ckpt_scale[2]; int64_t ld_ckpt_scale;
};

// A tiled product with its epilogue: one (A [M,K], B the weight), a pair (B[0] gate, B[1]
// up), or a gradient (A the planes hi and lo [M, branches * np], B the branches' weights,
// K the forward call's N, e.N its K, e.act_scale the rows' scales).
enum { FUSED_ONE = 0, FUSED_PAIR = 1, FUSED_GRAD = 2 };
struct FusedArgs {
    Epilogue e;
    const int8_t* A[2]; int64_t lda;
    const int8_t* B[2]; int64_t ldb[2];
    int K, branches;
    // Bytes that the rows along the sum hold, and columns that a [K,N] weight's rows hold: K and
    // e.N, or up to their padding's end.
    int k_bytes, b_cols;
    // NULL, or where `splits` workgroups a tile, of split_chunks chunks of 128 each, leave
    // their sums: int32 [splits, 1 or 2 (a pair's or a gradient's), e.M, ld_partial]
    int* partial; int splits, split_chunks; int64_t ld_partial;
    // Of a gradient: NULL, or partial sums [parts, bias_n], that workgroups behind the tiles' add
    // up to dbias.
    const float* part; int parts, bias_n; float* dbias;
};
// Rows and columns of sums of a tile; DEEP: more than two LDS stages; ANY: operands of any
// alignment.
enum FusedTile { FUSED_256x256, FUSED_128x128, FUSED_128x128_DEEP, FUSED_64x128_DEEP, FUSED_ANY_64x128, FUSED_TILES };
// kmajor: B's rows lie along the sum.
hipError_t launch_fused_one(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s);
hipError_t launch_fused_pair(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s);
hipError_t launch_fused_grad(const FusedArgs& a, FusedTile tile, bool kmajor, hipStream_t s);

// Matrices laid out with rows of whole 16-byte pieces, zeros behind them.
struct PadArgs {
    int count;
    const int8_t* src[3]; int64_t rows[3], cols[3], ld[3];
    int8_t* dst[3]; int64_t ldd[3];           // a multiple of 16
};
hipError_t launch_fused_pad(const PadArgs& a, hipStream_t s);

// Products of tm x tn outputs a workgroup (16, 32 or 64 rows, 16 or 32 columns; 32 with a
// checkpoint) of weights whose rows lie along the sum; any: rows of any alignment.
hipError_t launch_fused_direct(const FusedArgs& a, int form, int tm, int tn, bool any, hipStream_t s);
// Products of tm (16 or 32) rows by 64 columns of sums a workgroup of weights whose rows do not.
hipError_t launch_fused_direct_kn(const FusedArgs& a, int form, int tm, bool any, hipStream_t s);

// The second kernel of a divided sum.
hipError_t launch_fused_join(const FusedArgs& a, int form, hipStream_t s);

// The factors of a gradient, for each row of dy: `hi` and `lo` [M, branches * np]
// with zeros behind each branch's N, and the row's scale.
struct GradRowsArgs {
    int M, N, np;                             // np: N rounded up to 128
    const void* dy; int64_t ldy;
    const int8_t* ckpt[2]; int64_t ld_ckpt;   // NULL without an activation
    const float* ckpt_scale[2]; int64_t ld_ckpt_scale;
    const float* w_scale[2]; int ws_stride[2];
    int activation;
    int8_t* hi; int8_t* lo; int64_t ldq;
    float* row_scale;                         // [M]
    float* part; int parts;                   // NULL, or [parts,N] partial sums of dbias
};
// Zeros.
hipError_t launch_clear(float* x, int64_t n, hipStream_t s);
int grad_rows_parts(int64_t M, int64_t N);
hipError_t launch_grad_rows(const GradRowsArgs& a, bool pair, bool bf16, hipStream_t s);
struct Int8Args {
    int64_t M; int64_t n; int block;
    const void* x; int64_t ldx;               // quantise: values in
    void* out; int64_t ldo;                   // dequantise: values out
    int8_t* codes; int64_t ldc;
    float* scale; int64_t lds;
};
hipError_t launch_int8_quantize(const Int8Args& a, qg_dtype type, hipStream_t s);
hipError_t launch_int8_dequantize(const Int8Args& a, qg_dtype type, hipStream_t s);
// Of api.cpp.
void record_kernel(const char* name);

}  // namespace qg
