// C entry points of qgemm_mx.h: argument checks (before any HIP call), kernel
// choice and launch, with the launch-status convention of api.cpp.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include <hip/hip_runtime.h>

#include "mx_kernels.h"

namespace {

constexpr int64_t LIM = (int64_t)1 << 30;

bool is_float(qg_dtype t) { return t == QG_FP32 || t == QG_BF16 || t == QG_FP16; }
bool is_mx(qg_dtype t) { return t == QG_MXFP8 || t == QG_MXFP4; }
int64_t blocks_of(int64_t n) { return (n + 31) / 32; }
int64_t code_bytes(qg_dtype f, int64_t n) { return blocks_of(n) * (f == QG_MXFP8 ? 32 : 16); }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned_for(const void* p, qg_dtype t) { return aligned(p, t == QG_FP32 ? 4 : 2); }

qg_status done(hipError_t e, const char* name) {
    if (e != hipSuccess) return QG_ERR_HIP;
    qg::record_kernel(name);
    return QG_OK;
}

bool env_is(const char* name, const char* value) {
    const char* v = std::getenv(name);
    return v != nullptr && std::strcmp(v, value) == 0;
}

int env_int(const char* name, int dflt) {
    const char* v = std::getenv(name);
    return v != nullptr && *v ? std::atoi(v) : dflt;
}

// Kernels of the MX product.
enum MxKind { MX_256x256, MX_128x128, MX_64x128, MX_64x64, MX_64x32, MX_32x32, MX_DECODE };

// split: MXFP8 activations, whose codes are split in two, so every tile multiplies twice.
MxKind mx_kind(int64_t M, int64_t N, bool split) {
    const int forced = env_int("QGEMM_MX_TILE", -1);
    if (forced >= 0 && forced <= MX_DECODE && (forced != MX_DECODE || M <= qg::MX_DECODE_MAX_M)) return (MxKind)forced;
    auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    // up to 3584 columns; split, which costs tiles more than it does this kernel, up to
    // 4096, whose 16-column workgroups are one a CU (K = 8192, W from memory, M = 1 / 8:
    // 4096 8.5 / 9.5 us, 32 x 32 tiles 11.7 / 12.0; 6144 11.1 / 13.7, tiles 12.5 / 12.7)
    if (M <= qg::MX_DECODE_MAX_M && tiles(32, 32) <= (split ? 128 : 112)) return MX_DECODE;
    // the smallest tile of which every CU gets at most one
    if (tiles(32, 32) <= qg::MX_ROUND) return MX_32x32;
    if (tiles(64, 32) <= qg::MX_ROUND) return MX_64x32;
    if (tiles(64, 64) <= qg::MX_ROUND) return MX_64x64;
    if (tiles(64, 128) <= qg::MX_ROUND) return MX_64x128;
    // Beyond: by what the busiest CU gets.  A 256 x 256 tile, alone on its CU, takes as
    // long as three 128 x 128 tiles, which run two to a CU (split: 3.75, since its waves
    // then have no registers for the next fragments).  4096 x 4096 x 4096 MXFP4: one
    // large 38.8 us, four small 47.8; 2444 x 3355 x 2464: one 25.3, three 32.0; 4096 x
    // 4352 x 4096: two 59.2, five 57.3; 2560 x 2560 x 4096: one 29.5, two 24.5.  Split:
    // 4096 x 4096 x 4096 one 97, four 102; 2444 x 3355 x 2464 one 57, three 50; 4096 x 5120 x
    // 4096 two 160, five 132; 8192 x 8192 x 8192 four 668, sixteen 729.
    const int64_t large = (tiles(256, 256) + qg::MX_ROUND - 1) / qg::MX_ROUND;
    const int64_t small = (tiles(128, 128) + qg::MX_ROUND - 1) / qg::MX_ROUND;
    return 4 * small >= (split ? 15 : 12) * large ? MX_256x256 : MX_128x128;
}

qg_status nothing() {
    qg::record_kernel("none");
    return QG_OK;
}

}  // namespace

extern "C" {

qg_status rms_norm(int64_t M, int64_t n, const void* x, qg_dtype type, int64_t ldx, const void* residual,
                   int64_t ld_residual, const void* weight, qg_dtype weight_type, float eps, void* h, int64_t ldh,
                   void* out, qg_dtype format, int64_t ldo, uint8_t* block_scale, int64_t ld_block_scale,
                   float* row_scale, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM) return QG_ERR_INVALID_ARGUMENT;
    if (!is_float(type) || (weight_type != type && weight_type != QG_FP32)) return QG_ERR_INVALID_ARGUMENT;
    if (!(format == QG_INT8 || is_mx(format) || format == QG_FP32 || format == type)) return QG_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return QG_ERR_INVALID_ARGUMENT;
    if (n > QG_RMS_NORM_MAX_COLUMNS) return QG_ERR_UNSUPPORTED;
    if (M == 0) return nothing();
    if (x == nullptr || weight == nullptr || out == nullptr || ldx < n) return QG_ERR_INVALID_ARGUMENT;
    if (residual != nullptr && (h == nullptr || ld_residual < n || ldh < n)) return QG_ERR_INVALID_ARGUMENT;
    if (!aligned_for(x, type) || !aligned_for(residual, type) || !aligned_for(weight, weight_type) ||
        (residual != nullptr && !aligned_for(h, type)))
        return QG_ERR_INVALID_ARGUMENT;
    if (is_mx(format)) {
        if (block_scale == nullptr || ld_block_scale < blocks_of(n) || ldo < code_bytes(format, n))
            return QG_ERR_INVALID_ARGUMENT;
    } else {
        if (ldo < n || (format != QG_INT8 && !aligned_for(out, format))) return QG_ERR_INVALID_ARGUMENT;
    }
    if ((format == QG_INT8 || is_mx(format)) && row_scale == nullptr) return QG_ERR_INVALID_ARGUMENT;
    if (!aligned(row_scale, 4)) return QG_ERR_INVALID_ARGUMENT;
    (void)hipGetLastError();
    const qg::RmsNormArgs a{M, (int)n, x, ldx, residual, ld_residual, weight, eps, h, ldh,
                            out, ldo, block_scale, ld_block_scale, row_scale};
    const char* name = "";
    const hipError_t e = qg::launch_rms_norm(a, type, weight_type == QG_FP32, format, (hipStream_t)stream, &name);
    return done(e, name);
}

size_t rms_norm_grad_workspace_bytes(int64_t M, int64_t n) {
    if (M < 1 || M >= LIM || n < 1 || n > QG_RMS_NORM_MAX_COLUMNS) return 0;
    return (size_t)qg::rms_norm_grad_parts(M, n) * (size_t)n * 4;
}

qg_status rms_norm_grad(int64_t M, int64_t n, const void* dy, qg_dtype type, int64_t ld_dy, const void* h, int64_t ldh,
                        const void* weight, qg_dtype weight_type, const float* rstd, const void* dh, int64_t ld_dh,
                        void* dx, int64_t ld_dx, void* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM) return QG_ERR_INVALID_ARGUMENT;
    if (!is_float(type) || (weight_type != type && weight_type != QG_FP32)) return QG_ERR_INVALID_ARGUMENT;
    if (n > QG_RMS_NORM_MAX_COLUMNS) return QG_ERR_UNSUPPORTED;
    if (dweight == nullptr || !aligned_for(dweight, weight_type)) return QG_ERR_INVALID_ARGUMENT;
    if (M > 0) {
        if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr)
            return QG_ERR_INVALID_ARGUMENT;
        if (ld_dy < n || ldh < n || ld_dx < n || (dh != nullptr && ld_dh < n)) return QG_ERR_INVALID_ARGUMENT;
        if (!aligned_for(dy, type) || !aligned_for(h, type) || !aligned_for(dh, type) || !aligned_for(dx, type) ||
            !aligned_for(weight, weight_type) || !aligned(rstd, 4))
            return QG_ERR_INVALID_ARGUMENT;
        if (workspace == nullptr || !aligned(workspace, 16)) return QG_ERR_INVALID_ARGUMENT;
    }
    int parts = qg::rms_norm_grad_parts(M, n);
    const int64_t fit = (int64_t)(workspace_bytes / ((size_t)n * 4));
    if (M > 0 && fit < parts) {
        // Some larger shapes run fewer workgroups, never fewer than GRAD_PARTS_KEPT of
        // those this one has; with their workspace this one runs as many as it holds.
        if (fit < std::min(parts, qg::GRAD_PARTS_KEPT)) return QG_ERR_WORKSPACE;
        parts = (int)fit;
    }
    (void)hipGetLastError();
    const qg::RmsNormGradArgs a{M, (int)n, dy, ld_dy, h, ldh, weight, rstd, dh, ld_dh, dx, ld_dx, dweight,
                                (float*)workspace, parts};
    const char* name = "";
    const hipError_t e = qg::launch_rms_norm_grad(a, type, weight_type == QG_FP32, (hipStream_t)stream, &name);
    return done(e, name);
}

qg_status mx_quantize(int64_t M, int64_t n, const void* x, qg_dtype type, int64_t ldx, void* codes, qg_dtype format,
                      int64_t ldc, uint8_t* scale, int64_t lds, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM || !is_float(type) || !is_mx(format)) return QG_ERR_INVALID_ARGUMENT;
    if (M == 0) return nothing();
    if (x == nullptr || codes == nullptr || scale == nullptr || ldx < n || ldc < code_bytes(format, n) ||
        lds < blocks_of(n) || !aligned_for(x, type))
        return QG_ERR_INVALID_ARGUMENT;
    if (M * blocks_of(n) >= (int64_t)1 << 32) return QG_ERR_UNSUPPORTED;   // one launch's threads
    (void)hipGetLastError();
    const qg::MxCodecArgs a{M, n, x, ldx, nullptr, 0, (uint8_t*)codes, ldc, scale, lds};
    const char* name = "";
    return done(qg::launch_mx_quantize(a, type, format, (hipStream_t)stream, &name), name);
}

qg_status mx_dequantize(int64_t M, int64_t n, const void* codes, qg_dtype format, int64_t ldc, const uint8_t* scale,
                        int64_t lds, void* out, qg_dtype out_type, int64_t ldo, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM || !is_float(out_type) || !is_mx(format)) return QG_ERR_INVALID_ARGUMENT;
    if (M == 0) return nothing();
    if (out == nullptr || codes == nullptr || scale == nullptr || ldo < n || ldc < code_bytes(format, n) ||
        lds < blocks_of(n) || !aligned_for(out, out_type))
        return QG_ERR_INVALID_ARGUMENT;
    if (M * blocks_of(n) >= (int64_t)1 << 32) return QG_ERR_UNSUPPORTED;
    (void)hipGetLastError();
    const qg::MxCodecArgs a{M, n, nullptr, 0, out, ldo, (uint8_t*)const_cast<void*>(codes), ldc,
                            const_cast<uint8_t*>(scale), lds};
    const char* name = "";
    return done(qg::launch_mx_dequantize(a, out_type, format, (hipStream_t)stream, &name), name);
}

qg_status mx_matmul(int64_t M, int64_t N, int64_t K, const void* A, qg_dtype a_format, int64_t lda,
                    const uint8_t* a_scale, int64_t ld_a_scale, const void* W, int64_t ldw, const uint8_t* w_scale,
                    int64_t ld_w_scale, int scale_rows_padded, const float* act_scale, void* out, qg_dtype out_type,
                    int64_t ldo, void* stream) {
    if (M < 0 || N < 0 || K < 0 || M >= LIM || N >= LIM || K >= LIM) return QG_ERR_INVALID_ARGUMENT;
    if (!is_mx(a_format) || !is_float(out_type)) return QG_ERR_INVALID_ARGUMENT;
    if (M == 0 || N == 0) return nothing();
    if (K < 32 || K % 32 != 0) return QG_ERR_INVALID_ARGUMENT;
    if (A == nullptr || a_scale == nullptr || W == nullptr || w_scale == nullptr || out == nullptr)
        return QG_ERR_INVALID_ARGUMENT;
    if (lda < code_bytes(a_format, K) || ldw < K / 2 || ld_a_scale < K / 32 || ld_w_scale < K / 32 || ldo < N ||
        !aligned_for(out, out_type) || !aligned(act_scale, 4))
        return QG_ERR_INVALID_ARGUMENT;
    if (lda * 512 >= (int64_t)1 << 31 || ldw * 512 >= (int64_t)1 << 31 || ld_a_scale * 512 >= (int64_t)1 << 31 ||
        ld_w_scale * 512 >= (int64_t)1 << 31)
        return QG_ERR_UNSUPPORTED;
    const bool fast = lda % 16 == 0 && ldw % 16 == 0 && aligned(A, 16) && aligned(W, 16) && scale_rows_padded != 0 &&
                      (ld_a_scale % 4 == 0 || M == 1) && (ld_w_scale % 4 == 0 || N == 1) && aligned(a_scale, 4) &&
                      aligned(w_scale, 4) && !env_is("QGEMM_MX_KERNEL", "bytes");
    if (((M + 255) / 256) * ((N + 255) / 256) >= (int64_t)1 << 23) return QG_ERR_UNSUPPORTED;   // one launch's threads
    (void)hipGetLastError();
    qg::MxMatmulArgs a{};
    a.M = (int)M; a.N = (int)N; a.K = (int)K;
    a.A = (const uint8_t*)A; a.lda = lda; a.as = a_scale; a.ldas = ld_a_scale;
    a.W = (const uint8_t*)W; a.ldw = ldw; a.ws = w_scale; a.ldws = ld_w_scale;
    a.act_scale = act_scale; a.out = out; a.ldo = ldo; a.out_type = out_type;
    // A single row's stride may be anything.  The fast kernels ask for whole tiles of
    // rows, by 4-byte words, and leave it to the buffer's end that there is only one: at a
    // multiple of 4 the next ones start past that end, never inside its last word.
    if (M == 1) a.ldas = (a.ldas + 3) & ~(int64_t)3;
    if (N == 1) a.ldws = (a.ldws + 3) & ~(int64_t)3;
    const bool a8 = a_format == QG_MXFP8;
    const hipStream_t st = (hipStream_t)stream;
    const char* name = "";
    if (!fast) return done(qg::launch_mx_bytes(a, a8, st, &name), name);
    switch (mx_kind(M, N, a8)) {
        case MX_256x256: return done(qg::launch_mx_256x256(a, a8, st), "mx_tiled_256x256");
        case MX_128x128: return done(qg::launch_mx_128x128(a, a8, st), "mx_tiled_128x128");
        case MX_64x128: return done(qg::launch_mx_64x128(a, a8, st), "mx_tiled_64x128");
        case MX_64x64: return done(qg::launch_mx_64x64(a, a8, st), "mx_tiled_64x64");
        case MX_64x32: return done(qg::launch_mx_64x32(a, a8, st), "mx_tiled_64x32");
        case MX_32x32: return done(qg::launch_mx_32x32(a, a8, st), "mx_tiled_32x32");
        default: return done(qg::launch_mx_decode(a, a8, st), "mx_decode");
    }
}

}  // extern "C"
