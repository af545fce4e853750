// C entry points of qgemm_fused.h: argument checks (before any HIP call), workspace
// plans, kernel choice and launch, with the launch-status convention of api.cpp.
#include <algorithm>
#include <cstdlib>

#include <hip/hip_runtime.h>

#include "fused_kernels.h"

namespace {

constexpr int64_t LIM = (int64_t)1 << 30;
constexpr int64_t SPAN_LIMIT = (int64_t)1 << 31;   // 32-bit buffer offsets

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool is_float(qg_dtype t) { return t == QG_FP32 || t == QG_BF16 || t == QG_FP16; }
bool aligned_for(const void* p, qg_dtype t) { return aligned(p, t == QG_FP32 ? 4 : 2); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t blocks_of(int64_t n) { return (n + 31) / 32; }

qg_status nothing() {
    qg::record_kernel("none");
    return QG_OK;
}

qg_status done(hipError_t e, const char* name) {
    if (e != hipSuccess) return QG_ERR_HIP;
    qg::record_kernel(name);
    return QG_OK;
}

#define QG_TRY_HIP(call)                               \
    do {                                               \
        if ((call) != hipSuccess) return QG_ERR_HIP;   \
    } while (0)

// Spans that 32-bit offsets reach, as qgemm_a8w8 checks them.
bool span_ok(int64_t K, int64_t lda, int64_t ldw, int b_trans) {
    return 256 * lda + K + 256 < SPAN_LIMIT && (b_trans ? 256 * ldw + K + 256 : (K + 256) * ldw) < SPAN_LIMIT;
}

int env_int(const char* name, int dflt) {
    const char* v = std::getenv(name);
    return v != nullptr && *v ? std::atoi(v) : dflt;
}

// Rows of whole 16-byte pieces.
bool whole_pieces(const void* p, int64_t ld, int64_t n) { return aligned(p, 16) && ld % 16 == 0 && n % 16 == 0; }

// How a product runs: its tile, and in how many parts K is divided.
struct Choice {
    int tile, splits, split_chunks;
    size_t bytes;          // of their sums
    int64_t ld_partial;
};

// For `rows` x `cols` sums over `chunks` chunks of K (a pair's columns and a gradient's rows
// counted twice), out_cols columns of the output.  QGEMM_FUSED_TILE and QGEMM_FUSED_SPLITS force a
// tile (of an ANY tile's shape where the operands need that) and a number of parts, for
// tests and tuning.
Choice choose(int64_t rows, int64_t cols, int64_t chunks, int64_t out_cols, bool pieces) {
    auto tiles = [&](int64_t bm, int64_t bn) { return ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn); };
    const int forced = env_int("QGEMM_FUSED_TILE", -1);
    Choice c{forced, 1, 0, 0, (out_cols + 3) / 4 * 4};
    if (forced < 0 || forced >= qg::FUSED_TILES) {
        const int64_t large = tiles(256, 256), small = tiles(128, 128);
        if (large >= 512 || (large >= 160 && !(large > 256 && large <= 352))) c.tile = qg::FUSED_256x256;
        else if (chunks <= 16 && small <= 256) c.tile = qg::FUSED_64x128;
        else c.tile = qg::FUSED_128x128;
    }
    if (!pieces && c.tile < qg::FUSED_ANY_128x128)
        c.tile = c.tile == qg::FUSED_64x128 || c.tile == qg::FUSED_64x128_DEEP ? qg::FUSED_ANY_64x128 : qg::FUSED_ANY_128x128;
    const int64_t want = std::min<int64_t>(env_int("QGEMM_FUSED_SPLITS", 1), chunks);
    if (want > 1) {
        c.split_chunks = (int)((chunks + want - 1) / want);
        c.splits = (int)((chunks + c.split_chunks - 1) / c.split_chunks);
        c.bytes = (size_t)c.splits * (size_t)(rows * cols / out_cols) * c.ld_partial * 4;
    }
    return c;
}

hipError_t launch_fused(int form, const qg::FusedArgs& a, int tile, bool kmajor, hipStream_t s) {
    const qg::FusedTile t = (qg::FusedTile)tile;
    return form == qg::FUSED_ONE ? qg::launch_fused_one(a, t, kmajor, s)
           : form == qg::FUSED_PAIR ? qg::launch_fused_pair(a, t, kmajor, s) : qg::launch_fused_grad(a, t, kmajor, s);
}

const char* kernel_name(int form, const Choice& c) {
    static const char* const names[3][qg::FUSED_TILES] = {
        {"fused_one_256x256", "fused_one_128x128", "fused_one_128x128_deep", "fused_one_64x128", "fused_one_64x128_deep",
         "fused_one_any_128x128", "fused_one_any_64x128"},
        {"fused_pair_256x256", "fused_pair_128x128", "fused_pair_128x128_deep", "fused_pair_64x128", "fused_pair_64x128_deep",
         "fused_pair_any_128x128", "fused_pair_any_64x128"},
        {"fused_grad_256x256", "fused_grad_128x128", "fused_grad_128x128_deep", "fused_grad_64x128", "fused_grad_64x128_deep",
         "fused_grad_any_128x128", "fused_grad_any_64x128"}};
    static const char* const joined[3] = {"fused_one_joined", "fused_pair_joined", "fused_grad_joined"};
    return c.splits > 1 ? joined[form] : names[form][c.tile];
}

// The product, and the second kernel where K is divided.
qg_status run(int form, qg::FusedArgs& a, const Choice& c, bool kmajor, void* partial, hipStream_t s) {
    if (c.splits > 1) {
        a.partial = (int*)partial;
        a.splits = c.splits;
        a.split_chunks = c.split_chunks;
        a.ld_partial = c.ld_partial;
    }
    QG_TRY_HIP(launch_fused(form, a, c.tile, kmajor, s));
    if (c.splits > 1) QG_TRY_HIP(qg::launch_fused_join(a, form, s));
    return done(hipSuccess, kernel_name(form, c));
}

// A launch holds fewer than 2^32 threads: of the smallest tile's 256.
bool too_many_tiles(int64_t rows, int64_t cols) { return ((rows + 63) / 64) * ((cols + 127) / 128) >= (int64_t)1 << 24; }

struct Scales { const float* p; int64_t len; };

bool scale_ok(const Scales& s, int64_t n) { return s.p != nullptr && aligned(s.p, 4) && (s.len == 1 || s.len == n); }

// The forward calls.
struct Forward {
    int64_t M, N, K;
    const int8_t* A; int64_t lda;
    const int8_t* W[2]; int64_t ldw[2]; int b_trans;
    int pair;

    Choice choice() const {
        bool pieces = whole_pieces(A, lda, K);
        for (int h = 0; h < pair; ++h) pieces = pieces && whole_pieces(W[h], ldw[h], b_trans ? K : N);
        return choose(M, N * pair, (K + 127) / 128, N, pieces);
    }
};

bool sizes_bad(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= LIM || N >= LIM || K >= LIM;
}

size_t forward_workspace(const Forward& f) {
    if (sizes_bad(f.M, f.N, f.K) || f.M == 0 || f.N == 0 || f.K == 0) return 0;
    return up256(f.choice().bytes);
}

bool checkpoint_ok(const int8_t* c, int64_t ldc, const float* s, int64_t lds, int64_t N) {
    return c != nullptr && s != nullptr && aligned(s, 4) && ldc >= N && lds >= blocks_of(N);
}

qg_status forward(const Forward& f, const Scales& act, const Scales* ws, const float* bias, qg_activation activation,
                  const void* res, int64_t ldr, void* out, qg_dtype out_dtype, int64_t ldo, int8_t* ckpt, int64_t ld_ckpt,
                  float* ckpt_scale, int64_t ld_ckpt_scale, void* workspace, size_t workspace_bytes, void* stream) {
    const int64_t M = f.M, N = f.N, K = f.K;
    if (sizes_bad(M, N, K)) return QG_ERR_INVALID_ARGUMENT;
    if (!is_float(out_dtype) || activation < QG_ACT_NONE || activation > QG_ACT_GELU_TANH || (f.b_trans != 0 && f.b_trans != 1))
        return QG_ERR_INVALID_ARGUMENT;
    if (M == 0 || N == 0) return nothing();
    if (K == 0 || f.A == nullptr || out == nullptr || f.lda < K || ldo < N) return QG_ERR_INVALID_ARGUMENT;
    if (!scale_ok(act, M) || !aligned(bias, 4) || !aligned_for(out, out_dtype)) return QG_ERR_INVALID_ARGUMENT;
    for (int h = 0; h < f.pair; ++h)
        if (f.W[h] == nullptr || f.ldw[h] < (f.b_trans ? K : N) || !scale_ok(ws[h], N)) return QG_ERR_INVALID_ARGUMENT;
    if (res != nullptr && (ldr < N || !aligned_for(res, out_dtype))) return QG_ERR_INVALID_ARGUMENT;
    if ((ckpt != nullptr || ckpt_scale != nullptr) && !checkpoint_ok(ckpt, ld_ckpt, ckpt_scale, ld_ckpt_scale, N))
        return QG_ERR_INVALID_ARGUMENT;
    if (workspace != nullptr && !aligned(workspace, 256)) return QG_ERR_INVALID_ARGUMENT;
    for (int h = 0; h < f.pair; ++h)
        if (!span_ok(K, f.lda, f.ldw[h], f.b_trans)) return QG_ERR_UNSUPPORTED;
    if (too_many_tiles(M, N * f.pair)) return QG_ERR_UNSUPPORTED;
    const Choice c = f.choice();
    if (c.bytes > 0 && (workspace == nullptr || workspace_bytes < up256(c.bytes))) return QG_ERR_WORKSPACE;

    qg::Epilogue e{};
    e.M = (int)M; e.N = (int)N;
    e.act_scale = act.p; e.as_stride = act.len == 1 ? 0 : 1;
    for (int h = 0; h < f.pair; ++h) {
        e.w_scale[h] = ws[h].p;
        e.ws_stride[h] = ws[h].len == 1 ? 0 : 1;
        if (ckpt != nullptr) {
            e.ckpt[h] = ckpt + (int64_t)h * M * ld_ckpt;
            e.ckpt_scale[h] = ckpt_scale + (int64_t)h * M * ld_ckpt_scale;
        }
    }
    e.bias = bias; e.activation = activation;
    e.res = res; e.ldr = ldr;
    e.out = out; e.ldo = ldo; e.out_type = out_dtype;
    e.ld_ckpt = ld_ckpt; e.ld_ckpt_scale = ld_ckpt_scale;
    (void)hipGetLastError();
    qg::FusedArgs a{};
    a.e = e;
    a.A[0] = f.A; a.lda = f.lda;
    for (int h = 0; h < f.pair; ++h) {
        a.B[h] = f.W[h];
        a.ldb[h] = f.ldw[h];
    }
    a.K = (int)K; a.branches = 1;
    return run(f.pair == 2 ? qg::FUSED_PAIR : qg::FUSED_ONE, a, c, f.b_trans != 0, workspace, (hipStream_t)stream);
}

// The gradients.
struct Backward {
    int64_t M, N, K;
    const int8_t* W[2]; int64_t ldw[2]; int b_trans;
    int pair;
    bool with_bias;

    Choice choice() const {
        bool pieces = true;
        for (int h = 0; h < pair; ++h) pieces = pieces && whole_pieces(W[h], ldw[h], b_trans ? K : N);
        return choose(2 * M, K, (N + 127) / 128 * pair, K, pieces);
    }
};

// Where a gradient's workspace holds what.
struct GradPlan {
    int64_t np, ldq;
    size_t hi, lo, row_scale, part, sums, bytes;
    int parts;
    Choice c;
    explicit GradPlan(const Backward& b)
        : np((b.N + 127) / 128 * 128), ldq(np * b.pair), parts(b.with_bias ? qg::grad_rows_parts(b.M, b.N) : 0), c(b.choice()) {
        size_t at = 0;
        auto take = [&](size_t n) { const size_t here = at; at += up256(n); return here; };
        hi = take((size_t)b.M * ldq);
        lo = take((size_t)b.M * ldq);
        row_scale = take((size_t)b.M * 4);
        part = take((size_t)parts * b.N * 4);
        sums = take(c.bytes);
        bytes = at;
    }
};

size_t backward_workspace(const Backward& b) {
    if (sizes_bad(b.M, b.N, b.K) || b.M == 0 || b.N == 0 || b.K == 0 || b.N > QG_A8W8_GRAD_MAX_COLUMNS) return 0;
    return GradPlan(b).bytes;
}

qg_status backward(const Backward& b, const void* dy, qg_dtype dtype, int64_t ld_dy, const Scales* ws, const int8_t* ckpt,
                   int64_t ld_ckpt, const float* ckpt_scale, int64_t ld_ckpt_scale, qg_activation activation, void* dx,
                   int64_t ld_dx, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    const int64_t M = b.M, N = b.N, K = b.K;
    if (sizes_bad(M, N, K)) return QG_ERR_INVALID_ARGUMENT;
    if ((dtype != QG_BF16 && dtype != QG_FP16) || activation < QG_ACT_NONE || activation > QG_ACT_GELU_TANH ||
        (b.b_trans != 0 && b.b_trans != 1) || !aligned(dbias, 4))
        return QG_ERR_INVALID_ARGUMENT;
    if (N > QG_A8W8_GRAD_MAX_COLUMNS) return QG_ERR_UNSUPPORTED;
    if (M == 0) {
        if (dbias == nullptr || N == 0) return nothing();
        (void)hipGetLastError();
        qg::GradRowsArgs a{};
        a.N = (int)N;
        a.dbias = dbias;
        return done(qg::launch_grad_rows(a, false, true, (hipStream_t)stream), "grad_rows");
    }
    if (N == 0 || K == 0 || dy == nullptr || dx == nullptr || ld_dy < N || ld_dx < K) return QG_ERR_INVALID_ARGUMENT;
    if (!aligned_for(dy, dtype) || !aligned_for(dx, dtype)) return QG_ERR_INVALID_ARGUMENT;
    for (int h = 0; h < b.pair; ++h)
        if (b.W[h] == nullptr || b.ldw[h] < (b.b_trans ? K : N) || !scale_ok(ws[h], N)) return QG_ERR_INVALID_ARGUMENT;
    const bool no_ckpt = b.pair == 1 && activation == QG_ACT_NONE && ckpt == nullptr && ckpt_scale == nullptr;
    if (!no_ckpt && !checkpoint_ok(ckpt, ld_ckpt, ckpt_scale, ld_ckpt_scale, N)) return QG_ERR_INVALID_ARGUMENT;
    if (workspace != nullptr && !aligned(workspace, 256)) return QG_ERR_INVALID_ARGUMENT;
    const GradPlan p(b);
    for (int h = 0; h < b.pair; ++h)
        if (!span_ok(N, p.ldq, b.ldw[h], !b.b_trans)) return QG_ERR_UNSUPPORTED;
    if (too_many_tiles(2 * M, K)) return QG_ERR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < p.bytes) return QG_ERR_WORKSPACE;
    (void)hipGetLastError();
    const hipStream_t s = (hipStream_t)stream;
    char* const w = (char*)workspace;

    qg::GradRowsArgs a{};
    a.M = (int)M; a.N = (int)N; a.np = (int)p.np;
    a.dy = dy; a.ldy = ld_dy;
    for (int h = 0; h < b.pair; ++h) {
        if (ckpt != nullptr) {
            a.ckpt[h] = ckpt + (int64_t)h * M * ld_ckpt;
            a.ckpt_scale[h] = ckpt_scale + (int64_t)h * M * ld_ckpt_scale;
        }
        a.w_scale[h] = ws[h].p;
        a.ws_stride[h] = ws[h].len == 1 ? 0 : 1;
    }
    a.ld_ckpt = ld_ckpt; a.ld_ckpt_scale = ld_ckpt_scale;
    a.activation = activation;
    a.hi = (int8_t*)(w + p.hi); a.lo = (int8_t*)(w + p.lo); a.ldq = p.ldq;
    a.row_scale = (float*)(w + p.row_scale);
    a.part = (float*)(w + p.part); a.parts = p.parts;
    a.dbias = dbias;
    QG_TRY_HIP(qg::launch_grad_rows(a, b.pair == 2, dtype == QG_BF16, s));

    qg::FusedArgs f{};
    f.e.M = (int)M; f.e.N = (int)K;
    f.e.act_scale = a.row_scale; f.e.as_stride = 1;
    f.e.out = dx; f.e.ldo = ld_dx; f.e.out_type = dtype;
    f.A[0] = a.hi; f.A[1] = a.lo; f.lda = p.ldq;
    for (int h = 0; h < b.pair; ++h) {
        f.B[h] = b.W[h];
        f.ldb[h] = b.ldw[h];
    }
    f.K = (int)N; f.branches = b.pair;
    return run(qg::FUSED_GRAD, f, p.c, b.b_trans == 0, w + p.sums, s);
}

}  // namespace

extern "C" {

size_t qgemm_a8w8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* W,
                                         int64_t ldw, int b_trans) {
    return forward_workspace({M, N, K, A, lda, {W, nullptr}, {ldw, 0}, b_trans, 1});
}

qg_status qgemm_a8w8_linear(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* W, int64_t ldw,
                            int b_trans, const float* act_scale, int64_t act_scale_len, const float* weight_scale,
                            int64_t weight_scale_len, const float* bias, qg_activation activation, const void* residual,
                            int64_t ld_residual, void* out, qg_dtype out_dtype, int64_t ldo, int8_t* checkpoint,
                            int64_t ld_checkpoint, float* checkpoint_scale, int64_t ld_checkpoint_scale, void* workspace,
                            size_t workspace_bytes, void* stream) {
    const Scales ws[2] = {{weight_scale, weight_scale_len}, {nullptr, 0}};
    return forward({M, N, K, A, lda, {W, nullptr}, {ldw, 0}, b_trans, 1}, {act_scale, act_scale_len}, ws, bias, activation, residual,
                   ld_residual, out, out_dtype, ldo, checkpoint, ld_checkpoint, checkpoint_scale, ld_checkpoint_scale, workspace,
                   workspace_bytes, stream);
}

size_t qgemm_a8w8_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* W_gate,
                                        int64_t ld_gate, const int8_t* W_up, int64_t ld_up, int b_trans) {
    return forward_workspace({M, N, K, A, lda, {W_gate, W_up}, {ld_gate, ld_up}, b_trans, 2});
}

qg_status qgemm_a8w8_gated(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* W_gate, int64_t ld_gate,
                           const int8_t* W_up, int64_t ld_up, int b_trans, const float* act_scale, int64_t act_scale_len,
                           const float* gate_scale, int64_t gate_scale_len, const float* up_scale, int64_t up_scale_len,
                           qg_activation activation, void* out, qg_dtype out_dtype, int64_t ldo, int8_t* checkpoint,
                           int64_t ld_checkpoint, float* checkpoint_scale, int64_t ld_checkpoint_scale, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const Scales ws[2] = {{gate_scale, gate_scale_len}, {up_scale, up_scale_len}};
    return forward({M, N, K, A, lda, {W_gate, W_up}, {ld_gate, ld_up}, b_trans, 2}, {act_scale, act_scale_len}, ws, nullptr,
                   activation, nullptr, 0, out, out_dtype, ldo, checkpoint, ld_checkpoint, checkpoint_scale, ld_checkpoint_scale,
                   workspace, workspace_bytes, stream);
}

size_t qgemm_a8w8_linear_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, const int8_t* W, int64_t ldw, int b_trans,
                                              int with_bias) {
    return backward_workspace({M, N, K, {W, nullptr}, {ldw, 0}, b_trans, 1, with_bias != 0});
}

qg_status qgemm_a8w8_linear_grad(int64_t M, int64_t N, int64_t K, const void* dy, qg_dtype dtype, int64_t ld_dy, const int8_t* W,
                                 int64_t ldw, int b_trans, const float* weight_scale, int64_t weight_scale_len,
                                 const int8_t* checkpoint, int64_t ld_checkpoint, const float* checkpoint_scale,
                                 int64_t ld_checkpoint_scale, qg_activation activation, void* dx, int64_t ld_dx, float* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    const Scales ws[2] = {{weight_scale, weight_scale_len}, {nullptr, 0}};
    return backward({M, N, K, {W, nullptr}, {ldw, 0}, b_trans, 1, dbias != nullptr}, dy, dtype, ld_dy, ws, checkpoint, ld_checkpoint,
                    checkpoint_scale, ld_checkpoint_scale, activation, dx, ld_dx, dbias, workspace, workspace_bytes, stream);
}

size_t qgemm_a8w8_gated_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, const int8_t* W_gate, int64_t ld_gate,
                                             const int8_t* W_up, int64_t ld_up, int b_trans) {
    return backward_workspace({M, N, K, {W_gate, W_up}, {ld_gate, ld_up}, b_trans, 2, false});
}

qg_status qgemm_a8w8_gated_grad(int64_t M, int64_t N, int64_t K, const void* dy, qg_dtype dtype, int64_t ld_dy,
                                const int8_t* W_gate, int64_t ld_gate, const int8_t* W_up, int64_t ld_up, int b_trans,
                                const float* gate_scale, int64_t gate_scale_len, const float* up_scale, int64_t up_scale_len,
                                const int8_t* checkpoint, int64_t ld_checkpoint, const float* checkpoint_scale,
                                int64_t ld_checkpoint_scale, qg_activation activation, void* dx, int64_t ld_dx, void* workspace,
                                size_t workspace_bytes, void* stream) {
    const Scales ws[2] = {{gate_scale, gate_scale_len}, {up_scale, up_scale_len}};
    return backward({M, N, K, {W_gate, W_up}, {ld_gate, ld_up}, b_trans, 2, false}, dy, dtype, ld_dy, ws, checkpoint, ld_checkpoint,
                    checkpoint_scale, ld_checkpoint_scale, activation, dx, ld_dx, nullptr, workspace, workspace_bytes, stream);
}

qg_status int8_quantize(int64_t M, int64_t n, const void* x, qg_dtype type, int64_t ldx, int block, int8_t* codes, int64_t ldc,
                        float* scale, int64_t ld_scale, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM || !is_float(type) || (block != 0 && block != qg::INT8_BLOCK))
        return QG_ERR_INVALID_ARGUMENT;
    if (block == 0 && n > QG_INT8_ROW_MAX_COLUMNS) return QG_ERR_UNSUPPORTED;
    if (M == 0) return nothing();
    if (x == nullptr || codes == nullptr || scale == nullptr || ldx < n || ldc < n || ld_scale < (block == 0 ? 1 : blocks_of(n)) ||
        !aligned_for(x, type) || !aligned(scale, 4))
        return QG_ERR_INVALID_ARGUMENT;
    (void)hipGetLastError();
    const qg::Int8Args a{M, n, block, x, ldx, nullptr, 0, codes, ldc, scale, ld_scale};
    return done(qg::launch_int8_quantize(a, type, (hipStream_t)stream), block == 0 ? "int8_rows" : "int8_blocks");
}

qg_status int8_dequantize(int64_t M, int64_t n, const int8_t* codes, int64_t ldc, const float* scale, int64_t ld_scale, int block,
                          void* out, qg_dtype out_type, int64_t ldo, void* stream) {
    if (M < 0 || M >= LIM || n < 1 || n >= LIM || !is_float(out_type) || (block != 0 && block != qg::INT8_BLOCK))
        return QG_ERR_INVALID_ARGUMENT;
    if (M == 0) return nothing();
    if (out == nullptr || codes == nullptr || scale == nullptr || ldo < n || ldc < n ||
        ld_scale < (block == 0 ? 1 : blocks_of(n)) || !aligned_for(out, out_type) || !aligned(scale, 4))
        return QG_ERR_INVALID_ARGUMENT;
    (void)hipGetLastError();
    const qg::Int8Args a{M, n, block, nullptr, 0, out, ldo, const_cast<int8_t*>(codes), ldc, const_cast<float*>(scale), ld_scale};
    return done(qg::launch_int8_dequantize(a, out_type, (hipStream_t)stream), "int8_dequantize");
}

}  // extern "C"
