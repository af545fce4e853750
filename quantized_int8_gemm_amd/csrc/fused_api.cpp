// C entry points of qgemm_fused.h: argument checks (before any HIP call), workspace
// plans, kernel choice and launch, with the launch-status convention of api.cpp.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include <hip/hip_runtime.h>

#include "fused_kernels.h"

namespace {

constexpr int64_t LIM = (int64_t)1 << 30;
constexpr int64_t SPAN_LIMIT = (int64_t)1 << 31;   // 32-bit buffer offsets

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool is_float(qg_dtype t) { return t == QG_FP32 || t == QG_BF16 || t == QG_FP16; }
bool aligned_for(const void* p, qg_dtype t) { return aligned(p, t == QG_FP32 ? 4 : 2); }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
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

// QGEMM_FUSED="kind[/parts[/pad]]" forces a kind (its number), a number of parts of K and
// padding (0: none) where the call allows them, -1 for what is left open; for tests and tuning.
struct Forced {
    int kind = -1, parts = -1, pad = -1;
    Forced() {
        if (const char* v = std::getenv("QGEMM_FUSED")) std::sscanf(v, "%d/%d/%d", &kind, &parts, &pad);
    }
};

// Rows of whole 16-byte pieces.
bool whole_pieces(const void* p, int64_t ld, int64_t n) { return aligned(p, 16) && ld % 16 == 0 && n % 16 == 0; }

// How a product runs.  tile: a FusedTile; DIRECT + 0 .. 5 for workgroups of 16, 32 or 64 rows by
// 16 or 32 columns; DIRECT_KN + 0, 1 for 16 or 32 rows by 64 columns of sums.
constexpr int DIRECT = qg::FUSED_TILES, DIRECT_KN = DIRECT + 6, KINDS = DIRECT_KN + 2;
int direct_rows(int tile) { return 16 << (tile >= DIRECT_KN ? tile - DIRECT_KN : (tile - DIRECT) / 2); }
int direct_cols(int tile) { return tile >= DIRECT_KN ? 64 : (tile - DIRECT) % 2 == 0 ? 16 : 32; }

struct Choice {
    int tile, splits, split_chunks;
    bool pad;              // operands that need it are laid out once more
    size_t bytes;          // of the divided sums
    int64_t ld_partial;
};

struct Shape {
    int form;
    int64_t M, N, K;       // of the output, and of one weight's sum
    int branches;          // weights along the sum (a gradient's)
    bool kmajor, pieces;   // B's rows lie along the sum; all rows are whole 16-byte pieces
    bool blocks;           // with a checkpoint
    int64_t pad_bytes;     // of the operands whose rows are not; -1: they cannot be padded
};

// Microseconds that a kind takes, about, fitted to measured calls (those in parentheses).  A
// chunk of 128 of K costs a tile what its CU needs with the workgroups that run there at
// once: 1.7 for 256 x 256 (4000 x 4096 x 4096 71 us, 8192^3 446), 0.75 and 1.1 for one and two of
// 128 x 128 on two stages (1000 and 2000 x 4096 x 4096 29 and 40), 0.58 on four (24, 48; 1000 x
// 4096 x 14336 70, two stages 111), 0.4 for 64 x 128 on six (300 x 4096 x 14336 51, 90 x 1008 x 1008
// 7.9), 1.04 to 1.5 through registers (1000 x 4095 x 4095 71; 1 x 4095 x 4095 gated 54).  A direct
// workgroup takes its operands at 37 bytes a nanosecond (64 x 4096 x 4096 gated 15 us, 64 x 4096 x
// 14336 34; 300 x 1008 x 1008 6.6), 35 transposed ones (202 x 1904 x 3024 12), 16 unaligned ones (4 x 4095
// x 4095 gated 20; 27 of one [K,N] weight, 30 x 4095 x 4095 16), and faster where few run
// and L2 holds the weights (30 workgroups, 151 x 96 x 4576 gated, [K,N], 8; 49, 16 x 1552 x 5264, 18);
// a 257th takes as long as a second round (55 x 2064 x 384 gated, [K,N], 260 of 16 x 32 8.0, 130 of
// 32 x 32 5.6); what it adds up through LDS bounds short sums (1024 x 2816 x 64 gated 30 with 64 x
// 32, 33 with 32 x 32, tiles of 64 x 128 12).
double time_of(const Shape& s, int tile, int splits, bool pad) {
    const double chunks = (double)((s.K + 127) / 128 * s.branches);
    const double rows = (double)s.M * (s.form == qg::FUSED_GRAD ? 2 : 1), cols = (double)s.N * (s.form == qg::FUSED_PAIR ? 2 : 1);
    const double per = std::ceil(chunks / splits);
    auto tiles = [&](double bm, double bn) { return std::ceil(rows / bm) * std::ceil(cols / bn) * splits; };
    double t;
    switch (tile) {
        case qg::FUSED_256x256: {   // the epilogues: 4096 x 8192 x 1024 with GELU 72 us, 67 with 128 x 128; gated 4096 x 14336 x 1024 184, 198
            const double last = s.form == qg::FUSED_ONE ? 12.5 : s.form == qg::FUSED_PAIR ? 10 : 8;
            t = std::ceil(tiles(256, 256) / 256) * (per * 1.7 + last);
            break;
        }
        case qg::FUSED_128x128: {
            const double n = tiles(128, 128), full = std::floor(n / 512), rest = n - 512 * full;
            t = full * (per * 1.1 + 4) + (rest > 256 ? per * 1.1 + 4 : rest > 0 ? per * 0.75 + 3 : 0);
            break;
        }
        case qg::FUSED_128x128_DEEP: t = std::ceil(tiles(128, 128) / 256) * (per * 0.58 + 3.2); break;
        case qg::FUSED_64x128_DEEP: t = std::ceil(tiles(64, 128) / 256) * (per * 0.4 + 2.2); break;
        case qg::FUSED_ANY_64x128: { const double n = std::ceil(tiles(64, 128) / 256); t = std::max(1.25, n * 1.04) * per + 1 + 1.2 * n; break; }
        default: {
            // rows of A and of the weights that a workgroup reads, and how many there are
            const double tm = direct_rows(tile), tn = direct_cols(tile);
            const double a_rows = std::min<double>(tm, s.M) * (s.form == qg::FUSED_GRAD ? 2 : 1);
            const bool kn = tile >= DIRECT_KN, pair = s.form == qg::FUSED_PAIR;
            const double w_rows = pair && !kn ? 2 * tn : tn, out_cols = pair && kn ? tn / 2 : tn;
            const double n = std::ceil(s.M / tm) * std::ceil(s.N / out_cols) / 256;
            const double alone = cols * (double)s.K * s.branches < 8e6 ? std::max(0.0, 1 - n) : 0;
            const double rate = !s.pieces && !pad ? (!kn || s.form == qg::FUSED_GRAD ? 16e3 : s.form == qg::FUSED_ONE ? 27e3 : 16e3 + 10e3 * alone) : kn ? 35e3 + (s.form == qg::FUSED_GRAD ? 0 : 25e3) * alone : 37e3 + 20e3 * alone;
            const double each = (a_rows + w_rows) * (double)s.K * s.branches / rate + 0.35;
            const double sums = tm * out_cols * (s.form == qg::FUSED_ONE ? 1 : 2);
            t = 1.2 + 4e-4 * sums + each + (std::ceil(n) - 1) * std::max({each, kn ? 2.5 : 1.5, 1.3e-3 * sums});
        }
    }
    if (splits > 1) t += 5 + rows * cols * 8 * splits / 3e6;
    if (pad) t += 3 + 2 * (double)s.pad_bytes / 4e6;
    // No faster than the operands come from memory, and what direct workgroups read again from
    // L2 (1 and 16 x 14336 x 4096 gated 27 and 34 us, with 32 columns a workgroup 33 and 35, tiles 31;
    // 30 x 4096 x 4096 gated 10.8 with 32 x 16, 12.6 with 16 x 32).
    const double tm = direct_rows(tile), tn = direct_cols(tile);
    const double floor = tile < DIRECT ? (rows + cols) / 4.7e6
                                       : cols / (tn == 16 ? 4.9e6 : 4.1e6) +
                                             (rows * std::ceil(s.N / tn) + cols * (std::ceil(s.M / tm) - 1)) / 8.5e6;
    return std::max(t, floor * (double)s.K * s.branches) + 0.02 * t;
}

int64_t tiles_of(const Shape& s, int tile) {
    const int64_t rows = s.form == qg::FUSED_GRAD ? 2 * s.M : s.M, cols = s.form == qg::FUSED_PAIR ? 2 * s.N : s.N;
    const int64_t bm = tile == qg::FUSED_256x256 ? 256 : tile == qg::FUSED_128x128 || tile == qg::FUSED_128x128_DEEP ? 128 : 64;
    return ((rows + bm - 1) / bm) * ((cols + (bm == 256 ? 255 : 127)) / (bm == 256 ? 256 : 128));
}

// The kind that takes the least time by this reckoning.
Choice choose(const Shape& s) {
    const int64_t chunks = (s.K + 127) / 128 * s.branches;
    const Forced forced;
    Choice best{qg::FUSED_ANY_64x128, 1, 0, false, 0, (s.N + 3) / 4 * 4};
    double least = 1e30;
    static const int parts[] = {1, 2, 3, 4, 6, 8, 12, 16};
    for (int with_pad = 0; with_pad < 2; ++with_pad) {
        if (with_pad == 1 && (s.pieces || s.pad_bytes < 0)) continue;
        for (int k = 0; k < KINDS; ++k) {
            const bool direct = k >= DIRECT;
            if (direct && ((k < DIRECT_KN) != s.kmajor || (s.blocks && direct_cols(k) == 16) ||
                           (k == DIRECT_KN + 1 && s.form == qg::FUSED_GRAD) ||
                           ((s.M + 15) / direct_rows(k) + 1) * ((s.N + 15) / 16 + 1) >= (int64_t)1 << 23))
                continue;   // the last: threads of a launch
            if (k < qg::FUSED_ANY_64x128 && !s.pieces && with_pad == 0) continue;
            for (const int p : parts) {
                if (p > 1 && (direct || k == qg::FUSED_256x256 || p > chunks || s.M * ((s.N + 31) / 32) >= (int64_t)1 << 28)) break;
                // K is divided where workgroups would be missing
                if (p > 1 && forced.parts < 0 && tiles_of(s, k) * p > 384) break;
                // what is forced goes before what is not
                const double t = time_of(s, k, p, with_pad == 1) + (forced.kind >= 0 && k != forced.kind ? 1e12 : 0) +
                                 (forced.pad >= 0 && with_pad != forced.pad ? 1e9 : 0) + (forced.parts > 0 && p != forced.parts ? 1e6 : 0);
                if (t >= least) continue;
                least = t;
                best.tile = k;
                best.pad = with_pad == 1;
                best.splits = p;
            }
        }
    }
    if (best.splits > 1) {
        best.split_chunks = (int)((chunks + best.splits - 1) / best.splits);
        best.splits = (int)((chunks + best.split_chunks - 1) / best.split_chunks);
        best.bytes = (size_t)best.splits * (s.form == qg::FUSED_ONE ? 1 : 2) * (size_t)s.M * best.ld_partial * 4;
    }
    return best;
}

hipError_t launch_fused(int form, const qg::FusedArgs& a, int tile, bool kmajor, bool any, hipStream_t s) {
    if (tile >= DIRECT_KN) return qg::launch_fused_direct_kn(a, form, direct_rows(tile), any, s);
    if (tile >= DIRECT) return qg::launch_fused_direct(a, form, direct_rows(tile), direct_cols(tile), any, s);
    const qg::FusedTile t = (qg::FusedTile)tile;
    return form == qg::FUSED_ONE ? qg::launch_fused_one(a, t, kmajor, s)
           : form == qg::FUSED_PAIR ? qg::launch_fused_pair(a, t, kmajor, s) : qg::launch_fused_grad(a, t, kmajor, s);
}

const char* kernel_name(int form, const Choice& c) {
    static const char* const names[3][KINDS] = {
        {"fused_one_256x256", "fused_one_128x128", "fused_one_128x128_deep", "fused_one_64x128_deep",
         "fused_one_any_64x128", "fused_one_direct_16x16", "fused_one_direct_16x32", "fused_one_direct_32x16",
         "fused_one_direct_32x32", "fused_one_direct_64x16", "fused_one_direct_64x32", "fused_one_direct_kn_16",
         "fused_one_direct_kn_32"},
        {"fused_pair_256x256", "fused_pair_128x128", "fused_pair_128x128_deep", "fused_pair_64x128_deep",
         "fused_pair_any_64x128", "fused_pair_direct_16x16", "fused_pair_direct_16x32",
         "fused_pair_direct_32x16", "fused_pair_direct_32x32", "fused_pair_direct_64x16",
         "fused_pair_direct_64x32", "fused_pair_direct_kn_16", "fused_pair_direct_kn_32"},
        {"fused_grad_256x256", "fused_grad_128x128", "fused_grad_128x128_deep", "fused_grad_64x128_deep",
         "fused_grad_any_64x128", "fused_grad_direct_16x16", "fused_grad_direct_16x32",
         "fused_grad_direct_32x16", "fused_grad_direct_32x32", "fused_grad_direct_64x16",
         "fused_grad_direct_64x32", "fused_grad_direct_kn_16", ""}};
    static const char* const joined[3] = {"fused_one_joined", "fused_pair_joined", "fused_grad_joined"};
    return c.splits > 1 ? joined[form] : names[form][c.tile];
}

// An operand whose rows are laid out once more, and where.
struct Padded {
    const int8_t** p; int64_t* ld;
    int64_t rows, cols;
    bool needed() const { return !whole_pieces(*p, *ld, cols); }
    int64_t ldd() const { return up16(cols); }
    size_t bytes() const { return up256((size_t)rows * ldd()); }
};

// The product: its operands padded first where the choice says so, the second kernel behind
// it where K is divided.
qg_status run(int form, qg::FusedArgs& a, const Choice& c, bool kmajor, bool any, Padded* ops, int count, char* pad, void* partial,
              hipStream_t s) {
    a.b_cols = a.e.N;
    a.k_bytes = a.K;
    if (c.pad) {
        qg::PadArgs p{};
        for (int i = 0; i < count; ++i) {
            if (!ops[i].needed()) continue;
            p.src[p.count] = *ops[i].p; p.ld[p.count] = *ops[i].ld;
            p.rows[p.count] = ops[i].rows; p.cols[p.count] = ops[i].cols;
            p.dst[p.count] = (int8_t*)pad; p.ldd[p.count] = ops[i].ldd();
            ++p.count;
            *ops[i].p = (const int8_t*)pad; *ops[i].ld = ops[i].ldd();
            pad += ops[i].bytes();
        }
        QG_TRY_HIP(qg::launch_fused_pad(p, s));
        a.k_bytes = (int)up16(a.K);
        a.b_cols = (int)up16(a.e.N);
        any = false;
    }
    if (c.splits > 1) {
        a.partial = (int*)partial;
        a.splits = c.splits;
        a.split_chunks = c.split_chunks;
        a.ld_partial = c.ld_partial;
    }
    QG_TRY_HIP(launch_fused(form, a, c.tile, kmajor, any, s));
    if (c.splits > 1) QG_TRY_HIP(qg::launch_fused_join(a, form, s));
    return done(hipSuccess, kernel_name(form, c));
}

// A launch holds fewer than 2^32 threads: 512 to a tile of 64 x 128, and to 32 columns of a bias.
bool too_many_tiles(int64_t rows, int64_t cols) { return ((rows + 63) / 64) * ((cols + 127) / 128) >= ((int64_t)1 << 23) - 2048; }

struct Scales { const float* p; int64_t len; };

bool scale_ok(const Scales& s, int64_t n) { return s.p != nullptr && aligned(s.p, 4) && (s.len == 1 || s.len == n); }

// The forward calls.
struct Forward {
    int64_t M, N, K;
    const int8_t* A; int64_t lda;
    const int8_t* W[2]; int64_t ldw[2]; int b_trans;
    int pair;

    // Operands whose rows may have to be padded.
    int operands(Padded* o) {
        o[0] = {&A, &lda, M, K};
        for (int h = 0; h < pair; ++h) o[1 + h] = {&W[h], &ldw[h], b_trans ? N : K, b_trans ? K : N};
        return 1 + pair;
    }
    size_t pad_bytes() {
        Padded o[3];
        size_t n = 0;
        for (int i = operands(o); i-- > 0;) n += o[i].needed() ? o[i].bytes() : 0;
        return n;
    }
    Choice choice(bool blocks) {
        const size_t pad = pad_bytes();
        return choose({pair == 2 ? qg::FUSED_PAIR : qg::FUSED_ONE, M, N, K, 1, b_trans != 0, pad == 0, blocks,
                       span_ok(K, up16(lda), std::max(up16(ldw[0]), up16(ldw[pair - 1])), b_trans) && M * (up16(K) / 16) < (int64_t)1 << 32
                           ? (int64_t)pad : -1});
    }
};

bool sizes_bad(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= LIM || N >= LIM || K >= LIM;
}

size_t forward_workspace(Forward f, bool blocks) {
    if (sizes_bad(f.M, f.N, f.K) || f.M == 0 || f.N == 0 || f.K == 0) return 0;
    const Choice c = f.choice(blocks);
    return (c.pad ? f.pad_bytes() : 0) + up256(c.bytes);
}

// Rows of an output, residual or checkpoint of which a tile's 256 stay within 32-bit offsets.
bool rows_ok(int64_t ld) { return ld < (int64_t)1 << 22; }

bool checkpoint_ok(const int8_t* c, int64_t ldc, const float* s, int64_t lds, int64_t N) {
    return c != nullptr && s != nullptr && aligned(s, 4) && ldc >= N && lds >= blocks_of(N);
}

qg_status forward(Forward f, const Scales& act, const Scales* ws, const float* bias, qg_activation activation,
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
    if (too_many_tiles(M, N * f.pair) || !rows_ok(ldo) || (res != nullptr && !rows_ok(ldr)) ||
        (ckpt != nullptr && (!rows_ok(ld_ckpt) || !rows_ok(ld_ckpt_scale))))
        return QG_ERR_UNSUPPORTED;
    const Choice c = f.choice(ckpt != nullptr);
    const size_t pad = c.pad ? f.pad_bytes() : 0, need = pad + up256(c.bytes);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return QG_ERR_WORKSPACE;

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
    Padded ops[3];
    const int count = f.operands(ops);
    bool any = false;
    for (int i = 0; i < count; ++i) any = any || ops[i].needed();
    qg::FusedArgs a{};
    a.e = e;
    a.A[0] = f.A; a.lda = f.lda;
    ops[0].p = &a.A[0]; ops[0].ld = &a.lda;
    for (int h = 0; h < f.pair; ++h) {
        a.B[h] = f.W[h];
        a.ldb[h] = f.ldw[h];
        ops[1 + h].p = &a.B[h]; ops[1 + h].ld = &a.ldb[h];
    }
    a.K = (int)K; a.branches = 1;
    return run(f.pair == 2 ? qg::FUSED_PAIR : qg::FUSED_ONE, a, c, f.b_trans != 0, any, ops, count, (char*)workspace,
               (char*)workspace + pad, (hipStream_t)stream);
}

// The gradients.
struct Backward {
    int64_t M, N, K;
    const int8_t* W[2]; int64_t ldw[2]; int b_trans;
    int pair;
    bool with_bias;

    int operands(Padded* o) {
        for (int h = 0; h < pair; ++h) o[h] = {&W[h], &ldw[h], b_trans ? N : K, b_trans ? K : N};
        return pair;
    }
    size_t pad_bytes() {
        Padded o[2];
        size_t n = 0;
        for (int i = operands(o); i-- > 0;) n += o[i].needed() ? o[i].bytes() : 0;
        return n;
    }
    // the product's: outputs [M,K], sums over N
    Choice choice() {
        const size_t pad = pad_bytes();
        return choose({qg::FUSED_GRAD, M, K, N, pair, b_trans == 0, pad == 0, false,
                       span_ok(N, 0, std::max(up16(ldw[0]), up16(ldw[pair - 1])), !b_trans) ? (int64_t)pad : -1});
    }
};

// Where a gradient's workspace holds what.
struct GradPlan {
    int64_t np, ldq;
    size_t hi, lo, row_scale, part, pad, sums, bytes;
    int parts;
    Choice c;
    explicit GradPlan(Backward b)
        : np((b.N + 127) / 128 * 128), ldq(np * b.pair), parts(b.with_bias ? qg::grad_rows_parts(b.M, b.N) : 0), c(b.choice()) {
        size_t at = 0;
        auto take = [&](size_t n) { const size_t here = at; at += up256(n); return here; };
        hi = take((size_t)b.M * ldq);
        lo = take((size_t)b.M * ldq);
        row_scale = take((size_t)b.M * 4);
        part = take((size_t)parts * b.N * 4);
        pad = take(c.pad ? b.pad_bytes() : 0);
        sums = take(c.bytes);
        bytes = at;
    }
};

size_t backward_workspace(Backward b) {
    if (sizes_bad(b.M, b.N, b.K) || b.M == 0 || b.N == 0 || b.K == 0 || b.N > QG_A8W8_GRAD_MAX_COLUMNS) return 0;
    return GradPlan(b).bytes;
}

qg_status backward(Backward b, const void* dy, qg_dtype dtype, int64_t ld_dy, const Scales* ws, const int8_t* ckpt,
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
        return done(qg::launch_clear(dbias, N, (hipStream_t)stream), "fused_clear");
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
    if (too_many_tiles(2 * M, K) || !rows_ok(ld_dx)) return QG_ERR_UNSUPPORTED;
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
    a.part = dbias != nullptr ? (float*)(w + p.part) : nullptr; a.parts = p.parts;
    QG_TRY_HIP(qg::launch_grad_rows(a, b.pair == 2, dtype == QG_BF16, s));

    qg::FusedArgs f{};
    f.e.M = (int)M; f.e.N = (int)K;
    f.e.act_scale = a.row_scale; f.e.as_stride = 1;
    f.e.out = dx; f.e.ldo = ld_dx; f.e.out_type = dtype;
    f.A[0] = a.hi; f.A[1] = a.lo; f.lda = p.ldq;
    Padded ops[2];
    const int count = b.operands(ops);
    bool any = false;
    for (int h = 0; h < b.pair; ++h) {
        any = any || ops[h].needed();
        f.B[h] = b.W[h];
        f.ldb[h] = b.ldw[h];
        ops[h].p = &f.B[h]; ops[h].ld = &f.ldb[h];
    }
    f.K = (int)N; f.branches = b.pair;
    f.part = a.part; f.parts = p.parts; f.dbias = dbias; f.bias_n = (int)N;
    return run(qg::FUSED_GRAD, f, p.c, b.b_trans == 0, any, ops, count, w + p.pad, w + p.sums, s);
}

}  // namespace

extern "C" {

size_t qgemm_a8w8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* W,
                                         int64_t ldw, int b_trans, int with_checkpoint) {
    return forward_workspace({M, N, K, A, lda, {W, nullptr}, {ldw, 0}, b_trans, 1}, with_checkpoint != 0);
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
                                        int64_t ld_gate, const int8_t* W_up, int64_t ld_up, int b_trans, int with_checkpoint) {
    return forward_workspace({M, N, K, A, lda, {W_gate, W_up}, {ld_gate, ld_up}, b_trans, 2}, with_checkpoint != 0);
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
