// The factors of the fused products' gradients: for each row of dy the products of
// dy with what the 8-bit checkpoint gives (and the weight's scale of the column), in
// 16-bit fixed point as two int8 planes, the row's scale, and dbias.
//
// Mathematics: linear p = dy act'(z); gated p = dy u act'(g) and q = dy act(g).
// The product dx = (p s) W would need p s in bf16 and the int8 weight widened to
// bf16 in the kernel.  Held instead as t = rint(value * 32639 / a), a the row's largest
// magnitude, and split as t = 256 hi + lo with both in int8 (|hi| <= 127, -128 <= lo <=
// 127), it is two int8 products with the weight as it is: the same time on the
// matrix cores as one bf16 product, and sums that are exact.  The rounding is a /
// 65278 at most: half a bf16 step of a value of a / 128, so large factors are held
// more closely than bf16 would, and values below that less, in proportion to what
// they add to the sum.
//
// Bound by HBM: dy and the checkpoint are read once and stay packed in registers
// between the row's maximum and its codes, where p and q are computed again.
#include "fused_common.h"

namespace qg {
namespace {

constexpr float STEPS = 32639.f;   // 127 * 256 + 127

template <int G>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
#pragma unroll
    for (int off = G < 64 ? G / 2 : 32; off >= 1; off >>= 1) v = umax(v, (uint32_t)__shfl_xor((int)v, off));
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) v = umax(v, red[w]);
    }
    return v;
}

// Eight codes of a row of n from column c on, those past its end 0.
__device__ __forceinline__ uint2 load_codes(const int8_t* row, int c, int n) {
    uint2 r = make_uint2(0u, 0u);
    if (c + 8 <= n) {
        __builtin_memcpy(&r, row + c, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = c + i < n ? (uint32_t)(uint8_t)row[c + i] : 0u;
            if (i < 4) r.x |= b << (8 * i);
            else r.y |= b << (8 * (i - 4));
        }
    }
    return r;
}
__device__ __forceinline__ float code_at(uint2 r, int i) {
    return (float)(int8_t)((i < 4 ? r.x : r.y) >> (8 * (i & 3)));
}

// A weight's scales of columns c .. c + 7, 0 past the last.
__device__ __forceinline__ void load_scales(const float* w, int stride, int c, int n, float* s) {
    if (stride == 0) {
        const float one = w[0];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = c + e < n ? one : 0.f;
    } else {
        Pack8<float> v;
        if (c + 8 <= n) load8<false>(w, c, n, v);
        else load8<true>(w, c, n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = value(v, e);
    }
}

// G lanes a row, ITER groups of eight columns a lane; a workgroup walks rows.  HOLD, up to
// two groups a lane: the factors stay in registers between the row's maximum and their
// codes, the weights' scales, which every row needs again, lie in LDS, and the next row is on
// its way meanwhile (4096 x 14336 gated 232 us with none of that, a row a workgroup).  Wider
// rows are read, and their factors computed, again for the codes, one group at a time, and
// their sums for dbias lie in memory (300 x 60000 gated 361 us where the loops over groups were
// unrolled and spilled, 101 so).
template <typename T, int G, int ITER, bool PAIR, bool BIAS>
__global__ __launch_bounds__(G < 256 ? 256 : G) void grad_rows_kernel(GradRowsArgs a) {
    constexpr int RPW = G < 256 ? 256 / G : 1;
    constexpr int H = PAIR ? 2 : 1;
    constexpr bool HOLD = ITER <= 2;
    constexpr int TURNS = HOLD ? ITER : 1;   // unrolled where registers hold every group
    __shared__ uint32_t red[2][G < 64 ? 1 : G / 64];
    __shared__ float part[BIAS && RPW > 1 ? (RPW - 1) * G * ITER * 8 : 1];
    // a lane's own scales, four to a place: each lane reads what it wrote
    __shared__ __attribute__((aligned(16))) float ws[HOLD ? RPW * H * ITER * 2 * G * 4 : 1];
    const int t = threadIdx.x % G, group = threadIdx.x / G;
    const int N = a.N;
    auto place = [&](int h, int i, int half) { return ws + ((((group * H + h) * ITER + i) * 2 + half) * G + t) * 4; };
    float db[BIAS && HOLD ? ITER : 1][8];
#pragma unroll
    for (int i = 0; i < (BIAS && HOLD ? ITER : 1); ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) db[i][e] = 0.f;

    constexpr int WI = HOLD ? ITER : 1;
    struct Row {
        Pack8<T> y[WI];
        uint2 c[H][WI];
        float s[H][WI];
    };
    auto fetch_group = [&](int64_t r, Row& v, int i) {
        const int c = (i * G + t) * 8, w = HOLD ? i : 0;
        if (c + 8 <= N) load8<false>(reinterpret_cast<const T*>(a.dy) + r * a.ldy, c, N, v.y[w]);
        else load8<true>(reinterpret_cast<const T*>(a.dy) + r * a.ldy, c, N, v.y[w]);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (a.ckpt[h] == nullptr) continue;
            v.c[h][w] = load_codes(a.ckpt[h] + r * a.ld_ckpt, c, N);
            v.s[h][w] = c < N ? a.ckpt_scale[h][r * a.ld_ckpt_scale + c / INT8_BLOCK] : 0.f;
        }
    };
    auto fetch = [&](int64_t r, Row& v) {
        if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < ITER; ++i) fetch_group(r, v, i);
        }
    };
    // The factors of group i with the weight's scales; dy is 0 past the last column.
    auto factors = [&](const Row& row, int i, float (*v)[8], bool add, bool first) {
        const int w = HOLD ? i : 0;
        if (a.ckpt[0] == nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[0][e] = value(row.y[w], e);
        } else {
            with_activation(a.activation, [&](auto kind) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f, slope;
                    activate_both<decltype(kind)::value>(code_at(row.c[0][w], e) * row.s[0][w], f, slope);
                    const float y = value(row.y[w], e);
                    if constexpr (PAIR) {
                        v[0][e] = y * (code_at(row.c[1][w], e) * row.s[1][w]) * slope;
                        v[1][e] = y * f;
                    } else {
                        v[0][e] = y * slope;
                    }
                }
            });
        }
        if constexpr (BIAS) {
            if constexpr (HOLD) {
                if (add) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) db[i][e] += v[0][e];
                }
            } else if (add) {
                // the workgroup's own partial sums, in L2
                const int c = (i * G + t) * 8;
                float* own = a.part + (int64_t)blockIdx.x * N + c;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int count = N - c - 4 * half;
                    v4f sum = {v[0][4 * half], v[0][4 * half + 1], v[0][4 * half + 2], v[0][4 * half + 3]};
                    if (!first) sum = load4(own + 4 * half, count) + sum;
                    if (count > 0) store4(own + 4 * half, QG_FP32, count, sum);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float s[8];
            if constexpr (HOLD) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const v4f q = *reinterpret_cast<const v4f*>(place(h, i, half));
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[4 * half + e] = q[e];
                }
            } else {
                load_scales(a.w_scale[h], a.ws_stride[h], (i * G + t) * 8, N, s);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[h][e] *= s[e];
        }
    };
    // red: two in turn, since a wave may be one row ahead of the others' reads
    auto finish = [&](int64_t row, bool live, Row& v, int turn, bool first) {
        float held[HOLD ? ITER : 1][H][8];
        uint32_t top = 0u;
#pragma unroll TURNS
        for (int i = 0; i < ITER; ++i) {
            float (*f)[8] = held[HOLD ? i : 0];
            if constexpr (!HOLD) fetch_group(live ? row : a.M - 1, v, i);
            factors(v, i, f, live, first);
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = umax(top, abs_bits(f[h][e]));
            if constexpr (!HOLD) __builtin_amdgcn_sched_barrier(0);   // one group at a time
        }
        top = row_max<G>(top, red[turn]);
        if (!live) return;
        // a NaN or an infinity makes the row's scale NaN, and so every output of the row, whatever
        // its planes then hold (int8 values like any)
        const float most = __uint_as_float(top), up = most < 0x1p-90f ? 0x1p60f : 1.0f;   // STEPS / most stays finite
        const float inv = top >= INF_BITS || top == 0u ? 0.f : STEPS / (most * up);
        if (t == 0) a.row_scale[row] = top >= INF_BITS ? __uint_as_float(0x7fc00000u) : most / STEPS;
#pragma unroll TURNS
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
            if (c >= a.np) continue;
            float (*f)[8] = held[HOLD ? i : 0];
            if constexpr (!HOLD) {
                __builtin_amdgcn_sched_barrier(0);
                fetch_group(row, v, i);
                factors(v, i, f, false, false);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                uint32_t b[8], hi[2], lo[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = nearest_bits((f[h][e] * up) * inv);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    lo[q] = pack_bytes(b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
                    hi[q] = pack_bytes(b[4 * q] + 128u, b[4 * q + 1] + 128u, b[4 * q + 2] + 128u, b[4 * q + 3] + 128u, 1);
                }
                const int64_t at = row * a.ldq + (int64_t)h * a.np + c;
                *reinterpret_cast<uint2*>(a.hi + at) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(a.lo + at) = make_uint2(lo[0], lo[1]);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPW, M = a.M;
    int64_t row = (int64_t)blockIdx.x * RPW + group;   // whole groups; no barrier where a workgroup has several
    if constexpr (HOLD) {
        Row now, next;
        fetch(row < M ? row : M - 1, now);
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                float s[8];
                load_scales(a.w_scale[h], a.ws_stride[h], (i * G + t) * 8, N, s);
#pragma unroll
                for (int half = 0; half < 2; ++half) *reinterpret_cast<v4f*>(place(h, i, half)) = v4f{s[4 * half], s[4 * half + 1], s[4 * half + 2], s[4 * half + 3]};
            }
        for (int turn = 0; row - group < M; row += step, turn ^= 1) {
            if (row + step < M) fetch(row + step, next);
            finish(row, row < M, now, turn, false);
            now = next;
        }
    } else {
        const int64_t first = row;
        for (int turn = 0; row - group < M; row += step, turn ^= 1) {
            const bool live = row < M;
            Row now;
            finish(row, live, now, turn, row == first);
        }
    }
    if constexpr (BIAS && HOLD) {
        if constexpr (RPW > 1) {
            if (group > 0) {
#pragma unroll
                for (int i = 0; i < ITER; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) part[(((group - 1) * ITER + i) * 8 + e) * G + t] = db[i][e];
            }
            __syncthreads();
            if (group > 0) return;
            for (int g = 0; g < RPW - 1; ++g)
#pragma unroll
                for (int i = 0; i < ITER; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) db[i][e] += part[((g * ITER + i) * 8 + e) * G + t];
        }
        float* out = a.part + (int64_t)blockIdx.x * N;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * G + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < N) out[c + e] = db[i][e];
        }
    }
}

__global__ __launch_bounds__(256) void clear_kernel(float* x, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) x[i] = 0.f;
}

template <typename T, bool PAIR, bool BIAS>
hipError_t by_width(const GradRowsArgs& a, hipStream_t s) {
    bool done = false;
#define QG_ROWS(G, ITER, LIMIT)                                                                                     \
    if (!done && a.N <= LIMIT) {                                                                                    \
        constexpr int RPW = G < 256 ? 256 / G : 1;                                                                  \
        const int64_t groups = ((int64_t)a.M + RPW - 1) / RPW, most = G >= 1024 ? 256 : G == 512 ? 512 : 1024;      \
        const unsigned grid = (unsigned)(BIAS ? a.parts : groups < most ? groups : most);                           \
        hipLaunchKernelGGL((grad_rows_kernel<T, G, ITER, PAIR, BIAS>), dim3(grid), dim3(G < 256 ? 256 : G), 0, s, a); \
        done = true;                                                                                                \
    }
    // One group a lane as far as lanes go: more waves, fewer registers (8192 x 2816, gated 82 -> 75 us with the
    // product, linear 69 -> 62, of 512 x 1 after 256 x 2; 4096 x 8192 gated 97 -> 88 of 1024 x 1 after 512 x 2).
    QG_ROWS(64, 1, 512)
    QG_ROWS(256, 1, 2048)
    QG_ROWS(512, 1, 4096)
    QG_ROWS(1024, 1, 8192)
    QG_ROWS(1024, 2, 16384)
    QG_ROWS(1024, 4, 32768)
    QG_ROWS(1024, 8, 65536)
#undef QG_ROWS
    if (!done) return hipErrorInvalidValue;
    return hipGetLastError();
}

template <typename T>
hipError_t by_form(const GradRowsArgs& a, bool pair, hipStream_t s) {
    if (pair) return by_width<T, true, false>(a, s);
    return a.part != nullptr ? by_width<T, false, true>(a, s) : by_width<T, false, false>(a, s);
}

}  // namespace

// Workgroups of the row kernel where each leaves partial sums of dbias.
int grad_rows_parts(int64_t M, int64_t N) {
    // One to a compute unit for few rows and for wide ones, whose partial sums are many bytes (4096 x 8192
    // 73 us with 256, 77 with 512).
    const int64_t rows = N <= 512 ? 4 : 1, groups = (M + rows - 1) / rows, most = N > 4096 || M <= 1024 * rows ? 256 : 512;
    return (int)(groups < most ? groups : most);
}

hipError_t launch_clear(float* x, int64_t n, hipStream_t s) {
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, x, n);
    return hipGetLastError();
}

hipError_t launch_grad_rows(const GradRowsArgs& a, bool pair, bool bf16, hipStream_t s) {
    return bf16 ? by_form<__bf16>(a, pair, s) : by_form<_Float16>(a, pair, s);
}

}  // namespace qg
