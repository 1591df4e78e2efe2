// norm.hip -- root-mean-square norm of rows with the residual's addition,
// and 8-bit codes of rows with a scale each.
//
// With x and the optional residual r (both [rows, D]) and a weight w[D]:
//     h = x + r                          FP32, one addition
//     r <- round(h)                      in the residual's own type
//     rstd = 1 / sqrt(sum(h^2) / D + eps)
//     p = h * w,   y = p * rstd          (BF16 output)
//     m = max |p|, scale = m * rstd / 127, code = rint(p * 127 / m)
// The codes need no rstd: it scales a row's p and its m alike, so a code
// depends on h and w only.  Without the norm (quant_rows) p = x, scale =
// m / 127.  The norm takes the unrounded sum h, so y is as exact as if the
// residual stream were held in 32 bits for this layer.
//
// A row is read once and held in registers, 8 elements (16 bytes of BF16) a
// lane and step; sum(h^2) and max|p| are reduced together (DPP inside a
// wave, one LDS exchange between waves, so one barrier a row), and the
// outputs are written from the registers.  It is bound by HBM for many rows
// (8192 x 7168, BF16 residual and output: 74 us, 6.3 TB/s, where scaling a
// tensor in place runs at 6.0; 84 without the non-temporal loads of x; with
// an FP32 residual and codes 122 us, 5.3 TB/s; codes alone of 14560 x 7168 50 us,
// 6.2 TB/s) and by its one memory round trip for few (one row of 7168:
// 2.9 us, 64 rows with codes 4.0).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tp1_proj.h"
#include "args.hpp"
#include "device.hpp"

namespace tp1 {

namespace {

enum Residual { kNoResidual = 0, kBf16Residual = 1, kFp32Residual = 2 };

struct RowArgs {
    const uint16_t *x;
    long ldx;
    void *res;          // residual rows (type by template), read and rewritten
    long ldr;
    const uint16_t *w;  // norm weight [D], or nullptr
    uint16_t *y;        // BF16 output rows, contiguous, or nullptr
    int8_t *codes;      // 8-bit output rows, contiguous, or nullptr
    float *scale;       // one a row, with codes
    int rows, D;
    float eps;
};

// TPR threads share a row (a wave or more), holding IT groups of 8 elements
// each; a workgroup of T threads takes T / TPR rows.
template <int T, int TPR, int IT, int RES, bool NORM>
__global__ __launch_bounds__(T) void row_kernel(RowArgs a) {
    static_assert(TPR % 64 == 0 && T % TPR == 0, "whole waves share a row");
    constexpr int WPR = TPR / 64;
    constexpr int RPB = T / TPR;
    static_assert(WPR == 1 || RPB == 1, "one row a workgroup once it takes several waves");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int t = tid % TPR;
    const int row = scalar(blockIdx.x * RPB + tid / TPR);
    if (row >= a.rows) return;  // whole waves; with a barrier RPB is 1 and no row is past the end

    float p[IT][8];
    float ss = 0.f;
    unsigned top = 0;
    u32x4 xv[IT], wv[IT];
    f32x4 rv[IT][2];
    // every load of the row first
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c < a.D) {
            xv[i] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(a.x + (size_t)row * a.ldx + c));
            if constexpr (RES == kBf16Residual) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(
                    static_cast<const uint16_t *>(a.res) + (size_t)row * a.ldr + c);
                rv[i][0] = __builtin_bit_cast(f32x4, v);
            }
            if constexpr (RES == kFp32Residual) {
                const f32x4 *r = reinterpret_cast<const f32x4 *>(
                    static_cast<const float *>(a.res) + (size_t)row * a.ldr + c);
                rv[i][0] = r[0];
                rv[i][1] = r[1];
            }
            if constexpr (NORM) wv[i] = *reinterpret_cast<const u32x4 *>(a.w + c);
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c < a.D) {
            float h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[2 * j] = bf16_lo(xv[i][j]);
                h[2 * j + 1] = bf16_hi(xv[i][j]);
            }
            if constexpr (RES == kBf16Residual) {
                const u32x4 r = __builtin_bit_cast(u32x4, rv[i][0]);
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[2 * j] += bf16_lo(r[j]);
                    h[2 * j + 1] += bf16_hi(r[j]);
                    o[j] = pack_bf16(h[2 * j], h[2 * j + 1]);
                }
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.res) + (size_t)row * a.ldr +
                                           c) = o;
            }
            if constexpr (RES == kFp32Residual) {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] += rv[i][j / 4][j % 4];
                f32x4 *r = reinterpret_cast<f32x4 *>(static_cast<float *>(a.res) +
                                                     (size_t)row * a.ldr + c);
                r[0] = f32x4{h[0], h[1], h[2], h[3]};
                r[1] = f32x4{h[4], h[5], h[6], h[7]};
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (NORM) {
                    ss = __builtin_fmaf(h[j], h[j], ss);
                    p[i][j] = h[j] * ((j & 1) ? bf16_hi(wv[i][j / 2]) : bf16_lo(wv[i][j / 2]));
                } else {
                    p[i][j] = h[j];
                }
                const unsigned m = __float_as_uint(p[i][j]) & 0x7FFFFFFFu;
                top = m > top ? m : top;
            }
        }
    }
    if constexpr (NORM) ss = sum64(ss);
    top = max64(top);
    if constexpr (WPR > 1) {
        __shared__ float wave_ss[WPR];
        __shared__ unsigned wave_top[WPR];
        if (lane == 0) {
            wave_ss[tid >> 6] = ss;
            wave_top[tid >> 6] = top;
        }
        __syncthreads();
        ss = 0.f;
        top = 0;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            ss += wave_ss[w];
            top = wave_top[w] > top ? wave_top[w] : top;
        }
    }
    const float rstd = NORM ? rsqrtf(ss / (float)a.D + a.eps) : 1.f;
    if (a.y) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + t) * 8;
            if (c < a.D) {
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = pack_bf16(p[i][2 * j] * rstd, p[i][2 * j + 1] * rstd);
                *reinterpret_cast<u32x4 *>(a.y + (size_t)row * a.D + c) = o;
            }
        }
    }
    if (a.codes) {
        // A row with an infinity or a NaN has no codes: scale NaN, so that
        // whatever is computed from it is NaN, and codes 0.  A row whose
        // largest magnitude is so small that 127 / m would overflow is
        // scaled up by 2^100 first (exact).
        const float m = __uint_as_float(top);
        const bool live = top < 0x7F800000u && top > 0;
        const float up = m < 1e-30f ? 0x1p100f : 1.f;
        const float inv = live ? 127.f / (m * up) : 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + t) * 8;
            if (c < a.D) {
                unsigned o[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int code = live ? (int)rintf(p[i][j] * up * inv) : 0;
                    o[j / 4] |= ((unsigned)code & 0xFFu) << (8 * (j % 4));
                }
                *reinterpret_cast<u32x2 *>(a.codes + (size_t)row * a.D + c) = u32x2{o[0], o[1]};
            }
        }
        if (t == 0)
            a.scale[row] = top < 0x7F800000u ? (m / 127.f) * rstd
                                             : __uint_as_float(0x7FC00000u);
    }
}

template <int T, int TPR, int IT, bool NORM>
hipError_t launch_rows(const RowArgs &a, int res, hipStream_t st) {
    const unsigned g = (unsigned)((a.rows + T / TPR - 1) / (T / TPR));
    if constexpr (NORM) {
        if (res == kBf16Residual)
            hipLaunchKernelGGL((row_kernel<T, TPR, IT, kBf16Residual, true>), dim3(g), dim3(T), 0,
                               st, a);
        else if (res == kFp32Residual)
            hipLaunchKernelGGL((row_kernel<T, TPR, IT, kFp32Residual, true>), dim3(g), dim3(T), 0,
                               st, a);
        else
            hipLaunchKernelGGL((row_kernel<T, TPR, IT, kNoResidual, true>), dim3(g), dim3(T), 0,
                               st, a);
    } else {
        hipLaunchKernelGGL((row_kernel<T, TPR, IT, kNoResidual, false>), dim3(g), dim3(T), 0, st,
                           a);
    }
    return hipGetLastError();
}

// A wave a row up to 1024 elements (16384 rows of 1024: 24.3 us, 26.5 with a
// workgroup a row); above that a workgroup a row, with few elements a lane: a
// wave a row of 4096 takes 150 us against 134, and one row of 7168 3.4 us with
// 256 lanes against 2.9 with 512.
template <bool NORM>
hipError_t dispatch_rows(const RowArgs &a, int res, hipStream_t st) {
    const int groups = a.D / 8;
    if (groups <= 64) return launch_rows<256, 64, 1, NORM>(a, res, st);
    if (groups <= 128) return launch_rows<256, 64, 2, NORM>(a, res, st);
    if (groups <= 256) return launch_rows<256, 256, 1, NORM>(a, res, st);
    if (groups <= 512) return launch_rows<512, 512, 1, NORM>(a, res, st);
    if (groups <= 1024) return launch_rows<512, 512, 2, NORM>(a, res, st);
    if (groups <= 2048) return launch_rows<512, 512, 4, NORM>(a, res, st);
    return launch_rows<1024, 1024, 4, NORM>(a, res, st);
}

int check_rows(int rows, int D, const void *x, long *ldx) {
    if (rows < 0 || D <= 0 || D % 8 != 0 || D > PROJ_MAX_ROW) return PROJ_EINVAL;
    if (*ldx == 0) *ldx = D;
    if (*ldx < D) return PROJ_EINVAL;
    if (rows == 0) return PROJ_OK;
    if (!x) return PROJ_EINVAL;
    if (!is_aligned(x, 16) || *ldx % 8 != 0) return PROJ_EALIGN;
    return PROJ_OK;
}

}  // namespace
}  // namespace tp1

extern "C" int proj_rms_norm(int rows, int D, const void *x, long ldx, void *residual, long ldr,
                             int residual_fp32, const void *weight, float eps, void *y,
                             void *codes, void *scale, void *stream) {
    using namespace tp1;
    int rc = check_rows(rows, D, x, &ldx);
    if (rc != PROJ_OK) return rc;
    if (residual_fp32 != 0 && residual_fp32 != 1) return PROJ_EINVAL;
    if (!(eps >= 0.f)) return PROJ_EINVAL;
    if (ldr == 0) ldr = D;
    if (residual && ldr < D) return PROJ_EINVAL;
    if (rows == 0) return PROJ_OK;
    if (!weight || (!y && !codes) || (!codes != !scale)) return PROJ_EINVAL;
    if (!is_aligned(weight, 16) || !is_aligned(residual, 16) || !is_aligned(y, 16) ||
        !is_aligned(codes, 8) || !is_aligned(scale, 4) || (residual && ldr % 8 != 0))
        return PROJ_EALIGN;
    const size_t rsize = residual_fp32 ? 4 : 2;
    const Span in[] = {Span(x, span_bytes(rows, (size_t)D * 2, (size_t)ldx * 2)),
                       Span(weight, (size_t)D * 2)};
    const Span out[] = {
        Span(residual, residual ? span_bytes(rows, D * rsize, (size_t)ldr * rsize) : 0),
        Span(y, (size_t)rows * D * 2), Span(codes, (size_t)rows * D),
        Span(scale, (size_t)rows * 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (out[i].meets(s)) return PROJ_EINVAL;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return PROJ_EINVAL;
    }
    const RowArgs a{static_cast<const uint16_t *>(x), ldx, residual, ldr,
                    static_cast<const uint16_t *>(weight), static_cast<uint16_t *>(y),
                    static_cast<int8_t *>(codes), static_cast<float *>(scale), rows, D, eps};
    const int res = !residual ? kNoResidual : residual_fp32 ? kFp32Residual : kBf16Residual;
    if (dispatch_rows<true>(a, res, static_cast<hipStream_t>(stream)) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}

extern "C" int proj_quant_rows(int rows, int D, const void *x, long ldx, void *codes, void *scale,
                               void *stream) {
    using namespace tp1;
    int rc = check_rows(rows, D, x, &ldx);
    if (rc != PROJ_OK) return rc;
    if (rows == 0) return PROJ_OK;
    if (!codes || !scale) return PROJ_EINVAL;
    if (!is_aligned(codes, 8) || !is_aligned(scale, 4)) return PROJ_EALIGN;
    const Span in(x, span_bytes(rows, (size_t)D * 2, (size_t)ldx * 2));
    const Span c(codes, (size_t)rows * D), s(scale, (size_t)rows * 4);
    if (c.meets(in) || s.meets(in) || c.meets(s)) return PROJ_EINVAL;
    const RowArgs a{static_cast<const uint16_t *>(x), ldx, nullptr, 0, nullptr, nullptr,
                    static_cast<int8_t *>(codes), static_cast<float *>(scale), rows, D, 0.f};
    if (dispatch_rows<false>(a, kNoResidual, static_cast<hipStream_t>(stream)) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}
