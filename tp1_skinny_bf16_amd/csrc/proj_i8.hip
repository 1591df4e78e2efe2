// proj_i8.hip -- the decode projection in 8-bit integers.
//
//     y[b, n] = bf16( (sum_k xc[b, k] * wc[n, k]) * (xs[b] * ws[n]) )
//
// with codes xc [B, K] and wc [N, K] (int8, row-major) and one FP32 scale a
// row (a token of x, an output channel of W).  The integer sum is exact
// (|code| <= 128 and K <= PROJ_I8_MAX_K keep it inside 32 bits), so the
// result does not depend on how K is split or in which order slices arrive;
// it is rounded three times: the sum to FP32, the products with the scales,
// and the result to BF16.
//
// What bounds it: the weight is read once, N * K bytes, half of what the
// BF16 projection streams; at 16 rows and fewer that stream is all there is.
// From 64 rows on every compute unit also carries x (B * K bytes a row
// group) from the L2 beside it.
//
// i8_pipe_kernel: a workgroup owns a range of weight rows of one K slice and
// walks them in groups of 16 * NTB rows, KB bytes of K a step.  The step's x
// rows and weight rows go straight into a ring of D LDS stages
// (global_load_lds_dwordx4), D - 1 steps ahead of the one being multiplied,
// so loads in flight hold no registers; one barrier a step.  A 16-byte piece
// p of row r sits at position p ^ (r mod pieces-per-row) of its row, which
// spreads the 16 rows a fragment read touches over all LDS banks.
// v_mfma_i32_16x16x64_i8 takes 16 consecutive codes of one row a lane: lane l
// supplies row l % 16, K group l / 16; the accumulator's lane l holds rows
// 4 * (l / 16) + 0..3 of column l % 16.
// i8_reduce adds the slices of a split K (32-bit integers) and applies the
// scales.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <new>

#include "../../include/tp1_proj.h"
#include "args.hpp"
#include "device.hpp"
#include "plan.hpp"

namespace tp1 {

namespace {

// X(bcap, rows, waves, kw, kc, depth, nw): batch capacity, 16-row weight
// tiles a group, waves along the batch, waves along K, K bytes a step, LDS
// stages, waves a workgroup.
#define TP1_I8_INSTANCES(X)                                                                \
    X(16, 4, 1, 1, 512, 2, 4) X(16, 1, 1, 8, 512, 8, 8) X(16, 1, 1, 8, 512, 4, 8)          \
    X(32, 8, 2, 1, 256, 3, 8) X(32, 4, 1, 2, 512, 3, 8) X(64, 16, 2, 1, 128, 3, 8)         \
    X(64, 4, 4, 1, 256, 4, 8) X(128, 16, 2, 1, 128, 3, 8) X(128, 8, 2, 1, 128, 4, 8)       \
    X(128, 4, 4, 1, 128, 5, 8) X(256, 16, 4, 1, 64, 4, 8) X(256, 8, 4, 1, 128, 3, 8)       \
    X(256, 4, 4, 1, 128, 4, 8)

struct I8Args {
    const int8_t *x;
    long ldx;
    const float *xs;
    const int8_t *w;
    const float *ws;
    uint16_t *y;
    int *part;  // [S][B][N] integer sums when S > 1
    int N, K, B;
    int ks;     // K bytes a slice (a multiple of the step)
    int S;
    int stagger;
};

__device__ __align__(16) uint32_t kZeros[4];

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes a lane from src into LDS at base + 16 * lane (base uniform).  M0
// needs one wait state between its write and the load that reads it.
template <bool STREAM>
__device__ __forceinline__ void lds_load16(const void *src, uint32_t base) {
    if constexpr (STREAM)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt"
                     :
                     : "v"(src), "s"(base)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                     :
                     : "v"(src), "s"(base)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ float scaled(int acc, float xs, float ws) {
    return (float)acc * (xs * ws);
}

template <int MT, int NTB, int WM, int WK, int KB, int D, int NW>
__global__ __launch_bounds__(NW * 64) void i8_pipe_kernel(I8Args a) {
    constexpr int WN = NW / (WM * WK);        // waves along the weight rows
    constexpr int MTW = MT / WM;              // x tiles a wave
    constexpr int NTW = NTB / WN;             // weight tiles a wave
    constexpr int JW = KB / 64 / WK;          // 64-byte K steps a wave and stage
    constexpr int XR = 16 * MT;               // x rows a stage
    constexpr int GR = 16 * NTB;              // weight rows a group
    constexpr int PP = KB / 16;               // pieces a row
    constexpr int STAGE = (XR + GR) * KB;     // bytes a stage
    constexpr int NB = STAGE / 1024;          // load instructions a stage
    constexpr int XB = XR * KB / 1024;        // of which for x
    constexpr int NI = NB / NW;               // a wave
    static_assert(WM * WK * WN == NW && MTW * WM == MT && NTW * WN == NTB, "wave split");
    static_assert(JW * WK * 64 == KB, "K steps split over the waves along K");
    static_assert(PP >= 4 && (PP & (PP - 1)) == 0 && PP <= 64, "pieces a row");
    static_assert(NB % NW == 0 && (XR * KB) % 1024 == 0, "loads split over the waves");
    static_assert(D >= 2 && NI * (D - 2) <= 63, "loads in flight");
    extern __shared__ __align__(16) char stages[];
    const uint32_t lds0 = scalar((int)lds_offset(stages));

    const int lane = threadIdx.x & 63;
    const int wave = scalar(threadIdx.x >> 6);
    const int wk = wave / (WM * WN);
    const int wmn = wave - wk * (WM * WN);
    const int wm = wmn / WN, wn = wmn % WN;
    const int s = blockIdx.y;
    const int k0 = s * a.ks;
    const int klen = min(a.K - k0, a.ks);
    const int row0 = (int)((long)a.N * blockIdx.x / gridDim.x);
    const int rows = (int)((long)a.N * (blockIdx.x + 1) / gridDim.x) - row0;
    const int C = (klen + KB - 1) / KB;
    const int T = (rows + GR - 1) / GR * C;
    if (T == 0) return;  // uniform over the workgroup
    const int lrow = lane & 15, lgrp = lane >> 4;
    auto swz = [](int r) { return PP == 4 ? (r >> 1) & 3 : r & (PP - 1); };

    // this lane's piece of each of the wave's loads: stage row and K byte
    int lr[NI], lk[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int pos = (i * NW + wave) * 64 + lane;
        lr[i] = pos / PP;
        lk[i] = ((pos % PP) ^ swz(lr[i])) * 16;
    }
    const int c0 = a.stagger ? (int)(blockIdx.x % (unsigned)C) : 0;
    int it = 0, ig = 0, ic = 0;  // the next step to load
    auto issue = [&]() {
        const uint32_t st = lds0 + (uint32_t)((it % D) * STAGE);
        const int cc = ic + c0 < C ? ic + c0 : ic + c0 - C;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int bi = i * NW + wave;
            const int k = cc * KB + lk[i];
            // rows past the batch or the range repeat a live one: they feed
            // outputs that are not stored; only bytes past the slice's end,
            // which meet live rows, have to be zero
            if (bi < XB) {
                const int b = min(lr[i], a.B - 1);
                const void *src = k < klen ? (const void *)(a.x + (size_t)b * a.ldx + k0 + k)
                                           : (const void *)kZeros;
                lds_load16<false>(src, st + (uint32_t)bi * 1024u);
            } else {
                const int r = min(ig * GR + lr[i] - XR, rows - 1);
                const void *src = k < klen
                                      ? (const void *)(a.w + (size_t)(row0 + r) * a.K + k0 + k)
                                      : (const void *)kZeros;
                lds_load16<true>(src, st + (uint32_t)bi * 1024u);
            }
        }
        ++it;
        if (++ic == C) {
            ic = 0;
            ++ig;
        }
    };

    i32x4 acc[MTW][NTW];
#pragma unroll
    for (int m = 0; m < MTW; ++m)
#pragma unroll
        for (int n = 0; n < NTW; ++n) acc[m][n] = i32x4{0, 0, 0, 0};

#pragma unroll
    for (int p = 0; p < D - 1; ++p) issue();
    int g = 0, c = 0;
    for (int t = 0; t < T; ++t) {
        wait_loads<NI * (D - 2)>();  // this wave's pieces of step t have landed
        __syncthreads();             // everyone's have, and stage t - 1 is free
        issue();                     // step t + D - 1 into it
        const char *stg = stages + (t % D) * STAGE;
#pragma unroll
        for (int jj = 0; jj < JW; ++jj) {
            const int p = (jj * WK + wk) * 4 + lgrp;
            i32x4 wf[NTW];
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
                const int r = XR + (wn * NTW + n) * 16 + lrow;
                wf[n] = *reinterpret_cast<const i32x4 *>(stg + (r * PP + (p ^ swz(r))) * 16);
            }
#pragma unroll
            for (int m = 0; m < MTW; ++m) {
                const int r = (wm * MTW + m) * 16 + lrow;
                const i32x4 xf =
                    *reinterpret_cast<const i32x4 *>(stg + (r * PP + (p ^ swz(r))) * 16);
#pragma unroll
                for (int n = 0; n < NTW; ++n)
                    acc[m][n] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(xf, wf[n], acc[m][n], 0, 0, 0);
            }
        }
        if (c == C - 1) {
            if constexpr (WK > 1) {
                // the waves along K meet in LDS behind the ring
                i32x4 *part = reinterpret_cast<i32x4 *>(stages + D * STAGE);
                constexpr int TILES = MTW * NTW;
                if (wk > 0) {
#pragma unroll
                    for (int q = 0; q < TILES; ++q)
                        part[(((wk - 1) * WM * WN + wmn) * TILES + q) * 64 + lane] =
                            acc[q / NTW][q % NTW];
                }
                __syncthreads();
                if (wk == 0) {
#pragma unroll
                    for (int v = 1; v < WK; ++v)
#pragma unroll
                        for (int q = 0; q < TILES; ++q)
                            acc[q / NTW][q % NTW] +=
                                part[(((v - 1) * WM * WN + wmn) * TILES + q) * 64 + lane];
                }
            }
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
                const int r = g * GR + (wn * NTW + n) * 16 + lrow;
                const bool mine = wk == 0 && r < rows;
                const float ws = mine && a.S == 1 ? a.ws[row0 + r] : 0.f;
#pragma unroll
                for (int m = 0; m < MTW; ++m) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int b = (wm * MTW + m) * 16 + lgrp * 4 + v;
                        if (!mine || b >= a.B) continue;
                        if (a.S == 1)
                            a.y[(size_t)b * a.N + row0 + r] =
                                round_bf16(scaled(acc[m][n][v], a.xs[b], ws));
                        else
                            a.part[((size_t)s * a.B + b) * a.N + row0 + r] = acc[m][n][v];
                    }
                    acc[m][n] = i32x4{0, 0, 0, 0};
                }
            }
        }
        if (++c == C) {
            c = 0;
            ++g;
        }
    }
    wait_loads<0>();  // no wave leaves LDS writes in flight
}

// y = bf16( (sum over the S slices) * (xs * ws) ), V outputs a thread (V = 4
// where N allows it: one 16-byte load a slice, one 8-byte store).  Eight
// slices' loads are issued before any is added.
template <int V>
__global__ __launch_bounds__(256) void i8_reduce(const int *part, const float *xs, const float *ws,
                                                 uint16_t *y, int N, int B, int S) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * V;
    const int b = blockIdx.y;
    if (n >= N) return;
    const size_t slice = (size_t)B * N;
    const int *p = part + (size_t)b * N + n;
    int acc[V] = {};
    for (int s0 = 0; s0 < S; s0 += 8) {
        int v[8][V];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s0 + s >= S) continue;  // uniform
            if constexpr (V == 4)
                *reinterpret_cast<i32x4 *>(v[s]) = __builtin_nontemporal_load(
                    reinterpret_cast<const i32x4 *>(p + (s0 + s) * slice));
            else
                v[s][0] = p[(s0 + s) * slice];
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s0 + s < S)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += v[s][i];
    }
    uint16_t *to = y + (size_t)b * N + n;
    if constexpr (V == 4) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(ws + n);
        unsigned o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = round_bf16(scaled(acc[i], xs[b], w[i]));
        *reinterpret_cast<u32x2 *>(to) = u32x2{o[0] | o[1] << 16, o[2] | o[3] << 16};
    } else {
        *to = round_bf16(scaled(acc[0], xs[b], ws[n]));
    }
}

// ---------------------------------------------------------------- host side

int slice_bytes(int K, const proj_tactic_t &t) {
    const int per = (K + t.split - 1) / t.split;
    return (per + t.kc - 1) / t.kc * t.kc;
}
int slices(int K, const proj_tactic_t &t) {
    const int ks = slice_bytes(K, t);
    return (K + ks - 1) / ks;
}

size_t i8_lds_bytes(const proj_tactic_t &t) {
    const size_t ring = (size_t)t.depth * (t.bcap + 16 * t.rows) * t.kc;
    return ring + (size_t)(t.kw - 1) * (t.bcap / 16) * t.rows * 1024u;
}

size_t i8_workspace(int N, int K, const proj_tactic_t &t) {
    const int S = slices(K, t);
    return S > 1 ? (size_t)S * t.bcap * N * sizeof(int) : 0;
}

bool i8_instance_exists(const proj_tactic_t &t) {
#define TP1_I8_MATCH(BC, NTB, WM, WK, KB, D, NW)                                         \
    if (t.bcap == BC && t.rows == NTB && t.waves == WM && t.kw == WK && t.kc == KB &&    \
        t.depth == D && t.nw == NW)                                                      \
        return true;
    TP1_I8_INSTANCES(TP1_I8_MATCH)
#undef TP1_I8_MATCH
    return false;
}

int check_i8_tactic(int bin, const proj_tactic_t &t, size_t lds) {
    if (t.kernel != PROJ_KERNEL_I8_PIPE || !i8_instance_exists(t)) return PROJ_EINVAL;
    if (t.bcap < bin || t.split < 1 || t.split > 64 || t.wpc < 1 || t.wpc > 4) return PROJ_EINVAL;
    if (t.stagger != 0 && t.stagger != 1) return PROJ_EINVAL;
    return i8_lds_bytes(t) <= lds ? PROJ_OK : PROJ_EINVAL;
}

// The rule follows what was measured at the shapes of a layer and of its
// shards (us; the read of the weight alone takes 18.3 at 104 MB, 55 at 354 MB
// and 7 at 13 MB on the same card), by r, the weight rows a compute unit has
// of an even share:
//   r >= 100 (49376 x 7168, r = 193): the widest weight tiles, K whole.
//     B = 16: 58.2, 32: 60.6, 64: 59.5 (8-row-tile groups 72), 128: 80.2
//     (91 staggered), 256: 143.9 (156 and more with other tiles).
//   r >= 20 (14560 x 7168, r = 57; 7168 x 12288, r = 28): K split so that a
//     row range fills a group.  14560: B = 16: 21.4 (32.9 with K whole and 32-row
//     groups), 64: 23.9, 128: 34.8, 256: 56.1.  7168: 19.6, 23.6, 31.3, 45.0
//     (69 at half the split).
//   below (3640 and 1820 x 7168): 16-row groups whose waves split K, or 64-row
//     groups and more slices.  1820: B = 1: 8.6 (8.9 with two slices, whose sum is a
//     second launch), 32: 9.8, 128: 15.5 (22.5 with the tiles of large r);
//     3640: B = 16: 9.4 (12.7 with two slices), 200: 25.4 (28.5).  896 x 12288,
//     B = 1: 9.1 with four slices, 11.6 with one.
// Two workgroups of four waves a compute unit carry the narrow batches: 58.2
// against 64.3 for one of eight at 49376 x 7168.  A row pitch that is a
// multiple of 4 KB takes staggered chunks (7168 x 12288, B = 16: 19.6 against
// 19.8); others measured the same or worse with them.
proj_tactic_t i8_rule(int N, int K, int bin, int cus) {
    proj_tactic_t t{};
    t.kernel = PROJ_KERNEL_I8_PIPE;
    const double r = std::max(1.0, (double)N / cus);
    const bool wide = r >= 100, few = r < 20;
    auto tile = [&](int bcap, int rows, int waves, int kw, int kc, int depth, int nw, int fill) {
        t.bcap = bcap;
        t.rows = rows;
        t.waves = waves;
        t.kw = kw;
        t.kc = kc;
        t.depth = depth;
        t.nw = nw;
        t.wpc = nw == 4 ? 2 : 1;
        t.split = std::max(1, std::min(8, (int)(fill / r)));
        while (t.split > 1 && K / t.split < 2 * kc) --t.split;
    };
    if (bin <= 16) {
        if (few)
            tile(16, 1, 1, 8, 512, K <= 2048 ? 4 : 8, 8, 14);
        else
            tile(16, 4, 1, 1, 512, 2, 4, 128);
    } else if (bin <= 32) {
        if (few)
            tile(32, 4, 1, 2, 512, 3, 8, 64);
        else
            tile(32, 8, 2, 1, 256, 3, 8, 128);
    } else if (bin <= 64) {
        if (wide)
            tile(64, 16, 2, 1, 128, 3, 8, 64);
        else
            tile(64, 4, 4, 1, 256, 4, 8, 64);
    } else if (bin <= 128) {
        if (wide)
            tile(128, 16, 2, 1, 128, 3, 8, 64);
        else if (few)
            tile(128, 4, 4, 1, 128, 5, 8, 64);
        else
            tile(128, 8, 2, 1, 128, 4, 8, 128);
    } else {
        if (wide)
            tile(256, 16, 4, 1, 64, 4, 8, 64);
        else if (few)
            tile(256, 4, 4, 1, 128, 4, 8, 64);
        else
            tile(256, 8, 4, 1, 128, 3, 8, 128);
    }
    t.stagger = K % 4096 == 0;
    return t;
}

}  // namespace
}  // namespace tp1

struct proj_i8_plan_s {
    int N = 0, K = 0, nb = 0, device = -1, cus = 256;
    unsigned flags = 0;
    int batches[PROJ_MAX_BATCHES] = {};
    proj_tactic_t tactics[PROJ_MAX_BATCHES] = {};
    size_t lds = tp1::kLdsBytes;
    int *part = nullptr;
    size_t part_bytes = 0;
};

namespace tp1 {
namespace {

template <typename F>
hipError_t allow_lds(F *fn, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(fn),
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Every instance may use the LDS its ring needs; set once a device, so no
// launch (which may be captured) changes an attribute.
int prepare_i8(int dev, size_t lds) {
    static std::mutex mu;
    static bool done[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev]) return PROJ_OK;
    hipError_t e = hipSuccess;
#define TP1_I8_ALLOW(BC, NTB, WM, WK, KB, D, NW) \
    if (e == hipSuccess) e = allow_lds(&i8_pipe_kernel<BC / 16, NTB, WM, WK, KB, D, NW>, lds);
    TP1_I8_INSTANCES(TP1_I8_ALLOW)
#undef TP1_I8_ALLOW
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    if (dev >= 0 && dev < 64) done[dev] = true;
    return PROJ_OK;
}

int i8_alloc(proj_i8_plan_s *p, size_t bytes) {
    if (bytes <= p->part_bytes) return PROJ_OK;
    if (p->flags & PROJ_PLAN_HOST_ONLY) {
        p->part_bytes = bytes;
        return PROJ_OK;
    }
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != p->device) return PROJ_EINVAL;
    if (p->part && hipFree(p->part) != hipSuccess) return PROJ_EHIP;
    p->part = nullptr;
    p->part_bytes = 0;
    void *mem = nullptr;
    if (hipMalloc(&mem, bytes) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_ENOMEM;
    }
    p->part = static_cast<int *>(mem);
    p->part_bytes = bytes;
    return PROJ_OK;
}

int i8_bin(const proj_i8_plan_s &p, int B) {
    if (B < 1) return -1;
    for (int i = 0; i < p.nb; ++i)
        if (B <= p.batches[i]) return i;
    return -1;
}

hipError_t launch_i8(const I8Args &a, const proj_tactic_t &t, int cus, hipStream_t st) {
    const long g = std::max(1L, std::min((long)a.N, (long)cus * t.wpc / a.S));
    const size_t lds = i8_lds_bytes(t);
#define TP1_I8_CASE(BC, NTB, WM, WK, KB, D, NW)                                              \
    if (t.bcap == BC && t.rows == NTB && t.waves == WM && t.kw == WK && t.kc == KB &&        \
        t.depth == D && t.nw == NW) {                                                        \
        hipLaunchKernelGGL((i8_pipe_kernel<BC / 16, NTB, WM, WK, KB, D, NW>),                \
                           dim3((unsigned)g, a.S), dim3(NW * 64), lds, st, a);               \
        return hipGetLastError();                                                            \
    }
    TP1_I8_INSTANCES(TP1_I8_CASE)
#undef TP1_I8_CASE
    return hipErrorInvalidValue;
}

}  // namespace
}  // namespace tp1

extern "C" {

int proj_i8_plan(int N, int K, const int *batches, int n_batches, unsigned flags,
                 proj_i8_plan_t **out) {
    if (!out) return PROJ_EINVAL;
    *out = nullptr;
    if (flags & ~PROJ_PLAN_HOST_ONLY) return PROJ_EINVAL;
    if (K % 16 != 0 || K > PROJ_I8_MAX_K) return PROJ_EINVAL;
    int rc = tp1::check_plan_args(N, K, batches, n_batches, flags);
    if (rc != PROJ_OK) return rc;
    proj_i8_plan_s *p = new (std::nothrow) proj_i8_plan_s;
    if (!p) return PROJ_ENOMEM;
    p->N = N;
    p->K = K;
    p->nb = n_batches;
    p->flags = flags;
    if (!(flags & PROJ_PLAN_HOST_ONLY)) {
        int dev = -1, cus = 0, lds = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) !=
                hipSuccess ||
            hipDeviceGetAttribute(&lds, hipDeviceAttributeMaxSharedMemoryPerBlock, dev) !=
                hipSuccess) {
            (void)hipGetLastError();
            delete p;
            return PROJ_EHIP;
        }
        p->device = dev;
        if (cus > 0) p->cus = cus;
        if (lds > 0 && (size_t)lds < p->lds) p->lds = (size_t)lds;
        rc = tp1::prepare_i8(dev, p->lds);
    }
    size_t ws = 0;
    for (int i = 0; i < n_batches && rc == PROJ_OK; ++i) {
        p->batches[i] = batches[i];
        p->tactics[i] = tp1::i8_rule(N, K, batches[i], p->cus);
        rc = tp1::check_i8_tactic(batches[i], p->tactics[i], p->lds);
        ws = std::max(ws, tp1::i8_workspace(N, K, p->tactics[i]));
    }
    if (rc == PROJ_OK) rc = tp1::i8_alloc(p, ws);
    if (rc != PROJ_OK) {
        delete p;
        return rc;
    }
    *out = p;
    return PROJ_OK;
}

void proj_i8_free(proj_i8_plan_t *p) {
    if (!p) return;
    if (p->part) {
        int cur = -1;
        const bool other = hipGetDevice(&cur) == hipSuccess && cur != p->device;
        if (other) (void)hipSetDevice(p->device);
        (void)hipFree(p->part);
        if (other) (void)hipSetDevice(cur);
    }
    delete p;
}

int proj_i8_plan_tactic(const proj_i8_plan_t *p, int B, proj_tactic_t *tactic, int *bin) {
    if (!p || !tactic) return PROJ_EINVAL;
    const int i = tp1::i8_bin(*p, B);
    if (i < 0) return PROJ_EBATCH;
    *tactic = p->tactics[i];
    if (bin) *bin = p->batches[i];
    return PROJ_OK;
}

int proj_i8_plan_set_tactic(proj_i8_plan_t *p, int bin, const proj_tactic_t *tactic) {
    if (!p || !tactic) return PROJ_EINVAL;
    for (int i = 0; i < p->nb; ++i) {
        if (p->batches[i] != bin) continue;
        if (tp1::check_i8_tactic(bin, *tactic, p->lds) != PROJ_OK) return PROJ_EINVAL;
        const int rc = tp1::i8_alloc(p, tp1::i8_workspace(p->N, p->K, *tactic));
        if (rc == PROJ_OK) p->tactics[i] = *tactic;
        return rc;
    }
    return PROJ_EINVAL;
}

size_t proj_i8_plan_workspace_bytes(const proj_i8_plan_t *p) { return p ? p->part_bytes : 0; }

int proj_i8_run(const proj_i8_plan_t *p, int B, const void *x, long ldx, const void *x_scale,
                const void *W, const void *w_scale, void *y, void *stream) {
    using namespace tp1;
    if (!p) return PROJ_EINVAL;
    if (B < 0 || B > p->batches[p->nb - 1]) return PROJ_EBATCH;
    if (ldx == 0) ldx = p->K;
    if (ldx < p->K) return PROJ_EINVAL;
    if (B == 0) return PROJ_OK;
    if (!x || !x_scale || !W || !w_scale || !y) return PROJ_EINVAL;
    if (!is_aligned(x, 16) || !is_aligned(W, 16) || ldx % 16 != 0 || !is_aligned(y, 16) ||
        !is_aligned(x_scale, 4) || !is_aligned(w_scale, 4))
        return PROJ_EALIGN;
    const Span out(y, (size_t)B * p->N * 2);
    if (out.meets(Span(x, span_bytes(B, p->K, ldx))) || out.meets(Span(W, (size_t)p->N * p->K)) ||
        out.meets(Span(x_scale, (size_t)B * 4)) || out.meets(Span(w_scale, (size_t)p->N * 4)))
        return PROJ_EINVAL;
    if (p->flags & PROJ_PLAN_HOST_ONLY) return PROJ_ENODEV;
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != p->device) return PROJ_EINVAL;
    const int i = i8_bin(*p, B);
    if (i < 0) return PROJ_EBATCH;
    const proj_tactic_t &t = p->tactics[i];
    const int S = slices(p->K, t);
    if (S > 1 && (size_t)S * B * p->N * sizeof(int) > p->part_bytes) return PROJ_EINVAL;
    const I8Args a{static_cast<const int8_t *>(x), ldx, static_cast<const float *>(x_scale),
                   static_cast<const int8_t *>(W), static_cast<const float *>(w_scale),
                   static_cast<uint16_t *>(y), p->part, p->N, p->K, B, slice_bytes(p->K, t), S,
                   t.stagger};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = launch_i8(a, t, p->cus, st);
    if (e == hipSuccess && S > 1) {
        // four outputs a thread where rows of N stay 16-byte aligned
        if (p->N % 4 == 0 && is_aligned(w_scale, 16))
            hipLaunchKernelGGL(i8_reduce<4>, dim3((p->N + 1023) / 1024, B), dim3(256), 0, st,
                               a.part, a.xs, a.ws, a.y, a.N, a.B, S);
        else
            hipLaunchKernelGGL(i8_reduce<1>, dim3((p->N + 255) / 256, B), dim3(256), 0, st, a.part,
                               a.xs, a.ws, a.y, a.N, a.B, S);
        e = hipGetLastError();
    }
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}

}  // extern "C"
