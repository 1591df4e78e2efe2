// delta_chunk.hip -- the gated delta rule over sequences, 64 tokens at a time.
//
// Write G_i for the sum of the log decays of a chunk's tokens up to and with
// token i (a vector over the 128 key channels), S for the state before the
// chunk, and u_i for what token i adds (S <- S + k_i u_i^T).  Unrolling the
// recurrence inside the chunk,
//     u_i = beta_i (v_i - S^T (k_i e^{G_i}) - sum_{j<i} A_ij u_j),
//     A_ij = sum_c k_ic k_jc e^{G_ic - G_jc},
//     o_i = S^T (q_i e^{G_i}) + sum_{j<=i} P_ij u_j,   P_ij as A with q_i,
//     S'  = diag(e^{G_64}) S + sum_j (k_j e^{G_64 - G_j}) u_j^T.
// With N = diag(beta) A (strictly lower triangular) and T = (1 + N)^-1
// diag(beta), the u_i are U = T R, R = V - (K e^G) S.  Only R depends on the
// chunks before, so the work is in two parts:
//   prepare (one workgroup a chunk and head): K e^G, Q e^G, M = (K e^{G_64 -
//     G})^T T, P T and e^{G_64}, and V in operand order, to a workspace;
//   scan (workgroups of four waves, 16, 32 or 64 columns of a head's state each):
//     chunk after chunk R = V - (K e^G) S, O = (Q e^G) S + (P T) R,
//     S' = diag(e^{G_64}) S + M R.
//
// Numbers.  All products run on the 16-bit matrix cores with FP32 sums, and
// what reaches the state is as exact as FP32 operands would make it.  Keys
// and queries have unit length here (the chunked form is taken with l2norm
// only), so every update is a contraction, and T, M, K e^.. and Q e^.. stay
// within 1: they are held as two FP16 values hi + lo of 2^10 times the value,
// and hi hi + hi lo + lo hi summed, which drops 2^-23 of each (two BF16
// values would drop 2^-17, one 2^-9).  S and R have any range: they are
// scaled by a power of two under which a bound of their largest magnitude is
// 2^14.  What only reaches the BF16 output (Q, P T, and the hi parts of S and
// R against them) is one FP16 value each, 2^-12.
// Decays are products of factors e^x with x <= 0, the sums x taken inside
// blocks of 16 tokens from the token outward, so none is a difference of
// large numbers: with block a after block b, e^{G_i - G_j} = (e^{sum of a's
// tokens up to i}) (e^{whole blocks between}) (e^{sum of b's tokens after
// j}).  Inside a block the second factor is e^{-(sum up to j)} instead,
// which grows, so those products are FP32 ones (v_mfma_f32_16x16x4), and a
// block whose tokens decay a channel by more than 2^-112 takes an exact path
// on the vector unit (a running sum from i down to j).  A sum of up to 112 is
// off by 2^-18, and so is its factor, but only in a channel that a token of
// this block all but clears; the 128 channels' errors are independent.
//
// Layout.  A wave of `prepare` owns one block of 16 tokens; lane l holds
// token l % 16 and, for s = 0..3, channels 32 s + 8 (l / 16) + 0..7, which is
// the A and B operand of v_mfma_f32_16x16x32 over channels.  Sums over
// the tokens of a block are scans over 16 lanes (DPP).  Operands over tokens
// need the transpose, which a product with a selection matrix gives exactly
// (accumulator lane l holds rows 4 (l / 16) + 0..3 of column l % 16).  The
// order of the 32 summed values of a product is free, so accumulators are fed
// back as operands without any exchange of lanes: S tile 2 s + h has channel
// 32 s + 8 (r / 4) + 4 h + r % 4 as row r, and a step over tokens takes blocks
// 2 t and 2 t + 1, tokens 4 (l / 16) + 0..3 of each.  The workspace holds
// every operand in that order, 16 bytes a lane, 1 KB in one piece.
#include "delta.hpp"

#include "device.hpp"

namespace tp1 {

namespace {

constexpr int kC = kDeltaChunk;   // tokens a chunk

// Workspace of a chunk and head: what wave w of the scan takes, together.
//   token tile w:        -K e^G [4 s][hi, lo], Q e^G [4 s], V [8 value tiles] (8 bytes a lane),
//                        P T [2 steps]
//   channel tiles 2 w + h: M [2 h][2 steps][hi, lo]
// then e^{G_64} [128] and the largest |v| of each token tile [4].
constexpr int kWsWave = 26624;
constexpr int ws_k(int s) { return s * 2048; }
constexpr int ws_q(int s) { return 8192 + s * 1024; }
constexpr int ws_v(int vt) { return 12288 + vt * 512; }
constexpr int ws_p(int step) { return 16384 + step * 1024; }
constexpr int ws_m(int h, int step) { return 18432 + (h * 2 + step) * 2048; }
constexpr int kWsD = 4 * kWsWave;
constexpr int kWsTop = kWsD + 512;
static_assert(kWsTop + 512 == kDeltaItemBytes, "workspace of an item");

// LDS of `prepare`, in bytes.
constexpr int kLdsKr = 0;                     // [48 rows][hi, lo][128] FP16
constexpr int kLdsK = kLdsKr + 48 * 512;      // [8 channel tiles][2 steps][hi, lo][64][16]
constexpr int kLdsN = kLdsK + 32768;          // [10 blocks][16 rows][20] FP32
constexpr int kLdsP = kLdsN + 10 * 1280;      // [10 blocks][64][8]
constexpr int kLdsTot = kLdsP + 10 * 512;     // [4][128] FP32: a block's whole decay
constexpr int kLdsBeta = kLdsTot + 2048;      // [64] FP32
static_assert(kLdsBeta + 256 <= kDeltaLds, "LDS of prepare");
// LDS of `scan` with CT column tiles.
constexpr int lds_s(int ct, int s, int v) { return (s * ct + v) * 2048; }
constexpr int lds_r(int ct, int st, int v) { return ct * 8192 + (st * ct + v) * 2048; }
constexpr int lds_tops(int ct) { return ct * 12288; }  // of S [4], of R [4]
static_assert(lds_tops(4) + 32 <= kDeltaLds, "LDS of scan");

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma_bf(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_h(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// A block is mild if no channel decays by more than 2^-kMild over it: then
// 2^10 / (that decay) is still below FP32's largest value by 2^6.  At 2^-58,
// where ordinary gates (rates of 1 to 16) leave one block in three to the
// exact path, 8192 tokens of 96 heads take 1235 us, at 2^-112 974 us.
constexpr float kMild = 112.f;

// What unit-bounded values are multiplied by before they become FP16 pairs.
constexpr float kUnit = 1024.f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// log2 of a token's decay: -rate * ln(1 + e^z), z = f + dt_bias, where rate is
// exp(A_log) log2 e.  ln(1 + e^z) = max(z, 0) + 2 atanh(s) with s = e / (2 +
// e), e = e^-|z|; the series in s^2 <= 1/9 stops below 2^-25 of the value.
// (The rounding of e's exponent is an error relative to the gate itself,
// which weighs nothing where e is far from 1.)  Sums of gates stay in base
// 2, where e^x costs one instruction; infinite ones end as factors 0.
__device__ __forceinline__ float gate_of(float rate, float f, float bias) {
    const float z = f + bias;
    const float e = exp2_of(-1.442695041f * fabsf(z));
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), t = s * s;
    float p = 2.f / 13.f;
    p = __builtin_fmaf(p, t, 2.f / 11.f);
    p = __builtin_fmaf(p, t, 2.f / 9.f);
    p = __builtin_fmaf(p, t, 2.f / 7.f);
    p = __builtin_fmaf(p, t, 2.f / 5.f);
    p = __builtin_fmaf(p, t, 2.f / 3.f);
    p = __builtin_fmaf(p, t, 2.f);
    return -rate * __builtin_fmaf(s, p, fmaxf(z, 0.f));
}

__device__ __forceinline__ unsigned pack_h(float a, float b) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, f16x2_t{(_Float16)a, (_Float16)b});
}
__device__ __forceinline__ float h_lo(unsigned u) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}
__device__ __forceinline__ float h_hi(unsigned u) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(u >> 16));
}

// The bits v as they are: without this the compiler may round a product to
// FP16 twice, once fused with the product and once after its FP32 rounding,
// and store one hi but subtract the other, a whole step apart.
__device__ __forceinline__ unsigned settled(unsigned v) {
    asm("" : "+v"(v));
    return v;
}

__device__ __forceinline__ float settled(float v) {
    asm("" : "+v"(v));
    return v;
}

struct Split {
    u32x4 hi, lo;
};
// Eight values as FP16 pairs hi + lo; and one FP16 value each.
__device__ __forceinline__ Split split_h(const float *x) {
    Split o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned h = settled(pack_h(x[2 * i], x[2 * i + 1]));
        o.hi[i] = h;
        o.lo[i] = pack_h(x[2 * i] - h_lo(h), x[2 * i + 1] - h_hi(h));
    }
    return o;
}
__device__ __forceinline__ u32x4 round_h(const float *x) {
    return u32x4{pack_h(x[0], x[1]), pack_h(x[2], x[3]), pack_h(x[4], x[5]), pack_h(x[6], x[7])};
}
__device__ __forceinline__ Split split_h(f32x4 a, f32x4 b, float by) {
    const float x[8] = {a.x * by, a.y * by, a.z * by, a.w * by,
                        b.x * by, b.y * by, b.z * by, b.w * by};
    return split_h(x);
}
__device__ __forceinline__ u32x2 pack4_h(f32x4 a) {
    return u32x2{pack_h(a.x, a.y), pack_h(a.z, a.w)};
}

__device__ __forceinline__ void unpack8(u32x4 v, float *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
}

// A power of two that brings values of largest magnitude `top` (bits) to
// 2^14..2^15, and its inverse.  Zeros, subnormals, infinities and NaN are
// left as they are.
struct Scale {
    float up, down;
};
__device__ __forceinline__ Scale scale_for(unsigned top) {
    const int e = (int)(top >> 23);  // biased exponent
    int x = e == 0 || e == 255 ? 0 : 127 + 14 - e;
    x = x > 120 ? 120 : x < -113 ? -113 : x;
    return Scale{__uint_as_float((unsigned)(127 + x) << 23),
                 __uint_as_float((unsigned)(127 - x) << 23)};
}
__device__ __forceinline__ unsigned top_of(f32x4 v, unsigned top) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const unsigned m = __float_as_uint(v[r]) & 0x7FFFFFFFu;
        top = m > top ? m : top;
    }
    return top;
}

// Place of block (a, b), b <= a, among the lower triangle's ten.
__device__ __forceinline__ int block_of(int a, int b) { return a * (a + 1) / 2 + b; }

// Orders this wave's LDS writes before its later reads by other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sums over the lanes of a 16-lane row: up to and with this one, and after it.
__device__ __forceinline__ float sum_upto(float v) {
    v += dpp_move<0x111>(v);
    v += dpp_move<0x112>(v);
    v += dpp_move<0x114>(v);
    v += dpp_move<0x118>(v);
    return v;
}
__device__ __forceinline__ float sum_after(float v) {
    v += dpp_move<0x101>(v);
    v += dpp_move<0x102>(v);
    v += dpp_move<0x104>(v);
    v += dpp_move<0x108>(v);
    return dpp_move<0x101>(v);
}

// ---------------------------------------------------------------------------
// prepare: one workgroup of four waves a chunk and head, two a compute unit
// (by registers and LDS).  4128 chunks and heads take 209 us: 3460 vector
// instructions a wave fill half of the issue slots (a third of them are the
// gates), and 0.77 GB
// of inputs and operands move at 3.7 TB/s; the rest are the chains inside a
// chunk, which two waves a SIMD do not cover.
// ---------------------------------------------------------------------------
template <bool HEAD_GATE>
__device__ __forceinline__ void prepare_item(const DeltaArgs &a, int row0, int n, int h, char *ws,
                                             char *lds) {
    const int lane = threadIdx.x & 63;
    const int w = scalar(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int hk = h / a.rep;
    const bool live = w * 16 + lr < n;
    const long row = row0 + w * 16 + lr;
    float *tot = reinterpret_cast<float *>(lds + kLdsTot);
    float *betas = reinterpret_cast<float *>(lds + kLdsBeta);
    float *Nb = reinterpret_cast<float *>(lds + kLdsN);

    // ---- this lane's token: keys, queries, values, gates
    const u32x4 zero = {0u, 0u, 0u, 0u};
    char *wsw = ws + w * kWsWave;
    u32x4 kv[4], qv[4], fv[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + 8 * lg;
        kv[s] = qv[s] = fv[s] = zero;
        if (live) {
            kv[s] = *reinterpret_cast<const u32x4 *>(a.k + row * a.ldk + hk * kHead + c);
            qv[s] = *reinterpret_cast<const u32x4 *>(a.q + row * a.ldq + hk * kHead + c);
            if constexpr (!HEAD_GATE)
                fv[s] = *reinterpret_cast<const u32x4 *>(a.f + row * a.ldf + h * kHead + c);
        }
    }
    float rk, rq;  // to 2^10 times unit length
    {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k0 = bf16_lo(kv[s][i]), k1 = bf16_hi(kv[s][i]);
                const float q0 = bf16_lo(qv[s][i]), q1 = bf16_hi(qv[s][i]);
                sk = __builtin_fmaf(k0, k0, __builtin_fmaf(k1, k1, sk));
                sq = __builtin_fmaf(q0, q0, __builtin_fmaf(q1, q1, sq));
            }
        sk += __shfl_xor(sk, 16);
        sq += __shfl_xor(sq, 16);
        sk += __shfl_xor(sk, 32);
        sq += __shfl_xor(sq, 32);
        rk = rsqrtf(sk + kUnitEps) * kUnit;
        rq = rsqrtf(sq + kUnitEps) * kUnit;
    }
    const float rate = expf(a.a_log[h]) * 1.442695041f;
    if (lg == 0) betas[w * 16 + lr] = live ? sigmoid(bf16_value(a.b[row * a.ldb + h])) : 0.f;

    float el[4][8], er[4][8];  // decay of the block's tokens up to and with this one; after it
    float least = 0.f;
    auto gates = [&](int s, float *g) {  // log2 decays of channels 32 s + 8 lg + 0..7
        if constexpr (HEAD_GATE) {
            const float x = gate_of(rate, live ? bf16_value(a.f[row * a.ldf + h]) : 0.f,
                                    a.dt_bias[h]);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = live ? x : 0.f;
        } else {
            const f32x4 *bp =
                reinterpret_cast<const f32x4 *>(a.dt_bias + h * kHead + 32 * s + 8 * lg);
            const f32x4 b0 = bp[0], b1 = bp[1];
            unpack8(fv[s], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = settled(gate_of(rate, g[e], e < 4 ? b0[e & 3] : b1[e & 3]));
                g[e] = live ? x : 0.f;  // computed first: a branch a channel costs more
            }
        }
    };
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + 8 * lg;
        float g[8];
        if (!HEAD_GATE || s == 0) {
            gates(s, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (HEAD_GATE && e > 0) {
                    el[s][e] = el[s][0];
                    er[s][e] = er[s][0];
                    continue;
                }
                const float up = sum_upto(g[e]);
                least = fminf(least, up);
                el[s][e] = exp2_of(up);
                er[s][e] = exp2_of(sum_after(g[e]));
            }
            if (lr == 15) {
                f32x4 *t = reinterpret_cast<f32x4 *>(tot + w * kHead + c);
                t[0] = f32x4{el[s][0], el[s][1], el[s][2], el[s][3]};
                t[1] = f32x4{el[s][4], el[s][5], el[s][6], el[s][7]};
                if constexpr (HEAD_GATE) {
#pragma unroll
                    for (int o = 1; o < 4; ++o) t[8 * o] = t[8 * o + 1] = t[0];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                el[s][e] = el[0][0];
                er[s][e] = er[0][0];
            }
        }
        // keys scaled to the end of their block, for the blocks after
        if (w < 3) {
            float x[8];
            unpack8(kv[s], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= rk * er[s][e];
            const Split r = split_h(x);
            char *to = lds + kLdsKr + (w * 16 + lr) * 512 + (((4 * s + lg) ^ lr) * 16);
            *reinterpret_cast<u32x4 *>(to) = r.hi;
            *reinterpret_cast<u32x4 *>(to + 256) = r.lo;
        }
    }
    const bool mild = __all(least > -kMild);
    __syncthreads();  // 1: key rows, block totals and betas are there

    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    unsigned pick0 = 0, pick1 = 0;  // FP16 one for channel lr % 4 of four, in its lane group
    if (lg == lr >> 2) {
        const unsigned one = lr & 1 ? 0x3C000000u : 0x3C00u;
        pick0 = lr & 2 ? 0u : one;
        pick1 = lr & 2 ? one : 0u;
    }
    // A[i = 4 lg + r][j = lr] and P[j = 4 lg + r][i = lr] of blocks (w, b < w) and (w, w)
    f32x4 A[3], P[3], Ad = none, Pd = none;
#pragma unroll
    for (int b = 0; b < 3; ++b) A[b] = P[b] = none;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + 8 * lg;
        float kf[8], qf[8], x[8], y[8];
        unpack8(kv[s], kf);
        unpack8(qv[s], qf);
        // whole decays of the blocks before and behind this one
        f32x4 t[4][2], before[2], behind[2];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                t[b][i] = *reinterpret_cast<const f32x4 *>(tot + b * kHead + c + 4 * i);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            before[i] = behind[i] = f32x4{1.f, 1.f, 1.f, 1.f};
#pragma unroll
            for (int b = 0; b < 3; ++b)
                if (b < w) before[i] *= t[b][i];
#pragma unroll
            for (int b = 3; b > 0; --b)
                if (b > w) behind[i] *= t[b][i];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            kf[e] *= rk;
            x[e] = kf[e] * el[s][e];
            y[e] = qf[e] * rq * el[s][e];
        }
        // to the chunk's ends: K e^G and Q e^G to the workspace, K e^{G_64 - G} to LDS
        {
            float kt[8], kh[8], qt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kt[e] = -x[e] * before[e / 4][e % 4];
                qt[e] = y[e] * before[e / 4][e % 4];
                kh[e] = kf[e] * er[s][e] * behind[e / 4][e % 4];
            }
            *reinterpret_cast<u32x4 *>(wsw + ws_q(s) + lane * 16) = round_h(qt);
            if (w == 3 && lr == 15) {  // e^{G_64}: the decay of the whole chunk
                f32x4 *o = reinterpret_cast<f32x4 *>(ws + kWsD + c * 4);
                o[0] = f32x4{el[s][0], el[s][1], el[s][2], el[s][3]} * before[0];
                o[1] = f32x4{el[s][4], el[s][5], el[s][6], el[s][7]} * before[1];
            }
            const Split st = split_h(kt), sh = split_h(kh);
            *reinterpret_cast<u32x4 *>(wsw + ws_k(s) + lane * 16) = st.hi;
            *reinterpret_cast<u32x4 *>(wsw + ws_k(s) + 1024 + lane * 16) = st.lo;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                // column r of the selection picks channel 8 (r / 4) + 4 hf + r % 4
                const u32x4 sel =
                    hf ? u32x4{0u, 0u, pick0, pick1} : u32x4{pick0, pick1, 0u, 0u};
                char *to = lds + kLdsK + ((2 * s + hf) * 2 + (w >> 1)) * 2048 + lane * 16 +
                           (w & 1) * 8;
                *reinterpret_cast<u32x2 *>(to) = pack4_h(mfma_h(sh.hi, sel, none));
                *reinterpret_cast<u32x2 *>(to + 1024) = pack4_h(mfma_h(sh.lo, sel, none));
            }
        }
        // A and P, block row w: inside the block, then the blocks before
        if (mild) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // e^{-(sum up to j)}; el is at least 2^-112 here
                const float r = kf[e] * __builtin_amdgcn_rcpf(el[s][e]);
                Ad = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], r, Ad, 0, 0, 0);
                Pd = __builtin_amdgcn_mfma_f32_16x16x4f32(r, y[e], Pd, 0, 0, 0);
            }
        }
#pragma unroll
        for (int b = 2; b >= 0; --b) {
            if (b >= w) continue;  // uniform
            if (b < w - 1) {       // through block b + 1
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= t[b + 1][e / 4][e % 4];
                    y[e] *= t[b + 1][e / 4][e % 4];
                }
            }
            const Split l = split_h(x);
            const u32x4 q = round_h(y);
            const char *from = lds + kLdsKr + (b * 16 + lr) * 512 + (((4 * s + lg) ^ lr) * 16);
            const u32x4 rh = *reinterpret_cast<const u32x4 *>(from);
            const u32x4 rl = *reinterpret_cast<const u32x4 *>(from + 256);
            A[b] = mfma_h(l.hi, rl, A[b]);
            P[b] = mfma_h(rh, q, P[b]);
            A[b] = mfma_h(l.lo, rh, A[b]);
            A[b] = mfma_h(l.hi, rh, A[b]);
        }
    }
    if (!mild) {
        // Exact inside a block: for d = 0..15, token i with j = i - d, the
        // decay's exponent summed from i down.  Lane l holds i = l % 16.
        float pi[16], ai[16];  // row i of P and A, by distance
#pragma unroll
        for (int d = 0; d < 16; ++d) pi[d] = ai[d] = 0.f;
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
            float gs[8], ks[8], kf[8], qf[8], x[8];
            u32x4 kr = kv[0], qr = qv[0];
#pragma unroll
            for (int o = 1; o < 4; ++o) {
                kr = s == o ? kv[o] : kr;
                qr = s == o ? qv[o] : qr;
            }
            if constexpr (HEAD_GATE) {
                gates(0, gs);
            } else {
                u32x4 fr = fv[0];
#pragma unroll
                for (int o = 1; o < 4; ++o) fr = s == o ? fv[o] : fr;
                const float *bp = a.dt_bias + h * kHead + 32 * s + 8 * lg;
                unpack8(fr, gs);
#pragma unroll
                for (int e = 0; e < 8; ++e) gs[e] = live ? gate_of(rate, gs[e], bp[e]) : 0.f;
            }
            unpack8(kr, kf);
            unpack8(qr, qf);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kf[e] *= rk;
                qf[e] *= rq;
                ks[e] = kf[e];
                x[e] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < 16; ++d)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (d > 0) {
                        x[e] += gs[e];  // of token i - d + 1
                        gs[e] = dpp_move<0x111>(gs[e]);
                        ks[e] = dpp_move<0x111>(ks[e]);
                    }
                    const float y = ks[e] * exp2_of(x[e]);
                    ai[d] = __builtin_fmaf(kf[e], y, ai[d]);
                    pi[d] = __builtin_fmaf(qf[e], y, pi[d]);
                }
        }
        float *blk = Nb + block_of(w, w) * 320;  // this wave's own, free until below
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            ai[d] += __shfl_xor(ai[d], 16);
            pi[d] += __shfl_xor(pi[d], 16);
            ai[d] += __shfl_xor(ai[d], 32);
            pi[d] += __shfl_xor(pi[d], 32);
            if (lg == 0 && d <= lr) blk[lr * 20 + lr - d] = pi[d];
        }
        wave_sync();
#pragma unroll
        for (int r = 0; r < 4; ++r) Pd[r] = 4 * lg + r <= lr ? blk[lr * 20 + 4 * lg + r] : 0.f;
        wave_sync();
#pragma unroll
        for (int d = 0; d < 16; ++d)
            if (lg == 0 && d <= lr) blk[lr * 20 + lr - d] = ai[d];
        wave_sync();
#pragma unroll
        for (int r = 0; r < 4; ++r) Ad[r] = lr <= 4 * lg + r ? blk[(4 * lg + r) * 20 + lr] : 0.f;
        wave_sync();
    }
    // A and P come as 2^20 times their values
    const f32x4 beta4 = *reinterpret_cast<const f32x4 *>(betas + w * 16 + lg * 4) *
                        (1.f / (kUnit * kUnit));
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b > w) continue;  // uniform
        f32x4 Ab = Ad, Pb = Pd;
        if (b < 3 && b < w) {
            Ab = A[b < 3 ? b : 0];
            Pb = P[b < 3 ? b : 0];
        }
        float *blk = Nb + block_of(w, b) * 320;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (b == w && 4 * lg + r <= lr) Ab[r] = 0.f;  // strictly below the diagonal
            if (b == w && 4 * lg + r > lr) Pb[r] = 0.f;   // on it and below
            blk[(4 * lg + r) * 20 + lr] = Ab[r] * beta4[r];
        }
        *reinterpret_cast<u32x2 *>(lds + kLdsP + block_of(w, b) * 512 + lane * 8) =
            pack4_h(Pb * (1.f / kUnit));
    }
    // ---- inverse of this block's 1 + N by forward substitution, a column a lane
    {
        wave_sync();
        float *blk = Nb + block_of(w, w) * 320;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == lr ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) acc = __builtin_fmaf(-blk[i * 20 + j], x[j], acc);
            x[i] = acc;
        }
        wave_sync();
        if (lg == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) blk[i * 20 + lr] = x[i];
    }
    // ---- V in operand order: transposed, its own BF16 values.  Wave 0 takes
    // block 3 too: its A and P are the fewest, wave 3's the most.
    if (w < 3) {
#pragma unroll 1
        for (int vb = w; vb < 4; vb += 3) {
            const bool here = vb * 16 + lr < n;
            const uint16_t *from = a.v + (long)(row0 + vb * 16 + lr) * a.ldv + h * kHead + 8 * lg;
            u32x4 vv[4];
#pragma unroll
            for (int s = 0; s < 4; ++s)
                vv[s] = here ? *reinterpret_cast<const u32x4 *>(from + 32 * s) : zero;
            unsigned top = 0;
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    u32x4 sel = zero;  // column r picks value 16 hf + r
                    const int e = 16 * hf + lr - 8 * lg;
                    if (e >= 0 && e < 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sel[i] = e >> 1 == i ? (e & 1 ? 0x3F800000u : 0x3F80u) : 0u;
                    const f32x4 x = mfma_bf(vv[s], sel, none);
                    top = top_of(x, top);
                    *reinterpret_cast<u32x2 *>(ws + vb * kWsWave + ws_v(2 * s + hf) + lane * 8) =
                        u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
                }
            top = max64(top);
            if (lane == 0) reinterpret_cast<unsigned *>(ws + kWsTop)[vb] = top;
        }
    }
    __syncthreads();  // 2: N below the diagonal, the inverses, P and K e^{G_64 - G} are there

    // ---- column block w of T, a block at a time: T_ww is the block's inverse,
    // T_aw = -(inverse of a) (sum_c N_ac T_cw); rows i = 4 lg + r, column lr
    f32x4 T[4] = {none, none, none, none};
    {
        auto times = [&](int ai, int bi, f32x4 t, f32x4 acc) {  // block (ai, bi) of N times t
            const f32x4 nv =
                *reinterpret_cast<const f32x4 *>(Nb + block_of(ai, bi) * 320 + lr * 20 + lg * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(nv[r], t[r], acc, 0, 0, 0);
            return acc;
        };
        const float *d = Nb + block_of(w, w) * 320;
        f32x4 t, X[4] = {none, none, none, none};
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = d[(4 * lg + r) * 20 + lr];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c < w) continue;  // uniform
            T[c] = t;
#pragma unroll
            for (int i = c + 1; i < 4; ++i) X[i] = times(i, c, t, X[i]);
            if (c < 3) t = -times(c < 3 ? c + 1 : 3, c < 3 ? c + 1 : 3, X[c < 3 ? c + 1 : 3], none);
        }
    }
    // ---- columns of block w of M (as M^T: tokens j = 4 lg + r, channel lr of a tile) and of P T
    const float bj = betas[w * 16 + lr] * kUnit;
    const Split t0 = split_h(T[0], T[1], bj), t1 = split_h(T[2], T[3], bj);
    const int half = lane * 16 + (w & 1) * 8, step = w >> 1;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        f32x4 x = none, y = none;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if (st < step) continue;  // T is zero there; uniform
            const char *kp = lds + kLdsK + (t * 2 + st) * 2048 + lane * 16;
            const u32x4 kh = *reinterpret_cast<const u32x4 *>(kp);
            const u32x4 kl = *reinterpret_cast<const u32x4 *>(kp + 1024);
            const Split &ts = st ? t1 : t0;
            x = mfma_h(ts.hi, kl, x);
            y = mfma_h(ts.hi, kh, y);
            x = mfma_h(ts.lo, kh, x);
        }
        float m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = (x[r] + y[r]) * (1.f / kUnit);
        const unsigned h0 = settled(pack_h(m[0], m[1])), h1 = settled(pack_h(m[2], m[3]));
        char *to = ws + (t >> 1) * kWsWave + ws_m(t & 1, 0) + step * 2048 + half;
        *reinterpret_cast<u32x2 *>(to) = u32x2{h0, h1};
        *reinterpret_cast<u32x2 *>(to + 1024) =
            u32x2{pack_h(m[0] - h_lo(h0), m[1] - h_hi(h0)),
                  pack_h(m[2] - h_lo(h1), m[3] - h_hi(h1))};
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        if (it >> 1 < step) continue;  // the scan does not read these; uniform
        f32x4 x = none;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if (st < step || 2 * st > it) continue;  // uniform
            const char *pp = lds + kLdsP + block_of(it, 2 * st) * 512 + lane * 8;
            const u32x2 p0 = *reinterpret_cast<const u32x2 *>(pp);
            u32x2 p1 = {0u, 0u};
            if (2 * st + 1 <= it) p1 = *reinterpret_cast<const u32x2 *>(pp + 512);
            x = mfma_h((st ? t1 : t0).hi, u32x4{p0.x, p0.y, p1.x, p1.y}, x);
        }
        *reinterpret_cast<u32x2 *>(ws + it * kWsWave + ws_p(0) + step * 1024 + half) =
            pack4_h(x * (1.f / kUnit));
    }
}

// ---------------------------------------------------------------------------
// scan: a workgroup of four waves a head and 16 * CT columns of its state,
// chunk after chunk.  Wave w holds channel tiles 2 w and 2 w + 1 of S and
// computes token tile w of R and O, so each operand from the workspace goes
// to one wave only, straight into registers (those of the next chunk are
// loaded as soon as this one's are used); S and R meet in LDS as FP16 pairs.
// Two barriers a chunk.  A chunk is a chain (S's products, R, R's products,
// S') and takes 1.4 us alone with 16 columns, 1.9 with 32, 3.4 with 64.
//
// The scales of S and R are common to the waves without an exchange: a token
// adds at most |v| to the 2-norm of a column of S (|k| <= 1, beta <= 1, decays
// <= 1), so a bound of the column norms grows by 64 max |v| a chunk, and |R|
// <= max |v| + that bound.  The bound starts from the largest |S| and is
// taken from it again every 16 chunks, where it is at most 2^10 max |v| too
// large: FP16 pairs under a scale 2^13 too small still hold 2^-24 of the
// largest value.  (A maximum over a wave costs 300 cycles, two a chunk were a
// tenth of the scan.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ Scale scale_below(float bound) {
    return scale_for(__float_as_uint(fminf(bound, 3e38f)));
}
__device__ __forceinline__ float largest(u32x4 t) {
    const unsigned x = t.x > t.y ? t.x : t.y, y = t.z > t.w ? t.z : t.w;
    return __uint_as_float(x > y ? x : y);
}

// A chunk's operands of one wave.
template <int CT>
struct ChunkOperands {
    Split k[4], m[2][2];
    u32x4 q[4], p[2], vtop;
    u32x2 v[CT];
    f32x4 d[2];

    // what step s over channels of R takes
    __device__ __forceinline__ void load_step(const char *at, int s, int w, int lane) {
        const char *from = at + w * kWsWave + lane * 16;
        k[s].hi = *reinterpret_cast<const u32x4 *>(from + ws_k(s));
        k[s].lo = *reinterpret_cast<const u32x4 *>(from + ws_k(s) + 1024);
        q[s] = *reinterpret_cast<const u32x4 *>(from + ws_q(s));
    }
    __device__ __forceinline__ void load_values(const char *at, int w, int lane, int part) {
#pragma unroll
        for (int i = 0; i < CT; ++i)
            v[i] = *reinterpret_cast<const u32x2 *>(at + w * kWsWave + ws_v(0) +
                                                    (part * CT + i) * 512 + lane * 8);
        vtop = *reinterpret_cast<const u32x4 *>(at + kWsTop);
    }
    // what step st over tokens of S' takes
    __device__ __forceinline__ void load_tokens(const char *at, int st, int w, int lane) {
        const char *from = at + w * kWsWave + lane * 16;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            m[hf][st].hi = *reinterpret_cast<const u32x4 *>(from + ws_m(hf, st));
            m[hf][st].lo = *reinterpret_cast<const u32x4 *>(from + ws_m(hf, st) + 1024);
        }
        if (st == 0 || w >= 2) p[st] = *reinterpret_cast<const u32x4 *>(from + ws_p(st));
    }
    __device__ __forceinline__ void load_decays(const char *at, int w, int lane) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
            d[hf] = *reinterpret_cast<const f32x4 *>(
                at + kWsD + (32 * w + 8 * (lane >> 4) + 4 * hf) * 4);
    }
    __device__ __forceinline__ void load(const char *at, int w, int lane, int part) {
#pragma unroll
        for (int s = 0; s < 4; ++s) load_step(at, s, w, lane);
        load_values(at, w, lane, part);
        load_tokens(at, 0, w, lane);
        load_tokens(at, 1, w, lane);
        load_decays(at, w, lane);
    }
};

// AHEAD = 0: one set of operands, each half reloaded once it is used.  AHEAD
// = 1 or 2: that many chunks loaded ahead, between the products (a scan that
// has the compute unit to itself, where nothing else covers the latency): 21
// chunks of 12 heads take 39 us with 32 columns a workgroup, 58 with all loads
// at the chunk's start.
template <int CT, int AHEAD>
__device__ __forceinline__ void scan_columns(const DeltaArgs &a, int row0, int rows, int slot,
                                             int h, int part, const char *ws, size_t ws_step,
                                             char *lds) {
    const int lane = threadIdx.x & 63;
    const int w = scalar(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    unsigned *tops = reinterpret_cast<unsigned *>(lds + lds_tops(CT));
    float *state = a.state + ((size_t)slot * a.H + h) * (kHead * kHead) +
                   (size_t)(32 * w + 8 * lg) * kHead + part * (16 * CT) + lr;
    const int chunks = (rows + kC - 1) / kC;
    ChunkOperands<CT> ops[AHEAD + 1];
    // a chunk's place, or the last one's past the end (read again, unused)
    auto place = [&](int c) { return ws + (size_t)min(c, chunks - 1) * ws_step; };
    f32x4 S[2][CT];
#pragma unroll
    for (int i = 0; i < (AHEAD ? AHEAD : 1); ++i) {
        ops[i].load(place(i), w, lane, part);
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int v = 0; v < CT; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[hf][v][r] = state[(4 * hf + r) * kHead + v * 16];
    auto measure = [&]() {  // this wave's largest |S|, for the others
        unsigned top = 0;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int v = 0; v < CT; ++v) top = top_of(S[hf][v], top);
        top = max64(top);
        if (lane == 0) tops[w] = top;
    };
    auto measured = [&]() {  // a bound of the columns' norms from the largest |S| of all
        return 12.f * largest(*reinterpret_cast<const u32x4 *>(tops));
    };
    auto share = [&](float up) {  // this wave's channels of S, as operands of step s = w
#pragma unroll
        for (int v = 0; v < CT; ++v) {
            const Split x = split_h(S[0][v], S[1][v], up);
            char *to = lds + lds_s(CT, w, v) + lane * 16;
            *reinterpret_cast<u32x4 *>(to) = x.hi;
            *reinterpret_cast<u32x4 *>(to + 1024) = x.lo;
        }
    };
    measure();
    __syncthreads();
    float bound = measured();
    Scale ss = scale_below(bound);
    share(ss.up);
    uint16_t *out = a.out + (size_t)(row0 + w * 16 + lr) * a.ldo + h * kHead + part * (16 * CT) +
                    lg * 4;

    auto chunk = [&](int c, ChunkOperands<CT> &now, ChunkOperands<CT> &later) {
        const char *ahead = place(c + (AHEAD ? AHEAD : 1));
        __syncthreads();  // S is there
        if ((c & 15) == 15) bound = measured();
        const float vmax = largest(now.vtop);
        const Scale sr = scale_below(vmax + bound);
        f32x4 x[CT], y[CT], o[CT];
#pragma unroll
        for (int v = 0; v < CT; ++v) x[v] = y[v] = o[v] = none;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int v = 0; v < CT; ++v) {
                const char *at = lds + lds_s(CT, s, v) + lane * 16;
                const u32x4 bh = *reinterpret_cast<const u32x4 *>(at);
                const u32x4 bl = *reinterpret_cast<const u32x4 *>(at + 1024);
                x[v] = mfma_h(now.k[s].hi, bl, x[v]);
                y[v] = mfma_h(now.k[s].hi, bh, y[v]);
                o[v] = mfma_h(bh, now.q[s], o[v]);
                x[v] = mfma_h(now.k[s].lo, bh, x[v]);
                if (v == CT - 1) {
                    if constexpr (AHEAD > 0) later.load_step(ahead, s, w, lane);
                }
            }
        const float back = ss.down / kUnit;
#pragma unroll
        for (int v = 0; v < CT; ++v) {
            const float vv[4] = {bf16_lo(now.v[v].x), bf16_hi(now.v[v].x), bf16_lo(now.v[v].y),
                                 bf16_hi(now.v[v].y)};
            f32x4 R;
#pragma unroll
            for (int r = 0; r < 4; ++r) R[r] = __builtin_fmaf(x[v][r] + y[v][r], back, vv[r]);
            R *= sr.up;
            const unsigned h0 = settled(pack_h(R[0], R[1])), h1 = settled(pack_h(R[2], R[3]));
            char *to = lds + lds_r(CT, 0, v) + (w >> 1) * (CT * 2048) + lane * 16 + (w & 1) * 8;
            *reinterpret_cast<u32x2 *>(to) = u32x2{h0, h1};
            *reinterpret_cast<u32x2 *>(to + 1024) =
                u32x2{pack_h(R[0] - h_lo(h0), R[1] - h_hi(h0)),
                      pack_h(R[2] - h_lo(h1), R[3] - h_hi(h1))};
        }
        if constexpr (AHEAD == 0) {
#pragma unroll
            for (int s = 0; s < 4; ++s) now.load_step(ahead, s, w, lane);
            now.load_values(ahead, w, lane, part);
        } else {
            later.load_values(ahead, w, lane, part);
        }
        bound += 64.f * vmax;
        ss = scale_below(bound);
        __syncthreads();  // R is there; S's operands are free
        f32x4 u[2][CT], z[2][CT], ou[CT];
#pragma unroll
        for (int v = 0; v < CT; ++v) u[0][v] = u[1][v] = z[0][v] = z[1][v] = ou[v] = none;
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int v = 0; v < CT; ++v) {
                const char *at = lds + lds_r(CT, st, v) + lane * 16;
                const u32x4 bh = *reinterpret_cast<const u32x4 *>(at);
                const u32x4 bl = *reinterpret_cast<const u32x4 *>(at + 1024);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    u[hf][v] = mfma_h(now.m[hf][st].hi, bl, u[hf][v]);
                    z[hf][v] = mfma_h(now.m[hf][st].hi, bh, z[hf][v]);
                }
                if (st == 0 || w >= 2) ou[v] = mfma_h(bh, now.p[st], ou[v]);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) u[hf][v] = mfma_h(now.m[hf][st].lo, bh, u[hf][v]);
                if (v == CT - 1) {
                    if constexpr (AHEAD > 0) later.load_tokens(ahead, st, w, lane);
                }
            }
        const float rb = sr.down / kUnit;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int v = 0; v < CT; ++v)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[hf][v][r] = __builtin_fmaf(u[hf][v][r] + z[hf][v][r], rb,
                                                 S[hf][v][r] * now.d[hf][r]);
        share(ss.up);
        if constexpr (AHEAD == 0) {
            now.load_tokens(ahead, 0, w, lane);
            now.load_tokens(ahead, 1, w, lane);
            now.load_decays(ahead, w, lane);
        } else {
            later.load_decays(ahead, w, lane);
        }
        if ((c & 15) == 14) measure();
        const float os = back * a.scale, ob = rb * a.scale;
        if (c * kC + w * 16 + lr < rows) {
            uint16_t *to = out + (size_t)(c * kC) * a.ldo;
#pragma unroll
            for (int v = 0; v < CT; ++v) {
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) e[r] = __builtin_fmaf(o[v][r], os, ou[v][r] * ob);
                *reinterpret_cast<u32x2 *>(to + v * 16) =
                    u32x2{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3])};
            }
        }
    };
    if constexpr (AHEAD == 0) {
        for (int c = 0; c < chunks; ++c) chunk(c, ops[0], ops[0]);
    } else {
        constexpr int N = AHEAD + 1;  // the sets in turn
        for (int c = 0; c < chunks; c += N) {
            chunk(c, ops[0], ops[N - 1]);
            if (c + 1 < chunks) chunk(c + 1, ops[1], ops[0]);
            if constexpr (N == 3) {
                if (c + 2 < chunks) chunk(c + 2, ops[2], ops[1]);
            }
        }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int v = 0; v < CT; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) state[(4 * hf + r) * kHead + v * 16] = S[hf][v][r];
}

// Which head (of all sequences) and which of its columns a scan's workgroup
// takes.  Workgroups go to the eight XCDs in turn, each with an L2 of its
// own: the workgroups of a head, which load the same operands, are eight
// apart, so that one L2 fetches them once.
template <int PARTS>
__device__ __forceinline__ void scan_place(int i, int all, int *head, int *part) {
    const int g = i / (8 * PARTS), r = i % (8 * PARTS);
    const int heads = min(8, all - 8 * g);  // of this group
    *head = 8 * g + r % heads;
    *part = r / heads;
}

// A launch holds the scan of one segment (its workgroups come first) and the
// preparation of the next, which do not depend on each other.
template <int CT, bool HEAD_GATE>
__global__ __launch_bounds__(256, 2) void delta_chunk_kernel(DeltaArgs a, DeltaSegment scan,
                                                             DeltaSegment prep) {
    extern __shared__ __align__(16) char lds[];
    constexpr int PARTS = 8 / CT;  // workgroups a head in the scan
    const int all = scan.seqs * a.H, scans = all * PARTS;
    int i = blockIdx.x;
    if (i < scans) {
        int head, part;
        scan_place<PARTS>(i, all, &head, &part);
        const int h = head % a.H;
        const int *e = scan.seq_table + 4 * (head / a.H);
        scan_columns<CT, 0>(a, e[0], e[1], e[2], h, part,
                            scan.ws + ((size_t)e[3] * a.H + h) * kDeltaItemBytes,
                            (size_t)a.H * kDeltaItemBytes, lds);
        return;
    }
    i -= scans;
    const int h = i % a.H, c = i / a.H;
    const int *e = prep.chunk_table + 2 * c;
    prepare_item<HEAD_GATE>(a, e[0], e[1], h, prep.ws + (size_t)i * kDeltaItemBytes, lds);
}

// A scan alone: one workgroup a compute unit, with registers to load ahead.
template <int CT>
__global__ __launch_bounds__(256, 1) void delta_scan_kernel(DeltaArgs a, DeltaSegment scan) {
    extern __shared__ __align__(16) char lds[];
    constexpr int PARTS = 8 / CT;
    int head, part;
    scan_place<PARTS>(blockIdx.x, scan.seqs * a.H, &head, &part);
    const int h = head % a.H;
    const int *e = scan.seq_table + 4 * (head / a.H);
    scan_columns<CT, CT == 4 ? 1 : 2>(a, e[0], e[1], e[2], h, part,
                                      scan.ws + ((size_t)e[3] * a.H + h) * kDeltaItemBytes,
                                      (size_t)a.H * kDeltaItemBytes, lds);
}

template <int CT, bool HEAD_GATE>
hipError_t launch(const DeltaArgs &a, const DeltaSegment &scan, const DeltaSegment &prep,
                  hipStream_t st) {
    const dim3 grid((unsigned)(scan.seqs * a.H * (8 / CT) + prep.chunks * a.H));
    hipLaunchKernelGGL((delta_chunk_kernel<CT, HEAD_GATE>), grid, dim3(256), kDeltaLds, st, a,
                       scan, prep);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunks(const DeltaArgs &a, const DeltaSegment &scan,
                               const DeltaSegment &prep, bool head_gate, int cus,
                               hipStream_t st) {
    // Columns a workgroup: the fewer, the shorter a chunk takes (a head's
    // chunks are one chain), but each workgroup of a head loads its 104 KB of
    // operands.  By the heads at work on average (a short sequence is soon
    // done): 8192 tokens of 12 heads take 222 us with 16 columns, 277 with
    // 32, 413 with 64; of 24 heads 327, 358 and 492; of 40 heads 565, 464 and
    // 561; of 96 heads 1222, 1023 and 902.
    const long all = (long)scan.seqs * a.H;
    const long busy = scan.longest ? (long)scan.chunks * a.H / scan.longest : 0;
    const int ct = busy <= cus / 8 ? 1 : busy <= cus / 4 ? 2 : 4;
    if (prep.chunks == 0) {
        const dim3 grid((unsigned)(all * (8 / ct)));
        if (ct == 1)
            hipLaunchKernelGGL(delta_scan_kernel<1>, grid, dim3(256), kDeltaLds, st, a, scan);
        else if (ct == 2)
            hipLaunchKernelGGL(delta_scan_kernel<2>, grid, dim3(256), kDeltaLds, st, a, scan);
        else
            hipLaunchKernelGGL(delta_scan_kernel<4>, grid, dim3(256), kDeltaLds, st, a, scan);
        return hipGetLastError();
    }
    if (ct == 1)
        return head_gate ? launch<1, true>(a, scan, prep, st) : launch<1, false>(a, scan, prep, st);
    if (ct == 2)
        return head_gate ? launch<2, true>(a, scan, prep, st) : launch<2, false>(a, scan, prep, st);
    return head_gate ? launch<4, true>(a, scan, prep, st) : launch<4, false>(a, scan, prep, st);
}

hipError_t allow_delta_lds() {
    hipError_t e = hipSuccess;
    auto one = [&](const void *f) {
        if (e == hipSuccess)
            e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kDeltaLds);
    };
    one(reinterpret_cast<const void *>(&delta_scan_kernel<1>));
    one(reinterpret_cast<const void *>(&delta_scan_kernel<2>));
    one(reinterpret_cast<const void *>(&delta_scan_kernel<4>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<1, true>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<1, false>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<2, true>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<2, false>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<4, true>));
    one(reinterpret_cast<const void *>(&delta_chunk_kernel<4, false>));
    return e;
}

}  // namespace tp1
