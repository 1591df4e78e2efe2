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
// diag(beta), the u_i are U = T V - (T K e^G) S.  Everything but the terms
// in S is independent of the chunks before, so the work is in two parts:
//   prepare (one workgroup a chunk and head): W = -T K e^G, U0 = T V, P,
//     Q e^G, K e^{G_64 - G} and e^{G_64}, written to a workspace;
//   scan (eight waves a head, 16 columns of the state each): chunk after chunk,
//     U = U0 + W S, O = (Q e^G) S + P U, S' as above.
//
// Numbers.  All products run on the 16-bit matrix cores with FP32 sums, and
// what reaches the state is as exact as FP32 operands would make it.  Keys
// and queries have unit length here (the chunked form is taken with l2norm
// only), so every update is a contraction and T, W, K e^.. and Q e^.. stay
// within 1: they are held as two FP16 values hi + lo of 2^10 times the value,
// and hi hi + hi lo + lo hi summed, which drops 2^-23 of each (two BF16
// values would drop 2^-17, one 2^-9).  S, U and V have any range: a wave
// scales what it holds by a power of two that brings the largest magnitude
// to 2^14.  What only reaches the BF16 output (Q, P, and the hi parts of S
// and U against them) is one FP16 value each, 2^-12.
// Decays are products of factors e^x with x <= 0, the sums x taken inside
// blocks of 16 tokens from the token outward, so none is a difference of
// large numbers: with block a after block b, e^{G_i - G_j} = (e^{sum of a's
// tokens up to i}) (e^{whole blocks between}) (e^{sum of b's tokens after
// j}).  Inside a block the second factor is e^{-(sum up to j)} instead,
// which grows, so those products are FP32 ones (v_mfma_f32_16x16x4), and a
// block whose tokens decay a channel by more than 2^-58 takes an exact path
// on the vector unit (a running sum from i down to j).
//
// Layout.  A wave of `prepare` owns one block of 16 tokens; lane l holds
// token l % 16 and, for s = 0..3, channels 32 s + 8 (l / 16) + 0..7, which is
// the A and B operand of v_mfma_f32_16x16x32 over channels.  Sums over
// the tokens of a block are scans over 16 lanes (DPP).  Operands over tokens
// need the transpose, which a product with a selection matrix gives exactly
// (accumulator lane l holds rows 4 (l / 16) + 0..3 of column l % 16).  The
// order of the 32 summed values of a product is free, so the scan feeds its
// accumulators S and U back as operands without any exchange: S tile 2 s + h
// has channel 32 s + 8 (r / 4) + 4 h + r % 4 as row r, and a step over tokens
// takes blocks 2 t and 2 t + 1, tokens 4 (l / 16) + 0..3 of each.  The
// workspace holds every operand in that order, so each load is 16 bytes a
// lane, 1 KB in one piece.
#include "delta.hpp"

#include "device.hpp"

namespace tp1 {

namespace {

constexpr int kC = kDeltaChunk;   // tokens a chunk

// Workspace of a chunk and head: eight pieces of 12 KB, in the order the scan
// takes them, then U0.  Everything in operand order, 16 bytes a lane:
//   piece it = 0..3:      W of token tile it [4 s][hi, lo], Q e^G [4 s]
//   piece 4 + s, s = 0..3: K e^{G_64 - G} of channel tiles 2 s, 2 s + 1 [2 steps]
//                         [hi, lo], P of token tile s [2 steps], and (s = 0)
//                         e^{G_64} [128] FP32
//   U0:                   [4 token tiles][8 value tiles] FP32
constexpr int kPiece = 12288;
constexpr int kWsU = 8 * kPiece;
static_assert(kWsU + 32768 == kDeltaItemBytes, "workspace of an item");
constexpr int ws_w(int it, int s) { return it * kPiece + s * 2048; }
constexpr int ws_q(int it, int s) { return it * kPiece + 8192 + s * 1024; }
constexpr int ws_k(int tile, int step) {
    return (4 + tile / 2) * kPiece + (tile % 2 * 2 + step) * 2048;
}
constexpr int ws_p(int it, int step) { return (4 + it) * kPiece + 8192 + step * 1024; }
constexpr int kWsD = 4 * kPiece + 8192 + 2048;

// LDS of `prepare`, in bytes.
constexpr int kLdsKr = 0;                     // [48 rows][hi, lo][128] FP16, dead after barrier 2
constexpr int kLdsT = 0;                      // [hi, lo][10 blocks][16 rows][40]
constexpr int kLdsV = kLdsT + 2 * 10 * 640;   // [8 value tiles][2 steps][64][16]
constexpr int kLdsK = kLdsV + 16384;          // [8 channel tiles][2 steps][hi, lo][64][16]
constexpr int kLdsN = kLdsK + 32768;          // [10 blocks][16 rows][20] FP32
constexpr int kLdsTot = kLdsN + 10 * 1280;    // [4][128] FP32: a block's whole decay
constexpr int kLdsBeta = kLdsTot + 2048;      // [64] FP32
constexpr int kLdsTop = kLdsBeta + 256;       // [4] largest |v| of a block (bits)
static_assert(kLdsKr + 48 * 512 <= kLdsK, "the transposed values reuse the key rows");
static_assert(kLdsTop + 16 <= kDeltaLds, "LDS of prepare");
// LDS of `scan`: a ring of piece slots, each with the wave's U0 tiles behind.
constexpr int kSlots = 5;
constexpr int kSlot = kPiece + 4096;
static_assert(kSlots * kSlot <= kDeltaLds, "LDS of scan");

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma_bf(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_h(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// A block is mild if no channel decays by more than 2^-kMild over it.
constexpr float kMild = 58.f;

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

template <int I>
struct Place {
    static constexpr int value = I;
};

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
// prepare: one workgroup of four waves a chunk and head.
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
    u32x4 kv[4], qv[4], vv[4], fv[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = 32 * s + 8 * lg;
        kv[s] = qv[s] = vv[s] = fv[s] = zero;
        if (live) {
            kv[s] = *reinterpret_cast<const u32x4 *>(a.k + row * a.ldk + hk * kHead + c);
            qv[s] = *reinterpret_cast<const u32x4 *>(a.q + row * a.ldq + hk * kHead + c);
            vv[s] = *reinterpret_cast<const u32x4 *>(a.v + row * a.ldv + h * kHead + c);
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
    {
        unsigned top = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned lo = (vv[s][i] << 16) & 0x7FFFFFFFu, hi = vv[s][i] & 0x7FFF0000u;
                top = lo > top ? lo : top;
                top = hi > top ? hi : top;
            }
        top = max64(top);
        if (lane == 0) reinterpret_cast<unsigned *>(lds + kLdsTop)[w] = top;
    }
    __syncthreads();  // 1: key rows, block totals, betas and the values' range are there

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
        // to the chunk's ends: Q e^G and K e^{G_64 - G} to the workspace, K e^G to LDS
        {
            float kt[8], kh[8], qt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kt[e] = x[e] * before[e / 4][e % 4];
                qt[e] = y[e] * before[e / 4][e % 4];
                kh[e] = kf[e] * er[s][e] * behind[e / 4][e % 4];
            }
            *reinterpret_cast<u32x4 *>(ws + ws_q(0, s) + w * kPiece + lane * 16) = round_h(qt);
            if (w == 3 && lr == 15) {  // e^{G_64}: the decay of the whole chunk
                f32x4 *o = reinterpret_cast<f32x4 *>(ws + kWsD + c * 4);
                o[0] = f32x4{el[s][0], el[s][1], el[s][2], el[s][3]} * before[0];
                o[1] = f32x4{el[s][4], el[s][5], el[s][6], el[s][7]} * before[1];
            }
            const Split st = split_h(kt), sh = split_h(kh);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                // column r of the selection picks channel 8 (r / 4) + 4 hf + r % 4
                const u32x4 sel =
                    hf ? u32x4{0u, 0u, pick0, pick1} : u32x4{pick0, pick1, 0u, 0u};
                const int half = lane * 16 + (w & 1) * 8;
                char *kl = lds + kLdsK + ((2 * s + hf) * 2 + (w >> 1)) * 2048 + half;
                char *kg = ws + ws_k(2 * s + hf, 0) + (w >> 1) * 2048 + half;
                *reinterpret_cast<u32x2 *>(kl) = pack4_h(mfma_h(st.hi, sel, none));
                *reinterpret_cast<u32x2 *>(kl + 1024) = pack4_h(mfma_h(st.lo, sel, none));
                *reinterpret_cast<u32x2 *>(kg) = pack4_h(mfma_h(sh.hi, sel, none));
                *reinterpret_cast<u32x2 *>(kg + 1024) = pack4_h(mfma_h(sh.lo, sel, none));
            }
        }
        // A and P, block row w: inside the block, then the blocks before
        if (mild) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // e^{-(sum up to j)}; el is at least 2^-58 here
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
        char *po = ws + ws_p(0, b >> 1) + w * kPiece + lane * 16;
        *reinterpret_cast<u32x2 *>(po + (b & 1) * 8) = pack4_h(Pb * (1.f / kUnit));
        if (b == w && (b & 1) == 0) *reinterpret_cast<u32x2 *>(po + 8) = u32x2{0u, 0u};
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
    __syncthreads();  // 2: N below the diagonal and the inverses are there; key rows are free

    // ---- V transposed (scaled to FP16's range), and column block w of the whole inverse
    Scale sv;
    {
        const u32x4 t = *reinterpret_cast<const u32x4 *>(lds + kLdsTop);
        const unsigned x = t.x > t.y ? t.x : t.y, y = t.z > t.w ? t.z : t.w;
        sv = scale_for(x > y ? x : y);
    }
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
            *reinterpret_cast<u32x2 *>(lds + kLdsV + ((2 * s + hf) * 2 + (w >> 1)) * 1024 +
                                       lane * 16 + (w & 1) * 8) =
                pack4_h(mfma_bf(vv[s], sel, none) * sv.up);
        }
    {
        const float bj = betas[w * 16 + lr] * kUnit;
        auto store_t = [&](int ai, f32x4 t) {  // T_ab diag(beta), rows i = 4 lg + r, column lr
            char *o = lds + kLdsT + block_of(ai, w) * 640 + lr * 2;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x = t[r] * bj;
                const unsigned hi = settled(pack_h(x, 0.f));
                *reinterpret_cast<uint16_t *>(o + (4 * lg + r) * 40) = (uint16_t)hi;
                *reinterpret_cast<_Float16 *>(o + 6400 + (4 * lg + r) * 40) =
                    (_Float16)(x - h_lo(hi));
            }
        };
        auto times = [&](int ai, int bi, f32x4 t, f32x4 acc) {  // block (ai, bi) of N times t
            const f32x4 nv =
                *reinterpret_cast<const f32x4 *>(Nb + block_of(ai, bi) * 320 + lr * 20 + lg * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(nv[r], t[r], acc, 0, 0, 0);
            return acc;
        };
        // T_ww is the block's inverse; T_aw = -(inverse of a) (sum_c N_ac T_cw)
        const float *d = Nb + block_of(w, w) * 320;
        f32x4 t, X[4] = {none, none, none, none};
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = d[(4 * lg + r) * 20 + lr];
        store_t(w, t);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            if (c < w) continue;  // uniform
#pragma unroll
            for (int i = c + 1; i < 4; ++i) X[i] = times(i, c, t, X[i]);
            t = -times(c + 1, c + 1, X[c + 1], none);
            store_t(c + 1, t);
        }
    }
    __syncthreads();  // 3: T and the transposed values are there

    // ---- W = -T K e^G (channels 32 w + 0..31) and U0 = T V (the same columns)
    f32x4 Wt[2][4], U[4][2];  // W^T[channel tile][token tile], U0[token tile][value tile]
#pragma unroll
    for (int it = 0; it < 4; ++it) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) Wt[hf][it] = U[it][hf] = none;
#pragma unroll
        for (int st = 0; st <= it >> 1; ++st) {
            const char *t0 = lds + kLdsT + block_of(it, 2 * st) * 640 + lr * 40 + lg * 8;
            const u32x2 h0 = *reinterpret_cast<const u32x2 *>(t0);
            const u32x2 l0 = *reinterpret_cast<const u32x2 *>(t0 + 6400);
            u32x2 h1 = {0u, 0u}, l1 = {0u, 0u};
            if (2 * st + 1 <= it) {
                h1 = *reinterpret_cast<const u32x2 *>(t0 + 640);
                l1 = *reinterpret_cast<const u32x2 *>(t0 + 640 + 6400);
            }
            const u32x4 th = {h0.x, h0.y, h1.x, h1.y}, tl = {l0.x, l0.y, l1.x, l1.y};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const char *kp = lds + kLdsK + ((2 * w + hf) * 2 + st) * 2048 + lane * 16;
                const u32x4 kh = *reinterpret_cast<const u32x4 *>(kp);
                const u32x4 ko = *reinterpret_cast<const u32x4 *>(kp + 1024);
                const u32x4 vt = *reinterpret_cast<const u32x4 *>(
                    lds + kLdsV + ((2 * w + hf) * 2 + st) * 1024 + lane * 16);
                Wt[hf][it] = mfma_h(kh, tl, Wt[hf][it]);
                Wt[hf][it] = mfma_h(ko, th, Wt[hf][it]);
                Wt[hf][it] = mfma_h(kh, th, Wt[hf][it]);
                U[it][hf] = mfma_h(tl, vt, U[it][hf]);
                U[it][hf] = mfma_h(th, vt, U[it][hf]);
            }
        }
        const Split o = split_h(Wt[0][it], Wt[1][it], -1.f / kUnit);
        char *wp = ws + ws_w(it, 0) + w * 2048 + lane * 16;
        *reinterpret_cast<u32x4 *>(wp) = o.hi;
        *reinterpret_cast<u32x4 *>(wp + 1024) = o.lo;
        const float back = sv.down / kUnit;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
            *reinterpret_cast<f32x4 *>(ws + kWsU + ((it * 8 + 2 * w + hf) * 64 + lane) * 16) =
                U[it][hf] * back;
    }
}

// ---------------------------------------------------------------------------
// scan: a workgroup of four waves a head and 64 columns of its state, 16
// columns a wave, chunk after chunk.  A chunk's eight pieces go straight into
// a ring of LDS slots (global_load_lds_dwordx4), kSlots - 1 pieces ahead,
// and every wave reads its operands from there, so the state, which the next
// chunk waits for, never waits for memory.  One barrier a piece.
// ---------------------------------------------------------------------------
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes a lane from src into LDS at base + 16 * lane (base uniform).  M0
// needs one wait state between its write and the load that reads it.
__device__ __forceinline__ void lds_load16(const void *src, uint32_t base) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(src), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// A wave's loads of piece p: a quarter of the piece, and with W its own
// columns of U0.
constexpr int piece_loads(int p) { return p % 8 < 4 ? 4 : 3; }
// Loads of the kSlots - 2 pieces after piece p, which may be in flight when
// piece p is needed.
constexpr int loads_after(int p) {
    int n = 0;
    for (int i = 1; i <= kSlots - 2; ++i) n += piece_loads(p + i);
    return n;
}

__device__ void scan_columns(const DeltaArgs &a, int row0, int rows, int slot, int h, int part,
                             const char *ws, size_t ws_step, char *lds) {
    const int lane = threadIdx.x & 63;
    const int w = scalar(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int vt = part * 4 + w;  // this wave's value tile
    const int chunks = (rows + kC - 1) / kC;
    const uint32_t lds0 =
        scalar((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)lds);
    float *state = a.state + ((size_t)slot * a.H + h) * (kHead * kHead) + vt * 16 + lr;
    f32x4 S[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[t][r] = state[(size_t)(32 * (t >> 1) + 8 * lg + 4 * (t & 1) + r) * kHead];
    wait_loads<0>();  // the ring's loads are counted from here

    // the next piece to load: its place in the chunk is known where it is issued
    int slot_in = 0, chunk_in = 0;
    const char *ws_in = ws;
    auto issue = [&](int p) {  // p: place of the piece in its chunk
        const uint32_t to = lds0 + (uint32_t)(slot_in * kSlot);
        const char *from = ws_in + p * kPiece + w * 3072 + lane * 16;
#pragma unroll
        for (int j = 0; j < 3; ++j)
            lds_load16(from + j * 1024, to + (uint32_t)(w * 3072 + j * 1024));
        if (p < 4)
            lds_load16(ws_in + kWsU + (p * 8 + vt) * 1024 + lane * 16,
                       to + (uint32_t)(kPiece + w * 1024));
        slot_in = slot_in + 1 == kSlots ? 0 : slot_in + 1;
        // past the last chunk the ring reads it again: nothing uses that
        if (p == 7 && ++chunk_in < chunks) ws_in += ws_step;
    };
#pragma unroll
    for (int p = 0; p < kSlots - 1; ++p) issue(p);

    int slot_at = 0;
    const char *in = lds;
    auto next = [&](auto place) {  // piece `place` of the chunk has landed, the one before is free
        constexpr int p = decltype(place)::value;
        wait_loads<loads_after(p)>();
        __syncthreads();
        issue((p + kSlots - 1) % 8);
        in = lds + slot_at * kSlot;
        slot_at = slot_at + 1 == kSlots ? 0 : slot_at + 1;
    };

    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < rows; r0 += kC) {
        const int n = min(kC, rows - r0);
        unsigned top = 0;
#pragma unroll
        for (int t = 0; t < 8; ++t) top = top_of(S[t], top);
        const Scale ss = scale_for(max64(top));
        const float back = ss.down / kUnit;
        Split b[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) b[s] = split_h(S[2 * s], S[2 * s + 1], ss.up);
        f32x4 U[4], O[4];  // U[token][value]; O[value][token] of Q S
        top = 0;
        auto rows_of = [&](auto tile) {
            constexpr int it = decltype(tile)::value;
            next(tile);
            const char *at = in + lane * 16;
            f32x4 x = none, y = none, z = none, o = none;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const u32x4 wh = *reinterpret_cast<const u32x4 *>(at + s * 2048);
                const u32x4 wl = *reinterpret_cast<const u32x4 *>(at + s * 2048 + 1024);
                const u32x4 q = *reinterpret_cast<const u32x4 *>(at + 8192 + s * 1024);
                x = mfma_h(wh, b[s].lo, x);
                y = mfma_h(wl, b[s].hi, y);
                z = mfma_h(wh, b[s].hi, z);
                o = mfma_h(b[s].hi, q, o);
            }
            O[it] = o;
            const f32x4 u0 = *reinterpret_cast<const f32x4 *>(at + kPiece + w * 1024);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                U[it][r] = __builtin_fmaf((x[r] + y[r]) + z[r], back, u0[r]);
            top = top_of(U[it], top);
        };
        rows_of(Place<0>{});
        rows_of(Place<1>{});
        rows_of(Place<2>{});
        rows_of(Place<3>{});
        const Scale su = scale_for(max64(top));
        const float ub = su.down / kUnit;
        const float os = back * a.scale, ou = ub * a.scale;
        const Split u[2] = {split_h(U[0], U[1], su.up), split_h(U[2], U[3], su.up)};
        auto channels_of = [&](auto quarter) {
            constexpr int q = decltype(quarter)::value;
            next(Place<4 + q>{});
            const char *at = in + lane * 16;
            if (q == 0) {
                // the whole chunk's decays, of every piece's channels
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const f32x4 d = *reinterpret_cast<const f32x4 *>(
                        in + (kWsD - 4 * kPiece) + (32 * (t >> 1) + 8 * lg + 4 * (t & 1)) * 4);
                    S[t] *= d;
                }
            }
            f32x4 x[2] = {none, none}, y[2] = {none, none}, o = none;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const char *kp = at + (hf * 2 + st) * 2048;
                    const u32x4 kh = *reinterpret_cast<const u32x4 *>(kp);
                    const u32x4 kl = *reinterpret_cast<const u32x4 *>(kp + 1024);
                    x[hf] = mfma_h(kh, u[st].lo, x[hf]);
                    y[hf] = mfma_h(kh, u[st].hi, y[hf]);
                    x[hf] = mfma_h(kl, u[st].hi, x[hf]);
                }
#pragma unroll
            for (int st = 0; st <= q >> 1; ++st) {
                const u32x4 p = *reinterpret_cast<const u32x4 *>(at + 8192 + st * 1024);
                o = mfma_h(u[st].hi, p, o);
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[2 * q + hf][r] =
                        __builtin_fmaf(x[hf][r] + y[hf][r], ub, S[2 * q + hf][r]);
            if (q * 16 + lr < n) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(O[q][r], os, o[r] * ou);
                *reinterpret_cast<u32x2 *>(a.out + (size_t)(row0 + r0 + q * 16 + lr) * a.ldo +
                                           h * kHead + vt * 16 + lg * 4) =
                    u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            }
        };
        channels_of(Place<0>{});
        channels_of(Place<1>{});
        channels_of(Place<2>{});
        channels_of(Place<3>{});
    }
    wait_loads<0>();  // no wave leaves LDS writes in flight
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            state[(size_t)(32 * (t >> 1) + 8 * lg + 4 * (t & 1) + r) * kHead] = S[t][r];
}

// A launch holds the scan of one segment (its workgroups come first) and the
// preparation of the next, which do not depend on each other.
template <bool HEAD_GATE>
__global__ __launch_bounds__(256, 2) void delta_chunk_kernel(DeltaArgs a, DeltaSegment scan,
                                                             DeltaSegment prep) {
    extern __shared__ __align__(16) char lds[];
    const int scans = scan.seqs * a.H * 2;  // two workgroups of 64 columns a head
    int i = blockIdx.x;
    if (i < scans) {
        const int h = (i >> 1) % a.H;
        const int *e = scan.seq_table + 4 * ((i >> 1) / a.H);
        scan_columns(a, e[0], e[1], e[2], h, i & 1,
                     scan.ws + ((size_t)e[3] * a.H + h) * kDeltaItemBytes,
                     (size_t)a.H * kDeltaItemBytes, lds);
        return;
    }
    i -= scans;
    const int h = i % a.H, c = i / a.H;
    const int *e = prep.chunk_table + 2 * c;
    prepare_item<HEAD_GATE>(a, e[0], e[1], h, prep.ws + (size_t)i * kDeltaItemBytes, lds);
}

}  // namespace

hipError_t launch_delta_chunks(const DeltaArgs &a, const DeltaSegment &scan,
                               const DeltaSegment &prep, bool head_gate, hipStream_t st) {
    const dim3 grid((unsigned)(scan.seqs * a.H * 2 + prep.chunks * a.H));
    if (head_gate)
        hipLaunchKernelGGL(delta_chunk_kernel<true>, grid, dim3(256), kDeltaLds, st, a, scan, prep);
    else
        hipLaunchKernelGGL(delta_chunk_kernel<false>, grid, dim3(256), kDeltaLds, st, a, scan,
                           prep);
    return hipGetLastError();
}

hipError_t allow_delta_lds() {
    const auto attr = hipFuncAttributeMaxDynamicSharedMemorySize;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(&delta_chunk_kernel<true>), attr, kDeltaLds);
    if (e != hipSuccess) return e;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(&delta_chunk_kernel<false>), attr,
                               kDeltaLds);
}

}  // namespace tp1
