// delta_step.hip -- the gated delta rule, token by token.
//
// A head's state is a matrix S[key][value] (128 x 128, FP32).  A token with
// key k, query q, value v, decay a (a channel of the key, or a head) and
// strength beta does
//     S <- diag(a) S
//     u  = beta * (v - S^T k)
//     S <- S + k u^T
//     o  = S^T q = (diag(a) S)^T q + (k . q) u
// The second form of o lets one pass over the decayed state give both inner
// products, so a token costs one reduction over the key axis.
//
// For single tokens everything is the state: 64 KiB read and 64 KiB written
// a head, against 1.3 KiB of inputs, so HBM bounds it: 64 requests of 96
// heads take 141 us, 5.8 TB/s, where scaling a tensor of that size in place
// runs at 6.0.  A workgroup of 256 threads holds VC columns of one head's
// state in registers (all its loads issued before anything else), each
// thread 4 neighbouring columns of VC / 8 rows; the columns of a head are
// independent, so a head is split over 128 / VC workgroups.  The state's
// loads and stores are non-temporal (153 us without): the next step's come a
// whole model later.  The key axis is
// summed in the thread, across the lanes of a wave, then across the four
// waves through LDS in a fixed order.
// One barrier a token: the vectors (q, k, a) of the token after the next are
// made between barriers by waves 0 and 1, in one of three buffers.
#include "delta.hpp"

#include "device.hpp"

namespace tp1 {

namespace {

template <int VC, bool HEAD_GATE>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaArgs a, DeltaSeqs sq) {
    constexpr int VQ = VC / 4;        // lanes along the columns
    constexpr int KQ = 256 / VQ;      // threads along the keys
    constexpr int RT = kHead / KQ;    // key rows a thread
    __shared__ float vec[3][3][kHead];       // q, k, a of a token
    __shared__ float kq_dot[3];
    __shared__ f32x4 red[2][2][4][VQ];       // [parity][S^T k, S^T q][wave]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = scalar(tid >> 6);
    const int vq = tid % VQ, kq = tid / VQ;
    const int h = blockIdx.x / (kHead / VC);
    const int c0 = (blockIdx.x % (kHead / VC)) * VC + vq * 4;  // first column of this thread
    const int hk = h / a.rep;
    int i = blockIdx.y;
    const int slot = scalar(sq.table ? sq.table[3 * i + 2] : sq.slots[i]);
    if (slot < 0 || slot >= a.n_slots) {  // no state: padding of the batch
        if (kq == 0)
            for (int t = 0; t < sq.tokens; ++t)
                *reinterpret_cast<u32x2 *>(a.out + (size_t)(i * (long)sq.tokens + t) * a.ldo +
                                           h * kHead + c0) = u32x2{0u, 0u};
        return;
    }
    float *state = a.state + ((size_t)slot * a.H + h) * (kHead * kHead) + c0;
    f32x4 S[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        S[r] = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4 *>(state + (size_t)(kq + KQ * r) * kHead));

    // Requests that name one slot are taken in order by the first of them.
    bool shared = false;
    if (!sq.table) {
        bool any = false;
        for (int j = tid; j < sq.n; j += 256) any |= j != i && sq.slots[j] == slot;
        shared = __syncthreads_or(any);
        if (shared)
            for (int j = 0; j < i; ++j)
                if (sq.slots[j] == slot) return;
    }

    const float rate = expf(a.a_log[h]);
    for (;;) {
        const long row0 = sq.table ? sq.table[3 * i] : (long)i * sq.tokens;
        const int T = sq.table ? sq.table[3 * i + 1] : sq.tokens;
        auto prepare = [&](int t) {
            const long row = row0 + t;
            const int s = t % 3;
            if (wave == 0) {
                const unsigned qv = *reinterpret_cast<const unsigned *>(a.q + row * a.ldq +
                                                                        hk * kHead + lane * 2);
                const unsigned kv = *reinterpret_cast<const unsigned *>(a.k + row * a.ldk +
                                                                        hk * kHead + lane * 2);
                float q0 = bf16_lo(qv), q1 = bf16_hi(qv), k0 = bf16_lo(kv), k1 = bf16_hi(kv);
                float rq = a.scale, rk = 1.f;
                if (a.l2norm) {
                    rq *= rsqrtf(sum64(__builtin_fmaf(q0, q0, q1 * q1)) + kUnitEps);
                    rk = rsqrtf(sum64(__builtin_fmaf(k0, k0, k1 * k1)) + kUnitEps);
                }
                q0 *= rq, q1 *= rq, k0 *= rk, k1 *= rk;
                vec[s][0][2 * lane] = q0;
                vec[s][0][2 * lane + 1] = q1;
                vec[s][1][2 * lane] = k0;
                vec[s][1][2 * lane + 1] = k1;
                const float d = sum64(__builtin_fmaf(q0, k0, q1 * k1));
                if (lane == 0) kq_dot[s] = d;
            } else if (wave == 1) {
                if constexpr (HEAD_GATE) {
                    const float g =
                        expf(log_decay(rate, bf16_value(a.f[row * a.ldf + h]), a.dt_bias[h]));
                    vec[s][2][2 * lane] = g;
                    vec[s][2][2 * lane + 1] = g;
                } else {
                    const unsigned fv = *reinterpret_cast<const unsigned *>(
                        a.f + row * a.ldf + h * kHead + lane * 2);
                    const float *bias = a.dt_bias + h * kHead + lane * 2;
                    vec[s][2][2 * lane] = expf(log_decay(rate, bf16_lo(fv), bias[0]));
                    vec[s][2][2 * lane + 1] = expf(log_decay(rate, bf16_hi(fv), bias[1]));
                }
            }
        };
        __syncthreads();  // the buffers of the sequence before are free
        if (T > 0) prepare(0);
        __syncthreads();
        for (int t = 0; t < T; ++t) {
            const long row = row0 + t;
            const int s = t % 3;
            const u32x2 vv = *reinterpret_cast<const u32x2 *>(a.v + row * a.ldv + h * kHead + c0);
            const float beta = sigmoid(bf16_value(a.b[row * a.ldb + h]));
            f32x4 dk = {0.f, 0.f, 0.f, 0.f}, dq = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int key = kq + KQ * r;
                const float g = vec[s][2][key], kk = vec[s][1][key], qq = vec[s][0][key];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    S[r][c] *= g;
                    dk[c] = __builtin_fmaf(S[r][c], kk, dk[c]);
                    dq[c] = __builtin_fmaf(S[r][c], qq, dq[c]);
                }
            }
#pragma unroll
            for (int o = VQ; o < 64; o <<= 1)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    dk[c] += __shfl_xor(dk[c], o);
                    dq[c] += __shfl_xor(dq[c], o);
                }
            if (lane < VQ) {
                red[t & 1][0][wave][lane] = dk;
                red[t & 1][1][wave][lane] = dq;
            }
            if (t + 1 < T) prepare(t + 1);
            __syncthreads();
            f32x4 sk = red[t & 1][0][0][vq], sv = red[t & 1][1][0][vq];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                const f32x4 x = red[t & 1][0][w][vq], y = red[t & 1][1][w][vq];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sk[c] += x[c];
                    sv[c] += y[c];
                }
            }
            const float vf[4] = {bf16_lo(vv.x), bf16_hi(vv.x), bf16_lo(vv.y), bf16_hi(vv.y)};
            float u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] = beta * (vf[c] - sk[c]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float kk = vec[s][1][kq + KQ * r];
#pragma unroll
                for (int c = 0; c < 4; ++c) S[r][c] = __builtin_fmaf(kk, u[c], S[r][c]);
            }
            if (kq == 0) {
                const float d = kq_dot[s];
                float o[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(d, u[c], sv[c]);
                *reinterpret_cast<u32x2 *>(a.out + row * a.ldo + h * kHead + c0) =
                    u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
            }
        }
        if (!shared) break;
        do ++i;
        while (i < sq.n && sq.slots[i] != slot);
        if (i >= sq.n) break;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
        __builtin_nontemporal_store(
            S[r], reinterpret_cast<f32x4 *>(state + (size_t)(kq + KQ * r) * kHead));
}

template <int VC>
hipError_t launch_vc(const DeltaArgs &a, const DeltaSeqs &s, bool head_gate, hipStream_t st) {
    const dim3 grid((unsigned)(a.H * (kHead / VC)), (unsigned)s.n);
    if (head_gate)
        hipLaunchKernelGGL((delta_step_kernel<VC, true>), grid, dim3(256), 0, st, a, s);
    else
        hipLaunchKernelGGL((delta_step_kernel<VC, false>), grid, dim3(256), 0, st, a, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_steps(const DeltaArgs &a, const DeltaSeqs &s, bool head_gate, int cus,
                              hipStream_t st) {
    // 64 columns a workgroup, 32 while those are fewer than half the compute
    // units: 5.8 us against 5.9 at 96 heads in all (one request), 4.4 against
    // 4.8 at 12; but 23.7 against 20.8 at 768 and 41.1 against 38.6 at 1536
    if ((long)a.H * s.n * 2 >= cus) return launch_vc<64>(a, s, head_gate, st);
    return launch_vc<32>(a, s, head_gate, st);
}

}  // namespace tp1
