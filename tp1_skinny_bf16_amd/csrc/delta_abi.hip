// delta_abi.hip -- the entry points of the gated delta rule: argument checks,
// the plan of a batch of prompts, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <vector>

#include "../../include/tp1_proj.h"
#include "args.hpp"
#include "delta.hpp"

struct proj_delta_plan_s {
    int H = 0, Hk = 0, n = 0, n_slots = 0, device = -1, cus = 256;
    long rows = 0;               // of all sequences together
    unsigned flags = 0;
    int *table = nullptr;        // device: {first row, rows, slot} a sequence
};

namespace tp1 {
namespace {

// Checks of what both forms take; fills `a`.  `rows`: rows the call reads.
int check_io(const proj_delta_io_t *io, int H, int Hk, long rows, int n_slots, DeltaArgs *a) {
    if (!io || H < 1 || H > PROJ_DELTA_MAX_HEADS || Hk < 1 || H % Hk != 0 || n_slots < 1)
        return PROJ_EINVAL;
    if (io->head_gate != 0 && io->head_gate != 1) return PROJ_EINVAL;
    const long wq = (long)Hk * kHead, wv = (long)H * kHead, wf = io->head_gate ? H : wv;
    *a = DeltaArgs{static_cast<const uint16_t *>(io->q), static_cast<const uint16_t *>(io->k),
                   static_cast<const uint16_t *>(io->v), static_cast<const uint16_t *>(io->f),
                   static_cast<const uint16_t *>(io->b), io->ldq ? io->ldq : wq,
                   io->ldk ? io->ldk : wq, io->ldv ? io->ldv : wv, io->ldf ? io->ldf : wf,
                   io->ldb ? io->ldb : (long)H, static_cast<const float *>(io->a_log),
                   static_cast<const float *>(io->dt_bias), static_cast<float *>(io->state),
                   static_cast<uint16_t *>(io->out), io->ldo ? io->ldo : wv, io->scale,
                   io->l2norm != 0, H, H / Hk, n_slots};
    if (a->ldq < wq || a->ldk < wq || a->ldv < wv || a->ldf < wf || a->ldb < H || a->ldo < wv)
        return PROJ_EINVAL;
    if (rows == 0) return PROJ_OK;
    if (!a->q || !a->k || !a->v || !a->f || !a->b || !a->a_log || !a->dt_bias || !a->state ||
        !a->out)
        return PROJ_EINVAL;
    if (!is_aligned(a->q, 16) || !is_aligned(a->k, 16) || !is_aligned(a->v, 16) ||
        !is_aligned(a->state, 16) || !is_aligned(a->out, 16) || a->ldq % 8 || a->ldk % 8 ||
        a->ldv % 8 || a->ldo % 8 || !is_aligned(a->a_log, 4) || !is_aligned(a->dt_bias, 16) ||
        !is_aligned(a->b, 2) || !is_aligned(a->f, io->head_gate ? 2 : 16) ||
        (!io->head_gate && a->ldf % 8))
        return PROJ_EALIGN;
    const Span out(a->out, span_bytes(rows, wv * 2, a->ldo * 2));
    const Span state(a->state, (size_t)n_slots * H * kHead * kHead * 4);
    const Span in[] = {Span(a->q, span_bytes(rows, wq * 2, a->ldq * 2)),
                       Span(a->k, span_bytes(rows, wq * 2, a->ldk * 2)),
                       Span(a->v, span_bytes(rows, wv * 2, a->ldv * 2)),
                       Span(a->f, span_bytes(rows, wf * 2, a->ldf * 2)),
                       Span(a->b, span_bytes(rows, (size_t)H * 2, a->ldb * 2)),
                       Span(a->a_log, (size_t)H * 4), Span(a->dt_bias, (size_t)wf * 4)};
    if (out.meets(state)) return PROJ_EINVAL;
    for (const Span &s : in)
        if (out.meets(s) || state.meets(s)) return PROJ_EINVAL;
    return PROJ_OK;
}

}  // namespace
}  // namespace tp1

extern "C" {

int proj_delta_step(const proj_delta_io_t *io, int heads, int qk_heads, int requests, int tokens,
                    const void *slots, int n_slots, void *stream) {
    using namespace tp1;
    if (requests < 0 || requests > PROJ_DELTA_MAX_REQUESTS || tokens < 1 ||
        tokens > PROJ_DELTA_MAX_TOKENS)
        return PROJ_EINVAL;
    DeltaArgs a;
    const int rc = check_io(io, heads, qk_heads, (long)requests * tokens, n_slots, &a);
    if (rc != PROJ_OK) return rc;
    if (requests == 0) return PROJ_OK;
    if (!slots) return PROJ_EINVAL;
    if (!is_aligned(slots, 4)) return PROJ_EALIGN;
    const Span index(slots, (size_t)requests * 4);
    if (index.meets(Span(a.out, span_bytes((size_t)requests * tokens, (size_t)heads * kHead * 2,
                                           a.ldo * 2))) ||
        index.meets(Span(a.state, (size_t)n_slots * heads * kHead * kHead * 4)))
        return PROJ_EINVAL;
    int dev = -1, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    const DeltaSeqs s{nullptr, static_cast<const int *>(slots), tokens, requests};
    if (launch_delta_steps(a, s, io->head_gate, cus > 0 ? cus : 256,
                           static_cast<hipStream_t>(stream)) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}

int proj_delta_plan(int heads, int qk_heads, int n, const int *lens, const int *slots,
                    int n_slots, unsigned flags, proj_delta_plan_t **out) {
    using namespace tp1;
    if (!out) return PROJ_EINVAL;
    *out = nullptr;
    if (heads < 1 || heads > PROJ_DELTA_MAX_HEADS || qk_heads < 1 || heads % qk_heads != 0 ||
        n < 1 || n > PROJ_DELTA_MAX_REQUESTS || n_slots < 1 || !lens || !slots ||
        (flags & ~PROJ_PLAN_HOST_ONLY))
        return PROJ_EINVAL;
    long rows = 0;
    for (int i = 0; i < n; ++i) {
        if (lens[i] < 0 || slots[i] < 0 || slots[i] >= n_slots) return PROJ_EINVAL;
        rows += lens[i];
        for (int j = 0; j < i; ++j)
            if (slots[j] == slots[i]) return PROJ_EINVAL;  // one state, one sequence
    }
    if (rows > PROJ_DELTA_MAX_ROWS) return PROJ_EINVAL;
    proj_delta_plan_s *p = new (std::nothrow) proj_delta_plan_s;
    int *host = new (std::nothrow) int[3 * (size_t)n];
    if (!p || !host) {
        delete p;
        delete[] host;
        return PROJ_ENOMEM;
    }
    p->H = heads;
    p->Hk = qk_heads;
    p->n = n;
    p->n_slots = n_slots;
    p->rows = rows;
    p->flags = flags;
    long r = 0;
    for (int i = 0; i < n; ++i) {
        host[3 * i] = (int)r;
        host[3 * i + 1] = lens[i];
        host[3 * i + 2] = slots[i];
        r += lens[i];
    }
    int rc = PROJ_OK;
    if (!(flags & PROJ_PLAN_HOST_ONLY)) {
        int dev = -1, cus = 0;
        void *mem = nullptr;
        const size_t bytes = 3 * (size_t)n * sizeof(int);
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            rc = PROJ_EHIP;
        else if (hipMalloc(&mem, bytes) != hipSuccess)
            rc = PROJ_ENOMEM;
        else if (hipMemcpy(mem, host, bytes, hipMemcpyHostToDevice) != hipSuccess)
            rc = PROJ_EHIP;
        if (rc != PROJ_OK) {
            (void)hipGetLastError();
            if (mem) (void)hipFree(mem);
        } else {
            p->device = dev;
            if (cus > 0) p->cus = cus;
            p->table = static_cast<int *>(mem);
        }
    }
    delete[] host;
    if (rc != PROJ_OK) {
        delete p;
        return rc;
    }
    *out = p;
    return PROJ_OK;
}

void proj_delta_free(proj_delta_plan_t *p) {
    if (!p) return;
    if (p->table) {
        int cur = -1;
        const bool other = hipGetDevice(&cur) == hipSuccess && cur != p->device;
        if (other) (void)hipSetDevice(p->device);
        (void)hipFree(p->table);
        if (other) (void)hipSetDevice(cur);
    }
    delete p;
}

long proj_delta_plan_rows(const proj_delta_plan_t *p) { return p ? p->rows : 0; }

int proj_delta_run(const proj_delta_plan_t *p, const proj_delta_io_t *io, void *stream) {
    using namespace tp1;
    if (!p) return PROJ_EINVAL;
    DeltaArgs a;
    const int rc = check_io(io, p->H, p->Hk, p->rows, p->n_slots, &a);
    if (rc != PROJ_OK) return rc;
    if (p->rows == 0) return PROJ_OK;
    if (p->flags & PROJ_PLAN_HOST_ONLY) return PROJ_ENODEV;
    int cur = -1;
    if (hipGetDevice(&cur) != hipSuccess || cur != p->device) return PROJ_EINVAL;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const DeltaSeqs s{p->table, nullptr, 0, p->n};
    if (launch_delta_steps(a, s, io->head_gate, p->cus, st) != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}

}  // extern "C"
