// delta_abi.hip -- the entry points of the gated delta rule: argument checks,
// the plan of a batch of prompts, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "../../include/tp1_proj.h"
#include "args.hpp"
#include "delta.hpp"

struct proj_delta_plan_s {
    int H = 0, Hk = 0, n = 0, n_slots = 0, device = -1, cus = 256;
    long rows = 0;               // of all sequences together
    unsigned flags = 0;
    int shorts = 0;              // sequences that run token by token
    std::vector<tp1::DeltaSegment> segments;
    void *mem = nullptr;         // device: tables, then two workspaces
    const int *seq_table = nullptr;    // all sequences
    const int *short_table = nullptr;  // those that always run token by token
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

// Sequences of at most this many rows run token by token, unless they are
// few beside the others' chunks: a chunk costs about as much however few of
// its 64 tokens there are (20 us for all in one launch), a launch of the
// recurrent kernel beside the chunks' 5 us and more.
constexpr int kShortRows = 16;

// Chunks and heads a segment prepares at a time, by the heads at work on
// average.  Many: the launches' ragged ends cost, so few and large segments
// (8192 tokens of 96 heads: 902 us, 923 with 2048 and 970 with 1024; two
// workspaces of 440 MB).  Few: the scan's chain takes longer than the
// preparation, of which only the first segment's is not hidden (24 heads: 327
// us, 344 with 2048, 388 with 4096; 40 heads: 478, 464 and 522).
long segment_items(long busy) { return busy <= 32 ? 1024 : busy <= 64 ? 2048 : 4096; }

struct Tables {
    std::vector<int> words;                 // every table, one after another
    std::vector<tp1::DeltaSegment> segments;
    std::vector<size_t> chunk_at, seq_at;   // where a segment's tables start
    int shorts = 0, most = 0;               // most chunks of a segment
};

// Cuts the sequences' chunks into segments, first chunks of all sequences
// first, so that every segment carries many sequences on.
Tables cut(int H, int n, const int *lens, const int *slots) {
    Tables t;
    std::vector<long> row(n);
    long r = 0;
    for (int i = 0; i < n; ++i) {
        row[i] = r;
        r += lens[i];
        t.words.insert(t.words.end(), {(int)row[i], lens[i], slots[i]});
    }
    long shorts = 0, chunks = 0, longest = 1;
    for (int i = 0; i < n; ++i) {
        const long c = (lens[i] + (long)kDeltaChunk - 1) / kDeltaChunk;
        if (lens[i] > kShortRows) {
            chunks += c;
            longest = std::max(longest, c);
        } else if (lens[i] > 0) {
            ++shorts;
        }
    }
    const int shortest = shorts * 4 <= chunks ? 1 : kShortRows + 1;  // rows that make a chunk
    for (int i = 0; i < n; ++i)
        if (lens[i] > 0 && lens[i] < shortest) {
            t.words.insert(t.words.end(), {(int)row[i], lens[i], slots[i]});
            ++t.shorts;
        }
    // segments of one size: a small last one would leave the scan before it
    // without preparations to run beside
    if (shortest == 1) chunks += shorts;
    const double items = (double)chunks * H;
    const long parts =
        std::max(1L, std::lround(items / segment_items(chunks * H / longest)));
    const int per = (int)std::max(1L, (chunks + parts - 1) / parts);
    struct Chunk {
        int seq, at;
    };
    std::vector<Chunk> seg;
    auto close = [&]() {
        if (seg.empty()) return;
        std::stable_sort(seg.begin(), seg.end(),
                         [](const Chunk &x, const Chunk &y) { return x.seq < y.seq; });
        DeltaSegment s{};
        s.chunks = (int)seg.size();
        t.chunk_at.push_back(t.words.size());
        for (const Chunk &c : seg) {
            t.words.push_back((int)(row[c.seq] + (long)c.at * kDeltaChunk));
            t.words.push_back(std::min(kDeltaChunk, lens[c.seq] - c.at * kDeltaChunk));
        }
        t.seq_at.push_back(t.words.size());
        std::vector<std::pair<int, int>> runs;  // chunks of one sequence: {first, how many}
        for (size_t i = 0; i < seg.size();) {
            size_t j = i;
            while (j < seg.size() && seg[j].seq == seg[i].seq) ++j;
            runs.push_back({(int)i, (int)(j - i)});
            i = j;
        }
        // the longest first: whatever has to wait for a compute unit is short
        std::stable_sort(runs.begin(), runs.end(), [](const auto &x, const auto &y) {
            return x.second > y.second;
        });
        for (const auto &[i, m] : runs) {
            const Chunk &a = seg[i], &b = seg[i + m - 1];
            const int end = std::min(lens[a.seq], (b.at + 1) * kDeltaChunk);
            t.words.insert(t.words.end(), {(int)(row[a.seq] + (long)a.at * kDeltaChunk),
                                           end - a.at * kDeltaChunk, slots[a.seq], i});
        }
        s.seqs = (int)runs.size();
        s.longest = runs[0].second;
        t.most = std::max(t.most, s.chunks);
        t.segments.push_back(s);
        seg.clear();
    };
    std::vector<int> left;                  // sequences with chunks still to place
    for (int i = 0; i < n; ++i)
        if (lens[i] >= shortest) left.push_back(i);
    for (int at = 0; !left.empty(); ++at) {
        size_t keep = 0;
        for (const int i : left) {
            seg.push_back({i, at});
            if ((int)seg.size() == per) close();
            if (lens[i] - at * kDeltaChunk > kDeltaChunk) left[keep++] = i;
        }
        left.resize(keep);
    }
    close();
    return t;
}

int prepare_delta(int dev) {
    static std::mutex mu;
    static bool done[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev]) return PROJ_OK;
    if (allow_delta_lds() != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    if (dev >= 0 && dev < 64) done[dev] = true;
    return PROJ_OK;
}

// Tables and two workspaces on the current device.
int place(proj_delta_plan_s *p, Tables &t) {
    int dev = -1, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return PROJ_EHIP;
    p->device = dev;
    if (cus > 0) p->cus = cus;
    const int rc = prepare_delta(dev);
    if (rc != PROJ_OK) return rc;
    const size_t words = t.words.size() * sizeof(int);
    const size_t tables = (words + 255) / 256 * 256;
    const size_t ws = (size_t)t.most * p->H * kDeltaItemBytes;
    const size_t bytes = tables + ws * std::min<size_t>(2, t.segments.size());
    if (bytes == 0) return PROJ_OK;
    if (hipMalloc(&p->mem, bytes) != hipSuccess) {
        p->mem = nullptr;
        return PROJ_ENOMEM;
    }
    if (hipMemcpy(p->mem, t.words.data(), words, hipMemcpyHostToDevice) != hipSuccess)
        return PROJ_EHIP;
    const int *w = static_cast<const int *>(p->mem);
    p->shorts = t.shorts;
    p->seq_table = w;
    p->short_table = w + 3 * (size_t)p->n;
    for (size_t i = 0; i < t.segments.size(); ++i) {
        t.segments[i].chunk_table = w + t.chunk_at[i];
        t.segments[i].seq_table = w + t.seq_at[i];
        t.segments[i].ws = static_cast<char *>(p->mem) + tables + (i & 1) * ws;
    }
    p->segments.swap(t.segments);
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
    proj_delta_plan_s *p = nullptr;
    int rc = PROJ_OK;
    try {
        p = new proj_delta_plan_s;
        p->H = heads;
        p->Hk = qk_heads;
        p->n = n;
        p->n_slots = n_slots;
        p->rows = rows;
        p->flags = flags;
        if (!(flags & PROJ_PLAN_HOST_ONLY)) {
            Tables t = cut(heads, n, lens, slots);
            rc = place(p, t);
        }
    } catch (const std::bad_alloc &) {
        rc = PROJ_ENOMEM;
    }
    if (rc != PROJ_OK) {
        (void)hipGetLastError();
        proj_delta_free(p);
        return rc;
    }
    *out = p;
    return PROJ_OK;
}

void proj_delta_free(proj_delta_plan_t *p) {
    if (!p) return;
    if (p->mem) {
        int cur = -1;
        const bool other = hipGetDevice(&cur) == hipSuccess && cur != p->device;
        if (other) (void)hipSetDevice(p->device);
        (void)hipFree(p->mem);
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
    hipError_t e = hipSuccess;
    if (!a.l2norm) {
        const DeltaSeqs s{p->seq_table, nullptr, 0, p->n};
        e = launch_delta_steps(a, s, io->head_gate, p->cus, st);
        if (e == hipSuccess) return PROJ_OK;
    } else if (p->shorts) {
        const DeltaSeqs s{p->short_table, nullptr, 0, p->shorts};
        e = launch_delta_steps(a, s, io->head_gate, p->cus, st);
    }
    // segment i's scan shares a launch with segment i + 1's preparation
    const size_t n = p->segments.size();
    for (size_t i = 0; n && i <= n && e == hipSuccess; ++i) {
        const DeltaSegment none{};
        const DeltaSegment &scan = i ? p->segments[i - 1] : none;
        const DeltaSegment &prep = i < n ? p->segments[i] : none;
        e = launch_delta_chunks(a, scan, prep, io->head_gate, p->cus, st);
    }
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return PROJ_EHIP;
    }
    return PROJ_OK;
}

}  // extern "C"
