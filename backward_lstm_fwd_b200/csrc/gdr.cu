// gdr.cu -- C ABI of the gated delta rule (declared in include/liblstm.h):
// argument checks, workspace layout and the launches of gdr.cuh's kernels.
#include <algorithm>
#include <climits>

#include "gdr.cuh"

using namespace lstm;
using namespace lstm::gdr;

namespace {

bool dims_ok(const lstm_gdr_dims *d) {
    if (!d || d->T < 0 || d->B < 0 || d->Hk < 0 || d->Hv < 0 || d->K < 0 || d->V < 0) return false;
    if (!host::dtype_ok(d->dtype)) return false;
    if ((d->Hk == 0) != (d->Hv == 0) || (d->Hk > 0 && d->Hv % d->Hk != 0)) return false;
    // every row count fits an int
    return (long long)d->T * d->B <= INT_MAX && (long long)d->Hv * std::max(d->K, d->V) <= INT_MAX;
}

long long or_dense(long long ld, long long dense) { return ld ? ld : dense; }

int strides_check(const lstm_gdr_dims *d) {
    const long long q = or_dense(d->ldq, (long long)d->Hk * d->K), k = or_dense(d->ldk, (long long)d->Hk * d->K),
                    v = or_dense(d->ldv, (long long)d->Hv * d->V);
    if (q < (long long)d->Hk * d->K || k < (long long)d->Hk * d->K || v < (long long)d->Hv * d->V) return LSTM_ERR_INVALID_ARG;
    return LSTM_OK;
}

bool dims_supported(const lstm_gdr_dims *d) {
    if (d->K % 8 || d->V % 8 || d->K > 128 || d->V > 256 || d->T > INT_MAX - C) return false;
    if (or_dense(d->ldq, 0) % 8 || or_dense(d->ldk, 0) % 8 || or_dense(d->ldv, 0) % 8) return false;
    const long long nc = (d->T + C - 1) / C;
    return (long long)d->B * d->Hv * 4 <= INT_MAX && nc * d->B * std::max(d->Hk, d->Hv) <= INT_MAX;
}

int check(const lstm_gdr_dims *d) {
    if (!dims_ok(d)) return LSTM_ERR_INVALID_ARG;
    const int rc = strides_check(d);
    if (rc != LSTM_OK) return rc;
    return dims_supported(d) ? LSTM_OK : LSTM_ERR_UNSUPPORTED;
}

// Token by token or in chunks.  Measured for K = V = 128, us token by token /
// in chunks at 8, 16 and 24 tokens: 4 heads 10 / 18, 18 / 18, 26 / 18; 128
// heads 14 / 20, 24 / 19, 34 / 19; 1024 heads 66 / 105, 121 / 107, 178 / 109.
bool stepwise(const lstm_gdr_dims *d, bool save) { return !save && d->T <= LSTM_GDR_STEP_TOKENS; }

int terms_of(int dtype) { return dtype == LSTM_BF16 ? 1 : dtype == LSTM_F16 ? 2 : 3; }

// Segments of the chunk sequence (see SeqArgs): the number with the lowest
// estimate, from weights of a chunk of a pass that writes its outputs (4.0; it
// takes 5.1 us, 7.1 with the states), of one that does not (3.2; 4.1 us), of a
// joined segment (3.0; about 4 us) and of two more launches (8); 1 where
// splitting gains less than a tenth.  Measured for K = V = 128, bf16, us of a
// forward whole / split, heads x chunks: 4 x 8 53 / 56, 4 x 128 571 / 161, 16 x 32
// 166 / 106, 32 x 16 99 / 94, 64 x 32 225 / 229, 128 x 16 164 / 213; of a forward
// that keeps its states and its backward: 4 x 128 1548 / 409, 32 x 16 303 / 268, 64 x
// 32 734 / 720.  Of 4 to 128 heads and 8 to 128 chunks the choice is within 4 % of
// the best, but for 32 x 64 (302, where three segments take 278).
struct Split {
    int segments, chunks;
};
Split split_of(const lstm_gdr_dims *d) {
    const int nc = (d->T + C - 1) / C, sms = host::sm_count();
    const long long heads = (long long)d->B * d->Hv, vt = (d->V + LANES - 1) / LANES;
    auto waves = [&](long long blocks) { return (double)((blocks + sms - 1) / sms); };
    Split best = {1, std::max(nc, 1)};
    double cost = 0.9 * waves(heads * vt) * nc * 4.0;
    if (heads * vt > sms) return best;
    for (int n = 2; n <= 32 && 2 * n <= nc; ++n) {
        const int len = (nc + n - 1) / n, segs = (nc + len - 1) / len;
        if (segs < 2) continue;
        const long long scan = (segs - 1) * heads * (vt + 1) - heads;
        const double t = waves(scan) * len * 3.2 + (segs - 2) * 3.0 + waves(segs * heads * vt) * len * 4.0 + 8.0;
        if (t < cost) {
            cost = t;
            best = {segs, len};
        }
    }
    return best;
}

// Value heads that a block of the gradient kernel takes: the group of a key
// head, one after another, or one where a block a key head would leave more than
// half the SMs idle, with a sum of the parts more (T = 333, 3 sequences, 2 key
// heads of 3 value heads: 55 us against 25 + 5).
int heads_per_block(const lstm_gdr_dims *d) {
    const long long blocks = (long long)((d->T + C - 1) / C) * d->B * d->Hk;
    return 2 * blocks <= host::sm_count() ? 1 : d->Hv / std::max(d->Hk, 1);
}

struct Layout {
    size_t qk, tp, starts, first, trans, dstates, dvf, parts, total;
    Split split;
};
Layout layout(const lstm_gdr_dims *d, bool bwd) {
    Layout l;
    const size_t nc = (d->T + C - 1) / C, kd = d->K <= 64 ? 64 : 128;
    l.split = split_of(d);
    const size_t joints = (size_t)(l.split.segments - 1) * d->B * d->Hv;
    size_t o = kCtrlBytes;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    l.qk = take(nc * d->B * d->Hk * (terms_of(d->dtype) * kd * 256));
    l.tp = take(nc * d->B * d->Hv * (size_t)TP_BYTES);
    l.starts = take(joints * d->K * d->V * 4);
    l.first = take(joints ? (size_t)d->B * d->Hv * d->K * d->V * 4 : 0);  // a copy of the start, where the end replaces it
    l.trans = take(joints * (NT * kd * kd * 2));
    l.dstates = bwd ? take(nc * d->B * d->Hv * (size_t)d->K * d->V * 4) : 0;
    l.dvf = bwd ? take((size_t)d->T * d->B * d->Hv * d->V * 4) : 0;
    const int heads = heads_per_block(d);
    l.parts = bwd && d->Hk && d->Hv / d->Hk > heads ? take((size_t)(d->Hv / d->Hk) * 2 * d->T * d->B * d->Hk * d->K * 4) : 0;
    l.total = o;
    return l;
}

Shape shape_of(const lstm_gdr_dims *d, const lstm_gdr_options *opt) {
    Shape s = {};
    s.T = d->T;
    s.B = d->B;
    s.Hk = d->Hk;
    s.Hv = d->Hv;
    s.K = d->K;
    s.V = d->V;
    s.group = d->Hk ? d->Hv / d->Hk : 0;
    s.NC = (d->T + C - 1) / C;
    s.VT = (d->V + LANES - 1) / LANES;
    s.ldq = or_dense(d->ldq, (long long)d->Hk * d->K);
    s.ldk = or_dense(d->ldk, (long long)d->Hk * d->K);
    s.ldv = or_dense(d->ldv, (long long)d->Hv * d->V);
    s.scale = opt ? opt->scale : 1.0f;
    s.lengths = opt ? opt->lengths : nullptr;
    return s;
}

// (The attribute belongs to the function on the current device.)
template <class Kern> cudaError_t allow_smem(Kern kern, size_t bytes) {
    return cudaFuncSetAttribute((const void *)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <class E, int KD>
int prep(const Shape &s, const void *q, const void *k, const float *g, const float *beta, char *w, const Layout &l,
         cudaStream_t st) {
    const int blocks = s.NC * s.B * s.Hk;
    // A block a value head where blocks are few, though each makes the tiles again: us of a forward, a block
    // a value head / a key head: 36 blocks of key heads 45 / 57, 256 105 / 111, 512 100 / 97, 2048 279 / 267.
    const int heads = blocks <= 2 * host::sm_count() ? 1 : s.group;
    PrepArgs p = {s, q, k, g, beta, w + l.qk, w + l.tp, (Ctrl *)w, heads};
    LSTM_CUDA_TRY(allow_smem(prep_kernel<E, KD>, PrepSmem<E, KD>::smem));
    prep_kernel<E, KD><<<blocks * (s.group / heads), 128, PrepSmem<E, KD>::smem, st>>>(p);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

// The chunks in order, by segments where the split says so.
template <int KD, class Kern> int sequential(SeqArgs a, float *first, Kern scan, Kern run, size_t smem, cudaStream_t st) {
    const int heads = a.s.B * a.s.Hv;
    if (a.segments > 1) {
        if (a.s0 && a.s0 == a.sT) {  // the last segment's block may end before the first one's begins
            LSTM_CUDA_TRY(cudaMemcpyAsync(first, a.s0, (size_t)heads * a.s.K * a.s.V * 4, cudaMemcpyDeviceToDevice, st));
            a.s0 = first;
        }
        LSTM_CUDA_TRY(allow_smem(scan, smem));
        scan<<<(a.segments - 1) * heads * (a.s.VT + 1), SEQ_THREADS, smem, st>>>(a);
        LSTM_CUDA_TRY(host::launched());
        if (a.segments > 2) {
            LSTM_CUDA_TRY(allow_smem(scan_kernel<KD>, ScanSmem<KD>::smem));
            scan_kernel<KD><<<heads * a.s.VT, SEQ_THREADS, ScanSmem<KD>::smem, st>>>(a);
            LSTM_CUDA_TRY(host::launched());
        }
    }
    LSTM_CUDA_TRY(allow_smem(run, smem));
    run<<<a.segments * heads * a.s.VT, SEQ_THREADS, smem, st>>>(a);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

template <class E, int KD>
int chunked_fwd(const Shape &s, const void *q, const void *k, const void *v, const float *g, const float *beta,
                const float *s0, void *o, float *sT, float *states, float *deltas, char *w, const Layout &l,
                cudaStream_t st) {
    if (s.NC > 0) {
        const int rc = prep<E, KD>(s, q, k, g, beta, w, l, st);
        if (rc != LSTM_OK) return rc;
    }
    SeqArgs a = {s, w + l.qk, w + l.tp, v, s0, o, sT, states, deltas, (float *)(w + l.starts), w + l.trans,
                 l.split.segments, l.split.chunks, (Ctrl *)w};
    return sequential<KD>(a, (float *)(w + l.first), seq_fwd_kernel<E, KD, true>, seq_fwd_kernel<E, KD, false>, Seq<E, KD>::smem, st);
}

template <class E>
int stepwise_fwd(const Shape &s, const void *q, const void *k, const void *v, const float *g, const float *beta,
                 const float *s0, void *o, float *sT, char *w, cudaStream_t st) {
    StepArgs a = {s, q, k, v, g, beta, s0, o, sT, (Ctrl *)w, (s.V + STEP_COLS - 1) / STEP_COLS};
    step_kernel<E><<<s.B * s.Hv * a.tiles, STEP_THREADS, 0, st>>>(a);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

template <class E>
int fwd(const lstm_gdr_dims *d, const Shape &s, const void *q, const void *k, const void *v, const float *g,
        const float *beta, const float *s0, void *o, float *sT, float *states, float *deltas, char *w,
        cudaStream_t st) {
    if (stepwise(d, states != nullptr)) return stepwise_fwd<E>(s, q, k, v, g, beta, s0, o, sT, w, st);
    const Layout l = layout(d, false);
    if (s.K <= 64) return chunked_fwd<E, 64>(s, q, k, v, g, beta, s0, o, sT, states, deltas, w, l, st);
    return chunked_fwd<E, 128>(s, q, k, v, g, beta, s0, o, sT, states, deltas, w, l, st);
}

template <class E, int KD>
int chunked_bwd(const lstm_gdr_dims *d, const Shape &s, const void *dout, const float *dsT, const void *q,
                const void *k, const float *g, const float *beta, const float *states, const float *deltas, void *dq,
                void *dk, void *dv, float *dg, float *dbeta, float *ds0, const char *kept, char *w, cudaStream_t st) {
    const Layout l = layout(d, true);
    if (kept) {  // the forward's layout begins alike
        LSTM_CUDA_TRY(cudaMemsetAsync(w, 0, kCtrlBytes, st));
    } else if (s.NC > 0) {
        const int rc = prep<E, KD>(s, q, k, g, beta, w, l, st);
        if (rc != LSTM_OK) return rc;
    }
    const char *tiles = kept ? kept : w;
    float *dstates = (float *)(w + l.dstates), *dvf = (float *)(w + l.dvf);
    SeqArgs a = {s, tiles + l.qk, tiles + l.tp, dout, dsT, dv, ds0, dstates, dvf, (float *)(w + l.starts), w + l.trans,
                 l.split.segments, l.split.chunks, (Ctrl *)w};
    const int rc = sequential<KD>(a, (float *)(w + l.first), seq_bwd_kernel<E, KD, true>, seq_bwd_kernel<E, KD, false>, Seq<E, KD>::smem, st);
    if (rc != LSTM_OK || s.NC == 0) return rc;
    GradArgs ga = {s, tiles + l.qk, g, beta, dout, states, deltas, dstates, dvf, dq, dk, dg, dbeta, (float *)(w + l.parts), (Ctrl *)w};
    constexpr size_t smem = GradSmem<E, KD>::smem;
    const int blocks = s.NC * s.B * s.Hk;
    if (heads_per_block(d) == s.group) {
        LSTM_CUDA_TRY(allow_smem(grad_kernel<E, KD, false>, smem));
        grad_kernel<E, KD, false><<<blocks, GRAD_THREADS, smem, st>>>(ga);
        LSTM_CUDA_TRY(host::launched());
        return LSTM_OK;
    }
    LSTM_CUDA_TRY(allow_smem(grad_kernel<E, KD, true>, smem));
    grad_kernel<E, KD, true><<<blocks * s.group, GRAD_THREADS, smem, st>>>(ga);
    LSTM_CUDA_TRY(host::launched());
    const long long n8 = (long long)s.T * s.B * s.Hk * s.K / 8;
    if (n8 == 0) return LSTM_OK;
    sum_kernel<E><<<(unsigned)((2 * n8 + 255) / 256), 256, 0, st>>>((const float *)(w + l.parts), s.group, n8, (E *)dq, (E *)dk);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

template <class E, class... A> int bwd(const lstm_gdr_dims *d, A... args) {
    return d->K <= 64 ? chunked_bwd<E, 64>(d, args...) : chunked_bwd<E, 128>(d, args...);
}

bool scale_ok(const lstm_gdr_options *opt) { return !opt || (opt->scale == opt->scale && opt->scale - opt->scale == 0.f); }

}  // namespace

extern "C" {

size_t lstm_gdr_fwd_workspace_size(const lstm_gdr_dims *d, int save) {
    if (check(d) != LSTM_OK) return 0;
    return stepwise(d, save != 0) ? kCtrlBytes : layout(d, false).total;
}

size_t lstm_gdr_bwd_workspace_size(const lstm_gdr_dims *d) {
    if (check(d) != LSTM_OK) return 0;
    return layout(d, true).total;
}

int lstm_gdr_fwd(const lstm_gdr_dims *d, const lstm_gdr_options *opt, const void *q, const void *k, const void *v,
                 const float *g, const float *beta, const float *s0, void *o, float *sT, float *states, float *deltas,
                 void *ws, size_t ws_bytes, void *stream) {
    int rc = check(d);
    if (rc != LSTM_OK) return rc;
    if (!scale_ok(opt)) return LSTM_ERR_INVALID_ARG;
    const long long rows = (long long)d->T * d->B * d->Hv;
    const bool any = rows > 0, state = (long long)d->B * d->Hv * d->K * d->V > 0;
    if (!host::ptr_ok(q, any && d->K) || !host::ptr_ok(k, any && d->K) || !host::ptr_ok(v, any && d->V) ||
        !host::ptr_ok(g, any, 4) || !host::ptr_ok(beta, any, 4) || !host::ptr_ok(s0, false) ||
        !host::ptr_ok(o, any && d->V) || !host::ptr_ok(sT, state) || !host::ptr_ok(states, false) ||
        !host::ptr_ok(deltas, false) || !host::ptr_ok(opt ? opt->lengths : nullptr, false, 4) ||
        (states != nullptr) != (deltas != nullptr))
        return LSTM_ERR_INVALID_ARG;
    if (ws || !stepwise(d, states != nullptr)) {
        rc = host::ws_check(ws, ws_bytes, lstm_gdr_fwd_workspace_size(d, states != nullptr));
        if (rc != LSTM_OK) return rc;
    }
    if ((long long)d->B * d->Hv * d->V == 0) return LSTM_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const Shape s = shape_of(d, opt);
    char *w = (char *)ws;
    if (d->dtype == LSTM_F32) return fwd<float>(d, s, q, k, v, g, beta, s0, o, sT, states, deltas, w, st);
    if (d->dtype == LSTM_F16) return fwd<f16>(d, s, q, k, v, g, beta, s0, o, sT, states, deltas, w, st);
    return fwd<bf16>(d, s, q, k, v, g, beta, s0, o, sT, states, deltas, w, st);
}

int lstm_gdr_bwd(const lstm_gdr_dims *d, const lstm_gdr_options *opt, const void *dout, const float *dsT, const void *q,
                 const void *k, const void *v, const float *g, const float *beta, const float *states,
                 const float *deltas, void *dq, void *dk, void *dv, float *dg, float *dbeta, float *ds0,
                 const void *fwd_ws, void *ws, size_t ws_bytes, void *stream) {
    int rc = check(d);
    if (rc != LSTM_OK) return rc;
    if (!scale_ok(opt)) return LSTM_ERR_INVALID_ARG;
    const long long rows = (long long)d->T * d->B * d->Hv;
    const bool any = rows > 0, state = any && d->K && d->V;
    if (!host::ptr_ok(dout, false) || !host::ptr_ok(dsT, false) || !host::ptr_ok(q, any && d->K) ||
        !host::ptr_ok(k, any && d->K) || !host::ptr_ok(v, false) || !host::ptr_ok(g, any, 4) ||
        !host::ptr_ok(beta, any, 4) || !host::ptr_ok(states, state) || !host::ptr_ok(deltas, any && d->V) ||
        !host::ptr_ok(dq, any && d->K) || !host::ptr_ok(dk, any && d->K) || !host::ptr_ok(dv, any && d->V) ||
        !host::ptr_ok(dg, any, 4) || !host::ptr_ok(dbeta, any, 4) || !host::ptr_ok(ds0, false) ||
        !host::ptr_ok(fwd_ws, false, 256) ||
        !host::ptr_ok(opt ? opt->lengths : nullptr, false, 4))
        return LSTM_ERR_INVALID_ARG;
    rc = host::ws_check(ws, ws_bytes, layout(d, true).total);
    if (rc != LSTM_OK) return rc;
    if ((long long)d->B * d->Hv == 0) return LSTM_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (d->V == 0) {  // no outputs depend on q, k, g and beta
        if (any) {
            if (d->K) {
                const size_t n = (size_t)d->T * d->B * d->Hk * d->K * host::elem_bytes(d->dtype);
                LSTM_CUDA_TRY(cudaMemsetAsync(dq, 0, n, st));
                LSTM_CUDA_TRY(cudaMemsetAsync(dk, 0, n, st));
            }
            LSTM_CUDA_TRY(cudaMemsetAsync(dg, 0, (size_t)rows * 4, st));
            LSTM_CUDA_TRY(cudaMemsetAsync(dbeta, 0, (size_t)rows * 4, st));
        }
        return LSTM_OK;
    }
    const Shape s = shape_of(d, opt);
    const char *kept = (const char *)fwd_ws;
    char *w = (char *)ws;
    if (d->dtype == LSTM_F32)
        return bwd<float>(d, s, dout, dsT, q, k, g, beta, states, deltas, dq, dk, dv, dg, dbeta, ds0, kept, w, st);
    if (d->dtype == LSTM_F16)
        return bwd<f16>(d, s, dout, dsT, q, k, g, beta, states, deltas, dq, dk, dv, dg, dbeta, ds0, kept, w, st);
    return bwd<bf16>(d, s, dout, dsT, q, k, g, beta, states, deltas, dq, dk, dv, dg, dbeta, ds0, kept, w, st);
}

}  // extern "C"
