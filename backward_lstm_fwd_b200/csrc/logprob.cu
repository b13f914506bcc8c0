// logprob.cu -- log-probabilities of given tokens (declared in
// include/liblstm.h).  With z = logits / temperature, per row:
//   lse = log sum exp z,  logp = z_target - lse,
//   entropy = lse - sum p z,  p = exp(z - lse),
// and the `top` largest logits (ties: the lowest index first).  The gradient is
//   dlogits = (dlogp (1[target] - p) - dentropy p (z - lse + entropy)) / temperature.
//
// Bound: bytes.  The forward reads the logits once: with c = log2(e) /
// temperature, every thread keeps its largest logit m, s = sum 2^{c (x - m)}
// and w = sum 2^{c (x - m)} c (x - m), rescaled when a group of elements
// raises m, and the threads' triples are joined at the end.  An element costs
// one exponential and half of three packed operations (and its conversion), 32
// elements one look at the maximum.  Many
// rows: 128 threads a block and eight blocks an SM, so that one row's loads run
// beside another's joins.  Few rows: a cluster of up to eight blocks shares a row
// and joins its parts through distributed shared memory.
// The alternatives come from the same pass: the first quarter (a third
// above 16) of the range gives every thread its own maximum, the top-th largest
// of those is a lower bound of the answer, and only elements at or above it (a
// few times `top`) enter a candidate list; the quarter is looked at twice (the
// second time from L1 / L2).
// The backward reads the logits and writes the gradient once.
#include <climits>
#include <cmath>

#include "host.cuh"
#include "tc_ptx.cuh"

using namespace lstm;

namespace {

typedef __nv_bfloat16 bf16;
typedef __half f16;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr int kCand = 1024;     // candidate list of a block
constexpr int kNarrow = 128;    // threads of a block
constexpr int kWide = 512;      // alternatives of few long rows
constexpr int kMaxParts = 8;    // blocks that share a row (a portable cluster)
constexpr int kPartBytes = 16 << 10;  // a part's least share of a row
constexpr int kBwdThreads = 128;
static_assert(kMaxParts * LSTM_LOGPROB_MAX_TOP <= kCand, "the parts' alternatives fit the candidate list");

// ---------------------------------------------------------------- elements
// 2^x (the hardware's approximation: relative error about 2^-22, results
// below 2^-126 flush to zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max(x, least) that keeps NaN: -inf - m stays usable as a factor of zero.
__device__ __forceinline__ float floor_nan(float x, float least = -1e28f) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
    return y;
}
// Elements of one 16-byte group.
template <class T> struct Group { static constexpr int n = 16 / sizeof(T); };
template <class T> __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[Group<T>::n]);
template <> __device__ __forceinline__ void unpack<float>(const uint4 &v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void unpack<bf16>(const uint4 &v, float (&f)[8]) { x8_to_f32<bf16>(v, f); }
template <> __device__ __forceinline__ void unpack<f16>(const uint4 &v, float (&f)[8]) { x8_to_f32<f16>(v, f); }
template <class T> __device__ __forceinline__ uint4 pack(const float (&f)[Group<T>::n]);
template <> __device__ __forceinline__ uint4 pack<float>(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 pack<bf16>(const float (&f)[8]) { return f32x8_to<bf16>(f); }
template <> __device__ __forceinline__ uint4 pack<f16>(const float (&f)[8]) { return f32x8_to<f16>(f); }

// Order of alternatives: larger value first, then lower index; one 64-bit key,
// larger is better.  NaN sorts below every number.
__device__ __forceinline__ unsigned ordered(float x) {
    if (x != x) return 0u;
    if (x == 0.f) x = 0.f;  // -0 and +0 are equal
    const unsigned b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(unsigned o) {
    if (o == 0u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ float value_of(unsigned long long key) { return from_ordered((unsigned)(key >> 32)); }
__device__ __forceinline__ unsigned long long key_of(float x, int i) {
    return ((unsigned long long)ordered(x) << 32) | (unsigned)~i;
}
__device__ __forceinline__ int index_of(unsigned long long key) { return (int)~(unsigned)key; }

// --------------------------------------------------- running softmax triple
// With c = log2(e) / temperature and m the largest logit:
struct Stat {
    float m, s, w;  // m; sum 2^{c (x - m)}; sum 2^{c (x - m)} c (x - m)
};
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return Stat{m, a.s + b.s, a.w + b.w};  // nothing but -inf (or NaN) yet
    const float da = floor_nan((a.m - m) * c), db = floor_nan((b.m - m) * c), fa = ex2(da), fb = ex2(db);
    return Stat{m, a.s * fa + b.s * fb, (a.w + a.s * da) * fa + (b.w + b.s * db) * fb};
}
// Two floats at once.
struct F2 {
    float x, y;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// A thread takes the exponent c (x - m) as c x - round(c m), one fused operation, and
// corrects its sums by the remainder of c m at the end.  The remainder is half a
// unit of round(c m): at most half of one below 2^24, and at 2^31 the largest (64)
// that keeps a sum of exponentials in a float's range.  So:
// - logits at or below a.mask, the power of two with c |mask| in [2^30, 2^31), are
//   raised to it on the way in (NaN stays) and given no weight;
// - a part whose largest logit is a mask or has c |m| above kExact is summed again
//   as it stands, from c (x - m).  (In any other part the raised ones lie 2^29 and
//   more below it, their exponentials are zero.)
constexpr float kExact = 16777216.f;  // 2^24
__device__ __forceinline__ float raised(float x, float mask) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(mask));
    return y;
}

// A 16-byte group as pairs of floats raised to the mask value (as floats: the
// 16-bit maximum that keeps NaN costs more; 8192 x 32000 bf16 93 us against 103).
// float's largest() raises in place.
template <class T> struct Pairs {
    static constexpr int n = 4;
    typedef typename Elem<T>::E2 E2;
    __device__ static __forceinline__ float largest(uint4 &v, float mask) {
        E2 *h = reinterpret_cast<E2 *>(&v);
        const float2 m = Elem<T>::to_f2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(m.x, m.y);
    }
    __device__ static __forceinline__ F2 pair(const uint4 &v, int i, float mask) {
        const float2 f = Elem<T>::to_f2(reinterpret_cast<const E2 *>(&v)[i]);
        return F2{raised(f.x, mask), raised(f.y, mask)};
    }
    // bit i: element i is at or above the bound (or NaN)
    __device__ static __forceinline__ unsigned candidates(const uint4 &v, float bound) {
        const E2 *h = reinterpret_cast<const E2 *>(&v), b = Elem<T>::from_f2(bound, bound);
        unsigned bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned at = ~__hlt2_mask(h[i], b);
            bits |= ((at & 1u) | ((at >> 15) & 2u)) << (2 * i);
        }
        return bits;
    }
};
template <> struct Pairs<float> {
    static constexpr int n = 2;
    __device__ static __forceinline__ float largest(uint4 &v, float mask) {
        float *f = reinterpret_cast<float *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = raised(f[i], mask);
        return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    }
    __device__ static __forceinline__ F2 pair(const uint4 &v, int i, float mask) {
        const float *f = reinterpret_cast<const float *>(&v);
        return F2{f[2 * i], f[2 * i + 1]};
    }
    __device__ static __forceinline__ unsigned candidates(const uint4 &v, float bound) {
        const float *f = reinterpret_cast<const float *>(&v);
        unsigned bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) bits |= (unsigned)!(f[i] < bound) << i;
        return bits;
    }
};

// A group of masks.
template <class T> struct Elem16 { static constexpr unsigned neg_inf = 0xff80u; };
template <> struct Elem16<f16> { static constexpr unsigned neg_inf = 0xfc00u; };
template <class T> __device__ __forceinline__ uint4 masks() {
    const unsigned x = sizeof(T) == 4 ? 0xff800000u : Elem16<T>::neg_inf * 0x10001u;
    return make_uint4(x, x, x, x);
}

// A thread's own sums, with the rounded c m in the place of c m, so that an
// exponent is one fused multiply-add (half of a packed one).
struct Run {
    float mask, m, cm = 1e30f;  // masks only so far: every exponential is zero
    F2 s = {0.f, 0.f}, w = {0.f, 0.f};
    __device__ __forceinline__ explicit Run(float mask) : mask(mask), m(mask) {}
    __device__ __forceinline__ void see(float gmax, float c) {  // the next elements' largest
        if (gmax > m) {
            const float cn = gmax * c, d = m == mask ? 0.f : cm - cn, e = ex2(d);
            w.x = (w.x + s.x * d) * e;
            w.y = (w.y + s.y * d) * e;
            s.x *= e;
            s.y *= e;
            m = gmax;
            cm = cn;
        }
    }
    __device__ __forceinline__ void add(F2 x, float c) {
        const F2 d = fma2(x, F2{c, c}, F2{-cm, -cm}), e = F2{ex2(d.x), ex2(d.y)};
        s = add2(s, e);
        w = fma2(e, d, w);
    }
    __device__ __forceinline__ void add1(float x, float c) {
        see(x, c);
        const float d = fmaf(x, c, -cm), e = ex2(d);
        s.x += e;
        w.x = fmaf(e, d, w.x);
    }
    __device__ __forceinline__ Stat stat(float c) const {
        if (m == mask) return Stat{-INFINITY, s.x + s.y, w.x + w.y};  // zeros, or NaN
        const float d = fmaf(-m, c, cm), e = ex2(d);  // what the rounding of c m left
        const float st = s.x + s.y;
        return Stat{m, st * e, (w.x + w.y + st * d) * e};
    }
};
// Joins n (a power of two up to 16) triples of shared memory; the result is the
// same in every thread.
__device__ __forceinline__ Stat join_list(const Stat *list, int n, float c) {
    Stat a = list[(threadIdx.x & 31) % n];
    for (int o = n / 2; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_down_sync(~0u, a.m, o);
        b.s = __shfl_down_sync(~0u, a.s, o);
        b.w = __shfl_down_sync(~0u, a.w, o);
        a = join(a, b, c);
    }
    a.m = __shfl_sync(~0u, a.m, 0);
    a.s = __shfl_sync(~0u, a.s, 0);
    a.w = __shfl_sync(~0u, a.w, 0);
    return a;
}
template <int THREADS> __device__ __forceinline__ Stat block_join(Stat a, float c, Stat *warp_stats) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(~0u, a.m, o);
        b.s = __shfl_xor_sync(~0u, a.s, o);
        b.w = __shfl_xor_sync(~0u, a.w, o);
        a = join(a, b, c);
    }
    if ((threadIdx.x & 31) == 0) warp_stats[threadIdx.x >> 5] = a;
    __syncthreads();
    return join_list(warp_stats, THREADS / 32, c);
}

struct Args {
    const void *logits;
    const void *targets;
    int id64, N, vocab, top, parts;
    long long ld;
    float inv_temp, c, mask;  // c: times log2(e)
    float *logp, *entropy, *stats, *top_logp;
    int *top_ids;
};

// -1: an ignored row.
__device__ __forceinline__ int target_of(const void *t, int id64, int r, int vocab) {
    const long long x = id64 ? ((const long long *)t)[r] : (long long)((const int *)t)[r];
    return x >= 0 && x < vocab ? (int)x : -1;
}

// Row outputs from the row's triple, thread 0's target t and its logit x, and
// the row's sorted alternatives.
template <int THREADS>
__device__ __forceinline__ void finish(const Args &a, int r, Stat st, int t, float x, const unsigned long long *keys) {
    const bool empty = st.m == -INFINITY && st.s == 0.f;  // every logit is -inf
    const float ls = log2f(st.s);
    if (threadIdx.x == 0) {
        a.stats[2LL * r] = st.m;
        a.stats[2LL * r + 1] = empty ? 0.f : ls;
        if (a.entropy) a.entropy[r] = empty ? 0.f : (ls - st.w / st.s) * kLn2;
        if (a.logp) a.logp[r] = t < 0 ? 0.f : empty ? -INFINITY : (x - st.m) * a.inv_temp - ls * kLn2;
    }
    for (int i = threadIdx.x; i < a.top; i += THREADS) {
        const unsigned long long k = keys[i];
        a.top_ids[(long long)r * a.top + i] = index_of(k);
        a.top_logp[(long long)r * a.top + i] = empty ? -INFINITY : (value_of(k) - st.m) * a.inv_temp - ls * kLn2;
    }
}

// Of n <= kCand distinct keys in shared memory, the `top` largest in order:
// four lanes count the keys above one.
template <int THREADS>
__device__ __forceinline__ void rank_keys(const unsigned long long *keys, int n, int top, unsigned long long *out) {
    const int q = threadIdx.x & 3;
    for (int b = 0; b < n; b += THREADS / 4) {
        const int i = b + threadIdx.x / 4;
        const unsigned long long k = keys[min(i, n - 1)];
        int rank = 0;
        for (int j = q; j < n; j += 4) rank += keys[j] > k;
        rank += __shfl_xor_sync(~0u, rank, 1);
        rank += __shfl_xor_sync(~0u, rank, 2);
        if (i < n && q == 0 && rank < top) out[rank] = k;
    }
    __syncthreads();
}

// The top-th largest of the maxima of 32 (top <= 16) or 128 groups of threads:
// at least `top` elements are at or above it.  (It is the least of those with
// fewer than `top` above.)  Of 32, few more elements than `top` are (8: 9, 16:
// 22), and every warp ranks them all, a lane each; of 128 every group ranks its own.
__device__ __forceinline__ int above(const float *x, int n, float mine) {
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; j += 4) {
        const float4 o = *(const float4 *)(x + j);
        rank += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    return rank;
}
template <int THREADS>
__device__ __forceinline__ float bound_of(float mine, int top, float *maxima, unsigned *bound) {
    constexpr int each = THREADS / 128;
#pragma unroll
    for (int o = 1; o < each; o <<= 1) mine = fmaxf(mine, __shfl_xor_sync(~0u, mine, o));
    if (top <= 16) {
        mine = fmaxf(mine, __shfl_xor_sync(~0u, mine, each));
        mine = fmaxf(mine, __shfl_xor_sync(~0u, mine, 2 * each));
        if (threadIdx.x % (4 * each) == 0) maxima[threadIdx.x / (4 * each)] = mine;
        __syncthreads();
        mine = maxima[threadIdx.x & 31];
        return from_ordered(__reduce_min_sync(~0u, above(maxima, 32, mine) < top ? ordered(mine) : ~0u));
    }
    const int q = threadIdx.x % each;
    if (q == 0) maxima[threadIdx.x / each] = mine;
    if (threadIdx.x == 0) *bound = ~0u;
    __syncthreads();
    int rank = above(maxima + q * (128 / each), 128 / each, mine);
#pragma unroll
    for (int o = 1; o < each; o <<= 1) rank += __shfl_xor_sync(~0u, rank, o);
    const unsigned least = __reduce_min_sync(~0u, rank < top ? ordered(mine) : ~0u);
    if ((threadIdx.x & 31) == 0) atomicMin(bound, least);
    __syncthreads();
    return from_ordered(*bound);
}

// ----------------------------------------------------------------- forward
// 8192 x 32000 bf16: 97 us, 524 MB at 5.4 TB/s (the exponentials and their packed
// sums share the issue slots with the loads; a block that walks rows and loads the
// next one's beginning before it joins a row took 110 to 118); with 8
// alternatives 2048 x 100003 bf16 104 us, 410 MB at 3.9 TB/s: the quarter looked
// at twice and the joins of a row.  4 x 128000 float, 20 alternatives: 13 us, the
// latency of one row's steps.
// Block (r, p): part p of row r; the parts of a row are a cluster.  TOP:
// alternatives wanted.
template <class T, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kNarrow ? 8 : 1) fwd_kernel(Args a) {
    constexpr int n = Group<T>::n, U = TOP && THREADS == kNarrow ? 3 : 4, WARPS = THREADS / 32;
    __shared__ Stat warp_stats[WARPS > kMaxParts ? WARPS : kMaxParts], part_stat;
    __shared__ unsigned long long cand[TOP ? kCand : 1], best[TOP ? LSTM_LOGPROB_MAX_TOP : 1];
    __shared__ __align__(16) float maxima[TOP ? 128 : 4];
    __shared__ unsigned bound_s;
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31;
    const int r = blockIdx.x / a.parts, p = blockIdx.x % a.parts;
    const T *row = (const T *)a.logits + (long long)r * a.ld;
    const float c = a.c, mask = a.mask;
    // part p is the elements [e0, e1); its 16-byte groups [g0, g1)
    const int e0 = (int)((long long)a.vocab * p / a.parts), e1 = (int)((long long)a.vocab * (p + 1) / a.parts);
    const int mis = (int)(((uintptr_t)(row + e0) & 15u) / sizeof(T));
    const int h = min(e1, e0 + (mis ? n - mis : 0));  // [e0, h): before the first whole group
    const int groups = (e1 - h) / n;
    const uint4 *gp = (const uint4 *)(row + h);
    const int tail = h + groups * n;                  // [tail, e1): after the last one
    const int target = a.logp && p == 0 && tid == 0 ? target_of(a.targets, a.id64, r, a.vocab) : -1;
    Run sum(mask);
    float bound = -INFINITY;
    if (TOP && tid == 0) count = 0;

    // the elements of `bits`, from index i on and found at x, become candidates
    auto push = [&](int i, unsigned bits, const T *x) {
#pragma unroll 1
        for (; bits; bits &= bits - 1) {
            const int j = __ffs(bits) - 1, at = atomicAdd(&count, 1);
            if (at < kCand) cand[at] = key_of(to_f(x[j]), i + j);
        }
    };
    // groups b .. e-1, the next U of a thread loaded before it looks at the last
    // ones; look: candidates too.  (A warp goes round together: lanes that drift
    // apart at a candidate would go round one after another from there on, 65 us
    // instead of 38 on such a row of 128000.)
    auto fetch = [&](uint4 (&v)[U], int g, int e) {
        if (g + (U - 1) * THREADS < e) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = __ldg(gp + g + u * THREADS);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = g + u * THREADS < e ? __ldg(gp + g + u * THREADS) : masks<T>();
        }
    };
    uint4 ahead[U];  // what run() looks at first
    auto run = [&](int b, int e, bool look) {
#pragma unroll 1
        for (int g = b + tid; g - lane < e; g += U * THREADS) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ahead[u];
            fetch(ahead, g + U * THREADS, e);
            float gm[U], top = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                gm[u] = Pairs<T>::largest(v[u], mask);
                top = fmaxf(top, gm[u]);
            }
            sum.see(top, c);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < Pairs<T>::n; ++i) sum.add(Pairs<T>::pair(v[u], i, mask), c);
            if (TOP && look && __any_sync(~0u, !(top < bound))) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (g + u * THREADS < e && !(gm[u] < bound))
                        push(h + (g + u * THREADS) * n, Pairs<T>::candidates(v[u], bound), (const T *)(gp + g + u * THREADS));
                __syncwarp();
            }
        }
    };
    // How much is looked at twice: candidates against a second look.  (2048 x
    // 100003 bf16, us at an eighth, a sixth, a quarter, a third: 8 alternatives
    // 120, 115, 106, 110; 64 alternatives 3458 (the list overflows), 311, 217, 187.)
    const int first = TOP ? min(groups, max(groups / (a.top <= 16 ? 4 : 3), U * THREADS)) : 0;
    fetch(ahead, tid, TOP ? first : groups);
    // the elements outside whole groups: fewer than 2 n
    const int mine0 = e0 + tid < h ? e0 + tid : -1, mine1 = tail + tid < e1 ? tail + tid : -1;
    if (mine0 >= 0) sum.add1(raised(to_f(row[mine0]), mask), c);
    if (mine1 >= 0) sum.add1(raised(to_f(row[mine1]), mask), c);
    if (TOP) {
        run(0, first, false);
        fetch(ahead, first + tid, groups);  // under way while the bound is found
        bound = bound_of<THREADS>(sum.m, a.top, maxima, &bound_s);
        if (bound == mask) bound = -INFINITY;  // masks are among the alternatives
        if (mine0 >= 0) push(mine0, !(raised(to_f(row[mine0]), mask) < bound), row + mine0);
        if (mine1 >= 0) push(mine1, !(raised(to_f(row[mine1]), mask) < bound), row + mine1);
        __syncwarp();
#pragma unroll 2
        for (int g = tid; g - lane < first; g += THREADS) {
            uint4 v = g < first ? __ldg(gp + g) : masks<T>();
            const bool at = g < first && !(Pairs<T>::largest(v, mask) < bound);
            if (__any_sync(~0u, at)) {
                if (at) push(h + g * n, Pairs<T>::candidates(v, bound), (const T *)(gp + g));
                __syncwarp();
            }
        }
    }
    run(first, groups, TOP);
    const float chosen = target >= 0 ? to_f(row[target]) : 0.f;
    Stat st = block_join<THREADS>(sum.stat(c), c, warp_stats);  // its barrier also closes the candidate list
    if (!(fabsf(st.m) * c <= kExact)) {  // masks (or NaN) alone, or large logits: the part's plain sums
        Stat own = {-INFINITY, 0.f, 0.f};
        for (int i = e0 + tid; i < e1; i += THREADS) own.m = fmaxf(own.m, to_f(row[i]));
        __syncthreads();
        const float m = block_join<THREADS>(own, c, warp_stats).m;
        own.m = m;
        for (int i = e0 + tid; i < e1; i += THREADS) {
            const float x = to_f(row[i]);
            if (m == -INFINITY) {  // -inf counts nothing, NaN spoils the row
                own.s += x == m ? 0.f : x;
                continue;
            }
            const float d = floor_nan((x - m) * c), e = ex2(d);
            own.s += e;
            own.w = fmaf(e, d, own.w);
        }
        __syncthreads();
        st = block_join<THREADS>(own, c, warp_stats);
    }

    if (TOP) {
        if (count <= kCand) {
            rank_keys<THREADS>(cand, count, a.top, best);
        } else {
            // More candidates than the list holds (long runs of equal values, or
            // fewer unmasked ones than `top` in the first look): one exact pass
            // over the part per alternative.  2048 x 100003 bf16, three quarters
            // masked: 8 alternatives 2.3 ms, 64 16 ms; 4 x 128000 float 39 and 200 us.
            unsigned long long prev = ~0ull;
            for (int k = 0; k < a.top; ++k) {
                unsigned long long mine = 0;
                for (int i = e0 + tid; i < e1; i += THREADS) {
                    const unsigned long long key = key_of(to_f(row[i]), i);
                    if (key < prev && key > mine) mine = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long y = __shfl_xor_sync(~0u, mine, o);
                    mine = y > mine ? y : mine;
                }
                __syncthreads();
                if ((tid & 31) == 0) cand[tid >> 5] = mine;
                __syncthreads();
                for (int w = 0; w < WARPS; ++w) mine = cand[w] > mine ? cand[w] : mine;
                prev = mine;
                if (tid == 0) best[k] = mine;
            }
            __syncthreads();
        }
    }
    if (a.parts == 1) {
        finish<THREADS>(a, r, st, target, chosen, best);
        return;
    }
    // the first block of the cluster joins the parts
    if (tid == 0) part_stat = st;
    tc::cluster_sync_all();
    if (p == 0) {
        auto peer = [&](const void *x, int q) { return tc::map_rank(tc::smem_u32(x), q); };
        if (tid < a.parts) {
            const uint32_t at = peer(&part_stat, tid);
            Stat o;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.m) : "r"(at));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.s) : "r"(at + 4));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.w) : "r"(at + 8));
            warp_stats[tid] = o;
        }
        if (TOP) {
            const int all = a.parts * a.top;
            for (int i = tid; i < all; i += THREADS) {
                unsigned long long k;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(peer(&best[i % a.top], i / a.top)));
                cand[i] = k;
            }
        }
        __syncthreads();
        st = join_list(warp_stats, a.parts, c);
        if (TOP) rank_keys<THREADS>(cand, a.parts * a.top, a.top, best);
        finish<THREADS>(a, r, st, target, chosen, best);
    }
    tc::cluster_sync_all();  // no block leaves while its memory may be read
}

// ---------------------------------------------------------------- backward
// 8192 x 32000 bf16: 162 us, 1.05 GB at 6.5 TB/s, memory's rate.
struct BwdArgs {
    const void *logits, *targets;
    int id64, N, vocab, chunk, chunks;  // blocks of a row, elements each
    long long ld, ldd;
    float inv_temp;
    const float *stats, *entropy, *dlogp, *dentropy;
    void *dlogits;
};

template <class T, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) bwd_kernel(BwdArgs a) {
    constexpr int n = Group<T>::n, U = 2;
    const int tid = threadIdx.x;
    const int r = blockIdx.x / a.chunks, p = blockIdx.x % a.chunks;
    const T *x = (const T *)a.logits + (long long)r * a.ld;
    T *y = (T *)a.dlogits + (long long)r * a.ldd;
    const float m = a.stats[2LL * r], ls = a.stats[2LL * r + 1], c = a.inv_temp * kLog2e;
    const float dh = a.dentropy ? a.dentropy[r] : 0.f, ent = a.dentropy ? a.entropy[r] * kLog2e : 0.f;
    const int t = a.targets ? target_of(a.targets, a.id64, r, a.vocab) : -1;
    const float dl = t >= 0 && a.dlogp ? a.dlogp[r] * a.inv_temp : 0.f, dhc = dh * a.inv_temp * kLn2;
    const bool empty = m == -INFINITY && ls == ls;
    // dl 1[target] - p (dl + dh (log p + entropy)), dl and dh over the temperature
    auto grad = [&](float v, int i) {
        // log2 p, from -256 up (2^-127 and less is zero already): a finite factor of zero
        const float lp = floor_nan((v - m) * c - ls, -256.f);
        float g = -ex2(lp) * fmaf(dhc, lp + ent, dl);
        if (i == t) g += dl;
        return empty ? 0.f : g;
    };
    const int e0 = p * a.chunk, e1 = min(a.vocab, e0 + a.chunk);
    if (!VEC) {
        for (int i = e0 + tid; i < e1; i += kBwdThreads) y[i] = from_f<T>(grad(to_f(x[i]), i));
        return;
    }
    const int mis = (int)(((uintptr_t)(x + e0) & 15u) / sizeof(T));
    const int h = min(e1, e0 + (mis ? n - mis : 0));
    const int groups = (e1 - h) / n, tail = h + groups * n;
    if (tid < h - e0) y[e0 + tid] = from_f<T>(grad(to_f(x[e0 + tid]), e0 + tid));
    if (tid < e1 - tail) y[tail + tid] = from_f<T>(grad(to_f(x[tail + tid]), tail + tid));
    const uint4 *xv = (const uint4 *)(x + h);
    uint4 *yv = (uint4 *)(y + h);
    for (int g = tid; g < groups; g += U * kBwdThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g + u * kBwdThreads < groups) v[u] = xv[g + u * kBwdThreads];  // dlogits may be logits
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gg = g + u * kBwdThreads;
            if (gg >= groups) break;
            float f[n];
            unpack<T>(v[u], f);
#pragma unroll
            for (int i = 0; i < n; ++i) f[i] = grad(f[i], h + gg * n + i);
            yv[gg] = pack<T>(f);
        }
    }
}

// -------------------------------------------------------------------- host
bool dims_ok(const lstm_logprob_dims *d) {
    if (!d || d->N < 0 || d->vocab < 0 || d->ld < d->vocab || d->top < 0) return false;
    if (!host::dtype_ok(d->dtype) || (d->id_bytes != 4 && d->id_bytes != 8)) return false;
    if (d->top > d->vocab && d->N > 0) return false;
    return true;
}
bool dims_supported(const lstm_logprob_dims *d) {
    return d->top <= LSTM_LOGPROB_MAX_TOP && d->vocab <= (1 << 30) && d->N <= (1 << 30);
}

// (Within these limits the mask value and c = inv_temp log2(e) are ordinary floats.)
bool temp_ok(float inv_temp) { return inv_temp >= 1e-6f && inv_temp <= 1e6f; }

template <class T, bool TOP, int THREADS> int launch_fwd(Args &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * a.parts));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)a.parts, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = a.parts > 1 ? 1 : 0;
    LSTM_CUDA_TRY(cudaLaunchKernelEx(&cfg, fwd_kernel<T, TOP, THREADS>, a));
    note_launch();
    return LSTM_OK;
}

// Which blocks a row gets (us, bf16).  Rows share out over a cluster until every
// SM holds four blocks or a part is 16 KB: one row of 32000 takes 4.7 in 16 KB
// parts and 5.2 in 32 KB ones, 74 of 128000 take 8.9 in parts and 16.4 whole,
// 296 of 5000 take 4.0 whole and 5.0 in 8 KB parts.  Alternatives of so few rows
// that half the SMs hold a block each get 512 threads a block instead of 128
// (more loads in flight, and fewer turns over the candidates): 4 rows of 128000,
// 8 alternatives 8.9 against 12.1, 20 alternatives 11.5 against 16.4; one row of
// 32000, 64 alternatives 11.7 against 22.3.  Of more rows the clusters of 512
// threads no longer fit at once (16 rows of 128000: 16.4 against 12.8; 37: 24.0
// against 13.5), and below four parts there is little to win (5000: 8.5 against 6.4).
template <class T, bool TOP> int forward(Args &a, int sms, cudaStream_t s) {
    const long long bytes = (long long)a.vocab * (int)sizeof(T);
    a.parts = 1;
    while (a.parts < kMaxParts && (long long)a.N * a.parts <= 2 * sms && bytes > a.parts * kPartBytes) a.parts *= 2;
    if constexpr (TOP)
        if (a.parts >= 4 && 2LL * a.N * a.parts <= sms) return launch_fwd<T, TOP, kWide>(a, s);
    return launch_fwd<T, TOP, kNarrow>(a, s);
}

template <class T> int forward_t(Args &a, int sms, cudaStream_t s) {
    return a.top ? forward<T, true>(a, sms, s) : forward<T, false>(a, sms, s);
}

template <class T> int backward(BwdArgs &a, cudaStream_t s) {
    // Blocks of up to 8192 elements: 32 a thread, four 16-byte groups of a
    // 16-bit type.
    a.chunks = (a.vocab + 8191) / 8192;
    a.chunk = ((a.vocab + a.chunks - 1) / a.chunks + 7) / 8 * 8;
    const long long blocks = (long long)a.N * a.chunks;
    if (blocks > INT_MAX) return LSTM_ERR_UNSUPPORTED;
    // 16-byte groups need logits and dlogits rows that start alike
    const bool vec = (a.ld - a.ldd) * (long long)sizeof(T) % 16 == 0 && ((uintptr_t)a.logits - (uintptr_t)a.dlogits) % 16 == 0;
    if (vec)
        bwd_kernel<T, true><<<(unsigned)blocks, kBwdThreads, 0, s>>>(a);
    else
        bwd_kernel<T, false><<<(unsigned)blocks, kBwdThreads, 0, s>>>(a);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

}  // namespace

extern "C" {

int lstm_logprob_fwd(const lstm_logprob_dims *d, const void *logits, const void *targets, float inv_temp,
                     float *logp, float *entropy, float *stats, int *top_ids, float *top_logp, void *stream) {
    if (!dims_ok(d) || !temp_ok(inv_temp)) return LSTM_ERR_INVALID_ARG;
    if (!dims_supported(d)) return LSTM_ERR_UNSUPPORTED;
    const bool any = d->N > 0;
    if (!host::ptr_ok(logits, any && d->vocab > 0, host::elem_bytes(d->dtype)) ||
        !host::ptr_ok(targets, any && logp, d->id_bytes) || !host::ptr_ok(logp, any && targets, 4) ||
        !host::ptr_ok(entropy, false, 4) || !host::ptr_ok(stats, any, 4) ||
        !host::ptr_ok(top_ids, any && d->top > 0, 4) || !host::ptr_ok(top_logp, any && d->top > 0, 4))
        return LSTM_ERR_INVALID_ARG;
    if (!any) return LSTM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    Args a = {};
    a.logits = logits;
    a.targets = targets;
    a.id64 = d->id_bytes == 8;
    a.N = d->N;
    a.vocab = d->vocab;
    a.top = d->top;
    a.ld = d->ld;
    a.inv_temp = inv_temp;
    a.c = inv_temp * kLog2e;
    int e;
    (void)frexpf(a.c, &e);  // c in [2^(e-1), 2^e)
    a.mask = -ldexpf(1.f, 31 - e);
    a.logp = logp;
    a.entropy = entropy;
    a.stats = stats;
    a.top_ids = top_ids;
    a.top_logp = top_logp;
    const int sms = host::sm_count();
    if (d->dtype == LSTM_F32) return forward_t<float>(a, sms, s);
    if (d->dtype == LSTM_F16) return forward_t<f16>(a, sms, s);
    return forward_t<bf16>(a, sms, s);
}

int lstm_logprob_bwd(const lstm_logprob_dims *d, const void *logits, const void *targets, float inv_temp,
                     const float *stats, const float *entropy, const float *dlogp, const float *dentropy,
                     void *dlogits, long long ldd, void *stream) {
    if (!dims_ok(d) || ldd < d->vocab || !temp_ok(inv_temp)) return LSTM_ERR_INVALID_ARG;
    if (!dims_supported(d)) return LSTM_ERR_UNSUPPORTED;
    const bool any = d->N > 0 && d->vocab > 0;
    const size_t e = host::elem_bytes(d->dtype);
    if (!host::ptr_ok(logits, any, e) || !host::ptr_ok(targets, any && dlogp, d->id_bytes) || !host::ptr_ok(stats, any, 4) ||
        !host::ptr_ok(entropy, any && dentropy, 4) || !host::ptr_ok(dlogp, false, 4) ||
        !host::ptr_ok(dentropy, false, 4) || !host::ptr_ok(dlogits, any, e))
        return LSTM_ERR_INVALID_ARG;
    if (dlogits == logits && ldd != d->ld && any) return LSTM_ERR_INVALID_ARG;
    if (!any) return LSTM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    BwdArgs a = {};
    a.logits = logits;
    a.targets = targets;
    a.id64 = d->id_bytes == 8;
    a.N = d->N;
    a.vocab = d->vocab;
    a.ld = d->ld;
    a.ldd = ldd;
    a.inv_temp = inv_temp;
    a.stats = stats;
    a.entropy = entropy;
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    if (d->dtype == LSTM_F32) return backward<float>(a, s);
    if (d->dtype == LSTM_F16) return backward<f16>(a, s);
    return backward<bf16>(a, s);
}

}  // extern "C"
