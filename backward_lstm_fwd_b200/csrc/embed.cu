// embed.cu -- token embedding (declared in include/liblstm.h): the lookup
// x_r = scale table[id_r] and the gradient of the table,
//   dtable[w] = scale sum_{r : id_r = w} dx_r,
// summed in a fixed order (positions sorted stably by token), so that equal
// inputs give equal bits whatever the token frequencies.
//
// Bound: bytes.  The lookup reads each id and row once and writes x; the
// gradient reads dx once and writes every table row once, those with a token
// twice (first as zeros, in the shadow of the sort).
//
// Gradient, in launches on one stream:
//   sort    stable least-significant-digit radix sort of (token, position), 9
//           bits a pass: one launch of block histograms, then one a pass that
//           scatters and counts the next pass's histograms (integers: any
//           order of the additions gives the same).  Up to 4096 keys are
//           sorted by one block in shared memory, in one launch.  Further
//           blocks of these launches, bound by latency on few SMs, set the
//           table to zero meanwhile;
//   grad    units of 32 sorted positions x column tiles: a thread adds its
//           columns of up to 32 rows in order and stores each token that lies
//           inside the unit; a token that crosses a unit's border leaves
//           partial sums;
//   join    adds the partial sums of a token that spans units, in order and in
//           double.
#include "host.cuh"

#include <algorithm>
#include <climits>

using namespace lstm;

namespace {

typedef __nv_bfloat16 bf16;
typedef __half f16;

// A token id as a row of the table, or -1 for padding (any id outside it).
template <class ID> __device__ __forceinline__ int row_of(const ID *ids, long long r, int vocab) {
    const ID w = ids[r];
    return w >= 0 && w < (ID)vocab ? (int)w : -1;
}

// ------------------------------------------------------------------ lookup
// Vector path: rows of whole, aligned 16-byte groups.  One warp copies U x 32
// groups.  32768 rows x 1024 bf16 from a table of 32000: 14 us, 67 MB written at
// 4.8 TB/s beside as many read, most of them from L2.
template <class T> __device__ __forceinline__ uint4 scaled(uint4 v, float scale);
template <> __device__ __forceinline__ uint4 scaled<float>(uint4 v, float s) {
    return make_uint4(__float_as_uint(__uint_as_float(v.x) * s), __float_as_uint(__uint_as_float(v.y) * s),
                      __float_as_uint(__uint_as_float(v.z) * s), __float_as_uint(__uint_as_float(v.w) * s));
}
template <class T> __device__ __forceinline__ uint4 scaled16(uint4 v, float s) {
    float f[8];
    x8_to_f32<T>(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= s;
    return f32x8_to<T>(f);
}
template <> __device__ __forceinline__ uint4 scaled<bf16>(uint4 v, float s) { return scaled16<bf16>(v, s); }
template <> __device__ __forceinline__ uint4 scaled<f16>(uint4 v, float s) { return scaled16<f16>(v, s); }

template <class T, class ID, int U>
__global__ void __launch_bounds__(256) lookup_kernel(const ID *ids, const uint4 *table, float scale,
                                                     uint4 *x, int N, int vocab, int groups,
                                                     int tiles) {
    const long long job = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (job >= (long long)N * tiles) return;
    const int r = (int)(job / tiles), g0 = (int)(job % tiles) * (32 * U) + (threadIdx.x & 31);
    const int w = row_of(ids, r, vocab);
    const uint4 *src = table + (long long)max(w, 0) * groups;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        if (w >= 0 && g0 + 32 * u < groups) v[u] = __ldg(src + g0 + 32 * u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (g0 + 32 * u < groups)  // (padding: zeros, whatever the scale)
            x[(long long)r * groups + g0 + 32 * u] = w >= 0 ? scaled<T>(v[u], scale) : v[u];
}

// Element path: any other rows.
template <class T, class ID>
__global__ void __launch_bounds__(256) lookup_elem_kernel(const ID *ids, const T *table, float scale,
                                                          T *x, int N, int vocab, int I) {
    const int r = blockIdx.x;
    const int w = row_of(ids, r, vocab);
    for (int i = threadIdx.x; i < I; i += 256)
        x[(long long)r * I + i] = w >= 0 ? from_f<T>(to_f(table[(long long)w * I + i]) * scale) : from_f<T>(0.f);
}

template <class T, class ID>
int lookup(const lstm_embed_dims *d, const void *ids, const void *table, float scale, void *x,
           cudaStream_t s) {
    const size_t row = (size_t)d->I * sizeof(T);
    if (row % 16 || ((uintptr_t)table | (uintptr_t)x) % 16) {
        lookup_elem_kernel<T, ID><<<d->N, 256, 0, s>>>((const ID *)ids, (const T *)table, scale, (T *)x,
                                                      d->N, d->vocab, d->I);
        LSTM_CUDA_TRY(host::launched());
        return LSTM_OK;
    }
    const int groups = (int)(row / 16);
    // Four groups a lane keep enough loads in flight; of few rows one group a
    // lane spreads the call over more SMs.  (Rows of 128 groups, us with one / four:
    // 128 rows 1.9 / 2.1, 1024 2.3 / 2.2, 8192 6.1 / 4.4, 32768 24.8 / 16.1.)
    const bool wide = (long long)d->N * groups >= 1 << 17;
    const int tiles = (groups + (wide ? 128 : 32) - 1) / (wide ? 128 : 32);
    const long long blocks = ((long long)d->N * tiles + 7) / 8;
    if (blocks > INT_MAX) return LSTM_ERR_UNSUPPORTED;
    if (wide)
        lookup_kernel<T, ID, 4><<<(unsigned)blocks, 256, 0, s>>>((const ID *)ids, (const uint4 *)table, scale,
                                                                (uint4 *)x, d->N, d->vocab, groups, tiles);
    else
        lookup_kernel<T, ID, 1><<<(unsigned)blocks, 256, 0, s>>>((const ID *)ids, (const uint4 *)table, scale,
                                                                (uint4 *)x, d->N, d->vocab, groups, tiles);
    LSTM_CUDA_TRY(host::launched());
    return LSTM_OK;
}

// -------------------------------------------------------------------- sort
constexpr int kBits = 9, kBins = 1 << kBits;
constexpr int kSortWarps = 16, kSortThreads = 32 * kSortWarps;
constexpr int kWarpKeys = 64, kTile = kSortWarps * kWarpKeys;  // 1024 keys a tile
constexpr int kRounds = kWarpKeys / 32;
constexpr int kSortBlocks = 128;                                // most blocks of a sort
static_assert(kSortThreads == kBins, "one thread per digit");

// A piece of the table that the blocks behind a sort's own set to zero meanwhile.
struct Fill {
    float *p;
    long long n;
};
__device__ __forceinline__ void fill(const Fill &f, int block, int blocks) {
    const int head = (int)min(f.n, (long long)(-((uintptr_t)f.p / 4) & 3)), tid = threadIdx.x;
    const long long groups = (f.n - head) / 4, tail = head + groups * 4;
    if (block == 0 && tid < head) f.p[tid] = 0.f;
    if (block == 0 && tail + tid < f.n) f.p[tail + tid] = 0.f;
    float4 *q = (float4 *)(f.p + head);
    for (long long i = (long long)block * blockDim.x + tid; i < groups; i += (long long)blocks * blockDim.x)
        q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

struct SortArgs {
    const void *ids;         // pass 0: token ids (id64 or not); later passes: NULL
    int id64, vocab;
    const int *key_in, *pos_in;
    int *key_out, *pos_out;
    int *hist, *hist_next;   // [blocks][kBins]: of this pass; of the next one, or NULL
    int N, shift, blocks, tiles;  // every block sorts `tiles` consecutive tiles
    Fill zero;               // by the launch's blocks from `blocks` on
};

// The sort key of input i: its token, or vocab for padding.
__device__ __forceinline__ int sort_key(const SortArgs &a, int i) {
    if (!a.ids) return a.key_in[i];
    const int w = a.id64 ? row_of((const long long *)a.ids, i, a.vocab)
                         : row_of((const int *)a.ids, i, a.vocab);
    return w >= 0 ? w : a.vocab;
}

__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(SortArgs a) {
    if ((int)blockIdx.x >= a.blocks) return fill(a.zero, blockIdx.x - a.blocks, gridDim.x - a.blocks);
    __shared__ int h[kBins];
    h[threadIdx.x] = 0;
    __syncthreads();
    const long long b0 = (long long)blockIdx.x * a.tiles * kTile;
    const int i1 = (int)min((long long)a.N, b0 + (long long)a.tiles * kTile);
    for (int i = (int)min((long long)a.N, b0) + threadIdx.x; i < i1; i += kSortThreads)
        atomicAdd(&h[(sort_key(a, i) >> a.shift) & (kBins - 1)], 1);
    __syncthreads();
    a.hist[blockIdx.x * kBins + threadIdx.x] = h[threadIdx.x];
    a.hist_next[blockIdx.x * kBins + threadIdx.x] = 0;
}

// Exclusive prefix sum over the block's threads.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int add = 0;
    for (int w = 0; w < warp; ++w) add += warp_sums[w];
    __syncthreads();
    return add + x - v;
}

// Stable scatter by one digit.  Warp w of a tile owns 64 consecutive keys, taken
// 32 at a time in order; equal digits among 32 are ranked by lane.  Bound by the
// latency of its steps (the tile's histogram, two sums, the scatter): 7.7 us a
// pass on 32768 keys, of which two passes sort ids below 2^18; histograms 3.5 us.
// With their shares of 131 MB to clear 13 and 8 us, where the gradient's launch
// took 13 us more to write the rows without a token itself.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(SortArgs a) {
    if ((int)blockIdx.x >= a.blocks) return fill(a.zero, blockIdx.x - a.blocks, gridDim.x - a.blocks);
    __shared__ int base[kBins];                     // next output place of each digit
    __shared__ unsigned short cnt[kSortWarps][kBins];
    __shared__ int warp_sums[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long b0 = (long long)blockIdx.x * a.tiles * kTile;
    {
        int before = 0, total = 0;
#pragma unroll 16
        for (int b = 0; b < a.blocks; ++b) {
            const int h = __ldcg(a.hist + b * kBins + tid);
            if (b < (int)blockIdx.x) before += h;
            total += h;
        }
        const int off = block_exclusive(total, warp_sums);
        base[tid] = off + before;
    }
    for (int t = 0; t < a.tiles; ++t) {
        const long long t0 = b0 + (long long)t * kTile;
        if (t0 >= a.N) break;  // the same for every thread
        for (int i = tid; i < kSortWarps * kBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
        __syncthreads();
        int key[kRounds], rank[kRounds];
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const long long i = t0 + warp * kWarpKeys + j * 32 + lane;
            key[j] = i < a.N ? sort_key(a, (int)i) : -1;
            const int dg = key[j] < 0 ? kBins : (key[j] >> a.shift) & (kBins - 1);
            const unsigned peers = __match_any_sync(~0u, dg);
            rank[j] = 0;
            if (dg < kBins) {
                const int r = __popc(peers & ((1u << lane) - 1u));
                rank[j] = cnt[warp][dg] + r;
            }
            __syncwarp();
            if (dg < kBins && lane == __ffs(peers) - 1)
                cnt[warp][dg] = (unsigned short)(cnt[warp][dg] + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        {  // digit tid: counts of the warps -> first place of each warp
            int run = base[tid];
            const int first = run;
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = cnt[w][tid];
                cnt[w][tid] = (unsigned short)(run - first);
                run += c;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kRounds; ++j) {
                if (key[j] < 0) continue;
                const int dg = (key[j] >> a.shift) & (kBins - 1);
                const int o = base[dg] + cnt[warp][dg] + rank[j];
                const int i = (int)(t0 + warp * kWarpKeys + j * 32 + lane);
                a.key_out[o] = key[j];
                a.pos_out[o] = a.pos_in ? a.pos_in[i] : i;
                if (a.hist_next)
                    atomicAdd(&a.hist_next[o / (a.tiles * kTile) * kBins + ((key[j] >> (a.shift + kBits)) & (kBins - 1))], 1);
            }
            __syncthreads();
            base[tid] = run;
        }
        __syncthreads();
    }
}

// All passes of up to 4096 keys in one block: warp w holds keys 128 w .. in
// registers, four rounds of 32, and the passes trade places in shared memory.
// 10.4 us on 2049 keys (two passes), where the launches above took 19; with 52 MB
// of table cleared beside it 11.7.
constexpr int kOneWarps = 32, kOneThreads = 32 * kOneWarps, kOneRounds = 4, kOneKeys = kOneThreads * kOneRounds;
struct OneSmem {
    int key[kOneKeys];
    unsigned short pos[kOneKeys];
    unsigned short cnt[kOneWarps][kBins];  // counts, then first places, of a warp's digits
    int warp_sums[kOneWarps];
};
__global__ void __launch_bounds__(kOneThreads) sort_one_kernel(SortArgs a, int bits) {
    if (blockIdx.x > 0) return fill(a.zero, blockIdx.x - 1, gridDim.x - 1);
    extern __shared__ __align__(16) unsigned char one_raw[];
    OneSmem &m = *reinterpret_cast<OneSmem *>(one_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int key[kOneRounds], pos[kOneRounds], rank[kOneRounds];
#pragma unroll
    for (int j = 0; j < kOneRounds; ++j) {
        const int i = warp * (32 * kOneRounds) + j * 32 + lane;
        pos[j] = i;
        key[j] = i < a.N ? sort_key(a, i) : -1;
    }
    for (int shift = 0; shift < bits; shift += kBits) {
        for (int i = lane; i < kBins / 2; i += 32) ((unsigned *)m.cnt[warp])[i] = 0u;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kOneRounds; ++j) {
            const int dg = key[j] < 0 ? kBins : (key[j] >> shift) & (kBins - 1);
            const unsigned peers = __match_any_sync(~0u, dg);
            rank[j] = dg < kBins ? m.cnt[warp][dg] + __popc(peers & ((1u << lane) - 1u)) : 0;
            __syncwarp();
            if (dg < kBins && lane == __ffs(peers) - 1) m.cnt[warp][dg] = (unsigned short)(m.cnt[warp][dg] + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        int total = 0;
        if (tid < kBins)  // counts -> places among the digit's keys
            for (int w = 0; w < kOneWarps; ++w) {
                const int c = m.cnt[w][tid];
                m.cnt[w][tid] = (unsigned short)total;
                total += c;
            }
        const int first = block_exclusive(tid < kBins ? total : 0, m.warp_sums);  // of the digit
        if (tid < kBins)
            for (int w = 0; w < kOneWarps; ++w) m.cnt[w][tid] = (unsigned short)(m.cnt[w][tid] + first);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kOneRounds; ++j) {
            if (key[j] < 0) continue;
            const int o = m.cnt[warp][(key[j] >> shift) & (kBins - 1)] + rank[j];
            m.key[o] = key[j];
            m.pos[o] = (unsigned short)pos[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kOneRounds; ++j) {
            const int i = warp * (32 * kOneRounds) + j * 32 + lane;
            if (i < a.N) {
                key[j] = m.key[i];
                pos[j] = m.pos[i];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kOneRounds; ++j) {
        const int i = warp * (32 * kOneRounds) + j * 32 + lane;
        if (i < a.N) {
            a.key_out[i] = key[j];
            a.pos_out[i] = pos[j];
        }
    }
}

// ---------------------------------------------------------------- gradient
constexpr int kUnit = 32, kShortUnit = 8;  // sorted positions of a unit; of one where units are few
constexpr int kColThreads = 256;

struct GradArgs {
    const int *key, *pos;  // [N] sorted tokens (padding = vocab, last) and their positions
    const void *dx;
    float *dtable, *pfirst, *plast;
    Ctrl *ctrl;
    float scale;
    int N, vocab, I, units, accumulate;
};

// W consecutive columns a thread: 4 where the rows of both dx and dtable are
// whole, aligned groups of four, else 1.
template <class T, int W> __device__ __forceinline__ void load_cols(const T *p, float (&f)[W]);
template <> __device__ __forceinline__ void load_cols<float, 1>(const float *p, float (&f)[1]) { f[0] = __ldg(p); }
template <> __device__ __forceinline__ void load_cols<bf16, 1>(const bf16 *p, float (&f)[1]) { f[0] = to_f(*p); }
template <> __device__ __forceinline__ void load_cols<f16, 1>(const f16 *p, float (&f)[1]) { f[0] = to_f(*p); }
template <> __device__ __forceinline__ void load_cols<float, 4>(const float *p, float (&f)[4]) {
    const float4 v = __ldg((const float4 *)p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <class T> __device__ __forceinline__ void load4_16(const T *p, float (&f)[4]) {
    const uint2 v = __ldg((const uint2 *)p);
    const typename Elem<T>::E2 *h = (const typename Elem<T>::E2 *)&v;
    const float2 a = Elem<T>::to_f2(h[0]), b = Elem<T>::to_f2(h[1]);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
template <> __device__ __forceinline__ void load_cols<bf16, 4>(const bf16 *p, float (&f)[4]) { load4_16(p, f); }
template <> __device__ __forceinline__ void load_cols<f16, 4>(const f16 *p, float (&f)[4]) { load4_16(p, f); }
template <int W> __device__ __forceinline__ void store_cols(float *p, const float (&f)[W]) {
    if (W == 4)
        *(float4 *)p = make_float4(f[0], f[W > 1 ? 1 : 0], f[W > 2 ? 2 : 0], f[W > 3 ? 3 : 0]);
    else
        p[0] = f[0];
}
// A: float or double, what the sum was taken in; the product is rounded once.
template <int W, class A>
__device__ __forceinline__ void store_row(const GradArgs &a, int w, int col, const A (&acc)[W]) {
    float *p = a.dtable + (long long)w * a.I + col;
    float f[W];
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = (float)(acc[i] * (A)a.scale);
    if (a.accumulate) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] += p[i];
    }
    store_cols<W>(p, f);
}

// 32768 rows x 1024 float into a table of 32000 rows 28 us (134 MB read, 83
// written: 7.7 TB/s, the written part in L2); of 2049 x 260 the latency of eight
// rows.
template <class T, int W, int UNIT>
__global__ void __launch_bounds__(kColThreads) grad_kernel(GradArgs a) {
    __shared__ int skey[UNIT + 2], spos[UNIT];
    const int tid = threadIdx.x;
    const int col = (blockIdx.y * kColThreads + tid) * W;
    clear_ctrl(a.ctrl);
    const int u0 = blockIdx.x * UNIT, n = min(UNIT, a.N - u0);
    if (tid < n) {
        skey[tid + 1] = a.key[u0 + tid];
        spos[tid] = a.pos[u0 + tid];
    }
    if (tid == kColThreads - 1) skey[0] = u0 > 0 ? a.key[u0 - 1] : -1;
    if (tid == kColThreads - 2) skey[n + 1] = u0 + n < a.N ? a.key[u0 + n] : -1;
    __syncthreads();
    if (col >= a.I) return;
    const T *dx = (const T *)a.dx + col;
    float acc[W] = {};
    int start = 0;
    for (int i0 = 0; i0 < n; i0 += 8) {
        float f[8][W];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j;
            if (i < n && skey[i + 1] < a.vocab) load_cols<T, W>(dx + (long long)spos[i] * a.I, f[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j;
            if (i >= n) break;
            const int w = skey[i + 1];
            if (w >= a.vocab) return;  // padding is last
#pragma unroll
            for (int c = 0; c < W; ++c) acc[c] += f[j][c];
            const bool more = skey[i + 2] == w;  // the token goes on at i + 1
            if (!more || i == n - 1) {
                if (start == 0 && skey[0] == w)
                    store_cols<W>(a.pfirst + (long long)blockIdx.x * a.I + col, acc);
                else if (more)
                    store_cols<W>(a.plast + (long long)blockIdx.x * a.I + col, acc);
                else
                    store_row(a, w, col, acc);
                start = i + 1;
#pragma unroll
                for (int c = 0; c < W; ++c) acc[c] = 0.f;
            }
        }
    }
}

// One block per unit; only a unit in which a token begins that goes on in the
// next one has work.  Four thread groups take every fourth of the units the
// token goes on in; their sums are added in a fixed order.  The sums of units are
// added in double: of 131072 rows of one token a float chain of 1024 units lost
// 5e-7, and there is one to add per 32 rows.  13 us (10 in float)
// beside the 28 above: the most frequent tokens, whose units one block adds.
constexpr int kJoinGroups = 4, kJoinCols = 64;
template <int W, int UNIT>
__global__ void __launch_bounds__(kJoinGroups *kJoinCols) join_kernel(GradArgs a) {
    const int u = blockIdx.x, last = u * UNIT + UNIT - 1;
    if (last + 1 >= a.N) return;
    const int w = a.key[last], after = a.key[last + 1], before = u > 0 ? a.key[u * UNIT - 1] : -1;
    if (w >= a.vocab || after != w) return;
    if (before == w) return;  // began before this unit
    __shared__ double part[kJoinGroups][kJoinCols * W];
    // units u+1 .. end-1 hold the rest: those whose first token is w
    const int tid = threadIdx.x;
    int end = u + 1, more;
    do {
        const int v = end + tid;
        more = __syncthreads_count(v < a.units && a.key[(long long)min(v, a.units - 1) * UNIT] == w);
        end += more;
    } while (more == kJoinGroups * kJoinCols);
    const int g = tid / kJoinCols, c0 = tid % kJoinCols;
    const int col = (blockIdx.y * kJoinCols + c0) * W;
    double acc[W] = {};
    if (col < a.I) {
        if (g == 0) {
            float f[W];
            load_cols<float, W>(a.plast + (long long)u * a.I + col, f);
#pragma unroll
            for (int c = 0; c < W; ++c) acc[c] = f[c];
        }
        for (int v0 = u + 1 + g; v0 < end; v0 += 8 * kJoinGroups) {
            float f[8][W];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (v0 + j * kJoinGroups < end)
                    load_cols<float, W>(a.pfirst + (long long)(v0 + j * kJoinGroups) * a.I + col, f[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (v0 + j * kJoinGroups < end) {
#pragma unroll
                    for (int c = 0; c < W; ++c) acc[c] += (double)f[j][c];
                }
        }
    }
#pragma unroll
    for (int c = 0; c < W; ++c) part[g][c0 * W + c] = acc[c];
    __syncthreads();
    if (g == 0 && col < a.I) {
#pragma unroll
        for (int c = 0; c < W; ++c)
            acc[c] = ((part[0][c0 * W + c] + part[1][c0 * W + c]) + part[2][c0 * W + c]) + part[3][c0 * W + c];
        store_row(a, w, col, acc);
    }
}

// --------------------------------------------------------------- workspace
struct BwdLayout {
    size_t key[2], pos[2], hist[2], pfirst, plast, total;
    int unit, units;
};

// Units of 32 positions keep the partial sums few; where they would leave SMs
// without a block, units of 8.  (us, of 8 / of 32: 128 ids x 1024 into 32000 rows
// 27 / 33, 2049 x 260 into 50001 18 / 21, 4096 x 1024 36 / 37; 8192 x 1024 49 / 47,
// 16384 x 512 40 / 35, 32768 x 64 39 / 31.)
int unit_of(const lstm_embed_dims *d) {
    const long long blocks = (((long long)d->N + kUnit - 1) / kUnit) * ((d->I + 4 * kColThreads - 1) / (4 * kColThreads));
    return blocks < host::sm_count() ? kShortUnit : kUnit;
}
BwdLayout bwd_layout(const lstm_embed_dims *d) {
    BwdLayout l;
    size_t o = kCtrlBytes;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    l.unit = unit_of(d);
    l.units = (d->N + l.unit - 1) / l.unit;
    for (int i = 0; i < 2; ++i) {
        l.key[i] = take((size_t)d->N * 4);
        l.pos[i] = take((size_t)d->N * 4);
    }
    for (int i = 0; i < 2; ++i) l.hist[i] = take((size_t)kSortBlocks * kBins * 4);
    l.pfirst = take((size_t)l.units * d->I * 4);
    l.plast = take((size_t)l.units * d->I * 4);
    l.total = o;
    return l;
}

bool dims_ok(const lstm_embed_dims *d) {
    if (!d || d->N < 0 || d->vocab < 0 || d->I < 0) return false;
    if (!host::dtype_ok(d->dtype) || (d->id_bytes != 4 && d->id_bytes != 8)) return false;
    return true;
}

// A vocabulary of 2^30 rows or a row of 2^24 elements leaves room for every
// 32-bit index of the kernels (sort keys up to vocab, columns + tile).
bool dims_supported(const lstm_embed_dims *d) { return d->vocab <= (1 << 30) && d->I <= (1 << 24) && d->N <= INT_MAX - 4 * kTile * kSortBlocks; }

template <class T, int W, int UNIT> int grad(const lstm_embed_dims *d, GradArgs &a, cudaStream_t s) {
    const int tiles = (d->I + kColThreads * W - 1) / (kColThreads * W);
    const int jtiles = (d->I + kJoinCols * W - 1) / (kJoinCols * W);
    if (tiles > 65535 || jtiles > 65535) return LSTM_ERR_UNSUPPORTED;
    grad_kernel<T, W, UNIT><<<dim3(a.units, tiles), kColThreads, 0, s>>>(a);
    LSTM_CUDA_TRY(host::launched());
    if (a.units > 1) {
        join_kernel<W, UNIT><<<dim3(a.units, jtiles), kJoinGroups * kJoinCols, 0, s>>>(a);
        LSTM_CUDA_TRY(host::launched());
    }
    return LSTM_OK;
}

template <class T> int grad_w(const lstm_embed_dims *d, GradArgs &a, cudaStream_t s) {
    const bool wide = d->I % 4 == 0 && (uintptr_t)a.dx % (4 * sizeof(T)) == 0 && (uintptr_t)a.dtable % 16 == 0;
    if (unit_of(d) == kUnit) return wide ? grad<T, 4, kUnit>(d, a, s) : grad<T, 1, kUnit>(d, a, s);
    return wide ? grad<T, 4, kShortUnit>(d, a, s) : grad<T, 1, kShortUnit>(d, a, s);
}

}  // namespace

extern "C" {

int lstm_embed_fwd(const lstm_embed_dims *d, const void *ids, const void *table, float scale, void *x,
                   void *stream) {
    if (!dims_ok(d)) return LSTM_ERR_INVALID_ARG;
    if (!dims_supported(d)) return LSTM_ERR_UNSUPPORTED;
    const bool any = (long long)d->N * d->I > 0;
    const size_t e = host::elem_bytes(d->dtype);
    if (!host::ptr_ok(ids, any, d->id_bytes) || !host::ptr_ok(table, any && d->vocab > 0, e) ||
        !host::ptr_ok(x, any, e))
        return LSTM_ERR_INVALID_ARG;
    if (!any) return LSTM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const bool l = d->id_bytes == 8;
    if (d->dtype == LSTM_F32)
        return l ? lookup<float, long long>(d, ids, table, scale, x, s) : lookup<float, int>(d, ids, table, scale, x, s);
    if (d->dtype == LSTM_F16)
        return l ? lookup<f16, long long>(d, ids, table, scale, x, s) : lookup<f16, int>(d, ids, table, scale, x, s);
    return l ? lookup<bf16, long long>(d, ids, table, scale, x, s) : lookup<bf16, int>(d, ids, table, scale, x, s);
}

size_t lstm_embed_bwd_workspace_size(const lstm_embed_dims *d) {
    if (!dims_ok(d) || !dims_supported(d)) return 0;
    return bwd_layout(d).total;
}

int lstm_embed_bwd(const lstm_embed_dims *d, const void *ids, const void *dx, float scale, int accumulate,
                   float *dtable, void *ws, size_t ws_bytes, void *stream) {
    if (!dims_ok(d) || (accumulate != 0 && accumulate != 1)) return LSTM_ERR_INVALID_ARG;
    if (!dims_supported(d)) return LSTM_ERR_UNSUPPORTED;
    const bool any = (long long)d->N * d->I > 0, out = (long long)d->vocab * d->I > 0;
    if (!host::ptr_ok(ids, any, d->id_bytes) || !host::ptr_ok(dx, any, host::elem_bytes(d->dtype)) ||
        !host::ptr_ok(dtable, out, 4))
        return LSTM_ERR_INVALID_ARG;
    const BwdLayout l = bwd_layout(d);
    const int rc = host::ws_check(ws, ws_bytes, l.total);
    if (rc != LSTM_OK) return rc;
    if (!out) return LSTM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    char *w = (char *)ws;
    // sort: enough 9-bit passes for the largest key, which is vocab (padding)
    if (d->N == 0) {
        LSTM_CUDA_TRY(cudaMemsetAsync(ws, 0, kCtrlBytes, s));
        if (!accumulate) LSTM_CUDA_TRY(cudaMemsetAsync(dtable, 0, (size_t)d->vocab * d->I * 4, s));
        return LSTM_OK;
    }
    int cur = 0, bits = 1;
    while (bits < 31 && (d->vocab >> bits) != 0) ++bits;
    SortArgs a = {};
    const long long tiles = ((long long)d->N + kTile - 1) / kTile;
    a.tiles = (int)((tiles + kSortBlocks - 1) / kSortBlocks);
    a.blocks = (int)((tiles + a.tiles - 1) / a.tiles);
    a.id64 = d->id_bytes == 8;
    a.vocab = d->vocab;
    a.N = d->N;
    a.ids = ids;
    // a launch clears the parts from .. to - 1 of `of` of the table: its blocks for that
    const long long cells = accumulate ? 0 : (long long)d->vocab * d->I;
    auto share = [&](int from, int to, int of, int threads) {
        const long long b = cells / of * from, e = to == of ? cells : cells / of * to;
        a.zero = {dtable + b, e - b};
        return (int)std::min<long long>(2 * host::sm_count(), (a.zero.n + 4 * threads - 1) / (4 * threads));
    };
    if (d->N <= kOneKeys) {
        a.key_out = (int *)(w + l.key[0]);
        a.pos_out = (int *)(w + l.pos[0]);
        const int extra = share(0, 1, 1, kOneThreads);
        LSTM_CUDA_TRY(cudaFuncSetAttribute(sort_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(OneSmem)));
        sort_one_kernel<<<1 + extra, kOneThreads, sizeof(OneSmem), s>>>(a, bits);
        LSTM_CUDA_TRY(host::launched());
    } else {
        int *hist[2] = {(int *)(w + l.hist[0]), (int *)(w + l.hist[1])};
        const int passes = (bits + kBits - 1) / kBits, shares = 2 * passes + 1;  // a scatter takes twice as long as the histograms
        a.hist = hist[0];
        a.hist_next = hist[1];
        int extra = share(0, 1, shares, kSortThreads);
        sort_hist_kernel<<<a.blocks + extra, kSortThreads, 0, s>>>(a);
        LSTM_CUDA_TRY(host::launched());
        for (int pass = 0; pass < passes; ++pass) {
            const bool more = pass + 1 < passes;
            a.shift = pass * kBits;
            a.key_out = (int *)(w + l.key[cur]);
            a.pos_out = (int *)(w + l.pos[cur]);
            a.hist = hist[0];
            a.hist_next = more ? hist[1] : nullptr;
            if (more && pass > 0) LSTM_CUDA_TRY(cudaMemsetAsync(hist[1], 0, (size_t)a.blocks * kBins * 4, s));
            extra = share(2 * pass + 1, 2 * pass + 3, shares, kSortThreads);
            sort_scatter_kernel<<<a.blocks + extra, kSortThreads, 0, s>>>(a);
            LSTM_CUDA_TRY(host::launched());
            a.ids = nullptr;
            a.key_in = a.key_out;
            a.pos_in = a.pos_out;
            std::swap(hist[0], hist[1]);
            cur ^= 1;
        }
        cur ^= 1;
    }
    GradArgs g = {};
    g.key = (const int *)(w + l.key[cur]);
    g.pos = (const int *)(w + l.pos[cur]);
    g.dx = dx;
    g.dtable = dtable;
    g.pfirst = (float *)(w + l.pfirst);
    g.plast = (float *)(w + l.plast);
    g.ctrl = (Ctrl *)ws;
    g.scale = scale;
    g.N = d->N;
    g.vocab = d->vocab;
    g.I = d->I;
    g.units = l.units;
    g.accumulate = accumulate;
    if (d->dtype == LSTM_F32) return grad_w<float>(d, g, s);
    if (d->dtype == LSTM_F16) return grad_w<f16>(d, g, s);
    return grad_w<bf16>(d, g, s);
}

}  // extern "C"
