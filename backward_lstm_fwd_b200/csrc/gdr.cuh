// gdr.cuh -- kernels of the gated delta rule, a recurrent layer whose state
// of a head is a matrix S [K][V]:
//   S' = e^{g_t} S_{t-1},  x_t = v_t - S'^T k_t,  S_t = S' + beta_t k_t x_t^T,
//   o_t = scale S_t^T q_t.
//
// Chunked form (64 tokens).  With b_i the running sum of g in the chunk,
// gamma_i = e^{b_i}, Gamma_ij = e^{b_i - b_j} for i >= j, left_i = e^{b_63 - b_i}:
//   N  = strictly lower part of Gamma o (K K^T),   T2 = (1 + N diag(beta))^-1
//   P  = scale (lower part of Gamma o (Q K^T))
//   X  = T2 (V - diag(gamma) K S0),                U  = diag(beta) X
//   O  = scale diag(gamma) Q S0 + P U
//   S1 = gamma_63 S0 + K^T diag(left) U
// and backward, from dO and dS1:
//   dU  = P^T dO + diag(left) K dS1,               dV = T2^T diag(beta) dU
//   dS0 = gamma_63 dS1 + scale Q^T diag(gamma) dO - K^T diag(gamma) dV
//   Y = dO X^T, Z = dV X^T, E = X dS1^T, F = dO S0^T, G = dV S0^T
//   Yh = scale Gamma o Y diag(beta) (i >= j), Zh = Gamma o Z diag(beta) (i > j)
//   dQ = scale diag(gamma) F + Yh K
//   dK = Yh^T Q - (Zh + Zh^T) K + diag(left beta) E - diag(gamma) G
//   w_rj = Gamma_rj (scale (q_r.k_j) Y_rj - [r > j] (k_r.k_j) Z_rj)
//   dbeta_j = sum_r w_rj + left_j k_j.E_j
//   dg_i = sum_{r >= i > j} w_rj beta_j + sum_{r >= i} gamma_r (scale q_r.F_r - k_r.G_r)
//        + sum_{j < i} left_j beta_j k_j.E_j + gamma_63 <dS1, S0>
//
// Kernels: prep (every chunk at once: operand tiles, T2, P, gates), seq_fwd /
// seq_bwd (one block per head walks its chunks, the state in registers), grad
// (every chunk at once) and step (token by token, for a few tokens).
//
// Numbers.  The contractions run on the tensor cores in bf16 with float
// accumulators, every float operand split into three bf16 terms (8 + 8 + 8
// bits of its 24) and the products of orders 0, 1 and 2 kept: what is dropped
// is 2^-24 of the operands, below the rounding of a float sum.  (An accumulator
// drops what lies below its last place at every step; the small products come first,
// so that few steps meet the full sum.  Errors in norm: 1e-7 to 3e-7 of o, the states
// and their gradient, up to 1.7e-6 of dq and dk at V = 256, sums of four passes.)
// bf16 inputs are one term, fp16 two, fp32 three, each exactly the input.  Running
// sums of g are double: b_i - b_j of a float sum would lose the digits that a
// strong decay needs between its neighbours.
#pragma once

#include "host.cuh"
#include "tc_ptx.cuh"

namespace lstm {
namespace gdr {

typedef __nv_bfloat16 bf16;
typedef __half f16;

constexpr int C = LSTM_GDR_CHUNK;  // tokens of a chunk
static_assert(C == 64, "tiles and tensor-memory columns are laid out for 64 tokens");
constexpr int NT = 3;              // bf16 terms of a float operand
constexpr int TILE = C * 128;      // 64 rows x 64 bf16, 128-byte swizzled: 8 KB
constexpr int LANES = 128;         // columns of the state a block looks after (TMEM lanes)
constexpr int GATES = 3 * C * 4;   // bytes of a chunk's gates: gamma, left, beta [64] floats

template <class E> struct Terms;   // bf16 terms of an input type
template <> struct Terms<bf16> { static constexpr int n = 1; };
template <> struct Terms<f16> { static constexpr int n = 2; };
template <> struct Terms<float> { static constexpr int n = 3; };

// One chunk of one key head: for each term, KD / 64 chunks of [q 64 rows][k 64 rows] x 64.
template <class E, int KD> struct QK {
    static constexpr int term = KD / 64 * 2 * TILE, bytes = Terms<E>::n * term;
};
// One chunk of one value head: T2 terms, P terms, gates.
constexpr int TP_BYTES = 2 * NT * TILE + GATES;

struct Shape {
    int T, B, Hk, Hv, K, V, group, NC, VT;  // NC chunks, VT blocks of 128 state columns
    long long ldq, ldk, ldv;                // elements between tokens (rows t * B + b)
    float scale;
    const int *lengths;
};

__device__ __forceinline__ int length_of(const Shape &s, int b) {
    return s.lengths ? max(0, min(s.T, s.lengths[b])) : s.T;
}

// ------------------------------------------------------------ conversions
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Two floats -> n packed bf16 pairs whose sum is the floats (n = 3: to 2^-24).
template <int n> __device__ __forceinline__ void split2(float a, float b, uint32_t (&t)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
        t[i] = pack2(a, b);
        if (i + 1 < n)
            asm("{\n\t.reg .b64 x, y;\n\t"
                "mov.b64 x, {%0, %1};\n\t"
                "mov.b64 y, {%2, %3};\n\t"
                "sub.rn.f32x2 x, x, y;\n\t"
                "mov.b64 {%0, %1}, x;\n\t}"
                : "+f"(a), "+f"(b)
                : "f"(low_f(t[i])), "f"(high_f(t[i])));
    }
}

// (x, y) += a (bx, by)
__device__ __forceinline__ void fma2(float &x, float &y, float a, float bx, float by) {
    asm("{\n\t.reg .b64 d, a, b;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "fma.rn.f32x2 d, a, b, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(bx), "f"(by));
}

// byte offset of (row, byte column) in a 128-byte swizzled tile
__device__ __forceinline__ uint32_t swz(int row, int cb) { return row * 128 + (cb ^ ((row & 7) << 4)); }

// Eight consecutive elements, raw, and their terms.
template <class E> struct Raw8 { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };
template <class E> __device__ __forceinline__ Raw8<E> raw8(const E *p, bool in) {
    Raw8<E> r = {};
    if (in) {
        r.a = __ldg((const uint4 *)p);
        if constexpr (sizeof(E) == 4) r.b = __ldg((const uint4 *)p + 1);
    }
    return r;
}

// Eight consecutive elements as floats.
template <class E> __device__ __forceinline__ void load8(const E *p, float (&f)[8]) { x8_to_f32<E>(__ldg((const uint4 *)p), f); }
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&f)[8]) {
    const float4 a = __ldg((const float4 *)p), b = __ldg((const float4 *)p + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// n terms of eight floats as 16-byte groups.
template <int n> __device__ __forceinline__ void split8(const float (&f)[8], uint4 (&o)[n]) {
    uint32_t t[4][n];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<n>(f[2 * i], f[2 * i + 1], t[i]);
#pragma unroll
    for (int k = 0; k < n; ++k) o[k] = make_uint4(t[0][k], t[1][k], t[2][k], t[3][k]);
}

template <class E> __device__ __forceinline__ void terms8(const Raw8<E> &r, uint4 (&o)[Terms<E>::n]) {
    if constexpr (Terms<E>::n == 1) {
        o[0] = r.a;
    } else {
        float f[8];
        if constexpr (sizeof(E) == 4) {
            f[0] = __uint_as_float(r.a.x); f[1] = __uint_as_float(r.a.y); f[2] = __uint_as_float(r.a.z); f[3] = __uint_as_float(r.a.w);
            f[4] = __uint_as_float(r.b.x); f[5] = __uint_as_float(r.b.y); f[6] = __uint_as_float(r.b.z); f[7] = __uint_as_float(r.b.w);
        } else {
            x8_to_f32<E>(r.a, f);
        }
        split8<Terms<E>::n>(f, o);
    }
}

// ------------------------------------------------------------ descriptors
// Tiles are [rows][64] bf16, 128-byte swizzled.  As a K-major operand the rows
// are M or N and a K = 16 step moves 32 bytes; as an MN-major operand the rows
// are K (a step moves 16 rows, 2048 bytes) and 64-wide chunks are lbo apart.
__device__ __forceinline__ uint64_t k_major(uint32_t tile, int ks) { return tc::smem_desc_sw128(tile + ks * 32, 16, 1024); }
__device__ __forceinline__ uint64_t mn_major(uint32_t tile, int ks, uint32_t lbo) {
    return tc::smem_desc_sw128(tile + ks * 2048, lbo, 1024);
}

// Write 2 n floats of this thread's lane as terms: term t of pair i goes to
// column col + t * stride + i.  n a multiple of 8.
template <int n, int terms>
__device__ __forceinline__ void put_terms(uint32_t col, int stride, const float (&f)[2 * n]) {
#pragma unroll
    for (int i0 = 0; i0 < n; i0 += 8) {
        uint32_t r[terms][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t t[terms];
            split2<terms>(f[2 * (i0 + i)], f[2 * (i0 + i) + 1], t);
#pragma unroll
            for (int k = 0; k < terms; ++k) r[k][i] = t[k];
        }
#pragma unroll
        for (int k = 0; k < terms; ++k) tc::tmem_st8(col + k * stride + i0, r[k]);
    }
}

// One thread: D (+)= A B^T over the products of term t of A and u of B with
// t + u < orders, t < ta, u < tb, the smallest products first (a float
// accumulator of the tensor core drops what lies below its last bit, so the
// small ones are summed while it is small).  A in tensor memory (a_term
// columns between terms) or shared memory (A_SMEM: a is a descriptor); b a
// descriptor; term and step distances in 16-byte units.  steps K = 16 each,
// in chunks of four `chunk` apart.
struct Steps {
    uint32_t term, step, chunk;  // 16-byte units
};
__device__ __forceinline__ constexpr uint32_t at_step(const Steps &x, int t, int ks) {
    return t * x.term + (ks >> 2) * x.chunk + (ks & 3) * x.step;
}
template <int steps, int ta, int tb, int orders>
__device__ __forceinline__ void products_ts(uint32_t d, uint32_t a, uint32_t a_term, uint64_t b, const Steps bs,
                                            uint32_t idesc, uint32_t acc = 0) {
#pragma unroll
    for (int o = orders - 1; o >= 0; --o)
#pragma unroll
        for (int t = 0; t < ta; ++t) {
            if (t > o || o - t >= tb) continue;
#pragma unroll
            for (int ks = 0; ks < steps; ++ks) {
                tc::mma_bf16_ts(d, a + t * a_term + 8 * ks, b + at_step(bs, o - t, ks), idesc, acc);
                acc = 1;
            }
        }
}
// The sum of two such products, A in tensor memory.
template <int steps, int ta, int tb, int orders>
__device__ __forceinline__ void two_products_ts(uint32_t d, uint32_t a0, uint64_t b0, uint32_t a1, uint64_t b1,
                                                uint32_t a_term, const Steps bs, uint32_t idesc) {
    uint32_t acc = 0;
#pragma unroll
    for (int o = orders - 1; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int t = 0; t < ta; ++t) {
                if (t > o || o - t >= tb) continue;
#pragma unroll
                for (int ks = 0; ks < steps; ++ks) {
                    tc::mma_bf16_ts(d, (p ? a1 : a0) + t * a_term + 8 * ks, (p ? b1 : b0) + at_step(bs, o - t, ks), idesc, acc);
                    acc = 1;
                }
            }
}
template <int steps, int ta, int tb, int orders>
__device__ __forceinline__ void products_ss(uint32_t d, uint64_t a, const Steps as, uint64_t b, const Steps bs,
                                            uint32_t idesc, uint32_t acc = 0) {
#pragma unroll
    for (int o = orders - 1; o >= 0; --o)
#pragma unroll
        for (int t = 0; t < ta; ++t) {
            if (t > o || o - t >= tb) continue;
#pragma unroll
            for (int ks = 0; ks < steps; ++ks) {
                tc::mma_bf16(d, a + at_step(as, t, ks), b + at_step(bs, o - t, ks), idesc, acc);
                acc = 1;
            }
        }
}

__device__ __forceinline__ void get16(uint32_t col, float (&f)[16]) {
    uint32_t r[16];
    tc::tmem_ld16(col, r);
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void set16(uint32_t col, const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(f[i + j]);
        tc::tmem_st8(col + i, r);
    }
}

// A bounded wait of a whole warp, ordered before its tensor-memory accesses.
// The hint lets the hardware hold the warp for up to 20 us a try, so that
// waiting warps leave the issue slots to the others.  After a time-out (2 s)
// every later wait returns at once: the block runs to its end on what is
// there, and the status word says so.
__device__ __forceinline__ bool try_wait_hint(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, Ctrl *ctrl, volatile int *abort_flag, uint32_t site) {
    if (!try_wait_hint(bar, parity)) {
        const uint64_t t0 = tc::globaltimer_ns();
        while (!try_wait_hint(bar, parity) && !*abort_flag) {
            if (tc::globaltimer_ns() - t0 > 2000000000ull) {
                atomicCAS(&ctrl->status, 0u, 5u);
                atomicCAS(&ctrl->fail_site, 0u, site);
                *abort_flag = 1;
            }
        }
    }
    __syncwarp();
    tc::tc_fence_after();
}
// One lane of a converged warp (the same one every time).  A branch on it
// inside a warp-uniform branch keeps addresses and descriptors in uniform
// registers: 38 cycles per N = 64 product against 51 under threadIdx.x == 0.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int warp_id() { return __shfl_sync(~0u, threadIdx.x >> 5, 0); }

// Untiled bulk copy global -> this block's shared memory (16-byte aligned).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
        : "memory");
}

// ------------------------------------------------------------------- gates
// Running sums b of the chunk's g, times log2(e), as float pairs hi + lo of a
// double sum: b_i - b_j keeps its digits where a strong decay made both large,
// and e^{b_i - b_j} is three additions and one exponential (2^-22 relative).
struct Sums {
    float2 b[C];    // (hi, lo)
    float beta[C];
    float col[C], col_beta[C];  // prep: e^{b_r - b_j}, r the last token of j's 16, and times beta_j
};
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float decay(float2 i, float2 j) { return ex2((i.x - j.x) + (i.y - j.y)); }
__device__ __forceinline__ float decay(float2 i) { return ex2(i.x + i.y); }

// Warp 0, two tokens a lane.  Padding (t >= len) has g = 0 and beta = 0.  g =
// -inf (or below -1e5) counts as -1e5: its exponential is zero all the same.
__device__ __forceinline__ void load_gates(const Shape &s, const float *g, const float *beta, int c, int b,
                                           int h, int len, Sums &out) {
    const int lane = threadIdx.x & 31;
    double v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 2 * lane + i, t = c * C + j;
        const long long at = ((long long)t * s.B + b) * s.Hv + h;
        const float gv = t < len ? g[at] : 0.f;
        v[i] = (gv < -1e5f ? -1e5 : (double)gv) * 1.4426950408889634;
        out.beta[j] = t < len ? beta[at] : 0.f;
    }
    v[1] += v[0];
    double sum = v[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += y;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double x = sum - v[1] + v[i];
        const float hi = (float)x;
        out.b[2 * lane + i] = make_float2(hi, (float)(x - hi));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 2 * lane + i;
        out.col[j] = decay(out.b[j | 15], out.b[j]);
        out.col_beta[j] = out.col[j] * out.beta[j];
    }
}

// -------------------------------------------------------------------- prep
// Block (c, b, hk), 128 threads: the operand tiles of q and k (swizzled, in
// terms, zero for padding and past K), then per value head of the group T2,
// P and the gates, all in the layout the other kernels copy in bulk.  (Where
// that leaves SMs idle, a block per value head, the tiles from the first.)
//
// Bound by the latency of the substitution's steps between its loads: bf16, K =
// 128, 2048 blocks of two value heads 105 us (334 MB, 3.2 TB/s), 1024 blocks 57.
// Five blocks an SM (six need spills: no gain).
//
// Q K^T and K K^T are one product of the stacked [Q; K] with K.  T2 is the
// inverse of a unit lower triangular matrix [A 0; B D] of 32 x 32 blocks:
// [A' 0; -D' B A', D'].  A' and D' come from forward substitution, a thread a
// column, one warp a block, while the other two warps form P; the block below
// is two products by all four warps.
struct PrepArgs {
    Shape s;
    const void *q, *k;
    const float *g, *beta;
    char *qk, *tp;
    Ctrl *ctrl;
    int heads;  // value heads a block takes: the group, or 1
};
constexpr int PREP_LD = 68;                    // floats between rows of a 64 x 64 matrix in shared memory
constexpr int PREP_MAT = C * PREP_LD * 4;

template <class E, int KD> struct PrepSmem {
    // the triangle (then T2) and P go where the operand tiles were
    static constexpr size_t smem = (QK<E, KD>::bytes > 2 * PREP_MAT ? QK<E, KD>::bytes : 2 * PREP_MAT) + 1024;
};

template <class E, int KD>
__global__ void __launch_bounds__(128, 5) prep_kernel(PrepArgs a) {
    constexpr int TB = Terms<E>::n;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *tri = (float *)tiles, *pm = (float *)(tiles + PREP_MAT);
    __shared__ Sums sums;
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const Shape &s = a.s;
    const int tid = threadIdx.x, warp = warp_id(), lane = tid & 31;
    clear_ctrl(a.ctrl);
    const int split = s.group / a.heads, m0 = blockIdx.x % split * a.heads;
    int id = blockIdx.x / split;
    char *out = m0 == 0 ? a.qk + (size_t)id * QK<E, KD>::bytes : nullptr;
    const int hk = id % s.Hk;
    id /= s.Hk;
    const int b = id % s.B, c = id / s.B;
    const int len = length_of(s, b);
    if (tid == 0) {
        tc::mbar_init(&done, 1);
        abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&tmem_slot, 64);
        tc::tmem_relinquish();
    }
    // tiles: rows 0..63 q, 64..127 k; 16-byte groups of 8 dims, eight loads in flight a thread
    // (thread tid keeps its group gr and takes rows row0, row0 + step, ...)
    constexpr int step = 128 / (KD / 8), U = 8;
    const int row0 = tid / (KD / 8), gr = tid % (KD / 8);
    const uint32_t col = (gr >> 3) * 2 * TILE, cb = (gr & 7) * 16;
#pragma unroll 1
    for (int i0 = row0; i0 < 128; i0 += U * step) {
        Raw8<E> f[U];
#pragma unroll
        for (int n = 0; n < U; ++n) {
            const int row = i0 + n * step, t = c * C + (row & 63);
            const long long r = (long long)t * s.B + b;
            f[n] = raw8<E>((row < 64 ? (const E *)a.q + r * s.ldq : (const E *)a.k + r * s.ldk) + (long long)hk * s.K + gr * 8,
                           t < len && gr * 8 < s.K);
        }
#pragma unroll
        for (int n = 0; n < U; ++n) {
            uint4 o[TB];
            terms8<E>(f[n], o);
            const uint32_t off = col + swz(i0 + n * step, cb);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                *(uint4 *)(tiles + t * QK<E, KD>::term + off) = o[t];
                if (out) *(uint4 *)(out + t * QK<E, KD>::term + off) = o[t];
            }
        }
    }
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (warp == 0 && elect_one()) {
        const uint32_t base = tc::smem_u32(tiles);
        const Steps st = {QK<E, KD>::term >> 4, 2, 2 * TILE >> 4};
        products_ss<KD / 16, TB, TB, NT>(tmem, k_major(base, 0), st, k_major(base + TILE, 0), st, tc::idesc_bf16_f32(128, 64, 0, 0));
        tc::mma_commit(&done);
    }
    __syncwarp();
    if (warp == 0) load_gates(s, a.g, a.beta, c, b, hk * s.group + m0, len, sums);
    wait(&done, 0, a.ctrl, &abort_flag, 0x601);
    __syncthreads();
    const int row = tid & 63;  // warps 0, 1: Q K^T; warps 2, 3: K K^T
    const int half = warp & 1;  // rows 32 half ..
    for (int m = m0; m < m0 + a.heads; ++m) {
        const int h = hk * s.group + m;
        char *tp = a.tp + (((size_t)c * s.B + b) * s.Hv + h) * TP_BYTES;
        const float2 bi = sums.b[row];
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        float *dst = (warp < 2 ? pm : tri) + row * PREP_LD;
#pragma unroll 1
        for (int j0 = 0; j0 < 32 * (half + 1); j0 += 16) {
            float f[16];
            get16(lanes + j0, f);
            if (j0 + 16 <= 32 * half) {  // (of the whole warp) e^{b_i - b_r} e^{b_r - b_j}, r the block's last column
                const float di = decay(bi, sums.b[j0 + 15]) * (warp < 2 ? s.scale : 1.f);
                const float *col = (warp < 2 ? sums.col : sums.col_beta) + j0;
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] *= di * col[j];
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int jj = j0 + j;
                    const float dec = decay(bi, sums.b[jj]);
                    if (warp < 2) f[j] = jj <= row ? s.scale * dec * f[j] : 0.f;
                    else f[j] = jj < row ? dec * sums.beta[jj] * f[j] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4) *(float4 *)(dst + j0 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
        }
        if (warp < 2) {
            float *gates = (float *)(tp + 2 * NT * TILE);
            gates[tid] = decay(bi);
            gates[C + tid] = decay(sums.b[C - 1], bi);
            gates[2 * C + tid] = sums.beta[tid];
        } else {
            __syncwarp();
            // column `lane` of the inverse of block (half, half): x_i = [i == lane] - sum_{m < i} tri[i][m] x_m
            float *blk = tri + half * 32 * PREP_LD + half * 32;  // becomes its inverse
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float p0 = i == lane ? 1.f : 0.f, p1 = 0.f, p2 = 0.f, p3 = 0.f;
#pragma unroll
                for (int mm = 0; mm < i; mm += 4) {
                    const float4 v = *(const float4 *)(blk + i * PREP_LD + mm);
                    p0 = fmaf(-v.x, x[mm], p0);
                    if (mm + 1 < i) p1 = fmaf(-v.y, x[mm + 1], p1);
                    if (mm + 2 < i) p2 = fmaf(-v.z, x[mm + 2], p2);
                    if (mm + 3 < i) p3 = fmaf(-v.w, x[mm + 3], p3);
                }
                x[i] = (p0 + p1) + (p2 + p3);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i) blk[i * PREP_LD + lane] = x[i];
        }
        __syncthreads();
        {  // block (1, 0): W = B A', into the upper right corner; then -D' W in B's place.  A' and D' are
           // triangles: warp w does W's columns 8 w .. (k >= 8 w), then the rows 8 w .. (k < 8 w + 8)
            float *low = tri + 32 * PREP_LD, *corner = tri + 32;
            float acc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 2
            for (int k = 8 * warp; k < 32; k += 4) {  // row `lane`
                const float4 lv = *(const float4 *)(low + lane * PREP_LD + k);
                const float le[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 u = *(const float4 *)(tri + (k + q) * PREP_LD + 8 * warp),
                                 v = *(const float4 *)(tri + (k + q) * PREP_LD + 8 * warp + 4);
                    fma2(acc[0], acc[1], le[q], u.x, u.y);
                    fma2(acc[2], acc[3], le[q], u.z, u.w);
                    fma2(acc[4], acc[5], le[q], v.x, v.y);
                    fma2(acc[6], acc[7], le[q], v.z, v.w);
                }
            }
            *(float4 *)(corner + lane * PREP_LD + 8 * warp) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            *(float4 *)(corner + lane * PREP_LD + 8 * warp + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
            __syncthreads();
            // column `lane`, rows 8 warp ..
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll 2
            for (int k = 0; k < 8 * warp + 8; k += 4) {
                float w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = -corner[(k + q) * PREP_LD + lane];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 dv = *(const float4 *)(low + 32 + (8 * warp + j) * PREP_LD + k);
                    acc[j] = fmaf(dv.x, w[0], acc[j]);
                    acc[j] = fmaf(dv.y, w[1], acc[j]);
                    acc[j] = fmaf(dv.z, w[2], acc[j]);
                    acc[j] = fmaf(dv.w, w[3], acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) low[(8 * warp + j) * PREP_LD + lane] = acc[j];
        }
        __syncthreads();
        if (warp == 0 && m + 1 < m0 + a.heads) load_gates(s, a.g, a.beta, c, b, h + 1, len, sums);
        // terms of T2 and P: eight threads a row, whole 128-byte lines a warp
#pragma unroll 2
        for (int i = tid; i < 2 * C * 8; i += 128) {
            const int mat = i >> 9, r = (i >> 3) & 63, gr = i & 7;
            float f[8];
            const float4 *src = (const float4 *)((mat ? pm : tri) + r * PREP_LD + gr * 8);
            float4 u = src[0], v = src[1];
            if (r < 32 && gr >= 4) u = v = make_float4(0.f, 0.f, 0.f, 0.f);  // above the diagonal (T2: W's place)
            f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
            f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
            uint4 o[NT];
            split8<NT>(f, o);
#pragma unroll
            for (int t = 0; t < NT; ++t) *(uint4 *)(tp + (mat * NT + t) * TILE + swz(r, gr * 16)) = o[t];
        }
        __syncthreads();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, 64);
}

// -------------------------------------------------------------- sequential
// Block (b, h, 128 columns of V): the chunks of one head in order.  Thread
// (wg, lane) holds column `lane` of S^T -- the state is kept transposed, V on
// the tensor-memory lanes -- for a quarter of K in registers.  Every
// contraction of the chain has its left operand in tensor memory, where the
// thread that owns the lane writes it, so nothing in the chain crosses lanes
// or goes through shared memory:
//   K S  ->  R = V - gamma K S  ->  X = T2 R  ->  U  ->  S += K^T (left U).
// Q S and P U run beside the chain; their sum is stored a chunk later.  The
// chunks' tiles come by bulk copies, a chunk ahead where two stages fit.
// Bound: the chain's latency (three products and three passes over registers
// a chunk) where there are few heads.  512 threads rather than 256: a pass
// over the registers is short code for many warps (with 256 threads the warps
// waited for instructions more than for anything else).  bf16, K = V = 128: 7.1
// us a chunk forward with the states stored, 5.1 without, 6.8 backward; 256 heads of
// 16 chunks, up to two blocks an SM in turn, 227 us and 218 us.
constexpr int SEQ_THREADS = 512;
// tensor-memory columns: S terms, then left U terms | K S, Q S, then K^T (left
// U) | R terms, then U terms | X, then P U
constexpr uint32_t COL_S = 0, COL_D = 192, COL_R = 320, COL_X = 416, COL_W = 96;

template <class E, int KD> struct Seq {
    static constexpr int stage = QK<E, KD>::bytes + 2 * NT * TILE;  // tiles; the gates lie behind the stages
    static constexpr int extra = 1024 + 256;                        // alignment, barriers
    static constexpr int stages = 2 * (stage + GATES) + extra <= 232448 ? 2 : 1;
    static constexpr size_t smem = (size_t)stages * (stage + GATES) + extra;
    static constexpr int TB = Terms<E>::n;
};

// Few heads and many chunks: the chunks are split into segments.  A head's
// state is carried over a segment by S -> A S + B, with A [K][K] the same for
// every column, so a first pass (SCAN) runs the segments side by side from a
// zero state, which leaves B, and from the identity, which leaves A; scan_kernel
// joins them to every segment's start, and a second pass runs all segments at
// once.  (seg: chunks of a segment, in the order of the pass.)  16 heads of 128
// chunks on 8 key heads: 90 us to scan, 21 to join, 112 to run, 274 with the
// preparation (on 16 key heads 289, where 16 SMs that walk 128 chunks each take 648).
struct SeqArgs {
    Shape s;
    const char *qk, *tp;
    const void *v;            // forward: v; backward: dout
    const float *s0;          // forward: s0; backward: dsT
    void *o;                  // forward: o; backward: dv
    float *sT;                // forward: sT; backward: ds0
    float *states, *deltas;   // forward (or NULL): S and X; backward: dS and dV, in the workspace
    float *starts;            // [segments - 1][B][Hv][K][V]: B, then the start of the next segment
    char *trans;              // [segments - 1][B][Hv]: A as NT terms of KD rows, swizzled
    int segments, seg;
    Ctrl *ctrl;
};

struct SeqBars {
    uint64_t full[2], m1, m2, m3, m4;
    uint32_t tmem_slot;
    int abort_flag;
};

// What a block of the sequential kernels works on.  Only chunks with tokens in
// them (c < live) are walked: padding leaves the state as it is, whatever it holds.
template <bool SCAN> struct Job {
    int vt, h, b, seg, first, chunks, live;
    bool identity;  // SCAN: the state columns are those of the identity
    __device__ __forceinline__ explicit Job(const SeqArgs &a) {
        const Shape &s = a.s;
        const int width = s.VT + (SCAN ? 1 : 0);
        int id = blockIdx.x;
        vt = id % width;
        id /= width;
        h = id % s.Hv;
        id /= s.Hv;
        b = id % s.B;
        seg = id / s.B;
        first = seg * a.seg;
        chunks = min(a.seg, s.NC - first);
        live = (length_of(s, b) + C - 1) / C;
        identity = SCAN && vt == s.VT;
        if (identity) vt = 0;
    }
};

// One thread: copy the tiles of the segment's n-th chunk to its stage.  The
// caller has seen the last products that read that stage complete.
template <class E, int KD>
__device__ __forceinline__ void seq_load(const SeqArgs &a, uint8_t *smem, SeqBars *bar, int b, int h, int n, int first, bool reverse) {
    using Q = Seq<E, KD>;
    const Shape &s = a.s;
    const int st = n % Q::stages, c = reverse ? s.NC - 1 - first - n : first + n;
    uint8_t *dst = smem + st * Q::stage;
    tc::mbar_arrive_expect_tx(&bar->full[st], Q::stage + GATES);
    const size_t cb = (size_t)c * s.B + b;
    bulk_load(dst, a.qk + (cb * s.Hk + h / s.group) * QK<E, KD>::bytes, QK<E, KD>::bytes, &bar->full[st]);
    const char *tp = a.tp + (cb * s.Hv + h) * TP_BYTES;
    bulk_load(dst + QK<E, KD>::bytes, tp, 2 * NT * TILE, &bar->full[st]);
    bulk_load(smem + Q::stages * Q::stage + st * GATES, tp + 2 * NT * TILE, GATES, &bar->full[st]);
}
// After a time-out the block may leave only when its copies have landed.
template <class E, int KD> __device__ __forceinline__ void seq_drain(SeqBars *bar, int chunks) {
    using Q = Seq<E, KD>;
    for (int n = max(0, chunks - Q::stages); n < chunks; ++n)
        tc::mbar_wait(&bar->full[n % Q::stages], (n / Q::stages) & 1, nullptr, nullptr, 0, 200000000ull);
}
__device__ __forceinline__ void seq_setup(SeqBars *bar) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) tc::mbar_init(&bar->full[i], 1);
        tc::mbar_init(&bar->m1, 1);
        tc::mbar_init(&bar->m2, 1);
        tc::mbar_init(&bar->m3, 1);
        tc::mbar_init(&bar->m4, 1);
        bar->abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (threadIdx.x < 32) {
        tc::tmem_alloc(&bar->tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
}
__device__ __forceinline__ void seq_finish(SeqBars *bar) {
    tc::tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32) tc::tmem_dealloc(bar->tmem_slot, 512);
}
// Every thread's tensor-memory writes are done; one thread of warp 0 issues
// the products that read them, in the branch.
__device__ __forceinline__ bool hand_over(int warp) {
    tc::tmem_st_wait();
    tc::tc_fence_before();
    __syncthreads();
    if (warp != 0) return false;
    tc::tc_fence_after();
    return elect_one();
}

// 16 consecutive values of shared memory (16-byte aligned).
__device__ __forceinline__ void load16(const float *p, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = ((const float4 *)p)[i];
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
}
// Elements p[i stride], i < n, of up to N (zero past n); and their stores.
template <int N, class T> __device__ __forceinline__ void load_col(const T *p, long long stride, int n, T (&r)[N]) {
    if (n >= N) {
#pragma unroll
        for (int i = 0; i < N; ++i, p += stride) r[i] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i, p += stride) r[i] = i < n ? *p : from_f<T>(0.f);
    }
}
// 16 loaded elements, 16-bit ones two to a register.
template <class E> struct Col16 {
    uint32_t x[sizeof(E) * 4];
    __device__ __forceinline__ void load(const E *p, long long stride, int n) {
        E r[16];
        load_col(p, stride, n, r);
        if constexpr (sizeof(E) == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = reinterpret_cast<const uint16_t &>(r[2 * i]) |
                       ((uint32_t) reinterpret_cast<const uint16_t &>(r[2 * i + 1]) << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(r[i]);
        }
        __syncwarp();
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(E) == 2) {
            const uint16_t h = (uint16_t)(x[i >> 1] >> (16 * (i & 1)));
            return to_f(reinterpret_cast<const E &>(h));
        } else {
            return __uint_as_float(x[i]);
        }
    }
};
template <int N, class T> __device__ __forceinline__ void store_col(T *p, long long stride, int n, const float (&r)[N]) {
    if (n >= N) {
#pragma unroll
        for (int i = 0; i < N; ++i, p += stride) *p = from_f<T>(r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i, p += stride)
            if (i < n) *p = from_f<T>(r[i]);
    }
    __syncwarp();
}

// What a thread of the sequential kernels works on.
template <int KD> struct Lane {
    int wg, v, len;
    bool own;
    uint32_t lanes;
    long long head, row;  // row: elements of o, deltas between tokens
    __device__ __forceinline__ Lane(const Shape &s, uint32_t tmem, int b, int h, int vt, bool identity) {
        const int lane = threadIdx.x & 127;
        wg = threadIdx.x >> 7;
        v = vt * LANES + lane;
        own = v < s.V && !identity;
        len = length_of(s, b);
        lanes = tmem + ((uint32_t)(lane & 96) << 16);
        head = (long long)b * s.Hv + h;
        row = (long long)s.B * s.Hv * s.V;
    }
    // rows k of a [K][V] state at `base`, this thread's quarter
    __device__ __forceinline__ int rows(const Shape &s, const float *base) const { return base && own ? s.K - wg * (KD / 4) : 0; }
    __device__ __forceinline__ void load(const Shape &s, const float *base, float (&S)[KD / 4]) const {
        load_col(base + (long long)wg * (KD / 4) * s.V + v, s.V, rows(s, base), S);
        __syncwarp();
    }
    __device__ __forceinline__ void store(const Shape &s, float *base, const float (&S)[KD / 4]) const {
        store_col(base + (long long)wg * (KD / 4) * s.V + v, s.V, rows(s, base), S);
    }
    // quarters FROM .. TO - 1 of those rows
    template <int FROM, int TO> __device__ __forceinline__ void store_part(const Shape &s, float *base, const float (&S)[KD / 4]) const {
        constexpr int n = KD / 16 * (TO - FROM), i0 = KD / 16 * FROM;
        float r[n];
#pragma unroll
        for (int i = 0; i < n; ++i) r[i] = S[i0 + i];
        store_col(base + (long long)(wg * (KD / 4) + i0) * s.V + v, s.V, rows(s, base) - i0, r);
    }
    // column `lane` of the identity
    __device__ __forceinline__ void unit(const Shape &s, float (&S)[KD / 4]) const {
        const int lane = threadIdx.x & 127;
#pragma unroll
        for (int i = 0; i < KD / 4; ++i) S[i] = wg * (KD / 4) + i == lane && lane < s.K ? 1.f : 0.f;
    }
    // A's terms from its columns, one a lane
    __device__ __forceinline__ void store_trans(char *base, const float (&S)[KD / 4]) const {
        const int lane = threadIdx.x & 127;
        if (lane < KD) {
#pragma unroll
            for (int i = 0; i < KD / 4; i += 2) {
                uint32_t t[NT];
                split2<NT>(S[i], S[i + 1], t);
                const int k = wg * (KD / 4) + i;
                char *p = base + (lane >> 6) * (KD * 128);
#pragma unroll
                for (int n = 0; n < NT; ++n, p += KD * KD * 2) {
                    *(uint16_t *)(p + swz(k, (lane & 63) * 2)) = (uint16_t)t[n];
                    *(uint16_t *)(p + swz(k + 1, (lane & 63) * 2)) = (uint16_t)(t[n] >> 16);
                }
            }
        }
        __syncwarp();
    }
    // the rows of chunk c's padding are zero
    template <class T> __device__ __forceinline__ void clear_padding(const Shape &s, T *p, int c) const {
        const int t0 = c * C + wg * 16;
        p += head * s.V + v + t0 * row;
#pragma unroll 1
        for (int i = max(0, len - t0); i < tokens(t0, s.T) && i < 16; ++i) p[i * row] = from_f<T>(0.f);
        __syncwarp();
    }
    // how many of the 16 tokens from t0 on are below `end`, for a lane that has a column
    __device__ __forceinline__ int tokens(int t0, int end) const { return own ? end - t0 : 0; }
};

template <class E, int KD, bool SCAN>
__global__ void __launch_bounds__(SEQ_THREADS, 1) seq_fwd_kernel(const __grid_constant__ SeqArgs a) {
    using Q = Seq<E, KD>;
    constexpr int TB = Q::TB, H4 = KD / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    SeqBars *bar = (SeqBars *)(smem + Q::stages * (Q::stage + GATES));
    const Shape &s = a.s;
    const int tid = threadIdx.x, warp = warp_id();
    const Job<SCAN> J(a);
    if (J.identity && J.seg == 0) return;  // the first segment starts from s0: its A is not needed
    const int chunks = max(0, min(J.chunks, J.live - J.first));
    seq_setup(bar);
    const uint32_t tmem = bar->tmem_slot;
    const Lane<KD> L(s, tmem, J.b, J.h, J.vt, J.identity);
    volatile int *ab = &bar->abort_flag;
    constexpr Steps rows = {QK<E, KD>::term >> 4, 2, 2 * TILE >> 4};   // K-major q or k: K over the dims
    constexpr Steps cols = {QK<E, KD>::term >> 4, 2048 >> 4, 0};       // MN-major k: K over the tokens
    constexpr Steps mat = {TILE >> 4, 2, 0};                           // K-major T2, P
    if (s.NC == 0) clear_ctrl(a.ctrl);  // (else prep did)
    if (tid == 32 && chunks > 0) {
        seq_load<E, KD>(a, smem, bar, J.b, J.h, 0, J.first, false);
        if (Q::stages == 2 && chunks > 1) seq_load<E, KD>(a, smem, bar, J.b, J.h, 1, J.first, false);
    }
    __syncwarp();
    const long long KV = (long long)s.K * s.V, all = (long long)s.B * s.Hv * KV;  // a state; the states of all heads
    float S[H4], o[16];
    Col16<E> vr;
    if (J.identity) L.unit(s, S);
    else L.load(s, J.seg == 0 || (!SCAN && J.live == 0) ? (a.s0 ? a.s0 + L.head * KV : nullptr)  // (no token: of every segment)
                              : (SCAN ? nullptr : a.starts + (J.seg - 1) * all + L.head * KV), S);
    const E *vp = (const E *)a.v + (long long)J.b * s.ldv + (long long)J.h * s.V + L.v;
    auto load_v = [&](int c) {
        const int t0 = c * C + L.wg * 16;
        vr.load(vp + (long long)t0 * s.B * s.ldv, s.B * s.ldv, L.tokens(t0, L.len));
    };
    auto store_o = [&](int c) {
        const int t0 = c * C + L.wg * 16;
        store_col((E *)a.o + L.head * s.V + L.v + t0 * L.row, L.row, L.tokens(t0, L.len), o);
    };
    auto add_pu = [&](uint32_t ph, uint32_t site) {
        wait(&bar->m3, ph, a.ctrl, ab, site);
        float f[16];
        get16(L.lanes + COL_X + L.wg * 16, f);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] += f[i];
    };
    load_v(J.first);
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
        const int c = J.first + n, st = n % Q::stages, t0 = c * C + L.wg * 16;
        const uint32_t ph = n & 1;
        const uint32_t qk = tc::smem_u32(smem + st * Q::stage), tp = qk + QK<E, KD>::bytes;
        const float *gates = (const float *)(smem + Q::stages * Q::stage + st * GATES) + L.wg * 16;
        put_terms<H4 / 2, NT>(L.lanes + COL_S + L.wg * (H4 / 2), KD / 2, S);
        wait(&bar->full[st], (n / Q::stages) & 1, a.ctrl, ab, 0x612);
        if (hand_over(warp)) {  // D = K S and Q S, tokens on the columns
            products_ts<KD / 16, NT, TB, NT>(tmem + COL_D, tmem + COL_S, KD / 2, k_major(qk + TILE, 0), rows,
                                             tc::idesc_bf16_f32(128, 64, 0, 0));
            tc::mma_commit(&bar->m1);
            if (!SCAN)
                products_ts<KD / 16, NT, TB, NT>(tmem + COL_D + 64, tmem + COL_S, KD / 2, k_major(qk, 0), rows,
                                                 tc::idesc_bf16_f32(128, 64, 0, 0));
        }
        __syncwarp();
        if (!SCAN && n > 0) add_pu(ph ^ 1, 0x616);
        // (the products of chunk n - 1, whose stage this is, are complete)
        if (Q::stages == 2 && tid == 32 && n > 0 && n + 1 < chunks)
            seq_load<E, KD>(a, smem, bar, J.b, J.h, n + 1, J.first, false);
        __syncwarp();
        // (the state's rows go out a part in each product's shadow)
        float *kept = !SCAN && a.states ? a.states + c * all + L.head * KV : nullptr;
        if (!SCAN && n > 0) store_o(c - 1);
        if (kept) L.template store_part<0, 1>(s, kept, S);
        const float last = gates[C - 1 - L.wg * 16];  // gamma of token 63
        float f[16], be[16], u[16];
        load16(gates, u);  // gamma
        wait(&bar->m1, ph, a.ctrl, ab, 0x613);
        get16(L.lanes + COL_D + L.wg * 16, f);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = fmaf(-u[i], f[i], vr[i]);
        put_terms<8, NT>(L.lanes + COL_R + L.wg * 8, 32, f);
        if (hand_over(warp)) {  // X = T2 R
            products_ts<4, NT, NT, NT>(tmem + COL_X, tmem + COL_R, 32, k_major(tp, 0), mat,
                                       tc::idesc_bf16_f32(128, 64, 0, 0));
            tc::mma_commit(&bar->m2);
        }
        __syncwarp();
        if (n + 1 < chunks) load_v(c + 1);
        if (kept) L.template store_part<1, 3>(s, kept, S);
        load16(gates + C, u);
        load16(gates + 2 * C, be);
        wait(&bar->m2, ph, a.ctrl, ab, 0x614);  // Q S came before X
        get16(L.lanes + COL_X + L.wg * 16, f);
        if (!SCAN) get16(L.lanes + COL_D + 64 + L.wg * 16, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] *= f[i] * be[i];  // left U
        put_terms<8, NT>(L.lanes + COL_W + L.wg * 8, 32, u);
        if (hand_over(warp)) {  // D = K^T (left U)
            products_ts<4, NT, TB, NT>(tmem + COL_D, tmem + COL_W, 32, mn_major(qk + TILE, 0, 2 * TILE), cols,
                                       tc::idesc_bf16_f32(128, KD, 0, 1));
            tc::mma_commit(&bar->m4);
        }
        __syncwarp();
        if (!SCAN) {
            if (a.deltas) store_col(a.deltas + L.head * s.V + L.v + t0 * L.row, L.row, L.tokens(t0, L.len), f);
            load16(gates, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i] *= s.scale * u[i];
                f[i] *= be[i];  // U
            }
            put_terms<8, NT>(L.lanes + COL_R + L.wg * 8, 32, f);
            if (hand_over(warp)) {  // P U
                products_ts<4, NT, NT, NT>(tmem + COL_X, tmem + COL_R, 32, k_major(tp + NT * TILE, 0), mat,
                                           tc::idesc_bf16_f32(128, 64, 0, 0));
                tc::mma_commit(&bar->m3);
            }
            __syncwarp();
            if (kept) L.template store_part<3, 4>(s, kept, S);
        }
        wait(&bar->m4, ph, a.ctrl, ab, 0x615);
#pragma unroll
        for (int i0 = 0; i0 < H4; i0 += 16) {
            get16(L.lanes + COL_D + L.wg * H4 + i0, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i0 + i] = fmaf(last, S[i0 + i], f[i]);
        }
        if (Q::stages == 1) {
            if (!SCAN) wait(&bar->m3, ph, a.ctrl, ab, 0x617);
            if (tid == 32 && n + 1 < chunks) seq_load<E, KD>(a, smem, bar, J.b, J.h, n + 1, J.first, false);
            __syncwarp();
        }
    }
    if (!SCAN && chunks > 0) {
        add_pu((chunks - 1) & 1, 0x618);
        store_o(J.first + chunks - 1);
    }
    if (!SCAN) {
#pragma unroll 1
        for (int c = J.first + max(0, chunks - 1); c < J.first + J.chunks; ++c) {
            L.clear_padding(s, (E *)a.o, c);
            if (a.deltas) L.clear_padding(s, a.deltas, c);
            if (a.states && c >= J.live) L.store(s, a.states + c * all + L.head * KV, S);
        }
    }
    if (J.identity) L.store_trans(a.trans + ((J.seg * s.B + J.b) * (long long)s.Hv + J.h) * (NT * KD * KD * 2), S);
    else if (SCAN) L.store(s, a.starts + J.seg * all + L.head * KV, S);
    else if (J.seg == a.segments - 1) L.store(s, a.sT + L.head * KV, S);
    if (tid == 32) seq_drain<E, KD>(bar, chunks);
    seq_finish(bar);
}

// The adjoint, chunks in reverse, the same layout (dS^T in registers):
//   K dS and P^T dO  ->  dU  ->  dV = T2^T (beta dU)  ->  dS += scale Q^T gamma dO - K^T gamma dV.
// P^T dO of the next chunk runs beside the last product of this one.
template <class E, int KD, bool SCAN>
__global__ void __launch_bounds__(SEQ_THREADS, 1) seq_bwd_kernel(const __grid_constant__ SeqArgs a) {
    using Q = Seq<E, KD>;
    constexpr int TB = Q::TB, H4 = KD / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    SeqBars *bar = (SeqBars *)(smem + Q::stages * (Q::stage + GATES));
    const Shape &s = a.s;
    const int tid = threadIdx.x, warp = warp_id();
    const Job<SCAN> J(a);
    if (J.identity && J.seg == 0) return;
    // chunk n of the segment is NC - 1 - first - n: the first `skip` are padding
    const int skip = max(0, min(J.chunks, s.NC - J.first - J.live)), first = J.first + skip, chunks = J.chunks - skip;
    seq_setup(bar);
    const uint32_t tmem = bar->tmem_slot;
    const Lane<KD> L(s, tmem, J.b, J.h, J.vt, J.identity);
    volatile int *ab = &bar->abort_flag;
    constexpr Steps rows = {QK<E, KD>::term >> 4, 2, 2 * TILE >> 4};
    constexpr Steps cols = {QK<E, KD>::term >> 4, 2048 >> 4, 0};
    constexpr Steps mat = {TILE >> 4, 2048 >> 4, 0};                   // MN-major T2, P: transposed
    if (s.NC == 0) clear_ctrl(a.ctrl);
    if (tid == 32 && chunks > 0) seq_load<E, KD>(a, smem, bar, J.b, J.h, 0, first, true);
    __syncwarp();
    const long long KV = (long long)s.K * s.V, all = (long long)s.B * s.Hv * KV;
    float S[H4];
    Col16<E> d;
    if (J.identity) L.unit(s, S);
    else L.load(s, J.seg == 0 || (!SCAN && J.live == 0) ? (a.s0 ? a.s0 + L.head * KV : nullptr)  // (no token: of every segment)
                              : (SCAN ? nullptr : a.starts + (J.seg - 1) * all + L.head * KV), S);
    const E *dop = (const E *)a.v + L.head * s.V + L.v;
    auto load_do = [&](int c) {
        const int t0 = c * C + L.wg * 16;
        d.load(dop + t0 * L.row, L.row, a.v ? L.tokens(t0, L.len) : 0);
    };
    auto product_pdo = [&](int st) {  // X = P^T dO (one thread)
        const uint32_t tp = tc::smem_u32(smem + st * Q::stage) + QK<E, KD>::bytes;
        products_ts<4, TB, NT, NT>(tmem + COL_X, tmem + COL_R, 32, mn_major(tp + NT * TILE, 0, TILE), mat,
                                   tc::idesc_bf16_f32(128, 64, 0, 1));
    };
    auto put_do = [&]() {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = d[i];
        put_terms<8, TB>(L.lanes + COL_R + L.wg * 8, 32, x);
    };
    if (chunks > 0) load_do(s.NC - 1 - first);
    if (!SCAN) {
#pragma unroll 1
        for (int n = -skip; n < min(1, chunks); ++n) L.clear_padding(s, (E *)a.o, s.NC - 1 - first - n);
    }
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
        const int c = s.NC - 1 - first - n, st = n % Q::stages, t0 = c * C + L.wg * 16;
        const bool more = n + 1 < chunks;
        const uint32_t ph = n & 1;
        const uint32_t qk = tc::smem_u32(smem + st * Q::stage), tp = qk + QK<E, KD>::bytes;
        const float *gates = (const float *)(smem + Q::stages * Q::stage + st * GATES) + L.wg * 16;
        const bool early = Q::stages == 2 && n > 0;  // P^T dO was issued a chunk ago
        if (Q::stages == 2 && tid == 32 && more) seq_load<E, KD>(a, smem, bar, J.b, J.h, n + 1, first, true);
        __syncwarp();
        put_terms<H4 / 2, NT>(L.lanes + COL_S + L.wg * (H4 / 2), KD / 2, S);
        if (!early) put_do();
        wait(&bar->full[st], (n / Q::stages) & 1, a.ctrl, ab, 0x622);
        if (hand_over(warp)) {  // D = K dS
            if (!early) product_pdo(st);
            products_ts<KD / 16, NT, TB, NT>(tmem + COL_D, tmem + COL_S, KD / 2, k_major(qk + TILE, 0), rows,
                                             tc::idesc_bf16_f32(128, 64, 0, 0));
            tc::mma_commit(&bar->m1);
        }
        __syncwarp();
        float *kept = a.states + c * all + L.head * KV;
        if (!SCAN) L.template store_part<0, 1>(s, kept, S);
        const float last = gates[C - 1 - L.wg * 16];
        float f[16], e[16], left[16], be[16];
        load16(gates + C, left);
        load16(gates + 2 * C, be);
        wait(&bar->m1, ph, a.ctrl, ab, 0x623);
        get16(L.lanes + COL_D + L.wg * 16, f);
        get16(L.lanes + COL_X + L.wg * 16, e);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = be[i] * fmaf(left[i], f[i], e[i]);  // beta dU
        put_terms<8, NT>(L.lanes + COL_R + L.wg * 8, 32, f);
        if (hand_over(warp)) {  // dV = T2^T (beta dU)
            products_ts<4, NT, NT, NT>(tmem + COL_X, tmem + COL_R, 32, mn_major(tp, 0, TILE), mat,
                                       tc::idesc_bf16_f32(128, 64, 0, 1));
            tc::mma_commit(&bar->m2);
        }
        __syncwarp();
        load16(gates, be);  // gamma
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = s.scale * be[i] * d[i];
        put_terms<8, NT>(L.lanes + COL_S + L.wg * 8, 32, e);
        if (more) load_do(c - 1);
        if (!SCAN) L.template store_part<1, 3>(s, kept, S);
        wait(&bar->m2, ph, a.ctrl, ab, 0x624);
        get16(L.lanes + COL_X + L.wg * 16, f);
#pragma unroll
        for (int i = 0; i < 16; ++i) e[i] = -be[i] * f[i];
        put_terms<8, NT>(L.lanes + COL_W + L.wg * 8, 32, e);
        if (Q::stages == 2 && more) put_do();
        if (hand_over(warp)) {  // D = scale Q^T gamma dO - K^T gamma dV
            two_products_ts<4, NT, TB, NT>(tmem + COL_D, tmem + COL_S, mn_major(qk, 0, 2 * TILE), tmem + COL_W,
                                           mn_major(qk + TILE, 0, 2 * TILE), 32, cols, tc::idesc_bf16_f32(128, KD, 0, 1));
            tc::mma_commit(&bar->m4);
            if (Q::stages == 2 && more) {
                tc::mbar_wait(&bar->full[st ^ 1], ((n + 1) / Q::stages) & 1, a.ctrl, ab, 0x626);
                product_pdo(st ^ 1);
            }
        }
        __syncwarp();
        if (!SCAN) {
            store_col(a.deltas + L.head * s.V + L.v + t0 * L.row, L.row, L.tokens(t0, L.len), f);
            store_col((E *)a.o + L.head * s.V + L.v + t0 * L.row, L.row, L.tokens(t0, L.len), f);
            L.template store_part<3, 4>(s, kept, S);
        }
        wait(&bar->m4, ph, a.ctrl, ab, 0x625);
#pragma unroll
        for (int i0 = 0; i0 < H4; i0 += 16) {
            get16(L.lanes + COL_D + L.wg * H4 + i0, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i0 + i] = fmaf(last, S[i0 + i], f[i]);
        }
        if (Q::stages == 1 && tid == 32 && more) seq_load<E, KD>(a, smem, bar, J.b, J.h, n + 1, first, true);
        __syncwarp();
    }
    if (J.identity) L.store_trans(a.trans + ((J.seg * s.B + J.b) * (long long)s.Hv + J.h) * (NT * KD * KD * 2), S);
    else if (SCAN) L.store(s, a.starts + J.seg * all + L.head * KV, S);
    else if (J.seg == a.segments - 1) L.store(s, a.sT ? a.sT + L.head * KV : nullptr, S);
    if (tid == 32) seq_drain<E, KD>(bar, chunks);
    seq_finish(bar);
}

// Join the segments (4 us each, one after another: the products of a chain are
// bound by latency): starts[i] becomes A_i starts[i - 1] + B_i, i = 1 .. in
// order, block (b, h, 128 columns of V); S^T in registers and tensor memory as
// above, A's tiles by bulk copies one segment ahead.
template <int KD> struct ScanSmem {
    static constexpr int tile = NT * KD * KD * 2;
    static constexpr size_t smem = 2 * tile + 1024 + 256;
};
template <int KD>
__global__ void __launch_bounds__(SEQ_THREADS, 1) scan_kernel(const __grid_constant__ SeqArgs a) {
    constexpr int H4 = KD / 4, TILES = ScanSmem<KD>::tile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    SeqBars *bar = (SeqBars *)(smem + 2 * TILES);
    const Shape &s = a.s;
    const int tid = threadIdx.x, warp = warp_id();
    int id = blockIdx.x;
    const int vt = id % s.VT;
    id /= s.VT;
    const int h = id % s.Hv, b = id / s.Hv;
    seq_setup(bar);
    const uint32_t tmem = bar->tmem_slot;
    const Lane<KD> L(s, tmem, b, h, vt, false);
    volatile int *ab = &bar->abort_flag;
    constexpr Steps rows = {KD * KD * 2 >> 4, 2, KD * 128 >> 4};
    const long long KV = (long long)s.K * s.V, all = (long long)s.B * s.Hv * KV;
    const int last = a.segments - 2;  // the last start is starts[last]
    auto fetch = [&](int i) {
        tc::mbar_arrive_expect_tx(&bar->full[i & 1], TILES);
        bulk_load(smem + (i & 1) * TILES, a.trans + ((i * s.B + b) * (long long)s.Hv + h) * TILES, TILES, &bar->full[i & 1]);
    };
    if (tid == 32 && last >= 1) fetch(1);
    __syncwarp();
    float S[H4], B[H4];
    L.load(s, a.starts + L.head * KV, S);
#pragma unroll 1
    for (int i = 1; i <= last; ++i) {
        if (tid == 32 && i < last) fetch(i + 1);  // (segment i - 1's product is complete)
        __syncwarp();
        float *start = a.starts + i * all + L.head * KV;
        L.load(s, start, B);
        put_terms<H4 / 2, NT>(L.lanes + COL_S + L.wg * (H4 / 2), KD / 2, S);
        wait(&bar->full[i & 1], ((i - 1) >> 1) & 1, a.ctrl, ab, 0x641);
        if (hand_over(warp)) {
            products_ts<KD / 16, NT, NT, NT>(tmem + COL_D, tmem + COL_S, KD / 2,
                                             k_major(tc::smem_u32(smem + (i & 1) * TILES), 0), rows,
                                             tc::idesc_bf16_f32(128, KD, 0, 0));
            tc::mma_commit(&bar->m1);
        }
        __syncwarp();
        wait(&bar->m1, (i - 1) & 1, a.ctrl, ab, 0x642);
#pragma unroll
        for (int i0 = 0; i0 < H4; i0 += 16) {
            float f[16];
            get16(L.lanes + COL_D + L.wg * H4 + i0, f);
#pragma unroll
            for (int j = 0; j < 16; ++j) S[i0 + j] = f[j] + B[i0 + j];
        }
        L.store(s, start, S);
    }
    if (tid == 32)
        for (int i = max(1, last - 1); i <= last; ++i)  // after a time-out: the copies have landed
            tc::mbar_wait(&bar->full[i & 1], ((i - 1) >> 1) & 1, nullptr, nullptr, 0, 200000000ull);
    seq_finish(bar);
}

// ---------------------------------------------------------------- gradients
// Block (c, b, hk), 512 threads: dq, dk of the chunk, and dg, dbeta of every
// value head of the group, from the saved S0 and X and seq_bwd's dS1 and dV.
// (PARTS, where that leaves SMs idle: a block per value head, whose parts of dq
// and dk sum_kernel adds in order.)
// Rows are stacked so that every product has the 128 rows the tensor core
// takes: [dO; dV] with X gives Y over Z, with S0 gives F over G; X sits in the
// lower rows for E; [dQ; dK] += [Yh; -Zh] K, and dK += [Yh; -Zh]^T [Q; K] from
// the same tiles read the other way.  V is contracted 64 columns a pass.
// dg's double sum needs no matrix: sum_{r >= i > j} M_rj is the sum over
// r >= i of (row sum - column sum), for the lower triangle M.
//
// Bound by the conversions between the products (every operand is a float that
// becomes three terms) and by the one block an SM that the tiles leave room for:
// bf16, K = V = 128, 2048 blocks of two value heads 461 us, 0.94 GB at 2.0 TB/s,
// the tensor cores busy 36 % of the time.
constexpr int GRAD_THREADS = 512;
// [q; k] k^T | F over G, then Y over Z | E, then the transposed triangle's product | [dQ; dK]
constexpr uint32_t COL_QK = 0, COL_FG = 64, COL_E = 256, COL_OUT = 384;

// Tiles, 64 columns of V (NT terms each): `a` [dO; dV] 16 KB, `st` [S0 (KD
// rows); X (64 rows)], and dS1 in a buffer of its own where there is room,
// else in S0's rows after their products.  The triangle's operand [Yh; -Zh]
// lies over `a`.  (The 16 KB before `a`, q and k tiles, and the 64 rows before
// X, serve as rows of operands whose results are not used.)
template <class E, int KD> struct GradSmem {
    static constexpr int a = QK<E, KD>::bytes;
    static constexpr int st = a + NT * 2 * TILE, st_term = KD * 128 + TILE;
    static constexpr int ds = st + NT * st_term;
    static constexpr int fixed = 1024 + 8192;        // alignment; the static arrays
    static constexpr bool own_ds = ds + NT * KD * 128 + fixed <= 232448;
    static constexpr int ds_at = own_ds ? ds : st, ds_term = own_ds ? KD * 128 : st_term;
    static constexpr size_t smem = (own_ds ? ds + NT * KD * 128 : ds) + 1024;
};

struct GradArgs {
    Shape s;
    const char *qk;
    const float *g, *beta;
    const void *dout;
    const float *states, *deltas, *dstates, *dvf;
    void *dq, *dk;
    float *dg, *dbeta;
    float *parts;  // PARTS: [group][dq, dk][T][B][Hk][K]
    Ctrl *ctrl;
};

// Sums over the warp's 32 lanes of f[0..15]: lane 2 j (and 2 j + 1) returns the j-th.
__device__ __forceinline__ float transpose_sum(float (&f)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & (2 * o);
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? f[j + o] : f[j], give = up ? f[j] : f[j + o];
            f[j] = keep + __shfl_xor_sync(~0u, give, 2 * o);
        }
    }
    return f[0] + __shfl_xor_sync(~0u, f[0], 1);
}

template <class E, int KD, bool PARTS>
__global__ void __launch_bounds__(GRAD_THREADS, 1) grad_kernel(const __grid_constant__ GradArgs a) {
    using L = GradSmem<E, KD>;
    constexpr int TB = Terms<E>::n, TERM = QK<E, KD>::term, H4 = KD / 4, SI = KD / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ Sums sums;
    __shared__ float colp[4][C], rowp[4][2 * C], rp[4][2 * C], ep[4][C], dots[16], half_e;
    __shared__ double half_d;
    __shared__ uint64_t loaded, m1, m2, m3;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_s;
    const Shape &s = a.s;
    const int tid = threadIdx.x, warp = warp_id(), lane = tid & 31, wg = tid >> 7, r128 = tid & 127, r = r128 & 63;
    const bool isq = r128 < 64;
    const int heads = PARTS ? 1 : s.group, part = PARTS ? blockIdx.x % s.group : 0;
    int id = PARTS ? blockIdx.x / s.group : blockIdx.x;
    const char *tiles = a.qk + (size_t)id * QK<E, KD>::bytes;
    const int hk = id % s.Hk, h0 = hk * s.group + part;
    id /= s.Hk;
    const int b = id % s.B, c = id / s.B;
    const int len = length_of(s, b);
    volatile int *ab = &abort_s;
    if (c * C >= len) {  // (what seq_bwd keeps of a chunk ends with the tokens)
        const int n = min(C, s.T - c * C);
        const long long all = (long long)s.T * s.B * s.Hk * s.K;
        for (int i = tid; i < 2 * n * s.K; i += GRAD_THREADS) {
            const int of = i / (n * s.K), j = i % (n * s.K);
            const long long at = (((long long)(c * C + j / s.K) * s.B + b) * s.Hk + hk) * s.K + j % s.K;
            if constexpr (PARTS) a.parts[(2 * part + of) * all + at] = 0.f;
            else ((E *)(of ? a.dk : a.dq))[at] = from_f<E>(0.f);
        }
        for (long long i = tid; i < (long long)n * heads; i += GRAD_THREADS) {
            const long long at = ((c * C + i / heads) * s.B + b) * s.Hv + h0 + i % heads;
            a.dg[at] = a.dbeta[at] = 0.f;
        }
        return;
    }
    if (tid == 0) {
        tc::mbar_init(&loaded, 1);
        tc::mbar_init(&m1, 1);
        tc::mbar_init(&m2, 1);
        tc::mbar_init(&m3, 1);
        abort_s = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot, lanes = tmem + ((uint32_t)(r128 & 96) << 16);
    const uint32_t qk = tc::smem_u32(smem), sa = qk + L::a, ss = qk + L::st, sx = ss + KD * 128, sd = qk + L::ds_at;
    if (tid == 0) {
        tc::mbar_arrive_expect_tx(&loaded, QK<E, KD>::bytes);
        bulk_load(smem, tiles, QK<E, KD>::bytes, &loaded);
    }
    __syncwarp();
    const int row = tid >> 3, gr = tid & 7;  // loads: eight threads a row, eight columns each
    const int t_row = c * C + row;
    const uint32_t off = swz(row, gr * 16);  // rows 64 apart keep it
    const int passes = (s.V + 63) / 64;
    Raw8<E> ro;                                // dO, dV, X, S0, dS1 of the pass ahead
    Raw8<float> rv, rx, rs[SI], rd[SI];
    // where this thread's groups of the block's first value head, column 0, lie;
    // next_h, next_v: head and first column of the pass after the present one
    const long long tok0 = (((long long)t_row * s.B + b) * s.Hv + h0) * s.V + gr * 8;
    const long long st0 = ((((long long)c * s.B + b) * s.Hv + h0) * s.K + row) * s.V + gr * 8;
    int next_h = 0, next_v = 0;
    auto load_a = [&]() {
        const bool live = next_h < heads && next_v + gr * 8 < s.V && t_row < len;
        const long long at = tok0 + next_h * s.V + next_v;
        ro = raw8<E>((const E *)a.dout + at, live && a.dout);
        rv = raw8<float>(a.dvf + at, live);
    };
    auto load_x = [&]() {
        rx = raw8<float>(a.deltas + tok0 + next_h * s.V + next_v, next_h < heads && next_v + gr * 8 < s.V && t_row < len);
    };
    auto load_s = [&](const float *base, Raw8<float> (&o)[SI]) {
        const bool live = next_h < heads && next_v + gr * 8 < s.V;
        const float *q = base + st0 + (long long)next_h * s.K * s.V + next_v;
#pragma unroll
        for (int i = 0; i < SI; ++i) o[i] = raw8<float>(q + i * 64 * s.V, live && i * 64 + row < s.K);
    };
    auto put = [&](uint8_t *tile, int term, const Raw8<float> &x) {
        uint4 o[NT];
        terms8<float>(x, o);
#pragma unroll
        for (int k = 0; k < NT; ++k) *(uint4 *)(tile + k * term + off) = o[k];
    };
    constexpr Steps qk_rows = {TERM >> 4, 2, 2 * TILE >> 4}, a_rows = {2 * TILE >> 4, 2, 0}, x_rows = {L::st_term >> 4, 2, 0},
                    d_rows = {L::ds_term >> 4, 2, 0}, a_cols = {2 * TILE >> 4, 2048 >> 4, 4 * 2048 >> 4},
                    qk_cols = {TERM >> 4, 2048 >> 4, 4 * 2048 >> 4};
    load_s(a.states, rs);
    load_a();
    load_x();
    load_s(a.dstates, rd);
    wait(&loaded, 0, a.ctrl, ab, 0x631);
#pragma unroll 1
    for (int m = 0; m < heads; ++m) {
        const int h = h0 + m;
        float dot = 0.f;  // <dS1, S0>
        // A pass: the first products run beside the conversion of dS1, E beside
        // the next pass's conversions of S0, dO and dV; every buffer's next
        // values are loaded as soon as it is written.
#pragma unroll 1
        for (int p = 0; p < passes; ++p) {
            const int n = m * passes + p;
            next_h = p + 1 < passes ? m : m + 1;
            next_v = p + 1 < passes ? p * 64 + 64 : 0;
            if (n > 0) wait(&m1, (n - 1) & 1, a.ctrl, ab, 0x633);
            if (!L::own_ds && p > 0) wait(&m2, (n - 1) & 1, a.ctrl, ab, 0x634);  // dS1 lies in S0's rows
#pragma unroll
            for (int i = 0; i < SI; ++i) {
                put(smem + L::st + i * TILE, L::st_term, rs[i]);
                const uint4 *x = &rs[i].a, *y = &rd[i].a;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    dot = fmaf(__uint_as_float(x[j].x), __uint_as_float(y[j].x), dot);
                    dot = fmaf(__uint_as_float(x[j].y), __uint_as_float(y[j].y), dot);
                    dot = fmaf(__uint_as_float(x[j].z), __uint_as_float(y[j].z), dot);
                    dot = fmaf(__uint_as_float(x[j].w), __uint_as_float(y[j].w), dot);
                }
            }
            load_s(a.states, rs);
            if (m > 0 && p == 0) {
                wait(&m3, (m - 1) & 1, a.ctrl, ab, 0x632);  // the triangle's tiles are free
                if (!isq)  // dK's transposed part of the last head
#pragma unroll
                    for (int i0 = 0; i0 < H4; i0 += 16) {
                        float f[16], e[16];
                        get16(lanes + COL_OUT + wg * H4 + i0, f);
                        get16(lanes + COL_E + wg * H4 + i0, e);
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] += e[i];
                        set16(lanes + COL_OUT + wg * H4 + i0, f);
                    }
            }
            {
                uint4 o[TB];
                terms8<E>(ro, o);
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    *(uint4 *)(smem + L::a + k * 2 * TILE + off) = k < TB ? o[k < TB ? k : 0] : make_uint4(0, 0, 0, 0);
            }
            put(smem + L::a + TILE, 2 * TILE, rv);
            load_a();
            if (L::own_ds && p > 0) wait(&m2, (n - 1) & 1, a.ctrl, ab, 0x634);
            put(smem + L::st + KD * 128, L::st_term, rx);
            load_x();
            tc::fence_proxy_async_smem();
            if (hand_over(warp)) {
                if (n == 0)  // [q; k] k^T, once
                    products_ss<KD / 16, TB, TB, NT>(tmem + COL_QK, k_major(qk, 0), qk_rows, k_major(qk + TILE, 0), qk_rows,
                                                     tc::idesc_bf16_f32(128, 64, 0, 0));
                // [F; G | Y; Z] = [dO; dV] [S0; X]^T
                products_ss<4, NT, NT, NT>(tmem + COL_FG, k_major(sa, 0), a_rows, k_major(ss, 0), x_rows,
                                           tc::idesc_bf16_f32(128, KD + 64, 0, 0), p > 0);
                tc::mma_commit(&m1);
            }
            __syncwarp();
            if (p == 0 && warp == 2) load_gates(s, a.g, a.beta, c, b, h, len, sums);
            if (!L::own_ds) wait(&m1, n & 1, a.ctrl, ab, 0x636);
#pragma unroll
            for (int i = 0; i < SI; ++i) put(smem + L::ds_at + i * TILE, L::ds_term, rd[i]);
            load_s(a.dstates, rd);
            tc::fence_proxy_async_smem();
            if (hand_over(warp)) {  // rows 64..127: E = X dS1^T (the rows above X are not used)
                products_ss<4, NT, NT, NT>(tmem + COL_E, k_major(sx - TILE, 0), x_rows, k_major(sd, 0), d_rows,
                                           tc::idesc_bf16_f32(128, KD, 0, 0), p > 0);
                tc::mma_commit(&m2);
            }
            __syncwarp();
        }
        wait(&m2, (m * passes + passes - 1) & 1, a.ctrl, ab, 0x637);
        // ---- the triangle: weights w, their row and column sums, and [Yh; -Zh]
        {
            float y[16], kq[16];
            get16(lanes + COL_QK + wg * 16, kq);
            get16(lanes + COL_FG + KD + wg * 16, y);
            const float2 br = sums.b[r];
            const float sign = isq ? s.scale : -1.f;
            const int last = isq ? r : r - 1;  // last column of this row
            float rowsum = 0.f;
#pragma unroll
            for (int j0 = 0; j0 < 16; j0 += 8) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = wg * 16 + j0 + i;
                    const float z = j <= last ? decay(br, sums.b[j]) * sign * y[j0 + i] : 0.f;
                    kq[j0 + i] *= z;  // w_rj
                    e[i] = z * sums.beta[j];
                    rowsum = fmaf(sums.beta[j], kq[j0 + i], rowsum);
                }
                uint4 o[NT];
                split8<NT>(e, o);
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    *(uint4 *)(smem + L::a + k * 2 * TILE + swz(r128, (wg * 16 + j0) * 2)) = o[k];
            }
            rowp[wg][r128] = rowsum;
            __syncwarp();
            const float cs = transpose_sum(kq);
            if (!(lane & 1)) colp[warp & 3][wg * 16 + (lane >> 1)] = cs;
        }
        // ---- F | G and E: a quarter row of K a thread; their part of [dQ; dK]
        {
            const float gam = decay(sums.b[r]), lb = decay(sums.b[C - 1], sums.b[r]) * sums.beta[r];
            float dotf = 0.f, dote = 0.f;
#pragma unroll
            for (int i0 = 0; i0 < H4; i0 += 16) {
                float f[16], e[16], acc[16];
                get16(lanes + COL_FG + wg * H4 + i0, f);
                get16(lanes + COL_E + wg * H4 + i0, e);
                if (m > 0) {
                    get16(lanes + COL_OUT + wg * H4 + i0, acc);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
                }
#pragma unroll
                for (int g2 = 0; g2 < 2; ++g2) {
                    const int col = wg * H4 + i0 + g2 * 8;
                    float x[8] = {};
#pragma unroll
                    for (int t = 0; t < TB; ++t) {
                        float xt[8];
                        x8_to_f32<bf16>(*(const uint4 *)(smem + t * TERM + (col >> 6) * 2 * TILE + swz(r128, (col & 63) * 2)), xt);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] += xt[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int n = g2 * 8 + i;
                        dotf = fmaf(x[i], f[n], dotf);
                        if (isq) {
                            acc[n] = fmaf(s.scale * gam, f[n], acc[n]);
                        } else {
                            dote = fmaf(x[i], e[n], dote);
                            acc[n] += lb * e[n] - gam * f[n];
                        }
                    }
                }
                set16(lanes + COL_OUT + wg * H4 + i0, acc);
            }
            rp[wg][r128] = dotf;
            if (!isq) ep[wg][r] = dote;
            __syncwarp();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
            if (lane == 0) dots[warp] = dot;
        }
        tc::fence_proxy_async_smem();
        if (hand_over(warp)) {
            // [dQ; dK] += [Yh; -Zh] K; and in the lower rows of COL_E: [Yh; -Zh]^T [Q; K]
            products_ss<4, NT, TB, NT>(tmem + COL_OUT, k_major(sa, 0), a_rows, mn_major(qk + TILE, 0, 2 * TILE), qk_cols,
                                       tc::idesc_bf16_f32(128, KD, 0, 1), 1);
            products_ss<8, NT, TB, NT>(tmem + COL_E, mn_major(sa - 2 * TILE, 0, 2 * TILE), a_cols, mn_major(qk, 0, 2 * TILE),
                                       qk_cols, tc::idesc_bf16_f32(128, KD, 1, 1));
            tc::mma_commit(&m3);
        }
        __syncwarp();
        if (warp == 1 || warp == 5) {  // dg and dbeta, a token a lane
            const int j = (warp & 4) * 8 + lane, t = c * C + j;
            auto sum4 = [&](const float *x, int stride, int i) { return (x[i] + x[stride + i]) + (x[2 * stride + i] + x[3 * stride + i]); };
            const long long at = ((long long)min(t, s.T - 1) * s.B + b) * s.Hv + h;
            const float gt = a.g[at], be = sums.beta[j], gam = decay(sums.b[j]), left = decay(sums.b[C - 1], sums.b[j]);
            const float col = sum4(&colp[0][0], C, j), ke = left * sum4(&ep[0][0], C, j);
            const float rows = sum4(&rowp[0][0], 2 * C, j) + sum4(&rowp[0][0], 2 * C, C + j);
            const float inter = gam * (s.scale * sum4(&rp[0][0], 2 * C, j) - sum4(&rp[0][0], 2 * C, C + j));
            float all = lane < 16 ? dots[lane] : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
            all = __shfl_sync(~0u, all, 0) * decay(sums.b[C - 1]);
            // sums of d over the tokens from j on, of e over those before (double: most of d cancels)
            const double d = (double)rows - (double)(be * col) + (double)inter;
            const float e = be * ke;
            double sd = d;
            float se = e;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_down_sync(~0u, sd, o);
                const float y = __shfl_up_sync(~0u, se, o);
                if (lane + o < 32) sd += x;
                if (lane >= o) se += y;
            }
            if (warp == 5 && lane == 0) half_d = sd;
            if (warp == 1 && lane == 31) half_e = se;
            asm volatile("bar.sync 1, 64;" ::: "memory");
            if (t < s.T) {
                const double v = warp == 1 ? sd + half_d + (double)(se - e) : sd + (double)(half_e + (se - e));
                // (where e^g is zero so is its gradient, and not the rounding of the sums)
                a.dg[at] = t < len && !(gt < -104.f) ? (float)(v + (double)all) : 0.f;
                a.dbeta[at] = t < len ? col + ke : 0.f;
            }
        }
        __syncwarp();
    }
    wait(&m3, (heads - 1) & 1, a.ctrl, ab, 0x635);
    const int t = c * C + r;
    const long long at = (((long long)t * s.B + b) * s.Hk + hk) * s.K + wg * H4, all = (long long)s.T * s.B * s.Hk * s.K;
    E *out = (E *)(isq ? a.dq : a.dk) + at;
    float *out_part = PARTS ? a.parts + (2 * part + (isq ? 0 : 1)) * all + at : nullptr;
#pragma unroll
    for (int i0 = 0; i0 < H4; i0 += 16) {
        float f[16], e[16];
        get16(lanes + COL_OUT + wg * H4 + i0, f);
        get16(lanes + COL_E + wg * H4 + i0, e);
        if (t < s.T)
#pragma unroll
            for (int g2 = 0; g2 < 2; ++g2) {
                if (wg * H4 + i0 + g2 * 8 >= s.K) continue;
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = t < len ? f[g2 * 8 + i] + (isq ? 0.f : e[g2 * 8 + i]) : 0.f;
                if constexpr (PARTS) {
                    *(float4 *)(out_part + i0 + g2 * 8) = make_float4(x[0], x[1], x[2], x[3]);
                    *(float4 *)(out_part + i0 + g2 * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
                } else if constexpr (sizeof(E) == 4) {
                    *(float4 *)(out + i0 + g2 * 8) = make_float4(x[0], x[1], x[2], x[3]);
                    *(float4 *)(out + i0 + g2 * 8 + 4) = make_float4(x[4], x[5], x[6], x[7]);
                } else {
                    *(uint4 *)(out + i0 + g2 * 8) = f32x8_to<E>(x);
                }
            }
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// dq and dk from the parts of `split` blocks, eight elements a thread (5 us on
// the 2 MB of T = 333, 3 sequences, 2 key heads of 3).
template <class E> __global__ void __launch_bounds__(256) sum_kernel(const float *parts, int split, long long n8, E *dq, E *dk) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * n8) return;
    const float *src = parts + i * 8;  // dq's elements, then dk's
    float x[8] = {};
    for (int p = 0; p < split; ++p, src += 16 * n8) {
        float y[8];
        load8<float>(src, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += y[j];
    }
    E *out = i < n8 ? dq + i * 8 : dk + (i - n8) * 8;
    if constexpr (sizeof(E) == 4) {
        *(float4 *)out = make_float4(x[0], x[1], x[2], x[3]);
        *((float4 *)out + 1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *(uint4 *)out = f32x8_to<E>(x);
    }
}

// -------------------------------------------------------------------- step
// A few tokens, token by token: block (b, h, 64 columns of V), thread (part,
// columns) holds four columns of the state for eight rows of K in registers.
// Bound: the state's read and write.  16 heads, K = V = 128, one token: of 64
// sequences 26 us, 134 MB at 5.2 TB/s, of 256 85 us, 6.3 TB/s; a further token
// costs 6 us (1024 heads) or 1 us (4 heads).  (Blocks of 32 or 128 columns 26.3 and
// 30.5 us, of 8 parts 27.2, of 32 columns and 32 parts 28.8.)
constexpr int STEP_COLS = 64, STEP_LANES = STEP_COLS / 4, STEP_PARTS = 16, STEP_K = 128 / STEP_PARTS;
constexpr int STEP_THREADS = STEP_PARTS * STEP_LANES, STEP_WARPS = STEP_THREADS / 32;

struct StepArgs {
    Shape s;
    const void *q, *k, *v;
    const float *g, *beta, *s0;
    void *o;
    float *sT;
    Ctrl *ctrl;
    int tiles;  // blocks of 64 columns
};

template <class E>
__global__ void __launch_bounds__(STEP_THREADS, 1024 / STEP_THREADS) step_kernel(StepArgs a) {
    __shared__ float qs[128], ks[128];
    __shared__ float4 part[2][STEP_WARPS][STEP_LANES];  // a warp's parts together
    const Shape &s = a.s;
    if (a.ctrl) clear_ctrl(a.ctrl);
    const int tid = threadIdx.x, warp = tid >> 5, c4 = tid % STEP_LANES, v = blockIdx.x % a.tiles * STEP_COLS + c4 * 4;
    const int id = blockIdx.x / a.tiles, h = id % s.Hv, b = id / s.Hv, hk = h / s.group;
    const long long head = (long long)b * s.Hv + h;
    const int len = length_of(s, b), k0 = tid / STEP_LANES * STEP_K;
    const bool own = v < s.V;  // V is a multiple of 8: all four or none
    float4 S[STEP_K];
#pragma unroll
    for (int i = 0; i < STEP_K; ++i)
        S[i] = a.s0 && own && k0 + i < s.K ? __ldcs((const float4 *)(a.s0 + (head * s.K + k0 + i) * s.V + v))
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
    // the columns' sums over K of w[k] S[k], in every thread
    auto contract = [&](const float *w, int buf) {
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < STEP_K; ++i) {
            const float x = w[k0 + i];
            d.x = fmaf(x, S[i].x, d.x);
            d.y = fmaf(x, S[i].y, d.y);
            d.z = fmaf(x, S[i].z, d.z);
            d.w = fmaf(x, S[i].w, d.w);
        }
#pragma unroll
        for (int o = STEP_LANES; o < 32; o *= 2) {
            d.x += __shfl_xor_sync(~0u, d.x, o);
            d.y += __shfl_xor_sync(~0u, d.y, o);
            d.z += __shfl_xor_sync(~0u, d.z, o);
            d.w += __shfl_xor_sync(~0u, d.w, o);
        }
        if ((tid & 31) < STEP_LANES) part[buf][warp][c4] = d;
        __syncthreads();
        d = part[buf][0][c4];
#pragma unroll
        for (int i = 1; i < STEP_WARPS; ++i) {
            const float4 e = part[buf][i][c4];
            d.x += e.x;
            d.y += e.y;
            d.z += e.z;
            d.w += e.w;
        }
        return d;
    };
    for (int t = 0; t < s.T; ++t) {
        const long long r = (long long)t * s.B + b;
        E *o = (E *)a.o + (r * s.Hv + h) * s.V + v;
        const bool writes = tid < STEP_LANES && own;
        if (t >= len) {  // padding: the same for the whole block
            if (writes)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = from_f<E>(0.f);
            continue;
        }
        float x[4] = {};
        if (own)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = to_f(((const E *)a.v)[r * s.ldv + (long long)h * s.V + v + i]);
        const float gt = a.g[r * s.Hv + h], be = a.beta[r * s.Hv + h];
        for (int i = tid; i < 256; i += STEP_THREADS) {
            const bool isq = i < 128;
            const int j = i & 127;
            const E *w = isq ? (const E *)a.q + r * s.ldq : (const E *)a.k + r * s.ldk;
            (isq ? qs : ks)[j] = j < s.K ? to_f(w[(long long)hk * s.K + j]) : 0.f;
        }
        const float dec = expf(gt);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < STEP_K; ++i) {
            S[i].x *= dec;
            S[i].y *= dec;
            S[i].z *= dec;
            S[i].w *= dec;
        }
        float4 u = contract(ks, 0);
        u = make_float4(be * (x[0] - u.x), be * (x[1] - u.y), be * (x[2] - u.z), be * (x[3] - u.w));
#pragma unroll
        for (int i = 0; i < STEP_K; ++i) {
            const float k = ks[k0 + i];
            S[i].x = fmaf(k, u.x, S[i].x);
            S[i].y = fmaf(k, u.y, S[i].y);
            S[i].z = fmaf(k, u.z, S[i].z);
            S[i].w = fmaf(k, u.w, S[i].w);
        }
        const float4 y = contract(qs, 1);
        if (writes) {
            o[0] = from_f<E>(s.scale * y.x);
            o[1] = from_f<E>(s.scale * y.y);
            o[2] = from_f<E>(s.scale * y.z);
            o[3] = from_f<E>(s.scale * y.w);
        }
    }
#pragma unroll
    for (int i = 0; i < STEP_K; ++i)
        if (own && k0 + i < s.K) __stcs((float4 *)(a.sT + (head * s.K + k0 + i) * s.V + v), S[i]);
}

}  // namespace gdr
}  // namespace lstm
