// block_norm.cu -- what stands around the layer in a residual block, each as
// one pass over the token rows: the RMS norm in front of it (enter), and
// behind it the norm of its output, the gates, the residual scale and the norm
// in front of the next block (exit), with their gradients.
//
//   r(x)   = 1 / sqrt(mean_j x_j^2 + eps)
//   enter  n = x r(x) w
//   exit   out = a res + b s(gt_t) c_j w_j y r(y),  n = out r(out) w_next
//          (s the logistic function; r(y) only with w; each part optional;
//          the next norm reads `out` as it is stored)
// Gradients, with h = y r(y), m_j = w_j c_j, o = out r(out):
//   g    = dout + r(out) (dn w_next - o mean(dn w_next o))
//   dz   = b s g,  dh = dz m,  dot = sum_j dh h
//   dres = a g,  dy = r(y) (dh - h dot / d),  dgt = (1 - s) dot
//   S_j  = sum_t dz h:  dw = c S, dc = w S;  dw_next = sum_t dn o
// enter's are g with x for out.
//
// Bound by memory: every element is read from it and written to it once.  A
// group of warps owns a row, a thread the same columns of all its group's
// rows.  Each thread copies its columns of the next rows into shared memory
// itself (cp.async, up to kMaxDepth rows ahead) and reads only its own copies,
// so the loads need no barrier and no registers; a row is read from there as
// often as its passes need it.  Sums are fp32 in a fixed order.
//
// Measured: exit 4096 x 7168 bf16 43 us, 5.4 TB/s (a plain copy 6.55); its
// backward 8192 x 2048 bf16 53 us, 4.4 TB/s: its loads alone take 33 us, the
// arithmetic alone 30, both and the stores 49, the columns' launch 4.4.  fp32
// rows take about twice the time of their bytes (enter 8192 x 2048 43 us, 3.1
// TB/s; exit 4096 x 2048 36): a thread's eight elements are two 16-byte pieces
// side by side, so that a warp's load or store uses half of each 32-byte sector
// that it asks L2 for.
#include <cuda_bf16.h>

#include <initializer_list>

#include "beam_internal.h"
#include "beam_ptx.cuh"

namespace beam {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxD = 16384;
constexpr int kMaxDepth = 4;             // rows a thread loads ahead
constexpr int kRingBytes = 200 * 1024;   // shared memory of an SM for them

// Eight consecutive elements, as stored: one 16-byte piece of bf16, two of fp32.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 1;
    uint4 p[1];
    __device__ float2 two(int i) const {  // elements 2 i and 2 i + 1
        const uint32_t w = i == 0 ? p[0].x : i == 1 ? p[0].y : i == 2 ? p[0].z : p[0].w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ void set(const float2 (&v)[4]) {  // one rounding, to the stored type
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[i].x, v[i].y);
        p[0] = *reinterpret_cast<uint4 *>(h);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 2;
    uint4 p[2];
    __device__ float2 two(int i) const {
        const uint4 &q = p[i >> 1];
        return (i & 1) ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w))
                       : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    }
    __device__ void set(const float2 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y),
                              __float_as_uint(v[2 * i + 1].x), __float_as_uint(v[2 * i + 1].y));
    }
};
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T *p) {
    Vec<T> v;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) v.p[i] = reinterpret_cast<const uint4 *>(p)[i];
    return v;
}
template <typename T>
__device__ __forceinline__ void store_vec(T *p, const Vec<T> &v) {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) reinterpret_cast<uint4 *>(p)[i] = v.p[i];
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// v times eight consecutive weights.
template <typename T>
__device__ __forceinline__ void times(float2 (&v)[4], const T *w) {
    const Vec<T> q = load_vec(w);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], q.two(k));
}
template <typename T>
__device__ __forceinline__ void weights_of(float2 (&v)[4], const T *a, const T *b, int j) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = both(1.0f);
    if (a) times(v, a + j);
    if (b) times(v, b + j);
}

// ---------------------------------------------------------- loads ahead --
// Shared memory of a CTA: [depth][pieces][CTA's threads at most] 16-byte
// pieces.  A stage's pieces are those of one row's arrays, NV vectors each;
// strides are the same for every launch of a kernel, so that a piece's address
// is a constant from its stage's.  A thread whose last columns lie behind the
// row finds zeros there, so only its copies and stores are left out.

// Until at most `left` of the thread's copies (one group per row) are open.
__device__ __forceinline__ void cp_async_wait_for(int left) {
    if (left == 0)
        cp_async_wait<0>();
    else if (left == 1)
        cp_async_wait<1>();
    else if (left == 2)
        cp_async_wait<2>();
    else
        cp_async_wait<3>();
}

template <int THREADS, typename T>
__device__ __forceinline__ void copy_ahead(uint4 *piece, const T *src) {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
        cp_async_16(piece + i * THREADS, reinterpret_cast<const uint4 *>(src) + i);
}
template <int THREADS, typename T>
__device__ __forceinline__ Vec<T> read_copy(const uint4 *piece) {
    Vec<T> v;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) v.p[i] = piece[i * THREADS];
    return v;
}

// ------------------------------------------------------------- row sums --
// A row's warps, and two scratch buffers in turn, so that one barrier per
// reduction does (a buffer is written again only after every warp has passed
// the next reduction's barrier, so after it has read this one).
struct Row {
    int warps, group, lane, warp;  // warps per row, group in the CTA, lane, warp in the group
    float *now, *next;             // [warps][8] each, of this group
};

__device__ __forceinline__ Row this_row(int warps, float *scratch) {
    Row r;
    r.warps = warps;
    const int w = threadIdx.x >> 5;
    r.group = w / warps;
    r.warp = w - r.group * warps;
    r.lane = threadIdx.x & 31;
    r.now = scratch + r.group * warps * 16;
    r.next = r.now + warps * 8;
    return r;
}

// Every thread then reads the buffer this returns.
__device__ __forceinline__ const float *shared_by_group(Row &r) {
    asm volatile("bar.sync %0, %1;" ::"r"(r.group + 1), "r"(r.warps * 32) : "memory");
    const float *s = r.now;
    r.now = r.next;
    r.next = const_cast<float *>(s);
    return s;
}

// Two sums at once: half of the lanes carry each.
__device__ __forceinline__ void row_sum2(Row &r, float &a, float &b) {
    const bool up = (r.lane & 16) != 0;
    const float other = __shfl_xor_sync(kAll, up ? a : b, 16);
    float t = (up ? b : a) + other;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
    if (r.warps > 1) {
        if ((r.lane & 15) == 0) r.now[r.warp * 8 + (r.lane >> 4)] = t;
        const float *s = shared_by_group(r);
        const int w = r.lane & 15;  // at most 16 warps
        t = w < r.warps ? s[w * 8 + (r.lane >> 4)] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
    }
    a = __shfl_sync(kAll, t, 0);
    b = __shfl_sync(kAll, t, 16);
}

// Eight sums at once: each exchange halves the values a lane carries, nine
// shuffles instead of forty.
__device__ __forceinline__ void row_sum8(Row &r, float (&v)[8]) {
#pragma unroll
    for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
        const bool up = (r.lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n];
            v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(kAll, send, o);
        }
    }
    float t = v[0];  // of value lane / 4
    t += __shfl_xor_sync(kAll, t, 2);
    t += __shfl_xor_sync(kAll, t, 1);
    int step = 4;
    if (r.warps > 1) {
        if ((r.lane & 3) == 0) r.now[r.warp * 8 + (r.lane >> 2)] = t;
        const float *s = shared_by_group(r);
        t = 0.0f;
        for (int w = r.lane >> 3; w < r.warps; w += 4) t += s[w * 8 + (r.lane & 7)];
        t += __shfl_xor_sync(kAll, t, 8);
        t += __shfl_xor_sync(kAll, t, 16);
        step = 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(kAll, t, i * step);
}

// ------------------------------------------------------------- forward --
// Weights stay in registers where a thread has one or two vectors; the pair w,
// gate_c is multiplied once.  A thread's fixed costs per row (addresses, the
// reduction) are as large as the arithmetic of eight elements: hence up to
// four vectors a thread.  Two CTAs of 448 threads leave a thread 72 registers,
// which hold two bf16 vectors' state; with 512 (64 registers) some of it
// spilled.
template <int NV>
constexpr int kFwThreads = NV <= 2 ? 448 : 512;

template <typename T, int NV, bool BRANCH>
__global__ void __launch_bounds__(kFwThreads<NV>, NV <= 2 ? 2 : 1)
    block_forward_kernel(const BlockArgs a, int depth, int warps) {
    constexpr int THREADS = kFwThreads<NV>;
    constexpr bool KEEP = NV <= 1 || (NV == 2 && sizeof(T) == 2);
    constexpr int N = Vec<T>::N;
    constexpr int kVec = N * THREADS, kY = NV * kVec;  // next vector's pieces, y's first
    constexpr int kStage = (BRANCH ? 2 : 1) * NV * kVec;
    extern __shared__ uint4 s_ring[];
    __shared__ float scratch[2 * 16 * 8];
    griddep_wait();
    griddep_launch_dependents();
    Row row = this_row(warps, scratch);
    const int groups = (blockDim.x >> 5) / warps;
    const int lanes = warps * 32, me = row.warp * 32 + row.lane;
    const float inv_d = 1.0f / float(a.d), eps = a.eps, res_scale = a.res_scale;
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    const T *gt = static_cast<const T *>(a.gt), *wn = static_cast<const T *>(a.wn);
    const unsigned step = gridDim.x * groups, rows = a.T;
    unsigned t = blockIdx.x * groups + row.group;
    const long long hop = (long long)step * a.d;
    uint4 *const base = s_ring + threadIdx.x;
    const int wrap = depth * kStage;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        in[i] = (i * lanes + me) * 8 < a.d;
        if (!in[i])
            for (int s = 0; s < wrap; s += kStage)
#pragma unroll
                for (int q = 0; q < (BRANCH ? 2 : 1) * N; ++q)
                    base[s + (q / N) * kY + i * kVec + (q % N) * THREADS] = make_uint4(0u, 0u, 0u, 0u);
    }
    long long at = (long long)t * a.d + me * 8, ahead = at;
    unsigned t_ahead = t;
    auto fetch = [&](int stage) {
        if (t_ahead < rows) {
            const T *x = static_cast<const T *>(a.x) + ahead, *y = static_cast<const T *>(a.y) + ahead;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) {
                    copy_ahead<THREADS>(base + stage + i * kVec, x + i * lanes * 8);
                    if (BRANCH) copy_ahead<THREADS>(base + stage + kY + i * kVec, y + i * lanes * 8);
                }
        }
        cp_async_commit();
        t_ahead += step;
        ahead += hop;
    };
    for (int s = 0; s < wrap; s += kStage) fetch(s);
    float2 mw[KEEP ? NV : 1][4];
    Vec<T> nw[KEEP ? NV : 1];
    auto column = [&](int i) { return in[i] ? (i * lanes + me) * 8 : 0; };
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (BRANCH) weights_of(mw[i], w, gc, column(i));
            if (wn) nw[i] = load_vec(wn + column(i));
        }
    }
    // The square sum of the next row's y is taken before this row's out is
    // normed, so that one reduction per row does for both.
    auto squares = [&](int stage) {
        float2 yy = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Vec<T> v = read_copy<THREADS, T>(base + stage + kY + i * kVec);
#pragma unroll
            for (int k = 0; k < 4; ++k) yy = __ffma2_rn(v.two(k), v.two(k), yy);
        }
        return yy.x + yy.y;
    };
    const bool norm = BRANCH && w;
    cp_async_wait_for(depth - 1);
    float gate = gt && t < rows ? to_f(gt[t]) : 0.0f;
    float yy = norm && t < rows ? squares(0) : 0.0f, unused = 0.0f;
    if (norm && t < rows) row_sum2(row, yy, unused);
    for (int stage = 0; t < rows; t += step, at += hop) {
        float s = a.branch_scale;
        if (BRANCH) {
            if (gt) s *= 1.0f / (1.0f + expf(-gate));
            if (norm) s *= rsqrtf(fmaf(yy, inv_d, eps));
        }
        const bool more = t + step < rows;
        if (gt && more) gate = to_f(gt[t + step]);
        Vec<T> o[NV];
        float2 oo = both(0.0f);
        T *out = static_cast<T *>(a.out) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[i] = read_copy<THREADS, T>(base + stage + i * kVec);
            if (BRANCH) {
                const Vec<T> v = read_copy<THREADS, T>(base + stage + kY + i * kVec);
                float2 m[4], f[4];
                if constexpr (KEEP) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) m[k] = mw[i][k];
                } else {
                    weights_of(m, w, gc, column(i));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    f[k] = __ffma2_rn(both(res_scale), o[i].two(k),
                                      __fmul2_rn(__fmul2_rn(m[k], both(s)), v.two(k)));
                o[i].set(f);
                if (in[i]) store_vec(out + i * lanes * 8, o[i]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) oo = __ffma2_rn(o[i].two(k), o[i].two(k), oo);
        }
        fetch(stage);
        stage = stage + kStage == wrap ? 0 : stage + kStage;
        cp_async_wait_for(depth - 1);  // the next row's copies
        yy = norm && more ? squares(stage) : 0.0f;
        float sum = oo.x + oo.y;
        if (wn || norm) row_sum2(row, sum, yy);
        if (!wn) continue;
        const float r = rsqrtf(fmaf(sum, inv_d, eps));
        T *n = static_cast<T *>(a.n) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float2 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = __fmul2_rn(o[i].two(k), both(r));
            if constexpr (KEEP) {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = __fmul2_rn(f[k], nw[i].two(k));
            } else {
                times(f, wn + column(i));
            }
            o[i].set(f);
            if (in[i]) store_vec(n + i * lanes * 8, o[i]);
        }
    }
}

// ------------------------------------------------------------ backward --
// One reduction of six sums per row: dot is linear in g, so its three parts
// are summed before r(out) is known.  A thread owns its columns for all its
// rows; a CTA's groups add theirs up in order, and each CTA writes one slab
// [2][d] (S, dw_next) that block_columns_kernel adds up in order.
// BRANCH: exit's (else enter's, whose out is x); NEXT: with w_next.
// A thread's columns of the sums and the weights stay in registers: 512
// threads of 128 (640 of 96 spilled: 56 us became 90 at 8192 x 2048).
template <int NV>
constexpr int kBwThreads = NV == 1 ? 768 : 512;

template <typename T, int NV, bool BRANCH, bool NEXT>
__global__ void __launch_bounds__(kBwThreads<NV>, 1)
    block_backward_kernel(const BlockArgs a, int depth, int ring_n, int warps) {
    constexpr int THREADS = kBwThreads<NV>;
    constexpr bool KEEP = NV <= 2;
    constexpr int N = Vec<T>::N, kVec = N * THREADS;
    constexpr int kY = NEXT ? NV * kVec : 0, kG = kY + (BRANCH ? NV * kVec : 0), kN = kG + NV * kVec;
    constexpr int kStage = kN + (NEXT ? NV * 2 * THREADS : 0);
    constexpr bool ALWAYS = NV < 4 || sizeof(T) == 2;  // dn is copied too
    extern __shared__ uint4 s_ring[];
    __shared__ float scratch[2 * (THREADS / 32) * 8];
    griddep_wait();
    griddep_launch_dependents();
    Row row = this_row(warps, scratch);
    const int groups = (blockDim.x >> 5) / warps;
    const int d = a.d, lanes = warps * 32, me = row.warp * 32 + row.lane;
    const float inv_d = 1.0f / float(d), eps = a.eps, res_scale = a.res_scale;
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    const T *gt = static_cast<const T *>(a.gt), *wn = static_cast<const T *>(a.wn);
    const bool has_g = BRANCH || a.dout != nullptr;
    const unsigned step = gridDim.x * groups, rows = a.T;
    unsigned t = blockIdx.x * groups + row.group;
    const long long hop = (long long)step * d;
    uint4 *const base = s_ring + threadIdx.x;
    // dn is the last array of a stage, and of all where it is not copied
    const int stage_step = ALWAYS || ring_n ? kStage : kN, wrap = depth * stage_step;
    bool in[NV];
    float2 cs[NV][4], cn[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        in[i] = (i * lanes + me) * 8 < d;
#pragma unroll
        for (int k = 0; k < 4; ++k) cs[i][k] = cn[i][k] = both(0.0f);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int s = 0; s < wrap; s += stage_step) {
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const int at = s + i * kVec + q * THREADS;
                if (!in[i] && NEXT) base[at] = zero;
                if (!in[i] && BRANCH) base[at + kY] = zero;
                if (!in[i] || !has_g) base[at + kG] = zero;
            }
            if (NEXT && !in[i] && (ALWAYS || ring_n))
                base[s + kN + i * 2 * THREADS] = base[s + kN + i * 2 * THREADS + THREADS] = zero;
        }
    }
    long long at = (long long)t * d + me * 8, ahead = at;
    unsigned t_ahead = t;
    auto fetch = [&](int stage) {
        if (t_ahead < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) {
                    const long long q = ahead + i * lanes * 8;
                    uint4 *to = base + stage + i * kVec;
                    if (NEXT) copy_ahead<THREADS>(to, static_cast<const T *>(a.x) + q);
                    if (BRANCH) copy_ahead<THREADS>(to + kY, static_cast<const T *>(a.y) + q);
                    if (has_g) copy_ahead<THREADS>(to + kG, static_cast<const T *>(a.dout) + q);
                    if (NEXT && (ALWAYS || ring_n))
                        copy_ahead<THREADS>(base + stage + kN + i * 2 * THREADS, a.dn + q);
                }
        }
        cp_async_commit();
        t_ahead += step;
        ahead += hop;
    };
    for (int s = 0; s < wrap; s += stage_step) fetch(s);
    float2 mw[KEEP ? NV : 1][4], nw[KEEP ? NV : 1][4];
    auto column = [&](int i) { return in[i] ? (i * lanes + me) * 8 : 0; };
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (BRANCH) weights_of(mw[i], w, gc, column(i));
            if (NEXT) weights_of(nw[i], wn, static_cast<const T *>(nullptr), column(i));
        }
    }
    float gate = gt && t < rows ? to_f(gt[t]) : 0.0f;
    struct Pieces {
        Vec<T> o, y, g;
        Vec<float> n;
    };
    auto read = [&](Pieces &c, int stage, int i) {
        const uint4 *from = base + stage + i * kVec;
        if (NEXT) {
            c.o = read_copy<THREADS, T>(from);
            if (ALWAYS || ring_n)
                c.n = read_copy<THREADS, float>(base + stage + kN + i * 2 * THREADS);
            else if (in[i])
                c.n = load_vec(a.dn + at + i * lanes * 8);
            else
                c.n.p[0] = c.n.p[1] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (BRANCH) c.y = read_copy<THREADS, T>(from + kY);
        c.g = read_copy<THREADS, T>(from + kG);
    };
    auto weights = [&](float2(&m)[4], float2(&p)[4], int i) {
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = mw[i][k];
                p[k] = nw[i][k];
            }
        } else {
            if (BRANCH) weights_of(m, w, gc, column(i));
            if (NEXT) weights_of(p, wn, static_cast<const T *>(nullptr), column(i));
        }
    };
    for (int stage = 0; t < rows; t += step, at += hop) {
        const float z = gate;
        if (gt && t + step < rows) gate = to_f(gt[t + step]);
        cp_async_wait_for(depth - 1);
        float2 q[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) q[k] = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pieces c;
            read(c, stage, i);
            float2 m[4], p[4];
            weights(m, p, i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 o, pk, yk, mk;
                if (NEXT) {
                    o = c.o.two(k);
                    pk = __fmul2_rn(p[k], c.n.two(k));
                    q[0] = __ffma2_rn(o, o, q[0]);
                    q[1] = __ffma2_rn(pk, o, q[1]);
                }
                if (BRANCH) {
                    yk = c.y.two(k);
                    mk = __fmul2_rn(m[k], yk);
                    q[2] = __ffma2_rn(yk, yk, q[2]);
                    q[3] = __ffma2_rn(mk, c.g.two(k), q[3]);
                }
                if (BRANCH && NEXT) {
                    q[4] = __ffma2_rn(mk, pk, q[4]);
                    q[5] = __ffma2_rn(mk, o, q[5]);
                }
            }
        }
        float sum[8];
#pragma unroll
        for (int k = 0; k < 6; ++k) sum[k] = q[k].x + q[k].y;
        sum[6] = sum[7] = 0.0f;
        row_sum8(row, sum);
        const float ro = NEXT ? rsqrtf(fmaf(sum[0], inv_d, eps)) : 0.0f;
        // mean(dn w o) of the formula, o normed; no power of r(out) above one
        // is formed, which tiny rows would take past fp32
        const float mo = ro * sum[1] * inv_d;
        float sig = 1.0f, ry = 1.0f, back = 0.0f;
        if (BRANCH) {
            float rest = 0.0f;  // 1 - sig, which near 1 has no digits left of sig's
            if (gt) {
                sig = 1.0f / (1.0f + expf(-z));
                rest = 1.0f / (1.0f + expf(z));
            }
            if (w) ry = rsqrtf(fmaf(sum[2], inv_d, eps));
            const float dot =
                a.branch_scale * sig * ry * (sum[3] + ro * (sum[4] - mo * (ro * sum[5])));
            if (w) back = -(dot * inv_d) * ry * ry;
            if (gt && me == 0) a.dgt[t] = rest * dot;
        }
        const float zs = a.branch_scale * sig * ry;
        T *dres = static_cast<T *>(a.dres) + at, *dy = static_cast<T *>(a.dy) + at;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pieces c;
            read(c, stage, i);
            float2 m[4], p[4], g[4], f[4];
            weights(m, p, i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] = c.g.two(k);
                if (NEXT) {
                    const float2 o = __fmul2_rn(c.o.two(k), both(ro)), n = c.n.two(k);
                    const float2 u = __ffma2_rn(both(-mo), o, __fmul2_rn(p[k], n));
                    g[k] = __ffma2_rn(both(ro), u, g[k]);
                    cn[i][k] = __ffma2_rn(n, o, cn[i][k]);
                }
                f[k] = __fmul2_rn(both(res_scale), g[k]);
            }
            Vec<T> r;
            r.set(f);
            if (in[i]) store_vec(dres + i * lanes * 8, r);
            if constexpr (BRANCH) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = c.y.two(k), e = __fmul2_rn(both(zs), g[k]);  // r(y) dz
                    cs[i][k] = __ffma2_rn(e, y, cs[i][k]);
                    f[k] = __ffma2_rn(e, m[k], __fmul2_rn(both(back), y));
                }
                r.set(f);
                if (in[i]) store_vec(dy + i * lanes * 8, r);
            }
        }
        fetch(stage);
        stage = stage + stage_step == wrap ? 0 : stage + stage_step;
    }
    if (!a.part) return;
    // The CTA's slab: its groups' columns, [groups][2][d] in what was the
    // ring, added up in order.
    cp_async_wait<0>();
    __syncthreads();
    float *s_cols = reinterpret_cast<float *>(s_ring), *mine = s_cols + row.group * 2 * d;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
            const int j = (i * lanes + me) * 8;
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                *reinterpret_cast<float4 *>(mine + j + 2 * k) =
                    make_float4(cs[i][k].x, cs[i][k].y, cs[i][k + 1].x, cs[i][k + 1].y);
                *reinterpret_cast<float4 *>(mine + d + j + 2 * k) =
                    make_float4(cn[i][k].x, cn[i][k].y, cn[i][k + 1].x, cn[i][k + 1].y);
            }
        }
    __syncthreads();
    float *slab = a.part + (long long)blockIdx.x * 2 * d;
    const int from = a.dw || a.dgc ? 0 : d, to = a.dwn ? 2 * d : d;
    for (int j = from + threadIdx.x * 4; j < to; j += blockDim.x * 4) {
        float4 v = *reinterpret_cast<const float4 *>(s_cols + j);
        for (int g = 1; g < groups; ++g) {
            const float4 u = *reinterpret_cast<const float4 *>(s_cols + g * 2 * d + j);
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        *reinterpret_cast<float4 *>(slab + j) = v;
    }
}

// The slabs' sums and the weight gradients they give: 32 columns a CTA, thread
// (p, c) adds four columns of slabs p, p + 64, ..., then the 64 parts are
// added in order.
template <typename T>
__global__ void __launch_bounds__(512) block_columns_kernel(const BlockArgs a, int slabs) {
    __shared__ float4 s[2][64][8];
    griddep_wait();
    griddep_launch_dependents();
    const int c = threadIdx.x & 7, p = threadIdx.x >> 3, j4 = (blockIdx.x * 8 + c) * 4;
    const bool first = a.dw || a.dgc, second = a.dwn != nullptr;
    float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (j4 < a.d) {
#pragma unroll 4
        for (int b = p; b < slabs; b += 64) {
            const float *q = a.part + (long long)b * 2 * a.d + j4;
            if (first) {
                const float4 u = *reinterpret_cast<const float4 *>(q);
                v[0].x += u.x; v[0].y += u.y; v[0].z += u.z; v[0].w += u.w;
            }
            if (second) {
                const float4 u = *reinterpret_cast<const float4 *>(q + a.d);
                v[1].x += u.x; v[1].y += u.y; v[1].z += u.z; v[1].w += u.w;
            }
        }
    }
    s[0][p][c] = v[0];
    s[1][p][c] = v[1];
    __syncthreads();
    const int which = threadIdx.x >> 5, col = threadIdx.x & 31, j = blockIdx.x * 32 + col;
    if (which > 1 || j >= a.d) return;
    float t = 0.0f;
#pragma unroll
    for (int b = 0; b < 64; ++b) t += reinterpret_cast<const float *>(&s[which][b][0])[col];
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    auto put = [&](float *to, float v) { to[j] = a.accumulate ? to[j] + v : v; };
    if (which == 0) {
        if (a.dw) put(a.dw, gc ? to_f(gc[j]) * t : t);
        if (a.dgc) put(a.dgc, w ? to_f(w[j]) * t : t);
    } else if (a.dwn) {
        put(a.dwn, t);
    }
}

// --------------------------------------------------------------- launch --
// Warps per row: a row's vectors of eight over its lanes, nv each.
struct Shape {
    int nv, warps, groups, grid, per_sm;
};

int threads_of(int nv, bool backward) {
    if (backward) return nv == 1 ? kBwThreads<1> : nv == 2 ? kBwThreads<2> : kBwThreads<4>;
    return nv == 1 ? kFwThreads<1> : nv == 2 ? kFwThreads<2> : kFwThreads<4>;
}

Shape shape_of(const beam_block_desc *d, bool backward) {
    Shape s;
    const int vecs = d->d / 8, rows = d->T / kNominalSMs + (d->T % kNominalSMs != 0);
    s.nv = 1;
    while (vecs > s.nv * threads_of(s.nv, backward)) s.nv *= 2;
    // Many rows per SM: fewer, busier warps; few: more warps, sooner done.  8 M
    // elements, one vector a thread against two: exit bf16 d = 2048 19.3 / 15.6
    // us, d = 640 17.5 / 17.7, fp32 35.2 / 38.3; its backward bf16 d = 640 38.2 /
    // 35.7, d = 112 46.7 / 63.7, fp32 d = 2048 68.3 / 62.3, d = 5000 93 / 104.
    const bool bf16 = d->dtype == BEAM_BF16;
    const bool two = backward ? vecs >= 64 && (bf16 || vecs <= 512) : vecs >= 112 && bf16;
    if (s.nv == 1 && rows >= 4 && two) s.nv = 2;
    s.warps = (vecs + 32 * s.nv - 1) / (32 * s.nv);
    s.groups = threads_of(s.nv, backward) / 32 / s.warps;
    if (s.warps > 1 && s.groups > 15) s.groups = 15;  // named barriers 1..15
    // rather a row on every SM than several on a few
    s.per_sm = backward || s.nv > 2 ? 1 : 2;
    if (s.groups * s.per_sm > rows) s.groups = rows > s.per_sm ? rows / s.per_sm : 1;
    const long long want = ((long long)d->T + s.groups - 1) / s.groups;
    const long long cap = (long long)kNominalSMs * s.per_sm;
    s.grid = int(want < cap ? want : cap);
    return s;
}

// Rows ahead: as many as shared memory holds, and no more than there are.
int depth_for(size_t stage, const Shape &s, int T) {
    const long long at_once = (long long)s.grid * s.groups, rows = (T + at_once - 1) / at_once;
    int depth = kMaxDepth;
    while (depth > 1 && (depth * stage * s.per_sm > size_t(kRingBytes) || depth > rows)) --depth;
    return depth;
}

size_t slab_bytes(const beam_block_desc *d) {
    return d->T == 0 ? 0 : size_t(shape_of(d, true).grid) * 2 * size_t(d->d) * sizeof(float);
}

constexpr int kSmemMost = 208 * 1024;

template <typename T, int NV, bool BRANCH>
cudaError_t launch_forward_nv(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    auto kern = block_forward_kernel<T, NV, BRANCH>;
    static std::atomic<unsigned long long> attr_set{0};  // this instantiation only
    cudaError_t e = set_smem_once(kern, kSmemMost, attr_set);
    if (e != cudaSuccess) return e;
    const size_t stage = size_t(kFwThreads<NV>) * 16 * NV * (BRANCH ? 2 : 1) * (sizeof(T) / 2);
    const int depth = depth_for(stage, s, a.T);
    return launch_pdl(kern, dim3(s.grid), dim3(s.groups * s.warps * 32), depth * stage, st, a,
                      depth, s.warps);
}

template <typename T, bool BRANCH>
cudaError_t launch_forward(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    return s.nv == 1   ? launch_forward_nv<T, 1, BRANCH>(a, s, st)
           : s.nv == 2 ? launch_forward_nv<T, 2, BRANCH>(a, s, st)
                       : launch_forward_nv<T, 4, BRANCH>(a, s, st);
}

template <typename T, int NV, bool BRANCH, bool NEXT>
cudaError_t launch_backward_nv(const BlockArgs &a, Shape s, cudaStream_t st) {
    auto kern = block_backward_kernel<T, NV, BRANCH, NEXT>;
    static std::atomic<unsigned long long> attr_set{0};  // this instantiation only
    cudaError_t e = set_smem_once(kern, kSmemMost, attr_set);
    if (e != cudaSuccess) return e;
    // the widest fp32 rows leave no room for dn, which is then read in place
    const size_t plane = size_t(kBwThreads<NV>) * 16 * NV;
    size_t stage = plane * (1 + BRANCH + NEXT) * (sizeof(T) / 2);
    const int ring_n = NEXT && stage + 2 * plane <= size_t(kRingBytes);
    if (ring_n) stage += 2 * plane;
    const int depth = depth_for(stage, s, a.T);
    size_t smem = depth * stage;
    const size_t slab = size_t(s.groups) * a.d * 8;  // at most 32 KB a vector and thread
    if (a.part && smem < slab) smem = slab;
    return launch_pdl(kern, dim3(s.grid), dim3(s.groups * s.warps * 32), smem, st, a, depth, ring_n,
                      s.warps);
}

template <typename T, bool BRANCH, bool NEXT>
cudaError_t launch_backward(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    cudaError_t e = s.nv == 1   ? launch_backward_nv<T, 1, BRANCH, NEXT>(a, s, st)
                    : s.nv == 2 ? launch_backward_nv<T, 2, BRANCH, NEXT>(a, s, st)
                                : launch_backward_nv<T, 4, BRANCH, NEXT>(a, s, st);
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(block_columns_kernel<T>, dim3((a.d + 31) / 32), dim3(512), 0, st, a, s.grid);
}

bool bad16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

beam_status check_block_desc(const beam_block_desc *d) {
    if (!d) return BEAM_ERR_INVALID_ARG;
    if (d->T < 0 || d->d <= 0) return BEAM_ERR_INVALID_ARG;
    if (d->dtype != BEAM_BF16 && d->dtype != BEAM_F32) return BEAM_ERR_INVALID_ARG;
    // r(x)^2 has to stay far from fp32's end
    if (!(d->eps >= 1.0e-30f) || !(d->eps < 3.0e38f)) return BEAM_ERR_INVALID_ARG;
    if (!(d->res_scale - d->res_scale == 0.0f) || !(d->branch_scale - d->branch_scale == 0.0f))
        return BEAM_ERR_INVALID_ARG;  // infinite or NaN
    if (d->accumulate != 0 && d->accumulate != 1) return BEAM_ERR_INVALID_ARG;
    if (d->d % 8 != 0 || d->d > kMaxD) return BEAM_ERR_UNSUPPORTED_SHAPE;
    return BEAM_OK;
}

BlockArgs block_args(const beam_block_desc *d) {
    BlockArgs a = {};
    a.T = d->T;
    a.d = d->d;
    a.eps = d->eps;
    a.res_scale = d->res_scale;
    a.branch_scale = d->branch_scale;
    a.accumulate = d->accumulate;
    return a;
}

beam_status check_workspace(const beam_block_desc *d, const void *ws, size_t bytes) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || bytes < beam_block_workspace_size(d))
        return BEAM_ERR_WORKSPACE;
    return BEAM_OK;
}

// T = 0: the sums over no rows.
beam_status zero_columns(const beam_block_desc *d, std::initializer_list<float *> to,
                         cudaStream_t st) {
    if (!d->accumulate)
        for (float *p : to)
            if (p && cudaMemsetAsync(p, 0, sizeof(float) * size_t(d->d), st) != cudaSuccess)
                return BEAM_ERR_CUDA;
    return BEAM_OK;
}

beam_status done(cudaError_t e) { return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA; }

}  // namespace
}  // namespace beam

using namespace beam;

extern "C" {

size_t beam_block_workspace_size(const beam_block_desc *desc) {
    if (check_block_desc(desc) != BEAM_OK) return 0;
    return (slab_bytes(desc) + 511) & ~size_t(255);
}

beam_status beam_block_enter(const beam_block_desc *desc, const void *x, const void *w, void *n,
                             void *stream) {
    beam_status s = check_block_desc(desc);
    if (s != BEAM_OK) return s;
    for (const void *p : {x, w, static_cast<const void *>(n)})
        if (bad16(p) || (!p && desc->T > 0)) return BEAM_ERR_INVALID_ARG;
    if (desc->T == 0) return BEAM_OK;
    BlockArgs a = block_args(desc);
    a.x = x;
    a.wn = w;
    a.n = n;
    const Shape sh = shape_of(desc, false);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return done(desc->dtype == BEAM_BF16 ? launch_forward<__nv_bfloat16, false>(a, sh, st)
                                         : launch_forward<float, false>(a, sh, st));
}

beam_status beam_block_exit(const beam_block_desc *desc, const void *res, const void *y,
                            const void *w_out, const void *gate_c, const void *gate_t, void *out,
                            const void *w_next, void *n_next, void *stream) {
    beam_status s = check_block_desc(desc);
    if (s != BEAM_OK) return s;
    for (const void *p : {res, y, static_cast<const void *>(out)})
        if (bad16(p) || (!p && desc->T > 0)) return BEAM_ERR_INVALID_ARG;
    for (const void *p : {w_out, gate_c, gate_t, w_next, static_cast<const void *>(n_next)})
        if (bad16(p)) return BEAM_ERR_INVALID_ARG;
    if (desc->T == 0) return BEAM_OK;
    if (!w_next != !n_next) return BEAM_ERR_INVALID_ARG;
    BlockArgs a = block_args(desc);
    a.x = res;
    a.y = y;
    a.w = w_out;
    a.gc = gate_c;
    a.gt = gate_t;
    a.out = out;
    a.wn = w_next;
    a.n = n_next;
    const Shape sh = shape_of(desc, false);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return done(desc->dtype == BEAM_BF16 ? launch_forward<__nv_bfloat16, true>(a, sh, st)
                                         : launch_forward<float, true>(a, sh, st));
}

beam_status beam_block_enter_backward(const beam_block_desc *desc, const void *x, const void *w,
                                      const float *dn, const void *dskip, void *dx, float *dw,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    beam_status s = check_block_desc(desc);
    if (s != BEAM_OK) return s;
    for (const void *p : {x, w, static_cast<const void *>(dn), static_cast<const void *>(dx)})
        if (bad16(p) || (!p && desc->T > 0)) return BEAM_ERR_INVALID_ARG;
    if (!dw || bad16(dw) || bad16(dskip)) return BEAM_ERR_INVALID_ARG;
    s = check_workspace(desc, workspace, workspace_bytes);
    if (s != BEAM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) return zero_columns(desc, {dw}, st);
    BlockArgs a = block_args(desc);
    a.res_scale = 1.0f;
    a.x = x;
    a.wn = w;
    a.dn = dn;
    a.dout = dskip;
    a.dres = dx;
    a.dwn = dw;
    a.part = static_cast<float *>(workspace);
    const Shape sh = shape_of(desc, true);
    return done(desc->dtype == BEAM_BF16 ? launch_backward<__nv_bfloat16, false, true>(a, sh, st)
                                         : launch_backward<float, false, true>(a, sh, st));
}

beam_status beam_block_exit_backward(const beam_block_desc *desc, const void *y, const void *out,
                                     const void *w_out, const void *gate_c, const void *gate_t,
                                     const void *w_next, const void *dout, const float *dn_next,
                                     void *dres, void *dy, float *dw_out, float *dgate_c,
                                     float *dgate_t, float *dw_next, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    beam_status s = check_block_desc(desc);
    if (s != BEAM_OK) return s;
    for (const void *p : {y, dout, static_cast<const void *>(dres), static_cast<const void *>(dy)})
        if (bad16(p) || (!p && desc->T > 0)) return BEAM_ERR_INVALID_ARG;
    for (const void *p : {out, w_out, gate_c, gate_t, w_next, static_cast<const void *>(dn_next),
                          static_cast<const void *>(dw_out), static_cast<const void *>(dgate_c),
                          static_cast<const void *>(dgate_t), static_cast<const void *>(dw_next)})
        if (bad16(p)) return BEAM_ERR_INVALID_ARG;
    // each weight with its gradient; the next norm with its input's too
    if (!w_out != !dw_out || !gate_c != !dgate_c || !w_next != !dw_next) return BEAM_ERR_INVALID_ARG;
    if (desc->T > 0 && (!gate_t != !dgate_t || !w_next != !dn_next || (w_next && !out)))
        return BEAM_ERR_INVALID_ARG;
    s = check_workspace(desc, workspace, workspace_bytes);
    if (s != BEAM_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) return zero_columns(desc, {dw_out, dgate_c, dw_next}, st);
    BlockArgs a = block_args(desc);
    a.x = out;
    a.y = y;
    a.w = w_out;
    a.gc = gate_c;
    a.gt = gate_t;
    a.wn = w_next;
    a.dout = dout;
    a.dn = dn_next;
    a.dres = dres;
    a.dy = dy;
    a.dw = dw_out;
    a.dgc = dgate_c;
    a.dgt = dgate_t;
    a.dwn = dw_next;
    a.part = dw_out || dgate_c || dw_next ? static_cast<float *>(workspace) : nullptr;
    const Shape sh = shape_of(desc, true);
    if (desc->dtype == BEAM_BF16)
        return done(w_next ? launch_backward<__nv_bfloat16, true, true>(a, sh, st)
                           : launch_backward<__nv_bfloat16, true, false>(a, sh, st));
    return done(w_next ? launch_backward<float, true, true>(a, sh, st)
                       : launch_backward<float, true, false>(a, sh, st));
}

}  // extern "C"
