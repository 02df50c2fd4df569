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
// Bound by memory: every element is read and written once, in 16-byte (fp32:
// 32-byte) pieces that stay in registers between the sums and the results.
// A group of warps owns a row; its sums are fp32 in a fixed order.
#include <cuda_bf16.h>

#include <initializer_list>

#include "beam_internal.h"
#include "beam_ptx.cuh"

namespace beam {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxD = 16384;
constexpr int kMaxWarps = 16;  // of a CTA

// Eight consecutive elements, as stored.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    uint4 r;
    __device__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = r; }
    __device__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
    __device__ float get(int i) const {
        const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ void set(const float (&v)[8]) {  // one rounding, to the stored type
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        r = *reinterpret_cast<uint4 *>(h);
    }
};
template <>
struct Vec<float> {
    float4 a, b;
    __device__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ float get(int i) const {
        const float4 &q = i < 4 ? a : b;
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    }
    __device__ void set(const float (&v)[8]) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// v times eight consecutive weights.
template <typename T>
__device__ __forceinline__ void times(float (&v)[8], const T *w) {
    Vec<T> q;
    q.load(w);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= q.get(k);
}

// A row's warps.  `slot` counts its reductions: two buffers in turn let one
// barrier per reduction do (a buffer is written again only after every warp
// has passed the next reduction's barrier, so after it has read this one).
struct Row {
    int warps, group, lane, warp;  // warps per row, group in the CTA, lane, warp in the group
    float *scratch;                // [2][groups][warps][N] of this CTA
    int slot;
};

__device__ __forceinline__ void group_sync(const Row &r) {
    if (r.warps > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(r.group + 1), "r"(r.warps * 32) : "memory");
}

template <int N>
__device__ __forceinline__ void row_sum(Row &r, float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kAll, v[i], o);
    if (r.warps == 1) return;
    float *s = r.scratch + ((r.slot & 1) * kMaxWarps + r.group * r.warps) * N;
    ++r.slot;
    if (r.lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[r.warp * N + i] = v[i];
    group_sync(r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = 0.0f;
        for (int w = 0; w < r.warps; ++w) t += s[w * N + i];
        v[i] = t;
    }
}

__device__ __forceinline__ Row this_row(int warps, float *scratch) {
    Row r;
    r.warps = warps;
    const int w = threadIdx.x >> 5;
    r.group = w / warps;
    r.warp = w - r.group * warps;
    r.lane = threadIdx.x & 31;
    r.scratch = scratch;
    r.slot = 0;
    return r;
}

// ------------------------------------------------------------- forward --
// The next row of a group is loaded before the current one's sums are waited
// for, so the memory system never idles through a barrier.
template <int NV>
constexpr int kMinCtas = NV == 1 ? 2 : 1;

template <typename T, int NV, bool BRANCH>
__global__ void __launch_bounds__(512, kMinCtas<NV>)
    block_forward_kernel(const BlockArgs a, int warps) {
    __shared__ float scratch[2 * kMaxWarps];
    griddep_wait();
    griddep_launch_dependents();
    Row row = this_row(warps, scratch);
    const int groups = (blockDim.x >> 5) / warps;
    const int d = a.d, lanes = warps * 32, me = row.warp * 32 + row.lane;
    const float inv_d = 1.0f / float(d);
    const T *x = static_cast<const T *>(a.x), *y = static_cast<const T *>(a.y);
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    const T *gt = static_cast<const T *>(a.gt), *wn = static_cast<const T *>(a.wn);
    T *out = static_cast<T *>(a.out), *n = static_cast<T *>(a.n);
    const long long step = (long long)gridDim.x * groups;
    long long t = (long long)blockIdx.x * groups + row.group;
    Vec<T> nx[NV], ny[NV];
    auto fetch = [&](long long q) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * lanes + me) * 8;
            if (q < a.T && j < d) {
                nx[i].load(x + q * d + j);
                if (BRANCH) ny[i].load(y + q * d + j);
            } else {
                nx[i].zero();
                if (BRANCH) ny[i].zero();
            }
        }
    };
    fetch(t);
    for (; t < a.T; t += step) {
        const long long at = t * d;
        Vec<T> o[NV], v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[i] = nx[i];
            v[i] = ny[i];
        }
        fetch(t + step);
        if (BRANCH) {
            float s = a.branch_scale;
            if (gt) s *= 1.0f / (1.0f + expf(-to_f(gt[t])));
            if (w) {
                float yy[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) yy[0] = fmaf(v[i].get(k), v[i].get(k), yy[0]);
                row_sum(row, yy);
                s *= rsqrtf(fmaf(yy[0], inv_d, a.eps));
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * lanes + me) * 8;
                if (j >= d) continue;
                float m[8], f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) m[k] = s;
                if (w) times(m, w + j);
                if (gc) times(m, gc + j);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = fmaf(a.res_scale, o[i].get(k), m[k] * v[i].get(k));
                o[i].set(f);
                o[i].store(out + at + j);
            }
        }
        if (!wn) continue;
        float sq[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) sq[0] = fmaf(o[i].get(k), o[i].get(k), sq[0]);
        row_sum(row, sq);
        const float r = rsqrtf(fmaf(sq[0], inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * lanes + me) * 8;
            if (j >= d) continue;
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = o[i].get(k) * r;
            times(f, wn + j);
            o[i].set(f);
            o[i].store(n + at + j);
        }
    }
}

// ------------------------------------------------------------ backward --
// One reduction of six sums per row: dot is linear in g, so its three parts
// are summed before r(out) is known.  A thread owns its columns for all its
// rows; a CTA's groups add theirs up in order, and each CTA writes one slab
// [2][d] (S, dw_next) that block_columns_kernel adds up in order.
template <typename T, int NV, bool BRANCH>
__global__ void __launch_bounds__(512, 1) block_backward_kernel(const BlockArgs a, int warps) {
    constexpr bool AHEAD = NV * sizeof(T) <= 4;  // registers for the next row's loads
    __shared__ float scratch[2 * kMaxWarps * 6];
    extern __shared__ float s_cols[];  // [2][d]
    griddep_wait();
    griddep_launch_dependents();
    Row row = this_row(warps, scratch);
    const int groups = (blockDim.x >> 5) / warps;
    const int d = a.d, lanes = warps * 32, me = row.warp * 32 + row.lane;
    const float inv_d = 1.0f / float(d);
    const T *x = static_cast<const T *>(a.x), *y = static_cast<const T *>(a.y);
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    const T *gt = static_cast<const T *>(a.gt), *wn = static_cast<const T *>(a.wn);
    const T *dout = static_cast<const T *>(a.dout);
    T *dres = static_cast<T *>(a.dres), *dy = static_cast<T *>(a.dy);
    float cs[NV][8], cn[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) cs[i][k] = cn[i][k] = 0.0f;
    const long long step = (long long)gridDim.x * groups;
    long long t = (long long)blockIdx.x * groups + row.group;
    struct Loads {
        Vec<T> o, y, g;
        Vec<float> n;
    };
    Loads c[NV];
    auto fetch = [&](Loads(&to)[NV], long long q) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * lanes + me) * 8;
            const bool in = q < a.T && j < d;
            const long long at = q * d + j;
            to[i].o.zero();
            to[i].y.zero();
            to[i].g.zero();
            to[i].n.zero();
            if (in && wn) {
                to[i].o.load(x + at);
                to[i].n.load(a.dn + at);
            }
            if (in && BRANCH) to[i].y.load(y + at);
            if (in && dout) to[i].g.load(dout + at);
        }
    };
    fetch(c, t);
    for (; t < a.T; t += step) {
        const long long at = t * d;
        Loads ahead[AHEAD ? NV : 1];
        if constexpr (AHEAD) fetch(ahead, t + step);
        float q[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * lanes + me) * 8;
            if (j >= d) continue;
            float m[8], p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m[k] = c[i].y.get(k);
                p[k] = c[i].n.get(k);
            }
            if (BRANCH && w) times(m, w + j);
            if (BRANCH && gc) times(m, gc + j);
            if (wn) times(p, wn + j);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float o = c[i].o.get(k);
                q[0] = fmaf(o, o, q[0]);
                q[1] = fmaf(p[k], o, q[1]);
                if (BRANCH) {
                    const float yk = c[i].y.get(k);
                    q[2] = fmaf(yk, yk, q[2]);
                    q[3] = fmaf(m[k], c[i].g.get(k), q[3]);
                    q[4] = fmaf(m[k], p[k], q[4]);
                    q[5] = fmaf(m[k], o, q[5]);
                }
            }
        }
        if (BRANCH) {
            row_sum(row, q);
        } else {
            float q2[2] = {q[0], q[1]};
            row_sum(row, q2);
            q[0] = q2[0];
            q[1] = q2[1];
        }
        const float ro = wn ? rsqrtf(fmaf(q[0], inv_d, a.eps)) : 0.0f;
        // mean(dn w o) of the formula, o normed; no power of r(out) above one
        // is formed, which tiny rows would take past fp32
        const float mo = ro * q[1] * inv_d;
        float sig = 1.0f, ry = 1.0f, dot = 0.0f, back = 0.0f;
        if (BRANCH) {
            float rest = 0.0f;  // 1 - sig, which near 1 has no digits left of sig's
            if (gt) {
                const float z = to_f(gt[t]);
                sig = 1.0f / (1.0f + expf(-z));
                rest = 1.0f / (1.0f + expf(z));
            }
            if (w) ry = rsqrtf(fmaf(q[2], inv_d, a.eps));
            dot = a.branch_scale * sig * ry * (q[3] + ro * (q[4] - mo * (ro * q[5])));
            if (w) back = dot * inv_d;
            if (gt && me == 0) a.dgt[t] = rest * dot;
        }
        const float zs = a.branch_scale * sig;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = (i * lanes + me) * 8;
            if (j >= d) continue;
            float g[8], f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = c[i].n.get(k);
            if (wn) times(g, wn + j);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float o = c[i].o.get(k) * ro;
                g[k] = fmaf(ro, g[k] - mo * o, c[i].g.get(k));
                cn[i][k] = fmaf(c[i].n.get(k), o, cn[i][k]);
                f[k] = a.res_scale * g[k];
            }
            Vec<T> r;
            r.set(f);
            r.store(dres + at + j);
            if constexpr (BRANCH) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    g[k] *= zs;  // dz
                    cs[i][k] = fmaf(g[k], c[i].y.get(k) * ry, cs[i][k]);
                }
                if (w) times(g, w + j);
                if (gc) times(g, gc + j);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = ry * (g[k] - c[i].y.get(k) * ry * back);
                r.set(f);
                r.store(dy + at + j);
            }
        }
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = ahead[i];
        } else {
            fetch(c, t + step);
        }
    }
    if (!a.part) return;
    // The CTA's slab: its groups in order.
    for (int g = 0; g < groups; ++g) {
        if (row.group == g)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = (i * lanes + me) * 8;
                if (j >= d) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s_cols[j + k] = g ? s_cols[j + k] + cs[i][k] : cs[i][k];
                    s_cols[d + j + k] = g ? s_cols[d + j + k] + cn[i][k] : cn[i][k];
                }
            }
        __syncthreads();
    }
    float *slab = a.part + (long long)blockIdx.x * 2 * d;
    for (int j = threadIdx.x * 4; j < 2 * d; j += blockDim.x * 4)
        *reinterpret_cast<float4 *>(slab + j) = *reinterpret_cast<const float4 *>(s_cols + j);
}

// The slabs' sums, column by column in slab order (eight partial sums, then
// those in order), and the weight gradients they give.
template <typename T>
__global__ void __launch_bounds__(256) block_columns_kernel(const BlockArgs a, int slabs) {
    __shared__ float s[2][8][32];
    griddep_wait();
    griddep_launch_dependents();
    const int c = threadIdx.x & 31, p = threadIdx.x >> 5, j = blockIdx.x * 32 + c;
    float v0 = 0.0f, v1 = 0.0f;
    if (j < a.d)
        for (int b = p; b < slabs; b += 8) {
            const float *q = a.part + (long long)b * 2 * a.d + j;
            v0 += q[0];
            v1 += q[a.d];
        }
    s[0][p][c] = v0;
    s[1][p][c] = v1;
    __syncthreads();
    if (p != 0 || j >= a.d) return;
    v0 = v1 = 0.0f;
    for (int b = 0; b < 8; ++b) {
        v0 += s[0][b][c];
        v1 += s[1][b][c];
    }
    const T *w = static_cast<const T *>(a.w), *gc = static_cast<const T *>(a.gc);
    auto put = [&](float *to, float v) { to[j] = a.accumulate ? to[j] + v : v; };
    if (a.dw) put(a.dw, gc ? to_f(gc[j]) * v0 : v0);
    if (a.dgc) put(a.dgc, w ? to_f(w[j]) * v0 : v0);
    if (a.dwn) put(a.dwn, v1);
}

// --------------------------------------------------------------- launch --
// Warps per row: a row's vectors of eight over its lanes, NV each.
struct Shape {
    int nv, warps, groups, grid;
};

Shape shape_of(const beam_block_desc *d, bool backward) {
    Shape s;
    const int vecs = d->d / 8;
    s.nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
    s.warps = (vecs + 32 * s.nv - 1) / (32 * s.nv);
    s.groups = kMaxWarps / s.warps;
    if (s.groups > 15) s.groups = 15;  // named barriers 1..15
    // rather a row on every SM than several on a few
    const int rows = d->T / kNominalSMs;
    if (s.groups > rows) s.groups = rows > 1 ? rows : 1;
    const long long want = ((long long)d->T + s.groups - 1) / s.groups;
    const int threads = s.groups * s.warps * 32;
    const int per_sm = backward || s.nv > 1 ? 512 / threads : 1024 / threads;
    const long long cap = (long long)kNominalSMs * per_sm;
    s.grid = int(want < cap ? want : cap);
    return s;
}

size_t slab_bytes(const beam_block_desc *d) {
    return d->T == 0 ? 0 : size_t(shape_of(d, true).grid) * 2 * size_t(d->d) * sizeof(float);
}

template <typename T, bool BRANCH>
cudaError_t launch_forward(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    const dim3 grid(s.grid), block(s.groups * s.warps * 32);
    if (s.nv == 1) return launch_pdl(block_forward_kernel<T, 1, BRANCH>, grid, block, 0, st, a, s.warps);
    if (s.nv == 2) return launch_pdl(block_forward_kernel<T, 2, BRANCH>, grid, block, 0, st, a, s.warps);
    return launch_pdl(block_forward_kernel<T, 4, BRANCH>, grid, block, 0, st, a, s.warps);
}

template <typename T, int NV, bool BRANCH>
cudaError_t launch_backward_nv(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    auto kern = block_backward_kernel<T, NV, BRANCH>;
    static std::atomic<unsigned long long> attr_set{0};  // this instantiation only
    cudaError_t e = set_smem_once(kern, kMaxD * 8, attr_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(s.grid), dim3(s.groups * s.warps * 32),
                      a.part ? size_t(a.d) * 8 : 0, st, a, s.warps);
}

template <typename T, bool BRANCH>
cudaError_t launch_backward(const BlockArgs &a, const Shape &s, cudaStream_t st) {
    cudaError_t e = s.nv == 1   ? launch_backward_nv<T, 1, BRANCH>(a, s, st)
                    : s.nv == 2 ? launch_backward_nv<T, 2, BRANCH>(a, s, st)
                                : launch_backward_nv<T, 4, BRANCH>(a, s, st);
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(block_columns_kernel<T>, dim3((a.d + 31) / 32), dim3(256), 0, st, a, s.grid);
}

bool bad16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

beam_status check_block_desc(const beam_block_desc *d) {
    if (!d) return BEAM_ERR_INVALID_ARG;
    if (d->T < 0 || d->d <= 0) return BEAM_ERR_INVALID_ARG;
    if (d->dtype != BEAM_BF16 && d->dtype != BEAM_F32) return BEAM_ERR_INVALID_ARG;
    if (!(d->eps > 0.0f) || !(d->eps < 3.0e38f)) return BEAM_ERR_INVALID_ARG;
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
    return done(desc->dtype == BEAM_BF16 ? launch_backward<__nv_bfloat16, false>(a, sh, st)
                                         : launch_backward<float, false>(a, sh, st));
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
    return done(desc->dtype == BEAM_BF16 ? launch_backward<__nv_bfloat16, true>(a, sh, st)
                                         : launch_backward<float, true>(a, sh, st));
}

}  // extern "C"
