// balance.cu -- the router's balance loss with per-expert counts, and its
// gradient.
//
// The batch is S sequences of tokens, L_s long.  With p_t the softmax of token
// t's main-router logits over all E experts,
//   f_se = E / (K L_s) #{t in s: e is one of t's K candidates}   (or the kept)
//   P_se = 1 / L_s sum_{t in s} p_te
//   loss = coef / S sum_s sum_e f_se P_se
// (1 per sequence where the load is even), and since f only counts,
//   dr_te = dloss coef / (S L_s) p_te (f_se - sum_e' f_se' p_te').
//
// Forward: a CTA takes a chunk of one sequence, a warp a token at a time, lane
// l experts l, l + 32, ...; its probabilities and counts stay in registers
// over its tokens and are added up over the CTA's warps and the chunks in a
// fixed order, so the loss is bitwise repeatable.
#include "beam_internal.h"
#include "beam_ptx.cuh"

namespace beam {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBalWarps = 8;

// Sequence boundaries as given, made safe: inside [0, T] and not decreasing.
struct Span {
    int lo, hi;
    bool bad;
};
__device__ __forceinline__ Span span_of(const BalanceArgs &a, int s) {
    Span r;
    r.lo = a.seq_begin ? a.seq_begin[s] : 0;
    r.hi = a.seq_begin ? a.seq_begin[s + 1] : a.T;
    r.bad = r.lo < 0 || r.hi > a.T || r.lo > r.hi;
    if (r.bad) r.lo = r.hi = 0;
    return r;
}

// Which sequence and chunk of it the v-th chunk of the batch is: sequences
// have ceil(L / C) chunks each.  One warp; false if there are fewer chunks.
// *first: the index of the sequence's first chunk.
__device__ __forceinline__ bool find_chunk(const BalanceArgs &a, int v, int *seq, int *first) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int s0 = 0; s0 < a.S; s0 += 32) {
        int c = 0;
        if (s0 + lane < a.S) {
            const Span sp = span_of(a, s0 + lane);
            c = (sp.hi - sp.lo + a.C - 1) / a.C;
        }
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += u;
        }
        const unsigned past = __ballot_sync(kAll, base + sum > v);
        if (past) {
            const int l = __ffs(past) - 1;
            *seq = s0 + l;
            *first = base + __shfl_sync(kAll, sum - c, l);
            return true;
        }
        base += __shfl_sync(kAll, sum, 31);
    }
    return false;
}

// Larger logit -> larger key; -0 counts as +0, NaN as -infinity; 0 is taken.
__device__ __forceinline__ unsigned key_of(float r) {
    const float v = r == 0.0f ? 0.0f : (r != r) ? -INFINITY : r;
    const unsigned b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <int EPL>
__device__ __forceinline__ float row_max(const float (&r)[EPL]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = fmaxf(m, r[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    return m;
}

// r becomes the softmax of the row.  A row of -infinities has none: zeros.
template <int EPL>
__device__ __forceinline__ void softmax_row(float (&r)[EPL], int E) {
    const int lane = threadIdx.x & 31;
    const float m = row_max(r);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        // NaN logits reach the sum as NaN; fmaxf leaves them out of m
        r[i] = lane + 32 * i < E ? (r[i] == -INFINITY ? 0.0f : expf(r[i] - m)) : 0.0f;
        sum += r[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] *= inv;
}

template <int EPL>
__device__ __forceinline__ void load_row(const float *p, int E, float (&r)[EPL]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] = lane + 32 * i < E ? p[lane + 32 * i] : -INFINITY;
}

template <int EPL>
__global__ void __launch_bounds__(kBalWarps * 32) balance_chunk_kernel(const BalanceArgs a) {
    __shared__ float s_p[kBalWarps][32 * EPL];
    __shared__ int s_c[kMaxE], s_k[kMaxE];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    int seq, first;
    if (!find_chunk(a, blockIdx.x, &seq, &first)) return;  // the same in every warp
    const Span sp = span_of(a, seq);
    const int t0 = sp.lo + (int(blockIdx.x) - first) * a.C, t1 = min(sp.hi, t0 + a.C);
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_c[e] = s_k[e] = 0;
    __syncthreads();
    float acc[EPL];
    int cand[EPL], kept[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        acc[i] = 0.0f;
        cand[i] = kept[i] = 0;
    }
    for (int t = t0 + warp; t < t1; t += kBalWarps) {
        const float *row = a.logits + (long long)t * a.ld;
        float r[EPL];
        load_row(row, E, r);
        unsigned key[EPL], taken = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = lane + 32 * i < E ? key_of(r[i]) : 0u;
        for (int k = 0; k < a.K; ++k) {
            unsigned best = 0u;
            int at = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
            const unsigned top = __reduce_max_sync(kAll, best);
            // of the lanes that hold it, the lowest expert
            const unsigned id =
                __reduce_min_sync(kAll, best == top ? unsigned(lane + 32 * at) : ~0u);
            if (id == unsigned(lane + 32 * at)) {
                taken |= 1u << at;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i == at) key[i] = 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((taken >> i) & 1u) {
                ++cand[i];
                if (a.has_mask && row[E + lane + 32 * i] >= a.thr) ++kept[i];
            }
        softmax_row(r, E);
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] += r[i];
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        s_p[warp][e] = acc[i];
        if (cand[i]) atomicAdd(&s_c[e], cand[i]);
        if (kept[i]) atomicAdd(&s_k[e], kept[i]);
    }
    __syncthreads();
    const long long at = (long long)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) v += s_p[w][e];
        a.part_p[at + e] = v;
        a.part_c[at + e] = s_c[e];
        a.part_k[at + e] = s_k[e];
    }
}

// One CTA per sequence: its chunks in order, its counts, probabilities and
// loss; the last CTA to finish adds the sequences' losses up in order.
__global__ void __launch_bounds__(256) balance_final_kernel(const BalanceArgs a) {
    __shared__ float s_sum[8];
    __shared__ int s_last, s_first;
    griddep_wait();
    griddep_launch_dependents();
    const int s = blockIdx.x, e = threadIdx.x;
    const int lane = e & 31, warp = e >> 5;
    const Span sp = span_of(a, s);
    const int L = sp.hi - sp.lo, chunks = (L + a.C - 1) / a.C;
    if (warp == 0) {  // chunks before this sequence's
        int n = 0;
        for (int q = lane; q < s; q += 32) {
            const Span o = span_of(a, q);
            n += (o.hi - o.lo + a.C - 1) / a.C;
        }
        n = int(__reduce_add_sync(kAll, unsigned(n)));
        if (lane == 0) s_first = n;
    }
    __syncthreads();
    float term = 0.0f;
    if (e < a.E) {
        float p = 0.0f;
        int c = 0, k = 0;
        for (int q = 0; q < chunks && s_first + q < a.chunks; ++q) {
            const long long at = (long long)(s_first + q) * a.E + e;
            p += a.part_p[at];
            c += a.part_c[at];
            k += a.part_k[at];
        }
        const float len = float(L > 0 ? L : 1);
        const long long o = (long long)s * a.E + e;
        a.cand[o] = c;
        if (a.kept) a.kept[o] = k;
        if (a.prob) a.prob[o] = p / len;
        term = float(a.count_kept ? k : c) * float(a.E) / (float(a.K) * len) * (p / len);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kAll, term, o);
    if (lane == 0) s_sum[warp] = term;
    __syncthreads();
    if (e == 0) {
        float v = 0.0f;
        for (int w = 0; w < 8; ++w) v += s_sum[w];
        a.seq_loss[s] = sp.bad ? NAN : v;
        __threadfence();
        s_last = atomicAdd(a.ticket, 1) == a.S - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float v = 0.0f;  // thread e: sequences e, e + 256, ...; then a fixed tree
    for (int q = e; q < a.S; q += 256) v += __ldcg(a.seq_loss + q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    if (lane == 0) s_sum[warp] = v;
    __syncthreads();
    if (e == 0) {
        v = 0.0f;
        for (int w = 0; w < 8; ++w) v += s_sum[w];
        *a.loss = a.coef / float(a.S) * v;
    }
}

// A warp per token.  Tokens outside every sequence get zeros.
template <int EPL>
__global__ void __launch_bounds__(256) balance_grad_kernel(const BalanceArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, E = a.E;
    const int step = int(gridDim.x) * 8;
    const float up = a.coef / float(a.S) * (a.dloss ? *a.dloss : 1.0f);
    for (int t = int(blockIdx.x) * 8 + (threadIdx.x >> 5); t < a.T; t += step) {
        float r[EPL];
        load_row(a.logits + (long long)t * a.ld, E, r);
        // the first sequence that holds t (32 at a time)
        int s = -1;
        bool bad = false;
        for (int s0 = 0; s0 < a.S && s < 0; s0 += 32) {
            bool in = false;
            if (s0 + lane < a.S) {
                const Span sp = span_of(a, s0 + lane);
                in = t >= sp.lo && t < sp.hi;
                bad |= sp.bad;
            }
            const unsigned b = __ballot_sync(kAll, in);
            if (b) s = s0 + __ffs(b) - 1;
        }
        bad = __any_sync(kAll, bad);
        float g = 0.0f, f[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) f[i] = 0.0f;
        if (s >= 0) {
            const Span sp = span_of(a, s);
            const float len = float(sp.hi - sp.lo);
            const float scale = float(E) / (float(a.K) * len);
            const int *c = a.counts + (long long)s * E;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane + 32 * i < E) f[i] = float(c[lane + 32 * i]) * scale;
            g = up / len;
        }
        softmax_row(r, E);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) dot = fmaf(f[i], r[i], dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
        float *out = a.dlogits + (long long)t * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < E)
                out[lane + 32 * i] = bad ? NAN : s < 0 ? 0.0f : g * r[i] * (f[i] - dot);
    }
}

struct Layout {
    int C, chunks;
    size_t off_p, off_c, off_k, off_loss, bytes;
};

Layout layout_of(const beam_balance_desc *d) {
    Layout l;
    // about four CTAs per SM, at least two tokens per warp
    long long c = (d->T + 4ll * kNominalSMs - 1) / (4ll * kNominalSMs);
    c = (c + kBalWarps - 1) / kBalWarps * kBalWarps;
    l.C = int(c < 2 * kBalWarps ? 2 * kBalWarps : c);
    l.chunks = d->T / l.C + (d->n_seq < d->T ? d->n_seq : d->T);  // an unfilled one per sequence
    const size_t n = size_t(l.chunks) * size_t(d->E) * 4;
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    l.off_p = 256;
    l.off_c = up(l.off_p + n);
    l.off_k = up(l.off_c + n);
    l.off_loss = up(l.off_k + n);
    l.bytes = up(l.off_loss + 4 * size_t(d->n_seq));
    return l;
}

beam_status check_balance_desc(const beam_balance_desc *d) {
    if (!d) return BEAM_ERR_INVALID_ARG;
    if (d->T < 0 || d->E <= 0 || d->E > kMaxE || d->K <= 0 || d->K > d->E || d->K > kMaxK)
        return BEAM_ERR_INVALID_ARG;
    if (d->n_seq < 1 || (d->has_mask != 0 && d->has_mask != 1) ||
        (d->count_kept != 0 && d->count_kept != 1) || (d->count_kept && !d->has_mask))
        return BEAM_ERR_INVALID_ARG;
    if (d->logits_ld < (d->has_mask ? 2 * d->E : d->E)) return BEAM_ERR_INVALID_ARG;
    if (d->mask_logit_threshold != d->mask_logit_threshold) return BEAM_ERR_INVALID_ARG;
    if (!(d->coef - d->coef == 0.0f)) return BEAM_ERR_INVALID_ARG;
    // tokens are counted in 32 bits, with room for a grid's step; so are chunks,
    // at most 593 a sequence even where boundaries make sequences overlap
    if (d->T > 0x3fffffff || d->n_seq > (1 << 20)) return BEAM_ERR_UNSUPPORTED_SHAPE;
    return BEAM_OK;
}

bool bad16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

BalanceArgs balance_args(const beam_balance_desc *d) {
    BalanceArgs a = {};
    a.T = d->T;
    a.E = d->E;
    a.K = d->K;
    a.S = d->n_seq;
    a.ld = d->logits_ld;
    a.has_mask = d->has_mask;
    a.count_kept = d->count_kept;
    a.thr = d->mask_logit_threshold;
    a.coef = d->coef;
    return a;
}

template <template <int> class F>
cudaError_t by_experts(int E, const BalanceArgs &a, int grid, cudaStream_t st) {
    if (E <= 32) return F<1>::launch(a, grid, st);
    if (E <= 64) return F<2>::launch(a, grid, st);
    if (E <= 128) return F<4>::launch(a, grid, st);
    return F<8>::launch(a, grid, st);
}
template <int EPL>
struct Chunks {
    static cudaError_t launch(const BalanceArgs &a, int grid, cudaStream_t st) {
        return launch_pdl(balance_chunk_kernel<EPL>, dim3(grid), dim3(kBalWarps * 32), 0, st, a);
    }
};
template <int EPL>
struct Grad {
    static cudaError_t launch(const BalanceArgs &a, int grid, cudaStream_t st) {
        return launch_pdl(balance_grad_kernel<EPL>, dim3(grid), dim3(256), 0, st, a);
    }
};

}  // namespace
}  // namespace beam

using namespace beam;

extern "C" {

size_t beam_moe_balance_workspace_size(const beam_balance_desc *desc) {
    return check_balance_desc(desc) == BEAM_OK ? layout_of(desc).bytes : 0;
}

beam_status beam_moe_balance(const beam_balance_desc *desc, const float *logits,
                             const int32_t *seq_begin, float *loss, int32_t *cand_counts,
                             int32_t *kept_counts, float *mean_prob, void *workspace,
                             size_t workspace_bytes, void *stream) {
    beam_status s = check_balance_desc(desc);
    if (s != BEAM_OK) return s;
    if ((!logits && desc->T > 0) || !loss || !cand_counts || (!seq_begin && desc->n_seq != 1) ||
        (kept_counts && !desc->has_mask))
        return BEAM_ERR_INVALID_ARG;
    for (const void *p :
         {static_cast<const void *>(logits), static_cast<const void *>(seq_begin),
          static_cast<const void *>(loss), static_cast<const void *>(cand_counts),
          static_cast<const void *>(kept_counts), static_cast<const void *>(mean_prob)})
        if (bad16(p)) return BEAM_ERR_INVALID_ARG;
    const Layout l = layout_of(desc);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < l.bytes)
        return BEAM_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    BalanceArgs a = balance_args(desc);
    a.C = l.C;
    a.chunks = l.chunks;
    a.logits = logits;
    a.seq_begin = seq_begin;
    a.ticket = reinterpret_cast<int *>(ws);
    a.part_p = reinterpret_cast<float *>(ws + l.off_p);
    a.part_c = reinterpret_cast<int *>(ws + l.off_c);
    a.part_k = reinterpret_cast<int *>(ws + l.off_k);
    a.seq_loss = reinterpret_cast<float *>(ws + l.off_loss);
    a.loss = loss;
    a.cand = cand_counts;
    a.kept = kept_counts;
    a.prob = mean_prob;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = by_experts<Chunks>(desc->E, a, l.chunks > 0 ? l.chunks : 1, st);
    if (e == cudaSuccess) e = launch_pdl(balance_final_kernel, dim3(desc->n_seq), dim3(256), 0, st, a);
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

beam_status beam_moe_balance_backward(const beam_balance_desc *desc, const float *logits,
                                      const int32_t *seq_begin, const int32_t *counts,
                                      const float *dloss, float *dlogits, void *stream) {
    beam_status s = check_balance_desc(desc);
    if (s != BEAM_OK) return s;
    if (!counts || (!seq_begin && desc->n_seq != 1)) return BEAM_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(logits), static_cast<const void *>(seq_begin),
                          static_cast<const void *>(counts), static_cast<const void *>(dloss),
                          static_cast<const void *>(dlogits)})
        if (bad16(p)) return BEAM_ERR_INVALID_ARG;
    if (desc->T == 0) return BEAM_OK;
    if (!logits || !dlogits) return BEAM_ERR_INVALID_ARG;
    BalanceArgs a = balance_args(desc);
    a.logits = logits;
    a.seq_begin = seq_begin;
    a.counts = counts;
    a.dloss = dloss;
    a.dlogits = dlogits;
    const long long blocks = (desc->T + 7ll) / 8, cap = 8ll * device_sm_count();
    const cudaError_t e = by_experts<Grad>(desc->E, a, int(blocks < cap ? blocks : cap),
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

}  // extern "C"
