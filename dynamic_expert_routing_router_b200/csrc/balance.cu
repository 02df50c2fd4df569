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
// Forward: CTA v takes the tokens [v C, (v + 1) C) and adds up, per sequence
// that begins, ends or runs there, its probabilities and counts: part v + s of
// sequence s (one part per chunk or sequence begun, so no two share an index).
// A warp takes a token at a time, lane l experts l, l + 32, ..., the next
// token's logits being loaded meanwhile; a second launch adds the parts up.
// Every sum runs in a fixed order, in 32 bits: the loss is bitwise repeatable,
// and P is off by at most 2^-24 of itself for each term added in a row: T / 3552
// in a warp, 8 warps, up to 600 chunks (up to 10^8 tokens; 32768 in a warp and
// 4096 chunks at most).
//
// Bound by instructions: about 515 a token of 256 experts, half of them for the
// 8 largest, against 1 KB of logits and a 32-byte sector of mask logits for each
// candidate.  32768 such tokens with a mask take 28.5 us (1.5 TB/s), the second
// launch 5 of them; the gradient of 17937 x 239, about 400 instructions a token,
// 10.3 us (3.3 TB/s).
#include <cooperative_groups.h>

#include "beam_internal.h"
#include "beam_ptx.cuh"

namespace beam {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBalWarps = 8;
// One sequence of so many tokens goes to one cluster, up to eight CTAs of 32
// tokens.  A pass with K = 8 there against the two launches: 64 x 128 4.5 / 6.5
// us, 256 x 256 7.4 / 7.5.  Several sequences would take their turns there, a
// cluster barrier each: two of 64 x 128 7.6 / 6.4 us, of 256 x 128 11.2 / 6.3,
// four 13.0 / 6.5 and 20.3 / 6.6.
constexpr int kSmallTokens = 256;
constexpr int kMaxChunk = 1 << 18;  // tokens: a warp's counts fit 16 bits

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

// The first sequence that ends behind token t (S if none does), by one warp:
// each step leaves one of 32 parts of the boundaries.
__device__ __forceinline__ int first_ending_after(const BalanceArgs &a, int t) {
    if (!a.seq_begin) return t < a.T ? 0 : 1;
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.S;  // it is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
        const unsigned past = __ballot_sync(kAll, at >= hi || a.seq_begin[at + 1] > t);
        if (!past) return hi;  // not even the last one
        const int l = __ffs(past) - 1;
        hi = min(hi, lo + (l + 1) * step - 1);
        lo += l * step;
    }
    return lo;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <int EPL>
__device__ __forceinline__ void load_row(const float *p, int E, float (&r)[EPL]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] = lane + 32 * i < E ? __ldcs(p + lane + 32 * i) : -INFINITY;
}

// r, whose largest value (NaN left out) is m, becomes the softmax of the row
// but for the factor that is returned.  A row of -infinities has none: zeros.
// NaN logits reach the sum as NaN.
template <int EPL>
__device__ __forceinline__ float softmax_row(float (&r)[EPL], float m) {
    float sum = 0.0f;
    if (m == -INFINITY) m = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        r[i] = expf(r[i] - m);
        sum += r[i];
    }
    sum = warp_sum(sum);
    return sum == 0.0f ? 0.0f : 1.0f / sum;
}

// Which of the row's values are its K largest (ties to the lower id, NaN as
// -infinity): those >= the value returned, or in *ties, where that would be
// too many, bit i for expert lane + 32 i.  *m is the largest.  Each lane sorts
// its values; then the largest heads are taken off, all that are equal at
// once, until K are: the last one is the K-th largest.
template <int EPL>
__device__ __forceinline__ float kth_largest(const float (&r)[EPL], int E, int K, float *m,
                                             unsigned *ties) {
    const int lane = threadIdx.x & 31;
    float h[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) h[i] = fmaxf(r[i], -INFINITY);
    // odd-even merge sort, descending
#pragma unroll
    for (int p = 1; p < EPL; p <<= 1)
#pragma unroll
        for (int k = p; k > 0; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < EPL; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < EPL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const float x = h[i + j], y = h[i + j + k];
                        h[i + j] = fmaxf(x, y);
                        h[i + j + k] = fminf(x, y);
                    }
    // After k rounds a lane can give K - k more: only so many are kept sorted.
    float kth = warp_max(h[0]);
    *m = kth;
    int got = 0;
    bool done = false;
    auto take = [&](int keep) {  // the heads equal to kth, and the next kth
        const bool mine = h[0] == kth;
        got += __popc(__ballot_sync(kAll, mine));
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i < keep) h[i] = mine ? (i + 1 < EPL ? h[i + 1 < EPL ? i + 1 : 0] : -INFINITY) : h[i];
        const float next = warp_max(h[0]);
        if (got < K) {
            kth = next;
            return false;
        }
        // Exactly K reach the K-th.  (Equal values of one lane come off one
        // by one, so one may be left.)
        done = got == K && next != kth && kth != -INFINITY;
        return true;
    };
    if (K <= EPL) {
#pragma unroll
        for (int k = 0; k < EPL; ++k)
            if (take(EPL - k)) break;
    } else {
        while (!take(EPL)) {
        }
    }
    *ties = 0u;
    if (done) return kth;
    // Ties: those above, then the lowest ids of the equal ones.
    int left = K;
    unsigned taken = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) left -= __popc(__ballot_sync(kAll, r[i] > kth));
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const bool tie = lane + 32 * i < E && fmaxf(r[i], -INFINITY) == kth;
        const unsigned b = __ballot_sync(kAll, tie);
        const int before = __popc(b & ((1u << lane) - 1u));
        if (r[i] > kth || (tie && before < left)) taken |= 1u << i;
        left -= min(left, __popc(b));
    }
    *ties = taken;
    return NAN;  // nothing reaches it
}

// The warp's tokens t, t + kBalWarps, ... below hi: its probabilities, and its
// counts of candidates and, above bit 16, of kept ones, are added up.  r:
// token t's logits where `loaded`.
template <int EPL>
__device__ __forceinline__ void add_tokens(const BalanceArgs &a, bool mask, int t, int hi,
                                           float (&r)[EPL], bool loaded, float (&acc)[EPL],
                                           unsigned (&count)[EPL]) {
    const int lane = threadIdx.x & 31, E = a.E;
    float next[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        acc[i] = 0.0f;
        count[i] = 0u;
    }
    if (t < hi && !loaded) load_row(a.logits + (long long)t * a.ld, E, r);
    for (; t < hi; t += kBalWarps) {
        const float *row = a.logits + (long long)t * a.ld;
        if (t + kBalWarps < hi) load_row(row + (long long)kBalWarps * a.ld, E, next);
        float m;
        unsigned taken;
        const float kth = kth_largest(r, E, a.K, &m, &taken);
        // the mask's logits of the candidates alone; they arrive meanwhile
        float z[EPL];
        if (kth == kth) {
            taken = 0u;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (r[i] >= kth) taken |= 1u << i;
        }
        if (mask) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if ((taken >> i) & 1u) z[i] = __ldcs(row + E + lane + 32 * i);
        }
        const float inv = softmax_row(r, m);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            acc[i] = fmaf(r[i], inv, acc[i]);
            if ((taken >> i) & 1u) count[i] += mask && z[i] >= a.thr ? 0x10001u : 1u;
            r[i] = next[i];
        }
    }
}

// The CTA's warps' sums of expert e, in order.
template <int EPL>
struct WarpSums {
    float p[kBalWarps][32 * EPL];
    unsigned c[kBalWarps][32 * EPL];
    __device__ void put(const float (&acc)[EPL], const unsigned (&count)[EPL]) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[warp][lane + 32 * i] = acc[i];
            c[warp][lane + 32 * i] = count[i];
        }
    }
    __device__ void add(int e, float *v, int *cand, int *kept) const {
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) {
            *v += p[w][e];
            *cand += c[w][e] & 0xffffu;
            *kept += c[w][e] >> 16;
        }
    }
};

template <int EPL>
__global__ void __launch_bounds__(kBalWarps * 32, EPL <= 4 ? 4 : 3)
    balance_chunk_kernel(const BalanceArgs a) {
    __shared__ WarpSums<EPL> sums;
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, E = a.E;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    const int t0 = blockIdx.x * a.C, t1 = min(a.T, t0 + a.C);
    const bool mask = a.has_mask && (a.kept || a.count_kept);
    float r[EPL];  // the first token's logits come while the sequence is looked up
    if (t0 + warp < t1) load_row(a.logits + (long long)(t0 + warp) * a.ld, E, r);
    for (int s = first_ending_after(a, t0), first = t0; s < a.S; ++s) {
        const Span sp = span_of(a, s);
        if (sp.lo >= t1 && !sp.bad) break;
        const int lo = max(sp.lo, t0), hi = min(sp.hi, t1);
        if (lo >= hi) continue;
        float acc[EPL];
        unsigned count[EPL];
        add_tokens(a, mask, lo + warp, hi, r, lo == first, acc, count);
        first = -1;
        __syncthreads();  // the previous sequence's sums are out
        sums.put(acc, count);
        __syncthreads();
        const long long at = ((long long)blockIdx.x + s) * E;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float v = 0.0f;
            int c = 0, k = 0;
            sums.add(e, &v, &c, &k);
            a.part_p[at + e] = v;
            a.part_c[at + e] = c;
            if (mask) a.part_k[at + e] = k;
        }
    }
}

// Expert e of sequence s: what is written, and its term of the loss.
__device__ __forceinline__ float finish_expert(const BalanceArgs &a, int s, int e, const Span &sp,
                                               float p, int c, int k) {
    const float len = float(sp.hi > sp.lo ? sp.hi - sp.lo : 1);
    const long long o = (long long)s * a.E + e;
    a.cand[o] = c;
    if (a.kept) a.kept[o] = k;
    if (a.prob) a.prob[o] = p / len;
    return float(a.count_kept ? k : c) * float(a.E) / (float(a.K) * len) * (p / len);
}

// A small batch of one sequence in one launch: one cluster, CTA r takes the
// tokens [r C, (r + 1) C), and adds up the experts r, r + CTAs, ... of all CTAs
// through their shared memory.  128 tokens of 128 experts take 4.5 to 5.1 us on
// the GPU, by how the logits lie, and 5.0 to 5.4 a pass; two launches 6.0 and 6.5.
template <int EPL>
__global__ void __launch_bounds__(kBalWarps * 32) balance_small_kernel(const BalanceArgs a) {
    namespace cg = cooperative_groups;
    __shared__ WarpSums<EPL> sums;
    struct Part {
        float p[32 * EPL];
        int c[32 * EPL], k[32 * EPL];
    };
    __shared__ Part mine;
    __shared__ float s_terms[8];  // of rank 0: the CTAs' terms
    cg::cluster_group cluster = cg::this_cluster();
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int t0 = rank * a.C, t1 = min(a.T, t0 + a.C);
    const bool mask = a.has_mask && (a.kept || a.count_kept);
    float r[EPL];  // the first token's logits come while the boundaries do
    if (t0 + warp < t1) load_row(a.logits + (long long)(t0 + warp) * a.ld, a.E, r);
    const Span sp = span_of(a, 0);
    const int lo = max(sp.lo, t0);
    float acc[EPL];
    unsigned count[EPL];
    add_tokens(a, mask, lo + warp, min(sp.hi, t1), r, lo == t0, acc, count);
    sums.put(acc, count);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float v = 0.0f;
        int c = 0, k = 0;
        sums.add(e, &v, &c, &k);
        mine.p[e] = v;
        mine.c[e] = c;
        mine.k[e] = k;
    }
    cluster.sync();
    float term = 0.0f;  // of this thread's experts
    for (int e = rank + int(threadIdx.x) * ctas; e < a.E; e += blockDim.x * ctas) {
        float v = 0.0f;
        int c = 0, k = 0;
        for (int q = 0; q < ctas; ++q) {
            const Part *from = cluster.map_shared_rank(&mine, q);
            v += from->p[e];
            c += from->c[e];
            k += from->k[e];
        }
        term += finish_expert(a, 0, e, sp, v, c, k);
    }
    // the CTAs' terms, in order
    term = warp_sum(term);
    __syncthreads();
    if (lane == 0) sums.p[warp][0] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
        term = 0.0f;
        for (int w = 0; w < kBalWarps; ++w) term += sums.p[w][0];
        *cluster.map_shared_rank(&s_terms[rank], 0) = term;
    }
    cluster.sync();  // and nobody's part is read any more
    if (rank == 0 && threadIdx.x == 0) {
        float v = 0.0f;
        for (int r = 0; r < ctas; ++r) v += s_terms[r];
        *a.loss = sp.bad ? NAN : a.coef * v;
    }
}

// CTA (s, j): sequence s, experts [32 j, 32 j + 32); warp w adds up parts w, w
// + warps, ..., then warp 0 the warps' sums in order.  The last CTA to finish
// adds the losses of all in order.
__global__ void __launch_bounds__(1024) balance_final_kernel(const BalanceArgs a) {
    __shared__ float s_p[32][32];
    __shared__ int s_c[32][32], s_k[32][32];
    __shared__ int s_last;
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5, e = blockIdx.y * 32 + lane;
    // The boundaries are older than the chunk kernel, which lets this one start
    // only after its own wait: they may be read before this one's.
    const Span sp = span_of(a, s);
    griddep_wait();
    griddep_launch_dependents();
    const bool mask = a.has_mask && (a.kept || a.count_kept);
    float p = 0.0f;
    int c = 0, k = 0;
    if (e < a.E && sp.hi > sp.lo) {
        const int last = (sp.hi - 1) / a.C;
#pragma unroll 4
        for (int v = sp.lo / a.C + warp; v <= last; v += warps) {
            const long long at = ((long long)v + s) * a.E + e;
            p += a.part_p[at];
            c += a.part_c[at];
            if (mask) k += a.part_k[at];
        }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    s_k[warp][lane] = k;
    __syncthreads();
    if (warp == 0) {
        float term = 0.0f;
        if (e < a.E) {
            for (int w = 1; w < warps; ++w) {
                p += s_p[w][lane];
                c += s_c[w][lane];
                k += s_k[w][lane];
            }
            term = finish_expert(a, s, e, sp, p, c, k);
        }
        term = warp_sum(term);
        if (lane == 0) {
            const int n = gridDim.x * gridDim.y;
            a.seq_loss[s * gridDim.y + blockIdx.y] = sp.bad ? NAN : term;
            __threadfence();
            s_last = atomicAdd(a.ticket, 1) == n - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const int n = gridDim.x * gridDim.y;
    float v = 0.0f;  // thread i: terms i, i + threads, ...; then a fixed tree
    for (int q = threadIdx.x; q < n; q += blockDim.x) v += __ldcg(a.seq_loss + q);
    v = warp_sum(v);
    if (lane == 0) s_p[0][warp] = v;
    __syncthreads();
    if (warp == 0) {
        v = warp_sum(lane < warps ? s_p[0][lane] : 0.0f);
        if (lane == 0) *a.loss = a.coef / float(a.S) * v;
    }
}

// A warp takes a run of tokens, and its sequence's f once per sequence.
// Tokens outside every sequence get zeros.
template <int EPL>
__global__ void __launch_bounds__(256) balance_grad_kernel(const BalanceArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, E = a.E;
    const int t0 = (int(blockIdx.x) * 8 + int(threadIdx.x >> 5)) * a.C, t1 = min(a.T, t0 + a.C);
    if (t0 >= t1) return;
    const float up = a.coef / float(a.S) * (a.dloss ? *a.dloss : 1.0f);
    float next[EPL], f[EPL];
    load_row(a.logits + (long long)t0 * a.ld, E, next);
    int s = first_ending_after(a, t0), ends = t0;  // f is of the tokens before `ends`
    float g = 0.0f;
    for (int t = t0; t < t1; ++t) {
        if (t >= ends) {
            Span sp = {t, t1, false};  // behind the last sequence: none
            for (; s < a.S; ++s) {
                sp = span_of(a, s);
                if (sp.hi > t) break;
                sp.lo = t;
                sp.hi = t1;
            }
            const bool in = s < a.S && sp.lo <= t;
            ends = in || s >= a.S ? sp.hi : sp.lo;
            const float len = float(sp.hi - sp.lo);
            const float scale = float(E) / (float(a.K) * len);
            g = in ? up / len : 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                f[i] = in && lane + 32 * i < E
                           ? float(a.counts[(long long)s * E + lane + 32 * i]) * scale
                           : 0.0f;
        }
        float r[EPL], m = -INFINITY, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            r[i] = next[i];
            m = fmaxf(m, r[i]);
        }
        if (t + 1 < t1) load_row(a.logits + (long long)(t + 1) * a.ld, E, next);
        const float inv = softmax_row(r, warp_max(m));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            r[i] *= inv;
            dot = fmaf(f[i], r[i], dot);
        }
        dot = warp_sum(dot);
        // The probabilities add up to 1, so f may be taken less any f0: f - f0 -
        // <f - f0, p>.  With <f, p> as it came out for f0, its own error cancels,
        // and digits are left where one expert has nearly all of the probability
        // or f is the same everywhere.
        float rest = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) rest = fmaf(f[i] - dot, r[i], rest);
        rest = warp_sum(rest);
        float *out = a.dlogits + (long long)t * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < E)
                out[lane + 32 * i] = g == 0.0f ? 0.0f : g * r[i] * (f[i] - dot - rest);
    }
}

struct Layout {
    int C, chunks, slabs;
    size_t off_p, off_c, off_k, off_loss, bytes;
};

Layout layout_of(const beam_balance_desc *d) {
    Layout l;
    // one wave of CTAs (chunks of whole rounds of warps left a third of the SMs
    // a CTA short: 30.2 us for 28.5)
    const long long ctas = (d->E > 128 ? 3ll : 4ll) * kNominalSMs;
    long long c = (d->T + ctas - 1) / ctas;
    l.C = int(c < kBalWarps ? kBalWarps : c > kMaxChunk ? kMaxChunk : c);
    l.chunks = int((d->T + (long long)l.C - 1) / l.C);
    l.slabs = (d->E + 31) / 32;
    const size_t n = (size_t(l.chunks) + size_t(d->n_seq)) * size_t(d->E) * 4;
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    l.off_p = 256;
    l.off_c = up(l.off_p + n);
    l.off_k = up(l.off_c + n);
    l.off_loss = up(l.off_k + (d->has_mask ? n : 0));
    l.bytes = up(l.off_loss + 4 * size_t(d->n_seq) * size_t(l.slabs));
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
    // tokens and a chunk's end are counted in 32 bits
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
struct Small {
    static cudaError_t launch(const BalanceArgs &a, int grid, cudaStream_t st) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kBalWarps * 32);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = grid;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, balance_small_kernel<EPL>, a);
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
    if (desc->T <= kSmallTokens && desc->n_seq == 1) {
        const int ctas = desc->T <= 16 ? 1 : desc->T <= 32 ? 2 : desc->T <= 64 ? 4 : 8;
        a.C = (desc->T + ctas - 1) / ctas;
        return by_experts<Small>(desc->E, a, ctas, st) == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
    }
    cudaError_t e = by_experts<Chunks>(desc->E, a, l.chunks > 0 ? l.chunks : 1, st);
    // warps: the parts of a sequence of mean length, 8 to 32 (the longest one,
    // often several times the mean, sets the time: a quarter of them, 2 us more)
    int warps = 8;
    while (warps < 32 && (long long)warps * desc->n_seq < l.chunks) warps *= 2;
    if (e == cudaSuccess)
        e = launch_pdl(balance_final_kernel, dim3(desc->n_seq, l.slabs), dim3(32 * warps), 0, st, a);
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
    // a run of tokens per warp, eight CTAs per SM where there are as many
    const long long warps = 64ll * device_sm_count();
    a.C = int((desc->T + warps - 1) / warps);
    const long long runs = (desc->T + (long long)a.C - 1) / a.C;
    const cudaError_t e = by_experts<Grad>(desc->E, a, int((runs + 7) / 8),
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

}  // extern "C"
