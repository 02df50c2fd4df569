// mx4.cu -- microscaled 4-bit floating point (MXFP4): rows to 4 bits and back,
// and the grouped expert product of two such matrices.
//
// The format (OCP Microscaling v1.0): 32 consecutive values of a row share one
// power of two 2^X, X = floor(log2 max|v|) - 2, kept as the byte X + 127; each
// value is v / 2^X rounded to nearest-even on the grid +-{0, .5, 1, 1.5, 2, 3,
// 4, 6} (E2M1), larger magnitudes saturating at 6.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "beam_internal.h"
#include "beam_ptx.cuh"

namespace beam {
namespace {

// ------------------------------------------------------------- quantise --
// Four lanes share a block of 32 values, eight each: a warp reads 512
// contiguous bytes of bf16 per load and writes 128 of codes.  Scaling by 2^-X
// is exact, so each value is rounded once, by the conversion.  Bound by
// memory: kMxAhead loads of a thread are under way at a time, a CTA's side by
// side.  98304 x 2048 bf16: 79 us, 6.4 TB/s; read back 79.  With the scales in
// tiles 105: the divisions for their place make it 90 M instructions for 56 M.

constexpr int kMxAhead = 4, kMxAheadBack = 8;

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ float2 two(int i) const {
        const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    // The largest magnitude's bits as those of a float; NaN above infinity.
    __device__ uint32_t top() const {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(r.x & kAbs, r.y & kAbs), __vmaxu2(r.z & kAbs, r.w & kAbs));
        return max(m >> 16, m & 0xffffu) << 16;
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ float2 two(int i) const {
        const float4 &q = i < 2 ? a : b;
        return (i & 1) ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
    }
    __device__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = two(i);
            m = max(m, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu));
        }
        return m;
    }
};

// Two values to E2M1 (round to nearest even, saturating): lo in bits 0-3.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Byte of the scale of (row, block) in the tiled layout the product reads:
// tiles of 128 rows x 4 blocks of 512 bytes, row r of a tile at 16 (r % 32) +
// 4 (r / 32), its four blocks side by side.
__device__ __forceinline__ long long tiled_at(long long row, int block, int blocks) {
    const int r = int(row & 127);
    return ((row >> 7) * (blocks >> 2) + (block >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 +
           (block & 3);
}
// The same of the b-th block of a matrix; 64-bit divisions only where needed.
__device__ __forceinline__ long long tiled_at(long long b, int blocks) {
    if (b >> 32) return tiled_at(b / blocks, int(b % blocks), blocks);
    const uint32_t row = uint32_t(b) / uint32_t(blocks);
    return tiled_at((long long)row, int(uint32_t(b) - row * uint32_t(blocks)), blocks);
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const T *x, long long rows, int cols,
                                                           const int *n_rows, uint32_t *codes,
                                                           uint8_t *scales, int tiled) {
    griddep_wait();
    griddep_launch_dependents();
    if (n_rows) {
        const long long n = *n_rows;
        rows = n < 0 ? 0 : n < rows ? n : rows;
    }
    const long long total = rows * (cols >> 3);  // eights; a block's four never split
    const int blocks = cols >> 5;
    constexpr int step = 256;
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    for (long long i0 = (long long)blockIdx.x * (kMxAhead * step) + threadIdx.x; i0 < total;
         i0 += (long long)gridDim.x * (kMxAhead * step)) {
        Eight<T> v[kMxAhead];
#pragma unroll
        for (int q = 0; q < kMxAhead; ++q)
            if (i0 + q * step < total) v[q].load(x + (i0 + q * step) * 8);
#pragma unroll
        for (int q = 0; q < kMxAhead; ++q) {
            const long long i = i0 + q * step;
            if (i >= total) break;
            uint32_t m = v[q].top();
            m = max(m, __shfl_xor_sync(quad, m, 1));
            m = max(m, __shfl_xor_sync(quad, m, 2));
            const int field = int(m >> 23);  // exponent + 127 of the largest; 0: subnormal or zero
            const bool bad = field == 255;   // infinity or NaN: the whole block stands for NaN
            const int s = field > 2 ? field - 2 : 0;
            const float inv = __uint_as_float(uint32_t(254 - s) << 23);  // 2^-X
            uint32_t out = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = __fmul2_rn(v[q].two(j), make_float2(inv, inv));
                out |= to_e2m1x2(u.x, u.y) << (8 * j);
            }
            codes[i] = bad ? 0u : out;
            if ((threadIdx.x & 3) == 0) {
                const long long b = i >> 2;
                long long at = b;
                if (tiled) at = tiled_at(b, blocks);
                scales[at] = bad ? 255 : uint8_t(s);
            }
        }
    }
}

// ----------------------------------------------------------- read back --

// Two E2M1 values (bits 0-3 and 4-7) as floats; a half holds each exactly.
__device__ __forceinline__ float2 from_e2m1x2(uint32_t c) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.u8.u32 b, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h)
        : "r"(c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 16 bytes of output a lane and store: eight bf16 from 32 bits of codes, or
// four fp32 from 16.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    using Code = uint32_t;
    static __device__ void store(__nv_bfloat16 *p, uint32_t c, float f) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = __fmul2_rn(from_e2m1x2(c >> (8 * i)), make_float2(f, f));
            h[i] = __floats2bfloat162_rn(u.x, u.y);
        }
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
    }
};
template <>
struct Piece<float> {
    using Code = uint16_t;
    static __device__ void store(float *p, uint32_t c, float f) {
        const float2 u = __fmul2_rn(from_e2m1x2(c), make_float2(f, f));
        const float2 v = __fmul2_rn(from_e2m1x2(c >> 8), make_float2(f, f));
        *reinterpret_cast<float4 *>(p) = make_float4(u.x, u.y, v.x, v.y);
    }
};

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t *codes,
                                                             const uint8_t *scales,
                                                             long long rows, int cols, int tiled,
                                                             T *out) {
    using Code = typename Piece<T>::Code;
    constexpr int kValues = 2 * int(sizeof(Code)), kPerBlock = 32 / kValues;
    constexpr int kAhead = kMxAheadBack;
    griddep_wait();
    griddep_launch_dependents();
    const long long total = rows * (cols / kValues);
    const int blocks = cols >> 5;
    constexpr int step = 256;
    const Code *in = reinterpret_cast<const Code *>(codes);
    for (long long i0 = (long long)blockIdx.x * (kAhead * step) + threadIdx.x; i0 < total;
         i0 += (long long)gridDim.x * (kAhead * step)) {
        uint32_t c[kAhead], s[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const long long i = i0 + q * step;
            if (i >= total) break;
            c[q] = in[i];
            const long long b = i / kPerBlock;
            s[q] = scales[tiled ? tiled_at(b, blocks) : b];
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const long long i = i0 + q * step;
            if (i >= total) break;
            // 2^(s - 127); s = 0 is the subnormal 2^-127, s = 255 stands for NaN
            const float f = s[q] == 0 ? __uint_as_float(0x00400000u)
                                      : __uint_as_float(s[q] == 255u ? 0x7fc00000u : s[q] << 23);
            Piece<T>::store(out + i * kValues, c[q], f);
        }
    }
}

// -------------------------------------------------------------- product --
// out[i, :] = a_i . w_e^T for the rows i of expert e (rows grouped by expert,
// counts on the device), or SiLU(a_i . w_e^T) * (a_i . w3_e^T).
//
// tcgen05.mma kind::mxf4 takes both 4-bit operands and their scales as they
// are.  The weight rows are the MMA's M (128 per tile), the token rows its N
// (16..BN, following the tile's valid rows), so a decode batch, bound by the
// weights' bytes, wastes no tile on tokens it lacks.
//
// One persistent CTA per SM; unit = (token tile, 128 weight rows).  (Halves of a
// unit would even out the last round of a decode batch, but a stage costs its
// issue whatever its size: gate and up of 313 units, k = 2048, took 22.3 us in
// halves, 19.9 whole.)  Warps:
//   0      TMA of both code tiles (128 bytes = 256 values a row and stage) and
//          bulk copies of the weight scales, which lie in memory as tiled_at
//   1      TMEM owner and issuer: copies a stage's scales to TMEM
//          (tcgen05.cp, in order with the MMAs of the same thread), 4 MMAs
//   2..9   epilogue: a lane quadrant of TMEM each, two warps per quadrant that
//          take its columns by eights in turn
//   10..17 the token rows' scales: they start at any row, so these warps load
//          them row by row and lay them out in the stage, each for stages of
//          its own, the next one's loads under way: one warp alone had every
//          unit wait for several trips to memory.  (A warp has to see every
//          phase of a stage it fills, since a wait tells only odd from even.)
// Every wait is bounded; on expiry the CTA's status word says so.
//
// Decode is bound by the weights' bytes (gate and up of 154 rows, 128 experts
// of 768 x 2048: 19.8 us, 4.4 TB/s), prefill by what the SMs load from L2 and
// by the output (65536 rows, 2048 x 768, fp32 out: 111 us, 6.0 TB/s; under the
// power cap of a long run 137; gate and up of 65536 rows, 768 x 2048, bf16 out:
// 151 us, for which 1.4 GB go from L2 to the SMs).

constexpr int kMxWarps = 18;
constexpr int kMxThreads = 32 * kMxWarps;
constexpr int kMxScaleWarp = 10, kMxScaleWarps = 8;
constexpr int kMxStepK = 256;             // values per stage: one 128-byte row
constexpr uint32_t kMxSfCols = 64;        // TMEM columns of scales, behind the accumulators
constexpr uint32_t kMxTmemCols = 512;
constexpr uint32_t kMxSfChunk = 512;      // bytes of one 128 x 4 tile of scales

template <int NUM_A, int BN>
struct MxCfg {
    static constexpr uint32_t A_BYTES = 128 * 128;
    static constexpr uint32_t B_SF_TILES = (BN + 127) / 128;  // per 4 blocks of k
    // token rows per TMA box: a tile's boxes behind its last row stay out
    static constexpr uint32_t BOX = BN <= 64 ? BN : BN == 112 ? 56 : 64;
    static constexpr uint32_t SFA_BYTES = 2 * kMxSfChunk;
    static constexpr uint32_t OFF_B = NUM_A * A_BYTES;
    static constexpr uint32_t OFF_SFA = OFF_B + BN * 128;
    static constexpr uint32_t OFF_SFB = OFF_SFA + NUM_A * SFA_BYTES;
    static constexpr uint32_t STAGE_BYTES =
        (OFF_SFB + 2 * kMxSfChunk * B_SF_TILES + 1023) / 1024 * 1024;
    static constexpr int STAGES_FIT = int(220u * 1024u / STAGE_BYTES);
    static constexpr int STAGES = STAGES_FIT > 10 ? 10 : STAGES_FIT;
    static constexpr uint32_t SMEM_BYTES = STAGES * STAGE_BYTES + 1024;
    static constexpr uint32_t ACC_COLS = NUM_A * BN;
    static constexpr uint32_t ACC_BUFS = 2 * ACC_COLS <= kMxTmemCols - kMxSfCols ? 2 : 1;
    // scales of one stage in TMEM, two stages in turn
    static constexpr uint32_t SF_COLS = 2 * 4 * (NUM_A + B_SF_TILES);
    static_assert(ACC_BUFS * ACC_COLS <= kMxTmemCols - kMxSfCols, "accumulators and scales share TMEM");
    static_assert(2 * SF_COLS <= kMxSfCols, "scales in TMEM");
    static_assert(BN % 16 == 0 && BN >= 16 && BN <= 256, "MMA N");
    static_assert(BN % BOX == 0 && BOX % 8 == 0, "boxes of whole swizzle atoms");
    static_assert(STAGES >= 2 && SMEM_BYTES <= 227u * 1024u - 4096u, "shared memory");
};

// A role's place in the ring of stages, and which of its phases comes.
template <int N>
struct MxRing {
    int s = 0;
    uint32_t phase = 0u;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            phase ^= 1u;
        }
    }
};

// Instruction descriptor of kind::mxf4: A and B E2M1 (1) at [7,10) and
// [10,12), N >> 3 at [17,23), scales UE8M0 (1) at 23, M >> 7 at [27,29), the
// scale bytes' ids of B at [4,6) and of A at [29,31); both operands K-major,
// K = 64.
__device__ __forceinline__ uint32_t mxf4_idesc(int n, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (1u << 23) |
           (1u << 27) | (sf_id << 29);
}

// The issuing warps run converged, so that addresses and descriptors stay in
// uniform registers; `one` is set in the lane that issues.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void umma_mxf4(uint32_t one, uint32_t tmem_d, uint64_t adesc,
                                          uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)
        : "memory");
}

// One 512-byte tile of scales (32 rows of 16 bytes, no swizzle: 8-row groups
// of 128 bytes) to four TMEM columns, the same in all four lane quadrants.
__device__ __forceinline__ void tmem_cp_scales(uint32_t one, uint32_t taddr, uint32_t smem_addr) {
    uint64_t desc = 0;
    desc |= uint64_t((smem_addr & 0x3FFFFu) >> 4);
    desc |= uint64_t(128u >> 4) << 32;
    desc |= uint64_t(1u) << 46;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc), "r"(one)
        : "memory");
}

__device__ __forceinline__ void umma_commit_by(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(one)
        : "memory");
}

__device__ __forceinline__ void bulk_load(void *smem_dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(smem_dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

struct MxUnit {
    int e, mb;      // expert, block of 128 weight rows
    int row, rows;  // first token row, valid rows
};

// tile_end[e]: tiles of the experts up to e; row_end[e]: their rows.
__device__ __forceinline__ MxUnit mx_unit(int u, int n_mb, int bn, int E, const int *tile_end,
                                          const int *row_end) {
    MxUnit w;
    const int t = u / n_mb;
    w.mb = u - t * n_mb;
    int lo = 0, hi = E - 1;  // the first expert with tile_end > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tile_end[mid] > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    w.e = lo;
    const int t0 = lo ? tile_end[lo - 1] : 0, r0 = lo ? row_end[lo - 1] : 0;
    w.row = r0 + (t - t0) * bn;
    w.rows = min(bn, row_end[lo] - w.row);
    return w;
}

__device__ __forceinline__ int mx_cols(int rows) { return (rows + 15) & ~15; }

__device__ __forceinline__ void store_value(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_value(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The two words of scales (8 blocks) from word w0 of a row of `words`.
template <int VEC>
__device__ __forceinline__ uint2 load_scale_words(const uint32_t *row, int w0, int words) {
    if (VEC == 2) return *reinterpret_cast<const uint2 *>(row + w0);
    return make_uint2(row[w0], w0 + 1 < words ? row[w0 + 1] : 0u);
}

template <int NUM_A, int BN, int VEC, typename TOut>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_product_kernel(const __grid_constant__ Mx4Maps maps, const Mx4Args p) {
    using C = MxCfg<NUM_A, BN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
    __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
    __shared__ int s_tiles[kMaxE], s_rows[kMaxE];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh, bad_sh;
    // What an abort has to wait for: the stages issued, and the step that each
    // scale warp gave up at (none: all of its stages are laid out).
    __shared__ uint32_t issued_sh, gave_up_sh[kMxScaleWarps];
    uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const volatile int *abort_flag = &abort_sh;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 2);  // the TMA thread and the scales' warp
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], 256);
        }
        mbar_init(&drain_bar, 1);
        abort_sh = 0;
        bad_sh = 0;
        for (int i = 0; i < kMxScaleWarps; ++i) gave_up_sh[i] = ~0u;
        fence_barrier_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.a);
        if (NUM_A == 2) tma_prefetch_desc(&maps.w3);
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, kMxTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = tmem_base_sh;
    griddep_wait();
    griddep_launch_dependents();

    // Inclusive sums over the experts of their rows and of their tiles, eight
    // experts a lane.  Rows past p.N do not exist: counts that say otherwise
    // are cut and reported.
    if (warp == 0) {
        constexpr int kPer = kMaxE / 32;
        int r[kPer];
        bool bad = false;
        long long sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane * kPer + i;
            r[i] = e < p.E ? p.counts[e] : 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bad |= r[i] < 0 || r[i] > p.N;
            r[i] = r[i] < 0 ? 0 : min(r[i], p.N);
            sum += r[i];
        }
        long long end = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += v;
        }
        end -= sum;
        int tiles = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int lo = int(min(end, (long long)p.N));
            end += r[i];
            bad |= end > p.N;
            const int hi = int(min(end, (long long)p.N));
            tiles += (hi - lo + BN - 1) / BN;
            r[i] = tiles;
            if (lane * kPer + i < p.E) s_rows[lane * kPer + i] = hi;
        }
        int before = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        before -= tiles;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane * kPer + i < p.E) s_tiles[lane * kPer + i] = before + r[i];
        if (__any_sync(0xffffffffu, bad) && lane == 0) bad_sh = 1;
    }
    __syncthreads();
    const int n_mb = p.n >> 7;
    const int n_units = s_tiles[p.E - 1] * n_mb;
    const int nkb = (p.k + kMxStepK - 1) / kMxStepK, chunks = p.k >> 7;
    MxRing<STAGES> ring;

    if (warp == 0) {
        // -------------------------------------------- codes, weight scales --
        const uint32_t one = elect_one();
        uint32_t it = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
            const MxUnit w = mx_unit(u, n_mb, BN, p.E, s_tiles, s_rows);
            const int w_row = uniform(w.e * p.n + w.mb * 128);
            const int row = uniform(w.row), boxes = uniform((w.rows + int(C::BOX) - 1) / int(C::BOX));
            const long long sf = (long long)(w_row >> 7) * chunks * kMxSfChunk;
            for (int kb = 0; kb < nkb; ++kb, ++it, ring.next()) {
                uint64_t *bar = &full_bar[ring.s];
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty_bar[ring.s], ring.phase ^ 1u,
                                                               abort_flag, p.timeout_ns)) != 0;
                if (!ok) break;
                if (p.fault_skip && blockIdx.x == 0 && it == 0)
                    continue;  // test hook: this stage never fills
                if (one) {
                    uint8_t *st = smem + size_t(ring.s) * C::STAGE_BYTES;
                    const uint32_t sfb = min(2, chunks - 2 * kb) * kMxSfChunk;
                    mbar_arrive_expect_tx(bar, NUM_A * (C::A_BYTES + sfb) + boxes * C::BOX * 128);
                    tma_load_2d(st, &maps.w, kb * 128, w_row, bar);
                    if (NUM_A == 2) tma_load_2d(st + C::A_BYTES, &maps.w3, kb * 128, w_row, bar);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(st + C::OFF_B + i * C::BOX * 128, &maps.a, kb * 128,
                                    row + i * int(C::BOX), bar);
                    const long long o = sf + (long long)kb * 2 * kMxSfChunk;
                    bulk_load(st + C::OFF_SFA, p.w_scales + o, sfb, bar);
                    if (NUM_A == 2)
                        bulk_load(st + C::OFF_SFA + 2 * kMxSfChunk, p.w3_scales + o, sfb, bar);
                }
                __syncwarp();
            }
        }
        if (!ok) *reinterpret_cast<volatile int *>(&abort_sh) = 1;
        if (lane == 0) issued_sh = it;
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer --
        const uint32_t one = elect_one();
        uint32_t lu = 0, set = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t phase) {
            return __all_sync(0xffffffffu,
                              mbar_wait_bounded(bar, phase, abort_flag, p.timeout_ns)) != 0;
        };
        for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x, ++lu) {
            const MxUnit w = mx_unit(u, n_mb, BN, p.E, s_tiles, s_rows);
            const int cols = uniform(mx_cols(w.rows));
            const uint32_t a = lu % C::ACC_BUFS;
            ok = wait(&tempty_bar[a], ((lu / C::ACC_BUFS) & 1u) ^ 1u);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d0 = tmem_base + a * C::ACC_COLS;
            for (int kb = 0; kb < nkb; ++kb, ring.next(), set ^= 1u) {
                ok = wait(&full_bar[ring.s], ring.phase);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t sa = smem_u32(smem) + uint32_t(ring.s) * C::STAGE_BYTES;
                const uint32_t sf = tmem_base + kMxTmemCols - kMxSfCols + set * C::SF_COLS;
                const int nc = min(2, chunks - 2 * kb);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c >= nc) break;
                    // columns: [chunk][W, W3, B tiles] x 4
                    const uint32_t col = sf + c * 4 * (NUM_A + C::B_SF_TILES);
#pragma unroll
                    for (int m = 0; m < NUM_A; ++m)
                        tmem_cp_scales(one, col + 4 * m,
                                       sa + C::OFF_SFA + (m * 2 + c) * kMxSfChunk);
#pragma unroll
                    for (uint32_t j = 0; j < C::B_SF_TILES; ++j)
                        tmem_cp_scales(one, col + 4 * (NUM_A + j),
                                       sa + C::OFF_SFB + (c * C::B_SF_TILES + j) * kMxSfChunk);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t off = (c * 2 + h) * 32;
                        const uint64_t bdesc = umma_desc_sw128(sa + C::OFF_B + off);
                        const uint32_t id = mxf4_idesc(cols, 2 * h);
                        const uint32_t acc = (kb | c | h) ? 1u : 0u;
#pragma unroll
                        for (int m = 0; m < NUM_A; ++m)
                            umma_mxf4(one, d0 + m * BN,
                                      umma_desc_sw128(sa + m * C::A_BYTES + off),
                                      bdesc, id, col + 4 * m, col + 4 * NUM_A, acc);
                    }
                }
                umma_commit_by(one, &empty_bar[ring.s]);
            }
            if (!ok) break;
            umma_commit_by(one, &tfull_bar[a]);
        }
        if (!ok) {
            *reinterpret_cast<volatile int *>(&abort_sh) = 1;
            umma_commit_by(one, &drain_bar);  // wait for what was issued
            mbar_wait_bounded(&drain_bar, 0u, nullptr, p.timeout_ns);
        }
    } else if (warp >= kMxScaleWarp) {
        // ------------------------------------------------ token rows' scales --
        // Lane l carries rows l, l + 32, ...: a stage's words of a row are
        // exactly its bytes in the stage's two tiles.
        constexpr int RPL = (BN + 31) / 32;
        const int words = p.k >> 7;  // 32-bit words of scales per row
        const uint32_t *base = reinterpret_cast<const uint32_t *>(p.a_scales);
        const int first = warp - kMxScaleWarp;
        const int units = int(blockIdx.x) < n_units
                              ? (n_units - 1 - int(blockIdx.x)) / int(gridDim.x) + 1 : 0;
        const uint32_t total = first < STAGES ? uint32_t(units) * nkb : 0u;
        bool ok = true;
        uint2 next[RPL];
        int unit = -1;
        MxUnit w;
        auto load = [&](uint32_t it) {
            const int lu = int(it) / nkb, kb = int(it) - lu * nkb;
            if (lu != unit)
                w = mx_unit(int(blockIdx.x) + lu * int(gridDim.x), n_mb, BN, p.E, s_tiles,
                            s_rows);
            unit = lu;
#pragma unroll
            for (int q = 0; q < RPL; ++q) {
                const int r = lane + 32 * q;
                next[q] = make_uint2(0u, 0u);
                if (r < w.rows)
                    next[q] = load_scale_words<VEC>(base + (long long)(w.row + r) * words, kb * 2,
                                                    words);
            }
        };
        uint32_t lap = 0, it = uint32_t(first);  // stage s of a lap is step lap + s
        ring.s = first;
        if (it < total) load(it);
        while (it < total) {
            int s = ring.s + kMxScaleWarps;
            uint32_t then = it + kMxScaleWarps;
            if (s >= STAGES) {
                lap += uint32_t(STAGES);
                s = first;
                then = lap + uint32_t(first);
            }
            uint2 cur[RPL];
#pragma unroll
            for (int q = 0; q < RPL; ++q) cur[q] = next[q];
            if (then < total) load(then);
            ok = mbar_wait_bounded(&empty_bar[ring.s], ring.phase ^ 1u, abort_flag, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t *sfb = smem + size_t(ring.s) * C::STAGE_BYTES + C::OFF_SFB;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (uint32_t j = 0; j < C::B_SF_TILES; ++j) {
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int rq = int(j) * 4 + q;
                        v[q] = rq < RPL ? (c ? cur[rq < RPL ? rq : 0].y : cur[rq < RPL ? rq : 0].x) : 0u;
                    }
                    *reinterpret_cast<uint4 *>(sfb + (c * C::B_SF_TILES + j) * kMxSfChunk +
                                               lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            // the tensor core reads them through the async proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&full_bar[ring.s]);
            if (s <= ring.s) ring.phase ^= 1u;
            ring.s = s;
            it = then;
        }
        if (!ok && lane == 0) {
            *reinterpret_cast<volatile int *>(&abort_sh) = 1;
            gave_up_sh[first] = it;
        }
    } else {
        // -------------------------------------------------------- epilogue --
        const int q = warp & 3;  // TMEM lane quadrant of this warp
        uint32_t lu = 0;
        for (int u = blockIdx.x; u < n_units; u += gridDim.x, ++lu) {
            const MxUnit w = mx_unit(u, n_mb, BN, p.E, s_tiles, s_rows);
            const uint32_t a = lu % C::ACC_BUFS;
            bool ok = mbar_wait_bounded(&tfull_bar[a], (lu / C::ACC_BUFS) & 1u, abort_flag,
                                        p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) *reinterpret_cast<volatile int *>(&abort_sh) = 1;
                break;
            }
            tc_fence_after_sync();
            const uint32_t tb = tmem_base + (uint32_t(q * 32) << 16) + a * C::ACC_COLS;
            TOut *out = static_cast<TOut *>(p.out) + (long long)w.row * p.n + w.mb * 128 + q * 32 + lane;
            if constexpr (BN == 32) {
                // decode: few rows, and code that is fetched once per launch, so
                // short code counts (eight columns at a time: 4.5 us for 4.2 at 8
                // rows of 128, 20.4 for 20.2 at 154 rows of 128 experts)
                TOut *to = out + (long long)((warp - 2) >> 2) * p.n;
#pragma unroll 1
                for (int c = (warp - 2) >> 2; c < w.rows; c += 2, to += 2ll * p.n) {
                    uint32_t y1, v1 = 0u;
                    tmem_ld_1(tb + c, y1);
                    if (NUM_A == 2) tmem_ld_1(tb + BN + c, v1);
                    tmem_ld_wait();
                    asm volatile("" : "+r"(y1), "+r"(v1));
                    float y = __uint_as_float(y1);
                    if (NUM_A == 2) y = y / (1.0f + expf(-y)) * __uint_as_float(v1);
                    store_value(to, y);
                }
            } else {
#pragma unroll 1
                for (int c0 = ((warp - 2) >> 2) * 8; c0 < w.rows; c0 += 16) {
                    uint32_t y8[8], v[8];
                    tmem_ld_8(tb + c0, y8);
                    if (NUM_A == 2) tmem_ld_8(tb + BN + c0, v);
                    tmem_ld_wait();
                    reg_fence_8(y8);
                    if (NUM_A == 2) reg_fence_8(v);
                    TOut *to = out + (long long)c0 * p.n;
                    auto put = [&](int c) {
                        float y = __uint_as_float(y8[c]);
                        if (NUM_A == 2) y = y / (1.0f + expf(-y)) * __uint_as_float(v[c]);
                        store_value(to, y);
                        to += p.n;
                    };
                    if (c0 + 8 <= w.rows) {  // without a compare per row
#pragma unroll
                        for (int c = 0; c < 8; ++c) put(c);
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c0 + c < w.rows) put(c);
                    }
                }
            }
            tc_fence_before_sync();
            mbar_arrive(&tempty_bar[a]);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0) {
        // Own word of this CTA: no other call's or CTA's status can meet it.
        p.status[64 + blockIdx.x] =
            abort_sh ? int(DEV_ERR_TIMEOUT) : bad_sh ? int(DEV_ERR_INTERNAL) : int(DEV_OK);
        if (blockIdx.x == 0) p.status[0] = int(gridDim.x);
        // Whichever role gave up, this CTA's own copies land before it exits.
        // A stage completes with its bytes and its scales' arrival, which is
        // made here for the scale warps that left before it (nobody reads the
        // scales any more); the waits share one limit.
        if (abort_sh) {
            const uint32_t n = issued_sh;
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t j = n > uint32_t(STAGES) ? n - STAGES : 0u; j < n; ++j) {
                if (p.fault_skip && blockIdx.x == 0 && j == 0) continue;  // never issued
                const uint32_t s = j % STAGES;
                if (j >= gave_up_sh[s % kMxScaleWarps]) mbar_arrive(&full_bar[s]);
                const uint64_t spent = globaltimer_ns() - t0;
                mbar_wait_bounded(&full_bar[s], (j / STAGES) & 1u, nullptr,
                                  spent < p.timeout_ns ? p.timeout_ns - spent : 0u);
            }
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, kMxTmemCols);
    }
}

template <int NUM_A, int BN, int VEC, typename TOut>
cudaError_t launch_product_vec(const Mx4Maps &maps, const Mx4Args &a, int grid, cudaStream_t st) {
    using C = MxCfg<NUM_A, BN>;
    auto kern = mx4_product_kernel<NUM_A, BN, VEC, TOut>;
    static std::atomic<unsigned long long> attr_set{0};  // this instantiation only
    cudaError_t e = set_smem_once(kern, int(C::SMEM_BYTES), attr_set);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(kMxThreads), C::SMEM_BYTES, st, maps, a);
}

template <int NUM_A, int BN, typename TOut>
beam_status launch_product(Mx4Maps &maps, const uint8_t *a_codes, const Mx4Args &a, int grid,
                           cudaStream_t st) {
    if (!make_byte_tmap(&maps.a, a_codes, a.k / 2, a.N, MxCfg<NUM_A, BN>::BOX)) return BEAM_ERR_CUDA;
    // rows' scales by eight bytes where every row starts at such a boundary
    const cudaError_t e = (a.k >> 7) % 2 == 0
                              ? launch_product_vec<NUM_A, BN, 2, TOut>(maps, a, grid, st)
                              : launch_product_vec<NUM_A, BN, 1, TOut>(maps, a, grid, st);
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

template <typename TOut>
beam_status launch_product_bn(int swiglu, int bn, Mx4Maps &maps, const uint8_t *a_codes,
                              const Mx4Args &a, int grid, cudaStream_t st) {
    if (swiglu) {
        if (bn == 32) return launch_product<2, 32, TOut>(maps, a_codes, a, grid, st);
        if (bn == 64) return launch_product<2, 64, TOut>(maps, a_codes, a, grid, st);
        return launch_product<2, 112, TOut>(maps, a_codes, a, grid, st);
    }
    if (bn == 32) return launch_product<1, 32, TOut>(maps, a_codes, a, grid, st);
    if (bn == 64) return launch_product<1, 64, TOut>(maps, a_codes, a, grid, st);
    if (bn == 128) return launch_product<1, 128, TOut>(maps, a_codes, a, grid, st);
    return launch_product<1, 192, TOut>(maps, a_codes, a, grid, st);
}

// Token rows per tile, from the mean rows per expert a full batch would have.
// (A mask leaves fewer rows in wide tiles, which costs nothing, since MMAs and
// boxes follow the rows: 9830 rows, 77 an expert, in a batch for 65536 take
// gate and up 47.0 us and down 35.0; in one for 9830, with the next narrower
// tiles, 47.0 and 36.8.)
// Two accumulators have to fit TMEM beside the scales, so that one is read out
// while the other fills: 192 columns, with gate and up 112.
int product_bn(int N, int E, int swiglu) {
    const long long avg = ((long long)N + E - 1) / E;
    if (avg <= 16) return 32;
    if (avg <= 64) return 64;
    return swiglu ? 112 : avg <= 256 ? 128 : 192;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr size_t kMxWorkspace = 8192;  // status words: [0] CTAs, [64 + b] CTA b
constexpr int kMxMaxCtas = 1024;

beam_status check_mx4_desc(const beam_mx4_desc *d) {
    if (!d) return BEAM_ERR_INVALID_ARG;
    if (d->N < 0 || d->E <= 0 || d->E > kMaxE || d->n <= 0 || d->k <= 0) return BEAM_ERR_INVALID_ARG;
    if (d->swiglu != 0 && d->swiglu != 1) return BEAM_ERR_INVALID_ARG;
    if (d->out_dtype != BEAM_BF16 && d->out_dtype != BEAM_F32) return BEAM_ERR_INVALID_ARG;
    if (d->n % 128 != 0 || d->k % 128 != 0) return BEAM_ERR_UNSUPPORTED_SHAPE;
    // weight rows are 32-bit TMA coordinates, units 32-bit counters
    if ((long long)d->E * d->n > 0x7fffffffll) return BEAM_ERR_UNSUPPORTED_SHAPE;
    if (((long long)d->N / 16 + d->E) * (d->n / 128) > 0x3fffffffll || d->N > 0x3fffffff)
        return BEAM_ERR_UNSUPPORTED_SHAPE;
    return BEAM_OK;
}

beam_status check_rows(int dtype, long long rows, int cols, int tiled) {
    if (dtype != BEAM_BF16 && dtype != BEAM_F32) return BEAM_ERR_INVALID_ARG;
    if (rows < 0 || cols <= 0 || (tiled != 0 && tiled != 1)) return BEAM_ERR_INVALID_ARG;
    if (cols % 32 != 0) return BEAM_ERR_UNSUPPORTED_SHAPE;
    if (rows > 0x7fffffffffffll / cols) return BEAM_ERR_UNSUPPORTED_SHAPE;
    if (tiled && (rows % 128 != 0 || cols % 128 != 0)) return BEAM_ERR_UNSUPPORTED_SHAPE;
    return BEAM_OK;
}

// CTAs for this many pieces of a thread's step; a few rounds of them leave the
// SMs evenly loaded to the end (one round of 8 per SM: 6 % slower).
int rows_grid(long long pieces, int ahead) {
    const long long blocks = (pieces + 256 * ahead - 1) / (256 * ahead);
    const long long most = 64ll * device_sm_count();
    return int(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace beam

using namespace beam;

extern "C" {

beam_status beam_mx4_quantize(int dtype, long long rows, int cols, const void *x,
                              const int32_t *n_rows, uint8_t *codes, uint8_t *scales, int tiled,
                              void *stream) {
    beam_status s = check_rows(dtype, rows, cols, tiled);
    if (s != BEAM_OK) return s;
    if (tiled && n_rows) return BEAM_ERR_INVALID_ARG;
    if (rows == 0) return BEAM_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales))
        return BEAM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(n_rows) & 3u) return BEAM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(rows_grid(rows * (cols / 8), kMxAhead)), block(256);
    uint32_t *out = reinterpret_cast<uint32_t *>(codes);
    cudaError_t e =
        dtype == BEAM_BF16
            ? launch_pdl(mx4_quantize_kernel<__nv_bfloat16>, grid, block, 0, st,
                         static_cast<const __nv_bfloat16 *>(x), rows, cols, n_rows, out, scales, tiled)
            : launch_pdl(mx4_quantize_kernel<float>, grid, block, 0, st,
                         static_cast<const float *>(x), rows, cols, n_rows, out, scales, tiled);
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

beam_status beam_mx4_dequantize(int dtype, long long rows, int cols, const uint8_t *codes,
                                const uint8_t *scales, int tiled, void *out, void *stream) {
    beam_status s = check_rows(dtype, rows, cols, tiled);
    if (s != BEAM_OK) return s;
    if (rows == 0) return BEAM_OK;
    if (!out || !codes || !scales || !aligned16(out) || !aligned16(codes) || !aligned16(scales))
        return BEAM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(rows_grid(rows * (cols / (dtype == BEAM_BF16 ? 8 : 4)), kMxAheadBack)), block(256);
    cudaError_t e = dtype == BEAM_BF16
                        ? launch_pdl(mx4_dequantize_kernel<__nv_bfloat16>, grid, block, 0, st,
                                     codes, scales, rows, cols, tiled,
                                     static_cast<__nv_bfloat16 *>(out))
                        : launch_pdl(mx4_dequantize_kernel<float>, grid, block, 0, st, codes,
                                     scales, rows, cols, tiled, static_cast<float *>(out));
    return e == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
}

size_t beam_mx4_workspace_size(const beam_mx4_desc *desc) {
    return check_mx4_desc(desc) == BEAM_OK ? kMxWorkspace : 0;
}

beam_status beam_mx4_expert_product(const beam_mx4_desc *desc, const uint8_t *a_codes,
                                    const uint8_t *a_scales, const int32_t *expert_counts,
                                    const uint8_t *w_codes, const uint8_t *w_scales,
                                    const uint8_t *w3_codes, const uint8_t *w3_scales, void *out,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    beam_status s = check_mx4_desc(desc);
    if (s != BEAM_OK) return s;
    if (!expert_counts || !w_codes || !w_scales) return BEAM_ERR_INVALID_ARG;
    if (desc->swiglu ? (!w3_codes || !w3_scales) : (w3_codes || w3_scales))
        return BEAM_ERR_INVALID_ARG;
    for (const void *q : {static_cast<const void *>(a_codes), static_cast<const void *>(a_scales),
                          static_cast<const void *>(expert_counts),
                          static_cast<const void *>(w_codes), static_cast<const void *>(w_scales),
                          static_cast<const void *>(w3_codes),
                          static_cast<const void *>(w3_scales), static_cast<const void *>(out)})
        if (!aligned16(q)) return BEAM_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < kMxWorkspace)
        return BEAM_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (desc->N == 0)
        return cudaMemsetAsync(workspace, 0, 256, st) == cudaSuccess ? BEAM_OK : BEAM_ERR_CUDA;
    if (!a_codes || !a_scales || !out) return BEAM_ERR_INVALID_ARG;
    const int bn = product_bn(desc->N, desc->E, desc->swiglu);
    const unsigned long long row_bytes = desc->k / 2, w_rows = (unsigned long long)desc->E * desc->n;
    Mx4Maps maps;
    const uint8_t *w3 = desc->swiglu ? w3_codes : w_codes;
    if (!make_byte_tmap(&maps.w, w_codes, row_bytes, w_rows, 128) ||
        !make_byte_tmap(&maps.w3, w3, row_bytes, w_rows, 128))
        return BEAM_ERR_CUDA;
    Mx4Args a;
    a.N = desc->N;
    a.E = desc->E;
    a.n = desc->n;
    a.k = desc->k;
    a.counts = expert_counts;
    a.a_scales = a_scales;
    a.w_scales = w_scales;
    a.w3_scales = w3_scales;
    a.out = out;
    a.status = static_cast<int *>(workspace);
    a.timeout_ns = device_wait_limit_ns();
    a.fault_skip = device_fault_mode() == FAULT_MX4_STAGE;
    // No more CTAs than units there can be: a tile per full BN rows plus one
    // unfilled per expert that has rows.
    const long long tiles = desc->N / bn + (desc->N < desc->E ? desc->N : desc->E);
    long long grid = tiles * (desc->n / 128);
    const int n_sm = device_sm_count() < kMxMaxCtas ? device_sm_count() : kMxMaxCtas;
    if (grid > n_sm) grid = n_sm;
    return desc->out_dtype == BEAM_F32
               ? launch_product_bn<float>(desc->swiglu, bn, maps, a_codes, a, int(grid), st)
               : launch_product_bn<__nv_bfloat16>(desc->swiglu, bn, maps, a_codes, a, int(grid), st);
}

beam_status beam_mx4_check(const beam_mx4_desc *desc, void *workspace, void *stream) {
    beam_status s = check_mx4_desc(desc);
    if (s != BEAM_OK) return s;
    if (!workspace) return BEAM_ERR_WORKSPACE;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return BEAM_ERR_CUDA;
    int words[64 + kMxMaxCtas];
    if (cudaMemcpy(words, workspace, sizeof(words), cudaMemcpyDeviceToHost) != cudaSuccess)
        return BEAM_ERR_CUDA;
    const int n = words[0] < 0 ? 0 : words[0] > kMxMaxCtas ? kMxMaxCtas : words[0];
    int worst = DEV_OK;
    for (int b = 0; b < n; ++b) {
        if (words[64 + b] == DEV_ERR_TIMEOUT) return BEAM_ERR_TIMEOUT;
        if (words[64 + b] != DEV_OK) worst = DEV_ERR_INTERNAL;
    }
    return worst == DEV_OK ? BEAM_OK : BEAM_ERR_INTERNAL;
}

}  // extern "C"
