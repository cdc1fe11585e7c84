// moe.cu -- mixture-of-experts layer for a few tokens (decode batches) on sm_100a: the router and
// the experts' gated MLP on 4-bit weights.
//
// Router: z = x . Wr^T + bias, the k largest of each token's z (equal ones: the lower expert
// first), their softmax weights. Experts: y_t = sum_k w[t,k] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t))
// with e = ids[t,k]. With at most 64 tokens the cost is reading the met experts' weights once.
//
// The weights go to the FP4 tensor cores as they are stored. Those multiply FP4 by FP4 only, so an
// activation is split into eight FP4 terms, each the FP4 form of what the ones before leave
// (write_terms), and the eight products are added: the weights lose nothing and the activations
// about 2^-18 of their block's largest value, while the terms' columns cost the otherwise idle MMA
// 8 of its up to 256 columns a token. (Decoding the weights to f16 on the CUDA cores for mma.sync
// took 40-54 issue slots per 16 x 32 codes, as long as HBM takes to deliver them, and ran at a
// quarter of it: 64 tokens, 64 experts of 2048 x 1024, top 8: 135 us.)
#include <mutex>

#include "fp4_format.cuh"
#include "mxfp4_encode.cuh"
#include "nvfp4_internal.cuh"
#include "sm100_ptx.cuh"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------------------

constexpr int kRouteThreads = 256;
constexpr int kRouteCluster = 8;

struct RouteParams {
    const uint4 *x, *w; // bf16 [T x H], [E x H]
    const float *bias;  // [E] or null
    int64_t T, H;
    int E, k, renorm;
    int *ids;           // [T x k]
    float *weights;     // [T x k]
};

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v)
{
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// c = A B (16 x 8, K 16, bf16), and c += A B.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A cluster of 8 CTAs takes 8 tokens. Logits: 16 experts are the rows of bf16 MMAs, the tokens the
// columns; a CTA takes chunks of 16 experts (with few chunks, a slice of K too), its warps every
// eighth 32-wide block of K. Each block's 32 products are summed in fp32 by two MMAs and the blocks
// in fp64, so that the choice between two close experts does not hang on the order of a long sum.
// The logits go to the CTA that ranks the token: expert e is chosen if fewer than k experts precede
// it, counted by every thread at once. Bound by the latency of one round of loads (W is 1 MB at 128
// experts of 4096) and of the cluster barrier.
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
    moe_route_kernel(const RouteParams p)
{
    __shared__ double s_z[512];           // [slice][expert], then [expert]: this CTA's token
    __shared__ double s_part[8][16 * 8];  // [warp][expert][token]
    __shared__ int s_sel[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_ctarank();
    const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * 8;
    cluster_arrive(); // matched below: every CTA of the cluster runs before remote stores
    const int chunks = (p.E + 15) / 16;
    const int slices = chunks == 1 ? 8 : chunks == 2 ? 4 : chunks <= 4 ? 2 : 1;
    const int per = kRouteCluster / slices; // CTAs per slice of K
    const int slice = rank / per;
    const int64_t nvec = p.H >> 3;
    const int nblk = (int)(p.H >> 5);
    const int b0 = (int)((int64_t)nblk * slice / slices);
    const int b1 = (int)((int64_t)nblk * (slice + 1) / slices);
    const uint32_t zaddr = smem_u32(s_z);
    pdl_wait();
    const int64_t tok = t0 + g < p.T ? t0 + g : p.T - 1;
    for (int c = rank % per; c < chunks; c += per) {
        const uint4 *wa = p.w + (int64_t)min(c * 16 + g, p.E - 1) * nvec + t;
        const uint4 *wb = p.w + (int64_t)min(c * 16 + g + 8, p.E - 1) * nvec + t;
        const uint4 *xr = p.x + tok * nvec + t;
        double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
        for (int b = b0 + warp; b < b1; b += 8) {
            const uint4 a = __ldg(wa + 4 * b), d = __ldg(wb + 4 * b), x = __ldg(xr + 4 * b);
            float f[4]; // lane t's k indices: its 8 values of the block, whatever their order
            mma_bf16_first(f, a.x, d.x, a.y, d.y, x.x, x.y);
            mma_bf16(f, a.z, d.z, a.w, d.w, x.z, x.w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] += (double)f[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s_part[warp][(g + (j >> 1) * 8) * 8 + 2 * t + (j & 1)] = acc[j];
        __syncthreads();
        if (c < per)
            cluster_wait(); // (the first chunk) the other CTAs have started
        if (tid < 128) {
            const int e = c * 16 + (tid >> 3), j = tid & 7;
            double z = 0.0;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                z += s_part[w][tid];
            if (e < p.E)
                st_cluster_f64(mapa_shared(zaddr + 8u * (uint32_t)(slice * p.E + e), (uint32_t)j),
                               z);
        }
        __syncthreads();
    }
    if (rank % per >= chunks)
        cluster_wait();
    cluster_sync(); // this CTA's token has all its logits
    pdl_launch_dependents();
    const int64_t tk = t0 + rank;
    if (tk >= p.T)
        return;
    if (tid < 32)
        s_sel[tid] = -1;
    for (int e = tid; e < p.E; e += kRouteThreads) {
        double z = s_z[e];
        for (int q = 1; q < slices; ++q)
            z += s_z[q * p.E + e];
        if (p.bias)
            z += (double)__ldg(p.bias + e);
        s_z[e] = z == z ? z : -INFINITY; // a NaN logit is never chosen
    }
    __syncthreads();
    // parts threads share an expert's count (E <= 64: 4, <= 128: 2)
    const int parts = p.E <= 64 ? 4 : p.E <= 128 ? 2 : 1;
    const int part = tid % parts;
    for (int e0 = 0; e0 < p.E; e0 += kRouteThreads / parts) {
        const int e = e0 + tid / parts;
        const double z = e < p.E ? s_z[e] : -INFINITY;
        int n = 0;
        for (int q = part; q < p.E; q += parts) {
            const double o = s_z[q];
            n += (o > z || (o == z && q < e)) ? 1 : 0;
        }
        for (int o = 1; o < parts; o <<= 1)
            n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (part == 0 && e < p.E && n < p.k && z > -INFINITY)
            s_sel[n] = e;
    }
    __syncthreads();
    if (warp == 0) {
        const int e = lane < p.k ? s_sel[lane] : -1;
        const double top = s_sel[0] >= 0 ? s_z[s_sel[0]] : 0.0;
        // exp(z - top), 1 at the top itself (also where it is infinite)
        auto share = [&](int q) {
            const double z = s_z[q];
            return z == top ? 1.0f : expf((float)(z - top));
        };
        const float v = e >= 0 ? share(e) : 0.0f;
        float sum = 0.0f;
        if (p.renorm) {
            sum = v;
        } else if (s_sel[0] >= 0) {
            for (int q = lane; q < p.E; q += 32)
                sum += share(q);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane < p.k) {
            p.ids[tk * p.k + lane] = e;
            p.weights[tk * p.k + lane] = e >= 0 ? v / sum : 0.0f;
        }
    }
}

// ---------------------------------------------------------------------------------------
// Experts
// ---------------------------------------------------------------------------------------

constexpr int kTerms = 8;  // FP4 terms of an activation: the rows of one swizzle atom
constexpr int kCols = 16;  // tokens of a column tile: 128 MMA columns
constexpr int kUpRows = 64, kDownRows = 128; // rows of F, of H, per tile

// A column tile: up to kCols of the (expert, token) rows of one expert. Packed: 9 bits of expert, 11
// of row, 4 of columns - 1.
struct MoeUnit {
    int expert, row0, ncol;
};

__device__ __forceinline__ uint32_t pack_unit(int expert, int row0, int ncol)
{
    return (uint32_t)expert | (uint32_t)row0 << 9 | (uint32_t)(ncol - 1) << 20;
}

__device__ __forceinline__ MoeUnit unpack_unit(uint32_t u)
{
    return MoeUnit{(int)(u & 0x1FFu), (int)(u >> 9 & 0x7FFu), (int)(u >> 20) + 1};
}

// What the kernels of one call share in the workspace.
struct MoeShared {
    uint8_t *x_codes, *x_scales; // terms of x: [T * 8][H / 2], [T * 8][x_pitch]
    float *x_factor;             // [T] (NVFP4): the power of two a token was divided by
    int64_t x_pitch;
    float *h;                    // [rows][F]: silu(gate) * up of each (expert, token) row
    uint8_t *h_codes, *h_scales; // its terms
    float *h_factor;
    int64_t h_pitch;
    uint32_t *units;
    int *counts;                 // column tiles, rows
    uint8_t *tok;                // [rows] token
    float *wt;                   // [rows] weight
    float *partial;              // [128-row blocks of y][splits][T][128]
};

// ---- lists and terms ----------------------------------------------------------------------

constexpr int kPrepThreads = 512, kTermThreads = 256;

// The (expert, token) pairs that the ids name, in expert order, as rows: the row's token and weight
// (an expert that a token names twice gets one row with both weights), and the column tiles. ids
// outside [0, E) name no expert. One CTA.
__device__ __forceinline__ void build_lists(const MoeShared &sh, const int *ids,
                                            const float *weights, int T, int k, int E,
                                            uint8_t *smem)
{
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem); // [E][2]: the expert's tokens
    int *base = reinterpret_cast<int *>(mask + 2 * E);   // [E]: its first row
    int16_t *s_ids = reinterpret_cast<int16_t *>(base + E);
    const int tid = threadIdx.x, nthr = blockDim.x, n = T * k;
    auto count = [&](int e) { return __popc(mask[2 * e]) + __popc(mask[2 * e + 1]); };
    for (int i = tid; i < 2 * E; i += nthr)
        mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = __ldg(ids + i), t = i / k;
        const bool on = e >= 0 && e < E;
        s_ids[i] = on ? (int16_t)e : (int16_t)-1;
        if (on)
            atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    if (tid < 32) { // exclusive prefix of rows and of tiles over the experts
        const int per = (E + 31) / 32;
        int rows = 0, tiles = 0;
        for (int q = 0; q < per; ++q) {
            const int e = tid * per + q;
            const int c = e < E ? count(e) : 0;
            rows += c;
            tiles += (c + kCols - 1) / kCols;
        }
        int r0 = rows, u0 = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xFFFFFFFFu, r0, o);
            const int b = __shfl_up_sync(0xFFFFFFFFu, u0, o);
            if (tid >= o) {
                r0 += a;
                u0 += b;
            }
        }
        if (tid == 31) {
            sh.counts[0] = u0;
            sh.counts[1] = r0;
        }
        r0 -= rows;
        u0 -= tiles;
        for (int q = 0; q < per; ++q) {
            const int e = tid * per + q;
            if (e >= E)
                break;
            const int c = count(e);
            base[e] = r0;
            for (int c0 = 0; c0 < c; c0 += kCols)
                sh.units[u0++] = pack_unit(e, r0 + c0, min(kCols, c - c0));
            r0 += c;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = s_ids[i], t = i / k;
        if (e < 0)
            continue;
        bool first = true; // of the token's slots that name e
        float w = 0.0f;
        for (int s = t * k; s < (t + 1) * k; ++s)
            if (s_ids[s] == e) {
                first = first && s >= i;
                w += __ldg(weights + s);
            }
        if (first) {
            const uint32_t *m = mask + 2 * e;
            const int before = t < 32 ? __popc(m[0] & ((1u << t) - 1u))
                                      : __popc(m[0]) + __popc(m[1] & ((1u << (t - 32)) - 1u));
            const int row = base[e] + before;
            sh.tok[row] = (uint8_t)t;
            sh.wt[row] = w;
        }
    }
}

size_t lists_smem(int T, int k, int E) { return 12 * (size_t)E + 2 * (size_t)T * k; }

// One row of activations (load(i): values 4i .. 4i + 3) as kTerms FP4 rows: each term is the FP4
// form of what the terms before leave, so that the sum of the terms is the value up to the last
// remainder. MXFP4 terms have their own E8M0 scale per 32 values ("ceil": nothing saturates; a
// rounding is off by at most 1/5 of the block's largest remainder, 5^-8 = 2^-18.6 in all). NVFP4
// terms have an E4M3 scale per 16 values, of the row divided by a power of two that brings its
// largest value to 1344..2688 (off by at most 1/6 + 1/16 of the block's largest remainder a term,
// down to the smallest scale's 2^-18 of the row's largest value). A row with a NaN or an infinity
// gets NaN scales (MXFP4) or a NaN factor, and so NaN results. Eight lanes take 32 values.
template <bool NV, int THREADS, typename Load>
__device__ __forceinline__ void write_terms(int64_t cols, uint8_t *codes, uint8_t *scales,
                                            int64_t pitch, float *factor, Load load)
{
    const int tid = threadIdx.x, lane = tid & 31, sub = lane & 7;
    float inv_row = 1.0f;
    if constexpr (NV) { // the row's power of two
        __shared__ uint32_t s_max[THREADS / 32];
        uint32_t m = 0u;
        for (int64_t i = tid; i < cols / 4; i += THREADS) {
            const float4 v = load(i);
            m = max(max(m, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu)),
                    max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0)
            s_max[tid >> 5] = m;
        __syncthreads();
        m = s_max[lane & (THREADS / 32 - 1)];
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        // 2^k, k = floor(log2 max) - 10, kept where both it and its inverse are normal
        const int e = min(max((int)(m >> 23) - 10, 1), 253);
        inv_row = __uint_as_float((uint32_t)(254 - e) << 23);
        if (tid == 0)
            *factor = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                       : __uint_as_float((uint32_t)e << 23);
    }
    const int64_t groups = (pitch * (NV ? 16 : 32) + 31) / 32; // 32-value groups, padding included
    for (int64_t b = tid >> 3; b < groups; b += THREADS / 8) { // (whole warps in step)
        const bool on = b * 32 < cols;
        float4 v = on ? load(b * 8 + sub) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (NV) {
            v.x *= inv_row;
            v.y *= inv_row;
            v.z *= inv_row;
            v.w *= inv_row;
        }
#pragma unroll
        for (int j = 0; j < kTerms; ++j) {
            uint32_t m =
                max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                    max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            uint32_t sb;
            float s, inv;
            if constexpr (NV) {
                sb = m >= 0x7F800000u ? 0u : cvt_e4m3(__uint_as_float(m) * (1.0f / 6.0f));
                s = e4m3_to_f32(sb);
                inv = sb != 0u ? __frcp_rn(s) : 0.0f;
            } else {
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                sb = mx_scale_byte(m, true);
                s = sb == kMxNan ? 0.0f : mx_scale_f32(sb);
                inv = mx_inverse(sb);
            }
            const float y[8] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv, 0.0f, 0.0f, 0.0f, 0.0f};
            const uint32_t w = inv != 0.0f ? cvt_e2m1x8(y) & 0xFFFFu : 0u;
            const float2 lo = e2m1x2_to_f32x2(w & 0xFFu), hi = e2m1x2_to_f32x2(w >> 8);
            v.x = fmaf(-lo.x, s, v.x);
            v.y = fmaf(-lo.y, s, v.y);
            v.z = fmaf(-hi.x, s, v.z);
            v.w = fmaf(-hi.y, s, v.w);
            if (!NV && sb == kMxNan)
                v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (on)
                *reinterpret_cast<uint16_t *>(codes + j * (cols >> 1) + b * 16 + sub * 2) =
                    (uint16_t)w;
            if (NV) {
                if ((sub & 3) == 0 && 2 * b + (sub >> 2) < pitch)
                    scales[j * pitch + 2 * b + (sub >> 2)] = on ? (uint8_t)sb : (uint8_t)0;
            } else if (sub == 0 && b < pitch) {
                scales[j * pitch + b] = on ? (uint8_t)sb : (uint8_t)0;
            }
        }
    }
}

__device__ __forceinline__ float4 bf16x4(uint2 v)
{
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

// The tokens' terms (one CTA a token) and, in the last CTA, the lists.
template <bool NV>
__global__ void __launch_bounds__(kPrepThreads)
    moe_prepare_kernel(const MoeShared sh, const uint2 *x, const int *ids, const float *weights,
                       int T, int k, int E, int64_t H)
{
    extern __shared__ __align__(16) uint8_t list_smem[];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x;
    if (t == T) {
        build_lists(sh, ids, weights, T, k, E, list_smem);
        return;
    }
    const uint2 *row = x + t * (H >> 2);
    write_terms<NV, kPrepThreads>(H, sh.x_codes + (int64_t)t * kTerms * (H >> 1),
                    sh.x_scales + (int64_t)t * kTerms * sh.x_pitch, sh.x_pitch, sh.x_factor + t,
                    [&](int64_t i) { return bf16x4(__ldg(row + i)); });
}

// The terms of h, one CTA a row.
template <bool NV>
__global__ void __launch_bounds__(kTermThreads) moe_terms_kernel(const MoeShared sh, int64_t F)
{
    pdl_launch_dependents();
    pdl_wait();
    const int r = blockIdx.x;
    if (r >= sh.counts[1])
        return;
    const float4 *row = reinterpret_cast<const float4 *>(sh.h + (int64_t)r * F);
    write_terms<NV, kTermThreads>(F, sh.h_codes + (int64_t)r * kTerms * (F >> 1),
                    sh.h_scales + (int64_t)r * kTerms * sh.h_pitch, sh.h_pitch, sh.h_factor + r,
                    [&](int64_t i) { return __ldcg(row + i); });
}

// ---- products -----------------------------------------------------------------------------

constexpr int kThreads = 480;
constexpr uint32_t kWaitLimit = 1u << 20;
constexpr int kSfAhead = 2;  // a feeder group's k-tiles whose scales are on their way
constexpr int kSfRing = kSfAhead + 1;
constexpr int kMaxStages = 8;
constexpr int kMaxSmem = 232448 - 1024;

struct MoeGemm {
    MoeShared sh;
    int T, n_slots;          // tokens, T x top_k
    int64_t H, F;
    const uint8_t *a_scales; // the experts', linear
    int64_t a_rows;          // rows of the stacked weights
    const float *gs;         // [E] (NVFP4)
    int stages, b_rows;      // operand ring: stages, term rows of a stage
    int dense;               // gate/up: a stage holds all tokens' term rows, in token order
    int splits, blocks;      // down: CTAs per 128-row block of y, blocks
    __nv_bfloat16 *y;
    int *status;
};

// A run of k-tiles of one tile, whose sums stay in one accumulator.
struct MoeGroup {
    MoeUnit unit;
    int64_t ra0, ra1; // rows of the stacked weights of the tile's two 64-row halves
    int k0, k1;       // k-tiles (none: an empty job)
    int first;        // gate/up: first column of h; down: the block of y
    int split;
    bool last;        // down: the job's last run
};

// The groups of a CTA, in order; every role of the CTA walks them by itself. Gate/up: a run of the
// flat list of (column tile, 64 columns of F). Down: jobs (128-row block of y, split), whose run of
// the flat list of (column tile, k-tile) pairs is cut at the column tiles.
template <bool DOWN> struct MoeWalk {
    const MoeGemm &p;
    const uint32_t *units; // in shared memory
    int n_units, nkt, per;
    int64_t i, i1;       // gate/up
    int job, u, kt;      // down
    int64_t rest;

    __device__ __forceinline__ MoeWalk(const MoeGemm &q, const uint32_t *list, int n)
        : p(q), units(list), n_units(n)
    {
        const int64_t K = DOWN ? p.F : p.H;
        nkt = (int)((K + 255) >> 8);
        if constexpr (DOWN) {
            job = (int)blockIdx.x - (int)gridDim.x;
            rest = -1;
        } else {
            per = (int)((p.F + kUpRows - 1) / kUpRows);
            const int64_t n = (int64_t)n_units * per;
            i = n * blockIdx.x / gridDim.x;
            i1 = n * (blockIdx.x + 1) / gridDim.x;
        }
    }

    __device__ __forceinline__ bool next(MoeGroup &g)
    {
        if constexpr (!DOWN) {
            if (i >= i1)
                return false;
            g.unit = unpack_unit(units[(int)(i / per)]);
            g.first = (int)(i % per) * kUpRows;
            g.ra0 = (int64_t)g.unit.expert * 2 * p.F + g.first;
            g.ra1 = g.ra0 + p.F;
            g.k0 = 0;
            g.k1 = nkt;
            ++i;
        } else {
            if (rest <= 0) {
                job += gridDim.x;
                if (job >= p.blocks * p.splits)
                    return false;
                const int64_t total = (int64_t)n_units * nkt;
                g.split = job % p.splits;
                const int64_t a = total * g.split / p.splits;
                rest = total * (g.split + 1) / p.splits - a;
                u = (int)(a / nkt);
                kt = (int)(a % nkt);
            }
            g.first = job / p.splits;
            g.split = job % p.splits;
            if (rest == 0) {
                g.unit = MoeUnit{0, 0, 0};
                g.k0 = g.k1 = 0;
                g.last = true;
                return true;
            }
            g.unit = unpack_unit(units[u]);
            g.ra0 = (int64_t)g.unit.expert * p.H + (int64_t)g.first * kDownRows;
            g.ra1 = g.ra0 + 64;
            g.k0 = kt;
            g.k1 = (int)(rest < nkt - kt ? kt + rest : nkt);
            rest -= g.k1 - g.k0;
            ++u;
            kt = 0;
            g.last = rest == 0;
        }
        return true;
    }
};

template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const uint8_t *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(src))
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(src)), "n"(BYTES)
                     : "memory");
}

// One row's scale bytes of a k-tile where they are not a whole aligned piece: `have` of SB bytes,
// then zeros.
template <int SB>
__device__ __noinline__ void fetch_scales_general(uint32_t dst, const uint8_t *src, int have)
{
    if (have == SB && (reinterpret_cast<uintptr_t>(src) & 3) == 0) {
        for (int i = 0; i < SB; i += 4)
            cp_async<4>(dst + i, src + i);
        return;
    }
    for (int i = 0; i < SB; i += 4) {
        uint32_t w = 0u;
        for (int j = 0; j < 4; ++j)
            if (i + j < have)
                w |= (uint32_t)__ldg(src + i + j) << (8 * j);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + i), "r"(w) : "memory");
    }
}

// 128 rows' scale bytes (SB a row at `sm`) -> the TMEM columns of F::kAtoms atoms, this warp's lane
// quarter: lane r's word i of an atom is row r + 32 i's.
template <class F>
__device__ __forceinline__ void feed_rows(const uint8_t *sm, uint32_t tcol, int lane)
{
    constexpr int SB = 4 * F::kAtoms;
    uint32_t r[4 * F::kAtoms];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F::kMx) {
            const uint2 v = *reinterpret_cast<const uint2 *>(sm + (lane + 32 * i) * SB);
            r[i] = v.x;
            r[4 + i] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(sm + (lane + 32 * i) * SB);
            r[i] = v.x;
            r[4 + i] = v.y;
            r[8 + i] = v.z;
            r[12 + i] = v.w;
        }
    }
    if constexpr (F::kMx)
        tmem_st_32x32b_x8(tcol, r);
    else
        tmem_st_32x32b_x16(tcol, r);
}

// Gate/up (DOWN false) and down products on the FP4 tensor cores: 128 weight rows are the M side of
// block-scaled MMAs, eight term rows of each token of a column tile the N side (8..128 columns), so
// the weights go from HBM to the tensor cores as they are stored and the sum of a token's eight
// columns is the product with its full-precision value. One persistent CTA per SM:
//   warp 0      TMA producer of the weights: per 256-wide k-tile the tile's two 64-row halves;
//   warp 14     TMA producer of the term rows: one box (down; up to 16 tokens in all), or a box of
//               eight rows per token of the column tile;
//   warps 6..13 scale feeders, two groups in turn: the rows' linear scale bytes to shared memory by
//               cp.async ahead of time, then to the stage's TMEM columns in the MMA's layout (one
//               group takes 750 cycles for that);
//   warp 1      MMA issuer; accumulators alternate between two TMEM buffers, so that a tile's
//               epilogue overlaps the next tile's MMAs;
//   warps 2..5  epilogue. Gate/up: a tile is 64 gate rows and the same 64 up rows; they meet in
//               shared memory and silu(gate) * up goes to the workspace in fp32. Down: the weighted
//               sums of every column tile are added to [T][128] sums in shared memory, which go to y
//               or, split by split, to the workspace (moe_sum_kernel).
// A stage's bytes and scales complete one barrier, and the MMAs that have read them another.
// Bound by HBM: a k-tile's 16 KB take 370 ns of an SM's share, its four MMAs of N = 64 about 70 ns;
// a role must therefore take fewer than 700 cycles a k-tile, which is why each is a warp of its own
// with few instructions a step. Waits are bounded; after one that gave up the roles run on without
// waiting and the status word says so.
template <class F, bool DOWN>
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const MoeGemm p)
{
    constexpr int SB = 4 * F::kAtoms;          // scale bytes of a row and k-tile
    constexpr int kSfRows = 2 * 128 * SB;      // weights' and terms' rows of one k-tile
    constexpr uint32_t kAccCols = 128, kSfCol = 2 * kAccCols, kSlotCols = 32;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], drain_bar;
    __shared__ uint32_t tmem_slot;
    const int tid = threadIdx.x, lane = tid & 31;
    // the same in every lane, and known to be: the roles' loops then run on uniform registers
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    if ((smem_u32(smem) & 1023u) != 0) { // the same for every CTA
        if (tid == 0)
            atomicExch(p.status, (int)NVFP4_ERR_CUDA);
        return;
    }
    const int stage_bytes = 16384 + p.b_rows * 128;
    uint8_t *sf_ring = smem + p.stages * stage_bytes;
    float *s_out = reinterpret_cast<float *>(sf_ring + 2 * kSfRing * kSfRows);
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full_bar[s], 2 + 4); // the producers, a feeder group's warps
            mbar_init(&empty_bar[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 4);
        }
        mbar_init(&drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_launch_dependents();
    pdl_wait(); // the lists, the terms
    // the lists to shared memory: [rows] weights, [column tiles], [rows] tokens
    const int n_units = __ldg(p.sh.counts), n_rows = __ldg(p.sh.counts + 1);
    float *s_wt = s_out + (DOWN ? p.T : kCols) * 128;
    uint32_t *s_units = reinterpret_cast<uint32_t *>(s_wt + p.n_slots);
    uint8_t *s_tok = reinterpret_cast<uint8_t *>(s_units + p.n_slots);
    for (int i = tid; i < n_rows; i += kThreads) {
        s_wt[i] = __ldg(p.sh.wt + i);
        s_tok[i] = __ldg(p.sh.tok + i);
    }
    for (int i = tid; i < n_units; i += kThreads)
        s_units[i] = __ldg(p.sh.units + i);
    __syncthreads();

    bool dead = false; // a wait gave up: run on without waiting
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, kWaitLimit)) {
            dead = true;
            atomicExch(p.status, (int)NVFP4_ERR_TIMEOUT);
        }
    };
    int stage = 0;
    uint32_t phase = 0;
    auto next_stage = [&]() {
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
        }
    };
    MoeWalk<DOWN> walk(p, s_units, n_units);
    MoeGroup gr;
    if (warp == 0) {
        // ------------------------------- the weights' TMA producer ------------------
        if (lane == 0) {
            int issued = 0;
            while (walk.next(gr)) {
                const int y0 = (int)gr.ra0, y1 = (int)gr.ra1;
                for (int kt = gr.k0; kt < gr.k1; ++kt) {
                    uint8_t *a = smem + stage * stage_bytes;
                    uint64_t *bar = &full_bar[stage];
                    wait(&empty_bar[stage], phase ^ 1);
                    mbar_arrive_expect_tx(bar, 16384u);
                    tma_load_2d(a, &tmA, bar, kt * 128, y0);
                    tma_load_2d(a + 8192, &tmA, bar, kt * 128, y1);
                    ++issued;
                    next_stage();
                }
            }
            // every copy issued has landed before the CTA may exit
            const int last = issued < p.stages ? issued : p.stages;
            for (int i = 0; i < last; ++i) {
                if (--stage < 0) {
                    stage = p.stages - 1;
                    phase ^= 1;
                }
                wait(&full_bar[stage], phase);
            }
        }
        __syncwarp();
    } else if (warp == 14) {
        // ------------------------------- the term rows' TMA producer ----------------
        const bool one_box = DOWN || p.dense; // else a box of eight rows per token
        while (walk.next(gr)) {
            const int ncol = one_box ? 1 : gr.unit.ncol;
            const uint32_t bytes = one_box ? (uint32_t)p.b_rows * 128u : (uint32_t)ncol * 1024u;
            int row = 0;
            if (DOWN)
                row = gr.unit.row0 * kTerms;
            else if (!one_box && lane < ncol)
                row = (int)s_tok[gr.unit.row0 + lane] * kTerms;
            for (int kt = gr.k0; kt < gr.k1; ++kt) {
                uint64_t *bar = &full_bar[stage];
                wait(&empty_bar[stage], phase ^ 1);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, bytes);
                if (lane < ncol)
                    tma_load_2d(smem + stage * stage_bytes + 16384 + lane * 1024, &tmB, bar, kt * 128,
                                row);
                __syncwarp();
                next_stage();
            }
        }
    } else if (warp >= 6) {
        // ------------------------------- scale feeders ------------------------------
        const int group = (warp - 6) >> 2; // takes every other k-tile
        const int q = warp & 3;            // lane quarter of TMEM
        const int r = tid - 192 - 128 * group; // this thread's row
        const int srow = (int)((DOWN ? p.F : p.H) / F::kBlock);
        const int64_t pitch = DOWN ? p.sh.h_pitch : p.sh.x_pitch;
        const uint8_t *bs = DOWN ? p.sh.h_scales : p.sh.x_scales;
        const bool even = srow % SB == 0; // every piece of a row is whole and aligned
        uint8_t *my_ring = sf_ring + group * kSfRing * kSfRows;
        const uint32_t ring = smem_u32(my_ring) + r * SB;
        MoeWalk<DOWN> ahead(p, s_units, n_units); // kSfAhead of its k-tiles before the stores
        int akt = group, akend = 0, aslot = 0;    // (k-tiles count on into the next run)
        bool more = true, a_on = false, b_on = false;
        const uint8_t *asrc = p.a_scales, *bsrc = bs;
        auto zero = [&](uint32_t dst) {
#pragma unroll
            for (int i = 0; i < SB; i += 4)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + i), "r"(0u) : "memory");
        };
        auto load = [&]() {
            while (more && akt >= akend) {
                MoeGroup ga;
                more = ahead.next(ga);
                if (!more)
                    break;
                akt += ga.k0 - akend;
                akend = ga.k1;
                if (akt >= akend)
                    continue;
                const int64_t row = r < 64 ? ga.ra0 + r : ga.ra1 + (r - 64);
                a_on = row < p.a_rows;
                asrc = p.a_scales + (a_on ? row * srow + (int64_t)akt * SB : 0);
                const bool dense = !DOWN && p.dense;
                const int c = r / kTerms; // this row's token of the stage
                b_on = dense ? c < p.T : c < ga.unit.ncol;
                if (b_on) {
                    const int t = dense ? c
                                  : DOWN ? ga.unit.row0 + c
                                         : (int)s_tok[ga.unit.row0 + c];
                    bsrc = bs + ((int64_t)t * kTerms + r % kTerms) * pitch + (int64_t)akt * SB;
                }
            }
            if (more) {
                const uint32_t dst = ring + aslot * kSfRows;
                if (!a_on)
                    zero(dst);
                else if (even)
                    cp_async<SB>(dst, asrc);
                else
                    fetch_scales_general<SB>(dst, asrc, min(SB, srow - akt * SB));
                if (b_on)
                    cp_async<SB>(dst + 128 * SB, bsrc);
                else
                    zero(dst + 128 * SB);
                asrc += a_on ? 2 * SB : 0;
                bsrc += 2 * SB;
                akt += 2;
                aslot = aslot + 1 == kSfRing ? 0 : aslot + 1;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int i = 0; i < kSfAhead; ++i)
            load();
        int rslot = 0, turn = group;
        const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + kSfCol;
        while (walk.next(gr)) {
            for (int kt = gr.k0; kt < gr.k1; ++kt) {
                if (turn++ & 1) {
                    next_stage();
                    continue;
                }
                asm volatile("cp.async.wait_group %0;" ::"n"(kSfAhead - 1) : "memory");
                named_bar_sync(2 + group, 128); // the rows are here, and the last k-tile's have been read
                load();
                wait(&empty_bar[stage], phase ^ 1);
                __syncwarp();
                tc_fence_after();
                const uint8_t *src = my_ring + rslot * kSfRows;
                feed_rows<F>(src, tbase + stage * kSlotCols, lane);
                feed_rows<F>(src + 128 * SB, tbase + stage * kSlotCols + 16, lane);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full_bar[stage]);
                rslot = rslot + 1 == kSfRing ? 0 : rslot + 1;
                next_stage();
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == 1) {
        // ------------------------------- MMA issuer ---------------------------------
        int buf = 0;
        uint32_t aphase = 0;
        const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSwizzle128B);
        while (walk.next(gr)) {
            if (gr.k0 == gr.k1)
                continue;
            const int ncol = !DOWN && p.dense ? p.T : gr.unit.ncol;
            const uint32_t n = ncol <= 1 ? 8 : ncol <= 2 ? 16 : ncol <= 4 ? 32 : ncol <= 8 ? 64 : 128;
            const uint32_t idesc = F::kIdesc | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (8u << 24);
            const uint32_t acc = tmem + buf * kAccCols;
            wait(&acc_empty[buf], aphase ^ 1);
            uint32_t add = 0u;
            for (int kt = gr.k0; kt < gr.k1; ++kt) {
                wait(&full_bar[stage], phase);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t tsf = tmem + kSfCol + stage * kSlotCols;
                    const uint64_t adesc = desc0 + (uint64_t)((stage * stage_bytes) >> 4);
                    const uint64_t bdesc = adesc + (16384u >> 4);
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
                        tc_mma_fp4<F>(acc, adesc + (uint64_t)(2 * kb), bdesc + (uint64_t)(2 * kb),
                                      idesc | sf_id_bits<F>(kb), tsf + sf_atom<F>(kb) * 4,
                                      tsf + 16 + sf_atom<F>(kb) * 4, kb > 0 ? 1u : add);
                    tc_commit(&empty_bar[stage]);
                }
                add = 1u;
                __syncwarp();
                next_stage();
            }
            if (elect_one())
                tc_commit(&acc_full[buf]);
            __syncwarp();
            buf ^= 1;
            if (buf == 0)
                aphase ^= 1;
        }
        // every MMA issued completes before TMEM is freed (one lane issued them all)
        if (elect_one())
            tc_commit(&drain_bar);
        wait(&drain_bar, 0);
        __syncwarp();
    } else {
        // ------------------------------- epilogue (warps 2..5) ----------------------
        const int q = warp & 3, r = q * 32 + lane; // this thread's accumulator row
        const int et = tid - 64;
        int buf = 0;
        uint32_t aphase = 0;
        if constexpr (DOWN) {
            for (int i = et; i < p.T * 128; i += 128)
                s_out[i] = 0.0f; // [T][128]
            named_bar_sync(1, 128);
        }
        while (walk.next(gr)) {
            const int ncol = gr.unit.ncol;
            if (gr.k0 < gr.k1) {
                wait(&acc_full[buf], aphase);
                __syncwarp();
                tc_fence_after();
                const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccCols;
                const float gs = F::kMx ? 1.0f : __ldg(p.gs + gr.unit.expert);
                for (int c0 = 0; c0 < ncol; c0 += 4) { // four tokens' columns at a time
                    uint32_t v[4][8];
                    int tok[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int cc = min(c0 + c, ncol - 1);
                        tok[c] = (int)s_tok[gr.unit.row0 + cc];
                        tmem_ld_32x32b_x8(trow + (!DOWN && p.dense ? tok[c] : cc) * kTerms, v[c]);
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c0 + c >= ncol)
                            break;
                        float s = 0.0f; // the smallest terms first
#pragma unroll
                        for (int j = kTerms - 1; j >= 0; --j)
                            s += __uint_as_float(v[c][j]);
                        const int row = gr.unit.row0 + c0 + c;
                        if constexpr (!F::kMx)
                            s *= gs * __ldg(DOWN ? p.sh.h_factor + row : p.sh.x_factor + tok[c]);
                        if constexpr (DOWN)
                            s_out[tok[c] * 128 + r] = fmaf(s, s_wt[row], s_out[tok[c] * 128 + r]);
                        else
                            s_out[(c0 + c) * 128 + r] = s; // gate rows 0..63, up rows 64..127
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&acc_empty[buf]);
                buf ^= 1;
                if (buf == 0)
                    aphase ^= 1;
            }
            if constexpr (!DOWN) {
                named_bar_sync(1, 128);
                const int f = et & 63;
                if (gr.first + f < p.F)
                    for (int c = et >> 6; c < ncol; c += 2) {
                        const float ga = s_out[c * 128 + f], up = s_out[c * 128 + 64 + f];
                        p.sh.h[(int64_t)(gr.unit.row0 + c) * p.F + gr.first + f] =
                            ga / (1.0f + __expf(-ga)) * up;
                    }
                named_bar_sync(1, 128);
            } else if (gr.last) {
                // this job's sums: y, or a split's share of it
                const int64_t col = (int64_t)gr.first * kDownRows + r;
                float *part = p.sh.partial +
                              ((int64_t)gr.first * p.splits + gr.split) * p.T * kDownRows + r;
                for (int t = 0; t < p.T; ++t) {
                    const float s = s_out[t * 128 + r];
                    s_out[t * 128 + r] = 0.0f;
                    if (p.splits > 1)
                        part[t * kDownRows] = s;
                    else if (col < p.H)
                        p.y[t * p.H + col] = __float2bfloat16_rn(s);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// y from the splits' sums, in split order; four columns a thread.
__global__ void __launch_bounds__(256)
    moe_sum_kernel(const float *partial, int splits, int T, int64_t H, __nv_bfloat16 *y)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = (int64_t)T * (H >> 2);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / (H >> 2), c = (i % (H >> 2)) * 4;
        const float *src = partial + ((c / kDownRows) * splits * T + t) * kDownRows + c % kDownRows;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < splits; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + (int64_t)k * T * kDownRows));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2 *>(y + t * H + c) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

template <typename K, typename... Args>
cudaError_t launch_after(K kernel, int grid, int threads, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class F, bool DOWN>
cudaError_t launch_gemm(MoeGemm g, const CUtensorMap &tmA, const CUtensorMap &tmB, cudaStream_t s)
{
    static std::once_flag flags[64];
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = cudaSuccess;
    std::call_once(flags[dev & 63], [&]() {
        e = cudaFuncSetAttribute(moe_gemm_kernel<F, DOWN>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int fixed = 2 * kSfRing * 2 * 128 * 4 * F::kAtoms + (DOWN ? g.T : kCols) * 128 * 4 +
                      9 * g.n_slots;
    const int stage = 16384 + g.b_rows * 128;
    const int fit = (kMaxSmem - fixed) / stage;
    g.stages = fit < kMaxStages ? fit : kMaxStages;
    return launch_after(moe_gemm_kernel<F, DOWN>, num_sms(), kThreads,
                        (size_t)g.stages * stage + fixed, s, tmA, tmB, g);
}

// CTAs per 128-row block of y.
int moe_splits(int64_t H)
{
    const int64_t s = num_sms() / ((H + kDownRows - 1) / kDownRows);
    return (int)(s < 1 ? 1 : s);
}

// The workspace: offsets of MoeShared's arrays for T tokens of k experts.
struct MoeWs {
    size_t x_codes, x_scales, x_factor, h, h_codes, h_scales, h_factor, units, counts, tok, wt,
        partial, total;
};

MoeWs moe_ws(int64_t T, int64_t k, int64_t F, int64_t H)
{
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) & ~(size_t)255;
        return o;
    };
    const size_t n = (size_t)T * (size_t)k, blocks = (size_t)((H + kDownRows - 1) / kDownRows);
    const int splits = moe_splits(H);
    MoeWs w;
    const size_t x_pitch = (size_t)(H / 16 + 15) / 16 * 16, h_pitch = (size_t)(F / 16 + 15) / 16 * 16;
    w.x_codes = take((size_t)T * kTerms * (size_t)H / 2);
    w.x_scales = take((size_t)T * kTerms * x_pitch);
    w.x_factor = take((size_t)T * 4);
    w.h = take(n * (size_t)F * 4);
    w.h_codes = take(n * kTerms * (size_t)F / 2);
    w.h_scales = take(n * kTerms * h_pitch);
    w.h_factor = take(n * 4);
    w.units = take(n * 4);
    w.counts = take(8);
    w.tok = take(n);
    w.wt = take(n * 4);
    w.partial = take(splits > 1 ? blocks * splits * (size_t)T * kDownRows * 4 : 0);
    w.total = at;
    return w;
}

template <class F>
cudaError_t launch_experts(MoeGemm g, const uint2 *x, const int *ids,
                           const float *weights, int k, int E, const uint8_t *up_codes,
                           const uint8_t *up_scales, const float *up_gs, const uint8_t *down_codes,
                           const uint8_t *down_scales, const float *down_gs, cudaStream_t s)
{
    constexpr bool NV = !F::kMx;
    // scale bytes of a term row: whole 16-byte pieces, so that every k-tile's lie inside
    g.sh.x_pitch = (g.H / F::kBlock + 15) / 16 * 16;
    g.sh.h_pitch = (g.F / F::kBlock + 15) / 16 * 16;
    g.b_rows = (g.T < kCols ? g.T : kCols) * kTerms;
    g.dense = g.T <= kCols;
    CUtensorMap up, down, xt, ht;
    const int64_t n = (int64_t)g.T * k;
    if (!make_fp4_codes_map(&up, up_codes, (int64_t)E * 2 * g.F, g.H, 64) ||
        !make_fp4_codes_map(&down, down_codes, (int64_t)E * g.H, g.F, 64) ||
        !make_fp4_codes_map(&xt, g.sh.x_codes, (int64_t)g.T * kTerms, g.H,
                            g.dense ? g.b_rows : kTerms) ||
        !make_fp4_codes_map(&ht, g.sh.h_codes, n * kTerms, g.F, g.b_rows))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_after(moe_prepare_kernel<NV>, g.T + 1, kPrepThreads,
                                 lists_smem(g.T, k, E), s, g.sh, x, ids, weights, g.T, k, E,
                                 g.H);
    if (e != cudaSuccess)
        return e;
    MoeGemm u = g, d = g;
    u.a_scales = up_scales;
    u.a_rows = (int64_t)E * 2 * g.F;
    u.gs = up_gs;
    d.a_scales = down_scales;
    d.a_rows = (int64_t)E * g.H;
    d.gs = down_gs;
    if ((e = launch_gemm<F, false>(u, up, xt, s)) != cudaSuccess)
        return e;
    if ((e = launch_after(moe_terms_kernel<NV>, (int)n, kTermThreads, (size_t)0, s, g.sh, g.F)) !=
        cudaSuccess)
        return e;
    if ((e = launch_gemm<F, true>(d, down, ht, s)) != cudaSuccess || g.splits == 1)
        return e;
    const int64_t need = ((int64_t)g.T * (g.H / 4) + 255) / 256, cap = (int64_t)num_sms() * 4;
    return launch_after(moe_sum_kernel, (int)(need < cap ? need : cap), 256, (size_t)0, s,
                        g.sh.partial, g.splits, g.T, g.H, g.y);
}

} // namespace

size_t moe_workspace_bytes(int64_t T, int64_t k, int64_t F, int64_t H)
{
    return moe_ws(T, k, F, H).total;
}

cudaError_t launch_moe_route(const void *x, const void *w, const float *bias, int64_t T, int64_t H,
                             int E, int k, int renorm, int *ids, float *weights, cudaStream_t s)
{
    RouteParams p{reinterpret_cast<const uint4 *>(x), reinterpret_cast<const uint4 *>(w), bias, T,
                  H, E, k, renorm, ids, weights};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((T + 7) / 8 * kRouteCluster), 1, 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_route_kernel, p);
}

cudaError_t launch_moe_experts(const void *x, int64_t T, int64_t H, int64_t F, int E, int k,
                               const int *ids, const float *weights, int mx,
                               const uint8_t *up_codes, const uint8_t *up_scales,
                               const float *up_gs, const uint8_t *down_codes,
                               const uint8_t *down_scales, const float *down_gs, void *y, void *ws,
                               cudaStream_t s)
{
    const MoeWs w = moe_ws(T, k, F, H);
    uint8_t *b = reinterpret_cast<uint8_t *>(ws);
    auto f32 = [&](size_t o) { return reinterpret_cast<float *>(b + o); };
    auto i32 = [&](size_t o) { return reinterpret_cast<int *>(b + o); };
    MoeGemm g{};
    g.sh = MoeShared{b + w.x_codes, b + w.x_scales, f32(w.x_factor), 0,
                     f32(w.h), b + w.h_codes, b + w.h_scales, f32(w.h_factor), 0,
                     reinterpret_cast<uint32_t *>(b + w.units), i32(w.counts), b + w.tok, f32(w.wt),
                     f32(w.partial)};
    g.T = (int)T;
    g.n_slots = (int)T * k;
    g.H = H;
    g.F = F;
    g.splits = moe_splits(H);
    g.blocks = (int)((H + kDownRows - 1) / kDownRows);
    g.y = reinterpret_cast<__nv_bfloat16 *>(y);
    g.status = device_status_ptr();
    if (!g.status)
        return cudaErrorInvalidValue;
    const uint2 *xv = reinterpret_cast<const uint2 *>(x);
    return mx ? launch_experts<FmtMxfp4>(g, xv, ids, weights, k, E, up_codes, up_scales, up_gs,
                                         down_codes, down_scales, down_gs, s)
              : launch_experts<FmtNvfp4>(g, xv, ids, weights, k, E, up_codes, up_scales, up_gs,
                                         down_codes, down_scales, down_gs, s);
}

} // namespace nvfp4
