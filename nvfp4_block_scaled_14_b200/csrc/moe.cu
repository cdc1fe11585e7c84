// moe.cu -- mixture-of-experts layer for a few tokens (decode batches) on sm_100a: the router and
// the experts' gated MLP on 4-bit weights.
//
// Router: z = x . Wr^T + bias, the k largest of each token's z (equal ones: the lower expert
// first), their softmax weights. Experts: y_t = sum_k w[t,k] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t))
// with e = ids[t,k]. With at most 64 tokens the cost is reading the met experts' weights once.
//
// The weights go to the FP4 tensor cores as they are stored. Those multiply FP4 by FP4 only, so an
// activation is split into eight FP4 terms (put_terms) and the eight products are added: the weights
// lose nothing and the activations at most 2^-22 of their block's largest value, while the terms cost
// the otherwise idle MMA eight columns a token.
// (Decoding the weights to f16 on the CUDA cores for mma.sync took 40-54 issue slots per 16 x 32
// codes, as long as HBM takes to deliver them, and ran at a quarter of it: 64 tokens, 64 experts of
// 2048 x 1024, top 8: 135 us.)
#include <mutex>
#include <type_traits>

#include "fp4_format.cuh"
#include "grid_exchange.cuh"
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
// Blocks of K whose loads a warp has under way: 114 registers, two CTAs an SM. Eight: 154, one CTA (4096
// tokens, 128 experts of 4096: 265 us instead of 162; 64 tokens 7.0 instead of 7.6). Three: 174 and 7.9 us.
constexpr int kRouteAhead = 4;

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

__device__ __forceinline__ void max_cluster_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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

// Close calls of a token: every expert that fewer than k others precede by more than tol, and that is
// within tol of another, gets its exact logit (products of bf16, and their sum, in fp64), and s_sel the
// k experts in order. s_list: [E], part: [128][8]. By the whole CTA; apart from the kernel, whose
// registers it would take.
__device__ __noinline__ void route_close(const RouteParams &p, int64_t tk, double tol, double *s_z,
                                         int *s_sel, int16_t *s_list, int *s_close, double *part)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t nvec = p.H >> 3;
    if (tid < 32)
        s_sel[tid] = -1;
    if (tid == 32)
        *s_close = 0;
    __syncthreads();
    if (tol > 0.0) // (else a row of zeros: the logits are exact)
        for (int e = tid; e < p.E; e += kRouteThreads) {
            const double z = s_z[e], hi = z + tol, lo = z - tol;
            int sure = 0, all = 0;
            for (int q = 0; q < p.E; ++q) {
                sure += s_z[q] > hi ? 1 : 0;
                all += s_z[q] >= lo ? 1 : 0;
            }
            if (z > -INFINITY && sure < p.k && all - sure > 1)
                s_list[atomicAdd(s_close, 1)] = (int16_t)e; // in any order
        }
    __syncthreads();
    const int listed = *s_close;
    for (int i0 = 0; i0 < listed; i0 += 128) {
        const int m = min(listed - i0, 128);
        for (int i = 0; i < m; ++i) {
            const uint4 *x = p.x + tk * nvec, *w = p.w + s_list[i0 + i] * nvec;
            double z = 0.0;
#pragma unroll 2
            for (int64_t c = tid; c < nvec; c += kRouteThreads) {
                const uint4 a = __ldg(x + c), b = __ldg(w + c);
                const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z = fma((double)__uint_as_float(u[j] << 16),
                            (double)__uint_as_float(v[j] << 16), z);
                    z = fma((double)__uint_as_float(u[j] & 0xFFFF0000u),
                            (double)__uint_as_float(v[j] & 0xFFFF0000u), z);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
            if (lane == 0)
                part[i * 8 + warp] = z;
        }
        __syncthreads();
        if (tid < m) {
            const int e = s_list[i0 + tid];
            double z = 0.0;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                z += part[tid * 8 + w];
            if (p.bias)
                z += (double)__ldg(p.bias + e);
            s_z[e] = z == z ? z : -INFINITY;
        }
        __syncthreads();
    }
    for (int e = tid; e < p.E; e += kRouteThreads) {
        const double z = s_z[e];
        int n = 0;
        for (int q = 0; q < p.E; ++q)
            n += (s_z[q] > z || (s_z[q] == z && q < e)) ? 1 : 0;
        if (n < p.k && z > -INFINITY)
            s_sel[n] = e;
    }
    __syncthreads();
}

// A cluster of 8 CTAs takes 8 tokens. Logits: 16 experts are the rows of bf16 MMAs, the tokens the
// columns; a CTA takes chunks of 16 experts (with few chunks, a slice of K too), its warps every
// eighth 32-wide block of K. Each block's 32 products are summed in fp32 by two MMAs and the blocks
// in fp64; two more MMAs sum the products' sizes, S. The logits go to the CTA that ranks the token:
// expert e is chosen if fewer than k experts precede it, counted by every thread at once. A block's two
// MMAs are off by a unit in the last place of the sum of its sizes each, 2^-22 S a logit in all, so two
// logits that are 2^-21 S apart (S: the token's largest) have the order of the exact ones. An expert
// that may be chosen and is closer to another gets its sum in fp64 throughout, and the count runs again
// (one token in 500 or so of 128 random experts of 4096).
// Bound by the latency of one round of loads (W is 1 MB at 128 experts of 4096) and of the cluster barrier.
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads, 2)
    moe_route_kernel(const __grid_constant__ RouteParams p)
{
    __shared__ double s_z[512];           // [slice][expert], then [expert]: this CTA's token
    __shared__ double s_part[8][16 * 8];  // [warp][expert][token]
    __shared__ float s_size[8][16 * 8];   // as s_part: sizes
    __shared__ uint32_t s_most[8];        // [slice]: bits of the largest size of this CTA's token
    __shared__ int s_sel[32];
    __shared__ int s_close;               // experts of s_list
    __shared__ int16_t s_list[512];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_ctarank();
    const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * 8;
    if (tid < 8)
        s_most[tid] = 0u;
    cluster_arrive(); // matched below: every CTA of the cluster runs before remote stores
    const int chunks = (p.E + 15) / 16;
    const int slices = chunks == 1 ? 8 : chunks == 2 ? 4 : chunks <= 4 ? 2 : 1;
    const int per = kRouteCluster / slices; // CTAs per slice of K
    const int slice = rank / per;
    const int64_t nvec = p.H >> 3;
    const int nblk = (int)(p.H >> 5);
    const int b0 = (int)((int64_t)nblk * slice / slices);
    const int b1 = (int)((int64_t)nblk * (slice + 1) / slices);
    const uint32_t zaddr = smem_u32(s_z), maddr = smem_u32(s_most);
    pdl_wait();
    const int64_t tok = t0 + g < p.T ? t0 + g : p.T - 1;
    for (int c = rank % per; c < chunks; c += per) {
        const uint4 *wa = p.w + (int64_t)min(c * 16 + g, p.E - 1) * nvec + t;
        const uint4 *wb = p.w + (int64_t)min(c * 16 + g + 8, p.E - 1) * nvec + t;
        const uint4 *xr = p.x + tok * nvec + t;
        double acc[4] = {0.0, 0.0, 0.0, 0.0};
        float size[4] = {};
#pragma unroll 1
        for (int b = b0 + warp; b < b1; b += 8 * kRouteAhead) {
            uint4 a[kRouteAhead], d[kRouteAhead], x[kRouteAhead];
#pragma unroll
            for (int i = 0; i < kRouteAhead; ++i)
                if (b + 8 * i < b1) {
                    a[i] = __ldg(wa + 4 * (b + 8 * i));
                    d[i] = __ldg(wb + 4 * (b + 8 * i));
                    x[i] = __ldg(xr + 4 * (b + 8 * i));
                }
#pragma unroll
            for (int i = 0; i < kRouteAhead; ++i) {
                if (b + 8 * i >= b1)
                    break;
                float f[4]; // lane t's k indices: its 8 values of the block, whatever their order
                mma_bf16_first(f, a[i].x, d[i].x, a[i].y, d[i].y, x[i].x, x[i].y);
                mma_bf16(f, a[i].z, d[i].z, a[i].w, d[i].w, x[i].z, x[i].w);
                constexpr uint32_t kAbs = kAbs16x2;
                mma_bf16(size, a[i].x & kAbs, d[i].x & kAbs, a[i].y & kAbs, d[i].y & kAbs,
                         x[i].x & kAbs, x[i].y & kAbs);
                mma_bf16(size, a[i].z & kAbs, d[i].z & kAbs, a[i].w & kAbs, d[i].w & kAbs,
                         x[i].z & kAbs, x[i].w & kAbs);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[j] += (double)f[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (g + (j >> 1) * 8) * 8 + 2 * t + (j & 1);
            s_part[warp][at] = acc[j];
            s_size[warp][at] = size[j];
        }
        __syncthreads();
        if (c < per)
            cluster_wait(); // (the first chunk) the other CTAs have started
        if (tid < 128) {
            const int e = c * 16 + (tid >> 3), j = tid & 7;
            double z = 0.0;
            float size = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                z += s_part[w][tid];
                size += s_size[w][tid];
            }
            if (e < p.E)
                st_cluster_f64(mapa_shared(zaddr + 8u * (uint32_t)(slice * p.E + e), (uint32_t)j),
                               z);
            size = fmaxf(size, __shfl_xor_sync(0xFFFFFFFFu, size, 8)); // of four experts; no NaN
            size = fmaxf(size, __shfl_xor_sync(0xFFFFFFFFu, size, 16));
            if (lane < 8)
                max_cluster_u32(mapa_shared(maddr + 4u * (uint32_t)slice, (uint32_t)j),
                                __float_as_uint(size));
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
    int open_ = 0; // experts that may be chosen at all
    for (int e0 = 0; e0 < p.E; e0 += kRouteThreads) {
        const int e = e0 + tid;
        double z = -INFINITY;
        if (e < p.E) {
            z = s_z[e];
            for (int q = 1; q < slices; ++q)
                z += s_z[q * p.E + e];
            if (p.bias)
                z += (double)__ldg(p.bias + e);
            z = z == z ? z : -INFINITY; // a NaN logit is never chosen
            s_z[e] = z;
        }
        open_ += __syncthreads_count(z > -INFINITY);
    }
    float most = 0.0f; // (of the slices' largest: not below the largest sum)
    for (int q = 0; q < slices; ++q)
        most += __uint_as_float(s_most[q]);
    const double tol = most < INFINITY ? (double)most * 0x1p-21 : 0.0; // (else fp32 holds no sums)
    // An expert's place, if those within tol below it precede it: its own if there are none, a later one
    // if there are. So the first place of a close call stays empty. parts threads share an expert's count
    // (E <= 64: 4, <= 128: 2).
    const int parts = p.E <= 64 ? 4 : p.E <= 128 ? 2 : 1;
    const int part = tid % parts;
    for (int e0 = 0; e0 < p.E; e0 += kRouteThreads / parts) {
        const int e = e0 + tid / parts;
        const double lo = e < p.E ? s_z[e] - tol : -INFINITY;
        int n = -1; // (itself)
        for (int q = part; q < p.E; q += parts)
            n += s_z[q] >= lo ? 1 : 0;
        for (int o = 1; o < parts; o <<= 1)
            n += __shfl_xor_sync(0xFFFFFFFFu, n, o) + 1;
        if (part == 0 && lo > -INFINITY && n < p.k)
            s_sel[n] = e;
    }
    __syncthreads();
    if (__any_sync(0xFFFFFFFFu, lane < min(p.k, open_) && s_sel[lane] < 0)) {
        __syncthreads(); // every warp has seen it
        route_close(p, tk, tol, s_z, s_sel, s_list, &s_close, &s_part[0][0]);
    }
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

constexpr int kTerms = 8; // FP4 terms of an activation: the rows of one swizzle atom
// Tokens of a column tile: 128 MMA columns. An expert with more tokens streams its weights once per
// tile (tiles of 8: 64 tokens, 64 experts of 2048 x 1024, top 8, 77 us where these took 67; two
// accumulators of larger tiles and the scales pass TMEM, one would fit).
constexpr int kCols = 16;
// Groups of four scale-feeder warps, in turn: one takes 750 cycles a k-tile (64 tokens: 71 us where
// two took 67), a third gives nothing (68.9 against 68.5).
constexpr int kFeeders = 2;
constexpr int kThreads = 32 * (7 + 4 * kFeeders);
constexpr int kUpRows = 64, kDownRows = 128; // rows of F, of H, per tile

// A column tile: up to kCols of the (expert, token) rows of one expert. Packed: 9 bits of expert, 11
// of row, 4 of columns - 1, 2 each of the tile's index among the expert's and of their number - 1.
struct MoeUnit {
    int expert, row0, ncol;
};

__device__ __forceinline__ uint32_t pack_unit(int expert, int row0, int ncol, int index, int of)
{
    return (uint32_t)expert | (uint32_t)row0 << 9 | (uint32_t)(ncol - 1) << 20 |
           (uint32_t)index << 24 | (uint32_t)(of - 1) << 26;
}

__device__ __forceinline__ MoeUnit unpack_unit(uint32_t u)
{
    return MoeUnit{(int)(u & 0x1FFu), (int)(u >> 9 & 0x7FFu), (int)(u >> 20 & 0xFu) + 1};
}

__device__ __forceinline__ int unit_index(uint32_t u) { return (int)(u >> 24 & 3u); }
__device__ __forceinline__ int unit_siblings(uint32_t u) { return (int)(u >> 26 & 3u) + 1; }
static_assert(kMoeMaxTokens <= 4 * kCols, "an expert's column tiles count in two bits");

// What the CTAs of one call share in the workspace. Rows: the (expert, token) pairs, in expert order.
struct MoeShared {
    // terms of the rows' x and h = silu(gate) * up, k-tile by k-tile: [rows][k-tiles][8 terms][128
    // bytes]. NVFP4's h lies there in fp32 first, whose 256 values of a k-tile take the same bytes.
    uint8_t *x_codes, *h_codes;
    uint8_t *x_scales, *h_scales; // the terms' block scales (first term's): [rows][k-tiles][SB bytes]
    int64_t x_kt, h_kt;           // k-tiles of a row
    uint32_t *x_max, *h_max;      // [rows] (NVFP4): bits of the row's largest magnitude
    float *partial;               // [128-row blocks of y][splits][T][128]
};

// ---- lists and terms ----------------------------------------------------------------------

// The (expert, token) pairs that the ids name, in expert order, as rows: the row's token and weight
// (an expert that a token names twice gets one row with both weights), and the column tiles. ids
// outside [0, E) name no expert. In the CTA's shared memory.
struct MoeLists {
    float *wt;       // [rows]
    uint32_t *units; // [column tiles]
    int *counts;     // column tiles, rows
    uint8_t *tok;    // [rows]
};

// Built by the whole CTA. tmp: 12 E + 6 T k bytes.
__device__ __forceinline__ void build_lists(const MoeLists &l, const int *ids, const float *weights,
                                            int T, int k, int E, uint8_t *tmp)
{
    uint32_t *mask = reinterpret_cast<uint32_t *>(tmp); // [E][2]: the expert's tokens
    int *base = reinterpret_cast<int *>(mask + 2 * E);  // [E]: its first row
    float *s_w = reinterpret_cast<float *>(base + E);
    int16_t *s_ids = reinterpret_cast<int16_t *>(s_w + T * k);
    const int n = T * k, tid = threadIdx.x;
    auto count = [&](int e) { return __popc(mask[2 * e]) + __popc(mask[2 * e + 1]); };
    const int id = tid < n ? __ldg(ids + tid) : -1; // on their way while the masks are cleared
    const float wt = tid < n ? __ldg(weights + tid) : 0.0f;
    for (int i = tid; i < 2 * E; i += kThreads)
        mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int e = i == tid ? id : __ldg(ids + i), t = i / k;
        const bool on = e >= 0 && e < E;
        s_w[i] = i == tid ? wt : __ldg(weights + i);
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
            l.counts[0] = u0;
            l.counts[1] = r0;
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
                l.units[u0++] = pack_unit(e, r0 + c0, min(kCols, c - c0), c0 / kCols,
                                          (c + kCols - 1) / kCols);
            r0 += c;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int e = s_ids[i], t = i / k;
        if (e < 0)
            continue;
        bool first = true; // of the token's slots that name e
        float w = 0.0f;
        for (int s = t * k; s < (t + 1) * k; ++s)
            if (s_ids[s] == e) {
                first = first && s >= i;
                w += s_w[s];
            }
        if (first) {
            const uint32_t *m = mask + 2 * e;
            const int before = t < 32 ? __popc(m[0] & ((1u << t) - 1u))
                                      : __popc(m[0]) + __popc(m[1] & ((1u << (t - 32)) - 1u));
            const int row = base[e] + before;
            l.tok[row] = (uint8_t)t;
            l.wt[row] = w;
        }
    }
}

constexpr int kTileBytes = kTerms * 128; // a row's terms of a k-tile

// Activations as kTerms FP4 terms: the digits of a fixed-point number to base 8, X = v / 2^(E - 21),
// E the exponent of the block's largest value (32 values for MXFP4, 16 for NVFP4). -4 .. 3 are E2M1
// values, and with digits of that range the 3-bit fields of X + 4 (1 + 8 + 64 + ...) are the digits
// plus 4; one byte permute looks up four codes. Term j stands for digit * 2^(E - 3j). Off by at most
// half a unit: 2^-22 of the block's largest value (and 2^-128, where E < -106 is taken as -106).
//   MXFP4: term j's scale is 2^(E - 3j). Only 2^E is stored.
//   NVFP4: E4M3 holds the powers 2^8 .. 2^-9 only. Every term has the block's scale 2^(8 - (R - E)), R
//     the exponent of the row's largest value; the sums of term j's column are multiplied by
//     2^(R - 8 - 3j) instead, which is the same for the whole row (term_sum, row_factor). Blocks below
//     2^-17 of the row's largest value are taken at that exponent: off by 2^-39 of the row's largest.
//     (The eight scales spread over E4M3's range, one exponent a row, left 2^-18 of it.)
// Each term as the E2M1 rounding of what the ones before leave, at the best scale for that (a block
// maximum and a conversion both ways a term), took the 512 x 1024 values of 64 tokens 10 us, against 2.
// A NaN or an infinity: the block's scale is NaN (MXFP4), or the row's factor is (NVFP4), and so the
// row's results are.
//
// v: values c0 .. c0 + 7 of a row of `cols`, lane i's c0 being lane 0's + 8 i in aligned groups of four
// lanes; zeros behind the row's end. codes, scales: the row's; row_e: row_exponent of it (NVFP4). Codes
// behind the row's end are left: the weights are zero there. Called by whole warps.
template <bool NV>
__device__ __forceinline__ void put_terms(const float (&v)[8], int64_t c0, int64_t cols,
                                          uint8_t *codes, uint8_t *scales, int64_t kt, bool live,
                                          uint32_t row_e)
{
    constexpr float kMagic = 12582912.0f; // 1.5 * 2^23: the sum's low bits are the rounded integer
    constexpr uint32_t kDigits = 044444444u;
    constexpr int kBlock = NV ? 16 : 32, kPerTile = 256 / kBlock;
    const bool on = live && c0 < cols;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if constexpr (!NV)
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    uint32_t b = max(m >> 23, 21u); // E + 127, MXFP4's scale byte; 255: NaN or infinity
    const bool bad = b == 255u;
    uint32_t byte = b;
    if constexpr (NV) {
        b = min(max(b, row_e - min(row_e, 17u)), row_e);
        const uint32_t d = row_e - b; // E4M3 of 2^(8 - d)
        byte = d < 15u ? (15u - d) << 3 : 8u >> (d - 14u);
    } else {
        b = bad ? 254u : b;
    }
    const float unit = __uint_as_float((275u - b) << 23); // 2^(21 - E)
    if (live && c0 % kBlock == 0 && c0 / kBlock < kt * kPerTile)
        scales[c0 / kBlock] = on ? (uint8_t)byte : NV ? (uint8_t)0 : (uint8_t)21;
    uint32_t p[2][4]; // two values' codes, a byte a digit: digits 7..4, 3..0
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t u = __float_as_uint(fmaf(v[i], unit, kMagic)) - __float_as_uint(kMagic);
        u = bad ? kDigits : u + kDigits;
        u += (u & 0xFFF000u) * 15u; // 3-bit fields to nibbles: halves to 16 bits,
        u += (u & 0x0FC00FC0u) * 3u; // six bits to bytes,
        u += u & 0x38383838u;
        const uint32_t lo = i & 1 ? 0xA0C0D0E0u : 0x0A0C0D0Eu, hi = i & 1 ? 0x50402000u : 0x05040200u;
        const uint32_t a = __byte_perm(lo, hi, u), b4 = __byte_perm(lo, hi, u >> 16);
        p[0][i >> 1] = i & 1 ? p[0][i >> 1] | a : a;
        p[1][i >> 1] = i & 1 ? p[1][i >> 1] | b4 : b4;
    }
    codes += (c0 >> 8) * kTileBytes + ((c0 & 255) >> 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) { // four bytes of four words -> four words of one digit each
        const uint32_t t0 = __byte_perm(p[h][0], p[h][1], 0x5140);
        const uint32_t t1 = __byte_perm(p[h][2], p[h][3], 0x5140);
        const uint32_t t2 = __byte_perm(p[h][0], p[h][1], 0x7362);
        const uint32_t t3 = __byte_perm(p[h][2], p[h][3], 0x7362);
        const uint32_t w[4] = {__byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632),
                               __byte_perm(t2, t3, 0x5410), __byte_perm(t2, t3, 0x7632)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (on)
                *reinterpret_cast<uint32_t *>(codes + (7 - 4 * h - i) * 128) = w[i];
    }
}

// Scale bytes of term j of eight, four of a word of the first term's (MXFP4).
__device__ __forceinline__ uint32_t mx_term_scales(uint32_t first, int j)
{
    return first - 0x03030303u * (uint32_t)j;
}

// A token's product from its eight columns' sums, the smallest terms first. (NVFP4: in units of
// row_factor; term j counts 8^-j, an exact factor.)
template <bool NV> __device__ __forceinline__ float term_sum(const uint32_t (&v)[kTerms])
{
    float s = 0.0f;
#pragma unroll
    for (int j = kTerms - 1; j >= 0; --j)
        s = NV ? fmaf(s, 0.125f, __uint_as_float(v[j])) : s + __uint_as_float(v[j]);
    return s;
}

// R + 127 of a row with the largest magnitude m (bits), and what its first column is multiplied by,
// 2^(R - 8) (NaN where m is NaN or infinite).
__device__ __forceinline__ uint32_t row_exponent(uint32_t m)
{
    return min(max(m >> 23, 21u), 254u);
}

__device__ __forceinline__ float row_factor(uint32_t m)
{
    return __uint_as_float(m >= 0x7F800000u ? 0x7FC00000u : (row_exponent(m) - 8u) << 23);
}

// A CTA's share of the rows' 256-value chunks, one warp each.
struct MoeChunks {
    uint32_t per, first, last; // (32 bits, as in MoeStart)

    __device__ __forceinline__ MoeChunks(int rows, int64_t cols)
    {
        per = (uint32_t)((cols + 255) >> 8);
        const uint32_t n = (uint32_t)rows * per, q = n / gridDim.x, r = n % gridDim.x;
        first = blockIdx.x * q + min(blockIdx.x, r);
        last = first + q + (blockIdx.x < r ? 1u : 0u);
    }
};

// Terms of the CTA's chunks, by all warps but warp 0; load(row, c0, v): eight values; row_e(row):
// the row's exponent (NVFP4). A chunk's values may lie where its terms go.
template <bool NV, typename Load, typename RowE>
__device__ __forceinline__ void write_terms(const MoeChunks &ch, int64_t cols, uint8_t *codes,
                                            uint8_t *scales, int64_t kt, int warp, Load load,
                                            RowE row_e)
{
    const int lane = threadIdx.x & 31;
    if (warp == 0)
        return;
    for (uint32_t i = ch.first + warp - 1; i < ch.last; i += kThreads / 32 - 1) {
        const int64_t row = i / ch.per, c0 = (int64_t)(i - (uint32_t)row * ch.per) * 256 + lane * 8;
        float v[8] = {};
        if (c0 < cols)
            load(row, c0, v);
        __syncwarp(); // every lane has its values
        put_terms<NV>(v, c0, cols, codes + row * kt * kTileBytes,
                      scales + row * kt * (NV ? 16 : 8), kt, true, row_e(row));
    }
}

// ---- products -----------------------------------------------------------------------------

constexpr uint32_t kWaitLimit = kMoeWaits.wait_limit;
constexpr int kSfAhead = 2;  // a feeder group's k-tiles whose scales are on their way
constexpr int kSfRing = kSfAhead + 1;
constexpr int kMaxStages = 8;
constexpr int kMaxSmem = 232448 - 1024;

struct MoeGemm {
    MoeShared sh;
    const uint4 *x; // bf16 [T x H]
    const int *ids;
    const float *weights;
    int T, k, E;
    int64_t H, F;
    const uint8_t *up_scales, *down_scales; // linear
    const float *up_gs, *down_gs;           // [E] (NVFP4)
    int stages, stage_bytes; // operand ring
    int box;                 // tokens of a TMA box of terms
    int splits, blocks;      // down: CTAs per 128-row block of y, blocks
    __nv_bfloat16 *y;
    GridBarrier *barrier;
    int *status;
    MoeWaits waits;
};

// A run of k-tiles of one tile, whose sums stay in one accumulator.
struct MoeGroup {
    MoeUnit unit;
    int k0, k1;       // k-tiles (none: an empty job)
    int first;        // the tile's first column of h (gate/up) or of y (down)
    int split;
    bool last;        // down: the job's last run
};

// Where a CTA's share begins, computed once (in shared memory). 32 bits hold the tile counts: the
// weights' stacked rows are below 2^31, and an expert has at most four column tiles.
struct MoeStart {
    int up_kt, up_tiles, down_kt; // k-tiles of H, 64-column tiles of F, k-tiles of F
    int runs, u, tile, j;         // gate/up: runs of this CTA; the first one's expert's column tiles
                                  // (from u on), 64-column tile, and which of the former
    uint32_t q, r;                // down: (column tile, k-tile) pairs of a split, splits with one more

    __device__ __forceinline__ uint32_t cut(uint32_t split) const
    {
        return split * q + min(split, r);
    }
};

// The groups of a CTA, in order; every role of the CTA walks them by itself. Gate/up: a run of the
// flat list of (expert, 64 columns of F, column tile), so that an expert's column tiles take the
// weights one after the other, from L2 after the first (64 tokens on each of 8 experts of 4096 x 14336:
// 552 -> 512 us against column tile by column tile; where L2 holds the weights there is no
// difference). Down: jobs (128-row block of y, split), whose run of
// the flat list of (column tile, k-tile) pairs is cut at the column tiles.
template <bool DOWN> struct MoeWalk {
    const MoeGemm &p;
    const uint32_t *units; // in shared memory
    const MoeStart &st;
    int rest, u, tile; // runs (gate/up) or k-tiles (down) left, column tile, tile of it
    int j;             // gate/up: column tile u + j of the expert's
    int job;           // down

    __device__ __forceinline__ MoeWalk(const MoeGemm &q, const uint32_t *list, const MoeStart &s)
        : p(q), units(list), st(s)
    {
        rest = DOWN ? -1 : s.runs;
        u = s.u;
        tile = s.tile;
        j = s.j;
        job = (int)blockIdx.x - (int)gridDim.x;
    }

    __device__ __forceinline__ bool next(MoeGroup &g)
    {
        if constexpr (!DOWN) {
            if (rest == 0)
                return false;
            --rest;
            const uint32_t unit = units[u + j];
            g.unit = unpack_unit(unit);
            g.first = tile * kUpRows;
            g.k0 = 0;
            g.k1 = st.up_kt;
            if (++j == unit_siblings(unit)) {
                if (++tile == st.up_tiles) {
                    tile = 0;
                    u += j;
                }
                j = 0;
            }
        } else {
            if (rest <= 0) {
                job += gridDim.x;
                if (job >= p.blocks * p.splits)
                    return false;
                const uint32_t split = (uint32_t)job % (uint32_t)p.splits;
                const uint32_t a = st.cut(split);
                rest = (int)(st.cut(split + 1) - a);
                u = (int)(a / (uint32_t)st.down_kt);
                tile = (int)(a % (uint32_t)st.down_kt);
            }
            g.split = (int)((uint32_t)job % (uint32_t)p.splits);
            g.first = (int)((uint32_t)job / (uint32_t)p.splits) * kDownRows;
            if (rest == 0) {
                g.unit = MoeUnit{0, 0, 0};
                g.k0 = g.k1 = 0;
                g.last = true;
                return true;
            }
            g.unit = unpack_unit(units[u]);
            g.k0 = tile;
            g.k1 = min(tile + rest, st.down_kt);
            rest -= g.k1 - g.k0;
            ++u;
            tile = 0;
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

// 128 rows' scale bytes (SB a row at `sm`; MXFP4: less `less`; SHARE: eight rows have one row of
// bytes) -> the TMEM columns of F::kAtoms atoms, this warp's lane quarter: lane r's word i of an atom
// is row r + 32 i's.
template <class F, bool SHARE = false>
__device__ __forceinline__ void feed_rows(const uint8_t *sm, uint32_t tcol, int lane,
                                          uint32_t less = 0u)
{
    constexpr int SB = 4 * F::kAtoms;
    uint32_t r[4 * F::kAtoms];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F::kMx) {
            const uint2 v = *reinterpret_cast<const uint2 *>(sm + (lane + 32 * i) * SB);
            r[i] = v.x - less;
            r[4 + i] = v.y - less;
        } else {
            const int row = lane + 32 * i;
            const uint4 v = *reinterpret_cast<const uint4 *>(sm + (SHARE ? row >> 3 : row) * SB);
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

// A scale feeder thread's row: its scale bytes of every kFeeders-th k-tile, from `first` on (k-tiles
// count on from one run into the next), into a ring of kSfRing slots of 128 rows of weights and 128 of
// terms (NVFP4: 16 of tokens, whose eight terms share their scales).
template <class F, bool DOWN> struct ScaleRow {
    static constexpr int SB = 4 * F::kAtoms; // bytes of a row and k-tile
    static constexpr int kRowsPerToken = F::kMx ? kTerms : 1;
    static constexpr int kSlot = (128 + kCols * kRowsPerToken) * SB;
    const MoeGemm &p;
    MoeWalk<DOWN> walk;
    uint32_t ring; // this row's slot 0
    int r, srow, slot;
    int kt, kend = 0;
    bool more = true, a_on = false, b_on = false;
    const uint8_t *asrc, *bsrc;

    __device__ __forceinline__ ScaleRow(const MoeGemm &q, const uint32_t *units, const MoeStart &st,
                                        int row, uint32_t ring_row, int first, int first_slot)
        : p(q), walk(q, units, st), ring(ring_row), r(row), slot(first_slot), kt(first)
    {
        srow = (int)((DOWN ? p.F : p.H) / F::kBlock);
    }

    __device__ __forceinline__ static void zero(uint32_t dst)
    {
#pragma unroll
        for (int i = 0; i < SB; i += 4)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + i), "r"(0u) : "memory");
    }

    // The next k-tile's bytes (of the weights, of the terms), as one cp.async group.
    __device__ __forceinline__ void load(bool weights, bool terms)
    {
        while (more && kt >= kend) {
            MoeGroup g;
            more = walk.next(g);
            if (!more)
                break;
            kt += g.k0 - kend;
            kend = g.k1;
            if (kt >= kend)
                continue;
            // rows of the stacked weights; gate/up: 64 of gate, the same of up
            const int at = g.first + (DOWN ? r : r & 63);
            const int64_t row = DOWN ? g.unit.expert * p.H + at
                                     : (2 * g.unit.expert + (r >> 6)) * p.F + at;
            a_on = at < (DOWN ? p.H : p.F);
            asrc = (DOWN ? p.down_scales : p.up_scales) + (a_on ? row * srow + (int64_t)kt * SB : 0);
            const int token = r / kRowsPerToken;
            b_on = token < g.unit.ncol; // of the column tile
            bsrc = (DOWN ? p.sh.h_scales : p.sh.x_scales) +
                   ((int64_t)(g.unit.row0 + token) * (DOWN ? p.sh.h_kt : p.sh.x_kt) + kt) * SB;
        }
        if (more) {
            const uint32_t dst = ring + slot * kSlot;
            if (weights) {
                if (!a_on)
                    zero(dst);
                else if (srow % SB == 0) // every piece of a row is whole and aligned
                    cp_async<SB>(dst, asrc);
                else
                    fetch_scales_general<SB>(dst, asrc, min(SB, srow - kt * SB));
            }
            if (terms && b_on) // (the MMA reads no other columns)
                cp_async<SB>(dst + 128 * SB, bsrc);
            asrc += a_on ? kFeeders * SB : 0;
            bsrc += kFeeders * SB;
            kt += kFeeders;
            slot = slot + 1 == kSfRing ? 0 : slot + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// Four columns of y.
__device__ __forceinline__ void put_y(__nv_bfloat16 *y, const float4 &v)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(y) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
}

// The experts in one cooperative launch, one CTA per SM, five phases between grid barriers (a launch
// of its own for each cost 3 to 4 us more):
//   lists of the (expert, token) rows (every CTA its own) and the rows' terms of x;
//   gate/up products and, for MXFP4, the terms of h, whose blocks lie in one tile;
//   terms of h, for NVFP4, whose blocks' scales are relative to their row's largest value;
//   down products;
//   the splits' sums of y (where a block of y is shared by several CTAs).
// Products, on the FP4 tensor cores: 128 weight rows are the M side of block-scaled MMAs, eight term
// rows of each token of a column tile the N side (8..128 columns), so the weights go from HBM to the
// tensor cores as they are stored and the sum of a token's eight columns is the product with its value
// to 2^-22 of the largest of a block. Roles:
//   warp 0       TMA producer of the weights: per 256-wide k-tile one box of 128 rows (the next
//                phase's first stages before the barriers);
//   warp 14      TMA producer of the term rows: a box per four tokens of the column tile;
//   warps 6..13  scale feeders, two groups in turn: the rows' linear scale bytes to shared memory by
//                cp.async ahead of time, then to the stage's TMEM columns in the MMA's layout (one
//                group takes 750 cycles for that);
//   warp 1       MMA issuer; accumulators alternate between two TMEM buffers, so that a tile's
//                epilogue overlaps the next tile's MMAs;
//   warps 2..5   epilogue. Gate/up: a tile is 64 gate rows and the same 64 up rows; they meet in
//                shared memory and silu(gate) * up, in fp32, is split into terms or (NVFP4) goes to
//                the workspace. Down: the weighted sums of every column tile are added to [T][128]
//                sums in shared memory, which go to y or, split by split, to the workspace.
// A stage's bytes and scales complete one barrier, and the MMAs that have read them another.
// Measured, with the router, ids and inputs new each call: 64 tokens, 64 MXFP4 experts of 2048 x 1024,
// top 8: 63 us (214 MB of met weights: 3.4 TB/s); 16 tokens, 28 of 32 NVFP4 experts of 4096 x 1280, top
// 4: 69 us; one token, 6 experts of 2048 x 1408: 25 us. Of the 64 tokens' 52 us from this kernel's
// start to its end, gate/up take 22 to 25 (22 at the copy rate), down 13 to 14 (11), the rest are lists
// (3), terms (2.5), three barriers with the wait for the slowest CTA (10) and the sums. Products are
// bound by HBM and by the roles' latency
// together: a k-tile's 16 KB take 700 cycles of an SM's share, and the MMA warp's step (a completed
// wait is 95 cycles, four MMAs and a commit 300) leaves little of that; with the weights of eight
// experts for all, which L2 holds, the whole call took 60 us where it took 65, and separate rings for weights and
// terms, with a second wait and commit a step, took 77 where one took 67. So a role is a warp of its own
// with few instructions a step, and in a group
// of warps one polls while the others sleep at a named barrier. Waits are bounded. The first that gives
// up tells the CTA (s_dead) and the status word: no further tiles are copied and no stage completes any
// more, each other role stops waiting once one wait of its own has run out or at the next grid barrier,
// which the CTA does not enter any more, so that a call ends after about one limit.
template <class F>
__global__ void __launch_bounds__(kThreads, 1)
    moe_experts_kernel(const __grid_constant__ CUtensorMap tmUp,
                       const __grid_constant__ CUtensorMap tmDown,
                       const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmH, const MoeGemm p)
{
    constexpr bool NV = !F::kMx;
    constexpr int SB = 4 * F::kAtoms;          // scale bytes of a row and k-tile
    constexpr int kSfRows = ScaleRow<F, false>::kSlot;
    constexpr uint32_t kAccCols = 128, kSfCol = 2 * kAccCols, kSlotCols = 32;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_counts[2];
    __shared__ uint32_t s_max[kMoeMaxTokens];
    __shared__ MoeStart s_start;
    __shared__ volatile int s_dead; // a wait of this CTA gave up
    const int tid = threadIdx.x, lane = tid & 31;
    // the same in every lane, and known to be: the roles' loops then run on uniform registers
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const bool misaligned = (smem_u32(smem) & 1023u) != 0; // the same for every CTA
    if (misaligned) {
        if (tid == 0)
            atomicExch(p.status, (int)NVFP4_ERR_CUDA);
        return;
    }
    const int stage_bytes = p.stage_bytes;
    uint8_t *sf_ring = smem + p.stages * stage_bytes;
    float *s_out = reinterpret_cast<float *>(sf_ring + kFeeders * kSfRing * kSfRows);
    MoeLists l;
    l.wt = s_out + (p.T > kCols ? p.T : kCols) * 128;
    l.units = reinterpret_cast<uint32_t *>(l.wt + p.T * p.k);
    l.tok = reinterpret_cast<uint8_t *>(l.units + p.T * p.k);
    l.counts = s_counts;
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
        s_dead = 0;
    }
    if (tid == kThreads - 1) {
        tma_prefetch_desc(&tmUp);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmDown);
        tma_prefetch_desc(&tmH);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait(); // the ids, the activations
    for (int64_t i = blockIdx.x * kThreads + tid; i < p.T * (p.H >> 6); i += gridDim.x * kThreads)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.x + i * 8)); // while the lists are built

    bool dead = false; // this thread waits no more
    auto give_up = [&]() {
        dead = true;
        s_dead = 1;
        atomicExch(p.status, (int)NVFP4_ERR_TIMEOUT);
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, p.waits.wait_limit))
            give_up();
    };
    // Every CTA's writes so far are visible to every CTA, to its TMA loads too. Warp 0 has weights on
    // their way meanwhile, which its fences would wait for; it has written nothing and reads nothing
    // that others write.
    auto grid_sync = [&]() {
        if (warp != 0)
            asm volatile("fence.proxy.async;" ::: "memory");
        __syncthreads();
        // (A dead CTA stays away: its arrival would complete, for CTAs still polling, the barrier that
        // it gave up at.)
        if (tid == 32 && !s_dead && (int)blockIdx.x != p.waits.absent &&
            !grid_barrier_sync(p.barrier, (int)gridDim.x, (int)blockIdx.x, p.waits.barrier_limit))
            give_up();
        __syncthreads();
        dead = s_dead != 0;
        if (warp != 0)
            asm volatile("fence.proxy.async;" ::: "memory");
    };

    build_lists(l, p.ids, p.weights, p.T, p.k, p.E, smem);
    if (tid == 32) { // (the counts are there since the lists' last barrier)
        MoeStart st;
        st.up_kt = (int)((p.H + 255) >> 8);
        st.down_kt = (int)((p.F + 255) >> 8);
        st.up_tiles = (int)((p.F + kUpRows - 1) / kUpRows);
        const uint32_t n = (uint32_t)s_counts[0] * (uint32_t)st.up_tiles, g = gridDim.x;
        const uint32_t q = n / g, r = n % g, b = blockIdx.x; // the first r CTAs have one more
        const uint32_t i = b * q + min(b, r);
        st.runs = (int)(q + (b < r ? 1u : 0u));
        st.u = st.tile = st.j = 0;
        if (st.runs > 0) {
            const uint32_t at = i / (uint32_t)st.up_tiles, unit = l.units[at];
            st.u = (int)at - unit_index(unit);
            const uint32_t in = i - (uint32_t)st.u * (uint32_t)st.up_tiles;
            st.tile = (int)(in / (uint32_t)unit_siblings(unit));
            st.j = (int)(in % (uint32_t)unit_siblings(unit));
        }
        const uint32_t m = (uint32_t)s_counts[0] * (uint32_t)st.down_kt;
        st.q = m / (uint32_t)p.splits;
        st.r = m % (uint32_t)p.splits;
        s_start = st;
    }
    fence_proxy_async_smem(); // the lists' temporaries lay where TMA writes next
    __syncthreads();
    const int n_rows = s_counts[1];

    // ---- the roles' state, kept across the phases -----------------------------------------------
    int stage = 0, buf = 0;
    uint32_t phase = 0, aphase = 0;
    auto next_stage = [&]() {
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
        }
    };
    const int group = warp >= 6 && warp < 6 + 4 * kFeeders ? (warp - 6) >> 2 : 0; // a feeder's
    int rslot = 0, turn = group; // k-tiles until the group's next one
    uint8_t *my_ring = sf_ring + group * kSfRing * kSfRows;
    const int feed_row = (tid - 192) & 127; // a feeder thread's row
    const uint32_t ring_row = smem_u32(my_ring) + feed_row * SB;

    // The weights' tiles of a phase's k-tiles `skip` .. `count` - 1 (warp 0).
    auto load_weights = [&](auto down, int skip, int count) -> int {
        constexpr bool DOWN = decltype(down)::value;
        MoeWalk<DOWN> walk(p, l.units, s_start);
        MoeGroup gr;
        int n = 0;
        const CUtensorMap *tm = DOWN ? &tmDown : &tmUp;
        while (n < count && walk.next(gr)) {
            const int z = DOWN ? gr.unit.expert : 2 * gr.unit.expert; // gate's rows, then up's
            for (int kt = gr.k0; kt < gr.k1 && n < count; ++kt, ++n) {
                if (n < skip)
                    continue;
                uint64_t *bar = &full_bar[stage];
                wait(&empty_bar[stage], phase ^ 1);
                dead = __any_sync(0xFFFFFFFFu, s_dead != 0);
                if (dead)
                    return n;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, 16384u);
                    tma_load_3d(smem + stage * stage_bytes, tm, bar, kt * 128, gr.first, z);
                }
                next_stage();
            }
        }
        return n;
    };

    // What a phase can request before the barrier ahead of it: the first stages' weights and their
    // scales.
    int ahead = 0;
    auto start = [&](auto down) {
        constexpr bool DOWN = decltype(down)::value;
        if (warp == 0) {
            ahead = load_weights(down, 0, p.stages);
        } else if (warp >= 6 && warp < 6 + 4 * kFeeders) {
            named_bar_sync(3 + group, 128); // the ring's last rows have been read
            ScaleRow<F, DOWN> row(p, l.units, s_start, feed_row, ring_row, turn, rslot);
#pragma unroll 1
            for (int i = 0; i < kSfAhead; ++i)
                row.load(true, false);
        }
    };

    // One phase of products, after its start().
    auto products = [&](auto down) {
        constexpr bool DOWN = decltype(down)::value;
        MoeWalk<DOWN> walk(p, l.units, s_start);
        MoeGroup gr;
        if (warp == 0) {
            load_weights(down, ahead, 0x7FFFFFFF);
        } else if (warp == 6 + 4 * kFeeders) {
            // ------------------------------- the term rows' TMA producer --------------------
            const CUtensorMap *tm = DOWN ? &tmH : &tmX;
            while (walk.next(gr)) {
                const int row = gr.unit.row0 + lane * p.box;
                const int n = (gr.unit.ncol + p.box - 1) / p.box;
                const uint32_t bytes = (uint32_t)(n * p.box * kTileBytes);
                for (int kt = gr.k0; kt < gr.k1 && !dead; ++kt) {
                    uint64_t *bar = &full_bar[stage];
                    wait(&empty_bar[stage], phase ^ 1);
                    dead = __any_sync(0xFFFFFFFFu, s_dead != 0);
                    if (dead)
                        break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (lane < n)
                        tma_load_3d(smem + stage * stage_bytes + 16384 + lane * p.box * kTileBytes,
                                    tm, bar, 0, kt * kTerms, row);
                    __syncwarp();
                    next_stage();
                }
            }
        } else if (warp >= 6) {
            // ------------------------------- scale feeders ----------------------------------
            const int q = warp & 3;                // lane quarter of TMEM
            ScaleRow<F, DOWN> row(p, l.units, s_start, feed_row, ring_row, turn, rslot);
#pragma unroll 1
            for (int i = 0; i < kSfAhead; ++i)
                row.load(false, true); // (the weights' are on their way since before the barrier)
            const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + kSfCol;
            while (walk.next(gr)) {
                for (int kt = gr.k0; kt < gr.k1; ++kt) {
                    if (turn > 0) {
                        --turn;
                        next_stage();
                        continue;
                    }
                    turn = kFeeders - 1;
                    asm volatile("cp.async.wait_group %0;" ::"n"(kSfAhead - 1) : "memory");
                    if (q == 2) // one warp of the group polls, the others sleep at the barrier
                        wait(&empty_bar[stage], phase ^ 1);
                    named_bar_sync(3 + group, 128); // the rows are here, the last ones read
                    const bool live = s_dead == 0;
                    tc_fence_after();
                    const uint8_t *src = my_ring + rslot * kSfRows;
                    feed_rows<F>(src, tbase + stage * kSlotCols, lane);
                    if constexpr (F::kMx) // row r: term r % 8
                        feed_rows<F>(src + 128 * SB, tbase + stage * kSlotCols + 16, lane,
                                     mx_term_scales(0u, 0) - mx_term_scales(0u, lane & 7));
                    else // row r: token r / 8
                        feed_rows<F, true>(src + 128 * SB, tbase + stage * kSlotCols + 16, lane);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    // (once dead, the stage may still lack bytes of its last use: no arrival beyond)
                    if (lane == 0 && live)
                        mbar_arrive(&full_bar[stage]);
                    row.load(true, true);
                    rslot = rslot + 1 == kSfRing ? 0 : rslot + 1;
                    next_stage();
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else if (warp == 1) {
            // ------------------------------- MMA issuer -------------------------------------
            const uint64_t desc0 = smem_desc(smem_u32(smem), 16, 1024, kLayoutSwizzle128B);
            while (walk.next(gr)) {
                if (gr.k0 == gr.k1)
                    continue;
                const uint32_t idesc = F::kIdesc | (1u << 7) | (1u << 10) |
                                       ((uint32_t)gr.unit.ncol << 17) | (8u << 24); // N = 8 ncol
                const uint32_t acc = tmem + buf * kAccCols;
                wait(&acc_empty[buf], aphase ^ 1);
                uint32_t add = 0u;
                for (int kt = gr.k0; kt < gr.k1; ++kt) {
                    wait(&full_bar[stage], phase);
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
                    next_stage();
                }
                if (elect_one())
                    tc_commit(&acc_full[buf]);
                __syncwarp();
                buf ^= 1;
                if (buf == 0)
                    aphase ^= 1;
            }
        } else {
            // ------------------------------- epilogue (warps 2..5) --------------------------
            const int q = warp & 3, r = q * 32 + lane; // this thread's accumulator row
            const int et = tid - 64;
            [[maybe_unused]] const float *gsp = DOWN ? p.down_gs : p.up_gs;
            if constexpr (DOWN) {
                for (int i = et; i < p.T * 128; i += 128)
                    s_out[i] = 0.0f; // [T][128]
                named_bar_sync(1, 128);
            }
            while (walk.next(gr)) {
                const int ncol = gr.unit.ncol;
                if (gr.k0 < gr.k1) {
                    if (q == 2)
                        wait(&acc_full[buf], aphase);
                    named_bar_sync(1, 128);
                    tc_fence_after();
                    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + buf * kAccCols;
                    [[maybe_unused]] const float gs = F::kMx ? 1.0f : __ldg(gsp + gr.unit.expert);
                    for (int c0 = 0; c0 < ncol; c0 += 4) { // four tokens' columns at a time
                        uint32_t v[4][8];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_ld_32x32b_x8(trow + min(c0 + c, ncol - 1) * kTerms, v[c]);
                        }
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c0 + c >= ncol)
                                break;
                            float s = term_sum<NV>(v[c]);
                            const int row = gr.unit.row0 + c0 + c;
                            if constexpr (NV) // (this order: the two factors' product may vanish)
                                s = s * gs * row_factor(__ldcg((DOWN ? p.sh.h_max : p.sh.x_max) + row));
                            if constexpr (DOWN) {
                                float *sum = s_out + (int)l.tok[row] * 128 + r;
                                *sum = fmaf(s, l.wt[row], *sum);
                            } else
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
                    // eight columns of h a thread
                    const int c = et >> 3, f = (et & 7) * 8;
                    const int64_t col = gr.first + f, row = gr.unit.row0 + c;
                    const bool on = c < ncol && col < p.F;
                    float h[8] = {};
                    if (on) {
                        const float *ga = s_out + c * 128 + f;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            // (expf: the fast form loses bits with the gate, up to 2^-17 at -70)
                            h[i] = ga[i] / (1.0f + expf(-ga[i])) * ga[64 + i];
                    }
                    if constexpr (F::kMx) {
                        uint8_t *sc = p.sh.h_scales + row * p.sh.h_kt * SB;
                        put_terms<false>(h, col, p.F, p.sh.h_codes + row * p.sh.h_kt * kTileBytes, sc,
                                         p.sh.h_kt, c < ncol, 0u);
                        if (c < ncol && gr.first + kUpRows >= p.F) // finite scales behind the row
                            for (int64_t b = (gr.first + kUpRows) / 32 + (et & 7); b < p.sh.h_kt * SB;
                                 b += 8)
                                sc[b] = 21;
                    } else {
                        uint32_t m = 0u;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            m = max(m, __float_as_uint(h[i]) & 0x7FFFFFFFu);
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1)
                            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                        if (on) {
                            float4 *dst = reinterpret_cast<float4 *>(
                                p.sh.h_codes + row * p.sh.h_kt * kTileBytes + col * 4);
                            dst[0] = make_float4(h[0], h[1], h[2], h[3]);
                            dst[1] = make_float4(h[4], h[5], h[6], h[7]);
                        }
                        if (c < ncol && (et & 7) == 0)
                            atomicMax(p.sh.h_max + row, m); // in any order the same
                    }
                    named_bar_sync(1, 128);
                } else if (gr.last) {
                    // this job's sums, four columns a thread: y, or a split's share of it
                    named_bar_sync(1, 128);
                    const int64_t col = gr.first + (et & 31) * 4;
                    float *part = p.sh.partial +
                                  ((int64_t)(gr.first / kDownRows) * p.splits + gr.split) * p.T * kDownRows;
                    for (int i = et; i < p.T * 32; i += 128) {
                        float4 *sum = reinterpret_cast<float4 *>(s_out) + i;
                        const float4 v = *sum;
                        *sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (p.splits > 1)
                            reinterpret_cast<float4 *>(part)[i] = v;
                        else if (col < p.H)
                            put_y(p.y + (i >> 5) * p.H + col, v);
                    }
                    named_bar_sync(1, 128);
                }
            }
        }
    };

    const std::integral_constant<bool, false> kUp;
    const std::integral_constant<bool, true> kDown;
    start(kUp);
    {
        const MoeChunks ch(n_rows, p.H);
        if constexpr (NV) { // the largest values of the rows whose chunks this CTA has
            for (int i = blockIdx.x * kThreads + tid; i < n_rows; i += gridDim.x * kThreads)
                p.sh.h_max[i] = 0u;
            if (tid < kMoeMaxTokens)
                s_max[tid] = 0u;
            __syncthreads();
            const int64_t n = p.H >> 3;
            if (ch.first < ch.last)
                for (uint32_t r = ch.first / ch.per; r <= (ch.last - 1) / ch.per; ++r) {
                    const int t = l.tok[r];
                    uint32_t m = 0u; // of both halves' magnitudes
                    for (int64_t i = tid; i < n; i += kThreads) {
                        const uint4 v = __ldg(p.x + t * n + i);
                        m = max_u16x2(m, max_u16x2(max_u16x2(v.x & kAbs16x2, v.y & kAbs16x2),
                                                   max_u16x2(v.z & kAbs16x2, v.w & kAbs16x2)));
                    }
                    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
                    if (lane == 0)
                        atomicMax(&s_max[t], m << 16);
                }
            __syncthreads();
        }
        write_terms<NV>(ch, p.H, p.sh.x_codes, p.sh.x_scales, p.sh.x_kt, warp,
                        [&](int64_t row, int64_t c0, float(&v)[8]) {
                            const int t = l.tok[row];
                            const uint4 u = __ldg(p.x + ((t * p.H + c0) >> 3));
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[2 * i] = __uint_as_float(w[i] << 16);
                                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                            }
                            if (NV && c0 == 0)
                                p.sh.x_max[row] = s_max[t];
                        },
                        [&](int64_t row) { return NV ? row_exponent(s_max[l.tok[row]]) : 0u; });
    }
    grid_sync(); // the terms of x
    products(kUp);
    start(kDown);
    grid_sync(); // h
    if constexpr (NV) {
        write_terms<NV>(MoeChunks(n_rows, p.F), p.F, p.sh.h_codes, p.sh.h_scales, p.sh.h_kt,
                        warp,
                        [&](int64_t row, int64_t c0, float(&v)[8]) {
                            const float4 *src = reinterpret_cast<const float4 *>(
                                p.sh.h_codes + row * p.sh.h_kt * kTileBytes + c0 * 4);
                            const float4 a = __ldcg(src), b = __ldcg(src + 1);
                            const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[i] = u[i];
                        },
                        [&](int64_t row) { return row_exponent(__ldcg(p.sh.h_max + row)); });
        grid_sync(); // the terms of h
    }
    products(kDown);
    if (p.splits > 1) {
        grid_sync(); // the splits' sums
        const int64_t n = (int64_t)p.T * (p.H >> 2);
        for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < n;
             i += (int64_t)gridDim.x * kThreads) { // four columns a thread, in split order
            const int64_t t = i / (p.H >> 2), c = (i % (p.H >> 2)) * 4;
            const float *src =
                p.sh.partial + ((c / kDownRows) * p.splits * p.T + t) * kDownRows + c % kDownRows;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < p.splits; ++k) {
                const float4 v =
                    __ldcg(reinterpret_cast<const float4 *>(src + (int64_t)k * p.T * kDownRows));
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            put_y(p.y + t * p.H + c, s);
        }
    }
    if (warp == 1) { // every MMA issued has completed before TMEM is freed
        if (elect_one())
            tc_commit(&drain_bar);
        if (!mbar_wait(&drain_bar, 0, kWaitLimit))
            give_up();
        __syncwarp();
    }
    tc_fence_before();
    if (__syncthreads_or(dead || s_dead)) { // copies of a run that was given up land within microseconds
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Jobs per 128-row block of y: as many as give every SM at most one, whatever the number of k-tiles.
// (Two a CTA where that leaves SMs idle, 288 jobs instead of 128 for 32 blocks, costs more in sums
// written and read than it fills: 16 tokens, H 4096: 71.6 us against 72.6. Not measured at H above
// 9472, where a block has one job and up to half of the SMs none.)
int moe_splits(int64_t H)
{
    const int64_t s = num_sms() / ((H + kDownRows - 1) / kDownRows);
    return (int)(s < 1 ? 1 : s);
}

// The workspace: offsets of MoeShared's arrays for T tokens of k experts.
struct MoeWs {
    size_t x_codes, x_scales, x_max, h_codes, h_scales, h_max, partial, total;
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
    const size_t x_kt = (size_t)(H + 255) / 256, h_kt = (size_t)(F + 255) / 256;
    MoeWs w; // (of either format: MXFP4 has half the scales and no maxima)
    w.x_codes = take(n * x_kt * kTileBytes);
    w.x_scales = take(n * x_kt * 16);
    w.x_max = take(n * 4);
    w.h_codes = take(n * h_kt * kTileBytes);
    w.h_scales = take(n * h_kt * 16);
    w.h_max = take(n * 4);
    w.partial = take(splits > 1 ? blocks * splits * (size_t)T * kDownRows * 4 : 0);
    w.total = at;
    return w;
}

template <class F>
cudaError_t launch_experts(MoeGemm g, const uint8_t *up_codes, const uint8_t *down_codes,
                           cudaStream_t s)
{
    g.sh.x_kt = (g.H + 255) / 256;
    g.sh.h_kt = (g.F + 255) / 256;
    const int cols = g.T < kCols ? g.T : kCols; // tokens of a stage
    g.box = cols < 4 ? cols : 4;
    g.stage_bytes = 16384 + (cols + g.box - 1) / g.box * g.box * kTileBytes;
    CUtensorMap up, down, xt, ht;
    const int64_t n = (int64_t)g.T * g.k;
    if (!make_fp4_codes_map(&up, up_codes, 2 * g.E, g.F, g.H, 2, kUpRows) ||
        !make_fp4_codes_map(&down, down_codes, g.E, g.H, g.F, 1, kDownRows) ||
        // the terms, a row's k-tiles of 8 x 128 bytes: a box is one k-tile of g.box rows
        !make_fp4_codes_map(&xt, g.sh.x_codes, n, g.sh.x_kt * kTerms, 256, g.box, kTerms) ||
        !make_fp4_codes_map(&ht, g.sh.h_codes, n, g.sh.h_kt * kTerms, 256, g.box, kTerms))
        return cudaErrorInvalidValue;
    static std::once_flag flags[64];
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = cudaSuccess;
    std::call_once(flags[dev & 63], [&]() {
        e = cudaFuncSetAttribute(moe_experts_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int fixed = kFeeders * kSfRing * ScaleRow<F, false>::kSlot +
                      (g.T > kCols ? g.T : kCols) * 128 * 4 + 9 * g.T * g.k;
    const int fit = (kMaxSmem - fixed) / g.stage_bytes;
    g.stages = fit < kMaxStages ? fit : kMaxStages;
    // (build_lists' temporaries, 12 E + 6 T k <= 18 KB, lie in the first two stages)
    const size_t smem = (size_t)g.stages * g.stage_bytes + fixed;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_sms(), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative; // the CTAs wait for one another: all resident
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_experts_kernel<F>, up, down, xt, ht, g);
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
                               const MoeWaits *waits, cudaStream_t s)
{
    const MoeWs w = moe_ws(T, k, F, H);
    uint8_t *b = reinterpret_cast<uint8_t *>(ws);
    auto f32 = [&](size_t o) { return reinterpret_cast<float *>(b + o); };
    MoeGemm g{};
    auto u32 = [&](size_t o) { return reinterpret_cast<uint32_t *>(b + o); };
    g.sh = MoeShared{b + w.x_codes, b + w.h_codes, b + w.x_scales, b + w.h_scales, 0, 0,
                     u32(w.x_max), u32(w.h_max), f32(w.partial)};
    g.x = reinterpret_cast<const uint4 *>(x);
    g.ids = ids;
    g.weights = weights;
    g.T = (int)T;
    g.k = k;
    g.E = E;
    g.H = H;
    g.F = F;
    g.up_scales = up_scales;
    g.down_scales = down_scales;
    g.up_gs = up_gs;
    g.down_gs = down_gs;
    g.splits = moe_splits(H);
    g.blocks = (int)((H + kDownRows - 1) / kDownRows);
    g.y = reinterpret_cast<__nv_bfloat16 *>(y);
    g.waits = waits ? *waits : kMoeWaits;
    g.barrier = grid_barrier_for(s);
    g.status = device_status_ptr();
    if (!g.status || !g.barrier)
        return cudaErrorInvalidValue;
    return mx ? launch_experts<FmtMxfp4>(g, up_codes, down_codes, s)
              : launch_experts<FmtNvfp4>(g, up_codes, down_codes, s);
}

} // namespace nvfp4
