// moe.cu -- mixture-of-experts layer for a few tokens (decode batches) on sm_100a: the router and
// the experts' gated MLP on 4-bit weights.
//
// Router: z = x . Wr^T + bias, the k largest of each token's z (equal ones: the lower expert
// first), their softmax weights. Experts: y_t = sum_k w[t,k] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t))
// with e = ids[t,k]. With at most 64 tokens the cost is reading the met experts' weights once, so
// the activations stay in 16 bits: nothing is lost to quantizing them and the weights' bytes, not
// the products, bound the time.
//
// The products run on warp-level tensor-core MMAs (m16n8k16, f16 inputs, fp32 sums): the weights
// are the 16-row side, a column tile is 8 tokens of one expert. An E2M1 code is exact in f16; the
// block scales are applied to each block's fp32 partial sum, so weights lose nothing. The
// activations are scaled by a power of two per 32 values to a largest magnitude in [1, 2) (or
// [2, 4)) before they become f16: a bf16 value keeps its 8 bits down to 2^-14 of its block's
// largest and is off by at most 2^-25 of that below. The gate/up result is rounded to f16 (11
// bits) with such a block exponent, which adds 2^-12 relative to the down product's inputs, a
// sixteenth of the final bf16 rounding's 2^-8... see moe_up_kernel for where.
//
// A k order that suits the loads: an MMA sums 16 products whatever their order, so lane t of a
// quad takes 4 consecutive code bytes of a 32-code block (8 values, MXFP4; 2 + 2 bytes of the two
// 16-code blocks, NVFP4) as its k indices, and the same 8 activations, 16 bytes, of its column.
#include <mutex>

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

struct MoeParams {
    const uint4 *x; // bf16 [T x H]
    int T, k, E;
    int64_t H, F;
    const int *ids;
    const float *weights;
    const uint8_t *up_codes, *up_scales;     // [E][2F][H/2], [E][2F][H/block]
    const uint8_t *down_codes, *down_scales; // [E][H][F/2], [E][H][F/block]
    const float *up_gs, *down_gs;            // [E] (NVFP4)
    uint4 *h;        // f16 [rows][F]: silu(gate) * up of each (expert, token) pair, scaled
    uint8_t *h_exp;  // [rows][exp_pitch]: biased exponent of each 32-block's scale
    int64_t exp_pitch;
    __nv_bfloat16 *y; // [T x H]
    int panel;        // values of a token kept in shared memory at a time
    int splits;       // CTAs that share a 64-column block of y
    float *partial;   // [64-column blocks][splits][T][64] sums of each (splits > 1)
    int *arrived;     // [64-column blocks] CTAs whose sums are in place
    GridBarrier *barrier;
    int *status;
};

// What the ids say, in shared memory: for each expert the set of its tokens; the (expert, token)
// pairs in expert order as rows, with the row's token and weight (an expert that a token names
// twice gets one row with both weights); and the column tiles, up to cols rows of one expert each.
// ids outside [0, E) name no expert.
struct MoeLists {
    uint32_t *mask;   // [E][2]
    int *base;        // [E] first row of each expert
    float *wt;        // [rows]
    int *n_units;
    uint16_t *unit;   // [tiles] expert | first column of the tile << 9
    int16_t *ids;     // [T k], -1: no expert
    uint8_t *tok;     // [rows]
};

__host__ __device__ inline size_t moe_lists_bytes(int T, int k, int E)
{
    const size_t n = (size_t)T * k;
    return (12 * (size_t)E + 9 * n + 4 + 15) / 16 * 16;
}

__device__ __forceinline__ MoeLists moe_lists(uint8_t *s, int T, int k, int E)
{
    const int n = T * k;
    MoeLists l;
    l.mask = reinterpret_cast<uint32_t *>(s);
    l.base = reinterpret_cast<int *>(l.mask + 2 * E);
    l.wt = reinterpret_cast<float *>(l.base + E);
    l.n_units = reinterpret_cast<int *>(l.wt + n);
    l.unit = reinterpret_cast<uint16_t *>(l.n_units + 1);
    l.ids = reinterpret_cast<int16_t *>(l.unit + n);
    l.tok = reinterpret_cast<uint8_t *>(l.ids + n);
    return l;
}

__device__ __forceinline__ int mask_count(const uint32_t *m) { return __popc(m[0]) + __popc(m[1]); }

// Rows of the expert's tokens before token t.
__device__ __forceinline__ int mask_before(const uint32_t *m, int t)
{
    return t < 32 ? __popc(m[0] & ((1u << t) - 1u))
                  : __popc(m[0]) + __popc(m[1] & ((1u << (t - 32)) - 1u));
}

__device__ __forceinline__ int unit_expert(uint32_t u) { return (int)(u & 0x1FFu); }
__device__ __forceinline__ int unit_column(uint32_t u) { return (int)(u >> 9); }

__device__ __forceinline__ void build_lists(const MoeLists &l, const MoeParams &p, int cols)
{
    const int tid = threadIdx.x, nthr = blockDim.x, n = p.T * p.k;
    for (int i = tid; i < 2 * p.E; i += nthr)
        l.mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = __ldg(p.ids + i), t = i / p.k;
        const bool on = e >= 0 && e < p.E;
        l.ids[i] = on ? (int16_t)e : (int16_t)-1;
        if (on)
            atomicOr(&l.mask[2 * e + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    if (tid < 32) { // exclusive prefix of rows and of tiles over the experts
        const int per = (p.E + 31) / 32;
        int rows = 0, tiles = 0;
        for (int q = 0; q < per; ++q) {
            const int e = tid * per + q;
            const int c = e < p.E ? mask_count(l.mask + 2 * e) : 0;
            rows += c;
            tiles += (c + cols - 1) / cols;
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
        if (tid == 31)
            *l.n_units = u0;
        r0 -= rows;
        u0 -= tiles;
        for (int q = 0; q < per; ++q) {
            const int e = tid * per + q;
            if (e >= p.E)
                break;
            const int c = mask_count(l.mask + 2 * e);
            l.base[e] = r0;
            for (int c0 = 0; c0 < c; c0 += cols)
                l.unit[u0++] = (uint16_t)(e | c0 << 9);
            r0 += c;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = l.ids[i], t = i / p.k;
        if (e < 0)
            continue;
        bool first = true; // of the token's slots that name e
        float w = 0.0f;
        for (int s = t * p.k; s < (t + 1) * p.k; ++s)
            if (l.ids[s] == e) {
                first = first && s >= i;
                w += __ldg(p.weights + s);
            }
        if (first) {
            const int row = l.base[e] + mask_before(l.mask + 2 * e, t);
            l.tok[row] = (uint8_t)t;
            l.wt[row] = w;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Lane t's four code bytes of the 32-code block at `a`: bytes 4t.. (MXFP4), or bytes 2t, 2t + 1 of
// each of its two 16-code blocks (NVFP4).
template <bool NV> __device__ __forceinline__ uint32_t lane_codes(const uint8_t *a, int t)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a);
    if constexpr (NV)
        return __byte_perm(w[t >> 1], w[2 + (t >> 1)], (t & 1) ? 0x7632 : 0x5410);
    else
        return w[t];
}

// Code byte i of a word -> its two values as f16x2 (exact).
template <int I> __device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w)
{
    uint32_t h;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(h) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b1;\n\t}" : "=r"(h) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b2;\n\t}" : "=r"(h) : "r"(w));
    else
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b3;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

// c = A B (16 x 8, K 16), and c += A B.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Biased exponent of the power of two that a block of largest magnitude m (fp32 bits) is divided
// by: m / 2^(e - 127) lies in [1, 2) ([2, 4) for the top binade; below 1 for a subnormal m).
__device__ __forceinline__ uint32_t block_exponent(uint32_t m)
{
    const uint32_t e = m >> 23;
    return e < 1u ? 1u : e > 253u ? 253u : e;
}

// A warp's weight tile: 16 rows x 256 codes (128 bytes at a 144-byte pitch: the fragment loads of
// eight rows x four lanes hit 32 banks) and the rows' scale bytes of the tile (8 MXFP4, 16 NVFP4),
// fetched as the aligned words that hold them, since a row of scales may start at any byte.
constexpr int kTileK = 256, kTileBlocks = kTileK / 32;

template <bool NV> struct Tile {
    static constexpr int kPitch = 144;
    static constexpr int kScaleBytes = NV ? 16 : 8; // of one row and tile
    static constexpr int kWords = kScaleBytes / 4 + 1;
    static constexpr int kSlot = NV ? 32 : 16;
    static constexpr int kOffScales = 16 * kPitch;
    static constexpr int kBytes = kOffScales + 16 * kSlot;
};

// Where a lane reads its share of a warp's rows. Local rows 0..7 are rows row..row + 7 of the
// expert's matrix, 8..15 the same `half` rows further down.
struct TileSource {
    const uint8_t *codes;  // row + lane / 8, at the lane's 16-byte chunk
    const uint8_t *scales; // the expert's
    int64_t srow;          // byte offset of row (row + lane % 8 (+ half))'s scales
};

template <bool NV>
__device__ __forceinline__ TileSource tile_source(const uint8_t *codes, const uint8_t *scales,
                                                  int64_t K, int64_t row, int64_t half, int lane)
{
    TileSource s;
    s.codes = codes + (row + (lane >> 3)) * (K >> 1) + (lane & 7) * 16;
    s.scales = scales;
    s.srow = (row + (lane & 7) + ((lane & 8) ? half : 0)) * (NV ? K >> 4 : K >> 5);
    return s;
}

// Tile kt of the K codes of each row -> shared memory (cp.async; 16-byte pieces past the row's end
// are left out, and so are scale words that hold none of the row's bytes).
template <bool NV>
__device__ __forceinline__ void load_tile(uint32_t dst, const TileSource &s, int64_t K, int64_t half,
                                          int kt, int lane)
{
    using L = Tile<NV>;
    const int64_t krow = K >> 1;
    const int c = lane & 7;
    if (kt * kTileBlocks + c < (int)(K >> 5)) {
        const uint8_t *src = s.codes + (int64_t)kt * (kTileK / 2);
        const uint32_t d = dst + (lane >> 3) * L::kPitch + c * 16;
        cp_async16(d, src);
        cp_async16(d + 4 * L::kPitch, src + 4 * krow);
        cp_async16(d + 8 * L::kPitch, src + half * krow);
        cp_async16(d + 12 * L::kPitch, src + (half + 4) * krow);
    }
    const int64_t k0 = (int64_t)kt * L::kScaleBytes;
    const int64_t left = (NV ? K >> 4 : K >> 5) - k0;
    const int64_t off = s.srow + k0, a = off & ~(int64_t)3;
    const int64_t end = off + (left < L::kScaleBytes ? left : L::kScaleBytes);
    const uint32_t d = dst + L::kOffScales + (lane & 15) * L::kSlot;
#pragma unroll
    for (int w = 0; w < L::kWords; w += 2) { // lanes 16.. take the odd words
        const int q = w + (lane >> 4);
        if (a + 4 * q < end)
            cp_async4(d + 4 * q, s.scales + a + 4 * q);
    }
}

// Scale bytes of local row r as whole words; sh8: 8 x the byte in its word at which they start.
template <bool NV>
__device__ __forceinline__ void tile_scales(const uint8_t *tile, int r, uint32_t sh8,
                                            uint32_t (&s)[NV ? 4 : 2])
{
    const uint4 *a =
        reinterpret_cast<const uint4 *>(tile + Tile<NV>::kOffScales + r * Tile<NV>::kSlot);
    const uint4 w = a[0];
    s[0] = __funnelshift_r(w.x, w.y, sh8);
    s[1] = __funnelshift_r(w.y, w.z, sh8);
    if constexpr (NV) {
        s[2] = __funnelshift_r(w.z, w.w, sh8);
        s[3] = __funnelshift_r(w.w, a[1].x, sh8);
    }
}

// Whether a word has a byte 0 or 255 (MXFP4 scales that are not a shifted exponent field).
__device__ __forceinline__ bool odd_scale(uint32_t w)
{
    return ((((w - 0x01010101u) & ~w) | ((~w - 0x01010101u) & w)) & 0x80808080u) != 0u;
}

// acc += half a tile (four 32-blocks, nb of them live) x activations. frag(n, b) gives the
// activations of column tile n as MMA B fragments; colscale(n, b, j) the scale of this lane's j-th
// accumulator column (COLS). NL live column tiles. SPECIAL: the general form, for short tiles and
// for MXFP4 scale bytes 0 and 255; the other has no branch, so that the loads and MMAs of
// neighbouring blocks interleave.
template <int NT, int NL, bool NV, bool COLS, bool SPECIAL, typename Frag, typename ColScale>
__device__ __forceinline__ void half_blocks(float (&acc)[NT][4], const uint8_t *codes, int nb,
                                            int lane, const uint32_t *s0, const uint32_t *s1,
                                            Frag frag, ColScale colscale)
{
    const int g = lane >> 2, t = lane & 3;
    const uint8_t *ra = codes + g * Tile<NV>::kPitch, *rb = ra + 8 * Tile<NV>::kPitch;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (SPECIAL && b >= nb)
            break;
        const uint32_t w0 = lane_codes<NV>(ra + b * 16, t), w1 = lane_codes<NV>(rb + b * 16, t);
        // k16 step, fragment: rows g and g + 8, k indices 2t.. and 2t + 8..
        const uint32_t a[2][4] = {{e2m1x2_to_f16x2<0>(w0), e2m1x2_to_f16x2<0>(w1),
                                   e2m1x2_to_f16x2<1>(w0), e2m1x2_to_f16x2<1>(w1)},
                                  {e2m1x2_to_f16x2<2>(w0), e2m1x2_to_f16x2<2>(w1),
                                   e2m1x2_to_f16x2<3>(w0), e2m1x2_to_f16x2<3>(w1)}};
        float f0[2], f1[2]; // block scales of rows g, g + 8 (NVFP4: of each 16-block)
        if constexpr (NV) {
            const float2 p0 = e4m3x2_to_f32x2(s0[b >> 1] >> (16 * (b & 1)));
            const float2 p1 = e4m3x2_to_f32x2(s1[b >> 1] >> (16 * (b & 1)));
            f0[0] = p0.x;
            f0[1] = p0.y;
            f1[0] = p1.x;
            f1[1] = p1.y;
        } else if constexpr (SPECIAL) {
            f0[0] = mx_scale_f32((s0[0] >> (8 * b)) & 0xFFu);
            f1[0] = mx_scale_f32((s1[0] >> (8 * b)) & 0xFFu);
        } else { // the byte into bits 23..30
            f0[0] = __uint_as_float(__byte_perm(s0[0], 0u, 0x0444u | b << 12) >> 1);
            f1[0] = __uint_as_float(__byte_perm(s1[0], 0u, 0x0444u | b << 12) >> 1);
        }
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const uint4 u = frag(n, b);
            float q0 = 1.0f, q1 = 1.0f;
            if constexpr (COLS) {
                q0 = colscale(n, b, 0);
                q1 = colscale(n, b, 1);
            }
            float c[4];
            mma_f16_first(c, a[0], u.x, u.y);
            if constexpr (NV) {
                float d[4];
                mma_f16_first(d, a[1], u.z, u.w);
                acc[n][0] = fmaf(COLS ? c[0] * q0 : c[0], f0[0], acc[n][0]);
                acc[n][1] = fmaf(COLS ? c[1] * q1 : c[1], f0[0], acc[n][1]);
                acc[n][2] = fmaf(COLS ? c[2] * q0 : c[2], f1[0], acc[n][2]);
                acc[n][3] = fmaf(COLS ? c[3] * q1 : c[3], f1[0], acc[n][3]);
                acc[n][0] = fmaf(COLS ? d[0] * q0 : d[0], f0[1], acc[n][0]);
                acc[n][1] = fmaf(COLS ? d[1] * q1 : d[1], f0[1], acc[n][1]);
                acc[n][2] = fmaf(COLS ? d[2] * q0 : d[2], f1[1], acc[n][2]);
                acc[n][3] = fmaf(COLS ? d[3] * q1 : d[3], f1[1], acc[n][3]);
            } else {
                mma_f16(c, a[1], u.z, u.w);
                acc[n][0] = fmaf(COLS ? c[0] * q0 : c[0], f0[0], acc[n][0]);
                acc[n][1] = fmaf(COLS ? c[1] * q1 : c[1], f0[0], acc[n][1]);
                acc[n][2] = fmaf(COLS ? c[2] * q0 : c[2], f1[0], acc[n][2]);
                acc[n][3] = fmaf(COLS ? c[3] * q1 : c[3], f1[0], acc[n][3]);
            }
        }
    }
}

// The scales of a tile's rows g and g + 8, and whether they (or a short tile) need the general form.
template <bool NV> struct TileScales {
    uint32_t s0[NV ? 4 : 2], s1[NV ? 4 : 2];
    bool special;

    __device__ __forceinline__ void load(const uint8_t *tile, int nb, int lane, uint32_t sh0,
                                         uint32_t sh1)
    {
        tile_scales<NV>(tile, lane >> 2, sh0, s0);
        tile_scales<NV>(tile, (lane >> 2) + 8, sh1, s1);
        special = nb < kTileBlocks;
        if constexpr (!NV)
            special = special || __any_sync(0xFFFFFFFFu, odd_scale(s0[0]) || odd_scale(s0[1]) ||
                                                             odd_scale(s1[0]) || odd_scale(s1[1]));
    }
};

// Half HALF of a tile, nt live column tiles.
template <int HALF, int NT, bool NV, bool COLS, typename Frag, typename ColScale>
__device__ __forceinline__ void half_product(float (&acc)[NT][4], const uint8_t *tile, int nb,
                                             int nt, int lane, const TileScales<NV> &sc, Frag frag,
                                             ColScale colscale)
{
    constexpr int kW = NV ? 2 * HALF : HALF; // first scale word
    const uint8_t *codes = tile + HALF * 64;
    if (sc.special)
        half_blocks<NT, NT, NV, COLS, true>(acc, codes, nb - 4 * HALF, lane, sc.s0 + kW, sc.s1 + kW,
                                            frag, colscale);
    else if (nt == 1)
        half_blocks<NT, 1, NV, COLS, false>(acc, codes, 4, lane, sc.s0 + kW, sc.s1 + kW, frag,
                                            colscale);
    else
        half_blocks<NT, NT, NV, COLS, false>(acc, codes, 4, lane, sc.s0 + kW, sc.s1 + kW, frag,
                                             colscale);
}

// Place of value v (0..31) of a 32-block in the activations' layout: each lane's 8 values are
// consecutive (MXFP4: v itself; NVFP4: lane t takes 4t.. of both 16-blocks).
template <bool NV> __device__ __forceinline__ int lane_order(int v)
{
    if constexpr (NV)
        return (((v >> 2) & 3) * 2 + (v >> 4)) * 4 + (v & 3);
    else
        return v;
}

constexpr int kMaxSmem = 232448 - 64; // per CTA, beside the static part
constexpr int kWarps = 16, kGroups = kWarps / 4, kStages = 3;
constexpr int kRowBlock = 64;  // columns of y a CTA sums at a time: 16 a warp of a group
constexpr int kHPitch = 36;    // floats between columns of the h exchange: conflict-free
constexpr uint32_t kBarrierLimit = 1u << 21;

// Shared memory: rings; sums of the K-split; h exchange; token exponents; x panel (gate/up) or y
// sums (down); lists.
template <int NT, bool NV, int KS> struct Layout {
    static constexpr int kRed = (kGroups / KS) * KS * (KS - 1) * 4 * NT * 32 * 16;
    static constexpr int kOffRed = kWarps * kStages * Tile<NV>::kBytes;
    static constexpr int kOffH = kOffRed + kRed;
    static constexpr int kOffExp = kOffH + kGroups * 8 * NT * kHPitch * 4;
    static constexpr int kOffX = kOffExp + 128;
    // bytes between columns of the x panel: 64 past a multiple of 128, so that the 16-byte
    // fragment loads of two columns x four lanes hit 32 banks
    __host__ __device__ static int x_pitch(int panel)
    {
        return panel * 2 + (panel * 2 % 128 == 0 ? 64 : 0);
    }
    __host__ __device__ static int x_bytes(int T, int panel)
    {
        const int x = (T < 8 * NT ? T : 8 * NT) * x_pitch(panel), y = kWarps * 16 * T * 4;
        return x > y ? x : y;
    }
};

// The whole layer's experts in one cooperative launch, one CTA of 16 warps per SM.
//
// Gate/up: an item is 32 columns of F (64 weight rows) of one column tile. A team of KS groups of
// four warps takes an item; a warp has 8 of its columns, 8 gate rows and the same 8 up rows as its 16
// MMA rows, so that a lane's accumulators hold both sides of its products; the team's groups split
// the k-tiles, and take turns in adding the others' sums and finishing an item (h and its block
// exponents, to the workspace). A CTA's items are a run, so its tokens change seldom; they are kept in
// shared memory as f16, each divided by its power of two (whole rows, or panels of them where they
// do not fit).
//
// Grid barrier (every h is in place), behind which the rings already fill with the next tiles.
//
// Down: a CTA sums 64 columns of y, its groups' and `splits` CTAs' shares being runs of the flat list
// of (column tile, k-tile) pairs of all met experts. A warp weights its sums of a column tile into
// its own [T x 16] array; the arrays are added group by group, the CTAs' sums split by split by the
// CTA that comes last, so the order of every sum is fixed.
//
// Bound by the decode (35-40 issue slots per 16 x 32 codes and column tile, about the time HBM takes
// for them), so both have to run at once: the rings are private to the warps and run on across items.
template <int NT, bool NV, int KS>
__global__ void __launch_bounds__(kWarps * 32, 1) moe_experts_kernel(const MoeParams p)
{
    using L = Tile<NV>;
    using U = Layout<NT, NV, KS>;
    constexpr int NC = 8 * NT, kTeams = kGroups / KS;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int grp = warp >> 2, w4 = warp & 3, team = grp / KS, kg = grp % KS;
    const MoeLists l = moe_lists(smem + U::kOffX + U::x_bytes(p.T, p.panel), p.T, p.k, p.E);
    const int nrb = (int)((p.H + kRowBlock - 1) / kRowBlock);
    pdl_wait();
    if (blockIdx.x == 0)
        for (int i = tid; i < nrb; i += kWarps * 32)
            p.arrived[i] = 0;
    build_lists(l, p, NC);

    const int nf = (int)(p.F >> 5); // items per column tile
    const int n_units = *l.n_units;
    const int64_t items = (int64_t)n_units * nf;
    const int i0 = (int)(items * blockIdx.x / gridDim.x);
    const int i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
    const int upblk = (int)(p.H >> 5), upkt = (upblk + kTileBlocks - 1) / kTileBlocks;
    const int dnblk = (int)(p.F >> 5), dnkt = (dnblk + kTileBlocks - 1) / kTileBlocks;
    const int64_t uprow = NV ? p.H >> 4 : p.H >> 5, dnrow = NV ? p.F >> 4 : p.F >> 5;

    // ---- the tiles this warp loads, in the order in which it uses them -------------------------
    uint8_t *ring = smem + warp * kStages * L::kBytes;
    const uint32_t ring_addr = smem_u32(ring);
    int phase = 0;                      // 0 gate/up, 1 down, 2 none left
    int lu, li, lkt, left = 0, lslot = 0, job = 0;
    TileSource src;
    // the warp's run of (column tile, k-tile) pairs in down job j: [a, b)
    auto down_run = [&](int j, int &a, int &b) {
        const int64_t row = (int64_t)(j / p.splits) * kRowBlock + w4 * 16;
        const int64_t total = row < p.H ? (int64_t)n_units * dnkt : 0;
        const int run = (j % p.splits) * kGroups + grp, runs = p.splits * kGroups;
        a = (int)(total * run / runs);
        b = (int)(total * (run + 1) / runs);
    };
    auto down_source = [&]() {
        const int64_t e = unit_expert(l.unit[lu]);
        src = tile_source<NV>(p.down_codes + e * p.H * (p.F >> 1), p.down_scales + e * p.H * dnrow,
                              p.F, (int64_t)(job / p.splits) * kRowBlock + w4 * 16, 8, lane);
    };
    auto down_seek = [&]() { // to the first down job from `job` on with tiles for this warp
        phase = 2;
        for (; job < nrb * p.splits; job += gridDim.x) {
            int a, b;
            down_run(job, a, b);
            if (a < b) {
                left = b - a;
                lu = a / dnkt;
                lkt = a % dnkt;
                phase = 1;
                down_source();
                return;
            }
        }
    };
    auto up_seek = [&]() { // to this team's next item, of the same column tile or a later one
        while (li >= min(i1, (lu + 1) * nf)) {
            ++lu;
            li = lu * nf + team;
            if (lu * nf >= i1) {
                job = blockIdx.x;
                down_seek();
                return;
            }
        }
        const int64_t e = unit_expert(l.unit[lu]);
        src = tile_source<NV>(p.up_codes + e * 2 * p.F * (p.H >> 1),
                              p.up_scales + e * 2 * p.F * uprow, p.H,
                              (int64_t)(li - lu * nf) * 32 + w4 * 8, p.F, lane);
    };
    auto issue = [&]() {
        const uint32_t dst = ring_addr + lslot * L::kBytes;
        if (phase == 0) {
            load_tile<NV>(dst, src, p.H, p.F, lkt, lane);
            lkt += KS;
            if (lkt >= upkt) {
                lkt = kg;
                li += kTeams;
                up_seek();
            }
        } else if (phase == 1) {
            load_tile<NV>(dst, src, p.F, 8, lkt, lane);
            if (--left == 0) {
                job += gridDim.x;
                down_seek();
            } else if (++lkt == dnkt) {
                lkt = 0;
                ++lu;
                down_source();
            }
        }
        cp_async_commit();
        lslot = lslot + 1 == kStages ? 0 : lslot + 1;
    };
    if (i0 < i1 && kg < upkt) {
        lu = i0 / nf;
        li = i0 + team;
        lkt = kg;
        up_seek();
    } else {
        job = blockIdx.x;
        down_seek();
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        issue();
    int slot = 0;
    auto next_tile = [&]() -> const uint8_t * { // the oldest tile, once it has arrived
        issue();
        cp_async_wait<kStages - 1>();
        __syncwarp();
        return ring + slot * L::kBytes;
    };
    auto tile_done = [&]() {
        __syncwarp(); // the tile is read before its slot is filled again
        slot = slot + 1 == kStages ? 0 : slot + 1;
    };

    // ---- gate/up --------------------------------------------------------------------------------
    {
        const int pitch = U::x_pitch(p.panel);
        uint8_t *sx = smem + U::kOffX;
        uint32_t *s_ex = reinterpret_cast<uint32_t *>(smem + U::kOffExp);
        float *hx = reinterpret_cast<float *>(smem + U::kOffH) + grp * NC * kHPitch;
        // [team][turn][other group][w4][n][lane]
        float4 *red = reinterpret_cast<float4 *>(smem + U::kOffRed) +
                      team * KS * (KS - 1) * 4 * NT * 32;
        const uint8_t *xcol[NT]; // this lane's column of each column tile (past the last: that one)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            xcol[n] = sx + min(n * 8 + g, min(NC, p.T) - 1) * pitch + t * 16;
        int turn = 0; // the team's group that finishes the item
        for (int u = i0 / nf; u * nf < i1; ++u) {
            const int e = unit_expert(l.unit[u]), c0 = unit_column(l.unit[u]);
            const int row0 = l.base[e] + c0;
            const int ncol = min(NC, mask_count(l.mask + 2 * e) - c0);
            const int nt = (ncol + 7) >> 3;
            const int a = max(i0, u * nf), b = min(i1, (u + 1) * nf);
            const float gs = NV ? __ldg(p.up_gs + e) : 1.0f;
            for (int r = a; r < b; r += kTeams) {
                const int it = r + team;
                const bool on = it < b;
                const int64_t f0 = (int64_t)(it - u * nf) * 32;
                const uint32_t sh0 = (uint32_t)(((f0 + w4 * 8 + g) * uprow) & 3) * 8u;
                const uint32_t sh1 = (uint32_t)(((p.F + f0 + w4 * 8 + g) * uprow) & 3) * 8u;
                float acc[NT][4] = {};
                int kt = kg;
                for (int k0 = 0; k0 < (int)p.H; k0 += p.panel) {
                    const int k1 = min((int)p.H, k0 + p.panel);
                    if (r == a || p.panel < (int)p.H) {
                        __syncthreads(); // the last panel has been used
                        for (int c = warp; c < ncol; c += kWarps) {
                            const uint4 *x = p.x + (int64_t)l.tok[row0 + c] * (p.H >> 3);
                            uint32_t m = 0u;
#pragma unroll 4
                            for (int i = lane; i < (int)(p.H >> 3); i += 32) {
                                const uint4 v = __ldg(x + i);
                                m = max_u16x2(
                                    m, max_u16x2(max_u16x2(v.x & kAbs16x2, v.y & kAbs16x2),
                                                 max_u16x2(v.z & kAbs16x2, v.w & kAbs16x2)));
                            }
                            m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
                            const uint32_t ex = block_exponent(m << 16);
                            const float inv = __uint_as_float((254u - ex) << 23);
                            if (lane == 0)
                                s_ex[c] = ex;
#pragma unroll 4
                            for (int i = (k0 >> 3) + lane; i < k1 >> 3; i += 32) {
                                const uint4 v = __ldg(x + i);
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                                uint32_t h[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    h[q] = pack_f16x2(__uint_as_float(w[q] << 16) * inv,
                                                      __uint_as_float(w[q] & 0xFFFF0000u) * inv);
                                // eight values: two groups of four at their lanes' places
                                uint8_t *d = sx + c * pitch + ((i - (k0 >> 3)) >> 2) * 64;
                                const int v0 = (i & 3) * 8;
                                *reinterpret_cast<uint2 *>(d + lane_order<NV>(v0) * 2) =
                                    make_uint2(h[0], h[1]);
                                *reinterpret_cast<uint2 *>(d + lane_order<NV>(v0 + 4) * 2) =
                                    make_uint2(h[2], h[3]);
                            }
                        }
                        __syncthreads();
                    }
                    for (; on && kt * kTileK < k1; kt += KS) {
                        const uint8_t *tile = next_tile();
                        const int nb = min(kTileBlocks, upblk - kt * kTileBlocks);
                        TileScales<NV> sc;
                        sc.load(tile, nb, lane, sh0, sh1);
                        const int xt = (kt * kTileK - k0) * 2;
                        const auto one = [](int, int, int) { return 1.0f; };
                        half_product<0, NT, NV, false>(
                            acc, tile, nb, nt, lane, sc,
                            [&](int n, int b_) {
                                return *reinterpret_cast<const uint4 *>(xcol[n] + xt + b_ * 64);
                            },
                            one);
                        half_product<1, NT, NV, false>(
                            acc, tile, nb, nt, lane, sc,
                            [&](int n, int b_) {
                                return *reinterpret_cast<const uint4 *>(xcol[n] + xt + 256 +
                                                                        b_ * 64);
                            },
                            one);
                        tile_done();
                    }
                }
                if (!on)
                    continue;
                // The others hand their sums to the group whose turn it is. A turn's buffer comes
                // around after KS items: every other group has by then had its own turn, for which
                // it waited for this one's next arrival, made after the buffer was read.
                float4 *rt = red + turn * (KS - 1) * 4 * NT * 32;
                if (kg != turn) {
                    float4 *dst = rt + ((kg < turn ? kg : kg - 1) * 4 + w4) * NT * 32 + lane;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        dst[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                    named_bar_arrive(1 + team * KS + turn, KS * 128);
                } else {
                    named_bar_sync(1 + team * KS + turn, KS * 128);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int q = 0; q < KS; ++q) { // in group order
                            float4 v = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
                            if (q != kg)
                                v = rt[((q < kg ? q : q - 1) * 4 + w4) * NT * 32 + n * 32 + lane];
                            s.x += v.x;
                            s.y += v.y;
                            s.z += v.z;
                            s.w += v.w;
                        }
                        const float gate[2] = {s.x, s.y}, upv[2] = {s.z, s.w};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int c = n * 8 + 2 * t + j;
                            if (c < ncol) {
                                const float q = __uint_as_float(s_ex[c] << 23);
                                const float ga = gate[j] * q * gs, up = upv[j] * q * gs;
                                hx[c * kHPitch + w4 * 8 + g] = ga / (1.0f + __expf(-ga)) * up;
                            }
                        }
                    }
                    named_bar_sync(9 + grp, 128);
                    for (int c = w4; c < ncol; c += 4) {
                        const float v = hx[c * kHPitch + lane];
                        const uint32_t m =
                            __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
                        const uint32_t ex = block_exponent(m);
                        const int64_t row = row0 + c;
                        reinterpret_cast<__half *>(p.h)[row * p.F + f0 + lane_order<NV>(lane)] =
                            __float2half_rn(v * __uint_as_float((254u - ex) << 23));
                        if (lane == 0)
                            p.h_exp[row * p.exp_pitch + (f0 >> 5)] = (uint8_t)ex;
                    }
                }
                turn = turn + 1 == KS ? 0 : turn + 1;
            }
        }
    }

    // ---- every h in place -----------------------------------------------------------------------
    __syncthreads();
    if (tid == 0) {
        s_flag = grid_barrier_sync(p.barrier, (int)gridDim.x, (int)blockIdx.x, kBarrierLimit) ? 1 : 0;
        if (!s_flag)
            atomicExch(p.status, (int)NVFP4_ERR_TIMEOUT);
    }
    __syncthreads();
    if (!s_flag) {
        cp_async_wait<0>();
        return;
    }

    // ---- down -----------------------------------------------------------------------------------
    float *ysum = reinterpret_cast<float *>(smem + U::kOffX); // [group][w4][T][16]
    float *mysum = ysum + warp * 16 * p.T;
    for (int jb = blockIdx.x; jb < nrb * p.splits; jb += gridDim.x) {
        for (int i = lane; i < 16 * p.T; i += 32)
            mysum[i] = 0.0f;
        __syncwarp();
        const int64_t r0 = (int64_t)(jb / p.splits) * kRowBlock + w4 * 16;
        const uint32_t sh0 = (uint32_t)(((r0 + g) * dnrow) & 3) * 8u;
        const uint32_t sh1 = (uint32_t)(((r0 + g + 8) * dnrow) & 3) * 8u;
        int a, b;
        down_run(jb, a, b);
        float acc[NT][4] = {};
        for (int u = a / dnkt, kt = a % dnkt, rest = b - a; rest > 0; ++u, kt = 0) {
            const int e = unit_expert(l.unit[u]), c0 = unit_column(l.unit[u]);
            const int row = l.base[e] + c0;
            const int ncol = min(NC, mask_count(l.mask + 2 * e) - c0);
            const int nt = (ncol + 7) >> 3;
            const int kend = min(dnkt, kt + rest);
            rest -= kend - kt;
            const uint4 *hp[NT];
            const uint8_t *ep[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) { // dead columns read a live one's
                hp[n] = p.h + (int64_t)(row + min(n * 8 + g, ncol - 1)) * (p.F >> 3) + t;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ep[n][j] =
                        p.h_exp + (int64_t)(row + min(n * 8 + 2 * t + j, ncol - 1)) * p.exp_pitch;
            }
            // half a tile's activations and their exponents
            struct Half {
                uint4 h[NT][4];
                uint32_t e[NT][2];
            };
            auto fetch = [&](Half &f, int blk) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n > 0 && n >= nt)
                        break;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        f.h[n][q] = hp[n][min(blk + q, dnblk - 1) * 4];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        f.e[n][j] = *reinterpret_cast<const uint32_t *>(ep[n][j] + blk);
                }
            };
            auto scale_of = [](const Half &f, int n, int q, int j) {
                return __uint_as_float(__byte_perm(f.e[n][j], 0u, 0x0444u | q << 12) >> 1);
            };
            Half f0, f1;
            fetch(f0, kt * kTileBlocks);
            for (; kt < kend; ++kt) {
                const uint8_t *tile = next_tile();
                const int nb = min(kTileBlocks, dnblk - kt * kTileBlocks);
                TileScales<NV> sc;
                sc.load(tile, nb, lane, sh0, sh1);
                fetch(f1, kt * kTileBlocks + 4); // exponents past the row: its padding
                half_product<0, NT, NV, true>(
                    acc, tile, nb, nt, lane, sc, [&](int n, int q) { return f0.h[n][q]; },
                    [&](int n, int q, int j) { return scale_of(f0, n, q, j); });
                if (kt + 1 < kend)
                    fetch(f0, (kt + 1) * kTileBlocks);
                half_product<1, NT, NV, true>(
                    acc, tile, nb, nt, lane, sc, [&](int n, int q) { return f1.h[n][q]; },
                    [&](int n, int q, int j) { return scale_of(f1, n, q, j); });
                tile_done();
            }
            // the column tile's sums of this run
            const float gs = NV ? __ldg(p.down_gs + e) : 1.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = n * 8 + 2 * t + j;
                    if (c < ncol) {
                        const float w = l.wt[row + c];
                        float *y = mysum + l.tok[row + c] * 16 + g;
                        y[0] = fmaf(acc[n][j] * gs, w, y[0]);
                        y[8] = fmaf(acc[n][2 + j] * gs, w, y[8]);
                    }
                    acc[n][j] = acc[n][2 + j] = 0.0f;
                }
            __syncwarp(); // the next tile's columns may be other lanes' tokens
        }
        __syncthreads();
        // the groups' sums: y, or this split's share of it
        const int rb = jb / p.splits;
        float *part = p.partial + ((int64_t)rb * p.splits + jb % p.splits) * p.T * kRowBlock;
        for (int i = tid; i < kRowBlock * p.T; i += kWarps * 32) {
            const int r = i % kRowBlock, tk = i / kRowBlock;
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                s += ysum[((q * 4 + (r >> 4)) * p.T + tk) * 16 + (r & 15)];
            if (p.splits > 1)
                part[i] = s;
            else if ((int64_t)rb * kRowBlock + r < p.H)
                p.y[tk * p.H + (int64_t)rb * kRowBlock + r] = __float2bfloat16_rn(s);
        }
        if (p.splits > 1) {
            __threadfence();
            __syncthreads();
            if (tid == 0)
                s_flag = atomicAdd(p.arrived + rb, 1);
            __syncthreads();
            if (s_flag == p.splits - 1) { // the last of the block's CTAs adds them up
                __threadfence();
                const float *all = p.partial + (int64_t)rb * p.splits * p.T * kRowBlock;
                for (int i = tid; i < kRowBlock * p.T; i += kWarps * 32) {
                    const int r = i % kRowBlock, tk = i / kRowBlock;
                    float s = 0.0f;
                    for (int q = 0; q < p.splits; ++q)
                        s += __ldcg(all + (int64_t)q * p.T * kRowBlock + i);
                    if ((int64_t)rb * kRowBlock + r < p.H)
                        p.y[tk * p.H + (int64_t)rb * kRowBlock + r] = __float2bfloat16_rn(s);
                }
            }
        }
        __syncthreads(); // s_flag and the sums have been read
    }
    cp_async_wait<0>();
}

template <int NT, bool NV, int KS> cudaError_t launch_experts(MoeParams p, cudaStream_t s)
{
    using U = Layout<NT, NV, KS>;
    const int lists = (int)moe_lists_bytes(p.T, p.k, p.E);
    // the x panel: all of H where it fits beside the rings
    const int room = kMaxSmem - U::kOffX - lists;
    if (U::x_bytes(p.T, (int)p.H) <= room)
        p.panel = (int)p.H;
    else
        p.panel = (room / (p.T < 8 * NT ? p.T : 8 * NT) - 64) / 2 / kTileK * kTileK;
    const size_t smem = U::kOffX + U::x_bytes(p.T, p.panel) + lists;
    auto kernel = moe_experts_kernel<NT, NV, KS>;
    static std::once_flag flags[64];
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e = cudaSuccess;
    std::call_once(flags[dev & 63], [&]() {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    });
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_sms(), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative; // the CTAs wait for one another: all resident
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Whether a token panel of 16 whole rows fits.
template <bool NV> bool wide_fits(const MoeParams &p)
{
    using U = Layout<2, NV, 2>;
    return U::kOffX + U::x_bytes(p.T, (int)p.H) + (int)moe_lists_bytes(p.T, p.k, p.E) <=
           kMaxSmem;
}

template <bool NV> cudaError_t launch_experts_fmt(const MoeParams &p, cudaStream_t s)
{
    if (p.T <= 4)
        return launch_experts<1, NV, 4>(p, s);
    // column tiles of 16 where an expert may well meet more than 8 tokens
    if (p.T > 8 && p.T * p.k > 4 * p.E && wide_fits<NV>(p))
        return launch_experts<2, NV, 2>(p, s);
    return launch_experts<1, NV, 2>(p, s);
}

// CTAs per 64-column block of y.
int moe_splits(int64_t H)
{
    const int64_t nrb = (H + kRowBlock - 1) / kRowBlock;
    const int64_t s = num_sms() / nrb;
    return (int)(s < 1 ? 1 : s);
}

// Workspace: h, its exponents, the splits' sums of y, the arrival counters.
struct MoeWs {
    size_t exps, partial, arrived, total;
};

MoeWs moe_ws(int64_t T, int64_t k, int64_t F, int64_t H)
{
    auto align = [](size_t v) { return (v + 255) & ~(size_t)255; };
    const size_t rows = (size_t)T * (size_t)k, nrb = (size_t)((H + kRowBlock - 1) / kRowBlock);
    const int splits = moe_splits(H);
    MoeWs w;
    w.exps = align(rows * (size_t)F * 2);
    w.partial = w.exps + align(rows * (size_t)((F / 32 + 7) / 8 * 8));
    w.arrived = w.partial + (splits > 1 ? align(nrb * splits * (size_t)T * kRowBlock * 4) : 0);
    w.total = w.arrived + align(nrb * 4);
    return w;
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
    MoeParams p{};
    p.x = reinterpret_cast<const uint4 *>(x);
    p.T = (int)T;
    p.k = k;
    p.E = E;
    p.H = H;
    p.F = F;
    p.ids = ids;
    p.weights = weights;
    p.up_codes = up_codes;
    p.up_scales = up_scales;
    p.up_gs = up_gs;
    p.down_codes = down_codes;
    p.down_scales = down_scales;
    p.down_gs = down_gs;
    const MoeWs w = moe_ws(T, k, F, H);
    uint8_t *b = reinterpret_cast<uint8_t *>(ws);
    p.h = reinterpret_cast<uint4 *>(b);
    p.h_exp = b + w.exps;
    p.exp_pitch = (F / 32 + 7) / 8 * 8;
    p.y = reinterpret_cast<__nv_bfloat16 *>(y);
    p.splits = moe_splits(H);
    p.partial = reinterpret_cast<float *>(b + w.partial);
    p.arrived = reinterpret_cast<int *>(b + w.arrived);
    p.status = device_status_ptr();
    p.barrier = grid_barrier_for(s);
    if (!p.status || !p.barrier)
        return cudaErrorInvalidValue;
    return mx ? launch_experts_fmt<false>(p, s) : launch_experts_fmt<true>(p, s);
}

} // namespace nvfp4
