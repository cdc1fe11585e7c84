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

// Sum of the eight products of two 16-byte bf16 vectors: exact products, fp32 sums.
__device__ __forceinline__ float dot8(const uint4 &a, const float (&x)[8])
{
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(u[i] << 16), x[2 * i], s);
        s = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), x[2 * i + 1], s);
    }
    return s;
}

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v)
{
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// A cluster of 8 CTAs takes TG tokens: its warps share the experts out, one logit per expert and
// token by a warp (eight-term fp32 sums added up in fp64, so that the choice between two close
// experts does not hang on the order of a long sum), sent to the CTA that ranks the token.
// Expert e is chosen if fewer than k experts precede it: rank by counting, every thread at once.
template <int TG>
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
    moe_route_kernel(const RouteParams p)
{
    extern __shared__ __align__(16) double s_z[]; // [E], this CTA's token
    __shared__ int s_sel[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * TG;
    const int64_t nvec = p.H >> 3;
    cluster_arrive(); // matched below: every CTA of the cluster runs before remote stores
    pdl_wait();
    cluster_wait();
    const uint32_t zaddr = smem_u32(s_z);
    for (int e = (int)rank * 8 + warp; e < p.E; e += 8 * kRouteCluster) {
        double acc[TG];
#pragma unroll
        for (int j = 0; j < TG; ++j)
            acc[j] = 0.0;
#pragma unroll 4
        for (int64_t i = lane; i < nvec; i += 32) {
            const uint4 a = __ldg(p.w + (int64_t)e * nvec + i);
#pragma unroll
            for (int j = 0; j < TG; ++j) {
                if (t0 + j < p.T) {
                    const uint4 v = __ldg(p.x + (t0 + j) * nvec + i);
                    const float xf[8] = {
                        __uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                        __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u),
                        __uint_as_float(v.z << 16), __uint_as_float(v.z & 0xFFFF0000u),
                        __uint_as_float(v.w << 16), __uint_as_float(v.w & 0xFFFF0000u)};
                    acc[j] += (double)dot8(a, xf);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < TG; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
            double z = acc[j] + (p.bias ? (double)__ldg(p.bias + e) : 0.0);
            if (!(z == z))
                z = -INFINITY; // a NaN logit is never chosen
            if (lane == 0)
                st_cluster_f64(mapa_shared(zaddr + 8u * (uint32_t)e, (uint32_t)j), z);
        }
    }
    cluster_sync(); // this CTA's token has all its logits
    pdl_launch_dependents();
    const int64_t t = t0 + rank;
    if (rank >= TG || t >= p.T)
        return;
    if (tid < 32)
        s_sel[tid] = -1;
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
            p.ids[t * p.k + lane] = e;
            p.weights[t * p.k + lane] = e >= 0 ? v / sum : 0.0f;
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
};

// What the ids say, in shared memory: for each expert the set of its tokens; the (expert, token)
// pairs in expert order as rows, with the row's token and weight (an expert that a token names
// twice gets one row with both weights); and the column tiles, up to cols rows of one expert each.
// ids outside [0, E) name no expert.
struct MoeLists {
    uint32_t *mask;   // [E][2]
    int *base;        // [E] first row of each expert
    int *unit;        // [tiles] expert | first column of the tile << 16
    uint8_t *tok;     // [rows]
    float *wt;        // [rows]
    int *ids;         // [T k]
    int *n_units;
};

__host__ __device__ inline size_t moe_lists_bytes(int T, int k, int E)
{
    const size_t n = (size_t)T * k;
    return 8 * (size_t)E + 4 * (size_t)E + 4 * n + 4 * n + 4 * n + 16 + (n + 15) / 16 * 16;
}

__device__ __forceinline__ MoeLists moe_lists(uint8_t *s, int T, int k, int E)
{
    const int n = T * k;
    MoeLists l;
    l.mask = reinterpret_cast<uint32_t *>(s);
    l.base = reinterpret_cast<int *>(l.mask + 2 * E);
    l.unit = l.base + E;
    l.wt = reinterpret_cast<float *>(l.unit + n);
    l.ids = reinterpret_cast<int *>(l.wt + n);
    l.n_units = l.ids + n;
    l.tok = reinterpret_cast<uint8_t *>(l.n_units + 4);
    return l;
}

__device__ __forceinline__ int mask_count(const uint32_t *m) { return __popc(m[0]) + __popc(m[1]); }

// Rows of the expert's tokens before token t.
__device__ __forceinline__ int mask_before(const uint32_t *m, int t)
{
    return t < 32 ? __popc(m[0] & ((1u << t) - 1u))
                  : __popc(m[0]) + __popc(m[1] & ((1u << (t - 32)) - 1u));
}

template <bool WEIGHTS>
__device__ __forceinline__ void build_lists(const MoeLists &l, const MoeParams &p, int cols)
{
    const int tid = threadIdx.x, nthr = blockDim.x, n = p.T * p.k;
    for (int i = tid; i < 2 * p.E; i += nthr)
        l.mask[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = __ldg(p.ids + i), t = i / p.k;
        l.ids[i] = e;
        if (e >= 0 && e < p.E)
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
                l.unit[u0++] = e | c0 << 16;
            r0 += c;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
        const int e = l.ids[i], t = i / p.k;
        if (e < 0 || e >= p.E)
            continue;
        bool first = true; // of the token's slots that name e
        float w = 0.0f;
        for (int s = t * p.k; s < (t + 1) * p.k; ++s)
            if (l.ids[s] == e) {
                first = first && s >= i;
                if (WEIGHTS)
                    w += __ldg(p.weights + s);
            }
        if (first) {
            const int row = l.base[e] + mask_before(l.mask + 2 * e, t);
            l.tok[row] = (uint8_t)t;
            if (WEIGHTS)
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

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Lane t's four code bytes of the 32-code block at `a`: bytes 4t.. (MXFP4), or bytes 2t, 2t + 1 of
// each of its two 16-code blocks (NVFP4).
template <bool NV> __device__ __forceinline__ uint32_t lane_codes(uint32_t a, int t)
{
    if constexpr (NV) {
        const uint32_t h = a + 4 * (t >> 1);
        return __byte_perm(lds32(h), lds32(h + 8), (t & 1) ? 0x7632 : 0x5410);
    } else {
        return lds32(a + 4 * t);
    }
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

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Warp-private ring of weight tiles: MT x 16 rows x 128 codes (64 bytes at an 80-byte pitch: the
// fragment loads of eight rows x four lanes hit 32 banks) and the rows' scale bytes of the tile
// (4 MXFP4, 8 NVFP4), fetched as the aligned words that hold them, since a row of scales may start
// at any byte.
template <int MT, bool NV> struct Tile {
    static constexpr int kRows = MT * 16;
    static constexpr int kPitch = 80;
    static constexpr int kSlot = NV ? 16 : 8;
    static constexpr int kScaleBytes = NV ? 8 : 4; // of one row and tile
    static constexpr int kOffScales = kRows * kPitch;
    static constexpr int kBytes = kOffScales + kRows * kSlot;
};

// One tile's copies: local row r is row row_of(r) of the expert's matrix (K columns).
template <int MT, bool NV, typename RowOf>
__device__ __forceinline__ void load_tile(uint32_t dst, const uint8_t *codes, const uint8_t *scales,
                                          int64_t K, int kt, int lane, RowOf row_of)
{
    using L = Tile<MT, NV>;
    const int nblk = (int)(K >> 5);
#pragma unroll
    for (int j = 0; j < MT * 2; ++j) {
        const int r = j * 8 + (lane >> 2), c = lane & 3;
        if (kt * 4 + c < nblk)
            cp_async16(dst + r * L::kPitch + c * 16, codes + row_of(r) * (K >> 1) + kt * 64 + c * 16);
    }
    const int64_t srow = NV ? K >> 4 : K >> 5;
    const int64_t k0 = (int64_t)kt * L::kScaleBytes;
    const int64_t left = srow - k0;
    const int nb = left < L::kScaleBytes ? (int)left : L::kScaleBytes;
#pragma unroll
    for (int j = 0; j < (L::kRows + 31) / 32; ++j) {
        const int r = j * 32 + lane;
        if (r < L::kRows) {
            const int64_t off = row_of(r) * srow + k0;
            const int64_t a = off & ~(int64_t)3;
#pragma unroll
            for (int w = 0; w < (NV ? 3 : 2); ++w)
                if (a + 4 * w < off + nb)
                    cp_async4(dst + L::kOffScales + r * L::kSlot + 4 * w, scales + a + 4 * w);
        }
    }
}

// Scale bytes of local row r (whose row of scales starts at byte offset sh8 / 8 of a word):
// MXFP4 one word, NVFP4 two.
template <int MT, bool NV>
__device__ __forceinline__ void tile_scales(uint32_t tile, int r, uint32_t sh8, uint32_t (&s)[NV ? 2 : 1])
{
    using L = Tile<MT, NV>;
    const uint32_t a = tile + L::kOffScales + r * L::kSlot;
    const uint32_t w0 = lds32(a), w1 = lds32(a + 4);
    s[0] = __funnelshift_r(w0, w1, sh8);
    if constexpr (NV)
        s[1] = __funnelshift_r(w1, lds32(a + 8), sh8);
}

// Activations of one column tile and one 32-block as MMA B fragments: f16 pairs, and the scales of
// this lane's two accumulator columns.
struct BFrag {
    uint32_t u[4];
    float s0, s1;
};

// acc += tile x activations, over the tile's nb 32-blocks. frag(nt, b) gives the B fragments.
template <int MT, int NT, bool NV, typename Frag>
__device__ __forceinline__ void tile_product(float (&acc)[MT][NT][4], uint32_t tile, int nb, int lane,
                                             const uint32_t (&sh)[MT][2], Frag frag)
{
    using L = Tile<MT, NV>;
    const int g = lane >> 2, t = lane & 3;
    uint32_t sc[MT][2][NV ? 2 : 1];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        tile_scales<MT, NV>(tile, m * 16 + g, sh[m][0], sc[m][0]);
        tile_scales<MT, NV>(tile, m * 16 + g + 8, sh[m][1], sc[m][1]);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b >= nb)
            break;
        BFrag f[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            f[n] = frag(n, b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t ra = tile + (m * 16 + g) * L::kPitch + b * 16;
            const uint32_t rb = ra + 8 * L::kPitch;
            const uint32_t w0 = lane_codes<NV>(ra, t), w1 = lane_codes<NV>(rb, t);
            // k16 step, fragment: rows g and g + 8, k indices 2t.. and 2t + 8..
            const uint32_t a[2][4] = {
                {e2m1x2_to_f16x2<0>(w0), e2m1x2_to_f16x2<0>(w1), e2m1x2_to_f16x2<1>(w0),
                 e2m1x2_to_f16x2<1>(w1)},
                {e2m1x2_to_f16x2<2>(w0), e2m1x2_to_f16x2<2>(w1), e2m1x2_to_f16x2<3>(w0),
                 e2m1x2_to_f16x2<3>(w1)}};
            if constexpr (NV) {
                const uint32_t sa = sc[m][0][b >> 1] >> (16 * (b & 1));
                const uint32_t sb = sc[m][1][b >> 1] >> (16 * (b & 1));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float s0 = e4m3_to_f32(sa >> (8 * k)), s1 = e4m3_to_f32(sb >> (8 * k));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_f16(c, a[k][0], a[k][1], a[k][2], a[k][3], f[n].u[2 * k],
                                f[n].u[2 * k + 1]);
                        acc[m][n][0] = fmaf(c[0] * f[n].s0, s0, acc[m][n][0]);
                        acc[m][n][1] = fmaf(c[1] * f[n].s1, s0, acc[m][n][1]);
                        acc[m][n][2] = fmaf(c[2] * f[n].s0, s1, acc[m][n][2]);
                        acc[m][n][3] = fmaf(c[3] * f[n].s1, s1, acc[m][n][3]);
                    }
                }
            } else {
                const float s0 = mx_scale_f32((sc[m][0][0] >> (8 * b)) & 0xFFu);
                const float s1 = mx_scale_f32((sc[m][1][0] >> (8 * b)) & 0xFFu);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(c, a[0][0], a[0][1], a[0][2], a[0][3], f[n].u[0], f[n].u[1]);
                    mma_f16(c, a[1][0], a[1][1], a[1][2], a[1][3], f[n].u[2], f[n].u[3]);
                    acc[m][n][0] = fmaf(c[0] * f[n].s0, s0, acc[m][n][0]);
                    acc[m][n][1] = fmaf(c[1] * f[n].s1, s0, acc[m][n][1]);
                    acc[m][n][2] = fmaf(c[2] * f[n].s0, s1, acc[m][n][2]);
                    acc[m][n][3] = fmaf(c[3] * f[n].s1, s1, acc[m][n][3]);
                }
            }
        }
    }
}

// The 8 activations (16 bits each) of lane t's k indices of block blk of a row: consecutive
// (MXFP4), or 4 of each 16-block (NVFP4).
template <bool NV>
__device__ __forceinline__ uint4 load_b(const uint4 *row, int blk, int t)
{
    if constexpr (NV) {
        const uint2 *r = reinterpret_cast<const uint2 *>(row + 4 * blk);
        const uint2 a = r[t], b = r[4 + t];
        return make_uint4(a.x, a.y, b.x, b.y);
    } else {
        return row[4 * blk + t];
    }
}

constexpr int kUpWarps = 4, kUpStages = 4, kUpMt = 4;

// h = silu(gate) * up for 32 columns of F (64 weight rows) of one column tile. The warps split the
// k-tiles and their sums meet in shared memory. m-tile i holds gate rows f0 + 8i.. in its first
// eight rows and the same up rows in the other eight, so a lane's accumulators hold both sides of
// its products.
template <int NT, bool NV>
__global__ void __launch_bounds__(kUpWarps * 32, 2) moe_up_kernel(const MoeParams p)
{
    using L = Tile<kUpMt, NV>;
    constexpr int NC = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem;
    const MoeLists l = moe_lists(smem + kUpWarps * kUpStages * L::kBytes, p.T, p.k, p.E);
    pdl_wait();
    build_lists<false>(l, p, NC);
    pdl_launch_dependents(); // everything before this kernel is complete: see moe_down_kernel
    if ((int)blockIdx.y >= *l.n_units)
        return;
    const int unit = l.unit[blockIdx.y];
    const int e = unit & 0xFFFF, c0 = unit >> 16;
    const int row0 = l.base[e] + c0;
    const int ncol = min(NC, mask_count(l.mask + 2 * e) - c0);
    const int64_t f0 = (int64_t)blockIdx.x * 32;
    const int nblk = (int)(p.H >> 5), nkt = (nblk + 3) >> 2;
    const int64_t srow = NV ? p.H >> 4 : p.H >> 5;
    const uint8_t *codes = p.up_codes + (int64_t)e * 2 * p.F * (p.H >> 1);
    const uint8_t *scales = p.up_scales + (int64_t)e * 2 * p.F * srow;
    auto row_of = [&](int r) {
        return f0 + (r >> 4) * 8 + (r & 7) + ((r & 8) ? p.F : (int64_t)0);
    };
    const uint32_t my = smem_u32(ring) + warp * kUpStages * L::kBytes;
    const int mine = nkt > warp ? (nkt - warp + kUpWarps - 1) / kUpWarps : 0;
    auto issue = [&](int i) {
        if (i < mine)
            load_tile<kUpMt, NV>(my + (i % kUpStages) * L::kBytes, codes, scales, p.H,
                                 warp + i * kUpWarps, lane, row_of);
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kUpStages - 1; ++i)
        issue(i);
    const uint4 *xrow[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xrow[n] = n * 8 + g < ncol ? p.x + (int64_t)l.tok[row0 + n * 8 + g] * (p.H >> 3) : nullptr;
    uint4 bv[NT][4];
    auto fetch = [&](int i) {
        const int kt = warp + i * kUpWarps;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                bv[n][b] = xrow[n] && i < mine && kt * 4 + b < nblk ? load_b<NV>(xrow[n], kt * 4 + b, t)
                                                                   : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch(0);
    uint32_t sh[kUpMt][2];
#pragma unroll
    for (int m = 0; m < kUpMt; ++m) {
        sh[m][0] = (uint32_t)((row_of(m * 16 + g) * srow) & 3) * 8u;
        sh[m][1] = (uint32_t)((row_of(m * 16 + g + 8) * srow) & 3) * 8u;
    }
    float acc[kUpMt][NT][4] = {};
    for (int i = 0; i < mine; ++i) {
        issue(i + kUpStages - 1);
        cp_async_wait<kUpStages - 1>();
        __syncwarp();
        uint4 cur[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                cur[n][b] = bv[n][b];
        fetch(i + 1);
        const int nb = min(4, nblk - (warp + i * kUpWarps) * 4);
        tile_product<kUpMt, NT, NV>(
            acc, my + (i % kUpStages) * L::kBytes, nb, lane, sh, [&](int n, int b) {
                const uint4 v = cur[n][b];
                uint32_t m = max_u16x2(max_u16x2(v.x & kAbs16x2, v.y & kAbs16x2),
                                       max_u16x2(v.z & kAbs16x2, v.w & kAbs16x2));
                m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const uint32_t ex = block_exponent(max(m & 0xFFFFu, m >> 16) << 16);
                const float inv = __uint_as_float((254u - ex) << 23);
                BFrag f;
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f.u[q] = pack_f16x2(__uint_as_float(u[q] << 16) * inv,
                                        __uint_as_float(u[q] & 0xFFFF0000u) * inv);
                // this lane's accumulator columns are 2t and 2t + 1
                f.s0 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, ex, 8 * t) << 23);
                f.s1 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, ex, 8 * t + 4) << 23);
                return f;
            });
        __syncwarp(); // the tile is read before its slot is filled again
    }
    cp_async_wait<0>();
    __syncthreads();
    // sums of the warps, in warp order
    float4 *red = reinterpret_cast<float4 *>(ring); // [warp][m][n][lane]
#pragma unroll
    for (int m = 0; m < kUpMt; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            red[((warp * kUpMt + m) * NT + n) * 32 + lane] =
                make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
    float *s_h = reinterpret_cast<float *>(red + kUpWarps * kUpMt * NT * 32); // [NC][32]
    __syncthreads();
    const float gs = NV ? __ldg(p.up_gs + e) : 1.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) { // warp = m-tile
        float4 s = red[(warp * NT + n) * 32 + lane];
#pragma unroll
        for (int w = 1; w < kUpWarps; ++w) {
            const float4 q = red[((w * kUpMt + warp) * NT + n) * 32 + lane];
            s.x += q.x;
            s.y += q.y;
            s.z += q.z;
            s.w += q.w;
        }
        auto gated = [&](float a, float b) {
            const float ga = a * gs;
            return ga / (1.0f + __expf(-ga)) * (b * gs);
        };
        s_h[(n * 8 + 2 * t) * 32 + warp * 8 + g] = gated(s.x, s.z);
        s_h[(n * 8 + 2 * t + 1) * 32 + warp * 8 + g] = gated(s.y, s.w);
    }
    __syncthreads();
    for (int c = warp; c < ncol; c += kUpWarps) {
        const float v = s_h[c * 32 + lane];
        const uint32_t m =
            __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
        const uint32_t ex = block_exponent(m);
        const __half hv = __float2half_rn(v * __uint_as_float((254u - ex) << 23));
        const int64_t row = row0 + c;
        reinterpret_cast<__half *>(p.h)[row * p.F + f0 + lane] = hv;
        if (lane == 0)
            p.h_exp[row * p.exp_pitch + (f0 >> 5)] = (uint8_t)ex;
    }
}

constexpr int kDownWarps = 8, kDownStages = 8;

// y for 16 columns of H: the (column tile, k-tile) pairs of all met experts are shared out over
// the warps in runs; a warp's sums of one column tile are weighted and added to its own
// [16 x T] array, and the warps' arrays are added in warp order.
template <int NT, bool NV>
__global__ void __launch_bounds__(kDownWarps * 32) moe_down_kernel(const MoeParams p)
{
    using L = Tile<1, NV>;
    constexpr int NC = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem;
    float *ysum = reinterpret_cast<float *>(smem + kDownWarps * kDownStages * L::kBytes);
    const MoeLists l = moe_lists(reinterpret_cast<uint8_t *>(ysum + kDownWarps * 16 * p.T), p.T,
                                 p.k, p.E);
    for (int i = tid; i < kDownWarps * 16 * p.T; i += kDownWarps * 32)
        ysum[i] = 0.0f;
    // This grid starts once every CTA of moe_up_kernel is past its own wait for the stream's
    // earlier work, so the ids, the weights and the experts' codes are already complete; only h
    // (and y's readers) need the wait below.
    build_lists<true>(l, p, NC);
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    const int nblk = (int)(p.F >> 5), nkt = (nblk + 3) >> 2;
    const int64_t srow = NV ? p.F >> 4 : p.F >> 5;
    const int total = *l.n_units * nkt;
    const int u0 = (int)((int64_t)total * warp / kDownWarps);
    const int u1 = (int)((int64_t)total * (warp + 1) / kDownWarps);
    const uint32_t my = smem_u32(ring) + warp * kDownStages * L::kBytes;
    auto row_of = [&](int r) { return r0 + r; };
    auto issue = [&](int u) {
        if (u < u1) {
            const int64_t e = l.unit[u / nkt] & 0xFFFF;
            load_tile<1, NV>(my + ((u - u0) % kDownStages) * L::kBytes,
                             p.down_codes + e * p.H * (p.F >> 1), p.down_scales + e * p.H * srow,
                             p.F, u % nkt, lane, row_of);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDownStages - 1; ++i)
        issue(u0 + i);
    pdl_wait(); // h
    uint4 bv[NT][4];
    uint32_t ev[NT][2]; // exponents of this lane's accumulator columns, one byte per block
    auto fetch = [&](int u) {
        const bool on = u < u1;
        const int unit = on ? l.unit[u / nkt] : 0, kt = on ? u % nkt : 0;
        const int e = unit & 0xFFFF, c0 = unit >> 16;
        const int row = l.base[e] + c0;
        const int ncol = on ? min(NC, mask_count(l.mask + 2 * e) - c0) : 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 *hr = p.h + (int64_t)(row + n * 8 + g) * (p.F >> 3);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                bv[n][b] = n * 8 + g < ncol && kt * 4 + b < nblk ? load_b<NV>(hr, kt * 4 + b, t)
                                                                : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = n * 8 + 2 * t + j;
                ev[n][j] = c < ncol ? *reinterpret_cast<const uint32_t *>(
                                          p.h_exp + (int64_t)(row + c) * p.exp_pitch + kt * 4)
                                    : 0u;
            }
        }
    };
    fetch(u0);
    uint32_t sh[1][2];
    sh[0][0] = (uint32_t)(((r0 + g) * srow) & 3) * 8u;
    sh[0][1] = (uint32_t)(((r0 + g + 8) * srow) & 3) * 8u;
    float acc[1][NT][4] = {};
    float *mysum = ysum + warp * 16 * p.T;
    for (int u = u0; u < u1; ++u) {
        issue(u + kDownStages - 1);
        cp_async_wait<kDownStages - 1>();
        __syncwarp();
        uint4 cur[NT][4];
        uint32_t ec[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                cur[n][b] = bv[n][b];
            ec[n][0] = ev[n][0];
            ec[n][1] = ev[n][1];
        }
        fetch(u + 1);
        const int kt = u % nkt;
        tile_product<1, NT, NV>(acc, my + ((u - u0) % kDownStages) * L::kBytes,
                                min(4, nblk - kt * 4), lane, sh, [&](int n, int b) {
                                    BFrag f;
                                    f.u[0] = cur[n][b].x;
                                    f.u[1] = cur[n][b].y;
                                    f.u[2] = cur[n][b].z;
                                    f.u[3] = cur[n][b].w;
                                    f.s0 = __uint_as_float(((ec[n][0] >> (8 * b)) & 0xFFu) << 23);
                                    f.s1 = __uint_as_float(((ec[n][1] >> (8 * b)) & 0xFFu) << 23);
                                    return f;
                                });
        if (kt == nkt - 1 || u == u1 - 1) { // the column tile's last k-tile of this warp
            const int unit = l.unit[u / nkt];
            const int e = unit & 0xFFFF, c0 = unit >> 16;
            const int row = l.base[e] + c0;
            const int ncol = min(NC, mask_count(l.mask + 2 * e) - c0);
            const float gs = NV ? __ldg(p.down_gs + e) : 1.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = n * 8 + 2 * t + j;
                    if (c < ncol) {
                        const float w = l.wt[row + c];
                        const int tok = l.tok[row + c];
                        mysum[g * p.T + tok] = fmaf(acc[0][n][j] * gs, w, mysum[g * p.T + tok]);
                        mysum[(g + 8) * p.T + tok] =
                            fmaf(acc[0][n][2 + j] * gs, w, mysum[(g + 8) * p.T + tok]);
                    }
                    acc[0][n][j] = acc[0][n][2 + j] = 0.0f;
                }
        }
        __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    for (int i = tid; i < 16 * p.T; i += kDownWarps * 32) {
        const int r = i & 15, tk = i >> 4;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWarps; ++w)
            s += ysum[(w * 16 + r) * p.T + tk];
        p.y[tk * p.H + r0 + r] = __float2bfloat16_rn(s);
    }
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s,
                       const MoeParams &p)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int NT, bool NV> cudaError_t launch_experts(const MoeParams &p, cudaStream_t s)
{
    const size_t lists = moe_lists_bytes(p.T, p.k, p.E);
    // column tiles there can be at most: one per (token, expert) pair, and per expert the pairs
    // it may have beyond whole tiles
    const int n = p.T * p.k;
    const int units = n < p.E ? n : p.E + n / (8 * NT);
    cudaError_t e = launch_pdl(moe_up_kernel<NT, NV>,
                               dim3((unsigned)(p.F / 32), (unsigned)(units < n ? units : n), 1),
                               kUpWarps * 32,
                               kUpWarps * kUpStages * Tile<kUpMt, NV>::kBytes + lists, s, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(moe_down_kernel<NT, NV>, dim3((unsigned)(p.H / 16), 1, 1), kDownWarps * 32,
                      kDownWarps * kDownStages * Tile<1, NV>::kBytes +
                          (size_t)kDownWarps * 16 * p.T * 4 + lists,
                      s, p);
}

} // namespace

size_t moe_workspace_bytes(int64_t T, int64_t k, int64_t F)
{
    const size_t rows = (size_t)T * (size_t)k;
    const size_t h = (rows * (size_t)F * 2 + 255) & ~(size_t)255;
    return h + rows * (size_t)((F / 32 + 3) / 4 * 4);
}

cudaError_t launch_moe_route(const void *x, const void *w, const float *bias, int64_t T, int64_t H,
                             int E, int k, int renorm, int *ids, float *weights, cudaStream_t s)
{
    RouteParams p{reinterpret_cast<const uint4 *>(x), reinterpret_cast<const uint4 *>(w), bias, T,
                  H, E, k, renorm, ids, weights};
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)E * 8;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int tg = T <= 16 ? 1 : T <= 32 ? 2 : 4;
    cfg.gridDim = dim3((unsigned)((T + tg - 1) / tg * kRouteCluster), 1, 1);
    if (tg == 1)
        return cudaLaunchKernelEx(&cfg, moe_route_kernel<1>, p);
    if (tg == 2)
        return cudaLaunchKernelEx(&cfg, moe_route_kernel<2>, p);
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<4>, p);
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
    p.h = reinterpret_cast<uint4 *>(ws);
    p.h_exp = reinterpret_cast<uint8_t *>(ws) + (((size_t)T * k * F * 2 + 255) & ~(size_t)255);
    p.exp_pitch = (F / 32 + 3) / 4 * 4;
    p.y = reinterpret_cast<__nv_bfloat16 *>(y);
    // one column tile of 8 tokens per expert, two where an expert meets more than that on average
    const bool wide = T * k > 8 * (int64_t)E;
    if (mx)
        return wide ? launch_experts<2, false>(p, s) : launch_experts<1, false>(p, s);
    return wide ? launch_experts<2, true>(p, s) : launch_experts<1, true>(p, s);
}

} // namespace nvfp4
