// mxfp4.cu -- MXFP4 quantize (along rows, columns or both in one read) and dequantize on sm_100a.
//
// The arithmetic is in mxfp4_encode.cuh. A block's scale depends on its own 32 values only, so
// there is no tensor-wide pass: one read, one write, HBM-bound.
//
// Quantize: one CTA per 128 x 128 tile of x, because both outputs of such a tile are whole units
// of the operand layout: along the rows, 128 rows x 64 code bytes and one 512-byte scale atom
// (128 rows x 4 blocks); along the columns the same of x^T. Every atom, padding included, is
// written by exactly one CTA, as one 512-byte run. A row's 128 values are 8 lanes x 16 bf16 (16
// lanes x 8 fp32): two 16-byte loads a lane, the block maximum by one (two) shuffles. The column
// side keeps the tile in shared memory; a thread takes 32 rows of two adjacent bf16 columns (of
// one fp32 column), reading words that are contiguous across the warp, and the codes go through
// shared memory so that they leave as whole 64-byte row pieces (bf16: over the tile, which leaves the
// SM more L1: a lane's two 16-byte loads touch each sector twice, and where the second finds it gone
// both directions take 40 us instead of 33).
//
// 4096 x 12288 bf16: along rows 21.0 us (6.1 TB/s), columns 22.9 us (5.6 TB/s), both 33.2 us (4.6
// TB/s). fp32 4096 x 8192: rows 27.3 us (5.6 TB/s), columns 33.7 us (4.5 TB/s), both 42.9 us (4.0 TB/s).
// "Both" and fp32 columns are at neither limit (67 % of the issue slots for bf16, 36 to 49 % for fp32):
// a CTA's loads, directions and stores follow one another, and registers (bf16) or shared memory (fp32)
// leave an SM 4 CTAs (bf16 both), 3 (fp32 columns) or 2 (fp32 both) to overlap them.
#include <mutex>

#include "mxfp4_encode.cuh"
#include "nvfp4_internal.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kColPitch = 80; // staged transposed codes: 64 bytes a column
constexpr int kStageBytes = kTile * kColPitch + 64;

// Byte of column c's staged codes: even columns, then odd ones half a bank row further, so that
// neither a warp's 16-byte stores (every other column) nor its loads (whole columns) conflict.
__device__ __forceinline__ int stage_offset(int c)
{
    return (c >> 1) * kColPitch + (c & 1) * (kTile / 2 * kColPitch + 64);
}

struct MxQuantParams {
    const void *x;
    int64_t rows, cols;
    int64_t tiles_c;      // 128-column tiles
    int ceil_rule;
    int aligned32; // x begins on a 32-byte boundary (its rows then do)
    uint8_t *codes, *swz, *lin;       // along rows (may be null)
    uint8_t *codes_t, *swz_t, *lin_t; // along columns
};

// 32 bytes at once (4096 x 12288 bf16 along rows: 22.2 -> 21.0 us). Not where the tile goes to shared
// memory, whose stores then wait for both halves (along columns 33 us instead of 23).
__device__ __forceinline__ void ld_v8(const uint4 *src, uint4 &a, uint4 &b)
{
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                   "=r"(b.w)
                 : "l"(src));
}

// The tile's 128 x 4 scale bytes (s_sf, in atom order) to the swizzled atom and the linear array
// [rows x nblk] at rows r0.., blocks b0...
__device__ __forceinline__ void store_scales(const uint32_t *s_sf, uint8_t *swz_atom, uint8_t *lin,
                                             int64_t r0, int64_t rows, int64_t b0, int64_t nblk)
{
    const int t = threadIdx.x;
    if (swz_atom && t < 32)
        reinterpret_cast<uint4 *>(swz_atom)[t] = reinterpret_cast<const uint4 *>(s_sf)[t];
    if (lin && t >= 128 && r0 + t - 128 < rows) {
        const int r = t - 128;
        const uint32_t w = s_sf[4 * (r & 31) + (r >> 5)];
        uint8_t *dst = lin + (r0 + r) * nblk + b0;
        if ((nblk & 3) == 0) {
            *reinterpret_cast<uint32_t *>(dst) = w;
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b0 + b < nblk)
                    dst[b] = (uint8_t)(w >> (8 * b));
        }
    }
}

template <bool BF16, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(const MxQuantParams p)
{
    constexpr int kEsz = BF16 ? 2 : 4;
    constexpr int kVec = COLS && !BF16 && !ROWS ? 1 : 2;   // 16-byte vectors a lane
    constexpr int kLanesPerRow = kTile * kEsz / (16 * kVec);
    constexpr int kRowsPerPass = kThreads / kLanesPerRow;
    constexpr int kPasses = kTile / kRowsPerPass;
    constexpr int kPitch = kTile * kEsz;                    // shared tile row, bytes
    extern __shared__ __align__(16) uint8_t dyn[];          // COLS: tile, then staged codes
    __shared__ __align__(16) uint32_t s_sf[128];
    __shared__ __align__(16) uint32_t s_sft[128];

    // The next kernel may set up meanwhile: a GEMM's operands wait for this grid's end (777 x 1001 x
    // 2080 with its quantize: 17.0 -> 16.0 us). This kernel itself is launched without that: its CTAs
    // among a running GEMM's are spread unevenly (a step of three quantizes and three products: 67 us,
    // 71 us with it).
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int64_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c;
    const int64_t r0 = tr * kTile, c0 = tc * kTile;
    const int lane_r = tid / kLanesPerRow, lane_c = tid % kLanesPerRow;
    const int col = lane_c * (16 * kVec / kEsz); // this lane's first column of the tile
    const bool col_ok = c0 + col < p.cols;
    // Half of the lanes take their second vector first: eight lanes' 16-byte shared stores at a stride
    // of 32 bytes then meet every bank once.
    const int flip = COLS && kVec == 2 ? (lane_c >> 2) & 1 : 0;

    uint4 v[kPasses][kVec];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = r0 + i * kRowsPerPass + lane_r;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            v[i][j] = make_uint4(0u, 0u, 0u, 0u);
        if (col_ok && r < p.rows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const uint8_t *>(p.x) + (r * p.cols + c0 + col) * kEsz);
            if (!COLS && p.aligned32) {
                ld_v8(src, v[i][0], v[i][kVec - 1]);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    v[i][j] = __ldg(src + (j ^ flip));
            }
        }
    }
    if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            uint4 *dst =
                reinterpret_cast<uint4 *>(dyn + (i * kRowsPerPass + lane_r) * kPitch) + lane_c * kVec;
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                dst[j ^ flip] = v[i][j];
        }
    }
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int row = i * kRowsPerPass + lane_r;
            static_assert(kVec == 2, "32 bytes a lane: a block is 2 lanes of bf16, 4 of fp32");
            constexpr int kLpb = 32 * kEsz / (16 * kVec); // lanes per block
            const uint4 a = v[i][0], b = v[i][1];
            uint32_t m;
            if constexpr (BF16) {
                m = max_abs_bf16x2(
                    max_abs_bf16x2(max_abs_bf16x2(a.x, a.y), max_abs_bf16x2(a.z, a.w)),
                    max_abs_bf16x2(max_abs_bf16x2(b.x, b.y), max_abs_bf16x2(b.z, b.w)));
                m &= kAbs16x2;
                m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max(m & 0xFFFFu, m >> 16) << 16;
            } else {
                m = max(max(max(a.x & 0x7FFFFFFFu, a.y & 0x7FFFFFFFu),
                            max(a.z & 0x7FFFFFFFu, a.w & 0x7FFFFFFFu)),
                        max(max(b.x & 0x7FFFFFFFu, b.y & 0x7FFFFFFFu),
                            max(b.z & 0x7FFFFFFFu, b.w & 0x7FFFFFFFu)));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            }
            const uint32_t sb = mx_scale_byte(m, p.ceil_rule != 0);
            const float inv = mx_inverse(sb);
            const bool live = col_ok && r0 + row < p.rows;
            uint8_t *dst = p.codes + ((r0 + row) * p.cols + c0 + col) / 2;
            if constexpr (BF16) {
                const uint32_t lo = mx_codes_bf16x8(a.x, a.y, a.z, a.w, inv);
                const uint32_t hi = mx_codes_bf16x8(b.x, b.y, b.z, b.w, inv);
                if (live)
                    *reinterpret_cast<uint2 *>(dst) =
                        sb == kMxNan ? make_uint2(0u, 0u)
                                     : make_uint2(flip ? hi : lo, flip ? lo : hi);
            } else {
                const uint32_t ab = mx_codes_f32x8(a, b, inv); // four codes in either half
                const uint32_t w = flip ? __byte_perm(ab, 0u, 0x1032) : ab;
                if (live)
                    *reinterpret_cast<uint32_t *>(dst) = sb == kMxNan ? 0u : w;
            }
            // the row's four scale bytes (padding rows and blocks: 0) into the atom's word
            uint32_t w = live ? sb << (8 * (lane_c / kLpb)) : 0u;
            w |= __shfl_xor_sync(0xFFFFFFFFu, w, kLpb);
            w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2 * kLpb);
            if (lane_c == 0)
                s_sf[4 * (row & 31) + (row >> 5)] = w;
        }
    }
    __syncthreads();
    if constexpr (ROWS) {
        const int64_t atom = tr * p.tiles_c + tc;
        store_scales(s_sf, p.swz ? p.swz + atom * 512 : nullptr, p.lin, r0, p.rows, c0 / 32,
                     p.cols / 32);
    }
    if constexpr (COLS) {
        // bf16: over the tile, once every thread has its share of it in registers
        uint8_t *stage = BF16 ? dyn : dyn + kTile * kPitch;
        uint8_t *sft = reinterpret_cast<uint8_t *>(s_sft);
        auto put = [&](int c, int blk, const uint32_t (&w)[4], uint32_t sb) {
            const bool nan = sb == kMxNan;
            *reinterpret_cast<uint4 *>(stage + stage_offset(c) + blk * 16) =
                nan ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(w[0], w[1], w[2], w[3]);
            // blocks past the last row and columns past the last are padding: 0
            const bool live = c0 + c < p.cols && r0 + blk * 32 < p.rows;
            sft[16 * (c & 31) + 4 * (c >> 5) + blk] = live ? (uint8_t)sb : (uint8_t)0;
        };
        if constexpr (BF16) {
            // 64 column pairs x 4 blocks = 256 threads
            const int cp = tid & 63, blk = tid >> 6;
            uint32_t u[32], m = 0u;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                u[k] = *reinterpret_cast<const uint32_t *>(dyn + (blk * 32 + k) * kPitch + cp * 4);
                m = max_abs_bf16x2(m, u[k]);
            }
            m &= kAbs16x2;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sb =
                    mx_scale_byte(h ? m & 0xFFFF0000u : m << 16, p.ceil_rule != 0);
                const float inv = mx_inverse(sb);
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const uint32_t a = u[8 * q + k], b = u[8 * q + k + 1];
                        const float2 f = __fmul2_rn(
                            make_float2(__uint_as_float(h ? a & 0xFFFF0000u : a << 16),
                                        __uint_as_float(h ? b & 0xFFFF0000u : b << 16)),
                            make_float2(inv, inv));
                        y[k] = f.x;
                        y[k + 1] = f.y;
                    }
                    w[q] = cvt_e2m1x8(y);
                }
                put(2 * cp + h, blk, w, sb);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) { // 128 columns x 4 blocks
                const int c = tid & 127, blk = (tid >> 7) + 2 * i;
                float u[32];
                uint32_t m = 0u;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    u[k] = *reinterpret_cast<const float *>(dyn + (blk * 32 + k) * kPitch + c * 4);
                    m = max(m, __float_as_uint(u[k]) & 0x7FFFFFFFu);
                }
                const uint32_t sb = mx_scale_byte(m, p.ceil_rule != 0);
                const float inv = mx_inverse(sb);
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 f = __fmul2_rn(make_float2(u[8 * q + k], u[8 * q + k + 1]),
                                                    make_float2(inv, inv));
                        y[k] = f.x;
                        y[k + 1] = f.y;
                    }
                    w[q] = cvt_e2m1x8(y);
                }
                put(c, blk, w, sb);
            }
        }
        __syncthreads();
        const int64_t tiles_r = (p.rows + kTile - 1) / kTile;
        const int64_t nblk = (p.rows + 31) / 32; // blocks of a row of x^T
        const int64_t atom = tc * tiles_r + tr;
        store_scales(s_sft, p.swz_t ? p.swz_t + atom * 512 : nullptr, p.lin_t, c0, p.cols,
                     r0 / 32, nblk);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int idx = i * kThreads + tid, c = idx >> 2, q = idx & 3;
            if (c0 + c < p.cols && r0 / 32 + q < nblk)
                *reinterpret_cast<uint4 *>(p.codes_t + ((c0 + c) * nblk + r0 / 32 + q) * 16) =
                    *reinterpret_cast<const uint4 *>(stage + stage_offset(c) + q * 16);
        }
    }
}

template <bool BF16, bool ROWS, bool COLS>
cudaError_t launch_mx_quantize_t(const MxQuantParams &p, unsigned grid, cudaStream_t s)
{
    const int smem = !COLS ? 0 : BF16 ? kTile * kTile * 2 : kTile * kTile * 4 + kStageBytes;
    static_assert(kStageBytes <= kTile * kTile * 2, "bf16: the staged codes lie over the tile");
    if (COLS && !BF16) {
        static std::once_flag flags[64];
        int dev = 0;
        cudaGetDevice(&dev);
        cudaError_t e = cudaSuccess;
        std::call_once(flags[dev & 63], [&]() {
            e = cudaFuncSetAttribute(mx_quantize_kernel<BF16, ROWS, COLS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        });
        if (e != cudaSuccess)
            return e;
    }
    mx_quantize_kernel<BF16, ROWS, COLS><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

// ---- dequantize ----------------------------------------------------------------------

__device__ __forceinline__ void st_v8(void *p, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A lane decodes half a block (8 code bytes, 16 values) per step: a warp's loads are contiguous
// (256 bytes of codes) and so are its stores (1 KB of bf16), 32 bytes at a time where the output is
// aligned to that (V8; 16-byte stores at a 32-byte stride fill the store queue: 32 us instead of
// 24 us for 4096 x 12288 bf16). Four halves a step, the next step's loads in flight.
template <bool BF16, bool V8>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ lin,
                         int64_t halves, void *__restrict__ out)
{
    constexpr int kSteps = 4;
    const uint2 *cb = reinterpret_cast<const uint2 *>(codes);
    uint8_t *ob = reinterpret_cast<uint8_t *>(out);
    const int64_t stride = (int64_t)gridDim.x * kThreads * kSteps;
    int64_t h0 = (int64_t)blockIdx.x * kThreads * kSteps + threadIdx.x;
    uint2 c[kSteps], cn[kSteps];
    uint32_t sb[kSteps], sn[kSteps];
    auto load = [&](int64_t h1, uint2 (&cc)[kSteps], uint32_t (&ss)[kSteps]) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t h = h1 + (int64_t)i * kThreads;
            cc[i] = h < halves ? __ldg(cb + h) : make_uint2(0u, 0u);
            ss[i] = h < halves ? __ldg(lin + (h >> 1)) : 0u;
        }
    };
    load(h0, c, sb);
    for (; h0 < halves; h0 += stride) {
        load(h0 + stride, cn, sn);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t h = h0 + (int64_t)i * kThreads;
            if (h >= halves)
                break;
            const float s = mx_scale_f32(sb[i]);
            uint32_t w[BF16 ? 8 : 16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 e =
                    e2m1x2_to_f32x2(((j < 4 ? c[i].x : c[i].y) >> (8 * (j & 3))) & 0xFFu);
                const float lo = __fmul_rn(e.x, s), hi = __fmul_rn(e.y, s);
                if constexpr (BF16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
                    w[j] = *reinterpret_cast<const uint32_t *>(&b);
                } else {
                    w[2 * j] = __float_as_uint(lo);
                    w[2 * j + 1] = __float_as_uint(hi);
                }
            }
            constexpr int kWords = BF16 ? 8 : 16;
            uint8_t *o = ob + h * (kWords * 4);
#pragma unroll
            for (int j = 0; j < kWords; j += 8) {
                if constexpr (V8) {
                    st_v8(o + 4 * j, w + j);
                } else {
                    reinterpret_cast<uint4 *>(o + 4 * j)[0] =
                        make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                    reinterpret_cast<uint4 *>(o + 4 * j)[1] =
                        make_uint4(w[j + 4], w[j + 5], w[j + 6], w[j + 7]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            c[i] = cn[i];
            sb[i] = sn[i];
        }
    }
}

} // namespace

cudaError_t launch_quantize_mx(const void *x, int src_bf16, int64_t rows, int64_t cols,
                               int ceil_rule, uint8_t *codes, uint8_t *swz, uint8_t *lin,
                               uint8_t *codes_t, uint8_t *swz_t, uint8_t *lin_t, cudaStream_t s)
{
    if (rows == 0 || cols == 0)
        return cudaSuccess;
    const int aligned32 = (reinterpret_cast<uintptr_t>(x) & 31u) == 0;
    MxQuantParams p{x, rows, cols, (cols + kTile - 1) / kTile, ceil_rule, aligned32, codes, swz, lin,
                    codes_t, swz_t, lin_t};
    const unsigned grid = (unsigned)(((rows + kTile - 1) / kTile) * p.tiles_c);
    if (codes && codes_t)
        return src_bf16 ? launch_mx_quantize_t<true, true, true>(p, grid, s)
                        : launch_mx_quantize_t<false, true, true>(p, grid, s);
    if (codes_t)
        return src_bf16 ? launch_mx_quantize_t<true, false, true>(p, grid, s)
                        : launch_mx_quantize_t<false, false, true>(p, grid, s);
    return src_bf16 ? launch_mx_quantize_t<true, true, false>(p, grid, s)
                    : launch_mx_quantize_t<false, true, false>(p, grid, s);
}

cudaError_t launch_dequantize_mx(const uint8_t *codes, const uint8_t *lin, int64_t rows,
                                 int64_t cols, int out_bf16, void *out, cudaStream_t s)
{
    const int64_t halves = rows * (cols / 16);
    if (halves == 0)
        return cudaSuccess;
    int64_t g = (halves + kThreads * 4 - 1) / (kThreads * 4);
    const int64_t cap = (int64_t)num_sms() * 8;
    if (g > cap)
        g = cap;
    const bool v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    const dim3 grid((unsigned)g);
    if (out_bf16 && v8)
        mx_dequantize_kernel<true, true><<<grid, kThreads, 0, s>>>(codes, lin, halves, out);
    else if (out_bf16)
        mx_dequantize_kernel<true, false><<<grid, kThreads, 0, s>>>(codes, lin, halves, out);
    else if (v8)
        mx_dequantize_kernel<false, true><<<grid, kThreads, 0, s>>>(codes, lin, halves, out);
    else
        mx_dequantize_kernel<false, false><<<grid, kThreads, 0, s>>>(codes, lin, halves, out);
    return cudaGetLastError();
}

} // namespace nvfp4
