// fp4_format.cuh -- the two FP4 operand formats of the block-scaled tensor-core kernels: what their
// scale atoms look like, how they reach tensor memory, and the MMA that reads them.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace nvfp4 {

// Operand formats. Both hold E2M1 codes in 256-wide k-tiles of 128 bytes a row; they differ in
// the scales only. NVFP4: one E4M3 byte per 16 values, so a k-tile has four scale atoms (128
// rows x 4 blocks) and each K64 MMA takes the four bytes of one atom (scale_vec::4X). MXFP4: one
// E8M0 byte per 32 values, two atoms per k-tile, and each K64 MMA takes half of an atom's four
// bytes (scale_vec::2X; the scale-factor ids in the instruction descriptor, 0 or 2, say which).
// MXFP4 has no global scale: alpha = 1.
struct FmtNvfp4 {
    static constexpr bool kMx = false;
    static constexpr int kAtoms = 4;  // scale atoms per k-tile and 128-row band
    static constexpr int kBlock = 16; // values per scale
    static constexpr uint32_t kIdesc = 0u;
};
struct FmtMxfp4 {
    static constexpr bool kMx = true;
    static constexpr int kAtoms = 2;
    static constexpr int kBlock = 32;
    static constexpr uint32_t kIdesc = 1u << 23; // UE8M0 scales
};

// Scale atom, and instruction-descriptor bits, of the kb-th K64 MMA of a k-tile.
template <class F> __device__ __forceinline__ constexpr int sf_atom(int kb)
{
    return F::kMx ? kb >> 1 : kb;
}
template <class F> __device__ __forceinline__ constexpr uint32_t sf_id_bits(int kb)
{
    return F::kMx ? ((uint32_t)(kb & 1) * 2u) * ((1u << 29) | (1u << 4)) : 0u;
}

// alpha of the epilogue: sgA * sgW, 1 for MXFP4.
template <class F>
__device__ __forceinline__ float product_scale(const float *a_gs, const float *w_gs)
{
    if constexpr (F::kMx)
        return 1.0f;
    else
        return __fmul_rn(*a_gs, *w_gs);
}

// The scale atoms (F::kAtoms x 512 bytes) at shared address `ssf` -> TMEM columns tcol.. of this
// warp's lane quarter: 4 columns per atom, lane r holding the atom's 16-byte row r.
template <class F> __device__ __forceinline__ void feed_atoms(uint32_t ssf, uint32_t tcol, int lane)
{
    uint32_t r[4 * F::kAtoms];
#pragma unroll
    for (int kb = 0; kb < F::kAtoms; ++kb) {
        const uint4 w = lds128(ssf + kb * 512 + lane * 16);
        r[4 * kb] = w.x;
        r[4 * kb + 1] = w.y;
        r[4 * kb + 2] = w.z;
        r[4 * kb + 3] = w.w;
    }
    if constexpr (F::kMx)
        tmem_st_32x32b_x8(tcol, r);
    else
        tmem_st_32x32b_x16(tcol, r);
}

template <class F>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                           uint32_t accumulate)
{
    if constexpr (F::kMx)
        tc_mma_mxf4(d_tmem, adesc, bdesc, idesc, sfa_tmem, sfb_tmem, accumulate);
    else
        tc_mma_nvf4(d_tmem, adesc, bdesc, idesc, sfa_tmem, sfb_tmem, accumulate);
}

template <class F>
__device__ __forceinline__ void tc_mma_fp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                uint32_t idesc, uint32_t sfa_tmem,
                                                uint32_t sfb_tmem, uint32_t accumulate)
{
    if constexpr (F::kMx)
        tc_mma_mxf4_pair(d_tmem, adesc, bdesc, idesc, sfa_tmem, sfb_tmem, accumulate);
    else
        tc_mma_nvf4_pair(d_tmem, adesc, bdesc, idesc, sfa_tmem, sfb_tmem, accumulate);
}

} // namespace nvfp4
