// The paged 4-bit cache's cell format and the checks its calls share (not part of the ABI).
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "dl_common.cuh"

namespace dlp {

constexpr int kCell = 16;      // keys of a cell

// Byte offsets inside a cell of 16 keys (18 D bytes): K codes, K scales, V codes, V scales.
__host__ __device__ constexpr int cell_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int k_scale_off(int D) { return 8 * D; }
__host__ __device__ constexpr int v_code_off(int D) { return 9 * D; }
__host__ __device__ constexpr int v_scale_off(int D) { return 17 * D; }

// Place of lane group g's chunk in the V row of key pair j: the 8 (D = 128: 16-byte chunks) or 16
// (D = 64: 8-byte chunks) lanes of one shared-memory phase, which differ in c (pair) and g, then
// touch different banks.
__host__ __device__ constexpr int v_swizzle(int D, int j) { return D == 128 ? 2 * (j & 3) : 2 * (j & 2); }

// Byte offset of the word that holds channel d of key s (K), and of the 16-bit half (V).
__host__ __device__ constexpr int k_word_off(int D, int s, int d)
{
    return s * (D / 2) + ((d >> 3) & 3) * (D / 8) + (d >> 5) * 4;
}
__host__ __device__ constexpr int v_half_off(int D, int s, int d)
{
    return v_code_off(D) + (s >> 1) * D + ((((d >> 2) & 7) ^ v_swizzle(D, s >> 1)) * (D / 8)) + (d >> 5) * 4 + (s & 1) * 2;
}

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128 || page == 256; }

// A launch whose dynamic shared memory passes the default limit: the kernel asks once a device for `most`, the
// largest of its launches, and never for less, since the limit is one for all host threads.  A launch that finds
// it unset all the same (after a reset of the device) asks and launches again.  `asked`: of this kernel, a bit
// a device.
template <typename Launch>
int launch_wide(const void *kern, int most, std::atomic<uint64_t> &asked, const char *who, Launch launch)
{
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    for (bool ask = !(asked.load() & bit);; ask = true) {
        if (ask) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            if (e != cudaSuccess) return dl::cuda_fail(e, who);
            asked |= bit;
        }
        const int rc = launch();
        if (rc == DL_OK || ask) return rc;
        cudaGetLastError();
        dl::clear_error();
    }
}

// Checks of a cache and its tables that every call makes; DL_OK or the recorded failure.
int check_cache(const char *who, const dl_paged_kv *kv, const dl_block_tables *t, int n_q, bool want_mean);

}  // namespace dlp
