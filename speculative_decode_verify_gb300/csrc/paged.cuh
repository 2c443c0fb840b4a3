// Shared by the kernels over the paged 8-bit cache (include/kv_pages.h): sizes, the codes' decoding, and the
// reading of a sequence's length and live rows.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv_pages.h"
#include "va_internal.cuh"

namespace va {
namespace paged {

constexpr int kPage = VA_TILE;                  // positions per page
constexpr int kBlock = VA_B8_BLOCK;             // positions per scale
constexpr int kBlocks = kPage / kBlock;         // scales per page and head
constexpr int kHeadBytes = kPage * kD;          // code bytes of one page and head

// The largest code's value: a block's largest magnitude maps to it.
__host__ __device__ constexpr float top_code(bool int8) { return int8 ? 127.0f : 448.0f; }

// Four codes (one 32-bit word) to floats; exact for both formats.
template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if (kInt8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    } else {
        uint32_t lo, hi;
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
            : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[0] = p.x;
        x[1] = p.y;
        x[2] = q.x;
        x[3] = q.y;
    }
}

// Length and live rows of sequence b; what is out of range counts as an empty sequence and sets a status bit.
struct Seq {
    int len, live, status;
};
__device__ __forceinline__ Seq load_seq(const int32_t* __restrict__ lens, const int32_t* __restrict__ n_live, int b,
                                        int n_rows, int max_pages) {
    Seq s;
    s.len = __ldcg(lens + b);
    s.live = __ldcg(n_live + b);
    s.status = 0;
    if (s.live < 0 || s.live > n_rows || s.live > s.len) s.status |= VA_DEV_BAD_COUNT;
    if ((long long)s.len > (long long)max_pages * kPage) s.status |= VA_DEV_BEYOND_CACHE;
    if (s.status) s.len = s.live = 0;
    return s;
}

// Host-side checks that every call on a pool makes.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline va_status check_pool(const void* k_codes, const void* v_codes, const float* k_scale, const float* v_scale,
                            int n_layers, int n_pages, int n_kv_heads) {
    if (!k_codes || !v_codes || !k_scale || !v_scale) return VA_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_scale) || !aligned16(v_scale)) return VA_INVALID_ARG;
    if (n_layers < 1 || n_pages < 1 || n_kv_heads < 1 || n_kv_heads > VA_PAGED_MAX_KV_HEADS) return VA_INVALID_ARG;
    // one layer's pool is addressed by 32-bit row numbers
    if ((long long)n_pages * n_kv_heads * kPage > 0x7FFFFFFFll) return VA_UNSUPPORTED;
    return VA_OK;
}
inline va_status launched(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? VA_OK : VA_CUDA_ERROR;
}

}  // namespace paged
int device_sm_count();   // abi.cu: the current device's SMs (0 if unknown)
}  // namespace va
