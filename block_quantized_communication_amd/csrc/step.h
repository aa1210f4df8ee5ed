// step.h -- what adamw.hip and embedding.hip share: wide loads and stores of
// the three element types, host-side argument checks, and the lookup of a
// workgroup's tensor in a table of tensors.
#ifndef ZPQ_STEP_H
#define ZPQ_STEP_H

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zpq.h"

namespace zpq_step {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;                 // 4 waves of 64
constexpr int64_t kMaxElems = 1LL << 40;
constexpr int kI8 = 3;                        // INT8 codes, inside the lookup only

template <int DT>
constexpr int elem_bytes() { return DT == ZPQ_F32 ? 4 : DT == kI8 ? 1 : 2; }

// One element as fp32, and one fp32 value rounded to nearest even into DT.
template <int DT>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
    if constexpr (DT == ZPQ_F32) return static_cast<const float*>(base)[i];
    else if constexpr (DT == ZPQ_F16) return (float)static_cast<const _Float16*>(base)[i];
    else if constexpr (DT == ZPQ_BF16)
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[i] << 16);
    else return (float)static_cast<const int8_t*>(base)[i];
}

template <int DT>
__device__ __forceinline__ void store1(void* base, int64_t i, float x) {
    if constexpr (DT == ZPQ_F32) static_cast<float*>(base)[i] = x;
    else if constexpr (DT == ZPQ_F16) static_cast<_Float16*>(base)[i] = (_Float16)x;
    else static_cast<__bf16*>(base)[i] = (__bf16)x;
}

// 8 consecutive elements as raw words: 16-byte accesses (8-byte ones for
// INT8) at any byte address, which global memory allows in the unaligned access
// mode that every HSA process runs in.  NT: non-temporal, for what is read or
// written once.
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));

template <int DT>
struct Raw8 {
    static constexpr int WORDS = 8 * elem_bytes<DT>() / 4;
    uint32_t w[WORDS];

    template <bool NT = true>
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const char* p = static_cast<const char*>(base) + i * elem_bytes<DT>();
        if constexpr (WORDS == 2) {
            const u32x2 t = *reinterpret_cast<const u32x2_any*>(p);
            w[0] = t.x; w[1] = t.y;
        } else {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p) + k;
                u32x4 t;
                if constexpr (NT) t = __builtin_nontemporal_load(q); else t = *q;
                w[4 * k] = t.x; w[4 * k + 1] = t.y; w[4 * k + 2] = t.z; w[4 * k + 3] = t.w;
            }
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (DT == ZPQ_F32) return __uint_as_float(w[k]);
        else if constexpr (DT == ZPQ_F16)
            return (float)(__builtin_bit_cast(f16x2, w[k >> 1])[k & 1]);
        else if constexpr (DT == ZPQ_BF16)
            return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
        else return (float)(int8_t)(w[k >> 2] >> (8 * (k & 3)));
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        if constexpr (DT == ZPQ_F32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 f = {x[2 * k], x[2 * k + 1]};
                if constexpr (DT == ZPQ_F16)
                    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
                else
                    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
            }
        }
    }
    template <bool NT = true>
    __device__ __forceinline__ void store(void* base, int64_t i) const {
        char* p = static_cast<char*>(base) + i * elem_bytes<DT>();
        if constexpr (WORDS == 2) {
            *reinterpret_cast<u32x2_any*>(p) = u32x2{w[0], w[1]};
        } else {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const u32x4 t = {w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
                u32x4_any* q = reinterpret_cast<u32x4_any*>(p) + k;
                if constexpr (NT) __builtin_nontemporal_store(t, q); else *q = t;
            }
        }
    }
};

// The last i in [0, count) with starts[i] <= k, for non-decreasing starts and
// starts[0] = 0: each of the wave's 64 lanes looks at one of 64 evenly spaced
// entries, so 64 tensors take one load and 4096 take two.  The answer is the
// same in every lane.
__device__ __forceinline__ uint32_t find_start(const uint32_t* __restrict__ starts, uint32_t count,
                                               uint32_t k) {
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t lo = 0, n = count;
    while (n > 64) {
        const uint32_t gap = (n + 63) / 64, i = lane * gap;
        const uint64_t below = __ballot(i < n && starts[lo + i] <= k);
        const uint32_t j = ((uint32_t)__popcll(below) - 1) * gap;
        lo += j;
        n = n - j < gap ? n - j : gap;
    }
    const uint64_t below = __ballot(lane < n && starts[lo + lane] <= k);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(lo + (uint32_t)__popcll(below) - 1));
}

// ---------------------------------------------------------------------------
// Host side.
inline bool aligned(const void* p, uint64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}
inline int64_t dtype_bytes(int32_t t) {
    return t == ZPQ_F32 ? 4 : (t == ZPQ_F16 || t == ZPQ_BF16) ? 2 : 0;
}
inline zpq_status after_launch() {
    return hipGetLastError() == hipSuccess ? ZPQ_OK : ZPQ_ERR_LAUNCH;
}

}  // namespace zpq_step

#endif  // ZPQ_STEP_H
