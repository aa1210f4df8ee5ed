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

// Address of element i, for a scalar i: lanes then add 32-bit offsets.
template <int DT>
__device__ __forceinline__ const void* from(const void* base, int64_t i) {
    return static_cast<const char*>(base) + i * elem_bytes<DT>();
}
template <int DT>
__device__ __forceinline__ void* from(void* base, int64_t i) {
    return static_cast<char*>(base) + i * elem_bytes<DT>();
}

// E consecutive elements as raw words, accessed 4, 8 or 16 bytes at a time at any
// byte address, which global memory allows in the unaligned access mode that
// every HSA process runs in.  NT: non-temporal, for what is read or written once.
// E * elem_bytes is at most 16 where speed matters: then one access of a wave
// covers consecutive bytes.  (8 fp32 elements a lane, two 16-byte accesses that
// each cover every other 16 bytes, ran the 32-bit optimizer step at 4.9 TB/s; 4 a
// lane 5.9.)
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));

template <int DT, int E>
struct Raw {
    static_assert(E == 4 || E == 8, "4 or 8 elements");
    static constexpr int WORDS = E * elem_bytes<DT>() / 4;
    uint32_t w[WORDS];

    template <bool NT = true>
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const char* p = static_cast<const char*>(base) + i * elem_bytes<DT>();
        if constexpr (WORDS == 1) {
            const u32_any* q = reinterpret_cast<const u32_any*>(p);
            if constexpr (NT) w[0] = __builtin_nontemporal_load(q); else w[0] = *q;
        } else if constexpr (WORDS == 2) {
            const u32x2_any* q = reinterpret_cast<const u32x2_any*>(p);
            u32x2 t;
            if constexpr (NT) t = __builtin_nontemporal_load(q); else t = *q;
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
    template <bool NT = true>
    __device__ __forceinline__ void store(void* base, int64_t i) const {
        char* p = static_cast<char*>(base) + i * elem_bytes<DT>();
        if constexpr (WORDS == 1) {
            u32_any* q = reinterpret_cast<u32_any*>(p);
            if constexpr (NT) __builtin_nontemporal_store(w[0], q); else *q = w[0];
        } else if constexpr (WORDS == 2) {
            const u32x2 t = {w[0], w[1]};
            u32x2_any* q = reinterpret_cast<u32x2_any*>(p);
            if constexpr (NT) __builtin_nontemporal_store(t, q); else *q = t;
        } else {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const u32x4 t = {w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
                u32x4_any* q = reinterpret_cast<u32x4_any*>(p) + k;
                if constexpr (NT) __builtin_nontemporal_store(t, q); else *q = t;
            }
        }
    }
    __device__ __forceinline__ uint32_t byte(int k) const { return (w[k >> 2] >> (8 * (k & 3))) & 0xFFu; }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (DT == ZPQ_F32) return __uint_as_float(w[k]);
        else if constexpr (DT == ZPQ_F16)
            return (float)(__builtin_bit_cast(f16x2, w[k >> 1])[k & 1]);
        else if constexpr (DT == ZPQ_BF16)
            return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
        else return (float)(int8_t)byte(k);
    }
    __device__ __forceinline__ void set(const float (&x)[E]) {
        if constexpr (DT == ZPQ_F32) {
#pragma unroll
            for (int k = 0; k < E; ++k) w[k] = __float_as_uint(x[k]);
        } else {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                const f32x2 f = {x[2 * k], x[2 * k + 1]};
                if constexpr (DT == ZPQ_F16)
                    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
                else
                    w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
            }
        }
    }
    // the first `have` elements one by one (the rest as zeros; not written)
    __device__ __forceinline__ void load_some(const void* base, int64_t i, int have) {
        if constexpr (DT == kI8) {
#pragma unroll
            for (int k = 0; k < WORDS; ++k) w[k] = 0;
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (k < have)
                    w[k >> 2] |= (uint32_t)static_cast<const uint8_t*>(base)[i + k] << (8 * (k & 3));
        } else {
            float x[E];
#pragma unroll
            for (int k = 0; k < E; ++k) x[k] = k < have ? load1<DT>(base, i + k) : 0.0f;
            set(x);
        }
    }
    __device__ __forceinline__ void store_some(void* base, int64_t i, int have) const {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (k < have) {
                if constexpr (DT == kI8) static_cast<uint8_t*>(base)[i + k] = (uint8_t)byte(k);
                else if constexpr (DT == ZPQ_F32) static_cast<uint32_t*>(base)[i + k] = w[k];
                else static_cast<uint16_t*>(base)[i + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
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
