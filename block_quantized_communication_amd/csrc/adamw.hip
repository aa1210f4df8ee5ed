// adamw.hip -- the optimizer step over many tensors, the gradient norm it
// clips by, and the 8-bit states' conversions.
//
// One launch covers all tensors: a table in device memory (written by
// k_fill from kernel arguments, so that it is ordered with the stream, can be
// captured and needs no host memory to outlive the call) lists the tensors
// and where each one's share of workgroups starts; a workgroup finds its
// tensor by one or two 64-lane looks (find_start).
#include <math.h>

#include <atomic>

#include "step.h"

namespace {

using namespace zpq_step;

constexpr int kStateBlock = 256;              // elements of an 8-bit state block: one wave, 4 a lane
constexpr int kPart = kThreads * 4;           // elements that a workgroup takes at once, 4 a lane
constexpr int kParts = 2;                     // parts of a step tile, all loaded before any is computed
constexpr int kTile = kPart * kParts;

// ---------------------------------------------------------------------------
// Tables.
struct ListEntry { const void* ptr; int64_t n; };
struct PlanEntry {
    void* p;
    const void* g;
    void* m;
    void* v;
    uint8_t* me;
    uint8_t* ve;
    void* copy;
    int64_t n;
    int64_t base;                             // first random number
    double decay;
};
// A list's table: partial sums, counts of workgroups that are done (0 between
// calls; each on a cache line of its own), entries, starts.  A plan's: entries,
// starts.
constexpr int kSumParts = 2048, kSumGroup = 32, kSumGroups = kSumParts / kSumGroup;
struct Count { uint32_t n, unused[15]; };
struct ListHead {
    unsigned long long part[kSumParts];       // bits of binary64
    Count group[kSumGroups], all;
};
static_assert(sizeof(ListHead) + 64 <= ZPQ_LIST_BYTES(0) && sizeof(ListEntry) + 4 <= 32 &&
              sizeof(PlanEntry) + 4 <= 128, "ZPQ_*_BYTES");

template <class E, int N>
struct Fill {
    E entry[N];
    uint32_t start[N];
};

// Kernel arguments stay under 4 KB.
constexpr int kFillList = 128, kFillPlan = 40;
static_assert(sizeof(Fill<ListEntry, kFillList>) < 3800 && sizeof(Fill<PlanEntry, kFillPlan>) < 3800,
              "kernel arguments");

template <class E, int N>
__global__ __launch_bounds__(128) void k_fill(Fill<E, N> f, int32_t first, int32_t count, int32_t all,
                                              E* __restrict__ entries, uint32_t* __restrict__ starts,
                                              uint32_t total, ListHead* __restrict__ head) {
    const int i = threadIdx.x;
    if (head != nullptr && i <= kSumGroups) (i < kSumGroups ? head->group[i] : head->all).n = 0;
    if (i < count) {
        entries[first + i] = f.entry[i];
        starts[first + i] = f.start[i];
    }
    if (i == 0 && first + count == all) starts[all] = total;
}

template <class E>
uint32_t* starts_of(E* entries, int32_t count) {
    return reinterpret_cast<uint32_t*>(entries + count);
}
inline PlanEntry* plan_entries(void* table) { return static_cast<PlanEntry*>(table); }
inline ListEntry* list_entries(void* table) {
    return reinterpret_cast<ListEntry*>(static_cast<ListHead*>(table) + 1);
}

// ---------------------------------------------------------------------------
// Sum of squares.  Every square of a binary32 value is exact in binary64, and
// v_fma_f64 issues like v_fma_f32 here, so binary64 sums cost one conversion a
// value and no range checks.  Workgroup b of G takes the chunks
// [K*b/G, K*(b+1)/G): consecutive, so that the tensor is looked up once and
// then followed.  Bound by reading: 906 M fp16 elements 265 us, 6.8 TB/s (a bare read
// stream reaches 7.2).
template <int DT> constexpr int kSumEach = DT == ZPQ_F32 ? 4 : 8;       // elements a lane
constexpr int kSumChunk = 8192;               // elements of a workgroup's share

__device__ __forceinline__ double wg_sum(double x) {
    __shared__ double part[kThreads / 64];
    __syncthreads();                          // an earlier sum's reads
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) s += part[i];
    return s;
}

// Counts the caller; true for the last of n, which leaves the count at 0.
__device__ __forceinline__ bool count_to(uint32_t* count, uint32_t n) {
    if (__hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != n - 1) return false;
    (void)__hip_atomic_exchange(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// KEEP: plain loads, which leave what they read in the last-level cache (256 MB) for
// the optimizer step; non-temporal ones leave it alone.
template <int DT, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_sumsq(const ListEntry* __restrict__ entries,
                                                    const uint32_t* __restrict__ starts,
                                                    int32_t count, uint32_t chunks, ListHead* head,
                                                    int32_t accumulate, double* out) {
    const uint32_t k0 = (uint32_t)((uint64_t)chunks * blockIdx.x / gridDim.x);
    const uint32_t k1 = (uint32_t)((uint64_t)chunks * (blockIdx.x + 1) / gridDim.x);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    uint32_t t = find_start(starts, count, k0);
    for (uint32_t k = k0; k < k1; ++k) {
        while (k >= starts[t + 1]) ++t;       // starts[count] = chunks > k: ends
        const ListEntry e = entries[t];
        const int64_t at = (int64_t)(k - starts[t]) * kSumChunk;
        constexpr int E = kSumEach<DT>, N = kSumChunk / (kThreads * E);
        Raw<DT, E> r[N];
        if (at + kSumChunk <= e.n) {
#pragma unroll
            for (int u = 0; u < N; ++u) r[u].template load<!KEEP>(e.ptr, at + (u * kThreads + threadIdx.x) * E);
        } else {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int64_t i = at + (u * kThreads + threadIdx.x) * E, left = e.n - i;
                if (left >= E) r[u].template load<!KEEP>(e.ptr, i);
                else r[u].load_some(e.ptr, i, left > 0 ? (int)left : 0);
            }
        }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const double x = (double)r[u].get(i);
                s[i & 3] = __builtin_fma(x, x, s[i & 3]);
            }
    }
    const double sum = wg_sum((s[0] + s[1]) + (s[2] + s[3]));
    // The workgroup that finishes last adds the partial sums, always in the same
    // order.  Sums and counts are touched by read-modify-writes at agent scope only: these
    // are carried out where all XCDs' accesses meet, and one whose old value has come
    // back is done.  So a workgroup counts itself (waiting for its exchange) after
    // its sum can be read by all, and the one that counts to the end reads every sum.
    // Counting is in groups of 32 (where there are more), then the groups: with one count
    // for the 1024 workgroups of 256 compute units 50.3 M elements take 27.9 us, so 20.3, and
    // about 2 more with a second launch to join.  (A release and an acquire write back and
    // invalidate the L2 for each workgroup: 107 us.)
    __shared__ bool last;
    if (threadIdx.x == 0) {
        unsigned long long old = __hip_atomic_exchange(&head->part[blockIdx.x], __double_as_longlong(sum),
                                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(old) : : "memory");
        const uint32_t g = blockIdx.x / kSumGroup, groups = (gridDim.x + kSumGroup - 1) / kSumGroup;
        const uint32_t members = g + 1 < groups ? kSumGroup : gridDim.x - g * kSumGroup;
        last = groups == 1 ? count_to(&head->all.n, gridDim.x)
                           : count_to(&head->group[g].n, members) && count_to(&head->all.n, groups);
    }
    __syncthreads();
    if (!last) return;
    double all = 0.0;
    for (uint32_t b = 0; b < gridDim.x; b += 8 * kThreads) {
        unsigned long long x[8] = {};         // fetched together
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t i = b + u * kThreads + threadIdx.x;
            if (i < gridDim.x)
                x[u] = __hip_atomic_exchange(&head->part[i], 0ull, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) all += __longlong_as_double((long long)x[u]);
    }
    all = wg_sum(all);
    if (threadIdx.x == 0) out[0] = accumulate ? out[0] + all : all;
}

__global__ void k_zero(double* out) { out[0] = 0.0; }

// ---------------------------------------------------------------------------
// 8-bit states.  A state value is a binary32 pattern whose exponent field has
// been moved so that the block's top binade e lands on T (15 for m, 31 for
// v): then the pattern's bits from 20 up are the code, binary32's own
// subnormals are the code's subnormals, and rounding is an integer addition
// below bit 20.  ldexp moves the field, for any e, with one rounding where
// the result is subnormal.

// Maximum over the wave of unsigned values, as a scalar: within rows of 16 lanes
// by lane permutes, then lane 15 to the next row and lane 31 to the upper half,
// which leaves it in lane 63.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_dpp<0xB1>(v);                     // quad_perm [1,0,3,2]
    v = max_dpp<0x4E>(v);                     // quad_perm [2,3,0,1]
    v = max_dpp<0x141>(v);                    // row_half_mirror
    v = max_dpp<0x140>(v);                    // row_mirror
    v = max_dpp<0x142>(v);                    // row_bcast:15
    v = max_dpp<0x143>(v);                    // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Exponent byte of a block from the bits of its largest magnitude: up to
// 1.875 of a binade stays in it (a carry out of 3 fraction bits would not fit).
__device__ __forceinline__ uint32_t block_exp(uint32_t amax) {
    const uint32_t e = (amax + 0xFFFFFu) >> 23;
    return e < 1 ? 1 : e > 255 ? 255 : e;
}

// Value of byte i of w.
template <int MOMENT>
__device__ __forceinline__ float decode8(uint32_t w, int i, uint32_t e) {
    if constexpr (MOMENT == 1)                // the sign down to bit 31 and, masked off again, 27..30
        return __builtin_amdgcn_ldexpf(
            __uint_as_float((uint32_t)((int32_t)(w << (24 - 8 * i)) >> 4) & 0x87F00000u), (int)e - 15);
    else
        return __builtin_amdgcn_ldexpf(
            __uint_as_float((i < 3 ? w << (20 - 8 * i) : w >> 4) & 0x0FF00000u), (int)e - 31);
}

// Byte 3 of each of 4 words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(b, a, 0x0C0C0703u) | __builtin_amdgcn_perm(d, c, 0x07030C0Cu);
}

// Codes of 4 values of a block with exponent byte e.  add[i] is what goes in below
// bit 20: a random number for states; NEAREST: half a step (less one, plus the
// parity), for rounding to nearest even.
template <int MOMENT, bool NEAREST>
__device__ __forceinline__ uint32_t encode8(const float (&x)[4], uint32_t e, const uint32_t (&add)[4]) {
    if (e == 255) return MOMENT == 1 ? 0x7F7F7F7Fu : 0xFFFFFFFFu;
    uint32_t t[4];                            // the code in the top byte
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mag = __float_as_uint(
            __builtin_amdgcn_ldexpf(__builtin_fabsf(x[i]), (MOMENT == 1 ? 15 : 31) - (int)e));
        t[i] = (mag + (NEAREST ? 0x7FFFFu + ((mag >> 20) & 1u) : add[i])) << 4;
    }
    if constexpr (MOMENT == 2 && !NEAREST) {  // a value above 0 does not become 0
        if (__any(min(min(t[0], t[1]), min(t[2], t[3])) < 1u << 24)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = max(t[i], x[i] > 0.0f ? 1u << 24 : 0u);
        }
    }
    uint32_t c = top_bytes(t[0], t[1], t[2], t[3]);
    if constexpr (MOMENT == 1)
        c |= top_bytes(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                       __float_as_uint(x[3])) & 0x80808080u;
    return c;
}

// The random bits of element lo + 2^32 * hi for a key made of seed and step: a
// multiplicative counter and two rounds of xor-shift and multiply.  Low half
// for m, high half for v.
constexpr uint32_t kMulLo = 0x9E3779B1u, kMulHi = 0x85A308D3u;
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0xB7E15163u;
    x = (x ^ (x >> 15)) * 0x243F6A89u;
    return x ^ (x >> 16);
}
__host__ __device__ inline uint32_t random_key(uint64_t seed, uint64_t step) {
    uint64_t z = seed + step * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 31)) * 0xB7E151628AED2A6Bull;
    z = (z ^ (z >> 29)) * 0x243F6A8885A308D3ull;
    return (uint32_t)(z >> 32);
}

// ---------------------------------------------------------------------------
// The step.  The root and the quotient are the hardware's (1 ulp each; the IEEE
// sequences took 25 of about 110 instructions an element in the 8-bit step,
// which they bound).  With eps >= 1e-30 the quotient's denominator is a normal
// number.  The hardware's root of a v below 2^-126 is 0, but the true one is up to
// 2^-63, which counts beside a small eps: such a v is moved up by 2^64 and its root
// back by 2^-32, both exact (at no cost: 50.3 M elements 244 us without and with, 201 M
// with 8-bit states 529 and 530).
__device__ __forceinline__ float root(float v) {
    const bool low = v < 0x1p-126f;
    return __builtin_amdgcn_sqrtf(low ? v * 0x1p64f : v) * (low ? 0x1p-32f : 1.0f);
}
struct StepArgs {
    double lr, grad_scale, max_norm;
    float b1, ob1, b2, ob2, eps, rbc2, rate;  // ob: 1 - b; rbc2: 1/sqrt(1 - b2^t); rate: lr/(1 - b1^t)
    uint32_t key;
};

// The constants from the hyperparameters, in the same operations on the host and on
// the device (b^t by squaring, off by t * 2^-53 of itself, which 1 - b^t has to
// its rounding to 24 bits as long as 1 - b > 2^-29).
__host__ __device__ inline double power(double b, int64_t t) {
    double x = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) x *= b;
    return x;
}
__host__ __device__ inline bool finite_at_least(double x, double least) {
    return x >= least && x <= 1.7976931348623157e308;
}
// max_norm counts only where there is a norm.
__host__ __device__ inline bool hyper_ok(const zpq_adamw_hyper& h, bool norm) {
    return finite_at_least(h.lr, 0.0) && h.beta1 >= 0.0 && h.beta1 < 1.0 && h.beta2 >= 0.0 && h.beta2 < 1.0 &&
           finite_at_least(h.eps, 1e-30) && h.step >= 1 && h.grad_scale > 0.0 &&
           h.grad_scale <= 3.4028234663852886e38 && (!norm || h.max_norm > 0.0);
}
__host__ __device__ inline StepArgs step_args(const zpq_adamw_hyper& h) {
    StepArgs a;
    a.lr = h.lr;
    a.grad_scale = h.grad_scale;
    a.max_norm = h.max_norm;
    a.b1 = (float)h.beta1;
    a.ob1 = (float)(1.0 - h.beta1);
    a.b2 = (float)h.beta2;
    a.ob2 = (float)(1.0 - h.beta2);
    a.eps = (float)h.eps;
    a.rbc2 = (float)(1.0 / sqrt(1.0 - power(h.beta2, h.step)));
    a.rate = (float)(h.lr / (1.0 - power(h.beta1, h.step)));
    a.key = random_key(h.seed, (uint64_t)h.step);
    return a;
}

// Hyperparameters in device memory: a launch of its own turns them into the constants,
// in the plan's table behind the starts (lr -1 where they are out of range): norm and step
// 2 us more (50.3 M elements 249.6 -> 251.1, 12.5 K 10.9 -> 13.1).
static_assert(sizeof(PlanEntry) + 4 + 4 + 8 + sizeof(StepArgs) <= ZPQ_PLAN_BYTES(1) &&
              sizeof(PlanEntry) + 4 <= 128, "ZPQ_PLAN_BYTES");
inline StepArgs* args_of(void* table, int32_t count) {
    const uintptr_t end = reinterpret_cast<uintptr_t>(starts_of(plan_entries(table), count) + count + 1);
    return reinterpret_cast<StepArgs*>((end + 7) / 8 * 8);
}
__global__ void k_step_args(const zpq_adamw_hyper* __restrict__ h, int32_t norm, StepArgs* __restrict__ to) {
    StepArgs a = {};
    a.lr = -1.0;
    if (hyper_ok(*h, norm != 0)) a = step_args(*h);
    *to = a;
}

// 4 elements a lane of one part: loaded together, stepped, stored.  A wave holds
// 256 consecutive elements, which is a state block: the exponents of 8-bit
// states are scalars.
template <int PT, int GT, int CT, int BITS>
struct Part {
    static constexpr int ST = BITS == 32 ? ZPQ_F32 : kI8;
    Raw<PT, 4> p;
    Raw<GT, 4> g;
    Raw<ST, 4> m, v;
    uint32_t em, ev;
    int64_t at;                               // of the part: a scalar
    uint32_t lane;                            // this lane's first element in it
    int have;                                 // elements of this lane, 0 to 4

    __device__ __forceinline__ void load(const PlanEntry& e, int64_t at_) {
        at = at_;
        lane = threadIdx.x * 4;
        const int64_t left = e.n - at - kPart;                // past the part, or missing
        have = left >= 0 ? 4 : (int)(left + kPart - lane);
        have = have < 0 ? 0 : have > 4 ? 4 : have;
        em = ev = 1;
        if constexpr (BITS == 8) {
            const int64_t b = at / kStateBlock + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
            if (b * kStateBlock < e.n) { em = e.me[b]; ev = e.ve[b]; }
        }
        if (have == 4) {
            p.load(from<PT>(e.p, at), lane);
            g.load(from<GT>(e.g, at), lane);
            m.load(from<ST>(e.m, at), lane);
            v.load(from<ST>(e.v, at), lane);
        } else {
            p.load_some(e.p, at + lane, have);
            g.load_some(e.g, at + lane, have);
            m.load_some(e.m, at + lane, have);
            v.load_some(e.v, at + lane, have);
        }
    }

    __device__ __forceinline__ void step(const PlanEntry& e, const StepArgs& a, float c, float keep) {
        float pp[4], mm[4], vv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float m0, v0;
            if constexpr (BITS == 32) {
                m0 = m.get(i);
                v0 = v.get(i);
            } else {
                m0 = decode8<1>(m.w[0], i, em);
                v0 = decode8<2>(v.w[0], i, ev);
            }
            const float x = g.get(i) * c;
            mm[i] = m0 * a.b1 + x * a.ob1;
            vv[i] = v0 * a.b2 + (x * a.ob2) * x;
            const float den = root(vv[i]) * a.rbc2 + a.eps;
            pp[i] = p.get(i) * keep - mm[i] * __builtin_amdgcn_rcpf(den) * a.rate;
        }
        p.set(pp);
        if constexpr (BITS == 32) {
            m.set(mm);
            v.set(vv);
        } else {
            // lanes past the end hold zeros: m and v of zeros stay zeros
            uint32_t am = 0, av = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                am = max(am, __float_as_uint(mm[i]) & 0x7FFFFFFFu);
                av = max(av, __float_as_uint(vv[i]) & 0x7FFFFFFFu);
            }
            em = block_exp(wave_max(am));
            ev = block_exp(wave_max(av));
            // the wave's first element counts as a multiple of 256, so that none of its
            // 256 carries into the upper 32 bits
            const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
            const uint64_t n0 = (uint64_t)(e.base + at) + wave * kStateBlock;
            const uint32_t x0 = (uint32_t)n0 * kMulLo + (uint32_t)(n0 >> 32) * kMulHi + a.key +
                                (threadIdx.x & 63u) * 4 * kMulLo;
            uint32_t rm[4], rv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = mix(x0 + (uint32_t)i * kMulLo);
                rm[i] = (r << 4 & 0xFFFF0u) | 8u;
                rv[i] = (r >> 12 & 0xFFFF0u) | 8u;
            }
            m.w[0] = encode8<1, false>(mm, em, rm);
            v.w[0] = encode8<2, false>(vv, ev, rv);
        }
        // out
        Raw<CT < 0 ? ZPQ_F16 : CT, 4> copy;
        if constexpr (CT >= 0) copy.set(pp);
        if (have == 4) {
            p.store(from<PT>(e.p, at), lane);
            if constexpr (CT >= 0) copy.store(from<CT>(e.copy, at), lane);
            m.store(from<ST>(e.m, at), lane);
            v.store(from<ST>(e.v, at), lane);
        } else {
            p.store_some(e.p, at + lane, have);
            if constexpr (CT >= 0) copy.store_some(e.copy, at + lane, have);
            m.store_some(e.m, at + lane, have);
            v.store_some(e.v, at + lane, have);
        }
        if constexpr (BITS == 8) {
            if ((threadIdx.x & 63) == 0 && have > 0) {
                const int64_t b = (at + lane) / kStateBlock;
                e.me[b] = (uint8_t)em;
                e.ve[b] = (uint8_t)ev;
            }
        }
    }
};

// Workgroup k of the grid (and k + gridDim.x, ...) takes chunk k: one tile of one
// tensor.  Bound by HBM, every tensor read and written once: 50.3 M elements with fp32
// states 228 us (1.41 GB, 6.2 TB/s), 201 M with 8-bit states 493 us (3.22 GB, 6.5 TB/s).
// Two parts a tile: with one 266 and 545 us, with four 241 and 536, when two took 244 and
// 527.  16-bit weights without a copy, 50.3 M elements with 16-bit gradients: 181 us with
// fp32 states (1.11 GB, 6.1 TB/s), 108 with 8-bit ones (505 MB, 4.7 TB/s: 8 bytes a lane and
// access for weights and gradients, and the arithmetic).
template <int PT, int GT, int CT, int BITS>
__global__ __launch_bounds__(kThreads) void k_adamw(const PlanEntry* __restrict__ entries,
                                                    const uint32_t* __restrict__ starts,
                                                    int32_t count, uint32_t chunks, StepArgs a,
                                                    const StepArgs* __restrict__ device_args,
                                                    const double* __restrict__ sumsq) {
    if (device_args != nullptr) {
        a = *device_args;
        if (a.lr < 0.0) return;
    }
    float c = (float)a.grad_scale;
    if (sumsq != nullptr) {
        const double norm = __builtin_sqrt(*sumsq) * a.grad_scale;
        if (!(norm < __builtin_huge_val())) return;          // also NaN
        const double cut = a.max_norm / (norm + 1e-6);
        c = (float)(a.grad_scale * (cut < 1.0 ? cut : 1.0));
    }
    for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
        const uint32_t t = find_start(starts, count, k);
        const PlanEntry e = entries[t];
        const float keep = (float)(1.0 - a.lr * e.decay);
        const int64_t at = (int64_t)(k - starts[t]) * kTile;
        Part<PT, GT, CT, BITS> part[kParts];
#pragma unroll
        for (int u = 0; u < kParts; ++u) part[u].load(e, at + u * kPart);
#pragma unroll
        for (int u = 0; u < kParts; ++u) part[u].step(e, a, c, keep);
    }
}

// ---------------------------------------------------------------------------
// 8-bit states to floats and back.  Floats are written 16 bytes a lane: 201 M codes to
// bf16 102 us (604 MB, 5.9 TB/s; with one or two loads at once 127 and 107), with 8
// bytes a lane 140.
constexpr int kConvParts = 4;
template <int DT> constexpr int kConvEach = DT == ZPQ_F32 ? 4 : 8;
template <int DT, int MOMENT>
__global__ __launch_bounds__(kThreads) void k_unpack8(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ exps, int64_t n,
                                                      void* __restrict__ y) {
    constexpr int E = kConvEach<DT>;
    constexpr int64_t kAll = (int64_t)kThreads * E * kConvParts;
    for (int64_t at = blockIdx.x * kAll; at < n; at += gridDim.x * kAll) {
        Raw<kI8, E> r[kConvParts];
        uint32_t e[kConvParts];
        int have[kConvParts];
#pragma unroll
        for (int u = 0; u < kConvParts; ++u) {
            const uint32_t lane = (u * kThreads + threadIdx.x) * E;
            const int64_t left = n - at - lane;
            have[u] = left >= E ? E : left > 0 ? (int)left : 0;
            e[u] = have[u] > 0 ? (exps + at / kStateBlock)[lane / kStateBlock] : 1;
            if (have[u] == E) r[u].load(codes + at, lane);
            else r[u].load_some(codes + at, lane, have[u]);
        }
#pragma unroll
        for (int u = 0; u < kConvParts; ++u) {
            const uint32_t lane = (u * kThreads + threadIdx.x) * E;
            float x[E];
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = decode8<MOMENT>(r[u].w[i >> 2], i & 3, e[u]);
            Raw<DT, E> o;
            o.set(x);
            if (have[u] == E) o.store(from<DT>(y, at), lane);
            else o.store_some(from<DT>(y, at), lane, have[u]);
        }
    }
}

// 201 M values from fp32 177 us (1.01 GB, 5.7 TB/s), from bf16 150 (605 MB, 4.0 TB/s): one access
// of 16 or 8 bytes in flight a lane.
template <int DT, int MOMENT>
__global__ __launch_bounds__(kThreads) void k_pack8(const void* __restrict__ x, int64_t n,
                                                    uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ exps) {
    for (int64_t at = (int64_t)blockIdx.x * kPart; at < n; at += (int64_t)gridDim.x * kPart) {
        const int64_t i0 = at + threadIdx.x * 4;
        const int have = (int)(n - i0 < 0 ? 0 : n - i0 < 4 ? n - i0 : 4);
        Raw<DT, 4> r;
        if (have == 4) r.load(x, i0);
        else r.load_some(x, i0, have);
        float v[4];
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = r.get(i);
            a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        const uint32_t e = block_exp(wave_max(a));
        Raw<kI8, 4> c;
        c.w[0] = encode8<MOMENT, true>(v, e, {});
        if (have == 4) c.store(codes, i0);
        else c.store_some(codes, i0, have);
        if ((threadIdx.x & 63) == 0 && have > 0) exps[i0 / kStateBlock] = (uint8_t)e;
    }
}

// ---------------------------------------------------------------------------
// Host side.
// Compute units of the current device, cached per device (threads may race to
// fill an entry, with the same value).
inline unsigned cu_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
            n = 256;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return (unsigned)n;
}

inline unsigned grid_of(int64_t work) { return (unsigned)(work < (1 << 22) ? work : 1 << 22); }

// Gradients up to this size are left in the last-level cache for the step that
// follows: norm and step of 50.3 M elements 263 -> 250 us, 68.8 M fp32 ones 370 -> 336, 201 M
// 16-bit ones (403 MB, with both states read out) 796 -> 771.  Where no step follows the norm
// pays for it all the same: 18.9 -> 20.3 us, 46.0 -> 51.7, 66.9 -> 74.9.  Of 1.8 GB nothing would
// be left, and the norm takes 280 us, with plain loads 329.
constexpr int64_t kKeepBytes = 512LL << 20;

template <int DT>
void launch_sumsq(const zpq_list* list, int64_t parts, double* out, int32_t accumulate, hipStream_t st) {
    ListEntry* e = list_entries(list->table);
    const uint32_t* starts = starts_of(e, list->count);
    ListHead* head = static_cast<ListHead*>(list->table);
    const dim3 grid((unsigned)parts);
    if (list->elems * elem_bytes<DT>() <= kKeepBytes)
        hipLaunchKernelGGL((k_sumsq<DT, true>), grid, dim3(kThreads), 0, st, e, starts, list->count,
                           (uint32_t)list->chunks, head, accumulate, out);
    else
        hipLaunchKernelGGL((k_sumsq<DT, false>), grid, dim3(kThreads), 0, st, e, starts, list->count,
                           (uint32_t)list->chunks, head, accumulate, out);
}

bool list_ok(const zpq_list* l) {
    return l && l->count >= 0 && l->chunks >= 0 && l->chunks <= 0x7FFFFFFF && l->elems >= 0 &&
           dtype_bytes(l->dtype) != 0 && (l->chunks == 0 || (l->table && l->count > 0));
}

template <int PT, int GT, int CT, int BITS>
void launch_adamw(const zpq_adamw_plan* q, const StepArgs& a, const StepArgs* at, const double* sumsq,
                  hipStream_t st) {
    hipLaunchKernelGGL((k_adamw<PT, GT, CT, BITS>), dim3(grid_of(q->chunks)), dim3(kThreads), 0, st,
                       plan_entries(q->table), starts_of(plan_entries(q->table), q->count),
                       q->count, (uint32_t)q->chunks, a, at, sumsq);
}
template <int PT, int GT, int BITS>
void launch_adamw_c(const zpq_adamw_plan* q, const StepArgs& a, const StepArgs* at, const double* sumsq,
                  hipStream_t st) {
    if constexpr (PT == ZPQ_F32) {
        if (q->copy_dtype == ZPQ_F16) return launch_adamw<PT, GT, ZPQ_F16, BITS>(q, a, at, sumsq, st);
        if (q->copy_dtype == ZPQ_BF16) return launch_adamw<PT, GT, ZPQ_BF16, BITS>(q, a, at, sumsq, st);
    }
    launch_adamw<PT, GT, -1, BITS>(q, a, at, sumsq, st);
}
template <int PT, int BITS>
void launch_adamw_g(const zpq_adamw_plan* q, const StepArgs& a, const StepArgs* at, const double* sumsq,
                  hipStream_t st) {
    if (q->g_dtype == ZPQ_F32) launch_adamw_c<PT, ZPQ_F32, BITS>(q, a, at, sumsq, st);
    else if (q->g_dtype == ZPQ_F16) launch_adamw_c<PT, ZPQ_F16, BITS>(q, a, at, sumsq, st);
    else launch_adamw_c<PT, ZPQ_BF16, BITS>(q, a, at, sumsq, st);
}
template <int BITS>
void launch_adamw_p(const zpq_adamw_plan* q, const StepArgs& a, const StepArgs* at, const double* sumsq,
                  hipStream_t st) {
    if (q->p_dtype == ZPQ_F32) launch_adamw_g<ZPQ_F32, BITS>(q, a, at, sumsq, st);
    else if (q->p_dtype == ZPQ_F16) launch_adamw_g<ZPQ_F16, BITS>(q, a, at, sumsq, st);
    else launch_adamw_g<ZPQ_BF16, BITS>(q, a, at, sumsq, st);
}

zpq_status adamw(const zpq_adamw_plan* plan, const StepArgs& a, const StepArgs* at, const double* sumsq,
                 hipStream_t st) {
    if (plan->state_bits == 32) launch_adamw_p<32>(plan, a, at, sumsq, st);
    else launch_adamw_p<8>(plan, a, at, sumsq, st);
    return after_launch();
}

bool plan_ok(const zpq_adamw_plan* q) {
    return dtype_bytes(q->p_dtype) != 0 && dtype_bytes(q->g_dtype) != 0 &&
           (q->state_bits == 32 || q->state_bits == 8) && q->count >= 0 && q->chunks >= 0 &&
           q->chunks <= 0x7FFFFFFF && (q->chunks == 0 || (q->table && q->count > 0));
}

template <int DT>
void launch_unpack(const uint8_t* codes, const uint8_t* exps, int64_t n, int32_t moment,
                   void* y, hipStream_t st) {
    constexpr int64_t kAll = (int64_t)kThreads * kConvEach<DT> * kConvParts;
    const dim3 grid(grid_of((n + kAll - 1) / kAll));
    if (moment == 1)
        hipLaunchKernelGGL((k_unpack8<DT, 1>), grid, dim3(kThreads), 0, st, codes, exps, n, y);
    else
        hipLaunchKernelGGL((k_unpack8<DT, 2>), grid, dim3(kThreads), 0, st, codes, exps, n, y);
}
template <int DT>
void launch_pack(const void* x, int64_t n, int32_t moment, uint8_t* codes, uint8_t* exps,
                 hipStream_t st) {
    const dim3 grid(grid_of((n + kPart - 1) / kPart));
    if (moment == 1)
        hipLaunchKernelGGL((k_pack8<DT, 1>), grid, dim3(kThreads), 0, st, x, n, codes, exps);
    else
        hipLaunchKernelGGL((k_pack8<DT, 2>), grid, dim3(kThreads), 0, st, x, n, codes, exps);
}

zpq_status state8_check(const void* codes, const void* exps, const void* y, int64_t n, int32_t moment,
                        int32_t dtype) {
    if (moment != 1 && moment != 2) return ZPQ_ERR_ARG;
    if (n < 0 || n > kMaxElems) return ZPQ_ERR_SIZE;
    const int64_t eb = dtype_bytes(dtype);
    if (eb == 0) return ZPQ_ERR_DTYPE;
    if (n == 0) return ZPQ_OK;
    if (!codes || !exps || !y) return ZPQ_ERR_NULL;
    if (!aligned(y, eb)) return ZPQ_ERR_ALIGN;
    const uint64_t blocks = (uint64_t)(n + kStateBlock - 1) / kStateBlock;
    if (overlaps(codes, n, y, n * eb) || overlaps(exps, blocks, y, n * eb) ||
        overlaps(codes, n, exps, blocks))
        return ZPQ_ERR_ALIAS;
    return ZPQ_OK;
}

}  // namespace

extern "C" {

zpq_status zpq_list_make(const void* const* ptrs, const int64_t* sizes, int32_t count,
                         int32_t dtype, void* table, int64_t table_bytes, zpq_list* list,
                         zpq_stream stream) {
    if (count < 0) return ZPQ_ERR_ARG;
    const int64_t eb = dtype_bytes(dtype);
    if (eb == 0) return ZPQ_ERR_DTYPE;
    if (!list || (count > 0 && (!ptrs || !sizes || !table))) return ZPQ_ERR_NULL;
    if (table_bytes < ZPQ_LIST_BYTES(count)) return ZPQ_ERR_SIZE;
    if (count > 0 && !aligned(table, 16)) return ZPQ_ERR_ALIGN;
    int64_t elems = 0, chunks = 0;
    for (int32_t i = 0; i < count; ++i)
        if (sizes[i] < 0 || sizes[i] > kMaxElems || (elems += sizes[i]) > kMaxElems) return ZPQ_ERR_SIZE;
    for (int32_t i = 0; i < count; ++i) {
        if (sizes[i] > 0 && !ptrs[i]) return ZPQ_ERR_NULL;
        if (sizes[i] > 0 && !aligned(ptrs[i], eb)) return ZPQ_ERR_ALIGN;
        if (overlaps(ptrs[i], sizes[i] * eb, table, table_bytes)) return ZPQ_ERR_ALIAS;
        chunks += (sizes[i] + kSumChunk - 1) / kSumChunk;
    }
    if (chunks > 0x7FFFFFFF) return ZPQ_ERR_SIZE;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ListEntry* entries = list_entries(table);
    int64_t start = 0;
    for (int32_t first = 0; first < count; first += kFillList) {
        Fill<ListEntry, kFillList> f = {};
        const int32_t some = count - first < kFillList ? count - first : kFillList;
        for (int32_t i = 0; i < some; ++i) {
            f.entry[i] = ListEntry{ptrs[first + i], sizes[first + i]};
            f.start[i] = (uint32_t)start;
            start += (sizes[first + i] + kSumChunk - 1) / kSumChunk;
        }
        hipLaunchKernelGGL((k_fill<ListEntry, kFillList>), dim3(1), dim3(128), 0, st, f, first, some, count,
                           entries, starts_of(entries, count), (uint32_t)chunks, static_cast<ListHead*>(table));
    }
    *list = zpq_list{table, elems, chunks, count, dtype};
    return count > 0 ? after_launch() : ZPQ_OK;
}

zpq_status zpq_grad_sumsq(const zpq_list* list, double* out, int32_t accumulate, zpq_stream stream) {
    if (!list_ok(list)) return list ? ZPQ_ERR_ARG : ZPQ_ERR_NULL;
    if (!out) return ZPQ_ERR_NULL;
    if (!aligned(out, 8)) return ZPQ_ERR_ALIGN;
    if (overlaps(out, 8, list->table, ZPQ_LIST_BYTES(list->count))) return ZPQ_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (list->chunks == 0) {
        if (!accumulate) hipLaunchKernelGGL(k_zero, dim3(1), dim3(1), 0, st, out);
        return after_launch();
    }
    int64_t parts = (int64_t)cu_count() * 4;
    if (parts > kSumParts) parts = kSumParts;
    if (parts > list->chunks) parts = list->chunks;
    if (list->dtype == ZPQ_F32) launch_sumsq<ZPQ_F32>(list, parts, out, accumulate, st);
    else if (list->dtype == ZPQ_F16) launch_sumsq<ZPQ_F16>(list, parts, out, accumulate, st);
    else launch_sumsq<ZPQ_BF16>(list, parts, out, accumulate, st);
    return after_launch();
}

zpq_status zpq_adamw_plan_make(const zpq_adamw_tensor* tensors, int32_t count, int32_t p_dtype,
                               int32_t g_dtype, int32_t copy_dtype, int32_t state_bits,
                               void* table, int64_t table_bytes, zpq_adamw_plan* plan,
                               zpq_stream stream) {
    if (count < 0) return ZPQ_ERR_ARG;
    const int64_t pb = dtype_bytes(p_dtype), gb = dtype_bytes(g_dtype);
    if (pb == 0 || gb == 0) return ZPQ_ERR_DTYPE;
    if (copy_dtype != -1 && copy_dtype != ZPQ_F16 && copy_dtype != ZPQ_BF16) return ZPQ_ERR_DTYPE;
    if (copy_dtype != -1 && p_dtype != ZPQ_F32) return ZPQ_ERR_MODE;
    if (state_bits != 32 && state_bits != 8) return ZPQ_ERR_ARG;
    if (!plan || (count > 0 && (!tensors || !table))) return ZPQ_ERR_NULL;
    if (table_bytes < ZPQ_PLAN_BYTES(count)) return ZPQ_ERR_SIZE;
    if (count > 0 && !aligned(table, 16)) return ZPQ_ERR_ALIGN;
    const int64_t sb = state_bits / 8;
    int64_t elems = 0, chunks = 0;
    for (int32_t i = 0; i < count; ++i)
        if (tensors[i].n < 0 || tensors[i].n > kMaxElems || (elems += tensors[i].n) > kMaxElems)
            return ZPQ_ERR_SIZE;
    for (int32_t i = 0; i < count; ++i) {
        const zpq_adamw_tensor& t = tensors[i];
        if (!finite_at_least(t.weight_decay, 0.0)) return ZPQ_ERR_ARG;
        if (t.n == 0) continue;
        if ((copy_dtype == -1) != (t.copy == nullptr)) return ZPQ_ERR_MODE;
        if (!t.p || !t.g || !t.m || !t.v || (state_bits == 8 && (!t.m_exp || !t.v_exp))) return ZPQ_ERR_NULL;
        if (!aligned(t.p, pb) || !aligned(t.g, gb) || !aligned(t.m, sb) || !aligned(t.v, sb) ||
            !aligned(t.copy, 2))
            return ZPQ_ERR_ALIGN;
        const uint64_t blocks = state_bits == 8 ? (uint64_t)(t.n + kStateBlock - 1) / kStateBlock : 0;
        const void* at[8] = {t.p, t.g, t.m, t.v, t.copy, t.m_exp, t.v_exp, table};
        const uint64_t size[8] = {(uint64_t)(t.n * pb), (uint64_t)(t.n * gb), (uint64_t)(t.n * sb),
                                  (uint64_t)(t.n * sb), (uint64_t)t.n * 2, blocks, blocks,
                                  (uint64_t)table_bytes};
        for (int x = 0; x < 8; ++x)
            for (int y = x + 1; y < 8; ++y)
                if (overlaps(at[x], size[x], at[y], size[y])) return ZPQ_ERR_ALIAS;
        chunks += (t.n + kTile - 1) / kTile;
    }
    if (chunks > 0x7FFFFFFF) return ZPQ_ERR_SIZE;
    hipStream_t st = static_cast<hipStream_t>(stream);
    PlanEntry* entries = plan_entries(table);
    int64_t start = 0, base = 0;
    for (int32_t first = 0; first < count; first += kFillPlan) {
        Fill<PlanEntry, kFillPlan> f = {};
        const int32_t some = count - first < kFillPlan ? count - first : kFillPlan;
        for (int32_t i = 0; i < some; ++i) {
            const zpq_adamw_tensor& t = tensors[first + i];
            f.entry[i] = PlanEntry{t.p, t.g, t.m, t.v, t.m_exp, t.v_exp, t.copy, t.n, base,
                                   t.weight_decay};
            f.start[i] = (uint32_t)start;
            start += (t.n + kTile - 1) / kTile;
            base += (t.n + kStateBlock - 1) / kStateBlock * kStateBlock;
        }
        hipLaunchKernelGGL((k_fill<PlanEntry, kFillPlan>), dim3(1), dim3(128), 0, st, f, first, some, count,
                           entries, starts_of(entries, count), (uint32_t)chunks, (ListHead*)nullptr);
    }
    *plan = zpq_adamw_plan{table, elems, chunks, count, p_dtype, g_dtype, copy_dtype, state_bits};
    return count > 0 ? after_launch() : ZPQ_OK;
}

zpq_status zpq_adamw_step(const zpq_adamw_plan* plan, const zpq_adamw_hyper* h, const double* sumsq,
                          zpq_stream stream) {
    if (!plan || !h) return ZPQ_ERR_NULL;
    if (!plan_ok(plan) || !hyper_ok(*h, true)) return ZPQ_ERR_ARG;
    if (!sumsq && h->max_norm <= 1.7976931348623157e308) return ZPQ_ERR_ARG;
    if (!aligned(sumsq, 8)) return ZPQ_ERR_ALIGN;
    if (plan->chunks == 0) return ZPQ_OK;
    return adamw(plan, step_args(*h), nullptr, sumsq, static_cast<hipStream_t>(stream));
}

zpq_status zpq_adamw_step_at(const zpq_adamw_plan* plan, const zpq_adamw_hyper* h, const double* sumsq,
                             zpq_stream stream) {
    if (!plan || !h) return ZPQ_ERR_NULL;
    if (!plan_ok(plan)) return ZPQ_ERR_ARG;
    if (!aligned(h, 8) || !aligned(sumsq, 8)) return ZPQ_ERR_ALIGN;
    if (overlaps(h, sizeof *h, plan->table, ZPQ_PLAN_BYTES(plan->count))) return ZPQ_ERR_ALIAS;
    if (plan->chunks == 0) return ZPQ_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    StepArgs* at = args_of(plan->table, plan->count);
    hipLaunchKernelGGL(k_step_args, dim3(1), dim3(1), 0, st, h, (int32_t)(sumsq != nullptr), at);
    return adamw(plan, StepArgs{}, at, sumsq, st);
}

zpq_status zpq_state8_unpack(const uint8_t* codes, const uint8_t* exps, int64_t n, int32_t moment,
                             void* y, int32_t y_dtype, zpq_stream stream) {
    const zpq_status bad = state8_check(codes, exps, y, n, moment, y_dtype);
    if (bad != ZPQ_OK || n == 0) return bad;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (y_dtype == ZPQ_F32) launch_unpack<ZPQ_F32>(codes, exps, n, moment, y, st);
    else if (y_dtype == ZPQ_F16) launch_unpack<ZPQ_F16>(codes, exps, n, moment, y, st);
    else launch_unpack<ZPQ_BF16>(codes, exps, n, moment, y, st);
    return after_launch();
}

zpq_status zpq_state8_pack(const void* x, int32_t x_dtype, int64_t n, int32_t moment,
                           uint8_t* codes, uint8_t* exps, zpq_stream stream) {
    const zpq_status bad = state8_check(codes, exps, x, n, moment, x_dtype);
    if (bad != ZPQ_OK || n == 0) return bad;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (x_dtype == ZPQ_F32) launch_pack<ZPQ_F32>(x, n, moment, codes, exps, st);
    else if (x_dtype == ZPQ_F16) launch_pack<ZPQ_F16>(x, n, moment, codes, exps, st);
    else launch_pack<ZPQ_BF16>(x, n, moment, codes, exps, st);
    return after_launch();
}

}  // extern "C"
