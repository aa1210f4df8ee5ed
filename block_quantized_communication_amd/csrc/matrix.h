// matrix.h -- the tile loop of matrix products D = A * B^T on the matrix cores, for
// operands whose rows are consecutive along the sum: 8-bit floats with a power-of-two
// scale for each block of 128, or 16-bit floats.
//
// The unit along the sum is a slab, 128 bytes of a row: 128 8-bit or 64 16-bit
// elements.  Either way a lane's share of 16 rows is two 16-byte pieces and one
// slab of a 16 x 16 tile keeps the matrix core busy for 32 cycles, so both kinds
// share everything but the instruction.
//
// In LDS a slab is [row][128 bytes], the 16-byte piece c of row r at place c ^ (r & 7):
// 8 lanes that read the same piece of 8 rows then cover all banks.  The
// copy from global memory to LDS writes 16 bytes a lane in lane order, so the lanes'
// addresses are permuted instead.
#ifndef ZPQ_MATRIX_H
#define ZPQ_MATRIX_H

#include "step.h"

namespace zpq_matrix {

using namespace zpq_step;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kSlab = 128;                    // bytes of a row that one step takes
constexpr int kF16 = -1;                      // operand kind besides ZPQ_E4M3 and ZPQ_E5M2

// Rows of an operand: `rows` rows of `pitch` bytes (a multiple of 128, at most 2^23),
// and for 8-bit ones a row of exponent bytes, scale_pitch long (a multiple of 4),
// for each 2^scale_shift rows.
struct Operand {
    const uint8_t* data;
    const uint8_t* scale;
    int64_t rows;
    uint32_t pitch, scale_pitch, scale_shift;
};

// A buffer descriptor for reading [p, p + bytes): accesses past the end read nothing.
__device__ __forceinline__ i32x4 descriptor(const void* p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t n = bytes < 0 ? 0u : bytes > 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes;
    i32x4 d;
    d.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    d.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    d.z = __builtin_amdgcn_readfirstlane((int)n);
    d.w = 0x00020000;
    return d;
}

__device__ __forceinline__ uint32_t scalar(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// Copies 16 (or 4) bytes a lane from global memory to LDS at `to` (of the wave) + 16 (4) *
// lane.  Not the builtin: the compiler waits for it before any later LDS read.  These
// have no result register; whoever reads the bytes waits by wait_copies() and a barrier.
// `offset` and `to` are the same in all lanes.  (Five wait states: a scalar register that a vector
// instruction has written may be an operand.)
__device__ __forceinline__ void copy16(i32x4 from, uint32_t lane_offset, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(scalar(to)), "v"(lane_offset), "s"(from), "s"(scalar(offset)) : "m0", "memory");
}
__device__ __forceinline__ void copy4(i32x4 from, uint32_t lane_offset, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :: "s"(scalar(to)), "v"(lane_offset), "s"(from), "s"(scalar(offset)) : "m0", "memory");
}
// Until at most LEFT of the wave's memory accesses, the latest ones, are under way.
template <int LEFT = 0>
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LEFT) : "memory"); }
// Own LDS reads done, then all waves here.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// acc + one slab of 16 rows of B (rows of the result) times 16 rows of A (columns).
// Lane l gets rows 4 * (l / 16) .. + 3 of column l % 16.  The order of the slab's
// elements over the lanes does not matter as long as both operands share it, and
// the one scale of 128 elements is the instruction's four of 32.
template <int KA, int KB, int SEL>
__device__ __forceinline__ f32x4 product(i32x8 b, i32x8 a, f32x4 acc, int scale_b, int scale_a) {
    if constexpr (KA == kF16) {
        const i32x4 b0 = {b[0], b[1], b[2], b[3]}, b1 = {b[4], b[5], b[6], b[7]};
        const i32x4 a0 = {a[0], a[1], a[2], a[3]}, a1 = {a[4], a[5], a[6], a[7]};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b0), __builtin_bit_cast(f16x8, a0),
                                                     acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b1), __builtin_bit_cast(f16x8, a1),
                                                      acc, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, KB, KA, SEL, scale_b, SEL, scale_a);
    }
}

// 8 codes with their block's scale as bf16, which holds them exactly.
template <int KIND>
__device__ __forceinline__ bf16x8 widen8(int w0, int w1, float scale) {
    u32x4 r;
    if constexpr (KIND == ZPQ_E4M3) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w0, scale, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w0, scale, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w1, scale, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w1, scale, true));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w0, scale, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w0, scale, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w1, scale, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)w1, scale, true));
    }
    return __builtin_bit_cast(bf16x8, r);
}
// Byte SEL of a word of exponent bytes in the place where widen8 takes a scale's exponent from.
template <int SEL>
__device__ __forceinline__ float scale_byte(int word) {
    const uint32_t e = SEL == 3 ? (uint32_t)word >> 24 : ((uint32_t)word >> (8 * SEL)) & 0xFFu;
    return __uint_as_float(e << 23);
}

// acc[i][j] += one slab of a's 16 rows i times b's 16 rows j.  FULL: the 8-bit matrix
// instructions cut the products of 8 consecutive elements off, toward zero, 13 bits below the
// power of two of the largest before they add them, whichever instruction and whatever is in acc
// (as a root mean square 1.2e-5 of a sum of 128 normal values, 5e-5 with one in a hundred 30
// times as large); from there on, and in the 16-bit ones, sums keep binary32 (5e-8).  So with FULL
// the codes become bf16 with their scale, which is exact, at half the rate.
template <int KA, int KB, int SEL, bool FULL, int NA, int NB>
__device__ __forceinline__ void products(f32x4 (*acc)[NB], const i32x8 (&a)[NA], const i32x8 (&b)[NB], const int* sa,
                                         const int (&sb)[NB]) {
    if constexpr (FULL) {
        float fa[NA], fb[NB];
#pragma unroll
        for (int i = 0; i < NA; ++i) fa[i] = scale_byte<SEL>(sa[i]);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = scale_byte<SEL>(sb[j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            bf16x8 wb[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) wb[j] = widen8<KB>(b[j][2 * q], b[j][2 * q + 1], fb[j]);
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const bf16x8 wa = widen8<KA>(a[i][2 * q], a[i][2 * q + 1], fa[i]);
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[i][j] = product<KA, KB, SEL>(b[j], a[i], acc[i][j], KA == kF16 ? 0 : sb[j], KA == kF16 ? 0 : sa[i]);
    }
}

// What a wave does with its sums when the loop is over.  A lane holds 4 consecutive columns of 16 rows
// each; through the wave's own part of LDS they become 8 consecutive columns of a row, so that
// global memory sees whole rows:
//   l(row, column)         loads what f will need there, a group of 16 rows ahead of it
//   f(row, column, v, l)   the tile's row and first of 8 columns, their sums, what l loaded; may change the sums
//   g(column, row, h)      with TURN, what f made of them, rounded to binary16, the other way round: 8 consecutive rows
//                          of a column
// Written straight from the sums, 8 bytes a lane and 16 rows an instruction, a 256 x 256 tile's end
// took 25 us.
template <int MI, int NI, bool TURN, class L, class F, class G>
__device__ __forceinline__ void hand_out(const f32x4 (&acc)[MI][NI], uint8_t* shared, uint32_t wave, uint32_t row0, uint32_t col0,
                                         L&& l, F&& f, G&& g) {
    constexpr int COLS = NI * 16, CHUNKS = COLS / 4, LANES = COLS / 8, CALLS = 16 * LANES / 64;
    constexpr int HIGH = MI < 4 ? MI : 4, ROWS = HIGH * 16;      // rows that are turned at a time
    constexpr int STAGE = 16 * COLS * 4;
    meet();                                   // no wave reads operands any more
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));            // addresses are made here, not kept in registers through the loop
    uint8_t* stage = shared + wave * (STAGE + ROWS * COLS * 2);
    uint8_t* turned = stage + STAGE;
    decltype(l(0u, 0u)) here[CALLS], ahead[CALLS];
    const auto load = [&](int i, auto& to) {
#pragma unroll
        for (int k = 0; k < CALLS; ++k) to[k] = l(row0 + i * 16 + k * (64 / LANES) + lane / LANES, col0 + lane % LANES * 8);
    };
    load(0, ahead);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int k = 0; k < CALLS; ++k) here[k] = ahead[k];
        if (i + 1 < MI) load(i + 1, ahead);
        const uint32_t r = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < NI; ++j)
            *reinterpret_cast<f32x4*>(stage + r * (COLS * 4) + (((j * 4 + q) ^ (r & (CHUNKS - 1))) << 4)) = acc[i][j];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int k = 0; k < CALLS; ++k) {
            const uint32_t row = k * (64 / LANES) + lane / LANES, c = lane % LANES;
            const uint8_t* at = stage + row * (COLS * 4);
            const f32x4 x = *reinterpret_cast<const f32x4*>(at + (((c * 2) ^ (row & (CHUNKS - 1))) << 4));
            const f32x4 y = *reinterpret_cast<const f32x4*>(at + (((c * 2 + 1) ^ (row & (CHUNKS - 1))) << 4));
            float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            f(row0 + i * 16 + row, col0 + c * 8, v, here[k]);
            if constexpr (TURN) {
                const uint32_t high = (i % HIGH) * 16 + row;
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    *reinterpret_cast<_Float16*>(turned + (c * 8 + n) * (ROWS * 2) + (((high >> 3) ^ (c & (ROWS / 8 - 1))) << 4) + (high & 7) * 2) =
                        (_Float16)v[n];
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if constexpr (TURN) {
            if (i % HIGH == HIGH - 1) {
#pragma unroll
                for (int k = 0; k < COLS * (ROWS / 8) / 64; ++k) {
                    const uint32_t column = k * (64 / (ROWS / 8)) + lane / (ROWS / 8), c = lane % (ROWS / 8);
                    g(col0 + column, row0 + (i / HIGH) * ROWS + c * 8,
                      *reinterpret_cast<const u32x4*>(turned + column * (ROWS * 2) + ((c ^ ((column >> 3) & (ROWS / 8 - 1))) << 4)));
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
    }
}

// The loop of a 256 x 256 tile: 8 waves, each 128 rows of A by 64 of B, two waves on a
// SIMD; two buffers of one slab of both operands (128 KB of LDS), one barrier a slab.  The
// copy of the next slab starts right after the barrier, into the buffer that all waves have
// read by then, and has a whole slab's time to arrive.  Pieces of A are read two ahead of
// their products.
// Tried and slower: the two waves of a SIMD in turns, one reading and one multiplying (4 barriers a
// slab); half slabs in four buffers (64 bytes a row keep the address unit busier than the matrix cores);
// four waves of 128 x 128.
template <int KA, int KB, bool FULL = false>
struct Tile256 {
    static constexpr int BM = 256, BN = 256, kThreadsWg = 512, kWaves = 2, MI = 8, NI = 4;   // kWaves: on a SIMD
    static constexpr int kSide = 256 * kSlab, kBuffer = 2 * kSide;
    static constexpr bool kScaled = KA != kF16;
    static constexpr int kLds = 2 * kBuffer + (kScaled ? 2048 : 0);

    const uint8_t* lds;
    uint32_t base, wave, lane;
    i32x4 ra, rb, rs;
    uint32_t off[4], off_s;                    // both operands' rows have one pitch
    f32x4 acc[MI][NI];
    int sa[MI], sb[NI];

    __device__ __forceinline__ uint32_t wm() const { return wave >> 2; }
    __device__ __forceinline__ uint32_t wn() const { return wave & 3; }

    __device__ __forceinline__ void start_copy(int slab, int buffer) {
        const uint32_t to = base + buffer * kBuffer + wave * 4096;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            copy16(ra, off[i], (uint32_t)slab * kSlab, to + i * 1024);
            copy16(rb, off[i], (uint32_t)slab * kSlab, to + kSide + i * 1024);
        }
        if constexpr (kScaled)
            if ((slab & 3) == 0) copy4(rs, off_s, (uint32_t)slab, base + 2 * kBuffer + wave * 256);
    }
    __device__ __forceinline__ i32x8 piece(const uint8_t* side, uint32_t row) const {
        const uint32_t r = lane & 15, g = lane >> 4;
        const uint8_t* p = side + (row + r) * kSlab;
        const i32x4 x = *reinterpret_cast<const i32x4*>(p + ((g ^ (r & 7)) << 4));
        const i32x4 y = *reinterpret_cast<const i32x4*>(p + (((g + 4) ^ (r & 7)) << 4));
        return i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
    // Slab `slab` of [.., end), SEL = its number from the first one modulo 4.
    template <int SEL>
    __device__ __forceinline__ void step(int slab, int end) {
        constexpr int buffer = SEL & 1;
        const uint8_t* side_a = lds + buffer * kBuffer + wm() * 128 * kSlab;
        const uint8_t* side_b = lds + buffer * kBuffer + kSide + wn() * 64 * kSlab;
        wait_copies();
        meet();                               // the slab is there, and the other buffer read
        if constexpr (kScaled && SEL == 0) {
            const int* s = reinterpret_cast<const int*>(lds + 2 * kBuffer) + (lane & 15);
#pragma unroll
            for (int i = 0; i < MI; ++i) sa[i] = s[wm() * 128 + i * 16];
#pragma unroll
            for (int j = 0; j < NI; ++j) sb[j] = s[256 + wn() * 64 + j * 16];
        }
        i32x8 fb[NI], one[2], two[2];
        one[0] = piece(side_a, 0);
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[j] = piece(side_b, j * 16);
        one[1] = piece(side_a, 16);
        if (slab + 1 < end) start_copy(slab + 1, buffer ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        two[0] = piece(side_a, 32);
        two[1] = piece(side_a, 48);
        products<KA, KB, SEL, FULL>(acc, one, fb, sa, sb);
        pin<0>();
        __builtin_amdgcn_sched_barrier(0);
        one[0] = piece(side_a, 64);
        one[1] = piece(side_a, 80);
        products<KA, KB, SEL, FULL>(acc + 2, two, fb, sa + 2, sb);
        pin<2>();
        __builtin_amdgcn_sched_barrier(0);
        two[0] = piece(side_a, 96);
        two[1] = piece(side_a, 112);
        products<KA, KB, SEL, FULL>(acc + 4, one, fb, sa + 4, sb);
        pin<4>();
        __builtin_amdgcn_sched_barrier(0);
        products<KA, KB, SEL, FULL>(acc + 6, two, fb, sa + 6, sb);
        pin<6>();
        __builtin_amdgcn_sched_barrier(0);
    }
    // Here, not later: without this the compiler moves products behind branches and barriers.
    template <int FIRST>
    __device__ __forceinline__ void pin() {
#pragma unroll
        for (int i = FIRST; i < FIRST + 2; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    }

    // Sums slabs [first, end), none or some, first a multiple of 4 with scales, of the tile that starts
    // at row row_a of A and row_b of B (multiples of 256).
    __device__ __forceinline__ void run(const Operand& a, const Operand& b, int64_t row_a, int64_t row_b, int first,
                                        int end, uint8_t* shared) {
        first = (int)scalar((uint32_t)first);
        end = (int)scalar((uint32_t)end);
        lds = shared;
        base = lds_address(shared);
        lane = threadIdx.x & 63;
        wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        ra = descriptor(a.data + row_a * a.pitch, (a.rows - row_a) * a.pitch);
        rb = descriptor(b.data + row_b * b.pitch, (b.rows - row_b) * b.pitch);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = wave * 32 + i * 8 + (lane >> 3);
            off[i] = r * a.pitch + (((lane & 7) ^ (r & 7)) << 4);
        }
        if constexpr (kScaled) {
            const Operand& o = wave < 4 ? a : b;
            const int64_t row = (wave < 4 ? row_a : row_b) >> o.scale_shift;
            const int64_t rows = ((o.rows - 1) >> o.scale_shift) + 1;
            rs = descriptor(o.scale + row * o.scale_pitch, (rows - row) * o.scale_pitch);
            off_s = (((wave & 3) * 64 + lane) >> o.scale_shift) * o.scale_pitch;
        }
        clear();
        if (first >= end) return;
        start_copy(first, 0);
        for (int slab = first; slab < end; slab += 4) {
            step<0>(slab, end);
            if (slab + 1 < end) step<1>(slab + 1, end);
            if (slab + 2 < end) step<2>(slab + 2, end);
            if (slab + 3 < end) step<3>(slab + 3, end);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    }
    template <bool TURN, class L, class F, class G>
    __device__ __forceinline__ void finish(uint8_t* shared, L&& l, F&& f, G&& g) const {
        hand_out<MI, NI, TURN>(acc, shared, wave, wm() * 128, wn() * 64, l, f, g);
    }
};

// The loop of a smaller tile: 4 waves, 2 x 2, each MI * 16 rows of A by NI * 16 of B.  Several
// workgroups of a CU hide each other's waits. BUFFERS: 2, or 4 where there are few workgroups and a copy's
// way is what takes time (1024 x 1024 orthogonalised: 196 -> 149 us; but 999 x 4004 x 1001, 1008 tiles, 10.3 -> 11.4,
// since only two workgroups of four buffers fit a CU).
template <int KA, int KB, int MI_, int NI_, bool FULL = false, int BUFFERS = 2>
struct TileSmall {
    static constexpr int MI = MI_, NI = NI_, BM = 32 * MI, BN = 32 * NI, kThreadsWg = 256, kWaves = 2;
    static constexpr int kSideA = BM * kSlab, kSideB = BN * kSlab, kBuffer = kSideA + kSideB;
    static constexpr bool kScaled = KA != kF16;
    static constexpr int kScaleBytes = kScaled ? (BM + BN) * 4 : 0;
    static constexpr int kBuffers = BUFFERS, kCopies = MI + NI;       // copies of a slab, of a wave
    static constexpr int kLds = kBuffers * kBuffer + kScaleBytes;
    static_assert(BM + BN <= 256, "one exponent word a thread");

    const uint8_t* lds;
    uint32_t base, wave, lane;
    i32x4 ra, rb, rs;
    uint32_t off_a[MI], off_b[NI], off_s;
    f32x4 acc[MI][NI];
    int sa[MI], sb[NI];

    __device__ __forceinline__ uint32_t wm() const { return wave >> 1; }
    __device__ __forceinline__ uint32_t wn() const { return wave & 1; }

    // Waves past the exponent words' rows bring the others' again, so that all wait for the same number.
    __device__ __forceinline__ uint32_t scale_wave() const { return wave % ((BM + BN) / 64); }

    __device__ __forceinline__ void start_copy(int slab, int buffer) {
        const uint32_t to = base + buffer * kBuffer;
#pragma unroll
        for (int i = 0; i < MI; ++i) copy16(ra, off_a[i], (uint32_t)slab * kSlab, to + (wave * MI + i) * 1024);
#pragma unroll
        for (int j = 0; j < NI; ++j) copy16(rb, off_b[j], (uint32_t)slab * kSlab, to + kSideA + (wave * NI + j) * 1024);
    }
    __device__ __forceinline__ void start_scales(int slab) {
        if constexpr (kScaled)
            copy4(rs, off_s, (uint32_t)slab, base + kBuffers * kBuffer + scale_wave() * 256);
    }
    __device__ __forceinline__ i32x8 piece(const uint8_t* side, uint32_t row) const {
        const uint32_t r = lane & 15, g = lane >> 4;
        const uint8_t* p = side + (row + r) * kSlab;
        const i32x4 x = *reinterpret_cast<const i32x4*>(p + ((g ^ (r & 7)) << 4));
        const i32x4 y = *reinterpret_cast<const i32x4*>(p + (((g + 4) ^ (r & 7)) << 4));
        return i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
    template <int SEL>
    __device__ __forceinline__ void step(int slab, int end) {
        constexpr int buffer = SEL & (kBuffers - 1), freed = (SEL + kBuffers - 1) & (kBuffers - 1);
        // copies of the slabs between this one and those that are not started yet may be under way
        if constexpr (kBuffers == 2) {
            wait_copies();
        } else {
            if (slab + 2 < end) wait_copies<2 * kCopies + (kScaled && SEL >= 2)>();
            else if (slab + 1 < end) wait_copies<kCopies + (kScaled && SEL == 3)>();
            else wait_copies();
        }
        meet();                               // slab is there, and the buffer of the one before read
        if constexpr (kScaled && SEL == 0) {
            const int* s = reinterpret_cast<const int*>(lds + kBuffers * kBuffer) + (lane & 15);
#pragma unroll
            for (int i = 0; i < MI; ++i) sa[i] = s[(wm() * MI + i) * 16];
#pragma unroll
            for (int j = 0; j < NI; ++j) sb[j] = s[BM + (wn() * NI + j) * 16];
        }
        if (slab + kBuffers - 1 < end) {
            if constexpr (((SEL + kBuffers - 1) & 3) == 0) start_scales(slab + kBuffers - 1);
            start_copy(slab + kBuffers - 1, freed);
        }
        const uint8_t* side_a = lds + buffer * kBuffer + wm() * MI * 16 * kSlab;
        const uint8_t* side_b = lds + buffer * kBuffer + kSideA + wn() * NI * 16 * kSlab;
        i32x8 fb[NI], fa[MI];
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[j] = piece(side_b, j * 16);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = piece(side_a, i * 16);
        products<KA, KB, SEL, FULL>(acc, fa, fb, sa, sb);
    }
    // As Tile256::run; row_a and row_b multiples of BM and BN.
    __device__ __forceinline__ void run(const Operand& a, const Operand& b, int64_t row_a, int64_t row_b, int first,
                                        int end, uint8_t* shared) {
        first = (int)scalar((uint32_t)first);
        end = (int)scalar((uint32_t)end);
        lds = shared;
        base = lds_address(shared);
        lane = threadIdx.x & 63;
        wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        ra = descriptor(a.data + row_a * a.pitch, (a.rows - row_a) * a.pitch);
        rb = descriptor(b.data + row_b * b.pitch, (b.rows - row_b) * b.pitch);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const uint32_t r = (wave * MI + i) * 8 + (lane >> 3);
            off_a[i] = r * a.pitch + (((lane & 7) ^ (r & 7)) << 4);
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const uint32_t r = (wave * NI + j) * 8 + (lane >> 3);
            off_b[j] = r * b.pitch + (((lane & 7) ^ (r & 7)) << 4);
        }
        if constexpr (kScaled) {
            const bool of_a = scale_wave() * 64 < BM;
            const Operand& o = of_a ? a : b;
            const int64_t row = of_a ? row_a : row_b, within = scale_wave() * 64 + lane - (of_a ? 0 : BM);
            const int64_t first_scale = row >> o.scale_shift, rows = ((o.rows - 1) >> o.scale_shift) + 1;
            rs = descriptor(o.scale + first_scale * o.scale_pitch, (rows - first_scale) * o.scale_pitch);
            off_s = (uint32_t)(((row + within) >> o.scale_shift) - first_scale) * o.scale_pitch;
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        start_scales(first);
#pragma unroll
        for (int i = 0; i < kBuffers - 1; ++i)
            if (first + i < end) start_copy(first + i, i);
        for (int slab = first; slab < end; slab += 4) {
            step<0>(slab, end);
            if (slab + 1 < end) step<1>(slab + 1, end);
            if (slab + 2 < end) step<2>(slab + 2, end);
            if (slab + 3 < end) step<3>(slab + 3, end);
        }
    }
    template <bool TURN, class L, class F, class G>
    __device__ __forceinline__ void finish(uint8_t* shared, L&& l, F&& f, G&& g) const {
        hand_out<MI, NI, TURN>(acc, shared, wave, wm() * MI * 16, wn() * NI * 16, l, f, g);
    }
};

// Workgroup `id` of `count` to tile (i, j) of rows x columns tiles.  Workgroups go to the 8
// XCDs in turn, and each XCD has an L2 of its own: the ids of one XCD become consecutive
// tiles of bands of 4 tile rows, so that the 32 tiles it works on at a time share 4 row and
// 8 column strips (bands of 4 measured 5% faster than of 8 or 16, and 15% than no order).
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t count, uint32_t rows, uint32_t columns, uint32_t& i,
                                        uint32_t& j) {
    const uint32_t q = count / 8, r = count % 8, x = id % 8;
    const uint32_t t = x * q + (x < r ? x : r) + id / 8;
    const uint32_t band = t / (4 * columns), in = t - band * 4 * columns;
    const uint32_t high = rows - band * 4 < 4 ? rows - band * 4 : 4;
    j = in / high;
    i = band * 4 + (in - j * high);
}

constexpr int64_t kFewWorkgroups = 512;       // two a CU: up to here four buffers

}  // namespace zpq_matrix

#endif  // ZPQ_MATRIX_H
