// float8.hip -- 8-bit floating-point blocks of 128 with a power-of-two scale (quantizing along
// rows, along columns and in tiles; back to floats; transposing tiles) and the products of
// such operands.  Definitions: zpq.h.
#include <type_traits>

#include "matrix.h"

namespace {

using namespace zpq_matrix;

constexpr int kBlock = 128;                   // elements of a block, and rows of a tile
constexpr int64_t kMaxRow = 1 << 23;          // bytes of a row of codes (32-bit offsets in a tile of 256 rows)

// ---------------------------------------------------------------------------
// Quantizing.  A lane has 8 consecutive elements, 16 lanes a block.  The exponent byte
// is integer arithmetic on the largest magnitude's bits: one added to its exponent
// field where its fraction is over 0.75 (the largest value is 1.75 * 2^top), less top.
// The scale is a power of two, so the division is an exact product and the code's rounding
// the only one.
template <int KIND>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t most) {
    constexpr int top = KIND == ZPQ_E4M3 ? 8 : 15;
    const int e = (int)((most + 0x1FFFFFu) >> 23) - top;
    return most >= 0x7F800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}
// 2^(127 - byte); NaN for blocks with a value that is not finite.
__device__ __forceinline__ float unit_of(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : (254u - byte) << 23);
}
// 2^(byte - 127); infinite for 255, whose codes are NaNs.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}
template <int KIND>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int w = 0;
    if constexpr (KIND == ZPQ_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return (uint32_t)w;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    return umax(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}
// Maximum over the 16 lanes of a row: lane ^ 1, lane ^ 2, then mirrored halves and rows.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = max_dpp<0xB1>(x);
    x = max_dpp<0x4E>(x);
    x = max_dpp<0x141>(x);
    return max_dpp<0x140>(x);
}

template <int DT>
__device__ __forceinline__ void load8(Raw<DT, 8>& r, const void* x, int64_t at, int64_t have) {
    if (have >= 8) r.load(x, at);
    else r.load_some(x, at, have < 0 ? 0 : (int)have);
}
template <int DT>
__device__ __forceinline__ uint32_t most8(const Raw<DT, 8>& r) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = umax(m, __float_as_uint(r.get(k)) & 0x7FFFFFFFu);
    return m;
}
template <int DT, int KIND>
__device__ __forceinline__ u32x2 codes8(const Raw<DT, 8>& r, float unit) {
    return u32x2{codes4<KIND>(r.get(0) * unit, r.get(1) * unit, r.get(2) * unit, r.get(3) * unit),
                 codes4<KIND>(r.get(4) * unit, r.get(5) * unit, r.get(6) * unit, r.get(7) * unit)};
}

struct Quant {
    const void* x;
    int64_t rows, cols, ld;
    uint8_t *codes, *scales, *codes_t, *scales_t;
    uint32_t blocks, blocks4, blocks_t, blocks4_t;   // along a row; along a column
};

// Blocks along rows only: 16 lanes a block, kEach blocks of theirs in flight.
constexpr int kEach = 2;
template <int DT, int KIND>
__global__ __launch_bounds__(kThreads) void k_quant_rows(Quant q, int64_t count) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 16 * kEach);
    const int64_t row0 = first / q.blocks;
    const uint32_t rem = (uint32_t)(first - row0 * q.blocks), c = threadIdx.x & 15;
    Raw<DT, 8> raw[kEach];
    int64_t row[kEach];
    uint32_t block[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t k = i * (kThreads / 16) + (threadIdx.x >> 4), over = (rem + k) / q.blocks;
        row[i] = row0 + over;
        block[i] = rem + k - over * q.blocks;
        const int64_t col = (int64_t)block[i] * kBlock + c * 8;
        load8<DT>(raw[i], q.x, row[i] * q.ld + col, first + k < count ? q.cols - col : 0);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (first + i * (kThreads / 16) + (threadIdx.x >> 4) >= count) continue;   // all 16 lanes or none
        const uint32_t byte = exponent_byte<KIND>(max16(most8<DT>(raw[i])));
        *reinterpret_cast<u32x2*>(q.codes + (row[i] * q.blocks + block[i]) * kBlock + c * 8) =
            codes8<DT, KIND>(raw[i], unit_of(byte));
        // the last block's lanes also write the unused bytes behind it
        const uint32_t n = block[i] + 1 == q.blocks ? q.blocks4 - block[i] : 1;
        if (c < n) q.scales[row[i] * q.blocks4 + block[i] + c] = (uint8_t)(c == 0 ? byte : 0);
    }
}

// A tile of 128 x 128: every lane an 8 x 8 piece, which it rounds along its rows and, packed the other
// way, along its columns; the column codes go through LDS so that both are written in
// whole 128 bytes.  The input is read once for both.
template <int DT, int KIND, bool TILE, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads) void k_quant_tile(Quant q) {
    __shared__ uint32_t most_of[TILE ? 4 : 4 * kBlock];
    __shared__ __attribute__((aligned(16))) u32x2 turned[COLS ? kBlock * 16 : 1];
    static_assert(__alignof__(turned) >= alignof(u32x4), "read 16 bytes at a time");
    const uint32_t t = threadIdx.x, c = t & 15, r = t >> 4, wave = t >> 6;
    const uint32_t cb = blockIdx.x % q.blocks, rb = blockIdx.x / q.blocks;
    const int64_t row = (int64_t)rb * kBlock + r * 8, col = (int64_t)cb * kBlock + c * 8;
    Raw<DT, 8> raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) load8<DT>(raw[p], q.x, (row + p) * q.ld + col, row + p < q.rows ? q.cols - col : 0);

    uint32_t byte = 0, byte_t[8];
    if constexpr (TILE) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) m = umax(m, most8<DT>(raw[p]));
        m = max16(m);
        m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
        m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
        if ((t & 63) == 0) most_of[wave] = m;
        __syncthreads();
        byte = exponent_byte<KIND>(umax(umax(most_of[0], most_of[1]), umax(most_of[2], most_of[3])));
    } else if constexpr (COLS) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) m = umax(m, __float_as_uint(raw[p].get(k)) & 0x7FFFFFFFu);
            m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
            m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
            if ((t & 48) == 0) most_of[wave * kBlock + c * 8 + k] = m;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t at = c * 8 + k;
            byte_t[k] = exponent_byte<KIND>(umax(umax(most_of[at], most_of[kBlock + at]),
                                                 umax(most_of[2 * kBlock + at], most_of[3 * kBlock + at])));
        }
    }
    if constexpr (ROWS) {
        const uint32_t n = cb + 1 == q.blocks ? q.blocks4 - cb : 1;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if constexpr (!TILE) byte = exponent_byte<KIND>(max16(most8<DT>(raw[p])));
            if (row + p < q.rows) {
                *reinterpret_cast<u32x2*>(q.codes + ((row + p) * q.blocks + cb) * kBlock + c * 8) =
                    codes8<DT, KIND>(raw[p], unit_of(byte));
                if (!TILE && c < n) q.scales[(row + p) * q.blocks4 + cb + c] = (uint8_t)(c == 0 ? byte : 0);
            }
        }
        if (TILE && t < n) q.scales[(int64_t)rb * q.blocks4 + cb + t] = (uint8_t)(t == 0 ? byte : 0);
    }
    if constexpr (COLS) {
        const uint32_t n = rb + 1 == q.blocks_t ? q.blocks4_t - rb : 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float unit = unit_of(TILE ? byte : byte_t[k]);
            turned[(c * 8 + k) * 16 + (r ^ c)] =
                u32x2{codes4<KIND>(raw[0].get(k) * unit, raw[1].get(k) * unit, raw[2].get(k) * unit, raw[3].get(k) * unit),
                      codes4<KIND>(raw[4].get(k) * unit, raw[5].get(k) * unit, raw[6].get(k) * unit, raw[7].get(k) * unit)};
            if (!TILE && r < n && col + k < q.cols)
                q.scales_t[(col + k) * q.blocks4_t + rb + r] = (uint8_t)(r == 0 ? byte_t[k] : 0);
        }
        if (TILE && t < n) q.scales_t[(int64_t)cb * q.blocks4_t + rb + t] = (uint8_t)(t == 0 ? byte : 0);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t column = p * 32 + (t >> 3), pair = t & 7, h = column >> 3;
            const u32x4 w = *reinterpret_cast<const u32x4*>(&turned[column * 16 + ((pair ^ (h >> 1)) << 1)]);
            const int64_t at = (int64_t)cb * kBlock + column;
            if (at < q.cols)
                *reinterpret_cast<u32x4*>(q.codes_t + (at * q.blocks_t + rb) * kBlock + pair * 16) =
                    (h & 1) ? u32x4{w.z, w.w, w.x, w.y} : w;
        }
    }
}

// Codes of tiles the other way round, as k_quant_tile writes both.
__global__ __launch_bounds__(kThreads) void k_transpose(Quant q) {
    __shared__ __attribute__((aligned(16))) u32x2 turned[kBlock * 16];
    static_assert(__alignof__(turned) >= alignof(u32x4), "read 16 bytes at a time");
    const uint32_t t = threadIdx.x, c = t & 15, r = t >> 4;
    const uint32_t cb = blockIdx.x % q.blocks, rb = blockIdx.x / q.blocks;
    const int64_t row = (int64_t)rb * kBlock + r * 8;
    u32x2 in[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
        in[p] = row + p < q.rows ? *reinterpret_cast<const u32x2*>(q.codes + ((row + p) * q.blocks + cb) * kBlock + c * 8)
                                 : u32x2{0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        u32x2 o = {0, 0};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint32_t b = ((k < 4 ? in[p].x : in[p].y) >> (8 * (k & 3))) & 0xFFu;
            if (p < 4) o.x |= b << (8 * p);
            else o.y |= b << (8 * (p - 4));
        }
        turned[(c * 8 + k) * 16 + (r ^ c)] = o;
    }
    const uint32_t n = rb + 1 == q.blocks_t ? q.blocks4_t - rb : 1;
    if (t < n) q.scales_t[(int64_t)cb * q.blocks4_t + rb + t] = t == 0 ? q.scales[(int64_t)rb * q.blocks4 + cb] : 0;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t column = p * 32 + (t >> 3), pair = t & 7, h = column >> 3;
        const u32x4 w = *reinterpret_cast<const u32x4*>(&turned[column * 16 + ((pair ^ (h >> 1)) << 1)]);
        const int64_t at = (int64_t)cb * kBlock + column;
        if (at < q.cols)
            *reinterpret_cast<u32x4*>(q.codes_t + (at * q.blocks_t + rb) * kBlock + pair * 16) =
                (h & 1) ? u32x4{w.z, w.w, w.x, w.y} : w;
    }
}

// Values: a lane 8 of them.
template <int KIND, int DT>
__global__ __launch_bounds__(kThreads) void k_dequant(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                      int64_t cols, uint32_t blocks, uint32_t blocks4, int64_t count,
                                                      uint32_t shift, void* y, int64_t ld) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 16 * kEach);
    const int64_t row0 = first / blocks;
    const uint32_t rem = (uint32_t)(first - row0 * blocks), c = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t k = i * (kThreads / 16) + (threadIdx.x >> 4), over = (rem + k) / blocks;
        const int64_t row = row0 + over;
        const uint32_t block = rem + k - over * blocks;
        if (first + k >= count) continue;
        const u32x2 w = *reinterpret_cast<const u32x2*>(codes + (row * blocks + block) * kBlock + c * 8);
        const float s = scale_of(scales[(row >> shift) * blocks4 + block]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int word = (int)(j < 2 ? w.x : w.y);
            f32x2 f;
            if constexpr (KIND == ZPQ_E4M3)
                f = (j & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(word, true) : __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
            else
                f = (j & 1) ? __builtin_amdgcn_cvt_pk_f32_bf8(word, true) : __builtin_amdgcn_cvt_pk_f32_bf8(word, false);
            v[2 * j] = f.x * s;
            v[2 * j + 1] = f.y * s;
        }
        const int64_t col = (int64_t)block * kBlock + c * 8, have = cols - col;
        Raw<DT, 8> out;
        out.set(v);
        if (have >= 8) out.store(y, row * ld + col);
        else if (have > 0) out.store_some(y, row * ld + col, (int)have);
    }
}

// ---------------------------------------------------------------------------
// Products.
struct Result {
    void* out;
    int64_t m, n, ld;
    int32_t dtype, accumulate;
    float* parts;                              // of a sum that is split: [split][m][n]
    uint32_t tiles_m, tiles_n;
    int32_t slabs, per_split;
};

// E consecutive results of a row, `have` of them inside.
template <int DT, int E>
__device__ __forceinline__ void put(const Result& o, int64_t row, int64_t col, float (&x)[E], int have) {
    const int64_t at = row * o.ld + col;
    Raw<DT, E> r;
    if (o.accumulate) {
        if (have >= E) r.template load<false>(o.out, at);
        else r.load_some(o.out, at, have);
#pragma unroll
        for (int k = 0; k < E; ++k) x[k] += r.get(k);
    }
    r.set(x);
    if (have >= E) r.template store<false>(o.out, at);
    else r.store_some(o.out, at, have);
}
template <int E>
__device__ __forceinline__ void put(const Result& o, int64_t row, int64_t col, float (&x)[E]) {
    const int have = o.n - col < E ? (int)(o.n - col) : E;
    if (o.dtype == ZPQ_F32) put<ZPQ_F32, E>(o, row, col, x, have);
    else if (o.dtype == ZPQ_F16) put<ZPQ_F16, E>(o, row, col, x, have);
    else put<ZPQ_BF16, E>(o, row, col, x, have);
}

template <class TILE>
__global__ __launch_bounds__(TILE::kThreadsWg, TILE::kWaves) void k_matmul(Operand a, Operand b, Result o) {
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::kLds];
    const uint32_t tiles = o.tiles_m * o.tiles_n, split = blockIdx.x / tiles;
    uint32_t i, j;
    tile_of(blockIdx.x - split * tiles, tiles, o.tiles_m, o.tiles_n, i, j);
    const int64_t row_a = (int64_t)i * TILE::BM, row_b = (int64_t)j * TILE::BN;
    const int first = (int)split * o.per_split;
    TILE t;
    t.run(a, b, row_a, row_b, first, first + o.per_split < o.slabs ? first + o.per_split : o.slabs, shared);
    const auto none = [](uint32_t, uint32_t, u32x4) {};
    const auto nothing = [](uint32_t, uint32_t) { return 0; };
    if (o.parts != nullptr) {
        float* part = o.parts + (int64_t)split * o.m * o.n;
        t.template finish<false>(shared, nothing, [&](uint32_t x, uint32_t y, float (&v)[8], int) {
            const int64_t row = row_a + x, col = row_b + y;
            if (row >= o.m || col >= o.n) return;
            Raw<ZPQ_F32, 8> r;
            r.set(v);
            if (o.n - col >= 8) r.template store<false>(part, row * o.n + col);
            else r.store_some(part, row * o.n + col, (int)(o.n - col));
        }, none);
    } else {
        // binary32 results that are added to, whole pieces of a row: loaded ahead
        const bool ahead = o.accumulate && o.dtype == ZPQ_F32;
        t.template finish<false>(shared, [&](uint32_t x, uint32_t y) {
            Raw<ZPQ_F32, 8> old = {};
            if (ahead && row_a + x < o.m && row_b + y + 8 <= o.n)
                old.template load<false>(o.out, (row_a + x) * o.ld + row_b + y);
            return old;
        }, [&](uint32_t x, uint32_t y, float (&v)[8], const Raw<ZPQ_F32, 8>& old) {
            const int64_t row = row_a + x, col = row_b + y;
            if (row >= o.m || col >= o.n) return;
            if (ahead && col + 8 <= o.n) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += old.get(k);
                Raw<ZPQ_F32, 8> sum;
                sum.set(v);
                sum.template store<false>(o.out, row * o.ld + col);
            } else {
                put(o, row, col, v);
            }
        }, none);
    }
}

// Few rows of A (up to 16 * MI): the weight streams past once.  A workgroup has 16 rows of B; its 8 waves take
// four slabs (one exponent word) each in turn, straight from memory into registers, and add
// up in LDS.  Nothing is shared, so nothing goes through LDS on the way in.
constexpr int kFewWaves = 8;
template <int KA, int KB, bool FULL, int MI>
__global__ __launch_bounds__(kFewWaves * 64) void k_matmul_few(Operand a, Operand b, Result o) {
    __shared__ f32x4 sums[kFewWaves][MI][64];
    const uint32_t lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const uint32_t split = blockIdx.x / o.tiles_n;
    const int64_t col0 = (int64_t)(blockIdx.x - split * o.tiles_n) * 16;
    const int first = (int)split * o.per_split, end = first + o.per_split < o.slabs ? first + o.per_split : o.slabs;
    const int64_t row_b = col0 + r < o.n ? col0 + r : o.n - 1;             // rows past the end: the last one again
    const uint8_t *pb = b.data + row_b * b.pitch + g * 16, *sb = b.scale + (row_b >> b.scale_shift) * b.scale_pitch;
    const uint8_t *pa[MI], *sa[MI];
    f32x4 acc[1][1], all[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t row = i * 16 + r < o.m ? i * 16 + r : o.m - 1;
        pa[i] = a.data + row * a.pitch + g * 16;
        sa[i] = a.scale + (row >> a.scale_shift) * a.scale_pitch;
        all[i] = f32x4{0, 0, 0, 0};
    }
    const auto piece = [](const uint8_t* p) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(p), y = *reinterpret_cast<const i32x4*>(p + 64);
        return i32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };
    const auto one = [&](auto sel, const i32x8& fa, const i32x8& fb, int wa, int wb, f32x4& to) {
        const i32x8 x[1] = {fa}, y[1] = {fb};
        const int ya[1] = {wa}, yb[1] = {wb};
        acc[0][0] = to;
        products<KA, KB, decltype(sel)::value, FULL>(acc, x, y, ya, yb);
        to = acc[0][0];
    };
    for (int slab = first + (int)wave * 4; slab < end; slab += kFewWaves * 4) {
        const int wb = *reinterpret_cast<const int*>(sb + slab);
        int wa[MI];
        i32x8 fb[4], fa[MI][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = (int64_t)(slab + k < end ? slab + k : slab) * kSlab;
            fb[k] = piece(pb + at);
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i][k] = piece(pa[i] + at);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            wa[i] = *reinterpret_cast<const int*>(sa[i] + slab);
            one(std::integral_constant<int, 0>{}, fa[i][0], fb[0], wa[i], wb, all[i]);
            if (slab + 1 < end) one(std::integral_constant<int, 1>{}, fa[i][1], fb[1], wa[i], wb, all[i]);
            if (slab + 2 < end) one(std::integral_constant<int, 2>{}, fa[i][2], fb[2], wa[i], wb, all[i]);
            if (slab + 3 < end) one(std::integral_constant<int, 3>{}, fa[i][3], fb[3], wa[i], wb, all[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) sums[wave][i][lane] = all[i];
    __syncthreads();
    if (wave >= MI) return;
    f32x4 sum = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) sum += sums[w][wave][lane];
    const int64_t row = wave * 16 + r, col = col0 + g * 4;
    if (row >= o.m || col >= o.n) return;
    float v[4] = {sum.x, sum.y, sum.z, sum.w};
    if (o.parts == nullptr) {
        put(o, row, col, v);
    } else {
        float* part = o.parts + ((int64_t)split * o.m + row) * o.n + col;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (col + k < o.n) part[k] = v[k];
    }
}

// The parts of a split sum, in order.
__global__ __launch_bounds__(kThreads) void k_join(Result o, int32_t splits) {
    const int64_t per_row = (o.n + 3) / 4, all = o.m * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / per_row, col = (i - row * per_row) * 4;
        float sum[4] = {0, 0, 0, 0};
        for (int s = 0; s < splits; ++s) {
            const float* p = o.parts + ((int64_t)s * o.m + row) * o.n + col;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col + k < o.n) sum[k] += p[k];
        }
        put(o, row, col, sum);
    }
}

// A sum of nothing.
__global__ __launch_bounds__(kThreads) void k_empty(Result o) {
    const int64_t per_row = (o.n + 3) / 4, all = o.m * per_row;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / per_row;
        float zero[4] = {0, 0, 0, 0};
        put(o, row, (i - row * per_row) * 4, zero);
    }
}

// ---------------------------------------------------------------------------
// Host side.
constexpr int64_t kMaxGrid = (1 << 24) - 1;   // workgroups of 256: a dispatch holds fewer than 2^32 work-items
inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }
inline int64_t blocks4_of(int64_t n) { return (blocks_of(n) + 3) / 4 * 4; }
inline bool kind_ok(int32_t k) { return k == ZPQ_E4M3 || k == ZPQ_E5M2; }

struct Extent { const void* p; uint64_t bytes; };

template <int DT, int KIND>
void launch_quant(const Quant& q, bool tile, hipStream_t st) {
    if (!tile && !q.codes_t) {
        const int64_t count = q.rows * q.blocks, per = kThreads / 16 * kEach;
        hipLaunchKernelGGL((k_quant_rows<DT, KIND>), dim3((uint32_t)((count + per - 1) / per)), dim3(kThreads), 0, st, q, count);
        return;
    }
    const dim3 grid((uint32_t)(q.blocks * q.blocks_t)), wg(kThreads);
    if (tile) {
        if (q.codes && q.codes_t) hipLaunchKernelGGL((k_quant_tile<DT, KIND, true, true, true>), grid, wg, 0, st, q);
        else if (q.codes) hipLaunchKernelGGL((k_quant_tile<DT, KIND, true, true, false>), grid, wg, 0, st, q);
        else hipLaunchKernelGGL((k_quant_tile<DT, KIND, true, false, true>), grid, wg, 0, st, q);
    } else {
        if (q.codes) hipLaunchKernelGGL((k_quant_tile<DT, KIND, false, true, true>), grid, wg, 0, st, q);
        else hipLaunchKernelGGL((k_quant_tile<DT, KIND, false, false, true>), grid, wg, 0, st, q);
    }
}

template <int KIND>
void launch_quant(const Quant& q, int32_t dtype, bool tile, hipStream_t st) {
    if (dtype == ZPQ_F32) launch_quant<ZPQ_F32, KIND>(q, tile, st);
    else if (dtype == ZPQ_F16) launch_quant<ZPQ_F16, KIND>(q, tile, st);
    else launch_quant<ZPQ_BF16, KIND>(q, tile, st);
}

template <class TILE>
void launch_tiles(const Operand& a, const Operand& b, Result o, int64_t splits, hipStream_t st) {
    o.tiles_m = (uint32_t)((o.m + TILE::BM - 1) / TILE::BM);
    o.tiles_n = (uint32_t)((o.n + TILE::BN - 1) / TILE::BN);
    hipLaunchKernelGGL((k_matmul<TILE>), dim3((uint32_t)(o.tiles_m * (int64_t)o.tiles_n * splits)), dim3(TILE::kThreadsWg), 0, st, a, b,
                       o);
}

inline dim3 grid_of_quads(int64_t m, int64_t n) {
    const int64_t wgs = (m * ((n + 3) / 4) + kThreads - 1) / kThreads;
    return dim3((uint32_t)(wgs < 65536 ? wgs : 65536));
}

// How a product is cut: the tile's side and the parts of its sum.
struct Cut { int side; int64_t splits; int32_t per_split; };

// bf16 results: tiles of 256 where they keep half of the 256 CUs busy (3000 x 3000 x 8192, 144 tiles: 86 us, 118 with
// tiles of 64; 95 with 128), else of 64 (2048 x 2048 x 2048, 64 tiles of 256: 28 us, 16 with 64; 29 with 128).
// Others (full) spend twice the time on a slab, which tiles of 128 suffice for (3000 x 3300 x 2000: 48 us, 55 with
// 256, 52 with 64).
inline Cut cut_of(int64_t m, int64_t n, int64_t slabs, bool full) {
    const auto tiles = [&](int64_t s) { return ((m + s - 1) / s) * ((n + s - 1) / s); };
    Cut c{256, 1, (int32_t)slabs};
    if (m <= 32) {                             // 8 waves of 16 columns; 512 workgroups, but a turn of 32 slabs each
        c.side = 16;
        int64_t want = 512 / ((n + 15) / 16 > 0 ? (n + 15) / 16 : 1);
        if (want > slabs / 32) want = slabs / 32;
        if (want > 1) {
            c.per_split = (int32_t)(((slabs + want - 1) / want + 3) / 4 * 4);
            c.splits = (slabs + c.per_split - 1) / c.per_split;
        }
        return c;
    }
    if (full ? tiles(256) < 192 : tiles(256) < 128) c.side = full && tiles(128) >= 256 ? 128 : 64;
    int64_t want = 512 / (tiles(c.side) > 0 ? tiles(c.side) : 1);
    if (c.side == 256 || want < 2) want = 1;
    int64_t per = (slabs + want - 1) / want;
    per = (per + 3) / 4 * 4;
    if (per < 8) per = 8;
    c.splits = slabs > 0 ? (slabs + per - 1) / per : 1;
    if (c.splits > 1) c.per_split = (int32_t)per;
    return c;
}

template <int KA, int KB, bool FULL>
void launch_matmul(const Operand& a, const Operand& b, Result o, const Cut& c, hipStream_t st) {
    if (c.side == 16) {
        o.tiles_n = (uint32_t)((o.n + 15) / 16);
        const dim3 grid((uint32_t)(o.tiles_n * c.splits)), wg(kFewWaves * 64);
        if (o.m <= 16) hipLaunchKernelGGL((k_matmul_few<KA, KB, FULL, 1>), grid, wg, 0, st, a, b, o);
        else hipLaunchKernelGGL((k_matmul_few<KA, KB, FULL, 2>), grid, wg, 0, st, a, b, o);
    } else if (c.side == 256) launch_tiles<Tile256<KA, KB, FULL>>(a, b, o, c.splits, st);
    else if (FULL && c.side == 128) launch_tiles<TileSmall<KA, KB, 4, 4, true>>(a, b, o, c.splits, st);
    else if (((o.m + 63) / 64) * ((o.n + 63) / 64) * c.splits <= kFewWorkgroups)
        launch_tiles<TileSmall<KA, KB, 2, 2, FULL, 4>>(a, b, o, c.splits, st);
    else launch_tiles<TileSmall<KA, KB, 2, 2, FULL>>(a, b, o, c.splits, st);
    if (c.splits > 1) {
        hipLaunchKernelGGL(k_join, grid_of_quads(o.m, o.n), dim3(kThreads), 0, st, o, (int32_t)c.splits);
    }
}

// Which results get sums to binary32's precision (matrix.h, products). What the 8-bit instructions drop is, as a root mean
// square over activations with one column in a hundred 30 (1000) times as large, 5e-5 (9e-5) of the result: far
// below bf16's rounding, 1.7e-3, but a quarter (two fifths) of binary16's, 2.1e-4.
inline bool full_sums(int32_t dtype) { return dtype != ZPQ_BF16; }

template <int KA, int KB>
void launch_matmul(const Operand& a, const Operand& b, const Result& o, const Cut& c, hipStream_t st) {
    if (full_sums(o.dtype)) launch_matmul<KA, KB, true>(a, b, o, c, st);
    else launch_matmul<KA, KB, false>(a, b, o, c, st);
}

}  // namespace

extern "C" {

zpq_status zpq_quant_f8(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld, int32_t kind, int32_t tile,
                        uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, zpq_stream stream) {
    const int64_t xb = dtype_bytes(x_dtype);
    if (xb == 0 || !kind_ok(kind)) return ZPQ_ERR_DTYPE;
    if (rows < 0 || cols < 0 || rows > kMaxElems || cols > kMaxElems || (rows > 0 && cols > kMaxElems / rows)) return ZPQ_ERR_SIZE;
    if (rows > 1 && ld < cols) return ZPQ_ERR_SIZE;
    if (rows > 1 && ld > kMaxElems / rows) return ZPQ_ERR_SIZE;
    if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr)) return ZPQ_ERR_MODE;
    if (rows == 0 || cols == 0) return ZPQ_OK;
    if (!codes && !codes_t) return ZPQ_ERR_MODE;
    if (!x) return ZPQ_ERR_NULL;
    const int64_t kb = blocks_of(cols), kb4 = blocks4_of(cols), rb = blocks_of(rows), rb4 = blocks4_of(rows);
    if ((codes && kb * kBlock > kMaxRow) || (codes_t && rb * kBlock > kMaxRow)) return ZPQ_ERR_SIZE;
    if (kb * rb > kMaxGrid || rows * kb > kMaxGrid * 16) return ZPQ_ERR_SIZE;
    if (!aligned(x, xb) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(codes_t, 16) || !aligned(scales_t, 16))
        return ZPQ_ERR_ALIGN;
    const Extent e[5] = {{x, (uint64_t)((rows - 1) * ld + cols) * xb},
                         {codes, (uint64_t)(rows * kb * kBlock)}, {scales, (uint64_t)((tile ? rb : rows) * kb4)},
                         {codes_t, (uint64_t)(cols * rb * kBlock)}, {scales_t, (uint64_t)((tile ? kb : cols) * rb4)}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(e[i].p, e[i].bytes, e[j].p, e[j].bytes)) return ZPQ_ERR_ALIAS;
    const Quant q{x, rows, cols, ld, codes, scales, codes_t, scales_t, (uint32_t)kb, (uint32_t)kb4, (uint32_t)rb, (uint32_t)rb4};
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (kind == ZPQ_E4M3) launch_quant<ZPQ_E4M3>(q, x_dtype, tile != 0, st);
    else launch_quant<ZPQ_E5M2>(q, x_dtype, tile != 0, st);
    return after_launch();
}

zpq_status zpq_transpose_f8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint8_t* codes_t,
                            uint8_t* scales_t, zpq_stream stream) {
    if (rows < 0 || cols < 0 || rows > kMaxRow || cols > kMaxRow || (rows > 0 && cols > kMaxElems / rows)) return ZPQ_ERR_SIZE;
    if (rows == 0 || cols == 0) return ZPQ_OK;
    if (!codes || !scales || !codes_t || !scales_t) return ZPQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(codes_t, 16) || !aligned(scales_t, 16)) return ZPQ_ERR_ALIGN;
    const int64_t kb = blocks_of(cols), kb4 = blocks4_of(cols), rb = blocks_of(rows), rb4 = blocks4_of(rows);
    if (kb * rb > kMaxGrid) return ZPQ_ERR_SIZE;
    const Extent e[4] = {{codes, (uint64_t)(rows * kb * kBlock)}, {scales, (uint64_t)(rb * kb4)},
                         {codes_t, (uint64_t)(cols * rb * kBlock)}, {scales_t, (uint64_t)(kb * rb4)}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(e[i].p, e[i].bytes, e[j].p, e[j].bytes)) return ZPQ_ERR_ALIAS;
    const Quant q{nullptr, rows, cols, 0, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), codes_t, scales_t,
                  (uint32_t)kb, (uint32_t)kb4, (uint32_t)rb, (uint32_t)rb4};
    hipLaunchKernelGGL(k_transpose, dim3((uint32_t)(kb * rb)), dim3(kThreads), 0, static_cast<hipStream_t>(stream), q);
    return after_launch();
}

zpq_status zpq_dequant_f8(const uint8_t* codes, int32_t kind, const uint8_t* scales, int64_t rows, int64_t cols, int32_t tile,
                          void* y, int32_t y_dtype, int64_t ld, zpq_stream stream) {
    const int64_t yb = dtype_bytes(y_dtype);
    if (yb == 0 || !kind_ok(kind)) return ZPQ_ERR_DTYPE;
    if (rows < 0 || cols < 0 || cols > kMaxRow || rows > kMaxElems || (rows > 0 && cols > kMaxElems / rows)) return ZPQ_ERR_SIZE;
    if (rows > 1 && (ld < cols || ld > kMaxElems / rows)) return ZPQ_ERR_SIZE;
    if (rows == 0 || cols == 0) return ZPQ_OK;
    if (!codes || !scales || !y) return ZPQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(y, yb)) return ZPQ_ERR_ALIGN;
    const int64_t kb = blocks_of(cols), kb4 = blocks4_of(cols), count = rows * kb, per = kThreads / 16 * kEach;
    if (count > kMaxGrid * 16) return ZPQ_ERR_SIZE;
    const Extent e[3] = {{y, (uint64_t)((rows - 1) * ld + cols) * yb}, {codes, (uint64_t)(count * kBlock)},
                         {scales, (uint64_t)((tile ? blocks_of(rows) : rows) * kb4)}};
    if (overlaps(e[0].p, e[0].bytes, e[1].p, e[1].bytes) || overlaps(e[0].p, e[0].bytes, e[2].p, e[2].bytes)) return ZPQ_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid((uint32_t)((count + per - 1) / per)), wg(kThreads);
    const uint32_t shift = tile ? 7 : 0;
#define ZPQ_DEQUANT(K, D) hipLaunchKernelGGL((k_dequant<K, D>), grid, wg, 0, st, codes, scales, cols, (uint32_t)kb, (uint32_t)kb4, count, shift, y, ld)
    if (kind == ZPQ_E4M3) {
        if (y_dtype == ZPQ_F32) ZPQ_DEQUANT(ZPQ_E4M3, ZPQ_F32);
        else if (y_dtype == ZPQ_F16) ZPQ_DEQUANT(ZPQ_E4M3, ZPQ_F16);
        else ZPQ_DEQUANT(ZPQ_E4M3, ZPQ_BF16);
    } else {
        if (y_dtype == ZPQ_F32) ZPQ_DEQUANT(ZPQ_E5M2, ZPQ_F32);
        else if (y_dtype == ZPQ_F16) ZPQ_DEQUANT(ZPQ_E5M2, ZPQ_F16);
        else ZPQ_DEQUANT(ZPQ_E5M2, ZPQ_BF16);
    }
#undef ZPQ_DEQUANT
    return after_launch();
}

static zpq_status matmul_sizes(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0 || m > 0x7FFFFFFF || n > 0x7FFFFFFF || k > kMaxRow) return ZPQ_ERR_SIZE;
    if (m > 0 && (n > kMaxElems / m || k > kMaxElems / m)) return ZPQ_ERR_SIZE;
    if (n > 0 && k > kMaxElems / n) return ZPQ_ERR_SIZE;
    if (((m + 63) / 64) * ((n + 63) / 64) > 0x7FFFFF || n > (1 << 26)) return ZPQ_ERR_SIZE;
    return ZPQ_OK;
}

zpq_status zpq_matmul_f8_bytes(int64_t m, int64_t n, int64_t k, int64_t* bytes) {
    if (!bytes) return ZPQ_ERR_NULL;
    const zpq_status s = matmul_sizes(m, n, k);
    if (s != ZPQ_OK) return s;
    const int64_t a = cut_of(m, n, blocks_of(k), false).splits, b = cut_of(m, n, blocks_of(k), true).splits;
    const int64_t splits = a > b ? a : b;
    *bytes = splits > 1 ? splits * m * n * 4 : 0;
    return ZPQ_OK;
}

zpq_status zpq_matmul_f8(const zpq_f8_operand* a, const zpq_f8_operand* b, int64_t m, int64_t n, int64_t k, void* out,
                         int32_t out_dtype, int64_t ld, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                         zpq_stream stream) {
    const int64_t ob = dtype_bytes(out_dtype);
    if (!a || !b) return ZPQ_ERR_NULL;
    if (ob == 0 || !kind_ok(a->kind) || !kind_ok(b->kind)) return ZPQ_ERR_DTYPE;
    const zpq_status s = matmul_sizes(m, n, k);
    if (s != ZPQ_OK) return s;
    if (m > 1 && (ld < n || ld > kMaxElems / m)) return ZPQ_ERR_SIZE;
    if (m == 0 || n == 0) return ZPQ_OK;
    if (!out || (k > 0 && (!a->codes || !a->scales || !b->codes || !b->scales))) return ZPQ_ERR_NULL;
    const int64_t slabs = blocks_of(k), pitch = slabs * kBlock, kb4 = blocks4_of(k);
    const Cut c = cut_of(m, n, slabs, full_sums(out_dtype));
    const int64_t need = c.splits > 1 ? c.splits * m * n * 4 : 0;
    if (need > 0 && !workspace) return ZPQ_ERR_NULL;
    if (workspace_bytes < need) return ZPQ_ERR_SIZE;
    if (!aligned(a->codes, 16) || !aligned(a->scales, 16) || !aligned(b->codes, 16) || !aligned(b->scales, 16) ||
        !aligned(out, ob) || (need > 0 && !aligned(workspace, 16)))
        return ZPQ_ERR_ALIGN;
    const Extent e[6] = {{out, (uint64_t)((m - 1) * ld + n) * ob}, {workspace, (uint64_t)need},
                         {a->codes, (uint64_t)(m * pitch)}, {a->scales, (uint64_t)((a->tile ? blocks_of(m) : m) * kb4)},
                         {b->codes, (uint64_t)(n * pitch)}, {b->scales, (uint64_t)((b->tile ? blocks_of(n) : n) * kb4)}};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (overlaps(e[i].p, e[i].bytes, e[j].p, e[j].bytes)) return ZPQ_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Result o{out, m, n, ld, out_dtype, accumulate != 0, need > 0 ? static_cast<float*>(workspace) : nullptr, 0, 0,
                   (int32_t)slabs, c.per_split};
    if (k == 0) {
        if (accumulate) return ZPQ_OK;
        hipLaunchKernelGGL(k_empty, grid_of_quads(m, n), dim3(kThreads), 0, st, o);
        return after_launch();
    }
    const Operand oa{a->codes, a->scales, m, (uint32_t)pitch, (uint32_t)kb4, a->tile ? 7u : 0u};
    const Operand ob_{b->codes, b->scales, n, (uint32_t)pitch, (uint32_t)kb4, b->tile ? 7u : 0u};
    if (a->kind == ZPQ_E4M3) {
        if (b->kind == ZPQ_E4M3) launch_matmul<ZPQ_E4M3, ZPQ_E4M3>(oa, ob_, o, c, st);
        else launch_matmul<ZPQ_E4M3, ZPQ_E5M2>(oa, ob_, o, c, st);
    } else {
        if (b->kind == ZPQ_E4M3) launch_matmul<ZPQ_E5M2, ZPQ_E4M3>(oa, ob_, o, c, st);
        else launch_matmul<ZPQ_E5M2, ZPQ_E5M2>(oa, ob_, o, c, st);
    }
    return after_launch();
}

}  // extern "C"
