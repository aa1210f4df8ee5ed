// muon.hip -- orthogonalising matrices by Newton-Schulz products, and the Muon step that does
// so for the momenta of many matrices.  Definitions: zpq.h.
//
// A step of the iteration is three products: A = X X^T, B = b A + c A^2, X' = a X + B X,
// on the side of X that makes A the smaller one.  A and B are symmetric, so of the
// first two only tiles on and under the diagonal are computed, and written twice.  All three
// are of the form D = P Q^T with rows consecutive along the sum (matrix.h), X' with the
// transposed X for Q; so X is kept both ways round.
//
// Types: operands are 16-bit floats (binary16, scaled by kScale: 11 bits, and entries of a matrix of
// unit norm are far from its range's ends), sums binary32, and X itself is kept in
// binary32 beside its 16-bit copies.  That matters: the iteration multiplies small
// singular values by up to 485, and what rounding X to 16 bits puts into directions that
// the matrix does not have grows with them (a matrix of rank 8 comes out 4e-2 off
// with binary16 alone, 3e-1 with bf16); with X in binary32 the errors are, as a root mean square,
// 1.2e-3 (2048 x 2048) to 2.3e-3 (33 x 33) for normal values, 2e-4 to 1.3e-3 for ranks 1 to 8, and
// up to 3.3e-3 where only a few rows or columns differ or are not 0, so that the roundings of A and B
// add up instead of spreading.  A matrix that has only 2 rows would come out 1.2e-2 off.  Matrices with a side up to 32 go another way: all of X's powers commute,
// so the whole iteration is one small matrix P, a polynomial in A, in binary64 on
// one workgroup, and X is read twice, for A and for P X.
#include <math.h>

#include "matrix.h"

namespace {

using namespace zpq_matrix;

constexpr float kScale = 1024.0f;             // of 16-bit operands
constexpr int kCut = 128;                     // side of the elementwise kernels' tiles
constexpr int kGatherRows = 32;               // and of the gathering ones' tiles, 128 wide
constexpr int kMaxSteps = 32;
constexpr int64_t kMaxSide = 1 << 22;         // a row of 16-bit operands is at most 2^23 bytes
constexpr int kFew = 32;                      // sides that go by one small matrix
constexpr int kLong = 256;                    // of the other side, what a workgroup takes then
constexpr int kOneSide = 64, kOneLong = 256;  // matrices that one workgroup works on, in LDS
constexpr int64_t kGroup = 1 << 26;           // elements that are worked on at a time,
constexpr int64_t kGroupBytes = 1 << 30;      // and bytes of workspace: 14 an element, more for small matrices

struct Entry {
    const void* g;                            // input
    void* m;                                  // Muon: momentum
    void* p;                                  // Muon: weights; else the output
    void* copy;
    int64_t ld_g, ld_p;
    float* x32;                               // [rows][cols]
    _Float16 *x16, *t16;                      // [rows][pitch_x], [cols][pitch_t]
    _Float16* other;                          // of the one that X' is a product with, the next step's
    _Float16 *a16, *b16;                      // [small][pitch_a]
    float* pieces;                            // of A's sums that are split: [tile][split][256][256]
    double* part;                             // partial sums of squares
    double* inv;                              // 1 / norm, which binary32 cannot hold for subnormal matrices
    int32_t rows, cols;
    uint32_t pitch_x, pitch_t, pitch_a;       // elements, multiples of 64, zero past the end
    float decay, rate;                        // Muon: weight_decay, scale
    double* gram;                             // a side up to kFew: parts of A, [longs][kFew][kFew]
    float* poly;                              // and P, [kFew][kFew]
    uint32_t parts, longs;                    // parts: tiles of k_gather
    uint32_t start_part, start_cut, start_sym, start_full, start_long, start_large;
};
__host__ __device__ __forceinline__ bool one_workgroup(int64_t rows, int64_t cols) {
    const int64_t side = rows < cols ? rows : cols;
    return side > kFew && side <= kOneSide && rows + cols - side <= kOneLong;
}
__device__ __forceinline__ bool one_workgroup(const Entry& e) { return one_workgroup(e.rows, e.cols); }
__device__ __forceinline__ bool few(const Entry& e) { return (e.rows < e.cols ? e.rows : e.cols) <= kFew; }
constexpr int kFill = 16;
struct Fill { Entry entry[kFill]; };
static_assert(sizeof(Fill) < 3800, "kernel arguments");

__global__ __launch_bounds__(64) void k_fill(Fill f, int32_t first, int32_t count, Entry* entries, uint32_t* cut,
                                             uint32_t* sym, uint32_t* full, uint32_t* along, uint32_t* part, uint32_t* large) {
    const int i = threadIdx.x;
    if (i >= count) return;
    entries[first + i] = f.entry[i];
    cut[first + i] = f.entry[i].start_cut;
    sym[first + i] = f.entry[i].start_sym;
    full[first + i] = f.entry[i].start_full;
    along[first + i] = f.entry[i].start_long;
    part[first + i] = f.entry[i].start_part;
    large[first + i] = f.entry[i].start_large;
}

// What a launch works on: `count` consecutive entries and where their shares of workgroups start.
struct Work {
    const Entry* entries;
    const uint32_t* starts;
    uint32_t count;
};
__device__ __forceinline__ const Entry& entry_of(const Work& w, uint32_t& id) {
    const uint32_t i = find_start(w.starts, w.count, id);
    id -= w.starts[i];
    return w.entries[i];
}

struct Hyper {
    float momentum, lr;
    double grad_scale, max_norm;
    int32_t nesterov;
};

// A norm that is not finite leaves everything as it was.
__device__ __forceinline__ bool stopped(const double* sumsq) { return sumsq != nullptr && !(*sumsq < INFINITY); }

// u = [momentum and] gradient as binary32, and the sum of its squares; a 32 x 128 tile a workgroup, a
// lane 8 consecutive elements of 2 rows (of 8 rows: 35 us instead of 19 for three layers of hidden 250, too few
// workgroups).
template <int GT, bool MUON>
__global__ __launch_bounds__(kThreads) void k_gather(Work w, Hyper h, const double* __restrict__ sumsq) {
    if (MUON && stopped(sumsq)) return;
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const uint32_t across = (uint32_t)(e.cols + kCut - 1) / kCut, t = threadIdx.x;
    const int row = (int)(id / across) * kGatherRows + (t >> 4), col = (int)(id % across) * kCut + (t & 15) * 8;
    const int have = e.cols - col;
    float c = 1.0f;
    if (MUON) {
        double s = h.grad_scale;
        if (sumsq != nullptr) s *= fmin(1.0, h.max_norm / (h.grad_scale * sqrt(*sumsq) + 1e-6));
        c = (float)s;
    }
    double sum = 0;
#pragma unroll
    for (int p = 0; p < kGatherRows; p += 16) {
        if (row + p >= e.rows || have <= 0) continue;
        const int64_t at = (int64_t)(row + p) * e.cols + col, at_g = (int64_t)(row + p) * e.ld_g + col;
        Raw<GT, 8> g;
        if (have >= 8) g.load(e.g, at_g);
        else g.load_some(e.g, at_g, have);
        float u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = g.get(k);
        if constexpr (MUON) {
            Raw<ZPQ_F32, 8> m;
            if (have >= 8) m.load(e.m, at);
            else m.load_some(e.m, at, have);
            float next[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float gc = u[k] * c;
                next[k] = m.get(k) * h.momentum + gc;
                u[k] = h.nesterov ? gc + next[k] * h.momentum : next[k];
            }
            m.set(next);
            if (have >= 8) m.store(e.m, at);
            else m.store_some(e.m, at, have);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fma((double)u[k], (double)u[k], sum);
        Raw<ZPQ_F32, 8> x;
        x.set(u);
        if (have >= 8) x.template store<false>(e.x32, at);
        else x.store_some(e.x32, at, have);
    }
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    if ((t & 63) == 0) part[t >> 6] = sum;
    __syncthreads();
    if (t == 0) e.part[id] = part[0] + part[1] + part[2] + part[3];
}

// 1 / norm of each matrix; 0 for a matrix of zeros, NaN for one that is not finite.
__global__ __launch_bounds__(kThreads) void k_norms(const Entry* __restrict__ entries) {
    const Entry& e = entries[blockIdx.x];
    if (e.parts == 0 || few(e) || one_workgroup(e)) return;     // (no parts: an empty matrix)
    double sum = 0;
    for (uint32_t i = threadIdx.x; i < e.parts; i += kThreads) sum += e.part[i];
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = part[0] + part[1] + part[2] + part[3];
        *e.inv = sum == 0.0 ? 0.0 : sum < INFINITY ? 1.0 / sqrt(sum) : NAN;
    }
}

// The 16-bit copies of X = u / norm, both ways round, zero up to their pitches.
__global__ __launch_bounds__(kThreads) void k_halves(Work w) {
    __shared__ u32x4 turned[kCut * 16];
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const uint32_t across = (uint32_t)(e.cols + kCut - 1) / kCut, t = threadIdx.x, c = t & 15, r = t >> 4;
    const int row0 = (int)(id / across) * kCut, col0 = (int)(id % across) * kCut;
    const int row = row0 + r * 8, col = col0 + c * 8, have = e.cols - col;
    const double inv = *e.inv * kScale;
    Raw<ZPQ_F16, 8> x[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        float v[8] = {};
        if (row + p < e.rows && have > 0) {
            Raw<ZPQ_F32, 8> u;
            const int64_t at = (int64_t)(row + p) * e.cols + col;
            if (have >= 8) u.template load<false>(e.x32, at);
            else u.load_some(e.x32, at, have);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < have ? (float)(u.get(k) * inv) : 0.0f;
        }
        x[p].set(v);
        if (row + p < e.rows && col < (int)e.pitch_x)
            x[p].template store<false>(e.x16, (int64_t)(row + p) * e.pitch_x + col);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int p = 0; p < 8; p += 2) {
            const uint32_t a = (x[p].w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu, b = (x[p + 1].w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
            o[p >> 1] = a | b << 16;
        }
        turned[(c * 8 + k) * 16 + (r ^ c)] = u32x4{o[0], o[1], o[2], o[3]};
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint32_t column = p * 16 + r;
        const u32x4 v = turned[column * 16 + (c ^ (column >> 3))];
        if (col0 + (int)column < e.cols && row0 + (int)c * 8 < (int)e.pitch_t)
            *reinterpret_cast<u32x4*>(e.t16 + (int64_t)(col0 + column) * e.pitch_t + row0 + c * 8) = v;
    }
}

// ---------------------------------------------------------------------------
// A side up to kFew.  Element (i, j), i along that side, is x32[i * step_i + j * step_j].
struct Few {
    int side, length;
    int64_t step_i, step_j;
    __device__ __forceinline__ explicit Few(const Entry& e) {
        const bool wide = e.rows <= e.cols;
        side = wide ? e.rows : e.cols;
        length = wide ? e.cols : e.rows;
        step_i = wide ? e.cols : 1;
        step_j = wide ? 1 : e.cols;
    }
};

// A part of U U^T, over kLong elements of the long side: products of binary32 values are exact.
__global__ __launch_bounds__(kThreads) void k_gram(Work w) {
    __shared__ float x[kFew][kLong + 1];
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const Few f(e);
    const int j0 = (int)id * kLong, t = threadIdx.x;
    for (int i = 0; i < kFew; ++i)
        x[i][t] = i < f.side && j0 + t < f.length ? e.x32[i * f.step_i + (j0 + t) * f.step_j] : 0.0f;
    __syncthreads();
    const int r = (t >> 4) * 2, c = (t & 15) * 2;
    double s[2][2] = {};
    for (int j = 0; j < kLong; ++j) {
        const double a[2] = {x[r][j], x[r + 1][j]}, b[2] = {x[c][j], x[c + 1][j]};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < 2; ++q) s[p][q] = fma(a[p], b[q], s[p][q]);
    }
    double* to = e.gram + (int64_t)id * kFew * kFew;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q) to[(r + p) * kFew + c + q] = s[p][q];
}

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
struct Coeffs {
    float abc[3 * kMaxSteps];
    int32_t steps, g_dtype;
};
typedef double Square[kFew][kFew + 1];

// P and 1 / norm from the parts of U U^T, whose trace is the norm's square: with A = U U^T / norm^2, each step
// Q = a + b A + c A A;  P <- Q P;  A <- Q A Q.
__global__ __launch_bounds__(kThreads) void k_poly(const Entry* __restrict__ entries, Coeffs k) {
    const Entry& e = entries[blockIdx.x];
    if (e.longs == 0) return;
    __shared__ Square A, Q, P, T;
    const int t = threadIdx.x, r = (t >> 4) * 2, c = (t & 15) * 2;
    const auto put = [&](Square& to, const double (&v)[2][2]) {
        to[r][c] = v[0][0];
        to[r][c + 1] = v[0][1];
        to[r + 1][c] = v[1][0];
        to[r + 1][c + 1] = v[1][1];
    };
    const auto product = [&](const Square& a, const Square& b, double (&v)[2][2]) {
        v[0][0] = v[0][1] = v[1][0] = v[1][1] = 0;
        for (int j = 0; j < kFew; ++j) {
            const double a0 = a[r][j], a1 = a[r + 1][j], b0 = b[j][c], b1 = b[j][c + 1];
            v[0][0] = fma(a0, b0, v[0][0]);
            v[0][1] = fma(a0, b1, v[0][1]);
            v[1][0] = fma(a1, b0, v[1][0]);
            v[1][1] = fma(a1, b1, v[1][1]);
        }
    };
    double v[2][2] = {};
    for (uint32_t i = 0; i < e.longs; ++i) {
        const double* g = e.gram + (int64_t)i * kFew * kFew + r * kFew + c;
        v[0][0] += g[0];
        v[0][1] += g[1];
        v[1][0] += g[kFew];
        v[1][1] += g[kFew + 1];
    }
    put(A, v);
    __syncthreads();
    double size = 0;
    for (int i = 0; i < kFew; ++i) size += A[i][i];
    const double by = size == 0.0 ? 0.0 : size < INFINITY ? 1.0 / size : NAN;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q) v[p][q] *= by;
    put(A, v);
    if (t == 0) *e.inv = sqrt(by);
    const double one = r == c ? 1.0 : 0.0, unit[2][2] = {{one, 0.0}, {0.0, one}};
    put(P, unit);
    __syncthreads();
    for (int i = 0; i < k.steps; ++i) {
        product(A, A, v);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                v[p][q] = (double)k.abc[3 * i + 1] * A[r + p][c + q] + (double)k.abc[3 * i + 2] * v[p][q] +
                          (r + p == c + q ? (double)k.abc[3 * i] : 0.0);
        put(Q, v);
        __syncthreads();
        double u[2][2];
        product(Q, P, u);
        product(Q, A, v);
        __syncthreads();
        put(P, u);
        put(T, v);
        __syncthreads();
        product(T, Q, v);
        put(A, v);
        __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q) e.poly[(r + p) * kFew + c + q] = (float)P[r + p][c + q];
}

// ---------------------------------------------------------------------------
// The products.
struct Apply {
    float a, b, c;                             // of this step
    int32_t first, last, odd;
    int32_t out_dtype, copy_dtype;             // of the last step's results
    float lr;
};

__device__ __forceinline__ Operand operand(const _Float16* p, int64_t rows, uint32_t pitch) {
    return Operand{reinterpret_cast<const uint8_t*>(p), nullptr, rows, pitch * 2, 0, 0};
}
// Tile number k of the lower triangle: row i, column j <= i.
__device__ __forceinline__ void triangle(uint32_t k, uint32_t& i, uint32_t& j) {
    i = (uint32_t)((sqrtf(8.0f * (float)k + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > k) --i;
    while ((i + 1) * (i + 2) / 2 <= k) ++i;
    j = k - i * (i + 1) / 2;
}

// A = X X^T (SQUARE false) or B = b A + c A A^T (true): tiles on and under the diagonal.
template <class TILE, bool SQUARE>
__global__ __launch_bounds__(TILE::kThreadsWg, TILE::kWaves) void k_symmetric(Work w, Apply s) {
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::kLds];
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const bool wide = e.rows <= e.cols;
    const int small = wide ? e.rows : e.cols;
    const Operand x = SQUARE ? operand(e.a16, small, e.pitch_a)
                             : wide ? operand(e.x16, small, e.pitch_x) : operand(e.t16, small, e.pitch_t);
    uint32_t i, j;
    triangle(id, i, j);
    const int row0 = (int)i * TILE::BM, col0 = (int)j * TILE::BN;
    TILE t;
    t.run(x, x, row0, col0, 0, (int)(x.pitch / kSlab), shared);
    const int pitch = (int)e.pitch_a;
    _Float16* to = SQUARE ? e.b16 : e.a16;
    t.template finish<true>(shared, [&](uint32_t dr, uint32_t dc) {
        const int r = row0 + (int)dr, c = col0 + (int)dc;
        Raw<ZPQ_F16, 8> a = {};
        if (SQUARE && r < small && c < pitch) a.template load<false>(e.a16, (int64_t)r * pitch + c);
        return a;
    }, [&](uint32_t dr, uint32_t dc, float (&v)[8], Raw<ZPQ_F16, 8> a) {
        const int r = row0 + (int)dr, c = col0 + (int)dc;
        const bool in = r < small && c < pitch;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float x = v[k] * (1.0f / kScale);
            if constexpr (SQUARE) x = fmaf(s.b, a.get(k), s.c * x);
            v[k] = in && c + k < small ? x : 0.0f;
        }
        a.set(v);
        if (in) a.template store<false>(to, (int64_t)r * pitch + c);
    }, [&](uint32_t dc, uint32_t dr, u32x4 h) {   // tiles on the right edge bring the zeros up to the pitch
        const int r = row0 + (int)dr, c = col0 + (int)dc;
        if (i != j && c < small && r < pitch) *reinterpret_cast<u32x4*>(to + (int64_t)c * pitch + r) = h;
    });
}

// A = X X^T with each tile's sum over the long side in `splits` pieces: few large tiles leave part of the chip
// idle (136 of 256 CUs for a side of 4096), small ones cannot feed the matrix cores. 4096 x 16,384: 469 us in tiles of
// 128, 277 + 28 us to join 3 pieces, 274 + 41 with 5.
template <class TILE>
__global__ __launch_bounds__(TILE::kThreadsWg, 2) void k_symmetric_split(Work w, uint32_t tiles, int32_t splits) {
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::kLds];
    const uint32_t split = blockIdx.x / tiles;
    uint32_t id = blockIdx.x - split * tiles;
    const Entry& e = entry_of(w, id);
    const bool wide = e.rows <= e.cols;
    const Operand x = wide ? operand(e.x16, e.rows, e.pitch_x) : operand(e.t16, e.cols, e.pitch_t);
    uint32_t i, j;
    triangle(id, i, j);
    const int slabs = (int)(x.pitch / kSlab), per = (slabs + splits - 1) / splits, first = (int)split * per;
    TILE t;
    t.run(x, x, (int64_t)i * TILE::BM, (int64_t)j * TILE::BN, first, first + per < slabs ? first + per : slabs, shared);
    float* to = e.pieces + ((int64_t)id * splits + split) * (TILE::BM * TILE::BN);
    t.template finish<false>(shared, [](uint32_t, uint32_t) { return 0; }, [&](uint32_t r, uint32_t c, float (&v)[8], int) {
        Raw<ZPQ_F32, 8> x;
        x.set(v);
        x.template store<false>(to, r * TILE::BN + c);
    }, [](uint32_t, uint32_t, u32x4) {});
}

// The pieces added up, in order, into A and its mirror image; a 64 x 64 part of a tile a workgroup.
constexpr int kPart = 64;
template <int SIDE>
__global__ __launch_bounds__(kThreads) void k_symmetric_join(Work w, int32_t splits) {
    __shared__ __attribute__((aligned(16))) _Float16 turned[kPart * kPart];
    constexpr uint32_t along = SIDE / kPart, each = along * along;
    const uint32_t quarter = blockIdx.x % each, t = threadIdx.x;
    uint32_t id = blockIdx.x / each;
    const Entry& e = entry_of(w, id);
    const int small = e.rows <= e.cols ? e.rows : e.cols, pitch = (int)e.pitch_a;
    uint32_t i, j;
    triangle(id, i, j);
    const int in_row = (int)(quarter / along) * kPart, in_col = (int)(quarter % along) * kPart;
    const int row0 = (int)i * SIDE + in_row, col0 = (int)j * SIDE + in_col;
    if (row0 >= pitch || col0 >= pitch) return;                // the same in all lanes
    const float* from = e.pieces + (int64_t)id * splits * (SIDE * SIDE);
    const uint32_t c = t & 7;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t r = p * 32 + (t >> 3);
        float v[8] = {};
        for (int k = 0; k < splits; ++k) {
            Raw<ZPQ_F32, 8> x;
            x.template load<false>(from, (int64_t)k * (SIDE * SIDE) + (in_row + r) * SIDE + in_col + c * 8);
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] += x.get(n);
        }
        const int row = row0 + (int)r, col = col0 + (int)c * 8;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            v[n] = row < small && col + n < small ? v[n] * (1.0f / kScale) : 0.0f;
            turned[(c * 8 + n) * kPart + (((r >> 3) ^ c) << 3) + (r & 7)] = (_Float16)v[n];
        }
        Raw<ZPQ_F16, 8> h;
        h.set(v);
        if (row < small) h.template store<false>(e.a16, (int64_t)row * pitch + col);
    }
    if (i == j) return;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t column = p * 32 + (t >> 3);
        if (col0 + (int)column < small)
            *reinterpret_cast<u32x4*>(e.a16 + (int64_t)(col0 + (int)column) * pitch + row0 + c * 8) =
                *reinterpret_cast<const u32x4*>(&turned[column * kPart + ((c ^ (column >> 3)) << 3)]);
    }
}

template <int DT>
__device__ __forceinline__ void put_row(void* to, int64_t at, const float (&x)[8], int have) {
    Raw<DT, 8> r;
    r.set(x);
    if (have >= 8) r.template store<false>(to, at);
    else r.store_some(to, at, have);
}
__device__ __forceinline__ void put_row(int32_t dtype, void* to, int64_t at, const float (&x)[8], int have) {
    if (dtype == ZPQ_F32) put_row<ZPQ_F32>(to, at, x, have);
    else if (dtype == ZPQ_F16) put_row<ZPQ_F16>(to, at, x, have);
    else put_row<ZPQ_BF16>(to, at, x, have);
}
__device__ __forceinline__ float get_one(int32_t dtype, const void* from, int64_t at) {
    return dtype == ZPQ_F32 ? load1<ZPQ_F32>(from, at) : dtype == ZPQ_F16 ? load1<ZPQ_F16>(from, at) : load1<ZPQ_BF16>(from, at);
}
__device__ __forceinline__ void put_one(int32_t dtype, void* to, int64_t at, float x) {
    if (dtype == ZPQ_F32) store1<ZPQ_F32>(to, at, x);
    else if (dtype == ZPQ_F16) store1<ZPQ_F16>(to, at, x);
    else store1<ZPQ_BF16>(to, at, x);
}
__device__ __forceinline__ void get_row(int32_t dtype, const void* from, int64_t at, float (&x)[8], int have) {
    const auto get = [&](auto r) {
        if (have >= 8) r.template load<false>(from, at);
        else r.load_some(from, at, have);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = r.get(k);
    };
    if (dtype == ZPQ_F32) get(Raw<ZPQ_F32, 8>{});
    else if (dtype == ZPQ_F16) get(Raw<ZPQ_F16, 8>{});
    else get(Raw<ZPQ_BF16, 8>{});
}

// X' = a X + B X in X's own layout; the last step's goes to the output, or into the weights:
// p' = p (1 - lr decay) - lr scale X'.
template <class TILE, bool MUON>
__global__ __launch_bounds__(TILE::kThreadsWg, TILE::kWaves) void k_update(Work w, Apply s, const double* __restrict__ sumsq) {
    __shared__ __attribute__((aligned(16))) uint8_t shared[TILE::kLds];
    if (MUON && stopped(sumsq)) return;
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const bool wide = e.rows <= e.cols;
    const Operand b = operand(e.b16, wide ? e.rows : e.cols, e.pitch_a);
    // the operand that all workgroups read is written into the other buffer
    _Float16 *from = wide ? e.t16 : e.x16, *to = e.other;
    if (s.odd) {
        to = from;
        from = e.other;
    }
    const Operand x = wide ? operand(from, e.cols, e.pitch_t) : operand(from, e.rows, e.pitch_x);
    _Float16 *x16 = wide ? e.x16 : to, *t16 = wide ? to : e.t16;
    const uint32_t down = (uint32_t)(e.rows + TILE::BM - 1) / TILE::BM, across = (uint32_t)(e.cols + TILE::BN - 1) / TILE::BN;
    uint32_t i, j;
    tile_of(id, down * across, down, across, i, j);
    const int row0 = (int)i * TILE::BM, col0 = (int)j * TILE::BN;
    TILE t;
    t.run(wide ? b : x, wide ? x : b, row0, col0, 0, (int)(b.pitch / kSlab), shared);
    const double inv = s.first ? *e.inv : 1.0;
    const float keep = (float)(1.0 - (double)s.lr * e.decay), rate = s.lr * e.rate;
    const auto load = [&](uint32_t dr, uint32_t dc) {              // X
        const int r = row0 + (int)dr, c = col0 + (int)dc, have = e.cols - c;
        Raw<ZPQ_F32, 8> old = {};
        if (r < e.rows && have >= 8) old.template load<false>(e.x32, (int64_t)r * e.cols + c);
        else if (r < e.rows && have > 0) old.load_some(e.x32, (int64_t)r * e.cols + c, have);
        return old;
    };
    const auto sum = [&](int have, float (&v)[8], const Raw<ZPQ_F32, 8>& old) {     // X'
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float o = s.first ? (float)(old.get(k) * inv) : old.get(k);
            v[k] = k < have ? fmaf(v[k], 1.0f / (kScale * kScale), s.a * o) : 0.0f;
        }
    };
    if (s.last) {
        t.template finish<false>(shared, load, [&](uint32_t dr, uint32_t dc, float (&v)[8], const Raw<ZPQ_F32, 8>& old) {
            const int r = row0 + (int)dr, c = col0 + (int)dc, have = e.cols - c;
            if (r >= e.rows || have <= 0) return;
            sum(have, v, old);
            const int64_t at = (int64_t)r * e.ld_p + c;
            if constexpr (MUON) {
                float p[8];
                get_row(s.out_dtype, e.p, at, p, have);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = p[k] * keep - rate * v[k];
                if (s.copy_dtype >= 0) put_row(s.copy_dtype, e.copy, at, v, have);
            }
            put_row(s.out_dtype, e.p, at, v, have);
        }, [](uint32_t, uint32_t, u32x4) {});
        return;
    }
    t.template finish<true>(shared, load, [&](uint32_t dr, uint32_t dc, float (&v)[8], const Raw<ZPQ_F32, 8>& old) {
        const int r = row0 + (int)dr, c = col0 + (int)dc, have = e.cols - c;
        if (r >= e.rows || have <= 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0;
        } else {
            sum(have, v, old);
            Raw<ZPQ_F32, 8> x;
            x.set(v);
            const int64_t at = (int64_t)r * e.cols + c;
            if (have >= 8) x.template store<false>(e.x32, at);
            else x.store_some(e.x32, at, have);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= kScale;
        }
        if (r < e.rows && c < (int)e.pitch_x) {
            Raw<ZPQ_F16, 8> h;
            h.set(v);
            h.template store<false>(x16, (int64_t)r * e.pitch_x + c);
        }
    }, [&](uint32_t dc, uint32_t dr, u32x4 h) {
        const int r = row0 + (int)dr, c = col0 + (int)dc;
        if (c < e.cols && r < (int)e.pitch_t) *reinterpret_cast<u32x4*>(t16 + (int64_t)c * e.pitch_t + r) = h;
    });
}

// The whole iteration of a matrix of up to 64 x 256 on one workgroup, where launches would take far longer
// than the products: the same operands and sums as above, in LDS, X itself in registers.  8 waves;
// X' in tiles of 16 x 16, tile t of 4 down and 16 across is wave t / 8's.  Without a momentum it takes the input itself.
template <bool MUON>
__global__ __launch_bounds__(512) void k_one(const Entry* __restrict__ entries, Coeffs k, Apply s, const double* __restrict__ sumsq) {
    constexpr int PX = kOneLong + 8, PA = kOneSide + 8;        // pitches that spread rows over the banks
    __shared__ __attribute__((aligned(16))) _Float16 x16[kOneSide * PX], t16[kOneLong * PA], a16[kOneSide * PA], b16[kOneSide * PA];
    const Entry& e = entries[blockIdx.x];
    if (!one_workgroup(e)) return;             // an empty matrix neither
    if (MUON && stopped(sumsq)) return;
    const Few f(e);
    const bool wide = e.rows <= e.cols;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const bool deep = f.length > kOneLong / 2;
    float x[8][4];
    const auto row_of = [&](int n) { return ((wave * 8 + n) & 3) * 16 + r; };
    const auto col_of = [&](int n) { return ((wave * 8 + n) >> 2) * 16 + g * 4; };
    const auto keep16 = [&]() {                                // X both ways round, zeros outside
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int i = row_of(n), j = col_of(n);
            f16x4 h;
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = (_Float16)(x[n][q] * kScale);
            *reinterpret_cast<f16x4*>(x16 + i * PX + j) = h;
#pragma unroll
            for (int q = 0; q < 4; ++q) t16[(j + q) * PA + i] = h[q];
        }
    };
    const auto piece = [&](const _Float16* from, int pitch, int row, int step) {
        return *reinterpret_cast<const f16x8*>(from + (row + r) * pitch + step * 32 + g * 8);
    };
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const int i = row_of(n), j = col_of(n);
        if constexpr (MUON) {
            if (wide && i < f.side && j + 4 <= f.length) {
                Raw<ZPQ_F32, 4> u;
                u.load<false>(e.x32, i * f.step_i + j);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[n][q] = u.get(q);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) x[n][q] = i < f.side && j + q < f.length ? e.x32[i * f.step_i + (j + q) * f.step_j] : 0.0f;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = wide ? i * e.ld_g + j + q : (j + q) * e.ld_g + i;
                x[n][q] = i < f.side && j + q < f.length ? get_one(k.g_dtype, e.g, at) : 0.0f;
            }
        }
    }
    double size = 0;
    if constexpr (MUON) {
        for (uint32_t i = 0; i < e.parts; ++i) size += e.part[i];
    } else {
        __shared__ double sums[8];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) size = fma((double)x[n][q], (double)x[n][q], size);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) size += __shfl_xor(size, d);
        if (lane == 0) sums[wave] = size;
        __syncthreads();
        size = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) size += sums[i];
    }
    const double inv = size == 0.0 ? 0.0 : size < INFINITY ? 1.0 / sqrt(size) : NAN;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[n][q] = x[n][q] == 0.0f ? 0.0f : (float)(x[n][q] * inv);
    }
    for (int step = 0; step < k.steps; ++step) {
        const float a = k.abc[3 * step], b = k.abc[3 * step + 1], c = k.abc[3 * step + 2];
        keep16();
        __syncthreads();
        // A and B: tile t of 4 x 4 is wave t / 2's; lane: rows 4 g .. + 3 of column r, symmetric
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int ti = (wave * 2 + n) >> 2, tj = (wave * 2 + n) & 3;
            f32x4 acc = {0, 0, 0, 0};
            const auto add = [&](int d) {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(piece(x16, PX, ti * 16, d), piece(x16, PX, tj * 16, d), acc, 0, 0, 0);
            };
#pragma unroll
            for (int d = 0; d < kOneLong / 64; ++d) add(d);
            if (deep) {
#pragma unroll
                for (int d = kOneLong / 64; d < kOneLong / 32; ++d) add(d);
            }
            f16x4 h;
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = (_Float16)(acc[q] * (1.0f / kScale));
            *reinterpret_cast<f16x4*>(a16 + (tj * 16 + r) * PA + ti * 16 + g * 4) = h;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int ti = (wave * 2 + n) >> 2, tj = (wave * 2 + n) & 3;
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < 2; ++d)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(piece(a16, PA, ti * 16, d), piece(a16, PA, tj * 16, d), acc, 0, 0, 0);
            const int at = (tj * 16 + r) * PA + ti * 16 + g * 4;
            f16x4 h = *reinterpret_cast<const f16x4*>(a16 + at);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = (_Float16)fmaf(b, (float)h[q], c * (acc[q] * (1.0f / kScale)));
            *reinterpret_cast<f16x4*>(b16 + at) = h;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int ti = (wave * 8 + n) & 3, tj = (wave * 8 + n) >> 2;
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < 2; ++d)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(piece(t16, PA, tj * 16, d), piece(b16, PA, ti * 16, d), acc, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) x[n][q] = fmaf(acc[q], 1.0f / (kScale * kScale), a * x[n][q]);
        }
        __syncthreads();                       // before x16 and t16 are written again
    }
    const float keep = (float)(1.0 - (double)s.lr * e.decay), rate = s.lr * e.rate;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const int i = row_of(n), j = col_of(n);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (i >= f.side || j + q >= f.length) continue;
            const int64_t at = wide ? i * e.ld_p + j + q : (j + q) * e.ld_p + i;
            float y = x[n][q];
            if constexpr (MUON) {
                y = get_one(s.out_dtype, e.p, at) * keep - rate * y;
                if (s.copy_dtype >= 0) put_one(s.copy_dtype, e.copy, at, y);
            }
            put_one(s.out_dtype, e.p, at, y);
        }
    }
}

// The result of matrices with a side up to kFew: P X, a lane one place of the long side.
template <bool MUON>
__global__ __launch_bounds__(kThreads) void k_update_few(Work w, Apply s, const double* __restrict__ sumsq) {
    __shared__ float poly[kFew][kFew];
    if (MUON && stopped(sumsq)) return;
    uint32_t id = blockIdx.x;
    const Entry& e = entry_of(w, id);
    const Few f(e);
    for (int i = threadIdx.x; i < kFew * kFew; i += kThreads) (&poly[0][0])[i] = e.poly[i];
    __syncthreads();
    const int j = (int)id * kLong + threadIdx.x;
    if (j >= f.length) return;
    const bool wide = e.rows <= e.cols;
    const double inv = *e.inv;
    float x[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) x[i] = i < f.side ? (float)(e.x32[i * f.step_i + j * f.step_j] * inv) : 0.0f;
    const float keep = (float)(1.0 - (double)s.lr * e.decay), rate = s.lr * e.rate;
    for (int i = 0; i < f.side; ++i) {
        float y = 0;
#pragma unroll
        for (int k = 0; k < kFew; ++k) y = fmaf(poly[i][k], x[k], y);
        const int64_t at = wide ? i * e.ld_p + j : j * e.ld_p + i;
        if constexpr (MUON) {
            y = get_one(s.out_dtype, e.p, at) * keep - rate * y;
            if (s.copy_dtype >= 0) put_one(s.copy_dtype, e.copy, at, y);
        }
        put_one(s.out_dtype, e.p, at, y);
    }
}

// ---------------------------------------------------------------------------
// Host side.
inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
inline int64_t div_up(int64_t n, int64_t by) { return (n + by - 1) / by; }

struct Shape { int64_t rows, cols; };
inline int64_t small_of(Shape s) { return s.rows < s.cols ? s.rows : s.cols; }
inline int64_t cuts_of(Shape s) { return div_up(s.rows, kCut) * div_up(s.cols, kCut); }
inline int64_t parts_of(Shape s) { return div_up(s.rows, kGatherRows) * div_up(s.cols, kCut); }
inline bool few(Shape s) { return small_of(s) <= kFew; }
inline bool tiled(Shape s) { return !few(s) && !one_workgroup(s.rows, s.cols); }
inline int64_t longs_of(Shape s) { return few(s) ? div_up(s.rows < s.cols ? s.cols : s.rows, kLong) : 0; }
inline int64_t triangle_of(Shape s, int64_t side) {
    if (!tiled(s)) return 0;
    const int64_t t = div_up(small_of(s), side);
    return t * (t + 1) / 2;
}
inline int64_t tiles_of(Shape s, int64_t side) { return tiled(s) ? div_up(s.rows, side) * div_up(s.cols, side) : 0; }
inline bool shape_ok(Shape s) { return s.rows >= 0 && s.cols >= 0 && s.rows <= kMaxSide && s.cols <= kMaxSide && s.rows * s.cols <= (1LL << 34); }

// Bytes of a matrix's part of the workspace, and the addresses in it.
inline int64_t place(Shape s, int splits, char* at, Entry* e) {
    const int64_t px = up(s.cols, 64), pt = up(s.rows, 64), pa = up(small_of(s), 64), parts = parts_of(s), longs = longs_of(s);
    const int64_t halves = tiled(s) ? 2 : 0;
    int64_t used = 0;
    const auto take = [&](int64_t bytes) {
        char* p = at ? at + used : nullptr;
        used += up(bytes, 256);
        return p;
    };
    char *x32 = take(s.rows * s.cols * 4), *x16 = take(s.rows * px * halves), *t16 = take(s.cols * pt * halves);
    char* other = take((s.rows <= s.cols ? s.cols * pt : s.rows * px) * halves);
    char *a16 = take(small_of(s) * pa * halves), *b16 = take(small_of(s) * pa * halves);
    char *part = take(parts * 8), *inv = take(16), *gram = take(longs * kFew * kFew * 8), *poly = take(longs ? kFew * kFew * 4 : 0);
    char* pieces = take(splits > 1 ? triangle_of(s, 256) * splits * (256 * 256 * 4) : 0);
    if (e) {
        e->x32 = reinterpret_cast<float*>(x32);
        e->x16 = reinterpret_cast<_Float16*>(x16);
        e->t16 = reinterpret_cast<_Float16*>(t16);
        e->other = reinterpret_cast<_Float16*>(other);
        e->a16 = reinterpret_cast<_Float16*>(a16);
        e->b16 = reinterpret_cast<_Float16*>(b16);
        e->part = reinterpret_cast<double*>(part);
        e->inv = reinterpret_cast<double*>(inv);
        e->rows = (int32_t)s.rows;
        e->cols = (int32_t)s.cols;
        e->pitch_x = (uint32_t)px;
        e->pitch_t = (uint32_t)pt;
        e->pitch_a = (uint32_t)pa;
        e->pieces = reinterpret_cast<float*>(pieces);
        e->parts = (uint32_t)parts;
        e->longs = (uint32_t)longs;
        e->gram = reinterpret_cast<double*>(gram);
        e->poly = reinterpret_cast<float*>(poly);
    }
    return used;
}

// Matrices that are worked on at a time: consecutive ones up to kGroup elements and kGroupBytes (without pieces), one at
// least.
struct Group {
    int64_t first, end, bytes, parts, cuts, sym, large, full, longs, ones;
    int side_sym, side_full, splits;          // of square products (B), of X', pieces of A's sums (tiles of 256)
};
// Tiles of 256 where they keep half of the 256 CUs busy (4096 x 4096: 1603 us, with tiles of 128 for the
// symmetric products 1892), of 128 where they fill them once, else of 64.  For A of matrices of different lengths
// three quarters, measured at one set only: the four matrices of a layer of hidden 2048, 144 large tiles whose longest sums
// decide (177 us, 164 with tiles of 128).
constexpr int64_t kHalfBusy = 128;
template <class COUNT>
inline int side_of(COUNT count, int64_t least) { return count(256) >= least ? 256 : count(128) >= 256 ? 128 : 64; }

// Pieces of A's sums with tiles of 256 (1: none, and tiles of side_sym). Time in slabs of a tile of 256: rounds of the
// 256 CUs by slabs of a piece; writing and reading a piece costs a CU about as much as 10 slabs (measured: 256 KB
// twice, 1.4 us a slab), up to 23 where all CUs do. So pieces, and each further one, have to be better by more than
// that error: without the 0.95, 4096 x 16,384 took 5 pieces (5649 us as a whole, with 3 5563, a twelfth less memory),
// 2043 x 3411 7 (592, without 539), 498 x 3061 8 (244, without 193); what it loses is 6502 x 13,571 (11,317 with 2, without
// 11,584). For matrices of one length only: a layer's four matrices take 163 us without, 190 with. A slab of a 128 tile takes
// 2/3 of it, two at a time on a CU, of a 64 one 2/5, four at a time.
inline int splits_of(int64_t large, int64_t tiles, int side, int64_t longest) {
    const int64_t slabs = div_up(longest, 64);
    const double now = side == 256 ? (double)div_up(tiles, 256) * slabs
                     : side == 128 ? (double)div_up(tiles, 512) * slabs * 2 / 3 : (double)div_up(tiles, 1024) * slabs * 2 / 5;
    double best = now * 0.85;                 // worth its memory
    int splits = 1;
    for (int s = 2; s <= 8 && large > 0; ++s) {
        const double rounds = (double)div_up(large * s, 256), t = rounds * (div_up(slabs, s) + 10);
        if (t < best * 0.95) {
            best = t;
            splits = s;
        }
    }
    return splits;
}

template <class SHAPES>
Group group_at(const SHAPES& shape, int64_t first, int64_t count) {
    Group g{first, first, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    int64_t elems = 0, bytes = 0, longest = 0, shortest = kMaxSide;
    while (g.end < count) {
        const Shape s = shape(g.end);
        const int64_t more = s.rows > 0 && s.cols > 0 ? place(s, 1, nullptr, nullptr) : 0;
        if (elems > 0 && (elems + s.rows * s.cols > kGroup || bytes + more > kGroupBytes)) break;
        elems += s.rows * s.cols;
        bytes += more;
        if (s.rows > 0 && s.cols > 0) {
            g.parts += parts_of(s);
            g.cuts += tiled(s) ? cuts_of(s) : 0;
            if (tiled(s)) {
                const int64_t length = s.rows > s.cols ? s.rows : s.cols;
                longest = length > longest ? length : longest;
                shortest = length < shortest ? length : shortest;
            }
            g.longs += longs_of(s);
            g.ones += one_workgroup(s.rows, s.cols);
        }
        ++g.end;
    }
    const auto sum = [&](auto of, int64_t side) {
        int64_t n = 0;
        for (int64_t i = g.first; i < g.end; ++i) n += shape(i).rows > 0 && shape(i).cols > 0 ? of(shape(i), side) : 0;
        return n;
    };
    g.side_sym = side_of([&](int64_t side) { return sum(triangle_of, side); }, longest == shortest ? kHalfBusy : 192);
    g.side_full = side_of([&](int64_t side) { return sum(tiles_of, side); }, kHalfBusy);
    g.sym = sum(triangle_of, g.side_sym);
    g.large = sum(triangle_of, 256);
    g.splits = longest == shortest ? splits_of(g.large, g.sym, g.side_sym, longest) : 1;
    for (int64_t i = g.first; i < g.end; ++i)
        if (shape(i).rows > 0 && shape(i).cols > 0) g.bytes += place(shape(i), g.splits, nullptr, nullptr);
    g.full = sum(tiles_of, g.side_full);
    return g;
}

// The table: entries, then where each one's workgroups start, for the six kinds of launches.
struct Table {
    Entry* entries;
    uint32_t *cut, *sym, *full, *along, *part, *large;
};
inline Table table_of(void* at, int64_t count) {
    Table t;
    t.entries = static_cast<Entry*>(at);
    t.cut = reinterpret_cast<uint32_t*>(t.entries + count);
    t.sym = t.cut + count;
    t.full = t.sym + count;
    t.along = t.full + count;
    t.part = t.along + count;
    t.large = t.part + count;
    return t;
}
static_assert(sizeof(Entry) + 24 <= ZPQ_MUON_BYTES(1) - ZPQ_MUON_BYTES(0), "ZPQ_MUON_BYTES");

// Fills the table; `entry(i, Entry&)` sets what place() does not.
template <class SHAPES, class ENTRY>
void fill_table(const SHAPES& shape, const ENTRY& entry, int64_t count, void* table, void* workspace, hipStream_t st) {
    const Table t = table_of(table, count);
    for (int64_t first = 0; first < count;) {
        const Group g = group_at(shape, first, count);
        int64_t used = 0;
        uint32_t cut = 0, sym = 0, full = 0, along = 0, part = 0, large = 0;
        for (int64_t i = g.first; i < g.end; i += kFill) {
            Fill f = {};
            const int32_t some = (int32_t)(g.end - i < kFill ? g.end - i : kFill);
            for (int32_t k = 0; k < some; ++k) {
                const Shape s = shape(i + k);
                Entry& e = f.entry[k];
                e.start_cut = cut;
                e.start_sym = sym;
                e.start_full = full;
                e.start_long = along;
                e.start_part = part;
                e.start_large = large;
                if (s.rows == 0 || s.cols == 0) continue;
                used += place(s, g.splits, static_cast<char*>(workspace) + used, &e);
                entry(i + k, e);
                cut += (uint32_t)(tiled(s) ? cuts_of(s) : 0);
                part += (uint32_t)parts_of(s);
                large += (uint32_t)triangle_of(s, 256);
                sym += (uint32_t)triangle_of(s, g.side_sym);
                full += (uint32_t)tiles_of(s, g.side_full);
                along += (uint32_t)longs_of(s);
            }
            hipLaunchKernelGGL(k_fill, dim3(1), dim3(64), 0, st, f, (int32_t)i, some, t.entries, t.cut, t.sym, t.full,
                               t.along, t.part, t.large);
        }
        first = g.end;
    }
}

template <bool SQUARE>
void launch_symmetric(const Work& w, const Apply& s, const Group& g, hipStream_t st) {
    const dim3 grid((uint32_t)g.sym);
    if (g.side_sym == 256) hipLaunchKernelGGL((k_symmetric<Tile256<kF16, kF16>, SQUARE>), grid, dim3(512), 0, st, w, s);
    else if (g.side_sym == 128) hipLaunchKernelGGL((k_symmetric<TileSmall<kF16, kF16, 4, 4>, SQUARE>), grid, dim3(256), 0, st, w, s);
    else if (g.sym <= kFewWorkgroups)
        hipLaunchKernelGGL((k_symmetric<TileSmall<kF16, kF16, 2, 2, false, 4>, SQUARE>), grid, dim3(256), 0, st, w, s);
    else hipLaunchKernelGGL((k_symmetric<TileSmall<kF16, kF16, 2, 2>, SQUARE>), grid, dim3(256), 0, st, w, s);
}

template <bool MUON>
void launch_group(const Table& t, const Group& g, int32_t g_dtype, const Hyper& h, Apply s, const float* coeffs, int32_t steps,
                  const double* sumsq, hipStream_t st) {
    if (g.parts == 0) return;
    const Entry* entries = t.entries + g.first;
    const uint32_t count = (uint32_t)(g.end - g.first);
    const Work cut{entries, t.cut + g.first, count}, sym{entries, t.sym + g.first, count}, full{entries, t.full + g.first, count};
    const Work part{entries, t.part + g.first, count};
    const dim3 cuts((uint32_t)g.cuts), parts((uint32_t)g.parts), wg(kThreads);
    if (!MUON && g.ones > 0) {                 // of one shape: all of them
    } else if (g_dtype == ZPQ_F32) hipLaunchKernelGGL((k_gather<ZPQ_F32, MUON>), parts, wg, 0, st, part, h, sumsq);
    else if (g_dtype == ZPQ_F16) hipLaunchKernelGGL((k_gather<ZPQ_F16, MUON>), parts, wg, 0, st, part, h, sumsq);
    else hipLaunchKernelGGL((k_gather<ZPQ_BF16, MUON>), parts, wg, 0, st, part, h, sumsq);
    Coeffs k;
    for (int32_t i = 0; i < 3 * steps; ++i) k.abc[i] = coeffs[i];
    k.steps = steps;
    k.g_dtype = g_dtype;
    if (g.longs > 0) {
        const Work along{entries, t.along + g.first, count};
        const dim3 longs((uint32_t)g.longs);
        hipLaunchKernelGGL(k_gram, longs, wg, 0, st, along);
        hipLaunchKernelGGL(k_poly, dim3(count), wg, 0, st, entries, k);
        hipLaunchKernelGGL((k_update_few<MUON>), longs, wg, 0, st, along, s, sumsq);
    }
    if (g.ones > 0) hipLaunchKernelGGL((k_one<MUON>), dim3(count), dim3(512), 0, st, entries, k, s, sumsq);
    if (g.full == 0) return;
    hipLaunchKernelGGL(k_norms, dim3(count), wg, 0, st, entries);
    hipLaunchKernelGGL(k_halves, cuts, wg, 0, st, cut);
    for (int32_t i = 0; i < steps; ++i) {
        s.a = coeffs[3 * i];
        s.b = coeffs[3 * i + 1];
        s.c = coeffs[3 * i + 2];
        s.first = i == 0;
        s.last = i == steps - 1;
        s.odd = i & 1;
        if (g.splits > 1) {
            const Work large{entries, t.large + g.first, count};
            hipLaunchKernelGGL((k_symmetric_split<Tile256<kF16, kF16>>), dim3((uint32_t)(g.large * g.splits)), dim3(512), 0, st, large,
                               (uint32_t)g.large, g.splits);
            hipLaunchKernelGGL((k_symmetric_join<256>), dim3((uint32_t)(g.large * 16)), wg, 0, st, large, g.splits);
        } else {
            launch_symmetric<false>(sym, s, g, st);
        }
        if (g.large >= kHalfBusy)
            hipLaunchKernelGGL((k_symmetric<Tile256<kF16, kF16>, true>), dim3((uint32_t)g.large), dim3(512), 0, st,
                               Work{entries, t.large + g.first, count}, s);
        else launch_symmetric<true>(sym, s, g, st);
        const dim3 grid((uint32_t)g.full);
        if (g.side_full == 256) hipLaunchKernelGGL((k_update<Tile256<kF16, kF16>, MUON>), grid, dim3(512), 0, st, full, s, sumsq);
        else if (g.side_full == 128) hipLaunchKernelGGL((k_update<TileSmall<kF16, kF16, 4, 4>, MUON>), grid, dim3(256), 0, st, full, s, sumsq);
        else if (g.full <= kFewWorkgroups)
            hipLaunchKernelGGL((k_update<TileSmall<kF16, kF16, 2, 2, false, 4>, MUON>), grid, dim3(256), 0, st, full, s, sumsq);
        else hipLaunchKernelGGL((k_update<TileSmall<kF16, kF16, 2, 2>, MUON>), grid, dim3(256), 0, st, full, s, sumsq);
    }
}

template <class SHAPES>
int64_t workspace_of(const SHAPES& shape, int64_t count) {
    int64_t most = 0;
    for (int64_t first = 0; first < count;) {
        const Group g = group_at(shape, first, count);
        most = g.bytes > most ? g.bytes : most;
        first = g.end;
    }
    return most;
}

// Steps between 1 and kMaxSteps, finite numbers.
inline bool coeffs_ok(const double* coeffs, int32_t steps) {
    if (steps < 1 || steps > kMaxSteps) return false;
    for (int32_t i = 0; i < 3 * steps; ++i)
        if (!(fabs(coeffs[i]) <= 64.0)) return false;
    return true;
}

inline bool count_ok(int64_t count) { return count >= 0 && count <= (1 << 20); }

}  // namespace

extern "C" {

zpq_status zpq_orthogonalize_bytes(int64_t count, int64_t rows, int64_t cols, int64_t* bytes) {
    if (!bytes) return ZPQ_ERR_NULL;
    const Shape s{rows, cols};
    if (!count_ok(count) || !shape_ok(s) || (rows > 0 && cols > 0 && count > kMaxElems / (rows * cols))) return ZPQ_ERR_SIZE;
    *bytes = rows == 0 || cols == 0 || count == 0 ? 0 : up(ZPQ_MUON_BYTES(count), 256) + workspace_of([&](int64_t) { return s; }, count);
    return ZPQ_OK;
}

zpq_status zpq_orthogonalize(const void* x, int32_t x_dtype, int64_t count, int64_t rows, int64_t cols, int64_t ld_x,
                             int64_t stride_x, const double* coeffs, int32_t steps, void* out, int32_t out_dtype, int64_t ld_out,
                             int64_t stride_out, void* workspace, int64_t workspace_bytes, zpq_stream stream) {
    const int64_t xb = dtype_bytes(x_dtype), ob = dtype_bytes(out_dtype);
    if (xb == 0 || (out_dtype != ZPQ_F16 && out_dtype != ZPQ_BF16)) return ZPQ_ERR_DTYPE;
    if (!coeffs) return ZPQ_ERR_NULL;
    if (!coeffs_ok(coeffs, steps)) return ZPQ_ERR_ARG;
    int64_t need = 0;
    const zpq_status s = zpq_orthogonalize_bytes(count, rows, cols, &need);
    if (s != ZPQ_OK) return s;
    if (count == 0 || rows == 0 || cols == 0) return ZPQ_OK;
    if (rows > 1 && (ld_x < cols || ld_out < cols || ld_x > kMaxElems / rows || ld_out > kMaxElems / rows)) return ZPQ_ERR_SIZE;
    const int64_t span_x = (rows - 1) * ld_x + cols, span_out = (rows - 1) * ld_out + cols;
    if (count > 1 && (stride_x < span_x || stride_out < span_out || stride_x > kMaxElems / count || stride_out > kMaxElems / count))
        return ZPQ_ERR_SIZE;
    if (!x || !out || !workspace) return ZPQ_ERR_NULL;
    if (workspace_bytes < need) return ZPQ_ERR_SIZE;
    if (!aligned(x, xb) || !aligned(out, ob) || !aligned(workspace, 256)) return ZPQ_ERR_ALIGN;
    const uint64_t nx = (uint64_t)((count - 1) * stride_x + span_x) * xb, no = (uint64_t)((count - 1) * stride_out + span_out) * ob;
    if (overlaps(x, nx, out, no) || overlaps(x, nx, workspace, (uint64_t)need) || overlaps(out, no, workspace, (uint64_t)need))
        return ZPQ_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Shape one{rows, cols};
    const auto shape = [&](int64_t) { return one; };
    char* matrices = static_cast<char*>(workspace) + up(ZPQ_MUON_BYTES(count), 256);
    fill_table(shape, [&](int64_t i, Entry& e) {
        e.g = static_cast<const char*>(x) + i * stride_x * xb;
        e.p = static_cast<char*>(out) + i * stride_out * ob;
        e.ld_g = rows > 1 ? ld_x : cols;
        e.ld_p = rows > 1 ? ld_out : cols;
    }, count, workspace, matrices, st);
    const Table t = table_of(workspace, count);
    float c[3 * kMaxSteps];
    for (int32_t i = 0; i < 3 * steps; ++i) c[i] = (float)coeffs[i];
    for (int64_t first = 0; first < count;) {
        const Group g = group_at(shape, first, count);
        launch_group<false>(t, g, x_dtype, Hyper{}, Apply{0, 0, 0, 0, 0, 0, out_dtype, -1, 0.0f}, c, steps, nullptr, st);
        first = g.end;
    }
    return after_launch();
}

static zpq_status muon_shapes(const zpq_muon_matrix* matrices, int32_t count) {
    if (!count_ok(count)) return ZPQ_ERR_ARG;
    if (count > 0 && !matrices) return ZPQ_ERR_NULL;
    int64_t elems = 0;
    for (int32_t i = 0; i < count; ++i)
        if (!shape_ok(Shape{matrices[i].rows, matrices[i].cols}) || (elems += matrices[i].rows * matrices[i].cols) > kMaxElems)
            return ZPQ_ERR_SIZE;
    return ZPQ_OK;
}

zpq_status zpq_muon_plan_bytes(const zpq_muon_matrix* matrices, int32_t count, int64_t* bytes) {
    if (!bytes) return ZPQ_ERR_NULL;
    const zpq_status s = muon_shapes(matrices, count);
    if (s != ZPQ_OK) return s;
    *bytes = up(ZPQ_MUON_BYTES(count), 256) + workspace_of([&](int64_t i) { return Shape{matrices[i].rows, matrices[i].cols}; }, count);
    return ZPQ_OK;
}

zpq_status zpq_muon_plan_make(const zpq_muon_matrix* matrices, int32_t count, int32_t p_dtype, int32_t g_dtype, int32_t copy_dtype,
                              void* memory, int64_t memory_bytes, zpq_muon_plan* plan, zpq_stream stream) {
    const int64_t pb = dtype_bytes(p_dtype), gb = dtype_bytes(g_dtype);
    if (pb == 0 || gb == 0) return ZPQ_ERR_DTYPE;
    if (copy_dtype != -1 && copy_dtype != ZPQ_F16 && copy_dtype != ZPQ_BF16) return ZPQ_ERR_DTYPE;
    if (copy_dtype != -1 && p_dtype != ZPQ_F32) return ZPQ_ERR_MODE;
    if (!plan) return ZPQ_ERR_NULL;
    int64_t need = 0;
    const zpq_status s = zpq_muon_plan_bytes(matrices, count, &need);
    if (s != ZPQ_OK) return s;
    if (count > 0 && !memory) return ZPQ_ERR_NULL;
    if (memory_bytes < need) return ZPQ_ERR_SIZE;
    if (count > 0 && !aligned(memory, 256)) return ZPQ_ERR_ALIGN;
    for (int32_t i = 0; i < count; ++i) {
        const zpq_muon_matrix& t = matrices[i];
        if (!(t.weight_decay >= 0.0 && t.weight_decay < INFINITY) || !(t.scale >= 0.0 && t.scale < INFINITY)) return ZPQ_ERR_ARG;
        const int64_t n = t.rows * t.cols;
        if (n == 0) continue;
        if ((copy_dtype == -1) != (t.copy == nullptr)) return ZPQ_ERR_MODE;
        if (!t.p || !t.g || !t.m) return ZPQ_ERR_NULL;
        if (!aligned(t.p, pb) || !aligned(t.g, gb) || !aligned(t.m, 4) || !aligned(t.copy, 2)) return ZPQ_ERR_ALIGN;
        const void* at[5] = {t.p, t.g, t.m, t.copy, memory};
        const uint64_t size[5] = {(uint64_t)(n * pb), (uint64_t)(n * gb), (uint64_t)n * 4, (uint64_t)n * 2, (uint64_t)need};
        for (int a = 0; a < 5; ++a)
            for (int b = a + 1; b < 5; ++b)
                if (overlaps(at[a], size[a], at[b], size[b])) return ZPQ_ERR_ALIAS;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    fill_table([&](int64_t i) { return Shape{matrices[i].rows, matrices[i].cols}; }, [&](int64_t i, Entry& e) {
        const zpq_muon_matrix& t = matrices[i];
        e.g = t.g;
        e.m = t.m;
        e.p = t.p;
        e.copy = t.copy;
        e.ld_g = e.ld_p = t.cols;
        e.decay = (float)t.weight_decay;
        e.rate = (float)t.scale;
    }, count, memory, static_cast<char*>(memory) + up(ZPQ_MUON_BYTES(count), 256), st);
    *plan = zpq_muon_plan{memory, matrices, count, p_dtype, g_dtype, copy_dtype};
    return count > 0 ? after_launch() : ZPQ_OK;
}

zpq_status zpq_muon_step(const zpq_muon_plan* plan, const zpq_muon_hyper* hyper, const double* sumsq, zpq_stream stream) {
    if (!plan || !hyper) return ZPQ_ERR_NULL;
    if (plan->count < 0 || (plan->count > 0 && (!plan->memory || !plan->matrices)) || dtype_bytes(plan->p_dtype) == 0 ||
        dtype_bytes(plan->g_dtype) == 0)
        return ZPQ_ERR_ARG;
    if (!hyper->coeffs) return ZPQ_ERR_NULL;
    if (!(hyper->lr >= 0.0 && hyper->lr < INFINITY) || !(hyper->momentum >= 0.0 && hyper->momentum < 1.0) ||
        !(hyper->grad_scale > 0.0 && hyper->grad_scale < INFINITY) || !(hyper->max_norm > 0.0) || !coeffs_ok(hyper->coeffs, hyper->steps))
        return ZPQ_ERR_ARG;
    if (!sumsq && hyper->max_norm != INFINITY) return ZPQ_ERR_ARG;
    if (sumsq && !aligned(sumsq, 8)) return ZPQ_ERR_ALIGN;
    const auto shape = [&](int64_t i) { return Shape{plan->matrices[i].rows, plan->matrices[i].cols}; };
    const Table t = table_of(plan->memory, plan->count);
    const Hyper h{(float)hyper->momentum, (float)hyper->lr, hyper->grad_scale, hyper->max_norm, hyper->nesterov != 0};
    const Apply a{0, 0, 0, 0, 0, 0, plan->p_dtype, plan->copy_dtype, (float)hyper->lr};
    float c[3 * kMaxSteps];
    for (int32_t i = 0; i < 3 * hyper->steps; ++i) c[i] = (float)hyper->coeffs[i];
    hipStream_t st = static_cast<hipStream_t>(stream);
    for (int64_t first = 0; first < plan->count;) {
        const Group g = group_at(shape, first, plan->count);
        launch_group<true>(t, g, plan->g_dtype, h, a, c, hyper->steps, sumsq, st);
        first = g.end;
    }
    return plan->count > 0 ? after_launch() : ZPQ_OK;
}

}  // extern "C"
