// embedding.hip -- embedding lookup with scaling, from a float table or from
// qwZ's gathered INT8 blocks, and the embedding's gradient by sorted tokens.
//
// A row is cut into pieces of E elements, one a lane: 8, or 4 where a side is
// fp32, so that no access is wider than 16 bytes.  The last piece of a row whose
// length is no multiple of E is moved back so that it ends with the row (it
// reads, and in the lookup writes, some elements twice).  Rows shorter than E are
// one piece, handled element by element.
#include "step.h"

namespace {

using namespace zpq_step;

template <int A, int B>
constexpr int piece_elems() { return A == ZPQ_F32 || B == ZPQ_F32 ? 4 : 8; }

// n / d for n < 2^31 by a multiplication: with m = ceil(2^(31+s) / d) and 2^s >= d,
// n * m / 2^(31+s) exceeds n / d by less than (n / 2^31) / d < 1 / d, too little to
// reach the next integer.
struct Divisor {
    uint32_t d, m, s;
};
inline Divisor divisor(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return Divisor{d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, Divisor d) {
    return (uint32_t)(((uint64_t)n * d.m) >> d.s);
}

__device__ __forceinline__ int64_t load_id(const void* ids, int32_t id_bytes, int64_t t) {
    return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t]
                         : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// ---------------------------------------------------------------------------
// Lookup.  Number L of the grid's lanes is piece L % pieces of token L / pieces.
struct LookupArgs {
    const void* table;
    const float* scales;
    const void* ids;
    void* out;
    int64_t tokens, rows, dim, ld_table, first, ld_out;
    float scale;
    int32_t id_bytes, log_block;
    uint32_t lanes;                           // tokens of this launch * pieces, < 2^31
    Divisor pieces;
};

// Two pieces a lane: the way from id to row to store takes about 3 us, so the waves
// in flight have to carry more than one access each (16,384 x 8192: INT8 to bf16 55 us
// with one, 49 with two, 49 with four; fp32 to bf16 118, 95, 88; fp32 155, 130, 121; but
// bf16 54, 60, 64).  One number for all types, INT8's; 4-byte ids take the same times.
constexpr int kLookupPieces = 2;
template <int TT, int OT>
__global__ __launch_bounds__(kThreads) void k_lookup(LookupArgs a) {
    constexpr int E = piece_elems<TT, OT>(), U = kLookupPieces;
    uint32_t lane[U], token[U];
    int64_t row[U];
    int32_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        lane[u] = (blockIdx.x * U + u) * kThreads + threadIdx.x;
        token[u] = quotient(lane[u], a.pieces);
        col[u] = (int32_t)(lane[u] - token[u] * a.pieces.d) * E;
        row[u] = lane[u] < a.lanes ? load_id(a.ids, a.id_bytes, token[u])
                                  : (int64_t)((uint64_t)a.first - 1);
    }
    if (a.dim < E) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (lane[u] >= a.lanes) continue;
            const uint64_t r = (uint64_t)row[u] - (uint64_t)a.first;
            const bool there = r < (uint64_t)a.rows;
            for (int i = 0; i < (int)a.dim; ++i) {
                float x = 0.0f;
                if (there) {
                    x = load1<TT>(a.table, (int64_t)r * a.ld_table + i);
                    if constexpr (TT == kI8) x *= a.scales[((int64_t)r * a.dim + i) >> a.log_block];
                    x *= a.scale;
                }
                store1<OT>(a.out, token[u] * a.ld_out + i, x);
            }
        }
        return;
    }
    Raw<TT, E> in[U];
    float s0[U], s1[U];
    int32_t left[U];                          // elements of the piece that s0 scales
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (col[u] > a.dim - E) col[u] = (int32_t)a.dim - E;
        const uint64_t r = (uint64_t)row[u] - (uint64_t)a.first;
        const bool there = r < (uint64_t)a.rows;
#pragma unroll
        for (int i = 0; i < Raw<TT, E>::WORDS; ++i) in[u].w[i] = 0;
        s0[u] = s1[u] = 1.0f;
        left[u] = E;
        if (there) {
            const int64_t e = (int64_t)r * a.ld_table + col[u];
            in[u].template load<false>(a.table, e);
            if constexpr (TT == kI8) {
                s0[u] = a.scales[e >> a.log_block];
                left[u] = (1 << a.log_block) - (int32_t)(e & ((1 << a.log_block) - 1));
                s1[u] = left[u] < E ? a.scales[(e >> a.log_block) + 1] : s0[u];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (lane[u] >= a.lanes) continue;
        const bool there = (uint64_t)row[u] - (uint64_t)a.first < (uint64_t)a.rows;
        float x[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            x[i] = in[u].get(i);
            if constexpr (TT == kI8) x[i] *= i < left[u] ? s0[u] : s1[u];
            x[i] = there ? x[i] * a.scale : 0.0f;
        }
        Raw<OT, E> o;
        o.set(x);
        o.store(a.out, token[u] * a.ld_out + col[u]);
    }
}

// ---------------------------------------------------------------------------
// Sorting the tokens by row.  A token is the 64-bit number row * 2^32 + position
// (row = `rows` for what does not count).  All are different, so any correct sort
// is the stable one.
struct Ids {
    const void* ids;
    int64_t first, padding, rows;
    int32_t id_bytes;
    uint32_t tokens;
};
__device__ __forceinline__ uint32_t key_of(const Ids& a, uint32_t t) {
    const int64_t id = load_id(a.ids, a.id_bytes, t);
    const uint64_t r = (uint64_t)id - (uint64_t)a.first;
    return r < (uint64_t)a.rows && id != a.padding ? (uint32_t)r : (uint32_t)a.rows;
}

// A token's place in a tile is the number of the tile's tokens that come before it,
// counted by comparing it with all of them.  A workgroup places 64 tokens, one a
// lane; its waves share the tile's others, 64 at a time through LDS (a broadcast read
// gives 4, and each is one compare and one add with carry for 64 tokens).  Up to
// kRankTokens there is one tile and this is the whole sort; where rows are few as well,
// further workgroups count the same way what comes before each row: its first place.
// 300 tokens 3.8 us; of 4000 the whole gradient takes 21.6 us this way, with two tiles or
// more and a merge 22.5, of 6000 26.0 and 24.4.
constexpr uint32_t kRankTokens = 4096;
constexpr int kRankWaves = 16;
__global__ __launch_bounds__(64 * kRankWaves) void k_rank(Ids a, uint32_t tile, uint64_t* __restrict__ out,
                                                          uint32_t* __restrict__ starts) {
    __shared__ __align__(16) uint32_t keys[kRankWaves][64];
    __shared__ uint32_t counts[kRankWaves][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t blocks = (a.tokens + 63) / 64;
    const bool row_block = blockIdx.x >= blocks;
    const uint32_t own = row_block ? 0xFFFFFFFFu : blockIdx.x;
    const uint32_t t = (row_block ? blockIdx.x - blocks : blockIdx.x) * 64 + lane;     // token or row
    const uint32_t key = row_block ? t : t < a.tokens ? key_of(a, t) : 0xFFFFFFFEu;
    const uint32_t base = row_block ? 0 : blockIdx.x * 64 / tile * tile;                // of the tile
    const uint32_t first = base / 64, last = min(blocks, (base + tile) / 64);           // its blocks
    uint32_t before = 0;
    auto key_at = [&](uint32_t b) {
        const uint32_t j = b * 64 + lane;
        return b < last && j < a.tokens ? key_of(a, j) : 0xFFFFFFFFu;
    };
    uint32_t next = key_at(first + wave);
    for (uint32_t b = first + wave; b < last; b += kRankWaves) {
        __builtin_amdgcn_wave_barrier();
        keys[wave][lane] = next;
        next = key_at(b + kRankWaves);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const u32x4* other = reinterpret_cast<const u32x4*>(keys[wave]);
        if (b != own) {
            // equal rows of earlier tokens come before, those of later ones do not
            const uint32_t below = !row_block && b < own ? key + 1 : key;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const u32x4 k = other[i];
                before += (k.x < below) + (k.y < below) + (k.z < below) + (k.w < below);
            }
        } else {
#pragma unroll 8
            for (int i = 0; i < 64; ++i) before += keys[wave][i] < (i < (int)lane ? key + 1 : key);
        }
    }
    counts[wave][lane] = before;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < kRankWaves; ++w) before += counts[w][lane];
        if (!row_block && t < a.tokens) out[base + before] = (uint64_t)key << 32 | t;
        if (row_block && t <= a.rows) starts[t] = before;
    }
}

// Up to kMergeTokens: sorted tiles (runs of 2^log) are merged at once by places: a token's
// is its place in its own run plus, for each other run, how many there are smaller.
// kRuns lanes search for one token, a run each.  16,384 tokens: ranks and merge 11.5 us,
// radix sort 21; with the gradient of 24,000 x 1024 44.4 us, by radix sort 47.1, even at
// 32,768.
constexpr uint32_t kRuns = 16, kMergeTokens = 24576;
inline uint32_t run_log(uint32_t tokens) { return tokens <= kRuns * 1024 ? 10 : 11; }
__global__ __launch_bounds__(kThreads) void k_merge(const uint64_t* __restrict__ in, uint32_t tokens,
                                                    uint32_t log, uint64_t* __restrict__ out) {
    const uint32_t lane = blockIdx.x * kThreads + threadIdx.x, t = lane / kRuns, r = lane % kRuns;
    if (t >= tokens) return;                  // whole groups of kRuns lanes
    const uint64_t x = in[t];
    uint32_t at = r << log, n = at >= tokens ? 0 : min(tokens - at, 1u << log), less = 0;
    if (r == t >> log) { less = t - at; n = 0; }
    for (uint32_t left = 1u << log; left > 0; left >>= 1)          // n halves at least as fast
        if (n > 0) {
            const uint32_t half = n >> 1;
            if (in[at + half] < x) { at += half + 1; less += half + 1; n -= half + 1; }
            else n = half;
        }
#pragma unroll
    for (uint32_t d = 1; d < kRuns; d <<= 1) less += __shfl_xor(less, d);
    if (r == 0) out[less] = x;
}

// More tokens: a radix sort from the lowest digit, `bits` (at most 9) a pass, stable by
// construction.  k_digit_counts counts each tile's digits; k_digit_place gives every
// token its place: tokens with smaller digits, the same digit in earlier tiles, in
// earlier waves of the tile, and earlier in its wave (found by ballots).  131,072
// tokens 4.9 and 8.8 us a pass: latency, of the launches and of a few dependent accesses.
constexpr int kMaxDigits = 512, kSortThreads = 512, kSortTile = 4 * kSortThreads;
constexpr int kSortWaves = kSortThreads / 64;
static_assert(kSortThreads == kMaxDigits, "a digit a thread");
// Up to this many tiles k_digit_place sums their counts by itself; more take k_digit_scan, a
// third launch a pass.  The gradient of 65,536 x 8 into 50,000 rows (32 tiles) takes 32.6 us,
// with the scan 35.3; of 131,072 (64 tiles) 39.2 and 39.9; of 200,000 48.3 and 46.0, of
// 1,048,576 109 and 88.
constexpr uint32_t kDirectTiles = 64;

struct Pass {
    int32_t shift, bits;
    uint32_t tiles;
};

template <bool FIRST>
__device__ __forceinline__ uint64_t sort_item(const Ids& a, const uint64_t* __restrict__ in, uint32_t t) {
    if constexpr (FIRST) return (uint64_t)key_of(a, t) << 32 | t;
    else return in[t];
}

// counts[tile][digit]
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_digit_counts(Ids a, const uint64_t* __restrict__ in,
                                                               Pass p, uint32_t* __restrict__ counts) {
    __shared__ uint32_t n[kMaxDigits];
    n[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortTile / kSortThreads; ++k) {
        const uint32_t t = blockIdx.x * kSortTile + k * kSortThreads + threadIdx.x;
        if (t < a.tokens)
            atomicAdd(&n[(uint32_t)(sort_item<FIRST>(a, in, t) >> (32 + p.shift)) & ((1u << p.bits) - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < (1u << p.bits)) counts[(uint64_t)blockIdx.x << p.bits | threadIdx.x] = n[threadIdx.x];
}

// Many tiles: each digit's counts to the number in earlier tiles, in place, and
// its total; one wave a digit.
__global__ __launch_bounds__(64) void k_digit_scan(Pass p, uint32_t* __restrict__ counts,
                                                   uint32_t* __restrict__ totals) {
    uint32_t* row = counts + blockIdx.x;
    uint32_t sum = 0;
    for (uint32_t b = 0; b < p.tiles; b += 64) {
        const uint32_t i = b + threadIdx.x;
        const uint32_t x = i < p.tiles ? row[(uint64_t)i << p.bits] : 0;
        uint32_t s = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t y = __shfl_up(s, d);
            if ((int)threadIdx.x >= d) s += y;
        }
        if (i < p.tiles) row[(uint64_t)i << p.bits] = sum + s - x;
        sum += __shfl(s, 63);
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = sum;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_digit_place(Ids a, const uint64_t* __restrict__ in,
                                                              Pass p, const uint32_t* __restrict__ counts,
                                                              const uint32_t* __restrict__ totals,
                                                              uint64_t* __restrict__ out) {
    __shared__ uint32_t seen[kSortWaves][kMaxDigits];      // of each wave, then before each wave
    __shared__ uint32_t waves[kSortWaves];                 // totals of 64 digits each
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    constexpr int kEach = kSortTile / kSortThreads;
    uint64_t x[kEach];
    uint32_t digit[kEach], rank[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {         // wave w holds the tile's tokens [256 w, 256 w + 256)
        const uint32_t t = blockIdx.x * kSortTile + (wave * kEach + k) * 64 + lane;
        x[k] = t < a.tokens ? sort_item<FIRST>(a, in, t) : ~0ull;
    }
    for (uint32_t i = lane; i < kMaxDigits; i += 64) seen[wave][i] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // the digit's share of earlier tiles, and its total
    uint32_t total = 0, earlier = 0;
    if (threadIdx.x < (1u << p.bits)) {
        const uint32_t* row = counts + threadIdx.x;
        if (p.tiles <= kDirectTiles) {
            for (uint32_t b = 0; b < p.tiles; b += 32) {
                uint32_t n[32];               // loaded together
#pragma unroll
                for (uint32_t u = 0; u < 32; ++u) n[u] = b + u < p.tiles ? row[(b + u) << p.bits] : 0;
#pragma unroll
                for (uint32_t u = 0; u < 32; ++u) {
                    total += n[u];
                    earlier += b + u < blockIdx.x ? n[u] : 0;
                }
            }
        } else {
            total = totals[threadIdx.x];
            earlier = row[(uint64_t)blockIdx.x << p.bits];
        }
    }
    // exclusive sum of the totals over the digits, a digit a thread: within the wave ...
    uint32_t sum = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(sum, d);
        if ((int)lane >= d) sum += y;
    }
    if (lane == 63) waves[wave] = sum;
    const uint64_t lower = (1ull << lane) - 1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const uint32_t t = blockIdx.x * kSortTile + (wave * kEach + k) * 64 + lane;
        const bool there = t < a.tokens;
        digit[k] = (uint32_t)(x[k] >> (32 + p.shift)) & ((1u << p.bits) - 1);
        uint64_t same = __ballot(there);
        for (int b = 0; b < p.bits; ++b) {
            const uint64_t on = __ballot((digit[k] >> b) & 1u);
            same &= (digit[k] >> b) & 1u ? on : ~on;
        }
        rank[k] = seen[wave][digit[k]] + (uint32_t)__popcll(same & lower);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (there && (same & lower) == 0) seen[wave][digit[k]] += (uint32_t)__popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // ... and over the waves; then over the tile's waves of each digit
    uint32_t at = sum - total + earlier;
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) at += w < wave ? waves[w] : 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t n = seen[w][threadIdx.x];
        seen[w][threadIdx.x] = at;
        at += n;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const uint32_t t = blockIdx.x * kSortTile + (wave * kEach + k) * 64 + lane;
        if (t < a.tokens) out[seen[wave][digit[k]] + rank[k]] = x[k];
    }
}

// ---------------------------------------------------------------------------
// Sums.  A frequent token's row may have thousands of terms, so the sorted list
// is cut into aligned groups of G = 2^log, and of G * G, ...: a group that lies
// within one row is summed once, by lanes of its own, into the workspace
// (level 1 from dy, level l from level l - 1); a row then adds at most 2 (G - 1)
// terms a level.  Which terms are added in which order depends on the sorted
// list alone.
constexpr int kMaxLevels = 5;
// Loads in flight in a row's sum: with 8 (of 8 elements) the kernel has 5 waves a SIMD
// and took 204 us for the 16,384 x 8192 gradient, with 4 it took 173.
constexpr int kRowFlight = 4;

struct GradArgs {
    const uint64_t* sorted;
    const void* dy;
    void* grad;
    uint32_t* starts;                         // [rows + 1]: each row's first place in `sorted`
    float* part[kMaxLevels];                  // [tokens >> (log * l)][dim] sums of level l = 1, 2, ...
    int64_t ld_dy, ld_grad, dim, rows;
    uint32_t tokens;
    int32_t levels, log;
    float scale;
};

// acc += the E elements from `col` of `count` rows, FLIGHT rows' loads at a time;
// row(j) is the address of the j-th row.  `narrow`: rows of dim < E elements, whole.
template <int DT, int E, int FLIGHT, class Row>
__device__ __forceinline__ void add_rows(float (&acc)[E], uint32_t col, uint32_t count, bool narrow, int dim,
                                         Row row) {
    if (!narrow) {
        auto batch = [&](uint32_t j, uint32_t n) {
            Raw<DT, E> r[FLIGHT];
#pragma unroll
            for (uint32_t u = 0; u < FLIGHT; ++u)
                if (u < n) r[u].load(row(j + u), col);
#pragma unroll
            for (uint32_t u = 0; u < FLIGHT; ++u)
                if (u < n) {
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[i] += r[u].get(i);
                }
        };
        uint32_t j = 0;
        for (; j + FLIGHT <= count; j += FLIGHT) batch(j, FLIGHT);
        if (j < count) batch(j, count - j);
    } else {
        for (uint32_t j = 0; j < count; ++j) {
            const void* base = row(j);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < dim) acc[i] += load1<DT>(base, i);
        }
    }
}

// Reads of wave-uniform addresses through the scalar cache, of what earlier
// launches wrote.
template <class T>
__device__ __forceinline__ T load_uniform(const T* p, int64_t i) {
    typedef const T __attribute__((address_space(4))) scalar_t;
    return reinterpret_cast<scalar_t*>(reinterpret_cast<uintptr_t>(p))[i];
}
template <bool UNIFORM, class T>
__device__ __forceinline__ T load_from(const T* p, int64_t i) {
    if constexpr (UNIFORM) return load_uniform(p, i);
    else return p[i];
}

// How rows (or groups) are dealt out.  WIDE, for rows of more than 32 pieces: a wave
// takes 64 pieces of one row, so that the row's places and positions are scalars
// (131,072 x 2048: row sums 144 us, lane by lane 191).  Otherwise lanes one after the
// other, a piece each, several rows a wave.  `per` counts items a row, waves or lanes.
// (Two pieces a lane and row: 0 to 7% slower.)
struct Share {
    uint32_t items;
    Divisor per;
};
inline bool wide_rows(uint32_t pieces) { return pieces > 32; }
inline Share share_of(int64_t rows, uint32_t pieces) {
    const uint32_t per = wide_rows(pieces) ? (pieces + 63) / 64 : pieces;
    return Share{(uint32_t)(rows * per), divisor(per)};
}

// This lane's row and first column; false past the end.
template <bool WIDE, int E>
__device__ __forceinline__ bool my_share(const Share& s, uint32_t block, uint32_t& row, uint32_t& col) {
    const uint32_t lane = block * kThreads + threadIdx.x;
    const uint32_t item = WIDE ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(lane >> 6)) : lane;
    if (item >= s.items) return false;
    row = quotient(item, s.per);
    const uint32_t rest = item - row * s.per.d;
    col = (WIDE ? rest * 64 + (threadIdx.x & 63u) : rest) * E;
    return true;
}
// Elements that a piece from `col` writes (0: past the row); a short piece is moved
// back to end with the row.
template <int E>
__device__ __forceinline__ int piece_count(int64_t dim, bool narrow, uint32_t& col) {
    const int64_t left = dim - (int64_t)col;
    const int count = left >= E ? E : left > 0 ? (int)left : 0;
    if (!narrow && count < E) col = (uint32_t)(dim - E);
    return count;
}

// First place of the sorted list whose row is not below r.
__device__ __forceinline__ uint32_t lower_bound(const uint64_t* __restrict__ s, uint32_t n, uint64_t r) {
    uint32_t lo = 0;
    while (n > 0) {
        const uint32_t half = n >> 1;
        if (s[lo + half] >> 32 < r) { lo += half + 1; n -= half + 1; } else n = half;
    }
    return lo;
}

// Level `level` sums of whole groups that lie within one row: 39 us of 192 for 131,072 x
// 2048 (200 MB read), 17 of 196 for 16,384 x 8192.  On level 1 the
// workgroups from `start_blocks` on; those before find the rows' first places, a row a
// lane.
template <int DT, bool FIRST, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_group_sums(GradArgs a, int32_t level, uint32_t start_blocks,
                                                         Share share) {
    constexpr int E = FIRST ? piece_elems<DT, DT>() : 4;
    uint32_t block = blockIdx.x;
    if constexpr (FIRST) {
        if (block < start_blocks) {
            const uint32_t r = block * kThreads + threadIdx.x;
            if (r <= a.rows) a.starts[r] = lower_bound(a.sorted, a.tokens, r);
            return;
        }
        block -= start_blocks;
    }
    uint32_t group, col;
    if (!my_share<WIDE, E>(share, block, group, col)) return;
    const uint32_t lo = group << (a.log * level);
    const uint32_t hi = lo + (1u << (a.log * level)) - 1;
    const uint32_t key = (uint32_t)(load_from<WIDE>(a.sorted, lo) >> 32);
    if (key != (uint32_t)(load_from<WIDE>(a.sorted, hi) >> 32) || key >= a.rows) return;
    const bool narrow = !WIDE && a.dim < E;
    const int count = piece_count<E>(a.dim, narrow, col);
    if (count == 0) return;
    float acc[E] = {};
    if constexpr (FIRST) {
        add_rows<DT, E, 8>(acc, col, 1u << a.log, narrow, (int)a.dim, [&](uint32_t j) {
            return from<DT>(a.dy, (int64_t)(uint32_t)load_from<WIDE>(a.sorted, lo + j) * a.ld_dy);
        });
    } else {
        const int64_t below = (int64_t)group << a.log;
        add_rows<ZPQ_F32, E, 8>(acc, col, 1u << a.log, narrow, (int)a.dim, [&](uint32_t j) {
            return from<ZPQ_F32>((const void*)a.part[level - 2], (below + j) * a.dim);
        });
    }
    float* to = a.part[level - 1] + (int64_t)group * a.dim;
    if (narrow) {
        for (int i = 0; i < (int)a.dim; ++i) to[i] = acc[i];
    } else {
        Raw<ZPQ_F32, E> o;                    // a piece that was moved back writes the same again
        o.set(acc);
        o.template store<false>(to, col);
    }
}

// Rows: each lane sums its piece over the row's places [at, e) of the list.  Rows without
// a token are written at 6.6 TB/s where they are long (8192 bf16; non-temporal stores; plain
// ones 4.5), at 5.0 in 100,000 rows of 2000 bf16 (80 us); where rows have
// a few tokens each the chain of place, token, dy and store is what takes the time, and
// the waves in flight: 168 us for 16,384 x 8192 into 50,021 rows of bf16 (1.03 GB), 130 us
// for 131,072 x 2048 added to 65,536 rows of fp32 (762 MB).
// BY_TOKEN: the rows are those that tokens name, each found at its first token; `first`
// and the shares count tokens.
template <int DT, int OT, bool ADD, bool BY_TOKEN, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_row_sums(GradArgs a, int64_t first, Share share) {
    constexpr int E = piece_elems<DT, OT>();
    uint32_t r, col;
    if (!my_share<WIDE, E>(share, blockIdx.x, r, col)) return;
    int64_t row = first + r;
    uint32_t at, e;
    if constexpr (BY_TOKEN) {
        at = (uint32_t)row;
        row = (int64_t)(load_from<WIDE>(a.sorted, at) >> 32);
        if (row >= a.rows || (at > 0 && (int64_t)(load_from<WIDE>(a.sorted, at - 1) >> 32) == row)) return;
        e = load_from<WIDE>(a.starts, row + 1);
    } else {
        at = load_from<WIDE>(a.starts, row);
        e = load_from<WIDE>(a.starts, row + 1);
        if (ADD && at == e) return;
    }
    const bool narrow = !WIDE && a.dim < E;
    const int count = piece_count<E>(a.dim, narrow, col);
    if (count == 0) return;
    void* grad = from<OT>(a.grad, row * a.ld_grad);
    Raw<OT, E> old;
    if constexpr (ADD) {                      // early: it depends on nothing below
        if (!narrow) old.load(grad, col);
        else old.load_some(grad, 0, count);
    }
    const float scale = at < e ? a.scale : 0.0f;          // no token: zeros, whatever the scale
    float acc[E] = {};
#pragma unroll 1
    while (at < e) {
        int level = a.levels;
#pragma unroll 1
        while (level > 0 && ((at & ((1u << (a.log * level)) - 1)) != 0 ||
                             e - at < (1u << (a.log * level))))
            --level;
        if (level == 0) {
            // up to the next group that could be whole
            uint32_t stop = a.levels > 0 ? (at | ((1u << a.log) - 1)) + 1 : e;
            if (stop > e) stop = e;
            add_rows<DT, E, kRowFlight>(acc, col, stop - at, narrow, (int)a.dim, [&](uint32_t j) {
                return from<DT>(a.dy, (int64_t)(uint32_t)load_from<WIDE>(a.sorted, at + j) * a.ld_dy);
            });
            at = stop;
        } else {
            // groups of this level up to the end, or to where a larger one starts
            const uint32_t shift = a.log * level;
            uint32_t groups = (e - at) >> shift;
            if (level < a.levels) {
                const uint32_t next = (1u << a.log) - ((at >> shift) & ((1u << a.log) - 1));
                if (next < groups) groups = next;
            }
            const void* part = from<ZPQ_F32>((const void*)a.part[level - 1], (int64_t)(at >> shift) * a.dim);
            add_rows<ZPQ_F32, E, kRowFlight>(acc, col, groups, narrow, (int)a.dim, [&](uint32_t j) {
                return from<ZPQ_F32>(part, (int64_t)j * a.dim);
            });
            at += groups << shift;
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        acc[i] *= scale;
        if constexpr (ADD) acc[i] = old.get(i) + acc[i];
    }
    Raw<OT, E> out;
    out.set(acc);
    if (count == E) {
        out.store(grad, col);
    } else if (narrow) {
        out.store_some(grad, 0, count);
    } else {                                  // the last elements of a piece that was moved back
#pragma unroll
        for (int i = 1; i < E; ++i)
            if (i >= E - count) store1<OT>(grad, (int64_t)col + i, acc[i]);
    }
}

// ---------------------------------------------------------------------------
// Host side.
// Launches of at most 2^30 lanes: the division's range.
template <int TT, int OT>
void launch_lookup(LookupArgs a, hipStream_t st) {
    constexpr int E = piece_elems<TT, OT>();
    const uint32_t pieces = (uint32_t)((a.dim + E - 1) / E);
    a.pieces = divisor(pieces);
    const char* ids = static_cast<const char*>(a.ids);
    char* out = static_cast<char*>(a.out);
    const int64_t some = (1 << 30) / pieces;
    for (int64_t t = 0; t < a.tokens; t += some) {
        const int64_t n = a.tokens - t < some ? a.tokens - t : some;
        a.ids = ids + t * a.id_bytes;
        a.out = out + t * a.ld_out * elem_bytes<OT>();
        a.lanes = (uint32_t)(n * pieces);
        const unsigned grid = (a.lanes + kLookupPieces * kThreads - 1) / (kLookupPieces * kThreads);
        hipLaunchKernelGGL((k_lookup<TT, OT>), dim3(grid), dim3(kThreads), 0, st, a);
    }
}
template <int TT>
void launch_lookup_o(const LookupArgs& a, int32_t out_dtype, hipStream_t st) {
    if (out_dtype == ZPQ_F32) launch_lookup<TT, ZPQ_F32>(a, st);
    else if (out_dtype == ZPQ_F16) launch_lookup<TT, ZPQ_F16>(a, st);
    else launch_lookup<TT, ZPQ_BF16>(a, st);
}

// Bytes from the first to the last element of `rows` rows.
inline uint64_t span(int64_t rows, int64_t dim, int64_t ld, int64_t eb) {
    return rows > 0 ? (uint64_t)((rows - 1) * ld + dim) * (uint64_t)eb : 0;
}

constexpr int64_t kMaxRows = 0x7FFFFFFF;

zpq_status rows_ok(int64_t rows, int64_t tokens, int64_t dim, int64_t ld_a, int64_t ld_b) {
    if (rows < 0 || rows > kMaxRows || tokens < 0 || tokens > kMaxRows || dim < 1 || dim > (1 << 30) ||
        ld_a < dim || ld_b < dim || ld_a > kMaxElems || ld_b > kMaxElems)
        return ZPQ_ERR_SIZE;
    // element offsets within 2^60, bytes within 2^62
    if ((rows > 0 && ld_a > (1LL << 60) / rows) || (tokens > 0 && ld_b > (1LL << 60) / tokens))
        return ZPQ_ERR_SIZE;
    return ZPQ_OK;
}

zpq_status lookup(const LookupArgs& a, int32_t t_dtype, int32_t out_dtype, hipStream_t st) {
    if (t_dtype == ZPQ_F32) launch_lookup_o<ZPQ_F32>(a, out_dtype, st);
    else if (t_dtype == ZPQ_F16) launch_lookup_o<ZPQ_F16>(a, out_dtype, st);
    else if (t_dtype == ZPQ_BF16) launch_lookup_o<ZPQ_BF16>(a, out_dtype, st);
    else launch_lookup_o<kI8>(a, out_dtype, st);
    return after_launch();
}

struct GradWorkspace {
    int64_t sorted[2], counts, totals, starts, part[kMaxLevels], bytes;
    int32_t levels, log;
};

// Groups of 16 where the gradient is small and a frequent row's chain of additions
// is what takes the time (8000 tokens x 100: 39 us, with 64 56), of 64 where the sums' own
// traffic tells (131,072 x 2048: 204 us, with 16 216); about even at 2^25.  Level 1 pays from
// some hundred tokens on (its launch takes 3.5 us), a further level (a launch that
// mostly finds nothing to sum) only where a row could hold very many groups, or where
// rows average a group of it.
constexpr int64_t kSmallGrad = 1 << 25;       // tokens * dim
inline GradWorkspace grad_workspace(int64_t tokens, int64_t dim, int64_t rows) {
    GradWorkspace w = {};
    auto take = [&](int64_t bytes) {
        const int64_t at = w.bytes;
        w.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    w.starts = take((rows + 1) * 4);
    w.sorted[0] = take(tokens * 8);
    if (tokens > kRankTokens) w.sorted[1] = take(tokens * 8);
    if (tokens > kMergeTokens) {
        w.counts = take((tokens + kSortTile - 1) / kSortTile * kMaxDigits * 4);
        w.totals = take(kMaxDigits * 4);
    }
    w.log = tokens * dim <= kSmallGrad ? 4 : 6;
    for (int l = 1; l <= kMaxLevels && tokens >= 512; ++l) {
        const int64_t groups = tokens >> (w.log * l);
        if (l > 1 && (groups < 2 || (groups < 64 && groups < rows))) break;
        w.part[l - 1] = take(groups * dim * 4);
        w.levels = l;
    }
    return w;
}

// The sorted list; `list` and `other` are exchanged as the passes need.  True where
// the rows' first places have been found as well, by comparing every row with every
// token, which saves a launch (or, from 512 tokens on, binary searches in one).  That
// takes a workgroup of 16 waves for 64 rows whatever the tokens, 1024 such workgroups
// about as long as the launch: 5 tokens added to 65,000 rows of 64 6.8 us, by search 7.8;
// to 131,072 9.9 and 7.7, to 1,000,000 42.9 and 9.2.  And it takes the comparisons: 1000
// tokens into 16,000 rows (2^24) 9.9 and 11.8 us, 4000 into 16,000 (2^26) 16.9 and 16.1.
constexpr int64_t kRankRows = 1 << 16, kRankCompares = 1 << 24;
bool sort_tokens(const Ids& a, uint64_t*& list, uint64_t*& other, uint32_t* counts, uint32_t* totals,
                 uint32_t* starts, hipStream_t st) {
    if (a.tokens == 0) return false;
    if (a.tokens <= kRankTokens) {
        const bool rows = a.rows <= kRankRows && a.rows * a.tokens <= kRankCompares;
        const unsigned blocks = (a.tokens + 63) / 64 + (rows ? (unsigned)(a.rows / 64 + 1) : 0);
        hipLaunchKernelGGL(k_rank, dim3(blocks), dim3(64 * kRankWaves), 0, st, a, kRankTokens, list, starts);
        return rows;
    }
    if (a.tokens <= kMergeTokens) {
        const uint32_t log = run_log(a.tokens);
        hipLaunchKernelGGL(k_rank, dim3((a.tokens + 63) / 64), dim3(64 * kRankWaves), 0, st, a, 1u << log, other,
                           starts);
        hipLaunchKernelGGL(k_merge, dim3((a.tokens * kRuns + kThreads - 1) / kThreads), dim3(kThreads), 0, st,
                           other, a.tokens, log, list);
        return false;
    }
    int bits = 1;
    while (a.rows >> bits) ++bits;            // of the largest key, `rows`
    const int passes = (bits + 8) / 9;
    Pass p = {0, (bits + passes - 1) / passes, (a.tokens + kSortTile - 1) / kSortTile};
    for (int i = 0; i < passes; ++i, p.shift += p.bits) {
        const dim3 grid(p.tiles), block(kSortThreads);
        if (i == 0) hipLaunchKernelGGL(k_digit_counts<true>, grid, block, 0, st, a, list, p, counts);
        else hipLaunchKernelGGL(k_digit_counts<false>, grid, block, 0, st, a, list, p, counts);
        if (p.tiles > kDirectTiles)
            hipLaunchKernelGGL(k_digit_scan, dim3(1u << p.bits), dim3(64), 0, st, p, counts, totals);
        if (i == 0) hipLaunchKernelGGL(k_digit_place<true>, grid, block, 0, st, a, list, p, counts, totals, other);
        else hipLaunchKernelGGL(k_digit_place<false>, grid, block, 0, st, a, list, p, counts, totals, other);
        uint64_t* t = list;
        list = other;
        other = t;
    }
    return false;
}

// Workgroups of a share.
inline unsigned share_blocks(const Share& s, bool wide) {
    const unsigned items = wide ? kThreads / 64 : kThreads;
    return s.items / items + (s.items % items != 0);
}

template <int DT, bool FIRST>
void launch_group_level(const GradArgs& a, int32_t level, int64_t groups, uint32_t start_blocks, hipStream_t st) {
    constexpr int E = FIRST ? piece_elems<DT, DT>() : 4;
    const uint32_t pieces = (uint32_t)((a.dim + E - 1) / E);
    const bool wide = wide_rows(pieces);
    const Share s = share_of(groups, pieces);
    const dim3 grid(share_blocks(s, wide) + start_blocks), block(kThreads);
    if (wide)
        hipLaunchKernelGGL((k_group_sums<DT, FIRST, true>), grid, block, 0, st, a, level, start_blocks, s);
    else
        hipLaunchKernelGGL((k_group_sums<DT, FIRST, false>), grid, block, 0, st, a, level, start_blocks, s);
}
template <int DT>
void launch_groups(const GradArgs& a, bool starts_done, hipStream_t st) {
    const uint32_t start_blocks = starts_done ? 0 : (uint32_t)(a.rows / kThreads + 1);
    if (a.levels > 0 || start_blocks > 0)
        launch_group_level<DT, true>(a, 1, a.levels > 0 ? a.tokens >> a.log : 0, start_blocks, st);
    for (int l = 2; l <= a.levels; ++l) launch_group_level<DT, false>(a, l, a.tokens >> (a.log * l), 0, st);
}

// In launches of at most 2^30 lanes.
template <int DT, int OT, bool ADD, bool BY_TOKEN>
void launch_rows(const GradArgs& a, hipStream_t st) {
    constexpr int E = piece_elems<DT, OT>();
    const uint32_t pieces = (uint32_t)((a.dim + E - 1) / E);
    const bool wide = wide_rows(pieces);
    const int64_t all = BY_TOKEN ? a.tokens : a.rows;
    const int64_t some = (wide ? 1 << 24 : 1 << 30) / share_of(1, pieces).items;
    for (int64_t first = 0; first < all; first += some) {
        const Share s = share_of(all - first < some ? all - first : some, pieces);
        const dim3 grid(share_blocks(s, wide)), block(kThreads);
        if (wide)
            hipLaunchKernelGGL((k_row_sums<DT, OT, ADD, BY_TOKEN, true>), grid, block, 0, st, a, first, s);
        else
            hipLaunchKernelGGL((k_row_sums<DT, OT, ADD, BY_TOKEN, false>), grid, block, 0, st, a, first, s);
    }
}
template <int DT, int OT>
void launch_rows_add(const GradArgs& a, bool add, hipStream_t st) {
    // rows that get nothing are not touched: a launch over the tokens is smaller where
    // there are fewer of them
    if (add && (int64_t)a.tokens < a.rows) launch_rows<DT, OT, true, true>(a, st);
    else if (add) launch_rows<DT, OT, true, false>(a, st);
    else launch_rows<DT, OT, false, false>(a, st);
}
template <int DT>
void launch_grad(const GradArgs& a, int32_t grad_dtype, bool add, bool starts_done, hipStream_t st) {
    launch_groups<DT>(a, starts_done, st);
    if (grad_dtype == ZPQ_F32) launch_rows_add<DT, ZPQ_F32>(a, add, st);
    else if (grad_dtype == ZPQ_F16) launch_rows_add<DT, ZPQ_F16>(a, add, st);
    else launch_rows_add<DT, ZPQ_BF16>(a, add, st);
}

// A launch holds less than 2^32 work-items; groups of pieces are counted in 31
// bits, a launch's rows of pieces in 30.
bool grad_sizes_ok(int64_t tokens, int64_t dim, int64_t rows) {
    return tokens >= 0 && tokens <= (1LL << 28) && dim >= 1 && dim <= (1 << 28) && rows >= 0 &&
           rows <= (1LL << 27) && (tokens >> 6) * ((dim + 3) / 4) < (1LL << 31);
}

}  // namespace

extern "C" {

zpq_status zpq_embedding(const void* table, int32_t t_dtype, int64_t rows, int64_t dim,
                         int64_t ld_table, const void* ids, int32_t id_bytes, int64_t tokens,
                         int64_t first, float scale, void* out, int32_t out_dtype, int64_t ld_out,
                         zpq_stream stream) {
    if (const zpq_status bad = rows_ok(rows, tokens, dim, ld_table, ld_out)) return bad;
    const int64_t tb = dtype_bytes(t_dtype), ob = dtype_bytes(out_dtype);
    if (tb == 0 || ob == 0) return ZPQ_ERR_DTYPE;
    if (id_bytes != 4 && id_bytes != 8) return ZPQ_ERR_ARG;
    if (tokens == 0) return ZPQ_OK;
    if (!ids || !out || (rows > 0 && !table)) return ZPQ_ERR_NULL;
    if (!aligned(ids, id_bytes) || !aligned(out, ob) || !aligned(table, tb)) return ZPQ_ERR_ALIGN;
    const uint64_t on = span(tokens, dim, ld_out, ob);
    if (overlaps(out, on, table, span(rows, dim, ld_table, tb)) || overlaps(out, on, ids, tokens * id_bytes))
        return ZPQ_ERR_ALIAS;
    return lookup(LookupArgs{table, nullptr, ids, out, tokens, rows, dim, ld_table, first, ld_out, scale, id_bytes, 0,
                             0, {}},
                  t_dtype, out_dtype, static_cast<hipStream_t>(stream));
}

zpq_status zpq_embedding_i8(const int8_t* codes, const float* scales, int64_t rows, int64_t dim,
                            int32_t block, const void* ids, int32_t id_bytes, int64_t tokens,
                            int64_t first, float scale, void* out, int32_t out_dtype,
                            int64_t ld_out, zpq_stream stream) {
    int32_t log_block = 5;
    while (log_block < 10 && (1 << log_block) != block) ++log_block;
    if (log_block == 10) return ZPQ_ERR_BLOCK;
    if (const zpq_status bad = rows_ok(rows, tokens, dim, dim, ld_out)) return bad;
    const int64_t ob = dtype_bytes(out_dtype);
    if (ob == 0) return ZPQ_ERR_DTYPE;
    if (id_bytes != 4 && id_bytes != 8) return ZPQ_ERR_ARG;
    if (tokens == 0) return ZPQ_OK;
    if (!ids || !out || (rows > 0 && (!codes || !scales))) return ZPQ_ERR_NULL;
    if (!aligned(ids, id_bytes) || !aligned(out, ob) || !aligned(scales, 4)) return ZPQ_ERR_ALIGN;
    const uint64_t on = span(tokens, dim, ld_out, ob), tn = (uint64_t)rows * (uint64_t)dim;
    if (overlaps(out, on, codes, tn) || overlaps(out, on, scales, (tn + block - 1) / block * 4) ||
        overlaps(out, on, ids, tokens * id_bytes))
        return ZPQ_ERR_ALIAS;
    return lookup(LookupArgs{codes, scales, ids, out, tokens, rows, dim, dim, first, ld_out, scale, id_bytes,
                             log_block, 0, {}},
                  kI8, out_dtype, static_cast<hipStream_t>(stream));
}

zpq_status zpq_embedding_grad_bytes(int64_t tokens, int64_t rows, int64_t dim, int64_t* bytes) {
    if (!bytes) return ZPQ_ERR_NULL;
    if (!grad_sizes_ok(tokens, dim, rows)) return ZPQ_ERR_SIZE;
    *bytes = grad_workspace(tokens, dim, rows).bytes;
    return ZPQ_OK;
}

zpq_status zpq_embedding_grad(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* ids,
                              int32_t id_bytes, int64_t tokens, int64_t first, int64_t padding,
                              int64_t rows, int64_t dim, float scale, void* grad,
                              int32_t grad_dtype, int64_t ld_grad, int32_t accumulate,
                              void* workspace, int64_t workspace_bytes, zpq_stream stream) {
    if (!grad_sizes_ok(tokens, dim, rows)) return ZPQ_ERR_SIZE;
    if (const zpq_status bad = rows_ok(rows, tokens, dim, ld_grad, ld_dy)) return bad;
    const int64_t yb = dtype_bytes(dy_dtype), gb = dtype_bytes(grad_dtype);
    if (yb == 0 || gb == 0) return ZPQ_ERR_DTYPE;
    if (id_bytes != 4 && id_bytes != 8) return ZPQ_ERR_ARG;
    if (rows == 0) return ZPQ_OK;
    const GradWorkspace w = grad_workspace(tokens, dim, rows);
    if (!grad || !workspace || (tokens > 0 && (!dy || !ids))) return ZPQ_ERR_NULL;
    if (workspace_bytes < w.bytes) return ZPQ_ERR_SIZE;
    if (!aligned(grad, gb) || !aligned(dy, yb) || !aligned(ids, id_bytes) || !aligned(workspace, 16))
        return ZPQ_ERR_ALIGN;
    const void* at[4] = {grad, workspace, dy, ids};
    const uint64_t size[4] = {span(rows, dim, ld_grad, gb), (uint64_t)w.bytes,
                              span(tokens, dim, ld_dy, yb), (uint64_t)(tokens * id_bytes)};
    for (int x = 0; x < 2; ++x)
        for (int y = x + 1; y < 4; ++y)
            if (overlaps(at[x], size[x], at[y], size[y])) return ZPQ_ERR_ALIAS;
    if (accumulate && tokens == 0) return ZPQ_OK;

    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(ws + at); };
    uint64_t* list = reinterpret_cast<uint64_t*>(ws + w.sorted[0]);
    uint64_t* other = reinterpret_cast<uint64_t*>(ws + w.sorted[1]);
    const Ids sorted = {ids, first, padding, rows, id_bytes, (uint32_t)tokens};
    const bool starts_done = sort_tokens(sorted, list, other, words(w.counts), words(w.totals),
                                         words(w.starts), st);
    GradArgs a = {list, dy, grad, words(w.starts), {}, ld_dy, ld_grad, dim, rows, (uint32_t)tokens,
                  w.levels, w.log, scale};
    for (int l = 0; l < w.levels; ++l) a.part[l] = reinterpret_cast<float*>(ws + w.part[l]);
    if (dy_dtype == ZPQ_F32) launch_grad<ZPQ_F32>(a, grad_dtype, accumulate != 0, starts_done, st);
    else if (dy_dtype == ZPQ_F16) launch_grad<ZPQ_F16>(a, grad_dtype, accumulate != 0, starts_done, st);
    else launch_grad<ZPQ_BF16>(a, grad_dtype, accumulate != 0, starts_done, st);
    return after_launch();
}

}  // extern "C"
