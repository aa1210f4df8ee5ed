// embedding.hip -- embedding lookup with scaling, from a float table or from
// qwZ's gathered INT8 blocks, and the embedding's gradient by sorted tokens.
//
// A row is cut into pieces of 8 elements, one a lane; the last piece of a row
// whose length is no multiple of 8 is moved back so that it ends with the row
// (it reads, and in the lookup writes, some elements twice).  Rows shorter
// than 8 are one piece, handled element by element.
#include "step.h"

namespace {

using namespace zpq_step;

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
// Lookup.  Lane L of the grid takes piece L % pieces of token L / pieces.
struct LookupArgs {
    const void* table;
    const float* scales;
    const void* ids;
    void* out;
    int64_t rows, dim, ld_table, first, ld_out;
    float scale;
    int32_t id_bytes, log_block;
    uint32_t lanes;                           // tokens * pieces, < 2^31
    Divisor pieces;
};

template <int TT, int OT, int U>
__global__ __launch_bounds__(kThreads) void k_lookup(LookupArgs a) {
    uint32_t lane[U], token[U];
    int64_t row[U];
    int32_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        lane[u] = (blockIdx.x * U + u) * kThreads + threadIdx.x;
        token[u] = quotient(lane[u], a.pieces);
        col[u] = (int32_t)(lane[u] - token[u] * a.pieces.d) * 8;
        row[u] = lane[u] < a.lanes ? load_id(a.ids, a.id_bytes, token[u])
                                  : (int64_t)((uint64_t)a.first - 1);
    }
    if (a.dim < 8) {
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
    Raw8<TT> in[U];
    float s0[U], s1[U];
    int32_t left[U];                          // elements of the piece that s0 scales
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (col[u] > a.dim - 8) col[u] = (int32_t)a.dim - 8;
        const uint64_t r = (uint64_t)row[u] - (uint64_t)a.first;
        const bool there = r < (uint64_t)a.rows;
#pragma unroll
        for (int i = 0; i < Raw8<TT>::WORDS; ++i) in[u].w[i] = 0;
        s0[u] = s1[u] = 1.0f;
        left[u] = 8;
        if (there) {
            const int64_t e = (int64_t)r * a.ld_table + col[u];
            in[u].template load<false>(a.table, e);
            if constexpr (TT == kI8) {
                s0[u] = a.scales[e >> a.log_block];
                left[u] = (1 << a.log_block) - (int32_t)(e & ((1 << a.log_block) - 1));
                s1[u] = left[u] < 8 ? a.scales[(e >> a.log_block) + 1] : s0[u];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (lane[u] >= a.lanes) continue;
        const bool there = (uint64_t)row[u] - (uint64_t)a.first < (uint64_t)a.rows;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = in[u].get(i);
            if constexpr (TT == kI8) x[i] *= i < left[u] ? s0[u] : s1[u];
            x[i] = there ? x[i] * a.scale : 0.0f;
        }
        Raw8<OT> o;
        o.set(x);
        o.store(a.out, token[u] * a.ld_out + col[u]);
    }
}

// ---------------------------------------------------------------------------
// Sorting the tokens by row.  A token is the 64-bit number row * 2^32 + position
// (row = `rows` for what does not count): all different, so any correct sort
// is the stable one.  Tiles of N are sorted in LDS by a bitonic network; then
// runs are merged kFan at a time by ranks: an element's place in the merged run is
// its place in its own plus, for each other run, how many elements there are
// smaller (a binary search).  No counters, no atomics, two launches up to
// kFan * N tokens.
constexpr int kFan = 32;

template <int N, int THREADS>
__global__ __launch_bounds__(THREADS) void k_sort_tile(const void* __restrict__ ids,
                                                       int32_t id_bytes, uint32_t tokens,
                                                       int64_t first, int64_t padding, int64_t rows,
                                                       uint64_t* __restrict__ out) {
    __shared__ uint64_t s[N];
    const uint32_t base = blockIdx.x * N;
    for (int i = threadIdx.x; i < N; i += THREADS) {
        const uint32_t t = base + i;
        uint64_t x = ~0ull;
        if (t < tokens) {
            const int64_t id = load_id(ids, id_bytes, t);
            const uint64_t r = (uint64_t)id - (uint64_t)first;
            x = (r < (uint64_t)rows && id != padding ? r : (uint64_t)rows) << 32 | t;
        }
        s[i] = x;
    }
    __syncthreads();
    for (int k = 2; k <= N; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < N / 2; i += THREADS) {
                const int lo = (i & (j - 1)) | (i & ~(j - 1)) << 1, hi = lo | j;
                const uint64_t a = s[lo], b = s[hi];
                if ((a > b) == ((lo & k) == 0)) { s[lo] = b; s[hi] = a; }
            }
            __syncthreads();
        }
    for (int i = threadIdx.x; i < N; i += THREADS)
        if (base + i < tokens) out[base + i] = s[i];
}

// kLanes lanes search for one element, each in kFan / kLanes of the group's runs.
constexpr int kLanes = 8;
__global__ __launch_bounds__(kThreads) void k_merge(const uint64_t* __restrict__ in, uint32_t tokens,
                                                    uint32_t run, uint64_t* __restrict__ out) {
    const uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const uint32_t e = (uint32_t)(g / kLanes), part = (uint32_t)(g % kLanes);
    if (e >= tokens) return;                  // whole groups of lanes: tokens are counted in them
    const uint64_t x = in[e];
    const uint32_t own = e / run, group = own / kFan * kFan;
    const uint64_t start = (uint64_t)group * run;
    uint32_t lo[kFan / kLanes], n[kFan / kLanes];
    uint64_t at[kFan / kLanes];
#pragma unroll
    for (int r = 0; r < kFan / kLanes; ++r) {
        const uint32_t which = group + r * kLanes + part;
        at[r] = (uint64_t)which * run;
        n[r] = at[r] >= tokens ? 0 : tokens - at[r] < run ? (uint32_t)(tokens - at[r]) : run;
        lo[r] = 0;
        if (which == own) { lo[r] = e - own * run; n[r] = 0; }
    }
    for (uint32_t left = run; left > 0; left >>= 1) {   // n halves at least as fast as `left`
#pragma unroll
        for (int r = 0; r < kFan / kLanes; ++r)
            if (n[r] > 0) {
                const uint32_t half = n[r] >> 1;
                if (in[at[r] + lo[r] + half] < x) { lo[r] += half + 1; n[r] -= half + 1; }
                else n[r] = half;
            }
    }
    uint32_t rank = 0;
#pragma unroll
    for (int r = 0; r < kFan / kLanes; ++r) rank += lo[r];
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) rank += __shfl_xor(rank, d);
    if (part == 0) out[start + rank] = x;
}

// ---------------------------------------------------------------------------
// Sums.  A frequent token's row may have thousands of terms, so the sorted list
// is cut into aligned groups of 64, and of 64 * 64, ...: a group that lies
// within one row is summed once, by lanes of its own, into the workspace
// (level 1 from dy, level l from level l - 1); a row then adds at most 2 * 63
// terms a level.  Which terms are added in which order depends on the sorted
// list alone.
constexpr int kGroupLog = 6, kGroup = 1 << kGroupLog, kMaxLevels = 5;

struct GradArgs {
    const uint64_t* sorted;
    const void* dy;
    void* grad;
    float* part[kMaxLevels];                  // [tokens >> 6l][dim] sums of level l = 1, 2, ...
    int64_t ld_dy, ld_grad, dim, rows;
    uint32_t tokens;
    int32_t levels;
    float scale;
};

// acc += `count` rows of 8 floats, `stride` elements apart; or dy rows by position.
template <int DT, class Row>
__device__ __forceinline__ void add_rows(float (&acc)[8], uint32_t count, bool narrow, int dim, Row row) {
    uint32_t j = 0;
    if (!narrow) {
        for (; j + 4 <= count; j += 4) {
            Raw8<DT> r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const void* base;
                const int64_t at = row(j + u, base);
                r[u].load(base, at);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += r[u].get(i);
        }
        for (; j < count; ++j) {
            Raw8<DT> r;
            const void* base;
            const int64_t at = row(j, base);
            r.load(base, at);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += r.get(i);
        }
    } else {
        for (; j < count; ++j) {
            const void* base;
            const int64_t at = row(j, base);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < dim) acc[i] += load1<DT>(base, at + i);
        }
    }
}

// Level `level` sums: lane L takes piece L % pieces of group L / pieces.
template <int DT, bool FIRST>
__global__ __launch_bounds__(kThreads) void k_group_sums(GradArgs a, int32_t level, uint32_t lanes,
                                                         Divisor pieces) {
    const uint32_t lane = blockIdx.x * kThreads + threadIdx.x;
    if (lane >= lanes) return;
    const uint32_t group = quotient(lane, pieces);
    const uint32_t lo = group << (kGroupLog * level);            // whole groups only: in range
    const uint32_t hi = lo + (1u << (kGroupLog * level)) - 1;
    const uint64_t key = a.sorted[lo] >> 32;
    if (key != a.sorted[hi] >> 32 || key >= (uint64_t)a.rows) return;
    const bool narrow = a.dim < 8;
    int64_t col = (int64_t)(lane - group * pieces.d) * 8;
    if (!narrow && col > a.dim - 8) col = a.dim - 8;
    float acc[8] = {};
    if constexpr (FIRST) {
        add_rows<DT>(acc, kGroup, narrow, (int)a.dim, [&](uint32_t j, const void*& base) {
            base = a.dy;
            return (int64_t)(uint32_t)a.sorted[lo + j] * a.ld_dy + col;
        });
    } else {
        const int64_t below = (int64_t)group << kGroupLog;
        add_rows<ZPQ_F32>(acc, kGroup, narrow, (int)a.dim, [&](uint32_t j, const void*& base) {
            base = a.part[level - 2];
            return (below + j) * a.dim + col;
        });
    }
    float* to = a.part[level - 1];
    if (narrow) {
        for (int i = 0; i < (int)a.dim; ++i) to[(int64_t)group * a.dim + i] = acc[i];
    } else {
        Raw8<ZPQ_F32> o;
        o.set(acc);
        o.store<false>(to, (int64_t)group * a.dim + col);
    }
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

// Workgroup b takes rows b, b + G, b + 2G, ... (kRows of them): frequent tokens
// tend to have neighbouring ids, and this spreads them.
constexpr int kRows = 16;
template <int DT, int OT, bool ADD>
__global__ __launch_bounds__(kThreads) void k_row_sums(GradArgs a, Divisor pieces) {
    __shared__ uint32_t begin[kRows], end[kRows];
    if (threadIdx.x < 2 * kRows) {
        const uint32_t r = threadIdx.x >> 1;
        const uint64_t row = (uint64_t)r * gridDim.x + blockIdx.x;
        const uint32_t at = lower_bound(a.sorted, a.tokens, row + (threadIdx.x & 1));
        if (threadIdx.x & 1) end[r] = at; else begin[r] = at;
    }
    __syncthreads();
    const bool narrow = a.dim < 8;
    for (uint32_t k = threadIdx.x; k < kRows * pieces.d; k += kThreads) {
        const uint32_t r = quotient(k, pieces);
        const int64_t row = (int64_t)r * gridDim.x + blockIdx.x;
        if (row >= a.rows) break;             // later k: later rows
        const uint32_t e = end[r];
        uint32_t at = begin[r];
        if (ADD && at == e) continue;
        int64_t col = (int64_t)(k - r * pieces.d) * 8;
        const int count = (int)(a.dim - col < 8 ? a.dim - col : 8);    // elements this lane writes
        if (!narrow && count < 8) col = a.dim - 8;
        float acc[8] = {};
        while (at < e) {
            int level = a.levels;
            while (level > 0 && ((at & ((1u << (kGroupLog * level)) - 1)) != 0 ||
                                 e - at < (1u << (kGroupLog * level))))
                --level;
            if (level == 0) {
                // up to the next group that could be whole
                uint32_t stop = a.levels > 0 ? (at | (kGroup - 1)) + 1 : e;
                if (stop > e || stop == 0) stop = e;
                add_rows<DT>(acc, stop - at, narrow, (int)a.dim, [&](uint32_t j, const void*& base) {
                    base = a.dy;
                    return (int64_t)(uint32_t)a.sorted[at + j] * a.ld_dy + col;
                });
                at = stop;
            } else {
                // groups of this level up to the end, or to where a larger one starts
                const uint32_t shift = kGroupLog * level;
                uint32_t groups = (e - at) >> shift;
                if (level < a.levels) {
                    const uint32_t next = kGroup - ((at >> shift) & (kGroup - 1));
                    if (next < groups) groups = next;
                }
                const int64_t g0 = at >> shift;
                const float* part = a.part[level - 1];
                add_rows<ZPQ_F32>(acc, groups, narrow, (int)a.dim, [&](uint32_t j, const void*& base) {
                    base = part;
                    return (g0 + j) * a.dim + col;
                });
                at += groups << shift;
            }
        }
        const int64_t o = row * a.ld_grad + col;
        if (!narrow) {
            Raw8<OT> old;
            if constexpr (ADD) old.load(a.grad, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] *= a.scale;
                if constexpr (ADD) acc[i] = old.get(i) + acc[i];
            }
            if (count == 8) {
                Raw8<OT> out;
                out.set(acc);
                out.store(a.grad, o);
            } else {
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    if (i >= 8 - count) store1<OT>(a.grad, o + i, acc[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < count) {
                    float x = acc[i] * a.scale;
                    if constexpr (ADD) x = load1<OT>(a.grad, o + i) + x;
                    store1<OT>(a.grad, o + i, x);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.
template <int TT, int OT>
void launch_lookup(const LookupArgs& a, hipStream_t st) {
    const unsigned grid = (a.lanes + kThreads - 1) / kThreads;
    hipLaunchKernelGGL((k_lookup<TT, OT, 1>), dim3(grid), dim3(kThreads), 0, st, a);
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
    // element offsets within 2^62
    if ((rows > 0 && ld_a > (1LL << 62) / rows) || (tokens > 0 && ld_b > (1LL << 62) / tokens))
        return ZPQ_ERR_SIZE;
    return ZPQ_OK;
}

zpq_status lookup(const void* table, int32_t t_dtype, const float* scales, int32_t log_block, int64_t rows,
                  int64_t dim, int64_t ld_table, const void* ids, int32_t id_bytes, int64_t tokens,
                  int64_t first, float scale, void* out, int32_t out_dtype, int64_t ld_out,
                  hipStream_t st) {
    const uint32_t pieces = (uint32_t)((dim + 7) / 8);
    LookupArgs a = {table, scales, ids, out, rows, dim, ld_table, first, ld_out, scale, id_bytes,
                    log_block, 0, divisor(pieces)};
    // launches of at most 2^30 lanes: the division's range
    const int64_t some = (1 << 30) / pieces;
    const int64_t ob = dtype_bytes(out_dtype);
    for (int64_t t = 0; t < tokens; t += some) {
        const int64_t n = tokens - t < some ? tokens - t : some;
        a.ids = static_cast<const char*>(ids) + t * id_bytes;
        a.out = static_cast<char*>(out) + t * ld_out * ob;
        a.lanes = (uint32_t)(n * pieces);
        if (t_dtype == ZPQ_F32) launch_lookup_o<ZPQ_F32>(a, out_dtype, st);
        else if (t_dtype == ZPQ_F16) launch_lookup_o<ZPQ_F16>(a, out_dtype, st);
        else if (t_dtype == ZPQ_BF16) launch_lookup_o<ZPQ_BF16>(a, out_dtype, st);
        else launch_lookup_o<kI8>(a, out_dtype, st);
    }
    return after_launch();
}

struct GradWorkspace {
    int64_t sorted[2], part[kMaxLevels], bytes;
    int32_t levels;
};

// Levels are used from where a row could hold a whole group and more: 2 groups
// of tokens.
inline GradWorkspace grad_workspace(int64_t tokens, int64_t dim) {
    GradWorkspace w = {};
    const int64_t list = (tokens * 8 + 255) / 256 * 256;
    w.sorted[0] = 0;
    w.sorted[1] = list;
    w.bytes = 2 * list;
    for (int l = 1; l <= kMaxLevels && (tokens >> (kGroupLog * l)) >= 2; ++l) {
        w.part[l - 1] = w.bytes;
        w.bytes += ((tokens >> (kGroupLog * l)) * dim * 4 + 255) / 256 * 256;
        w.levels = l;
    }
    return w;
}

template <int DT>
void launch_groups(const GradArgs& a, hipStream_t st) {
    const uint32_t pieces = (uint32_t)((a.dim + 7) / 8);
    for (int l = 1; l <= a.levels; ++l) {
        const uint32_t lanes = (a.tokens >> (kGroupLog * l)) * pieces;
        const dim3 grid((lanes + kThreads - 1) / kThreads);
        if (l == 1)
            hipLaunchKernelGGL((k_group_sums<DT, true>), grid, dim3(kThreads), 0, st, a, l, lanes,
                               divisor(pieces));
        else
            hipLaunchKernelGGL((k_group_sums<DT, false>), grid, dim3(kThreads), 0, st, a, l, lanes,
                               divisor(pieces));
    }
}
template <int DT, int OT>
void launch_rows(const GradArgs& a, bool add, hipStream_t st) {
    const dim3 grid((unsigned)((a.rows + kRows - 1) / kRows));
    const Divisor pieces = divisor((uint32_t)((a.dim + 7) / 8));
    if (add)
        hipLaunchKernelGGL((k_row_sums<DT, OT, true>), grid, dim3(kThreads), 0, st, a, pieces);
    else
        hipLaunchKernelGGL((k_row_sums<DT, OT, false>), grid, dim3(kThreads), 0, st, a, pieces);
}
template <int DT>
void launch_grad(const GradArgs& a, int32_t grad_dtype, bool add, hipStream_t st) {
    launch_groups<DT>(a, st);
    if (grad_dtype == ZPQ_F32) launch_rows<DT, ZPQ_F32>(a, add, st);
    else if (grad_dtype == ZPQ_F16) launch_rows<DT, ZPQ_F16>(a, add, st);
    else launch_rows<DT, ZPQ_BF16>(a, add, st);
}

// A launch holds less than 2^32 work-items, kLanes a token and kThreads for
// kRows rows; rows of pieces and groups of pieces are counted in 31 bits.
bool grad_sizes_ok(int64_t tokens, int64_t dim, int64_t rows) {
    return tokens >= 0 && tokens <= (1LL << 28) && dim >= 1 && dim <= (1 << 28) && rows <= (1LL << 27) &&
           (tokens >> kGroupLog) * ((dim + 7) / 8) < (1LL << 31) && kRows * ((dim + 7) / 8) < (1LL << 31);
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
    return lookup(table, t_dtype, nullptr, 0, rows, dim, ld_table, ids, id_bytes, tokens, first, scale, out,
                  out_dtype, ld_out, static_cast<hipStream_t>(stream));
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
    return lookup(codes, kI8, scales, log_block, rows, dim, dim, ids, id_bytes, tokens, first, scale, out,
                  out_dtype, ld_out, static_cast<hipStream_t>(stream));
}

zpq_status zpq_embedding_grad_bytes(int64_t tokens, int64_t dim, int64_t* bytes) {
    if (!bytes) return ZPQ_ERR_NULL;
    if (!grad_sizes_ok(tokens, dim, 0)) return ZPQ_ERR_SIZE;
    *bytes = grad_workspace(tokens, dim).bytes;
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
    const GradWorkspace w = grad_workspace(tokens, dim);
    if (!grad || (tokens > 0 && (!dy || !ids || !workspace))) return ZPQ_ERR_NULL;
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
    uint64_t* list = reinterpret_cast<uint64_t*>(ws + w.sorted[0]);
    uint64_t* other = reinterpret_cast<uint64_t*>(ws + w.sorted[1]);
    const uint32_t n = (uint32_t)tokens;
    uint32_t run = 1024;
    if (n > 0 && n <= 256) {
        hipLaunchKernelGGL((k_sort_tile<256, 128>), dim3(1), dim3(128), 0, st, ids, id_bytes, n, first, padding,
                           rows, list);
    } else if (n > 0 && n <= 1024 * kFan) {
        hipLaunchKernelGGL((k_sort_tile<1024, 512>), dim3((n + 1023) / 1024), dim3(512), 0, st, ids, id_bytes, n,
                           first, padding, rows, list);
    } else if (n > 0) {
        run = 4096;
        hipLaunchKernelGGL((k_sort_tile<4096, 1024>), dim3((n + 4095) / 4096), dim3(1024), 0, st, ids, id_bytes, n,
                           first, padding, rows, list);
    }
    for (uint64_t r = run; r < n; r *= kFan) {
        const uint64_t lanes = (uint64_t)n * kLanes;
        hipLaunchKernelGGL(k_merge, dim3((unsigned)((lanes + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                           list, n, (uint32_t)r, other);
        uint64_t* t = list;
        list = other;
        other = t;
    }
    GradArgs a = {list, dy, grad, {}, ld_dy, ld_grad, dim, rows, n, w.levels, scale};
    for (int l = 0; l < w.levels; ++l) a.part[l] = reinterpret_cast<float*>(ws + w.part[l]);
    if (dy_dtype == ZPQ_F32) launch_grad<ZPQ_F32>(a, grad_dtype, accumulate != 0, st);
    else if (dy_dtype == ZPQ_F16) launch_grad<ZPQ_F16>(a, grad_dtype, accumulate != 0, st);
    else launch_grad<ZPQ_BF16>(a, grad_dtype, accumulate != 0, st);
    return after_launch();
}

}  // extern "C"
