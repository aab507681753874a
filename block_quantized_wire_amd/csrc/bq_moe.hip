// bq_moe.hip -- tokens sorted by expert, their rows out and back, and both gradients.
//
// The order.  A slot is one (token, choice) pair; the sort is a stable counting sort of the
// slots by expert id, ids outside [0, E) counted as a bucket E of their own at the end.
// Every block of slots counts its ids, takes the counts of all blocks for where its share
// of each bucket starts, and places its slots: within a wave the rank of a slot among the
// equal ids before it comes from ballots over the id's bits, so the order is the slot
// order and no atomic decides it.
//
// Measured on MI355X: 16384 tokens x 8 choices over 256 experts (64 workgroups of 2048 slots)
// sort in 12 us, 28 before eight ids were asked for at a time; 256 slots in 3.3 us, one
// workgroup.  Bound by the latency of its steps, not by its 1.5 MB.
//
// The rows.  gather and combine move whole rows: a token's row out to its topk sorted rows,
// and the topk rows back into a weighted sum.  Both are streams bound by memory: a thread
// takes one 16-byte unit of a token's columns for all of its slots, so the token's side is
// read (written) once; the units of all tokens are dealt out evenly, whatever the width.
// Measured on MI355X (a large copy reaches 4.9 TB/s): gather of 16384 x 7168 bf16 rows to
// 4 slots each 199 us (5.9 TB/s, the rows of x coming from the last-level cache in part),
// combine of 8 rows of 7168 for 16384 tokens 405 us (5.2 TB/s; 448 before the rows of four
// slots were asked for at once), its gradient for 8192 x 8 rows of 4096 217 us (4.9 TB/s).
// Rows may start anywhere their type allows: gfx950 loads and stores unaligned vectors in
// hardware, and the last unit of a row falls back to single values.  Unaligned rows cost a
// third more (rows of 2055 binary16 values 36.8 us, of 2056 27.3); units of 8 or 4 bytes cost
// more yet (37.8 and 47.2).
#include "bq_device.h"
#include "bq_launch.h"

namespace bq {

namespace {

// ---- sort -------------------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBuckets = 1024 + 1;

struct SortArgs {
    const int32_t* expert;
    int32_t* off;
    int32_t* src;
    int32_t* pos;
    int32_t* counts;     // [blocks][E + 1], where there is more than one block
    int32_t slots, E, per;   // slots per block
    int32_t blocks, bits;    // bits of a bucket number
};

// The buckets of 8 slots of a lane, `stride` apart from `s` on (-1 at or past `end`): all 8 ids are
// asked for before the first is used.
constexpr int kIds = 8;
__device__ __forceinline__ void load_buckets(const SortArgs& p, int s, int stride, int end,
                                             int e[kIds]) {
#pragma unroll
    for (int i = 0; i < kIds; ++i)
        e[i] = s + i * stride < end ? p.expert[s + i * stride] : 0;
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
        e[i] = (uint32_t)e[i] < (uint32_t)p.E ? e[i] : p.E;
        if (s + i * stride >= end)
            e[i] = -1;
    }
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs p) {
    __shared__ int count[kMaxBuckets];
    const int nb = p.E + 1;
    for (int e = threadIdx.x; e < nb; e += kSortThreads)
        count[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * p.per, hi = min(lo + p.per, p.slots);
    for (int s = lo + (int)threadIdx.x; s < hi; s += kIds * kSortThreads) {
        int e[kIds];
        load_buckets(p, s, kSortThreads, hi, e);
#pragma unroll
        for (int i = 0; i < kIds; ++i)
            if (e[i] >= 0)
                atomicAdd(&count[e[i]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nb; e += kSortThreads)
        p.counts[blockIdx.x * nb + e] = count[e];
}

__global__ __launch_bounds__(kSortThreads) void k_sort_place(SortArgs p) {
    __shared__ int next[kSortWaves][kMaxBuckets];   // counts, then the next row, per wave
    __shared__ int total[kMaxBuckets];              // over all blocks, then the bucket's first row
    __shared__ int part[kSortWaves];
    const int nb = p.E + 1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = lane; e < nb; e += 64)
        next[wave][e] = 0;
    __syncthreads();

    // this wave's run of the block's slots, and its counts
    const int lo = blockIdx.x * p.per, hi = min(lo + p.per, p.slots);
    const int run = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) & ~63;
    const int first = lo + wave * run, last = min(first + run, hi);
    for (int s = first + lane; s < last; s += kIds * 64) {
        int e[kIds];
        load_buckets(p, s, 64, last, e);
#pragma unroll
        for (int i = 0; i < kIds; ++i)
            if (e[i] >= 0)
                atomicAdd(&next[wave][e[i]], 1);
    }
    __syncthreads();

    // bucket totals, and the rows that earlier blocks take in each bucket
    for (int e = tid; e < nb; e += kSortThreads) {
        int sum = 0, before = 0;
        if (p.blocks > 1) {
#pragma unroll 8
            for (int b = 0; b < p.blocks; ++b) {
                const int v = p.counts[b * nb + e];
                before += b < (int)blockIdx.x ? v : 0;
                sum += v;
            }
        } else {
            for (int w = 0; w < kSortWaves; ++w)
                sum += next[w][e];
        }
        total[e] = sum;
        // each wave's first row, counted from the bucket's
        for (int w = 0; w < kSortWaves; ++w) {
            const int v = next[w][e];
            next[w][e] = before;
            before += v;
        }
    }
    __syncthreads();

    // exclusive prefix of the totals, 512 buckets at a time
    int carry = 0;
    for (int base = 0; base < nb; base += kSortThreads) {
        const int e = base + tid;
        const int v = e < nb ? total[e] : 0;
        int inc = v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            inc += lane >= d ? o : 0;
        }
        if (lane == 63)
            part[wave] = inc;
        __syncthreads();
        int pre = carry, all = carry;
        for (int w = 0; w < kSortWaves; ++w) {
            pre += w < wave ? part[w] : 0;
            all += part[w];
        }
        if (e < nb) {
            total[e] = pre + inc - v;
            if (blockIdx.x == 0)
                p.off[e] = pre + inc - v;
        }
        carry = all;
        __syncthreads();
    }

    // place: 64 slots of the wave's run at a time, in order
    for (int s0 = first; s0 < last; s0 += kIds * 64) {
        int e[kIds];
        load_buckets(p, s0 + lane, 64, last, e);
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int s = s0 + i * 64 + lane;
            if (s - lane >= last)
                break;
            uint64_t same = __ballot(e[i] >= 0);
            for (int b = 0; b < p.bits; ++b) {
                const bool bit = (e[i] >> b) & 1;
                const uint64_t m = __ballot(bit);
                same &= bit ? m : ~m;
            }
            if (e[i] >= 0) {
                const int rank = __popcll(same & ((1ull << lane) - 1));
                const int leader = __ffsll((unsigned long long)same) - 1;
                int row = 0;
                if (rank == 0)
                    row = atomicAdd(&next[wave][e[i]], __popcll(same));
                row = __shfl(row, leader) + total[e[i]] + rank;
                p.src[row] = s;
                p.pos[s] = row;
            }
        }
    }
}

// ---- rows ---------------------------------------------------------------------------------

constexpr int kThreads = 256;

// The element types: the values of one 32-bit word as binary32, and back.
struct Bf16 {
    uint16_t b;
};

template <typename E>
struct Values;
template <>
struct Values<Bf16> {
    static __device__ __forceinline__ void open(uint32_t w, float f[2]) {
        f[0] = bf16_lo(w);
        f[1] = bf16_hi(w);
    }
    static __device__ __forceinline__ uint32_t close(const float f[2]) {
        return pack_bf16x2(f[0], f[1]);
    }
};
template <>
struct Values<_Float16> {
    static __device__ __forceinline__ void open(uint32_t w, float f[2]) {
        const h16x2 h = __builtin_bit_cast(h16x2, w);
        f[0] = (float)h.x;
        f[1] = (float)h.y;
    }
    static __device__ __forceinline__ uint32_t close(const float f[2]) {
        // The binary32 value is rounded to binary16, as the definitions say.  Left to itself the
        // compiler folds a product into a mixed-precision instruction that rounds the exact
        // product once; the empty asm keeps the two roundings apart.
        float a = f[0], b = f[1];
        asm("" : "+v"(a), "+v"(b));
        return __builtin_bit_cast(uint32_t, h16x2{(_Float16)a, (_Float16)b});
    }
};
template <>
struct Values<float> {
    static __device__ __forceinline__ void open(uint32_t w, float f[1]) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t close(const float f[1]) {
        return __float_as_uint(f[0]);
    }
};

// A unit of a row: 16 bytes, loaded from and stored to any address that suits the element.
constexpr int kUnitBytes = 16, kUnitWords = kUnitBytes / 4;
struct Unit {
    uint32_t w[kUnitWords];
};
typedef uint32_t LooseUnit __attribute__((ext_vector_type(4), aligned(2)));

template <typename E>
__device__ __forceinline__ void open(const Unit& u, float* f) {
#pragma unroll
    for (int i = 0; i < kUnitWords; ++i)
        Values<E>::open(u.w[i], f + i * (4 / sizeof(E)));
}
template <typename E>
__device__ __forceinline__ Unit close(const float* f) {
    Unit u;
#pragma unroll
    for (int i = 0; i < kUnitWords; ++i)
        u.w[i] = Values<E>::close(f + i * (4 / sizeof(E)));
    return u;
}

// One unit of a row, `n` of its values inside the row (the others read as zero).
template <typename E>
__device__ __forceinline__ Unit load(const E* p, int n) {
    constexpr int V = kUnitBytes / sizeof(E);
    if (n >= V)
        return __builtin_bit_cast(Unit, *reinterpret_cast<const LooseUnit*>(p));
    struct {
        E v[V];
    } u{};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            u.v[i] = p[i];
    return __builtin_bit_cast(Unit, u);
}

template <typename E>
__device__ __forceinline__ void store(E* p, const Unit& u, int n) {
    constexpr int V = kUnitBytes / sizeof(E);
    if (n >= V) {
        *reinterpret_cast<LooseUnit*>(p) = __builtin_bit_cast(LooseUnit, u);
        return;
    }
    struct Parts {
        E v[V];
    };
    const Parts v = __builtin_bit_cast(Parts, u);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            p[i] = v.v[i];
}

struct RowArgs {
    const void* in;        // gather: x; combine: rows; combine_bwd: rows
    const void* dy;        // combine_bwd
    void* out;             // gather: out; combine: y; combine_bwd: drows
    const int32_t* pos;
    const int32_t* off;
    const float* weight;
    float* dweight;
    int64_t ldi, ldd, ldo;
    int32_t topk, E, slots;
    int32_t cols;
    uint32_t per_row;      // units of a row, the last one perhaps partial
    uint64_t units;        // ... of all tokens
    uint64_t recip;        // ceil(2^64 / per_row)
};

// The token and the first column of unit `at`.  floor(at * ceil(2^64 / d) / 2^64) is at / d
// for at * d < 2^64, and there are less than 2^44 units (a tensor spans at most 2^48 bytes) of
// at most 2^20 in a row.
template <int V>
__device__ __forceinline__ int64_t token_of(const RowArgs& p, uint64_t at, int& col) {
    const uint64_t t = p.per_row == 1 ? at : __umul64hi(at, p.recip);
    col = (int)(uint32_t)(at - t * p.per_row) * V;
    return (int64_t)t;
}

// Slots are taken four at a time: their rows' addresses, then their rows, are all asked for
// before the first is used.
constexpr int kBatch = 4;

template <typename E>
__global__ __launch_bounds__(kThreads) void k_gather(RowArgs p) {
    constexpr int V = kUnitBytes / sizeof(E);
    const int kept = p.off[p.E];
    for (uint64_t at = blockIdx.x * (uint64_t)kThreads + threadIdx.x; at < p.units;
         at += gridDim.x * (uint64_t)kThreads) {
        int c;
        const int64_t t = token_of<V>(p, at, c);
        const int n = p.cols - c;
        const int32_t* pos = p.pos + t * p.topk;
        const Unit u = load(static_cast<const E*>(p.in) + t * p.ldi + c, n);
        for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
            int row[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                row[j] = j0 + j < p.topk ? pos[j0 + j] : -1;
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if ((uint32_t)row[j] < (uint32_t)p.slots)
                    store(static_cast<E*>(p.out) + row[j] * p.ldo + c,
                          row[j] < kept ? u : Unit{}, n);
        }
    }
}

template <typename E, bool W>
__global__ __launch_bounds__(kThreads) void k_combine(RowArgs p) {
    constexpr int V = kUnitBytes / sizeof(E);
    const uint32_t kept = (uint32_t)max(min(p.off[p.E], p.slots), 0);
    for (uint64_t at = blockIdx.x * (uint64_t)kThreads + threadIdx.x; at < p.units;
         at += gridDim.x * (uint64_t)kThreads) {
        int c;
        const int64_t t = token_of<V>(p, at, c);
        const int n = p.cols - c;
        const int64_t s0 = t * p.topk;
        float acc[V] = {};
        for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
            bool live[kBatch];
            Unit u[kBatch];
            float w[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int row = j0 + j < p.topk ? p.pos[s0 + j0 + j] : -1;
                live[j] = (uint32_t)row < kept;
                w[j] = W && live[j] ? p.weight[s0 + j0 + j] : 1.0f;
                // a dropped slot's row is left unread: its unit stays zero
                u[j] = Unit{};
                if (live[j])
                    u[j] = load(static_cast<const E*>(p.in) + row * p.ldi + c, n);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                float f[V];
                open<E>(u[j], f);
                if (live[j]) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        acc[i] += w[j] * f[i];
                }
            }
        }
        store(static_cast<E*>(p.out) + t * p.ldo + c, close<E>(acc), n);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// One workgroup for one slot: its row's dot product with dy ends in LDS.  It has 256, 128 or 64
// threads, by the units of a row, so that short rows leave few of them idle.
template <typename E>
__global__ __launch_bounds__(kThreads) void k_combine_bwd(RowArgs p) {
    constexpr int V = kUnitBytes / sizeof(E);
    __shared__ float part[kThreads / 64];
    const uint32_t kept = (uint32_t)max(min(p.off[p.E], p.slots), 0);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t s = blockIdx.x; s < p.slots; s += gridDim.x) {
        const int64_t t = s / p.topk;
        const int row = p.pos[s];
        const bool live = (uint32_t)row < kept;
        const bool mine = (uint32_t)row < (uint32_t)p.slots;
        const float w = live ? p.weight[s] : 0.0f;
        float dot = 0.0f;
        for (int c = (int)threadIdx.x * V; c < p.cols; c += (int)blockDim.x * V) {
            const int n = p.cols - c;
            Unit d{};
            if (live) {
                float g[V], u[V];
                open<E>(load(static_cast<const E*>(p.dy) + t * p.ldd + c, n), g);
                open<E>(load(static_cast<const E*>(p.in) + row * p.ldi + c, n), u);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot += u[i] * g[i];
                    g[i] = w * g[i];
                }
                d = close<E>(g);
            }
            if (mine)
                store(static_cast<E*>(p.out) + row * p.ldo + c, d, n);
        }
        dot = wave_sum(dot);
        if (lane == 0)
            part[wave] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = part[0];
            for (uint32_t i = 1; i < blockDim.x / 64; ++i)
                sum += part[i];
            p.dweight[s] = sum;
        }
        __syncthreads();
    }
}

RowArgs row_args(const MoeRows& r) {
    RowArgs a{};
    a.pos = r.pos;
    a.off = r.off;
    a.topk = r.topk;
    a.E = r.experts;
    a.slots = (int32_t)(r.tokens * r.topk);
    a.cols = (int32_t)r.cols;
    return a;
}

// Most workgroups of one launch (a launch holds less than 2^32 threads); beyond it they walk on.
constexpr int64_t kMaxGrid = 1 << 22;

dim3 grid_of(int64_t groups) { return dim3((unsigned)(groups < kMaxGrid ? groups : kMaxGrid)); }

// The grid over all tokens' units.
template <typename E>
dim3 rows_grid(RowArgs& a, int64_t tokens) {
    constexpr int V = kUnitBytes / (int)sizeof(E);
    a.per_row = (uint32_t)((a.cols + V - 1) / V);
    a.units = (uint64_t)tokens * a.per_row;
    a.recip = ~(uint64_t)0 / a.per_row + 1;
    return grid_of((int64_t)((a.units + kThreads - 1) / kThreads));
}

template <typename E>
hipError_t gather(RowArgs a, int64_t tokens, hipStream_t st) {
    const dim3 grid = rows_grid<E>(a, tokens);
    return launch1(k_gather<E>, grid, dim3(kThreads), st, a);
}

template <typename E>
hipError_t combine(RowArgs a, int64_t tokens, hipStream_t st) {
    const dim3 grid = rows_grid<E>(a, tokens);
    return a.weight ? launch1(k_combine<E, true>, grid, dim3(kThreads), st, a)
                    : launch1(k_combine<E, false>, grid, dim3(kThreads), st, a);
}

template <typename E>
hipError_t combine_bwd(RowArgs a, hipStream_t st) {
    constexpr int V = kUnitBytes / (int)sizeof(E);
    const int units = (a.cols + V - 1) / V;
    const dim3 threads(units > 128 ? 256 : units > 64 ? 128 : 64);
    return launch1(k_combine_bwd<E>, grid_of(a.slots), threads, st, a);
}

}  // namespace

hipError_t launch_moe_sort(const int32_t* expert, int64_t slots, int experts, int32_t* off,
                           int32_t* src, int32_t* pos, void* ws, hipStream_t stream) {
    SortArgs a{};
    a.expert = expert;
    a.off = off;
    a.src = src;
    a.pos = pos;
    a.counts = static_cast<int32_t*>(ws);
    a.slots = (int32_t)slots;
    a.E = experts;
    while ((1 << a.bits) < experts + 1)
        ++a.bits;
    if (slots <= kMoeSortOneBlock) {
        a.per = (int32_t)slots;
        a.blocks = 1;
        return launch1(k_sort_place, dim3(1), dim3(kSortThreads), stream, a);
    }
    // at most kMoeSortBlocks blocks of at least 2048 slots
    int64_t per = (slots + kMoeSortBlocks - 1) / kMoeSortBlocks;
    per = per < 2048 ? 2048 : (per + 511) / 512 * 512;
    a.per = (int32_t)per;
    a.blocks = (int32_t)((slots + per - 1) / per);
    const hipError_t e =
        launch1(k_sort_count, dim3((unsigned)a.blocks), dim3(kSortThreads), stream, a);
    if (e != hipSuccess)
        return e;
    return launch1(k_sort_place, dim3((unsigned)a.blocks), dim3(kSortThreads), stream, a);
}

hipError_t launch_moe_gather(const MoeRows& r, const void* x, int64_t ldx, int esize, void* out,
                             int64_t ldo, hipStream_t stream) {
    RowArgs a = row_args(r);
    a.in = x;
    a.ldi = ldx;
    a.out = out;
    a.ldo = ldo;
    return esize == 2 ? gather<uint16_t>(a, r.tokens, stream) : gather<uint32_t>(a, r.tokens, stream);
}

hipError_t launch_moe_combine(const MoeRows& r, MoeType type, const void* rows, int64_t ldr,
                              const float* weight, void* y, int64_t ldy, hipStream_t stream) {
    RowArgs a = row_args(r);
    a.in = rows;
    a.ldi = ldr;
    a.weight = weight;
    a.out = y;
    a.ldo = ldy;
    return type == MoeType::kBf16 ? combine<Bf16>(a, r.tokens, stream)
         : type == MoeType::kF16  ? combine<_Float16>(a, r.tokens, stream)
                                  : combine<float>(a, r.tokens, stream);
}

hipError_t launch_moe_combine_bwd(const MoeRows& r, MoeType type, const void* dy, int64_t lddy,
                                  const void* rows, int64_t ldr, const float* weight, void* drows,
                                  int64_t lddr, float* dweight, hipStream_t stream) {
    RowArgs a = row_args(r);
    a.in = rows;
    a.ldi = ldr;
    a.dy = dy;
    a.ldd = lddy;
    a.weight = weight;
    a.out = drows;
    a.ldo = lddr;
    a.dweight = dweight;
    return type == MoeType::kBf16 ? combine_bwd<Bf16>(a, stream)
         : type == MoeType::kF16  ? combine_bwd<_Float16>(a, stream)
                                  : combine_bwd<float>(a, stream);
}

}  // namespace bq
