// bq_moe.hip -- tokens sorted by expert, their rows out and back, and both gradients.
//
// The order.  A slot is one (token, choice) pair; the sort is a stable counting sort of the
// slots by expert id, ids outside [0, E) counted as a bucket E of their own at the end.
// Every block of slots counts its ids, takes the counts of all blocks for where its share
// of each bucket starts, and places its slots: within a wave the rank of a slot among the
// equal ids before it comes from ballots over the id's bits, so the order is the slot
// order and no atomic decides it.
//
// The rows.  gather and combine move whole rows: a token's row out to its topk sorted rows,
// and the topk rows back into a weighted sum.  Both are streams bound by memory: a thread
// takes one 16-byte unit of a token's columns for all of its slots, so the token's side is
// read (written) once.  Rows may start anywhere their type allows: gfx950 loads and stores
// unaligned vectors in hardware, and the last unit of a row falls back to single values.
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

__device__ __forceinline__ int bucket_of(const SortArgs& p, int slot) {
    const int e = p.expert[slot];
    return (uint32_t)e < (uint32_t)p.E ? e : p.E;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortArgs p) {
    __shared__ int count[kMaxBuckets];
    const int nb = p.E + 1;
    for (int e = threadIdx.x; e < nb; e += kSortThreads)
        count[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * p.per, hi = min(lo + p.per, p.slots);
    for (int s = lo + (int)threadIdx.x; s < hi; s += kSortThreads)
        atomicAdd(&count[bucket_of(p, s)], 1);
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
    for (int i = tid; i < kSortWaves * kMaxBuckets; i += kSortThreads)
        next[i / kMaxBuckets][i % kMaxBuckets] = 0;
    __syncthreads();

    // this wave's run of the block's slots, and its counts
    const int lo = blockIdx.x * p.per, hi = min(lo + p.per, p.slots);
    const int run = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) & ~63;
    const int first = lo + wave * run, last = min(first + run, hi);
    for (int s = first + lane; s < last; s += 64)
        atomicAdd(&next[wave][bucket_of(p, s)], 1);
    __syncthreads();

    // bucket totals, and the rows that earlier blocks take in each bucket
    for (int e = tid; e < nb; e += kSortThreads) {
        int sum = 0, before = 0;
        if (p.blocks > 1) {
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
    for (int s0 = first; s0 < last; s0 += 64) {
        const int s = s0 + lane;
        const bool on = s < last;
        const int e = on ? bucket_of(p, s) : 0;
        uint64_t same = __ballot(on);
        for (int b = 0; b < p.bits; ++b) {
            const bool bit = (e >> b) & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        if (on) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int leader = __ffsll((unsigned long long)same) - 1;
            int row = 0;
            if (rank == 0)
                row = atomicAdd(&next[wave][e], __popcll(same));
            row = __shfl(row, leader) + total[e] + rank;
            p.src[row] = s;
            p.pos[s] = row;
        }
    }
}

// ---- rows ---------------------------------------------------------------------------------

constexpr int kThreads = 256;

// The element types: values per 16-byte unit, and a unit's values as binary32 and back.
struct Bf16 {
    uint16_t b;
};

template <typename E>
struct Values;
template <>
struct Values<Bf16> {
    static constexpr int kCount = 8;
    static __device__ __forceinline__ void open(u32x4 w, float f[8]) { unpack_bf16x8(w, f); }
    static __device__ __forceinline__ u32x4 close(const float f[8]) { return pack_bf16x8(f); }
};
template <>
struct Values<_Float16> {
    static constexpr int kCount = 8;
    static __device__ __forceinline__ void open(u32x4 w, float f[8]) { unpack_f16x8(w, f); }
    static __device__ __forceinline__ u32x4 close(const float f[8]) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // The binary32 value is rounded to binary16, as the definitions say.  Left to itself
            // the compiler folds a product into a mixed-precision instruction that rounds the
            // exact product once; the empty asm keeps the two roundings apart.
            float a = f[2 * i], b = f[2 * i + 1];
            asm("" : "+v"(a), "+v"(b));
            w[i] = __builtin_bit_cast(uint32_t, h16x2{(_Float16)a, (_Float16)b});
        }
        return w;
    }
};
template <>
struct Values<float> {
    static constexpr int kCount = 4;
    static __device__ __forceinline__ void open(u32x4 w, float f[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ u32x4 close(const float f[4]) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
    }
};

// A 16-byte vector at any address that suits the element.
template <int Bytes>
struct Loose;
template <>
struct Loose<2> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Loose<4> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};

// One 16-byte unit of a row, `n` of its values inside the row (the others read as zero).
template <typename E>
__device__ __forceinline__ u32x4 load(const E* p, int n) {
    constexpr int V = 16 / sizeof(E);
    if (n >= V)
        return *reinterpret_cast<const typename Loose<sizeof(E)>::type*>(p);
    struct {
        E v[V];
    } u{};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            u.v[i] = p[i];
    return __builtin_bit_cast(u32x4, u);
}

template <typename E>
__device__ __forceinline__ void store(E* p, u32x4 w, int n) {
    constexpr int V = 16 / sizeof(E);
    if (n >= V) {
        *reinterpret_cast<typename Loose<sizeof(E)>::type*>(p) = w;
        return;
    }
    struct Parts {
        E v[V];
    };
    const Parts u = __builtin_bit_cast(Parts, w);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            p[i] = u.v[i];
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
    uint32_t per_token;    // workgroups' worth of columns of one token
    int64_t groups;        // ... of all tokens
};

template <typename E>
__global__ __launch_bounds__(kThreads) void k_gather(RowArgs p) {
    constexpr int V = 16 / sizeof(E);
    const int kept = p.off[p.E];
    for (int64_t b = blockIdx.x; b < p.groups; b += gridDim.x) {
        const int64_t t = b / p.per_token;
        const int c = (int)((b - t * p.per_token) * kThreads + threadIdx.x) * V;
        if (c >= p.cols)
            continue;
        const int n = p.cols - c;
        const int32_t* pos = p.pos + t * p.topk;
        const u32x4 u = load(static_cast<const E*>(p.in) + t * p.ldi + c, n);
        for (int j = 0; j < p.topk; ++j) {
            const int row = pos[j];
            if ((uint32_t)row < (uint32_t)p.slots)
                store(static_cast<E*>(p.out) + row * p.ldo + c, row < kept ? u : u32x4{}, n);
        }
    }
}

template <typename E, bool W>
__global__ __launch_bounds__(kThreads) void k_combine(RowArgs p) {
    constexpr int V = Values<E>::kCount;
    const uint32_t kept = (uint32_t)max(min(p.off[p.E], p.slots), 0);
    for (int64_t b = blockIdx.x; b < p.groups; b += gridDim.x) {
        const int64_t t = b / p.per_token;
        const int c = (int)((b - t * p.per_token) * kThreads + threadIdx.x) * V;
        if (c >= p.cols)
            continue;
        const int n = p.cols - c;
        const int64_t s0 = t * p.topk;
        float acc[V] = {};
        for (int j = 0; j < p.topk; ++j) {
            const int row = p.pos[s0 + j];
            if ((uint32_t)row >= kept)
                continue;
            float f[V];
            Values<E>::open(load(static_cast<const E*>(p.in) + row * p.ldi + c, n), f);
            const float w = W ? p.weight[s0 + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] += w * f[i];
        }
        store(static_cast<E*>(p.out) + t * p.ldo + c, Values<E>::close(acc), n);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

template <typename E>
__global__ __launch_bounds__(kThreads) void k_combine_bwd(RowArgs p) {
    constexpr int V = Values<E>::kCount;
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
        for (int c = (int)threadIdx.x * V; c < p.cols; c += kThreads * V) {
            const int n = p.cols - c;
            u32x4 d{};
            if (live) {
                float g[V], u[V];
                Values<E>::open(load(static_cast<const E*>(p.dy) + t * p.ldd + c, n), g);
                Values<E>::open(load(static_cast<const E*>(p.in) + row * p.ldi + c, n), u);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot += u[i] * g[i];
                    g[i] = w * g[i];
                }
                d = Values<E>::close(g);
            }
            if (mine)
                store(static_cast<E*>(p.out) + row * p.ldo + c, d, n);
        }
        dot = wave_sum(dot);
        if (lane == 0)
            part[wave] = dot;
        __syncthreads();
        if (threadIdx.x == 0)
            p.dweight[s] = (part[0] + part[1]) + (part[2] + part[3]);
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

// Most workgroups of one launch (a launch holds less than 2^32 threads); beyond it the
// workgroups walk on.
constexpr int64_t kMaxGrid = 1 << 22;

dim3 grid_of(int64_t groups) { return dim3((unsigned)(groups < kMaxGrid ? groups : kMaxGrid)); }

// The grid over all tokens' columns, 256 units of 16 bytes to a workgroup.
template <typename E>
dim3 rows_grid(RowArgs& a, int64_t tokens) {
    constexpr int64_t per = kThreads * (16 / (int64_t)sizeof(E));
    a.per_token = (uint32_t)((a.cols + per - 1) / per);
    a.groups = tokens * a.per_token;
    return grid_of(a.groups);
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
    const dim3 grid = grid_of(a.slots);
    return type == MoeType::kBf16 ? launch1(k_combine_bwd<Bf16>, grid, dim3(kThreads), stream, a)
         : type == MoeType::kF16  ? launch1(k_combine_bwd<_Float16>, grid, dim3(kThreads), stream, a)
                                  : launch1(k_combine_bwd<float>, grid, dim3(kThreads), stream, a);
}

}  // namespace bq
