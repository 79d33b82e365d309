// mx_moe.cu -- tokens sorted by expert and back, on B200 (sm_100a): the sort
// of (token, choice) slots by expert, the copy of token rows into expert
// order, and the weighted sum of a token's rows with its gradient.
//
// All of it is bound by memory (the sort, for few tokens, by latency).  The
// row kernels go by token, not by sorted row: a token's row is then read once
// from HBM and written `choices` times (dispatch), or its `choices` rows are
// read and one written (combine); by sorted row a token's row would be read
// `choices` times, far apart.  Sums run in 32 bits in the order of a token's
// choices, with no atomics, so every call gives the same bits.
//
// On a B200, 16384 tokens x 8 choices x 7168 bf16: dispatch 330 us (6.4 TB/s),
// combine 355 us (5.9 TB/s), its gradient 608 us (6.6 TB/s); a copy of those rows
// runs at 6.6 TB/s.  16 tokens: 2.3, 2.5 and 5.1 us.

#include <climits>

#include "mx_ops.cuh"

namespace mx {
namespace {

// ------------------------------------------------------------------ sort
// A stable counting sort of S slots by expert (E <= 64).  A CTA takes one
// contiguous range of slots, each of its warps a contiguous part of that, 32
// slots a step.  Within a step match_any gives each slot the lanes with the
// same expert: the slot's rank is the number of lower ones among them.
//   count:  per-warp counters, then (several CTAs) the CTA's sums to `counts`;
//   place:  a slot's row = expert's start + earlier CTAs + earlier warps +
//           earlier steps + rank in the step.
// One CTA does both in one launch up to kSortOneCta slots; above, two
// launches, because a CTA needs the counts of all earlier ones.  On a B200, 64
// experts: 2.8 us for 128 slots, 4.6 for 1024, 9.0 for 131072; 8192 slots take
// 17.2 us in one CTA and 8.2 in eight.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortOneCta = 2048;
constexpr int64_t kSortChunk = 1024;   // slots of a CTA, at least
constexpr int kSortMaxCtas = 148;

template <typename Id>
__device__ __forceinline__ int load_expert(const Id *ids, int64_t s, int64_t end, int E) {
    if (s >= end) return -1;
    const Id v = ids[s];
    return v >= 0 && v < (Id)E ? (int)v : -1;
}

struct SortShared {
    int warp[kSortWarps][kMaxGroups + 1]; // counts, then next row of the warp's slots
    int total[kMaxGroups];              // the CTA's counts
    int before[kMaxGroups];             // counts of earlier CTAs
    int all[kMaxGroups];                // counts of all CTAs
    int start[kMaxGroups + 1];
};

// Per-warp counts of slots [begin, end) in sh.warp.
template <typename Id>
__device__ __forceinline__ void sort_count(const Id *ids, int64_t begin, int64_t end, int64_t per_warp, int E,
                                           SortShared &sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    sh.warp[w][lane] = 0;
    sh.warp[w][lane + 32] = 0;
    __syncwarp();
    const int64_t from = begin + w * per_warp, to = min(end, from + per_warp);
    for (int64_t at = from; at < to; at += 32) {
        const int e = load_expert(ids, at + lane, to, E);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) sh.warp[w][e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

// Warp w turns the per-warp counts of experts w and w + 32 into exclusive sums
// over the warps, and leaves the CTA's count in sh.total.
__device__ __forceinline__ void sort_scan_warps(SortShared &sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = w + 32 * h;
        const int n = sh.warp[lane][e];
        const int sum = warp_scan_sum(n, lane);
        sh.warp[lane][e] = sum - n;
        if (lane == 31) sh.total[e] = sum;
    }
    __syncthreads();
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const Id *__restrict__ ids, int64_t S, int64_t per_cta, int64_t per_warp, int E, int *__restrict__ counts) {
    __shared__ SortShared sh;
    grid_dependency_wait();
    const int64_t begin = blockIdx.x * per_cta, end = min(S, begin + per_cta);
    sort_count(ids, begin, end, per_warp, E, sh);
    sort_scan_warps(sh);
    if (threadIdx.x < kMaxGroups) counts[blockIdx.x * kMaxGroups + threadIdx.x] = sh.total[threadIdx.x];
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const Id *__restrict__ ids, int64_t S, int64_t per_cta, int64_t per_warp, int E,
                  const int *__restrict__ counts, int *__restrict__ group_ends, int *__restrict__ row_of_slot,
                  int *__restrict__ slot_of_row) {
    __shared__ SortShared sh;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    grid_dependency_wait();
    const int64_t begin = blockIdx.x * per_cta, end = min(S, begin + per_cta);
    if (tid < kMaxGroups) sh.before[tid] = sh.all[tid] = 0;
    sort_count(ids, begin, end, per_warp, E, sh);
    sort_scan_warps(sh);
    if (counts != nullptr) {
        // 16 threads an expert add up the CTAs' counts
        const int e = tid & (kMaxGroups - 1);
        int before = 0, all = 0;
        for (int b = tid / kMaxGroups; b < (int)gridDim.x; b += kSortThreads / kMaxGroups) {
            const int n = counts[b * kMaxGroups + e];
            all += n;
            if (b < (int)blockIdx.x) before += n;
        }
        atomicAdd(&sh.before[e], before);   // whole numbers: the order does not matter
        atomicAdd(&sh.all[e], all);
    } else if (tid < kMaxGroups) {
        sh.all[tid] = sh.total[tid];
    }
    __syncthreads();
    if (w == 0) {
        const int n0 = sh.all[lane], n1 = sh.all[lane + 32];
        const int s0 = warp_scan_sum(n0, lane);
        const int s1 = warp_scan_sum(n1, lane) + __shfl_sync(0xffffffffu, s0, 31);
        sh.start[lane] = s0 - n0;
        sh.start[lane + 32] = s1 - n1;
        if (lane == 31) sh.start[kMaxGroups] = s1;
        if (blockIdx.x == 0) {
            if (lane < E) group_ends[lane] = s0;
            if (lane + 32 < E) group_ends[lane + 32] = s1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = lane + 32 * h;
        sh.warp[w][e] += sh.start[e] + sh.before[e];
    }
    __syncwarp();
    const int64_t from = begin + w * per_warp, to = min(end, from + per_warp);
    for (int64_t at = from; at < to; at += 32) {
        const int e = load_expert(ids, at + lane, to, E);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = sh.warp[w][e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) sh.warp[w][e] += __popc(same);
        __syncwarp();
        if (at + lane < to) {
            row_of_slot[at + lane] = row;
            // below S unless the ids or the workspace changed since they were counted
            if (row >= 0 && row < S) slot_of_row[row] = (int)(at + lane);
        }
    }
    // rows behind the last group
    for (int64_t r = sh.start[kMaxGroups] + (int64_t)blockIdx.x * kSortThreads + tid; r < S;
         r += (int64_t)gridDim.x * kSortThreads)
        slot_of_row[r] = -1;
}

// ------------------------------------------------------------------ rows
// A CTA of 256 threads takes 256 / tpr tokens and one chunk of their rows: kPacks
// packs a thread, tpr packs apart (tpr a power of two: the packs of a row, at
// most 256).  Chunks of a token are neighbours in the grid, so their rows are
// touched together.  A pack is 16 bytes, 8, 4, or one element, whichever all rows
// are aligned to; the copy of rows off 8-byte boundaries has a kernel of its own.
constexpr int kRowThreads = 256;

struct RowShape {
    int64_t tokens, rows;   // tokens; rows = tokens * choices
    int32_t k;              // choices a token
    int32_t packs;          // packs of a row
    int32_t tpr_log2;
    int32_t chunks;
};

// Packs of a thread that are in flight for each row: enough small loads, and
// enough of 16 bytes where a token has few rows.
constexpr int packs_of(int bytes, int ahead) { return bytes == 16 ? 8 / ahead : bytes == 8 ? 16 / ahead : ahead == 2 ? 8 : 4; }

template <typename P>
__device__ __forceinline__ void zero_rows(P *__restrict__ out, int64_t stride, int64_t from, const RowShape &s) {
    const int64_t n = (s.rows - from) * s.packs;
    P zero;
    memset(&zero, 0, sizeof(zero));
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kRowThreads) {
        const int64_t r = i / s.packs;
        out[(from + r) * stride + (i - r * s.packs)] = zero;
    }
}

// This thread's token and first pack.
template <int kPacks>
__device__ __forceinline__ void place_of(const RowShape &s, int64_t &t, int &p) {
    const int64_t slab = blockIdx.x / s.chunks;
    const int chunk = (int)(blockIdx.x - slab * s.chunks);
    t = (slab << (8 - s.tpr_log2)) + (threadIdx.x >> s.tpr_log2);
    p = chunk * (kPacks << s.tpr_log2) + (threadIdx.x & ((1 << s.tpr_log2) - 1));
}

// Rows off 8-byte boundaries, as elements of 16 bits (32-bit ones are two).  Loads
// are of whole words (one that holds a wanted element is always readable), shifted
// by an element where the row starts between two; stores are of 16 bytes from the
// row's first boundary on, so that no sector of a token's row is written in parts but
// at its ends.  48033 tokens x 4 x 2201 bf16: 235 us, element by element 393; 2202,
// 4-byte boundaries: 228, in packs of 4 bytes 260; 29144 x 1 x 2463: 87 and 145.  Rows
// behind the last group are still zeroed 4 or 2 bytes at a time: with half of those
// slots dropped the first takes 494 us, with seven of eight 725.

// Elements at .. at + 15 of a row; those past its `cols` are undefined.
__device__ __forceinline__ void load_sixteen(const uint16_t *row, int at, int cols, uint32_t (&w)[8]) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + at);
    const uint32_t *src = reinterpret_cast<const uint32_t *>(a & ~uintptr_t(3));
    const int odd = (int)(a >> 1 & 1);
    uint32_t last = 0;
    if (at + 16 <= cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ldg(src + i);
        if (odd) last = __ldg(src + 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = at - odd + 2 * i < cols ? __ldg(src + i) : 0u;
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(w[i], i < 7 ? w[i + 1] : last, 16);
    }
}
// Eight of them, from element `from` (0..7) on.
__device__ __forceinline__ uint4 eight_of(const uint32_t (&w)[8], int from) {
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = from & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) b[i] = from & 2 ? a[i + 1] : a[i];
    return from & 1 ? make_uint4(__funnelshift_r(b[0], b[1], 16), __funnelshift_r(b[1], b[2], 16),
                                 __funnelshift_r(b[2], b[3], 16), __funnelshift_r(b[3], b[4], 16))
                    : make_uint4(b[0], b[1], b[2], b[3]);
}

// dispatch_kernel for such rows: a thread holds 15 elements of the token's row at a
// time, of which each destination takes the eight that it stores as a whole.
constexpr int kDispatchPieces = 2;
template <typename P>
__global__ void __launch_bounds__(kRowThreads)
dispatch_elements_kernel(const uint16_t *__restrict__ x, int64_t x_stride, const int *__restrict__ row_of_slot,
                         const int *__restrict__ ends, int E, uint16_t *__restrict__ out, int64_t out_stride, int cols, RowShape s) {
    grid_dependency_wait();
    int64_t t;
    int p;
    place_of<kDispatchPieces>(s, t, p);
    if (t < s.tokens) {
        const int tpr = 1 << s.tpr_log2;
        uint32_t w[kDispatchPieces][8];
#pragma unroll
        for (int i = 0; i < kDispatchPieces; ++i)
            if (p + i * tpr < s.packs) load_sixteen(x + t * x_stride, (p + i * tpr) * 8, cols, w[i]);
        const int *rows = row_of_slot + t * s.k;
        for (int j = 0; j < s.k; ++j) {
            const int64_t r = rows[j];
            if (r < 0 || r >= s.rows) continue;
            uint16_t *row = out + r * out_stride;
            const int first = -(int)(reinterpret_cast<uintptr_t>(row) >> 1) & 7;   // elements before the row's first boundary
#pragma unroll
            for (int i = 0; i < kDispatchPieces; ++i) {
                if (p + i * tpr >= s.packs) break;
                const int at = (p + i * tpr) * 8 + first;
                const uint4 v = eight_of(w[i], first);
                if (at + 8 <= cols) {
                    *reinterpret_cast<uint4 *>(row + at) = v;
                } else {
                    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (at + u < cols) row[at + u] = (uint16_t)(e[u / 2] >> (16 * (u & 1)));
                }
                if (at == first) {   // the row's first elements
#pragma unroll
                    for (int u = 0; u < 7; ++u)
                        if (u < first && u < cols) row[u] = (uint16_t)(w[i][u / 2] >> (16 * (u & 1)));
                }
            }
        }
    }
    constexpr int kOfPack = sizeof(P) / 2;
    s.packs = cols / kOfPack;
    zero_rows(reinterpret_cast<P *>(out), out_stride / kOfPack, rows_in_groups(ends, E), s);
}

// out[row_of_slot[t, j]] = x[t]; rows behind the last group = 0.  Strides in packs.
constexpr int dispatch_packs(int bytes) { return 16 / bytes; }
template <typename P>
__global__ void __launch_bounds__(kRowThreads)
dispatch_kernel(const P *__restrict__ x, int64_t x_stride, const int *__restrict__ row_of_slot,
                const int *__restrict__ ends, int E, P *__restrict__ out, int64_t out_stride, RowShape s) {
    constexpr int kPacks = dispatch_packs(sizeof(P));
    grid_dependency_wait();
    int64_t t;
    int p;
    place_of<kPacks>(s, t, p);
    if (t < s.tokens) {
        const int tpr = 1 << s.tpr_log2;
        P v[kPacks];
#pragma unroll
        for (int i = 0; i < kPacks; ++i)
            if (p + i * tpr < s.packs) v[i] = x[t * x_stride + p + i * tpr];
        const int *rows = row_of_slot + t * s.k;
        for (int j = 0; j < s.k; ++j) {
            const int64_t r = rows[j];
            if (r < 0 || r >= s.rows) continue;
#pragma unroll
            for (int i = 0; i < kPacks; ++i)
                if (p + i * tpr < s.packs) out[r * out_stride + p + i * tpr] = v[i];
        }
    }
    zero_rows(out, out_stride, rows_in_groups(ends, E), s);
}

// y[t] = sum_j w[t, j] * rows[row_of_slot[t, j]] over the slots that have a row;
// kAhead rows' loads are in flight together.  Strides in packs.
template <typename T, int N, int kAhead>
__global__ void __launch_bounds__(kRowThreads)
combine_kernel(const Raw<T, N> *__restrict__ rows, int64_t rows_stride, const int *__restrict__ row_of_slot,
               const float *__restrict__ weights, Raw<T, N> *__restrict__ y, int64_t y_stride, RowShape s) {
    using P = Raw<T, N>;
    constexpr int kPacks = packs_of(sizeof(P), kAhead);
    grid_dependency_wait();
    int64_t t;
    int p;
    place_of<kPacks>(s, t, p);
    if (t >= s.tokens || p >= s.packs) return;
    const int tpr = 1 << s.tpr_log2;
    float sum[kPacks][N] = {};
    for (int j0 = 0; j0 < s.k; j0 += kAhead) {
        P v[kAhead][kPacks];
        float w[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t slot = t * s.k + j0 + u;
            const int64_t r = j0 + u < s.k ? row_of_slot[slot] : -1;
            live[u] = r >= 0 && r < s.rows;
            w[u] = 1.f;
            if (live[u]) {
#pragma unroll
                for (int i = 0; i < kPacks; ++i)
                    if (p + i * tpr < s.packs) v[u][i] = rows[r * rows_stride + p + i * tpr];
                if (weights != nullptr) w[u] = weights[slot];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (live[u]) {
#pragma unroll
                for (int i = 0; i < kPacks; ++i) {
                    float f[N];
                    unpack<T, N>(v[u][i], f);
#pragma unroll
                    for (int e = 0; e < N; ++e) sum[i][e] = fmaf(w[u], f[e], sum[i][e]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < kPacks; ++i)
        if (p + i * tpr < s.packs) y[t * y_stride + p + i * tpr] = pack<T, N>(sum[i]);
}

// d_rows[row_of_slot[t, j]] = w[t, j] * grad[t]; d_weights[t, j] = <grad[t], rows[...]>.
// kTpt threads take one token and walk its whole row, because the inner
// products run over it: a warp a token for short rows, a CTA for long ones.
template <typename T, int N, int kTpt, int kAhead>
__global__ void __launch_bounds__(kRowThreads)
combine_backward_kernel(const Raw<T, N> *__restrict__ grad, int64_t grad_stride, const Raw<T, N> *__restrict__ rows,
                        int64_t rows_stride, const int *__restrict__ row_of_slot, const int *__restrict__ ends, int E,
                        const float *__restrict__ weights, Raw<T, N> *__restrict__ d_rows, int64_t d_rows_stride,
                        float *__restrict__ d_weights, RowShape s) {
    using P = Raw<T, N>;
    constexpr int kPacks = packs_of(sizeof(P), kAhead);
    __shared__ float part[kRowThreads / 32][kAhead];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / kTpt) + threadIdx.x / kTpt;
    if (t < s.tokens) {   // the same for all threads of a warp, and of the CTA where it takes one token
        for (int j0 = 0; j0 < s.k; j0 += kAhead) {
            int64_t at[kAhead];
            float wt[kAhead], dot[kAhead];
            bool live[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t slot = t * s.k + j0 + u;
                const int64_t r = j0 + u < s.k ? row_of_slot[slot] : -1;
                live[u] = r >= 0 && r < s.rows;
                at[u] = r;
                wt[u] = live[u] ? weights[slot] : 0.f;
                dot[u] = 0.f;
            }
            for (int p = threadIdx.x % kTpt; p < s.packs; p += kTpt * kPacks) {
                P g[kPacks], v[kAhead][kPacks];
#pragma unroll
                for (int i = 0; i < kPacks; ++i)
                    if (p + i * kTpt < s.packs) g[i] = grad[t * grad_stride + p + i * kTpt];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (live[u]) {
#pragma unroll
                        for (int i = 0; i < kPacks; ++i)
                            if (p + i * kTpt < s.packs) v[u][i] = rows[at[u] * rows_stride + p + i * kTpt];
                    }
#pragma unroll
                for (int i = 0; i < kPacks; ++i) {
                    if (p + i * kTpt >= s.packs) break;
                    float gf[N];
                    unpack<T, N>(g[i], gf);
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (live[u]) {
                            float f[N], o[N];
                            unpack<T, N>(v[u][i], f);
#pragma unroll
                            for (int e = 0; e < N; ++e) {
                                dot[u] = fmaf(gf[e], f[e], dot[u]);
                                o[e] = wt[u] * gf[e];
                            }
                            d_rows[at[u] * d_rows_stride + p + i * kTpt] = pack<T, N>(o);
                        }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], d);
            }
            if (kTpt == 32) {
                if (lane == 0)
                    for (int u = 0; u < kAhead && j0 + u < s.k; ++u) d_weights[t * s.k + j0 + u] = dot[u];
            } else {
                __syncthreads();
                if (lane == 0) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) part[w][u] = dot[u];
                }
                __syncthreads();
                if (threadIdx.x < kAhead && j0 + threadIdx.x < s.k) {
                    float sum = 0.f;
                    for (int q = 0; q < kRowThreads / 32; ++q) sum += part[q][threadIdx.x];
                    d_weights[t * s.k + j0 + threadIdx.x] = sum;
                }
            }
        }
    }
    zero_rows(d_rows, d_rows_stride, rows_in_groups(ends, E), s);
}

// ------------------------------------------------------------------ host side
int64_t sort_ctas(int64_t S) {
    if (S <= kSortOneCta) return 1;
    const int64_t n = div_up(S, kSortChunk);
    return n < kSortMaxCtas ? n : kSortMaxCtas;
}

bool slots_ok(int64_t tokens, int32_t choices) {
    return tokens >= 0 && choices >= 1 && tokens <= kOpsMaxExtent && tokens * choices <= kOpsMaxExtent;
}

int element_bytes(mx_dtype t) {
    return t == MX_F32 ? 4 : t == MX_BF16 || t == MX_F16 ? 2 : 0;
}

template <typename Id>
mx_status sort_typed(const void *ids, int64_t S, int32_t E, int32_t *group_ends, int32_t *row_of_slot,
                     int32_t *slot_of_row, int32_t *workspace, cudaStream_t stream) {
    const int64_t ctas = sort_ctas(S);
    const int64_t per_warp = up_to(div_up(S, ctas * kSortWarps), 32);
    const int64_t per_cta = per_warp * kSortWarps;
    const Id *p = static_cast<const Id *>(ids);
    if (ctas > 1)
        if (mx_status st = launch(sort_count_kernel<Id>, ctas, kSortThreads, 0, stream, p, S, per_cta, per_warp, E, workspace);
            st != MX_OK)
            return st;
    return launch(sort_place_kernel<Id>, ctas, kSortThreads, 0, stream, p, S, per_cta, per_warp, E,
                  static_cast<const int *>(ctas > 1 ? workspace : nullptr), group_ends, row_of_slot, slot_of_row);
}

// Bytes of a pack: the most of 16, 8 and 4 that every row of every matrix starts on
// and is made of, else one element's.
struct Mat { const void *p; int64_t stride; };
template <int n>
int pack_bytes(int es, int64_t cols, const Mat (&m)[n]) {
    for (int bytes : {16, 8, 4}) {
        bool fits = cols * es % bytes == 0;
        for (const Mat &a : m) fits = fits && aligned_to(a.p, bytes) && a.stride * es % bytes == 0;
        if (fits) return bytes;
    }
    return es;
}

mx_status row_shape(int64_t tokens, int32_t choices, int64_t packs, int per_thread, RowShape *s, int64_t *grid) {
    s->tokens = tokens;
    s->rows = tokens * choices;
    s->k = choices;
    s->packs = (int32_t)packs;
    s->tpr_log2 = 0;
    while (s->tpr_log2 < 8 && (per_thread << s->tpr_log2) < packs) ++s->tpr_log2;
    s->chunks = (int32_t)div_up(packs, (int64_t)per_thread << s->tpr_log2);
    *grid = div_up(tokens, kRowThreads >> s->tpr_log2) * s->chunks;
    return *grid > INT_MAX ? MX_ERR_UNSUPPORTED : MX_OK;
}

template <typename P>
mx_status dispatch_typed(const void *x, int64_t x_bytes, const int32_t *row_of_slot, const int32_t *ends, int E, void *out,
                         int64_t out_bytes, int64_t tokens, int32_t choices, int64_t row_bytes, cudaStream_t stream) {
    constexpr int64_t n = sizeof(P);
    RowShape s;
    int64_t grid;
    if (mx_status st = row_shape(tokens, choices, row_bytes / n, dispatch_packs(n), &s, &grid); st != MX_OK) return st;
    return launch(dispatch_kernel<P>, grid, kRowThreads, 0, stream, static_cast<const P *>(x), x_bytes / n, row_of_slot,
                  ends, E, static_cast<P *>(out), out_bytes / n, s);
}

template <typename P>
mx_status dispatch_elements(const void *x, int64_t x_bytes, const int32_t *row_of_slot, const int32_t *ends, int E, void *out,
                            int64_t out_bytes, int64_t tokens, int32_t choices, int64_t row_bytes, cudaStream_t stream) {
    RowShape s;
    int64_t grid;
    if (mx_status st = row_shape(tokens, choices, div_up(row_bytes, 16), kDispatchPieces, &s, &grid); st != MX_OK) return st;
    return launch(dispatch_elements_kernel<P>, grid, kRowThreads, 0, stream, static_cast<const uint16_t *>(x), x_bytes / 2, row_of_slot,
                  ends, E, static_cast<uint16_t *>(out), out_bytes / 2, (int)(row_bytes / 2), s);
}

template <typename T, int N, int kAhead>
mx_status combine_typed(const void *rows, int64_t rows_stride, const int32_t *row_of_slot, const float *weights, void *y,
                        int64_t y_stride, int64_t tokens, int32_t choices, int64_t cols, cudaStream_t stream) {
    using P = Raw<T, N>;
    RowShape s;
    int64_t grid;
    if (mx_status st = row_shape(tokens, choices, cols / N, packs_of(sizeof(P), kAhead), &s, &grid); st != MX_OK) return st;
    return launch(combine_kernel<T, N, kAhead>, grid, kRowThreads, 0, stream, static_cast<const P *>(rows), rows_stride / N,
                  row_of_slot, weights, static_cast<P *>(y), y_stride / N, s);
}

template <typename T, int N, int kAhead>
mx_status backward_typed(const void *grad, int64_t grad_stride, const void *rows, int64_t rows_stride,
                         const int32_t *row_of_slot, const int32_t *ends, int E, const float *weights, void *d_rows,
                         int64_t d_rows_stride, float *d_weights, int64_t tokens, int32_t choices, int64_t cols,
                         cudaStream_t stream) {
    using P = Raw<T, N>;
    RowShape s;
    int64_t grid;
    if (mx_status st = row_shape(tokens, choices, cols / N, 1, &s, &grid); st != MX_OK) return st;
    const bool warp = s.packs <= 128 * packs_of(sizeof(P), kAhead);
    const int64_t ctas = warp ? div_up(tokens, kRowThreads / 32) : tokens;
    return launch(warp ? combine_backward_kernel<T, N, 32, kAhead> : combine_backward_kernel<T, N, kRowThreads, kAhead>, ctas,
                  kRowThreads, 0, stream, static_cast<const P *>(grad), grad_stride / N, static_cast<const P *>(rows),
                  rows_stride / N, row_of_slot, ends, E, weights, static_cast<P *>(d_rows), d_rows_stride / N, d_weights, s);
}

}  // namespace
}  // namespace mx

extern "C" {

size_t mx_expert_sort_workspace(int64_t tokens, int32_t choices) {
    if (!mx::slots_ok(tokens, choices)) return 0;
    const int64_t ctas = mx::sort_ctas(tokens * choices);
    return ctas > 1 ? (size_t)(ctas * mx::kMaxGroups * 4) : 0;
}

mx_status mx_expert_sort(const void *expert_ids, int32_t id_bytes, int64_t tokens, int32_t choices, int32_t num_experts,
                         int32_t *group_ends, int32_t *row_of_slot, int32_t *slot_of_row, void *workspace,
                         cudaStream_t stream) {
    if (!mx::slots_ok(tokens, choices) || num_experts < 1 || num_experts > MX_MAX_GROUPS) return MX_ERR_INVALID_ARG;
    if (id_bytes != 4 && id_bytes != 8) return MX_ERR_INVALID_ARG;
    const int64_t S = tokens * choices;
    if (group_ends == nullptr || (S > 0 && (expert_ids == nullptr || row_of_slot == nullptr || slot_of_row == nullptr)))
        return MX_ERR_INVALID_ARG;
    if (mx_expert_sort_workspace(tokens, choices) > 0 && workspace == nullptr) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(expert_ids, id_bytes) || !mx::aligned_to(group_ends, 4) || !mx::aligned_to(row_of_slot, 4) ||
        !mx::aligned_to(slot_of_row, 4) || !mx::aligned_to(workspace, 4))
        return MX_ERR_MISALIGNED;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    auto *ws = static_cast<int32_t *>(workspace);
    return id_bytes == 4 ? mx::sort_typed<int32_t>(expert_ids, S, num_experts, group_ends, row_of_slot, slot_of_row, ws, stream)
                         : mx::sort_typed<int64_t>(expert_ids, S, num_experts, group_ends, row_of_slot, slot_of_row, ws, stream);
}

mx_status mx_dispatch_rows(const void *x, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t x_stride,
                           const int32_t *row_of_slot, int32_t choices, const int32_t *group_ends, int32_t num_experts,
                           void *out, int64_t out_stride, cudaStream_t stream) {
    const int es = mx::element_bytes(dtype);
    if (es == 0 || !mx::slots_ok(tokens, choices) || cols < 0 || cols > mx::kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (num_experts < 1 || num_experts > MX_MAX_GROUPS || x_stride < cols || out_stride < cols) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(x_stride, es) || !mx::stride_fits(out_stride, es)) return MX_ERR_UNSUPPORTED;
    if (tokens == 0 || cols == 0) return MX_OK;
    if (x == nullptr || out == nullptr || row_of_slot == nullptr || group_ends == nullptr) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(x, es) || !mx::aligned_to(out, es) || !mx::aligned_to(row_of_slot, 4) || !mx::aligned_to(group_ends, 4))
        return MX_ERR_MISALIGNED;
    const mx::Mat mats[] = {{x, x_stride}, {out, out_stride}};
    const int bytes = mx::pack_bytes(es, cols, mats);
    if (bytes < 8 && cols * es / 2 > mx::kOpsMaxExtent) return MX_ERR_UNSUPPORTED;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
#define MX_DISPATCH(F, P) mx::F<P>(x, x_stride * es, row_of_slot, group_ends, num_experts, out, out_stride * es, tokens, choices, cols * es, stream)
    return bytes == 16  ? MX_DISPATCH(dispatch_typed, uint4)
           : bytes == 8 ? MX_DISPATCH(dispatch_typed, uint2)
           : bytes == 4 ? MX_DISPATCH(dispatch_elements, uint32_t)
                        : MX_DISPATCH(dispatch_elements, uint16_t);
#undef MX_DISPATCH
}

mx_status mx_combine_rows(const void *rows, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t rows_stride,
                          const int32_t *row_of_slot, int32_t choices, const float *weights, void *y, int64_t y_stride,
                          cudaStream_t stream) {
    const int es = mx::element_bytes(dtype);
    if (es == 0 || !mx::slots_ok(tokens, choices) || cols < 0 || cols > mx::kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (rows_stride < cols || y_stride < cols) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(rows_stride, es) || !mx::stride_fits(y_stride, es)) return MX_ERR_UNSUPPORTED;
    if (tokens == 0 || cols == 0) return MX_OK;
    if (rows == nullptr || y == nullptr || row_of_slot == nullptr) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(rows, es) || !mx::aligned_to(y, es) || !mx::aligned_to(row_of_slot, 4) || !mx::aligned_to(weights, 4))
        return MX_ERR_MISALIGNED;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    const mx::Mat mats[] = {{rows, rows_stride}, {y, y_stride}};
    const int bytes = mx::pack_bytes(es, cols, mats);
#define MX_COMBINE_K(T, N, K) mx::combine_typed<T, N, K>(rows, rows_stride, row_of_slot, weights, y, y_stride, tokens, choices, cols, stream)
#define MX_COMBINE(T, N) (choices <= 2 ? MX_COMBINE_K(T, N, 2) : choices <= 4 ? MX_COMBINE_K(T, N, 4) : MX_COMBINE_K(T, N, 8))
#define MX_COMBINE_16(T) (bytes == 16 ? MX_COMBINE(T, 8) : bytes == 8 ? MX_COMBINE(T, 4) : bytes == 4 ? MX_COMBINE(T, 2) : MX_COMBINE(T, 1))
    if (dtype == MX_F32) return bytes == 16 ? MX_COMBINE(float, 4) : bytes == 8 ? MX_COMBINE(float, 2) : MX_COMBINE(float, 1);
    return dtype == MX_BF16 ? MX_COMBINE_16(__nv_bfloat16) : MX_COMBINE_16(__half);
#undef MX_COMBINE_16
#undef MX_COMBINE
#undef MX_COMBINE_K
}

mx_status mx_combine_rows_backward(const void *grad, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t grad_stride,
                                   const void *rows, int64_t rows_stride, const int32_t *row_of_slot, int32_t choices,
                                   const int32_t *group_ends, int32_t num_experts, const float *weights, void *d_rows,
                                   int64_t d_rows_stride, float *d_weights, cudaStream_t stream) {
    const int es = mx::element_bytes(dtype);
    if (es == 0 || !mx::slots_ok(tokens, choices) || cols < 1 || cols > mx::kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (num_experts < 1 || num_experts > MX_MAX_GROUPS) return MX_ERR_INVALID_ARG;
    if (grad_stride < cols || rows_stride < cols || d_rows_stride < cols) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(grad_stride, es) || !mx::stride_fits(rows_stride, es) || !mx::stride_fits(d_rows_stride, es))
        return MX_ERR_UNSUPPORTED;
    if (tokens == 0) return MX_OK;
    if (grad == nullptr || rows == nullptr || row_of_slot == nullptr || group_ends == nullptr || weights == nullptr ||
        d_rows == nullptr || d_weights == nullptr)
        return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(grad, es) || !mx::aligned_to(rows, es) || !mx::aligned_to(d_rows, es) ||
        !mx::aligned_to(row_of_slot, 4) || !mx::aligned_to(group_ends, 4) || !mx::aligned_to(weights, 4) ||
        !mx::aligned_to(d_weights, 4))
        return MX_ERR_MISALIGNED;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    const mx::Mat mats[] = {{grad, grad_stride}, {rows, rows_stride}, {d_rows, d_rows_stride}};
    const int bytes = mx::pack_bytes(es, cols, mats);
#define MX_BACKWARD_K(T, N, K)                                                                                            \
    mx::backward_typed<T, N, K>(grad, grad_stride, rows, rows_stride, row_of_slot, group_ends, num_experts, weights,      \
                                d_rows, d_rows_stride, d_weights, tokens, choices, cols, stream)
#define MX_BACKWARD(T, N) (choices <= 2 ? MX_BACKWARD_K(T, N, 2) : choices <= 4 ? MX_BACKWARD_K(T, N, 4) : MX_BACKWARD_K(T, N, 8))
#define MX_BACKWARD_16(T) (bytes == 16 ? MX_BACKWARD(T, 8) : bytes == 8 ? MX_BACKWARD(T, 4) : bytes == 4 ? MX_BACKWARD(T, 2) : MX_BACKWARD(T, 1))
    if (dtype == MX_F32) return bytes == 16 ? MX_BACKWARD(float, 4) : bytes == 8 ? MX_BACKWARD(float, 2) : MX_BACKWARD(float, 1);
    return dtype == MX_BF16 ? MX_BACKWARD_16(__nv_bfloat16) : MX_BACKWARD_16(__half);
#undef MX_BACKWARD_16
#undef MX_BACKWARD
#undef MX_BACKWARD_K
}

}  // extern "C"
