// mx_quantize.cu -- 8-bit floating point with one power-of-two scale (E8M0)
// for each block of values, on B200 (sm_100a).
//
// For a block with largest magnitude A the scale is 2^e, e the smallest whole
// number with A <= F * 2^e, where F = 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2)
// is the type's largest value: nothing saturates.  With A = m * 2^a, 1 <= m < 2,
// that is e = a - 8 (or 15), plus one if m > 1.75: read off A's bits, with no
// logarithm.  x * 2^-e is exact in 32 bits wherever it does not vanish, so the
// only rounding is the one to 8 bits (to nearest, ties to even).  The scale
// byte is e + 127, at least 0; a block that holds a NaN or an infinity gets
// the byte 255 (NaN) and NaN elements.  A block of zeros gets the byte 0.
//
// Everything here is bound by memory.  A thread holds 8 or 16 consecutive
// elements, because a block of 128 is then 16 or 8 neighbouring lanes and its
// maximum 4 or 3 shuffles.  On a B200, 131072 x 7168 bf16: rows 411 us (6.85
// TB/s; 8 elements a lane 522; blocks of 32 439), columns of 8 groups 470 us (6.0 TB/s), 128 x 128
// blocks 455 us (6.2 TB/s); 16384 tokens to 131072 rows in expert order 217 us
// (5.4 TB/s), 23 of them for the scales, whose bytes go to scattered rows.

#include <climits>

#include <cuda_fp8.h>

#include "mx_ops.cuh"

namespace mx {
namespace {

constexpr int kQThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

// Magnitudes are compared as bits: the order of finite values is that of their
// bits, and infinities and NaNs lie above all of them.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, int fexp) {
    if (amax >= kInfBits) return 255u;
    const int b = (int)(amax >> 23) - fexp + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax < 0x800000u || b < 0 ? 0u : (uint32_t)b;
}

// 2^-e of a finite scale byte: its exponent field is 254 - byte, 7 .. 254.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

template <__nv_fp8_interpretation_t kTo>
__device__ __forceinline__ uint2 eight_bytes(const float (&v)[8]) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, kTo);
    return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
}
__device__ __forceinline__ uint2 eight_bytes(const float (&v)[8], bool e5m2) {
    return e5m2 ? eight_bytes<__NV_E5M2>(v) : eight_bytes<__NV_E4M3>(v);
}
constexpr uint32_t kNanBytes = 0x7f7f7f7fu;   // four NaNs in both types

// Eight consecutive elements of a row from column c on, zeros past `cols`, as
// the words that hold them.  kIn: rows start on 16-byte boundaries, or anywhere;
// kWide, of the 8-bit rows, on 8-byte ones.  kWhole: on 16-byte and 8-byte ones, and
// cols is a multiple of 8: without the code for a rest, tiles of 128 x 128 take 455
// us where they take 523 with it.  Anywhere costs about twice the time of whole
// rows (48033 x 2201 bf16: rows 85 us, blocks 103; 2202: 79 and 76).
enum In { kAnywhere = 0, kVectors = 1, kWhole = 2 };
template <typename T> struct Eight { uint4 q[sizeof(T) / 2]; };
template <typename T, int kIn>
__device__ __forceinline__ Eight<T> load8(const T *row, int c, int cols) {
    Eight<T> v;
    if constexpr (kIn == kWhole) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            v.q[i] = c < cols ? __ldg(reinterpret_cast<const uint4 *>(row + c) + i) : make_uint4(0u, 0u, 0u, 0u);
        return v;
    }
    if (kIn == kVectors && c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v.q[i] = __ldg(reinterpret_cast<const uint4 *>(row + c) + i);
    } else if (sizeof(T) == 2 && c + 8 <= cols) {
        // off a 4-byte boundary: the five words that hold the elements, each of
        // which holds at least one
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
        const uint32_t *src = reinterpret_cast<const uint32_t *>(at & ~uintptr_t(3));
        v.q[0] = make_uint4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
        if (at & 2) {
            const uint32_t last = __ldg(src + 4);
            v.q[0] = make_uint4(__funnelshift_r(v.q[0].x, v.q[0].y, 16), __funnelshift_r(v.q[0].y, v.q[0].z, 16),
                                __funnelshift_r(v.q[0].z, v.q[0].w, 16), __funnelshift_r(v.q[0].w, last, 16));
        }
    } else {
        using W = Raw<T, 1>;
        const W *src = reinterpret_cast<const W *>(row);
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? src[c + i] : 0u;
        if constexpr (sizeof(T) == 4) {
            v.q[0] = make_uint4(e[0], e[1], e[2], e[3]);
            v.q[1] = make_uint4(e[4], e[5], e[6], e[7]);
        } else {
            v.q[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        }
    }
    return v;
}
template <typename T> __device__ __forceinline__ Eight<T> no_eight() {
    Eight<T> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v.q[i] = make_uint4(0u, 0u, 0u, 0u);
    return v;
}
template <typename T> __device__ __forceinline__ void floats_of(const Eight<T> &v, float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        float lo[4], hi[4];
        unpack<T, 4>(v.q[0], lo);
        unpack<T, 4>(v.q[1], hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = lo[i], f[4 + i] = hi[i];
    } else {
        unpack<T, 8>(v.q[0], f);
    }
}

// The largest magnitudes so far, as bits: two 16-bit ones a word (their order is
// that of their bits too), or one of 32 bits.
template <typename T> struct Top { uint32_t w[sizeof(T) == 4 ? 8 : 4] = {}; };
template <typename T> __device__ __forceinline__ void raise(Top<T> &t, const Eight<T> &v) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t e[8] = {v.q[0].x, v.q[0].y, v.q[0].z, v.q[0].w, v.q[1].x, v.q[1].y, v.q[1].z, v.q[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) t.w[i] = max(t.w[i], e[i] & 0x7fffffffu);
    } else {
        const uint32_t e[4] = {v.q[0].x, v.q[0].y, v.q[0].z, v.q[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) t.w[i] = __vmaxu2(t.w[i], e[i] & 0x7fff7fffu);
    }
}
// Each column's, as bits of a 32-bit float.
template <typename T> __device__ __forceinline__ void columns_of(const Top<T> &t, uint32_t (&m)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = t.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = two_floats<T>(t.w[i]);
            m[2 * i] = __float_as_uint(f.x);
            m[2 * i + 1] = __float_as_uint(f.y);
        }
    }
}
// The largest of all of them.
template <typename T> __device__ __forceinline__ uint32_t top_of(const Top<T> &t) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = t.w[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, t.w[i]);
        return m;
    } else {
        const uint32_t p = __vmaxu2(__vmaxu2(t.w[0], t.w[1]), __vmaxu2(t.w[2], t.w[3]));
        return __float_as_uint(two_floats<T>(max(p & 0xffffu, p >> 16)).x);
    }
}

template <bool kWide, int kIn>
__device__ __forceinline__ void store8(uint8_t *row, int c, int cols, uint2 q) {
    if constexpr (kIn == kWhole) {
        if (c < cols) *reinterpret_cast<uint2 *>(row + c) = q;
    } else if (kWide && c + 8 <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
}

// ------------------------------------------------------------------ rows
struct RowsArgs {
    uint8_t *q;
    int64_t q_stride;
    uint8_t *scales;
    int64_t scale_row, scale_block;   // bytes between the scales of neighbouring rows and blocks
    const int *row_of_slot;           // kOrder: the rows that each token goes to
    const int *ends;
    int32_t G;
    int64_t in_rows, out_rows;
    int32_t cols, k, segments;
    int32_t per_warp;                 // rows of a warp, 1 to 4
    bool e5m2;
};

// A CTA takes 32 * kPer columns of 8 to 32 rows, a warp 1 to 4 of them: that many
// rows' loads are in flight a lane, fewer where there are too few rows to fill
// the SMs.  A lane holds kPer consecutive elements: 16 where rows allow it (half
// the shuffles, scales and stores of 8 for the same bytes), else 8.  kOrder: row
// t is written to the rows row_of_slot[t, :], so a token is read and rounded once
// however many experts it goes to.
template <typename T, int kIn, bool kWide, int kPer, int kBlock, bool kOrder>
__global__ void __launch_bounds__(kQThreads)
quantize_rows_kernel(const T *__restrict__ x, int64_t x_stride, RowsArgs a) {
    constexpr int kEights = kPer / 8, kLanes = kBlock / kPer;   // lanes of a block
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t band = blockIdx.x / a.segments;
    const int c = (int)(blockIdx.x - band * a.segments) * (32 * kPer) + lane * kPer;
    const int64_t r0 = (band * 8 + w) * a.per_warp;
    const int fexp = a.e5m2 ? 15 : 8;
    Eight<T> v[4][kEights];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < kEights; ++h)
            v[i][h] = i < a.per_warp && r0 + i < a.in_rows ? load8<T, kIn>(x + (r0 + i) * x_stride, c + 8 * h, a.cols) : no_eight<T>();
    const bool scaler = lane % kLanes == 0;
    const int64_t block_at = (int64_t)(c / kBlock) * a.scale_block;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= a.per_warp) break;
        Top<T> top;
#pragma unroll
        for (int h = 0; h < kEights; ++h) raise(top, v[i][h]);
        uint32_t amax = top_of(top);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        const uint32_t byte = scale_byte(amax, fexp);
        uint2 q[kEights];
#pragma unroll
        for (int h = 0; h < kEights; ++h) {
            q[h] = make_uint2(kNanBytes, kNanBytes);
            if (byte != 255u) {
                const float s = inverse_scale(byte);
                float f[8];
                floats_of(v[i][h], f);
#pragma unroll
                for (int u = 0; u < 8; ++u) f[u] *= s;
                q[h] = eight_bytes(f, a.e5m2);
            }
        }
        auto store = [&](int64_t r) {
            uint8_t *row = a.q + r * a.q_stride;
            if constexpr (kPer == 16) *reinterpret_cast<uint4 *>(row + c) = make_uint4(q[0].x, q[0].y, q[kEights - 1].x, q[kEights - 1].y);
            else store8<kWide, kIn>(row, c, a.cols, q[0]);
            if (scaler) a.scales[r * a.scale_row + block_at] = (uint8_t)byte;
        };
        const int64_t t = r0 + i;
        if (t < a.in_rows && c < a.cols) {
            if (!kOrder) {
                store(t);
            } else {
                for (int j = 0; j < a.k; ++j) {
                    const int64_t r = a.row_of_slot[t * a.k + j];
                    if (r >= 0 && r < a.out_rows) store(r);
                }
            }
        }
    }
    if (kOrder) {   // rows behind the last group
        const int64_t from = rows_in_groups(a.ends, a.G);
        const int64_t units = (a.cols + 7) / 8, n = (a.out_rows - from) * units;
        for (int64_t i = (int64_t)blockIdx.x * kQThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kQThreads) {
            const int64_t r = from + i / units;
            const int at = (int)(i % units) * 8;
            store8<kWide, kIn>(a.q + r * a.q_stride, at, a.cols, make_uint2(0u, 0u));
            if (at % kBlock == 0) a.scales[r * a.scale_row + (int64_t)(at / kBlock) * a.scale_block] = 0;
        }
    }
}

// ------------------------------------------------------------------ tiles
// 128 x 128 tiles, 256 threads: thread (ty, tx) holds rows ty + 16 i (i < 8) of
// columns 8 tx .. 8 tx + 7, 8 loads in flight; a warp covers two rows of 128
// columns.  Column blocks (one scale a column) and square blocks (one a tile)
// differ in how far the maximum is reduced.  Four CTAs an SM (16-bit input, 64
// registers) overlap one tile's stores with another's loads: with two, columns
// took 720 us where they took 497.
struct TileArgs {
    int64_t x_stride, x_group;      // elements
    uint8_t *q;
    int64_t q_stride, q_group;
    uint8_t *scales;
    int64_t scale_stride;           // columns: bytes between 128-row blocks
    const int *ends;                // columns: group ends
    int64_t rows, tiles;            // rows of x (of each group); tiles in all
    int32_t G, cols, row_tiles, col_tiles;
    bool e5m2;
};

template <typename T, int kIn, bool kWide, bool kSquare>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 4 : 2)
quantize_tiles_kernel(const T *__restrict__ x, TileArgs a) {
    __shared__ alignas(16) uint32_t top[16][128];
    __shared__ uint32_t bytes[128];
    __shared__ GroupTable table;
    grid_dependency_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, w = tid >> 5;
    const int fexp = a.e5m2 ? 15 : 8;
    if (!kSquare) {
        if (w == 0) build_group_table<true>(a.ends, a.G, (int)a.rows, 1, table);
        __syncthreads();
    }
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int64_t rb = tile / a.col_tiles;
        const int c0 = (int)(tile - rb * a.col_tiles) * 128, c = c0 + tx * 8;
        const T *src = x;
        uint8_t *dst = a.q;
        int64_t valid, dst_rows = 128;   // rows of the tile that hold data, and that exist in q
        int64_t scale_at;
        if (kSquare) {
            const int64_t g = rb / a.row_tiles, r0 = (rb - g * a.row_tiles) * 128;
            src += g * a.x_group + r0 * a.x_stride;
            dst += g * a.q_group + r0 * a.q_stride;
            valid = dst_rows = min((int64_t)128, a.rows - r0);
            scale_at = rb * a.col_tiles + c0 / 128;
        } else {
            valid = 0;
            const int64_t p = rb * 128;
            if (p < table.pstart[kMaxGroups]) {
                const int g = find_group_pstart(table, kMaxGroups, (int)p);
                const int64_t r0 = p - table.pstart[g];
                valid = min((int64_t)128, table.size[g] - r0);
                src += (table.begin[g] + r0) * a.x_stride;
            }
            dst += p * a.q_stride;
            scale_at = rb * a.scale_stride + c0;
        }
        if (!kSquare && valid <= 0) {   // behind the last group: zeros, and nothing to wait for
#pragma unroll
            for (int i = 0; i < 8; ++i) store8<kWide, kIn>(dst + (ty + 16 * i) * a.q_stride, c, a.cols, make_uint2(0u, 0u));
            if (tid < 128 && c0 + tid < a.cols) a.scales[scale_at + tid] = 0;
            continue;
        }
        Eight<T> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = ty + 16 * i;
            v[i] = r < valid ? load8<T, kIn>(src + r * a.x_stride, c, a.cols) : no_eight<T>();
        }
        Top<T> mine;
#pragma unroll
        for (int i = 0; i < 8; ++i) raise(mine, v[i]);
        uint32_t m[8];
        if (kSquare) {
            uint32_t all = __reduce_max_sync(0xffffffffu, top_of(mine));
            if (lane == 0) top[0][w] = all;
            __syncthreads();
            all = top[0][0];
#pragma unroll
            for (int u = 1; u < kQThreads / 32; ++u) all = max(all, top[0][u]);
            const uint32_t byte = scale_byte(all, fexp);
            if (tid == 0) a.scales[scale_at] = (uint8_t)byte;
#pragma unroll
            for (int u = 0; u < 8; ++u) m[u] = byte;
        } else {
            columns_of(mine, m);
#pragma unroll
            for (int u = 0; u < 8; u += 4)
                *reinterpret_cast<uint4 *>(&top[ty][tx * 8 + u]) = make_uint4(m[u], m[u + 1], m[u + 2], m[u + 3]);
            __syncthreads();
            if (tid < 128) {
                uint32_t all = 0;
#pragma unroll
                for (int u = 0; u < 16; ++u) all = max(all, top[u][tid]);
                const uint32_t byte = scale_byte(all, fexp);
                bytes[tid] = byte;
                if (c0 + tid < a.cols) a.scales[scale_at + tid] = (uint8_t)byte;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < 8; ++u) m[u] = bytes[tx * 8 + u];
        }
        uint32_t nan[2] = {0u, 0u};   // bytes of the columns whose block holds no finite scale
        float s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (m[u] == 255u) nan[u >> 2] |= 0xffu << (8 * (u & 3));
            s[u] = inverse_scale(min(m[u], 254u));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = ty + 16 * i;
            float f[8];
            floats_of(v[i], f);
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] *= s[u];
            uint2 q = eight_bytes(f, a.e5m2);
            if (r < valid) {
                q.x = (q.x & ~nan[0]) | (kNanBytes & nan[0]);
                q.y = (q.y & ~nan[1]) | (kNanBytes & nan[1]);
            }
            if (r < dst_rows) store8<kWide, kIn>(dst + r * a.q_stride, c, a.cols, q);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host side
int in_bytes(mx_dtype t) { return t == MX_F32 ? 4 : t == MX_BF16 || t == MX_F16 ? 2 : 0; }

// How rows of the input are aligned, and whether those of the output are.
int in_of(const void *x, int64_t x_stride, int64_t x_group, int es) {
    const auto on = [&](int64_t n) { return aligned_to(x, n) && x_stride * es % n == 0 && x_group * es % n == 0; };
    return on(16) ? kVectors : kAnywhere;
}
bool wide_of(const void *q, int64_t q_stride, int64_t q_group, int64_t n) {
    return aligned_to(q, n) && q_stride % n == 0 && q_group % n == 0;
}

template <typename T, int kIn, bool kWide, int kPer>
mx_status rows_typed(const void *x, int64_t x_stride, const RowsArgs &a, int block, int64_t grid, cudaStream_t stream) {
    const T *p = static_cast<const T *>(x);
    const bool order = a.row_of_slot != nullptr;
    if (block == 128)
        return order ? launch(quantize_rows_kernel<T, kIn, kWide, kPer, 128, true>, grid, kQThreads, 0, stream, p, x_stride, a)
                     : launch(quantize_rows_kernel<T, kIn, kWide, kPer, 128, false>, grid, kQThreads, 0, stream, p, x_stride, a);
    return order ? launch(quantize_rows_kernel<T, kIn, kWide, kPer, 32, true>, grid, kQThreads, 0, stream, p, x_stride, a)
                 : launch(quantize_rows_kernel<T, kIn, kWide, kPer, 32, false>, grid, kQThreads, 0, stream, p, x_stride, a);
}

// Rows of the output that are not aligned are rare (the torch calls align theirs): they share one kernel.
template <typename T>
mx_status rows_any(const void *x, int64_t x_stride, const RowsArgs &a, int block, int64_t grid, int in, bool wide, bool sixteen,
                   cudaStream_t stream) {
    if (sixteen) return rows_typed<T, kWhole, true, 16>(x, x_stride, a, block, grid, stream);
    if (!wide) return rows_typed<T, kAnywhere, false, 8>(x, x_stride, a, block, grid, stream);
    if (in == kVectors) return rows_typed<T, kVectors, true, 8>(x, x_stride, a, block, grid, stream);
    return rows_typed<T, kAnywhere, true, 8>(x, x_stride, a, block, grid, stream);
}

template <typename T, bool kSquare>
mx_status tiles_typed(const void *x, const TileArgs &a, int in, bool wide, cudaStream_t stream) {
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    const int64_t cap = (int64_t)sms * 4;
    const int64_t grid = a.tiles < cap ? a.tiles : cap;
    const T *p = static_cast<const T *>(x);
    if (wide && in == kVectors && a.cols % 8 == 0)
        return launch(quantize_tiles_kernel<T, kWhole, true, kSquare>, grid, kQThreads, 0, stream, p, a);
    if (!wide) return launch(quantize_tiles_kernel<T, kAnywhere, false, kSquare>, grid, kQThreads, 0, stream, p, a);
    if (in == kVectors) return launch(quantize_tiles_kernel<T, kVectors, true, kSquare>, grid, kQThreads, 0, stream, p, a);
    return launch(quantize_tiles_kernel<T, kAnywhere, true, kSquare>, grid, kQThreads, 0, stream, p, a);
}

template <bool kSquare>
mx_status tiles_any(const void *x, mx_dtype dtype, const TileArgs &a, int in, bool wide, cudaStream_t stream) {
    if (dtype == MX_F32) return tiles_typed<float, kSquare>(x, a, in, wide, stream);
    if (dtype == MX_BF16) return tiles_typed<__nv_bfloat16, kSquare>(x, a, in, wide, stream);
    return tiles_typed<__half, kSquare>(x, a, in, wide, stream);
}

bool eight_bit_type(mx_dtype t) { return t == MX_E4M3 || t == MX_E5M2; }

}  // namespace
}  // namespace mx

extern "C" {

mx_status mx_quantize_rows(const void *x, mx_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride, int32_t block,
                           mx_dtype out_dtype, const int32_t *row_of_slot, int32_t choices, const int32_t *group_ends,
                           int32_t num_experts, uint8_t *q, int64_t q_stride, uint8_t *scales, int64_t scale_row_stride,
                           int64_t scale_block_stride, cudaStream_t stream) {
    const int es = mx::in_bytes(dtype);
    if (es == 0 || !mx::eight_bit_type(out_dtype) || (block != 128 && block != 32)) return MX_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || rows > mx::kOpsMaxExtent || cols > mx::kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (x_stride < cols || q_stride < cols || scale_row_stride < 1 || scale_block_stride < 1) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(x_stride, es) || !mx::stride_fits(q_stride, 1) || !mx::stride_fits(scale_row_stride, 1) ||
        !mx::stride_fits(scale_block_stride, 1))
        return MX_ERR_UNSUPPORTED;
    const bool order = row_of_slot != nullptr;
    if (order && (choices < 1 || rows * choices > mx::kOpsMaxExtent || num_experts < 1 || num_experts > MX_MAX_GROUPS ||
                  group_ends == nullptr))
        return MX_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MX_OK;
    if (x == nullptr || q == nullptr || scales == nullptr) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(x, es) || !mx::aligned_to(row_of_slot, 4) || !mx::aligned_to(group_ends, 4)) return MX_ERR_MISALIGNED;
    mx::RowsArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.scales = scales;
    a.scale_row = scale_row_stride;
    a.scale_block = scale_block_stride;
    a.row_of_slot = row_of_slot;
    a.ends = group_ends;
    a.G = num_experts;
    a.in_rows = rows;
    a.out_rows = order ? rows * choices : rows;
    a.cols = (int32_t)cols;
    a.k = choices;
    const int in = mx::in_of(x, x_stride, 0, es);
    const bool wide = mx::wide_of(q, q_stride, 0, 8);
    const bool sixteen = in == mx::kVectors && mx::wide_of(q, q_stride, 0, 16) && cols % 16 == 0;
    a.segments = (int32_t)mx::div_up(cols, sixteen ? 512 : 256);
    a.e5m2 = out_dtype == MX_E5M2;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    a.per_warp = 4;
    while (a.per_warp > 1 && mx::div_up(rows, 8 * a.per_warp) * a.segments < 2 * sms) a.per_warp /= 2;
    const int64_t grid = mx::div_up(rows, 8 * a.per_warp) * a.segments;
    if (grid > INT_MAX) return MX_ERR_UNSUPPORTED;
#define MX_ROWS(T) mx::rows_any<T>(x, x_stride, a, block, grid, in, wide, sixteen, stream)
    if (dtype == MX_F32) return MX_ROWS(float);
    if (dtype == MX_BF16) return MX_ROWS(__nv_bfloat16);
    return MX_ROWS(__half);
#undef MX_ROWS
}

int64_t mx_padded_rows(int64_t rows, int32_t num_groups) {
    if (rows < 0 || rows > mx::kOpsMaxExtent || num_groups < 1 || num_groups > MX_MAX_GROUPS) return 0;
    return mx::up_to(rows, 128) + 128ll * num_groups;
}

mx_status mx_quantize_cols(const void *x, mx_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride,
                           const int32_t *group_ends, int32_t num_groups, mx_dtype out_dtype, uint8_t *q, int64_t q_stride,
                           uint8_t *scales, int64_t scale_stride, cudaStream_t stream) {
    const int es = mx::in_bytes(dtype);
    if (es == 0 || !mx::eight_bit_type(out_dtype) || num_groups < 1 || num_groups > MX_MAX_GROUPS) return MX_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || rows > mx::kOpsMaxExtent || cols > mx::kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (x_stride < cols || q_stride < cols || scale_stride < cols) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(x_stride, es) || !mx::stride_fits(q_stride, 1) || !mx::stride_fits(scale_stride, 1))
        return MX_ERR_UNSUPPORTED;
    if (cols == 0) return MX_OK;
    if ((rows > 0 && x == nullptr) || q == nullptr || scales == nullptr || group_ends == nullptr) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(x, es) || !mx::aligned_to(group_ends, 4)) return MX_ERR_MISALIGNED;
    mx::TileArgs a = {};
    a.x_stride = x_stride;
    a.q = q;
    a.q_stride = q_stride;
    a.scales = scales;
    a.scale_stride = scale_stride;
    a.ends = group_ends;
    a.rows = rows;
    a.G = num_groups;
    a.cols = (int32_t)cols;
    a.col_tiles = (int32_t)mx::div_up(cols, 128);
    a.tiles = mx_padded_rows(rows, num_groups) / 128 * a.col_tiles;
    a.e5m2 = out_dtype == MX_E5M2;
    return mx::tiles_any<false>(x, dtype, a, mx::in_of(x, x_stride, 0, es), mx::wide_of(q, q_stride, 0, 8), stream);
}

mx_status mx_quantize_blocks(const void *x, mx_dtype dtype, int64_t groups, int64_t rows, int64_t cols, int64_t x_group_stride,
                             int64_t x_stride, mx_dtype out_dtype, uint8_t *q, int64_t q_group_stride, int64_t q_stride,
                             uint8_t *scales, cudaStream_t stream) {
    const int es = mx::in_bytes(dtype);
    if (es == 0 || !mx::eight_bit_type(out_dtype)) return MX_ERR_INVALID_ARG;
    if (groups < 0 || rows < 0 || cols < 0 || groups > mx::kOpsMaxExtent || rows > mx::kOpsMaxExtent || cols > mx::kOpsMaxExtent)
        return MX_ERR_INVALID_ARG;
    if (x_stride < cols || q_stride < cols || x_group_stride < 0 || q_group_stride < 0) return MX_ERR_INVALID_ARG;
    if (!mx::stride_fits(x_stride, es) || !mx::stride_fits(q_stride, 1) ||
        (groups > 1 && (!mx::stride_fits(x_group_stride, es) || !mx::stride_fits(q_group_stride, 1))))
        return MX_ERR_UNSUPPORTED;
    if (groups == 0 || rows == 0 || cols == 0) return MX_OK;
    if (x == nullptr || q == nullptr || scales == nullptr) return MX_ERR_INVALID_ARG;
    if (groups > 1 && !mx::rows_fit(rows, q_stride, cols, q_group_stride)) return MX_ERR_INVALID_ARG;
    if (!mx::aligned_to(x, es)) return MX_ERR_MISALIGNED;
    mx::TileArgs a = {};
    a.x_stride = x_stride;
    a.x_group = groups > 1 ? x_group_stride : 0;
    a.q = q;
    a.q_stride = q_stride;
    a.q_group = groups > 1 ? q_group_stride : 0;
    a.scales = scales;
    a.rows = rows;
    a.cols = (int32_t)cols;
    a.row_tiles = (int32_t)mx::div_up(rows, 128);
    a.col_tiles = (int32_t)mx::div_up(cols, 128);
    if (mx::div_up(rows, 128) * a.col_tiles > INT64_MAX / mx::kOpsMaxExtent) return MX_ERR_UNSUPPORTED;
    a.tiles = groups * a.row_tiles * a.col_tiles;
    a.e5m2 = out_dtype == MX_E5M2;
    return mx::tiles_any<true>(x, dtype, a, mx::in_of(x, x_stride, a.x_group, es), mx::wide_of(q, q_stride, a.q_group, 8), stream);
}

}  // extern "C"
