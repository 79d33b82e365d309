// mx_matmul.cu -- grouped 8-bit matrix product with E8M0 scales on the tensor
// cores of B200 (sm_100a).
//
//   rows in groups (forward, input gradient):
//     out[r, n] = sum_k a[r, k] 2^sa(r, k) * b[g(r), n, k] 2^sb(g, n, k)
//   contraction in groups (weight gradient):
//     out[g, m, n] = sum_{r in g} a[r, m] 2^sa(r, m) * b[r, n] 2^sb(r, n)
//
// A scale covers 128 values along the contraction (and 128 columns of a weight
// matrix), or 32 in the blocked 128x4 layout.  A matrix instruction takes 32
// values of the contraction and one scale byte per row for them, from tensor
// memory, where 128 rows x 4 such bytes are four columns: exactly one 512-byte
// tile of the blocked layout, copied there whole.  For scales of 128 a warp
// writes such a tile with each byte four times, so both kinds run the same
// loop, and the scales cost no arithmetic outside the tensor cores.
//
// A CTA per SM walks output tiles of 128 x kN.  Its warps: 0 loads operands by
// TMA into a ring of stages of 128 along the contraction; 1 issues the matrix
// instructions; 2 brings the scales; 3 holds the tensor memory; 4..7 empty the
// accumulators into the output.  Operands whose contraction is the outer
// dimension in memory (weights read for the input gradient, both operands of
// the weight gradient) are loaded as they are and read through descriptors of
// that order: nothing is transposed in memory.

#include <climits>
#include <mutex>

#include "mx_ops.cuh"
#include "mx_tcgen05.cuh"

// A tensor map over bytes, with the 128-byte swizzle (defined in mx_rearrange.cu).
mx_status mx_encode_bytes_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                              const uint32_t *box);

namespace mx {
namespace {

__device__ unsigned int g_matmul_flags = 0;

enum Form { kFormNK = 0, kFormKN = 1, kFormOuter = 2 };
enum ScaleForm { kScales128 = 0, kScales32 = 1 };

constexpr int kTileM = 128;
constexpr int kTileK = 128;
constexpr int kMatThreads = 256;
constexpr int kOperandBytes = kTileM * kTileK;   // a 128 x 128 panel of either operand
constexpr int kTmemColumns = 512;
constexpr int kScaleColumn = 480;                // 2 sets of 4 + 8 columns of scales

struct MatArgs {
    const int *ends;
    const uint8_t *sa, *sb;
    int64_t sa_row, sa_block;               // bytes between scales along rows and along the contraction
    int64_t sb_group, sb_row, sb_block;
    void *out;
    int64_t out_stride, out_group;          // elements
    int32_t G, rows;                        // rows: of a (row groups), of both operands (contraction groups)
    int32_t M, N, K;                        // M: contraction groups only
    int32_t n_tiles, m_tiles, k_tiles;      // m_tiles: contraction groups only
    int32_t out_type;                       // 0 f32, 1 bf16, 2 f16
    uint32_t idesc;
    bool wide_out;
};

template <int kN>
struct Shared {
    static constexpr int kStages = kN == 256 ? 4 : 6;
    static constexpr int kPanels = kN / 128;
    static constexpr int kAccs = kN == 256 ? 1 : 2;
    static constexpr int kStageBytes = (1 + kPanels) * kOperandBytes;
    static constexpr int kScaleBytes = (1 + kPanels) * 512;
    alignas(1024) uint8_t operands[kStages][kStageBytes];
    alignas(128) uint8_t scales[kStages][kScaleBytes];
    GroupTable table;
    alignas(8) uint64_t full[kStages], empty[kStages], acc_full[kAccs], acc_empty[kAccs], drain;
    uint32_t tmem;
    volatile int abort;
};

struct Tile {
    int32_t g, row0, rows, n0, k_tiles;   // row0: first row of a (row groups) or column of a (contraction groups)
    int32_t k_base;                       // contraction groups: first row of the operands
    int32_t scale_row;                    // blocked scales: the 128-row tile of a's scales
};

template <int kForm, int kN>
__device__ __forceinline__ Tile tile_at(const GroupTable &table, const MatArgs &a, int t) {
    Tile o;
    if (kForm == kFormOuter) {
        const int per = a.m_tiles * a.n_tiles;
        o.g = t / per;
        const int local = t - o.g * per, mt = local / a.n_tiles;
        o.row0 = mt * kTileM;
        o.rows = min(kTileM, a.M - o.row0);
        o.n0 = (local - mt * a.n_tiles) * kN;
        o.k_base = table.pstart[o.g];
        o.k_tiles = (table.size[o.g] + kTileK - 1) / kTileK;
        o.scale_row = 0;
    } else {
        o.g = find_group(table, kMaxGroups, t);
        const int local = t - table.istart[o.g], mt = local / a.n_tiles;
        o.row0 = table.begin[o.g] + mt * kTileM;
        o.rows = min(kTileM, table.size[o.g] - mt * kTileM);
        o.n0 = (local - mt * a.n_tiles) * kN;
        o.k_base = 0;
        o.k_tiles = a.k_tiles;
        o.scale_row = table.pstart[o.g] / kTileM + mt;
    }
    return o;
}

// A bounded wait that also ends when another warp of the CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > (1ll << 31)) {
            *abort = 1;
            atomicOr(&g_matmul_flags, kFlagWaitTimeout);
            return false;
        }
    }
}

// Scale bytes of four rows (lane, lane + 32, ...) for four steps of the
// contraction, one word a step.
struct RowScales { uint32_t step[4]; };
__device__ __forceinline__ RowScales load_row_scales(const uint8_t *s, int64_t row_stride, int64_t block_stride, int row0,
                                                     int rows, int block0, int blocks, int lane) {
    RowScales o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        o.step[k] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row0 + lane + 32 * i;
            uint32_t b = 127;
            if (r < rows && block0 + k < blocks) b = s[r * row_stride + (block0 + k) * block_stride];
            o.step[k] |= b << (8 * i);
        }
    }
    return o;
}
// A line of the tile: rows lane + 32 i, each byte for all four groups of 32.
__device__ __forceinline__ uint4 scale_line(uint32_t rows4) {
    return make_uint4(__byte_perm(rows4, 0, 0x0000), __byte_perm(rows4, 0, 0x1111), __byte_perm(rows4, 0, 0x2222),
                      __byte_perm(rows4, 0, 0x3333));
}

template <typename T>
__device__ __forceinline__ void store_row(T *dst, const uint32_t (&v)[32], int valid, bool wide) {
    if (wide && valid >= 32) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 32; i += N) {
            Pack<T, N> p;
#pragma unroll
            for (int u = 0; u < N; ++u) p.v[u] = from_f32<T>(__uint_as_float(v[i + u]));
            *reinterpret_cast<Pack<T, N> *>(dst + i) = p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < valid) dst[i] = from_f32<T>(__uint_as_float(v[i]));
    }
}

template <int kForm, int kScales, int kN>
__global__ void __launch_bounds__(kMatThreads, 1)
grouped_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const MatArgs a) {
    using Sh = Shared<kN>;
    constexpr int kStages = Sh::kStages, kPanels = Sh::kPanels, kAccs = Sh::kAccs;
    constexpr bool kOuterA = kForm == kFormOuter, kOuterB = kForm != kFormNK;
    extern __shared__ uint8_t dyn_smem[];
    Sh &sh = *reinterpret_cast<Sh *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;

    if (w == 0 && lane == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);    // operands, scales
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 4);   // the four warps that empty it
        }
        mbar_init(&sh.drain, 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    if (w == 3) tmem_alloc(&sh.tmem, kTmemColumns);
    if (w == 2) build_group_table<true>(a.ends, a.G, a.rows, a.n_tiles, sh.table);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int total = kForm == kFormOuter ? a.G * a.m_tiles * a.n_tiles : sh.table.istart[kMaxGroups];

    if (w == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
                const Tile o = tile_at<kForm, kN>(sh.table, a, t);
                for (int k = 0; k < o.k_tiles; ++k, ++it) {
                    const uint32_t s = it % kStages, phase = it / kStages & 1;
                    if (!(ok = wait_or_abort(&sh.empty[s], phase ^ 1, &sh.abort))) break;
                    uint8_t *pa = sh.operands[s], *pb = pa + kOperandBytes;
                    mbar_arrive_expect_tx(&sh.full[s], Sh::kStageBytes);
                    if (kOuterA) tma_load_2d(pa, &map_a, o.row0, o.k_base + k * kTileK, &sh.full[s]);
                    else tma_load_2d(pa, &map_a, k * kTileK, o.row0, &sh.full[s]);
                    if (kForm == kFormNK) {
                        tma_load_3d(pb, &map_b, k * kTileK, o.n0, o.g, &sh.full[s]);
                    } else {
#pragma unroll
                        for (int p = 0; p < kPanels; ++p) {
                            if (kForm == kFormKN)
                                tma_load_3d(pb + p * kOperandBytes, &map_b, o.n0 + 128 * p, k * kTileK, o.g, &sh.full[s]);
                            else
                                tma_load_2d(pb + p * kOperandBytes, &map_b, o.n0 + 128 * p, o.k_base + k * kTileK, &sh.full[s]);
                        }
                    }
                }
            }
            if (!ok)   // copies in flight land before the CTA leaves
                for (uint32_t i = it < (uint32_t)kStages ? 0 : it - kStages; i < it; ++i)
                    mbar_wait_bounded(&sh.full[i % kStages], i / kStages & 1, 1ll << 24);
        }
    } else if (w == 1) {
        if (lane == 0) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
                const Tile o = tile_at<kForm, kN>(sh.table, a, t);
                if (o.k_tiles == 0) continue;
                const uint32_t acc = n % kAccs;
                if (!(ok = wait_or_abort(&sh.acc_empty[acc], (n / kAccs & 1) ^ 1, &sh.abort))) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * kN;
                for (int k = 0; k < o.k_tiles; ++k, ++it) {
                    const uint32_t s = it % kStages;
                    if (!(ok = wait_or_abort(&sh.full[s], it / kStages & 1, &sh.abort))) break;
                    tc_fence_after();
                    const uint32_t pa = smem_addr(sh.operands[s]), pb = pa + kOperandBytes, ps = smem_addr(sh.scales[s]);
                    const uint32_t ta = tmem + kScaleColumn + (it & 1) * 16, tb = ta + 4;
                    tc_copy_scales(ta, smem_desc(ps, 128, 128, 0));
#pragma unroll
                    for (int p = 0; p < kPanels; ++p) tc_copy_scales(tb + 4 * p, smem_desc(ps + 512 * (1 + p), 128, 128, 0));
                    // contraction inner: 8 rows x 128 bytes apart by 1024, a step of 32 is 32 bytes;
                    // contraction outer: panels of 128 columns, a step of 32 is 32 rows of 128 bytes
                    const uint64_t da = kOuterA ? smem_desc(pa, kOperandBytes, 1024, 2) : smem_desc(pa, 16, 1024, 2);
                    const uint64_t db = kOuterB ? smem_desc(pb, kOperandBytes, 1024, 2) : smem_desc(pb, 16, 1024, 2);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tc_mma_scaled(d, da + q * (kOuterA ? 256 : 2), db + q * (kOuterB ? 256 : 2),
                                      with_scale_byte(a.idesc, q), ta, tb, k > 0 || q > 0);
                    tc_commit(&sh.empty[s]);
                }
                if (ok) tc_commit(&sh.acc_full[acc]);
                ++n;
            }
            if (!ok) {   // matrix instructions in flight end before the tensor memory is freed
                tc_commit(&sh.drain);
                mbar_wait_bounded(&sh.drain, 0, 1ll << 24);
            }
        }
    } else if (w == 2) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
            const Tile o = tile_at<kForm, kN>(sh.table, a, t);
            if (kScales == kScales32) {
                if (lane == 0) {
                    const int nb = a.N < o.n0 + kN ? (a.N - o.n0 + 127) / 128 : kPanels;   // panels that exist
                    const uint8_t *sa = a.sa + (int64_t)o.scale_row * a.k_tiles * 512;
                    const uint8_t *sb = a.sb + ((int64_t)o.g * ((a.N + 127) / 128) + o.n0 / 128) * a.k_tiles * 512;
                    for (int k = 0; k < o.k_tiles; ++k, ++it) {
                        const uint32_t s = it % kStages;
                        if (!(ok = wait_or_abort(&sh.empty[s], (it / kStages & 1) ^ 1, &sh.abort))) break;
                        mbar_arrive_expect_tx(&sh.full[s], 512 * (1 + nb));
                        bulk_load(sh.scales[s], sa + (int64_t)k * 512, 512, &sh.full[s]);
                        for (int p = 0; p < nb; ++p)
                            bulk_load(sh.scales[s] + 512 * (1 + p), sb + ((int64_t)p * a.k_tiles + k) * 512, 512, &sh.full[s]);
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            } else {
                // four steps' bytes are loaded ahead of the four that are written
                const int b0 = o.k_base / kTileK;
                const int a_blocks = kForm == kFormOuter ? a.rows / kTileK : a.k_tiles;
                const int a_rows = kForm == kFormOuter ? a.M : a.rows;
                RowScales na, nb[kPanels];
                auto fetch = [&](int k) {
                    na = load_row_scales(a.sa, a.sa_row, a.sa_block, o.row0, a_rows, b0 + k, a_blocks, lane);
#pragma unroll
                    for (int p = 0; p < kPanels; ++p) {
                        if (kForm == kFormOuter) {
                            nb[p] = load_row_scales(a.sb, a.sb_row, a.sb_block, o.n0 + 128 * p, a.N, b0 + k, a_blocks, lane);
                        } else {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int n = o.n0 + 128 * p;
                                uint32_t b = 127;
                                if (n < a.N && k + u < o.k_tiles)
                                    b = a.sb[o.g * a.sb_group + (n / 128) * a.sb_row + (k + u) * a.sb_block];
                                nb[p].step[u] = b * 0x01010101u;
                            }
                        }
                    }
                };
                fetch(0);
                for (int k = 0; ok && k < o.k_tiles; k += 4) {
                    const RowScales ca = na;
                    RowScales cb[kPanels];
#pragma unroll
                    for (int p = 0; p < kPanels; ++p) cb[p] = nb[p];
                    if (k + 4 < o.k_tiles) fetch(k + 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (!ok || k + u >= o.k_tiles) break;
                        const uint32_t s = it % kStages;
                        ok = wait_or_abort(&sh.empty[s], (it / kStages & 1) ^ 1, &sh.abort);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        *reinterpret_cast<uint4 *>(sh.scales[s] + 16 * lane) = scale_line(ca.step[u]);
#pragma unroll
                        for (int p = 0; p < kPanels; ++p)
                            *reinterpret_cast<uint4 *>(sh.scales[s] + 512 * (1 + p) + 16 * lane) = scale_line(cb[p].step[u]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.full[s]);
                        ++it;
                    }
                }
            }
        }
    } else if (w >= 4) {
        const int quarter = w & 3;
        uint32_t n = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
            const Tile o = tile_at<kForm, kN>(sh.table, a, t);
            const uint32_t acc = n % kAccs;
            const bool empty = o.k_tiles == 0;   // a group with no rows: its product is zero
            if (!empty) {
                ok = wait_or_abort(&sh.acc_full[acc], n / kAccs & 1, &sh.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            const int r = quarter * 32 + lane;
            const int64_t at = (kForm == kFormOuter ? o.g * a.out_group : 0) + (int64_t)(o.row0 + r) * a.out_stride + o.n0;
            for (int c = 0; c < kN; c += 32) {
                uint32_t v[32];
                if (!empty) {
                    tc_load32(tmem + ((uint32_t)quarter << 21) + acc * kN + c, v);
                    tc_wait_load();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0;
                }
                const int valid = min(32, a.N - o.n0 - c);
                if (r < o.rows && valid > 0) {
                    if (a.out_type == 0) store_row(static_cast<float *>(a.out) + at + c, v, valid, a.wide_out);
                    else if (a.out_type == 1) store_row(static_cast<__nv_bfloat16 *>(a.out) + at + c, v, valid, a.wide_out);
                    else store_row(static_cast<__half *>(a.out) + at + c, v, valid, a.wide_out);
                }
            }
            if (!empty) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[acc]);
                ++n;
            }
        }
        if (kForm != kFormOuter) {   // rows behind the last group
            const int last = sh.table.begin[a.G - 1] + sh.table.size[a.G - 1];
            const int64_t cells = (int64_t)(a.rows - last) * a.N;
            for (int64_t i = (int64_t)blockIdx.x * 128 + (tid - 128); i < cells; i += (int64_t)gridDim.x * 128) {
                const int64_t r = i / a.N, at = (last + r) * a.out_stride + (i - r * a.N);
                if (a.out_type == 0) static_cast<float *>(a.out)[at] = 0.f;
                else static_cast<uint16_t *>(a.out)[at] = 0;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 3) tmem_free(tmem, kTmemColumns);
}

// ------------------------------------------------------------------ host side
constexpr int kMatMaxDevices = 128;

template <int kForm, int kScales, int kN>
mx_status launch_product(const CUtensorMap &ma, const CUtensorMap &mb, const MatArgs &a, int64_t tiles, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(Shared<kN>) + 1024;
    auto kernel = grouped_product<kForm, kScales, kN>;
    static std::mutex mu;
    static bool ready[kMatMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return mx_record_cuda_error(e);
    if (dev < 0 || dev >= kMatMaxDevices) return MX_ERR_UNSUPPORTED;
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); e != cudaSuccess)
                return mx_record_cuda_error(e);
            ready[dev] = true;
        }
    }
    return launch(kernel, tiles < sms ? tiles : sms, kMatThreads, smem, stream, ma, mb, a);
}

int out_code(mx_dtype t) { return t == MX_F32 ? 0 : t == MX_BF16 ? 1 : t == MX_F16 ? 2 : -1; }
bool eight(mx_dtype t) { return t == MX_E4M3 || t == MX_E5M2; }

bool operand_ok(const void *p, int64_t stride) { return aligned_to(p, 16) && stride % 16 == 0; }

}  // namespace
}  // namespace mx

// Read (and optionally clear) the product's error flags; part of mx_device_flags.
cudaError_t mx_matmul_flags(unsigned int *flags, int clear) {
    if (cudaError_t e = cudaMemcpyFromSymbol(flags, mx::g_matmul_flags, sizeof(*flags)); e != cudaSuccess) return e;
    if (clear) {
        const unsigned int zero = 0;
        if (cudaError_t e = cudaMemcpyToSymbol(mx::g_matmul_flags, &zero, sizeof(zero)); e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

extern "C" {

mx_status mx_grouped_matmul_m(const void *a, mx_dtype a_dtype, int64_t a_stride, const uint8_t *a_scales,
                              int64_t a_scale_row_stride, int64_t a_scale_block_stride, const void *b, mx_dtype b_dtype,
                              mx_b_layout b_layout, int64_t b_group_stride, int64_t b_stride, const uint8_t *b_scales,
                              int64_t b_scale_group_stride, int64_t b_scale_n_stride, int64_t b_scale_k_stride,
                              int32_t block, int64_t rows, int64_t n, int64_t k, const int32_t *group_ends,
                              int32_t num_groups, void *out, mx_dtype out_dtype, int64_t out_stride, cudaStream_t stream) {
    using namespace mx;
    if (!eight(a_dtype) || !eight(b_dtype) || out_code(out_dtype) < 0 || (block != 128 && block != 32)) return MX_ERR_INVALID_ARG;
    if (b_layout != MX_B_NK && b_layout != MX_B_KN) return MX_ERR_INVALID_ARG;
    if (num_groups < 1 || num_groups > MX_MAX_GROUPS || rows < 0 || n < 0 || k < 1) return MX_ERR_INVALID_ARG;
    if (rows > kOpsMaxExtent || n > kOpsMaxExtent || k > kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    const bool nk = b_layout == MX_B_NK;
    if (a_stride < k || b_stride < (nk ? k : n) || out_stride < n) return MX_ERR_INVALID_ARG;
    if (num_groups > 1 && b_group_stride < b_stride * ((nk ? n : k) - 1) + (nk ? k : n)) return MX_ERR_INVALID_ARG;
    if (block == 32 && !nk) return MX_ERR_UNSUPPORTED;
    if (rows == 0 || n == 0) return MX_OK;
    if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr || group_ends == nullptr || out == nullptr)
        return MX_ERR_INVALID_ARG;
    const int os = out_dtype == MX_F32 ? 4 : 2;
    if (!operand_ok(a, a_stride) || !operand_ok(b, b_stride) || (num_groups > 1 && b_group_stride % 16 != 0) ||
        !aligned_to(out, os) || !aligned_to(group_ends, 4))
        return MX_ERR_MISALIGNED;
    if (block == 32 && (!aligned_to(a_scales, 16) || !aligned_to(b_scales, 16))) return MX_ERR_MISALIGNED;

    MatArgs m = {};
    m.ends = group_ends;
    m.sa = a_scales;
    m.sb = b_scales;
    m.sa_row = a_scale_row_stride;
    m.sa_block = a_scale_block_stride;
    m.sb_group = b_scale_group_stride;
    m.sb_row = b_scale_n_stride;
    m.sb_block = b_scale_k_stride;
    m.out = out;
    m.out_stride = out_stride;
    m.G = num_groups;
    m.rows = (int32_t)rows;
    m.N = (int32_t)n;
    m.K = (int32_t)k;
    m.k_tiles = (int32_t)div_up(k, kTileK);
    m.out_type = out_code(out_dtype);
    m.wide_out = aligned_to(out, 16) && (out_stride * os) % 16 == 0;
    const int tile_n = 256;
    m.n_tiles = (int32_t)div_up(n, tile_n);
    m.idesc = block_scaled_idesc(a_dtype == MX_E5M2, b_dtype == MX_E5M2, false, !nk, kTileM, tile_n);
    const int64_t tiles = (div_up(rows, kTileM) + num_groups) * m.n_tiles;
    if (tiles > INT_MAX / 2) return MX_ERR_UNSUPPORTED;

    CUtensorMap ma, mb;
    const uint64_t da[2] = {(uint64_t)k, (uint64_t)rows}, sa[1] = {(uint64_t)a_stride};
    const uint32_t ba[2] = {128, 128};
    if (mx_status st = mx_encode_bytes_map(&ma, a, 2, da, sa, ba); st != MX_OK) return st;
    const uint64_t db[3] = {(uint64_t)(nk ? k : n), (uint64_t)(nk ? n : k), (uint64_t)num_groups};
    const uint64_t sb[2] = {(uint64_t)b_stride, (uint64_t)(num_groups > 1 ? b_group_stride : b_stride)};
    const uint32_t bb[3] = {128, nk ? (uint32_t)tile_n : 128u, 1};
    if (mx_status st = mx_encode_bytes_map(&mb, b, 3, db, sb, bb); st != MX_OK) return st;
    if (block == 32) return launch_product<kFormNK, kScales32, 256>(ma, mb, m, tiles, stream);
    if (nk) return launch_product<kFormNK, kScales128, 256>(ma, mb, m, tiles, stream);
    return launch_product<kFormKN, kScales128, 256>(ma, mb, m, tiles, stream);
}

mx_status mx_grouped_matmul_k(const void *a, mx_dtype a_dtype, int64_t a_stride, const uint8_t *a_scales,
                              int64_t a_scale_stride, const void *b, mx_dtype b_dtype, int64_t b_stride,
                              const uint8_t *b_scales, int64_t b_scale_stride, int64_t padded_rows, int64_t m, int64_t n,
                              const int32_t *group_ends, int32_t num_groups, void *out, mx_dtype out_dtype,
                              int64_t out_group_stride, int64_t out_stride, cudaStream_t stream) {
    using namespace mx;
    if (!eight(a_dtype) || !eight(b_dtype) || out_code(out_dtype) < 0) return MX_ERR_INVALID_ARG;
    if (num_groups < 1 || num_groups > MX_MAX_GROUPS || padded_rows < 128 || padded_rows % 128 != 0 || m < 0 || n < 0)
        return MX_ERR_INVALID_ARG;
    if (padded_rows > kOpsMaxExtent || m > kOpsMaxExtent || n > kOpsMaxExtent) return MX_ERR_INVALID_ARG;
    if (a_stride < m || b_stride < n || a_scale_stride < m || b_scale_stride < n || out_stride < n) return MX_ERR_INVALID_ARG;
    if (num_groups > 1 && m > 0 && out_group_stride < (m - 1) * out_stride + n) return MX_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return MX_OK;
    if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr || group_ends == nullptr || out == nullptr)
        return MX_ERR_INVALID_ARG;
    const int os = out_dtype == MX_F32 ? 4 : 2;
    if (!operand_ok(a, a_stride) || !operand_ok(b, b_stride) || !aligned_to(out, os) || !aligned_to(group_ends, 4))
        return MX_ERR_MISALIGNED;

    MatArgs g = {};
    g.ends = group_ends;
    g.sa = a_scales;
    g.sb = b_scales;
    g.sa_row = 1;
    g.sa_block = a_scale_stride;
    g.sb_row = 1;
    g.sb_block = b_scale_stride;
    g.out = out;
    g.out_stride = out_stride;
    g.out_group = num_groups > 1 ? out_group_stride : 0;
    g.G = num_groups;
    g.rows = (int32_t)padded_rows;
    g.M = (int32_t)m;
    g.N = (int32_t)n;
    g.out_type = out_code(out_dtype);
    g.wide_out = aligned_to(out, 16) && (out_stride * os) % 16 == 0 && (g.out_group * os) % 16 == 0;
    const int tile_n = 256;
    g.n_tiles = (int32_t)div_up(n, tile_n);
    g.m_tiles = (int32_t)div_up(m, kTileM);
    g.idesc = block_scaled_idesc(a_dtype == MX_E5M2, b_dtype == MX_E5M2, true, true, kTileM, tile_n);
    const int64_t tiles = (int64_t)g.m_tiles * g.n_tiles;
    if (tiles > INT_MAX / 2 / num_groups) return MX_ERR_UNSUPPORTED;

    CUtensorMap ma, mb;
    const uint64_t da[2] = {(uint64_t)m, (uint64_t)padded_rows}, sa[1] = {(uint64_t)a_stride};
    const uint64_t db[2] = {(uint64_t)n, (uint64_t)padded_rows}, sb[1] = {(uint64_t)b_stride};
    const uint32_t box[2] = {128, 128};
    if (mx_status st = mx_encode_bytes_map(&ma, a, 2, da, sa, box); st != MX_OK) return st;
    if (mx_status st = mx_encode_bytes_map(&mb, b, 2, db, sb, box); st != MX_OK) return st;
    return launch_product<kFormOuter, kScales128, 256>(ma, mb, g, tiles * num_groups, stream);
}

}  // extern "C"
