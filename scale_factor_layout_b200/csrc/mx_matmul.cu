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
// A CTA, or a pair of CTAs of a cluster, per SM (or two) walks output tiles of
// kTileRows x kN.  The warps of a CTA: 0 loads operands by TMA into a ring of
// stages of 128 along the contraction; 1 issues the matrix instructions (in a
// pair, that of rank 0 for both); 2 and 3 bring the scales, each for every
// other stage; 4..11 empty the accumulators into the output, two warps for
// each quarter of the rows.  A pair works on 256 rows x 256 columns: each CTA
// holds 128 rows of a and half of b's 256, so a stage brings 32 KB for the work
// that takes 48 KB alone.  Shared memory bounds the loop (a stage is written
// once and read once, 128 bytes a clock), so that is what a pair wins.
// Where there are too few tiles for the SMs (few rows, few groups), tiles are
// 128 x 128 and the contraction of one is split over a cluster of CTAs, which
// add their parts up through each other's shared memory, in the order of the
// parts.
// Operands whose contraction is the outer dimension in memory (weights read
// for the input gradient, both operands of the weight gradient) are loaded as
// they are and read through descriptors of that order: nothing is transposed
// in memory.
//
// On a B200, 8192 x 8192 x 8192 takes 385 us (2.85 PFLOP/s; a stage of the loop
// 530 clocks, 512 of them the matrix instructions'), and 446 us (2.46 PFLOP/s)
// after seconds of it, when the power limit holds the SMs near 1.3 GHz; a
// library product of the same operands without scales per block takes 357 and
// 418.  131072 x 1408 x 7168 in 8 ragged groups: 1140 to 1180 us of it (2.25 to 2.33
// PFLOP/s), 960 us on a cool GPU.  Few rows are bound by the weights' bytes: 128 rows
// over 64 experts of 1408 x 7168, about 50 of them in use, 88 to 106 us by the GPU, 4.8
// to 5.7 TB/s.
//
// The sums are those of the tensor cores: 32 bits, but cut rather than rounded
// at each step of 32, and in one accumulator however long they are; sums of 8192
// positive products are off by 3.7e-6, of 131072 by 1.5e-4 at most.

#include <climits>
#include <mutex>

#include "mx_ops.cuh"
#include "mx_tcgen05.cuh"

// A tensor map over bytes with a swizzle, or over 32-bit words without (defined in mx_rearrange.cu).
mx_status mx_encode_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                        const uint32_t *box, CUtensorMapSwizzle swizzle);

namespace mx {
namespace {

__device__ unsigned int g_matmul_flags = 0;

enum Form { kFormNK = 0, kFormKN = 1, kFormOuter = 2 };
enum ScaleForm { kScales128 = 0, kScales32 = 1 };

constexpr int kTileK = 128;
constexpr int kMatThreads = 384;
constexpr int kDrainWarps = 8;
constexpr int kOutRow = 64, kOutBytes = 32 * kOutRow;   // bytes of a row, and of a warp's rows, in a store
constexpr int kPanelBytes = 128 * kTileK;   // 128 rows (or columns) of an operand in a stage
constexpr int kTmemColumns = 512;
constexpr int kScaleColumn = 480;           // 2 sets of 4 + 8 columns of scales
constexpr int kTileSlots = 4;
constexpr int kStrip = 8;                   // tiles of a strip of columns

struct MatArgs {
    const int *ends;
    const uint8_t *sa, *sb;
    int64_t sa_row, sa_block;               // bytes between scales along rows and along the contraction
    int64_t sb_group, sb_row, sb_block;
    void *out;
    int64_t out_stride, out_group;          // elements
    int32_t G, rows;                        // rows: of a (row groups), of both operands (contraction groups)
    int32_t M, N;                           // M: contraction groups only
    int32_t n_tiles, m_tiles, k_tiles;      // m_tiles: contraction groups only
    int32_t out_type;                       // 0 f32, 1 bf16, 2 f16
    uint32_t idesc;
    bool tma_out;                           // out's rows start and end on 16-byte boundaries
    bool swapped;                           // contraction groups: tiles are of out's transpose
};

struct Maps { CUtensorMap a, b, sa, sb, out; };   // sa, sb: scales of 32 only

template <int kScales, int kN, bool kPair>
struct Shared {
    static constexpr int kTileRows = kPair ? 256 : 128;
    static constexpr int kPanels = kN / 128;                  // 128-column panels of the tile
    static constexpr int kPanelsHere = kPair ? 1 : kPanels;   // of them in this CTA
    static constexpr int kStages = 192 / (16 + 16 * kPanelsHere);
    static constexpr int kStageBytes = (1 + kPanelsHere) * kPanelBytes;
    static constexpr int kScaleBytes = (1 + kPanels) * 512;
    // scales of 128: a slot holds those of four stages; of 32: of one, and comes with its operands
    static constexpr int kScaleSlots = kScales == kScales128 ? 4 : kStages;
    alignas(1024) uint8_t operands[kStages][kStageBytes];
    alignas(1024) uint8_t out[kDrainWarps][kOutBytes];
    alignas(128) uint8_t scales[kScaleSlots][kScaleBytes];
    GroupTable table;
    alignas(8) uint64_t full[kStages], empty[kStages], scale_full[kScaleSlots], scale_empty[kScaleSlots];
    alignas(8) uint64_t acc_full, acc_empty, drain;
    alignas(16) uint4 answer;   // about a cancelled launch
    alignas(8) uint64_t answered, tile_full[kTileSlots], tile_empty[kTileSlots];
    int tiles[kTileSlots];
    uint32_t tmem;
    volatile int abort;
};

struct Tile {
    int32_t g, row0, rows, n0, n, k_tiles;   // n: columns of the tile, a multiple of 32; row0: this CTA's first row of a (row groups) or column of a (contraction groups)
    int32_t k_base;                       // contraction groups: first row of the operands
    int32_t scale_row;                    // scales of 32: the 128-row tile of a's scales
};

// The group table in a warp's registers: lane l holds groups l and l + 32.  A
// role looks a tile up between two tiles, where the tensor cores wait for it, so
// the search is two ballots and not six dependent loads, and no division is a
// full one.
struct Groups {
    int first0, first1;   // tiles of rows before the group
    int tiles;            // of all groups
    int begin0, begin1, size0, size1, pstart0, pstart1;
    __device__ __forceinline__ Groups(const GroupTable &t, int tile_rows, int lane)
        : begin0(t.begin[lane]), begin1(t.begin[lane + 32]), size0(t.size[lane]), size1(t.size[lane + 32]),
          pstart0(t.pstart[lane]), pstart1(t.pstart[lane + 32]) {
        const int n0 = (size0 + tile_rows - 1) / tile_rows, n1 = (size1 + tile_rows - 1) / tile_rows;
        const int s0 = warp_scan_sum(n0, lane);
        const int s1 = warp_scan_sum(n1, lane) + __shfl_sync(0xffffffffu, s0, 31);
        first0 = s0 - n0;
        first1 = s1 - n1;
        tiles = __shfl_sync(0xffffffffu, s1, 31);
    }
    // the group of tile v of rows: the last one that starts at or before it
    __device__ __forceinline__ int find(int v) const {
        return __popc(__ballot_sync(0xffffffffu, first0 <= v)) + __popc(__ballot_sync(0xffffffffu, first1 <= v)) - 1;
    }
    __device__ __forceinline__ static int of(int lo, int hi, int g) {
        return __shfl_sync(0xffffffffu, g < 32 ? lo : hi, g & 31);
    }
    __device__ __forceinline__ int last_end() const { return __shfl_sync(0xffffffffu, begin1 + size1, 31); }
};

// n / d for n >= 0, d > 0: a rounded quotient is at most one off below 2^22.
__device__ __forceinline__ int quotient(int n, int d) {
    if (n >= 1 << 22) return n / d;
    int q = (int)__fdividef((float)n, (float)d);
    const int r = n - q * d;
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}

// Tiles of a group go in strips of kStrip tiles of columns, row by row within
// a strip, so that the tiles in flight share both operands in L2.  Behind the
// groups' tiles come those of the rows behind the last group, which have no
// contraction and are written as zeros.
template <int kForm, int kN, int kTileRows>
__device__ __forceinline__ Tile tile_at(const Groups &groups, int row_tiles, const MatArgs &a, int t, int rank) {
    Tile o;
    if (kForm != kFormOuter && t >= row_tiles * a.n_tiles) {
        t -= row_tiles * a.n_tiles;
        const int mt = quotient(t, a.n_tiles);
        o.g = 0;
        o.row0 = groups.last_end() + mt * kTileRows + rank * 128;
        o.rows = min(128, a.rows - o.row0);
        o.n0 = (t - mt * a.n_tiles) * kN;
        o.n = kN;
        o.k_base = o.k_tiles = o.scale_row = 0;
        return o;
    }
    int local, m_tiles;
    if (kForm == kFormOuter) {
        m_tiles = a.m_tiles;
        o.g = quotient(t, m_tiles * a.n_tiles);
        local = t - o.g * (m_tiles * a.n_tiles);
    } else {
        o.g = groups.find(quotient(t, a.n_tiles));
        local = t - Groups::of(groups.first0, groups.first1, o.g) * a.n_tiles;
        m_tiles = (Groups::of(groups.size0, groups.size1, o.g) + kTileRows - 1) / kTileRows;
    }
    const int strip = quotient(local, m_tiles * kStrip);
    local -= strip * m_tiles * kStrip;
    const int width = min(kStrip, a.n_tiles - strip * kStrip);
    const int mt = quotient(local, width), nt = strip * kStrip + local - mt * width;
    const int row = mt * kTileRows + rank * 128;
    const int size = Groups::of(groups.size0, groups.size1, o.g), pstart = Groups::of(groups.pstart0, groups.pstart1, o.g);
    o.n0 = nt * kN;
    o.n = min(kN, (a.N - o.n0 + 31) & ~31);
    if (kForm == kFormOuter) {
        o.row0 = row;
        o.rows = min(128, a.M - row);
        o.k_base = pstart;
        o.k_tiles = (size + kTileK - 1) / kTileK;
        o.scale_row = 0;
    } else {
        o.row0 = Groups::of(groups.begin0, groups.begin1, o.g) + row;
        o.rows = min(128, size - row);
        o.k_base = 0;
        o.k_tiles = a.k_tiles;
        o.scale_row = (pstart + row) / 128;
    }
    return o;   // rows may be 0 or less in the second CTA of a pair
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

// Scale bytes of rows lane + 32 i of a panel for four steps of the contraction:
// a line of the 128 x 4 tile.  Rows past the last are read as the last one,
// since what they scale is not stored; so are steps.
struct LineSource {
    const uint8_t *p[4];
    __device__ __forceinline__ LineSource() {}
    __device__ __forceinline__ LineSource(const uint8_t *s, int64_t stride, int row0, int rows, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = s + (int64_t)max(0, min(row0 + lane + 32 * i, rows - 1)) * stride;
    }
    __device__ __forceinline__ void load(uint32_t (&b)[16], int k, int last, int64_t stride) const {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t at = (int64_t)min(k + u, last) * stride;
#pragma unroll
            for (int i = 0; i < 4; ++i) b[4 * i + u] = __ldg(p[i] + at);
        }
    }
};
__device__ __forceinline__ uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return a | b << 8 | c << 16 | d << 24;
}
__device__ __forceinline__ uint4 tile_line(const uint32_t (&b)[16]) {
    return make_uint4(four_bytes(b[0], b[1], b[2], b[3]), four_bytes(b[4], b[5], b[6], b[7]),
                      four_bytes(b[8], b[9], b[10], b[11]), four_bytes(b[12], b[13], b[14], b[15]));
}

template <typename T>
__device__ __forceinline__ void store_row(void *out, int64_t at, const uint32_t *v, int valid) {
    T *dst = static_cast<T *>(out) + at;
    constexpr int N = 16 / sizeof(T);
    if (valid >= 32) {
#pragma unroll
        for (int i = 0; i < 32; i += N) {
            float f[N];
#pragma unroll
            for (int u = 0; u < N; ++u) f[u] = __uint_as_float(v[i + u]);
            *reinterpret_cast<uint4 *>(dst + i) = pack<T, N>(f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < valid) dst[i] = from_f32<T>(__uint_as_float(v[i]));
    }
}

// This lane's values, `stride` elements apart.
template <typename T, int n>
__device__ __forceinline__ void store_across(void *out, int64_t at, int64_t stride, const uint32_t (&v)[n], int valid) {
    T *p = static_cast<T *>(out) + at;
#pragma unroll
    for (int c = 0; c < n; ++c, p += stride)
        if (c < valid) *p = from_f32<T>(__uint_as_float(v[c]));
}

// 64 bytes of this lane's row into the warp's box of 32 rows, with the 64-byte
// swizzle: 16-byte piece c of row r sits at piece c ^ (r / 2 % 4).
template <typename T>
__device__ __forceinline__ void stage_row(uint8_t *box, const uint32_t *v, int lane) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float f[N];
#pragma unroll
        for (int u = 0; u < N; ++u) f[u] = __uint_as_float(v[c * N + u]);
        *reinterpret_cast<uint4 *>(box + lane * kOutRow + ((c ^ (lane >> 1 & 3)) << 4)) = pack<T, N>(f);
    }
}

// The box's rows into rows of `out` that start anywhere: a half or whole warp
// writes the 64 bytes of a row, so that a store touches two lines at most and not
// 32.
template <typename W>
__device__ __forceinline__ void store_box(const uint8_t *box, W *out, int64_t at, int64_t stride, int rows, int cols, int lane) {
    constexpr int kLine = kOutRow / sizeof(W), kAtOnce = 32 / kLine;   // elements of a row; rows of a store
    const int e = lane % kLine, piece = e * sizeof(W) / 16, byte = e * sizeof(W) % 16;
#pragma unroll 8
    for (int r = lane / kLine; r < rows; r += kAtOnce)
        if (e < cols) out[at + r * stride + e] = *reinterpret_cast<const W *>(box + r * kOutRow + ((piece ^ (r >> 1 & 3)) << 4) + byte);
}

// The tiles of a CTA (of a pair).  The first is its own block's; for each that it
// begins, the producer of rank 0 cancels the launch of a block that has not
// started, takes over its tile and tells every warp.  So faster SMs do more
// tiles, which the clocks and distances to memory of 148 SMs, groups' uneven
// ends and narrow last columns of tiles all ask for.
template <typename Sh, bool kPair>
struct TileStream {
    Sh &sh;
    uint32_t n = 0;
    int tile;
    __device__ __forceinline__ TileStream(Sh &s, int first) : sh(s), tile(first) {}
    // For the warps that are told: the next tile; false after the last.
    __device__ __forceinline__ bool next(int lane) {
        const uint32_t slot = n % kTileSlots;
        const bool ok = wait_or_abort(&sh.tile_full[slot], n / kTileSlots & 1, &sh.abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tile = *reinterpret_cast<volatile int *>(&sh.tiles[slot]);
        // The arrival lets the slot be overwritten, and must not overtake the load: behind a
        // queue of stores that can take longer than the arrival and the next announcement.  The
        // vote needs every lane's value (all are -1 or more), and the arrival needs the vote.
        if (__all_sync(0xffffffffu, tile >= -1) && lane == 0) mbar_arrive_at(leader_addr<kPair>(&sh.tile_empty[slot]));
        ++n;
        return tile >= 0;
    }
    // For the producer of rank 0: ask for a tile, and take and announce it.
    __device__ __forceinline__ void ask() {
        if (elect_one()) {
            mbar_arrive_expect_tx(&sh.answered, 16);
            cancel_launch(&sh.answer, &sh.answered);
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool take() {
        const uint32_t slot = n % kTileSlots;
        bool ok = wait_or_abort(&sh.answered, n & 1, &sh.abort);
        ok = ok && wait_or_abort(&sh.tile_empty[slot], (n / kTileSlots & 1) ^ 1, &sh.abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        tile = cancelled_block(&sh.answer);
        if (tile >= 0) tile /= kPair ? 2 : 1;
        fence_proxy_async_smem();   // the answer is read before the next one is written
        __syncwarp();
        if (elect_one()) {
#pragma unroll
            for (int c = 0; c < (kPair ? 2 : 1); ++c) {
                const uint32_t bar = addr_in<kPair>(&sh.tile_full[slot], c);
                mbar_expect_at(bar, 4);
                store_word_at(addr_in<kPair>(&sh.tiles[slot], c), (uint32_t)tile, bar);
            }
        }
        __syncwarp();
        ++n;
        return tile >= 0;
    }
};

// The parts of a split tile, added up.  Each CTA of the cluster owns an equal
// share of the tile's columns and gets the other parts' values of them in its
// stages, which no load or matrix instruction uses any more once all have
// emptied their accumulators (the first barrier); after the second it adds them
// in the order of the parts and writes them out.
template <int kForm, int kN>
__device__ __forceinline__ void add_parts(uint8_t *stages, const Tile &o, const MatArgs &a, const uint32_t (&v)[kN / 2],
                                          int part, int parts, int row, int half, int thread) {
    const int share = kN / parts;   // columns of a CTA: 16 to 64
    // [part][128][share], rows 4 words further apart: a warp writes 32 rows at once, 16 bytes of
    // each, which a distance of 64, 128 or 256 bytes would put into the same banks
    float *mine = reinterpret_cast<float *>(stages);
    const int pitch = share + 4;
    __syncwarp();
    cluster_sync();
    if (row < o.rows) {
#pragma unroll
        for (int c = 0; c < kN / 2; c += 4) {
            const int col = half * (kN / 2) + c, owner = col / share;
            float *at = mine + (part * 128 + row) * pitch + (col - owner * share);
            if (owner == part) *reinterpret_cast<uint4 *>(at) = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
            else asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};"
                              ::"r"(addr_in<true>(at, owner)), "r"(v[c]), "r"(v[c + 1]), "r"(v[c + 2]), "r"(v[c + 3]) : "memory");
        }
    }
    __syncwarp();
    cluster_sync();
    const int es = a.out_type == 0 ? 4 : 2;
    for (int i = thread; i < 128 * share / 8; i += 32 * kDrainWarps) {   // eight columns of a row at a time
        const int r = i / (share / 8), c0 = (i - r * (share / 8)) * 8, n = o.n0 + part * share + c0;
        if (r >= o.rows || n >= a.N) continue;
        float sum[8] = {};
        for (int q = 0; q < parts; ++q) {
            const float4 *src = reinterpret_cast<const float4 *>(mine + (q * 128 + r) * pitch + c0);
            const float4 x = src[0], y = src[1];
            sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
            sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
        }
        const int64_t at = (kForm == kFormOuter ? o.g * a.out_group : 0) + (int64_t)(o.row0 + r) * a.out_stride + n;
        if (a.tma_out && es == 2) {   // N is then a multiple of 8
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) =
                a.out_type == 1 ? pack<__nv_bfloat16, 8>(sum) : pack<__half, 8>(sum);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (n + u >= a.N) break;
                if (a.out_type == 0) static_cast<float *>(a.out)[at + u] = sum[u];
                else if (a.out_type == 1) static_cast<__nv_bfloat16 *>(a.out)[at + u] = from_f32<__nv_bfloat16>(sum[u]);
                else static_cast<__half *>(a.out)[at + u] = from_f32<__half>(sum[u]);
            }
        }
    }
}

// Steps of the contraction that part `part` of `parts` takes: whole slots of scales.
__device__ __forceinline__ int split_begin(int k_tiles, int part, int parts) {
    const int each = ((k_tiles + parts - 1) / parts + 3) & ~3;
    return min(k_tiles, part * each);
}

enum Work { kAlone = 0, kPairs = 1, kSplits = 2 };   // a CTA, two CTAs, or a cluster of parts a tile

template <int kForm, int kScales, int kN, int kWork>
__global__ void __launch_bounds__(kMatThreads, 1)
grouped_product(const __grid_constant__ Maps maps, const MatArgs a) {
    constexpr bool kPair = kWork == kPairs, kSplit = kWork == kSplits;
    using Sh = Shared<kScales, kN, kPair>;
    constexpr int kScaleSlots = Sh::kScaleSlots;
    constexpr int kStages = Sh::kStages, kPanels = Sh::kPanels, kPanelsHere = Sh::kPanelsHere, kTileRows = Sh::kTileRows;
    constexpr bool kOuterA = kForm == kFormOuter, kOuterB = kForm != kFormNK;
    constexpr int kCtas = kPair ? 2 : 1;
    constexpr int kScaleSteps = kScales == kScales128 ? 4 : 1;   // stages whose scales are in one slot
    extern __shared__ uint8_t dyn_smem[];
    Sh &sh = *reinterpret_cast<Sh *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rank = kPair ? (int)cluster_rank() : 0;

    if (w == 0 && lane == 0) {
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], kCtas);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.scale_full[i], kCtas);
            mbar_init(&sh.scale_empty[i], 1);
        }
        mbar_init(&sh.acc_full, 1);
        mbar_init(&sh.acc_empty, kDrainWarps * kCtas);
        mbar_init(&sh.drain, 1);
        mbar_init(&sh.answered, 1);
        for (int i = 0; i < kTileSlots; ++i) {
            mbar_init(&sh.tile_full[i], 1);
            // the matrix warp, the scale warps, the draining warps, the other CTA's producer
            mbar_init(&sh.tile_empty[i], 1 + (kScales == kScales128 ? 2 : 0) * kCtas + kDrainWarps * kCtas + (kCtas - 1));
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    __syncwarp();
    grid_dependency_wait();
    if (w == 3) tmem_alloc<kPair>(&sh.tmem, kTmemColumns);
    if (w == 2) build_group_table<true>(a.ends, a.G, a.rows, 1, sh.table);
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();   // the barriers are there before the other CTA arrives on them
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const Groups groups(sh.table, kTileRows, lane);
    const int row_tiles = groups.tiles;
    // tiles in all: the launch has an upper bound of blocks, the last of them without work
    const int total = kForm == kFormOuter ? a.G * a.m_tiles * a.n_tiles
                                          : (row_tiles + (a.rows - groups.last_end() + kTileRows - 1) / kTileRows) * a.n_tiles;
    // a split tile is its cluster's only one
    const int parts = kSplit ? (int)cluster_size() : 1, part = kSplit ? (int)cluster_rank() : 0;
    TileStream<Sh, kPair> tiles(sh, blockIdx.x / (kSplit ? parts : kCtas));

    if (w == 0) {
        uint32_t it = 0;
        bool ok = true;
        do {
            if (!kSplit && rank == 0) tiles.ask();
            if (tiles.tile >= total) continue;
            const Tile o = tile_at<kForm, kN, kTileRows>(groups, row_tiles, a, tiles.tile, rank);
            const int k_begin = kSplit ? split_begin(o.k_tiles, part, parts) : 0;
            const int k_end = kSplit ? split_begin(o.k_tiles, part + 1, parts) : o.k_tiles;
            const int n0 = o.n0 + (kPair ? rank * (o.n / 2) : 0);
            const int panels = (o.n + 127) / 128;   // of scales of 32
            const int sb0 = (o.g * ((a.N + 127) / 128) + o.n0 / 128) * a.k_tiles;
            for (int k = k_begin; k < k_end; ++k, ++it) {
                const uint32_t s = it % kStages, phase = it / kStages & 1;
                ok = __all_sync(0xffffffffu, wait_or_abort(&sh.empty[s], phase ^ 1, &sh.abort));
                if (!ok) break;
                if (elect_one()) {
                    uint8_t *pa = sh.operands[s], *pb = pa + kPanelBytes;
                    const uint32_t full = leader_addr<kPair>(&sh.full[s]);
                    mbar_expect_at(full, Sh::kStageBytes + (kScales == kScales32 ? 512 * ((o.rows > 0) + panels) : 0));
                    if (kScales == kScales32) {
                        if (o.rows > 0) tma_load_2d_to<kPair>(sh.scales[s], &maps.sa, 0, o.scale_row * a.k_tiles + k, full);
                        for (int p = 0; p < panels; ++p)
                            tma_load_2d_to<kPair>(sh.scales[s] + 512 * (1 + p), &maps.sb, 0, sb0 + p * a.k_tiles + k, full);
                    }
                    if (kOuterA) tma_load_2d_to<kPair>(pa, &maps.a, o.row0, o.k_base + k * kTileK, full);
                    else tma_load_2d_to<kPair>(pa, &maps.a, k * kTileK, o.row0, full);
                    if (kForm == kFormNK) {
                        tma_load_3d_to<kPair>(pb, &maps.b, k * kTileK, n0, o.g, full);
                    } else {
#pragma unroll
                        for (int p = 0; p < kPanelsHere; ++p) {
                            if (kForm == kFormKN)
                                tma_load_3d_to<kPair>(pb + p * kPanelBytes, &maps.b, n0 + 128 * p, k * kTileK, o.g, full);
                            else
                                tma_load_2d_to<kPair>(pb + p * kPanelBytes, &maps.b, n0 + 128 * p, o.k_base + k * kTileK, full);
                        }
                    }
                }
                __syncwarp();
            }
        } while (!kSplit && ok && (rank == 0 ? tiles.take() : tiles.next(lane)));
        if (sh.abort) {   // copies in flight, a few microseconds' worth, land before the CTA leaves
            const long long t0 = clock64();
            while (clock64() - t0 < (1ll << 22)) {}
        }
    } else if (w == 1) {
        uint32_t it = 0, n = 0, sc = 0;
        bool ok = rank == 0;
        // contraction inner: 8 rows x 128 bytes apart by 1024, a step of 32 is 32 bytes;
        // contraction outer: panels of 128 columns, a step of 32 is 32 rows of 128 bytes
        const uint32_t p0 = smem_addr(sh.operands[0]), s0 = smem_addr(sh.scales[0]);
        const uint64_t desc_a = smem_desc(p0, kOuterA ? kPanelBytes : 16, 1024, 2);
        const uint64_t desc_b = smem_desc(p0 + kPanelBytes, kOuterB ? kPanelBytes : 16, 1024, 2);
        const uint64_t desc_s = smem_desc(s0, 128, 128, 0);
        if (ok) do {
            if (tiles.tile >= total) continue;
            const Tile o = tile_at<kForm, kN, kTileRows>(groups, row_tiles, a, tiles.tile, 0);
            const int k_begin = kSplit ? split_begin(o.k_tiles, part, parts) : 0;
            const int k_end = kSplit ? split_begin(o.k_tiles, part + 1, parts) : o.k_tiles;
            if (k_begin == k_end) continue;
            const uint32_t idesc = a.idesc | (uint32_t)(o.n / 8) << 17 | (uint32_t)(kTileRows / 16) << 24;
            ok = __all_sync(0xffffffffu, wait_or_abort(&sh.acc_empty, (n & 1) ^ 1, &sh.abort));
            if (!ok) break;
            tc_fence_after();
            for (int k = k_begin; k < k_end; ++k, ++it) {
                const uint32_t s = it % kStages, slot = sc % kScaleSlots;
                const bool scales = k % kScaleSteps == 0;   // this stage brings new ones
                if (kScales == kScales128 && scales)
                    ok = __all_sync(0xffffffffu, wait_or_abort(&sh.scale_full[slot], sc / kScaleSlots & 1, &sh.abort));
                ok = ok && __all_sync(0xffffffffu, wait_or_abort(&sh.full[s], it / kStages & 1, &sh.abort));
                if (!ok) break;
                tc_fence_after();
                if (scales) ++sc;
                const uint32_t ta = tmem + kScaleColumn + ((sc - 1) & 1) * 16, tb = ta + 4;
                if (elect_one()) {
                    if (scales) {
                        const uint64_t ds = desc_s + slot * (Sh::kScaleBytes / 16);
                        tc_copy_scales<kPair>(ta, ds);
#pragma unroll
                        for (int p = 0; p < kPanels; ++p) tc_copy_scales<kPair>(tb + 4 * p, ds + 32 * (1 + p));
                        if (kScales == kScales128) tc_commit<kPair>(&sh.scale_empty[slot]);
                    }
                    const uint64_t da = desc_a + s * (Sh::kStageBytes / 16), db = desc_b + s * (Sh::kStageBytes / 16);
                    // scales of 128: the stage's byte for all four steps; of 32: a byte a step
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        tc_mma_scaled<kPair>(tmem, da + q * (kOuterA ? 256 : 2), db + q * (kOuterB ? 256 : 2),
                                             with_scale_byte(idesc, kScaleSteps == 4 ? k & 3 : q), ta, tb, k > k_begin || q > 0);
                    tc_commit<kPair>(&sh.empty[s]);
                    if (k == k_end - 1) tc_commit<kPair>(&sh.acc_full);
                }
                __syncwarp();
            }
            ++n;
        } while (!kSplit && ok && tiles.next(lane));
        if (sh.abort && rank == 0) {   // matrix instructions in flight end before the tensor memory is freed
            if (elect_one()) tc_commit<kPair>(&sh.drain);
            __syncwarp();
            mbar_wait_bounded(&sh.drain, 0, 1ll << 24);
        }
    } else if (w < 4) {
        uint32_t sc = 0;   // slots before this tile; a warp fills every other one
        const uint32_t half = w & 1;
        bool ok = kScales == kScales128;
        if (ok) do {
            if (tiles.tile >= total) continue;
            const Tile o = tile_at<kForm, kN, kTileRows>(groups, row_tiles, a, tiles.tile, rank);
            const int k_begin = kSplit ? split_begin(o.k_tiles, part, parts) : 0;
            const int k_end = kSplit ? split_begin(o.k_tiles, part + 1, parts) : o.k_tiles;
            const int slots = (k_end - k_begin + kScaleSteps - 1) / kScaleSteps;
            constexpr bool kRowsB = kForm == kFormOuter;
            const int b0 = o.k_base / kTileK + k_begin;
            const int last = (kRowsB ? a.rows / kTileK : a.k_tiles) - 1;   // last step whose scales exist
            const LineSource sa(a.sa, a.sa_row, o.row0, kRowsB ? a.M : a.rows, lane);
            LineSource sb[kPanels];
            const uint8_t *sq[kPanels];
#pragma unroll
            for (int p = 0; p < kPanels; ++p) {
                if (kRowsB) sb[p] = LineSource(a.sb, a.sb_row, o.n0 + 128 * p, a.N, lane);
                else sq[p] = a.sb + o.g * a.sb_group + min(o.n0 / 128 + p, (a.N - 1) / 128) * a.sb_row;
            }
            for (int i = (sc ^ half) & 1; i < slots; i += 2) {
                // the bytes are on their way while the slot is still in use
                uint32_t ba[16], bb[kPanels][16];
                sa.load(ba, b0 + 4 * i, last, a.sa_block);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    if (kRowsB) {
                        sb[p].load(bb[p], b0 + 4 * i, last, a.sb_block);
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u) bb[p][u] = __ldg(sq[p] + min(k_begin + 4 * i + u, last) * a.sb_block);
                    }
                }
                const uint32_t s = (sc + i) % kScaleSlots;
                ok = wait_or_abort(&sh.scale_empty[s], ((sc + i) / kScaleSlots & 1) ^ 1, &sh.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint4 *to = reinterpret_cast<uint4 *>(sh.scales[s]) + lane;
                to[0] = tile_line(ba);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    const uint32_t q = four_bytes(bb[p][0], bb[p][1], bb[p][2], bb[p][3]);
                    to[32 * (1 + p)] = kRowsB ? tile_line(bb[p]) : make_uint4(q, q, q, q);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_release_at(leader_addr<kPair>(&sh.scale_full[s]));
            }
            sc += slots;
        } while (!kSplit && ok && tiles.next(lane));
    } else {
        const int quarter = w & 3, part_of_columns = (w - 4) >> 2;   // rows 32 * quarter.., columns part_of_columns * kN / 2..
        constexpr int kCols = kN / 2;
        uint32_t n = 0;
        bool ok = true;
        do {
            if (tiles.tile >= total) continue;
            const Tile o = tile_at<kForm, kN, kTileRows>(groups, row_tiles, a, tiles.tile, rank);
            uint32_t v[kCols];
            if (kSplit ? split_begin(o.k_tiles, part, parts) < split_begin(o.k_tiles, part + 1, parts) : o.k_tiles > 0) {
                ok = wait_or_abort(&sh.acc_full, n & 1, &sh.abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // all of it into registers, so that the next tile can begin
#pragma unroll
                for (int c = 0; c < kCols; c += 32)
                    tc_load32(tmem + ((uint32_t)quarter << 21) + part_of_columns * kCols + c, v + c);
                tc_wait_load();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(leader_addr<kPair>(&sh.acc_empty));
                ++n;
            } else {   // a group with no rows (or a part with no steps): its product is zero
#pragma unroll
                for (int i = 0; i < kCols; ++i) v[i] = 0;
            }
            if (kSplit) {
                add_parts<kForm, kN>(sh.operands[0], o, a, v, part, parts, quarter * 32 + lane, part_of_columns, tid - 128);
                continue;
            }
            const int r0 = quarter * 32, n0 = o.n0 + part_of_columns * kCols, es = a.out_type == 0 ? 4 : 2;
            const int wanted = a.N - n0;   // columns from n0 on that exist
            if (kForm == kFormOuter && kPair && a.swapped) {
                // a lane's row is a column of out: 32 lanes write 32 neighbours of each of their columns
                const int64_t at = o.g * a.out_group + (int64_t)n0 * a.out_stride + o.row0 + r0 + lane;
                if (r0 + lane < o.rows) {
                    if (a.out_type == 0) store_across<float, kCols>(a.out, at, a.out_stride, v, wanted);
                    else if (a.out_type == 1) store_across<__nv_bfloat16, kCols>(a.out, at, a.out_stride, v, wanted);
                    else store_across<__half, kCols>(a.out, at, a.out_stride, v, wanted);
                }
            } else if (a.tma_out && r0 + 32 <= o.rows) {
                // whole rows of the warp: through shared memory, since a lane holds a row and
                // 32 rows a store instruction would be 32 separate lines
                uint8_t *box = sh.out[w - 4];
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    if (es == 2 && c % 32 != 0) continue;
                    if (c >= wanted) break;
                    if (lane == 0) bulk_wait_read<0>();   // the box is free
                    __syncwarp();
                    if (a.out_type == 0) stage_row<float>(box, v + c, lane);
                    else if (a.out_type == 1) stage_row<__nv_bfloat16>(box, v + c, lane);
                    else stage_row<__half>(box, v + c, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&maps.out, (n0 + c) * es, o.row0 + r0, kForm == kFormOuter ? o.g : 0, box);
                        bulk_commit();
                    }
                }
            } else if (a.tma_out) {   // some rows of the warp
                if (r0 + lane < o.rows) {
                    const int64_t at = (kForm == kFormOuter ? o.g * a.out_group : 0) + (int64_t)(o.row0 + r0 + lane) * a.out_stride + n0;
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        const int valid = wanted - c;
                        if (a.out_type == 0) store_row<float>(a.out, at + c, v + c, valid);
                        else if (a.out_type == 1) store_row<__nv_bfloat16>(a.out, at + c, v + c, valid);
                        else store_row<__half>(a.out, at + c, v + c, valid);
                    }
                }
            } else if (r0 < o.rows) {
                uint8_t *box = sh.out[w - 4];
                const int rows = min(32, o.rows - r0);
                const int64_t at = (kForm == kFormOuter ? o.g * a.out_group : 0) + (int64_t)(o.row0 + r0) * a.out_stride + n0;
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    if (es == 2 && c % 32 != 0) continue;
                    if (c >= wanted) break;
                    if (a.out_type == 0) stage_row<float>(box, v + c, lane);
                    else if (a.out_type == 1) stage_row<__nv_bfloat16>(box, v + c, lane);
                    else stage_row<__half>(box, v + c, lane);
                    __syncwarp();
                    if (es == 4) store_box(box, static_cast<uint32_t *>(a.out), at + c, a.out_stride, rows, wanted - c, lane);
                    else store_box(box, static_cast<uint16_t *>(a.out), at + c, a.out_stride, rows, wanted - c, lane);
                    __syncwarp();
                }
            }
        } while (!kSplit && ok && tiles.next(lane));
        if (lane == 0) bulk_wait_all();
        if (kSplit && !(ok && tiles.tile < total)) {   // the barriers of add_parts, without a part
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    }
    if (kSplit && w < 4) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();   // neither CTA leaves while the other may signal it or read its shared memory
    tc_fence_after();
    if (w == 3) tmem_free<kPair>(tmem, kTmemColumns);
}

// ------------------------------------------------------------------ host side
constexpr int kMatMaxDevices = 128;

// The most 128-row (or `tile`-row) tiles that groups of `rows` rows in all, and
// the rows behind them, can make: each has a row at least.
int64_t most_row_tiles(int64_t rows, int64_t groups, int64_t tile) {
    const int64_t n = div_up(rows, tile) + groups;
    return n < rows ? n : rows;
}

template <int kForm, int kScales, int kN, int kWork>
mx_status launch_product(const Maps &maps, MatArgs a, int parts, cudaStream_t stream) {
    using Sh = Shared<kScales, kN, kWork == kPairs>;
    constexpr int smem = (int)sizeof(Sh) + 1024;
    const int ctas = kWork == kPairs ? 2 : kWork == kSplits ? parts : 1;
    auto kernel = grouped_product<kForm, kScales, kN, kWork>;
    a.n_tiles = (int32_t)div_up(a.N, kN);
    a.m_tiles = (int32_t)div_up(a.M, Sh::kTileRows);
    // an upper bound on the tiles, known without the group ends
    const int64_t tiles = kForm == kFormOuter ? (int64_t)a.m_tiles * a.n_tiles * a.G
                                              : most_row_tiles(a.rows, a.G, Sh::kTileRows) * a.n_tiles;
    if (tiles > INT_MAX / 8) return MX_ERR_UNSUPPORTED;

    static std::mutex mu;
    static bool ready[kMatMaxDevices] = {};
    int dev = 0, sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return mx_record_cuda_error(e);
    if (dev < 0 || dev >= kMatMaxDevices) return MX_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); e != cudaSuccess)
                return mx_record_cuda_error(e);
            ready[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(tiles * ctas));
    cfg.blockDim = dim3(kMatThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, maps, a);
    return e == cudaSuccess ? MX_OK : mx_record_cuda_error(e);
}

// Operand bytes as the loads take them: contraction inner, 128 of it and
// `rows` rows a box; contraction outer, 128 columns and 128 rows a box.
mx_status operand_map(CUtensorMap *map, const void *p, int64_t inner, int64_t outer, int64_t stride, int64_t groups,
                      int64_t group_stride, uint32_t rows) {
    const uint64_t dims[3] = {(uint64_t)inner, (uint64_t)outer, (uint64_t)groups};
    const uint64_t strides[2] = {(uint64_t)stride, (uint64_t)group_stride};
    const uint32_t box[3] = {128, rows, 1};
    return mx_encode_map(map, p, groups > 0 ? 3 : 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// 512-byte tiles of blocked scales.
mx_status tiles_map(CUtensorMap *map, const void *p, int64_t tiles) {
    const uint64_t dims[2] = {128, (uint64_t)tiles}, strides[1] = {512};
    const uint32_t box[2] = {128, 1};
    return mx_encode_map(map, p, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Whether the output may be stored as boxes of a tensor map.  A row has to end on a
// 16-byte boundary too: a store of bytes is cut at the row's end rounded up to 16 (what
// lay behind 2441 columns of bf16 was overwritten up to the 2448th), so that it would
// reach into whatever lies between the rows.
bool boxes_out(const void *p, int64_t n, int64_t es, int64_t stride, int64_t group_stride) {
    return aligned_to(p, 16) && n * es % 16 == 0 && stride * es % 16 == 0 && group_stride * es % 16 == 0;
}

// The output in bytes, 32 rows x 64 bytes a box.
mx_status out_map(CUtensorMap *map, const void *p, int64_t row_bytes, int64_t rows, int64_t stride, int64_t groups, int64_t group_stride) {
    const uint64_t dims[3] = {(uint64_t)row_bytes, (uint64_t)rows, (uint64_t)groups};
    const uint64_t strides[2] = {(uint64_t)stride, (uint64_t)group_stride};
    const uint32_t box[3] = {kOutRow, 32, 1};
    return mx_encode_map(map, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

// A tile's contraction has to end well within the time limit of a wait, and a
// row's bytes are an int in the stores.
constexpr int64_t kMaxContraction = 1ll << 25;
bool too_long(int64_t contraction, int64_t n, int out_bytes) { return contraction > kMaxContraction || n * out_bytes > INT_MAX; }

int out_code(mx_dtype t) { return t == MX_F32 ? 0 : t == MX_BF16 ? 1 : t == MX_F16 ? 2 : -1; }
bool eight(mx_dtype t) { return t == MX_E4M3 || t == MX_E5M2; }

// How a product is spread over the SMs.  `row_tiles`: 128-row tiles if the groups
// are even; `most`: the most that there can be; `rows`: rows of a group, on
// average; `steps`: of the contraction.
struct Plan { Work work; bool narrow; int parts; };
Plan plan_of(int64_t row_tiles, int64_t most, int64_t n, int64_t rows, int64_t steps, int sms) {
    // 128 x 128 tiles where they fit the SMs at once (128 rows, 4 groups of 4096 x
    // 4096, 128 of them: 18.6 us, 26.2 with tiles of 256 columns; 16 groups of 1408 x
    // 1024, 176 of them: 12.0 and 9.7), and of their contraction as many parts as
    // clusters of that size run at once on a B200 (74 of 2 CTAs, 33 of 4, 15 of 8:
    // clusters do not cross the borders of its processor groups; one group of 1408 x
    // 7168: 14.2 us in four parts, 23.6 whole)
    const int64_t tiles = row_tiles * div_up(n, 128);
    if (tiles <= sms) {
        const int64_t clusters = most * div_up(n, 128);
        int parts = 1;
        if (steps >= 8 && clusters <= sms / 2) parts = 2;
        if (steps >= 16 && clusters <= 33) parts = 4;
        if (steps >= 32 && clusters <= 15) parts = 8;
        return {parts > 1 ? kSplits : kAlone, true, parts};
    }
    // Pairs where groups have more than 128 rows on average: 32 groups of 2048 x 2048,
    // with 64 rows each 31 us alone and 38 in pairs, 128: 33 and 40, 160: 44 and 44,
    // 256: 50 and 44, 512: 75 and 75; 8192 rows of one 8192 x 8192: 420 and 385.
    return {rows > 128 ? kPairs : kAlone, false, 1};
}
Plan plan_of_rows(int64_t rows, int64_t n, int64_t k, int64_t groups, int sms) {
    const int64_t each = div_up(rows, groups), even = div_up(each, 128) * groups;
    return plan_of(even < rows ? even : rows, most_row_tiles(rows, groups, 128), n, each, div_up(k, kTileK), sms);
}
Plan plan_of_contraction(int64_t m, int64_t n, int64_t padded_rows, int64_t groups, int sms) {
    const int64_t row_tiles = div_up(m, 128) * groups;
    return plan_of(row_tiles, row_tiles, n, m, padded_rows / kTileK / groups, sms);
}
// Pairs round their rows up to 256 and their columns to 32: where that makes the
// transpose of a weight gradient cheaper, its tiles are computed and written across.
// bf16 out, as it is and across: 1408 x 7168 in 8 groups of 131072 rows 958 and 926
// us, 1152 x 8192 in 4 of 65536 533 and 498, 1408 x 2560 in 4 of 16384 86 and 85, but
// 1300 x 5120 in 8 of 131072 772 and 778, 1408 x 4096 in 16 of 65536 347 and 367.
bool across(const Plan &plan, int64_t m, int64_t n) {
    return plan.work == kPairs && 1.03 * up_to(n, 256) * up_to(m, 32) < (double)up_to(m, 256) * up_to(n, 32);
}

template <int kForm, int kScales>
mx_status launch_planned(const Plan &p, const Maps &maps, const MatArgs &a, cudaStream_t stream) {
    if (p.work == kPairs) return launch_product<kForm, kScales, 256, kPairs>(maps, a, 1, stream);
    if (p.work == kSplits) return launch_product<kForm, kScales, 128, kSplits>(maps, a, p.parts, stream);
    return p.narrow ? launch_product<kForm, kScales, 128, kAlone>(maps, a, 1, stream)
                    : launch_product<kForm, kScales, 256, kAlone>(maps, a, 1, stream);
}

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
    const int os = out_dtype == MX_F32 ? 4 : 2;
    if (!stride_fits(a_stride, 1) || !stride_fits(b_stride, 1) || (num_groups > 1 && !stride_fits(b_group_stride, 1)) ||
        !stride_fits(out_stride, os))
        return MX_ERR_UNSUPPORTED;
    if (num_groups > 1 && !rows_fit(nk ? n : k, b_stride, nk ? k : n, b_group_stride)) return MX_ERR_INVALID_ARG;
    if (block == 32 && !nk) return MX_ERR_UNSUPPORTED;
    if (rows == 0 || n == 0) return MX_OK;
    if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr || group_ends == nullptr || out == nullptr)
        return MX_ERR_INVALID_ARG;
    if (!operand_ok(a, a_stride) || !operand_ok(b, b_stride) || (num_groups > 1 && b_group_stride % 16 != 0) ||
        !aligned_to(out, os) || !aligned_to(group_ends, 4))
        return MX_ERR_MISALIGNED;
    if (too_long(k, n, os)) return MX_ERR_UNSUPPORTED;
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
    m.k_tiles = (int32_t)div_up(k, kTileK);
    m.out_type = out_code(out_dtype);
    m.tma_out = boxes_out(out, n, os, out_stride, 0);
    m.idesc = block_scaled_idesc(a_dtype == MX_E5M2, b_dtype == MX_E5M2, false, !nk);
    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    const Plan plan = plan_of_rows(rows, n, k, num_groups, sms);
    const bool pair = plan.work == kPairs;
    Maps maps = {};
    if (mx_status st = operand_map(&maps.a, a, k, rows, a_stride, 0, 0, 128); st != MX_OK) return st;
    if (mx_status st = operand_map(&maps.b, b, nk ? k : n, nk ? n : k, b_stride, num_groups,
                                   num_groups > 1 ? b_group_stride : b_stride, nk && !pair && !plan.narrow ? 256 : 128);
        st != MX_OK)
        return st;
    if (m.tma_out)
        if (mx_status st = out_map(&maps.out, out, n * os, rows, out_stride * os, 1, out_stride * os); st != MX_OK) return st;
    if (block == 32) {
        const int64_t a_tiles = (rows + 128ll * num_groups) / 128 * m.k_tiles, b_tiles = num_groups * div_up(n, 128) * m.k_tiles;
        if (a_tiles > INT_MAX || b_tiles > INT_MAX) return MX_ERR_UNSUPPORTED;
        if (mx_status st = tiles_map(&maps.sa, a_scales, a_tiles); st != MX_OK) return st;
        if (mx_status st = tiles_map(&maps.sb, b_scales, b_tiles); st != MX_OK) return st;
        return launch_planned<kFormNK, kScales32>(plan, maps, m, stream);
    }
    return nk ? launch_planned<kFormNK, kScales128>(plan, maps, m, stream)
              : launch_planned<kFormKN, kScales128>(plan, maps, m, stream);
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
    const int os = out_dtype == MX_F32 ? 4 : 2;
    if (!stride_fits(a_stride, 1) || !stride_fits(b_stride, 1) || !stride_fits(out_stride, os) ||
        (num_groups > 1 && !stride_fits(out_group_stride, os)))
        return MX_ERR_UNSUPPORTED;
    if (num_groups > 1 && !rows_fit(m, out_stride, n, out_group_stride)) return MX_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return MX_OK;
    if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr || group_ends == nullptr || out == nullptr)
        return MX_ERR_INVALID_ARG;
    if (!operand_ok(a, a_stride) || !operand_ok(b, b_stride) || !aligned_to(out, os) || !aligned_to(group_ends, 4))
        return MX_ERR_MISALIGNED;

    if (too_long(padded_rows, n, os)) return MX_ERR_UNSUPPORTED;

    int sms = 0;
    if (mx_status st = mx_device_sms(&sms); st != MX_OK) return st;
    const Plan plan = plan_of_contraction(m, n, padded_rows, num_groups, sms);
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
    g.tma_out = boxes_out(out, n, os, out_stride, g.out_group);
    g.idesc = block_scaled_idesc(a_dtype == MX_E5M2, b_dtype == MX_E5M2, true, true);
    Maps maps = {};
    if (mx_status st = operand_map(&maps.a, a, m, padded_rows, a_stride, 0, 0, 128); st != MX_OK) return st;
    if (mx_status st = operand_map(&maps.b, b, n, padded_rows, b_stride, 0, 0, 128); st != MX_OK) return st;
    if (g.tma_out)
        if (mx_status st = out_map(&maps.out, out, n * os, m, out_stride * os, num_groups,
                                   (num_groups > 1 ? out_group_stride : out_stride) * os);
            st != MX_OK)
            return st;
    if (across(plan, m, n)) {
        const CUtensorMap t = maps.a;
        maps.a = maps.b;
        maps.b = t;
        g.sa = b_scales;
        g.sb = a_scales;
        g.sa_block = b_scale_stride;
        g.sb_block = a_scale_stride;
        g.M = (int32_t)n;
        g.N = (int32_t)m;
        g.idesc = block_scaled_idesc(b_dtype == MX_E5M2, a_dtype == MX_E5M2, true, true);
        g.swapped = true;
    }
    return launch_planned<kFormOuter, kScales128>(plan, maps, g, stream);
}

mx_tiles mx_select_tiles(mx_group_dim dim, int64_t m, int64_t n, int64_t k, int32_t num_groups, int32_t sms) {
    using namespace mx;
    if ((dim != MX_GROUPS_M && dim != MX_GROUPS_K) || m < 1 || n < 1 || k < 1 || sms < 1 || num_groups < 1 ||
        num_groups > MX_MAX_GROUPS || m > kOpsMaxExtent || n > kOpsMaxExtent || k > kOpsMaxExtent)
        return MX_TILES_NONE;
    const bool rows = dim == MX_GROUPS_M;
    const Plan plan = rows ? plan_of_rows(m, n, k, num_groups, sms) : plan_of_contraction(m, n, k, num_groups, sms);
    if (plan.work == kPairs) return !rows && across(plan, m, n) ? MX_TILES_PAIRS_ACROSS : MX_TILES_PAIRS;
    return plan.work == kSplits ? (mx_tiles)plan.parts : plan.narrow ? MX_TILES_NARROW : MX_TILES_WIDE;
}

}  // extern "C"
