// q4_mx_gemm.cu -- products with microscaled 4-bit matrices: q4_gemm_mx (one
// matrix) and q4_gemm_experts (rows grouped by expert, one matrix per group).
//
// Mathematics.  y[m][n] = sum_k W[n][k] x[m][k], W = e2m1 * 2^e with one e for
// 32 k, x bfloat16.  The tensor cores multiply such blocks natively
// (tcgen05.mma kind::mxf8f6f4, a scale factor per row and 32 k on either
// side), so W's codes and exponents go from memory to the tensor core as
// they are stored; nothing is decoded.  x, with 8 significant bits, is split
// into two e4m3 parts with exponents per 32 k of their own:
//     s = 2^(floor(log2 max|x|) - 7),  hi = e4m3(x / s),
//     lo = e4m3((x / s - hi) * 32),    x = s * hi + (s / 32) * lo.
// hi takes the leading 4 significant bits, and the remainder's bits fit lo
// exactly wherever |x| >= 2^-14 of the group's largest; a smaller x is off by
// at most half of lo's smallest step, 2^-15 s or 2^-22 of that largest.  (A
// third part would hold five octaves more, for half as many MMAs again.  In
// normally distributed x one element in 17,000 is off at all.  It shows where
// W is zero or small at a spike of the group; the caller can split such a row
// exactly, see q4.h.)
// Products are exact.  The tensor core
// adds them to its binary32 accumulator by truncation: measured, the relative
// error grows by 7e-8 for each 128 k.  For a binary32 y the accumulator is
// therefore read out every kFlush32 blocks of k and added up in registers,
// rounded to nearest (5e-7 measured at K = 1024); a bfloat16 y, whose own
// rounding is 2^-9, takes kFlush16 blocks at a time.
// The bound on y.  A step of 32 k adds 32 products to the accumulator, aligned
// to the largest of the 33 and cut below 2^-24 of it: 33 * 2^-24 S, S = sum
// |W x|, for 32 steps a reading (binary32 y) or 256 (bfloat16).  Readings are
// added in binary32, 2^-24 S each, K / 1024 or K / 8192 of them, hi and lo
// once more, and at most 64 parts of a tile.  That is (1056 + K / 1024 + 66)
// 2^-24 S, 8.2e-5 S up to K = 2^18 and 1.3e-4 S at 2^20; for bfloat16
// (8448 + K / 8192 + 66) 2^-24 S, 5.2e-4 S at 2^20.  The split adds 2^-22 of
// its group's largest |x| times sum |W| for each group.
//
// Work.  The hi rows and lo rows of kTokens tokens are the N = 2 kTokens
// columns of one MMA, 128 rows of W its M; the epilogue adds the two halves.
// An output tile is (expert, 128 rows of W, kTokens tokens) and its K is Kb
// blocks; all tiles' blocks form one list of units, cut into equal runs, one
// per persistent CTA, so that there is no tail (fewer tiles than CTAs: see
// q4_mx_runs.cuh).  Where a tile is cut, each CTA stores its part to the workspace and counts
// itself in; the last to come adds all parts in CTA order, so results do not
// depend on timing and no CTA waits for another.
//
// Up to 64 tokens a tile belongs to one CTA (kCtas = 1).  More tokens go to
// pairs of CTAs with 256 rows of W (kCtas = 2, see Shape), which bring each
// byte of x to half as many SMs: with one CTA a tile, 512 tokens asked L2 for
// 42 KB a k block and SM, and that was the limit.
//
// Roles in a CTA: warp 0 streams stages of one or two k blocks (codes by a TMA
// load that spreads 16 nibbles over 16 bytes, exponents, x's parts); warp 1
// copies the exponents to tensor memory and issues four MMAs per block; warps
// 2-5 read the accumulator and write y.  The weights' first stages are
// requested before the x conversion that precedes on the stream has finished
// (programmatic dependent launch).
//
// Measured on B200: 13 tokens x 128256 x 4096 52 us (5.5 TB/s; six exponent
// copies and eight MMAs a stage take three quarters of its time), 64 tokens x
// 57344 x 8192 70 us (3.8 TB/s; MMAs and copies), 512 tokens 349 us to
// bfloat16 and 360 us to binary32 in short runs (1.38 and 1.34 PFLOP/s of 1.64;
// three copies to every four MMAs, 14 % of the time, and waits for stages), 410
// to 460 us once the power cap has lowered the clock.
// Every wait is bounded; one that runs out sets an error bit and the CTA
// drains its copies, frees its tensor memory and exits.
#include <algorithm>

#include "q4_mx_runs.cuh"
#include "q4_mx_tc.cuh"

namespace q4 {

__device__ unsigned int g_gemm_mx_error;

namespace {

constexpr int kThreads = 192;     // producer, MMA, four epilogue warps
constexpr int kFlush32 = 8;       // k blocks per accumulation in tensor memory, binary32 y
constexpr int kFlush16 = 64;      // ... bfloat16 y
constexpr int kPairTokens = 120;  // most tokens of a pair's tile: two accumulators of 240 columns

struct MxGemm {
    const uint8_t* wsf;           // exponent bytes of W
    const uint8_t* xsf;           // exponent bytes of x's parts, [tile][x_blocks][Kb][512]
    const int32_t* offsets;       // first row of each expert; nullptr: one matrix
    float* partial;               // [2 * CTAs][tokens][128]
    uint32_t* counters;           // one for each 128 rows of an output tile
    void* y;
    int64_t N;
    int tile_limit;               // token tiles that the workspace holds
    int T, E, Nb, Kb, y_bf16;
    int tokens;                   // of a tile
    int Nt;                       // row tiles of W: Nb, or pairs of row blocks
    int Ku;                       // units (stages) of k of a tile
    int flush;                    // units per accumulation in tensor memory
    RunCost cost;
};

// Layout of the workspace, all parts multiples of 1024 bytes.
struct Workspace {
    int64_t tiles;  // bound on the number of token tiles
    size_t counters, xq, xsf, partial, bytes;
};

// Blocks of 128 columns (x rows, hi and lo) whose exponents a tile has.
int x_blocks(int tokens, bool pair) { return pair ? 2 : (2 * tokens + kMxBlock - 1) / kMxBlock; }

// Tokens of a tile, and whether pairs of CTAs take it.  Up to 64 tokens an
// expert one CTA: for one matrix its tokens in whole eights, which are then
// the MMA's columns.  Experts differ, and one with more rows than a tile reads
// its codes again, which costs more than wider MMAs: their tiles hold twice the
// average share (64 experts of 2048 x 4096, tiles of the share or of twice:
// 32 tokens x 8 58 or 51 us, 64 67 or 58 us, 256 102 or 98 us), up to 64 for
// shares from 17 to 64 (512 tokens: 154 us; pairs 168 us).  More: pairs, in
// tiles of at most 120 tokens: equal ones for one matrix, of 120 where experts
// differ (a pair's tile with fewer tokens has shorter MMAs).
struct Plan {
    int tokens;
    bool pair;
};
Plan plan_for(int64_t T, int64_t E) {
    const int64_t share = (T + E - 1) / E;
    if (E > 1) {
        if (share > 64) return {kPairTokens, true};
        return {share <= 2 ? 8 : share <= 8 ? 16 : share <= 16 ? 32 : 64, false};
    }
    if (share <= 64) return {static_cast<int>((share + 7) / 8 * 8), false};
    const int64_t tiles = (share + kPairTokens - 1) / kPairTokens;
    return {static_cast<int>(((share + tiles - 1) / tiles + 7) / 8 * 8), true};
}

Workspace workspace_layout(int64_t T, int64_t E, int64_t N, int64_t K, const Plan& plan) {
    auto up = [](size_t n) { return (n + 1023) / 1024 * 1024; };
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    const int tokens = plan.tokens;
    Workspace w{};
    // an expert with c > 0 rows has at most c / tokens + 1 tiles
    w.tiles = E == 1 ? (T + tokens - 1) / tokens : std::min(T, T / tokens + E);
    w.counters = 0;
    w.xq = up(static_cast<size_t>(w.tiles) * (Nb + 1) * sizeof(uint32_t));
    w.xsf = w.xq + up(static_cast<size_t>(w.tiles) * 2 * tokens * Kb * kMxBlock);
    w.partial = w.xsf + up(static_cast<size_t>(w.tiles) * x_blocks(tokens, plan.pair) * Kb * kMxScaleBytes);
    w.bytes = w.partial + up(static_cast<size_t>(2) * kMxMaxSms * tokens * kMxBlock * sizeof(float));
    return w;
}

// ---------------------------------------------------------------------------
// x to its two parts, in the order of the token tiles
// ---------------------------------------------------------------------------
// Tokens that a pair's MMA computes for a tile of `count`: N has to be a multiple of 16.
__device__ __forceinline__ int pair_tokens(int count) { return (count + 7) / 8 * 8; }

struct Convert {
    const uint16_t* x;
    const int32_t* rows;  // x row of each of the T rows; nullptr: the row itself
    const int32_t* offsets;
    uint8_t* xq;
    uint8_t* xsf;
    uint32_t* counters;
    void* y;
    int64_t Mx, K, N, counter_count, tile_limit;
    int T, E, Kb, y_bf16, tokens, x_blocks, pair;
    int split;  // warps that share a row, a power of two
};

// A warp converts 256 k of a row at a time: 4 lanes a group of 32, 8 values a lane.
template <bool kVector>
__global__ void __launch_bounds__(256) convert_kernel(const Convert p) {
    __shared__ Table table;
    pdl_launch();
    fill_table(table, p.offsets, p.E, p.T, p.tokens);
    const int64_t thread = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = thread; i < p.counter_count; i += threads) p.counters[i] = 0;
    // rows of y behind the last expert's
    const int64_t behind = table.offset[p.E] * p.N, all = static_cast<int64_t>(p.T) * p.N;
    for (int64_t i = behind + thread; i < all; i += threads) {
        if (!Q4_IN_BOUNDS(i, 1, all)) continue;
        if (p.y_bf16)
            static_cast<uint16_t*>(p.y)[i] = 0;
        else
            static_cast<float*>(p.y)[i] = 0.0f;
    }
    // A warp takes every p.split-th run of 256 k of a row, kFlight of them at a
    // time so that their loads are in flight together.
    constexpr int kFlight = 4;
    const int lane = threadIdx.x & 31;
    const int pieces = (p.Kb + 1) / 2;
    const int part = static_cast<int>(thread / 32) & (p.split - 1), step = p.split;
    const int64_t row_step = threads / 32 / p.split;
    const int64_t Kp = static_cast<int64_t>(p.Kb) * kMxBlock;
    for (int64_t r = thread / 32 / p.split; r < table.offset[p.E]; r += row_step) {
        const int row = static_cast<int>(r);
        const int e = find_expert(table.offset, p.E, row);
        const int in = row - table.offset[e];
        const int64_t tile = table.tile[e] + in / p.tokens;
        if (row < table.offset[0] || tile >= p.tile_limit) continue;  // offsets that do not start at 0
        const int m = in % p.tokens;
        const int64_t src = p.rows ? static_cast<int64_t>(__ldg(p.rows + row)) : row;
        const bool have = src >= 0 && src < p.Mx;
        // the row's hi and lo columns; a pair's tile has as many as tokens need
        const int lo_m = (p.pair ? pair_tokens(min(p.tokens, table.offset[e + 1] - (row - m))) : p.tokens) + m;
        const int64_t first = (have ? src : 0) * p.K;
        for (int p0 = part; p0 < pieces; p0 += step * kFlight) {
            uint4 q[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int64_t k = static_cast<int64_t>(p0 + i * step) * 256 + 8 * lane;
                q[i] = load_x8<kVector>(p.x, have, first + k, k, p.K, p.Mx * p.K);
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const int piece = p0 + i * step;
                if (piece >= pieces) break;
                const int64_t k = static_cast<int64_t>(piece) * 256 + 8 * lane;
                const int kb = 2 * piece + lane / 16;
                const XParts parts = split_x(q[i]);
                uint32_t four, four_lo;
                gather_bytes(parts.byte, lane, four, four_lo);
                if (kb >= p.Kb) continue;
                [[maybe_unused]] const int64_t extent = p.tile_limit * 2 * p.tokens * Kp;
                const int64_t at = (tile * 2 * p.tokens + m) * Kp + k;
                if (Q4_IN_BOUNDS(at, 8, extent) && Q4_IN_BOUNDS(at + p.tokens * Kp, 8, extent)) {
                    *reinterpret_cast<uint2*>(p.xq + at) = parts.hi;
                    *reinterpret_cast<uint2*>(p.xq + at + p.tokens * Kp) = parts.lo;
                }
                if ((lane & 15) != 0) continue;
                // the four groups of a k block: one 32-bit store per part
                [[maybe_unused]] const int64_t sf_extent = p.tile_limit * p.x_blocks * p.Kb * kMxScaleBytes;
                const int64_t sf =
                    ((tile * p.x_blocks + m / kMxBlock) * p.Kb + kb) * kMxScaleBytes + mx_scale_at(m % kMxBlock, 0);
                const int64_t sf_lo =
                    ((tile * p.x_blocks + lo_m / kMxBlock) * p.Kb + kb) * kMxScaleBytes + mx_scale_at(lo_m % kMxBlock, 0);
                if (Q4_IN_BOUNDS(sf, 4, sf_extent) && Q4_IN_BOUNDS(sf_lo, 4, sf_extent)) {
                    *reinterpret_cast<uint32_t*>(p.xsf + sf) = four;
                    *reinterpret_cast<uint32_t*>(p.xsf + sf_lo) = four_lo;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
// kTokens: the most a tile may have.  A pair's (kCtas = 2) MMA has 256 rows of
// W, 128 in each CTA, and reads its columns from both: the first CTA holds the
// hi rows of x, the second the lo rows, so each byte of x is brought to one SM
// for 256 rows of W.
template <int kTokens, int kCtas>
struct Shape {
    static constexpr int kCols = 2 * kTokens;                    // MMA N
    static constexpr int kXBlocks = (kCols + kMxBlock - 1) / kMxBlock;
    // k blocks of a stage: two for few tokens, whose MMAs are short beside a
    // stage's bookkeeping
    static constexpr int kUnit = kTokens <= 32 ? 2 : 1;
    static constexpr int kABytes = kMxBlock * 128;               // a block's codes spread over bytes
    static constexpr int kBBytes = kCols / kCtas * 128;
    // a stage: kUnit blocks of A, of B, A's exponents, B's (by row block, then k block)
    static constexpr int kBAt = kUnit * kABytes;
    static constexpr int kSfaAt = kBAt + kUnit * kBBytes;
    static constexpr int kSfbAt = kSfaAt + kUnit * kMxScaleBytes;
    static constexpr int kStage = kSfbAt + kUnit * kXBlocks * kMxScaleBytes;
    static constexpr int kStagePitch = (kStage + 1023) / 1024 * 1024;
    static constexpr int kRoom = 222 * 1024 - static_cast<int>(sizeof(Table));
    static constexpr int kStages = kRoom / kStagePitch < 12 ? kRoom / kStagePitch : 12;
    static constexpr uint32_t kScaleSet = 4 * kUnit * (1 + kXBlocks);
    static constexpr uint32_t kScaleCol = 2 * kCols;               // after two accumulators, two sets of exponents
    static constexpr int kSmem = 1024 + kStages * kStagePitch + static_cast<int>(sizeof(Table)) + 512;
    static_assert(kStages >= 3, "the ring needs stages");
    static_assert(kScaleCol + 2 * kScaleSet <= kTmemCols, "tensor memory");
};

// The run of units of a CTA or pair, a unit being kUnit k blocks of one output tile.
// Tiles are numbered by expert, then rows of W, then token tile, so that the
// token tiles of the same rows follow each other and find their codes in L2.
struct Segment {
    int out;              // output tile
    int e, nt, tile, in;  // expert, row tile, token tile, its number in the expert
    int first, count;     // its rows of y
    int k0, k1;           // units of k
};
// All counts fit 31 bits (the API refuses more units than that).
struct Runs {
    RunCut cut;
    int u, u1;
    __device__ Runs(const MxGemm& p, const Table& t, int c, int groups)
        : cut(min(t.tile[p.E], p.tile_limit) * p.Nt, groups, p.Ku, p.cost) {
        u = c < cut.ctas ? cut.start(c) : cut.units;
        u1 = c < cut.ctas ? cut.start(c + 1) : cut.units;
    }
    __device__ bool next(const MxGemm& p, const Table& t, Segment& s) {
        if (u >= u1) return false;
        s.out = u / p.Ku;
        s.k0 = u - s.out * p.Ku;
        s.k1 = min(p.Ku, s.k0 + u1 - u);
        u += s.k1 - s.k0;
        s.e = p.E == 1 ? 0 : find_expert(t.tile, p.E, s.out / p.Nt);
        const int local = s.out - t.tile[s.e] * p.Nt, mine = t.tile[s.e + 1] - t.tile[s.e];
        s.nt = mine == 1 ? local : local / mine;
        s.in = local - s.nt * mine;
        s.tile = t.tile[s.e] + s.in;
        s.first = t.offset[s.e] + s.in * p.tokens;
        s.count = min(p.tokens, t.offset[s.e + 1] - s.first);
        return true;
    }
};

// acc[0 .. count) to `out` and every N-th element behind it.  (Short on
// purpose: with the address and the bounds worked out for each token, 120
// unrolled stores were so much code that a tile's took 14 us.)
template <int kTokens, typename T>
__device__ __forceinline__ void store_column(T* out, int64_t N, const float (&acc)[kTokens], int count) {
#pragma unroll
    for (int m0 = 0; m0 < kTokens; m0 += 8) {
        if (m0 >= count) break;
#pragma unroll
        for (int m = m0; m < m0 + 8; ++m) {
            if (m < count) *out = Element<T>::put(acc[m]);
            out += N;
        }
    }
}

// Four consecutive outputs n .. n + 3 of row `at` / N.
__device__ __forceinline__ void store4(const MxGemm& p, int64_t at, int64_t n, const float4& v) {
    const float f[4] = {v.x, v.y, v.z, v.w};
    if ((p.N & 3) == 0) {  // then rows are aligned for it
        if (n >= p.N || !Q4_IN_BOUNDS(at, 4, static_cast<int64_t>(p.T) * p.N)) return;
        if (p.y_bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
            uint2 w;
            w.x = *reinterpret_cast<const uint32_t*>(&a);
            w.y = *reinterpret_cast<const uint32_t*>(&b);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) = w;
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= p.N || !Q4_IN_BOUNDS(at + i, 1, static_cast<int64_t>(p.T) * p.N)) continue;
        if (p.y_bf16)
            static_cast<__nv_bfloat16*>(p.y)[at + i] = __float2bfloat16_rn(f[i]);
        else
            static_cast<float*>(p.y)[at + i] = f[i];
    }
}

template <int kTokens, int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_mx_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const __grid_constant__ CUtensorMap wsfmap, const __grid_constant__ CUtensorMap xsfmap,
                   const MxGemm p) {
    using S = Shape<kTokens, kCtas>;
    const int tokens = p.tokens;
    const uint32_t rank = kCtas == 1 ? 0u : cluster_rank();
    const int group = blockIdx.x / kCtas, groups = gridDim.x / kCtas;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    Table& table = *reinterpret_cast<Table*>(smem + S::kStages * S::kStagePitch);
    uint8_t* tail = smem + S::kStages * S::kStagePitch + sizeof(Table);
    const uint32_t bars = (smem_u32(tail) + 7u) & ~7u;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
    auto dfull = [&](int b) { return bars + 8u * (2 * S::kStages + b); };
    auto dempty = [&](int b) { return bars + 8u * (2 * S::kStages + 2 + b); };
    const uint32_t drain = bars + 8u * (2 * S::kStages + 4);
    const uint32_t words = bars + 8u * (2 * S::kStages + 5);  // tensor-memory base, abort, last arrival
    volatile uint32_t* word = reinterpret_cast<volatile uint32_t*>(smem + (words - base));
    volatile uint32_t* abort_flag = word + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull(b), 1);
            mbar_init(dempty(b), 4 * kCtas);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensor_map(&wmap);
        prefetch_tensor_map(&xmap);
    }
    if (warp == 1) {
        tmem_alloc_all<kCtas>(words);
    }
    tc_fence_before();
    fill_table(table, p.offsets, p.E, p.T, tokens);  // ends in __syncthreads
    if (kCtas > 1) cluster_sync();                   // the other CTA's barriers exist
    tc_fence_after();
    const uint32_t tmem = *word;

    if (warp == 0) {
        // ------------------------------ producer ------------------------------
        bool ok = true;
        // A pair's loads all complete on the first CTA's barrier, which expects
        // the bytes of both (a count of bytes may run ahead of that).
        const uint32_t leader_full = kCtas == 1 ? bars : in_first_cta(bars);
        auto load_w = [&](int64_t block, int blocks, int slot) {
            const uint32_t dst = base + slot * S::kStagePitch, bar = leader_full + 8u * slot;
            // the load that spreads the nibbles counts the bytes it reads
            const int brows = 2 * tokens / kCtas;
            if (rank == 0)
                mbar_arrive_expect_tx(full(slot), kCtas * (S::kUnit * (kMxCodeBytes + brows * 128) +
                                                           blocks * kMxScaleBytes * (1 + S::kXBlocks)));
            if (kCtas > 1) {
                tma_load_2d_pair(dst, &wmap, 0, static_cast<int>(block * kMxBlock), bar);
                tma_load_2d_pair(dst + S::kSfaAt, &wsfmap, 0, static_cast<int>(block), bar);
                return;
            }
            tma_load_2d(dst, &wmap, 0, static_cast<int>(block * kMxBlock), bar);
            if (Q4_IN_BOUNDS(block, blocks, static_cast<int64_t>(p.E) * p.Nb * p.Kb))
                bulk_load(dst + S::kSfaAt, p.wsf + block * kMxScaleBytes, blocks * kMxScaleBytes, bar);
        };
        auto load_x = [&](int tile, int kb, int blocks, int slot) {
            const uint32_t dst = base + slot * S::kStagePitch, bar = leader_full + 8u * slot;
            if (kCtas > 1) {
                tma_load_3d_pair(dst + S::kBAt, &xmap, 0, (2 * tile + static_cast<int>(rank)) * tokens, kb, bar);
#pragma unroll
                for (int b = 0; b < S::kXBlocks; ++b)
                    tma_load_2d_pair(dst + S::kSfbAt + b * kMxScaleBytes, &xsfmap, 0,
                                     (tile * S::kXBlocks + b) * p.Kb + kb, bar);
                return;
            }
            tma_load_3d(dst + S::kBAt, &xmap, 0, 2 * tile * tokens, kb, bar);
#pragma unroll
            for (int b = 0; b < S::kXBlocks; ++b) {
                const int64_t at = (static_cast<int64_t>(tile) * S::kXBlocks + b) * p.Kb + kb;
                if (Q4_IN_BOUNDS(at, blocks, static_cast<int64_t>(p.tile_limit) * S::kXBlocks * p.Kb))
                    bulk_load(dst + S::kSfbAt + b * S::kUnit * kMxScaleBytes, p.xsf + at * kMxScaleBytes,
                              blocks * kMxScaleBytes, bar);
            }
        };
        // a pair's second CTA without rows of its own reads the first's
        auto row_block = [&](const Segment& s) { return min(s.nt * kCtas + static_cast<int>(rank), p.Nb - 1); };
        // the ring's first filling: W before the x conversion is known to be done
        Segment s;
        {
            Runs runs(p, table, group, groups);
            for (int n = 0; n < S::kStages && runs.next(p, table, s);) {
                const int64_t block = (static_cast<int64_t>(s.e) * p.Nb + row_block(s)) * p.Kb;
                for (int k = s.k0; k < s.k1 && n < S::kStages; ++k, ++n)
                    if (elect_one()) load_w(block + k * S::kUnit, min(S::kUnit, p.Kb - k * S::kUnit), n);
            }
        }
        pdl_wait();
        asm volatile("fence.proxy.async;" ::: "memory");  // x's parts were written by plain stores
        Runs runs(p, table, group, groups);
        Ring<S::kStages> ring;
        int64_t issued = 0;
        while (ok && runs.next(p, table, s)) {
            const int64_t block = (static_cast<int64_t>(s.e) * p.Nb + row_block(s)) * p.Kb;
            for (int k = s.k0; k < s.k1; ++k) {
                const bool first = issued < S::kStages;
                if (!first && !wait_bar(empty(ring.slot), ring.parity ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const int kb = k * S::kUnit, blocks = min(S::kUnit, p.Kb - kb);
                    if (!first) load_w(block + kb, blocks, ring.slot);
                    load_x(s.tile, kb, blocks, ring.slot);
                }
                __syncwarp();
                ++issued;
                ring.next();
            }
        }
        if (!ok && lane == 0) {
            atomicOr(&g_gemm_mx_error, 1u);
            *abort_flag = 1;
        }
        // Leave only once every copy issued has landed and, in a pair's second
        // CTA, the first one's arrivals for its stages have come: they are
        // sent into this CTA's shared memory.  (Bounded, and without the error
        // flag, so that an error leaves them time.)
        for (int64_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i) {
            const int slot = static_cast<int>(i % S::kStages);
            if (!mbar_wait(rank == 0 ? full(slot) : empty(slot), static_cast<uint32_t>(i / S::kStages) & 1u)) break;
        }
    } else if (warp == 1 && rank != 0) {
        // the pair's first CTA issues for both
    } else if (warp == 1) {
        // -------------------------------- MMA ---------------------------------
        bool ok = true;
        Runs runs(p, table, group, groups);
        Segment s;
        Ring<S::kStages> ring;
        Ring<2> dring;
        uint32_t set = 0;
        bool reused = false;  // the accumulator's earlier contents have to be read first
        const uint64_t adesc = smem_desc_sw128(base, 1024), sdesc = scale_desc(base);
        while (ok && runs.next(p, table, s)) {
            const uint32_t idesc = mx_idesc(kMxBlock * kCtas, 2 * (kCtas == 1 ? tokens : pair_tokens(s.count)), 0);
            for (int k0 = s.k0; ok && k0 < s.k1; k0 += p.flush) {
                const int k1 = min(s.k1, k0 + p.flush);
                if (reused && !wait_bar(dempty(dring.slot), dring.parity ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + dring.slot * S::kCols;
                for (int k = k0; k < k1; ++k) {
                    if (!wait_bar(full(ring.slot), ring.parity, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = static_cast<uint32_t>(ring.slot) * (S::kStagePitch >> 4);
                        const uint32_t sf = tmem + S::kScaleCol + set * S::kScaleSet;
                        const int blocks = S::kUnit == 1 ? 1 : min(S::kUnit, p.Kb - k * S::kUnit);
#pragma unroll
                        for (int u = 0; u < S::kUnit; ++u) {
                            if (u >= blocks) break;
                            const uint32_t sfa = sf + 4 * u * (1 + S::kXBlocks), sfb = sfa + 4;
                            tc_copy_scales<kCtas>(sfa, sdesc + at + (S::kSfaAt + u * kMxScaleBytes) / 16);
#pragma unroll
                            for (int b = 0; b < S::kXBlocks; ++b)
                                tc_copy_scales<kCtas>(sfb + 4 * b,
                                               sdesc + at + (S::kSfbAt + (b * S::kUnit + u) * kMxScaleBytes) / 16);
                        }
#pragma unroll
                        for (int u = 0; u < S::kUnit; ++u) {
                            if (u >= blocks) break;
                            const uint32_t sfa = sf + 4 * u * (1 + S::kXBlocks), sfb = sfa + 4;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                tc_mma_mx<kCtas>(d, adesc + at + (u * S::kABytes + 32 * q) / 16,
                                          adesc + at + (S::kBAt + 32 * q) / 16 + u * (2 * tokens / kCtas * 128 / 16),
                                          idesc | mx_idesc(0, 0, q), sfa, sfb, (k > k0 || u > 0 || q > 0) ? 1u : 0u);
                        }
                        tc_commit_all<kCtas>(empty(ring.slot));
                        if (k == k1 - 1) tc_commit_all<kCtas>(dfull(dring.slot));
                    }
                    __syncwarp();
                    set ^= 1u;
                    ring.next();
                }
                dring.next();
                if (dring.slot == 0) reused = true;
            }
        }
        if (!ok && lane == 0) {
            atomicOr(&g_gemm_mx_error, 2u);
            *abort_flag = 1;
        }
        __syncwarp();
        if (elect_one()) tc_commit_own<kCtas>(drain);
        if (!mbar_wait(drain, 0u) && lane == 0) atomicOr(&g_gemm_mx_error, 4u);
        __syncwarp();
    } else {
        // ------------------------------ epilogue ------------------------------
        const int quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        constexpr int kLoad = kTokens % 32 == 0 ? 32 : 8;                    // columns of a tensor-memory load
        constexpr int kWait = kTokens % 24 == 0 ? 24 : kTokens < 32 ? kTokens : 32;  // ... of a wait for them
        Ring<2> dring;
        bool ok = true;
        Runs runs(p, table, group, groups);
        Segment s;
        pdl_wait();  // the counters' zeros, and whoever read the workspace before
        while (ok && runs.next(p, table, s)) {
            const int cols = kCtas == 1 ? tokens : pair_tokens(s.count);  // of either part
            float acc[kTokens];
#pragma unroll
            for (int i = 0; i < kTokens; ++i) acc[i] = 0.0f;
            for (int k0 = s.k0; k0 < s.k1; k0 += p.flush) {
                ok = wait_bar(dfull(dring.slot), dring.parity, abort_flag);
                if (!ok) break;
                const uint32_t d = lanes + dring.slot * S::kCols;
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < kTokens; c0 += kWait) {
                    if (c0 >= cols) break;
                    uint32_t hi[kWait], lo[kWait];
#pragma unroll
                    for (int c = 0; c < kWait; c += kLoad) {
                        if (c0 + c >= cols) break;
                        if constexpr (kLoad == 8) {
                            tc_ld_x8(d + c0 + c, hi + c);
                            tc_ld_x8(d + cols + c0 + c, lo + c);
                        } else {
                            tc_ld_x32(d + c0 + c, hi + c);
                            tc_ld_x32(d + cols + c0 + c, lo + c);
                        }
                    }
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < kWait; c += kLoad) {
                        if (c0 + c >= cols) break;
#pragma unroll
                        for (int i = 0; i < kLoad; ++i)
                            acc[c0 + c + i] += __uint_as_float(hi[c + i]) + __uint_as_float(lo[c + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0)
                        mbar_arrive(dempty(dring.slot));
                    else
                        arrive_cluster(in_first_cta(dempty(dring.slot)));
                }
                dring.next();
            }
            ok = epilogue_sync(ok);
            if (!ok) break;
            const int first = s.first, count = s.count;
            const int64_t n0 = (static_cast<int64_t>(s.nt) * kCtas + rank) * kMxBlock, n = n0 + row;
            if (s.k0 == 0 && s.k1 == p.Ku) {
                // one row of W a thread: a warp's store is 32 outputs of a token in a row
                const int64_t at = static_cast<int64_t>(first) * p.N + n;
                if (n < p.N && Q4_IN_BOUNDS(at + (count - 1) * p.N, 1, static_cast<int64_t>(p.T) * p.N)) {
                    if (p.y_bf16)
                        store_column<kTokens>(static_cast<__nv_bfloat16*>(p.y) + at, p.N, acc, count);
                    else
                        store_column<kTokens>(static_cast<float*>(p.y) + at, p.N, acc, count);
                }
                continue;
            }
            // A part of a tile.  A run that begins inside the tile owns slot
            // 2 c, one that begins with it (or before) slot 2 c + 1.
            auto slot_of = [&](int c, bool inside) {
                return p.partial + static_cast<int64_t>((2 * c + (inside ? 0 : 1)) * kCtas + static_cast<int>(rank)) * tokens * kMxBlock;
            };
            float* mine = slot_of(group, s.k0 > 0) + row;
#pragma unroll
            for (int m = 0; m < kTokens; ++m)
                if (m < count) __stcg(mine + m * kMxBlock, acc[m]);
            __threadfence();
            epilogue_sync(true);
            const int u0 = s.out * p.Ku, c0 = runs.cut.owner(u0), c1 = runs.cut.owner(u0 + p.Ku - 1);
            if (tid == 64) word[2] = atomicAdd(p.counters + s.out * kCtas + rank, 1u) == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
            epilogue_sync(true);
            if (word[2] == 0u) continue;
            __threadfence();
            // each warp adds up every fourth token, four rows of W a lane,
            // with kBatch tokens' loads of a part in flight
            constexpr int kBatch = kTokens / 4 < 8 ? kTokens / 4 : 8;
            const int64_t n4 = n0 + 4 * lane;
            for (int m0 = warp - 2; m0 < count; m0 += 4 * kBatch) {
                float4 sum[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) sum[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
                for (int c = c0; c <= c1; ++c) {
                    const float* part = slot_of(c, runs.cut.start(c) > u0) + 4 * lane;
                    float4 v[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b)
                        v[b] = __ldcg(reinterpret_cast<const float4*>(part + min(m0 + 4 * b, count - 1) * kMxBlock));
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        sum[b].x += v[b].x;
                        sum[b].y += v[b].y;
                        sum[b].z += v[b].z;
                        sum[b].w += v[b].w;
                    }
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (m0 + 4 * b < count) store4(p, static_cast<int64_t>(first + m0 + 4 * b) * p.N + n4, n4, sum[b]);
            }
        }
        if (!ok && lane == 0) {
            atomicOr(&g_gemm_mx_error, 8u);
            *abort_flag = 1;
        }
    }

    // -------------------------------- teardown --------------------------------
    __syncwarp();  // a role may have left its loop lane by lane
    pdl_wait();  // no CTA ends before the conversion has: it writes y's last rows
    tc_fence_before();
    __syncthreads();
    if (kCtas > 1) cluster_sync();  // neither CTA's memory goes while the other may use it
    if (warp == 1) {
        tc_fence_after();
        tmem_free_all<kCtas>(tmem);
    }
}

template <int kTokens, int kCtas>
cudaError_t launch_as(const Plan& plan, const uint8_t* codes, const uint8_t* scales, const uint16_t* x, const int32_t* rows,
                      const int32_t* offsets, void* y, int y_type, int64_t Mx, int64_t T, int64_t E, int64_t N,
                      int64_t K, uint8_t* ws, cudaStream_t s, const DeviceInfo& dev) {
    using S = Shape<kTokens, kCtas>;
    const Workspace l = workspace_layout(T, E, N, K, plan);
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    Convert c{};
    c.x = x;
    c.rows = rows;
    c.offsets = offsets;
    c.xq = ws + l.xq;
    c.xsf = ws + l.xsf;
    c.counters = reinterpret_cast<uint32_t*>(ws + l.counters);
    c.y = y;
    c.Mx = Mx;
    c.K = K;
    c.N = N;
    c.counter_count = l.tiles * (Nb + 1);
    c.tile_limit = l.tiles;
    c.T = static_cast<int>(T);
    c.E = static_cast<int>(E);
    c.Kb = static_cast<int>(Kb);
    c.y_bf16 = y_type == Q4_BF16;
    c.tokens = plan.tokens;
    c.x_blocks = x_blocks(plan.tokens, plan.pair);
    c.pair = plan.pair;
    // as many warps to a row as leave each four runs of 256 k, and more where
    // rows are too few for the SMs
    const int64_t pieces = (Kb + 1) / 2;
    c.split = 1;
    while (c.split < pieces && (pieces > 4 * c.split || T * c.split < 8 * dev.sm_count) && c.split < 1024) c.split *= 2;
    while (c.split > 1 && T * c.split > 64 * static_cast<int64_t>(dev.sm_count) && pieces < 16 * c.split) c.split /= 2;
    const int64_t warps = std::max<int64_t>(T * c.split, (c.counter_count + 255) / 256);
    // whole groups of warps that share rows: 8 warps a block
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 8;
    int64_t blocks = std::min<int64_t>((warps + 7) / 8, std::max<int64_t>(most, (c.split + 7) / 8));
    const int64_t whole = std::max<int64_t>(1, c.split / 8);
    blocks = (blocks + whole - 1) / whole * whole;
    const int grid = static_cast<int>(blocks);
    if (K % 8 == 0)
        convert_kernel<true><<<grid, 256, 0, s>>>(c);
    else
        convert_kernel<false><<<grid, 256, 0, s>>>(c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    CUtensorMap wmap, xmap, wsfmap, xsfmap;
    e = encode_tensor_map_2d(&wmap, codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 0,
                             static_cast<uint64_t>(E * Nb * Kb * kMxBlock), kMxBlock, 64, S::kUnit * kMxBlock, kMxBlock,
                             CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    e = encode_tensor_map_rows_by_block(&xmap, c.xq, static_cast<uint64_t>(l.tiles * 2 * plan.tokens),
                                        static_cast<uint64_t>(Kb), 2 * plan.tokens / kCtas, S::kUnit);
    if (e != cudaSuccess) return e;
    wsfmap = xsfmap = wmap;  // not used by one CTA, which copies exponents without a map
    if (kCtas > 1) {
        const uint64_t x_rows = static_cast<uint64_t>(l.tiles) * c.x_blocks * Kb;
        e = encode_tensor_map_2d(&wsfmap, scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, static_cast<uint64_t>(E * Nb * Kb),
                                 128, kMxScaleBytes, 1, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (e == cudaSuccess)
            e = encode_tensor_map_2d(&xsfmap, c.xsf, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, x_rows, 128, kMxScaleBytes, 1,
                                     128, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (e != cudaSuccess) return e;
    }
    MxGemm p{};
    p.wsf = scales;
    p.xsf = c.xsf;
    p.offsets = offsets;
    p.partial = reinterpret_cast<float*>(ws + l.partial);
    p.counters = c.counters;
    p.y = y;
    p.N = N;
    p.tile_limit = static_cast<int>(l.tiles);
    p.T = c.T;
    p.E = c.E;
    p.Nb = static_cast<int>(Nb);
    p.Kb = c.Kb;
    p.tokens = plan.tokens;
    p.Nt = static_cast<int>((Nb + kCtas - 1) / kCtas);
    p.y_bf16 = c.y_bf16;
    p.Ku = static_cast<int>((Kb + S::kUnit - 1) / S::kUnit);
    p.flush = (c.y_bf16 ? kFlush16 : kFlush32) / S::kUnit;

    // ns of a k block, of adding a tile's parts up, and of each part
    p.cost = run_cost(Kb * (kCtas > 1 ? 370 : kTokens > 32 ? 270 : 190), 2000 + 70 * plan.tokens, 300 + 14 * plan.tokens,
                      p.Ku);
    const void* fn = reinterpret_cast<const void*>(gemm_mx_kernel<kTokens, kCtas>);
    constexpr int kSlot = kTokens == 8 ? 100 : kTokens == 16 ? 101 : kTokens == 32 ? 102 : kTokens == 64 ? 103 : 104;
    if (S::kSmem > dev.smem_optin) return cudaErrorNotSupported;
    e = ensure_smem_attr(fn, S::kSmem, kSlot, dev.device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    const int64_t groups = std::min<int64_t>(std::min(dev.sm_count, kMxMaxSms) / kCtas,
                                             std::max<int64_t>(1, l.tiles * p.Nt * p.Ku));
    cfg.gridDim = dim3(static_cast<unsigned>(groups * kCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = kCtas == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, gemm_mx_kernel<kTokens, kCtas>, wmap, xmap, wsfmap, xsfmap, p);
}

}  // namespace

// Whether a product of few tokens runs on q4_mx_decode.cu, in tiles of 8, and
// how: the CTAs that share a tile's K (0: not at all), and how many such groups.
// Counted in stages of 256 k, 0.31 us each on one SM (0.42 us with more than 4
// tokens, whose x takes longer to prepare than the codes to come): a turn of a
// group costs half a stage beside its own, sharing a tile 5 stages once, and
// the kernel above 21 for its second launch and its sums' way through memory,
// 30 from 9 to 16 tokens, where the decode kernel reads the codes twice.
// Measured on B200 (us, 1 token; 1, 2, 4 CTAs a tile; the kernel above):
//   4096 x 4096   8.0  6.8  5.8;  9.5     28672 x 4096  14.9 16.1 14.4; 17.7
//   4096 x 14336 21.0 13.5 10.0; 12.1     28672 x 8192  26.0 27.6 24.4; 26.6
//   128256 x 4096 44.7 46.0 47.3; 49.6    28672 x 8192, 8 tokens 32.2 33.6 31.6; 27.0
// The least of every row is taken but for 28672 x 4096, which the rule gives to
// one CTA a tile (14.9 us): its three differ by less than the rule resolves.
struct DecodePlan {
    int split, groups;
};
constexpr int kDecodeSplits[3] = {1, 2, 4};
constexpr int kDecodeGroups[3] = {148, 74, 33};  // clusters that run at once, of 148 SMs in one, two and four
constexpr double kTurnStages = 0.5, kShareStages = 5.0, kAboveStages = 21.0, kAboveStages16 = 30.0;

// Stages that `turns` turns take with `split` CTAs a tile, and that the kernel
// above takes for `tiles` of its tiles.
static double decode_stages(double turns, int64_t Ku, int split) {
    return turns * (static_cast<double>((Ku + split - 1) / split) + kTurnStages) + (split == 1 ? 0.0 : kShareStages);
}
static double above_stages(double tiles, int64_t Ku, double fixed) { return tiles * static_cast<double>(Ku) / 148 + fixed; }

static DecodePlan decode_plan(int64_t T, int64_t E, int64_t N, int64_t K, const Plan& plan) {
    DecodePlan best{0, 0};
    const int64_t share = (T + E - 1) / E;
    if (share > 16 || (E > 1 && plan.tokens > 8)) return best;
    const int64_t Nb = mx_blocks(N), Ku = (mx_blocks(K) + 1) / 2;
    const int64_t tiles = workspace_layout(T, E, N, K, {8, false}).tiles * Nb;  // of 8 tokens
    const int64_t above = E > 1 ? tiles : Nb;                                    // the kernel above's
    const double stage = share > 4 ? 1.35 : 1.0;
    double least = above_stages(static_cast<double>(above), Ku, share > 8 ? kAboveStages16 : kAboveStages);
    for (int i = 0; i < 3; ++i) {
        const int most = kDecodeGroups[i];
        const int64_t turns = (tiles + most - 1) / most;
        const double cost = decode_stages(static_cast<double>(turns), Ku, kDecodeSplits[i]) * stage;
        if (cost < least) {
            least = cost;
            best = {kDecodeSplits[i], static_cast<int>(std::min<int64_t>(tiles, most))};
        }
    }
    return best;
}

// Whether every batch of E > 1 experts that makes lo .. hi token tiles of 8 runs
// on q4_mx_decode.cu.  Costs are straight lines in the tiles but for the whole
// turns, which the line through their upper ends bounds: one split that wins
// at both ends of a range wins in all of it.  (May say no where yes holds.)
static bool all_decode(int64_t lo, int64_t hi, int64_t Nb, int64_t Ku) {
    for (int i = 0; i < 3; ++i) {
        bool wins = true;
        for (const int64_t t : {lo, hi}) {
            const int64_t tiles = t * Nb, most = kDecodeGroups[i];
            const double turns = lo == hi ? static_cast<double>((tiles + most - 1) / most)
                                          : static_cast<double>(tiles - 1) / static_cast<double>(most) + 1.0;
            wins = wins && decode_stages(turns, Ku, kDecodeSplits[i]) < above_stages(static_cast<double>(tiles), Ku, kAboveStages);
        }
        if (wins) return true;
    }
    if (lo == hi) return false;
    const int64_t mid = lo + (hi - lo) / 2;
    return all_decode(lo, mid, Nb, Ku) && all_decode(mid + 1, hi, Nb, Ku);
}

// Bytes that the call itself uses: 0 none, -1 too many units.
static int64_t workspace_used(int64_t T, int64_t E, int64_t N, int64_t K) {
    const Plan plan = plan_for(T, E);
    const Workspace l = workspace_layout(T, E, N, K, plan);
    if (l.tiles > INT32_MAX / (mx_blocks(N) * mx_blocks(K))) return -1;
    if (decode_plan(T, E, N, K, plan).split > 0) return 0;
    return static_cast<int64_t>(l.bytes);
}

// The most that T rows or fewer use, so that a workspace made for the largest
// batch serves every smaller one.  Within a class of tile sizes the bytes grow
// with T, so the last T of each class below are all there is to compare.
int64_t gemm_mx_workspace(int64_t T, int64_t E, int64_t N, int64_t K) {
    int64_t most = workspace_used(T, E, N, K);
    if (most < 0) return most;
    if (E == 1) {
        // one token tile of up to 64 (the decode kernel's rule changes at 4, 8 and 16), then of up to 120 each
        for (const int64_t last : {int64_t{4}, int64_t{8}, int64_t{16}, int64_t{64}, (T - 1) / kPairTokens * kPairTokens})
            if (last > 0 && last < T) most = std::max(most, workspace_used(last, E, N, K));
        return most;
    }
    for (const int64_t share : {2, 8, 16, 64})
        if (share * E < T) most = std::max(most, workspace_used(share * E, E, N, K));
    const int64_t few = std::min(T, 2 * E);  // rows of which some batches run on the decode kernel
    const Workspace l = workspace_layout(few, E, N, K, plan_for(few, E));
    if (static_cast<int64_t>(l.bytes) > most && !all_decode(1, l.tiles, mx_blocks(N), (mx_blocks(K) + 1) / 2))
        most = static_cast<int64_t>(l.bytes);
    return most;
}

cudaError_t launch_gemm_mx(const uint8_t* codes, const uint8_t* scales, const uint16_t* x, const int32_t* rows,
                           const int32_t* offsets, void* y, int y_type, int64_t Mx, int64_t T, int64_t E, int64_t N,
                           int64_t K, void* workspace, cudaStream_t s, const DeviceInfo& dev) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Plan plan = plan_for(T, E);
    const DecodePlan d = decode_plan(T, E, N, K, plan);
    if (d.split > 0)
        return launch_decode_mx(codes, scales, x, rows, offsets, y, y_type, Mx, T, E, N, K, d.split, d.groups, s, dev);
    const auto launch = plan.pair           ? launch_as<kPairTokens, 2>
                        : plan.tokens <= 8  ? launch_as<8, 1>
                        : plan.tokens <= 16 ? launch_as<16, 1>
                        : plan.tokens <= 32 ? launch_as<32, 1> : launch_as<64, 1>;
    return launch(plan, codes, scales, x, rows, offsets, y, y_type, Mx, T, E, N, K, ws, s, dev);
}

cudaError_t take_gemm_mx_error(unsigned int* out) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_gemm_mx_error, sizeof(unsigned int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_gemm_mx_error, &zero, sizeof(unsigned int));
    return e;
}

Q4_DEFINE_TAKE_BOUNDS(mx_gemm)

}  // namespace q4
