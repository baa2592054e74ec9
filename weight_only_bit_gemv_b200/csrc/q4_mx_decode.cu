// q4_mx_decode.cu -- products with microscaled matrices in tiles of 8 tokens, for
// decode: one launch, no workspace.
//
// The mathematics is q4_mx_gemm.cu's: hi and lo rows of 8 tokens are the 16
// columns of one block-scaled MMA.  What differs is who prepares x and who
// adds up a tile's parts, because at one token a projection streams for a
// microsecond or two and a launch before it or counters in memory cost more
// than that:
//  * x's parts are made by five warps of the CTA that uses them, straight into
//    the stage's shared memory, while the codes of the same stage are on their
//    way.  A stage takes a warp some 700 cycles, most of them latency, so the
//    warps take the stages in turn (all on each stage, they were the limit);
//  * a tile's K is cut in kSplit equal parts over the CTAs of a cluster, and
//    the first CTA adds the others' sums, which they put into its shared memory.
// Clusters take the tiles in turn.  With kSplit = 1 a CTA takes whole tiles.
// Roles: warp 0 streams codes and exponents, warp 1 issues the MMAs, warps 2-5
// read the accumulators and write y, warps 6-10 prepare x.
// Measured on B200 at one token, back to back in a graph: 4096 x 4096 6.1 us, of
// which 3 us are launch, prologue, first load and epilogue; 28672 x 4096 15.0 us
// (4.2 TB/s; an SM takes a stage of 17 KB in 0.31 us); 28672 x 8192 24.9 us (5.0
// TB/s); 128256 x 4096 44.7 us (6.3 TB/s).
// Every wait is bounded, as in q4_mx_gemm.cu.
#include <algorithm>

#include "q4_mx_tc.cuh"

namespace q4 {

__device__ unsigned int g_decode_mx_error;

namespace {

constexpr int kTokens = 8;
constexpr int kCols = 2 * kTokens;
constexpr int kUnit = 2;                     // k blocks of a stage
constexpr int kFlush = 4;                    // stages per accumulation in tensor memory (1024 k)
constexpr int kABytes = kMxBlock * 128;      // a block's codes spread over bytes
constexpr int kBBytes = kCols * 128;
constexpr int kBAt = kUnit * kABytes;
constexpr int kSfaAt = kBAt + kUnit * kBBytes;
constexpr int kSfbAt = kSfaAt + kUnit * kMxScaleBytes;
constexpr int kStagePitch = kSfbAt + kUnit * kMxScaleBytes;  // 38 KB
constexpr int kStages = 5;
constexpr int kXWarps = kStages;             // warps that prepare x, one for each slot of the ring
constexpr int kThreads = (6 + kXWarps) * 32;
constexpr int kMaxSplit = 4;
constexpr int kPartBytes = kTokens * kMxBlock * 4;           // one CTA's sums of a tile
constexpr int kPartsAt = kStages * kStagePitch;              // [2][kMaxSplit - 1] parts
constexpr int kTableAt = kPartsAt + 2 * (kMaxSplit - 1) * kPartBytes;
constexpr int kTailAt = (kTableAt + static_cast<int>(sizeof(Table)) + 15) / 16 * 16;
constexpr int kSmem = 1024 + kTailAt + 256;
constexpr uint32_t kScaleCol = 2 * kCols;                    // after two accumulators, two sets of exponents
constexpr uint32_t kScaleSet = 8 * kUnit;
constexpr uint32_t kDecodeCols = 64;
constexpr unsigned long long kSumsLandNs = 1000000;          // a store to another CTA's shared memory takes about 1 us
static_assert(kStagePitch % 1024 == 0 && kScaleCol + 2 * kScaleSet <= kDecodeCols, "layout");

struct MxDecode {
    const uint8_t* wsf;      // exponent bytes of W
    const uint16_t* x;
    const int32_t* rows;     // x row of each of the T rows; nullptr: the row itself
    const int32_t* offsets;  // first row of each expert; nullptr: one matrix
    void* y;
    int64_t Mx, N, K;
    int T, E, Nb, Kb, Ku, y_bf16;
};

// A tile of a cluster's turn, and the CTA's part of its K in stages.
struct Tile {
    int e, nb, first, count;
};

// Tiles in order of expert, row block, token tile.
struct Turns {
    int next, step, tiles;
    __device__ Turns(const MxDecode& p, const Table& t, int group, int groups)
        : next(group), step(groups), tiles(t.tile[p.E] * p.Nb) {}
    __device__ bool take(const MxDecode& p, const Table& t, Tile& s) {
        if (next >= tiles) return false;
        s.e = p.E == 1 ? 0 : find_expert(t.tile, p.E, next / p.Nb);
        const int local = next - t.tile[s.e] * p.Nb, mine = t.tile[s.e + 1] - t.tile[s.e];
        s.nb = mine == 1 ? local : local / mine;
        s.first = t.offset[s.e] + (local - s.nb * mine) * kTokens;
        s.count = min(kTokens, t.offset[s.e + 1] - s.first);
        next += step;
        return true;
    }
};

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
// Four floats into another CTA's shared memory, counted by a barrier there:
// the reader needs no more than that barrier (stores with a release and an
// acquire on the cluster's scope took 1.4 us a tile).
__device__ __forceinline__ void store_counted(uint32_t addr, const float* v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar)
                 : "memory");
}

template <int kSplit, bool kVector>
__global__ void __launch_bounds__(kThreads, 1)
    decode_mx_kernel(const __grid_constant__ CUtensorMap wmap, const MxDecode p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    Table& table = *reinterpret_cast<Table*>(smem + kTableAt);
    const uint32_t bars = base + kTailAt;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto dfull = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto dempty = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };
    auto parts_in = [&](int b) { return bars + 8u * (2 * kStages + 4 + b); };    // the others' sums are here
    auto parts_free = [&](int b) { return bars + 8u * (2 * kStages + 6 + b); };  // the first CTA has read them
    const uint32_t drain = bars + 8u * (2 * kStages + 8);
    const uint32_t words = drain + 8u;  // tensor-memory base, abort
    volatile uint32_t* word = reinterpret_cast<volatile uint32_t*>(smem + (words - base));
    volatile uint32_t* abort_flag = word + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int rank = kSplit == 1 ? 0 : static_cast<int>(cluster_rank());
    const int group = blockIdx.x / kSplit, groups = gridDim.x / kSplit;
    // this CTA's part of every tile's K, in stages
    const int k_begin = p.Ku * rank / kSplit, k_end = p.Ku * (rank + 1) / kSplit;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 2);  // the loads' bytes and the warp that prepares x
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull(b), 1);
            mbar_init(dempty(b), 4);
            mbar_init(parts_in(b), 1);
            mbar_init(parts_free(b), 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensor_map(&wmap);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(words), "r"(kDecodeCols)
                     : "memory");
        tmem_relinquish();
    }
    tc_fence_before();
    // all that follows may read what earlier kernels of the stream wrote
    pdl_wait();
    fill_table(table, p.offsets, p.E, p.T, kTokens);  // ends in __syncthreads
    if (kSplit > 1) cluster_sync();                   // the others' barriers exist
    tc_fence_after();
    const uint32_t tmem = *word;

    int issued = 0;  // stages that the producer has asked for

    if (warp == 0) {
        // ------------------------------ producer ------------------------------
        bool ok = true, filled = false;
        Turns turns(p, table, group, groups);
        Tile s;
        Ring<kStages> ring;
        while (ok && turns.take(p, table, s)) {
            const int64_t block = (static_cast<int64_t>(s.e) * p.Nb + s.nb) * p.Kb;
            for (int k = k_begin; k < k_end; ++k) {
                if (filled && !wait_bar(empty(ring.slot), ring.parity ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const int kb = k * kUnit, blocks = min(kUnit, p.Kb - kb);
                    const uint32_t dst = base + ring.slot * kStagePitch, bar = full(ring.slot);
                    mbar_arrive_expect_tx(bar, kUnit * kMxCodeBytes + blocks * kMxScaleBytes);
                    tma_load_2d(dst, &wmap, 0, static_cast<int>((block + kb) * kMxBlock), bar);
                    if (Q4_IN_BOUNDS(block + kb, blocks, static_cast<int64_t>(p.E) * p.Nb * p.Kb))
                        bulk_load(dst + kSfaAt, p.wsf + (block + kb) * kMxScaleBytes, blocks * kMxScaleBytes, bar);
                }
                __syncwarp();
                ++issued;
                ring.next();
                if (ring.slot == 0) filled = true;
            }
        }
        if (!ok && lane == 0) {
            atomicOr(&g_decode_mx_error, 1u);
            *abort_flag = 1;
        }
    } else if (warp == 1) {
        // -------------------------------- MMA ---------------------------------
        bool ok = true, reused = false;
        Turns turns(p, table, group, groups);
        Tile s;
        Ring<kStages> ring;
        Ring<2> dring;
        uint32_t set = 0;
        const uint64_t adesc = smem_desc_sw128(base, 1024), sdesc = scale_desc(base);
        while (ok && turns.take(p, table, s)) {
            for (int k0 = k_begin; ok && k0 < k_end; k0 += kFlush) {
                const int k1 = min(k_end, k0 + kFlush);
                if (reused && !wait_bar(dempty(dring.slot), dring.parity ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + dring.slot * kCols;
                for (int k = k0; k < k1; ++k) {
                    if (!wait_bar(full(ring.slot), ring.parity, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = static_cast<uint32_t>(ring.slot) * (kStagePitch >> 4);
                        const uint32_t sf = tmem + kScaleCol + set * kScaleSet;
                        const int blocks = min(kUnit, p.Kb - k * kUnit);
#pragma unroll
                        for (int u = 0; u < kUnit; ++u) {
                            if (u >= blocks) break;
                            tc_copy_scales<1>(sf + 8 * u, sdesc + at + (kSfaAt + u * kMxScaleBytes) / 16);
                            tc_copy_scales<1>(sf + 8 * u + 4, sdesc + at + (kSfbAt + u * kMxScaleBytes) / 16);
                        }
#pragma unroll
                        for (int u = 0; u < kUnit; ++u) {
                            if (u >= blocks) break;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                tc_mma_mx<1>(d, adesc + at + (u * kABytes + 32 * q) / 16,
                                             adesc + at + (kBAt + u * kBBytes + 32 * q) / 16,
                                             mx_idesc(kMxBlock, kCols, q), sf + 8 * u, sf + 8 * u + 4,
                                             (k > k0 || u > 0 || q > 0) ? 1u : 0u);
                        }
                        tc_commit(empty(ring.slot));
                        if (k == k1 - 1) tc_commit(dfull(dring.slot));
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
            atomicOr(&g_decode_mx_error, 2u);
            *abort_flag = 1;
        }
        __syncwarp();
        if (elect_one()) tc_commit(drain);
        if (!mbar_wait(drain, 0u) && lane == 0) atomicOr(&g_decode_mx_error, 4u);
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------ epilogue ------------------------------
        const int quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        Ring<2> dring, pring;
        bool ok = true, reused = false;
        Turns turns(p, table, group, groups);
        Tile s;
        while (ok && turns.take(p, table, s)) {
            float acc[kTokens];
#pragma unroll
            for (int i = 0; i < kTokens; ++i) acc[i] = 0.0f;
            for (int k0 = k_begin; k0 < k_end; k0 += kFlush) {
                ok = wait_bar(dfull(dring.slot), dring.parity, abort_flag);
                if (!ok) break;
                tc_fence_after();
                uint32_t hi[kTokens], lo[kTokens];
                tc_ld_x8(lanes + dring.slot * kCols, hi);
                tc_ld_x8(lanes + dring.slot * kCols + kTokens, lo);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < kTokens; ++i) acc[i] += __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty(dring.slot));
                dring.next();
            }
            if (!ok) break;
            // a part: 128 rows of 8 sums, the second four only for more than 4 tokens
            const uint32_t part0 = base + kPartsAt + pring.slot * (kMaxSplit - 1) * kPartBytes + row * kTokens * 4;
            if (rank > 0) {
                // to the first CTA, once it has read what was there before
                ok = !reused || wait_bar(parts_free(pring.slot), pring.parity ^ 1u, abort_flag);
                if (!ok) break;
                const uint32_t to = in_cta(part0 + static_cast<uint32_t>((rank - 1) * kPartBytes), 0);
                const uint32_t bar = in_cta(parts_in(pring.slot), 0);
                store_counted(to, acc, bar);
                if (s.count > 4) store_counted(to + 16, acc + 4, bar);
            } else {
                if (kSplit > 1) {
                    if (tid == 64)
                        mbar_arrive_expect_tx(parts_in(pring.slot), (kSplit - 1) * kMxBlock * 16 * (s.count > 4 ? 2 : 1));
                    ok = wait_bar(parts_in(pring.slot), pring.parity, abort_flag);
                    if (!ok) break;
#pragma unroll
                    for (int c = 0; c < kSplit - 1; ++c) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (4 * h >= s.count) break;
                            const float4 v = ld_smem<float4>(smem, part0 - base + c * kPartBytes + 16 * h);
                            acc[4 * h] += v.x;
                            acc[4 * h + 1] += v.y;
                            acc[4 * h + 2] += v.z;
                            acc[4 * h + 3] += v.w;
                        }
                    }
                    __syncwarp();
                    if (lane < kSplit - 1) arrive_cluster(in_cta(parts_free(pring.slot), lane + 1));
                }
                const int64_t n = static_cast<int64_t>(s.nb) * kMxBlock + row;
                const int64_t at = static_cast<int64_t>(s.first) * p.N + n;
                if (n < p.N && Q4_IN_BOUNDS(at + (s.count - 1) * p.N, 1, static_cast<int64_t>(p.T) * p.N)) {
#pragma unroll
                    for (int m = 0; m < kTokens; ++m) {
                        if (m >= s.count) break;
                        if (p.y_bf16)
                            static_cast<__nv_bfloat16*>(p.y)[at + m * p.N] = __float2bfloat16_rn(acc[m]);
                        else
                            static_cast<float*>(p.y)[at + m * p.N] = acc[m];
                    }
                }
            }
            pring.next();
            if (pring.slot == 0) reused = true;
        }
        if (!ok && lane == 0) {
            atomicOr(&g_decode_mx_error, 8u);
            *abort_flag = 1;
        }
    } else {
        // -------------------------------- x's parts -----------------------------
        // rows of y behind the last expert's
        const int64_t behind = table.offset[p.E] * p.N, all = static_cast<int64_t>(p.T) * p.N;
        for (int64_t i = behind + blockIdx.x * (kXWarps * 32) + (tid - 192); i < all;
             i += static_cast<int64_t>(gridDim.x) * (kXWarps * 32)) {
            if (!Q4_IN_BOUNDS(i, 1, all)) continue;
            if (p.y_bf16)
                static_cast<uint16_t*>(p.y)[i] = 0;
            else
                static_cast<float*>(p.y)[i] = 0.0f;
        }
        // Each warp prepares the stages of one slot, for all tokens, and has the
        // x of its next one on the way.  (As many warps as slots: a warp that
        // came to a slot two uses late or early could not tell them apart by
        // the barrier's parity.)
        bool ok = true, more = k_begin < k_end;
        const int slot = warp - 6;
        int k = k_begin + slot, count = 0;
        uint32_t parity = 1;  // of the use before this one
        bool filled = false;
        Turns turns(p, table, group, groups);
        Tile s;
        more = more && turns.take(p, table, s);
        uint4 q[kTokens], ahead[kTokens];
        auto fetch = [&] {
            while (more && k >= k_end) {
                k -= k_end - k_begin;
                more = turns.take(p, table, s);
            }
            if (!more) return;
            const int64_t kx = static_cast<int64_t>(k) * kUnit * kMxBlock + 8 * lane;
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                if (m >= s.count && m % 2 == 0) break;  // tokens go in pairs, the last perhaps with zeros
                const int64_t src = m >= s.count ? -1 : p.rows ? static_cast<int64_t>(__ldg(p.rows + s.first + m)) : s.first + m;
                const bool have = src >= 0 && src < p.Mx;
                ahead[m] = load_x8<kVector>(p.x, have, (have ? src * p.K : 0) + kx, kx, p.K, p.Mx * p.K);
            }
            count = s.count;
            k += kXWarps;
        };
        fetch();
        const int kb_of = lane / 16, c = lane % 16 / 2;  // k block of the stage and 16-byte piece of the lane's eight k
        while (ok && more) {
#pragma unroll
            for (int m = 0; m < kTokens; ++m) q[m] = ahead[m];
            const int tokens = count;
            fetch();
            if (filled && !wait_bar(empty(slot), parity, abort_flag)) {
                ok = false;
                break;
            }
            uint8_t* stage = smem + slot * kStagePitch;
#pragma unroll
            for (int m0 = 0; m0 < kTokens; m0 += 2) {
                if (m0 >= tokens) break;
                XParts parts[2];
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    parts[j] = split_x(q[m0 + j]);
                    gather_bytes(parts[j].byte, lane, hi[j], lo[j]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int m = m0 + j;
                    // 128-byte rows in the 128-byte swizzle: 16-byte piece c of row r is at c ^ (r % 8)
                    uint8_t* to = stage + kBAt + kb_of * kBBytes + m * 128 + ((c ^ m) * 16) + (lane & 1) * 8;
                    *reinterpret_cast<uint2*>(to) = parts[j].hi;
                    *reinterpret_cast<uint2*>(to + kTokens * 128) = parts[j].lo;
                    if ((lane & 15) == 0) {
                        uint8_t* sf = stage + kSfbAt + kb_of * kMxScaleBytes;
                        *reinterpret_cast<uint32_t*>(sf + mx_scale_at(m, 0)) = hi[j];
                        *reinterpret_cast<uint32_t*>(sf + mx_scale_at(m + kTokens, 0)) = lo[j];
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full(slot));
            parity ^= 1u;
            filled = true;
        }
        if (!ok && lane == 0) {
            atomicOr(&g_decode_mx_error, 16u);
            *abort_flag = 1;
        }
    }

    // -------------------------------- teardown --------------------------------
    // The MMAs waited for every load and the first CTA for the others' sums, so
    // nothing is in flight here unless some role gave up.  Then the producer
    // waits for its last stages (one without its x ends by the limit, which is
    // far longer than a copy takes), and a first CTA stays until what was still
    // on its way to it has landed.
    __syncwarp();  // a role may have left its loop lane by lane
    tc_fence_before();
    __syncthreads();
    const bool gave_up = *abort_flag != 0u;
    if (gave_up && warp == 0)
        for (int i = max(issued - kStages, 0); i < issued; ++i)
            if (!mbar_wait(full(i % kStages), static_cast<uint32_t>(i / kStages) & 1u)) break;
    __syncwarp();
    if (kSplit > 1) {
        cluster_sync();  // no CTA's memory goes while another may use it
        if (gave_up && rank == 0) {
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kSumsLandNs) {
            }
        }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kDecodeCols);
    }
}

template <int kSplit>
cudaError_t launch_split(const CUtensorMap& wmap, const MxDecode& p, int groups, cudaStream_t s, const DeviceInfo& dev) {
    const bool vector = p.K % 8 == 0;
    const auto kernel = vector ? decode_mx_kernel<kSplit, true> : decode_mx_kernel<kSplit, false>;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem,
                                           107 + (kSplit == 1 ? 0 : kSplit == 2 ? 1 : 2) * 2 + vector, dev.device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSplit;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(groups * kSplit));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = kSplit == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, wmap, p);
}

}  // namespace

cudaError_t launch_decode_mx(const uint8_t* codes, const uint8_t* scales, const uint16_t* x, const int32_t* rows,
                             const int32_t* offsets, void* y, int y_type, int64_t Mx, int64_t T, int64_t E, int64_t N,
                             int64_t K, int split, int groups, cudaStream_t s, const DeviceInfo& dev) {
    const int64_t Nb = mx_blocks(N), Kb = mx_blocks(K);
    CUtensorMap wmap;
    const cudaError_t e = encode_tensor_map_2d(&wmap, codes, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 0,
                                               static_cast<uint64_t>(E * Nb * Kb * kMxBlock), kMxBlock, 64,
                                               kUnit * kMxBlock, kMxBlock, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    if (kSmem > dev.smem_optin) return cudaErrorNotSupported;
    MxDecode p{};
    p.wsf = scales;
    p.x = x;
    p.rows = rows;
    p.offsets = offsets;
    p.y = y;
    p.Mx = Mx;
    p.N = N;
    p.K = K;
    p.T = static_cast<int>(T);
    p.E = static_cast<int>(E);
    p.Nb = static_cast<int>(Nb);
    p.Kb = static_cast<int>(Kb);
    p.Ku = static_cast<int>((Kb + kUnit - 1) / kUnit);
    p.y_bf16 = y_type == Q4_BF16;
    if (split == 1) return launch_split<1>(wmap, p, groups, s, dev);
    if (split == 2) return launch_split<2>(wmap, p, groups, s, dev);
    return launch_split<4>(wmap, p, groups, s, dev);
}

cudaError_t take_decode_mx_error(unsigned int* out) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(out, g_decode_mx_error, sizeof(unsigned int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_decode_mx_error, &zero, sizeof(unsigned int));
    return e;
}

Q4_DEFINE_TAKE_BOUNDS(mx_decode)

}  // namespace q4
