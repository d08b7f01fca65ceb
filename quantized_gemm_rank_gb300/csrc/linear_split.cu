// linear_split.cu -- the fused-epilogue matrix product when there are few tiles:
// few rows (a decode step, a short chunk) or a small output.
//
// What bounds it is reading the weight once, so every SM has to read.  The
// weight's columns are the MMA's rows and the tokens its N columns (16 to 256), so
// a single token wastes a 16-wide MMA and no weight traffic; the contraction is
// split over the CTAs (or CTA pairs) of a cluster, which send one another
// their partial sums by bulk copies between shared memories and add them in rank
// order (the result does not depend on timing).
//   kG = 1  up to 64 tokens, of int8 codes up to 128: a CTA takes 128 columns, M = 128
//   kG = 2  more tokens: a CTA pair takes 256 columns, M = 256; each CTA loads 128
//           columns of the weight and half the tokens, which halves what the
//           tokens cost in L2 reads
//   warp 1      TMEM allocation, MMA issue (the pair's first CTA)
//   warps 0, 2  TMA producers, every other stage each
//   the others  bring what the epilogue will read into L1; of int8 codes, widen them (below)
//   all warps   then: partial sums from TMEM to shared memory, the sum over the
//               cluster, and the epilogue, four columns a thread
// Next to that, a stage's time was its issue: one lane took 460 clocks for a stage's two copies
// (a wait, the count of bytes, 170 clocks a copy), two warps hide it; five elections and 64-bit
// offsets took 360 clocks for its MMAs, which take 128 to 512 (now 220 to 255 where the MMAs are shorter).
// That and a set-up free of divisions took 16% off 512 tokens, 4096 x 4096 (now 14.2 us), 15% off 128 tokens (9.5) and 29% off
// 512 x 1024 x 8192 (11.4).
// (Reading the other CTAs' sums with loads ran at 9 bytes a clock: 7.3 us for a pair's
// 256 x 256 sums, the longest part of the call.)
// The tensor core adds at the size of its running sum, so each 1024-deep part of
// the contraction goes to an accumulator of its own while TMEM has room, and
// these are added in fp32 with round-to-nearest.  Beyond that they are used again (two for 256
// tokens: 6144 deep each for 2000 x 1024 x 24576, split in two).
//
// Int8 codes (EPI_SCALED) come as bytes, 128 deep a stage, and warps bring them to fp16 between the copies and the MMAs: the
// weight to TMEM, from where the MMA takes its A, the tokens (and an M-major weight) to shared memory.  Blocks of 1024 stay in
// accumulators of their own, so every sum is an exact integer, in any shape.  A stage then takes 0.24 us and 2.4 ns a
// token where three teams of warps fit, 0.26 and 2.8 where two do (M-major 0.31 and 4.5): 64 tokens, 4096 x 4096 9.4 us, 256 15.5,
// 64 tokens, 28672 x 8192 58 (4.0 TB/s).  Codes go by single CTAs: of a pair, one CTA's warps would have to tell the other's that their
// half is widened, and an arrival that publishes to the cluster takes about a microsecond a stage (256 tokens 16.8 us).
#include <atomic>
#include <cmath>
#include <type_traits>

#include "epilogue.cuh"
#include "host.h"
#include "internal.h"
#include "linear.h"
#include "sm103_ptx.cuh"

namespace mc2 {

namespace {

constexpr int kTileN = 128;      // weight columns a tile (MMA M)
constexpr int kDepth = 64;       // contraction a stage
constexpr int kDepth8 = 128;     // ... of int8 codes
constexpr int kMaxStages = 16;
constexpr int kMaxCluster = 8;
constexpr int kProducers = 2;
// Threads a CTA: the pairs' tiles have more to bring out of TMEM and one CTA an SM; codes have warps that widen them.
__host__ __device__ constexpr int split_threads(int group, bool codes) { return group == 2 || codes ? 512 : 256; }
constexpr int kWidenFirst = 4;   // the first of those warps; the others are producers, MMA, and one that is idle
constexpr int kWidenTeam = 4;    // warps that widen a stage together, one for each quarter of TMEM's lanes
constexpr int kMaxTeams = 3;
static_assert(kWidenFirst % 4 == 0 && kWidenFirst + kMaxTeams * kWidenTeam <= split_threads(1, true) / 32, "warps of the teams");
constexpr int kBlockDepth = 1024;   // of one accumulator
constexpr uint32_t kWBytes = kTileN * kDepth * 2;
constexpr uint32_t kSmemPerSm = 228 * 1024;
constexpr uint32_t kSmemStatic = 288;            // this kernel's static shared memory ...
constexpr uint32_t kSmemStaticCodes = 544;       // ... and with the barriers of a ring of codes
constexpr uint32_t kMostSmem = 227 * 1024 - kSmemStatic, kMostSmemCodes = 227 * 1024 - kSmemStaticCodes;
constexpr uint32_t kSmemOverhead = 1024 + kSmemStatic;   // with the system's part of each CTA's

struct SplitParams {
    CUtensorMap w_map, x_map;
    const void *bias, *aux;
    void *out, *preact;
    int64_t ldaux, ldo, ldp;
    int m, n;
    int steps, more;          // 64-deep stages of a rank; the first `more` ranks have one more
    int share;                // tokens of a tile that a rank finishes (the last ones' may be fewer, or none)
    uint64_t m_tiles_inv;     // 2^64 / m_tiles, rounded up
    int w_kn;                 // the weight is (k, n): read M-major
    int rows;                 // tokens a tile (MMA N), a multiple of 16
    int m_tiles, split;       // token tiles; CTAs (or pairs) that share a tile's contraction
    int stages, accs, tmem_cols;
    uint32_t recv_off;        // the other CTAs' sums arrive here, (split - 1) slots of ceil(rows / split) rows
    int late;                 // ... which the ring reaches into: only once the whole cluster's MMAs are done
    int prefetch;             // the weight's first stages into L2 ahead of time
    Activation act;
    int *status;
    uint64_t wait_limit_ns;
    // int8 codes (EPI_SCALED)
    const float *x_scale, *w_scale;
    int bias_f32;
    int raws, teams;          // stages of codes, from raw_off on; teams that widen them
    uint32_t raw_off, a_cols; // ... and the weight's widened stages in TMEM, from this column on (K-major)
    int words;                // rows of out and aux begin at multiples of 8 bytes
};

// Four columns of a row, of which the first `n` (4 or more: all) are in it; whole ones in one access, where rows allow it (`words`).
template <bool kBF16>
__device__ __forceinline__ void store4(uint16_t *p, int n, const float *v, bool words) {
    const uint32_t pk[2] = {pack2<kBF16>(v[0], v[1]), pack2<kBF16>(v[2], v[3])};
    if (n >= 4 && words) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pk[0], pk[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(pk[i >> 1] >> ((i & 1) * 16));
    }
}

__device__ __forceinline__ void load4(const uint16_t *p, int n, uint32_t *w, bool words) {
    if (n >= 4 && words) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << ((i & 1) * 16);
    }
}

// kT tokens of a tile from token t on, four columns a lane: the partial sums in rank order, the
// epilogue, the outputs.  kWhole: all four columns are in the row.  `from`: the token's sums from rank 0 on, `slot`
// apart but for this CTA's own (rank `rank`), which are at `own`.  EPI_SCALED: the sums are int32, x_scale that of the tokens.
template <bool kBF16, int kEpi, int kT, bool kWhole>
__device__ __forceinline__ void finish_tokens(const SplitParams &p, const float4 *own, const float4 *from, int slot, int rank, const float *b4,
                                              const float *w4, const float *x_scale, const uint16_t *aux_row, uint16_t *pre_row, uint16_t *out_row,
                                              int n) {
    constexpr bool kCodes = kEpi == EPI_SCALED;
    if constexpr (kWhole) n = 4;
    const bool words = !kCodes || p.words != 0;
    uint32_t aux[2 * kT] = {};
    if (aux_row) {
#pragma unroll
        for (int u = 0; u < kT; ++u) load4(aux_row + u * p.ldaux, n, &aux[2 * u], words);
    }
    float v[4 * kT];
    const auto add = [](float a, float b) {
        if constexpr (kCodes) return __int_as_float(__float_as_int(a) + __float_as_int(b));
        return __fadd_rn(a, b);
    };
    auto source = [&](int r) {
        const float4 *at = r == rank ? own : from;
        if (r != rank) from += slot;
        return at;
    };
    const float4 *at = source(0);
#pragma unroll
    for (int u = 0; u < kT; ++u) {
        const float4 s = at[u * (kTileN / 4)];
        v[4 * u] = s.x, v[4 * u + 1] = s.y, v[4 * u + 2] = s.z, v[4 * u + 3] = s.w;
    }
#pragma unroll 1
    for (int r = 1; r < p.split; ++r) {
        at = source(r);
#pragma unroll
        for (int u = 0; u < kT; ++u) {
            const float4 s = at[u * (kTileN / 4)];
            v[4 * u] = add(v[4 * u], s.x), v[4 * u + 1] = add(v[4 * u + 1], s.y);
            v[4 * u + 2] = add(v[4 * u + 2], s.z), v[4 * u + 3] = add(v[4 * u + 3], s.w);
        }
    }
    if constexpr (kCodes) {
#pragma unroll
        for (int u = 0; u < kT; ++u) {
            const float s = x_scale[u];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * u + i] = __fmul_rn(__fmul_rn(__int2float_rn(__float_as_int(v[4 * u + i])), s), w4[i]);
        }
    }
    // (codes: a sum's negative zero stays one without a bias, as in the other kernels)
    if (!kCodes || p.bias) {
#pragma unroll
        for (int i = 0; i < 4 * kT; ++i) v[i] = __fadd_rn(v[i], b4[i & 3]);
    }
    if (pre_row) {
#pragma unroll
        for (int u = 0; u < kT; ++u) store4<kBF16>(pre_row + u * p.ldp, n, &v[4 * u], words);
    }
    epilogue<kBF16, kEpi>(v, aux, p.act, aux_row != nullptr);
#pragma unroll
    for (int u = 0; u < kT; ++u) store4<kBF16>(out_row + u * p.ldo, n, &v[4 * u], words);
}

// Where a lane's four columns of the tokens from `first` on are.
struct Place {
    const uint16_t *aux;
    uint16_t *pre, *out;
    int n;          // columns from the lane's first on; none: 0 or less
    float b4[4];    // their biases
    const float *x_scale;   // EPI_SCALED: the tokens' scales
    float w4[4];            // and the columns'
};

template <bool kBF16, int kEpi>
__device__ __forceinline__ Place place(const SplitParams &p, int64_t row, int col) {
    Place at = {};
    at.n = p.n - col;
    if (p.aux) at.aux = static_cast<const uint16_t *>(p.aux) + row * p.ldaux + col;
    if (p.preact) at.pre = static_cast<uint16_t *>(p.preact) + row * p.ldp + col;
    at.out = static_cast<uint16_t *>(p.out) + row * p.ldo + col;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < at.n) at.b4[i] = kEpi == EPI_SCALED && p.bias_f32 ? static_cast<const float *>(p.bias)[col + i] : load16<kBF16>(p.bias, col + i);
    }
    if constexpr (kEpi == EPI_SCALED) {
        at.x_scale = p.x_scale + row;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < at.n) at.w4[i] = p.w_scale[col + i];
    }
    return at;
}

// The tokens [first, last) of a tile, over the CTA's warps.
template <bool kBF16, int kEpi, int kThreads>
__device__ __forceinline__ void finish(const SplitParams &p, const Place &at, int first, int last, int rank, const float4 *own,
                                       const float4 *recv) {
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5;
    const int slot = (last - first) * (kTileN / 4);
    own += first * (kTileN / 4);
    const int count = last - first;
    int t = 0;   // from `first` on
    // four tokens at a time hide one another's latency, where there are that many
    if (count > kWarps) {
        for (t = 4 * warp; t + 4 <= count; t += 4 * kWarps) {
            const float4 *o = own + t * (kTileN / 4), *r = recv + t * (kTileN / 4);
            if (at.n >= 4) {
                finish_tokens<kBF16, kEpi, 4, true>(p, o, r, slot, rank, at.b4, at.w4, at.x_scale + t, at.aux ? at.aux + t * p.ldaux : nullptr,
                                                    at.pre ? at.pre + t * p.ldp : nullptr, at.out + t * p.ldo, 4);
            } else {
#pragma unroll 1
                for (int u = 0; u < 4; ++u)
                    finish_tokens<kBF16, kEpi, 1, false>(p, o + u * (kTileN / 4), r + u * (kTileN / 4), slot, rank, at.b4, at.w4, at.x_scale + t + u,
                                                         at.aux ? at.aux + (t + u) * p.ldaux : nullptr,
                                                         at.pre ? at.pre + (t + u) * p.ldp : nullptr, at.out + (t + u) * p.ldo, at.n);
            }
        }
        t = count & ~3;   // the rest, fewer than four
    }
#pragma unroll 1
    for (t += warp; t < count; t += kWarps)
        finish_tokens<kBF16, kEpi, 1, false>(p, own + t * (kTileN / 4), recv + t * (kTileN / 4), slot, rank, at.b4, at.w4, at.x_scale + t,
                                             at.aux ? at.aux + t * p.ldaux : nullptr, at.pre ? at.pre + t * p.ldp : nullptr,
                                             at.out + t * p.ldo, at.n);
}

template <bool kBF16, int kEpi, int kG>
__global__ void __launch_bounds__(split_threads(kG, kEpi == EPI_SCALED), 1) linear_split_kernel(const __grid_constant__ SplitParams p) {
    constexpr bool kCodes = kEpi == EPI_SCALED;   // int8 operands
    static_assert(!kCodes || kG == 1, "codes by single CTAs");
    constexpr int kThreads = split_threads(kG, kCodes);
    constexpr int kStep = kCodes ? kDepth8 : kDepth;      // contraction a stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar, recv_bar;
    __shared__ __align__(8) uint64_t raw_full[kCodes ? kMaxStages : 1], raw_empty[kCodes ? kMaxStages : 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;

    // (broadcast from a lane: what the compiler knows to be the same in a warp it keeps in uniform registers, where the MMA
    // and copy instructions take their operands)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int S = p.stages;
    const int ctas = p.split * kG;                       // of the cluster
    const int crank = ctas > 1 ? __shfl_sync(0xffffffffu, static_cast<int>(ptx::cluster_ctarank()), 0) : 0;
    const int half = kG == 2 ? crank & 1 : 0;            // of the pair
    const int rank = crank / kG;                         // share of the contraction
    const int x_rows = p.rows / kG;                      // tokens this CTA loads
    // (codes: of the weight, the widened stages are in TMEM where it is K-major)
    const uint32_t w_bytes = !kCodes ? kWBytes : (p.w_kn ? 2 * kWBytes : 0);
    const uint32_t stage_bytes = w_bytes + static_cast<uint32_t>(x_rows) * kStep * 2;
    const uint32_t raw_bytes = (kTileN + static_cast<uint32_t>(x_rows)) * kDepth8;
    // (no divisions: seven of them, one after another, took 0.5 us of each call.  A quotient of 32-bit numbers is the
    // high word of the product with the reciprocal rounded up to 64 bits: its error, below 2^-64 x tile, does not
    // reach the next integer.)
    const uint32_t tile = ctas > 1 ? ptx::cluster_id() : blockIdx.x;
    const uint32_t n_tile = p.m_tiles == 1 ? tile : static_cast<uint32_t>(__umul64hi(tile, p.m_tiles_inv));
    // clusters next to one another share the weight's tile
    const int n0 = static_cast<int>(n_tile * kG + half) * kTileN;
    const int m0 = static_cast<int>(tile - n_tile * p.m_tiles) * p.rows;
    const int step0 = p.steps * rank + min(rank, p.more);
    const int count = p.steps + (rank < p.more ? 1 : 0);

    // the tile's tokens, and this CTA's share of them to finish
    const int live = min(p.rows, p.m - m0);
    const auto share_from = [&](int r) { return min(live, r * p.share); };
    const int t0 = share_from(rank), t1 = share_from(rank + 1);
    const uint32_t recv_bytes = static_cast<uint32_t>((p.split - 1) * (t1 - t0)) * (kTileN * 4);

    if (warp == 1) {
        ptx::tmem_alloc<kG>(ptx::smem_u32(&tmem_slot), static_cast<uint32_t>(p.tmem_cols));
        ptx::tmem_relinquish<kG>();
    } else if (warp == 0) {
        if (lane < S) {
            ptx::mbar_init(ptx::smem_u32(&full_bar[lane]), kCodes ? kWidenTeam : 1);
            ptx::mbar_init(ptx::smem_u32(&empty_bar[lane]), 1);
        }
        if (kCodes && lane < p.raws) {
            ptx::mbar_init(ptx::smem_u32(&raw_full[lane]), 1);
            ptx::mbar_init(ptx::smem_u32(&raw_empty[lane]), kWidenTeam);
        }
        if (lane == 0) {
            failed = 0;
            ptx::mbar_init(ptx::smem_u32(&done_bar), 1);
            ptx::mbar_init(ptx::smem_u32(&recv_bar), 1);
        }
        ptx::fence_mbar_init();
        __syncwarp();
    }
    if (threadIdx.x == 0 && recv_bytes) ptx::mbar_arrive_expect_tx(ptx::smem_u32(&recv_bar), recv_bytes);
    ptx::tc_fence_before();
    __syncthreads();
    // the barriers of the cluster are ready (one CTA a share: needed when its sums are sent)
    if (ctas > 1) ptx::cluster_arrive_relaxed();
    if constexpr (kG == 2) ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    // A producer's wait for a stage tells the stage's last use from the one before only while
    // the ring is at least as long as there are producers: it has issued the step
    // `producers` back, so what the ring held before that one is consumed.
    const int ring = kCodes ? p.raws : S;
    const int producers = kCodes ? 1 : min(kProducers, ring), producer = warp == 0 ? 0 : warp - 1;   // (warp 1 issues the MMAs)
    if (warp != 1 && producer < producers && lane == 0) {
        ptx::prefetch_tmap(&p.w_map);
        ptx::prefetch_tmap(&p.x_map);
        // The weight's first stages into L2 while the stream's previous kernel ends.  Nothing is
        // read by this: were that kernel to write the weight, L2 would hold what it wrote.
        for (int i = producer; i < min(count, ring) && p.prefetch; i += producers) {
            const int k0 = (step0 + i) * kStep;
            if (p.w_kn) {
                ptx::tma_prefetch_2d(&p.w_map, n0, k0);
                if (!kCodes) ptx::tma_prefetch_2d(&p.w_map, n0 + 64, k0);
            } else {
                ptx::tma_prefetch_2d(&p.w_map, k0, n0);
            }
        }
    }
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    if (kCodes && warp != 1 && producer < producers) {
        // codes as they are, each CTA its own: 128 columns of the weight and x_rows tokens, 128 deep
        int i = 0, stage = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (; i < count; ++i) {
            const bool got = ptx::mbar_wait(ptx::smem_u32(&raw_empty[stage]), phase, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint32_t full = ptx::smem_u32(&raw_full[stage]);
            const uint32_t sw = ptx::smem_u32(smem) + p.raw_off + stage * raw_bytes;
            const int k0 = (step0 + i) * kStep;
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(full, raw_bytes);
                ptx::tma_load_2d(sw, &p.w_map, p.w_kn ? n0 : k0, p.w_kn ? k0 : n0, full);
                ptx::tma_load_2d(sw + kTileN * kStep, &p.x_map, k0, m0 + half * x_rows, full);
            }
            __syncwarp();
            if (++stage == ring) stage = 0, phase ^= 1u;
        }
        if (!ok && lane == 0) {
            atomicExch(&failed, 1);
            // the copies in flight land before the CTA can exit
            for (int back = 0; back < ring && i > 0; ++back) {
                --i;
                (void)ptx::mbar_wait(ptx::smem_u32(&raw_full[i % ring]), static_cast<uint32_t>((i / ring) & 1), p.wait_limit_ns);
            }
            ptx::nanosleep(20000);
        }
    } else if (kCodes && warp >= kWidenFirst && warp < kWidenFirst + kWidenTeam * p.teams) {
        // Codes to fp16: a team of four warps takes a 128-deep stage, the teams take turns, so that the latencies of one stage's
        // loads, stores and fences are hidden by the others' (all warps at one stage after another: 1640 clocks a stage).
        // A K-major weight goes to TMEM, a row a lane.  (Through shared memory it crosses that four times, 48 KiB in and out
        // a 64-deep stage, which takes 384 clocks; this way 16.)  An M-major one, whose rows are depth, and the tokens go to shared
        // memory, half of eight rows of 128 bytes a warp's turn: 64 codes of each, 16 a lane.  Codes and operands have the
        // 128-byte swizzle (chunk c of row r at c ^ r % 8), and the lanes' rows in the order 0 5 1 4 2 7 3 6 meet all
        // banks in eight lanes at a time, in the loads (neighbouring rows differ in bit 2) and in the stores (and in bit 0).
        // (A wait on a barrier's parity tells a phase from the one two before it only if that one cannot still be open.  With at
        // most as many teams as widened stages, a team at step i has seen the MMAs of the step two turns of them before done;
        // with a ring that is a multiple of the teams, the last user of a slot was itself.)
        const int team = (warp - kWidenFirst) / kWidenTeam, member = warp % kWidenTeam;
        const int row_in = (lane >> 3) ^ ((lane >> 2) & 1 ? 5 : 0), chunk = lane & 3, h = member & 1;
        const uint32_t rows0 = static_cast<uint32_t>((member >> 1) * 1024 + row_in * 128);   // of the first turn, either side
        const uint32_t from0 = rows0 + (((4 * h + chunk) ^ row_in) << 4);
        const uint32_t to0 = rows0 + (((2 * chunk) ^ row_in) << 4), to1 = rows0 + (((2 * chunk + 1) ^ row_in) << 4);
        // kTurns turns, 16 rows apart; from the fifth on `jump` further
        const auto widen = [&](const uint8_t *from, uint8_t *to, auto turns, uint32_t jump) {
            constexpr int kTurns = decltype(turns)::value;
            uint4 q[kTurns];
#pragma unroll
            for (int i = 0; i < kTurns; ++i) q[i] = *reinterpret_cast<const uint4 *>(from + i * 2048);
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const uint2 a = widen4(q[i].x), b = widen4(q[i].y), c = widen4(q[i].z), d = widen4(q[i].w);
                uint8_t *at = to + i * 2048 + (i >= 4 ? jump : 0);
                *reinterpret_cast<uint4 *>(at + to0) = make_uint4(a.x, a.y, b.x, b.y);
                *reinterpret_cast<uint4 *>(at + to1) = make_uint4(c.x, c.y, d.x, d.y);
            }
        };
        int rs = 0, stage = 0;
        uint32_t raw_phase = 0, phase = 1;
        const auto skip = [&](int n) {
            for (rs += n; rs >= ring; rs -= ring) raw_phase ^= 1u;
            for (stage += n; stage >= S; stage -= S) phase ^= 1u;
        };
        skip(team);
        bool ok = true;
        for (int i = team; i < count; i += p.teams) {
            const bool got = ptx::mbar_wait(ptx::smem_u32(&raw_full[rs]), raw_phase, p.wait_limit_ns) &&
                             ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), phase, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint8_t *raw = smem + p.raw_off + rs * raw_bytes;
            uint8_t *to = smem + stage * stage_bytes;
            // the tokens' turns, in fours
            const uint8_t *from = raw + kTileN * kDepth8 + from0;
            uint8_t *x_to = to + w_bytes + h * x_rows * 128;
            int left = x_rows / 16;
            for (; left >= 4; left -= 4, from += 4 * 2048, x_to += 4 * 2048) widen(from, x_to, std::integral_constant<int, 4>{}, 0);
            for (; left > 0; --left, from += 2048, x_to += 2048) widen(from, x_to, std::integral_constant<int, 1>{}, 0);
            if (p.w_kn) {
                // depth 64 on is another 64-deep part, half h a slab 8 KiB on
                widen(raw + from0, to + h * (kWBytes / 2), std::integral_constant<int, 8>{}, kWBytes / 2);
            } else {
                const uint8_t *row = raw + (32 * member + lane) * 128;
                const uint32_t a = tmem + p.a_cols + static_cast<uint32_t>(stage * (kDepth8 / 2)) + (static_cast<uint32_t>(32 * member) << 16);
                ptx::tc_fence_after();
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(row + (((4 * d + c) ^ (lane & 7)) << 4));
                        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint2 v = widen4(words[e]);
                            w[8 * c + 2 * e] = v.x, w[8 * c + 2 * e + 1] = v.y;
                        }
                    }
                    ptx::tmem_st_32x32b_x32(a + 32 * d, w);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ptx::smem_u32(&raw_empty[rs]));
                ptx::mbar_arrive(ptx::smem_u32(&full_bar[stage]));
            }
            skip(p.teams);
        }
        if (!ok && lane == 0) atomicExch(&failed, 1);
    } else if (!kCodes && warp != 1 && producer < producers) {
        // stages producer, producer + producers, ...; the warp stays converged, an elected lane issues
        int i = producer, stage = producer;
        uint32_t phase = 1;
        while (stage >= S) stage -= S, phase ^= 1u;
        bool ok = true;
        auto load = [&](uint32_t dst, const CUtensorMap *m, int c0, int c1, uint32_t bar) {
            if constexpr (kG == 2)
                ptx::tma_load_2d_pair(dst, m, c0, c1, bar);
            else
                ptx::tma_load_2d(dst, m, c0, c1, bar);
        };
        for (; i < count; i += producers) {
            const bool got = ptx::mbar_wait(ptx::smem_u32(&empty_bar[stage]), phase, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint32_t mine = ptx::smem_u32(&full_bar[stage]);
            const uint32_t full = kG == 2 && half ? ptx::mapa(mine, crank - 1) : mine;
            const uint32_t sw = ptx::smem_u32(smem) + stage * stage_bytes;
            const int k0 = (step0 + i) * kDepth;
            if (ptx::elect_one()) {
                // (the pair's first CTA counts the bytes of both)
                if (!half) ptx::mbar_arrive_expect_tx(mine, stage_bytes * kG);
                if (p.w_kn) {
                    load(sw, &p.w_map, n0, k0, full);
                    load(sw + kWBytes / 2, &p.w_map, n0 + 64, k0, full);
                } else {
                    load(sw, &p.w_map, k0, n0, full);
                }
                load(sw + kWBytes, &p.x_map, k0, m0 + half * x_rows, full);
            }
            __syncwarp();
            stage += producers;
            while (stage >= S) stage -= S, phase ^= 1u;
        }
        if (!ok && lane == 0) {
            atomicExch(&failed, 1);
            // the copies in flight, among this warp's last ones, land before the CTA can exit
            for (int back = 0; back <= S && i - producers >= 0 && !half; back += producers) {
                i -= producers;
                (void)ptx::mbar_wait(ptx::smem_u32(&full_bar[i % S]), static_cast<uint32_t>((i / S) & 1), p.wait_limit_ns);
            }
            ptx::nanosleep(20000);
        }
    } else if (warp == 1 && !half) {
        const uint32_t idesc = ptx::idesc_f16(kBF16 && !kCodes, false, kTileN * kG, p.rows, p.w_kn != 0);
        const uint32_t s0 = ptx::smem_u32(smem);
        const uint64_t w_desc = p.w_kn ? ptx::smem_desc_sw128(s0, kDepth * 128, 1024) : ptx::smem_desc_sw128(s0, 16, 1024);
        const uint64_t x_desc = ptx::smem_desc_sw128(s0 + w_bytes, 16, 1024);
        // (a stage's addresses stay within the descriptors' low words)
        const uint32_t w_hi = static_cast<uint32_t>(w_desc >> 32), w_lo0 = static_cast<uint32_t>(w_desc);
        const uint32_t x_hi = static_cast<uint32_t>(x_desc >> 32), x_lo0 = static_cast<uint32_t>(x_desc);
        const uint32_t w_kk = p.w_kn ? (2048u >> 4) : (32u >> 4);
        const uint32_t x_kk = 32u >> 4;
        const uint32_t full0 = ptx::smem_u32(&full_bar[0]), to_empty = ptx::smem_u32(&empty_bar[0]) - full0;
        const uint32_t full_end = full0 + 8u * static_cast<uint32_t>(S), advance = stage_bytes >> 4;
        const uint16_t pair = static_cast<uint16_t>(3u << crank);
        uint32_t full = full0, off = 0, phase = 0;
        bool ok = true;
        bool ready = ptx::mbar_test(full, 0);
        for (int done = 0, block = 0, acc = 0; done < count && ok; ++block) {
            const uint32_t d = tmem + static_cast<uint32_t>(acc * p.rows);
            uint32_t add = block >= p.accs ? 1u : 0u;   // an accumulator's first stage starts it from zero
            const int end = min(done + kBlockDepth / kStep, count);
            for (; done < end; ++done) {
                if (!__all_sync(0xffffffffu, ready)) {
                    ready = ptx::mbar_wait(full, phase, p.wait_limit_ns);
                    if (!__all_sync(0xffffffffu, ready)) {
                        ok = false;
                        break;
                    }
                }
                ptx::tc_fence_after();
                const uint32_t bar = full + to_empty, w_lo = w_lo0 + off, x_lo = x_lo0 + off;
                // the next stage's barrier is asked before this stage's MMAs are issued
                full += 8;
                off += advance;
                if (full == full_end) full = full0, off = 0, phase ^= 1u;
                ready = ptx::mbar_test(full, phase);
                if constexpr (kCodes) {
                    const uint32_t x_half = static_cast<uint32_t>(x_rows * 128) >> 4;
                    if (p.w_kn) {
                        ptx::mma_four_f16_ss(d, w_lo, w_hi, w_kk, x_lo, x_hi, x_kk, idesc, add);
                        ptx::mma_stage_f16_ss<kG>(d, w_lo + (kWBytes >> 4), w_hi, w_kk, x_lo + x_half, x_hi, x_kk, idesc, 1, bar, pair);
                    } else {
                        ptx::mma_stage_f16_ts(d, tmem + p.a_cols + static_cast<uint32_t>((bar - to_empty - full0) * (kDepth8 / 16)), x_lo, x_hi, x_kk,
                                              x_half, idesc, add, bar);
                    }
                } else {
                    ptx::mma_stage_f16_ss<kG>(d, w_lo, w_hi, w_kk, x_lo, x_hi, x_kk, idesc, add, bar, pair);
                }
                add = 1;
            }
            if (++acc == p.accs) acc = 0;
        }
        if (!ok && lane == 0) atomicExch(&failed, 1);
        // (also after giving up: the MMAs issued so far complete before TMEM is freed)
        if constexpr (kG == 2)
            ptx::mma_commit_pair(ptx::smem_u32(&done_bar), pair);
        else
            ptx::mma_commit<1>(ptx::smem_u32(&done_bar));
    } else if (!kCodes && warp > kProducers && p.aux) {
        // the other warps: the part of aux that this CTA will need, into L1
        constexpr int kIdle = kThreads / 32 - kProducers - 1;
        const uint16_t *aux = static_cast<const uint16_t *>(p.aux) + (static_cast<int64_t>(m0) + t0) * p.ldaux + n0;
        for (int e = (warp - kProducers - 1) * 32 + lane; e < 2 * (t1 - t0); e += 32 * kIdle)
            if (n0 + (e & 1) * 64 < p.n) ptx::prefetch_l1(aux + (e >> 1) * p.ldaux + (e & 1) * 64);
    }
    __syncwarp();
    const Place at = place<kBF16, kEpi>(p, static_cast<int64_t>(m0) + t0, n0 + 4 * lane);
    // every thread waits (bounded) for the MMAs: from here on the ring is idle
    if (!ptx::mbar_wait(ptx::smem_u32(&done_bar), 0u, p.wait_limit_ns)) atomicExch(&failed, 1);
    __syncthreads();
    bool ok = failed == 0;
    if (kG == 1 && ctas > 1) ptx::cluster_wait();
    // Others' sums are about to be copied over the ring.  What was there of 16-bit operands only copies and MMAs wrote and read, and their ends
    // have been waited for; codes were widened by this CTA's warps, whose loads and stores the arrival publishes (0.5 us).
    if (p.late) {
        if constexpr (kCodes) {
            ptx::cluster_sync();
        } else {
            ptx::cluster_arrive_relaxed();
            ptx::cluster_wait();
        }
    }
    float *part = reinterpret_cast<float *>(smem);   // [rows][128], over the ring
    // The sums leave TMEM a chunk of tokens at a time, four warps (one for each 32 columns) at a
    // chunk: first the chunks with tokens that another CTA finishes, which are sent to it, to
    // its slot of this rank among the ranks without its own; then, while those are on their
    // way, this CTA's own.
    {
        constexpr int kChunk = kG == 1 ? 16 : 32;
        const int group = warp >> 2, q = warp & 3;
        const int used = min(p.accs, (count + kBlockDepth / kStep - 1) / (kBlockDepth / kStep));
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
        // chunks [own0, own1) hold own tokens only; the others come in the order own1, ..., then 0, ...
        const int chunks = (live + kChunk - 1) / kChunk;
        const int own0 = min((t0 + kChunk - 1) / kChunk, chunks), own1 = max(own0, t1 == live ? chunks : t1 / kChunk);
        ptx::tc_fence_after();
        auto bring = [&](int c) {
            float sum[kChunk];
#pragma unroll
            for (int e = 0; e < kChunk; ++e) sum[e] = 0.0f;
            for (int a = 0; a < used; ++a) {
                uint32_t r[kChunk];
                if constexpr (kChunk == 32) {
                    ptx::tmem_ld_32x32b_x32(lanes + a * p.rows + c, r);
                    ptx::tmem_ld_wait32(r);
                } else {
                    ptx::tmem_ld_32x32b_x16(lanes + a * p.rows + c, r);
                    ptx::tmem_ld_wait16(r);
                }
#pragma unroll
                for (int e = 0; e < kChunk; ++e) {
                    if constexpr (kCodes)   // an int32, as its bits
                        sum[e] = __int_as_float(__float_as_int(sum[e]) + __float2int_rn(__uint_as_float(r[e])));
                    else
                        sum[e] = __fadd_rn(sum[e], __uint_as_float(r[e]));
                }
            }
            float *to = part + c * kTileN + 32 * q + lane;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) to[e * kTileN] = sum[e];
        };
        const int others = chunks - (own1 - own0);
        if (p.split > 1) {
            for (int i = group; i < others && ok; i += kThreads / 128) bring((i < chunks - own1 ? own1 + i : i - (chunks - own1)) * kChunk);
            ptx::fence_proxy_async_smem();
            __syncthreads();
            if (threadIdx.x < p.split && static_cast<int>(threadIdx.x) != rank) {
                const int r = threadIdx.x, first = share_from(r), n = share_from(r + 1) - first;
                const uint32_t bytes = static_cast<uint32_t>(n) * (kTileN * 4);
                if (bytes)
                    ptx::bulk_copy_to_cta(
                        ptx::mapa(ptx::smem_u32(smem) + p.recv_off + (rank < r ? rank : rank - 1) * bytes, r * kG + half),
                        ptx::smem_u32(part) + static_cast<uint32_t>(first) * (kTileN * 4), bytes,
                        ptx::mapa(ptx::smem_u32(&recv_bar), r * kG + half));
            }
            __syncwarp();
        }
        for (int i = own0 + group; i < own1 && ok; i += kThreads / 128) bring(i * kChunk);
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (p.split > 1) {
        if (recv_bytes && !ptx::mbar_wait(ptx::smem_u32(&recv_bar), 0u, p.wait_limit_ns)) ok = false;
        __syncwarp();
        ptx::cluster_arrive_relaxed();   // (what this CTA was sent is here)
    }
    if (!ok && p.status) atomicExch(p.status, -7);
    if (ok && at.n > 0) {
        const float4 *own = reinterpret_cast<const float4 *>(part) + lane;
        const float4 *recv = reinterpret_cast<const float4 *>(smem + p.recv_off) + lane;
        finish<kBF16, kEpi, kThreads>(p, at, t0, t1, rank, own, recv);
    }
    // no CTA leaves while its sums are on their way to another, nor half a pair before its MMAs' other half
    // (nothing is published by this: an arrival with release would wait for the outputs' stores, 0.9 us)
    __syncwarp();
    if (kG == 2 && p.split == 1) ptx::cluster_arrive_relaxed();
    if (ctas > 1) ptx::cluster_wait();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<kG>(tmem, static_cast<uint32_t>(p.tmem_cols));
    }
}

// The shape of a launch.
struct SplitShape {
    int group, rows, m_tiles, split, per_sm, stages, accs, tmem_cols, late, prefetch;
    int raws, teams, a_cols;   // int8 codes: stages of them as they are (0: 16-bit operands), teams, TMEM column of the weight's
    uint32_t smem, recv_off, raw_off;
    int64_t tiles;
    float us;   // what it is expected to take
};

// Fetching the weight's first stages into L2 ahead of the stream's previous kernel's end
// pays where two CTAs share most SMs (one token, 4096 x 4096, 256 CTAs: 0.9 us less), and
// costs where the loads follow at once (32 tokens, 1024 x 8192, 64 CTAs: 0.6 us more).
bool prefetch_pays(const SplitShape &s, int num_sms) {
    return s.group == 1 && s.per_sm == 2 && s.tiles * s.split * 8 >= num_sms * 13ll;
}

// Shared memory and TMEM of a launch whose tiles and split are chosen; false if it has none.
bool fit_split(SplitShape &s, int steps, int num_sms, bool codes, bool w_kn) {
    const int most = (steps + s.split - 1) / s.split;   // stages of one CTA
    const int block_steps = kBlockDepth / (codes ? kDepth8 : kDepth);
    const uint32_t x_rows = static_cast<uint32_t>(s.rows / s.group);
    const uint32_t stage = codes ? (kTileN + x_rows) * kDepth8 : kWBytes + x_rows * kDepth * 2;   // (of codes, as they are)
    const uint32_t room = s.per_sm == 2 ? 110u * 1024u : (codes ? 225u : 220u) * 1024u;
    const uint32_t sums = static_cast<uint32_t>(s.rows) * kTileN * 4;   // this CTA's, over the ring
    const uint32_t recv = static_cast<uint32_t>((s.split - 1) * ((s.rows + s.split - 1) / s.split)) * kTileN * 4;
    const int blocks = (most + block_steps - 1) / block_steps;
    s.accs = (s.per_sm == 2 ? 256 : 512) / s.rows;
    // (integer sums stay exact in an accumulator of their own for each block)
    if (codes && s.accs < blocks) return false;
    if (s.accs > blocks) s.accs = blocks;
    int columns = s.accs * s.rows, widened = 0, unit = 1;
    s.teams = 0, s.a_cols = 0;
    if (codes) {
        // teams and widened stages, the first of these that leave room for a ring of two stages a team.  A stage more than teams hides
        // the MMAs of the last one: 64 tokens, 28672 x 4096 37.5 us with (3, 4), 38.4 with (3, 3), 40.6 with (2, 3); 256 of them
        // 91.7 with (2, 3), 94.8 with (3, 3) and a ring of three, 100.9 with (2, 2).  Not beside three where the others' sums then
        // have no room beside the ring and would without it (64 tokens, 4096 x 4096 9.4 us with (3, 3), 9.7 with (3, 4); 256 of them 15.5
        // with (2, 3), 16.9 with (2, 2) all the same).
        const struct { int teams, widened; } forms[5] = {{3, 4}, {3, 3}, {2, 3}, {2, 2}, {1, 2}};
        const uint32_t wide = (w_kn ? 2 * kWBytes : 0u) + x_rows * kDepth8 * 2;
        s.a_cols = (columns + 63) / 64 * 64;
        for (const auto &f : forms) {
            const uint32_t need = f.widened * wide + 2 * f.teams * stage;
            if (need > room || (!w_kn && s.a_cols + f.widened * (kDepth8 / 2) > 512)) continue;
            if (f.teams == 3 && f.widened > 3 && need + recv > room && need - wide + recv <= room) continue;
            widened = f.widened, s.teams = unit = f.teams;
            break;
        }
        if (!w_kn) columns = s.a_cols + widened * (kDepth8 / 2);
        if (widened == 0 || columns > 512) return false;
        s.raw_off = widened * wide;
    } else {
        s.raw_off = 0;
    }
    int full = static_cast<int>((room - s.raw_off) / stage);
    if (full > kMaxStages) full = kMaxStages;
    if (codes)
        full = full / unit * unit;   // (see the kernel)
    else if (full > most)
        full = most;
    // the others' sums beside the ring, or, where that would shorten it, over it (256 tokens,
    // 4096 x 4096, split in two: 0.6 us less than with a shorter ring)
    int ring_stages = recv + s.raw_off < room ? static_cast<int>((room - s.raw_off - recv) / stage) : 0;
    if (codes) ring_stages = ring_stages / unit * unit;
    s.late = ring_stages < full && (s.group == 2 || codes);
    if (s.late || ring_stages > full) ring_stages = full;
    if (ring_stages < unit) return false;
    const uint32_t ring = s.raw_off + ring_stages * stage;
    s.stages = codes ? widened : ring_stages;
    s.raws = codes ? ring_stages : 0;
    s.recv_off = s.late || ring < sums ? sums : ring;
    const uint32_t bytes = ring > s.recv_off + recv ? ring : s.recv_off + recv;
    s.smem = bytes + 1024;   // (slack to align the ring)
    s.tmem_cols = 32;
    while (s.tmem_cols < columns) s.tmem_cols *= 2;
    // A CTA that waits for TMEM while its cluster's others hold theirs could wait for
    // ever on a CTA that waits for it, were TMEM oversubscribed by launches of two
    // streams.  So a CTA that takes 1/2^i of TMEM takes at least that part of the
    // SM's shared memory too (its static part and the system's 1 KiB included):
    // CTAs that fit beside one another find their columns free.
    const uint32_t share = static_cast<uint32_t>(s.tmem_cols) * (kSmemPerSm / 512) - 1024 - (codes ? kSmemStaticCodes : kSmemStatic);
    if (s.smem < share) s.smem = share;
    if (codes && s.smem > kMostSmemCodes) return false;
    s.prefetch = codes || prefetch_pays(s, num_sms);
    return true;
}

// Clusters of `ctas` CTAs, one an SM, that the device runs at once.  A cluster stays inside
// one GPC, so they are fewer than the SMs would hold (15 of 8 CTAs, not 19); asked once for each size.
int clusters_at_once(int ctas, int num_sms) {
    if (ctas == 1) return num_sms;
    static std::atomic<int> known[64][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) {
        (void)cudaGetLastError();
        return num_sms / ctas;
    }
    std::atomic<int> &slot = known[dev][ctas];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = linear_split_kernel<true, EPI_FORWARD, 1>;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas * num_sms), 1, 1);
        cfg.blockDim = dim3(split_threads(1, false), 1, 1);
        cfg.dynamicSmemBytes = 222 * 1024;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = num_sms / ctas > 0 ? num_sms / ctas : 1;
        }
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

// What a shape takes, in us, fitted to 1440 measurements on GB300: launch and set-up; the stages,
// each bound by its MMAs or by its bytes at 175 a ns (fitted), and the rate of device memory,
// which reads the weight once (the root of the squares' sum, since the two do not overlap
// wholly); another set-up for each further wave; per token of the tile the way from
// TMEM to the output, and to the other CTAs; less what an early prefetch saves.  Rows that are not a multiple of 128 bytes
// apart take longer to receive: a stage's 128 bytes of each lie in two lines (judged by the
// sizes: a result does not depend on the strides).
// Over 117 products (1 to 1536 tokens, 256 to 14336 columns, 1024 to 8192 deep) the
// shape it chose took 1% more than the best one on average, and at most 13%.
float split_us(const SplitShape &s, const LinearParams &p, int steps, int num_sms) {
    const int beside = s.smem <= kSmemPerSm / 2 - kSmemOverhead ? 2 : 1;   // CTAs that fit an SM
    const int64_t clusters = static_cast<int64_t>(clusters_at_once(s.group * s.split, num_sms)) * beside;
    const int64_t units = s.tiles;   // a cluster each
    // (with two CTAs an SM about a tenth more fit: 32 clusters of 8 run at once)
    const int64_t slots = beside == 2 ? clusters * 11 / 10 : clusters;
    const float waves = static_cast<float>((units + slots - 1) / slots);
    const float share = (units < clusters ? units : clusters) * s.group * s.split > num_sms ? 2.0f : 1.0f;
    const float bytes = static_cast<float>(kWBytes) + static_cast<float>(s.rows / s.group) * kDepth * 2;
    const float receive = (p.k % 64 != 0 || (!p.w_nk && p.n % 64 != 0) ? 1.87f : 1.0f) * share * bytes / 175e3f;
    const float stages = waves * ((steps + s.split - 1) / s.split) * fmaxf(0.00102f * s.rows, receive);
    const float read = static_cast<float>(p.n) * static_cast<float>(p.k) * 2.0f / 7.0e6f;
    const float stream = sqrtf(stages * stages + read * read);
    float join = 0.017f * s.rows;
    if (s.split > 1) join += 0.14f + 0.063f * s.split + 0.0116f * s.rows * (s.split - 1) / s.split;
    return 2.1f + (s.group == 2 ? 0.17f : 0.0f) + stream + waves * join + 2.0f * (waves - 1.0f) - (s.prefetch ? fminf(0.5f, 0.1f * read) : 0.0f);
}

// The same for int8 codes, fitted to 60700 measurements (10 to 1024 tokens, 512 to 28672 columns, 1024 to 16384 deep): a 128-deep
// stage is bound by what widens it, three teams or fewer, longer where they have no stage to spare; launch and set-up; per token of the tile
// the way from TMEM to the output, and to the other CTAs, longer where the sums wait for the ring; another set-up for each further wave.  The shape that it chose took
// 0.4% more than the best one on average, 8% for one in a hundred, and at most 25%.  Clusters that run at once are those of a
// GB300, so that a plan, and with it the size of a workspace, is the same wherever it is asked for: what the occupancy query says
// there, but for clusters of 3 and 5, whose last one or two (of 46 and 28) often find no place beside the last kernel's.
float split_codes_us(const SplitShape &s, const LinearParams &p, int steps) {
    constexpr int kClusters[kMaxCluster + 1] = {0, 152, 76, 45, 36, 26, 23, 15, 15};
    const int64_t clusters = kClusters[s.split];
    const float waves = static_cast<float>((s.tiles + clusters - 1) / clusters);
    const float rows = static_cast<float>(s.rows);
    float stage, join = 0.0044f * rows;
    if (p.w_nk) {
        stage = s.teams == 3 ? 0.244f + 0.0024f * rows : 0.263f + 0.0028f * rows;
        if (s.stages == s.teams) stage += s.teams == 3 ? 0.014f : 0.074f;
        if (s.teams < 3) join += 0.23f;
    } else {
        stage = s.teams > 1 ? 0.309f + 0.0045f * rows : 0.92f;
    }
    const float stages = waves * ((steps + s.split - 1) / s.split) * stage;
    const float read = static_cast<float>(p.n) * static_cast<float>(p.k) * 1.09f / 7.0e6f;
    if (s.split > 1) join += 0.0203f * rows * (s.split - 1) / s.split - 0.46f + (s.late ? 0.6f : 0.0f);
    return 4.2f + sqrtf(stages * stages + read * read) + waves * join + 3.9f * (waves - 1.0f);
}

SplitShape search_split(const LinearParams &p, int num_sms) {
    const bool codes = p.codes != 0;
    const int steps = codes ? (p.k + kDepth8 - 1) / kDepth8 : (p.k + kDepth - 1) / kDepth;
    SplitShape best = {};
    // tiles of at most 64 tokens by single CTAs; of 64, 128 or 256 by pairs, of codes of 128 by single CTAs
    const struct { int group, most; } forms[4] = {{1, 64}, {codes ? 1 : 2, codes ? 128 : 64}, {2, 128}, {2, 256}};
    for (const auto &f : forms) {
        if (codes && f.group == 2) break;
        if (f.group == 2 && p.m <= 32) continue;
        if (f.most > 64 && p.m <= f.most / 2) continue;   // the smaller tile does the same
        SplitShape s = {};
        s.group = f.group;
        const int unit = f.group == 1 ? 16 : 32, cols = kTileN * f.group;
        s.m_tiles = (p.m + f.most - 1) / f.most;
        s.rows = ((p.m + s.m_tiles - 1) / s.m_tiles + unit - 1) / unit * unit;
        s.tiles = static_cast<int64_t>(s.m_tiles) * ((p.n + cols - 1) / cols);
        for (s.split = 1; s.split <= kMaxCluster / f.group && s.split <= steps; ++s.split) {
            // two CTAs an SM where there are more than SMs and their stages are short: 0.2 us less for one token, 4096 x 4096;
            // but 1.7 us more for 32 tokens, 1024 x 8192, 64 CTAs
            s.per_sm = !codes && f.group == 1 && s.rows <= 32 && s.tiles > clusters_at_once(s.split, num_sms) ? 2 : 1;
            if (!fit_split(s, steps, num_sms, codes, !p.w_nk)) continue;
            s.us = codes ? split_codes_us(s, p, steps) : split_us(s, p, steps, num_sms);
            if (best.group == 0 || s.us < best.us) best = s;
        }
    }
    return best;
}

// The shape for p.  A product of codes asks for it as its workspace is asked for, as it is planned and as it is launched, so a host
// thread keeps the last one of these (it goes by the sizes alone; a search takes 1 us).
SplitShape best_split(const LinearParams &p, int num_sms) {
    if (!p.codes) return search_split(p, num_sms);
    thread_local struct { int m, n, k, w_nk; SplitShape shape; } last = {};
    if (last.m != p.m || last.n != p.n || last.k != p.k || last.w_nk != p.w_nk) last = {p.m, p.n, p.k, p.w_nk, search_split(p, num_sms)};
    return last.shape;
}

template <bool kBF16, int kEpi, int kG>
cudaError_t launch_split(const SplitParams &p, const SplitShape &s, cudaStream_t stream) {
    auto kern = linear_split_kernel<kBF16, kEpi, kG>;
    thread_local unsigned long long ready_ctx = 0;
    const unsigned long long ctx = current_context_id();
    if (ctx == 0 || ctx != ready_ctx) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kEpi == EPI_SCALED ? kMostSmemCodes : kMostSmem);
        if (e != cudaSuccess) return e;
        ready_ctx = ctx;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.split * kG);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(s.tiles * s.split * kG), 1, 1);
    cfg.blockDim = dim3(split_threads(kG, kEpi == EPI_SCALED), 1, 1);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = s.split * kG > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// what a tensor map takes: 16-byte units, and rows less than 2^40 bytes apart
bool rows_fit(const void *p, int64_t ld) { return !p || (host::aligned16(p) && ld % 8 == 0 && ld < (1ll << 39)); }

}  // namespace

bool linear_layout_fits(const LinearParams &p) {
    // the kernels count rows, columns and stages in 32 bits, up to a tile past the end
    constexpr int kMost = INT32_MAX - 512;
    if (p.m > kMost || p.n > kMost || p.k > kMost) return false;
    return rows_fit(p.x, p.ldx) && rows_fit(p.w, p.ldw) && rows_fit(p.out, p.ldo) && rows_fit(p.preact, p.ldp) &&
           rows_fit(p.aux, p.ldaux);
}

bool linear_prefers_split(const LinearParams &p, int num_sms) {
    // the tiles' outputs leave by tensor copies, which write whole 16-byte units: a row
    // that ends inside one would have up to 7 elements past its end overwritten
    if (p.n % 8 != 0) return true;
    if (p.m <= 64) return true;
    // the 256 x 256 tiles: 6.3 us and 0.29 a 64-deep stage for each wave of them (1024 deep 10.6 to
    // 12.5 us, 4096 deep 24.0 to 25.6, 8192 deep 40.5 to 43.5, two waves 42.7 to 45).  Where the two cross, at
    // (m, 4096) with k = 4096, both in one run: 512 tokens 15.1 us split against 24.4, 777 21.6 against 25.0, 1024
    // 24.0 against 25.5, 1536 43.8 against 42.7.
    const int64_t tiles = ((p.m + 255ll) / 256) * ((p.n + 255ll) / 256), pairs = num_sms / 2;
    const SplitShape s = best_split(p, num_sms);
    const int steps = (p.k + kDepth - 1) / kDepth, blocks = ((steps + s.split - 1) / s.split * kDepth + kBlockDepth - 1) / kBlockDepth;
    // where the tiles fill the device, no sum is left deeper in one accumulator than it would be in theirs
    if (tiles >= pairs && (blocks + s.accs - 1) / s.accs * (kBlockDepth / kDepth) > linear_tiles_block(p.k)) return false;
    const float us = 6.3f + 0.29f * static_cast<float>((tiles + pairs - 1) / pairs) * steps;
    return s.us < us;
}

float linear_split_codes_us(const LinearParams &p) {
    const SplitShape s = best_split(p, 0);   // (asks for no number of SMs)
    return s.group == 0 ? -1.0f : s.us;
}

cudaError_t launch_linear_split(bool bf16, const LinearParams &lp, int num_sms, cudaStream_t stream) {
    const SplitShape s = best_split(lp, num_sms);
    if (s.group == 0 || s.tiles * s.split * s.group > INT32_MAX) return cudaErrorInvalidValue;
    SplitParams p = {};
    const uint64_t m = lp.m, n = lp.n, k = lp.k;
    bool ok;
    if (lp.codes)
        ok = host::make_map8(&p.x_map, lp.x, k, m, static_cast<uint32_t>(s.rows / s.group), lp.ldx) &&
             host::make_map8(&p.w_map, lp.w, lp.w_nk ? k : n, lp.w_nk ? n : k, 128, lp.ldw);
    else
        ok = host::make_map16(&p.x_map, lp.x, k, m, kDepth, static_cast<uint32_t>(s.rows / s.group), lp.ldx);
    if (!lp.codes)
        ok = ok && (lp.w_nk ? host::make_map16(&p.w_map, lp.w, k, n, kDepth, kTileN, lp.ldw)
                            : host::make_map16(&p.w_map, lp.w, n, k, 64, kDepth, lp.ldw));
    if (!ok) return cudaErrorInvalidValue;
    p.bias = lp.bias, p.aux = lp.aux_mode == AUX_NONE ? nullptr : lp.aux, p.out = lp.out, p.preact = lp.preact;
    p.ldaux = lp.ldaux, p.ldo = lp.ldo, p.ldp = lp.ldp;
    p.m = lp.m, p.n = lp.n;
    const int steps = lp.codes ? (lp.k + kDepth8 - 1) / kDepth8 : (lp.k + kDepth - 1) / kDepth;
    p.steps = steps / s.split, p.more = steps % s.split;
    p.share = ((lp.m < s.rows ? lp.m : s.rows) + s.split - 1) / s.split;
    p.m_tiles_inv = UINT64_MAX / static_cast<uint64_t>(s.m_tiles) + 1;   // (0 for one tile: not used)
    p.w_kn = !lp.w_nk;
    p.rows = s.rows, p.m_tiles = s.m_tiles, p.split = s.split;
    p.stages = s.stages, p.accs = s.accs, p.tmem_cols = s.tmem_cols;
    p.recv_off = s.recv_off, p.late = s.late, p.prefetch = s.prefetch;
    p.act = activation_of(lp.act);
    p.status = device_status_word();
    p.wait_limit_ns = host::kWaitLimitNs;
    if (lp.codes) {
        p.x_scale = lp.x_scale, p.w_scale = lp.w_scale, p.bias_f32 = lp.bias_f32;
        p.raws = s.raws, p.teams = s.teams, p.raw_off = s.raw_off, p.a_cols = static_cast<uint32_t>(s.a_cols);
        const auto words = [](const void *q, int64_t ld) { return reinterpret_cast<uintptr_t>(q) % 8 == 0 && ld % 4 == 0; };
        p.words = words(lp.out, lp.ldo) && (!p.aux || words(p.aux, lp.ldaux));
        return bf16 ? launch_split<true, EPI_SCALED, 1>(p, s, stream) : launch_split<false, EPI_SCALED, 1>(p, s, stream);
    }
    const bool back = lp.aux_mode == AUX_ACT_GRAD;
    if (s.group == 1) {
        if (back) return bf16 ? launch_split<true, EPI_BACKWARD, 1>(p, s, stream) : launch_split<false, EPI_BACKWARD, 1>(p, s, stream);
        return bf16 ? launch_split<true, EPI_FORWARD, 1>(p, s, stream) : launch_split<false, EPI_FORWARD, 1>(p, s, stream);
    }
    if (back) return bf16 ? launch_split<true, EPI_BACKWARD, 2>(p, s, stream) : launch_split<false, EPI_BACKWARD, 2>(p, s, stream);
    return bf16 ? launch_split<true, EPI_FORWARD, 2>(p, s, stream) : launch_split<false, EPI_FORWARD, 2>(p, s, stream);
}

}  // namespace mc2
