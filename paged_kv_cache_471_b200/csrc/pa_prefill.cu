// Prefill attention over the paged cache (pa_prefill; see include/pagedattn.h
// for the contract): the last n_s tokens of each sequence attend causally over
// the sequence's cached keys and values, their own among them.
//
// One CTA per (group of query tokens, kv head, key partition).  Its rows are
// (query token, head of the kv head's group) pairs, tokens slowest, in two
// tiles of 128 rows; key tiles of 128 tokens pass by once for all 256 rows:
//   * the loader warps, from 8 on, gather the tile's pages into shared memory as
//     tensor-core operands.  Both page layouts are K-major already (K: 16-byte
//     columns of 8 head dims; V: rows of B tokens), so two warps' TMA copies put
//     bf16 pages in place without a register; 8-bit codes are widened to f16
//     (exact) on the way, by three warps;
//   * the warp after them issues the products: S = Q K^T into TMEM, then O += P V
//     with P read from TMEM, where it lies over the S it came from;
//   * warps 0-3 and 4-7 hold a row of one tile per thread: the running maximum
//     and sum, P = 2^(x - m) back to TMEM.  While one tile is in softmax, the
//     tensor cores work on the other's products.
// O is rescaled only when a row's maximum has grown by more than 2^8 since the
// last time: until then the weights are simply up to 256, which bf16 and f16
// carry at the same relative precision.
//
// Bound: 4 D flops per (row, key) on the tensor cores, against one exponential
// per (row, key): 16 a clock and SM, so at D = 128 both need the same time, 2048
// clocks a step of the 256 rows.  A step takes 3500, 4000 when a row rescales: a
// tile's chain of softmax (1980: scores loaded 240, maximum 350, weights 1390),
// hand-overs (620) and its own products.  Measured, D = 128:
//   1 prompt of 8192 tokens, 32/8 heads, bf16        557-632 us, 870-985 TFLOP/s
//   4 chunks of 257-1025 tokens behind up to 4001,
//   64/8 heads, e4m3 blocks                          355-357 us, 665-670 TFLOP/s
// (the first at the card's power limit).  At 168 registers every form spills: 64
// to 124 bytes of stores, 200 in the e4m3 block forms of D = 128, whose second
// loop (see kNarrow) counts with it.  Part of the exponentials as a
// polynomial on the FMA pipes made it slower: a quarter of them 671, half 732 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "pa_launch.cuh"
#include "pa_query_start.cuh"
#include "pa_tcgen05.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

constexpr int kRows = 128;        // rows of a tile (M of the products)
constexpr int kTiles = 2;         // tiles per CTA
constexpr int kKeys = 128;        // keys of a tile
constexpr int kStages = 2;        // K tiles, and V tiles, in shared memory
constexpr int kInfo = 4;          // key tiles whose page info is kept
constexpr int kSoftmaxWarps = 8;
// Loader warps (8-bit pages go through registers, and take one more), then the
// warp that issues the products.  Either way a thread can have 168 registers.
constexpr int load_warps(bool bf16) { return bf16 ? 2 : 3; }
constexpr int cta_threads(bool bf16) { return (kSoftmaxWarps + load_warps(bf16) + 1) * 32; }
constexpr uint32_t kTmemColumns = 512;  // S of both tiles, then O of both
// The weights of a tile go to the product in two parts, the first of
// kFirstKeys keys, so that it begins before the last weight is there (32, 64
// and 96 keys measured within 1%).
constexpr int kFirstKeys = 96;
constexpr int kRawBytes = 8192;   // of codes in flight, per loader warp (8-bit pages)
constexpr float kLazyRescale = 8.f;     // log2 of the largest weight
constexpr int kMaxSplits = 32;          // partials per row (merge_slots)
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr unsigned long long kDrainNs = 20000000ull;  // after a wait that ran out
// The partials start behind the decode's merge counts, which have to stay 0
// where calls of both share a workspace.
constexpr size_t kBodyOffset = PA_WORKSPACE_HEADER_BYTES + PA_WORKSPACE_MERGE_COUNT_BYTES;

enum Format : int { kFmtBf16 = 0, kFmtE4m3 = 1, kFmtE4m3Block = 2, kFmtInt8Block = 3 };

struct PrefillParams {
    __nv_bfloat16* out;          // [T, Hq, D]
    const uint16_t* q;           // bf16 bits [T, Hq, D]
    const uint8_t* kc;
    const uint8_t* vc;
    const float* k_scale;
    const float* v_scale;
    const int32_t* bt;           // [S, max_blocks]
    const int32_t* seq_lens;     // [S]
    const int32_t* query_start;  // [S + 1]
    float* ws_o;                 // [T, Hq, P, D] (P > 1)
    float* ws_m;                 // [T, Hq, P]
    float* ws_l;
    uint32_t* status;
    long long num_blocks;
    int T, S, Hq, Hk, G, max_blocks;
    int tokens_per_tile;   // 128 / G
    int P, tiles_per_part;
    int units;             // token groups (an upper bound)
    float scale_log2;      // |scale| log2(e)
    int negate;            // scale < 0: the queries are negated
    int v_pages;           // num_blocks * Hk: pages of the tensor maps
};

// Tensor maps of the bf16 caches: K as rows of one page each, V as pages of D
// rows of B tokens.
struct PageMaps {
    CUtensorMap k, v;
};

template <int D, int B, bool BF16>
struct Layout {  // shared memory, in bytes
    static constexpr int kTile = kKeys * D * 2;  // a K tile
    // A Q tile: 8 head dims of every row, 16 bytes each.  The step between these
    // columns is off the banks' period, so that lanes along a row store at once.
    static constexpr int kQStep = kRows * 16 + 16;
    static constexpr int kQTile = D / 8 * kQStep;
    // A V tile of bf16 pages: the pages as the TMA unit lays them down, rows of
    // B tokens with the 32- or 64-byte swizzle.  Of 8-bit pages: 8 keys of every
    // head dim, 16 bytes each, a step apart that is off the 128-byte period of
    // the banks by as much as makes a warp's stores -- rows of V, 16-byte pieces
    // fastest -- hit every bank once.
    static constexpr int kVStep = D * 16 + (B == 16 ? 64 : 32);
    static constexpr int kVTile = BF16 ? kTile : kKeys / 8 * kVStep;
    static constexpr int q = 0;
    static constexpr int k = (q + kTiles * kQTile + 1023) / 1024 * 1024;
    static constexpr int v = k + kStages * kTile;
    static constexpr int info = v + kStages * kVTile;         // per key tile: 32 floats
    static constexpr int q_mul = info + kInfo * 32 * 4;       // per row: float (8-bit pages)
    static constexpr int bad = q_mul + kTiles * kRows * 4;    // 8 words: see scrub
    static constexpr int bars = bad + 32;
    static constexpr int n_bars = 5 * kStages + 3 * kTiles + kInfo + 2;
    static constexpr int tmem_slot = bars + 8 * n_bars;
    // 8-bit pages as they come from the cache, kRawBytes for each loader warp.
    static constexpr int raw = (tmem_slot + 16 + 127) / 128 * 128;
    static constexpr int total = BF16 ? raw : raw + load_warps(BF16) * kRawBytes;
};

// Page info of a key tile: word 0, a bit per page with a legal block id; word 1,
// whether its pages are wide (see kNarrow); from word 8, the pages' K scales;
// from word 16, log2 of their V scales (block formats; 8 pages at most).
constexpr int kInfoK = 8, kInfoV = 16;

constexpr float kTinyFactor = 1.17549435e-38f;  // of a logit: what is below counts as it

template <int D, int B, int FMT>
__global__ void __launch_bounds__(cta_threads(FMT == kFmtBf16), 1)
    pa_prefill_kernel(const PrefillParams p, const __grid_constant__ PageMaps maps) {
    using L = Layout<D, B, FMT == kFmtBf16>;
    constexpr bool BF16 = FMT == kFmtBf16;
    constexpr bool BLOCK = FMT == kFmtE4m3Block || FMT == kFmtInt8Block;
    constexpr bool INT8 = FMT == kFmtInt8Block;
    constexpr int ELEM = BF16 ? 2 : 1;
    constexpr int PAGE = D * B * ELEM;
    constexpr int NPG = kKeys / B;  // pages of a key tile
    constexpr int kLoadWarps = load_warps(BF16), kMmaWarp = kSoftmaxWarps + kLoadWarps;
    extern __shared__ __align__(1024) uint8_t prefill_smem[];
    uint8_t* const smem = prefill_smem;
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---------------- this CTA's work; the last units (the longest rows of a
    // sequence) come first
    const unsigned per_unit = static_cast<unsigned>(p.Hk) * p.P;
    const int u = p.units - 1 - static_cast<int>(blockIdx.x / per_unit);
    const int rest = static_cast<int>(blockIdx.x % per_unit);
    const int kvh = rest % p.Hk, part = rest / p.Hk;
    const int tokens_per_cta = kTiles * p.tokens_per_tile;
    auto first_unit = [&](int s) {
        return max(0, min(__ldg(p.query_start + s), p.T)) / tokens_per_cta + s;
    };
    // (Unit u looks after entry u: a bad one may leave its sequence no unit.)
    if (rest == 0 && threadIdx.x == 0 && u < p.S && bad_rows(p.query_start, u, p.T))
        atomicOr(p.status, PA_DEV_BAD_QUERY_START);
    const int s = find_sequence(p.S, lane, first_unit, u);
    if (s < 0 || bad_rows(p.query_start, s, p.T)) return;
    const int a = __ldg(p.query_start + s), n = __ldg(p.query_start + s + 1) - a;
    const int tok0 = (u - first_unit(s)) * tokens_per_cta;  // first query token of the CTA
    if (tok0 < 0 || tok0 >= n) return;
    const int T = __ldg(p.seq_lens + s);
    if (T < n || T > static_cast<long long>(p.max_blocks) * B) {
        if (threadIdx.x == 0) atomicOr(p.status, PA_DEV_SEQ_LEN_OUT_OF_RANGE);
        return;
    }
    // Query token i sees the keys [0, T - n + i].  Key tiles of this partition,
    // for each row tile: [j0, j0 + count(t)).
    // (Sums with a length that reaches 2^31 - 1 stay below it.)
    const int seen0 = T - n + tok0 + 1;                                  // by the first row
    auto seen_by = [&](int i) { return seen0 + min(T - seen0, i); };     // by i tokens later
    const int seen_end = seen_by(tokens_per_cta - 1);                    // by the last
    const int pages = (seen_end - 1) / B + 1;
    const int j0 = part * p.tiles_per_part;
    auto count = [&](int t) {
        if (tok0 + t * p.tokens_per_tile >= n) return 0;
        const int seen = seen_by((t + 1) * p.tokens_per_tile - 1);
        // (The last partition takes all that is left, also behind max_seq_len.)
        const int tiles = (seen - 1) / kKeys + 1 - j0;
        return max(0, part == p.P - 1 ? tiles : min(tiles, p.tiles_per_part));
    };
    const int n0 = count(0), n1 = count(1);
    const int steps = max(n0, n1);

    const uint32_t sbase = smem_addr(smem);
    const uint32_t bars = sbase + L::bars;
    const uint32_t k_full = bars, k_empty = k_full + 8 * kStages, v_full = k_empty + 8 * kStages,
                   v_empty = v_full + 8 * kStages, s_ready = v_empty + 8 * kStages,
                   p_first = s_ready + 8 * kTiles, p_ready = p_first + 8 * kTiles,
                   i_full = p_ready + 8 * kTiles,
                   q_full = i_full + 8 * kInfo, v_land = q_full + 8,
                   drained = v_land + 8 * kStages;
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::bad);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full + 8 * i, BF16 ? 1 : 32 * kLoadWarps);
            mbar_init(v_full + 8 * i, BF16 ? 2 : 32 * kLoadWarps);
            mbar_init(v_land + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(s_ready + 8 * t, 1);
            mbar_init(p_first + 8 * t, kRows);
            mbar_init(p_ready + 8 * t, kRows);
        }
        for (int i = 0; i < kInfo; ++i) mbar_init(i_full + 8 * i, 1);
        mbar_init(q_full, kTiles * kRows);
        mbar_init(drained, 1);
        fence_mbar_init();
        for (int i = 0; i < 8; ++i) bad[i] = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(sbase + L::tmem_slot, kTmemColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::tmem_slot);
    bool lost = false;  // a wait ran out: leave every loop
    auto wait_one = [&](uint32_t bar, int phase) {
        if (!lost && !mbar_wait_bounded(bar, static_cast<uint32_t>(phase) & 1u, kWaitNs))
            lost = true;
        return !lost;
    };
    auto wait = [&](uint32_t bar, int phase) {  // with the whole warp's verdict
        lost = !__all_sync(kFull, wait_one(bar, phase));
        return !lost;
    };

    if (warp >= kSoftmaxWarps && warp < kMmaWarp) {
        // ================================================ loaders
        const int32_t* btrow = p.bt + static_cast<long long>(s) * p.max_blocks;
        const size_t block_stride = static_cast<size_t>(p.Hk) * PAGE;
        const size_t head_off = static_cast<size_t>(kvh) * PAGE;
        // Lane l < NPG: the id of page l of key tile j (-1: none, or not legal).
        auto page_id = [&](int j) {
            const int pg = (j0 + j) * NPG + lane;
            if (lane >= NPG || j >= steps || pg >= pages) return -1;
            const int id = __ldg(btrow + pg);
            if (id >= 0 && id < p.num_blocks) return id;
            atomicOr(p.status, PA_DEV_BAD_BLOCK_ID);
            return -1;
        };
        int next = page_id(0);
        auto widen = [&](uint32_t w, uint32_t& lo, uint32_t& hi) {
            lo = INT8 ? int8_lo_pair(w) : e4m3_lo_pair(w);
            hi = INT8 ? int8_hi_pair(w) : e4m3_hi_pair(w);
        };
        auto put16 = [&](uint32_t lo_at, uint32_t hi_at, const uint4& w) {  // 16 codes
            uint4 x, y;
            widen(w.x, x.x, x.y);
            widen(w.y, x.z, x.w);
            widen(w.z, y.x, y.y);
            widen(w.w, y.z, y.w);
            sts128(lo_at, x);
            sts128(hi_at, y);
        };
        // Values of keys that not every row sees, or none: non-finite ones are
        // kept out of the product (0 times NaN is NaN), and noted where some row
        // does see them.  For a 16-byte piece of one head dim from key `key` on:
        // which of its elements those keys are (their top bits), ...
        constexpr int kBits = ELEM * 8, kPer = 32 / kBits;
        struct Late {
            uint32_t top[4];
        };
        auto late_keys = [&](int key) {
            Late m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m.top[i] = 0;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (key + i * kPer + e >= seen0) m.top[i] |= 1u << ((e + 1) * kBits - 1);
            }
            return m;
        };
        // ... which of them are not finite (an exponent, or a code, of all ones
        // carries into the top bit), ...
        auto odd_of = [&](uint32_t x, uint32_t top) -> uint32_t {
            if constexpr (BF16) return ((x & 0x7f807f80u) + 0x00800080u) & top;
            if constexpr (INT8) return 0u;
            return ((x & 0x7f7f7f7fu) + 0x01010101u) & top;
        };
        auto odd_any = [&](const uint4& w, const Late& m) -> uint32_t {
            return odd_of(w.x, m.top[0]) | odd_of(w.y, m.top[1]) | odd_of(w.z, m.top[2]) |
                   odd_of(w.w, m.top[3]);
        };
        // ... and the piece without those.
        auto scrub = [&](uint4& w, const Late& m, int key) {
            uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 1
            for (int e = 0; e < 4 * kPer; ++e) {
                const int i = e / kPer, k = key + e - seen0;
                const uint32_t top = i == 0 ? m.top[0] : i == 1 ? m.top[1] : i == 2 ? m.top[2]
                                                                                    : m.top[3];
                const uint32_t v = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3];
                if (!((odd_of(v, top) >> ((e % kPer + 1) * kBits - 1)) & 1u)) continue;
                const uint32_t keep = ~(((1u << kBits) - 1u) << (e % kPer * kBits));
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] &= u == i ? keep : kFull;
                if (key + e < seen_end) atomicOr(bad + (k >> 5), 1u << (k & 31));
            }
            w = make_uint4(x[0], x[1], x[2], x[3]);
        };
        // Block scales of a tile's pages (the first loader warp's business).
        [[maybe_unused]] ScaleRange range;
        auto scales_of = [&](int ids) {
            PageScales ps = {};
            if constexpr (BLOCK) {
                if (warp == kSoftmaxWarps)
                    ps = load_page_scales(p.k_scale, p.v_scale, ids, -1, p.num_blocks, p.Hk, kvh);
            }
            return ps;
        };
        auto page_info = [&](int j, int ids, [[maybe_unused]] PageScales ps) {
            // (kInfo tiles deep: the slot's last user is done once K of tile
            // j - 2 has been released.)
            float* info = reinterpret_cast<float*>(smem + L::info) + (j % kInfo) * 32;
            const unsigned legal = __ballot_sync(kFull, lane < NPG && ids >= 0);
            if (lane == 0) reinterpret_cast<uint32_t*>(info)[0] = legal;
            if constexpr (BLOCK) {
                finish_page_scales(ps, range);
                if (lane == 0) reinterpret_cast<uint32_t*>(info)[1] = range.wide();
                if (lane < NPG) {
                    info[kInfoK + lane] = ps.k[0];
                    info[kInfoV + lane] = ps.v_log2[0];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(i_full + 8 * (j % kInfo));
        };
        // Tiles with keys that some row does not see.
        auto edge = [&](int j) { return j0 + j >= seen0 / kKeys; };
        if constexpr (BF16) {
            // K: a gather of four pages brings one 16-byte column of each (B
            // tokens of 8 head dims) to consecutive addresses of the tile's
            // column; each warp takes half the columns.  V: a page at a time,
            // swizzled as the product wants its rows of B tokens.  Few, large
            // requests matter: one costs its warp about 60 cycles, and loads
            // through registers would take the issue slots and the memory pipe
            // that the softmax warps read TMEM with.
            constexpr int CG = D / 8;  // columns of a K page
            const bool first = warp == kSoftmaxWarps;
            int landed[kStages] = {};
            for (int j = 0; j < steps; ++j) {
                const int st = j % kStages;
                const int ids = next;
                next = page_id(j + 1);
                if (!wait(k_empty + 8 * st, j / kStages + 1)) break;
                if (first) {
                    page_info(j, ids, PageScales{});
                    if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * st, L::kTile);
                    __syncwarp();
                }
                const uint32_t kdst = sbase + L::k + st * L::kTile;
#pragma unroll
                for (int g = 0; g < NPG / 4; ++g) {
                    int page[4];  // (an illegal page's keys are masked: any page will do)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int id = __shfl_sync(kFull, ids, 4 * g + i);
                        page[i] = (id < 0 ? 0 : id) * p.Hk + kvh;
                    }
                    if (lane < CG / 2) {
                        const int c = lane + (first ? 0 : CG / 2);
                        tma_gather4(kdst + c * (kKeys * 16) + g * (4 * B * 16), &maps.k, c * B * 8,
                                    page[0], page[1], page[2], page[3], k_full + 8 * st);
                    }
                    __syncwarp();
                }
                if (!wait(v_empty + 8 * st, j / kStages + 1)) break;
                const bool late = edge(j);
                if (first) {
                    const uint32_t bar = (late ? v_land : v_full) + 8 * st;
                    if (lane == 0) mbar_arrive_expect_tx(bar, NPG * PAGE);
                    __syncwarp();
                    if (lane < NPG)  // (an illegal page is outside the map: zeros)
                        tma_load_3d(sbase + L::v + st * L::kVTile + lane * PAGE, &maps.v, 0, 0,
                                    ids >= 0 ? ids * p.Hk + kvh : p.v_pages, bar);
                } else if (!late && lane == 0) {
                    mbar_arrive(v_full + 8 * st);
                }
                if (late) {
                    // Each warp scrubs half the pages that some row does not see.
                    if (!wait(v_land + 8 * st, landed[st]++)) break;
                    constexpr int PC = B / 8;  // 16-byte pieces of a row, a lane's always the same
                    constexpr int kPieces = D * PC / 32;  // of a page, per lane
                    constexpr int U = kPieces < 8 ? kPieces : 8;
                    static_assert(kPieces % U == 0, "a page's pieces, no more");
#pragma unroll 1
                    for (int pg = first ? 0 : 1; pg < NPG; pg += 2) {
                        const int key = (j0 + j) * kKeys + pg * B + lane % PC * 8;
                        const int page_key = (j0 + j) * kKeys + pg * B;
                        if (page_key + B <= seen0 || page_key >= seen_end) continue;
                        const Late m = late_keys(key);
                        const uint32_t page = sbase + L::v + st * L::kVTile + pg * PAGE;
#pragma unroll 1
                        for (int i0 = lane; i0 < D * PC; i0 += 32 * U) {
                            uint4 w[U];
                            uint32_t at[U];
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                // The swizzle: bit 4 of the offset by bit 7 (rows
                                // of 32 bytes), or bits 4, 5 by 7, 8 (of 64).
                                const uint32_t off = (i0 + 32 * u) * 16;
                                at[u] = page + (off ^ ((off >> 3) & (B == 16 ? 0x10u : 0x30u)));
                                w[u] = lds128(at[u]);
                            }
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                if (odd_any(w[u], m)) {
                                    scrub(w[u], m, key);
                                    sts128(at[u], w[u]);
                                }
                            }
                        }
                    }
                    fence_smem_to_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_full + 8 * st);
                }
            }
            if (lost) {
                // Copies in flight land before the CTA's memory is another's.
                for (int i = 0; i < kStages; ++i)
                    for (int ph = 0; ph < 2; ++ph) {
                        (void)mbar_wait_bounded(k_full + 8 * i, ph, kDrainNs);
                        (void)mbar_wait_bounded(v_full + 8 * i, ph, kDrainNs);
                        (void)mbar_wait_bounded(v_land + 8 * i, ph, kDrainNs);
                    }
            }
        } else {
            // ---- 8-bit pages.  Those of all tiles, K's and V's of each tile in
            // turn, are dealt to the loader warps one by one.  A page is 16-byte
            // pieces, of K (column group, token), of V (head dim, tokens), taken by
            // consecutive lanes; a lane's next piece of the page is a fixed step
            // further at both ends.  Pages go through a ring of slots: asynchronous
            // copies bring some while the one before is widened, and a lane reads
            // what it copied itself.  The loop is kept short: unrolled over a tile
            // it missed the instruction cache, and a tile took 2.5 times as long.
            constexpr int NQ = PAGE / 512;  // pieces of a page per lane
            constexpr int VR = B / 16;      // pieces of a V row
            constexpr int kSlots = kRawBytes / PAGE < NPG / 2 ? kRawBytes / PAGE : NPG / 2;
            static_assert(NQ * 512 == PAGE && 32 % B == 0, "");
            static_assert(kSlots * kLoadWarps < 2 * NPG, "copies run ahead into the next tile");
            const int me = warp - kSoftmaxWarps;
            const uint32_t ring = sbase + L::raw + me * kRawBytes + lane * 16;
            // Page i of a tile (K's, then V's) to a slot; ids are the tile's.
            auto copy = [&](int ids, int i, uint32_t slot) {
                const int id = __shfl_sync(kFull, ids, i % NPG);
                const uint8_t* src = (i < NPG ? p.kc : p.vc) + (id < 0 ? 0 : id) * block_stride +
                                     head_off + lane * 16;
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    cp_async16(slot + q * 512, src + q * 512, id < 0 ? 0u : 16u);
                cp_async_commit();
            };
            int ids = next;
            PageScales scales = scales_of(ids);
            next = page_id(1);
            for (int i = 0; i < kSlots; ++i) copy(ids, me + i * kLoadWarps, ring + i * PAGE);
            int slot = 0, i = me;  // the next page of this warp, within tile j
            for (int j = 0; j < steps && !lost; ++j) {
                const int st = j % kStages;
                const PageScales now = scales;
                scales = scales_of(next);
                for (int v = 0; v < 2; ++v) {  // K's pages, then V's
                    if (!wait((v ? v_empty : k_empty) + 8 * st, j / kStages + 1)) break;
                    if (!v && me == 0) page_info(j, ids, now);
                    // K: column group lane / B, token lane % B.  V: head dim lane /
                    // VR, part lane % VR.  A piece becomes two 16-byte columns.
                    const uint32_t column = v ? L::kVStep : kKeys * 16;
                    const uint32_t dst =
                        v ? sbase + L::v + st * L::kVTile + 2 * (lane % VR) * column + lane / VR * 16
                          : sbase + L::k + st * L::kTile + 2 * (lane / B) * column + lane % B * 16;
                    const uint32_t page_step = v ? B / 8 * L::kVStep : B * 16;
                    const uint32_t piece_step = v ? 32 / VR * 16 : 2 * (32 / B) * column;
                    const bool late = !INT8 && v && edge(j);
#pragma unroll 1
                    for (; i < (v + 1) * NPG; i += kLoadWarps) {
                        cp_async_wait<kSlots - 1>();
                        const uint32_t raw = ring + slot * PAGE;
                        const int pg = i % NPG;
                        uint4 w[NQ];
#pragma unroll
                        for (int q = 0; q < NQ; ++q) w[q] = lds128(raw + q * 512);
                        if (late) {
                            const int key = (j0 + j) * kKeys + pg * B + lane % VR * 16;
                            const Late m = late_keys(key);
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                if (odd_any(w[q], m)) scrub(w[q], m, key);
                        }
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const uint32_t at = dst + pg * page_step + q * piece_step;
                            put16(at, at + column, w[q]);
                        }
                        // The slot's next page: of this tile, or of the next one
                        // (none behind the last tile: zeros).
                        const int ahead = i + kSlots * kLoadWarps;
                        copy(ahead < 2 * NPG ? ids : next, ahead % (2 * NPG), raw);
                        slot = slot + 1 == kSlots ? 0 : slot + 1;
                    }
                    fence_smem_to_async();
                    mbar_arrive((v ? v_full : k_full) + 8 * st);
                }
                i -= 2 * NPG;
                ids = next;
                next = page_id(j + 2);
            }
            cp_async_wait<0>();
        }
    } else if (warp == kMmaWarp) {
        // ================================================ products
        if (lane == 0) {
            constexpr uint32_t kQk = mma_shape(BF16, kRows, kKeys);
            constexpr uint32_t kPv = mma_shape(BF16, kRows, D);
            auto scores = [&](int t, int st) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(tmem + t * kKeys,
                           smem_operand(sbase + L::q + t * L::kQTile + k * (2 * L::kQStep),
                                        L::kQStep),
                           smem_operand(sbase + L::k + st * L::kTile + k * (2 * kKeys * 16),
                                        kKeys * 16),
                           kQk, k > 0);
            };
            auto values = [&](int t, int st, int k0, int k1, bool add) {
#pragma unroll
                for (int k = k0; k < k1; ++k)
                {
                    const uint32_t v = sbase + L::v + st * L::kVTile;
                    const uint64_t operand =
                        !BF16     ? smem_operand(v + k * (2 * L::kVStep), L::kVStep)
                        : B == 16 ? smem_operand_swizzled<32>(v + k * PAGE)
                                  : smem_operand_swizzled<64>(v + k / 2 * PAGE + k % 2 * 32);
                    mma_ts(tmem + kTiles * kKeys + t * 128, tmem + t * kKeys + 8 * k, operand, kPv,
                           add || k > 0);
                }
            };
            if (steps > 0 && wait_one(q_full, 0) && wait_one(k_full, 0)) {
                tmem_fence_after();
                if (n0 > 0) {
                    scores(0, 0);
                    mma_commit(s_ready);
                }
                if (n1 > 0) {
                    scores(1, 0);
                    mma_commit(s_ready + 8);
                }
                mma_commit(k_empty);
            }
            for (int j = 0; j < steps && !lost; ++j) {
                const int st = j % kStages, nx = (j + 1) % kStages;
                if (!wait_one(v_full + 8 * st, j / kStages)) break;
                for (int t = 0; t < kTiles; ++t) {
                    const int nt = t ? n1 : n0;
                    if (j >= nt) continue;
                    if (!wait_one(p_first + 8 * t, j)) break;
                    tmem_fence_after();
                    values(t, st, 0, kFirstKeys / 16, j > 0);
                    if (!wait_one(p_ready + 8 * t, j)) break;
                    tmem_fence_after();
                    values(t, st, kFirstKeys / 16, kKeys / 16, true);
                    if (j + 1 < nt) {
                        if (!wait_one(k_full + 8 * nx, (j + 1) / kStages)) break;
                        tmem_fence_after();
                        scores(t, nx);
                    }
                    // S of the next tile, or O, is there (and P consumed).
                    mma_commit(s_ready + 8 * t);
                }
                if (lost) break;
                mma_commit(v_empty + 8 * st);
                if (j + 1 < steps) mma_commit(k_empty + 8 * nx);
            }
            if (lost) {
                // The products in flight still write TMEM: wait for them (bounded).
                mma_commit(drained);
                (void)mbar_wait_bounded(drained, 0u, kWaitNs);
            }
        }
        __syncwarp();
    } else {
        // ================================================ softmax, one row per thread
        const int t = warp / 4;
        const int r = threadIdx.x - t * kRows;
        const int nt = t ? n1 : n0;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const uint32_t s_at = tmem + lanes + t * kKeys;
        const uint32_t o_at = tmem + lanes + kTiles * kKeys + t * 128;
        const int qt = tok0 + t * p.tokens_per_tile + r / p.G;
        const bool row_ok = r < p.tokens_per_tile * p.G && qt < n;
        // Keys of this row; a row of no query token counts as seeing all, so that
        // it does not make its warp mask (its results go nowhere).
        const int seen = row_ok ? T - n + qt + 1 : 0x7fffffff;
        float mul = p.scale_log2, out_mul = 1.f;
        const uint32_t stage = sbase + L::q + t * L::kQTile + warp % 4 * (32 * D * 2);
        const int head = kvh * p.G + r % p.G;
        const long long row = (static_cast<long long>(a) + qt) * p.Hq + head;
        {
            // The warp's 32 query rows, 16 bytes a lane, into the tile's operand.
            // f16 operands (8-bit caches) are scaled per row by a power of two,
            // which puts the largest |q| in [2^14, 2^15).
            constexpr int LR = D / 8, RI = 32 / LR;  // lanes per row, rows at a time
            // (Factors of a logit stay above 0; a sign goes to the query.)
            bool negate = p.negate != 0;
            if constexpr (FMT == kFmtE4m3) negate ^= __ldg(p.k_scale) < 0.f;
            const uint32_t flip = negate ? 0x80008000u : 0u;
            float* muls = reinterpret_cast<float*>(smem + L::q_mul) + t * kRows + warp % 4 * 32;
            constexpr int QB = 8;  // loads in flight
#pragma unroll 1
            for (int i0 = 0; i0 < LR; i0 += QB) {
                uint4 w[QB];
#pragma unroll
                for (int u = 0; u < QB; ++u) {
                    const long long from =
                        __shfl_sync(kFull, row_ok ? row : -1ll, (i0 + u) * RI + lane / LR);
                    w[u] = make_uint4(0, 0, 0, 0);
                    if (from >= 0)
                        w[u] = __ldg(reinterpret_cast<const uint4*>(p.q + from * D) + lane % LR);
                }
#pragma unroll
                for (int u = 0; u < QB; ++u) {
                    const int of = (i0 + u) * RI + lane / LR;  // row of the warp
                    uint32_t x[4] = {w[u].x ^ flip, w[u].y ^ flip, w[u].z ^ flip, w[u].w ^ flip};
                    if constexpr (!BF16) {
                        float amax = 0.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
#pragma unroll
                        for (int o = LR / 2; o > 0; o >>= 1)
                            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                        int e = 0;  // amax in [2^(14 + e), 2^(15 + e))
                        if (amax > 0.f && amax < INFINITY)
                            e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
                        e = max(-110, min(113, e));
                        const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                        if (lane % LR == 0)
                            muls[of] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = pack_f16x2(bf16_lo(x[k]) * up, bf16_hi(x[k]) * up);
                    }
                    sts128(sbase + L::q + t * L::kQTile + lane % LR * L::kQStep +
                               (warp % 4 * 32 + of) * 16,
                           make_uint4(x[0], x[1], x[2], x[3]));
                }
            }
            fence_smem_to_async();
            mbar_arrive(q_full);
            if constexpr (!BF16) {
                __syncwarp();
                mul *= muls[lane];
                if constexpr (!BLOCK) {
                    mul *= fabsf(__ldg(p.k_scale));
                    out_mul = __ldg(p.v_scale);
                }
            }
            // (Above 0, so that the -inf of a hidden key stays one.)
            mul = fmaxf(mul, kTinyFactor);
        }
        // A warp without a row of a query token has nothing to weigh: whatever its
        // rows' products are, they go nowhere.
        const bool idle = !__any_sync(kFull, row_ok);
        float m = -INFINITY, l = 0.f;
        int j = 0;
        // The tiles from j on, up to the first wide one (see kNarrow) unless WIDE
        // (the unusual form has a loop of its own, out of the usual one's registers).
        auto weigh = [&](auto form) {
            constexpr bool WIDE = decltype(form)::value;
            for (; j < nt && !lost; ++j) {
                if (!wait(s_ready + 8 * t, j)) break;
                if (!wait(i_full + 8 * (j % kInfo), j / kInfo)) break;
                tmem_fence_after();
                if (idle) {
                    mbar_arrive(p_first + 8 * t);
                    mbar_arrive(p_ready + 8 * t);
                    continue;
                }
                const float* info =
                    reinterpret_cast<const float*>(smem + L::info) + (j % kInfo) * 32;
                const uint32_t legal = reinterpret_cast<const uint32_t*>(info)[0];
                if (BLOCK && !WIDE && reinterpret_cast<const uint32_t*>(info)[1]) return;
                const int left = seen - (j0 + j) * kKeys;  // keys of this tile that the row sees
                const bool masked = __any_sync(kFull, left < kKeys) || legal != (1u << NPG) - 1u;
                // ---- the tile's scores, and their maximum (of x + log2 vs with
                // block scales)
                float x[kKeys], mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_at + c, x + c);
                tmem_wait_ld(x);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < kKeys; ++c)
                        if (c >= left || !((legal >> (c / B)) & 1u)) x[c] = -INFINITY;
                }
                if constexpr (BLOCK) {
#pragma unroll
                    for (int pg = 0; pg < NPG; ++pg) {
                        float y = x[pg * B];
#pragma unroll
                        for (int c = 1; c < B; ++c) y = fmaxf(y, x[pg * B + c]);
                        const float f = fmaxf(mul * info[kInfoK + pg], kTinyFactor);
                        mx = fmaxf(mx, fmaf(y, f, info[kInfoV + pg]));
                    }
                } else {
                    float y[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < kKeys; ++c) y[c % 4] = fmaxf(y[c % 4], x[c]);
                    mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * mul;
                }
                // ---- O in the units of a new maximum, only when it grew by a lot
                const bool grow = mx > m + kLazyRescale || (m == -INFINITY && mx > -INFINITY);
                if (__any_sync(kFull, grow)) {
                    const float to = grow ? mx : m;
                    const float fall = to == -INFINITY ? 0.f : m - to;
                    const float alpha = fast_exp2(fall);
                    m = to;
                    if constexpr (WIDE) {  // (alpha itself may vanish)
                        const float half = fast_exp2(0.5f * fall);
                        l = l * half * half;
                    } else {
                        l *= alpha;
                    }
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_ld32(o_at + c, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            tmem_st32(o_at + c, o);
                        }
                    }
                }
                const float m_use = m == -INFINITY ? 0.f : m;
                // ---- weights back to TMEM over the scores; their sum
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kKeys; c += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int g = 0; g < 32; g += 16) {
                        const int pg = (c + g) / B;
                        float f = mul, add = -m_use;
                        if constexpr (BLOCK) {
                            f = fmaxf(mul * info[kInfoK + pg], kTinyFactor);
                            add = info[kInfoV + pg] - m_use;
                        }
                        const float2 f2 = make_float2(f, f), add2 = make_float2(add, add);
                        [[maybe_unused]] const float2 plain2 = make_float2(-m_use, -m_use);
                        float2 part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 y =
                                __ffma2_rn(make_float2(x[c + g + i], x[c + g + i + 1]), f2, add2);
                            const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            if constexpr (WIDE) {  // (see WarpAttn::page)
                                const float2 z = __ffma2_rn(
                                    make_float2(x[c + g + i], x[c + g + i + 1]), f2, plain2);
                                sum = __fadd2_rn(sum, make_float2(fast_exp2(z.x), fast_exp2(z.y)));
                            } else {
                                part = __fadd2_rn(part, e);
                            }
                            w[(g + i) / 2] = BF16 ? pack_bf16x2(e.x, e.y) : pack_f16x2(e.x, e.y);
                        }
                        if constexpr (!BLOCK) {
                            sum = __fadd2_rn(sum, part);
                        } else if constexpr (!WIDE) {
                            const float back = fast_exp2(-info[kInfoV + pg]);
                            sum = __ffma2_rn(part, make_float2(back, back), sum);
                        }
                    }
                    tmem_st16(s_at + c / 2, w);
                    if (c + 32 == kFirstKeys || c + 32 == kKeys) {
                        tmem_wait_st();
                        tmem_fence_before();
                        mbar_arrive((c + 32 == kKeys ? p_ready : p_first) + 8 * t);
                    }
                }
                l += sum.x + sum.y;
            }
        };
        weigh(std::false_type{});
        if constexpr (BLOCK) {
            if (j < nt && !lost) weigh(std::true_type{});
        }
        // ---- the rows' results
        if (nt > 0) (void)wait(s_ready + 8 * t, nt);
        tmem_fence_after();
        const long long prow = row * p.P + part;
        const bool empty = nt == 0 || lost;
        if (BLOCK && l == INFINITY) l = 3.4e38f;  // (rows of V scales of 2^-100: o is near 0)
        if (p.P > 1 && row_ok) {
            // (A sum of NaN goes to the merge as an overriding row of NaNs.)
            const int e = BLOCK ? sum_exponent(l) : 0;
            p.ws_m[prow] = l != l ? 1e30f : e ? m + static_cast<float>(e) : m;
            p.ws_l[prow] = empty ? 0.f : l != l ? 1.f : e ? l * exp2_int(-e) : l;
        }
        const float inv = l > 0.f || l != l ? out_mul / l : 0.f;
        if (nt > 0 && !idle) {
            uint32_t any_bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) any_bad |= bad[i];
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(o_at + c, o);
                tmem_wait_ld(o);
                if (any_bad && row_ok) {
                    // Non-finite values of keys that not every row of the CTA
                    // sees were left out: they make the rows that do see them
                    // what they are.
                    for (int key = seen0; key < seen; ++key) {
                        if (!((bad[(key - seen0) >> 5] >> ((key - seen0) & 31)) & 1u)) continue;
                        const int jk = key / kKeys - j0;
                        if (jk < 0 || jk >= nt) continue;  // another partition's
                        const int id = __ldg(p.bt + static_cast<long long>(s) * p.max_blocks +
                                             key / B);
                        if (id < 0 || id >= p.num_blocks) continue;
                        const uint8_t* v = p.vc + static_cast<size_t>(id) * p.Hk * PAGE +
                                           static_cast<size_t>(kvh) * PAGE;
                        for (int i = 0; i < 32; ++i) {
                            const int at = (c + i) * B + key % B;
                            float y = 0.f;
                            if constexpr (BF16) {
                                y = __uint_as_float(static_cast<uint32_t>(
                                        __ldg(reinterpret_cast<const uint16_t*>(v) + at)) << 16);
                            } else if constexpr (!INT8) {
                                y = (__ldg(v + at) & 0x7f) == 0x7f ? NAN : 0.f;
                            }
                            if (!(fabsf(y) < INFINITY)) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if (k == i) o[k] += y;
                            }
                        }
                    }
                }
                if (p.P > 1) {
                    if (!row_ok || lost) continue;
                    float4* dst = reinterpret_cast<float4*>(p.ws_o + prow * D + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv,
                                             o[4 * i + 2] * inv, o[4 * i + 3] * inv);
                } else {
                    // Through the warp's rows of the (spent) Q tile, 16-byte
                    // pieces rotated by the row, so that whole rows are stored.
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sts128(stage + lane * (D * 2) + (((c / 8 + i) ^ lane) & (D / 8 - 1)) * 16,
                               make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv),
                                          pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                          pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                          pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv)));
                }
            }
            if (p.P == 1 && !lost) {
                __syncwarp();
                constexpr int LR = D / 8, RI = 32 / LR;  // lanes per row, rows at a time
#pragma unroll 1
                for (int i0 = 0; i0 < LR; i0 += 8) {
                    uint4 w[8];
                    long long to[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int from = (i0 + u) * RI + lane / LR;  // row of the warp
                        to[u] = __shfl_sync(kFull, row_ok ? row : -1ll, from);
                        w[u] = lds128(stage + from * (D * 2) + ((lane ^ from) & (LR - 1)) * 16);
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (to[u] >= 0)
                            *reinterpret_cast<uint4*>(p.out + to[u] * D + lane % LR * 8) = w[u];
                }
            }
        }
    }
    if (lost && lane == 0) atomicOr(p.status, PA_DEV_WAIT_TIMEOUT);
    tmem_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tmem_fence_after();
        tmem_free(tmem, kTmemColumns);
    }
}

// Merges the P partials of each (token, head) row, a warp per row.  Rows that
// no sequence owns, or whose sequence was skipped, are left alone.
template <int D>
__global__ void __launch_bounds__(kThreads)
    pa_prefill_merge_kernel(const PrefillParams p, int block_size) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (row >= static_cast<long long>(p.T) * p.Hq) return;
    merge_slots<D>(p.ws_o, p.ws_m, p.ws_l, p.out, row * p.P, p.P, lane, [&]() -> SlotRow {
        const int token = static_cast<int>(row / p.Hq);
        const int s = find_sequence(
            p.S, lane, [&](int i) { return max(0, min(__ldg(p.query_start + i), p.T)); }, token);
        if (s < 0 || bad_rows(p.query_start, s, p.T)) return {-1, row};
        const int a = __ldg(p.query_start + s), b = __ldg(p.query_start + s + 1);
        const int len = __ldg(p.seq_lens + s);
        const bool mine = token >= a && token < b && len >= b - a &&
                          len <= static_cast<long long>(p.max_blocks) * block_size;
        return {mine ? p.P : -1, row};
    });
}

// The maps of bf16 caches; false when the driver cannot make them.
bool encode_maps(PageMaps* maps, const PrefillParams& p, int D, int B) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<Encode>(f);
        (void)cudaGetLastError();
    });
    if (!encode) return false;
    const auto u64 = [](long long x) { return static_cast<cuuint64_t>(x); };
    const auto u32 = [](int x) { return static_cast<cuuint32_t>(x); };
    const cuuint64_t v_dims[3] = {u64(B), u64(D), u64(p.v_pages)};
    const cuuint64_t v_strides[2] = {u64(B * 2), u64(B * D * 2)};
    const cuuint32_t v_box[3] = {u32(B), u32(D), 1};
    const cuuint64_t k_dims[2] = {u64(B * D), u64(p.v_pages)};
    const cuuint64_t k_strides[1] = {u64(B * D * 2)};
    const cuuint32_t k_box[2] = {u32(B * 8), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(&maps->v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t*>(p.vc),
                  v_dims, v_strides, v_box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  B == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           encode(&maps->k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t*>(p.kc),
                  k_dims, k_strides, k_box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int B, int FMT>
cudaError_t launch_prefill(const PrefillParams& p, unsigned grid, cudaStream_t st) {
    static std::atomic<int> done[kMaxDevices];
    constexpr bool kBf16 = FMT == kFmtBf16;
    auto kern = pa_prefill_kernel<D, B, FMT>;
    cudaError_t e = ensure_smem(kern, done);
    if (e != cudaSuccess) return e;
    PageMaps maps;
    std::memset(&maps, 0, sizeof maps);
    if (kBf16 && !encode_maps(&maps, p, D, B)) return cudaErrorInvalidValue;
    return launch_pdl(kern, grid, cta_threads(kBf16), Layout<D, B, kBf16>::total, st, p, maps);
}

template <int D, int B>
cudaError_t launch_format(const PrefillParams& p, pa_kv_dtype t, unsigned grid, cudaStream_t st) {
    switch (t) {
        case PA_KV_BF16: return launch_prefill<D, B, kFmtBf16>(p, grid, st);
        case PA_KV_FP8_E4M3: return launch_prefill<D, B, kFmtE4m3>(p, grid, st);
        case PA_KV_FP8_E4M3_BLOCK: return launch_prefill<D, B, kFmtE4m3Block>(p, grid, st);
        default: return launch_prefill<D, B, kFmtInt8Block>(p, grid, st);
    }
}

struct PrefillPlan {
    long long units;
    int P, tiles_per_part;
    size_t workspace_bytes;
};

pa_status check_sizes(int num_tokens, int num_seqs, int num_heads,
                      int num_kv_heads, int head_size, int block_size, int max_seq_len,
                      pa_kv_dtype kv_dtype, const pa_options* opts) {
    if (num_tokens < 0 || num_seqs < 0)
        return fail(PA_ERR_INVALID_ARG, "%s", "num_tokens or num_seqs < 0");
    if (num_heads <= 0 || num_kv_heads <= 0)
        return fail(PA_ERR_INVALID_ARG, "%s", "num_heads and num_kv_heads must be > 0");
    if (num_heads % num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "%s", "num_heads must be a multiple of num_kv_heads");
    if (num_heads / num_kv_heads > 16)
        return fail(PA_ERR_UNSUPPORTED, "%s", "num_heads / num_kv_heads > 16");
    if (head_size != 64 && head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "%s", "head_size must be 64 or 128");
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "%s", "block_size must be 16 or 32");
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3 && !block_scales(kv_dtype))
        return fail(PA_ERR_UNSUPPORTED, "%s", "kv_dtype");
    if (max_seq_len < 0) return fail(PA_ERR_INVALID_ARG, "%s", "max_seq_len < 0");
    if (opts) {
        if (opts->num_sms < 0 || opts->partition_pages < 0)
            return fail(PA_ERR_INVALID_ARG, "%s", "opts->num_sms or opts->partition_pages < 0");
        if (opts->stages || opts->shared_prefix_blocks || opts->alibi_slopes ||
            opts->fp8_compute || opts->test_stall_copies || opts->schedule || opts->mha_cuda_cores)
            return fail(PA_ERR_UNSUPPORTED, "%s",
                        "prefill takes partition_pages and num_sms only");
    }
    return PA_OK;
}

// Sizes that check_sizes has passed.
pa_status plan_prefill(PrefillPlan* pl, int num_tokens, int num_seqs, int num_heads,
                       int num_kv_heads, int head_size, int block_size, int max_seq_len,
                       const pa_options* opts) {
    int sms = opts ? opts->num_sms : 0;
    if (sms == 0 && device_sms(&sms) != 0)
        return fail(PA_ERR_CUDA, "%s", "cannot query the SM count of the current device");
    const int tokens_per_cta = kTiles * (kRows / (num_heads / num_kv_heads));
    pl->units = num_tokens / tokens_per_cta + static_cast<long long>(num_seqs);
    const long long ctas = pl->units * num_kv_heads;
    const long long tiles = (static_cast<long long>(max_seq_len) + kKeys - 1) / kKeys;
    long long per;
    if (opts && opts->partition_pages > 0) {
        per = (static_cast<long long>(opts->partition_pages) * block_size + kKeys - 1) / kKeys;
    } else {
        // A batch of fewer than two waves of CTAs (one per SM) splits the keys
        // where that is expected to end sooner: P partitions take
        // ceil(ctas P / sms) waves of ceil(tiles / P) steps, and about six steps
        // more for a CTA's start and end, eight with the merge.  Measured with 3
        // sequences x 32 kv heads, 4 tokens over 12086 int8 keys: 96 CTAs 229 us,
        // 3 partitions 167 us.
        long long P = 1;
        long long best = 0;
        for (long long n = 1; n <= kMaxSplits; ++n) {
            if (n > 1 && (ctas >= 2 * static_cast<long long>(sms) || n > tiles / 2)) break;
            const long long waves = (ctas * n + sms - 1) / sms;
            const long long cost = waves * ((tiles + n - 1) / n + (n > 1 ? 8 : 6));
            if (n == 1 || cost < best) {
                best = cost;
                P = n;
            }
        }
        per = (tiles + P - 1) / P;
    }
    if (per < 1) per = 1;
    const long long P = tiles > 0 ? (tiles + per - 1) / per : 1;
    if (P > kMaxSplits)
        return fail(PA_ERR_INVALID_ARG, "%s",
                    "opts->partition_pages makes more than 32 partitions of max_seq_len");
    if (ctas * P > 0x7fffffffll ||
        static_cast<long long>(num_tokens) * num_heads > 0x7fffffffll)
        return fail(PA_ERR_INVALID_ARG, "%s", "too many tokens, sequences and heads for one call");
    pl->P = static_cast<int>(P);
    pl->tiles_per_part = static_cast<int>(per);
    pl->workspace_bytes = PA_WORKSPACE_HEADER_BYTES;
    if (P > 1) {
        pl->workspace_bytes = kBodyOffset + static_cast<size_t>(num_tokens) * num_heads * P *
                                                (static_cast<size_t>(head_size) + 2) *
                                                sizeof(float);
        pl->workspace_bytes = (pl->workspace_bytes + 255) & ~static_cast<size_t>(255);
    }
    return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_prefill_workspace_size(int num_tokens, int num_seqs, int num_heads,
                                            int num_kv_heads, int head_size, int block_size,
                                            int max_seq_len, pa_kv_dtype kv_dtype,
                                            const pa_options* opts) {
    pa::clear_detail();
    pa::PrefillPlan pl;
    if (pa::check_sizes(num_tokens, num_seqs, num_heads, num_kv_heads, head_size, block_size,
                        max_seq_len, kv_dtype, opts) != PA_OK ||
        pa::plan_prefill(&pl, num_tokens, num_seqs, num_heads, num_kv_heads, head_size, block_size,
                         max_seq_len, opts) != PA_OK)
        return 0;
    return pl.workspace_bytes;
}

extern "C" pa_status pa_prefill(void* out, const void* query, const void* key_cache,
                                const void* value_cache, int num_tokens, int num_seqs,
                                int num_heads, int num_kv_heads, int head_size, float scale,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* seq_lens, const int32_t* query_start,
                                int block_size, int max_seq_len, int64_t num_blocks,
                                pa_kv_dtype kv_dtype, const float* k_scale, const float* v_scale,
                                void* workspace, size_t workspace_bytes, void* stream,
                                const pa_options* opts) {
    using pa::aligned;
    using pa::fail;
    pa::clear_detail();
    pa_status status = pa::check_sizes(num_tokens, num_seqs, num_heads, num_kv_heads, head_size,
                                       block_size, max_seq_len, kv_dtype, opts);
    if (status != PA_OK) return status;
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "%s", "scale is not finite");
    if (max_blocks_per_seq < 1) return fail(PA_ERR_INVALID_ARG, "%s", "max_blocks_per_seq < 1");
    if (static_cast<long long>(max_seq_len) >
        static_cast<long long>(max_blocks_per_seq) * block_size)
        return fail(PA_ERR_INVALID_ARG, "%s", "max_seq_len > max_blocks_per_seq * block_size");
    if (num_blocks < 1 || num_blocks > 0x7ffffffeLL / num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "%s",
                    "num_blocks and num_blocks * num_kv_heads must be in [1, 2^31 - 1)");
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    const struct {
        const void* p;
        size_t a;
        const char* name;
    } ptrs[] = {{out, 16, "out"},
                {query, 16, "query"},
                {key_cache, 16, "key_cache"},
                {value_cache, 16, "value_cache"},
                {block_tables, 4, "block_tables"},
                {seq_lens, 4, "seq_lens"},
                {query_start, 4, "query_start"},
                {workspace, 16, "workspace"}};
    for (const auto& q : ptrs) {
        if (!q.p) return fail(PA_ERR_INVALID_ARG, "%s is NULL", q.name);
        if (!aligned(q.p, q.a)) return fail(PA_ERR_INVALID_ARG, "%s is misaligned", q.name);
    }
    if (kv_dtype != PA_KV_BF16) {
        if (!k_scale || !v_scale)
            return fail(PA_ERR_INVALID_ARG, "%s",
                        "k_scale and v_scale are required for an 8-bit cache");
        if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
            return fail(PA_ERR_INVALID_ARG, "%s", "k_scale / v_scale misaligned");
    }
    pa::PrefillPlan pl;
    status = pa::plan_prefill(&pl, num_tokens, num_seqs, num_heads, num_kv_heads, head_size,
                              block_size, max_seq_len, opts);
    if (status != PA_OK) return status;
    if (workspace_bytes < pl.workspace_bytes)
        return fail(PA_ERR_WORKSPACE_TOO_SMALL, "%s",
                    "workspace_bytes < pa_prefill_workspace_size");
    pa::PrefillParams p;
    std::memset(&p, 0, sizeof p);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.q = static_cast<const uint16_t*>(query);
    p.kc = static_cast<const uint8_t*>(key_cache);
    p.vc = static_cast<const uint8_t*>(value_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.bt = block_tables;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t rows = static_cast<size_t>(num_tokens) * num_heads * pl.P;
    p.ws_o = reinterpret_cast<float*>(ws + pa::kBodyOffset);
    p.ws_m = p.ws_o + rows * head_size;
    p.ws_l = p.ws_m + rows;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.num_blocks = num_blocks;
    p.T = num_tokens;
    p.S = num_seqs;
    p.Hq = num_heads;
    p.Hk = num_kv_heads;
    p.G = num_heads / num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.tokens_per_tile = pa::kRows / p.G;
    p.P = pl.P;
    p.tiles_per_part = pl.tiles_per_part;
    p.units = static_cast<int>(pl.units);
    p.scale_log2 = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
    p.negate = scale < 0.f;
    p.v_pages = static_cast<int>(num_blocks * num_kv_heads);
    const unsigned grid = static_cast<unsigned>(pl.units * num_kv_heads * pl.P);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_size == 64)
        e = block_size == 16 ? pa::launch_format<64, 16>(p, kv_dtype, grid, st)
                             : pa::launch_format<64, 32>(p, kv_dtype, grid, st);
    else
        e = block_size == 16 ? pa::launch_format<128, 16>(p, kv_dtype, grid, st)
                             : pa::launch_format<128, 32>(p, kv_dtype, grid, st);
    if (e == cudaSuccess && pl.P > 1) {
        const unsigned merge = static_cast<unsigned>(
            (static_cast<long long>(num_tokens) * num_heads + pa::kWarps - 1) / pa::kWarps);
        e = head_size == 64
                ? pa::launch_pdl(pa::pa_prefill_merge_kernel<64>, merge, pa::kThreads, 0, st, p,
                                 block_size)
                : pa::launch_pdl(pa::pa_prefill_merge_kernel<128>, merge, pa::kThreads, 0, st, p,
                                 block_size);
    }
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
    return PA_OK;
}
