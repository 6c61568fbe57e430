// Appending keys and values to the paged cache, with the position rotation on
// the way (pa_append_kv; see include/pagedattn.h for the contract).
//
// Work is cut into (block of a sequence's run, task) pairs, one warp each:
//   * task h < Hk: the new keys of kv head h in the block;
//   * task Hk + h: its new values;
//   * the tasks after them: the query rows of the block's new tokens.
// Warps share nothing and never wait for one another.  A warp takes a few rows
// at a time in short loops -- what hides the loads' latency is many warps of
// few registers, and straight-line code for a whole page of rows misses the
// instruction cache.  A block whose scale is to be found is read twice, the
// second time from L1; so are the rotation's table rows, by each head.
//
// Bound: every row is read once and every element written once, so DRAM for
// prompts; for single tokens the launch and two dependent rounds of loads
// (length -> block id and angles -> scale).
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>

#include "pa_launch.cuh"
#include "pa_query_start.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

constexpr int kAppendWarps = 4;
// CTAs per SM that the kernel's registers are held to (64 a thread: 32 warps).
// Measured on 16 prompts of 18301 tokens, 64/8 heads, bf16, and on 12271 tokens
// in chunks, 32/8 heads, int8 blocks of 32, before the loops prefetched: 6 CTAs
// 132 and 69 us, 8 CTAs 125 and 64, 10 CTAs (which spill) 123 and 67.  Now:
// 115-119 us, 6300-6500 GB/s of rows and caches, and 57-62 us.
constexpr int kAppendCtasPerSm = 8;
constexpr int kQueryRows = 32;  // rows of a query task (then: 16 131 us, 32 125, 64 126)
constexpr int kStep = 16;  // slots of a V row that leave at once

// Cache formats, as template argument.
enum Format : int { kFmtBf16 = 0, kFmtE4m3 = 1, kFmtE4m3Block = 2, kFmtInt8Block = 3 };

struct AppendParams {
    uint8_t* kc;
    uint8_t* vc;
    float* k_scale;  // one value (kFmtE4m3) or [num_blocks, Hk] (block formats)
    float* v_scale;
    const uint16_t* k;  // bf16 bits [T, Hk, D], token rows *_stride elements apart
    const uint16_t* v;
    const uint16_t* q;  // [T, Hq, D] or nullptr
    uint16_t* q_out;
    long long k_stride, v_stride, q_stride, qo_stride;
    const int32_t* bt;           // [S, max_blocks]
    const int32_t* seq_lens;     // [S], with the new tokens
    const int32_t* query_start;  // [S + 1], or nullptr: one row per sequence
    const int32_t* positions;    // [T], or nullptr: a token's index in its sequence
    const float* cos_sin;        // [max_position, rot] or nullptr
    uint32_t* status;            // or nullptr
    long long num_blocks;
    int T, S, Hq, Hk, max_blocks;
    int max_position, rot, interleaved;
    int chunks;        // CTAs per unit (kAppendWarps tasks each)
    int q_tokens, q_heads, q_groups;  // a query task: tokens, heads; head groups of a token
    int wide_v;        // value_cache is 32-byte aligned
};

__device__ __forceinline__ void flag(const AppendParams& p, uint32_t bits) {
    if (p.status) atomicOr(p.status, bits);
}

// Which two 8-element chunks of a head's row lane-pair j of D / 16 owns, and
// whether they turn.  Turned chunks c < rot / 8 are taken as (j, j + rot / 16),
// the pairs of a half-split rotation; the others in order.
struct ChunkPair {
    int a, b;
    bool turn;
    __device__ __forceinline__ ChunkPair(int j, int rot) {
        const int half = rot >> 4;
        turn = j < half;
        a = turn ? j : 2 * j;
        b = turn ? j + half : 2 * j + 1;
    }
};

// Two fp32 products at once (a packed sum after them would be fused into an
// fma, whatever its rounding modifier says; see Turn::two).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// The cosines and sines that a chunk pair turns by at one position.
struct Turn {
    float2 c[4], s[4];
    template <bool INTERLEAVED>
    __device__ __forceinline__ void load(const AppendParams& p, const ChunkPair& cp, int pos) {
        if (!cp.turn) return;
        const float* cs = p.cos_sin + static_cast<long long>(pos) * p.rot;
        const float* sn = cs + (p.rot >> 1);
        const int i0 = INTERLEAVED ? 4 * cp.a : 8 * cp.a;  // first angles: of chunk a ...
        const int i1 = INTERLEAVED ? 4 * cp.b : i0 + 4;    // ... and of b (or a's second half)
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(cs + i0));
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(cs + i1));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + i0));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(sn + i1));
        c[0] = make_float2(c0.x, c0.y);
        c[1] = make_float2(c0.z, c0.w);
        c[2] = make_float2(c1.x, c1.y);
        c[3] = make_float2(c1.z, c1.w);
        s[0] = make_float2(s0.x, s0.y);
        s[1] = make_float2(s0.z, s0.w);
        s[2] = make_float2(s1.x, s1.y);
        s[3] = make_float2(s1.z, s1.w);
    }
    // a' = a cos - b sin, b' = a sin + b cos for two pairs: each product and
    // each sum rounded once in fp32 (no contraction), so that the result does
    // not depend on how a compiler fuses them -- it fixes the 8-bit codes and
    // scales that follow.
    __device__ __forceinline__ void two(float2& a, float2& b, int i) const {
        const float2 ac = mul2(a, c[i]), bs = mul2(b, s[i]);
        const float2 as = mul2(a, s[i]), bc = mul2(b, c[i]);
        a = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
        b = make_float2(__fadd_rn(as.x, bc.x), __fadd_rn(as.y, bc.y));
    }
};

// A chunk pair in fp32, turned: element pairs x[0 .. 3] of chunk a, x[4 .. 7]
// of chunk b.
struct Chunks {
    float2 x[8];
    template <bool INTERLEAVED>
    __device__ __forceinline__ void turned(const uint4& wa, const uint4& wb, const ChunkPair& cp,
                                           const Turn& t) {
        const uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
        if (!cp.turn) return;
        if constexpr (INTERLEAVED) {  // pairs are a word's halves, angle i for word i
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 a = make_float2(x[2 * i].x, x[2 * i + 1].x);
                float2 b = make_float2(x[2 * i].y, x[2 * i + 1].y);
                t.two(a, b, i);
                x[2 * i] = make_float2(a.x, b.x);
                x[2 * i + 1] = make_float2(a.y, b.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) t.two(x[i], x[4 + i], i);
        }
    }
    __device__ __forceinline__ uint4 bf16(int chunk) const {
        const float2* y = x + 4 * chunk;
        return make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                          pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
    }
};

// A token's position, kept inside the table (flagged when it is not).
__device__ __forceinline__ int position_of(const AppendParams& p, int row, int index) {
    if (!p.cos_sin) return 0;
    const int pos = p.positions ? __ldg(p.positions + row) : index;
    if (pos >= 0 && pos < p.max_position) return pos;
    flag(p, PA_DEV_POSITION_OUT_OF_RANGE);
    return pos < 0 ? 0 : p.max_position - 1;
}

// ------------------------------------------------------------------ 8-bit codes
template <int FMT>
__device__ __forceinline__ constexpr float code_max() {
    return FMT == kFmtInt8Block ? 127.f : 448.f;
}

// x / scale for a power of two: by its reciprocal, exactly.
struct PowerOfTwo {
    float y;
    __device__ __forceinline__ explicit PowerOfTwo(float scale) {
        y = __uint_as_float((254u << 23) - __float_as_uint(scale));
    }
    static __device__ __forceinline__ bool is(float scale) {  // 2^-126 .. 2^126
        const uint32_t b = __float_as_uint(scale);
        return (b & 0x7fffffu) == 0 && b >= (1u << 23) && b <= (253u << 23);
    }
    __device__ __forceinline__ float operator()(float x) const { return x * y; }
};

// x / scale, correctly rounded, without a division per element: with y the
// correctly rounded reciprocal, q = x y is off by an ulp at most, and
// q + y (x - q scale), the remainder being exact in an fma, is the rounded
// quotient (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Where q is not finite it stands.
struct Divisor {
    float s, y;
    __device__ __forceinline__ explicit Divisor(float scale) {
        s = scale;
        y = __frcp_rn(scale);
    }
    __device__ __forceinline__ float operator()(float x) const {
        const float q = x * y;
        const float r = fmaf(fmaf(-q, s, x), y, q);
        return fabsf(q) < INFINITY ? r : q;
    }
};

// The nearest int8 code (ties to even), saturating at -127 and 127; a NaN
// becomes 0.
__device__ __forceinline__ uint32_t int8_code(float x) {
    uint32_t r;
    asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, 0fC2FE0000;\n\t"  // -127
        "cvt.rni.sat.s8.f32 %0, t;\n\t}"
        : "=r"(r)
        : "f"(x));
    return r;
}

// Two values to two codes (nearest, ties to even, saturating; a NaN becomes
// the e4m3 NaN, or int8 0), the first in the low byte; the upper half is not
// defined.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(float x, float y) {
    if constexpr (FMT == kFmtInt8Block)
        return __byte_perm(int8_code(x), int8_code(y), 0x0040);
    else
        return f32x2_to_e4m3x2(x, y);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3) {
    return __byte_perm(codes2<FMT>(x0, x1), codes2<FMT>(x2, x3), 0x5410);
}

// The smallest exponent e with amax <= code_max 2^e, within [-100, 100]:
// code_max is 1.75 2^8 (e4m3) or 1.984375 2^6 (int8), so amax's own exponent
// and a comparison of mantissas give it without rounding.
template <int FMT>
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - 127;
    const uint32_t m = b & 0x7fffffu;
    const int r = FMT == kFmtInt8Block ? e - 6 + (m > 0x7e0000u) : e - 8 + (m > 0x600000u);
    return max(-100, min(100, r));  // (0 and subnormals end at -100)
}

// The block's scale for a largest |x| of amax, joined with that of the tokens
// it already holds unless the run begins the block; *old is the scale that
// those tokens' codes have.
template <int FMT>
__device__ __forceinline__ float block_scale(const float* at, bool holds_tokens, float amax,
                                             float* old) {
    const float need =
        __uint_as_float(static_cast<uint32_t>(127 + scale_exponent<FMT>(amax)) << 23);
    *old = need;
    if (!holds_tokens) return need;
    constexpr float kLo = 7.888609052210118e-31f, kHi = 1.2676506002282294e30f;  // 2^-100, 2^100
    *old = fminf(fmaxf(*at, kLo), kHi);  // (a NaN becomes 2^-100)
    return fmaxf(*old, need);
}

// Four codes of a word in a scale `ratio` (<= 1) times finer than before.
template <int FMT>
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
    if constexpr (FMT == kFmtInt8Block) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xffu)) * ratio;
        return codes4<FMT>(x[0], x[1], x[2], x[3]);
    } else {
        const uint32_t lo = e4m3_lo_pair(w), hi = e4m3_hi_pair(w);
        return codes4<FMT>(f16_lo(lo) * ratio, f16_hi(lo) * ratio, f16_lo(hi) * ratio,
                           f16_hi(hi) * ratio);
    }
}

constexpr float kFltMax = 3.402823466e38f;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

// 32 bytes to consecutive addresses: one store where the cache's base allows
// it, so that a sector is written at once.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                     "r"(w[7])
                     : "memory");
    } else {
        uint4* d = static_cast<uint4*>(dst);
        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The part of one block that a sequence's run covers: slots [off, off + m),
// input rows row0 .., sequence indices index0 ...
struct Run {
    int row0, index0, off, m;
};

// ------------------------------------------------------------------------ keys
// Lane: chunk pair j = lane % (D / 16) of tokens lane / (D / 16) + TPI i.  A
// key's 16-byte chunks of one column group are contiguous over tokens, so a
// store instruction covers whole sectors of several groups.
template <int D, int B, int FMT, bool INTERLEAVED>
__device__ __forceinline__ void append_keys(const AppendParams& p, const Run& r, int h,
                                            long long pb, int lane) {
    constexpr int PJ = D / 16, TPI = 32 / PJ;
    constexpr bool BLOCK = FMT == kFmtE4m3Block || FMT == kFmtInt8Block;
    constexpr int PAGE = D * B * (FMT == kFmtBf16 ? 2 : 1);
    uint8_t* page = p.kc + (static_cast<size_t>(pb) * p.Hk + h) * PAGE;
    const ChunkPair cp(lane % PJ, p.rot);
    // Token t of the run: its chunks, turned.
    auto token = [&](int t, Chunks& x, uint4& wa, uint4& wb) {
        const uint16_t* src = p.k + static_cast<long long>(r.row0 + t) * p.k_stride + h * D;
        wa = __ldg(reinterpret_cast<const uint4*>(src + 8 * cp.a));
        wb = __ldg(reinterpret_cast<const uint4*>(src + 8 * cp.b));
        if (t + TPI < r.m) {
            prefetch_l1(src + TPI * p.k_stride + 8 * cp.a);
            prefetch_l1(src + TPI * p.k_stride + 8 * cp.b);
        }
        Turn turn;
        turn.load<INTERLEAVED>(p, cp, position_of(p, r.row0 + t, r.index0 + t));
        x.turned<INTERLEAVED>(wa, wb, cp, turn);
    };
    Chunks x;
    uint4 wa, wb;
    float scale = 1.f;
    if constexpr (BLOCK) {
        // The largest finite |x|: infinities saturate and NaNs stay NaN, and
        // neither may push a neighbour's code to 0.  (fmaxf drops NaNs; an
        // infinity is seen at the end, and then left out.)
        auto amax_below = [&](float limit) {
            float amax = 0.f;
#pragma unroll 1
            for (int t = lane / PJ; t < r.m; t += TPI) {
                token(t, x, wa, wb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = fabsf(x.x[e].x), v = fabsf(x.x[e].y);
                    amax = fmaxf(amax, u <= limit ? u : 0.f);
                    amax = fmaxf(amax, v <= limit ? v : 0.f);
                }
            }
            __syncwarp();
            return warp_max(amax);
        };
        float amax = amax_below(INFINITY);
        if (amax == INFINITY) amax = amax_below(kFltMax);
        float* at = p.k_scale + pb * p.Hk + h;
        float old;
        scale = block_scale<FMT>(at, r.off > 0, amax, &old);
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *at = scale;
        if (scale > old) {  // the block's earlier tokens, in the new scale
            const float ratio = __fdiv_rn(old, scale);
            uint32_t* words = reinterpret_cast<uint32_t*>(page);
#pragma unroll 1
            for (int w = lane; w < PAGE / 4; w += 32)
                if (w / 4 % B < r.off) words[w] = rescaled<FMT>(words[w], ratio);
        }
    } else if constexpr (FMT == kFmtE4m3) {
        scale = __ldg(p.k_scale);
    }
    auto store = [&](const auto& div) {
#pragma unroll 1
        for (int t = lane / PJ; t < r.m; t += TPI) {
            const int tok = r.off + t;
            token(t, x, wa, wb);
            if constexpr (FMT == kFmtBf16) {
                uint4* dst = reinterpret_cast<uint4*>(page);
                dst[cp.a * B + tok] = cp.turn ? x.bf16(0) : wa;
                dst[cp.b * B + tok] = cp.turn ? x.bf16(1) : wb;
            } else {
                auto eight = [&](const float2* y) {
                    return make_uint2(
                        codes4<FMT>(div(y[0].x), div(y[0].y), div(y[1].x), div(y[1].y)),
                        codes4<FMT>(div(y[2].x), div(y[2].y), div(y[3].x), div(y[3].y)));
                };
                uint8_t* da = page + ((cp.a >> 1) * B + tok) * 16 + (cp.a & 1) * 8;
                uint8_t* db = page + ((cp.b >> 1) * B + tok) * 16 + (cp.b & 1) * 8;
                *reinterpret_cast<uint2*>(da) = eight(x.x);
                *reinterpret_cast<uint2*>(db) = eight(x.x + 4);
            }
        }
    };
    if constexpr (FMT == kFmtBf16)
        store(0);
    else if (PowerOfTwo::is(scale))
        store(PowerOfTwo(scale));
    else
        store(Divisor(scale));
}

// ---------------------------------------------------------------------- values
// A V page holds a row of B tokens per head dim: lane l owns dims DV l ..
// DV l + DV - 1 of every token (DV = D / 32), and the transposition happens in
// its registers.  Where the run fills 16 slots each of the lane's rows leaves as
// one piece (32 bytes of bf16, 16 of codes), else as words of the slots that it
// fills; at its ends, and for single tokens, elements are stored one by one.
template <int D, int B, int FMT>
__device__ __forceinline__ void append_values(const AppendParams& p, const Run& r, int h,
                                              long long pb, int lane) {
    constexpr int DV = D / 32, NW = DV / 2;  // head dims and input words per lane and token
    constexpr bool BLOCK = FMT == kFmtE4m3Block || FMT == kFmtInt8Block;
    constexpr int ELEM = FMT == kFmtBf16 ? 2 : 1;
    constexpr int PAGE = D * B * ELEM;
    uint8_t* rows = p.vc + (static_cast<size_t>(pb) * p.Hk + h) * PAGE +
                    static_cast<size_t>(lane) * DV * B * ELEM;
    const uint16_t* src = p.v + static_cast<long long>(r.row0) * p.v_stride + h * D + DV * lane;
    auto load = [&](int t, uint32_t (&w)[NW]) {  // token t of the run
        const uint16_t* at = src + static_cast<long long>(t) * p.v_stride;
        if constexpr (NW == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            w[0] = v.x;
            w[1] = v.y;
        } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
        }
    };
    auto value = [&](const uint32_t (&w)[NW], int d) {
        return d % 2 ? bf16_hi(w[d / 2]) : bf16_lo(w[d / 2]);
    };
    float scale = 1.f;
    if constexpr (BLOCK) {
        // The largest finite |x|, as for the keys, on pairs of bf16 magnitudes
        // (which order like integers); those above `limit` are left out.
        auto amax_below = [&](uint32_t limit) {
            uint32_t amax = 0;
#pragma unroll 8
            for (int t = 0; t < r.m; ++t) {
                uint32_t w[NW];
                load(t, w);
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const uint32_t m = w[i] & 0x7fff7fffu;
                    amax = __vmaxu2(amax, limit == kFull ? m : m & __vcmpleu2(m, limit));
                }
            }
            amax = max(amax & 0xffffu, amax >> 16);
            return __reduce_max_sync(kFull, amax);
        };
        uint32_t bits = amax_below(kFull);
        if (bits >= 0x7f80u) bits = amax_below(0x7f7f7f7fu);
        const float amax = __uint_as_float(bits << 16);
        float* at = p.v_scale + pb * p.Hk + h;
        float old;
        scale = block_scale<FMT>(at, r.off > 0, amax, &old);
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *at = scale;
        if (scale > old) {
            // The block's earlier tokens, in the new scale; the bytes behind
            // them in a word are written back as they were.
            const float ratio = __fdiv_rn(old, scale);
#pragma unroll 1
            for (int i = 0; i < DV * (B / 4); ++i) {
                const int left = r.off - 4 * (i % (B / 4));  // earlier tokens in this word
                if (left <= 0) continue;
                uint32_t* at4 = reinterpret_cast<uint32_t*>(rows) + i;
                const uint32_t v = *at4, n = rescaled<FMT>(v, ratio);
                const uint32_t keep = left >= 4 ? 0u : kFull << (8 * left);
                *at4 = (n & ~keep) | (v & keep);
            }
        }
    } else if constexpr (FMT == kFmtE4m3) {
        scale = __ldg(p.v_scale);
    }
    const int end = r.off + r.m;
    constexpr int kPerWord = 4 / ELEM;  // slots of a 32-bit word of a row
    auto store = [&](const auto& div) {
#pragma unroll 1
        for (int t0 = 0; t0 < B; t0 += kStep) {  // slots t0 .. t0 + 15
            const int lo = max(t0, r.off), hi = min(t0 + kStep, end);
            // Slots [wlo, whi) leave as whole words, those around them one by one.
            const int wlo = (lo + kPerWord - 1) / kPerWord * kPerWord;
            const int whi = hi / kPerWord * kPerWord;
            if (wlo < whi) {
                const bool whole = hi - lo == kStep;
                uint32_t w[kStep][NW];
#pragma unroll
                for (int i = 0; i < kStep; ++i)
                    if (t0 + i >= wlo && t0 + i < whi) load(t0 + i - r.off, w[i]);
#pragma unroll
                for (int d = 0; d < DV; ++d) {
                    uint8_t* out = rows + (d * B + t0) * ELEM;
                    constexpr int NX = kStep / kPerWord;
                    uint32_t x[NX];
#pragma unroll
                    for (int i = 0; i < NX; ++i) {
                        if constexpr (FMT == kFmtBf16)
                            x[i] = __byte_perm(w[2 * i][d / 2], w[2 * i + 1][d / 2],
                                               d % 2 ? 0x7632 : 0x5410);
                        else
                            x[i] = codes4<FMT>(
                                div(value(w[4 * i], d)), div(value(w[4 * i + 1], d)),
                                div(value(w[4 * i + 2], d)), div(value(w[4 * i + 3], d)));
                    }
                    if (whole) {
                        if constexpr (FMT == kFmtBf16)
                            store32(out, x, p.wide_v != 0);
                        else
                            *reinterpret_cast<uint4*>(out) = make_uint4(x[0], x[1], x[2], x[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < NX; ++i)
                            if (t0 + i * kPerWord >= wlo && t0 + i * kPerWord < whi)
                                *reinterpret_cast<uint32_t*>(out + 4 * i) = x[i];
                    }
                }
                if (whole) continue;
            }
#pragma unroll 1
            for (int t = lo; t < hi; ++t) {
                if (t == wlo && wlo < whi) t = whi;
                if (t >= hi) break;
                uint32_t w[NW];
                load(t - r.off, w);
#pragma unroll
                for (int d = 0; d < DV; ++d) {
                    uint8_t* at = rows + (d * B + t) * ELEM;
                    if constexpr (FMT == kFmtBf16)
                        *reinterpret_cast<uint16_t*>(at) =
                            static_cast<uint16_t>(w[d / 2] >> (16 * (d % 2)));
                    else
                        *at = static_cast<uint8_t>(codes2<FMT>(div(value(w, d)), 0.f));
                }
            }
        }
    };
    if constexpr (FMT == kFmtBf16)
        store(0);
    else if (PowerOfTwo::is(scale))
        store(PowerOfTwo(scale));
    else
        store(Divisor(scale));
}

// --------------------------------------------------------------------- queries
// Task: tokens [t0, t0 + q_tokens) of the run, heads [h0, h0 + q_heads).  A
// token's angles are loaded once for all its heads.  A lane reads both chunks
// of a pair before it writes them, so query_out may be query itself.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void append_queries(const AppendParams& p, const Run& r, int t0, int h0,
                                               int lane) {
    constexpr int PJ = D / 16, TPI = 32 / PJ;
    const ChunkPair cp(lane % PJ, p.rot);
    const int t1 = min(t0 + p.q_tokens, r.m), h1 = min(h0 + p.q_heads, p.Hq);
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
        Turn turn;
        turn.load<INTERLEAVED>(p, cp, position_of(p, r.row0 + t, r.index0 + t));
        const uint16_t* src = p.q + static_cast<long long>(r.row0 + t) * p.q_stride;
        uint16_t* dst = p.q_out + static_cast<long long>(r.row0 + t) * p.qo_stride;
#pragma unroll 1
        for (int h = h0 + lane / PJ; h < h1; h += TPI) {
            const int a = h * D + 8 * cp.a, b = h * D + 8 * cp.b;
            const uint4 wa = *reinterpret_cast<const uint4*>(src + a);
            const uint4 wb = *reinterpret_cast<const uint4*>(src + b);
            // (To L1 two passes ahead: 124 -> 116 us on the 16 prompts.)
            if (h + 2 * TPI < h1) {
                prefetch_l1(src + a + 2 * TPI * D);
                prefetch_l1(src + b + 2 * TPI * D);
            }
            Chunks x;
            x.turned<INTERLEAVED>(wa, wb, cp, turn);
            *reinterpret_cast<uint4*>(dst + a) = cp.turn ? x.bf16(0) : wa;
            *reinterpret_cast<uint4*>(dst + b) = cp.turn ? x.bf16(1) : wb;
        }
    }
}

// ---------------------------------------------------------------------- kernel
// Units: sequence s owns the units from f(s) = query_start[s] / B + 2 s up to
// f(s + 1), enough for the blocks that its n_s rows can touch (n_s / B + 2 at
// most), so a unit finds its sequence from query_start alone, by a 32-way
// search; units past a sequence's blocks have nothing to do.  Without
// query_start, unit u is sequence u and its one row, if it has a length.
template <int D, int B, int FMT, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendCtasPerSm) pa_append_kernel(const AppendParams p) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int u = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.chunks));
    int task = static_cast<int>(blockIdx.x - static_cast<unsigned>(u) * p.chunks) * kAppendWarps +
               (threadIdx.x >> 5);
    int s = u, a = u, b = u + 1, j = 0;
    if (p.query_start) {
        // (Unit u looks after entry u: a bad one may leave its sequence no unit.)
        if (task == 0 && lane == 0 && u < p.S && bad_rows(p.query_start, u, p.T))
            flag(p, PA_DEV_BAD_QUERY_START);
        auto f = [&](int i) {
            return max(0, min(__ldg(p.query_start + i), p.T)) / B + 2 * i;
        };
        s = find_sequence(p.S, lane, f, u);
        if (s < 0 || bad_rows(p.query_start, s, p.T)) return;
        a = __ldg(p.query_start + s);
        b = __ldg(p.query_start + s + 1);
        j = u - f(s);
        if (j < 0 || a == b) return;
    }
    const int T = __ldg(p.seq_lens + s);
    if (!p.query_start && T == 0) return;  // a padded batch's row
    const int start = T - (b - a);  // the run's first index
    if (start < 0 || T > static_cast<long long>(p.max_blocks) * B) {
        if (lane == 0) flag(p, PA_DEV_SEQ_LEN_OUT_OF_RANGE);
        return;
    }
    const int blk = start / B + j;
    if (blk > (T - 1) / B) return;
    Run r;
    r.index0 = max(start, blk * B);
    r.off = r.index0 - blk * B;
    r.m = min(T - r.index0, B - r.off);
    r.row0 = a + (r.index0 - start);
    if (task >= 2 * p.Hk) {
        if (!p.q) return;
        const int q_task = task - 2 * p.Hk;
        const int t0 = q_task / p.q_groups * p.q_tokens;
        if (t0 < r.m)
            append_queries<D, INTERLEAVED>(p, r, t0, q_task % p.q_groups * p.q_heads, lane);
        return;
    }
    const int pb = __ldg(p.bt + static_cast<long long>(s) * p.max_blocks + blk);
    if (pb < 0 || pb >= p.num_blocks) {
        if (lane == 0) flag(p, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    if (task < p.Hk)
        append_keys<D, B, FMT, INTERLEAVED>(p, r, task, pb, lane);
    else
        append_values<D, B, FMT>(p, r, task - p.Hk, pb, lane);
}

template <int D, int B, int FMT>
cudaError_t launch_append(const AppendParams& p, unsigned grid, cudaStream_t st) {
    return p.interleaved
               ? launch_pdl(pa_append_kernel<D, B, FMT, true>, grid, kAppendWarps * 32, 0, st, p)
               : launch_pdl(pa_append_kernel<D, B, FMT, false>, grid, kAppendWarps * 32, 0, st, p);
}

template <int D, int B>
cudaError_t launch_format(const AppendParams& p, pa_kv_dtype t, unsigned grid, cudaStream_t st) {
    switch (t) {
        case PA_KV_BF16: return launch_append<D, B, kFmtBf16>(p, grid, st);
        case PA_KV_FP8_E4M3: return launch_append<D, B, kFmtE4m3>(p, grid, st);
        case PA_KV_FP8_E4M3_BLOCK: return launch_append<D, B, kFmtE4m3Block>(p, grid, st);
        default: return launch_append<D, B, kFmtInt8Block>(p, grid, st);
    }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_append_kv(void* key_cache, void* value_cache, const void* key,
                                  const void* value, int num_tokens, int num_seqs,
                                  int num_kv_heads, int head_size, const int32_t* block_tables,
                                  int max_blocks_per_seq, const int32_t* seq_lens,
                                  const int32_t* query_start, int block_size, int64_t num_blocks,
                                  pa_kv_dtype kv_dtype, float* k_scale, float* v_scale,
                                  uint32_t* status, void* stream, const pa_append_options* opts) {
    using pa::aligned;
    using pa::fail;
    pa::clear_detail();
    if (num_tokens < 0 || num_seqs < 0)
        return fail(PA_ERR_INVALID_ARG, "%s", "num_tokens or num_seqs < 0");
    if (num_kv_heads < 1) return fail(PA_ERR_INVALID_ARG, "%s", "num_kv_heads must be > 0");
    if (head_size != 64 && head_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "%s", "head_size must be 64 or 128");
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "%s", "block_size must be 16 or 32");
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3 && !pa::block_scales(kv_dtype))
        return fail(PA_ERR_UNSUPPORTED, "%s", "kv_dtype");
    if (max_blocks_per_seq < 1) return fail(PA_ERR_INVALID_ARG, "%s", "max_blocks_per_seq < 1");
    if (num_blocks < 1 || num_blocks > 0x7fffffffLL)
        return fail(PA_ERR_INVALID_ARG, "%s", "num_blocks must be in [1, 2^31)");
    if (!query_start && num_tokens != num_seqs)
        return fail(PA_ERR_INVALID_ARG, "%s",
                    "without query_start every sequence has one row: num_tokens != num_seqs");
    pa_append_options o;
    if (opts)
        o = *opts;
    else
        std::memset(&o, 0, sizeof o);
    const long long dense = static_cast<long long>(num_kv_heads) * head_size;
    if (!o.key_stride) o.key_stride = dense;
    if (!o.value_stride) o.value_stride = dense;
    if (o.key_stride < dense || o.value_stride < dense || o.key_stride % 8 || o.value_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "%s",
                    "key_stride and value_stride must be multiples of 8 elements, at least "
                    "num_kv_heads * head_size");
    if (o.cos_sin) {
        if (o.rotary_dim < 16 || o.rotary_dim > head_size || o.rotary_dim % 16)
            return fail(PA_ERR_UNSUPPORTED, "%s",
                        "rotary_dim must be a multiple of 16 in [16, head_size]");
        if (o.max_position < 1) return fail(PA_ERR_INVALID_ARG, "%s", "max_position < 1");
        if (!aligned(o.cos_sin, 16)) return fail(PA_ERR_INVALID_ARG, "%s", "cos_sin is misaligned");
        if (!aligned(o.positions, 4))
            return fail(PA_ERR_INVALID_ARG, "%s", "positions is misaligned");
    } else if (o.rotary_dim || o.positions || o.query || o.query_out) {
        return fail(PA_ERR_INVALID_ARG, "%s",
                    "rotary_dim, positions, query and query_out need cos_sin");
    }
    if (!o.query != !o.query_out)
        return fail(PA_ERR_INVALID_ARG, "%s", "query and query_out go together");
    if (o.query) {
        if (o.num_heads < 1 || o.num_heads > 65536)
            return fail(PA_ERR_INVALID_ARG, "%s", "num_heads must be in [1, 65536]");
        const long long dense_q = static_cast<long long>(o.num_heads) * head_size;
        if (!o.query_stride) o.query_stride = dense_q;
        if (!o.query_out_stride) o.query_out_stride = dense_q;
        if (o.query_stride < dense_q || o.query_out_stride < dense_q || o.query_stride % 8 ||
            o.query_out_stride % 8)
            return fail(PA_ERR_INVALID_ARG, "%s",
                        "query_stride and query_out_stride must be multiples of 8 elements, at "
                        "least num_heads * head_size");
        if (!aligned(o.query, 16) || !aligned(o.query_out, 16))
            return fail(PA_ERR_INVALID_ARG, "%s", "query or query_out is misaligned");
    }
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    const struct {
        const void* p;
        size_t a;
        const char* name;
    } ptrs[] = {{key_cache, 16, "key_cache"}, {value_cache, 16, "value_cache"},
                {key, 16, "key"},             {value, 16, "value"},
                {block_tables, 4, "block_tables"}, {seq_lens, 4, "seq_lens"}};
    for (const auto& q : ptrs) {
        if (!q.p) return fail(PA_ERR_INVALID_ARG, "%s is NULL", q.name);
        if (!aligned(q.p, q.a)) return fail(PA_ERR_INVALID_ARG, "%s is misaligned", q.name);
    }
    if (!aligned(query_start, 4) || !aligned(status, 4))
        return fail(PA_ERR_INVALID_ARG, "%s", "query_start or status is misaligned");
    if (kv_dtype != PA_KV_BF16) {
        if (!k_scale || !v_scale)
            return fail(PA_ERR_INVALID_ARG, "%s",
                        "k_scale and v_scale are required for an 8-bit cache");
        if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
            return fail(PA_ERR_INVALID_ARG, "%s", "k_scale / v_scale misaligned");
    }
    const long long units = query_start ? num_tokens / block_size + 2ll * num_seqs : num_seqs;
    const long long tokens = query_start ? (num_tokens < block_size ? num_tokens : block_size) : 1;
    // Query tasks: about 32 rows of a page's tokens; in a decode step, where a
    // row is waited for, no more than one pass of a warp.
    const int rows_per_pass = 512 / head_size;
    const int q_rows = query_start ? pa::kQueryRows : rows_per_pass;
    const int q_heads = o.num_heads < q_rows ? o.num_heads : q_rows;
    const int q_tokens = o.query && q_rows / o.num_heads > 1 ? q_rows / o.num_heads : 1;
    const int q_groups = o.query ? (o.num_heads + q_heads - 1) / q_heads : 1;
    const long long q_tasks = o.query ? (tokens + q_tokens - 1) / q_tokens * q_groups : 0;
    const long long tasks = 2ll * num_kv_heads + q_tasks;
    const long long chunks = (tasks + pa::kAppendWarps - 1) / pa::kAppendWarps;
    if (units > 0x7fffffffll || units * chunks > 0x7fffffffll)
        return fail(PA_ERR_INVALID_ARG, "%s", "too many tokens, sequences and heads for one call");
    pa::AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.kc = static_cast<uint8_t*>(key_cache);
    p.vc = static_cast<uint8_t*>(value_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k = static_cast<const uint16_t*>(key);
    p.v = static_cast<const uint16_t*>(value);
    p.q = static_cast<const uint16_t*>(o.query);
    p.q_out = static_cast<uint16_t*>(o.query_out);
    p.k_stride = o.key_stride;
    p.v_stride = o.value_stride;
    p.q_stride = o.query_stride;
    p.qo_stride = o.query_out_stride;
    p.bt = block_tables;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    p.positions = o.positions;
    p.cos_sin = o.cos_sin;
    p.status = status;
    p.num_blocks = num_blocks;
    p.T = num_tokens;
    p.S = num_seqs;
    p.Hq = o.query ? o.num_heads : 1;
    p.Hk = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.max_position = o.max_position;
    p.rot = o.cos_sin ? o.rotary_dim : 0;
    p.interleaved = o.interleaved;
    p.chunks = static_cast<int>(chunks);
    p.q_tokens = q_tokens;
    p.q_heads = q_heads;
    p.q_groups = q_groups;
    p.wide_v = aligned(value_cache, 32);
    const unsigned grid = static_cast<unsigned>(units * chunks);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_size == 64)
        e = block_size == 16 ? pa::launch_format<64, 16>(p, kv_dtype, grid, st)
                             : pa::launch_format<64, 32>(p, kv_dtype, grid, st);
    else
        e = block_size == 16 ? pa::launch_format<128, 16>(p, kv_dtype, grid, st)
                             : pa::launch_format<128, 32>(p, kv_dtype, grid, st);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
    return PA_OK;
}
