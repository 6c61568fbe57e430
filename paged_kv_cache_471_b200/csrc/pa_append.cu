// Appending keys and values to the paged cache, with the position rotation on
// the way (pa_append_kv; see include/pagedattn.h for the contract).
//
// Work is cut into (block of a sequence's run, task) pairs, one warp each:
//   * task h < Hk: the new keys of kv head h in the block;
//   * task Hk + h: its new values;
//   * the tasks after them: the query rows of the block's new tokens.
// A warp holds what it loads in registers (a whole page of new tokens is 4 KiB
// at head size 128, 16 tokens), so every load is in flight before the first is
// used, and a (block, head)'s largest |x| -- which fixes its scale -- needs one
// warp reduction and no second pass over memory.  Warps share nothing and
// never wait for one another: the rotation's table rows are re-read by each
// head from L1, at twice the bytes of the bf16 rows they turn.
//
// Bound: every row is read once and every element written once, so DRAM for
// prompts; for single tokens the launch and two dependent rounds of loads
// (length -> block id and angles -> scale).
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>

#include "pa_launch.cuh"
#include "pagedattn.h"

namespace pa {
namespace {

constexpr int kAppendWarps = 4;

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
    int wide_v;        // value_cache is 32-byte aligned
};

__device__ __forceinline__ void flag(const AppendParams& p, uint32_t bits) {
    if (p.status) atomicOr(p.status, bits);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
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

// a' = a cos - b sin, b' = a sin + b cos: each product and each sum rounded
// once in fp32 (no contraction), so that the result does not depend on how a
// compiler fuses them -- it fixes the 8-bit codes and scales that follow.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float y = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    a = x;
    b = y;
}

// The two chunks of one row at position `pos`, in fp32, turned.
__device__ __forceinline__ void turned_chunks(const AppendParams& p, const ChunkPair& cp, int pos,
                                              const uint4& wa, const uint4& wb, float (&xa)[8],
                                              float (&xb)[8]) {
    unpack8(wa, xa);
    unpack8(wb, xb);
    if (!cp.turn) return;
    const float* cs = p.cos_sin + static_cast<long long>(pos) * p.rot;
    const float* sn = cs + (p.rot >> 1);
    const int i0 = p.interleaved ? 4 * cp.a : 8 * cp.a;  // first angles: of chunk a ...
    const int i1 = p.interleaved ? 4 * cp.b : i0 + 4;    // ... and of b (or a's second half)
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(cs + i0));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(cs + i1));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + i0));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(sn + i1));
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn_pair(xa[2 * i], xa[2 * i + 1], c[i], s[i]);
            turn_pair(xb[2 * i], xb[2 * i + 1], c[4 + i], s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(xa[i], xb[i], c[i], s[i]);
    }
}

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

// x / scale, correctly rounded; for a power of two by its (exact) reciprocal.
struct Divisor {
    float s, inv;
    bool pow2;
    __device__ __forceinline__ explicit Divisor(float s_) {
        s = s_;
        const uint32_t b = __float_as_uint(s_);
        const uint32_t e = b >> 23;  // (the sign counts: a negative scale is no power of two)
        pow2 = (b & 0x7fffffu) == 0 && e >= 1 && e <= 253;
        inv = pow2 ? __uint_as_float((254u - e) << 23) : 0.f;
    }
    __device__ __forceinline__ float operator()(float x) const {
        return pow2 ? x * inv : __fdiv_rn(x, s);
    }
};

// Two values to two codes (nearest, ties to even, saturating; a NaN becomes
// the e4m3 NaN, or int8 0), the first in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(float x, float y) {
    if constexpr (FMT == kFmtInt8Block) {
        const int a = max(-127, min(127, __float2int_rn(x)));
        const int b = max(-127, min(127, __float2int_rn(y)));
        return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
    } else {
        return f32x2_to_e4m3x2(x, y);
    }
}
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const Divisor& d, float x0, float x1, float x2,
                                           float x3) {
    return codes2<FMT>(d(x0), d(x1)) | (codes2<FMT>(d(x2), d(x3)) << 16);
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

// The largest finite |x| (infinities saturate and NaNs stay NaN; neither may
// push a neighbour's code to 0).
__device__ __forceinline__ float amax_of(float amax, float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? fmaxf(amax, a) : amax;
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
        return codes2<FMT>(x[0], x[1]) | (codes2<FMT>(x[2], x[3]) << 16);
    } else {
        const uint32_t lo = e4m3_lo_pair(w), hi = e4m3_hi_pair(w);
        return codes2<FMT>(f16_lo(lo) * ratio, f16_hi(lo) * ratio) |
               (codes2<FMT>(f16_lo(hi) * ratio, f16_hi(hi) * ratio) << 16);
    }
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
template <int D, int B, int FMT>
__device__ __forceinline__ void append_keys(const AppendParams& p, const Run& r, int h,
                                            long long pb, int lane) {
    constexpr int PJ = D / 16, TPI = 32 / PJ, IT = B / TPI;
    constexpr bool BLOCK = FMT == kFmtE4m3Block || FMT == kFmtInt8Block;
    constexpr int PAGE = D * B * (FMT == kFmtBf16 ? 2 : 1);
    uint8_t* page = p.kc + (static_cast<size_t>(pb) * p.Hk + h) * PAGE;
    const ChunkPair cp(lane % PJ, p.rot);
    const int tok0 = lane / PJ;
    uint4 wa[IT], wb[IT];
    int pos[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int t = tok0 + i * TPI - r.off;  // token of the run, if in [0, m)
        wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
        pos[i] = 0;
        if (t < 0 || t >= r.m) continue;
        const uint16_t* src = p.k + static_cast<long long>(r.row0 + t) * p.k_stride + h * D;
        wa[i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * cp.a));
        wb[i] = __ldg(reinterpret_cast<const uint4*>(src + 8 * cp.b));
        pos[i] = position_of(p, r.row0 + t, r.index0 + t);
    }
    float scale = 1.f;
    if constexpr (BLOCK) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int t = tok0 + i * TPI - r.off;
            if (t < 0 || t >= r.m) continue;
            float xa[8], xb[8];
            turned_chunks(p, cp, pos[i], wa[i], wb[i], xa, xb);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = amax_of(amax_of(amax, xa[e]), xb[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
        float* at = p.k_scale + pb * p.Hk + h;
        float old;
        scale = block_scale<FMT>(at, r.off > 0, amax, &old);
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *at = scale;
        if (scale > old) {  // the block's earlier tokens, in the new scale
            const float ratio = __fdiv_rn(old, scale);
            uint4* words = reinterpret_cast<uint4*>(page);
            for (int w = lane; w < PAGE / 16; w += 32) {
                if (w % B >= r.off) continue;
                uint4 v = words[w];
                v.x = rescaled<FMT>(v.x, ratio);
                v.y = rescaled<FMT>(v.y, ratio);
                v.z = rescaled<FMT>(v.z, ratio);
                v.w = rescaled<FMT>(v.w, ratio);
                words[w] = v;
            }
        }
    } else if constexpr (FMT == kFmtE4m3) {
        scale = __ldg(p.k_scale);
    }
    const Divisor div(scale);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int tok = tok0 + i * TPI;
        const int t = tok - r.off;
        if (t < 0 || t >= r.m) continue;
        float xa[8], xb[8];
        turned_chunks(p, cp, pos[i], wa[i], wb[i], xa, xb);
        if constexpr (FMT == kFmtBf16) {
            uint4* dst = reinterpret_cast<uint4*>(page);
            dst[cp.a * B + tok] = cp.turn ? pack8(xa) : wa[i];
            dst[cp.b * B + tok] = cp.turn ? pack8(xb) : wb[i];
        } else {
            uint8_t* da = page + ((cp.a >> 1) * B + tok) * 16 + (cp.a & 1) * 8;
            uint8_t* db = page + ((cp.b >> 1) * B + tok) * 16 + (cp.b & 1) * 8;
            *reinterpret_cast<uint2*>(da) =
                make_uint2(codes4<FMT>(div, xa[0], xa[1], xa[2], xa[3]),
                           codes4<FMT>(div, xa[4], xa[5], xa[6], xa[7]));
            *reinterpret_cast<uint2*>(db) =
                make_uint2(codes4<FMT>(div, xb[0], xb[1], xb[2], xb[3]),
                           codes4<FMT>(div, xb[4], xb[5], xb[6], xb[7]));
        }
    }
}

// ---------------------------------------------------------------------- values
// A V page holds a row of B tokens per head dim: lane l owns dims DV l ..
// DV l + DV - 1 of every token (DV = D / 32), so the transposition happens in
// its registers and each of its rows leaves in pieces as wide as the run
// fills: 32 or 16 bytes, else single words or elements.
template <int D, int B, int FMT>
__device__ __forceinline__ void append_values(const AppendParams& p, const Run& r, int h,
                                              long long pb, int lane) {
    constexpr int DV = D / 32, NW = DV / 2;  // head dims and input words per lane and token
    constexpr bool BLOCK = FMT == kFmtE4m3Block || FMT == kFmtInt8Block;
    constexpr int ELEM = FMT == kFmtBf16 ? 2 : 1;
    constexpr int PAGE = D * B * ELEM;
    uint8_t* rows = p.vc + (static_cast<size_t>(pb) * p.Hk + h) * PAGE +
                    static_cast<size_t>(lane) * DV * B * ELEM;
    const int end = r.off + r.m;
    uint32_t w[B][NW];
    const uint16_t* src =
        p.v + static_cast<long long>(r.row0 - r.off) * p.v_stride + h * D + DV * lane;
#pragma unroll
    for (int t = 0; t < B; ++t) {
        const bool in = t >= r.off && t < end;
        const uint16_t* at = src + static_cast<long long>(t) * p.v_stride;
        if constexpr (NW == 2) {
            const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
            w[t][0] = v.x;
            w[t][1] = v.y;
        } else {
            w[t][0] = in ? __ldg(reinterpret_cast<const uint32_t*>(at)) : 0u;
        }
    }
    if constexpr (FMT == kFmtBf16) {
#pragma unroll
        for (int d = 0; d < DV; ++d) {
            uint8_t* row = rows + d * B * 2;
            // Words of two tokens' elements of this dim.
            uint32_t x[B / 2];
#pragma unroll
            for (int t = 0; t < B / 2; ++t)
                x[t] = __byte_perm(w[2 * t][d / 2], w[2 * t + 1][d / 2], d % 2 ? 0x7632 : 0x5410);
#pragma unroll
            for (int s = 0; s < B / 16; ++s) {  // 16 tokens, one 32-byte sector
                if (r.off <= 16 * s && end >= 16 * s + 16) {
                    const uint32_t v[8] = {x[8 * s],     x[8 * s + 1], x[8 * s + 2], x[8 * s + 3],
                                           x[8 * s + 4], x[8 * s + 5], x[8 * s + 6], x[8 * s + 7]};
                    store32(row + 32 * s, v, p.wide_v != 0);
                    continue;
                }
#pragma unroll
                for (int t = 8 * s; t < 8 * s + 8; ++t) {
                    const bool lo = 2 * t >= r.off && 2 * t < end;
                    const bool hi = 2 * t + 1 >= r.off && 2 * t + 1 < end;
                    if (lo && hi) {
                        *reinterpret_cast<uint32_t*>(row + 4 * t) = x[t];
                    } else if (lo) {
                        *reinterpret_cast<uint16_t*>(row + 4 * t) = static_cast<uint16_t>(x[t]);
                    } else if (hi) {
                        *reinterpret_cast<uint16_t*>(row + 4 * t + 2) =
                            static_cast<uint16_t>(x[t] >> 16);
                    }
                }
            }
        }
        return;
    } else {
        auto value = [&](int t, int d) {
            return d % 2 ? bf16_hi(w[t][d / 2]) : bf16_lo(w[t][d / 2]);
        };
        float scale;
        if constexpr (BLOCK) {
            float amax = 0.f;  // (rows outside the run are zeros)
#pragma unroll
            for (int t = 0; t < B; ++t)
#pragma unroll
                for (int d = 0; d < DV; ++d) amax = amax_of(amax, value(t, d));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            float* at = p.v_scale + pb * p.Hk + h;
            float old;
            scale = block_scale<FMT>(at, r.off > 0, amax, &old);
            __syncwarp();  // every lane has read the old scale
            if (lane == 0) *at = scale;
            if (scale > old) {
                // The block's earlier tokens, in the new scale; the bytes behind
                // them in a word are written back as they were.
                const float ratio = __fdiv_rn(old, scale);
                for (int i = 0; i < DV * (B / 4); ++i) {
                    const int left = r.off - 4 * (i % (B / 4));  // earlier tokens in this word
                    if (left <= 0) continue;
                    uint32_t* at4 = reinterpret_cast<uint32_t*>(rows) + i;
                    const uint32_t v = *at4, n = rescaled<FMT>(v, ratio);
                    const uint32_t keep = left >= 4 ? 0u : kFull << (8 * left);
                    *at4 = (n & ~keep) | (v & keep);
                }
            }
        } else {
            scale = __ldg(p.v_scale);
        }
        const Divisor div(scale);
#pragma unroll
        for (int d = 0; d < DV; ++d) {
            uint8_t* row = rows + d * B;
            uint32_t x[B / 4];
#pragma unroll
            for (int t = 0; t < B / 4; ++t)
                x[t] = codes4<FMT>(div, value(4 * t, d), value(4 * t + 1, d),
                                   value(4 * t + 2, d), value(4 * t + 3, d));
#pragma unroll
            for (int s = 0; s < B / 16; ++s) {
                if (r.off <= 16 * s && end >= 16 * s + 16) {
                    *reinterpret_cast<uint4*>(row + 16 * s) =
                        make_uint4(x[4 * s], x[4 * s + 1], x[4 * s + 2], x[4 * s + 3]);
                    continue;
                }
#pragma unroll
                for (int t = 4 * s; t < 4 * s + 4; ++t) {
                    if (r.off <= 4 * t && end >= 4 * t + 4) {
                        *reinterpret_cast<uint32_t*>(row + 4 * t) = x[t];
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * t + e >= r.off && 4 * t + e < end)
                            row[4 * t + e] = static_cast<uint8_t>(x[t] >> (8 * e));
                }
            }
        }
    }
}

// --------------------------------------------------------------------- queries
// Query rows a task covers: 4 KiB of them.
template <int D>
constexpr int query_rows() {
    return 2048 / D;
}

// Rows [first, first + query_rows) of the run's (token, head) rows, heads
// fastest.  A lane reads both chunks of a pair before it writes them, so
// query_out may be query itself.
template <int D>
__device__ __forceinline__ void append_queries(const AppendParams& p, const Run& r, int first,
                                               int lane) {
    constexpr int PJ = D / 16, TPI = 32 / PJ, IT = query_rows<D>() / TPI;
    const ChunkPair cp(lane % PJ, p.rot);
    uint4 wa[IT], wb[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int n = first + lane / PJ + i * TPI;
        const int t = n / p.Hq, h = n - t * p.Hq;
        wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
        if (t >= r.m) continue;
        const uint16_t* src = p.q + static_cast<long long>(r.row0 + t) * p.q_stride + h * D;
        wa[i] = *reinterpret_cast<const uint4*>(src + 8 * cp.a);
        wb[i] = *reinterpret_cast<const uint4*>(src + 8 * cp.b);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int n = first + lane / PJ + i * TPI;
        const int t = n / p.Hq, h = n - t * p.Hq;
        if (t >= r.m) continue;
        float xa[8], xb[8];
        turned_chunks(p, cp, position_of(p, r.row0 + t, r.index0 + t), wa[i], wb[i], xa, xb);
        uint16_t* dst = p.q_out + static_cast<long long>(r.row0 + t) * p.qo_stride + h * D;
        *reinterpret_cast<uint4*>(dst + 8 * cp.a) = cp.turn ? pack8(xa) : wa[i];
        *reinterpret_cast<uint4*>(dst + 8 * cp.b) = cp.turn ? pack8(xb) : wb[i];
    }
}

// ---------------------------------------------------------------------- kernel
// Units: sequence s owns the units from f(s) = query_start[s] / B + 2 s up to
// f(s + 1), enough for the blocks that its n_s rows can touch (n_s / B + 2 at
// most), so a unit finds its sequence from query_start alone, by a 32-way
// search; units past a sequence's blocks have nothing to do.  Without
// query_start, unit u is sequence u and its one row.
template <int D, int B, int FMT>
__global__ void __launch_bounds__(kAppendWarps * 32) pa_append_kernel(const AppendParams p) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int u = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.chunks));
    int task = static_cast<int>(blockIdx.x - static_cast<unsigned>(u) * p.chunks) * kAppendWarps +
               (threadIdx.x >> 5);
    int s = u, a = u, b = u + 1, j = 0;
    if (p.query_start) {
        auto f = [&](int i) {
            return max(0, min(__ldg(p.query_start + i), p.T)) / B + 2 * i;
        };
        int lo = 0, hi = p.S;
        for (;;) {
            const int step = (hi - lo + 31) / 32;
            const int i = lo + lane * step;
            const unsigned before = __ballot_sync(kFull, i < hi && f(i) <= u);
            if (before == 0) return;  // rows before query_start[0] belong to nobody
            lo += (__popc(before) - 1) * step;
            hi = min(hi, lo + step);
            if (step == 1) break;
        }
        s = lo;
        a = __ldg(p.query_start + s);
        b = __ldg(p.query_start + s + 1);
        if (a < 0 || b < a || b > p.T) {
            if (lane == 0) flag(p, PA_DEV_BAD_QUERY_START);
            return;
        }
        j = u - f(s);
        if (a == b) return;
    }
    const int T = __ldg(p.seq_lens + s);
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
    r.m = min(T, (blk + 1) * B) - r.index0;
    r.row0 = a + (r.index0 - start);
    if (task >= 2 * p.Hk) {
        if (!p.q) return;
        const long long first = static_cast<long long>(task - 2 * p.Hk) * query_rows<D>();
        if (first < static_cast<long long>(r.m) * p.Hq)
            append_queries<D>(p, r, static_cast<int>(first), lane);
        return;
    }
    const int pb = __ldg(p.bt + static_cast<long long>(s) * p.max_blocks + blk);
    if (pb < 0 || pb >= p.num_blocks) {
        if (lane == 0) flag(p, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    if (task < p.Hk)
        append_keys<D, B, FMT>(p, r, task, pb, lane);
    else
        append_values<D, B, FMT>(p, r, task - p.Hk, pb, lane);
}

template <int D, int B>
cudaError_t launch_format(const AppendParams& p, int fmt, unsigned grid, cudaStream_t st) {
    constexpr unsigned kThreadsPerCta = kAppendWarps * 32;
    switch (fmt) {
        case kFmtBf16:
            return launch_pdl(pa_append_kernel<D, B, kFmtBf16>, grid, kThreadsPerCta, 0, st, p);
        case kFmtE4m3:
            return launch_pdl(pa_append_kernel<D, B, kFmtE4m3>, grid, kThreadsPerCta, 0, st, p);
        case kFmtE4m3Block:
            return launch_pdl(pa_append_kernel<D, B, kFmtE4m3Block>, grid, kThreadsPerCta, 0, st,
                              p);
        default:
            return launch_pdl(pa_append_kernel<D, B, kFmtInt8Block>, grid, kThreadsPerCta, 0, st,
                              p);
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
    const long long rows_per_task = 2048 / head_size;
    const long long q_tasks =
        o.query ? (tokens * o.num_heads + rows_per_task - 1) / rows_per_task : 0;
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
    p.wide_v = aligned(value_cache, 32);
    const int fmt = kv_dtype == PA_KV_BF16             ? pa::kFmtBf16
                    : kv_dtype == PA_KV_FP8_E4M3       ? pa::kFmtE4m3
                    : kv_dtype == PA_KV_FP8_E4M3_BLOCK ? pa::kFmtE4m3Block
                                                       : pa::kFmtInt8Block;
    const unsigned grid = static_cast<unsigned>(units * chunks);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (head_size == 64)
        e = block_size == 16 ? pa::launch_format<64, 16>(p, fmt, grid, st)
                             : pa::launch_format<64, 32>(p, fmt, grid, st);
    else
        e = block_size == 16 ? pa::launch_format<128, 16>(p, fmt, grid, st)
                             : pa::launch_format<128, 32>(p, fmt, grid, st);
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
    return PA_OK;
}
