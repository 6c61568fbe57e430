// The decode kernel's forms for 8-bit pages with a scale per (block, kv head).
//
// Bound: DRAM, as with one scale per tensor; a page's scales are 8 bytes beside
// 4 KiB of codes.  Measured, one box, us on one set of inputs repeated, then on
// three sets in turn (per tensor e4m3 / e4m3 blocks / int8 blocks):
//   128 sequences of 512-8192 tokens, 64/8 heads (floor 174)
//                               178 / 190 / 208     191 / 201 / 221
//   32 sequences of 4001-4096 tokens, 32/32 heads (floor 162)
//                               167 / 177 / 188     172 / 182 / 200
//   1 sequence of 131072 tokens, 32/8 heads, B = 32 (floor 41)
//                               51.4 / 51.9 / 57.8  50.3 / 51.7 / 56.5
// The scales cost a multiply-add per logit and an exponential per page; int8
// codes cost three more instructions per four codes than e4m3's conversion.
#include "pa_launch.cuh"

namespace pa {
namespace {

template <int D, int B, int CODES>
cudaError_t launch_codes(const DecodeParams& p, long long grid, size_t smem, cudaStream_t st) {
    // Shared-prefix units pack 16 query rows, so they need the 16-row form.
    return (p.G > 8 || p.prefix_pages > 0)
               ? launch_decode<D, B, true, 2, false, false, CODES>(p, grid, smem, st)
               : launch_decode<D, B, true, 1, false, false, CODES>(p, grid, smem, st);
}

template <int D, int B>
cudaError_t launch_page(const DecodeParams& p, bool int8, long long grid, size_t smem,
                        cudaStream_t st) {
    return int8 ? launch_codes<D, B, kInt8Block>(p, grid, smem, st)
                : launch_codes<D, B, kE4m3Block>(p, grid, smem, st);
}

}  // namespace

cudaError_t launch_decode_block(const DecodeParams& p, int D, int B, bool int8, long long grid,
                                size_t smem, cudaStream_t st) {
    if (D == 64)
        return B == 16 ? launch_page<64, 16>(p, int8, grid, smem, st)
                       : launch_page<64, 32>(p, int8, grid, smem, st);
    return B == 16 ? launch_page<128, 16>(p, int8, grid, smem, st)
                   : launch_page<128, 32>(p, int8, grid, smem, st);
}

}  // namespace pa
