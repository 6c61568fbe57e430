// The decode kernel's forms for 8-bit pages with a scale per (block, kv head).
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
