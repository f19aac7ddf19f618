// attn_internal.h -- launchers of libsvattention's translation units.
#pragma once

#include "attn_common.cuh"

namespace sva {

// One side (keys or values) of the packed arrays of an append or a read.
struct Packed {
    uint8_t* x[2];
    int64_t token_stride[2], head_stride[2];  // bytes
    int64_t tokens;
    int32_t* status;
};

cudaError_t launch_append(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s);
cudaError_t launch_read(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s);

// Head sizes up to kMaxTileDim.
constexpr int64_t kMaxTileDim = 128;
size_t tiles_workspace(int64_t max_chunk, int64_t G, int64_t D);
cudaError_t launch_attention_tiles(const Attn& a, bool f16, bool e4m3, void* workspace,
                                   cudaStream_t s);

// The same, kFewRows rows of a sequence and key/value head at a time, any head size.
constexpr int64_t kFewRows = 16;
cudaError_t launch_attention_few(const Attn& a, bool f16, bool e4m3, void* workspace,
                                 cudaStream_t s);

// A cache without pages.
cudaError_t launch_attention_no_pages(const Attn& a, bool f16, cudaStream_t s);

}  // namespace sva
