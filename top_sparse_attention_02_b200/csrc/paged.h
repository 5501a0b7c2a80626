// paged.h -- host-side launchers of the paged-cache kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.h"

namespace tsa {

constexpr int kMaxGroup = 16;     // query heads per kv-head that the paged attention takes
constexpr int kPageRows = 16;     // a page holds a multiple of this many rows
constexpr int kMaxPrefixSplits = 128;  // partials of a shared prefix's pass a row
constexpr int kPartFloats = 132;  // a partial of one head: acc[128], M, L, 2 pad (528 B)

// A cache in pages: row j of (sequence b, kv-head h) lies in page
// table[b][j / page_size], at element page * page_stride + h * head_stride +
// (j % page_size) * row_stride of K and of V.
struct Pages {
    void* K = nullptr;
    void* V = nullptr;
    const int32_t* table = nullptr;  // [B][width]
    long long page_stride = 0, head_stride = 0, row_stride = 0;
    int num_pages = 0, page_size = 0, width = 0, B = 0, Hkv = 0, half = 0;  // half: fp16 elements, else bf16
    // rows a sequence's table can name (as far as int32 row numbers reach)
    __host__ __device__ int rows_cap() const {
        const long long r = (long long)width * page_size;
        return r > 0x7fffffc0LL ? 0x7fffffc0 : (int)r;
    }
};

struct Rotation {
    const double* inv_freq = nullptr;  // [rot_dim / 2] radians a position
    int rot_dim = 0, interleaved = 0;
};

struct Heads {  // [T][H][128], strides in elements
    const void* p = nullptr;
    long long st = 0, sh = 0;
};

cudaError_t launch_qk_norm_rope(const Heads& q, const Heads& k, const Heads& qo, const Heads& ko, int T, int Hq, int Hkv,
                                int half, const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const Rotation& rot, cudaStream_t st);

cudaError_t launch_paged_append(const Pages& c, const Heads& k, const Heads& v, int T, const int32_t* seq,
                                const int32_t* row, const int32_t* positions, const Rotation& rot, unsigned* flag,
                                cudaStream_t st);

// Partials of a shared prefix's pass: [splits][B][Hq][kPartFloats], counted only
// for the sequences that hold the whole prefix (len >= prefix_len); and room for
// those of each sequence's own rows.
struct PrefixParts {
    float* parts = nullptr;
    float* own = nullptr;  // [B][Hq][kPartFloats]
    int splits = 0, prefix_len = 0;
};

// the shared prefix's pass into parts [prefix_max_splits][B][Hq][kPartFloats]; fills *out for the paged attention after it
int prefix_max_splits(int Hkv, int rows, int prefix_len);  // rows = B * Hq / Hkv; grows with prefix_len
cudaError_t launch_prefix(const Pages& c, const void* Q, int Hq, const int32_t* lens, int prefix_len, float scale,
                          float* parts, PrefixParts* out, unsigned* flag, cudaStream_t st);

int paged_ctas();  // CTAs of the paged attention's grid
cudaError_t launch_paged_attn(const Pages& c, const void* Q, int Hq, const int32_t* lens, const int32_t* idx,
                              const int32_t* kreq, int k_max, float scale, void* O, float* lse, float* pieces,
                              const PrefixParts& pre, unsigned* flag, cudaStream_t st);

}  // namespace tsa
