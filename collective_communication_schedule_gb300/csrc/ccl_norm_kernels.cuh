// The norm's kernels of one pair of types, one translation unit a type.
#pragma once

#include <vector>

#include "ccl_norm.cuh"

namespace ccl {
namespace tensor {

// Kernels for rows on 16 bytes and for any others, from the narrowest up, then
// for rows of any length.
struct NormKernels {
    struct Forward {
        int64_t width;             // elements of the longest row
        int threads, rows;         // of a threadblock
        void (*kernel)(const Norm);
        int blocks;                // an SM in the grid, which take rows in turn; 0: as many as the rows need
        int smem, stage;           // bytes of shared memory, and where rows of y lie apart
    };
    struct Backward {
        int64_t width;
        int threads, across;       // of a threadblock, of a row
        int pieces, each;          // of a thread, elements of one
        void (*kernel)(const Norm);
    };
    std::vector<Forward> forward[2];
    Backward backward[2][6];
    void (*forward_long)(const Norm);
    void (*backward_long)(const Norm);
    void (*sums_long)(const Norm);
    void (*sums)(const Norm);
};

template <int T, int TW>
NormKernels norm_kernels_of()
{
    // (f32: half the elements a piece, twice the pieces)
    // Forward, the narrowest that holds a row, with 2 to 4 pieces of 16 bytes a thread on
    // their way.  bf16, us with the next wider form instead: 20000 x 1024 12.8 and 22.1,
    // 8192 x 2048 11.7 and 13.8, 8192 x 4096 22.1 and 42.2 (in 512 threads of 2
    // pieces; 8192 columns in them 29.2, in 256 threads of 4 23.0), 1000 x 32768 33.9 and,
    // read three times, 60.8.
    constexpr int W = Type<T>::kVec, M = 8 / W;
#define FORWARD(tpr, v, vec) {(tpr) * (v) * ((vec) ? W : 1), (tpr) < 128 ? 128 : (tpr), (tpr) < 128 ? 128 / (tpr) : 1, norm_kernel_rows<T, TW, tpr, v, vec>}
#define SHIFTED(tpr, v)                                                                                            \
    {(tpr) * (v) * W - (W - 1), kShiftedThreads, kShiftedThreads / (tpr), norm_kernel_shifted<T, TW, tpr, v>,          \
     shifted_blocks((v) * W), 8 * W * plane_of<W, tpr, v>(), kShiftedThreads * (v) * 16}
    // Backward, likewise.  us: rows of 16-bit elements in 512 threads of 2 or 4 pieces or in
    // 1024 of half as many, 8192 x 8192 81.2 and 84.6, 8192 x 12288 133 and 248, 8192 x 4096
    // 43.0 and 42.2, 20000 x 1024 28.8 and 27.7; f32 8192 x 4096 89.4 and 71.1; element by
    // element, 10 a thread or 5, 8191 x 2057 bf16 34.2 and 40.9, f32 42.2 and 48.9,
    // 4097 x 4097 37.7 and 48.2.  The last form of single elements, 8 for each of 1024
    // threads with 64 registers, spills 290 bytes a thread (4097 x 7001 bf16 123 us, 1.4
    // TB/s), those of 5 for 1024 threads 40 to 48.  Wider rows, f32 and single elements
    // from 8193 columns on and 16-bit ones from 16385, are read three times by
    // elements: f32 4096 x 8192 65 us (6.2 TB/s), 4096 x 8196 151 (2.7), 2048 x 16384 147.
    constexpr int D = W == 8 ? 512 : 1024;
#define BACKWARD(threads, across, v, vec) {(across) * (v) * ((vec) ? W : 1), threads, across, v, (vec) ? W : 1, norm_grad_kernel_rows<T, TW, threads, across, v, vec>}
    NormKernels k = {
        {{FORWARD(32, M, true), FORWARD(32, 4 * M, true), FORWARD(128, 2 * M, true), FORWARD(128, 4 * M, true),
          FORWARD(256, 4 * M, true), FORWARD(512, 4 * M, true), FORWARD(1024, 4 * M, true)}},
        {{BACKWARD(1024, 32, 1, true), BACKWARD(1024, 128, 1, true), BACKWARD(1024, 256, 1, true), BACKWARD(1024, 512, 1, true),
          BACKWARD(D, D, 1024 / D, true), BACKWARD(512, 512, 4, true)},
         {BACKWARD(1024, 32, 5, false), BACKWARD(1024, 128, 5, false), BACKWARD(512, 128, 10, false), BACKWARD(512, 256, 10, false),
          BACKWARD(512, 512, 10, false), BACKWARD(1024, 1024, 8, false)}},
        norm_kernel_long<T, TW>,
        norm_grad_kernel_long<T, TW>,
        norm_sums_kernel_long<T>,
        norm_sums_kernel<TW>};
    if constexpr (T == CCL_F32)
        k.forward[1] = {FORWARD(32, 4, false), FORWARD(32, 16, false), FORWARD(128, 16, false), FORWARD(256, 10, false),
                        FORWARD(256, 16, false), FORWARD(512, 16, false), FORWARD(1024, 16, false)};
    else
        k.forward[1] = {FORWARD(32, 4, false), SHIFTED(32, 3), SHIFTED(128, 3), SHIFTED(256, 3), SHIFTED(256, 5), FORWARD(1024, 16, false)};
#undef FORWARD
#undef SHIFTED
#undef BACKWARD
    return k;
}

}  // namespace tensor
}  // namespace ccl
