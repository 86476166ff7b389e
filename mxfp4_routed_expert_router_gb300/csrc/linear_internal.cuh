// linear_internal.cuh -- what the files of the linear layers share.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// A call of at most this many tokens streams the FRAG store through the
// warp-level MMAs (linear.cu); more tokens run on the tcgen05 GEMM
// (linear_tc.cu).  Eight tokens fill the columns of a warp-level MMA.  Measured
// (device time in us, this kernel and the GEMM): MXFP4 7168 x 7168 12.4 and 16.0
// for 8 tokens, 17.7 (two MMAs per weight fragment) and 16.3 for 16; group-32 INT4
// 7168 x 18432 33 and 46 for 8, 52 and 46 for 16; BF16 2048 x 7168 10.0 and 9.3 for
// 8, 12.1 and 9.5 for 16.
constexpr int LINEAR_STREAM_MAX_T = 8;

// Operands of the tcgen05 GEMM: FP16 (MXFP4 whose exponents span at most
// TILE_F16_MAX_SPREAD in every row), BF16 (BF16 weights, other MXFP4), FP16 hi +
// lo pairs (group-32 INT4).
enum LinearOp { LIN_F16 = 0, LIN_BF16 = 1, LIN_I4 = 2 };

struct LinearGemm {
    const WeightStore *w;  // TILE-family store of one group
    int fmt, op;
    int N, K, T;
    const void *x;         // BF16 or MXFP8 rows
    const uint8_t *xscales;
    long long x_ld;
    bool x_mx;
    void *y;
    long long y_ld;
    bool y_f32, accumulate;
    uint8_t *workspace;    // linear_gemm_workspace() bytes
    int *err;
};

size_t linear_gemm_workspace(int K, int T);
cudaError_t launch_linear_gemm(const LinearGemm &a, cudaStream_t st);

}  // namespace moe
