// linear_internal.cuh -- what the files of the linear layers share.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// A call of at most this many tokens streams the FRAG store through the
// warp-level MMAs (linear.cu); more tokens, and MXFP4 weights with scales outside
// LINEAR_STREAM_MIN_E8M0 .. MAX_E8M0, run on the tcgen05 GEMM (linear_tc.cu).  INT4
// weights whose scales the GEMM's FP16 operands do not hold run here in slices of
// this many tokens, each of which reads the weights once.  Eight tokens fill the columns of a warp-level MMA.  Measured
// (device time in us, weights from HBM, 8 tokens here and 9 in the GEMM): MXFP4
// 7168 x 7168 10.8 and 14.1, 7168 x 18432 21.2 and 26.4; group-32 INT4 7168 x 18432
// 25.0 and 46 (F32 rows 51); BF16 256 x 7168 3.8 and 6.6, 2048 x 7168 8.4 and 8.7,
// 7168 x 7168 19.0 and 19.0.  Sixteen tokens here would take two MMAs per weight
// fragment (measured with the weights in L2): MXFP4 7168 x 7168 17.7 (the GEMM 13.0),
// 36864 x 7168 55 (33); INT4 7168 x 18432 52 (46, F32 rows 52).
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
