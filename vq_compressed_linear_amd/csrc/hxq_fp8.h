// The 8-bit path: device helpers and launchers shared by its kernels.
//
// An 8-bit tensor holds e4m3 values (OCP: largest 448, no infinities).
// Activations carry one power of two for each 128 columns of a row, weights
// one for each 128 x 128 block, as e8m0 bytes (2^(byte - 127)): the form in
// which the matrix cores take an operand's block scale, so the products need
// no multiplication by scales on the vector ALUs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hxq {

constexpr int kFp8Block = 128;

inline int64_t fp8_padded(int64_t k) { return (k + 127) / 128 * 128; }       // bytes of a row of k values
inline int64_t fp8_scale_row(int64_t k) { return (k + 511) / 512 * 4; }      // bytes of its row of scales

// ------------------------------------------------------------ row operators

struct NormArgs {
  const void* x;          // [M][K]
  const void* residual;   // [M][K] or nullptr
  const float* weight;    // [K] or nullptr (ones)
  void* sum_out;          // [M][K], the residual's type, or nullptr
  void* out;              // [M][K], or [M][Kp] e4m3
  uint8_t* scales;        // [M][Gs] (e4m3 output)
  float* rstd;            // [M] or nullptr
  float eps;
  int64_t M;
  int K;
  int x_dtype, res_dtype, out_dtype;  // res_dtype: -1 without a residual
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
  const void* dy;         // [M][K]
  const void* h;          // [M][K]
  const float* weight;    // [K] or nullptr
  const float* rstd;      // [M]
  const float* dsum;      // [M][K] or nullptr
  float* dx;              // [M][K]
  float* dweight;         // [K] or nullptr
  float* part;            // [norm_bwd_parts()][K] when dweight
  int64_t M;
  int K;
  int dy_dtype, h_dtype;
};
int64_t norm_bwd_parts(int64_t M, int64_t K);  // partial rows of the weight's gradient
hipError_t launch_rms_norm_bwd(const NormBwdArgs& a, hipStream_t stream);

hipError_t launch_quant_rows(const void* x, int x_dtype, uint8_t* q, uint8_t* scales, int64_t M, int K,
                             hipStream_t stream);
hipError_t launch_quant_weight(const void* w, int w_dtype, uint8_t* q, uint8_t* scales, uint8_t* qt,
                               uint8_t* scales_t, int64_t E, int64_t N, int64_t K, hipStream_t stream);

// ------------------------------------------------------------- the products

struct Fp8Args {
  const uint8_t* x;        // [Mx][Kp] e4m3
  const uint8_t* xs;       // [Mx][Gs]
  const void* xf;          // [Mx][K] float32 or bf16, where the kernel converts x itself
  int x_dtype;             // its type then, else HXQ_E4M3
  const int32_t* rows;     // [M] row of x for each row of y, or nullptr (the row itself); experts only
  const int32_t* offsets;  // [E + 1] first row of each expert, or nullptr (one layer)
  const uint8_t* w;        // [E][N][Kp] e4m3
  const uint8_t* ws;       // [E][ceil(N / 128)][Gs]
  const float* bias;       // [E][N] or nullptr
  void* y;                 // [M][N]
  int y_bf16;
  float* part;             // [S][M][N] partial sums when S > 1
  int64_t Mx;
  int M, N, K, Kp, Gs, E;
  int S, kbs;              // splits of the sum, 128-blocks in each
};

// How a product is run (host): which kernel, and how its sum is split.
struct Fp8Plan {
  int kernel;       // one of Fp8Kernel
  bool wide;        // operands widened to bf16 (tile kernels)
  bool converts;    // the kernel converts a float32 or bf16 x itself
  int waves, depth; // skinny kernel: waves that share a tile's sum, blocks of a wave in flight
  int S, kbs;
  int64_t tiles_m, tiles_n;
  int64_t part_bytes;
  bool ok;          // the tiles can be numbered in 31 bits
};
enum Fp8Kernel { kFp8Skinny, kFp8Tile32, kFp8Tile64, kFp8Tile128, kFp8Tile256 };

hipError_t launch_fp8_skinny(const Fp8Args& a, const Fp8Plan& p, hipStream_t stream);
hipError_t launch_fp8_tile(const Fp8Args& a, const Fp8Plan& p, hipStream_t stream);
hipError_t launch_fp8_sum(const Fp8Args& a, hipStream_t stream);

}  // namespace hxq
