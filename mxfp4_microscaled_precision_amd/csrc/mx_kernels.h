// Internal launch interface between the C ABI (mx_api.cpp) and the kernels.
// Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>
#include <utility>

namespace mx {

// Launch `kernel` and return that launch's own status (never a sticky error
// left behind by an unrelated earlier HIP call). Arguments are converted to
// the kernel's exact parameter types before their addresses are taken.
template <typename... KArgs, typename... Args>
inline hipError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t shmem,
                         hipStream_t stream, Args... args) {
  static_assert(sizeof...(KArgs) == sizeof...(Args), "kernel argument count");
  std::tuple<KArgs...> params{static_cast<KArgs>(args)...};
  void *ptrs[sizeof...(KArgs)];
  std::apply([&](auto &...p) {
    int i = 0;
    ((ptrs[i++] = static_cast<void *>(&p)), ...);
  }, params);
  return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, ptrs, shmem, stream);
}

enum { MX_K_ROT_NONE = 0, MX_K_ROT_HADAMARD = 1, MX_K_ROT_RAND_SIGN = 2, MX_K_ROT_HADAMARD16 = 3 };
enum { MX_K_ROUND_RNE = 0, MX_K_ROUND_SR = 1 };

struct QuantArgs {
  const uint16_t *x;   // bf16 [rows, cols], leading dimension ld
  int64_t rows, cols, ld;
  int axis;            // 0 or 1
  int rotate, round;
  uint32_t seed_lo, seed_hi;
  uint8_t *codes;      // tiled codes
  uint8_t *scales;     // tiled scales
  int rb;              // axis-0 row blocks per lane (0 = default)
  int fmt;             // 0: E2M1 (MXFP4), 1: E4M3 (MXFP8 comparator, RNE only)
};

hipError_t quantize_launch(const QuantArgs &a, hipStream_t stream);

// Two axis-1 MXFP4 quantizations of sources with the same column count (and
// the same rotation and rounding) in one launch.
hipError_t quantize_pair_launch(const QuantArgs &a, const QuantArgs &b, hipStream_t stream);

// Both orientations of one source (rows % 32 == 0, cols % 32 == 0).
struct DualArgs {
  const uint16_t *x;   // bf16 [rows, cols], leading dimension ld
  int64_t rows, cols, ld;
  int rotate, round;
  uint32_t seed1_lo, seed1_hi;   // axis-1 operand
  uint32_t seed0_lo, seed0_hi;   // axis-0 operand
  uint8_t *codes1, *scales1;
  uint8_t *codes0, *scales0;
};

hipError_t quantize_dual_launch(const DualArgs &a, hipStream_t stream);

// Operands and output of one GEMM of a grouped launch.
struct GemmEntry {
  const uint8_t *a_codes, *a_scales;
  const uint8_t *b_codes, *b_scales;
  void *c;
};

constexpr int kMaxGemmBatch = 4;

struct GemmArgs {
  const uint8_t *a_codes, *a_scales;  // [M][K/2], [M][K/32]
  const uint8_t *b_codes, *b_scales;  // [N][K/2], [N][K/32]
  void *c;                            // [M][N], leading dimension ldc
  int64_t M, N, K, ldc;
  int out_bf16;
  // Set by the launcher: the output tiles (in its ordering) one launch of
  // the MXFP4 GEMM covers, [tile_base, tile_base + tile_count).
  int tile_base, tile_count;
  // Grouped launch (MXFP4 only): `batch` GEMMs of this one shape, entry 0 in
  // the fields above and entry e > 0 in more[e - 1]. Their tile rows are
  // stacked into one tall grid: tile row i of entry e is row e * tiles_m + i.
  int batch = 1;
  GemmEntry more[kMaxGemmBatch - 1] = {};
};

hipError_t gemm_launch(const GemmArgs &g, hipStream_t stream);

// The MXFP8 (E4M3) comparator GEMM on the same tiled operands (2 KB code
// tiles); same arguments.
hipError_t gemm_e4m3_launch(const GemmArgs &g, hipStream_t stream);

// Compute units of the current device (one persistent GEMM workgroup each).
int cu_count();

// fp32 values of a packed operand in its source's shape.
struct DequantArgs {
  const uint8_t *codes, *scales;   // tiled (E2M1 or E4M3 codes)
  int64_t mn, k, mnp, kp;          // operand extents and their padded ones
  int axis;                        // source orientation: 1 -> [mn][k], 0 -> [k][mn]
  int fmt;                         // 0: E2M1, 1: E4M3
  float *out;                      // leading dimension ld
  int64_t ld;
};

hipError_t dequantize_launch(const DequantArgs &a, hipStream_t stream);

// RMS norm into the axis-1 operand and, unless codes0 is null, the axis-0 one
// (rows % 32 == 0).
struct NormArgs {
  const void *x, *residual;        // [rows, cols] bf16 or fp32; residual may be null
  const void *weight;              // [cols] bf16 or fp32
  void *h;                         // x + residual (x itself without a residual)
  float *rstd;                     // [rows]
  int64_t rows, cols, ldx, ldr, ldh;
  int f32, wf32;                   // rows / weight are fp32
  double eps, inv_cols;            // inv_cols = 1 / cols
  int rotate, round, fmt;
  uint32_t seed1_lo, seed1_hi;     // axis-1 operand
  uint32_t seed0_lo, seed0_hi;     // axis-0 operand
  uint8_t *codes1, *scales1;
  uint8_t *codes0, *scales0;
};

hipError_t norm_launch(const NormArgs &a, hipStream_t stream);
// The two-operand case (codes0 != nullptr) of the above.
hipError_t norm_dual_launch(const NormArgs &a, hipStream_t stream);

// Gradient of the norm.
struct NormGradArgs {
  const void *dy, *h, *dres;       // [rows, cols] bf16 or fp32; dres may be null
  const float *rstd;               // [rows]
  const void *weight;              // [cols]
  void *dh;                        // [rows, cols]
  float *dweight;                  // [cols]
  float *partial;                  // [norm_grad_groups(rows, cols)][cols]
  int64_t rows, cols, lddy, ldh, ldres, lddh;
  int f32, wf32;
};

// Workgroups of the gradient's row pass, one partial weight gradient each: 16
// waves to a compute unit where that leaves each at least eight rows, up to 512
// workgroups of them where there are fewer rows (2048 x 8192: 30.8 us with the
// 256 that fit, 36.8 us with 512). A function of the shape alone, so
// that the order of the sums is too.
inline int norm_grad_groups(int64_t rows, int64_t cols) {
  const int64_t waves = cols >= 16 * 512 ? 16 : (cols + 511) / 512;
  const int64_t full = waves > 0 ? 4096 / waves : 4096;
  const int64_t some = full < rows / 8 ? full : rows / 8;
  const int64_t low = full < 512 ? full : 512;
  const int64_t most = some > low ? some : low;
  return (int)(rows < most ? rows : most);
}

// Few rows take one launch without partial rows: 16 x 512 4.0 us (two launches
// 5.2 us), 32 x 512 5.1 (5.2), 1 x 4096 4.9 (5.8), 8 x 4096 5.7 (6.0), 32 x 1024
// 5.9 (5.5), 16 x 4096 6.6 (6.0), 32 x 4096 10.0 (6.2); a call that is not
// captured is 3.7 us shorter on the host by a launch and a workspace.
constexpr int kFewRows = 32;
inline bool norm_grad_few(int64_t rows, int64_t cols) {
  return rows > 0 && rows <= kFewRows && cols <= 4096 && rows * cols <= 32768;
}

hipError_t norm_grad_launch(const NormGradArgs &a, hipStream_t stream);

// Gradient tensors and their chunks, as a table in device memory.
struct GradTensor {
  void *data;
  int64_t rows, cols, ld;          // ld == cols: no gaps
  int64_t f32;                     // fp32, else bf16
};
struct GradChunk {
  uint32_t tensor, at;             // elements [at * chunk, (at + 1) * chunk) of a tensor
};
struct GradTable {
  const GradTensor *tensors;
  const GradChunk *chunk_of;
  int64_t chunks, chunk;
  int64_t bytes;                   // of all tensors
  int64_t once;                    // chunks before this one are not read again soon
};

constexpr int kGradGroups = 1280;  // workgroups, and partial sums, at most

hipError_t grad_norm_launch(const GradTable &t, double *partial, float *norm, hipStream_t stream);
hipError_t grad_clip_launch(const GradTable &in, const GradTable &out, double *partial,
                            float max_norm, float *norm, hipStream_t stream);

}  // namespace mx
