// Layer norm and its gradient.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), n = (x - mu) r
//   y  = n gamma + beta
// and with u = dy gamma, means taken over a row's columns:
//   dx = r (u - mean(u) - n mean(u n))
//   dgamma = sum_rows dy n,   dbeta = sum_rows dy
//
// The mean is subtracted before squaring (a second pass over the row), so a
// large common offset costs no digits; every sum is held in fp32.
#include "device.hpp"
#include "host.hpp"

#include <algorithm>

namespace pbs {

struct NormArgs {
  const void* x;
  const void* dy;       // gradient only
  const void* gamma;    // may be null: 1
  const void* beta;     // may be null: 0
  int w_bf16;
  int64_t rows, ldx, ldy;
  int cols;
  float eps;
  void* y;
  float* mean;
  float* rstd;
  uint32_t* amax;
  void* dx;
  int64_t lddx;
  float* part;          // [2][strips][cols]: partial sums of dgamma, dbeta
  int strips;
};

template <typename T>
__device__ __forceinline__ float ld1(const void* p, int64_t i);
template <>
__device__ __forceinline__ float ld1<bf16_t>(const void* p, int64_t i) {
  return bf16_to_float(((const bf16_t*)p)[i]);
}
template <>
__device__ __forceinline__ float ld1<float>(const void* p, int64_t i) {
  return ((const float*)p)[i];
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Stores v and returns the bits of |v| as stored, in fp32.
template <typename T>
__device__ __forceinline__ uint32_t st1(void* p, int64_t i, float v);
template <>
__device__ __forceinline__ uint32_t st1<bf16_t>(void* p, int64_t i, float v) {
  const uint32_t b = bf16_bits(v);
  ((bf16_t*)p)[i] = (bf16_t)b;
  return (b & 0x7FFFu) << 16;
}
template <>
__device__ __forceinline__ uint32_t st1<float>(void* p, int64_t i, float v) {
  ((float*)p)[i] = v;
  return __float_as_uint(v) & 0x7FFFFFFFu;
}

__device__ __forceinline__ float ldw(const void* p, int i, int w_bf16, float none) {
  if (!p) return none;
  return w_bf16 ? ld1<bf16_t>(p, i) : ld1<float>(p, i);
}

constexpr int WIDE_THR = 256;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the workgroup, to every thread; `part` is this reduction's own.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < WIDE_THR / 64; ++i) s += part[i];
  return s;
}

__device__ __forceinline__ void block_amax(uint32_t m, uint32_t* out, uint32_t* part) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t u = (uint32_t)__shfl_xor((int)m, o, 64);
    m = m > u ? m : u;
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < (int)(blockDim.x >> 6); ++i) m = m > part[i] ? m : part[i];
    const uint32_t cur = __builtin_nontemporal_load(out);
    if (m > cur) atomicMax(out, m);
  }
}

// Rows of any width: a workgroup reads its row three times.
template <typename TX, typename TY>
__global__ __launch_bounds__(WIDE_THR) void layernorm_wide_kernel(NormArgs a) {
  __shared__ float part[3][WIDE_THR / 64];
  uint32_t mx = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t ox = row * a.ldx, oy = row * a.ldy;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += WIDE_THR) s += ld1<TX>(a.x, ox + c);
    const float mu = block_sum(s, part[0]) / (float)a.cols;
    s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += WIDE_THR) {
      const float d = ld1<TX>(a.x, ox + c) - mu;
      s += d * d;
    }
    const float r = 1.0f / sqrtf(block_sum(s, part[1]) / (float)a.cols + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
    for (int c = threadIdx.x; c < a.cols; c += WIDE_THR) {
      const float n = (ld1<TX>(a.x, ox + c) - mu) * r;
      const uint32_t b =
          st1<TY>(a.y, oy + c, n * ldw(a.gamma, c, a.w_bf16, 1.0f) + ldw(a.beta, c, a.w_bf16, 0.0f));
      mx = mx > b ? mx : b;
    }
  }
  if (a.amax) block_amax(mx, a.amax, (uint32_t*)part[2]);
}

template <typename TX, typename TY>
__global__ __launch_bounds__(WIDE_THR) void layernorm_dx_wide_kernel(NormArgs a) {
  __shared__ float part[2][WIDE_THR / 64];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t ox = row * a.ldx, oy = row * a.ldy, od = row * a.lddx;
    const float mu = a.mean[row], r = a.rstd[row];
    float su = 0.0f, sn = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += WIDE_THR) {
      const float u = ld1<TY>(a.dy, oy + c) * ldw(a.gamma, c, a.w_bf16, 1.0f);
      su += u;
      sn += u * ((ld1<TX>(a.x, ox + c) - mu) * r);
    }
    su = block_sum(su, part[0]) / (float)a.cols;
    sn = block_sum(sn, part[1]) / (float)a.cols;
    for (int c = threadIdx.x; c < a.cols; c += WIDE_THR) {
      const float u = ld1<TY>(a.dy, oy + c) * ldw(a.gamma, c, a.w_bf16, 1.0f);
      const float n = (ld1<TX>(a.x, ox + c) - mu) * r;
      st1<TX>(a.dx, od + c, r * (u - su - n * sn));
    }
  }
}

// Partial column sums of a strip of rows: a thread owns one column.
template <typename TX, typename TY>
__global__ __launch_bounds__(WIDE_THR) void layernorm_dw_wide_kernel(NormArgs a) {
  const int c = blockIdx.x * WIDE_THR + threadIdx.x;
  if (c >= a.cols) return;
  const int64_t r0 = a.rows * blockIdx.y / a.strips, r1 = a.rows * (blockIdx.y + 1) / a.strips;
  float sg = 0.0f, sb = 0.0f;
  for (int64_t row = r0; row < r1; ++row) {
    const float dy = ld1<TY>(a.dy, row * a.ldy + c);
    sg += dy * ((ld1<TX>(a.x, row * a.ldx + c) - a.mean[row]) * a.rstd[row]);
    sb += dy;
  }
  a.part[(int64_t)blockIdx.y * a.cols + c] = sg;
  a.part[(int64_t)(a.strips + blockIdx.y) * a.cols + c] = sb;
}

// dgamma / dbeta from the strips' partial sums, in the strips' order.
__global__ __launch_bounds__(WIDE_THR) void layernorm_dw_join_kernel(const float* part, int strips, int cols,
                                                                     float* dgamma, float* dbeta) {
  const int c = blockIdx.x * WIDE_THR + threadIdx.x;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (c >= cols || !out) return;
  const float* p = part + (int64_t)blockIdx.y * strips * cols + c;
  float s = 0.0f;
  for (int i = 0; i < strips; ++i) s += p[(int64_t)i * cols];
  out[c] = s;
}

__global__ void norm_fill_kernel(uint32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0u;
}

static int norm_strips(int64_t rows) { return (int)std::min<int64_t>(std::max<int64_t>(rows, 1), 512); }

}  // namespace pbs

using namespace pbs;

static pbs_status norm_check(const char* what, pbs_format x_fmt, pbs_format y_fmt, pbs_format w_fmt, int64_t rows,
                             int64_t cols, const void* x, int64_t ldx, const void* y, int64_t ldy) {
  PBS_REQUIRE((x_fmt == PBS_FMT_BF16 || x_fmt == PBS_FMT_F32) && (y_fmt == PBS_FMT_BF16 || y_fmt == PBS_FMT_F32) &&
                  (w_fmt == PBS_FMT_BF16 || w_fmt == PBS_FMT_F32),
              PBS_ERR_UNSUPPORTED, "%s: formats must be BF16 or F32", what);
  PBS_REQUIRE(rows >= 0 && cols >= 1 && cols <= (1 << 24) && rows <= (1ll << 40), PBS_ERR_SHAPE,
              "%s: needs rows in [0, 2^40] and cols in [1, 2^24] (got %lld x %lld)", what, (long long)rows,
              (long long)cols);
  PBS_REQUIRE(ldx >= cols && ldy >= cols && ldx <= (1ll << 40) && ldy <= (1ll << 40), PBS_ERR_SHAPE,
              "%s: row strides must be in [cols, 2^40]", what);
  if (rows == 0) return PBS_OK;
  PBS_REQUIRE(x && y, PBS_ERR_INVALID_ARG, "%s: null tensor", what);
  PBS_REQUIRE(((uintptr_t)x & (x_fmt == PBS_FMT_BF16 ? 1 : 3)) == 0 &&
                  ((uintptr_t)y & (y_fmt == PBS_FMT_BF16 ? 1 : 3)) == 0,
              PBS_ERR_INVALID_ARG, "%s: tensors must be aligned to their elements", what);
  return PBS_OK;
}

static bool norm_misaligned(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

#define PBS_NORM_LAUNCH(kernel, grid, thr, a)                                                       \
  do {                                                                                              \
    if (x_fmt == PBS_FMT_BF16) {                                                                    \
      if (y_fmt == PBS_FMT_BF16) hipLaunchKernelGGL((kernel<bf16_t, bf16_t>), grid, dim3(thr), 0, stream, a); \
      else hipLaunchKernelGGL((kernel<bf16_t, float>), grid, dim3(thr), 0, stream, a);              \
    } else {                                                                                        \
      if (y_fmt == PBS_FMT_BF16) hipLaunchKernelGGL((kernel<float, bf16_t>), grid, dim3(thr), 0, stream, a); \
      else hipLaunchKernelGGL((kernel<float, float>), grid, dim3(thr), 0, stream, a);               \
    }                                                                                               \
  } while (0)

extern "C" {

pbs_status pbs_layernorm(const void* x, pbs_format x_fmt, int64_t rows, int64_t cols, int64_t ldx,
                         const void* gamma, const void* beta, pbs_format w_fmt, float eps, void* y,
                         pbs_format y_fmt, int64_t ldy, float* mean, float* rstd, float* amax_out,
                         hipStream_t stream) {
  const pbs_status st = norm_check("pbs_layernorm", x_fmt, y_fmt, w_fmt, rows, cols, x, ldx, y, ldy);
  if (st != PBS_OK) return st;
  const int wb = w_fmt == PBS_FMT_BF16 ? 2 : 4;
  PBS_REQUIRE(eps >= 0.0f && eps <= 3.4e38f, PBS_ERR_INVALID_ARG, "pbs_layernorm: eps must be finite and >= 0");
  PBS_REQUIRE(!norm_misaligned(gamma, wb) && !norm_misaligned(beta, wb) && !norm_misaligned(mean, 4) &&
                  !norm_misaligned(rstd, 4) && !norm_misaligned(amax_out, 4),
              PBS_ERR_INVALID_ARG, "pbs_layernorm: a vector is not aligned to its elements");
  if (amax_out) hipLaunchKernelGGL(norm_fill_kernel, dim3(1), dim3(64), 0, stream, (uint32_t*)amax_out, (int64_t)1);
  if (rows > 0) {
    NormArgs a = {};
    a.x = x; a.gamma = gamma; a.beta = beta; a.w_bf16 = wb == 2;
    a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldy = ldy; a.eps = eps;
    a.y = y; a.mean = mean; a.rstd = rstd; a.amax = (uint32_t*)amax_out;
    const int grid = (int)std::min<int64_t>(rows, 2048);
    log_dispatch("layernorm_wide rows=%lld cols=%lld grid=%d", (long long)rows, (long long)cols, grid);
    PBS_NORM_LAUNCH(layernorm_wide_kernel, dim3(grid), WIDE_THR, a);
  }
  return check_launch("pbs_layernorm");
}

pbs_status pbs_layernorm_grad_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  PBS_REQUIRE(bytes, PBS_ERR_INVALID_ARG, "pbs_layernorm_grad_bytes: bytes is null");
  PBS_REQUIRE(rows >= 0 && cols >= 1 && cols <= (1 << 24) && rows <= (1ll << 40), PBS_ERR_SHAPE,
              "pbs_layernorm_grad_bytes: needs rows in [0, 2^40] and cols in [1, 2^24] (got %lld x %lld)",
              (long long)rows, (long long)cols);
  *bytes = (size_t)norm_strips(rows) * 2 * (size_t)cols * 4;
  return PBS_OK;
}

pbs_status pbs_layernorm_grad(const void* dy, pbs_format y_fmt, int64_t lddy, const void* x, pbs_format x_fmt,
                              int64_t ldx, int64_t rows, int64_t cols, const void* gamma, pbs_format w_fmt,
                              const float* mean, const float* rstd, void* dx, int64_t lddx, float* dgamma,
                              float* dbeta, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const pbs_status st = norm_check("pbs_layernorm_grad", x_fmt, y_fmt, w_fmt, rows, cols, x, ldx, dy, lddy);
  if (st != PBS_OK) return st;
  PBS_REQUIRE(!dx || (lddx >= cols && lddx <= (1ll << 40)), PBS_ERR_SHAPE,
              "pbs_layernorm_grad: row strides must be in [cols, 2^40]");
  PBS_REQUIRE(rows == 0 || (mean && rstd), PBS_ERR_INVALID_ARG, "pbs_layernorm_grad: mean or rstd is null");
  PBS_REQUIRE(!norm_misaligned(gamma, w_fmt == PBS_FMT_BF16 ? 2 : 4) &&
                  !norm_misaligned(dx, x_fmt == PBS_FMT_BF16 ? 2 : 4) && !norm_misaligned(mean, 4) &&
                  !norm_misaligned(rstd, 4) && !norm_misaligned(dgamma, 4) && !norm_misaligned(dbeta, 4),
              PBS_ERR_INVALID_ARG, "pbs_layernorm_grad: a tensor is not aligned to its elements");
  if (rows == 0) {
    if (dgamma) hipLaunchKernelGGL(norm_fill_kernel, dim3(64), dim3(256), 0, stream, (uint32_t*)dgamma, cols);
    if (dbeta) hipLaunchKernelGGL(norm_fill_kernel, dim3(64), dim3(256), 0, stream, (uint32_t*)dbeta, cols);
    return check_launch("pbs_layernorm_grad");
  }
  NormArgs a = {};
  a.strips = norm_strips(rows);
  const bool sums = dgamma || dbeta;
  if (sums) {
    PBS_REQUIRE(workspace && ((uintptr_t)workspace & 15) == 0, PBS_ERR_INVALID_ARG,
                "pbs_layernorm_grad: the workspace is null or not 16-byte aligned");
    PBS_REQUIRE(workspace_bytes >= (size_t)a.strips * 2 * (size_t)cols * 4, PBS_ERR_INVALID_ARG,
                "pbs_layernorm_grad: the workspace holds %zu bytes, pbs_layernorm_grad_bytes asks for %zu",
                workspace_bytes, (size_t)a.strips * 2 * (size_t)cols * 4);
  }
  a.x = x; a.dy = dy; a.gamma = gamma; a.w_bf16 = w_fmt == PBS_FMT_BF16;
  a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldy = lddy; a.lddx = lddx;
  a.mean = (float*)mean; a.rstd = (float*)rstd; a.dx = dx; a.part = (float*)workspace;
  const unsigned cb = (unsigned)ceil_div(cols, WIDE_THR);
  log_dispatch("layernorm_grad_wide rows=%lld cols=%lld strips=%d", (long long)rows, (long long)cols, a.strips);
  if (sums) {
    PBS_NORM_LAUNCH(layernorm_dw_wide_kernel, dim3(cb, a.strips), WIDE_THR, a);
    hipLaunchKernelGGL(layernorm_dw_join_kernel, dim3(cb, 2), dim3(WIDE_THR), 0, stream, a.part, a.strips, a.cols,
                       dgamma, dbeta);
  }
  // last: dx may take the place of x or dy
  if (dx) PBS_NORM_LAUNCH(layernorm_dx_wide_kernel, dim3((unsigned)std::min<int64_t>(rows, 2048)), WIDE_THR, a);
  return check_launch("pbs_layernorm_grad");
}

}  // extern "C"
