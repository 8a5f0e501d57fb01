// Layer norm and its gradient, bound by memory.  15872 x 4096 bf16 takes 51 us
// forward (5.1 TB/s of the 260 MB it must read and write) and 75 us backward
// (5.2 TB/s of 390 MB); a large device copy reaches 4.8 to 5.0 TB/s.
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
#include <cstdlib>

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

// Rows of any width: a workgroup reads its row three times, the gradient reads x
// and dy once more for the columns' sums (8192 x 16392 bf16 347 us forward, 520
// backward, where 16384 columns take 98 and 161).
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

// ---------------------------------------------------------------------------
// Rows held in registers: a row is read once.
//
// TPR threads share a row (16 or 64: part of a wave or one wave, no barrier;
// 192 and more: a workgroup), each with NCH chunks of 8 consecutive values, so
// a lane's loads and stores are 16 bytes (32 in fp32) at any element address.
// Workgroups stay and walk over the rows, the next row's loads in flight while
// a row is reduced; the weights stay in registers.
// ---------------------------------------------------------------------------
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4 w;
  __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
  // the values, as something the compiler knows nothing about
  __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
  __device__ __forceinline__ void load(const void* p, int64_t i) { w = *(const u32x4a2*)((const bf16_t*)p + i); }
  __device__ __forceinline__ void set(int k, const void* p, int64_t i) {
    const uint32_t v = ((const bf16_t*)p)[i];
    w[k >> 1] = (k & 1) ? (w[k >> 1] & 0xFFFFu) | (v << 16) : (w[k >> 1] & 0xFFFF0000u) | v;
  }
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
  }
};
template <>
struct Raw8<float> {
  f32x4a4 a, b;
  __device__ __forceinline__ void zero() { a = b = f32x4a4{0, 0, 0, 0}; }
  __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(a), "+v"(b)); }
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float* q = (const float*)p + i;
    a = *(const f32x4a4*)q;
    b = *(const f32x4a4*)(q + 4);
  }
  __device__ __forceinline__ void set(int k, const void* p, int64_t i) {
    const float v = ((const float*)p)[i];
    if (k < 4) a[k & 3] = v;
    else b[k & 3] = v;
  }
  __device__ __forceinline__ float get(int k) const { return k < 4 ? a[k & 3] : b[k & 3]; }
};

// A thread's chunk of 8 values of a row: those from column c on, or, where the
// row ends inside them, its last 8, of which the first `skip` are another
// thread's (they are left out of every sum, and stored as the same values).
// Rows narrower than 8 have no such window: their values are fetched one by
// one, and those past the end are 0.  RAGGED: cols is no multiple of 8; else
// every chunk is whole or not there, and no value needs its own test (2 to 5%
// on aligned rows; the windows in place of single values took 4099-wide
// gradients from 103 to 67 us).
template <bool RAGGED>
struct Chunk {
  int c, skip;
  bool any;
  __device__ __forceinline__ Chunk(int first, int cols) {
    any = first < cols;
    c = !RAGGED || first + 8 <= cols || cols < 8 ? first : cols - 8;
    skip = any ? first - c : 8;
  }
  __device__ __forceinline__ bool mine(int k, int cols) const { return RAGGED ? k >= skip && c + k < cols : any; }
};

template <typename T, bool RAGGED>
__device__ __forceinline__ void row_load8(Raw8<T>& r, const void* p, int64_t row0, const Chunk<RAGGED>& h, int cols) {
  if ((!RAGGED || cols >= 8) && h.any) {
    r.load(p, row0 + h.c);
  } else {
    r.zero();
    if (RAGGED && cols < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (h.c + k < cols) r.set(k, p, row0 + h.c + k);
    }
  }
}

__device__ __forceinline__ uint32_t pk2(float lo, float hi) { return bf16_bits(lo) | (bf16_bits(hi) << 16); }

// Stores 8 values; returns the bits of the largest |v| as stored, in fp32.
template <typename T, bool RAGGED>
__device__ __forceinline__ uint32_t row_store8(void* p, int64_t row0, const Chunk<RAGGED>& h, int cols,
                                               const float (&v)[8], bool want) {
  uint32_t mx = 0;
  if (RAGGED && cols < 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (h.c + k < cols) {
        const uint32_t b = st1<T>(p, row0 + h.c + k, v[k]);
        mx = mx > b ? mx : b;
      }
  } else if (h.any) {
    if (sizeof(T) == 2) {
      const u32x4 w = {pk2(v[0], v[1]), pk2(v[2], v[3]), pk2(v[4], v[5]), pk2(v[6], v[7])};
      *(u32x4a2*)((bf16_t*)p + row0 + h.c) = w;
      if (want) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = (w[k] & 0x7FFFu) << 16, hi = w[k] & 0x7FFF0000u;
          mx = mx > lo ? mx : lo;
          mx = mx > hi ? mx : hi;
        }
      }
    } else {
      float* q = (float*)p + row0 + h.c;
      *(f32x4a4*)q = f32x4a4{v[0], v[1], v[2], v[3]};
      *(f32x4a4*)(q + 4) = f32x4a4{v[4], v[5], v[6], v[7]};
      if (want) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
          mx = mx > b ? mx : b;
        }
      }
    }
  }
  return mx;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}
// Sum over 16 consecutive lanes, to each of them (row rotations by 8, 4, 2, 1).
__device__ __forceinline__ float sum16(float v) {
  return dpp_add<0x121>(dpp_add<0x122>(dpp_add<0x124>(dpp_add<0x128>(v))));
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// Sum over the TPR threads of a row; `part`: TPR / 64 floats of this reduction's own.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  if (TPR == 16) return sum16(v);
  v = sum64(v);
  if (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < TPR / 64; ++i) s += part[i];
  return s;
}
// The same for two sums with one barrier.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* part) {
  if (TPR == 16) {
    a = sum16(a);
    b = sum16(b);
    return;
  }
  a = sum64(a);
  b = sum64(b);
  if (TPR == 64) return;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  a = b = 0.0f;
#pragma unroll
  for (int i = 0; i < TPR / 64; ++i) {
    const float2 u = part[i];
    a += u.x;
    b += u.y;
  }
}

// A chunk's weights; `none` where there are none.
template <bool RAGGED>
__device__ __forceinline__ void weights8(float (&v)[8], const void* p, int w_bf16, const Chunk<RAGGED>& h, int cols,
                                         float none) {
  if (p && w_bf16) {
    Raw8<bf16_t> r;
    row_load8(r, p, 0, h, cols);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.get(k);
  } else if (p) {
    Raw8<float> r;
    row_load8(r, p, 0, h, cols);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.get(k);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = none;
  }
}

template <int TPR, bool RAGGED>
struct Chunks {
  int sub, cols;
  __device__ __forceinline__ Chunk<RAGGED> operator[](int j) const { return Chunk<RAGGED>((sub + j * TPR) * 8, cols); }
};

constexpr int norm_threads(int tpr) { return tpr <= 64 ? 256 : tpr; }

template <typename TX, typename TY, int TPR, int NCH, bool RAGGED>
__global__ __launch_bounds__(norm_threads(TPR)) void layernorm_kernel(NormArgs a) {
  constexpr int THR = norm_threads(TPR), RPW = THR / TPR;
  __shared__ float part[3][THR / 64];
  const int sub = threadIdx.x % TPR;
  const Chunks<TPR, RAGGED> at{sub, a.cols};
  const int64_t step = (int64_t)gridDim.x * RPW;
  const float inv = 1.0f / (float)a.cols;
  float gam[NCH][8], bet[NCH][8];
  uint32_t mx = 0;
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  Raw8<TX> next[NCH];
  if (row < a.rows) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) row_load8(next[j], a.x, row * a.ldx, at[j], a.cols);
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    weights8(gam[j], a.gamma, a.w_bf16, at[j], a.cols, 1.0f);
    weights8(bet[j], a.beta, a.w_bf16, at[j], a.cols, 0.0f);
  }
  for (; row < a.rows; row += step) {
    float x[NCH][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[j][k] = next[j].get(k);
        s += at[j].mine(k, a.cols) ? x[j][k] : 0.0f;
      }
    if (row + step < a.rows) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) row_load8(next[j], a.x, (row + step) * a.ldx, at[j], a.cols);
    }
    const float mu = row_sum<TPR>(s, part[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[j][k] -= mu;
        const float d = at[j].mine(k, a.cols) ? x[j][k] : 0.0f;
        s = __builtin_fmaf(d, d, s);
      }
    const float r = 1.0f / sqrtf(__builtin_fmaf(row_sum<TPR>(s, part[1]), inv, a.eps));
    if (sub == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __builtin_fmaf(x[j][k] * r, gam[j][k], bet[j][k]);
      const uint32_t b = row_store8<TY>(a.y, row * a.ldy, at[j], a.cols, y, a.amax != nullptr);
      mx = mx > b ? mx : b;
    }
  }
  if (a.amax) block_amax(mx, a.amax, (uint32_t*)part[2]);
}

template <typename TX, typename TY, int TPR, int NCH, bool RAGGED>
__global__ __launch_bounds__(norm_threads(TPR)) void layernorm_grad_kernel(NormArgs a) {
  constexpr int THR = norm_threads(TPR), RPW = THR / TPR;
  __shared__ float2 part[2][THR / 64];
  __shared__ float fold[RPW > 1 ? THR * 8 : 1];
  const int sub = threadIdx.x % TPR;
  const Chunks<TPR, RAGGED> at{sub, a.cols};
  const int64_t step = (int64_t)gridDim.x * RPW;
  const float inv = 1.0f / (float)a.cols;
  float gam[NCH][8], sg[NCH][8], sb[NCH][8];
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  Raw8<TX> x[NCH], nx[NCH];
  Raw8<TY> dy[NCH], ndy[NCH];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](int64_t q) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      row_load8(nx[j], a.x, q * a.ldx, at[j], a.cols);
      row_load8(ndy[j], a.dy, q * a.ldy, at[j], a.cols);
    }
    nmu = a.mean[q];
    nr = a.rstd[q];
  };
  // 1024 threads have 128 registers each: the next row's values would spill
  // (8192 x 16384, fp32 in and bf16 dy: 483 us with them, 257 without, unpacking
  // again for dx; 3 registers still spill there).  Beyond 8192 columns of fp32 a
  // width that is no multiple of 8, whose window costs registers, spills all the
  // same, 50 of them with 512 x 3 and 143 with 1024 x 2: 15872 x 8201 fp32 403 us
  // (3.9 TB/s) against 290 at 8200, 8192 x 16383 481 us (3.4 TB/s) against 307 at
  // 16384.
  constexpr bool AHEAD = TPR < 1024;
  if (AHEAD && row < a.rows) fetch(row);
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    weights8(gam[j], a.gamma, a.w_bf16, at[j], a.cols, 1.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) sg[j][k] = sb[j][k] = 0.0f;
  }
  int slot = 0;
  for (; row < a.rows; row += step, slot ^= 1) {
    if (!AHEAD) fetch(row);
    const float mu = nmu, r = nr;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      x[j] = nx[j];
      dy[j] = ndy[j];
    }
    if (AHEAD && row + step < a.rows) fetch(row + step);
    float su = 0.0f, sn = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (a chunk that is not there was loaded as zeros; its n is 0 too, as
        // mu r may overflow where the row's own n do not)
        const bool mine = !RAGGED || at[j].mine(k, a.cols);
        const float d = mine ? dy[j].get(k) : 0.0f;
        const float n = RAGGED ? (mine ? (x[j].get(k) - mu) * r : 0.0f) : (x[j].get(k) - (at[j].any ? mu : 0.0f)) * r;
        const float u = d * gam[j][k];
        sg[j][k] = __builtin_fmaf(d, n, sg[j][k]);
        sb[j][k] += d;
        su += u;
        sn = __builtin_fmaf(u, n, sn);
      }
    if (a.dx) {
      row_sum2<TPR>(su, sn, part[slot]);
      su *= inv;
      sn *= inv;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        if (!AHEAD) {
          x[j].opaque();
          dy[j].opaque();
        }
        float d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          d[k] = r * (__builtin_fmaf(-((x[j].get(k) - mu) * r), sn, dy[j].get(k) * gam[j][k]) - su);
        row_store8<TX>(a.dx, row * a.lddx, at[j], a.cols, d, false);
      }
    }
  }
  if (!a.part) return;
  // the workgroup's sums: one strip
  float* pg = a.part + (int64_t)blockIdx.x * a.cols;
  float* pb = pg + (int64_t)a.strips * a.cols;
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = h ? sb[j][k] : sg[j][k];
      if constexpr (RPW > 1) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) fold[k * THR + threadIdx.x] = v[k];
        __syncthreads();
        if (threadIdx.x >= TPR) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          for (int q = 1; q < RPW; ++q) v[k] += fold[k * THR + q * TPR + sub];
      }
      const Chunk<RAGGED> ch = at[j];
      float* to = h ? pb : pg;
      if (!RAGGED || (ch.skip == 0 && a.cols >= 8)) {
        row_store8<float>(to, 0, ch, a.cols, v, false);
      } else {                                         // the columns before `skip` are another thread's sums
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (ch.mine(k, a.cols)) to[ch.c + k] = v[k];
      }
    }
}

// dgamma / dbeta from the strips' partial sums: 32 columns a workgroup, 32
// threads a column, in the strips' order.
constexpr int JOIN_THR = 1024;
__global__ __launch_bounds__(JOIN_THR) void layernorm_dw_join_kernel(const float* part, int strips, int cols,
                                                                     float* dgamma, float* dbeta) {
  __shared__ float sums[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const float* p = part + (int64_t)blockIdx.y * strips * cols + c;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int i = q; i < strips; i += 32) s += p[(int64_t)i * cols];
  }
  sums[q][threadIdx.x & 31] = s;
  __syncthreads();
  if (threadIdx.x < 32 && c < cols) {
    s = 0.0f;
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    out[c] = s;
  }
}

__global__ void norm_fill_kernel(uint32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0u;
}

// Threads a row and chunks of 8 values a thread; 0: the row is too wide for
// registers.  The widest row of a shape is 8 tpr nch; a shape is taken where
// the row fills most of it, as threads without a chunk cost bandwidth, more of
// it the shorter the row is in bytes.  65536 rows of bf16, forward / gradient,
// in us, against the next shape: 16 threads x 2 chunks at 136 and 256 columns
// 13 / 26 and 14 / 29 (64 x 1: 23 / 33 and 24 / 34), 16 x 3 at 320 17 (24), 64 x
// 3 at 1032 and 1280 59 / 84 and 62 / 99 (256 x 1: 93 / 130 and 97 / 132), 192 x
// 2 on 52428 x 2560 110 / 148 (256 x 2: 116, 512 x 1: 211).
//
// The wider the values, the sooner the next shape is the better one, as its
// empty threads cost less and its fuller ones take longer.  Forward, 65536 x
// 1536: bf16 79 by 64 x 3 and 98 by 256 x 1, bf16 to fp32 130 and 116, fp32 166
// and 156.  Gradient: fp32 with bf16 dy, 65536 x 1100 149 by 64 x 3 and 152 by
// 256 x 1, at 1200 159 and 156; 65280 x 2056 266 by 192 x 2 and 279 by 512 x 1, at
// 2304 262 and 256; fp32 with fp32 dy, 65536 x 1032 166 and 162, at 1200 185 and
// 174, 52428 x 2560 298 and 275.
//
// The gradient, which keeps two
// sums a column in registers, takes a row of 4096 by 512 threads (15872 rows:
// 74.6 us; 78.7 with 256 threads of two chunks each), the forward pass, which
// has one more barrier a row, by 256 (50 us; 51 to 62 with 512).  Widths just
// past 4096 would leave the second chunk of 512 threads empty: three chunks of
// 256 threads take 33.9 us on 8192 x 5120 bf16 against 39.8, and 34 against 62
// at 4099; at 6144 they lose, 56.8 against 53.6.  Three chunks of 512 threads
// from 8193 on: 32 us on 4096 x 10240 against 41 with two of 1024.
//
// Workgroups (cap) are few enough that their start (weights, the first row's
// latency) is paid over several rows, and many enough to fill memory's queues.
// Forward: 768 (15872 x 4096 bf16 45.4 us, at 512 48.7; 65536 x 768 fp32 to bf16
// 53 us, at 256 69); from fp32 to fp32, past the 256 MiB of the last-level cache,
// rows of about 4 MiB in flight (65536 x 2048 at 512 183 us, at 768 218; 32768 x
// 4096 at 256 184, at 768 196; but 4096 x 3579 26 and 22.5), where a multiple of
// 256 workgroups of one row each comes within a fifth of that (52428 x 2560 at
// 512 220, at 256 225, at 768 204).
// Gradient: each leaves a strip of sums to be joined: 512 of 256 threads (4099 x
// 1537 fp32 21.6 us, at 768 22.6), 256 of 512.
struct NormShape {
  int tpr, nch, cap;
};
static int norm_rows_per_group(int tpr) { return tpr > 0 && tpr <= 64 ? 256 / tpr : 1; }

static NormShape norm_shape_forward(int64_t rows, int64_t cols, bool x_bf16, bool y_bf16) {
  if (cols > 16384) return {0, 0, 2048};
  if (cols > 12288) return {1024, 2, 512};
  if (cols > 8192) return {512, 3, 256};
  if (cols > 5632) return {512, 2, 256};
  NormShape f = cols <= 128                      ? NormShape{16, 1, 768}
                : cols <= 256                    ? NormShape{16, 2, 1024}
                : cols <= 384                    ? NormShape{16, 3, 1024}
                : cols <= 512                    ? NormShape{64, 1, 768}
                : cols <= 1024                   ? NormShape{64, 2, 768}
                : cols <= (x_bf16 && y_bf16 ? 1536 : 1280) ? NormShape{64, 3, 512}
                : cols <= 2048                   ? NormShape{256, 1, 768}
                : cols <= 2816 && x_bf16         ? NormShape{192, 2, 768}
                : cols <= 4096                   ? NormShape{256, 2, 768}
                                                 : NormShape{256, 3, 768};
  if (!x_bf16 && !y_bf16 && rows > (256ll << 20) / (cols * 4)) {
    const int64_t want = 4 << 20, each = cols * 4 * norm_rows_per_group(f.tpr) * 256;
    const int64_t n = std::min<int64_t>(4, std::max<int64_t>(1, (want + each / 2) / each));
    if (f.tpr <= 64 || 5 * std::abs(n * each - want) <= want) f.cap = 256 * (int)n;
  }
  return f;
}

static NormShape norm_shape_grad(int64_t cols, bool x_bf16, bool dy_bf16) {
  if (cols <= 128) return {16, 1, 768};
  if (cols <= 256) return {16, 2, 512};
  if (cols <= 512) return {64, 1, 512};
  if (cols <= 1024) return {64, 2, 512};
  if (cols <= (x_bf16 ? 1280 : dy_bf16 ? 1152 : 1024)) return {64, 3, 512};
  if (cols <= 2048) return {256, 1, 512};
  if (cols <= (x_bf16 ? 2816 : dy_bf16 ? 2176 : 2048)) return {192, 2, 512};
  if (cols <= 4096) return {512, 1, 256};
  if (cols <= 8192) return {512, 2, 256};
  if (cols <= 12288) return {512, 3, 256};
  if (cols <= 16384) return {1024, 2, 256};
  return {0, 0, 512};
}

static int norm_grid(const NormShape& f, int64_t rows) {
  return (int)std::min<int64_t>(ceil_div(std::max<int64_t>(rows, 1), norm_rows_per_group(f.tpr)), f.cap);
}

// Bytes for the partial column sums of a gradient's strips of rows, one strip
// for each workgroup of its pass, whatever its formats.
static size_t norm_grad_bytes(int64_t rows, int64_t cols) {
  int strips = 0;
  for (int t = 0; t < 4; ++t) strips = std::max(strips, norm_grid(norm_shape_grad(cols, t & 1, t >> 1), rows));
  return (size_t)strips * 2 * (size_t)cols * 4;
}

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

// Whether an output may stand where it does: in an input's place only with the input's type and rows.
static bool norm_in_place(const void* out, pbs_format out_fmt, int64_t ldo, const void* in, pbs_format in_fmt,
                          int64_t ldi, int64_t rows) {
  return out != in || (out_fmt == in_fmt && (rows <= 1 || ldo == ldi));
}

static bool norm_misaligned(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

// One launch of kernel<TX, TY ...> for the call's formats.
#define PBS_NORM_LAUNCH(kernel, grid, thr, a, ...)                                                  \
  do {                                                                                              \
    const dim3 block(thr);                                                                          \
    if (x_fmt == PBS_FMT_BF16 && y_fmt == PBS_FMT_BF16)                                             \
      hipLaunchKernelGGL((kernel<bf16_t, bf16_t __VA_ARGS__>), grid, block, 0, stream, a);          \
    else if (x_fmt == PBS_FMT_BF16)                                                                 \
      hipLaunchKernelGGL((kernel<bf16_t, float __VA_ARGS__>), grid, block, 0, stream, a);           \
    else if (y_fmt == PBS_FMT_BF16)                                                                 \
      hipLaunchKernelGGL((kernel<float, bf16_t __VA_ARGS__>), grid, block, 0, stream, a);           \
    else                                                                                            \
      hipLaunchKernelGGL((kernel<float, float __VA_ARGS__>), grid, block, 0, stream, a);            \
  } while (0)

#define PBS_NORM_COMMA ,
#define PBS_NORM_RAGGED(kernel, grid, thr, a, T, N)                                                 \
  do {                                                                                              \
    if (a.cols % 8) PBS_NORM_LAUNCH(kernel, grid, thr, a, PBS_NORM_COMMA T, N, true);                \
    else PBS_NORM_LAUNCH(kernel, grid, thr, a, PBS_NORM_COMMA T, N, false);                          \
  } while (0)
#define PBS_NORM_CASE(kernel, f, grid, a, T, N) \
  if (f.tpr == T && f.nch == N) PBS_NORM_RAGGED(kernel, grid, norm_threads(T), a, T, N)
// the shapes that both passes use
#define PBS_NORM_SHAPED(kernel, f, grid, a)             \
  do {                                                  \
    PBS_NORM_CASE(kernel, f, grid, a, 16, 1);           \
    else PBS_NORM_CASE(kernel, f, grid, a, 16, 2);      \
    else PBS_NORM_CASE(kernel, f, grid, a, 64, 1);      \
    else PBS_NORM_CASE(kernel, f, grid, a, 64, 2);      \
    else PBS_NORM_CASE(kernel, f, grid, a, 64, 3);      \
    else PBS_NORM_CASE(kernel, f, grid, a, 192, 2);     \
    else PBS_NORM_CASE(kernel, f, grid, a, 256, 1);     \
    else PBS_NORM_CASE(kernel, f, grid, a, 512, 2);     \
    else PBS_NORM_CASE(kernel, f, grid, a, 512, 3);     \
    else PBS_NORM_RAGGED(kernel, grid, 1024, a, 1024, 2); \
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
  PBS_REQUIRE(rows == 0 || norm_in_place(y, y_fmt, ldy, x, x_fmt, ldx, rows), PBS_ERR_INVALID_ARG,
              "pbs_layernorm: y is x with another type or row stride");
  if (amax_out) hipLaunchKernelGGL(norm_fill_kernel, dim3(1), dim3(64), 0, stream, (uint32_t*)amax_out, (int64_t)1);
  if (rows > 0) {
    NormArgs a = {};
    a.x = x; a.gamma = gamma; a.beta = beta; a.w_bf16 = wb == 2;
    a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldy = ldy; a.eps = eps;
    a.y = y; a.mean = mean; a.rstd = rstd; a.amax = (uint32_t*)amax_out;
    const NormShape f = norm_shape_forward(rows, cols, x_fmt == PBS_FMT_BF16, y_fmt == PBS_FMT_BF16);
    const unsigned grid = (unsigned)norm_grid(f, rows);
    log_dispatch("layernorm rows=%lld cols=%lld threads/row=%d chunks=%d grid=%u", (long long)rows, (long long)cols,
                 f.tpr, f.nch, grid);
    if (!f.tpr) PBS_NORM_LAUNCH(layernorm_wide_kernel, dim3(grid), WIDE_THR, a);
    else PBS_NORM_CASE(layernorm_kernel, f, dim3(grid), a, 16, 3);
    else PBS_NORM_CASE(layernorm_kernel, f, dim3(grid), a, 256, 2);
    else PBS_NORM_CASE(layernorm_kernel, f, dim3(grid), a, 256, 3);
    else PBS_NORM_SHAPED(layernorm_kernel, f, dim3(grid), a);
  }
  return check_launch("pbs_layernorm");
}

pbs_status pbs_layernorm_grad_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  PBS_REQUIRE(bytes, PBS_ERR_INVALID_ARG, "pbs_layernorm_grad_bytes: bytes is null");
  PBS_REQUIRE(rows >= 0 && cols >= 1 && cols <= (1 << 24) && rows <= (1ll << 40), PBS_ERR_SHAPE,
              "pbs_layernorm_grad_bytes: needs rows in [0, 2^40] and cols in [1, 2^24] (got %lld x %lld)",
              (long long)rows, (long long)cols);
  *bytes = norm_grad_bytes(rows, cols);
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
  PBS_REQUIRE(rows == 0 || !dx || (norm_in_place(dx, x_fmt, lddx, x, x_fmt, ldx, rows) &&
                                   norm_in_place(dx, x_fmt, lddx, dy, y_fmt, lddy, rows)),
              PBS_ERR_INVALID_ARG, "pbs_layernorm_grad: dx is x or dy with another type or row stride");
  if (rows == 0) {
    if (dgamma) hipLaunchKernelGGL(norm_fill_kernel, dim3(64), dim3(256), 0, stream, (uint32_t*)dgamma, cols);
    if (dbeta) hipLaunchKernelGGL(norm_fill_kernel, dim3(64), dim3(256), 0, stream, (uint32_t*)dbeta, cols);
    return check_launch("pbs_layernorm_grad");
  }
  NormArgs a = {};
  const NormShape f = norm_shape_grad(cols, x_fmt == PBS_FMT_BF16, y_fmt == PBS_FMT_BF16);
  a.strips = norm_grid(f, rows);
  const bool sums = dgamma || dbeta;
  if (sums) {
    PBS_REQUIRE(workspace && ((uintptr_t)workspace & 15) == 0, PBS_ERR_INVALID_ARG,
                "pbs_layernorm_grad: the workspace is null or not 16-byte aligned");
    const size_t need = norm_grad_bytes(rows, cols);
    PBS_REQUIRE(workspace_bytes >= need, PBS_ERR_INVALID_ARG,
                "pbs_layernorm_grad: the workspace holds %zu bytes, pbs_layernorm_grad_bytes asks for %zu",
                workspace_bytes, need);
  }
  a.x = x; a.dy = dy; a.gamma = gamma; a.w_bf16 = w_fmt == PBS_FMT_BF16;
  a.rows = rows; a.cols = (int)cols; a.ldx = ldx; a.ldy = lddy; a.lddx = lddx;
  a.mean = (float*)mean; a.rstd = (float*)rstd; a.dx = dx; a.part = (float*)workspace;
  log_dispatch("layernorm_grad rows=%lld cols=%lld threads/row=%d chunks=%d strips=%d", (long long)rows,
               (long long)cols, f.tpr, f.nch, a.strips);
  if (!sums) a.part = nullptr;
  PBS_NORM_CASE(layernorm_grad_kernel, f, dim3(a.strips), a, 512, 1);
  else if (f.tpr) PBS_NORM_SHAPED(layernorm_grad_kernel, f, dim3(a.strips), a);
  else if (sums) {
    PBS_NORM_LAUNCH(layernorm_dw_wide_kernel, dim3((unsigned)ceil_div(cols, WIDE_THR), a.strips), WIDE_THR, a);
  }
  if (sums)
    hipLaunchKernelGGL(layernorm_dw_join_kernel, dim3((unsigned)ceil_div(cols, 32), 2), dim3(JOIN_THR), 0, stream,
                       a.part, a.strips, a.cols, dgamma, dbeta);
  // last: dx may take the place of x or dy
  if (!f.tpr && dx)
    PBS_NORM_LAUNCH(layernorm_dx_wide_kernel, dim3((unsigned)std::min<int64_t>(rows, 2048)), WIDE_THR, a);
  return check_launch("pbs_layernorm_grad");
}

}  // extern "C"
