// Orthogonalisation of a matrix by Newton-Schulz products and Muon's update of a
// weight with it.  With m = min(rows, cols), n the other one, X taken as [m, n]:
//
//   M' = beta M + (1 - beta) G,  U = beta M' + (1 - beta) G (Nesterov) or M'
//   X = U / (||U||_F + eps)
//   A = X X^T,  P = b A + c A^2,  X' = a X + P X         for each step (a, b, c)
//   W' = (1 - lr decay) W - lr scale X
//
// Number formats.  The products run on fp16 operands and add in fp32.  Every X,
// A and P is bounded (the singular values of X start within [0, 1] and the
// steps' polynomials keep them within a bound that the host computes), so one
// power of two for the whole call puts them into fp16's range, whose three
// more bits of mantissa than bf16's make the roundings 8 times smaller at the same
// rate.  What remains of them:
//  * Small singular directions grow by `a` a step next to large ones that stay
//    near 1, and with them what X's rounding adds.  X is therefore kept as a pair,
//    hi + lo 2^-11, of which the sum enters a X and only hi the products: an error
//    of hi there is multiplied by P, which is small but in the large directions.
//    A matrix of eight directions 30 times above its noise: error 4% of the
//    result with hi alone, 0.08% with the pair (bf16 alone: 34%).
//  * P's diagonal, near b + c, is much larger than the rest of its row and
//    cancels against a: it is kept apart in fp32 and joins a in a X (a random
//    matrix 0.17% -> 0.05 to 0.1%).
// They move the result by 0.01 to 0.2% (Frobenius norm) beside its own rounding to bf16
// (0.17%), and by up to 1% where one direction stands thousands of times above the rest:
// there A's entries are nearly alike, and half a step of them outweighs the others' part.
//
// A and P are symmetric: the tiles on and below the diagonal are formed and
// stored twice, once transposed.
//
// Where the longer side exceeds the shorter, steps are taken two and two: with R =
// X X^T and q = a I + b R + c R^2 of one step, the next step's R is q R q and its X
// is q' q X, so the long side is gone through once a pair and not once a step.  A
// step alone takes 3 m^2 n + m^3 multiplications (symmetric products by half),
// two together 3 m^2 n + 5 m^3: 16384 x 4096 in five steps 3.38 ms where one by one
// takes 4.45.  R's rounding errors grow by
// q^2 until X X^T is formed anew, which is why no more go together (ns_pairs).
#include "device.hpp"
#include "gemm_common.hpp"
#include "host.hpp"
#include "mfma_tile.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace pbs {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16_t;
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float NS_LO = 2048.0f;           // a pair's lo is held times this
constexpr int NS_PART = 2048;              // most partial sums of a matrix's norm

// ---------------------------------------------------------------------------
// Momentum, norm and the first X
// ---------------------------------------------------------------------------
struct MuonIn {
  const void* g;           // gradient, or the matrix to orthogonalise
  void* m;                 // momentum; may be null: U = G
  int64_t ldg, sg, ldm, sm;// row and batch strides, elements
  int rows, cols;          // of the weight
  int g_bf16, m_bf16, g_transposed, nesterov;
  float beta, one_less;    // one_less: 1 - beta
  int mp, np, tall;        // X: [mp][np], the matrix transposed if tall
  int parts;
  double* part;            // [batch][parts]
  float eps, scale;
  uint8_t *hi, *lo;        // [batch][mp][np] fp16
};

template <typename T> __device__ __forceinline__ float muon_get(const void* p, int64_t i);
template <> __device__ __forceinline__ float muon_get<bf16_t>(const void* p, int64_t i) { return bf16_to_float(((const bf16_t*)p)[i]); }
template <> __device__ __forceinline__ float muon_get<float>(const void* p, int64_t i) { return ((const float*)p)[i]; }

// Four values of a row from column c on; those at or past cols are 0.
template <typename T>
__device__ __forceinline__ float4 muon_get4(const T* row, int c, int cols, bool vec) {
  if (vec && c + 4 <= cols) {
    if constexpr (sizeof(T) == 4) return *(const float4*)(row + c);
    else {
      const uint2 u = *(const uint2*)(row + c);
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xFFFF0000u));
    }
  }
  float4 v;
  v.x = c < cols ? muon_get<T>(row, c) : 0.0f;
  v.y = c + 1 < cols ? muon_get<T>(row, c + 1) : 0.0f;
  v.z = c + 2 < cols ? muon_get<T>(row, c + 2) : 0.0f;
  v.w = c + 3 < cols ? muon_get<T>(row, c + 3) : 0.0f;
  return v;
}
template <typename T>
__device__ __forceinline__ void muon_put4(T* row, int c, int cols, bool vec, float4 v) {
  if constexpr (sizeof(T) == 4) {
    if (vec && c + 4 <= cols) { *(float4*)(row + c) = v; return; }
    if (c < cols) row[c] = v.x;
    if (c + 1 < cols) row[c + 1] = v.y;
    if (c + 2 < cols) row[c + 2] = v.z;
    if (c + 3 < cols) row[c + 3] = v.w;
  } else {
    const uint32_t lo = pk_bf16(v.x, v.y), hi = pk_bf16(v.z, v.w);
    if (vec && c + 4 <= cols) { *(uint2*)(row + c) = make_uint2(lo, hi); return; }
    if (c < cols) row[c] = (bf16_t)lo;
    if (c + 1 < cols) row[c + 1] = (bf16_t)(lo >> 16);
    if (c + 2 < cols) row[c + 2] = (bf16_t)hi;
    if (c + 3 < cols) row[c + 3] = (bf16_t)(hi >> 16);
  }
}
// Four aligned values as they lie in memory.
template <typename T>
struct MuonQuad {
  typedef typename std::conditional<sizeof(T) == 4, u32x4, u32x2>::type raw;
  raw v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    if constexpr (sizeof(T) == 4) v = __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    else v = __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
  }
  // keep * them - step * x
  __device__ __forceinline__ float4 moved(float keep, float step, float4 x) const {
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (sizeof(T) == 4) o[i] = __uint_as_float(v[i]);
      else o[i] = __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    return make_float4(keep * o[0] - step * x.x, keep * o[1] - step * x.y, keep * o[2] - step * x.z, keep * o[3] - step * x.w);
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t at, float4 x) {
    if constexpr (sizeof(T) == 4)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, at, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{pk_bf16(x.x, x.y), pk_bf16(x.z, x.w)}, r, at, 0, 0);
  }
};
template <typename T>
__device__ __forceinline__ bool muon_vec(const void* p, int64_t ld, int64_t batch_stride) {
  return (((uintptr_t)p & (4 * sizeof(T) - 1)) | (uint64_t)(ld & 3) | (uint64_t)(batch_stride & 3)) == 0;
}

// All waves meet with their LDS work done; loads and stores stay in flight
// (__syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// (Each product and sum is rounded by itself, as the formulas stand: a momentum
// kept in bf16 then comes out as any fp32 evaluation of them has it.  A value
// rounded the other way, 2^-8 of it, may move the small directions of the next
// step's X by as much as they are.)
// A 64 x 64 tile of U: thread t holds four values of the rows t / 16 + 16 k
// from column 4 (t % 16) on.  m4: M', for the momentum's store.
constexpr int MT = 64, MPITCH = 65;
template <typename TG, typename TM>
struct MuonTile {
  float4 u[4], m4[4];
  __device__ __forceinline__ void load(const MuonIn& a, int batch, int r0, int c0, float (*lds)[MPITCH]) {
    const int t = threadIdx.x, tr = t >> 4, tc = 4 * (t & 15);
    const TG* g = (const TG*)a.g + batch * a.sg;
    const bool vg = muon_vec<TG>(a.g, a.ldg, a.sg);
    // the momentum's loads first: they are in flight while the gradient is turned
    float4 gv[4], o4[4];
    if (a.m) {
      const TM* m = (const TM*)a.m + batch * a.sm;
      const bool vm = muon_vec<TM>(a.m, a.ldm, a.sm);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + tr + 16 * k;
        o4[k] = r < a.rows ? muon_get4<TM>(m + r * a.ldm, c0 + tc, a.cols, vm) : make_float4(0, 0, 0, 0);
      }
    }
    if (a.g_transposed) {
      float4 turned[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = tr + 16 * k;
        turned[k] = c0 + c < a.cols ? muon_get4<TG>(g + (c0 + c) * a.ldg, r0 + tc, a.rows, vg) : make_float4(0, 0, 0, 0);
      }
      lds_barrier();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = tr + 16 * k;
        lds[tc][c] = turned[k].x; lds[tc + 1][c] = turned[k].y; lds[tc + 2][c] = turned[k].z; lds[tc + 3][c] = turned[k].w;
      }
      lds_barrier();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* p = &lds[tr + 16 * k][tc];
        gv[k] = make_float4(p[0], p[1], p[2], p[3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + tr + 16 * k;
        gv[k] = r < a.rows ? muon_get4<TG>(g + r * a.ldg, c0 + tc, a.cols, vg) : make_float4(0, 0, 0, 0);
      }
    }
    if (!a.m) {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = gv[k];
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 o = o4[k];
      const float4 s = make_float4(a.one_less * gv[k].x, a.one_less * gv[k].y, a.one_less * gv[k].z, a.one_less * gv[k].w);
      float4 n;
      n.x = a.beta * o.x + s.x; n.y = a.beta * o.y + s.y; n.z = a.beta * o.z + s.z; n.w = a.beta * o.w + s.w;
      m4[k] = n;
      if (a.nesterov) {
        n.x = a.beta * n.x + s.x; n.y = a.beta * n.y + s.y; n.z = a.beta * n.z + s.z; n.w = a.beta * n.w + s.w;
      }
      u[k] = n;
    }
  }
};

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Partial sums of U's squares in 64 bits (gradients of 1e-25 or 1e25 square past
// fp32), a fixed set of tiles a workgroup.
template <typename TG, typename TM>
__global__ __launch_bounds__(256) void muon_norm_kernel(MuonIn a) {
  __shared__ float lds[MT][MPITCH];
  __shared__ double sums[4];
  const int tc = (a.cols + MT - 1) / MT, tr = (a.rows + MT - 1) / MT;
  double s = 0.0;
  for (int64_t i = blockIdx.x; i < (int64_t)tc * tr; i += a.parts) {
    MuonTile<TG, TM> t;
    t.load(a, blockIdx.y, (int)(i / tc) * MT, (int)(i % tc) * MT, lds);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double x = t.u[k].x, y = t.u[k].y, z = t.u[k].z, w = t.u[k].w;
      s += x * x + y * y + (z * z + w * w);
    }
  }
  s = wave_sum_d(s);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.part[(int64_t)blockIdx.y * a.parts + blockIdx.x] = sums[0] + sums[1] + (sums[2] + sums[3]);
}

// x as hi + lo 2^-11 in fp16.
__device__ __forceinline__ void ns_split(float x, f16_t& hi, f16_t& lo) {
  hi = (f16_t)x;
  lo = (f16_t)((x - (float)hi) * NS_LO);
}

// The momentum's store and the first X, zeros past the matrix's end.  Tiles in
// reverse, eight at a time (so each stays on its XCD): the norm's pass has left the
// last ones in the caches (16384 x 4096 193 -> 178 us).
template <typename TG, typename TM>
__global__ __launch_bounds__(256) void muon_start_kernel(MuonIn a) {
  __shared__ float lds[MT][MPITCH];
  __shared__ double sums[4];
  const int t = threadIdx.x, tr = t >> 4, tc = 4 * (t & 15);
  const int batch = gridDim.y - 1 - blockIdx.y;
  double s = 0.0;
#pragma unroll 8
  for (int i = t; i < a.parts; i += 256) s += a.part[(int64_t)batch * a.parts + i];
  s = wave_sum_d(s);
  if ((t & 63) == 0) sums[t >> 6] = s;
  __syncthreads();
  const double norm = sqrt(sums[0] + sums[1] + (sums[2] + sums[3])) + (double)a.eps;
  // a matrix of zeros stays one; one with an infinity or a NaN becomes NaN
  const double f = norm == 0.0 ? 0.0 : norm < __builtin_inf() ? (double)a.scale / norm : __builtin_nan("");
  const int wr = a.tall ? a.np : a.mp, wc = a.tall ? a.mp : a.np;           // the weight's padded shape
  const int tiles_c = wc / MT;
  const int id = blockIdx.x, whole = gridDim.x / NXCD * NXCD;
  const int tile = id < whole ? whole - NXCD - id / NXCD * NXCD + id % NXCD : id;
  const int r0 = tile / tiles_c * MT, c0 = tile % tiles_c * MT;
  if (r0 >= wr) return;
  MuonTile<TG, TM> u;
  u.load(a, batch, r0, c0, lds);
  if (a.m) {
    TM* m = (TM*)a.m + batch * a.sm;
    const bool vm = muon_vec<TM>(a.m, a.ldm, a.sm);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + tr + 16 * k;
      if (r < a.rows) muon_put4<TM>(m + r * a.ldm, c0 + tc, a.cols, vm, u.m4[k]);
    }
  }
  if (a.tall) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float* p = &lds[tr + 16 * k][tc];
      p[0] = u.u[k].x; p[1] = u.u[k].y; p[2] = u.u[k].z; p[3] = u.u[k].w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      u.u[k] = make_float4(lds[tc][tr + 16 * k], lds[tc + 1][tr + 16 * k], lds[tc + 2][tr + 16 * k], lds[tc + 3][tr + 16 * k]);
  }
  const int x0 = a.tall ? c0 : r0, y0 = a.tall ? r0 : c0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t at = ((int64_t)batch * a.mp + x0 + tr + 16 * k) * a.np + y0 + tc;
    f16x4 h, l;
    const float v[4] = {(float)(u.u[k].x * f), (float)(u.u[k].y * f), (float)(u.u[k].z * f), (float)(u.u[k].w * f)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f16_t hh, ll;
      ns_split(v[e], hh, ll);
      h[e] = hh;
      l[e] = ll;
    }
    *(f16x4*)((f16_t*)a.hi + at) = h;
    *(f16x4*)((f16_t*)a.lo + at) = l;
  }
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
// The products.  Symmetric, by half: A = X X^T; P from A^2; T = (D + P) R; Q from P
// Q'.  Whole: the next X, and the last one into the weight.
enum { NS_GRAM = 0, NS_POLY = 1, NS_TURN = 2, NS_JOIN = 3, NS_STEP = 4, NS_LAST = 5 };
constexpr bool ns_symmetric(int mode) { return mode < NS_STEP; }

struct NsArgs {
  const uint8_t *hi, *lo;  // X
  uint8_t *hi2, *lo2;      // the next X
  // symmetric products: operands [batch][mp][mp] fp16, of which src1 and src2 enter the
  // sum by row1 (its row's value, times f1) and col2 (its column's, times f2)
  const uint8_t *left, *right, *src1, *src2;
  const float *row1, *col2;
  float f1, f2, f;         // f: the product's own factor
  uint8_t* out;
  float* diag;             // the result's diagonal, [batch][mp]; whole products: Q's
  const uint8_t* q;        // whole products: Q without its diagonal
  int mp, np, batch;
  int tiles_m, tiles_n, per; // tiles of a matrix
  float a;
  float inv;               // 1 / the power of two that X is held times
  // the last step: to y, or into the weight
  void* w;
  int64_t ldw, sw;
  int rows, cols;          // of the weight
  int w_bf16, tall, update;
  float lr, decay, scale;  // W' = (1 - lr decay) W - lr scale X
  const float* lr_by;      // may be null: 1
};

// A tile has 64 T x 64 T outputs; wave (wm, wn) holds its 32 x 32 tiles
// (2 i + wm, 2 j + wn), i, j < T.
template <int T> constexpr int ns_pitch() { return 128 * T + 16; }      // staged rows of fp16
template <int T> constexpr int ns_pitch4() { return 256 * T + 16; }     // and of fp32
constexpr int NS_TALL_PITCH = 68;                                       // floats: staged columns of 64 rows
// D: stages that loads are ahead of the products
template <int T> constexpr int ns_smem(int mode, int d) {
  return cmax((2 * d + 1) * tile_bytes<T>(), mode == NS_GRAM ? 64 * T * ns_pitch<T>()
                                   : mode == NS_LAST ? 128 * ns_pitch<T>() + 64 * T * NS_TALL_PITCH * 4
                                                     : 256 * ns_pitch<T>());
}

template <int T>
struct NsHalf {
  i32x4 x[T][2];
};
template <int LD, int T> constexpr int ns_reads() { return LD == KMAJ ? 2 * T : 4 * T; }

// LDS read d of half H of a stage.  K-major: the row's chunk 4 H + 2 part + lg
// under its swizzle key, which for row 32 (2 i + w) + lr is the lane's XOR
// 2 (2 i + w).  MN-major: the transposing read of 4 K rows.
template <int H, int LD, int T>
__device__ __forceinline__ void ns_read(NsHalf<T>& f, int d, const uint8_t* base, uint32_t lb) {
  if (LD == KMAJ) {
    const int tile = d >> 1, part = d & 1;
    f.x[tile][part] = *(const i32x4*)(base + tile * 8192 + (lb ^ (uint32_t)(((4 * H) ^ ((4 * tile) & 7)) << 4) ^
                                                            (uint32_t)(part << 5)));
  } else {
    const int tile = d >> 2, s = (d >> 1) & 1, q = d & 1;
    const i16x4 v = read_lds_tr16(base + (16 * (2 * H + s) + 4 * q) * (128 * T) + (lb ^ (uint32_t)(128 * tile)));
    const int2 w2 = __builtin_bit_cast(int2, v);
    if (q == 0) {
      f.x[tile][s].x = w2.x;
      f.x[tile][s].y = w2.y;
    } else {
      f.x[tile][s].z = w2.x;
      f.x[tile][s].w = w2.y;
    }
  }
}

// Tile `id` of the lower triangle of tiles: rows walked four together, so that
// neighbours in time share operand rows.
__device__ __forceinline__ void ns_triangle(int id, int n, int& row, int& col) {
  int g = (int)((sqrtf(4.0f + 32.0f * (float)id) - 2.0f) * 0.0625f);      // 8 g^2 + 2 g tiles lie ahead of group g
  while (g > 0 && 8 * g * g + 2 * g > id) --g;
  while (8 * (g + 1) * (g + 1) + 2 * (g + 1) <= id) ++g;
  int in = id - 8 * g * g - 2 * g;
  const int have = n - 4 * g < 4 ? n - 4 * g : 4;
  if (in < 4 * g * have) {
    row = 4 * g + in % have;
    col = in / have;
    return;
  }
  in -= 4 * g * have;
  int c = 0;
  while (in >= have - c) in -= have - c++;
  col = 4 * g + c;
  row = col + in;
}

// The last stages but one.
template <int LEFT, typename Body>
__device__ __forceinline__ void ns_tail(int nk, Body& body) {
  if constexpr (LEFT > 1) {
    if (nk >= LEFT) body(nk - LEFT, std::integral_constant<int, LEFT>{});
    ns_tail<LEFT - 1>(nk, body);
  }
}

template <int T, int D, int MODE, typename TW>
__global__ __launch_bounds__(256, T >= 3 ? 1 : (T == 2 ? 4 : 8) / D) void ns_product_kernel(NsArgs g) {
  __shared__ __align__(16) uint8_t smem[ns_smem<T>(MODE, D)];
  constexpr int LDA = MODE >= NS_STEP ? MNMAJ : KMAJ;
  constexpr int TILE = 64 * T;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w >> 1, wn = w & 1;

  // XCD b % 8 takes a contiguous range of the matrices' tiles
  const int total = g.per * g.batch;
  const int x = (int)blockIdx.x % NXCD, share = total / NXCD, left = total % NXCD;
  const int id = x * share + (x < left ? x : left) + (int)blockIdx.x / NXCD;
  const int mat = id / g.per;
  int tm, tn;
  if constexpr (MODE >= NS_STEP) {
    const int in = id - mat * g.per, group = GROUP_M * g.tiles_n, q = in / group;
    const int gm = g.tiles_m - q * GROUP_M < GROUP_M ? g.tiles_m - q * GROUP_M : GROUP_M, r = in - q * group;
    tm = q * GROUP_M + r % gm;
    tn = r / gm;
  } else {
    ns_triangle(id - mat * g.per, g.tiles_n, tn, tm);
  }
  const int m0 = tm * TILE, n0 = tn * TILE;
  const int64_t xs = (int64_t)mat * g.mp * g.np, ps = (int64_t)mat * g.mp * g.mp;    // a matrix's X; its A and P
  // M, the results' contiguous axis, and the contraction's stages
  const int M = MODE >= NS_STEP ? g.np : g.mp, nk = (MODE == NS_GRAM ? g.np : g.mp) / 64;

  auto tileA = [&](int kt) { return smem + kt % D * tile_bytes<T>(); };
  auto tileB = [&](int kt) { return smem + D * tile_bytes<T>() + kt % (D + 1) * tile_bytes<T>(); };

  f32x16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  typename std::conditional<LDA == KMAJ, KLoad<T>, MnLoad<T == 3 ? 4 : T>>::type la;
  KLoad<T> lb;
  if constexpr (MODE == NS_GRAM) {
    la.init(g.hi + 2 * xs, (int64_t)g.np * 2, m0, g.mp, w);
    lb.init(g.hi + 2 * xs, (int64_t)g.np * 2, n0, g.mp, w);
  } else if constexpr (ns_symmetric(MODE)) {
    la.init(g.right + 2 * ps, (int64_t)g.mp * 2, m0, g.mp, w);
    lb.init(g.left + 2 * ps, (int64_t)g.mp * 2, n0, g.mp, w);
  } else {
    la.init(g.hi + 2 * xs, (int64_t)g.np * 2, m0, g.np, g.mp, w);
    lb.init(g.q + 2 * ps, (int64_t)g.mp * 2, n0, g.mp, w);
  }

  const int lr = lane & 31, lg = lane >> 5;
  const int jj = (lr & 15) >> 2;
  const uint32_t kb = (uint32_t)(lr * 128 + ((lg ^ swz_key(lr)) << 4));
  const uint32_t fba = LDA == KMAJ ? kb ^ (uint32_t)(wm << 5)
                                   : (uint32_t)((8 * lg + jj) * (128 * T) + ((64 * (T == 1 ? jj >> 1 : jj)) ^ (64 * wm)) + 32 * (lr >> 4) +
                                                16 * ((lr & 3) >> 1) + 8 * (lr & 1));
  const uint32_t fbb = kb ^ (uint32_t)(wn << 5);
  const int offA = LDA == KMAJ ? wm * 4096 : 0, offB = wn * 4096;

  constexpr int NMFMA = 2 * T * T, OVER = NMFMA * 3 / 4, NL = 2 * T;
  constexpr int RA = ns_reads<LDA, T>(), RB = ns_reads<KMAJ, T>();
  NsHalf<T> a0, a1, b0, b1;
  auto load_a = [&](int kt, int v) { la.load(kt, 0, tileA(kt), w, v); };
  auto load_b = [&](int kt, int v) { lb.load(kt, 0, tileB(kt), w, v); };
  auto mfma = [&](const NsHalf<T>& a, const NsHalf<T>& b, int m) {
    const int s = m / (T * T), i = (m / T) % T, j = m % T;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a.x[i][s]),
                                                       __builtin_bit_cast(f16x8, b.x[j][s]), acc[i][j], 0, 0, 0);
  };

#pragma unroll
  for (int k = 0; k < D; ++k)
    if (k < nk) {
#pragma unroll
      for (int v = 0; v < NL; ++v) load_a(k, v);
#pragma unroll
      for (int v = 0; v < NL; ++v) load_b(k, v);
    }
  if (nk >= D) stage_barrier<(D - 1) * 2 * NL>();
  else stage_barrier<0>();
#pragma unroll
  for (int d = 0; d < RA; ++d) ns_read<0, LDA, T>(a0, d, tileA(0) + offA, fba);
#pragma unroll
  for (int d = 0; d < RB; ++d) ns_read<0, KMAJ, T>(b0, d, tileB(0) + offB, fbb);

  // A's stages go through D LDS buffers, B's through D + 1, so that the loads of
  // stage kt + D spread over the whole of stage kt: B's while the first half of
  // the stage is multiplied, A's, into the buffer that was just read out, while
  // the second is.  LEFT: stages from this one on, D + 1 if more than D, which
  // are then loaded ahead.
  auto body = [&](int kt, auto left_c) {
    constexpr int LEFT = decltype(left_c)::value;
    constexpr bool ISSUE = LEFT > D, NEXT = LEFT > 1;
    const uint8_t* curA = tileA(kt) + offA;
    const uint8_t* curB = tileB(kt) + offB;
    const uint8_t* nxtA = tileA(kt + 1) + offA;
    const uint8_t* nxtB = tileB(kt + 1) + offB;
#pragma unroll
    for (int m = 0; m < NMFMA; ++m) {
      mfma(a0, b0, m);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = part_lo(RA + RB, OVER, m); d < part_hi(RA + RB, OVER, m); ++d) {
        if (d < RA) ns_read<1, LDA, T>(a1, d, curA, fba);
        else ns_read<1, KMAJ, T>(b1, d - RA, curB, fbb);
      }
      if (ISSUE) {
#pragma unroll
        for (int v = part_lo(NL, NMFMA, m); v < part_hi(NL, NMFMA, m); ++v) load_b(kt + D, v);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // (the last stage's loads were waited for in the one before; what is in flight then is the epilogue's)
    if constexpr (ISSUE) stage_barrier<(D - 2) * 2 * NL + NL>();
    else if constexpr (NEXT) stage_barrier<(LEFT - 2) * 2 * NL>();
    else lds_barrier();
    constexpr int NDS = NEXT ? RA + RB : 0;
#pragma unroll
    for (int m = 0; m < NMFMA; ++m) {
      mfma(a1, b1, m);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = part_lo(NDS, OVER, m); d < part_hi(NDS, OVER, m); ++d) {
        if (d < RA) ns_read<0, LDA, T>(a0, d, nxtA, fba);
        else ns_read<0, KMAJ, T>(b0, d - RA, nxtB, fbb);
      }
      if (ISSUE) {
#pragma unroll
        for (int v = part_lo(NL, NMFMA, m); v < part_hi(NL, NMFMA, m); ++v) load_a(kt + D, v);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int kt = 0; kt < nk - D; ++kt) body(kt, std::integral_constant<int, D + 1>{});
  ns_tail<D>(nk, body);
  // The epilogue's sources of 64 rows, A or X's pair, a pass ahead in
  // registers: the first behind the last stage's products.
  constexpr int CHUNKS = 8 * T, PER = 2 * T;                  // 16-byte chunks a row, and a thread in 64 rows
  const uint8_t* src = ns_symmetric(MODE) ? g.src1 + 2 * ps : g.hi + 2 * xs;
  const uint8_t* src2 = ns_symmetric(MODE) ? g.src2 + 2 * ps : g.lo + 2 * xs;
  u32x4 v1[PER], v2[PER];
  auto fetch = [&](int j) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int at = t + 256 * k;
      const int r = n0 + 64 * j + at / CHUNKS, c = m0 + 8 * (at % CHUNKS);
      const int64_t o = 2 * ((int64_t)(r < g.mp ? r : g.mp - 1) * M + (c < M ? c : M - 8));
      v1[k] = *(const u32x4*)(src + o);
      if constexpr (MODE >= NS_JOIN) v2[k] = *(const u32x4*)(src2 + o);
    }
  };
  if constexpr (MODE != NS_GRAM && MODE != NS_LAST) fetch(0);
  const int srow = 32 * wn + lr;                              // the lane's row of 64
  float own[T];                                               // Q's or row1's value there
  if constexpr (MODE >= NS_TURN) {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const int row = n0 + 64 * j + srow;
      own[j] = (ns_symmetric(MODE) ? g.row1 : g.diag)[(int64_t)mat * g.mp + (row < g.mp ? row : g.mp - 1)];
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  body(nk - 1, std::integral_constant<int, 1>{});

  // Every LDS read of the loop finished before its last barrier, and no load to
  // LDS is in flight.  acc[i][j][4 q + r] is row n0 + 32 (2 j + wn) + lr, column m0 + 32
  // (2 i + wm) + 8 q + 4 lg + r.  The results are staged 64 rows at a time (those
  // of one j) and stored from there in whole rows.
  constexpr int PITCH = ns_pitch<T>(), PITCH4 = ns_pitch4<T>();
  auto scol = [&](int i, int q) { return 32 * (2 * i + wm) + 8 * q + 4 * lg; };
  // Stores go through buffer resources that begin at the tile's first row and end
  // with the matrix, and what lies past its columns is sent past that end: the
  // hardware drops it.  (Behind a condition the compiler no longer knows how many
  // stores are in flight and waits for all of them ahead of the next pass's
  // sources.)
  constexpr uint32_t NOWHERE = 0xFFFFFFF0u;
  auto rows_of = [](uint8_t* p, int first, int rows, int64_t ld) {
    return buffer_rows(p + 2 * first * ld, (uint32_t)(2 * (rows - first) * ld < 0xFFFFFFF0ll ? 2 * (rows - first) * ld : 0xFFFFFFF0ll));
  };
  // 64 staged rows from the tile's row r0 on, of a matrix with ld columns
  auto store_rows = [&](const uint8_t* from, const BufferRows& to, int r0, int64_t ld) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int at = t + 256 * k, r = at / CHUNKS, c = at % CHUNKS;
      const u32x4 v = *(const u32x4*)(from + r * PITCH + 16 * c);
      const uint32_t o = (uint32_t)(r0 + r) * (uint32_t)(2 * ld) + (uint32_t)(2 * (m0 + 8 * c));
      __builtin_amdgcn_raw_buffer_store_b128(v, to.r, m0 + 8 * c < M ? o : NOWHERE, 0, 0);
    }
  };
  // and transposed: 8 rows of 16 columns at a time, by the transposing read
  auto store_transposed = [&](const uint8_t* from, const BufferRows& to, int r0) {
    const int gq = lane >> 4, li = lane & 15;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int block = w + 4 * k, c0 = 16 * (block >> 1), o = 8 * (4 * (block & 1) + gq);
      const uint8_t* p = from + (o + (li >> 2)) * PITCH + 2 * (c0 + 4 * (li & 3));
      const u32x2 lo = __builtin_bit_cast(u32x2, read_lds_tr16(p));
      const u32x2 hi = __builtin_bit_cast(u32x2, read_lds_tr16(p + 4 * PITCH));
      const uint32_t at = (uint32_t)(c0 + li) * (uint32_t)(2 * g.mp) + (uint32_t)(2 * (n0 + r0 + o));
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo.x, lo.y, hi.x, hi.y}, to.r, n0 + r0 + o < g.mp ? at : NOWHERE, 0, 0);
    }
  };

  if constexpr (MODE == NS_GRAM) {
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f16x4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = (f16_t)(acc[i][j][4 * q + r] * g.f);
          *(f16x4*)(smem + (64 * j + srow) * PITCH + 2 * scol(i, q)) = v;
        }
    lds_barrier();
    const BufferRows to = rows_of(g.out + 2 * ps, n0, g.mp, g.mp), over = rows_of(g.out + 2 * ps, m0, g.mp, g.mp);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      store_rows(smem + 64 * j * PITCH, to, 64 * j, g.mp);
      if (tm != tn) store_transposed(smem + 64 * j * PITCH, over, 64 * j);
    }
  } else {
    constexpr int AREA = 64 * PITCH;
    const BufferRows to1 = ns_symmetric(MODE) ? rows_of(g.out + 2 * ps, n0, g.mp, g.mp) : rows_of(g.hi2 + 2 * xs, n0, g.mp, g.np);
    const BufferRows to2 = ns_symmetric(MODE) ? rows_of(g.out + 2 * ps, m0, g.mp, g.mp) : rows_of(g.lo2 + 2 * xs, n0, g.mp, g.np);
    // The last step: four values of a row of the weight at a time, QPT a thread
    // and pass.  A tall weight's rows are the tile's columns, which are then
    // staged as rows.  Value 4 of step k in pass j lies k * krows rows on from the
    // thread's first, and j * 64 rows (columns, if tall).
    constexpr int QUADS = 16 * T, QPT = 64 * QUADS / 256, AHEAD = sizeof(TW) == 2 || QPT < 2 ? QPT : QPT / 2;
    const float lr_now = MODE == NS_LAST && g.lr_by ? g.lr * *g.lr_by : g.lr;
    const float keep = 1.0f - lr_now * g.decay, step = g.update ? lr_now * g.scale : -1.0f;
    const int row_step = g.tall ? 1 : PITCH4 / 4, col_step = g.tall ? NS_TALL_PITCH : 1;      // of the staged fp32
    const int krows = g.tall ? 16 : 256 / QUADS, kstage = g.tall ? 16 * NS_TALL_PITCH : 256 / QUADS * (PITCH4 / 4);
    const int first = g.tall ? (t >> 4) * NS_TALL_PITCH + 4 * (t & 15) : t / QUADS * (PITCH4 / 4) + 4 * (t % QUADS);
    const int w0 = g.tall ? m0 : n0, qrow = g.tall ? t >> 4 : t / QUADS, wcol = g.tall ? n0 + 4 * (t & 15) : m0 + 4 * (t % QUADS);
    // whole quads of rows that one buffer resource reaches
    const int64_t ldb = g.ldw * (int64_t)sizeof(TW);
    const bool quads = g.cols % 4 == 0 && muon_vec<TW>(g.w, g.ldw, g.sw) && 256 * ldb < 0x7FFFFFFFll;
    TW* const weight = (TW*)g.w + mat * g.sw + w0 * g.ldw;                // the tile's first row
    BufferRows wb;
    {
      const int64_t have = ((int64_t)(g.rows - w0 - 1) * g.ldw + g.cols) * (int64_t)sizeof(TW);
      wb = buffer_rows((const uint8_t*)weight, (uint32_t)(have < 0 ? 0 : have < 0xFFFFFFF0ll ? have : 0xFFFFFFF0ll));
    }
    const uint32_t ldb32 = (uint32_t)ldb;
    auto w_at = [&](int j, int k) {
      const int c = wcol + (g.tall ? 64 * j : 0), r = qrow + k * krows + (g.tall ? 0 : 64 * j);
      return quads && c < g.cols && w0 + r < g.rows ? (uint32_t)r * ldb32 + (uint32_t)(c * (int)sizeof(TW)) : NOWHERE;
    };
    MuonQuad<TW> old[AHEAD];
    auto fetch_w = [&](int j, int from) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) old[k].load(wb.r, g.update ? w_at(j, from + k) : NOWHERE);
    };
    auto put_w = [&](int j, int from, const float* f) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        float4 v = *(const float4*)(f + first + (from + k) * kstage);
        v = old[k].moved(keep, step, v);                       // (no update: 0 and x)
        MuonQuad<TW>::store(wb.r, w_at(j, from + k), v);
      }
    };
#pragma unroll
    for (int j = 0; j < T; ++j) {
      uint8_t* s1 = smem + (MODE == NS_LAST ? 0 : (j & 1) * 2 * AREA);
      uint8_t* s2 = s1 + AREA;
      // (the last step has the weight to fetch ahead: with X's pair a pass ahead too,
      // registers spill, and a spilled load is waited for, 10 us a pass)
      if constexpr (MODE == NS_LAST) fetch(j);
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int at = t + 256 * k, o = at / CHUNKS * PITCH + 16 * (at % CHUNKS);
        *(u32x4*)(s1 + o) = v1[k];
        if constexpr (MODE >= NS_JOIN) *(u32x4*)(s2 + o) = v2[k];
      }
      if (MODE != NS_LAST && j + 1 < T) fetch(j + 1);
      if constexpr (MODE == NS_LAST) fetch_w(j, 0);
      const int row = n0 + 64 * j + srow;
      // the diagonal: where the lane's row meets the tile's columns
      const int dcol = (MODE == NS_POLY || MODE == NS_JOIN) && tm == tn ? row - m0 : -64 * T;
      float dval = 0.0f;
      bool has = false;
      lds_barrier();
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f16x4* p1 = (f16x4*)(s1 + srow * PITCH + 2 * scol(i, q));
          const f16x4 h = *p1;
          float v[4];
          if constexpr (ns_symmetric(MODE)) {
            const int at = dcol - scol(i, q);
            f16x4 o, h2;
            float4 c2;
            if constexpr (MODE == NS_JOIN) {
              h2 = *(const f16x4*)(s2 + srow * PITCH + 2 * scol(i, q));
              const int col = m0 + scol(i, q);
              c2 = *(const float4*)(g.col2 + (int64_t)mat * g.mp + (col < g.mp ? col : g.mp - 4));
            }
            const float r1 = MODE == NS_POLY ? g.f1 : own[j] * g.f1;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = r1 * (float)h[r] + acc[i][j][4 * q + r] * g.f;
              if constexpr (MODE == NS_JOIN) v[r] += (r == 0 ? c2.x : r == 1 ? c2.y : r == 2 ? c2.z : c2.w) * g.f2 * (float)h2[r];
              dval = at == r ? v[r] : dval;
              o[r] = (f16_t)(at == r ? 0.0f : v[r]);
            }
            has = has || (at >= 0 && at < 4);
            *p1 = o;
          } else {
            f16x4* p2 = (f16x4*)(s2 + srow * PITCH + 2 * scol(i, q));
            const f16x4 l = *p2;
            f16x4 oh, ol;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = own[j] * ((float)h[r] + (float)l[r] * (1.0f / NS_LO)) + acc[i][j][4 * q + r] * g.f;
              f16_t hh, ll;
              ns_split(v[r], hh, ll);
              oh[r] = hh;
              ol[r] = ll;
            }
            if constexpr (MODE == NS_STEP) {
              *p1 = oh;
              *p2 = ol;
            } else {
              // (strides, not a branch: ahead of one the accumulators of all passes are read and fill the registers)
              float* f = (float*)(smem + 2 * AREA) + srow * row_step + scol(i, q) * col_step;
#pragma unroll
              for (int r = 0; r < 4; ++r) f[r * col_step] = v[r] * g.inv;
            }
          }
        }
      if (has && row < g.mp) {
        const int64_t at = (int64_t)mat * g.mp + row;
        if (MODE == NS_POLY) g.diag[at] = g.a + dval * g.inv;
        if (MODE == NS_JOIN) g.diag[at] = own[j] * g.col2[at] + dval * g.inv;
      }
      lds_barrier();
      if constexpr (ns_symmetric(MODE)) {
        store_rows(s1, to1, 64 * j, g.mp);
        if (tm != tn) store_transposed(s1, to2, 64 * j);
      } else if constexpr (MODE == NS_STEP) {
        store_rows(s1, to1, 64 * j, g.np);
        store_rows(s2, to2, 64 * j, g.np);
      } else {
        const float* f = (const float*)(smem + 2 * AREA);
        put_w(j, 0, f);
        if constexpr (AHEAD < QPT) {
          fetch_w(j, AHEAD);
          put_w(j, AHEAD, f);
        }
        if (!quads) {
          const int r = w0 + qrow + (g.tall ? 0 : 64 * j), c = wcol + (g.tall ? 64 * j : 0);
          TW* p = weight + (r - w0) * g.ldw;
#pragma unroll 1
          for (int k = 0; k < QPT && r + k * krows < g.rows; ++k, p += krows * g.ldw) {
            float4 v = *(const float4*)(f + first + k * kstage);
            if (g.update) {
              const float4 o = muon_get4<TW>(p, c, g.cols, false);
              v = make_float4(keep * o.x - step * v.x, keep * o.y - step * v.y, keep * o.z - step * v.z, keep * o.w - step * v.w);
            }
            muon_put4<TW>(p, c, g.cols, false, v);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Short sides up to 64
//
// The steps' polynomials are polynomials of R = U U^T / (||U||_F + eps)^2 alone,
// whose trace gives the norm: X = Q U / (||U||_F + eps) with Q the product of the
// steps' a I + b R + c R^2, and R <- (a I + b R + c R^2)^2 R after each.  So the
// long side is gone through twice, for R and for Q U, and the steps between run
// in one workgroup a matrix: three launches instead of 2 + 3 a step, of which
// each takes 5 us or more here (16 x 4096 291 -> 24 us, 64 x 1000
// 147 -> 65).  Small ones have a kernel of their own, below.  What R's rounding adds to the small directions grows by a^2 = 12 a
// step, 2e4 in five, and nothing takes it back as X X^T formed anew would: R is
// held in 64 bits, and its products run on the 64-bit matrix instruction (a
// product of 64 x 64 x 64 1.3 us; for 128 it would be 10).  The result is fp32's
// own roundings away from 64 bits, grown by a a step in directions that U lacks; many
// steps are taken otherwise, below.
// ---------------------------------------------------------------------------
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int NS_SHORT = 64;               // the longest short side
constexpr int SB = 16;                     // a matrix instruction's tile
constexpr int SPITCH = 66;                 // doubles: a row of a staged matrix
constexpr int STILES = 10;                 // tiles of 16 x 16 on and below a 64 x 64 diagonal
constexpr int SUPITCH = 68;                // floats: a row of a staged piece of U

struct ShortArgs {
  MuonIn in;               // mp, np unused
  int blocks;              // 16-row blocks of the short side
  int chunks;              // workgroups that share a matrix's long side; 0: small matrices, all in one launch
  double* part;            // [batch][chunks][blocks (blocks + 1) / 2][256]: R's tiles as the instruction holds them
  float* q;                // [batch][side][side], side = 16 blocks
  double* inv;             // [batch]: 1 / (||U||_F + eps)
  float coef[3 * 64];
  int steps;
  float hold;              // small matrices: the power of two that X, A and P are held times
  // in 64 bits:
  double* x;               // X [batch][short][long], ahead of the first step U
  double* p;               // P of step `step`, or Q; [batch][side][side]
  int step;                // -1: all steps together
  void* w;
  int64_t ldw, sw;
  int update;
  float lr, decay, scale;
  const float* lr_by;
};

__device__ __forceinline__ void short_tile(int p, int& row, int& col) {
  row = p < 1 ? 0 : p < 3 ? 1 : p < 6 ? 2 : 3;
  col = p - row * (row + 1) / 2;
}

// 64 values of the long side from `at` on: U as [short][64] in LDS.  The tile's
// own registers hold it as the weight lies.
template <typename TG, typename TM>
__device__ __forceinline__ void short_load(const MuonIn& a, int batch, int at, MuonTile<TG, TM>& u, float (*turn)[MPITCH]) {
  u.load(a, batch, a.tall ? at : 0, a.tall ? 0 : at, turn);
}
template <typename TG, typename TM>
__device__ __forceinline__ void short_stage(const MuonIn& a, const MuonTile<TG, TM>& u, double f, float* lds) {
  const int t = threadIdx.x, tr = t >> 4, tc = 4 * (t & 15);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = make_float4((float)(u.u[k].x * f), (float)(u.u[k].y * f), (float)(u.u[k].z * f), (float)(u.u[k].w * f));
    const int r = tr + 16 * k;
    if (a.tall) {
      lds[tc * SUPITCH + r] = v.x;
      lds[(tc + 1) * SUPITCH + r] = v.y;
      lds[(tc + 2) * SUPITCH + r] = v.z;
      lds[(tc + 3) * SUPITCH + r] = v.w;
    } else {
      *(float4*)(lds + r * SUPITCH + tc) = v;
    }
  }
}

// What 64 staged columns add to U U^T: wave w takes every fourth step of 4 of them.
template <int PITCH, typename T>
__device__ __forceinline__ void short_gram_add(const T* u, int blocks, f64x4 (&acc)[STILES]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    double x[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) x[b] = (double)u[(SB * b + lane % 16) * PITCH + 4 * (4 * s + w) + lane / 16];
#pragma unroll
    for (int p = 0; p < STILES; ++p) {
      int i, j;
      short_tile(p, i, j);
      if (i < blocks) acc[p] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[i], x[j], acc[p], 0, 0, 0);
    }
  }
}
// The four waves' sums, in their order, to the workgroup's part.
__device__ __forceinline__ void short_gram_put(const ShortArgs& a, const f64x4 (&acc)[STILES], double* sums) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, tiles = a.blocks * (a.blocks + 1) / 2;
  for (int q = 0; q < 4; ++q) {
    __syncthreads();
    if (w == q) {
#pragma unroll
      for (int p = 0; p < STILES; ++p)
        if (p < tiles) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            double* to = sums + p * 256 + 64 * r + lane;
            *to = q ? *to + acc[p][r] : acc[p][r];
          }
        }
    }
  }
  __syncthreads();
  double* to = a.part + ((int64_t)blockIdx.y * a.chunks + blockIdx.x) * tiles * 256;
  for (int i = t; i < tiles * 256; i += 256) to[i] = sums[i];
}

// Partial sums of U U^T.
template <typename TG, typename TM>
__global__ __launch_bounds__(256) void short_gram_kernel(ShortArgs a) {
  __shared__ float turn[MT][MPITCH];
  __shared__ __align__(16) float u[NS_SHORT * SUPITCH];
  __shared__ double sums[STILES * 256];
  const int batch = blockIdx.y, n = a.in.tall ? a.in.rows : a.in.cols;
  f64x4 acc[STILES];
#pragma unroll
  for (int p = 0; p < STILES; ++p) acc[p] = f64x4{0, 0, 0, 0};
  for (int at = blockIdx.x * 64; at < n; at += a.chunks * 64) {
    MuonTile<TG, TM> v;
    short_load(a.in, batch, at, v, turn);
    __syncthreads();
    short_stage(a.in, v, 1.0, u);
    __syncthreads();
    short_gram_add<SUPITCH>(u, a.blocks, acc);
  }
  short_gram_put(a, acc, sums);
}

// Tile (i, j) of x y^T: lane l holds rows 4 r + l / 16, r < 4, of column l % 16.
// Sixteen columns of both at a time, read ahead of the products.
__device__ __forceinline__ f64x4 short_product(const double* x, const double* y, int i, int j, int blocks, int lane) {
  f64x4 c = {0, 0, 0, 0};
  const double* p = x + (SB * i + lane % 16) * SPITCH + lane / 16;
  const double* q = y + (SB * j + lane % 16) * SPITCH + lane / 16;
  double u[2][4], v[2][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u[0][k] = p[4 * k];
    v[0][k] = q[4 * k];
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b >= blocks) break;
    if (b + 1 < blocks) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[(b + 1) & 1][k] = p[16 * (b + 1) + 4 * k];
        v[(b + 1) & 1][k] = q[16 * (b + 1) + 4 * k];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f64_16x16x4f64(u[b & 1][k], v[b & 1][k], c, 0, 0, 0);
  }
  return c;
}

// Row r (of 4) of tile (i, j), as a product's lanes hold it, into a symmetric matrix.  (Of a tile on the diagonal the
// lower half: the two halves' roundings differ.)
__device__ __forceinline__ void short_put(double* m, int i, int j, int r, int lane, double v) {
  const int row = SB * i + 4 * r + lane / 16, col = SB * j + lane % 16;
  if (row < col) return;
  m[row * SPITCH + col] = v;
  m[col * SPITCH + row] = v;
}
constexpr int SSTEP_THR = 64 * STILES;
// The parts' sum; wave w of STILES.
__device__ __forceinline__ void short_gram_join(const ShortArgs& a, int batch, int w, int lane, double* R) {
  const int tiles = a.blocks * (a.blocks + 1) / 2;
  const double* from = a.part + (int64_t)batch * a.chunks * tiles * 256;
  for (int e = w; e < 4 * tiles; e += STILES) {           // rows e % 4 of tile e / 4, as the instruction holds them
    double s = 0.0;
    for (int c = 0; c < a.chunks; c += 16) {
      double v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = from[(int64_t)(c + k < a.chunks ? c + k : 0) * tiles * 256 + 64 * e + lane];
#pragma unroll
      for (int k = 0; k < 16; ++k) s += c + k < a.chunks ? v[k] : 0.0;
    }
    int i, j;
    short_tile(e >> 2, i, j);
    short_put(R, i, j, e & 3, lane, s);
  }
}
// U U^T in R becomes that of U / (||U||_F + eps); the factor 1 / (||U||_F + eps) is returned.
__device__ __forceinline__ double short_normed(const ShortArgs& a, int side, int lane, double* R) {
  const double norm = sqrt(wave_sum_d(lane < side ? R[lane * (SPITCH + 1)] : 0.0)) + (double)a.in.eps;
  // a matrix of zeros stays one; one with an infinity or a NaN becomes NaN
  const double inv = norm == 0.0 ? 0.0 : norm < __builtin_inf() ? 1.0 / norm : __builtin_nan("");
  __syncthreads();
  for (int i = threadIdx.x; i < side * side; i += SSTEP_THR) R[i / side * SPITCH + i % side] *= inv * inv;
  __syncthreads();
  return inv;
}

// The steps, a wave for each tile.  Every matrix is a polynomial of R, symmetric
// and commuting with the others, so products are formed as X Y^T, by half, and
// stored twice.
__global__ __launch_bounds__(SSTEP_THR) void short_steps_kernel(ShortArgs a) {
  __shared__ double R[NS_SHORT * SPITCH], P[NS_SHORT * SPITCH], Q[NS_SHORT * SPITCH];
  const int t = threadIdx.x, lane = t & 63, batch = blockIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int tiles = a.blocks * (a.blocks + 1) / 2, side = SB * a.blocks;
  int ti, tj;
  short_tile(w, ti, tj);
  auto put = [&](double* m, int i, int j, int r, double v) { short_put(m, i, j, r, lane, v); };
  short_gram_join(a, batch, w, lane, R);
  __syncthreads();
  const double inv = short_normed(a, side, lane, R);
  const bool here = w < tiles;
  f64x4 acc = {0, 0, 0, 0};
  auto store = [&](double* m) {
    if (here)
#pragma unroll
      for (int r = 0; r < 4; ++r) put(m, ti, tj, r, acc[r]);
  };
  for (int s = 0; s < a.steps; ++s) {
    const double ca = a.coef[3 * s], cb = a.coef[3 * s + 1], cc = a.coef[3 * s + 2];
    if (here) {
      acc = short_product(R, R, ti, tj, a.blocks, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = SB * ti + 4 * r + lane / 16, col = SB * tj + lane % 16;
        const double v = cb * R[row * SPITCH + col] + cc * acc[r] + (row == col ? ca : 0.0);
        put(P, ti, tj, r, v);
        if (s == 0) put(Q, ti, tj, r, v);
      }
    }
    __syncthreads();
    f64x4 next = {0, 0, 0, 0};
    if (here && s > 0) next = short_product(P, Q, ti, tj, a.blocks, lane);
    if (here && s + 1 < a.steps) acc = short_product(P, R, ti, tj, a.blocks, lane);
    __syncthreads();
    if (s + 1 < a.steps) store(R);
    if (s > 0) {
      acc = next;
      store(Q);
    }
    __syncthreads();
    if (s + 1 < a.steps) {
      if (here) acc = short_product(P, R, ti, tj, a.blocks, lane);
      __syncthreads();
      store(R);
      __syncthreads();
    }
  }
  for (int i = t; i < side * side; i += SSTEP_THR) {
    const int64_t to = (int64_t)batch * side * side + i;
    if (a.p) a.p[to] = Q[i / side * SPITCH + i % side];
    else a.q[to] = (float)Q[i / side * SPITCH + i % side];
  }
  if (t == 0) a.inv[batch] = inv;
}

// X = Q U inv for 64 values of the long side, the momentum's store and the weight.
template <typename TG, typename TM, typename TW>
__global__ __launch_bounds__(256) void short_apply_kernel(ShortArgs a) {
  __shared__ float turn[MT][MPITCH];
  __shared__ __align__(16) float u[NS_SHORT * SUPITCH], q[NS_SHORT * SUPITCH];
  const int t = threadIdx.x, tr = t >> 4, tc = 4 * (t & 15), batch = blockIdx.y, side = SB * a.blocks;
  const MuonIn& in = a.in;
  const int at = blockIdx.x * 64, r0 = in.tall ? at : 0, c0 = in.tall ? 0 : at;
  MuonTile<TG, TM> v;
  short_load(in, batch, at, v, turn);
  const double inv = a.inv[batch];
  for (int i = t; i < side * side; i += 256) q[i / side * SUPITCH + i % side] = a.q[(int64_t)batch * side * side + i];
  short_stage(in, v, inv, u);
  const float lr_now = a.lr_by ? a.lr * *a.lr_by : a.lr, keep = 1.0f - lr_now * a.decay, step = lr_now * a.scale;
  if (in.m) {
    TM* m = (TM*)in.m + batch * in.sm;
    const bool vm = muon_vec<TM>(in.m, in.ldm, in.sm);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r0 + tr + 16 * k < in.rows) muon_put4<TM>(m + (r0 + tr + 16 * k) * in.ldm, c0 + tc, in.cols, vm, v.m4[k]);
  }
  __syncthreads();
  // x[k][e]: the weight's row tr + 16 k, column tc + e of the tile
  float x[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[k][e] = 0.0f;
  if (!in.tall) {
#pragma unroll 4
    for (int j = 0; j < side; ++j) {
      const float4 b = *(const float4*)(u + j * SUPITCH + tc);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = k < a.blocks ? q[(tr + 16 * k) * SUPITCH + j] : 0.0f;
        x[k][0] = __builtin_fmaf(f, b.x, x[k][0]); x[k][1] = __builtin_fmaf(f, b.y, x[k][1]);
        x[k][2] = __builtin_fmaf(f, b.z, x[k][2]); x[k][3] = __builtin_fmaf(f, b.w, x[k][3]);
      }
    }
  } else if (tc < side) {
#pragma unroll 4
    for (int j = 0; j < side; ++j) {
      const float4 b = *(const float4*)(q + j * SUPITCH + tc);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = u[j * SUPITCH + tr + 16 * k];
        x[k][0] = __builtin_fmaf(f, b.x, x[k][0]); x[k][1] = __builtin_fmaf(f, b.y, x[k][1]);
        x[k][2] = __builtin_fmaf(f, b.z, x[k][2]); x[k][3] = __builtin_fmaf(f, b.w, x[k][3]);
      }
    }
  }
  TW* wp = (TW*)a.w + batch * a.sw;
  const bool vw = muon_vec<TW>(a.w, a.ldw, a.sw);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = r0 + tr + 16 * k;
    if (r >= in.rows) continue;
    TW* p = wp + r * a.ldw;
    float4 o = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
    if (a.update) {
      const float4 old = muon_get4<TW>(p, c0 + tc, in.cols, vw);
      o = make_float4(keep * old.x - step * o.x, keep * old.y - step * o.y, keep * old.z - step * o.z, keep * old.w - step * o.w);
    }
    muon_put4<TW>(p, c0 + tc, in.cols, vw, o);
  }
}

// ---------------------------------------------------------------------------
// Short sides, many steps
//
// In directions that U does not have Q grows by a in each step, and with it what is
// rounded off Q and off the product Q U; and R <- q R q multiplies what 64
// bits round off R by q^2 a step there, of either sign, where X X^T is never less
// than 0: once such a value nears -1 the polynomials run away (a matrix of rank 1,
// Muon's step: 10 times the result after 16, NaN after 20).  So beyond a growth of
// SHORT_GROWTH Q U is formed in 64 bits, from a copy of U in the workspace, and beyond
// SHORT_WIDE_GROWTH the steps are taken one by one, with X in 64 bits and X X^T formed
// anew for each: what X's rounding adds to such a direction still grows by a, from
// 2^-53, but no singular value leaves the polynomials' range.  a X stays apart from
// P X there, so that equal rows stay equal.  Both on the 64-bit matrix instruction,
// bound by latency: 16 x 4096 six steps 27 us, eight 32, sixteen (one by one) 225;
// 64 x 1000 72, 98 and 612.
// ---------------------------------------------------------------------------
// Five of Muon's steps grow by 485, six by 1670: a matrix of ones, 64 x 1000, is then 0.03% and 0.12% off, and would be
// 0.5% after eight.
constexpr double SHORT_GROWTH = 2048.0;
// Nine steps grow by 68000.  A wave adds at most 4096 products of four to an entry of R one after the other, so R is off by
// 2^12 2^-53 of its trace, and grown by 2^34 by less than 0.01.
constexpr double SHORT_WIDE_GROWTH = 131072.0;

// U, and the momentum's store.
template <typename TG, typename TM>
__global__ __launch_bounds__(256) void short_wide_start_kernel(ShortArgs a) {
  __shared__ float turn[MT][MPITCH];
  __shared__ __align__(16) float u[NS_SHORT * SUPITCH];
  const MuonIn& in = a.in;
  const int t = threadIdx.x, tr = t >> 4, tc = 4 * (t & 15), batch = blockIdx.y, at = blockIdx.x * 64;
  const int m = in.tall ? in.cols : in.rows, n = in.tall ? in.rows : in.cols;
  const int r0 = in.tall ? at : 0, c0 = in.tall ? 0 : at;
  MuonTile<TG, TM> v;
  short_load(in, batch, at, v, turn);
  short_stage(in, v, 1.0, u);
  if (in.m) {
    TM* p = (TM*)in.m + batch * in.sm;
    const bool vm = muon_vec<TM>(in.m, in.ldm, in.sm);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r0 + tr + 16 * k < in.rows) muon_put4<TM>(p + (r0 + tr + 16 * k) * in.ldm, c0 + tc, in.cols, vm, v.m4[k]);
  }
  __syncthreads();
  const int c = t & 63;
  if (at + c < n)
    for (int r = t >> 6; r < m; r += 4) a.x[((int64_t)batch * m + r) * n + at + c] = (double)u[r * SUPITCH + c];
}

// 64 columns of X from `at` on into LDS, zeros behind its rows (up to whole blocks) and columns.
__device__ __forceinline__ void short_wide_load(const ShortArgs& a, int batch, int at, double* u) {
  const int m = a.in.tall ? a.in.cols : a.in.rows, n = a.in.tall ? a.in.rows : a.in.cols, c = threadIdx.x & 63;
  for (int r = threadIdx.x >> 6; r < SB * a.blocks; r += 4)
    u[r * SPITCH + c] = r < m && at + c < n ? a.x[((int64_t)batch * m + r) * n + at + c] : 0.0;
}

// Partial sums of X X^T.
__global__ __launch_bounds__(256) void short_wide_gram_kernel(ShortArgs a) {
  __shared__ double u[NS_SHORT * SPITCH], sums[STILES * 256];
  const int batch = blockIdx.y, n = a.in.tall ? a.in.rows : a.in.cols;
  for (int i = threadIdx.x; i < NS_SHORT * SPITCH; i += 256) u[i] = 0.0;
  f64x4 acc[STILES];
#pragma unroll
  for (int p = 0; p < STILES; ++p) acc[p] = f64x4{0, 0, 0, 0};
  for (int at = blockIdx.x * 64; at < n; at += a.chunks * 64) {
    __syncthreads();
    short_wide_load(a, batch, at, u);
    __syncthreads();
    short_gram_add<SPITCH>(u, a.blocks, acc);
  }
  short_gram_put(a, acc, sums);
}

// P = b R + c R^2; ahead of the first step R is U U^T and gives the norm.
__global__ __launch_bounds__(SSTEP_THR) void short_poly_kernel(ShortArgs a) {
  __shared__ double R[NS_SHORT * SPITCH], P[NS_SHORT * SPITCH];
  const int t = threadIdx.x, lane = t & 63, batch = blockIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int tiles = a.blocks * (a.blocks + 1) / 2, side = SB * a.blocks;
  short_gram_join(a, batch, w, lane, R);
  __syncthreads();
  if (a.step == 0) {
    const double inv = short_normed(a, side, lane, R);
    if (t == 0) a.inv[batch] = inv;
  }
  const double cb = a.coef[3 * a.step + 1], cc = a.coef[3 * a.step + 2];
  if (w < tiles) {
    int ti, tj;
    short_tile(w, ti, tj);
    const f64x4 acc = short_product(R, R, ti, tj, a.blocks, lane);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = SB * ti + 4 * r + lane / 16, col = SB * tj + lane % 16;
      short_put(P, ti, tj, r, lane, cb * R[row * SPITCH + col] + cc * acc[r]);
    }
  }
  __syncthreads();
  for (int i = t; i < side * side; i += SSTEP_THR)
    a.p[(int64_t)batch * side * side + i] = P[i / side * SPITCH + i % side];
}

// X' = a X + P X, or Q X, for 64 values of the long side: in place, or the last one into the weight.  Wave w takes
// columns 16 w on.
template <typename TW>
__global__ __launch_bounds__(256) void short_wide_step_kernel(ShortArgs a) {
  __shared__ double u[NS_SHORT * SPITCH], p[NS_SHORT * SPITCH];
  const MuonIn& in = a.in;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, batch = blockIdx.y, at = blockIdx.x * 64, side = SB * a.blocks;
  const int m = in.tall ? in.cols : in.rows, n = in.tall ? in.rows : in.cols;
  short_wide_load(a, batch, at, u);
  for (int i = t; i < side * side; i += 256) p[i / side * SPITCH + i % side] = a.p[(int64_t)batch * side * side + i];
  __syncthreads();
  // U is not divided by its norm yet
  const double f = a.step <= 0 ? a.inv[batch] : 1.0, ca = a.step < 0 ? 0.0 : (double)a.coef[3 * a.step];
  const bool last = a.step < 0 || a.step + 1 == a.steps;
  const int c = SB * w + lane % 16;
  f64x4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f64x4{0, 0, 0, 0};
  for (int k = lane / 16; k < side; k += 4) {
    const double v = u[k * SPITCH + c];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < a.blocks) x[i] = __builtin_amdgcn_mfma_f64_16x16x4f64(p[(SB * i + lane % 16) * SPITCH + k], v, x[i], 0, 0, 0);
  }
  if (at + c >= n) return;
  const float lr_now = a.lr_by ? a.lr * *a.lr_by : a.lr, keep = 1.0f - lr_now * a.decay, step = lr_now * a.scale;
  TW* wp = (TW*)a.w + batch * a.sw;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = SB * i + 4 * r + lane / 16;
      if (row >= m) continue;
      const double v = f * (ca * u[row * SPITCH + c] + x[i][r]);
      if (!last) {
        a.x[((int64_t)batch * m + row) * n + at + c] = v;
        continue;
      }
      TW* to = in.tall ? wp + (int64_t)(at + c) * a.ldw + row : wp + row * a.ldw + at + c;
      float o = (float)v;
      if (a.update) o = keep * muon_get<TW>(to, 0) - step * o;
      if constexpr (sizeof(TW) == 4) *to = o;
      else *to = (bf16_t)pk_bf16(o, o);
    }
}

// ---------------------------------------------------------------------------
// Small matrices: short sides of 33 to 64, long ones up to 256
//
// All of X sits in one workgroup's LDS and the steps run there, in one launch that
// reads the gradient and the momentum once; the three launches above take 42 us for
// the steps alone of sides over 48 (64 x 64 61 -> 22 us, 64 x 128 64 -> 29, 64 x 256
// 64 -> 44, 300 of 64 x 64 108 -> 42).  X, A and P are pairs of fp16, hi + lo 2^-11, and
// each product three of fp16 (hi hi, hi lo, lo hi) with fp32 sums: what is left out is
// 2^-22 of a value.  Bound by latency, 1.5 us a step for 64 columns where the matrix
// instructions take 0.3 and the LDS reads as long; the next operands read ahead gained
// nothing (46 us).
// ---------------------------------------------------------------------------
constexpr int TINY_LONG = 256, TINY_TILES = TINY_LONG / 64;
constexpr int TINY_XP = TINY_LONG + 8, TINY_PP = 64 + 8;      // values a row: 16 rows' 16-byte reads take all banks

struct TinyPair {
  f16x8 hi, lo;
};
// A matrix instruction's operand: rows row0 + lane % 32, 8 values from k0 + 8 (lane / 32) on.
__device__ __forceinline__ TinyPair tiny_rows(const f16_t* hi, const f16_t* lo, int pitch, int row0, int k0) {
  const int lane = threadIdx.x & 63, at = (row0 + (lane & 31)) * pitch + k0 + 8 * (lane >> 5);
  return {*(const f16x8*)(hi + at), *(const f16x8*)(lo + at)};
}
// The same of the matrix transposed: columns c0 + lane % 32, 8 rows, by two transposing reads.
__device__ __forceinline__ f16x8 tiny_turned(const f16_t* m, int pitch, int c0, int k0) {
  const int lane = threadIdx.x & 63, li = lane & 15;
  const uint8_t* p = (const uint8_t*)(m + (k0 + 8 * (lane >> 5) + (li >> 2)) * pitch + c0 + 16 * ((lane >> 4) & 1) + 4 * (li & 3));
  const int2 u = __builtin_bit_cast(int2, read_lds_tr16(p)), v = __builtin_bit_cast(int2, read_lds_tr16(p + 8 * pitch));
  return __builtin_bit_cast(f16x8, i32x4{u.x, u.y, v.x, v.y});
}
// hi hi, and hi lo + lo hi, which counts 2^-11.  (A third sum of their own: 6% slower.)
struct TinySum {
  f32x16 big, small;
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < 16; ++r) big[r] = small[r] = 0.0f;
  }
  __device__ __forceinline__ void add(const TinyPair& a, const TinyPair& b) {
    big = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.hi, b.hi, big, 0, 0, 0);
    small = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.hi, b.lo, small, 0, 0, 0);
    small = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.lo, b.hi, small, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int r) const { return big[r] + small[r] * (1.0f / NS_LO); }
};
// Four values of a row as a pair.
__device__ __forceinline__ void tiny_put(f16_t* hi, f16_t* lo, int at, const float (&v)[4]) {
  f16x4 h, l;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f16_t x, y;
    ns_split(v[r], x, y);
    h[r] = x;
    l[r] = y;
  }
  *(f16x4*)(hi + at) = h;
  *(f16x4*)(lo + at) = l;
}
__device__ __forceinline__ void tiny_get(const f16_t* hi, const f16_t* lo, int at, float (&v)[4]) {
  const f16x4 h = *(const f16x4*)(hi + at), l = *(const f16x4*)(lo + at);
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = (float)h[r] + (float)l[r] * (1.0f / NS_LO);
}

template <typename TG, typename TM, typename TW>
__global__ __launch_bounds__(256) void tiny_kernel(ShortArgs a) {
  __shared__ __align__(16) f16_t xh[NS_SHORT * TINY_XP], xl[NS_SHORT * TINY_XP];
  __shared__ __align__(16) f16_t ah[NS_SHORT * TINY_PP], al[NS_SHORT * TINY_PP], ph[NS_SHORT * TINY_PP], pl[NS_SHORT * TINY_PP];
  __shared__ float turn[MT][MPITCH];
  __shared__ double sums[4];
  const MuonIn& in = a.in;
  const int t = threadIdx.x, lane = t & 63, tr = t >> 4, tc = 4 * (t & 15), batch = blockIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6), lr = lane & 31, lg = lane >> 5;
  const int tiles = ((in.tall ? in.rows : in.cols) + 63) / 64;         // of the long side
  // U, the momentum's store and the norm
  MuonTile<TG, TM> u[TINY_TILES];
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < TINY_TILES; ++k)
    if (k < tiles) {
      const int r0 = in.tall ? 64 * k : 0, c0 = in.tall ? 0 : 64 * k;
      u[k].load(in, batch, r0, c0, turn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double x = u[k].u[i].x, y = u[k].u[i].y, z = u[k].u[i].z, v = u[k].u[i].w;
        s += x * x + y * y + (z * z + v * v);
      }
      if (in.m) {
        TM* m = (TM*)in.m + batch * in.sm;
        const bool vm = muon_vec<TM>(in.m, in.ldm, in.sm);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + tr + 16 * i < in.rows) muon_put4<TM>(m + (r0 + tr + 16 * i) * in.ldm, c0 + tc, in.cols, vm, u[k].m4[i]);
      }
    }
  s = wave_sum_d(s);
  if (lane == 0) sums[w] = s;
  __syncthreads();
  const double norm = sqrt(sums[0] + sums[1] + (sums[2] + sums[3])) + (double)in.eps;
  // a matrix of zeros stays one; one with an infinity or a NaN becomes NaN
  const double f = norm == 0.0 ? 0.0 : norm < __builtin_inf() ? (double)a.hold / norm : __builtin_nan("");
#pragma unroll
  for (int k = 0; k < TINY_TILES; ++k)
    if (k < tiles) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v[4] = {(float)(u[k].u[i].x * f), (float)(u[k].u[i].y * f), (float)(u[k].u[i].z * f), (float)(u[k].u[i].w * f)};
        const int r = tr + 16 * i;
        if (!in.tall) {
          tiny_put(xh, xl, r * TINY_XP + 64 * k + tc, v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) ns_split(v[e], xh[(tc + e) * TINY_XP + 64 * k + r], xl[(tc + e) * TINY_XP + 64 * k + r]);
        }
      }
    }
  __syncthreads();
  const float inv = 1.0f / a.hold;
  const float lr_now = a.lr_by ? a.lr * *a.lr_by : a.lr, keep = 1.0f - lr_now * a.decay, step = a.update ? lr_now * a.scale : -1.0f;
  // A and P: wave w's 32 x 32 of them, of which a lane holds row i0 + lr, columns j0 + 8 q + 4 lg on
  const int i0 = 32 * (w & 1), j0 = 32 * (w >> 1);
  for (int n = 0; n < a.steps; ++n) {
    const float ca = a.coef[3 * n], cb = a.coef[3 * n + 1], cc = a.coef[3 * n + 2];
    TinySum sum;
    sum.zero();
    for (int k = 0; k < tiles; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        sum.add(tiny_rows(xh, xl, TINY_XP, j0, 64 * k + 16 * c), tiny_rows(xh, xl, TINY_XP, i0, 64 * k + 16 * c));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = sum.get(4 * q + r) * inv;
      tiny_put(ah, al, (i0 + lr) * TINY_PP + j0 + 8 * q + 4 * lg, v);
    }
    __syncthreads();
    sum.zero();
#pragma unroll
    for (int c = 0; c < 4; ++c) sum.add(tiny_rows(ah, al, TINY_PP, j0, 16 * c), tiny_rows(ah, al, TINY_PP, i0, 16 * c));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int at = (i0 + lr) * TINY_PP + j0 + 8 * q + 4 * lg;
      float v[4];
      tiny_get(ah, al, at, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = cb * v[r] + cc * inv * sum.get(4 * q + r);
      tiny_put(ph, pl, at, v);
    }
    __syncthreads();
    // P X: rows i0 + lr, columns j0 + 64 k + 8 q + 4 lg on
    TinyPair p[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) p[c] = tiny_rows(ph, pl, TINY_PP, i0, 16 * c);
    f32x16 px[TINY_TILES];
#pragma unroll
    for (int k = 0; k < TINY_TILES; ++k)
      if (k < tiles) {
        sum.zero();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sum.add({tiny_turned(xh, TINY_XP, j0 + 64 * k, 16 * c), tiny_turned(xl, TINY_XP, j0 + 64 * k, 16 * c)}, p[c]);
#pragma unroll
        for (int r = 0; r < 16; ++r) px[k][r] = sum.get(r);
      }
    __syncthreads();                                                   // X is read out
#pragma unroll
    for (int k = 0; k < TINY_TILES; ++k)
      if (k < tiles) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = i0 + lr, j = j0 + 64 * k + 8 * q + 4 * lg;
          float v[4];
          tiny_get(xh, xl, i * TINY_XP + j, v);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = ca * v[r] + px[k][4 * q + r] * inv;
          if (n + 1 < a.steps) {
            tiny_put(xh, xl, i * TINY_XP + j, v);
            continue;
          }
          TW* wp = (TW*)a.w + batch * a.sw;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] *= inv;
          if (!in.tall) {
            if (i < in.rows) {
              const bool vw = muon_vec<TW>(a.w, a.ldw, a.sw);
              float4 o = make_float4(v[0], v[1], v[2], v[3]);
              if (a.update) {
                const float4 old = muon_get4<TW>(wp + i * a.ldw, j, in.cols, vw);
                o = make_float4(keep * old.x - step * o.x, keep * old.y - step * o.y, keep * old.z - step * o.z, keep * old.w - step * o.w);
              }
              muon_put4<TW>(wp + i * a.ldw, j, in.cols, vw, o);
            }
          } else if (i < in.cols) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (j + r >= in.rows) continue;
              TW* at = wp + (j + r) * a.ldw + i;
              float o = v[r];
              if (a.update) o = keep * muon_get<TW>(at, 0) - step * o;
              if constexpr (sizeof(TW) == 4) *at = o;
              else *at = (bf16_t)pk_bf16(o, o);
            }
          }
        }
      }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// The least short side from which two steps go together (see ns_pairs).
constexpr int64_t NS_PAIRS_FROM = 512;

struct NsPlan {
  int64_t mp, np, x, p;                       // padded sides; bytes of a matrix's X (hi or lo) and of its A or P
  int parts;
  size_t hi[2], lo[2], gram, poly, turn, poly2, join, diag, part, bytes;
  int blocks;                                 // short sides: 16-row blocks; else 0
  int chunks;                                 // and workgroups that share the long one; 0: all in one launch
  size_t q, inv, x64;
};

static NsPlan ns_plan(int64_t batch, int64_t rows, int64_t cols) {
  NsPlan h = {};
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  h.mp = ceil_div(m, 64) * 64;
  h.np = ceil_div(n, 64) * 64;
  h.x = h.mp * h.np * 2;
  h.p = h.mp * h.mp * 2;
  h.parts = (int)std::min<int64_t>(ceil_div(rows, MT) * ceil_div(cols, MT), NS_PART);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  if (m <= NS_SHORT) {
    h.blocks = (int)ceil_div(m, SB);
    // (of up to 32 the Gram matrix's steps are short themselves: 32 x 256 27 us there and 44 here, 32 x 64 26 and 22)
    if (n <= TINY_LONG && h.blocks > 2) {
      h.bytes = 256;                          // unused: every size's call wants a workspace
      return h;
    }
    const int64_t side = SB * h.blocks;
    // fewer where their sums take long to join: of 6 or 10 tiles against 1 or 3
    h.chunks = (int)std::min<int64_t>(ceil_div(n, 64), m > 32 ? 16 : 32);
    h.part = take((size_t)(batch * h.chunks * (h.blocks * (h.blocks + 1) / 2)) * 256 * 8);
    h.q = take((size_t)(batch * side * side) * 8);  // Q, or P in 64 bits
    h.inv = take((size_t)batch * 8);
    h.x64 = take((size_t)(batch * m * n) * 8);
    h.bytes = at;
    return h;
  }
  for (int i = 0; i < 2; ++i) {
    h.hi[i] = take((size_t)(batch * h.x));
    h.lo[i] = take((size_t)(batch * h.x));
  }
  h.gram = take((size_t)(batch * h.p));
  h.poly = take((size_t)(batch * h.p));
  if (h.mp >= NS_PAIRS_FROM && h.np > h.mp) {             // several steps together
    h.turn = take((size_t)(batch * h.p));
    h.poly2 = take((size_t)(batch * h.p));
    h.join = take((size_t)(batch * h.p));
  }
  h.diag = take((size_t)(3 * batch * h.mp) * 4);
  h.part = take((size_t)(batch * h.parts) * 8);
  h.bytes = at;
  return h;
}

constexpr int64_t NS_MOST_SIDE = 1 << 20, NS_MOST_SHORT = 32768, NS_MOST_STEPS = 64, NS_MOST_BATCH = 65535;

static pbs_status ns_check_dims(const char* what, int64_t batch, int64_t rows, int64_t cols) {
  PBS_REQUIRE(batch >= 0 && batch <= NS_MOST_BATCH && rows >= 0 && cols >= 0 && rows <= NS_MOST_SIDE && cols <= NS_MOST_SIDE &&
                  std::min(rows, cols) <= NS_MOST_SHORT,
              PBS_ERR_SHAPE, "%s: needs a batch of at most 65535, sides up to 2^20, the shorter up to 32768 (got %lld x %lld x %lld)",
              what, (long long)batch, (long long)rows, (long long)cols);
  PBS_REQUIRE(batch * ceil_div(std::max(rows, cols), 64) * ceil_div(std::min(rows, cols), 64) < (1ll << 31), PBS_ERR_SHAPE,
              "%s: too many values for one call", what);
  return PBS_OK;
}

static pbs_status ns_check_matrix(const char* what, const char* name, const void* p, pbs_format fmt, int64_t batch, int64_t rows,
                                  int64_t cols, int64_t ld, int64_t stride, bool out) {
  PBS_REQUIRE(fmt == PBS_FMT_BF16 || fmt == PBS_FMT_F32, PBS_ERR_UNSUPPORTED, "%s: %s must be BF16 or F32", what, name);
  const int64_t most = 1ll << 40;
  PBS_REQUIRE(ld >= 0 && stride >= 0 && ld <= most && stride <= most, PBS_ERR_SHAPE, "%s: strides of %s must be in [0, 2^40]", what, name);
  PBS_REQUIRE(p, PBS_ERR_INVALID_ARG, "%s: %s is null", what, name);
  PBS_REQUIRE(((uintptr_t)p & (fmt == PBS_FMT_BF16 ? 1 : 3)) == 0, PBS_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", what,
              name);
  if (out) {
    // rows apart, matrices apart, or matrices that lie between each other's rows
    const int64_t ns = std::min(ld, stride), nl = std::max(ld, stride);
    const bool both = rows > 1 && batch > 1;
    const bool apart = both ? ns >= cols && nl >= ns * ((ld <= stride ? rows : batch) - 1) + cols
                            : (rows <= 1 || ld >= cols) && (batch <= 1 || stride >= cols);
    PBS_REQUIRE(apart, PBS_ERR_SHAPE, "%s: rows of %s overlap", what, name);
  }
  return PBS_OK;
}

// The largest |f(x)| for x in [0, end]: at an end or at one of the roots of f', e0 + e1 x + e2 x^2.
template <typename F>
static double ns_largest(F f, double end, double e0, double e1, double e2) {
  double most = std::max(std::fabs(f(0.0)), std::fabs(f(end)));
  auto at = [&](double x) {
    if (x > 0.0 && x < end) most = std::max(most, std::fabs(f(x)));
  };
  const double d = e1 * e1 - 4 * e2 * e0;
  if (d >= 0.0) {
    const double h = -0.5 * (e1 + std::copysign(std::sqrt(d), e1));     // (no difference of near values)
    at(h / e2);
    at(e0 / h);
  }
  return most;
}

// The power of two that X, A and P are held times: the largest up to 2^14 that
// keeps all of them below fp16's largest value, 65504, with a third to spare for
// roundings.  top: the largest singular value ahead of each step, at most 1 at
// first, then the largest |p(s)| for s up to it and NS_ROUNDING of it, by which A's and
// P's roundings move it (a = 8.3, b = -23.6, c = 17.3: 7e-5 of it where rank 1 is random, 3e-3 in a constant
// matrix, whose roundings are alike): polynomials that rise
// steeply at the end of their range, as some published schedules have them, let a matrix of
// rank 1 run away from there (seven steps of one: 11 times the result in emulation; with arguments 1% within
// their ranges 2% off).  qmax: the largest |a + b s^2 + c s^4| of a step.
constexpr double NS_ROUNDING = 1.0 / 1024;
static pbs_status ns_scale(const char* what, const float* coef, int steps, float* scale, double* qmax) {
  double top = 1.0, most = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double a = coef[3 * k], b = coef[3 * k + 1], c = coef[3 * k + 2];
    PBS_REQUIRE(std::isfinite(a) && std::isfinite(b) && std::isfinite(c), PBS_ERR_INVALID_ARG, "%s: coefficients of step %d are not finite",
                what, k);
    const double t2 = top * top;                          // x: s^2
    const double poly = ns_largest([&](double x) { return x * (b + c * x); }, t2, b, 2 * c, 0.0);
    const double next = (1.0 + NS_ROUNDING) * ns_largest([&](double x) { return std::sqrt(x) * (a + x * (b + c * x)); }, t2, a, 3 * b, 5 * c);
    most = std::max({most, t2, poly, next});              // A, P, X; T, top * next at most, lies between A and the next A
    qmax[k] = ns_largest([&](double x) { return a + x * (b + c * x); }, t2, b, 2 * c, 0.0);
    top = next;
    PBS_REQUIRE(most < 4096.0, PBS_ERR_INVALID_ARG, "%s: the coefficients let singular values grow past fp16's range (step %d)", what, k);
  }
  float s = 16384.0f;
  while (s * most > 49152.0) s *= 0.5f;
  *scale = s;
  return PBS_OK;
}

// A product's tile: the one that takes least by this account, in us.  A stage of
// 64 K values takes a compute unit `stage` for each tile that it holds, but a tile
// no less than `alone`; what a tile takes beside its stages, `fixed`, is behind
// another tile's stages where several share a compute unit (sides of 64 and 128).
// Taken from A, A^2 and P X at 4 x 384 x 1100 to 16384 x 4096, with each tile
// size; measured there in us (A): 1024 x 1024 7.0, 11.9, 17.3 and 27 with tiles
// of 64, 128, 192 and 256; 2048 x 2048 22.6, 20.2, 28 and 44; 4096 x 4096 122, 95,
// 74 and 92; three of these 328, 225, 213 and 208.
constexpr int NS_CUS = 256;
static int ns_tile(int64_t mp, int64_t np, int64_t nk, int64_t batch, bool symmetric, double* time = nullptr) {
  struct Cost { double stage, alone, fixed; };
  static const Cost half[5] = {{}, {0.19, 0.27, 3.0}, {0.5, 0.5, 4.0}, {1.06, 1.06, 6.0}, {1.6, 1.6, 9.0}};
  static const Cost whole[5] = {{}, {0.25, 0.29, 4.0}, {0.5, 0.5, 6.0}, {}, {1.6, 1.6, 20.0}};
  int best = 4;
  double least = 1e300;
  for (int t = 4; t >= 1; --t) {
    if (t == 3 && !symmetric) continue;
    const Cost& c = symmetric ? half[t] : whole[t];
    const int64_t a = ceil_div(mp, 64 * t), b = ceil_div(np, 64 * t);
    const double held = (double)ceil_div(batch * (symmetric ? a * (a + 1) / 2 : a * b), NS_CUS);
    const double us = t >= 3 ? held * (nk * c.stage + c.fixed) : nk * std::max(c.alone, held * c.stage) + c.fixed;
    if (us < least) { least = us; best = t; }
  }
  if (time) *time = least;
  return best;
}

template <int MODE, typename TW = float>
static void ns_launch(NsArgs g, hipStream_t stream) {
  constexpr bool SYM = ns_symmetric(MODE);
  const int t = ns_tile(g.mp, g.np, (MODE == NS_GRAM ? g.np : g.mp) / 64, g.batch, SYM);
  g.tiles_n = (int)ceil_div(g.mp, 64 * t);
  g.tiles_m = SYM ? g.tiles_n : (int)ceil_div(g.np, 64 * t);
  g.per = SYM ? g.tiles_n * (g.tiles_n + 1) / 2 : g.tiles_m * g.tiles_n;
  const dim3 grid((unsigned)(g.per * g.batch)), block(256);
  // Loads further ahead where few tiles leave LDS to spare: 136 tiles of 64 and 16
  // stages 7.0 us instead of 9.9, but 528 of them and 32 stages 24 instead of 21;
  // 136 tiles of 128 and 32 stages 19.4 instead of 21.0.  Eight stages ahead gained
  // nothing over four.
  const int64_t tiles = (int64_t)g.per * g.batch;
  if (t == 4) hipLaunchKernelGGL((ns_product_kernel<4, 2, MODE, TW>), grid, block, 0, stream, g);
  else if (t == 2 && tiles <= NS_CUS) hipLaunchKernelGGL((ns_product_kernel<2, 4, MODE, TW>), grid, block, 0, stream, g);
  else if (t == 2) hipLaunchKernelGGL((ns_product_kernel<2, 2, MODE, TW>), grid, block, 0, stream, g);
  else if (t == 1 && tiles <= 2 * NS_CUS) hipLaunchKernelGGL((ns_product_kernel<1, 4, MODE, TW>), grid, block, 0, stream, g);
  else if (t == 1) hipLaunchKernelGGL((ns_product_kernel<1, 2, MODE, TW>), grid, block, 0, stream, g);
  else if constexpr (SYM) hipLaunchKernelGGL((ns_product_kernel<3, 2, MODE, TW>), grid, block, 0, stream, g);
}

// The time of steps together: A, P and the whole product, and for each step after the first
// T, R, P and Q.
static double ns_group_us(int64_t mp, int64_t np, int64_t batch, int steps) {
  double gram, small, whole;
  ns_tile(mp, np, np / 64, batch, true, &gram);
  ns_tile(mp, np, mp / 64, batch, true, &small);
  ns_tile(mp, np, mp / 64, batch, false, &whole);
  return gram + whole + small * (1 + 4 * (steps - 1));
}

// Whether steps are taken two and two.  How far R = A's rounding errors may grow
// within a pair: max(a + b s^2 + c s^4)^2, 12 for the Muon optimiser's step.
// Errors of the result in emulation, one by one, in pairs, and with three at the
// beginning, of noise, eight directions 30 times above it, and one (a constant)
// 100 and 1000 times above it: 1024 x 2048 0.06, 0.1, 0.06%; 0.01, 0.02, 0.08%; 0.01, 0.03,
// 0.3%; 0.1, 0.2, 1.2%; 256 x 1024 0.08, 0.07, 0.15% and 0.06, 0.13, 0.34%; 128 x 512 0.07,
// 0.06, 0.14% and 0.10, 0.19, 0.47%.  So two steps go together from 512 on and
// three nowhere, although they would save another pass over the long side (16384 x
// 4096 2.88 ms): with R and T as pairs of fp16, as X is, the three's error stays where
// it is, for P's rounding makes it.
constexpr double NS_PAIR_GROWTH = 16.0;

static bool ns_pairs(int64_t mp, int64_t np, int64_t batch, int steps, const double* qmax) {
  if (mp < NS_PAIRS_FROM || np <= mp) return false;
  for (int k = 0; k + 1 < steps; ++k)
    if (qmax[k] * qmax[k] > NS_PAIR_GROWTH) return false;
  return ns_group_us(mp, np, batch, 2) < 2 * ns_group_us(mp, np, batch, 1);
}

template <typename TG, typename TM>
static void muon_begin(const MuonIn& in, int64_t batch, hipStream_t stream) {
  hipLaunchKernelGGL((muon_norm_kernel<TG, TM>), dim3((unsigned)in.parts, (unsigned)batch), dim3(256), 0, stream, in);
  hipLaunchKernelGGL((muon_start_kernel<TG, TM>), dim3((unsigned)((in.mp / MT) * (in.np / MT)), (unsigned)batch), dim3(256), 0,
                     stream, in);
}

template <typename TG, typename TM>
static void short_run(ShortArgs a, int64_t batch, bool w_bf16, double growth, hipStream_t stream) {
  const int64_t n = a.in.tall ? a.in.rows : a.in.cols;
  if (a.chunks == 0) {
    if (w_bf16) hipLaunchKernelGGL((tiny_kernel<TG, TM, bf16_t>), dim3((unsigned)batch), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((tiny_kernel<TG, TM, float>), dim3((unsigned)batch), dim3(256), 0, stream, a);
    return;
  }
  const dim3 grid((unsigned)ceil_div(n, 64), (unsigned)batch), parts((unsigned)a.chunks, (unsigned)batch);
  if (growth > SHORT_GROWTH) {
    auto step = [&] {
      if (w_bf16) hipLaunchKernelGGL((short_wide_step_kernel<bf16_t>), grid, dim3(256), 0, stream, a);
      else hipLaunchKernelGGL((short_wide_step_kernel<float>), grid, dim3(256), 0, stream, a);
    };
    hipLaunchKernelGGL((short_wide_start_kernel<TG, TM>), grid, dim3(256), 0, stream, a);
    if (growth <= SHORT_WIDE_GROWTH) {
      a.step = -1;
      hipLaunchKernelGGL(short_wide_gram_kernel, parts, dim3(256), 0, stream, a);
      hipLaunchKernelGGL(short_steps_kernel, dim3((unsigned)batch), dim3(SSTEP_THR), 0, stream, a);
      step();
      return;
    }
    for (a.step = 0; a.step < a.steps; ++a.step) {
      hipLaunchKernelGGL(short_wide_gram_kernel, parts, dim3(256), 0, stream, a);
      hipLaunchKernelGGL(short_poly_kernel, dim3((unsigned)batch), dim3(SSTEP_THR), 0, stream, a);
      step();
    }
    return;
  }
  a.p = nullptr;
  hipLaunchKernelGGL((short_gram_kernel<TG, TM>), parts, dim3(256), 0, stream, a);
  hipLaunchKernelGGL(short_steps_kernel, dim3((unsigned)batch), dim3(SSTEP_THR), 0, stream, a);
  if (w_bf16) hipLaunchKernelGGL((short_apply_kernel<TG, TM, bf16_t>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((short_apply_kernel<TG, TM, float>), grid, dim3(256), 0, stream, a);
}

// X from `in`, the steps, and the last of them into g's weight.
static void ns_run(const NsPlan& h, MuonIn in, NsArgs g, int64_t batch, const float* coef, int steps, float scale, const double* qmax, uint8_t* ws,
                   hipStream_t stream) {
  if (h.blocks) {
    ShortArgs a = {};
    a.in = in;
    a.in.tall = in.rows > in.cols;
    a.blocks = h.blocks;
    a.chunks = h.chunks;
    a.part = (double*)(ws + h.part); a.q = (float*)(ws + h.q); a.inv = (double*)(ws + h.inv);
    a.x = (double*)(ws + h.x64); a.p = (double*)(ws + h.q);
    double grown = 1.0, most = 1.0;             // by any run of steps
    for (int k = 0; k < steps; ++k) {
      grown = std::max(grown, 1.0) * qmax[k];
      most = std::max(most, grown);
    }
    std::copy(coef, coef + 3 * steps, a.coef);
    a.steps = steps;
    a.hold = scale;
    a.w = g.w; a.ldw = g.ldw; a.sw = g.sw; a.update = g.update;
    a.lr = g.lr; a.lr_by = g.lr_by; a.decay = g.decay; a.scale = g.scale;
    if (in.g_bf16) {
      if (in.m_bf16) short_run<bf16_t, bf16_t>(a, batch, g.w_bf16, most, stream);
      else short_run<bf16_t, float>(a, batch, g.w_bf16, most, stream);
    } else {
      if (in.m_bf16) short_run<float, bf16_t>(a, batch, g.w_bf16, most, stream);
      else short_run<float, float>(a, batch, g.w_bf16, most, stream);
    }
    return;
  }
  in.mp = (int)h.mp; in.np = (int)h.np; in.tall = in.rows > in.cols; in.parts = h.parts;
  in.part = (double*)(ws + h.part);
  in.scale = scale;
  in.hi = ws + h.hi[0]; in.lo = ws + h.lo[0];
  if (in.g_bf16) {
    if (in.m_bf16) muon_begin<bf16_t, bf16_t>(in, batch, stream);
    else muon_begin<bf16_t, float>(in, batch, stream);
  } else {
    if (in.m_bf16) muon_begin<float, bf16_t>(in, batch, stream);
    else muon_begin<float, float>(in, batch, stream);
  }
  g.mp = (int)h.mp; g.np = (int)h.np; g.batch = (int)batch;
  g.inv = 1.0f / scale;
  g.tall = in.tall; g.rows = in.rows; g.cols = in.cols;
  const bool pairs = ns_pairs(h.mp, h.np, batch, steps, qmax);
  uint8_t *R = ws + h.gram, *T = ws + h.turn, *P = ws + h.poly, *P2 = ws + h.poly2, *J = ws + h.join;
  float* diag[3] = {(float*)(ws + h.diag), (float*)(ws + h.diag) + batch * h.mp, (float*)(ws + h.diag) + 2 * batch * h.mp};
  int turn = 0;
  for (int k = 0; k < steps; ++turn) {
    const int n = pairs && k + 2 <= steps ? 2 : 1;
    g.hi = ws + h.hi[turn & 1]; g.lo = ws + h.lo[turn & 1];
    g.hi2 = ws + h.hi[(turn + 1) & 1]; g.lo2 = ws + h.lo[(turn + 1) & 1];
    g.f = g.inv; g.out = R;
    ns_launch<NS_GRAM>(g, stream);
    // the pair's Q, held times qs, in q with its diagonal in dq
    uint8_t* q = P;
    float *dq = diag[0], qs = scale;
    double most = qmax[k];
    for (int i = 0; i < n; ++i, ++k) {
      const float* c = coef + 3 * k;
      uint8_t* p = i == 0 ? P : P2;
      float* dp = diag[i];
      g.a = c[0];
      g.left = g.right = g.src1 = R; g.f1 = c[1]; g.f = c[2] * g.inv; g.out = p; g.diag = dp;
      ns_launch<NS_POLY>(g, stream);
      if (i > 0) {
        most *= qmax[k];
        float to = qs;
        while (to * most > 49152.0) to *= 0.5f;
        g.left = p; g.right = q; g.src1 = q; g.row1 = dp; g.f1 = to / qs; g.src2 = p; g.col2 = dq; g.f2 = to / scale;
        g.f = to / (qs * scale); g.out = J; g.diag = diag[2];
        const float inv = g.inv;
        g.inv = 1.0f / to;
        ns_launch<NS_JOIN>(g, stream);
        g.inv = inv;
        q = J; dq = diag[2]; qs = to;
      }
      if (i + 1 < n) {
        g.left = p; g.row1 = dp; g.f1 = 1.0f; g.f = g.inv;
        g.right = g.src1 = R; g.out = T;
        ns_launch<NS_TURN>(g, stream);
        g.right = g.src1 = T; g.out = R;
        ns_launch<NS_TURN>(g, stream);
      }
    }
    g.q = q; g.diag = dq; g.f = 1.0f / qs;
    if (k < steps) ns_launch<NS_STEP>(g, stream);
    else if (g.w_bf16) ns_launch<NS_LAST, bf16_t>(g, stream);
    else ns_launch<NS_LAST, float>(g, stream);
  }
}

static pbs_status ns_check_call(const char* what, const float* coef, int64_t steps, float eps, const void* ws, size_t have, size_t need) {
  PBS_REQUIRE(coef && steps >= 1 && steps <= NS_MOST_STEPS, PBS_ERR_INVALID_ARG, "%s: needs the coefficients of 1 to %d steps", what,
              (int)NS_MOST_STEPS);
  PBS_REQUIRE(eps >= 0.0f && eps <= 3.4e38f, PBS_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", what);
  PBS_REQUIRE(need == 0 || (ws && ((uintptr_t)ws & 255) == 0), PBS_ERR_INVALID_ARG, "%s: the workspace is null or not 256-byte aligned",
              what);
  PBS_REQUIRE(have >= need, PBS_ERR_INVALID_ARG, "%s: the workspace holds %zu bytes, pbs_orthogonalize_bytes asks for %zu", what, have,
              need);
  return PBS_OK;
}

}  // namespace pbs

using namespace pbs;

extern "C" {

pbs_status pbs_orthogonalize_bytes(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  PBS_REQUIRE(bytes, PBS_ERR_INVALID_ARG, "pbs_orthogonalize_bytes: bytes is null");
  const pbs_status st = ns_check_dims("pbs_orthogonalize_bytes", batch, rows, cols);
  if (st != PBS_OK) return st;
  *bytes = batch && rows && cols ? ns_plan(batch, rows, cols).bytes : 0;
  return PBS_OK;
}

pbs_status pbs_orthogonalize(const void* x, pbs_format x_fmt, int64_t ldx, int64_t x_batch_stride, int64_t batch, int64_t rows,
                             int64_t cols, const float* coefficients, int steps, float eps, void* y, int64_t ldy,
                             int64_t y_batch_stride, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* what = "pbs_orthogonalize";
  pbs_status st = ns_check_dims(what, batch, rows, cols);
  if (st != PBS_OK) return st;
  const bool none = batch == 0 || rows == 0 || cols == 0;
  const NsPlan h = none ? NsPlan{} : ns_plan(batch, rows, cols);
  if ((st = ns_check_call(what, coefficients, steps, eps, workspace, workspace_bytes, h.bytes)) != PBS_OK) return st;
  float scale;
  double qmax[NS_MOST_STEPS];
  if ((st = ns_scale(what, coefficients, steps, &scale, qmax)) != PBS_OK) return st;
  if (none) return PBS_OK;
  if ((st = ns_check_matrix(what, "x", x, x_fmt, batch, rows, cols, ldx, x_batch_stride, false)) != PBS_OK) return st;
  if ((st = ns_check_matrix(what, "y", y, PBS_FMT_BF16, batch, rows, cols, ldy, y_batch_stride, true)) != PBS_OK) return st;
  PBS_REQUIRE(y != workspace && x != workspace, PBS_ERR_INVALID_ARG, "%s: a matrix is on the workspace's memory", what);
  PBS_REQUIRE(y != x || (x_fmt == PBS_FMT_BF16 && (rows == 1 || ldy == ldx) && (batch == 1 || y_batch_stride == x_batch_stride)),
              PBS_ERR_INVALID_ARG, "%s: y is x with another type or other strides", what);
  MuonIn in = {};
  in.g = x; in.ldg = ldx; in.sg = x_batch_stride; in.g_bf16 = x_fmt == PBS_FMT_BF16;
  in.rows = (int)rows; in.cols = (int)cols; in.eps = eps;
  NsArgs g = {};
  g.w = y; g.ldw = ldy; g.sw = y_batch_stride; g.w_bf16 = 1;
  log_dispatch("orthogonalize batch=%lld rows=%lld cols=%lld steps=%d scale=%g", (long long)batch, (long long)rows,
               (long long)cols, steps, scale);
  ns_run(h, in, g, batch, coefficients, steps, scale, qmax, (uint8_t*)workspace, stream);
  return check_launch(what);
}

pbs_status pbs_muon(void* w, pbs_format w_fmt, int64_t ldw, int64_t w_batch_stride, void* momentum, pbs_format m_fmt, int64_t ldm,
                    int64_t m_batch_stride, const void* grad, pbs_format g_fmt, int grad_transposed, int64_t ldg,
                    int64_t g_batch_stride, int64_t batch, int64_t rows, int64_t cols, double beta, int nesterov, float lr,
                    const float* lr_factor, float weight_decay, float scale, const float* coefficients, int steps, float eps,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* what = "pbs_muon";
  pbs_status st = ns_check_dims(what, batch, rows, cols);
  if (st != PBS_OK) return st;
  const bool none = batch == 0 || rows == 0 || cols == 0;
  const NsPlan h = none ? NsPlan{} : ns_plan(batch, rows, cols);
  if ((st = ns_check_call(what, coefficients, steps, eps, workspace, workspace_bytes, h.bytes)) != PBS_OK) return st;
  PBS_REQUIRE(beta >= 0.0 && beta <= 1.0, PBS_ERR_INVALID_ARG, "%s: beta must be in [0, 1]", what);
  PBS_REQUIRE(std::isfinite(lr) && std::isfinite(weight_decay) && std::isfinite(scale), PBS_ERR_INVALID_ARG,
              "%s: lr, weight_decay and scale must be finite", what);
  PBS_REQUIRE(((uintptr_t)lr_factor & 3) == 0, PBS_ERR_INVALID_ARG, "%s: lr_factor is not aligned to its elements", what);
  float hold;
  double qmax[NS_MOST_STEPS];
  if ((st = ns_scale(what, coefficients, steps, &hold, qmax)) != PBS_OK) return st;
  if (none) return PBS_OK;
  if ((st = ns_check_matrix(what, "w", w, w_fmt, batch, rows, cols, ldw, w_batch_stride, true)) != PBS_OK) return st;
  if ((st = ns_check_matrix(what, "momentum", momentum, m_fmt, batch, rows, cols, ldm, m_batch_stride, true)) != PBS_OK) return st;
  if ((st = ns_check_matrix(what, "grad", grad, g_fmt, batch, grad_transposed ? cols : rows, grad_transposed ? rows : cols, ldg,
                            g_batch_stride, false)) != PBS_OK)
    return st;
  PBS_REQUIRE(w != momentum && w != grad && momentum != grad, PBS_ERR_INVALID_ARG, "%s: w, momentum and grad must lie apart", what);
  PBS_REQUIRE(w != workspace && momentum != workspace && grad != workspace, PBS_ERR_INVALID_ARG,
              "%s: a matrix is on the workspace's memory", what);
  MuonIn in = {};
  in.g = grad; in.ldg = ldg; in.sg = g_batch_stride; in.g_bf16 = g_fmt == PBS_FMT_BF16; in.g_transposed = grad_transposed != 0;
  in.m = momentum; in.ldm = ldm; in.sm = m_batch_stride; in.m_bf16 = m_fmt == PBS_FMT_BF16;
  in.rows = (int)rows; in.cols = (int)cols; in.eps = eps;
  in.beta = (float)beta; in.one_less = (float)(1.0 - beta); in.nesterov = nesterov != 0;
  NsArgs g = {};
  g.w = w; g.ldw = ldw; g.sw = w_batch_stride; g.w_bf16 = w_fmt == PBS_FMT_BF16;
  g.update = 1; g.lr = lr; g.lr_by = lr_factor; g.decay = weight_decay; g.scale = scale;
  log_dispatch("muon batch=%lld rows=%lld cols=%lld steps=%d scale=%g", (long long)batch, (long long)rows, (long long)cols,
               steps, hold);
  ns_run(h, in, g, batch, coefficients, steps, hold, qmax, (uint8_t*)workspace, stream);
  return check_launch(what);
}

}  // extern "C"
