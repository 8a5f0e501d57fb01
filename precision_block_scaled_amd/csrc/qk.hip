// Norm of the queries and keys of each head and their rotation by position, in
// one pass, and its gradient.  For a token at position p and a row x [dim] of a
// head, with pairs (u_i, u_i') of the first `rot` values and angles p f_i:
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  u = n w
//   y_i = u_i cos - u_i' sin,  y_i' = u_i' cos + u_i sin,  the rest of y is u
// and from dy, with the rotation taken back:
//   g_i = dy_i cos + dy_i' sin,  g_i' = dy_i' cos - dy_i sin
//   dw = sum g n,  v = g w,  dx = r (v - n mean(v n))
//
// The angle is formed in 64 bits, in turns, and reduced before it is rounded
// to 32, so far positions lose nothing; everything else is fp32, rounded once
// at the store.  dw is summed in registers over a workgroup's strip of tokens
// and its strips are joined in their order, so identical inputs give identical
// bytes.
//
// Bound by memory: on 15872 tokens of 32 + 32 heads of 128 in bf16 the forward
// pass takes 101 us (5.15 TB/s of the 520 MB it must read and write, a large
// copy's rate) and the gradient, with 32 heads of values, 211 us (4.95 TB/s of
// 1040 MB).  Few tokens are bound by latency: 16 of 32 + 8 heads 7 us.
//
// A row is spread over G lanes; a lane holds units of two chunks of CH values,
// the two that the rotation takes together, so it turns its values by itself.
// A wave takes one token and several of its heads, of which all need the same
// cosines: each is formed once and handed round through LDS.
#include "device.hpp"
#include "host.hpp"

#include <algorithm>

namespace pbs {

constexpr int QK_WAVES = 4, QK_THR = 64 * QK_WAVES, QK_MOST_DIM = 512;

// A tensor [batch, seq, heads, dim], the last axis contiguous.
struct QkTensor {
  const void* p;
  int64_t sb, ss, sh;
};

// Queries, keys, or the values that the gradient only copies.
struct QkPart {
  QkTensor x, dy, out;     // dy: gradient only.  Values: dy is copied to out.
  const void* w;           // may be null: 1
  int heads, blocks;       // blocks: groups of heads that a token's row is cut into
  int strips;              // gradient: workgroups that share the part's tokens
  int first;               // gradient: the part's first workgroup
};

struct QkArgs {
  QkPart part[3];
  const int64_t* pos;      // may be null: the place in the sequence
  int64_t pos_sb;
  const double* freqs;     // [rot / 2]
  int64_t tokens, items;   // items: tokens x blocks of all parts
  int seq, dim, rot, interleaved, norm, w_bf16;
  int heads_each;          // heads of a block
  float eps;
  uint32_t* most;          // gradient: a workgroup's max |value| as stored; may be null
  float* dw;               // gradient: [workgroups of q and k][dim]; may be null
};

__device__ __forceinline__ uint32_t qk_pk(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const f2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

// CH consecutive values as they lie in memory; CH 4 and 8 take aligned
// addresses (8 or 16 bytes).
template <typename T, int CH>
struct QkRaw {
  static constexpr int WORDS = CH * (int)sizeof(T) / 4;
  uint32_t w[WORDS ? WORDS : 1];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (WORDS ? WORDS : 1); ++k) w[k] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (CH == 1) {
      if constexpr (sizeof(T) == 4) w[0] = *(const uint32_t*)p;
      else w[0] = *(const uint16_t*)p;
    } else if constexpr (WORDS == 2) {
      const uint2 u = *(const uint2*)p;
      w[0] = u.x; w[1] = u.y;
    } else {
#pragma unroll
      for (int k = 0; k < WORDS / 4; ++k) {
        const uint4 u = ((const uint4*)p)[k];
        w[4 * k] = u.x; w[4 * k + 1] = u.y; w[4 * k + 2] = u.z; w[4 * k + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(CH > 1 && (i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

// CH values rounded to T, as they go to memory, and their largest magnitude as
// stored, as fp32 bits.  (Rounded ahead of the condition that the store hangs
// on: a branch around both made the compiler keep the values in scratch.)
template <typename T, int CH>
struct QkOut {
  static constexpr int WORDS = QkRaw<T, CH>::WORDS ? QkRaw<T, CH>::WORDS : 1;
  uint32_t w[WORDS], most;
  __device__ __forceinline__ QkOut(const float (&v)[2 * CH], int first) {
    most = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        w[k] = __float_as_uint(v[first + k]);
        most = max(most, w[k] & 0x7FFFFFFFu);
      }
    } else if constexpr (CH == 1) {
      w[0] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[first]);
      most = (w[0] & 0x7FFFu) << 16;
    } else {
#pragma unroll
      for (int k = 0; k < CH / 2; ++k) {
        w[k] = qk_pk(v[first + 2 * k], v[first + 2 * k + 1]);
        most = max(most, max((w[k] & 0x7FFFu) << 16, w[k] & 0x7FFF0000u));
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (CH == 1) {
      if constexpr (sizeof(T) == 4) *(uint32_t*)p = w[0];
      else *(uint16_t*)p = (uint16_t)w[0];
    } else if constexpr (WORDS == 2) {
      *(uint2*)p = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < WORDS / 4; ++k) ((uint4*)p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
  }
};

// Sum over the G lanes of a group, to each of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Where a unit's two chunks begin in a row, and whether they are turned and
// there at all.  Pairs that lie half of `rot` apart: the chunks at CH u and rot
// / 2 + CH u; neighbouring pairs, and what is not turned: two chunks in a row.
struct QkUnit {
  int a, b, pair;          // pair: the unit's first angle, -1: not turned
  bool has_a, has_b;
};
template <int CH>
__device__ __forceinline__ QkUnit qk_unit(int u, int dim, int rot, int interleaved) {
  QkUnit q;
  const int turned = rot / 2 / CH;
  if (u < turned) {
    q.pair = CH * u;
    q.a = interleaved ? 2 * CH * u : CH * u;
    q.b = interleaved ? q.a + CH : rot / 2 + CH * u;
    q.has_a = q.has_b = true;
  } else {
    q.pair = -1;
    q.a = rot + 2 * CH * (u - turned);
    q.b = q.a + CH;
    q.has_a = q.a < dim;
    q.has_b = q.b < dim;
    if (!q.has_a) q.a = 0;
    if (!q.has_b) q.b = 0;
  }
  return q;
}

// Turns a unit's values by +- its angles.  INTER: pairs are neighbours (a
// kernel of its own: a branch here made the compiler choose between addresses
// and keep the values in scratch); single values lie as pairs either way.
template <int CH, bool INTER>
__device__ __forceinline__ void qk_turn(float (&v)[2 * CH], const float2 (&cs)[CH], float sign) {
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float& u = v[INTER ? 2 * k : k];
    float& w = v[INTER ? 2 * k + 1 : CH + k];
    const float p = u, q = w, c = cs[k].x, s = sign * cs[k].y;
    u = p * c - q * s;
    w = q * c + p * s;
  }
}

// cos and sin of a token's angles into the wave's part of LDS.
__device__ __forceinline__ void qk_angles(const QkArgs& a, int64_t pos, float2* cs) {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int i = threadIdx.x & 63; i < a.rot / 2; i += 64) {
    double t = (double)pos * a.freqs[i] * 0.15915494309189533577;      // 1 / (2 pi)
    t -= rint(t);
    float s, c;
    sincospif(2.0f * (float)t, &s, &c);
    cs[i] = make_float2(c, s);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One token's heads h0 .. h1 of a part.  UN rounds of 64 / G heads are loaded
// before the first is used.
template <typename TX, typename TY, int CH, bool INTER, int G, int NU, int UN, bool GRAD>
struct QkRows {
  static constexpr int PER = 64 / G;
  QkUnit u[NU];
  float w[NU][2 * CH];
  float dw[GRAD ? NU : 1][2 * CH];

  __device__ __forceinline__ void init(const QkArgs& a, const QkPart& p) {
    const int li = (threadIdx.x & 63) % G;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      u[k] = qk_unit<CH>(li + G * k, a.dim, a.rot, a.interleaved);
#pragma unroll
      for (int i = 0; i < 2 * CH; ++i) {
        const bool has = i < CH ? u[k].has_a : u[k].has_b;
        const int at = i < CH ? u[k].a + i : u[k].b + i - CH;
        w[k][i] = !has ? 0.0f : !p.w ? 1.0f : a.w_bf16 ? bf16_to_float(((const bf16_t*)p.w)[at]) : ((const float*)p.w)[at];
        if (GRAD) dw[k][i] = 0.0f;
      }
    }
  }

  template <typename T>
  __device__ __forceinline__ void load(const T* row, bool there, QkRaw<T, CH> (&v)[NU][2]) const {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      v[k][0].zero();
      v[k][1].zero();
      if (there && u[k].has_a) v[k][0].load(row + u[k].a);
      if (there && u[k].has_b) v[k][1].load(row + u[k].b);
    }
  }
  template <typename T>
  __device__ __forceinline__ uint32_t store(T* row, bool there, const float (&v)[NU][2 * CH]) const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const QkOut<T, CH> a(v[k], 0), b(v[k], CH);
      if (there && u[k].has_a) {
        a.store(row + u[k].a);
        m = max(m, a.most);
      }
      if (there && u[k].has_b) {
        b.store(row + u[k].b);
        m = max(m, b.most);
      }
    }
    return m;
  }

  __device__ __forceinline__ uint32_t run(const QkArgs& a, const QkPart& p, int64_t token, int h0, int h1, float2* lds) {
    const int b = (int)(token / a.seq), s = (int)(token - (int64_t)b * a.seq);
    const int64_t pos = a.rot && a.pos ? a.pos[b * a.pos_sb + s] : s;
    const TX* x = (const TX*)p.x.p + b * p.x.sb + s * p.x.ss;
    const TY* dy = GRAD ? (const TY*)p.dy.p + b * p.dy.sb + s * p.dy.ss : nullptr;
    const int64_t o = b * p.out.sb + s * p.out.ss;
    const float inv = 1.0f / (float)a.dim;
    uint32_t mx = 0;
    const int g0 = (threadIdx.x & 63) / G;
    QkRaw<TX, CH> rx[UN][NU][2];
    QkRaw<TY, CH> ry[GRAD ? UN : 1][NU][2];
    auto fetch = [&](int h) {
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        load(x + (h + n * PER) * p.x.sh, h + n * PER < h1, rx[n]);
        if constexpr (GRAD) load(dy + (h + n * PER) * p.dy.sh, h + n * PER < h1, ry[n]);
      }
    };
    // the first rows are on their way while the angles are formed
    fetch(h0 + g0);
    if (a.rot) qk_angles(a, pos, lds);
    float2 cs[NU][CH];
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i) cs[k][i] = u[k].pair >= 0 ? lds[u[k].pair + i] : make_float2(1.0f, 0.0f);
    for (int h = h0 + g0; h - g0 < h1; h += PER * UN) {
      if (h - g0 > h0) fetch(h);
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        const bool there = h + n * PER < h1;
        float v[NU][2 * CH], g[NU][2 * CH];
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2 * CH; ++i) {
            v[k][i] = rx[n][k][i / CH].get(i % CH);
            if constexpr (GRAD) g[k][i] = ry[n][k][i / CH].get(i % CH);
          }
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2 * CH; ++i) sum = __builtin_fmaf(v[k][i], v[k][i], sum);
        if constexpr (!GRAD) {
          const float r = a.norm ? 1.0f / sqrtf(group_sum<G>(sum) * inv + a.eps) : 1.0f;
#pragma unroll
          for (int k = 0; k < NU; ++k) {
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) v[k][i] = v[k][i] * r * w[k][i];
            if (u[k].pair >= 0) qk_turn<CH, INTER>(v[k], cs[k], 1.0f);
          }
          store((TY*)p.out.p + o + (h + n * PER) * p.out.sh, there, v);
        } else {
          float dot = 0.0f;
#pragma unroll
          for (int k = 0; k < NU; ++k) {
            if (u[k].pair >= 0) qk_turn<CH, INTER>(g[k], cs[k], -1.0f);
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) dot = __builtin_fmaf(g[k][i] * w[k][i], v[k][i], dot);
          }
          // (a row past the heads adds nothing to dw: with eps 0 its zeros would give 0 / 0)
          const float squares = group_sum<G>(sum) * inv + a.eps;
          const float r = a.norm ? there ? 1.0f / sqrtf(squares) : 0.0f : 1.0f;
          const float mean = a.norm ? group_sum<G>(dot) * inv * r : 0.0f;       // mean(v n)
#pragma unroll
          for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int i = 0; i < 2 * CH; ++i) {
              const float nrm = v[k][i] * r;
              dw[k][i] = __builtin_fmaf(g[k][i], nrm, dw[k][i]);
              // (without the norm dx does not depend on x, whatever x is)
              v[k][i] = r * (g[k][i] * w[k][i] - (a.norm ? nrm * mean : 0.0f));
            }
          mx = max(mx, store((TX*)p.out.p + o + (h + n * PER) * p.out.sh, there, v));
        }
      }
    }
    return mx;
  }
};

template <typename TX, typename TY, int CH, bool INTER, int G, int NU>
__global__ __launch_bounds__(QK_THR) void qk_norm_rope_kernel(QkArgs a) {
  __shared__ float2 cs[QK_WAVES][QK_MOST_DIM / 2];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t item = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * QK_WAVES + w;
  if (item >= a.items) return;
  const int64_t queries = a.tokens * a.part[0].blocks;
  const int which = item < queries ? 0 : 1;
  const QkPart& p = a.part[which];
  if (which) item -= queries;
  const int64_t token = item / p.blocks;
  const int h0 = (int)(item - token * p.blocks) * a.heads_each;
  QkRows<TX, TY, CH, INTER, G, NU, CH == 8 ? 4 : 2, false> rows;
  rows.init(a, p);
  rows.run(a, p, token, h0, min(h0 + a.heads_each, p.heads), cs[w]);
}

// A workgroup takes every strips-th group of QK_WAVES tokens of one part.
template <typename TX, typename TY, int CH, bool INTER, int G, int NU>
__global__ __launch_bounds__(QK_THR) void qk_norm_rope_grad_kernel(QkArgs a) {
  __shared__ float2 cs[QK_WAVES][QK_MOST_DIM / 2];
  __shared__ float sums[QK_WAVES][QK_MOST_DIM];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = blockIdx.x;
  const int which = block < a.part[1].first ? 0 : block < a.part[2].first ? 1 : 2;
  const QkPart& p = a.part[which];
  const int strip = block - p.first;
  uint32_t mx = 0;
  if (which == 2) {
    // chunk lane + 64 j of a token's values; eight loads ahead of their stores
    constexpr int AHEAD = 8;
    const int n = a.dim / CH, all = n * p.heads, dh = 64 / n, dc = 64 - dh * n;
    for (int64_t t = (int64_t)strip * QK_WAVES + w; t < a.tokens; t += (int64_t)p.strips * QK_WAVES) {
      const int b = (int)(t / a.seq), s = (int)(t - (int64_t)b * a.seq);
      const TY* from = (const TY*)p.dy.p + b * p.dy.sb + s * p.dy.ss;
      TX* to = (TX*)p.out.p + b * p.out.sb + s * p.out.ss;
      int h = lane / n, c = lane - h * n;
      for (int i = lane; i < all; i += 64 * AHEAD) {
        QkRaw<TY, CH> r[AHEAD];
        int64_t at[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          if (i + 64 * j < all) r[j].load(from + h * p.dy.sh + c * CH);
          at[j] = h * p.out.sh + c * CH;
          c += dc;
          h += dh + (c >= n ? 1 : 0);
          c -= c >= n ? n : 0;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          float v[2 * CH];
#pragma unroll
          for (int k = 0; k < CH; ++k) v[k] = r[j].get(k);
          const QkOut<TX, CH> o(v, 0);
          if (i + 64 * j < all) {
            o.store(to + at[j]);
            mx = max(mx, o.most);
          }
        }
      }
    }
  } else {
    QkRows<TX, TY, CH, INTER, G, NU, 2, true> rows;
    rows.init(a, p);
    for (int64_t t = (int64_t)strip * QK_WAVES + w; t < a.tokens; t += (int64_t)p.strips * QK_WAVES)
      mx = max(mx, rows.run(a, p, t, 0, p.heads, cs[w]));
    if (a.dw) {
      // the wave's groups, then its waves
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2 * CH; ++i) {
          float v = rows.dw[k][i];
#pragma unroll
          for (int o = G; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
          const bool has = i < CH ? rows.u[k].has_a : rows.u[k].has_b;
          if (lane < G && has) sums[w][i < CH ? rows.u[k].a + i : rows.u[k].b + i - CH] = v;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < a.dim; i += QK_THR) {
        float v = sums[0][i];
#pragma unroll
        for (int q = 1; q < QK_WAVES; ++q) v += sums[q][i];
        a.dw[(int64_t)block * a.dim + i] = v;
      }
    }
  }
  if (a.most) {
    __shared__ uint32_t most[QK_WAVES];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o, 64));
    if (lane == 0) most[w] = mx;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int q = 1; q < QK_WAVES; ++q) mx = max(mx, most[q]);
      a.most[block] = mx;
    }
  }
}

__global__ void qk_fill_kernel(uint32_t* p, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0u;
}

// dw = the sum of its strips, a column's by 64 threads, each every 64th strip
// (16 threads of it took 8 us for 512 strips, these 4); and the maximum over the
// workgroups, by a workgroup of its own.
constexpr int QK_JOIN_COLS = 16, QK_JOIN_ROWS = 64, QK_JOIN_THR = QK_JOIN_COLS * QK_JOIN_ROWS;
__global__ __launch_bounds__(QK_JOIN_THR) void qk_join_kernel(QkArgs a, float* dqw, float* dkw, uint32_t* amax, int all) {
  __shared__ float part[QK_JOIN_ROWS][QK_JOIN_COLS];
  if (blockIdx.y == 2) {
    if (!amax || blockIdx.x) return;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < all; i += QK_JOIN_THR) m = max(m, a.most[i]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    uint32_t* most = (uint32_t*)part;
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < QK_JOIN_THR / 64; ++i) m = max(m, most[i]);
      *amax = m;
    }
    return;
  }
  const QkPart& p = a.part[blockIdx.y];
  float* out = blockIdx.y ? dkw : dqw;
  if (!out) return;
  const int c = blockIdx.x * QK_JOIN_COLS + threadIdx.x % QK_JOIN_COLS, r = threadIdx.x / QK_JOIN_COLS;
  float s = 0.0f;
  if (c < a.dim) {
    const float* from = a.dw + (int64_t)p.first * a.dim + c;
#pragma unroll 4
    for (int i = r; i < p.strips; i += QK_JOIN_ROWS) s += from[(int64_t)i * a.dim];
  }
  part[r][threadIdx.x % QK_JOIN_COLS] = s;
  __syncthreads();
  if (r == 0 && c < a.dim) {
#pragma unroll
    for (int i = 1; i < QK_JOIN_ROWS; ++i) s += part[i][threadIdx.x];
    out[c] = s;
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Workgroups of a gradient: what the card holds at a time (three a compute
// unit), shared out by the parts' cost a token (a fixed part, the angles and the
// first loads' latency, and the rounds of heads).  15872 tokens of 32 + 32 + 32
// heads take 211 us, 8191 of 32 + 8 + 8 70 us; with 1024 workgroups 14 and 18%
// longer, with 2048 10 and 16%, four rounds of heads ahead instead of two 28 and
// 50% (registers).
constexpr int QK_STRIPS = 768;
static int qk_strips(int64_t tokens, int64_t cost, int64_t all) {
  const int64_t most = ceil_div(tokens, QK_WAVES);
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, QK_STRIPS * cost / std::max<int64_t>(all, 1)));
}
// Sums of the weights' gradients, dim a workgroup of q and k, and every workgroup's maximum.
static int64_t qk_most_strips(int64_t tokens) { return std::max<int64_t>(1, std::min<int64_t>(ceil_div(tokens, QK_WAVES), QK_STRIPS)); }
static size_t qk_grad_bytes(int64_t tokens, int64_t dim) {
  return (size_t)qk_most_strips(tokens) * (2 * (size_t)dim + 3) * 4;
}

// The widest chunks that the call's sizes, strides and addresses allow.
struct QkCall {
  const char* what;
  int64_t batch, seq, dim, rot;
  int interleaved, norm;
  float eps;
  bool x_bf16, y_bf16, w_bf16;
};

static bool qk_fits(const QkTensor& t, int bytes, int ch) {
  const int align = std::min(16, ch * bytes);
  return !t.p || (((uintptr_t)t.p & (align - 1)) == 0 && t.sb * bytes % align == 0 && t.ss * bytes % align == 0 &&
                  t.sh * bytes % align == 0);
}
static int qk_chunk(const QkCall& c, const QkArgs& a, bool grad) {
  for (int ch = grad ? 4 : 8; ch > 1; ch -= 4) {
    bool ok = c.dim % ch == 0 && c.rot / 2 % ch == 0;
    for (int i = 0; i < 3; ++i) {
      const QkPart& p = a.part[i];
      ok = ok && qk_fits(p.x, c.x_bf16 ? 2 : 4, ch) && qk_fits(p.dy, c.y_bf16 ? 2 : 4, ch) &&
           qk_fits(p.out, (grad ? c.x_bf16 : c.y_bf16) ? 2 : 4, ch);
    }
    if (ok) return ch;
  }
  return 1;
}

#define PBS_QK_TYPED(kernel, grid, ...)                                                                            \
  do {                                                                                                             \
    if (c.x_bf16 && c.y_bf16) hipLaunchKernelGGL((kernel<bf16_t, bf16_t, __VA_ARGS__>), grid, dim3(QK_THR), 0, stream, a);  \
    else if (c.x_bf16) hipLaunchKernelGGL((kernel<bf16_t, float, __VA_ARGS__>), grid, dim3(QK_THR), 0, stream, a); \
    else if (c.y_bf16) hipLaunchKernelGGL((kernel<float, bf16_t, __VA_ARGS__>), grid, dim3(QK_THR), 0, stream, a); \
    else hipLaunchKernelGGL((kernel<float, float, __VA_ARGS__>), grid, dim3(QK_THR), 0, stream, a);                \
  } while (0)
// Lanes a row: units of 16 values (chunks of 8, the forward pass), 8 (of 4) or 2 (single values).
#define PBS_QK_EIGHT(kernel, grid, INTER)                            \
  do {                                                               \
    if (c.dim <= 64) PBS_QK_TYPED(kernel, grid, 8, INTER, 4, 1);     \
    else if (c.dim <= 128) PBS_QK_TYPED(kernel, grid, 8, INTER, 8, 1);   \
    else if (c.dim <= 256) PBS_QK_TYPED(kernel, grid, 8, INTER, 16, 1);  \
    else PBS_QK_TYPED(kernel, grid, 8, INTER, 32, 1);                \
  } while (0)
#define PBS_QK_FOUR(kernel, grid, INTER)                             \
  do {                                                               \
    if (c.dim <= 64) PBS_QK_TYPED(kernel, grid, 4, INTER, 8, 1);     \
    else if (c.dim <= 128) PBS_QK_TYPED(kernel, grid, 4, INTER, 16, 1);  \
    else if (c.dim <= 256) PBS_QK_TYPED(kernel, grid, 4, INTER, 32, 1);  \
    else PBS_QK_TYPED(kernel, grid, 4, INTER, 64, 1);                \
  } while (0)
#define PBS_QK_FOUR_OR_ONE(kernel, grid)                             \
  do {                                                               \
    if (ch == 1) PBS_QK_TYPED(kernel, grid, 1, false, 64, 4);        \
    else if (c.interleaved) PBS_QK_FOUR(kernel, grid, true);         \
    else PBS_QK_FOUR(kernel, grid, false);                           \
  } while (0)
static int qk_per_wave(int ch, int64_t dim) {
  const int lanes = ch == 1 ? 64 : dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64;
  return 64 / (ch == 8 ? lanes / 2 : lanes);
}

static pbs_status qk_check_tensor(const QkCall& c, const char* name, const QkTensor& t, bool bf16) {
  PBS_REQUIRE(t.p, PBS_ERR_INVALID_ARG, "%s: %s is null", c.what, name);
  PBS_REQUIRE(((uintptr_t)t.p & (bf16 ? 1 : 3)) == 0, PBS_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", c.what,
              name);
  const int64_t most = 1ll << 40;
  PBS_REQUIRE(t.sb >= 0 && t.ss >= 0 && t.sh >= 0 && t.sb <= most && t.ss <= most && t.sh <= most, PBS_ERR_SHAPE,
              "%s: strides of %s must be in [0, 2^40]", c.what, name);
  return PBS_OK;
}

// An output's rows may not share memory: of the axes longer than one, from the
// smallest stride up, each steps over all that the smaller ones cover.
static bool qk_rows_apart(const QkCall& c, const QkTensor& t, int64_t heads) {
  int64_t n[3] = {c.batch, c.seq, heads}, s[3] = {t.sb, t.ss, t.sh};
  int64_t cover = c.dim;
  bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) break;
    if (s[at] < cover) return false;
    cover = s[at] * (n[at] - 1) + cover;
    used[at] = true;
  }
  return true;
}

static pbs_status qk_check(const QkCall& c, pbs_format x, pbs_format y, pbs_format w, int64_t heads, int64_t kv,
                           const double* freqs, const int64_t* pos, int64_t pos_sb) {
  PBS_REQUIRE((x == PBS_FMT_BF16 || x == PBS_FMT_F32) && (y == PBS_FMT_BF16 || y == PBS_FMT_F32) &&
                  (w == PBS_FMT_BF16 || w == PBS_FMT_F32),
              PBS_ERR_UNSUPPORTED, "%s: formats must be BF16 or F32", c.what);
  PBS_REQUIRE(c.batch >= 0 && c.seq >= 0 && heads >= 0 && kv >= 0 && heads <= 65536 && kv <= 65536 &&
                  c.batch <= (1 << 24) && c.seq <= (1 << 24) && c.batch * c.seq <= (1ll << 30),
              PBS_ERR_SHAPE, "%s: needs batch, seq in [0, 2^24], at most 2^30 tokens and 65536 heads (got %lld x %lld, %lld and %lld)",
              c.what, (long long)c.batch, (long long)c.seq, (long long)heads, (long long)kv);
  PBS_REQUIRE(c.dim >= 1 && c.dim <= QK_MOST_DIM, PBS_ERR_SHAPE, "%s: head_dim must be in [1, %d] (got %lld)", c.what,
              QK_MOST_DIM, (long long)c.dim);
  PBS_REQUIRE(c.rot >= 0 && c.rot <= c.dim && c.rot % 2 == 0, PBS_ERR_SHAPE,
              "%s: rot_dim must be even and in [0, head_dim] (got %lld)", c.what, (long long)c.rot);
  PBS_REQUIRE(c.rot == 0 || (freqs && ((uintptr_t)freqs & 7) == 0), PBS_ERR_INVALID_ARG,
              "%s: freqs is null or not aligned to its elements", c.what);
  PBS_REQUIRE(((uintptr_t)pos & 7) == 0, PBS_ERR_INVALID_ARG, "%s: positions are not aligned to their elements", c.what);
  PBS_REQUIRE(!pos || pos_sb == 0 || pos_sb >= c.seq, PBS_ERR_SHAPE,
              "%s: the positions' batch stride must be 0 or at least seq", c.what);
  PBS_REQUIRE(!c.norm || (c.eps >= 0.0f && c.eps <= 3.4e38f), PBS_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", c.what);
  return PBS_OK;
}

static QkTensor qk_tensor(const void* p, const int64_t* s) {
  QkTensor t = {p, 0, 0, 0};
  if (p && s) { t.sb = s[0]; t.ss = s[1]; t.sh = s[2]; }
  return t;
}

static bool qk_same_place(const QkTensor& out, bool out_bf16, const QkTensor& in, bool in_bf16) {
  return out.p == in.p && out_bf16 == in_bf16 && out.sb == in.sb && out.ss == in.ss && out.sh == in.sh;
}

}  // namespace pbs

using namespace pbs;

extern "C" {

pbs_status pbs_qk_norm_rope(const void* q, const int64_t* q_strides, int64_t heads, const void* k,
                            const int64_t* k_strides, int64_t kv_heads, pbs_format x_fmt, int64_t batch, int64_t seq,
                            int64_t head_dim, const void* q_weight, const void* k_weight, pbs_format w_fmt, int norm,
                            float eps, const int64_t* positions, int64_t pos_batch_stride, const double* freqs,
                            int64_t rot_dim, int interleaved, void* q_out, const int64_t* q_out_strides, void* k_out,
                            const int64_t* k_out_strides, pbs_format y_fmt, hipStream_t stream) {
  const QkCall c = {"pbs_qk_norm_rope", batch, seq, head_dim, rot_dim, interleaved != 0, norm != 0, eps,
                    x_fmt == PBS_FMT_BF16, y_fmt == PBS_FMT_BF16, w_fmt == PBS_FMT_BF16};
  pbs_status st = qk_check(c, x_fmt, y_fmt, w_fmt, heads, kv_heads, freqs, positions, pos_batch_stride);
  if (st != PBS_OK) return st;
  const int wb = c.w_bf16 ? 2 : 4;
  PBS_REQUIRE(((uintptr_t)q_weight & (wb - 1)) == 0 && ((uintptr_t)k_weight & (wb - 1)) == 0, PBS_ERR_INVALID_ARG,
              "pbs_qk_norm_rope: a weight is not aligned to its elements");
  QkArgs a = {};
  a.part[0].x = qk_tensor(q, q_strides); a.part[0].out = qk_tensor(q_out, q_out_strides);
  a.part[1].x = qk_tensor(k, k_strides); a.part[1].out = qk_tensor(k_out, k_out_strides);
  a.part[0].w = q_weight; a.part[1].w = k_weight;
  a.part[0].heads = (int)heads; a.part[1].heads = (int)kv_heads;
  a.tokens = batch * seq;
  const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
  const int64_t* strides[2][2] = {{q_strides, q_out_strides}, {k_strides, k_out_strides}};
  for (int i = 0; i < 2; ++i) {
    QkPart& p = a.part[i];
    if (p.heads == 0 || a.tokens == 0) { p.x = p.out = QkTensor{}; p.heads = 0; continue; }
    PBS_REQUIRE(strides[i][0] && strides[i][1], PBS_ERR_INVALID_ARG, "pbs_qk_norm_rope: strides of %s or %s are missing",
                names[i][0], names[i][1]);
    if ((st = qk_check_tensor(c, names[i][0], p.x, c.x_bf16)) != PBS_OK) return st;
    if ((st = qk_check_tensor(c, names[i][1], p.out, c.y_bf16)) != PBS_OK) return st;
    PBS_REQUIRE(qk_rows_apart(c, p.out, p.heads), PBS_ERR_SHAPE, "pbs_qk_norm_rope: rows of %s overlap", names[i][1]);
    for (int j = 0; j < 2; ++j)
      PBS_REQUIRE(p.out.p != a.part[j].x.p || (i == j && qk_same_place(p.out, c.y_bf16, p.x, c.x_bf16)), PBS_ERR_INVALID_ARG,
                  "pbs_qk_norm_rope: %s is on an input's memory with another type or other strides", names[i][1]);
  }
  if (a.part[0].heads + a.part[1].heads == 0) return PBS_OK;
  PBS_REQUIRE(a.part[0].out.p != a.part[1].out.p, PBS_ERR_INVALID_ARG, "pbs_qk_norm_rope: q_out and k_out are one tensor");
  a.pos = positions; a.pos_sb = pos_batch_stride; a.freqs = freqs;
  a.seq = (int)seq; a.dim = (int)head_dim; a.rot = (int)rot_dim;
  a.interleaved = c.interleaved; a.norm = c.norm; a.eps = eps; a.w_bf16 = c.w_bf16;
  const int ch = qk_chunk(c, a, false), per = qk_per_wave(ch, head_dim);
  // all of a token's heads for one wave, or fewer where that leaves the card's waves idle
  const int most = std::max(a.part[0].heads, a.part[1].heads);
  a.heads_each = (int)ceil_div(most, per) * per;
  while (a.heads_each > per && a.tokens * ceil_div(most, a.heads_each) < 4096)
    a.heads_each = (int)ceil_div(a.heads_each / per, 2) * per;
  for (int i = 0; i < 2; ++i) {
    a.part[i].blocks = (int)ceil_div(a.part[i].heads, a.heads_each);
    a.items += a.tokens * a.part[i].blocks;
  }
  // (an axis of a launch holds less than 2^32 threads)
  const int64_t groups = ceil_div(a.items, QK_WAVES), along = std::min<int64_t>(groups, 1 << 22);
  const dim3 grid((unsigned)along, (unsigned)ceil_div(groups, along));
  log_dispatch("qk_norm_rope tokens=%lld heads=%d+%d dim=%d rot=%d chunk=%d heads/wave=%d", (long long)a.tokens,
               a.part[0].heads, a.part[1].heads, a.dim, a.rot, ch, a.heads_each);
  if (ch != 8) PBS_QK_FOUR_OR_ONE(qk_norm_rope_kernel, grid);
  else if (c.interleaved) PBS_QK_EIGHT(qk_norm_rope_kernel, grid, true);
  else PBS_QK_EIGHT(qk_norm_rope_kernel, grid, false);
  return check_launch("pbs_qk_norm_rope");
}

pbs_status pbs_qk_norm_rope_grad_bytes(int64_t batch, int64_t seq, int64_t head_dim, size_t* bytes) {
  PBS_REQUIRE(bytes, PBS_ERR_INVALID_ARG, "pbs_qk_norm_rope_grad_bytes: bytes is null");
  PBS_REQUIRE(batch >= 0 && seq >= 0 && batch <= (1 << 24) && seq <= (1 << 24) && batch * seq <= (1ll << 30) &&
                  head_dim >= 1 && head_dim <= QK_MOST_DIM,
              PBS_ERR_SHAPE, "pbs_qk_norm_rope_grad_bytes: needs at most 2^30 tokens and head_dim in [1, %d]", QK_MOST_DIM);
  *bytes = qk_grad_bytes(batch * seq, head_dim);
  return PBS_OK;
}

pbs_status pbs_qk_norm_rope_grad(const void* dq, const int64_t* dq_strides, const void* dk, const int64_t* dk_strides,
                                 const void* dv, const int64_t* dv_strides, pbs_format y_fmt, const void* q,
                                 const int64_t* q_strides, int64_t heads, const void* k, const int64_t* k_strides,
                                 int64_t kv_heads, pbs_format x_fmt, int64_t batch, int64_t seq, int64_t head_dim,
                                 const void* q_weight, const void* k_weight, pbs_format w_fmt, int norm, float eps,
                                 const int64_t* positions, int64_t pos_batch_stride, const double* freqs,
                                 int64_t rot_dim, int interleaved, void* dq_out, const int64_t* dq_out_strides,
                                 void* dk_out, const int64_t* dk_out_strides, void* dv_out,
                                 const int64_t* dv_out_strides, float* dq_weight, float* dk_weight, float* amax_out,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const QkCall c = {"pbs_qk_norm_rope_grad", batch, seq, head_dim, rot_dim, interleaved != 0, norm != 0, eps,
                    x_fmt == PBS_FMT_BF16, y_fmt == PBS_FMT_BF16, w_fmt == PBS_FMT_BF16};
  pbs_status st = qk_check(c, x_fmt, y_fmt, w_fmt, heads, kv_heads, freqs, positions, pos_batch_stride);
  if (st != PBS_OK) return st;
  const int wb = c.w_bf16 ? 2 : 4;
  PBS_REQUIRE(((uintptr_t)q_weight & (wb - 1)) == 0 && ((uintptr_t)k_weight & (wb - 1)) == 0 &&
                  (((uintptr_t)dq_weight | (uintptr_t)dk_weight | (uintptr_t)amax_out) & 3) == 0,
              PBS_ERR_INVALID_ARG, "pbs_qk_norm_rope_grad: a vector is not aligned to its elements");
  PBS_REQUIRE((dv == nullptr) == (dv_out == nullptr), PBS_ERR_INVALID_ARG,
              "pbs_qk_norm_rope_grad: dv and dv_out go together");
  QkArgs a = {};
  a.part[0].x = qk_tensor(q, q_strides); a.part[0].dy = qk_tensor(dq, dq_strides); a.part[0].out = qk_tensor(dq_out, dq_out_strides);
  a.part[1].x = qk_tensor(k, k_strides); a.part[1].dy = qk_tensor(dk, dk_strides); a.part[1].out = qk_tensor(dk_out, dk_out_strides);
  a.part[2].dy = qk_tensor(dv, dv_strides); a.part[2].out = qk_tensor(dv_out, dv_out_strides);
  a.part[0].w = q_weight; a.part[1].w = k_weight;
  a.part[0].heads = (int)heads; a.part[1].heads = (int)kv_heads; a.part[2].heads = dv ? (int)kv_heads : 0;
  a.tokens = batch * seq;
  const char* names[3][3] = {{"q", "dq", "dq_out"}, {"k", "dk", "dk_out"}, {"v", "dv", "dv_out"}};
  const int64_t* strides[3][3] = {{q_strides, dq_strides, dq_out_strides}, {k_strides, dk_strides, dk_out_strides},
                                  {dv_strides, dv_strides, dv_out_strides}};
  for (int i = 0; i < 3; ++i) {
    QkPart& p = a.part[i];
    if (p.heads == 0 || a.tokens == 0) { p.x = p.dy = p.out = QkTensor{}; p.heads = 0; continue; }
    PBS_REQUIRE(strides[i][0] && strides[i][1] && strides[i][2], PBS_ERR_INVALID_ARG,
                "pbs_qk_norm_rope_grad: strides of %s, %s or %s are missing", names[i][0], names[i][1], names[i][2]);
    if (i < 2 && (st = qk_check_tensor(c, names[i][0], p.x, c.x_bf16)) != PBS_OK) return st;
    if ((st = qk_check_tensor(c, names[i][1], p.dy, c.y_bf16)) != PBS_OK) return st;
    if ((st = qk_check_tensor(c, names[i][2], p.out, c.x_bf16)) != PBS_OK) return st;
    PBS_REQUIRE(qk_rows_apart(c, p.out, p.heads), PBS_ERR_SHAPE, "pbs_qk_norm_rope_grad: rows of %s overlap", names[i][2]);
    for (int j = 0; j < 3; ++j) {
      const QkPart& o = a.part[j];
      PBS_REQUIRE(p.out.p != o.x.p || (i == j && qk_same_place(p.out, c.x_bf16, o.x, c.x_bf16)), PBS_ERR_INVALID_ARG,
                  "pbs_qk_norm_rope_grad: %s is on an input's memory with another type or other strides", names[i][2]);
      PBS_REQUIRE(p.out.p != o.dy.p || (i == j && qk_same_place(p.out, c.x_bf16, o.dy, c.y_bf16)), PBS_ERR_INVALID_ARG,
                  "pbs_qk_norm_rope_grad: %s is on an input's memory with another type or other strides", names[i][2]);
    }
  }
  const int all = a.part[0].heads + a.part[1].heads + a.part[2].heads;
  for (int i = 0; i < 3; ++i)
    PBS_REQUIRE(!a.part[i].out.p || a.part[i].out.p != a.part[(i + 1) % 3].out.p, PBS_ERR_INVALID_ARG,
                "pbs_qk_norm_rope_grad: %s and %s are one tensor", names[i][2], names[(i + 1) % 3][2]);
  PBS_REQUIRE(!dq_weight || dq_weight != dk_weight, PBS_ERR_INVALID_ARG, "pbs_qk_norm_rope_grad: dq_weight and dk_weight are one vector");
  const bool sums = all && (dq_weight || dk_weight);
  if (sums || (all && amax_out)) {
    PBS_REQUIRE(workspace && ((uintptr_t)workspace & 15) == 0, PBS_ERR_INVALID_ARG,
                "pbs_qk_norm_rope_grad: the workspace is null or not 16-byte aligned");
    const size_t need = qk_grad_bytes(a.tokens, head_dim);
    PBS_REQUIRE(workspace_bytes >= need, PBS_ERR_INVALID_ARG,
                "pbs_qk_norm_rope_grad: the workspace holds %zu bytes, pbs_qk_norm_rope_grad_bytes asks for %zu",
                workspace_bytes, need);
  }
  if (amax_out && all == 0) hipLaunchKernelGGL(qk_fill_kernel, dim3(1), dim3(64), 0, stream, (uint32_t*)amax_out, 1);
  // a part that has no rows leaves its weight's gradient zero
  for (int i = 0; i < 2; ++i)
    if (a.part[i].heads == 0 && (i ? dk_weight : dq_weight))
      hipLaunchKernelGGL(qk_fill_kernel, dim3(1), dim3(256), 0, stream, (uint32_t*)(i ? dk_weight : dq_weight), (int)head_dim);
  if (all == 0) return check_launch("pbs_qk_norm_rope_grad");
  a.pos = positions; a.pos_sb = pos_batch_stride; a.freqs = freqs;
  a.seq = (int)seq; a.dim = (int)head_dim; a.rot = (int)rot_dim;
  a.interleaved = c.interleaved; a.norm = c.norm; a.eps = eps; a.w_bf16 = c.w_bf16;
  a.most = amax_out ? (uint32_t*)workspace : nullptr;
  a.dw = sums ? (float*)workspace + 3 * qk_most_strips(a.tokens) : nullptr;
  const int ch = qk_chunk(c, a, true), per = qk_per_wave(ch, head_dim);
  auto cost = [&](int i) { return a.part[i].heads ? 6 + (i < 2 ? 6 : 2) * ceil_div(a.part[i].heads, 2 * per) : 0; };
  int grid = 0;
  for (int i = 0; i < 3; ++i) {
    QkPart& p = a.part[i];
    p.first = grid;
    p.strips = p.heads ? qk_strips(a.tokens, cost(i), cost(0) + cost(1) + cost(2)) : 0;
    grid += p.strips;
  }
  log_dispatch("qk_norm_rope_grad tokens=%lld heads=%d+%d+%d dim=%d rot=%d chunk=%d strips=%d+%d+%d", (long long)a.tokens,
               a.part[0].heads, a.part[1].heads, a.part[2].heads, a.dim, a.rot, ch, a.part[0].strips, a.part[1].strips,
               a.part[2].strips);
  PBS_QK_FOUR_OR_ONE(qk_norm_rope_grad_kernel, dim3((unsigned)grid));
  if (sums || amax_out)
    hipLaunchKernelGGL(qk_join_kernel, dim3((unsigned)ceil_div(head_dim, QK_JOIN_COLS), 3), dim3(QK_JOIN_THR), 0, stream, a,
                       a.part[0].heads ? dq_weight : nullptr, a.part[1].heads ? dk_weight : nullptr, (uint32_t*)amax_out, grid);
  return check_launch("pbs_qk_norm_rope_grad");
}

}  // extern "C"
