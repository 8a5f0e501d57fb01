// Losses of a linear head, from the hidden states and the head's weight,
// without keeping the logits:
//
//   z = x W^T / tau        x [tokens, hidden], W [vocab, hidden], both bf16
//   lse_t = log sum_v exp z_tv,   q_tv = exp(z_tv - lse_t)
//   loss_t = sum_s p_ts (log p_ts - z_t,id(t,s) + lse_t)
//   dz_tv = dloss_t / tau (q_tv - sum over the slots s with id(t,s) = v of p_ts)
//   dx = dz W,   dW = dz^T x
//
// Cross entropy is one slot with p = 1 and tau = 1; distillation has the
// softmax of a teacher's highest logits over tau in its slots.
//
// The loss multiplies x by W^T tile by tile and keeps, of each token's logits,
// the maximum and the sum of exponentials above it over half a tile's ids, and
// the slots' own logits; a second kernel joins them.  The
// gradient forms z again for a piece of the vocabulary at a time, turns it
// into dz (bf16, in the workspace) in the product's epilogue and multiplies
// that by W and, transposed, by x; what the rounding to bf16 leaves out of a
// token's few large values is added in fp32.  Tokens that take no part are left out:
// the others' rows are gathered first, so a masked token costs nothing and
// whatever its row of x holds reaches no sum.
//
// The products use the tiling of the library's BF16 GEMM: 256 x 256 outputs
// per workgroup of 4 waves (or 128 x 128, two workgroups a compute unit, where
// those would leave compute units idle), K stages of 64 values filled by
// LDS-DMA, v_mfma_f32_32x32x16_bf16.
//
// What bounds them: the matrix cores and the power they draw.  On 8192 x
// 131072 x 4096 the loss runs at 1430 TFLOP/s (6.1 ms) and the gradient at 1390
// (19.0 ms) with the matrix cores busy 80% of the time (dz 76%) at 1.6 to 1.67
// GHz; a large library product reaches 1490 on the same operands.  A K stage of a
// 256 x 256 tile takes 2220 cycles, 2048 of them matrix instructions, or 1.32
// to 1.4 us; a tile's fixed cost (first loads 2.3 us, the loss's epilogue 4) is
// 7% at hidden = 4096 and 13% at 2048.  Workgroups that stay and issue the next
// tile's loads ahead of the loss's epilogue, all at once or spread over it,
// took 1 to 2% fewer cycles a tile and no less time (within 1%).
#include "device.hpp"
#include "gemm_common.hpp"
#include "host.hpp"

#include <algorithm>
#include <type_traits>

namespace pbs {

enum { KMAJ = 0, MNMAJ = 1 };                    // how an operand is stored
enum { EPI_STATS = 0, EPI_DZ = 1, EPI_DX = 2, EPI_DW = 3 };
enum { ROW_OUT = 0, ROW_LIVE = 1, ROW_BAD = 2 }; // a token: no part, part, an id past the vocabulary

// dz goes into the products as bf16, each value off by up to 2^-8 of itself.
// Of a token's values one or a few stand out, those at the ids its teacher
// thinks likely: a row of dx, and the rows of dW that these ids have, hang on
// them alone, so their roundings do not average out and come to as much as the
// results' own rounding to bf16 (errors against 64 bits, in 2-norms, of dx and
// dW alike: 0.0023 to 0.0024, where their store alone is 0.0017).  What the
// rounding left out there is kept in fp32 and added to the products' sums ahead
// of their own rounding: rest * W's row to dx, rest * x's row to dW (0.0017 in
// cross entropy, 0.0018 in distillation).  These are the heavy slots: cross
// entropy's one, and distillation's with p > 1/5 (four at most; with those
// above 1/16 the error would be 0.0017 too, but they are three times as many).
// It costs 1 to 7% of a gradient, the more the shorter it is: 8192 x 131072 x
// 4096 18.77 -> 18.93 ms, 2048 x 32768 x 4096 1258 -> 1290 us, 512 x 32000 x 2048
// 195 -> 208, 129 x 5000 x 1024 36 -> 37.5; two terms for all of dz would cost
// half as much again.
// A row of dW whose id is heavy for many tokens averages their roundings after
// all: it is left as it is where they are more than MOST_SHARED.
constexpr int MOST_HEAVY = 4, MOST_SHARED = 8;
constexpr float HEAVY_P = 0.2f;
// The row of side of an id whose list begins at head, -1: none.
__device__ __forceinline__ int side_row(int head, int id, int by_id) { return head < 0 || !by_id ? head : id; }
// What rounding v to bf16 leaves out (nothing where that overflows).
__device__ __forceinline__ float bf16_rest(float v) {
  const float b = (float)(__bf16)v;
  return __builtin_fabsf(b) < __builtin_inff() ? v - b : 0.0f;
}

// Puts a place at the head of its id's list, in two steps around the exchange's
// latency; every lane of the wave takes part, those that are `here` with a
// place.  Lanes with the same id make one piece of the list and one exchange
// (gradient of 15872 tokens against 5000 ids of 1024, all with one target:
// 486 us, 606 with an exchange each, which queue at the one address).
struct Push {
  int before, last;        // lanes: the one below with the same id or -1, the highest with it
  int old;                 // there: what was at the head
};
__device__ __forceinline__ Push push_place(int* head, int id, int place, bool here) {
  const int lane = threadIdx.x & 63;
  Push q = {-1, lane, -1};
  for (uint64_t left = __ballot(here); left;) {
    const bool mine = here && id == __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    const uint64_t same = __ballot(mine), below = same & ((1ull << lane) - 1);
    if (mine) {
      q.before = below ? 63 - __clzll((long long)below) : -1;
      q.last = 63 - __clzll((long long)same);
    }
    left &= ~same;
  }
  if (here && q.last == lane) q.old = atomicExch(head + id, place);
  return q;
}
// What comes next in the list after the lane's place.
__device__ __forceinline__ int pushed_next(const Push& q, int place) {
  const int old = __shfl(q.old, q.last, 64), before = __shfl(place, q.before & 63, 64);
  return q.before < 0 ? old : before;
}

// v += f * (eight bf16 values)
__device__ __forceinline__ void add_bf16x8(float (&v)[8], float f, const uint4& u) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t b = k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w;
    v[2 * k] = __builtin_fmaf(f, __uint_as_float(b << 16), v[2 * k]);
    v[2 * k + 1] = __builtin_fmaf(f, __uint_as_float(b & 0xFFFF0000u), v[2 * k + 1]);
  }
}

struct HeadArgs {
  const uint8_t* x;        // [tokens, hidden]
  const uint8_t* xc;       // the live tokens' rows, used when not all are live
  const uint8_t* w;        // first row of this piece of W
  const int* live;         // {live rows, splits of dx, splits of dW}
  const int* row_of;       // live row -> token
  const int64_t* targets;  // cross entropy: the token's one slot, p = 1; else null and
  const int* state;        //   per token: ROW_*
  const int* ids;          //   [tokens][slots]: vocabulary ids, -1 unused
  const float* p;          //   [tokens][slots]
  float* zsel;             // [tokens][slots]: the slots' logits / tau
  float2* stats;           // [parts][rows]: maximum of a part of a row over log 2, sum of exponentials above it
  const float* lse;        // per token
  const float* dloss;      // per token
  uint16_t* dz;            // [rows][dz_ld]; PAIR: [rows][2][dz_ld], dz rounded and what that left out
  uint16_t* dx;            // dx itself, where one product gives all of it; else null and
  float* dx_part;          //   partial products of dx
  float* dw_part;          // partial products of dW
  const int* heavy;        // [tokens][heavy_n]: ids of the token's heavy slots, -1: none (null: dz is a pair)
  float* rest;             // [tokens][heavy_n]: what dz's rounding left out there
  int* head;               // [vocab]: one of the places of heavy that hold the id, -1: none (null: dW stays as it is)
  int* next;               // for every place another one with its id, -1: none (lists, in no order)
  float* side;             // rows of a bf16 dW before their rounding, those of the ids that a place holds
  int side_by_id;          // ... an id's row at the id, else at its head
  void* dw;                // this piece of dW
  int dx_blocks;           // workgroups of dx ahead of dW's
  int tokens, rows, hidden, slots;   // rows: tokens, rounded up to whole tiles
  int heavy_n;             // 1 in cross entropy, MOST_HEAVY in distillation
  int v0, nv;              // this piece: first id, ids in it
  int dz_ld;
  int vocab;
  int add;                 // the product is added to out
  int out_bf16;
  float inv_tau;
};

// Stage geometry for a tile of 64 TI x 64 TJ outputs: each of the 2 x 2 waves
// holds TI x TJ 32 x 32 tiles.
template <int T> constexpr int tile_bytes() { return 64 * T * ROWB; }
// Staging of a result tile in LDS: fp32, 128 rows a pass, or bf16, all rows at
// once.  16 bytes of padding a row: 16 lanes' 16-byte (32 lanes' 8-byte)
// accesses to consecutive rows then cover every bank.
constexpr int STAGE_ROWS = 128, STAGE_PAD = 16;
template <int TI, int TJ> constexpr int head_smem() {
  return cmax(cmax(2 * tile_bytes<TI>() + 3 * tile_bytes<TJ>(),
                   STAGE_ROWS * (64 * cmax(TI, TJ) * 4 + STAGE_PAD) + 64 * TJ * 4),
              64 * TJ * (64 * TI * 2 + STAGE_PAD));
}

// `bytes` bytes from p as one buffer resource, and a 16-byte load from it to LDS.
struct BufferRows {
  __amdgpu_buffer_rsrc_t r;
};
__device__ __forceinline__ BufferRows buffer_rows(const uint8_t* p, uint32_t bytes) {
  BufferRows b;
  b.r = __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, BUF_RSRC_WORD3);
  return b;
}
__device__ __forceinline__ void buffer_to_lds(const BufferRows& b, uint8_t* lds, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b.r, (lds_ptr_t)lds, 16, lane_off, off, 0, 0);
}

// K-major operand: load i (of 2 T) of wave w fills LDS rows 16 T w + 8 i ..
// + 7; lane l owns row + l / 8 and the chunk that the swizzle puts at l % 8.
// Rows past the end re-read the last one.
template <int T>
struct KLoad {
  BufferRows b;
  uint32_t off[2 * T];
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld, int row0, int rows, int w) {
    const int lane = threadIdx.x & 63;
    const int64_t span = (int64_t)(rows - row0) * ld;
    b = buffer_rows(p + (int64_t)row0 * ld, (uint32_t)(span < 0xFFFFFFFFll ? span : 0xFFFFFFFFll));
    const int last = rows - row0 - 1;
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) {
      const int t = 16 * T * w + 8 * i + (lane >> 3);
      off[i] = (uint32_t)(t < last ? t : last) * (uint32_t)ld + (uint32_t)(((lane & 7) ^ swz_key(t)) << 4);
    }
  }
  // K stage kt, `along` bytes further in every row
  __device__ __forceinline__ void load(int kt, int64_t along, uint8_t* tile, int w, int i) const {
    buffer_to_lds(b, tile + (w * 2 * T + i) * 1024, off[i], (uint32_t)(kt * ROWB + along));
  }
};

// MN-major operand (stored [K][MN]): a stage's 64 K rows of the tile's 64 T
// values go to LDS as they are, 16-byte chunk c of row k at chunk c ^ 4 (k &
// 3).  Chunks past the operand's width re-read its last one; K rows past its
// end (krows) re-read the last row, whose products the other operand's zeros
// take away.
template <int T>
struct MnLoad {
  static constexpr int CH = 8 * T;             // chunks per row
  static constexpr int RPL = 64 / CH;          // rows per load
  const uint8_t* base;
  int64_t ld;
  int krows;
  uint32_t off[2 * T];
  uint32_t c[2];                               // the lane's chunk in loads of even / odd i
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld_, int mn0, int nmn, int krows_, int w) {
    const int lane = threadIdx.x & 63;
    base = p + (int64_t)mn0 * 2;
    ld = ld_;
    krows = krows_;
    const int lastc = (nmn - mn0 - 8) >> 3;
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) {
      const int row = RPL * (2 * T * w + i) + lane / CH;
      int lc = (lane % CH) ^ (4 * (row & 3));
      lc = lc < lastc ? lc : lastc;
      if (i < 2) c[i] = (uint32_t)(lc << 4);
      off[i] = (uint32_t)row * (uint32_t)ld + (uint32_t)(lc << 4);
    }
  }
  __device__ __forceinline__ void load(int kt, int64_t along, uint8_t* tile, int w, int i) const {
    const int left = krows - 64 * kt;
    const uint32_t top = (uint32_t)((left < 64 ? left : 64) - 1) * (uint32_t)ld + c[i & 1];
    buffer_to_lds(buffer_rows(base + (int64_t)kt * 64 * ld + along, (uint32_t)(64 * ld)), tile + (w * 2 * T + i) * 1024,
                  off[i] < top ? off[i] : top, 0);
  }
};

typedef short i16x4 __attribute__((ext_vector_type(4)));
// The restrict-qualified pointer gives the transposing read the alias
// information by which the compiler tells it apart from LDS-DMA loads into
// the other stage; without it every such read waits for all of them.
__device__ __forceinline__ i16x4 head_read_tr16(const uint8_t* __restrict__ p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
}

// Fragments of one half stage (32 K values): x[tile][s] is the operand of
// K=16 step s of the half, lane (lr, lg) holding 8 K values of its row.
template <int T>
struct Half {
  i32x4 x[T][2];
};

template <int LD, int T>
constexpr int half_reads() { return LD == KMAJ ? 2 * T : 4 * T; }

template <int H, int LD, int T>
__device__ __forceinline__ void half_read(Half<T>& f, int d, const uint8_t* base, uint32_t lb) {
  if (LD == KMAJ) {
    const int tile = d >> 1, part = d & 1;
    f.x[tile][part] = *(const i32x4*)(base + tile * 4096 + (lb ^ (uint32_t)(((4 * H) ^ (2 * tile)) << 4) ^
                                                            (uint32_t)(part << 5)));
  } else {
    const int tile = d >> 2, s = (d >> 1) & 1, q = d & 1;
    const i16x4 v = head_read_tr16(base + (16 * (2 * H + s) + 4 * q) * (128 * T) + (lb ^ (uint32_t)(64 * tile)));
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

// Waits for all but this wave's last N loads and for its LDS reads, then for
// every wave.  (__syncthreads would wait for every load.)
template <int N>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ constexpr int part_lo(int n, int over, int m) { return m < over ? n * m / over : n; }
__device__ __forceinline__ constexpr int part_hi(int n, int over, int m) { return m < over ? n * (m + 1) / over : n; }

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// The product and its epilogues.
//
// A's K stages go through two LDS buffers, B's through three.  Phase A of
// stage kt multiplies its first half while its second half is read from LDS
// and the loads of B's stage kt + 2 are issued; then the wave waits for its
// own loads of stage kt + 1 (all but those just issued, an explicit vmcnt) and
// all waves meet; phase C multiplies the second half while the first half of
// stage kt + 1 is read and the loads of A's stage kt + 2 go into the buffer
// that was just read out.  The third B buffer is what lets the loads spread
// over the whole stage: issued over phase C alone, they fill the address
// unit's time there and hold up the wave.
// ---------------------------------------------------------------------------
template <int TI, int TJ, int LDA, int LDB, int EPI, bool MULTI, bool PAIR>
__device__ __forceinline__ void head_product(const HeadArgs& g, int block, uint8_t* smem) {
  constexpr int M_T = 64 * TI, N_T = 64 * TJ;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w >> 1, wn = w & 1;
  const int n = g.live[0], splits = EPI <= EPI_DZ ? 1 : g.live[EPI == EPI_DX ? 1 : 2];
  const uint8_t* xs = n == g.tokens ? g.x : g.xc;
  const int64_t ldx = (int64_t)g.hidden * 2, ldz = (int64_t)g.dz_ld * (PAIR ? 4 : 2);
  // every product is formed transposed: M is the result's contiguous axis (ids
  // of z and dz, hidden of dx and dW), N its rows.  A lane then holds 16 TI
  // values of each of TJ rows, four consecutive ones at a time: a token's
  // maximum, sum and gradient need one other lane, and stores are wide.
  const int M = EPI <= EPI_DZ ? g.nv : g.hidden;
  const int N = EPI == EPI_DW ? g.nv : n;
  // PAIR: a stage of dz's rounded part and one of the rest, with the same
  // stage of the other operand, by turns
  constexpr int TURNS = PAIR && EPI >= EPI_DX ? 2 : 1;
  const int nk = EPI <= EPI_DZ ? g.hidden / 64 : ((EPI == EPI_DX ? g.nv : n) + 63) / 64 * TURNS;
  const int tiles_m = (M + M_T - 1) / M_T, tiles_n = (N + N_T - 1) / N_T;
  const int tiles = tiles_m * tiles_n * splits;
  if (block >= tiles) return;
  int tm, tn;
  tile_of(block, tiles_m, tiles_n * splits, tm, tn);
  const int split = tn / tiles_n;
  tn -= split * tiles_n;
  const int m0 = tm * M_T, n0 = tn * N_T;
  const int k0 = (int)((int64_t)nk * split / splits), k1 = (int)((int64_t)nk * (split + 1) / splits);

  auto tileA = [&](int kt) { return smem + ((kt - k0) & 1) * tile_bytes<TI>(); };
  auto tileB = [&](int kt) { return smem + 2 * tile_bytes<TI>() + (kt - k0) % 3 * tile_bytes<TJ>(); };

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  typename std::conditional<LDA == KMAJ, KLoad<TI>, MnLoad<TI>>::type la;
  typename std::conditional<LDB == KMAJ, KLoad<TJ>, MnLoad<TJ>>::type lb;
  if constexpr (EPI <= EPI_DZ) {
    la.init(g.w, ldx, m0, g.nv, w);
    lb.init(xs, ldx, n0, n, w);
  } else if constexpr (EPI == EPI_DX) {
    la.init(g.w, ldx, m0, g.hidden, g.nv, w);
    lb.init((const uint8_t*)g.dz, ldz, n0, n, w);
  } else {
    la.init(xs, ldx, m0, g.hidden, n, w);
    lb.init((const uint8_t*)g.dz, ldz, n0, g.dz_ld, 64 * nk / TURNS, w);
  }

  const int lr = lane & 31, lg = lane >> 5;
  const int jj = (lr & 15) >> 2;
  // per-lane part of a fragment read: K-major, the row's chunk lg under its
  // swizzle key; MN-major, K row 8 lg + jj, the chunk swizzle 64 jj and the
  // wave's columns
  auto frag_base = [&](int ld, int T, int wv) {
    if (ld == KMAJ) return (uint32_t)(lr * 128 + ((lg ^ swz_key(lr) ^ ((2 * wv * T) & 7)) << 4));
    return (uint32_t)((8 * lg + jj) * (128 * T) + ((64 * jj) ^ (64 * T * wv)) + 32 * (lr >> 4) +
                      16 * ((lr & 3) >> 1) + 8 * (lr & 1));
  };
  const uint32_t fba = frag_base(LDA, TI, wm), fbb = frag_base(LDB, TJ, wn);
  const int offA = LDA == KMAJ ? wm * TI * 4096 : 0, offB = LDB == KMAJ ? wn * TJ * 4096 : 0;

  constexpr int NMFMA = 2 * TI * TJ;                         // per half stage
  constexpr int OVER = NMFMA * 3 / 4;                        // MFMAs that a half stage's fragment reads are spread over
  constexpr int NA = 2 * TI, NB = 2 * TJ;                    // loads per stage and wave
  constexpr int RA = half_reads<LDA, TI>(), RB = half_reads<LDB, TJ>();
  Half<TI> a0, a1;
  Half<TJ> b0, b1;

  auto load_a = [&](int kt, int v) { la.load(kt / TURNS, 0, tileA(kt), w, v); };
  auto load_b = [&](int kt, int v) {
    lb.load(kt / TURNS, TURNS == 2 ? (int64_t)(kt & 1) * g.dz_ld * 2 : 0, tileB(kt), w, v);
  };
  auto mfma = [&](const Half<TI>& a, const Half<TJ>& b, int m) {
    const int s = m / (TI * TJ), i = (m / TJ) % TI, j = m % TJ;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.x[i][s]),
                                                        __builtin_bit_cast(bf16x8, b.x[j][s]), acc[i][j], 0, 0, 0);
  };

  // What the epilogue needs of the lane's tokens: loaded behind the last two
  // stages' products.
  int tok[TJ], state[TJ];
  int64_t target[TJ];
  float lse[TJ], dloss[TJ];
  // A bf16 dW: the rows of side that the lane's ids' rows go to, -1: none
  // (loaded ahead of the first stage: the barrier in the last one would wait
  // for them, 0.5 us a tile)
  int own[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    own[j] = -1;
    if constexpr (EPI == EPI_DW && !PAIR) {
      const int id = n0 + wn * 32 * TJ + 32 * j + lr;
      if (g.head && g.out_bf16 && id < N) own[j] = side_row(g.head[g.v0 + id], g.v0 + id, g.side_by_id);
    }
  }
  // The staged tokens, one a pass, whose slots (MULTI) the thread looks through or whose heavy slots it fetches
  constexpr int PASSES = N_T / STAGE_ROWS;
  const int srow = t % STAGE_ROWS, half = t / STAGE_ROWS;
  auto staged = [&](int p) { return 32 * TJ * (srow / 64) + 64 * p + srow % 64; };
  int slot_tok[PASSES];
  auto token_rows = [&]() {
    if (MULTI || (EPI == EPI_DX && !PAIR && g.dx)) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) slot_tok[p] = g.row_of[n0 + staged(p) < n ? n0 + staged(p) : n - 1];
    }
    if constexpr (EPI <= EPI_DZ) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int col = n0 + wn * 32 * TJ + 32 * j + lr;
        tok[j] = g.row_of[col < n ? col : n - 1];
      }
    }
  };
  auto token_data = [&]() {
    if constexpr (EPI <= EPI_DZ) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if (!MULTI) target[j] = g.targets[tok[j]];
        if (EPI == EPI_DZ) {
          if (MULTI) state[j] = g.state[tok[j]];
          lse[j] = g.lse[tok[j]];
          dloss[j] = g.dloss[tok[j]];
        }
      }
    }
  };

  if (k1 > k0) {
#pragma unroll
    for (int v = 0; v < NA; ++v) load_a(k0, v);
#pragma unroll
    for (int v = 0; v < NB; ++v) load_b(k0, v);
    if (k1 > k0 + 1) {
#pragma unroll
      for (int v = 0; v < NA; ++v) load_a(k0 + 1, v);
#pragma unroll
      for (int v = 0; v < NB; ++v) load_b(k0 + 1, v);
      stage_barrier<NA + NB>();
    } else {
      stage_barrier<0>();
    }
#pragma unroll
    for (int d = 0; d < RA; ++d) half_read<0, LDA, TI>(a0, d, tileA(k0) + offA, fba);
#pragma unroll
    for (int d = 0; d < RB; ++d) half_read<0, LDB, TJ>(b0, d, tileB(k0) + offB, fbb);

    auto body = [&](int kt, auto issue_c, auto next_c) {
      constexpr bool ISSUE = decltype(issue_c)::value;
      constexpr bool NEXT = decltype(next_c)::value;
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
          if (d < RA) half_read<1, LDA, TI>(a1, d, curA, fba);
          else half_read<1, LDB, TJ>(b1, d - RA, curB, fbb);
        }
        if (ISSUE) {
#pragma unroll
          for (int v = part_lo(NB, NMFMA, m); v < part_hi(NB, NMFMA, m); ++v) load_b(kt + 2, v);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      stage_barrier<ISSUE ? NB : 0>();
      constexpr int NDS = NEXT ? RA + RB : 0;
#pragma unroll
      for (int m = 0; m < NMFMA; ++m) {
        mfma(a1, b1, m);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = part_lo(NDS, OVER, m); d < part_hi(NDS, OVER, m); ++d) {
          if (d < RA) half_read<0, LDA, TI>(a0, d, nxtA, fba);
          else half_read<0, LDB, TJ>(b0, d - RA, nxtB, fbb);
        }
        if (ISSUE) {
#pragma unroll
          for (int v = part_lo(NA, NMFMA, m); v < part_hi(NA, NMFMA, m); ++v) load_a(kt + 2, v);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using T_ = std::integral_constant<bool, true>;
    using F_ = std::integral_constant<bool, false>;
    for (int kt = k0; kt < k1 - 2; ++kt) body(kt, T_{}, T_{});
    token_rows();
    if (k1 - k0 >= 2) body(k1 - 2, F_{}, T_{});
    token_data();
    body(k1 - 1, F_{}, F_{});
  }
  // Every LDS read of the loop finished before its last barrier, and no load
  // is in flight: the tiles' space may now stage the result.  Lane (lr, lg)
  // holds, in acc[i][j][4 q + r], row 32 TI wm + 32 i + 8 q + 4 lg + r of column
  // 32 TJ wn + 32 j + lr.
  const float none = -__builtin_inff();
  constexpr int PITCH = M_T + STAGE_PAD / 4, PITCHB = M_T * 2 + STAGE_PAD;
  float* stage = (float*)smem;                                 // [STAGE_ROWS][PITCH], or bf16 [N_T][PITCHB]
  const int row0 = wm * 32 * TI;                               // the wave's first value of the tile's rows
  auto stage_bf16 = [&](int j) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(uint2*)(smem + (wn * 32 * TJ + 32 * j + lr) * PITCHB + (row0 + 32 * i + 8 * q + 4 * lg) * 2) = make_uint2(
            pk_bf16(acc[i][j][4 * q], acc[i][j][4 * q + 1]), pk_bf16(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]));
  };
  // rows 32 TJ wn + 64 p .. of the wave's columns, to staged rows 64 wn ..: a
  // pass p stages row s of the tile's row 32 TJ (s / 64) + 64 p + s % 64
  auto stage_f32 = [&](int p) {
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = 2 * p + jj;
          *(float4*)(stage + (wn * 64 + 32 * jj + lr) * PITCH + row0 + 32 * i + 8 * q + 4 * lg) =
              make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        }
  };
  if constexpr (EPI <= EPI_DZ) {
    float* scale = (float*)(smem + STAGE_ROWS * PITCH * 4);     // MULTI: dloss / tau of the tile's tokens
    const int have = g.nv - m0 < M_T ? g.nv - m0 : M_T;        // ids of the tile that exist
    // MULTI: a token's slots lie in groups of four; its two threads take the
    // even and the odd ones.  The first AHEAD of each are loaded ahead of the
    // statistics, or of the pass before (read where they are used, they and
    // the row's token cost 4 us a tile in latency).
    constexpr int AHEAD = 8, HELD = EPI == EPI_STATS ? PASSES : 1;
    const int groups = g.slots / 4;
    int4 sid[HELD][AHEAD];
    float4 sp[AHEAD];
    int4 heavy4;
    auto load_slots = [&](int p) {
      const int64_t at = (int64_t)slot_tok[p] * groups;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int q = half + 2 * k;                            // past the last group: that one, for nothing
        sid[HELD == 1 ? 0 : p][k] = ((const int4*)g.ids)[at + (q < groups ? q : groups - 1)];
        if (EPI == EPI_DZ) sp[k] = ((const float4*)g.p)[at + (q < groups ? q : groups - 1)];
      }
      if (EPI == EPI_DZ && !PAIR) heavy4 = ((const int4*)g.heavy)[slot_tok[p]];
    };
    if constexpr (MULTI) {
#pragma unroll
      for (int p = 0; p < HELD; ++p) load_slots(p);
    }
    const float c2 = g.inv_tau * LOG2E;
    int want[TJ];                                              // the token's target less this lane's first id
    float lse2[TJ], cz[TJ];                                    // lse / log 2, dloss / tau
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const bool there = n0 + wn * 32 * TJ + 32 * j + lr < n;  // past the last row: exp(-inf) 0 = 0
      const int64_t local = MULTI ? -1 : target[j] - (g.v0 + m0 + row0);
      want[j] = there && local >= 0 && local < 32 * TI && local < have - row0 ? (int)local - 4 * lg : -1;
      if (EPI == EPI_DZ) {
        const bool bad = MULTI ? state[j] == ROW_BAD : target[j] >= g.vocab;
        lse2[j] = there ? lse[j] * LOG2E : __builtin_inff();
        cz[j] = !there ? 0.0f : bad ? __builtin_nanf("") : dloss[j] * g.inv_tau;
      }
    }
    // Each token's heavy place goes to the head of its id's list; what stood there comes next.
    Push push[TJ];
    bool here[TJ];
    if constexpr (!MULTI && EPI == EPI_DZ && !PAIR) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int64_t local = target[j] - (g.v0 + m0);
        here[j] = g.head && wm == 0 && lg == 0 && n0 + wn * 32 * TJ + 32 * j + lr < n && local >= 0 && local < have;
        push[j] = push_place(g.head, (int)target[j], tok[j], here[j]);
      }
    }
    // Token j: its statistics or its dz, staged.  FULL: no id of the tile is
    // past the last one (-inf in its place).  The accumulators are read here
    // and not earlier: hoisted ahead of the choice between the two instances
    // they filled the vector registers and spilled (loss 0.5 to 1.5% slower).
    auto column = [&](auto full_c, int j) {
      constexpr bool FULL = decltype(full_c)::value;
      float v[TI][16];
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          v[i][r] = acc[i][j][r];
          if (TI == 4) asm volatile("" : "+v"(v[i][r]));
        }
      auto z = [&](int i, int r) {
        return FULL || row0 + 32 * i + 8 * (r >> 2) + 4 * lg + (r & 3) < have ? v[i][r] : none;
      };
      if constexpr (EPI == EPI_STATS) {
        float mx = none;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) mx = fmaxf(mx, z(i, r));
        mx *= c2;                                            // everything in units of log 2 from here
        const float safe = mx == none ? 0.0f : mx;           // nothing but -inf: the sum stays 0
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          // sixteen independent exponentials, then a tree: one running sum
          // would wait out the instruction's latency 16 TI times
          float e[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(z(i, r), c2, -safe));
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
            for (int r = 0; r < o; ++r) e[r] += e[r + o];
          sum += e[0];
        }
        const float mo = __shfl_xor(mx, 32, 64), so = __shfl_xor(sum, 32, 64);
        const float m1 = fmaxf(mx, mo), safe1 = m1 == none ? 0.0f : m1;
        sum = sum * __builtin_amdgcn_exp2f(mx - safe1) + so * __builtin_amdgcn_exp2f(mo - safe1);
        if (lg == 0)
          g.stats[(int64_t)(tm * 2 + wm) * g.rows + n0 + wn * 32 * TJ + 32 * j + lr] = make_float2(m1, sum);
      } else {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            v[i][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(z(i, r), c2, -lse2[j])) * cz[j];
      }
      if (!MULTI && __any(want[j] >= 0)) {
        float at = 0.0f;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool hit = want[j] == 32 * i + 8 * (r >> 2) + (r & 3);
            if (EPI == EPI_DZ) v[i][r] -= hit ? cz[j] : 0.0f;
            at = hit ? v[i][r] : at;
            mine |= hit;
          }
        if (EPI == EPI_STATS && mine) g.zsel[tok[j]] = at * g.inv_tau;
        if (EPI == EPI_DZ && !PAIR && mine) g.rest[tok[j]] = bf16_rest(at);
      }
      if constexpr (MULTI) {
        const float f = EPI == EPI_STATS ? g.inv_tau : 1.0f;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *(float4*)(stage + (wn * 64 + 32 * (j % 2) + lr) * PITCH + row0 + 32 * i + 8 * q + 4 * lg) =
                make_float4(v[i][4 * q] * f, v[i][4 * q + 1] * f, v[i][4 * q + 2] * f, v[i][4 * q + 3] * f);
      } else if constexpr (EPI == EPI_DZ) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = v[i][r];
        if (!PAIR) stage_bf16(j);
      }
    };
    auto columns = [&](int j0, int j1) {
      if (have == M_T) {
#pragma unroll
        for (int j = j0; j < j1; ++j) column(std::integral_constant<bool, true>{}, j);
      } else {
#pragma unroll
        for (int j = j0; j < j1; ++j) column(std::integral_constant<bool, false>{}, j);
      }
    };
    if (!MULTI) columns(0, TJ);
    constexpr int LPR = M_T / 8;                               // lanes a row, 8 values each
    constexpr int PARTS = PAIR ? 2 : 1;
    if constexpr (!MULTI && EPI == EPI_DZ) {
      if constexpr (!PAIR) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const int next = pushed_next(push[j], tok[j]);
          if (here[j]) g.next[tok[j]] = next;
        }
      }
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        if (PAIR) {
          if (h) __syncthreads();
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            if (h) {
#pragma unroll
              for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] -= (float)(__bf16)acc[i][j][r];
            }
            stage_bf16(j);
          }
        }
        __syncthreads();
#pragma unroll 4
        for (int s = t / LPR; s < N_T; s += 256 / LPR)
          *(uint4*)(g.dz + ((int64_t)(n0 + s) * PARTS + h) * g.dz_ld + m0 + (t % LPR) * 8) =
              *(const uint4*)(smem + s * PITCHB + (t % LPR) * 16);
      }
    }
    if constexpr (MULTI) {
      // fp32, 128 tokens a pass
      if (EPI == EPI_DZ && wm == 0 && lg == 0) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) scale[wn * 32 * TJ + 32 * j + lr] = cz[j];
      }
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int some = n0 + staged(p) < n ? have : 0;        // ids in reach
        const int first = g.v0 + m0;
        Push push[MOST_HEAVY];
        auto heavy_id = [&](int e) { return e == 0 ? heavy4.x : e == 1 ? heavy4.y : e == 2 ? heavy4.z : heavy4.w; };
        if constexpr (EPI == EPI_DZ && !PAIR) {
#pragma unroll
          for (int e = 0; e < MOST_HEAVY; ++e)                 // (half: whole waves)
            push[e] = push_place(g.head, heavy_id(e), slot_tok[p] * MOST_HEAVY + e,
                                 g.head && half == 0 && (uint32_t)(heavy_id(e) - first) < (uint32_t)some);
        }
        columns(2 * p, 2 * p + 2);
        stage_barrier<63>();
        float* mine = stage + srow * PITCH;
        const int64_t at = (int64_t)slot_tok[p] * g.slots;
        // (an unused slot's id is -1, which is in no tile)
        auto group = [&](int q, const int4& id4, const float4& p4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = (k == 0 ? id4.x : k == 1 ? id4.y : k == 2 ? id4.z : id4.w) - first;
            if ((uint32_t)c >= (uint32_t)some) continue;
            if (EPI == EPI_STATS) g.zsel[at + 4 * q + k] = mine[c];
            else mine[c] -= (k == 0 ? p4.x : k == 1 ? p4.y : k == 2 ? p4.z : p4.w) * scale[staged(p)];
          }
        };
        auto look = [&]() {
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
            if (half + 2 * k < groups) group(half + 2 * k, sid[HELD == 1 ? 0 : p][k], sp[k]);
          for (int q = half + 2 * AHEAD; q < groups; q += 2)
            group(q, ((const int4*)g.ids)[at / 4 + q],
                  EPI == EPI_DZ ? ((const float4*)g.p)[at / 4 + q] : make_float4(0, 0, 0, 0));
        };
        if (EPI == EPI_STATS) {
          look();
        } else {
          // slots of one id add up in one place: one thread of the two after the other
          if (half == 0) look();
          stage_barrier<63>();
          if (half == 1) look();
        }
        stage_barrier<63>();
        if constexpr (EPI == EPI_DZ && !PAIR) {
          if (half == 0) {
#pragma unroll
            for (int e = 0; e < MOST_HEAVY; ++e) {
              const int c = heavy_id(e) - first, place = slot_tok[p] * MOST_HEAVY + e;
              const int next = pushed_next(push[e], place);
              if ((uint32_t)c >= (uint32_t)some) continue;
              g.rest[place] = bf16_rest(mine[c]);
              if (g.head) g.next[place] = next;
            }
          }
        }
        if (EPI == EPI_DZ && p + 1 < PASSES) load_slots(p + 1);
        if (EPI == EPI_DZ) {
#pragma unroll 4
          for (int s2 = t / LPR; s2 < STAGE_ROWS; s2 += 256 / LPR) {
            const float* q = stage + s2 * PITCH + (t % LPR) * 8;
            float4 lo = *(const float4*)q, hi = *(const float4*)(q + 4);
            uint16_t* to = g.dz + (int64_t)(n0 + 32 * TJ * (s2 / 64) + 64 * p + s2 % 64) * PARTS * g.dz_ld + m0 +
                           (t % LPR) * 8;
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
              *(uint4*)(to + h * g.dz_ld) =
                  make_uint4(pk_bf16(lo.x, lo.y), pk_bf16(lo.z, lo.w), pk_bf16(hi.x, hi.y), pk_bf16(hi.z, hi.w));
              if (h + 1 < PARTS) {
                auto rest = [](float& v) { v -= (float)(__bf16)v; };
                rest(lo.x); rest(lo.y); rest(lo.z); rest(lo.w);
                rest(hi.x); rest(hi.y); rest(hi.z); rest(hi.w);
              }
            }
          }
          if (p + 1 < PASSES) stage_barrier<63>();
        }
      }
    }
  } else {
    constexpr int LPR = M_T / 8, RPI = 256 / LPR;              // lanes a row, 8 values each; rows a round
    const int col = m0 + (t % LPR) * 8;
    if (EPI == EPI_DX ? PAIR && g.dx : splits == 1 && g.out_bf16) {
      uint16_t* out = EPI == EPI_DX ? g.dx : (uint16_t*)g.dw;
      if constexpr (EPI == EPI_DW && !PAIR) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          if (own[j] >= 0) {
            float* to = g.side + (int64_t)own[j] * g.hidden + m0 + row0 + 4 * lg;
#pragma unroll
            for (int i = 0; i < TI; ++i) {
              if (m0 + row0 + 32 * i >= M) break;              // (hidden is a multiple of 64)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *(float4*)(to + 32 * i + 8 * q) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) stage_bf16(j);
      stage_barrier<63>();
#pragma unroll 4
      for (int s = t / LPR; s < N_T; s += RPI)
        if (n0 + s < N && col < M)
          *(uint4*)(out + (int64_t)(EPI == EPI_DX ? g.row_of[n0 + s] : n0 + s) * g.hidden + col) =
              *(const uint4*)(smem + s * PITCHB + (t % LPR) * 16);
      return;
    }
    // dx partials: the splits' live rows, in whole tiles, one after the other, or dx itself with its heavy slots' part
    // (W is one piece then); dW itself, or its partials
    float* out = EPI == EPI_DW && splits == 1
                     ? (float*)g.dw
                     : (EPI == EPI_DX ? g.dx_part + (int64_t)split * tiles_n * N_T * g.hidden
                                        : g.dw_part + (int64_t)split * g.dz_ld * g.hidden);
#pragma unroll
    for (int p = 0; p < N_T / STAGE_ROWS; ++p) {
      if (EPI == EPI_DX && !PAIR && g.dx) {
        // dx itself: the rows' tokens and heavy slots go to LDS, and the rows of W for eight results are fetched at once
        // (each where it is used, gradient 15872 x 69 x 4096 took 212 us)
        struct Row {
          int tok, id[MOST_HEAVY];
          float rest[MOST_HEAVY];
        };
        static_assert(STAGE_ROWS * (PITCH * 4 + (int)sizeof(Row)) <= head_smem<TI, TJ>(), "no room for the rows");
        Row* rows = (Row*)(smem + STAGE_ROWS * PITCH * 4);
        if (half == 0) {
          Row r;
          r.tok = n0 + staged(p) < n ? slot_tok[p] : -1;
#pragma unroll
          for (int e = 0; e < MOST_HEAVY; ++e) {
            const int64_t at = (int64_t)slot_tok[p] * g.heavy_n + e;
            r.id[e] = e < g.heavy_n ? g.heavy[at] : -1;
            r.rest[e] = r.id[e] >= 0 ? g.rest[at] : 0.0f;
          }
          rows[srow] = r;
        }
        stage_f32(p);
        stage_barrier<0>();
        constexpr int AT_ONCE = 8;
        for (int s0 = t / LPR; s0 < STAGE_ROWS; s0 += AT_ONCE * RPI) {
          uint4 u[AT_ONCE];
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) {      // (no heavy slot: some row, times 0)
            const int id = rows[s0 + k * RPI].id[0];
            u[k] = *(const uint4*)(g.w + (id > 0 ? id : 0) * ldx + (col < M ? col : 0) * 2);
          }
#pragma unroll
          for (int k = 0; k < AT_ONCE; ++k) {
            const Row* r = rows + s0 + k * RPI;
            if (r->tok < 0 || col >= M) continue;
            const float* q = stage + (s0 + k * RPI) * PITCH + (t % LPR) * 8;
            float v[8];
            *(float4*)v = *(const float4*)q;
            *(float4*)(v + 4) = *(const float4*)(q + 4);
            add_bf16x8(v, r->rest[0], u[k]);
            for (int e = 1; e < MOST_HEAVY && r->id[e] >= 0; ++e)   // (they stand first)
              add_bf16x8(v, r->rest[e], *(const uint4*)(g.w + r->id[e] * ldx + col * 2));
            *(uint4*)(g.dx + (int64_t)r->tok * g.hidden + col) =
                make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
          }
        }
        if (p + 1 < N_T / STAGE_ROWS) stage_barrier<63>();
        continue;
      }
      stage_f32(p);
      stage_barrier<63>();
#pragma unroll 4
      for (int s = t / LPR; s < STAGE_ROWS; s += RPI) {
        const float* q = stage + s * PITCH + (t % LPR) * 8;
        float4 lo = *(const float4*)q, hi = *(const float4*)(q + 4);
        const int row = n0 + 32 * TJ * (s / 64) + 64 * p + s % 64;
        if (row < N && col < M) {
          float4* o = (float4*)(out + (int64_t)row * g.hidden + col);
          if (EPI == EPI_DX && g.add) {
            const float4 u = o[0], v = o[1];
            lo = make_float4(lo.x + u.x, lo.y + u.y, lo.z + u.z, lo.w + u.w);
            hi = make_float4(hi.x + v.x, hi.y + v.y, hi.z + v.z, hi.w + v.w);
          }
          o[0] = lo;
          o[1] = hi;
        }
      }
      if (p + 1 < N_T / STAGE_ROWS) stage_barrier<63>();
    }
  }
}

// z's statistics or dz, T x T tiles of 64 values.
template <int T, int EPI, bool MULTI, bool PAIR>
__global__ __launch_bounds__(256, T >= 4 ? 1 : 2) void head_logits_kernel(HeadArgs g) {
  __shared__ __align__(16) uint8_t smem[head_smem<T, T>()];
  head_product<T, T, KMAJ, KMAJ, EPI, MULTI, PAIR>(g, blockIdx.x, smem);
}

// dx and dW of a piece in one launch: the two need nothing of each other, and
// the tiles of one fill the compute units that the other's last round leaves
// idle.  dx's tiles, the longer ones, come first.
template <int T, bool PAIR>
__global__ __launch_bounds__(256, T >= 4 ? 1 : 2) void head_grads_kernel(HeadArgs g) {
  __shared__ __align__(16) uint8_t smem[head_smem<T, T>()];
  if ((int)blockIdx.x < g.dx_blocks) head_product<T, T, MNMAJ, KMAJ, EPI_DX, false, PAIR>(g, blockIdx.x, smem);
  else head_product<T, T, MNMAJ, MNMAJ, EPI_DW, false, PAIR>(g, blockIdx.x - g.dx_blocks, smem);
}

// ---------------------------------------------------------------------------
// Around the products.
// ---------------------------------------------------------------------------
struct TeacherArgs {
  const int64_t* ids;      // [tokens][top]
  const void* logits;      // [tokens][top]
  int bf16, top, slots, tokens, vocab;
  float inv_tau;
  int* state;
  int* ids32;
  float* p;
  float* ent;              // sum p log p
  int4* heavy;             // per token: its heavy slots' ids, each once, -1: none (null: not wanted)
};

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The teacher's probabilities: one wave per token.  A slot with a negative id
// is unused, whatever its logit holds; a token without a used slot, or whose
// used slots all hold -inf, takes no part.  The maximum is subtracted before
// the division by tau, so the type's lowest value in every slot is a uniform
// distribution and overflows nowhere.
// The first 64 slots, mostly all there are, are read once.
__global__ __launch_bounds__(256) void head_teacher_kernel(TeacherArgs a) {
  const int tok = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (tok >= a.tokens) return;
  const int64_t in = (int64_t)tok * a.top, out = (int64_t)tok * a.slots;
  const float none = -__builtin_inff();
  struct Slot {
    int64_t id;
    float v;
  };
  auto read = [&](int s) {
    Slot u = {-1, none};
    if (s < a.top) {
      u.id = a.ids[in + s];
      u.v = a.bf16 ? bf16_to_float(((const bf16_t*)a.logits)[in + s]) : ((const float*)a.logits)[in + s];
      if (u.id < 0) u.v = none;
    }
    return u;
  };
  const Slot first = read(lane);
  float mx = none;
  bool bad = false, nan = false;
  for (int s = lane; s < a.slots; s += 64) {
    const Slot u = s < 64 ? first : read(s);
    nan |= u.v != u.v;
    bad |= u.id >= a.vocab;
    mx = fmaxf(mx, u.v);
  }
  mx = wave_max_f(mx);
  nan = __any(nan);
  bad = __any(bad);
  const bool live = mx > none || nan || bad;
  const float safe = mx > none ? mx : 0.0f;
  float sum = 0.0f;
  for (int s = lane; s < a.slots; s += 64) sum += expf(((s < 64 ? first : read(s)).v - safe) * a.inv_tau);
  sum = wave_sum_f(sum);
  const float ls = logf(sum);
  float ent = 0.0f;
  int4 heavy = make_int4(-1, -1, -1, -1);
  for (int s = lane; s < a.slots; s += 64) {
    const Slot u = s < 64 ? first : read(s);
    const float e = (u.v - safe) * a.inv_tau;
    const float p = live ? expf(e) / sum : 0.0f;
    if (!(p == 0.0f)) ent += p * (e - ls);
    const int id = u.id >= 0 && u.id < a.vocab ? (int)u.id : -1;
    a.p[out + s] = p;
    a.ids32[out + s] = id;
    // (slots are a multiple of 4: lane 0 is here whenever one is)
    for (uint64_t m = __ballot(p > HEAVY_P && id >= 0); m; m &= m - 1) {
      const int h = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)m) - 1);
      if (h != heavy.x && h != heavy.y && h != heavy.z && h != heavy.w) heavy = make_int4(h, heavy.x, heavy.y, heavy.z);
    }
  }
  ent = wave_sum_f(ent);
  if (lane == 0) {
    if (a.heavy) a.heavy[tok] = heavy;
    a.ent[tok] = ent;
    a.state[tok] = bad ? ROW_BAD : live ? ROW_LIVE : ROW_OUT;
  }
}

// Splits of a product's K loop over nk stages when its tiles alone leave
// workgroup slots idle: the number that minimises rounds of tiles times
// (stages + a tile's fixed cost) plus the partial products' traffic, all in
// stages.  Never more than 2 x 256 tiles' worth of partial products.  Lanes 0
// to 15 of a wave weigh 1 to 16 splits each; every lane gets the answer.
// `beside`: stages that each slot has to do for the other product of the
// launch.  Its tiles come after these and fill what they leave idle, so the
// fewest splits do whose tiles end before both products would if spread evenly
// (gradient, against as many splits as fill the card: 1433 x 49999 x 2048 806
// -> 770 us, 512 x 32000 x 2048 213 -> 197, 8 x 100000 x 4096 675 -> 614; with
// 3/4 of that time as the limit 781, 205 and 624).
constexpr int HEAD_FIXED = 6, HEAD_LEAST_STAGES = 8, HEAD_MOST_SPLITS = 16, HEAD_SPLIT_TILES = 512;
__device__ __forceinline__ int head_splits(int tiles, int nk, int slots, int beside) {
  const int s = (threadIdx.x & (HEAD_MOST_SPLITS - 1)) + 1;
  const bool may = s == 1 || (nk / s >= HEAD_LEAST_STAGES && tiles <= HEAD_SPLIT_TILES / s);
  const uint32_t rounds = (uint32_t)((tiles - 1) / slots + 1);
  uint32_t cost = rounds * (uint32_t)(nk + HEAD_FIXED);
  if (s > 1) cost = (uint32_t)((tiles * s + slots - 1) / slots * ((nk + s - 1) / s + HEAD_FIXED) + tiles * s / 23);
  // (where tiles are too many to be split, one split's cost may wrap: it still
  // is at most the others', and comes first among equals)
  cost = may && cost < 0x07FFFFFFu ? cost : 0x07FFFFFFu;
  uint32_t key = cost * 16 + (uint32_t)(s - 1);
#pragma unroll
  for (int o = HEAD_MOST_SPLITS / 2; o >= 1; o >>= 1) {
    const uint32_t u = (uint32_t)__shfl_xor((int)key, o, 64);
    key = key < u ? key : u;
  }
  const int best = (int)(key & 15u) + 1;
  const int all = beside + (int)((int64_t)tiles * (nk + HEAD_FIXED) / slots);
  const uint64_t fit = __ballot(beside > 0 && may && (nk + s - 1) / s + HEAD_FIXED <= all);
  const int few = fit ? __ffsll((unsigned long long)fit) : best;
  return few < best ? few : best;
}

struct RowsArgs {
  const int64_t* targets;  // cross entropy; null: state is set
  const int* state;
  int tokens;
  int* live;               // out: {live rows, splits of dx, splits of dW}
  int* row_of;
  int* pos_of;             // token -> live row, or -1
  float* loss;             // of the tokens that take no part: 0 (null in the gradient)
  float* lse;
  const uint4* x;
  uint4* xc;
  int chunks;              // 16-byte chunks of a row of x
  int tile, dx_tn, dx_nk, dw_tiles, turns, slots;  // the gradient's products, for their splits
  int together;            // dx and dW share their launches
  int dx_whole;            // dx is not split
  uint4* zero_dx;          // the rows of dx that nothing else writes, those of the tokens left out (or null)
  int* heavy;              // out, cross entropy: the token's target, -1 where it has none (or null)
  int* head;               // out: -1 for every id (or null)
  int vocab;
};

// The live tokens in order, and their rows of x one after the other (unless
// every token is live: the products then read x itself).  Every workgroup
// counts all tokens, 8 x 64 consecutive ones a wave and step by ballots, and
// so knows how many are live ahead of its own share of the tokens, which it
// then ranks and copies: one launch instead of a scan and a copy (7 us for
// 8192 live tokens; a scan by one workgroup and a copy took 8 + 5).
constexpr int ROWS_THR = 1024, ROWS_PER = 8, ROWS_WAVES = ROWS_THR / 64;
__global__ __launch_bounds__(ROWS_THR) void head_rows_kernel(RowsArgs a) {
  __shared__ int wave_n[2][ROWS_WAVES][2];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (a.head)
    for (int64_t i = (int64_t)blockIdx.x * ROWS_THR + threadIdx.x; i < a.vocab; i += (int64_t)gridDim.x * ROWS_THR)
      a.head[i] = -1;
  auto is_live = [&](int64_t t) { return a.targets ? a.targets[t] >= 0 : a.state[t] != ROW_OUT; };
  // this workgroup's tokens: [lo, hi)
  const int64_t lo = (int64_t)a.tokens * blockIdx.x / gridDim.x;
  const int64_t hi = (int64_t)a.tokens * (blockIdx.x + 1) / gridDim.x;
  int n = 0, before = 0, buf = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += ROWS_THR * ROWS_PER, buf ^= 1) {
    const int64_t first = t0 + w * 64 * ROWS_PER;
    bool on[ROWS_PER];
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      const int64_t t = first + 64 * i + lane;
      on[i] = t < a.tokens && is_live(t);
    }
    int all = 0, ahead = 0;
#pragma unroll
    for (int i = 0; i < ROWS_PER; ++i) {
      all += __popcll(__ballot(on[i]));
      ahead += __popcll(__ballot(on[i] && first + 64 * i + lane < lo));
    }
    if (lane == 0) {
      wave_n[buf][w][0] = all;
      wave_n[buf][w][1] = ahead;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS_WAVES; ++i) {
      n += wave_n[buf][i][0];
      before += wave_n[buf][i][1];
    }
  }
  if (blockIdx.x == 0 && w == 0) {
    int dx = 1, dw = 1;
    if (!a.loss) {
      const int dw_nk = (n + 63) / 64 * a.turns;
      const int beside = a.together ? (int)((int64_t)a.dw_tiles * (dw_nk + HEAD_FIXED) / a.slots) : 0;
      if (!a.dx_whole) dx = head_splits((n + a.tile - 1) / a.tile * a.dx_tn, a.dx_nk, a.slots, beside);
      dw = head_splits(a.dw_tiles, dw_nk, a.slots, 0);
    }
    if (lane == 0) {
      a.live[0] = n;
      a.live[1] = dx;
      a.live[2] = dw;
    }
  }
  // the own tokens, up to 64 at a time; a wave copies 1 KiB of a row at a time
  const int segs = (a.chunks + 63) / 64;
  for (int64_t t0 = lo; t0 < hi; t0 += 64) {
    const int64_t t = t0 + lane;
    const bool in = t < hi, on = in && is_live(t);
    const uint64_t mask = __ballot(on);
    const int pos = before + __popcll(mask & ((1ull << lane) - 1));
    if (in && w == 0) {
      a.pos_of[t] = on ? pos : -1;
      if (on) a.row_of[pos] = (int)t;
      if (a.heavy) a.heavy[t] = on && a.targets[t] < a.vocab ? (int)a.targets[t] : -1;
      if (!on && a.loss) {
        a.loss[t] = 0.0f;
        a.lse[t] = 0.0f;
      }
    }
    if (n < a.tokens) {
      const int items = (int)(hi - t0 < 64 ? hi - t0 : 64) * segs;
      for (int i = w; i < items; i += ROWS_WAVES) {
        const int k = i / segs, c = (i - k * segs) * 64 + lane;
        if (c >= a.chunks) continue;
        if ((mask >> k) & 1)
          a.xc[(int64_t)(before + __popcll(mask & ((1ull << k) - 1))) * a.chunks + c] = a.x[(t0 + k) * a.chunks + c];
        else if (a.zero_dx)
          a.zero_dx[(t0 + k) * a.chunks + c] = make_uint4(0, 0, 0, 0);
      }
    }
    before += __popcll(mask);
  }
}

struct JoinArgs {
  const int* live;
  const int* row_of;
  const int64_t* targets;  // cross entropy, or null and
  const int* state;
  const int* ids;
  const float* p;
  const float* ent;
  const float* zsel;
  const float2* stats;
  int parts, rows, slots, vocab;
  float* loss;
  float* lse;
};

// lse and loss of 32 live rows: 32 threads a row share its parts, then its slots.
constexpr int JOIN_ROWS = 32, JOIN_Q = 32;
__global__ __launch_bounds__(JOIN_ROWS * JOIN_Q) void head_join_kernel(JoinArgs a) {
  __shared__ float2 sm[JOIN_Q][JOIN_ROWS + 1];
  const int r = threadIdx.x % JOIN_ROWS, q = threadIdx.x / JOIN_ROWS;
  const int row = blockIdx.x * JOIN_ROWS + r;
  const int n = a.live[0];
  if ((int)blockIdx.x * JOIN_ROWS >= n) return;
  const bool ok = row < n;
  const float none = -__builtin_inff();
  // the token's own data, ahead of the sums
  const int tok = a.row_of[ok ? row : n - 1];
  const int64_t target = a.targets ? a.targets[tok] : 0;
  const float zt = a.targets ? a.zsel[tok] : 0.0f;
  float2 u = make_float2(none, 0.0f);
  auto add = [&](float2 v) {
    const float m1 = fmaxf(u.x, v.x), safe = m1 == none ? 0.0f : m1;
    u = make_float2(m1, u.y * __builtin_amdgcn_exp2f(u.x - safe) + v.y * __builtin_amdgcn_exp2f(v.x - safe));
  };
  if (ok) {
    const float2* st = a.stats + row;
    int i = q;
    for (; i + 3 * JOIN_Q < a.parts; i += 4 * JOIN_Q) {
      const float2 v0 = st[(int64_t)i * a.rows], v1 = st[(int64_t)(i + JOIN_Q) * a.rows];
      const float2 v2 = st[(int64_t)(i + 2 * JOIN_Q) * a.rows], v3 = st[(int64_t)(i + 3 * JOIN_Q) * a.rows];
      const float m1 = fmaxf(fmaxf(u.x, fmaxf(v0.x, v1.x)), fmaxf(v2.x, v3.x)), safe = m1 == none ? 0.0f : m1;
      const float s01 = v0.y * __builtin_amdgcn_exp2f(v0.x - safe) + v1.y * __builtin_amdgcn_exp2f(v1.x - safe);
      const float s23 = v2.y * __builtin_amdgcn_exp2f(v2.x - safe) + v3.y * __builtin_amdgcn_exp2f(v3.x - safe);
      u = make_float2(m1, u.y * __builtin_amdgcn_exp2f(u.x - safe) + (s01 + s23));
    }
    for (; i < a.parts; i += JOIN_Q) add(st[(int64_t)i * a.rows]);
  }
  sm[q][r] = u;
  __syncthreads();
  // every thread of the row joins the 32 sums, in the same order
  float mx = none, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < JOIN_Q; ++i) mx = fmaxf(mx, sm[i][r].x);
  const float safe = mx == none ? 0.0f : mx;
#pragma unroll
  for (int i = 0; i < JOIN_Q; ++i) sum = __builtin_fmaf(sm[i][r].y, __builtin_amdgcn_exp2f(sm[i][r].x - safe), sum);
  const float lse = (mx + __builtin_amdgcn_logf(sum)) * LN2;
  if (a.targets) {
    if (q == 0 && ok) {
      a.lse[tok] = lse;
      a.loss[tok] = target >= a.vocab ? __builtin_nanf("") : lse - zt;
    }
    return;
  }
  float loss = 0.0f;
  if (ok) {
    const int64_t at = (int64_t)tok * a.slots;
    for (int s = q; s < a.slots; s += JOIN_Q) {
      const float p = a.p[at + s];
      if (a.ids[at + s] >= 0 && !(p == 0.0f)) loss -= p * (a.zsel[at + s] - lse);
    }
  }
  __syncthreads();
  sm[q][r].x = loss;
  __syncthreads();
  if (q != 0 || !ok) return;
  for (int i = 1; i < JOIN_Q; ++i) loss += sm[i][r].x;
  a.lse[tok] = lse;
  a.loss[tok] = a.state[tok] == ROW_BAD ? __builtin_nanf("") : loss + a.ent[tok];
}

// dW of a piece from its splits' partial products.
__global__ __launch_bounds__(256) void head_dw_kernel(const float* part, const int* live, int64_t split_stride,
                                                      int64_t chunks8, void* dw, int bf16, const int* head, float* side,
                                                      int side_by_id, int v0, int per_row) {
  const int splits = live[2];
  if (splits == 1) return;                     // the product stored dW itself
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks8; i += (int64_t)gridDim.x * 256) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float* q = part + i * 8;
    for (int s = 0; s < splits; ++s, q += split_stride) {
      const float4 lo = *(const float4*)q, hi = *(const float4*)(q + 4);
      v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
      v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    const int64_t row = i / per_row;
    const int own = bf16 && head ? side_row(head[v0 + row], v0 + (int)row, side_by_id) : -1;
    if (own >= 0) {
      float4* o = (float4*)side + ((int64_t)own * per_row + (i - row * per_row)) * 2;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    if (bf16) {
      *(uint4*)((uint16_t*)dw + i * 8) =
          make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
    } else {
      ((float4*)dw)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
      ((float4*)dw)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

struct FinishArgs {
  const int* live;
  const int* pos_of;
  const float* dx_part;    // partial products of dx
  const int* heavy;
  const float* rest;
  const int* head;
  const int* next;
  const float* side;
  const uint4* x;
  const uint4* w;
  uint16_t* dx;
  void* dw;
  int64_t chunks8;         // 8-value chunks of dx
  int dx_blocks;           // workgroups of dx ahead of dW's
  int tile, hidden, per_row, heavy_n;   // per_row: 8-value chunks of a row
  int dw_bf16, side_by_id;
};

// dx [tokens, hidden] bf16 from the partial products of the live rows and their
// heavy slots; zeros for the tokens that take no part.  8 values a thread.
__device__ __forceinline__ void finish_dx(const FinishArgs& a) {
  const int splits = a.live[1];
  const int64_t split_stride = (int64_t)((a.live[0] + a.tile - 1) / a.tile) * a.tile * a.hidden;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.chunks8; i += (int64_t)a.dx_blocks * 256) {
    const int64_t tok = i / a.per_row;
    const int c = (int)(i - tok * a.per_row);
    const int pos = a.pos_of[tok];
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (pos >= 0) {
      const float* q = a.dx_part + ((int64_t)pos * a.per_row + c) * 8;
      for (int s = 0; s < splits; ++s, q += split_stride) {
        const float4 lo = *(const float4*)q, hi = *(const float4*)(q + 4);
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
      }
      for (int64_t e = tok * a.heavy_n; e < (tok + 1) * a.heavy_n; ++e) {
        const int id = a.heavy[e];
        if (id >= 0) add_bf16x8(v, a.rest[e], a.w[(int64_t)id * a.per_row + c]);
      }
    }
    *(uint4*)(a.dx + i * 8) =
        make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
  }
}

// The heavy slots' part of dW, 8 columns a thread: the token whose place is the
// head of an id's list adds rest * x's row of each of its places, in the order of
// the tokens, to the id's row.
__device__ __forceinline__ void finish_dw(const FinishArgs& a, int64_t i) {
  const int tok = (int)(i / a.per_row), c = (int)(i - (int64_t)tok * a.per_row);
  for (int place = tok * a.heavy_n; place < (tok + 1) * a.heavy_n; ++place) {
    const int64_t id = a.heavy[place];
    if (id < 0) break;                             // (a token's heavy slots stand first)
    if (a.head[id] != place) continue;
    const float4* from = a.dw_bf16 ? (const float4*)a.side + ((a.side_by_id ? id : place) * a.per_row + c) * 2
                                   : (const float4*)a.dw + (id * a.per_row + c) * 2;
    const float4 lo = from[0], hi = from[1];
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    int places[MOST_SHARED], more = place;
#pragma unroll
    for (int k = 0; k < MOST_SHARED; ++k) {
      places[k] = more;
      if (more >= 0) more = a.next[more];
    }
    if (more >= 0) continue;
    for (int last = -1;;) {
      int low = 0x7FFFFFFF;                        // the lowest place above the last one
#pragma unroll
      for (int k = 0; k < MOST_SHARED; ++k)
        if (places[k] > last && places[k] < low) low = places[k];
      if (low == 0x7FFFFFFF) break;
      add_bf16x8(v, a.rest[low], a.x[(int64_t)(low / a.heavy_n) * a.per_row + c]);
      last = low;
    }
    if (a.dw_bf16) {
      ((uint4*)a.dw)[id * a.per_row + c] =
          make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
    } else {
      float4* to = (float4*)a.dw + (id * a.per_row + c) * 2;
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

__global__ __launch_bounds__(256) void head_finish_kernel(FinishArgs a) {
  if ((int)blockIdx.x < a.dx_blocks) {
    finish_dx(a);
  } else {
    for (int64_t i = (int64_t)(blockIdx.x - a.dx_blocks) * 256 + threadIdx.x; i < a.chunks8;
         i += (int64_t)(gridDim.x - a.dx_blocks) * 256)
      finish_dw(a, i);
  }
}

__global__ void head_zero_kernel(uint4* p, int64_t n16) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Host side: the workspace's layout and the calls.
// ---------------------------------------------------------------------------
// Tiles: 256 x 256, one workgroup per compute unit, or 128 x 128, two.
constexpr int HEAD_TILE = 256, HEAD_SMALL = 128, HEAD_CUS = 256;

// Up to this many tokens dz is kept as two bf16 terms, the rounded value and
// what the rounding left (2^-16 together), and both are multiplied, in place of
// the heavy slots' rests: these calls are bound by reading w, not by the matrix
// cores (gradient 8 x 100000 x 4096 612 -> 694 us, 128 x 50000 x 2048 179 -> 210;
// with more tokens it would be half as much again).
constexpr int HEAD_PAIR_TOKENS = 128;

struct HeadPlan {
  int64_t rows, slots, parts, piece;
  int loss_tile, dz_tile, grad_tile, wg_slots;                    // the gradient's workgroups at a time
  int64_t dx_grid, dw_grid;                              // most tiles, splits included
  bool pair, dw_can_split, apart, dx_whole, heavy_dw, side_by_id;
  int heavy_n;                                           // 0: a pair has none
  size_t live, row_of, pos_of, state, ids, p, ent, xc;
  size_t zsel, stats, loss_bytes;                        // the loss
  size_t dz, dxp, dwp, heavy, rest, head, next, side, grad_bytes;   // the gradient
};

// The tile of a product of rows x cols outputs.  A round of 256 x 256 tiles,
// one a compute unit, takes 1.64 times a round of 128 x 128 ones, two a
// compute unit (100 and 61 us at 64 K stages; on 4096 x 32768 outputs 0.80
// against 0.98 ms), so the small tile pays where rounds are few and unfilled.
static int head_tile(int64_t rows, int64_t cols) {
  const int64_t big = ceil_div(ceil_div(rows, HEAD_TILE) * ceil_div(cols, HEAD_TILE), HEAD_CUS);
  const int64_t small = ceil_div(ceil_div(rows, HEAD_SMALL) * ceil_div(cols, HEAD_SMALL), 2 * HEAD_CUS);
  return big * 164 <= small * 100 ? HEAD_TILE : HEAD_SMALL;
}

static HeadPlan head_plan(int64_t tokens, int64_t vocab, int64_t hidden, int64_t top, bool xent, int64_t piece) {
  HeadPlan h = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const int64_t tm = ceil_div(tokens, HEAD_TILE), th = ceil_div(hidden, HEAD_TILE);
  h.pair = tokens <= HEAD_PAIR_TOKENS;
  // rows of dz and of the statistics, in whole tiles: those few tokens only meet small ones
  const int64_t row_tile = h.pair ? HEAD_SMALL : HEAD_TILE;
  h.rows = ceil_div(tokens, row_tile) * row_tile;
  h.slots = xent ? 1 : ceil_div(top, 4) * 4;
  h.loss_tile = h.pair ? HEAD_SMALL : head_tile(tokens, vocab);
  h.parts = ceil_div(vocab, h.loss_tile) * 2;
  h.live = take(12);
  h.row_of = take(4 * tokens);
  h.pos_of = take(4 * tokens);
  h.state = take(xent ? 0 : 4 * tokens);
  h.ids = take(xent ? 0 : 4 * tokens * h.slots);
  h.p = take(xent ? 0 : 4 * tokens * h.slots);
  h.ent = take(xent ? 0 : 4 * tokens);
  h.xc = take(2 * tokens * hidden);
  const size_t shared = at;
  h.zsel = take(4 * tokens * h.slots);
  h.stats = take(8 * h.parts * h.rows);
  h.loss_bytes = at;
  at = shared;
  // default piece: dz of a piece (both its terms) at most 1 GiB, or 2048 ids where these take more
  const int64_t dz_row = h.pair ? 4 : 2;
  if (piece <= 0)
    piece = std::max<int64_t>(2048, (1ll << 30) / (dz_row * std::max<int64_t>(h.rows, 1)) / HEAD_TILE * HEAD_TILE);
  h.piece = ceil_div(std::min(piece, vocab), HEAD_TILE) * HEAD_TILE;
  h.dz_tile = h.pair ? HEAD_SMALL : head_tile(tokens, std::min(h.piece, vocab));
  // dx and dW together, dx counted as the splits it may have: small tiles while both leave compute units idle
  h.grad_tile = h.pair || (h.piece / HEAD_TILE + tm) * th < HEAD_CUS / 2 ? HEAD_SMALL : HEAD_TILE;
  h.wg_slots = h.grad_tile == HEAD_TILE ? HEAD_CUS : 2 * HEAD_CUS;
  const int64_t hn = ceil_div(hidden, h.grad_tile);
  h.dx_grid = ceil_div(std::max<int64_t>(ceil_div(tokens, h.grad_tile) * hn, HEAD_SPLIT_TILES), NXCD) * NXCD;
  h.dw_grid = std::max<int64_t>(h.piece / h.grad_tile * hn, HEAD_SPLIT_TILES);
  h.dz = take(dz_row * h.rows * h.piece);
  // A vocabulary of one piece whose product for dx is too short to be split, or
  // short (a tile of 64 stages takes 90 us) and with tiles enough: its result is
  // dx, stored as such.  Otherwise dx goes through fp32 partial products and
  // head_finish_kernel (gradient 15872 x 69 x 4096: 157 us, 264 through them;
  // 15872 x 1000 x 4096: 404 us and 489).
  const int64_t dx_nk = h.piece / 64 * (h.pair ? 2 : 1);
  h.dx_whole = vocab <= h.piece &&
               (dx_nk < 2 * HEAD_LEAST_STAGES ||
                (dx_nk <= 64 && ceil_div(tokens, h.grad_tile) * hn * 2 > HEAD_SPLIT_TILES));
  // partial products: the tiles of one product, or of all splits of one that
  // is split (fewer live rows may be split more often, but not into more tiles
  // than HEAD_SPLIT_TILES nor more often than HEAD_MOST_SPLITS)
  const int64_t tile_values = (int64_t)h.grad_tile * hidden;
  auto partial = [&](int64_t tile_rows) {
    return 4 * tile_values * std::max(tile_rows, std::min<int64_t>(HEAD_SPLIT_TILES / hn, HEAD_MOST_SPLITS * tile_rows));
  };
  h.dxp = take(h.dx_whole ? 0 : partial(ceil_div(tokens, h.grad_tile)));
  // Two full rounds of dx tiles need nothing to fill up with, and the two
  // products then run apart, each with its own operands in the caches (8192 x
  // 131072 x 4096: 19.26 ms apart, 19.58 together; 512 x 32000 x 2048: 239 us
  // apart, 221 together).
  h.apart = ceil_div(tokens, h.grad_tile) * hn >= 2 * h.wg_slots;
  // as head_splits decides for any number of live rows
  h.dw_can_split = h.piece / h.grad_tile * hn * 2 <= HEAD_SPLIT_TILES &&
                   ceil_div(tokens, 64) * (h.pair ? 2 : 1) / 2 >= HEAD_LEAST_STAGES;
  h.dwp = take(h.dw_can_split ? partial(h.piece / h.grad_tile) : 0);
  h.heavy_n = h.pair ? 0 : xent ? 1 : MOST_HEAVY;
  // (with more tokens than that hardly an id is heavy for so few)
  h.heavy_dw = !h.pair && tokens <= MOST_SHARED * vocab;
  h.heavy = take(4 * tokens * h.heavy_n);
  h.rest = take(4 * tokens * h.heavy_n);
  h.head = take(h.heavy_dw ? 4 * vocab : 0);
  h.next = take(h.heavy_dw ? 4 * tokens * h.heavy_n : 0);
  h.side_by_id = vocab < tokens * h.heavy_n;
  h.side = take(h.heavy_dw ? 4 * std::min(vocab, tokens * h.heavy_n) * hidden : 0);
  h.grad_bytes = at;
  return h;
}

// top: 0 for cross entropy
static pbs_status head_check_dims(const char* what, int64_t tokens, int64_t vocab, int64_t hidden, int64_t top) {
  PBS_REQUIRE(tokens >= 0 && tokens <= (1 << 24) && vocab >= 1 && vocab <= (1 << 22), PBS_ERR_SHAPE,
              "%s: needs tokens in [0, 2^24] and vocab in [1, 2^22] (got %lld, %lld)", what, (long long)tokens,
              (long long)vocab);
  PBS_REQUIRE(hidden >= 64 && hidden % 64 == 0 && hidden <= (1 << 16), PBS_ERR_SHAPE,
              "%s: hidden must be a multiple of 64 in [64, 65536] (got %lld)", what, (long long)hidden);
  PBS_REQUIRE(top >= 0 && top <= 1024, PBS_ERR_SHAPE, "%s: top must be in [1, 1024] (got %lld)", what, (long long)top);
  PBS_REQUIRE(ceil_div(tokens, 64) * ceil_div(vocab, 64) < (1ll << 31) / 16, PBS_ERR_SHAPE,
              "%s: tokens x vocab is too large for one call", what);
  return PBS_OK;
}

struct HeadCall {
  const char* what;
  bool xent;
  const void* x;
  const void* w;
  int64_t tokens, vocab, hidden;
  const int64_t* targets;      // cross entropy
  const int64_t* top_ids;      // distillation
  const void* top_logits;
  pbs_format top_fmt;
  int64_t top;
  float tau;
  float* loss;
  float* lse;                  // the gradient reads it
  const float* dloss;
  int64_t piece;
  void* dx;
  void* dw;
  pbs_format dw_fmt;
  void* ws;
  size_t ws_bytes;
};

static bool off_by(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

static pbs_status head_check(const HeadCall& c, bool grad, HeadPlan* plan) {
  const pbs_status st = head_check_dims(c.what, c.tokens, c.vocab, c.hidden, c.top);
  if (st != PBS_OK) return st;
  PBS_REQUIRE(c.xent || c.top >= 1, PBS_ERR_SHAPE, "%s: top must be in [1, 1024] (got 0)", c.what);
  PBS_REQUIRE(c.tau > 0.0f && c.tau <= 1e30f && c.tau >= 1e-30f, PBS_ERR_INVALID_ARG,
              "%s: temperature must be in [1e-30, 1e30]", c.what);
  PBS_REQUIRE(c.tokens == 0 || (c.xent ? c.targets != nullptr : c.top_ids && c.top_logits), PBS_ERR_INVALID_ARG,
              "%s: null targets", c.what);
  PBS_REQUIRE(!c.top_logits || c.top_fmt == PBS_FMT_F32 || c.top_fmt == PBS_FMT_BF16, PBS_ERR_UNSUPPORTED,
              "%s: teacher logits must be BF16 or F32", c.what);
  PBS_REQUIRE(!off_by(c.targets, 8) && !off_by(c.top_ids, 8) &&
                  !off_by(c.top_logits, c.top_fmt == PBS_FMT_BF16 ? 2 : 4),
              PBS_ERR_INVALID_ARG, "%s: targets not aligned to their elements", c.what);
  PBS_REQUIRE(c.w && !off_by(c.w, 16) && !off_by(c.x, 16), PBS_ERR_INVALID_ARG,
              "%s: x and w must be 16-byte aligned, w not null", c.what);
  PBS_REQUIRE(c.tokens == 0 || (c.x && c.lse), PBS_ERR_INVALID_ARG, "%s: x or lse is null", c.what);
  PBS_REQUIRE(!off_by(c.lse, 4) && !off_by(c.loss, 4) && !off_by(c.dloss, 4), PBS_ERR_INVALID_ARG,
              "%s: loss, lse and dloss must be 4-byte aligned", c.what);
  if (grad) {
    PBS_REQUIRE(c.tokens == 0 || c.dloss, PBS_ERR_INVALID_ARG, "%s: dloss is null", c.what);
    PBS_REQUIRE(c.piece >= 0, PBS_ERR_INVALID_ARG, "%s: piece is negative", c.what);
    PBS_REQUIRE(c.dx || c.dw || c.tokens == 0, PBS_ERR_INVALID_ARG, "%s: dx and dw are both null", c.what);
    PBS_REQUIRE(!off_by(c.dx, 16) && !off_by(c.dw, 16), PBS_ERR_INVALID_ARG, "%s: dx and dw must be 16-byte aligned",
                c.what);
    PBS_REQUIRE(!c.dw || c.dw_fmt == PBS_FMT_F32 || c.dw_fmt == PBS_FMT_BF16, PBS_ERR_UNSUPPORTED,
                "%s: dw must be F32 or BF16", c.what);
  } else {
    PBS_REQUIRE(c.tokens == 0 || c.loss, PBS_ERR_INVALID_ARG, "%s: loss is null", c.what);
  }
  *plan = head_plan(c.tokens, c.vocab, c.hidden, c.top, c.xent, c.piece);
  const size_t need = grad ? plan->grad_bytes : plan->loss_bytes;
  PBS_REQUIRE(c.tokens == 0 || (c.ws && !off_by(c.ws, 256)), PBS_ERR_INVALID_ARG,
              "%s: the workspace is null or not 256-byte aligned", c.what);
  PBS_REQUIRE(c.tokens == 0 || c.ws_bytes >= need, PBS_ERR_INVALID_ARG,
              "%s: the workspace holds %zu bytes, pbs_linear_loss_bytes asks for %zu", c.what, c.ws_bytes, need);
  return PBS_OK;
}

// The live rows, their slots, and the products' common arguments.
static HeadArgs head_rows(const HeadCall& c, const HeadPlan& h, hipStream_t stream) {
  uint8_t* ws = (uint8_t*)c.ws;
  if (!c.xent) {
    TeacherArgs a = {};
    a.ids = c.top_ids; a.logits = c.top_logits; a.bf16 = c.top_fmt == PBS_FMT_BF16;
    a.top = (int)c.top; a.slots = (int)h.slots; a.tokens = (int)c.tokens; a.vocab = (int)c.vocab;
    a.inv_tau = 1.0f / c.tau;
    a.state = (int*)(ws + h.state); a.ids32 = (int*)(ws + h.ids); a.p = (float*)(ws + h.p);
    a.ent = (float*)(ws + h.ent);
    a.heavy = c.loss || h.pair ? nullptr : (int4*)(ws + h.heavy);
    hipLaunchKernelGGL(head_teacher_kernel, dim3((unsigned)ceil_div(c.tokens, 4)), dim3(256), 0, stream, a);
  }
  RowsArgs r = {};
  r.targets = c.targets; r.state = (const int*)(ws + h.state); r.tokens = (int)c.tokens;
  r.live = (int*)(ws + h.live); r.row_of = (int*)(ws + h.row_of); r.pos_of = (int*)(ws + h.pos_of);
  r.loss = c.loss; r.lse = c.loss ? c.lse : nullptr;
  r.x = (const uint4*)c.x; r.xc = (uint4*)(ws + h.xc); r.chunks = (int)(c.hidden / 8);
  r.tile = h.grad_tile; r.dx_tn = (int)ceil_div(c.hidden, h.grad_tile); r.turns = h.pair ? 2 : 1;
  r.dx_nk = (int)(h.piece / 64) * r.turns;
  r.dw_tiles = (int)(h.piece / h.grad_tile) * r.dx_tn; r.slots = h.wg_slots;
  r.together = c.dx && c.dw && !h.apart;
  r.dx_whole = h.dx_whole;
  r.zero_dx = h.dx_whole ? (uint4*)c.dx : nullptr;
  r.vocab = (int)c.vocab;
  if (!c.loss) {
    r.heavy = c.xent && !h.pair ? (int*)(ws + h.heavy) : nullptr;
    r.head = h.heavy_dw && c.dw ? (int*)(ws + h.head) : nullptr;
  }
  hipLaunchKernelGGL(head_rows_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(c.tokens, 16), HEAD_CUS)),
                     dim3(ROWS_THR), 0, stream, r);
  HeadArgs g = {};
  g.x = (const uint8_t*)c.x; g.xc = ws + h.xc; g.w = (const uint8_t*)c.w; g.targets = c.targets;
  g.live = r.live; g.row_of = r.row_of; g.state = r.state; g.ids = (const int*)(ws + h.ids);
  g.p = (const float*)(ws + h.p); g.tokens = (int)c.tokens; g.rows = (int)h.rows; g.hidden = (int)c.hidden;
  g.slots = (int)h.slots; g.nv = g.vocab = (int)c.vocab; g.inv_tau = 1.0f / c.tau;
  return g;
}

template <int T, int EPI, bool PAIR>
static void head_logits(const HeadArgs& g, hipStream_t stream) {
  const dim3 grid((unsigned)(ceil_div(g.tokens, 64 * T) * ceil_div(g.nv, 64 * T)));
  if (g.targets) hipLaunchKernelGGL((head_logits_kernel<T, EPI, false, PAIR>), grid, dim3(256), 0, stream, g);
  else hipLaunchKernelGGL((head_logits_kernel<T, EPI, true, PAIR>), grid, dim3(256), 0, stream, g);
}

static void head_grads(const HeadPlan& h, int64_t dx_blocks, int64_t dw_blocks, HeadArgs g, hipStream_t stream) {
  g.dx_blocks = (int)dx_blocks;
  const dim3 grid((unsigned)(dx_blocks + dw_blocks));
  if (h.pair) hipLaunchKernelGGL((head_grads_kernel<2, true>), grid, dim3(256), 0, stream, g);
  else if (h.grad_tile == HEAD_SMALL) hipLaunchKernelGGL((head_grads_kernel<2, false>), grid, dim3(256), 0, stream, g);
  else hipLaunchKernelGGL((head_grads_kernel<4, false>), grid, dim3(256), 0, stream, g);
}

static pbs_status head_loss(const HeadCall& c, hipStream_t stream) {
  HeadPlan h;
  const pbs_status st = head_check(c, false, &h);
  if (st != PBS_OK || c.tokens == 0) return st;
  uint8_t* ws = (uint8_t*)c.ws;
  HeadArgs g = head_rows(c, h, stream);
  g.zsel = (float*)(ws + h.zsel); g.stats = (float2*)(ws + h.stats);
  log_dispatch("%s tokens=%lld vocab=%lld hidden=%lld top=%lld tile=%d", c.what, (long long)c.tokens,
               (long long)c.vocab, (long long)c.hidden, (long long)c.top, h.loss_tile);
  if (h.loss_tile == HEAD_TILE) head_logits<4, EPI_STATS, false>(g, stream);
  else head_logits<2, EPI_STATS, false>(g, stream);
  JoinArgs j = {};
  j.live = g.live; j.row_of = g.row_of; j.targets = g.targets; j.state = g.state; j.ids = g.ids; j.p = g.p;
  j.ent = (const float*)(ws + h.ent); j.zsel = g.zsel; j.stats = g.stats;
  j.parts = (int)h.parts; j.rows = g.rows; j.slots = g.slots; j.vocab = g.vocab; j.loss = c.loss; j.lse = c.lse;
  hipLaunchKernelGGL(head_join_kernel, dim3((unsigned)ceil_div(c.tokens, JOIN_ROWS)), dim3(JOIN_ROWS * JOIN_Q), 0,
                     stream, j);
  return check_launch(c.what);
}

static pbs_status head_grad(const HeadCall& c, hipStream_t stream) {
  HeadPlan h;
  const pbs_status st = head_check(c, true, &h);
  if (st != PBS_OK) return st;
  const int dwb = c.dw_fmt == PBS_FMT_BF16 ? 2 : 4;
  if (c.tokens == 0) {
    if (c.dw)
      hipLaunchKernelGGL(head_zero_kernel, dim3(1024), dim3(256), 0, stream, (uint4*)c.dw,
                         c.vocab * c.hidden * dwb / 16);
    return check_launch(c.what);
  }
  uint8_t* ws = (uint8_t*)c.ws;
  HeadArgs g = head_rows(c, h, stream);
  g.lse = c.lse; g.dloss = c.dloss; g.dz = (uint16_t*)(ws + h.dz); g.dz_ld = (int)h.piece; g.out_bf16 = dwb == 2;
  g.dx = h.dx_whole ? (uint16_t*)c.dx : nullptr;
  g.dx_part = (float*)(ws + h.dxp); g.dw_part = (float*)(ws + h.dwp);
  g.heavy = h.pair ? nullptr : (const int*)(ws + h.heavy); g.heavy_n = h.heavy_n; g.rest = (float*)(ws + h.rest);
  g.head = h.heavy_dw && c.dw ? (int*)(ws + h.head) : nullptr; g.next = (int*)(ws + h.next);
  g.side = (float*)(ws + h.side); g.side_by_id = h.side_by_id;
  const int per_row = (int)(c.hidden / 8);
  log_dispatch("%s tokens=%lld vocab=%lld hidden=%lld top=%lld piece=%lld tiles=%d,%d", c.what, (long long)c.tokens,
               (long long)c.vocab, (long long)c.hidden, (long long)c.top, (long long)h.piece, h.dz_tile, h.grad_tile);
  for (int64_t v0 = 0; v0 < c.vocab; v0 += h.piece) {
    const int64_t nv = std::min(h.piece, c.vocab - v0);
    g.v0 = (int)v0;
    g.nv = (int)nv;
    g.w = (const uint8_t*)c.w + v0 * c.hidden * 2;
    g.add = v0 > 0;
    g.dw = c.dw ? (uint8_t*)c.dw + v0 * c.hidden * dwb : nullptr;
    if (h.pair) head_logits<2, EPI_DZ, true>(g, stream);
    else if (h.dz_tile == HEAD_SMALL) head_logits<2, EPI_DZ, false>(g, stream);
    else head_logits<4, EPI_DZ, false>(g, stream);
    if (h.apart && c.dx && c.dw) {
      head_grads(h, h.dx_grid, 0, g, stream);
      head_grads(h, 0, h.dw_grid, g, stream);
    } else {
      head_grads(h, c.dx ? h.dx_grid : 0, c.dw ? h.dw_grid : 0, g, stream);
    }
    if (c.dw && h.dw_can_split)
      hipLaunchKernelGGL(head_dw_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(nv * c.hidden / 8, 256), 2048)),
                         dim3(256), 0, stream, g.dw_part, g.live, h.piece * c.hidden, nv * c.hidden / 8, g.dw,
                         g.out_bf16, g.head, g.side, g.side_by_id, g.v0, per_row);
  }
  FinishArgs a = {};
  a.live = g.live; a.pos_of = (const int*)(ws + h.pos_of); a.dx_part = g.dx_part; a.heavy = g.heavy; a.rest = g.rest;
  a.head = g.head; a.next = g.next; a.side = g.side; a.x = (const uint4*)c.x; a.w = (const uint4*)c.w;
  a.dx = (uint16_t*)c.dx; a.dw = c.dw; a.chunks8 = c.tokens * per_row; a.tile = h.grad_tile; a.hidden = g.hidden;
  a.per_row = per_row; a.heavy_n = h.heavy_n; a.dw_bf16 = g.out_bf16; a.side_by_id = h.side_by_id;
  if (c.dx && !h.dx_whole) a.dx_blocks = (int)std::min<int64_t>(ceil_div(a.chunks8, 256), 2048);
  const int64_t blocks = a.dx_blocks + (g.head ? std::min<int64_t>(ceil_div(a.chunks8, 256), 1 << 20) : 0);
  if (blocks > 0) hipLaunchKernelGGL(head_finish_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return check_launch(c.what);
}

}  // namespace pbs

using namespace pbs;

extern "C" {

pbs_status pbs_linear_loss_bytes(int64_t tokens, int64_t vocab, int64_t hidden, int64_t top, int64_t piece,
                                 size_t* loss_bytes, size_t* grad_bytes) {
  PBS_REQUIRE(loss_bytes && grad_bytes, PBS_ERR_INVALID_ARG, "pbs_linear_loss_bytes: null output pointer");
  const pbs_status st = head_check_dims("pbs_linear_loss_bytes", tokens, vocab, hidden, top);
  if (st != PBS_OK) return st;
  PBS_REQUIRE(piece >= 0, PBS_ERR_INVALID_ARG, "pbs_linear_loss_bytes: piece is negative");
  const HeadPlan h = head_plan(tokens, vocab, hidden, top, top == 0, piece);
  *loss_bytes = h.loss_bytes;
  *grad_bytes = h.grad_bytes;
  return PBS_OK;
}

pbs_status pbs_linear_xent(const void* x, const void* w, int64_t tokens, int64_t vocab, int64_t hidden,
                           const int64_t* targets, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  HeadCall c = {};
  c.what = "pbs_linear_xent"; c.x = x; c.w = w; c.tokens = tokens; c.vocab = vocab; c.hidden = hidden;
  c.xent = true; c.targets = targets; c.tau = 1.0f; c.loss = loss; c.lse = lse; c.ws = workspace;
  c.ws_bytes = workspace_bytes;
  return head_loss(c, stream);
}

pbs_status pbs_linear_xent_grad(const float* dloss, const void* x, const void* w, int64_t tokens, int64_t vocab,
                                int64_t hidden, const int64_t* targets, const float* lse, int64_t piece, void* dx,
                                void* dw, pbs_format dw_fmt, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  HeadCall c = {};
  c.what = "pbs_linear_xent_grad"; c.x = x; c.w = w; c.tokens = tokens; c.vocab = vocab; c.hidden = hidden;
  c.xent = true; c.targets = targets; c.tau = 1.0f; c.lse = (float*)lse; c.dloss = dloss; c.piece = piece; c.dx = dx;
  c.dw = dw; c.dw_fmt = dw_fmt; c.ws = workspace; c.ws_bytes = workspace_bytes;
  return head_grad(c, stream);
}

pbs_status pbs_linear_distill(const void* x, const void* w, int64_t tokens, int64_t vocab, int64_t hidden,
                              const int64_t* top_ids, const void* top_logits, pbs_format top_fmt, int64_t top,
                              float temperature, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  HeadCall c = {};
  c.what = "pbs_linear_distill"; c.x = x; c.w = w; c.tokens = tokens; c.vocab = vocab; c.hidden = hidden;
  c.top_ids = top_ids; c.top_logits = top_logits; c.top_fmt = top_fmt; c.top = top; c.tau = temperature;
  c.loss = loss; c.lse = lse; c.ws = workspace; c.ws_bytes = workspace_bytes;
  return head_loss(c, stream);
}

pbs_status pbs_linear_distill_grad(const float* dloss, const void* x, const void* w, int64_t tokens, int64_t vocab,
                                   int64_t hidden, const int64_t* top_ids, const void* top_logits, pbs_format top_fmt,
                                   int64_t top, float temperature, const float* lse, int64_t piece, void* dx, void* dw,
                                   pbs_format dw_fmt, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  HeadCall c = {};
  c.what = "pbs_linear_distill_grad"; c.x = x; c.w = w; c.tokens = tokens; c.vocab = vocab; c.hidden = hidden;
  c.top_ids = top_ids; c.top_logits = top_logits; c.top_fmt = top_fmt; c.top = top; c.tau = temperature;
  c.lse = (float*)lse; c.dloss = dloss; c.piece = piece; c.dx = dx; c.dw = dw; c.dw_fmt = dw_fmt; c.ws = workspace;
  c.ws_bytes = workspace_bytes;
  return head_grad(c, stream);
}

}  // extern "C"
