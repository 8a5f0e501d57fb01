// Pieces shared by the products of head.hip and muon.hip: operand stages of 64
// 16-bit K values filled by LDS-DMA, the transposing LDS read, and the barrier
// that leaves a wave's last loads in flight.
#pragma once
#include "gemm_common.hpp"

namespace pbs {

enum { KMAJ = 0, MNMAJ = 1 };                    // how an operand is stored

// Bytes of one K stage of a tile's 64 T rows.
template <int T> constexpr int tile_bytes() { return 64 * T * ROWB; }

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
// 3), or, in rows of 8 chunks (T = 1), c ^ 4 (k / 2 & 1).  Chunks past the operand's width re-read its last one; K rows past its
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
      int lc = (lane % CH) ^ (4 * (T == 1 ? row >> 1 & 1 : row & 3));
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
__device__ __forceinline__ i16x4 read_lds_tr16(const uint8_t* __restrict__ p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
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

}  // namespace pbs
