// qmm_records.h -- where the bytes of a repacked record come from (the layout is
// described in qmm_repack.hip).
#pragma once

#include "qmm_device.h"

namespace qmm {
namespace rp {

struct Shape {
  int B;            // bytes of one row's k-block
  int n_lane;       // lane sections
  int n_row;        // row sections
  int width[4];     // bytes per row of each row section
};

template <int KIND> struct Map;

// The 4-bit-code kinds: lane section c, slot (G, j), byte i holds code byte
// 4G + i%4 of block 4c + i/4 (code bytes start at `at` in a block of `bb`).
template <int BB, int AT>
struct NibMap {
  __device__ static int lane(int c, int G, int i) { return BB * (4 * c + i / 4) + AT + 4 * G + i % 4; }
};

template <> struct Map<Q4_0> : NibMap<18, 2> {
  static constexpr Shape shape{144, 2, 1, {16, 0}};
  __device__ static int row(int, int i) { return 18 * (i / 2) + i % 2; }  // the f16 scales
};
template <> struct Map<IQ4_NL> : Map<Q4_0> {};
template <> struct Map<MXFP4> : NibMap<17, 1> {
  static constexpr Shape shape{136, 2, 1, {8, 0}};
  __device__ static int row(int, int i) { return 17 * i; }  // the E8M0 bytes
};
template <> struct Map<Q5_0> : NibMap<22, 6> {
  static constexpr Shape shape{176, 2, 2, {32, 16}};
  __device__ static int row(int sec, int i) {
    return sec == 0 ? 22 * (i / 4) + 2 + i % 4   // the 32-bit qh words
                    : 22 * (i / 2) + i % 2;      // the f16 scales
  }
};
template <> struct Map<Q8_0> {
  static constexpr Shape shape{272, 4, 1, {16, 0}};
  // Section c: code bytes 8G .. 8G+7 of blocks 2c and 2c+1.
  __device__ static int lane(int c, int G, int i) { return 34 * (2 * c + i / 8) + 2 + 8 * G + i % 8; }
  __device__ static int row(int, int i) { return 34 * (i / 2) + i % 2; }
};
template <> struct Map<IQ4_XS> {
  static constexpr Shape shape{136, 2, 1, {8, 0}};
  __device__ static int lane(int c, int G, int i) { return 8 + 16 * (4 * c + i / 4) + 4 * G + i % 4; }
  __device__ static int row(int, int i) { return i; }  // d, scales_h, scales_l
};
template <> struct Map<Q4_K> {
  static constexpr Shape shape{144, 2, 1, {16, 0}};
  __device__ static int lane(int c, int G, int i) { return 16 + 32 * G + 16 * c + i; }
  __device__ static int row(int, int i) { return i; }  // d, dmin, scales and mins
};
template <> struct Map<Q6_K> {
  static constexpr Shape shape{210, 3, 2, {16, 2}};
  __device__ static int lane(int c, int G, int i) {
    const int h = G >> 1, a = G & 1;
    return c == 0 ? 64 * h + 16 * a + i : c == 1 ? 64 * h + 32 + 16 * a + i : 128 + 32 * h + 16 * a + i;
  }
  __device__ static int row(int sec, int i) { return sec == 0 ? 192 + i : 208 + i; }  // scales, d
};

// Q5_K: the Q4_K code sections, then qh[32] and the 16-byte header as row
// sections (every group of a row reads all 32 fifth-bit bytes).
template <> struct Map<Q5_K> {
  static constexpr Shape shape{176, 2, 2, {32, 16}};
  __device__ static int lane(int c, int G, int i) { return 48 + 32 * G + 16 * c + i; }
  __device__ static int row(int sec, int i) { return sec == 0 ? 16 + i : i; }  // qh, then d, dmin, scales
};
// Q2_K and Q3_K: group G = 2n + a takes code bytes 32n + 16a .. + 15.
template <> struct Map<Q2_K> {
  static constexpr Shape shape{84, 1, 2, {16, 4}};
  __device__ static int lane(int, int G, int i) { return 16 + 16 * G + i; }
  __device__ static int row(int sec, int i) { return sec == 0 ? i : 80 + i; }  // scales, then d, dmin
};
template <> struct Map<Q3_K> {
  static constexpr Shape shape{110, 1, 4, {32, 8, 4, 2}};
  __device__ static int lane(int, int G, int i) { return 32 + 16 * G + i; }
  __device__ static int row(int sec, int i) {  // hmask, scale bytes 0-7, scale bytes 8-11, d
    return sec == 0 ? i : sec == 1 ? 96 + i : sec == 2 ? 104 + i : 108 + i;
  }
};

// Row j (in the tile) and offset in its k-block of record byte o.
template <int KIND>
__device__ void source(int o, int &j, int &off) {
  using Mp = Map<KIND>;
  constexpr Shape sh = Mp::shape;
  if (o < 1024 * sh.n_lane) {
    const int c = o >> 10, slot = (o & 1023) >> 4;
    j = slot & 15;
    off = Mp::lane(c, slot >> 4, o & 15);
    return;
  }
  o -= 1024 * sh.n_lane;
#pragma unroll
  for (int sec = 0; sec < sh.n_row; ++sec) {
    if (o < 16 * sh.width[sec] || sec == sh.n_row - 1) {
      j = o / sh.width[sec];
      off = Mp::row(sec, o % sh.width[sec]);
      return;
    }
    o -= 16 * sh.width[sec];
  }
}

}  // namespace rp
}  // namespace qmm
