// fd_rotary.cu -- table of rotary positions: amplitude * cos(p g_i) and
// amplitude * sin(p g_i) for every position p and pair i.
//
// The angle p g_i reaches 10^5 radians, where a 32-bit product has lost it.
// It is kept as a 64-bit fraction of a turn instead (g_i / 2 pi in units of
// 2^-64): the product with p modulo 2^64 is the exact reduction, and the
// distance to the nearest quarter turn, at most an eighth, converts to fp32
// with full relative precision.  There cos and sin are their Taylor sums
// around zero (remainders below 2^-31), swapped and negated by the quarter.
//
// One thread holds four neighbouring pairs and walks down the positions, so a
// step is four 64-bit additions and two 16-byte stores.  131072 positions of
// 128 (67 MB) take 22 us, 3.0 TB/s into a flushed L2: the arithmetic (about 40
// operations a pair) and the launch bound it, not the stores.
#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int kThreads = 256;

// cos and sin of t / 2^64 turns.
__device__ __forceinline__ void cos_sin_turns(unsigned long long t, float& c, float& s) {
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);   // nearest, mod 4
  const long long r = (long long)(t - ((unsigned long long)quarter << 62));
  // radians in [-pi/4, pi/4]: 2 pi / 2^64
  const float y = __ll2float_rn(r) * 3.4061215800304e-19f;
  const float z = y * y;
  // sum_{k} (-1)^k y^(2k+1) / (2k+1)!  and  sum_{k} (-1)^k y^(2k) / (2k)!
  float sp = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sp = fmaf(z, sp, 8.3333333e-3f);
  sp = fmaf(z, sp, -1.6666667e-1f);
  const float sn = fmaf(y * z, sp, y);
  float cp = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cp = fmaf(z, cp, -1.3888889e-3f);
  cp = fmaf(z, cp, 4.1666667e-2f);
  cp = fmaf(z, cp, -0.5f);
  const float cn = fmaf(z, cp, 1.f);
  // turned on by `quarter` quarters: (c, s) -> (-s, c) for each
  const bool swap = quarter & 1u;
  c = swap ? sn : cn;
  s = swap ? cn : sn;
  if (quarter == 1u || quarter == 2u) c = -c;
  if (quarter & 2u) s = -s;
}

__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const __grid_constant__ RotaryTable p,
                                                                int steps) {
  const int quads = p.rot_dim / 8;           // threads per position
  const int per_block = kThreads / quads;    // positions a block takes per step
  const int lane = threadIdx.x % quads, slot = threadIdx.x / quads;
  if (slot >= per_block) return;
  long long pos = (long long)blockIdx.x * per_block * steps + slot;
  unsigned long long t[4], dt[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long g = p.turns[4 * lane + k];
    t[k] = g * (unsigned long long)pos;
    dt[k] = g * (unsigned long long)per_block;
  }
  float* row = p.table + pos * p.rot_dim + 4 * lane;
  const long long step = (long long)per_block * p.rot_dim;
  for (int i = 0; i < steps && pos < p.positions; ++i, pos += per_block, row += step) {
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      cos_sin_turns(t[k], c[k], s[k]);
      t[k] += dt[k];
    }
    const float a = p.amplitude;
    *reinterpret_cast<float4*>(row) = make_float4(a * c[0], a * c[1], a * c[2], a * c[3]);
    *reinterpret_cast<float4*>(row + p.rot_dim / 2) =
        make_float4(a * s[0], a * s[1], a * s[2], a * s[3]);
  }
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryTable& p, int sms, cudaStream_t stream) {
  const int per_block = kThreads / (p.rot_dim / 8);
  const long long groups = (p.positions + per_block - 1) / per_block;
  // eight blocks fill an SM; a thread walks several positions where there are
  // more than that
  long long steps = (groups + 8ll * sms - 1) / (8ll * sms);
  if (steps > 64) steps = 64;
  const long long blocks = (groups + steps - 1) / steps;
  rotary_table_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(p, (int)steps);
  return cudaGetLastError();
}

}  // namespace fd
