// fd_rotary.cu -- table of rotary positions: amplitude * cos(p g_i) and
// amplitude * sin(p g_i) for every position p and pair i.
//
// The angle p g_i reaches 10^5 radians, where a 32-bit product has lost it.
// It is kept as a 64-bit fraction of a turn instead (g_i / 2 pi in units of
// 2^-64): the product with p modulo 2^64 is the exact reduction, and the
// distance to the nearest quarter turn, at most an eighth, converts to fp32
// with full relative precision.  There cos and sin are their Taylor sums
// around zero (remainders below 2^-33 and 2^-29), swapped and negated by the
// quarter.
//
// A block takes several steps of a few positions each, the grid's blocks side
// by side in every step.  Position P + j (P the step's first, j the place of a
// thread group) is the turn of P followed by the turn of j,
//   cos(P + j) = cos P cos j - sin P sin j,  sin(P + j) = sin P cos j + cos P sin j,
// so that the series are summed for the steps' P (shared memory) and once for
// j (registers) instead of for every element: one level of sums, no error
// that grows with p.  In units of 2^-24 of the amplitude a sum rounds by 0.6
// (its angle carries a second word) and leaves out 0.03, the amplitude rounds by
// 1, the product and the last sum by 1 of their values: at most 4.52
// altogether.  A table of one step
// sums the series at P + j itself.
//
// The stores bound it: 131072 positions of 128 (67 MB) take 12.4 us in a row,
// 5.4 TB/s, the time of a plain fill (18.5 us with the series summed for every
// element and the frequencies read from parameter space, where lanes that
// differ are served one by one).  Small tables are bound by the launch.
#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSteps = 16;
constexpr int kBlocksPerSm = 8;   // one wave (16: 13.4 us in place of 12.4, 32: 18.4)

// cos and sin of t / 2^64 turns.
__device__ __forceinline__ void cos_sin_turns(unsigned long long t, float& c, float& s) {
  const unsigned quarter = (unsigned)((t + (1ull << 61)) >> 62);   // nearest, mod 4
  const long long r = (long long)(t - ((unsigned long long)quarter << 62));
  // radians y + e in [-pi/4, pi/4]: 2 pi / 2^32 and 2 pi / 2^64, in two words;
  // r = 2^32 (h0 + d) + lo
  constexpr float kHi = 1.4629180793e-9f, kLo = -4.07094e-17f, kUnit = 3.4061216e-19f;
  const int hi = (int)((r + (1ll << 31)) >> 32), lo = (int)(unsigned)r;
  const float h0 = __int2float_rn(hi);
  const float low = fmaf(__int2float_rn(hi - __float2int_rn(h0)), 4294967296.f,
                         __int2float_rn(lo));
  const float y = h0 * kHi;
  const float e = fmaf(low, kUnit, fmaf(h0, kLo, fmaf(h0, kHi, -y)));
  const float z = y * y;
  // sum_{k} (-1)^k y^(2k+1) / (2k+1)!  and  sum_{k} (-1)^k y^(2k) / (2k)!
  float sp = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sp = fmaf(z, sp, 8.3333333e-3f);
  sp = fmaf(z, sp, -1.6666667e-1f);
  float cp = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cp = fmaf(z, cp, -1.3888889e-3f);
  cp = fmaf(z, cp, 4.1666667e-2f);
  cp = fmaf(z, cp, -0.5f);
  const float cn = 1.f + fmaf(z, cp, -e * y);
  const float sn = y + fmaf(y * z, sp, e * cn);
  // turned on by `quarter` quarters: (c, s) -> (-s, c) for each
  const bool swap = quarter & 1u;
  c = swap ? sn : cn;
  s = swap ? cn : sn;
  if (quarter == 1u || quarter == 2u) c = -c;
  if (quarter & 2u) s = -s;
}

__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const __grid_constant__ RotaryTable p,
                                                                int steps) {
  __shared__ float4 cos_p[kMaxSteps * kMaxRotDim / 8], sin_p[kMaxSteps * kMaxRotDim / 8];
  __shared__ unsigned long long turns[kMaxRotDim / 2];
  const int pairs = p.rot_dim / 2, quads = pairs / 4;   // quads: threads per position
  const int per_step = kThreads / quads;                // positions of a step
  const int lane = threadIdx.x % quads, slot = threadIdx.x / quads;
  const long long first = (long long)blockIdx.x * per_step, apart = (long long)gridDim.x * per_step;
  if (threadIdx.x < pairs) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  for (int i = threadIdx.x; i < steps * pairs; i += kThreads) {
    float c = 1.f, s = 0.f;
    if (steps > 1)
      cos_sin_turns(turns[i % pairs] * (unsigned long long)(first + i / pairs * apart), c, s);
    reinterpret_cast<float*>(cos_p)[i] = p.amplitude * c;
    reinterpret_cast<float*>(sin_p)[i] = p.amplitude * s;
  }
  float cj[4], sj[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    cos_sin_turns(turns[4 * lane + k] * (unsigned long long)(steps > 1 ? slot : first + slot),
                  cj[k], sj[k]);
  __syncthreads();
  if (slot >= per_step) return;
  long long pos = first + slot;
  float* row = p.table + pos * p.rot_dim + 4 * lane;
  const long long step = apart * p.rot_dim;
  for (int i = 0; i < steps && pos < p.positions; ++i, pos += apart, row += step) {
    const float4 c = cos_p[i * quads + lane], s = sin_p[i * quads + lane];
    *reinterpret_cast<float4*>(row) =
        make_float4(fmaf(c.x, cj[0], -(s.x * sj[0])), fmaf(c.y, cj[1], -(s.y * sj[1])),
                    fmaf(c.z, cj[2], -(s.z * sj[2])), fmaf(c.w, cj[3], -(s.w * sj[3])));
    *reinterpret_cast<float4*>(row + pairs) =
        make_float4(fmaf(s.x, cj[0], c.x * sj[0]), fmaf(s.y, cj[1], c.y * sj[1]),
                    fmaf(s.z, cj[2], c.z * sj[2]), fmaf(s.w, cj[3], c.w * sj[3]));
  }
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryTable& p, int sms, cudaStream_t stream) {
  const int per_step = kThreads / (p.rot_dim / 8);
  const long long groups = (p.positions + per_step - 1) / per_step;
  // one wave of blocks; beyond kMaxSteps steps each, more of them
  const long long wave = (long long)kBlocksPerSm * sms;
  long long steps = (groups + wave - 1) / wave;
  if (steps > kMaxSteps) steps = kMaxSteps;
  const long long blocks = (groups + steps - 1) / steps;
  rotary_table_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(p, (int)steps);
  return cudaGetLastError();
}

}  // namespace fd
