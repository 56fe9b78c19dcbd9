// rotary.cu -- rotary positions with several axes, and the write of the rotated
// keys and the values into the cache.
//
// Pair i of a head turns by a = p[axis(i)] f_i.  A float product p f_i is off
// by up to half an ulp of the angle itself (0.03 rad at 10^6), so the angle is
// taken in turns and reduced in fp64, u = p (f_i / 2 pi), u - rint(u), and
// only the fraction, exact to 2^-53 of u, goes on in fp32 (sincospi).
//
// Bound by HBM: every q, k and v element is read and written once (2 + 2
// bytes), plus 8 + 4 A bytes per token.  A CTA takes `tok` tokens: first every
// thread has its loads of 16-byte chunks in flight, then the CTA computes the
// tok * P angles into shared memory (once per token, not once per head), then
// each thread turns and stores what it loaded.  A thread's item is a pair of
// chunks of one head that its pairs lie in: chunks i and i + P/8 for pairs
// (i, i + P), neighbours for interleaved pairs, for the dims behind the rotary
// ones, and for v.
#include "ksa_device.cuh"
#include "ksa_internal.h"

namespace ksa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // items (two 16-byte loads each) a thread has in flight
constexpr int kMaxTok = 4;  // tokens per CTA, large calls

struct Item {
  uint4 lo, hi;
};

__device__ __forceinline__ void turn2(uint32_t &a, uint32_t &b, float4 cs) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(a0 * cs.x - b0 * cs.y, a1 * cs.z - b1 * cs.w);
  b = pack_bf16x2(a0 * cs.y + b0 * cs.x, a1 * cs.w + b1 * cs.z);
}

__device__ __forceinline__ uint32_t turn1(uint32_t ab, float c, float s) {
  const float a = bf16_lo(ab), b = bf16_hi(ab);
  return pack_bf16x2(a * c - b * s, a * s + b * c);
}

__global__ void __launch_bounds__(kThreads)
    rotary_append_kernel(const __grid_constant__ RotaryArgs a, int tok) {
  // (cos, sin) of two pairs as one float4, [token][4][P/8]: item i reads its 8 pairs as four
  // rows at column i, so the lanes of a head read neighbouring float4 (no bank conflicts)
  __shared__ float4 cs[kMaxTok * 32];
  __shared__ int slot[kMaxTok];  // < 2^31: the caches' rows are
  pdl_wait();
  pdl_launch_dependents();
  const int n0 = blockIdx.x * tok, nt = min(tok, a.N - n0);
  const int P = a.rotary_dim >> 1, per = a.D / 16;  // items of a head
  const int heads = (a.q != nullptr ? a.Hq : 0) + (a.k != nullptr ? 2 * a.Hkv : 0);
  const int q_heads = a.q != nullptr ? a.Hq : 0;
  const int items = nt * heads * per;
  if (threadIdx.x < nt) {
    long long s = a.slots != nullptr ? a.slots[n0 + threadIdx.x] : 0;
    if (a.slots != nullptr && s >= a.num_slots) {
      flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
      s = -1;
    }
    slot[threadIdx.x] = s < 0 ? -1 : static_cast<int>(s);
  }
  __syncthreads();
  for (int base = 0; base < items; base += kThreads * kUnroll) {
    Item it[kUnroll];
    const uint4 *src[kUnroll];
    uint16_t *dst[kUnroll];
    int lo[kUnroll], hi[kUnroll], at[kUnroll];  // chunks of the item; its column in cs, or -1
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = base + u * kThreads + threadIdx.x;
      dst[u] = nullptr;
      if (e < items) {
        const int i = e % per, nh = e / per, t = nh / heads, h = nh - t * heads;
        const int s = slot[t];
        const long long n = n0 + t;
        if (s >= 0) {
          const bool is_v = h >= q_heads + a.Hkv;
          if (h < q_heads) {
            src[u] = reinterpret_cast<const uint4 *>(a.q + n * a.q_stride + h * a.D);
            dst[u] = a.q_out + n * a.q_out_stride + h * a.D;
          } else {
            const int g = h - q_heads - (is_v ? a.Hkv : 0);
            src[u] = reinterpret_cast<const uint4 *>(
                (is_v ? a.v + n * a.v_stride : a.k + n * a.k_stride) + g * a.D);
            const int page = s / a.slots_per_page, off = s - page * a.slots_per_page;
            dst[u] = (is_v ? a.V : a.K) +
                     ((static_cast<long long>(page) * a.Hkv + g) * a.slots_per_page + off) * a.D;
          }
          const bool turned = !is_v && i < P / 8;
          at[u] = turned ? t * 32 + i : -1;
          lo[u] = a.interleaved || is_v ? 2 * i : turned ? i : 2 * i;
          hi[u] = turned && !a.interleaved ? i + P / 8 : lo[u] + 1;
          it[u].lo = src[u][lo[u]];  // plain loads: q_out may be q
          it[u].hi = src[u][hi[u]];
        }
      }
    }
    if (base == 0 && P > 0) {
      for (int e = threadIdx.x; e < nt * P; e += kThreads) {
        const int t = e / P, i = e - t * P;
        const double turns =
            static_cast<double>(a.positions[static_cast<long long>(a.axis[i]) * a.N + n0 + t]) *
            a.turns_per_step[i];
        float s, c;
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
        reinterpret_cast<float2 *>(cs)[(t * 32 + ((i & 7) >> 1) * (P / 8) + (i >> 3)) * 2 +
                                       (i & 1)] = make_float2(c, s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (dst[u] == nullptr) continue;
      if (at[u] >= 0) {
        const float4 *w = cs + at[u];
        const int step = P / 8;
        const float4 w0 = w[0], w1 = w[step], w2 = w[2 * step], w3 = w[3 * step];
        if (a.interleaved) {
          it[u].lo.x = turn1(it[u].lo.x, w0.x, w0.y);
          it[u].lo.y = turn1(it[u].lo.y, w0.z, w0.w);
          it[u].lo.z = turn1(it[u].lo.z, w1.x, w1.y);
          it[u].lo.w = turn1(it[u].lo.w, w1.z, w1.w);
          it[u].hi.x = turn1(it[u].hi.x, w2.x, w2.y);
          it[u].hi.y = turn1(it[u].hi.y, w2.z, w2.w);
          it[u].hi.z = turn1(it[u].hi.z, w3.x, w3.y);
          it[u].hi.w = turn1(it[u].hi.w, w3.z, w3.w);
        } else {
          turn2(it[u].lo.x, it[u].hi.x, w0);
          turn2(it[u].lo.y, it[u].hi.y, w1);
          turn2(it[u].lo.z, it[u].hi.z, w2);
          turn2(it[u].lo.w, it[u].hi.w, w3);
        }
      }
      uint4 *out = reinterpret_cast<uint4 *>(dst[u]);
      out[lo[u]] = it[u].lo;
      out[hi[u]] = it[u].hi;
    }
  }
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryArgs &a, int num_sms, cudaStream_t stream) {
  // one token per CTA while that leaves SMs without work, so a decode step's few tokens spread
  const int tok = a.N <= 4 * num_sms ? 1 : kMaxTok;
  return launch_pdl(rotary_append_kernel, dim3(static_cast<unsigned>((a.N + tok - 1) / tok)),
                    dim3(kThreads), 0, stream, a, tok);
}

}  // namespace ksa
