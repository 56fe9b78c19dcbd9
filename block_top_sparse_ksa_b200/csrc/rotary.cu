// rotary.cu -- rotary positions with several axes, and the write of the rotated
// keys and the values into the cache.
//
// Pair i of a head turns by a = p[axis(i)] f_i.  A float product p f_i is off
// by up to half an ulp of the angle itself (0.03 rad at 10^6), so the angle is
// taken in turns and reduced in fp64, u = p (f_i / 2 pi), u - rint(u), and
// only the fraction, exact to 2^-53 of u, goes on in fp32 (sincospi).
//
// Bound by HBM: every q, k and v element is read and written once (2 + 2
// bytes), plus 8 + 4 A bytes per token.  A CTA takes `tok` tokens: first all
// its loads (positions, slots and 16-byte chunks of data) are put in flight
// together, for with one memory latency a CTA instead of three the bandwidth is
// there; then it computes the tok * P angles into shared memory (once per token,
// not once per head), and each thread turns and stores what it loaded.  A
// thread's item is a pair of chunks of one head that its pairs lie in: chunks i
// and i + P/8 for pairs (i, i + P), neighbours for interleaved pairs, for the
// dims behind the rotary ones, and for v.
#include "ksa_device.cuh"
#include "ksa_internal.h"

namespace ksa {

namespace {

constexpr int kThreads = 256;
// Measured on 16411 tokens of 32 + 8 + 8 heads of 128 (403 MB): 68 us with two items (two 16-byte
// loads each) in flight per thread, three such rounds per CTA and four CTAs per SM (62 registers);
// 70 with four or eight rounds; 82 with three items and one round (three CTAs per SM: between a
// CTA's start and its last store lie two memory latencies, which more CTAs cover).
constexpr int kUnroll = 2, kCtas = 4;
constexpr int kMaxTok = 8;  // tokens per CTA, at most

__device__ __forceinline__ void turn2(uint32_t &a, uint32_t &b, float4 cs) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(a0 * cs.x - b0 * cs.y, a1 * cs.z - b1 * cs.w);
  b = pack_bf16x2(a0 * cs.y + b0 * cs.x, a1 * cs.w + b1 * cs.z);
}

__device__ __forceinline__ uint32_t turn1(uint32_t ab, float c, float s) {
  const float a = bf16_lo(ab), b = bf16_hi(ab);
  return pack_bf16x2(a * c - b * s, a * s + b * c);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtas)
    rotary_append_kernel(const __grid_constant__ RotaryArgs a, int tok, uint32_t per_head) {
  // (cos, sin) of two pairs as one float4, [token][4][P/8]: item i reads its 8 pairs as four
  // rows at column i, so the lanes of a head read neighbouring float4 (no bank conflicts)
  __shared__ float4 cs[kMaxTok * 32];
  __shared__ long long place[kMaxTok];  // of a token's row of kv-head 0 in the cache; -1: padding
  constexpr int kPer = D / 16;   // items of a head
  constexpr int kAngles = kMaxTok * 64 / kThreads;  // a thread's angles, at most
  pdl_wait();
  pdl_launch_dependents();
  const int n0 = blockIdx.x * tok, nt = min(tok, a.N - n0), tid = threadIdx.x;
  const int P = a.rotary_dim >> 1;
  const int q_heads = a.q != nullptr ? a.Hq : 0;
  const int heads = q_heads + (a.k != nullptr ? 2 * a.Hkv : 0);
  const int items = nt * heads * kPer;
  // elements between the kv-heads of a row or page (a contiguous row may hold 2^31 and more)
  const long long head_pitch = static_cast<long long>(a.slots_per_page) * D;
  // first every load that the CTA needs: positions, slots, data
  int pos[kAngles];
#pragma unroll
  for (int i = 0; i < kAngles; ++i) {
    const int e = tid + i * kThreads;
    if (e < nt * P)
      pos[i] = a.positions[static_cast<long long>(a.axis[e % P]) * a.N + n0 + e / P];
  }
  long long my_slot = 0;
  if (tid < nt && a.slots != nullptr) my_slot = a.slots[n0 + tid];
  for (int base = 0; base < items; base += kThreads * kUnroll) {
    uint4 lo[kUnroll], hi[kUnroll];
    int clo[kUnroll], chi[kUnroll], head[kUnroll], t[kUnroll];  // chunks, head and token
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int e = base + u * kThreads + tid;
      t[u] = -1;
      if (e < items) {
        const int i = e % kPer, nh = e / kPer;
        t[u] = tok == 1 ? 0 : heads == 1 ? nh : __umulhi(nh, per_head);  // nh / heads
        head[u] = nh - t[u] * heads;
        const long long n = n0 + t[u];
        const int g = head[u] - q_heads;  // of k and v
        const uint16_t *src = head[u] < q_heads ? a.q + n * a.q_stride + head[u] * D
                              : g < a.Hkv       ? a.k + n * a.k_stride + g * D
                                                : a.v + n * a.v_stride + (g - a.Hkv) * D;
        const bool apart = g < a.Hkv && i < P / 8 && !a.interleaved;
        clo[u] = apart ? i : 2 * i;
        chi[u] = apart ? i + P / 8 : 2 * i + 1;
        lo[u] = reinterpret_cast<const uint4 *>(src)[clo[u]];  // plain loads: q_out may be q
        hi[u] = reinterpret_cast<const uint4 *>(src)[chi[u]];
      }
    }
    if (base == 0) {
#pragma unroll
      for (int i = 0; i < kAngles; ++i) {
        const int e = tid + i * kThreads;
        if (e < nt * P) {
          const int tk = e / P, pair = e - tk * P;
          const double turns = static_cast<double>(pos[i]) * a.turns_per_step[pair];
          float s, c;
          sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
          reinterpret_cast<float2 *>(
              cs)[(tk * 32 + ((pair & 7) >> 1) * (P / 8) + (pair >> 3)) * 2 + (pair & 1)] =
              make_float2(c, s);
        }
      }
      if (tid < nt) {
        if (a.k == nullptr) my_slot = min(my_slot, 0LL);  // no cache: padding or not
        if (my_slot >= a.num_slots) {
          flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
          my_slot = -1;
        }
        long long at = -1;
        if (my_slot >= 0) {
          const int s = static_cast<int>(my_slot), page = s / a.slots_per_page;
          at = (static_cast<long long>(page) * a.Hkv * a.slots_per_page +
                (s - page * a.slots_per_page)) * D;
        }
        place[tid] = at;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (t[u] < 0) continue;
      const long long at = place[t[u]];
      if (at < 0) continue;
      const int g = head[u] - q_heads;
      const bool is_v = g >= a.Hkv;
      const int i = (base + u * kThreads + tid) % kPer;
      if (!is_v && i < P / 8) {
        const int step = P / 8;
        const float4 *w = cs + t[u] * 32 + i;
        const float4 w0 = w[0], w1 = w[step], w2 = w[2 * step], w3 = w[3 * step];
        if (a.interleaved) {
          lo[u].x = turn1(lo[u].x, w0.x, w0.y);
          lo[u].y = turn1(lo[u].y, w0.z, w0.w);
          lo[u].z = turn1(lo[u].z, w1.x, w1.y);
          lo[u].w = turn1(lo[u].w, w1.z, w1.w);
          hi[u].x = turn1(hi[u].x, w2.x, w2.y);
          hi[u].y = turn1(hi[u].y, w2.z, w2.w);
          hi[u].z = turn1(hi[u].z, w3.x, w3.y);
          hi[u].w = turn1(hi[u].w, w3.z, w3.w);
        } else {
          turn2(lo[u].x, hi[u].x, w0);
          turn2(lo[u].y, hi[u].y, w1);
          turn2(lo[u].z, hi[u].z, w2);
          turn2(lo[u].w, hi[u].w, w3);
        }
      }
      uint16_t *dst =
          g < 0 ? a.q_out + static_cast<long long>(n0 + t[u]) * a.q_out_stride + head[u] * D
                : (is_v ? a.V : a.K) + at + (is_v ? g - a.Hkv : g) * head_pitch;
      reinterpret_cast<uint4 *>(dst)[clo[u]] = lo[u];
      reinterpret_cast<uint4 *>(dst)[chi[u]] = hi[u];
    }
  }
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryArgs &a, int num_sms, cudaStream_t stream) {
  // tokens per CTA: the least waves x (rounds + 1 for a CTA's start), so that a decode step's
  // tokens spread over the SMs and a large call ends with full waves (5001 tokens of 48 heads of
  // 64: 5 tokens in two waves instead of 8 in one and a bit)
  const int heads = (a.q != nullptr ? a.Hq : 0) + (a.k != nullptr ? 2 * a.Hkv : 0);
  int tok = 1;
  long long best = -1;
  for (int t = 1; t <= (heads <= 4096 ? kMaxTok : 1); ++t) {
    const long long ctas = (a.N + t - 1) / t, slots = kCtas * num_sms;
    const long long waves = (ctas + slots - 1) / slots;
    const long long per = static_cast<long long>(t) * heads * (a.D / 16);
    const long long cost = waves * ((per + kThreads * kUnroll - 1) / (kThreads * kUnroll) + 1);
    if (best < 0 || cost < best) {
      best = cost;
      tok = t;
    }
  }
  const dim3 grid(static_cast<unsigned>((a.N + tok - 1) / tok)), block(kThreads);
  // x / heads = umulhi(x, per_head) for x < tok * heads: the quotient's error, below x / 2^32,
  // stays below 1 / heads, since tok * heads^2 < 2^32
  const uint32_t per_head = static_cast<uint32_t>((0x100000000ull + heads - 1) / heads);
  if (a.D == 128)
    return launch_pdl(rotary_append_kernel<128>, grid, block, 0, stream, a, tok, per_head);
  return launch_pdl(rotary_append_kernel<64>, grid, block, 0, stream, a, tok, per_head);
}

}  // namespace ksa
