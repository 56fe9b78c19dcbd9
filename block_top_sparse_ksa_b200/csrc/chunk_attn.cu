// chunk_attn.cu -- attention of several query tokens per row over the cache.
//
// One warp per (query token, head), keys 32 at a time: lane l scores key l,
// the running maximum and sum follow the online softmax, and for the output
// each lane owns D/32 dims of the values.  Exact fp32 throughout; the baseline
// that the tensor-core form is measured against.
#include "ksa_device.cuh"
#include "ksa_internal.h"

namespace ksa {

namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) chunk_attn_simple_kernel(const ChunkArgs a) {
  __shared__ float qs[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += blockDim.x)
      if (a.cu_q[b] < 0 || a.cu_q[b] > a.cu_q[b + 1] || a.cu_q[b + 1] > a.N)
        flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
  }
  if (w >= static_cast<long long>(a.N) * a.Hq) return;
  const int n = static_cast<int>(w / a.Hq), h = static_cast<int>(w - static_cast<long long>(n) * a.Hq);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= n)
      lo = mid;
    else
      hi = mid;
  }
  const int b = lo, s0 = max(a.cu_q[b], 0), s1 = min(a.cu_q[b + 1], a.N);
  if (n < s0 || n >= s1) return;
  const int L0 = a.seq_lens[b], L = min(max(L0, 0), a.T);
  if (L != L0 && lane == 0) flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
  const int end = a.causal ? min(static_cast<long long>(L), static_cast<long long>(L) - (s1 - s0) + (n - s0) + 1) : L;
  const int g = h / (a.Hq / a.Hkv);
  for (int d = lane; d < D; d += 32)
    qs[warp][d] = bf16_bits_to_f32(a.q[n * a.q_stride + static_cast<long long>(h) * D + d]) * a.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32];
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int t0 = 0; t0 < end; t0 += 32) {
    const int t = t0 + lane;
    float z = -INFINITY;
    long long row = -1;
    if (t < end) {
      row = kv_row(a.kv, b, g, a.Hkv, a.T, t);
      if (row < 0) {
        flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
      } else {
        const uint4 *k = reinterpret_cast<const uint4 *>(a.K + row * D);
        z = 0.f;
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = k[c];
          const float *q = &qs[warp][c * 8];
          z += q[0] * bf16_lo(x.x) + q[1] * bf16_hi(x.x) + q[2] * bf16_lo(x.y) +
               q[3] * bf16_hi(x.y) + q[4] * bf16_lo(x.z) + q[5] * bf16_hi(x.z) +
               q[6] * bf16_lo(x.w) + q[7] * bf16_hi(x.w);
        }
      }
    }
    float mt = z;
    for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
    const float mn = fmaxf(m, mt);
    if (mn == -INFINITY) continue;
    const float fix = __expf(m - mn), p = __expf(z - mn);
    float ps = p;
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    l = l * fix + ps;
    for (int i = 0; i < D / 32; ++i) o[i] *= fix;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const long long rj = __shfl_sync(0xffffffffu, row, j);
      if (rj < 0) continue;
      for (int i = 0; i < D / 32; ++i) o[i] += pj * bf16_bits_to_f32(a.V[rj * D + i * 32 + lane]);
    }
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const long long at = static_cast<long long>(n) * a.Hq + h;
  for (int i = 0; i < D / 32; ++i) a.out[at * D + i * 32 + lane] = f32_to_bf16_bits(o[i] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[at] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t chunk_attn_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_chunk_attn(const ChunkArgs &a, void *, int, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.N) * a.Hq;
  const dim3 grid(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), block(kWarps * 32);
  if (a.D == 128) return launch_pdl(chunk_attn_simple_kernel<128>, grid, block, 0, stream, a);
  return launch_pdl(chunk_attn_simple_kernel<64>, grid, block, 0, stream, a);
}

}  // namespace ksa
