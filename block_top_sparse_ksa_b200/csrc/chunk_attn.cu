// chunk_attn.cu -- attention of several query tokens per row over the cache, on
// the 5th-generation tensor cores.
//
// Mathematics.  The G query heads of a kv-head see the same keys, so the rows
// of a product are (token, head) pairs, TQ = 128 / G tokens by G heads: a query
// tile of 128 rows.  Over key tiles of 128 tokens, with running row maximum m,
// sum l and output O (online softmax):
//   S = Q K^T;  m' = max(m, max S);  P = 2^(c (S - m'));   c = scale log2 e
//   l = l 2^(c (m - m')) + sum P;  O = O 2^(c (m - m')) + P V.
// m only moves when a row's maximum rose by more than a factor 2^8 in weight
// (P then stays below 2^8 and l and O far inside fp32), so O is rescaled a few
// times per row and not once per tile; the quotient O / l does not depend on m.
//
// Layout.  One CTA holds two streams, each with its S (whose first half P
// overwrites) and O in tensor memory, four softmax warps of one row per thread:
// no shuffles.  While one stream's softmax runs, the tensor cores work for the
// other.  PAIR: the streams are two query tiles over the same key tiles.
// Otherwise (few query rows per sequence) they are one query tile over the even
// and the odd key tiles, joined at the end.  One warp loads (TMA; a page's rows
// of one kv-head are one box), one issues the products.  Keys and values share
// one ring of stages.  When there are fewer (tile, kv-head) pairs than SMs, the
// keys are split between CTAs; the last CTA of a tile to finish joins the parts
// in their order (so results do not depend on timing).
#include "ksa_device.cuh"
#include "ksa_internal.h"
#include "tcgen05_device.cuh"

namespace ksa {

namespace {

constexpr int kQ = 128;         // query rows of a tile
constexpr int kKeys = 64;       // key tokens of a tile
constexpr int kSoftWarps = 8;   // four per stream
constexpr int kThreads = (kSoftWarps + 2) * 32;
constexpr int kBadRing = 64;    // key tiles whose page marks are kept (above any stage count)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kLead = 4, kLag = 10;  // stagger of the weights' loop, in pairs of keys
constexpr float kRescale = 8.f;  // log2 of the largest weight before m moves

template <int D, bool PAIR>
struct Cfg {
  static constexpr int kQBytes = kQ * D * 2, kTileBytes = kKeys * D * 2;  // of a Q, of a K or V tile
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr int kFit = (224 * 1024 - kQTiles * kQBytes) / kTileBytes;
  static constexpr int kStages = kFit < 20 ? kFit : 20;
  static constexpr int kRows = kQ * kQTiles;  // query rows of a CTA
  static constexpr int kAhead = PAIR ? 2 : 4;  // key tiles whose scores are in flight or in use
  // 1 KB for the alignment of the tiles, the rest for barriers beside them
  static constexpr int kSmem = kQTiles * kQBytes + kStages * kTileBytes + 1024 + 2048;
};

struct Ctl {  // in shared memory
  uint64_t q_full, full[20], empty[20];
  // per stream and score buffer: scores ready, weights ready, product with V done
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2], drain;
  uint32_t tmem;
  int abort, row, last;
  uint32_t bad[kBadRing];
};

struct Plan {
  int pair, tokens, slots, splits;  // tokens: query tokens of a CTA
};

struct Params {
  ChunkArgs a;
  uint32_t *sem;
  float *part;
  int tq, slots, splits;  // tq: query tokens of a tile
};

// Waits with a limit; false (and the CTA's abort mark) when it runs out.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int *>(abort) != 0) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      *reinterpret_cast<volatile int *>(abort) = 1;
      return false;
    }
  }
  return true;
}

// Largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void exp2_in_place(uint32_t &x) {  // kept in program order
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+r"(x));
}

// Offset of row b's first tile slot: rows b in order, each with at least
// ceil(tokens / TT) slots, without a prefix sum over the rows.
__device__ __forceinline__ int first_slot(const ChunkArgs &a, int b, int TT) {
  return min(max(a.cu_q[b], 0), a.N) / TT + b;
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ Params p) {
  using C = Cfg<D, PAIR>;
  constexpr int NST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *tiles = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Ctl &ctl = *reinterpret_cast<Ctl *>(tiles + C::kQTiles * C::kQBytes + NST * C::kTileBytes);
  static_assert(sizeof(Ctl) <= 2048 && NST <= 20 && NST < kBadRing, "");
  const ChunkArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv, TQ = p.tq, TT = TQ * C::kQTiles;

  // slots run backwards: a row's last tiles see the most keys when causal
  int x = blockIdx.x;
  const int z = x / (p.slots * a.Hkv);
  x -= z * p.slots * a.Hkv;
  const int g = x / p.slots, slot = p.slots - 1 - (x - g * p.slots);

  if (blockIdx.x == 0) {
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_q[b] < 0 || a.cu_q[b] > a.cu_q[b + 1] || a.cu_q[b + 1] > a.N)
        flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
  }
  if (warp == 0) {  // the row of this slot: 32-way search
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const bool le = at < hi && first_slot(a, at, TT) <= slot;
      const uint32_t no = ~__ballot_sync(0xffffffffu, le);
      const int cnt = no == 0u ? 32 : __ffs(no) - 1;
      lo += cnt * step;
      hi = min(hi, lo + step);
    }
    if (lane == 0) {
      ctl.row = lo;
      ctl.abort = 0;
    }
  } else if (warp == kSoftWarps) {
    if (lane == 0) {
      mbar_init(&ctl.q_full, 1);
      for (int i = 0; i < NST; ++i) {
        mbar_init(&ctl.full[i], 1);
        mbar_init(&ctl.empty[i], 1);
      }
      for (int s = 0; s < 2; ++s) {
        for (int i = 0; i < 2; ++i) {
          mbar_init(&ctl.s_full[s][i], 1);
          mbar_init(&ctl.p_full[s][i], 4);
          mbar_init(&ctl.o_done[s][i], 1);
        }
      }
      mbar_init(&ctl.drain, 1);
      fence_mbar_init();
    }
  } else if (warp == kSoftWarps + 1) {
    if (lane == 0) {
      prefetch_tensormap(&q_map);
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
  }
  __syncthreads();

  const int b = ctl.row;
  const int s0 = min(max(a.cu_q[b], 0), a.N), s1 = max(s0, min(a.cu_q[b + 1], a.N));
  const int n = s1 - s0, tok0 = (slot - (s0 / TT + b)) * TT;  // first token, within the row
  if (tok0 < 0 || tok0 >= n) return;
  const int L0 = a.seq_lens[b], L = min(max(L0, 0), a.T);
  if (L != L0 && tid == 0) flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
  const int tokens = min(TT, n - tok0);  // of this CTA
  // keys that the CTA's last token sees, in tiles, and this CTA's share of them
  const int kend = a.causal ? max(0, L - n + tok0 + tokens) : L;
  const int all = (kend + kKeys - 1) / kKeys, share = (all + p.splits - 1) / p.splits;
  const int parts = share == 0 ? 1 : (all + share - 1) / share;
  if (z >= parts) return;
  const int t0 = z * share, nt = min(share, all - t0);
  const int q_tiles = PAIR && tokens > TQ ? 2 : 1;

  uint32_t tmem = 0;
  if (nt > 0) {
    if (warp == kSoftWarps) {
      tmem_alloc(&ctl.tmem, 512);
      tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    tmem = ctl.tmem;
  }
  uint8_t *ring = tiles + C::kQTiles * C::kQBytes;

  // the ring's order is the order of use: K0 ... K(A-1), V0, K(A), V1, K(A+1), ...
  constexpr int A = C::kAhead;

  if (nt > 0 && warp == kSoftWarps + 1) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      mbar_arrive_expect_tx(&ctl.q_full, static_cast<uint32_t>(q_tiles * G * TQ * D * 2));
      for (int s = 0; s < q_tiles; ++s)
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(tiles + s * C::kQBytes + h * (kQ * 128), &q_map, h * 64, g * G,
                      s0 + tok0 + s * TQ, &ctl.q_full);
    }
    const bool paged = a.kv.table != nullptr;
    const int bs = paged ? a.kv.bs : kKeys, ppt = kKeys / bs;  // boxes of a tile and half
    const int groups = 32 / ppt;                               // tiles whose ids 32 lanes hold
    const int box = lane % ppt, half = lane / ppt;
    const long long rows =
        paged ? static_cast<long long>(a.kv.num_pages) * a.Hkv * bs
              : static_cast<long long>(a.B) * a.Hkv * a.T;
    const int none = static_cast<int>(rows);  // a row past the pool: the box reads as zeros
    const int32_t *table = paged ? a.kv.table + static_cast<size_t>(b) * a.kv.max_blocks : nullptr;
    const int blocks = (kend + bs - 1) / bs;
    auto load_ids = [&](int group) {  // the page of block (t0 + group * groups) * ppt + lane
      const int j = (t0 + group * groups) * ppt + lane;
      return paged && j < blocks && j < a.kv.max_blocks ? __ldg(table + j) : -1;
    };
    int ids = load_ids(0), next = load_ids(1);
    int stage = 0, puts = 0;
    uint32_t drained = 1;  // a place's first filling waits for nothing
    bool ok = true;
    auto put = [&](const CUtensorMap *map, int y) {  // one tile into the next place
      ok = wait_bar(&ctl.empty[stage], drained, &ctl.abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(&ctl.full[stage], C::kTileBytes);
      __syncwarp();
      if (lane < ppt * (D / 64))
        tma_load_2d(ring + stage * C::kTileBytes + half * (kKeys * 128) + box * bs * 128, map,
                    half * 64, y, &ctl.full[stage]);
      ++puts;
      if (++stage == NST) {
        stage = 0;
        drained ^= 1u;
      }
    };
    // K runs A tiles ahead of V; the rows of the tiles between wait in registers
    int group = 0, y_ring[A];
    for (int j = 0; j < nt + A && ok; ++j) {
      if (j >= A) put(&v_map, y_ring[0]);  // of tile j - A
#pragma unroll
      for (int i = 0; i + 1 < A; ++i) y_ring[i] = y_ring[i + 1];
      if (j >= nt || !ok) continue;
      int y = none;
      if (paged) {
        if (j / groups != group) {
          ids = next;
          next = load_ids(++group + 1);
        }
        const int block = (t0 + j) * ppt + box;
        const int id = __shfl_sync(0xffffffffu, ids, (j % groups) * ppt + box);
        const bool inside = block < blocks, good = id >= 0 && id < a.kv.num_pages;
        if (inside && good) y = (id * a.Hkv + g) * bs;
        const uint32_t bad = __ballot_sync(0xffffffffu, lane < ppt && inside && !good);
        if (lane == 0) {
          ctl.bad[j % kBadRing] = bad;
          if (bad != 0u) flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
        }
      } else {
        y = (b * a.Hkv + g) * a.T + (t0 + j) * kKeys;
        if (lane == 0) ctl.bad[j % kBadRing] = 0u;
      }
      put(&k_map, y);
      y_ring[A - 1] = y;
    }
    // leave no copy in flight behind (also after an aborted wait)
    for (int i = max(0, puts - NST); i < puts; ++i)
      wait_bar(&ctl.full[i % NST], (i / NST) & 1, &ctl.abort);
    wait_bar(&ctl.q_full, 0, &ctl.abort);
  } else if (nt > 0 && warp == kSoftWarps) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idesc_s = mma_idesc_bf16(kQ, kKeys, false);
    constexpr uint32_t idesc_o = mma_idesc_bf16(kQ, D, true);
    bool ok = wait_bar(&ctl.q_full, 0, &ctl.abort);
    const int streams = PAIR ? q_tiles : 2;
    const uint64_t q_desc = smem_desc_128b(smem_addr(tiles), 16, 1024);
    const uint64_t k_desc = smem_desc_128b(smem_addr(ring), 16, 1024);
    const uint64_t v_desc = smem_desc_128b(smem_addr(ring), kKeys * 128, 1024);
    const uint32_t one = elect_one();
    int stage = 0;  // next place of the ring, and the parity of its filling
    uint32_t fill = 0;
    auto take = [&]() {  // waits for the next place and returns it
      const int st = stage;
      ok = ok && wait_bar(&ctl.full[st], fill, &ctl.abort);
      if (++stage == NST) {
        stage = 0;
        fill ^= 1u;
      }
      return st;
    };
    // scores of stream s's k-th tile, its keys in place st: to buffer k % 2
    auto scores = [&](int s, int k, int st) {
      const uint64_t qd = q_desc + static_cast<uint64_t>((PAIR ? s : 0) * C::kQBytes >> 4);
      const uint64_t kd = k_desc + static_cast<uint64_t>(st * C::kTileBytes >> 4);
      const uint32_t to = tmem + s * 2 * kKeys + (k & 1) * kKeys;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        mma_ss(one, to, qd + static_cast<uint64_t>(((i / 4) * (kQ * 128) + (i % 4) * 32) >> 4),
               kd + static_cast<uint64_t>(((i / 4) * (kKeys * 128) + (i % 4) * 32) >> 4), idesc_s,
               i > 0);
      mma_commit(one, &ctl.s_full[s][k & 1]);
      if (!PAIR || s == streams - 1) mma_commit(one, &ctl.empty[st]);
    };
    for (int j = 0; j < min(A, nt); ++j) {
      const int st = take();
      if (!ok) break;
      tmem_fence_after();
      if (PAIR)
        for (int s = 0; s < streams; ++s) scores(s, j, st);
      else
        scores(j & 1, j >> 1, st);
    }
    for (int j = 0; j < nt && ok; ++j) {
      const int sv = take();
      int sk = 0;
      if (!ok) break;
      if ((t0 + j + 1) * kKeys > L) {
        // the cache behind the row's last token: P is 0 there, but 0 x NaN is not
        const int r0 = L - (t0 + j) * kKeys;
        for (int e = r0 * 8 + lane; e < kKeys * 8; e += 32)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<uint4 *>(ring + sv * C::kTileBytes + h * (kKeys * 128) + e * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint64_t vd = v_desc + static_cast<uint64_t>(sv * C::kTileBytes >> 4);
      const int k = PAIR ? j : j >> 1;
      for (int i = 0; i < (PAIR ? streams : 1); ++i) {
        const int s = PAIR ? i : j & 1;
        ok = wait_bar(&ctl.p_full[s][k & 1], (k >> 1) & 1, &ctl.abort);
        if (!ok) break;
        tmem_fence_after();
#pragma unroll
        for (int e = 0; e < kKeys / 16; ++e)
          mma_ts(one, tmem + 4 * kKeys + s * D, tmem + s * 2 * kKeys + (k & 1) * kKeys + e * 8,
                 vd + static_cast<uint64_t>(e * 16 * 128 >> 4), idesc_o, k > 0 || e > 0);
        mma_commit(one, &ctl.o_done[s][k & 1]);
        if (!PAIR || s == streams - 1) mma_commit(one, &ctl.empty[sv]);
        if (j + A < nt) {
          if (i == 0) sk = take();
          if (!ok) break;
          tmem_fence_after();
          scores(s, k + 2, sk);
        }
      }
    }
    if (!ok) {  // the tensor memory goes back only when no product runs
      mma_commit(one, &ctl.drain);
      const uint64_t since = global_timer_ns();
      while (!mbar_try_wait(&ctl.drain, 0) && global_timer_ns() - since < kWaitTimeoutNs) {
      }
    }
  } else if (nt > 0 && warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;  // stream, row of the query tile
    const int tok = r / G + (PAIR ? s * TQ : 0);          // token within the CTA
    const int h = g * G + r % G;
    const bool valid = r < G * TQ && tok < tokens;
    const bool active = __any_sync(0xffffffffu, valid);
    const int end = valid ? (a.causal ? L - n + tok0 + tok + 1 : L) : 0;  // visible: t < end
    const float c = a.scale * kLog2e;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + 4 * kKeys + s * D;
    const int steps = PAIR ? (s < q_tiles ? nt : 0) : (nt - s + 1) / 2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int k = 0; k < steps; ++k) {
      const int j = PAIR ? k : 2 * k + s;
      ok = wait_bar(&ctl.s_full[s][k & 1], (k >> 1) & 1, &ctl.abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tmem_fence_after();
      if (active) {
        const uint32_t ts = tmem + lanes + s * 2 * kKeys + (k & 1) * kKeys;
        uint32_t v[kKeys];
        tmem_load64(ts, v);
        const int lim = end - (t0 + j) * kKeys;
        const uint32_t bad = ctl.bad[j % kBadRing];
        if (lim < kKeys) {
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (i >= lim) v[i] = 0xff800000u;
        }
        if (bad != 0u) {
          const int sh = __ffs(a.kv.bs) - 1;
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if ((bad >> (i >> sh)) & 1u) v[i] = 0xff800000u;
        }
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
        for (int i = 0; i < kKeys; i += 2)
          mx[(i >> 1) & 7] = max3_nan(mx[(i >> 1) & 7], __uint_as_float(v[i]),
                                      __uint_as_float(v[i + 1]));
        const float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), max3_nan(mx[3], mx[4], mx[5]),
                                   max3_nan(mx[6], mx[7], -INFINITY));
        if (!(top < INFINITY)) l = NAN;  // a NaN or infinite score: so is the row's softmax
        if (k == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, (top - m) * c > kRescale)) {
          const float up = fmaxf(m, top);
          const float f = up == -INFINITY ? 1.f : fast_exp2((m - up) * c);
          m = up;
          l *= f;
          // the product of the step before has to be in O first
          ok = wait_bar(&ctl.o_done[s][(k - 1) & 1], ((k - 1) >> 1) & 1, &ctl.abort);
          tmem_fence_after();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tmem_load32(to + i, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_store32(to + i, o);
          }
        }
        const float ms = m == -INFINITY ? 0.f : m * c;
        const uint64_t cc = f32x2(c, c), mm = f32x2(-ms, -ms);
        uint64_t sum[2] = {0, 0};
        uint32_t w[kKeys / 2];
        // pair e's scale, exponential, and sum and rounding run staggered, so that the
        // exponential unit (8 cycles a warp instruction, what bounds this loop) never waits
#pragma unroll
        for (int e = 0; e < kKeys / 2 + kLag; ++e) {
          if (e < kKeys / 2) {
            float x0, x1;
            f32x2_split(fma2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), cc,
                             mm), x0, x1);
            v[2 * e] = __float_as_uint(x0);
            v[2 * e + 1] = __float_as_uint(x1);
          }
          if (e >= kLead && e - kLead < kKeys / 2) {
            exp2_in_place(v[2 * (e - kLead)]);
            exp2_in_place(v[2 * (e - kLead) + 1]);
          }
          if (e >= kLag) {
            const int d = e - kLag;
            const float p0 = __uint_as_float(v[2 * d]), p1 = __uint_as_float(v[2 * d + 1]);
            sum[d & 1] = add2(sum[d & 1], f32x2(p0, p1));
            w[d] = pack_bf16x2(p0, p1);
            if ((d & 15) == 15) tmem_store16(ts + (d & ~15), w + (d & ~15));
          }
        }
        float l0, l1;
        f32x2_split(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        tmem_wait_st();
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.p_full[s][k & 1]);
    }
    // -------------------------------------------------------- output
    // all products of a stream are in once its last one is
    if (PAIR) {
      if (steps > 0)
        ok = ok && wait_bar(&ctl.o_done[s][(steps - 1) & 1], ((steps - 1) >> 1) & 1, &ctl.abort);
    } else {
      for (int i = 0; i < min(nt, 2); ++i) {
        const int last = (nt - i + 1) / 2 - 1;
        ok = ok && wait_bar(&ctl.o_done[i][last & 1], (last >> 1) & 1, &ctl.abort);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    tmem_fence_after();
    float f0 = 1.f, f1 = 0.f;
    if (!PAIR) {  // join the streams: each half of the warps writes half of the dims
      float2 *ml = reinterpret_cast<float2 *>(tiles);  // the products have read Q
      ml[s * kQ + r] = make_float2(m, l);
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
      const float2 x0 = ml[r], x1 = ml[kQ + r];
      m = fmaxf(x0.x, x1.x);
      f0 = x0.x == -INFINITY ? 0.f : fast_exp2((x0.x - m) * c);
      f1 = x1.x == -INFINITY ? 0.f : fast_exp2((x1.x - m) * c);
      l = x0.y * f0 + x1.y * f1;
    }
    if (active && ok && (steps > 0 || !PAIR)) {
      constexpr int kCols = PAIR ? D : D / 2;
      const int col0 = PAIR ? 0 : s * kCols;
      const uint32_t o0 = tmem + lanes + 4 * kKeys + (PAIR ? s * D : 0) + col0;
      const long long at = (static_cast<long long>(s0) + tok0 + tok) * a.Hq + h;
      const int row = PAIR ? s * kQ + r : r;
      float *part = p.part + (static_cast<size_t>(slot * a.Hkv + g) * p.splits + z) *
                                 (C::kRows * (D + 2));
      const float inv = parts > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      if (valid && (PAIR || s == 0)) {
        if (parts > 1)
          reinterpret_cast<float2 *>(part)[row] = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[at] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
      }
#pragma unroll
      for (int i = 0; i < kCols; i += 32) {
        uint32_t v[32];
        tmem_load32(o0 + i, v);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(v[e]) * f0;
        if (!PAIR && nt > 1) {
          tmem_load32(o0 + D + i, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] += __uint_as_float(v[e]) * f1;
        }
        if (!valid) continue;
        if (parts > 1) {
          float4 *dst = reinterpret_cast<float4 *>(part + 2 * C::kRows + row * D + col0 + i);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * D + col0 + i);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]),
                                pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16x2(o[8 * e + 4], o[8 * e + 5]),
                                pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
        }
      }
    }
    tmem_fence_before();
  }

  if (nt > 0) {
    __syncthreads();
    if (warp == kSoftWarps) {
      tmem_fence_after();
      tmem_dealloc(tmem, 512);
    }
    if (ctl.abort != 0) {
      if (tid == 0) flag_status(a.status, KSA_FLAG_WAIT_TIMEOUT);
      return;
    }
  } else {  // the CTA's queries see nothing
    for (int e = tid; e < tokens * G * (D / 8); e += kThreads) {
      const int row = e / (D / 8);
      const long long at =
          (static_cast<long long>(s0) + tok0 + row / G) * a.Hq + g * G + row % G;
      reinterpret_cast<uint4 *>(a.out + at * D)[e % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
      if (e % (D / 8) == 0 && a.lse != nullptr) a.lse[at] = -INFINITY;
    }
    return;
  }
  if (parts == 1) return;

  // ---------------------------------------------------------- join of the parts
  uint32_t *sem = p.sem + slot * a.Hkv + g;
  if (tid == 0) {
    __threadfence();
    ctl.last = atomicAdd(sem, 1u) == static_cast<uint32_t>(parts) - 1u;
    if (ctl.last) *sem = 0u;
  }
  __syncthreads();
  if (!ctl.last) return;
  __threadfence();
  const float c = a.scale * kLog2e;
  const size_t pitch = C::kRows * (D + 2);
  const float *base = p.part + static_cast<size_t>(slot * a.Hkv + g) * p.splits * pitch;
  for (int e = tid; e < tokens * G * (D / 8); e += kThreads) {
    const int rr = e / (D / 8), d = (e % (D / 8)) * 8, tok = rr / G, hh = rr % G;
    const int row = (PAIR ? (tok / TQ) * kQ + (tok % TQ) * G : tok * G) + hh;
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int q = 0; q < parts; ++q) m = fmaxf(m, __ldcg(base + q * pitch + 2 * row));
    for (int q = 0; q < parts; ++q) {
      const float2 ml = __ldcg(reinterpret_cast<const float2 *>(base + q * pitch) + row);
      if (ml.x == -INFINITY) continue;
      const float f = fast_exp2((ml.x - m) * c);
      l += ml.y * f;
      const float4 *src =
          reinterpret_cast<const float4 *>(base + q * pitch + 2 * C::kRows + row * D + d);
      const float4 x = __ldcg(src), y = __ldcg(src + 1);
      o[0] += x.x * f;
      o[1] += x.y * f;
      o[2] += x.z * f;
      o[3] += x.w * f;
      o[4] += y.x * f;
      o[5] += y.y * f;
      o[6] += y.z * f;
      o[7] += y.w * f;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at = (static_cast<long long>(s0) + tok0 + tok) * a.Hq + g * G + hh;
    *reinterpret_cast<uint4 *>(a.out + at * D + d) =
        make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                   pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    if (d == 0 && a.lse != nullptr) a.lse[at] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
  }
}

// Two query tiles per CTA where the rows of an average sequence fill more than
// one; the keys split where the tiles leave SMs idle (a part has at least two
// key tiles).
Plan make_plan(int B, int Hq, int Hkv, int D, int T, int N, int num_sms) {
  const int G = Hq / Hkv, TQ = kQ / G;
  Plan pl;
  pl.pair = static_cast<long long>(N) * G > static_cast<long long>(kQ) * B;
  pl.tokens = pl.pair ? 2 * TQ : TQ;
  pl.slots = N / pl.tokens + B;
  const long long items = static_cast<long long>(pl.slots) * Hkv;
  long long splits = items > 0 ? num_sms / items : 1;
  const int most = (T + 4 * kKeys - 1) / (4 * kKeys);
  if (splits > most) splits = most;
  pl.splits = splits < 1 ? 1 : static_cast<int>(splits);
  return pl;
}

size_t sem_bytes(const Plan &pl, int Hkv) {
  return (static_cast<size_t>(pl.slots) * Hkv * 4 + 255) / 256 * 256;
}

template <int D, bool PAIR>
cudaError_t launch(const Params &p, const CUtensorMap *maps, cudaStream_t stream) {
  int occ = 0;
  auto kernel = chunk_attn_kernel<D, PAIR>;
  const cudaError_t err = kernel_occupancy(reinterpret_cast<const void *>(kernel), kThreads,
                                           Cfg<D, PAIR>::kSmem, &occ);
  if (err != cudaSuccess) return err;
  const dim3 grid(static_cast<unsigned>(p.slots) * p.a.Hkv * p.splits);
  kernel<<<grid, kThreads, Cfg<D, PAIR>::kSmem, stream>>>(maps[0], maps[1], maps[2], p);
  return cudaGetLastError();
}

}  // namespace

size_t chunk_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int T, int N, int num_sms) {
  const Plan pl = make_plan(B, Hq, Hkv, D, T, N, num_sms);
  const size_t rows = (pl.pair ? 2 : 1) * kQ;
  const size_t parts = pl.splits == 1 ? 0
                                      : static_cast<size_t>(pl.slots) * Hkv * pl.splits * rows *
                                            (D + 2) * 4;
  return sem_bytes(pl, Hkv) + (parts + 255) / 256 * 256;
}

cudaError_t launch_chunk_attn(const ChunkArgs &a, void *ws, int num_sms, cudaStream_t stream) {
  const Plan pl = make_plan(a.B, a.Hq, a.Hkv, a.D, a.T, a.N, num_sms);
  Params p;
  p.a = a;
  p.sem = static_cast<uint32_t *>(ws);
  p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + sem_bytes(pl, a.Hkv));
  p.tq = kQ / (a.Hq / a.Hkv);
  p.slots = pl.slots;
  p.splits = pl.splits;
  const bool paged = a.kv.table != nullptr;
  const uint64_t rows = paged ? static_cast<uint64_t>(a.kv.num_pages) * a.Hkv * a.kv.bs
                              : static_cast<uint64_t>(a.B) * a.Hkv * a.T;
  const int box = paged ? a.kv.bs : kKeys;
  CUtensorMap maps[3];
  if (!encode_q_tensor_map(&maps[0], a.q, a.D, a.Hq, a.N, a.q_stride, a.Hq / a.Hkv, p.tq) ||
      !encode_kv_tensor_map(&maps[1], a.K, rows, a.D, box) ||
      !encode_kv_tensor_map(&maps[2], a.V, rows, a.D, box))
    return cudaErrorInvalidValue;
  if (a.D == 128)
    return pl.pair ? launch<128, true>(p, maps, stream) : launch<128, false>(p, maps, stream);
  return pl.pair ? launch<64, true>(p, maps, stream) : launch<64, false>(p, maps, stream);
}

}  // namespace ksa
