// pages.cu -- block tables and token slots of a paged cache from request lengths.
//
// Assignment.  Row b needs need_b = ceil(L_b / bs) - ceil(c_b / bs) pages and
// has n_b new tokens; with the exclusive prefix sums first_b of the needs and
// cu_b of the tokens, everything else is local: token t of row b sits at
// position c_b + t - cu_b, in block j = position / bs, and
//   page(j) = table[b][j]                              j <  ceil(c_b / bs)
//           = free_pages[F - 1 - (first_b + j - ceil(c_b / bs))]   otherwise.
// So no CTA waits for another: each scans the rows' lengths itself (they are a
// few KB out of L2), 1024 rows at a time in shared memory, and expands its own
// token places by binary search over the prefix sums.  A new block's first
// token is always a new token, so the thread that has it writes the block's
// table entry.  Release is the same with the released blocks as the places.
//
// The lengths and the stack's count may be carried in place, so they are
// written by the CTA that is the last to have read them (a counter in the
// workspace, which it sets back to zero).
//
// Bound by latency: three dependent loads (lengths, page, then the store).  256
// rows of one token take 3.9 us, 64 rows of 139000 tokens 6.1 us; with 500 rows
// of 625000 tokens the scans in 611 CTAs count, 11.0 us (11.3 with half as many
// CTAs of twice the places), and the release of their 39000 pages takes 5.6.
#include "ksa_device.cuh"
#include "ksa_internal.h"

namespace ksa {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;
constexpr int kChunk = kThreads * kRowsPerThread;  // rows scanned together
constexpr int kTokens = 1024;                      // token places per CTA
constexpr int kPages = 512;                        // released pages per CTA and turn

struct Chunk {           // one chunk of rows, in shared memory
  int place[kChunk + 1];  // first place of each row: cu_b, or pages released before it
  int first[kChunk];      // pages taken by the rows before; -1: the row is refused
  int ctx[kChunk];        // c_b
  int len[kChunk];        // the row's seq_lens after the call
};

// Blocks of 2^sh tokens that n tokens fill or begin (block sizes are 16, 32 and 64).
__device__ __forceinline__ int blocks_of(int n, int sh) { return (n + (1 << sh) - 1) >> sh; }

// Exclusive prefix sums over the block of two values per thread, and the totals.
__device__ __forceinline__ void block_scan2(int &a, int &b, int &ta, int &tb, int2 *scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, off), v = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) scratch[warp] = make_int2(x, y);
  __syncthreads();
  int ba = 0, bb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 s = scratch[w];
    if (w < warp) {
      ba += s.x;
      bb += s.y;
    }
    ta += s.x;
    tb += s.y;
  }
  a = ba + x - a;
  b = bb + y - b;
  __syncthreads();
}

// Last chunk row whose first place is <= t (rows with no place are passed over,
// since the next row starts at the same place).
__device__ __forceinline__ int find_row(const Chunk &c, int rows, int t) {
  int lo = 0, hi = rows;  // place[lo] <= t < place[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.place[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// True in every thread of the last CTA to arrive (which resets the counter).
__device__ __forceinline__ bool last_cta(uint32_t *counter, int *flag) {
  if (gridDim.x == 1) return true;
  __syncthreads();  // all of this CTA's reads are done
  if (threadIdx.x == 0) {
    __threadfence();
    *flag = atomicAdd(counter, 1u) == gridDim.x - 1u;
    if (*flag) {
      *counter = 0u;
      __threadfence();
    }
  }
  __syncthreads();
  return *flag != 0;
}

// Scans rows [base, base + kChunk) into `c`; `tokens` and `pages` carry the
// sums over the chunks before and are advanced.  Returns the rows in the chunk.
__device__ __forceinline__ int scan_assign(const AssignArgs &a, int base, int F, Chunk &c,
                                           int2 *scratch, int &tokens, int &pages,
                                           bool report) {
  const int rows = min(kChunk, a.B - base), sh = __ffs(a.bs) - 1;
  int n[kRowsPerThread], need[kRowsPerThread], ctx[kRowsPerThread];
  bool bad[kRowsPerThread];
  int sn = 0, sp = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int r = threadIdx.x * kRowsPerThread + i;
    n[i] = need[i] = ctx[i] = 0;
    bad[i] = false;
    if (r < rows) {
      const int c0 = a.ctx_lens[base + r], n0 = a.new_lens[base + r];
      ctx[i] = min(max(c0, 0), a.T);
      n[i] = min(max(n0, 0), a.T);
      bad[i] = ctx[i] != c0 || n[i] != n0 || n[i] > a.T - ctx[i];
      if (!bad[i]) need[i] = blocks_of(ctx[i] + n[i], sh) - blocks_of(ctx[i], sh);
    }
    sn += n[i];
  }
  // token places first: a row past num_tokens is refused and needs no page
  int en = sn, dummy = 0, tn, td;
  block_scan2(en, dummy, tn, td, scratch);
  en += tokens;
  int place[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    place[i] = en;
    en += n[i];
    if (en > a.N && n[i] > 0) {
      bad[i] = true;
      need[i] = 0;
    }
    sp += need[i];
  }
  int ep = sp, tp;
  dummy = 0;
  block_scan2(ep, dummy, tp, td, scratch);
  ep += pages;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int r = threadIdx.x * kRowsPerThread + i;
    const bool none = need[i] > F - ep && need[i] > 0;
    if (r < rows) {
      c.place[r] = place[i];
      c.first[r] = (bad[i] || none) ? -1 : ep;
      c.ctx[r] = ctx[i];
      c.len[r] = (bad[i] || none) ? ctx[i] : ctx[i] + n[i];
      if (report && bad[i]) flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
      if (report && none) flag_status(a.status, KSA_FLAG_NO_PAGE);
    }
    ep += need[i];
  }
  tokens += tn;
  pages += tp;
  if (threadIdx.x == 0) c.place[rows] = tokens;
  __syncthreads();
  return rows;
}

__global__ void __launch_bounds__(kThreads) assign_pages_kernel(const AssignArgs a) {
  __shared__ Chunk c;
  __shared__ int2 scratch[kThreads / 32];
  __shared__ int flag;
  pdl_wait();
  pdl_launch_dependents();
  const bool reporter = blockIdx.x == 0;
  const int sh = __ffs(a.bs) - 1;
  const int F0 = *a.num_free, F = min(max(F0, 0), a.num_pages);
  if (reporter && threadIdx.x == 0 && F != F0) flag_status(a.status, KSA_FLAG_NO_PAGE);
  const int t0 = blockIdx.x * kTokens, t1 = min(t0 + kTokens, a.N);
  int tokens = 0, pages = 0, rows = 0, base = 0;
  for (; base < a.B; base += kChunk) {
    const int before = tokens;
    // CTA 0 reads every row (it reports, and writes cu_new); others stop at their last place
    if (!reporter && before >= t1) break;
    rows = scan_assign(a, base, F, c, scratch, tokens, pages, reporter);
    if (reporter) {
      for (int r = threadIdx.x; r < rows; r += kThreads) a.cu_new[base + r] = min(c.place[r], a.N);
      if (threadIdx.x == 0 && base + kChunk >= a.B) a.cu_new[a.B] = min(tokens, a.N);
    }
    // a thread's places together: their pages' loads are in flight at once
    const int lo = max(t0, before) + threadIdx.x, hi = min(t1, tokens);
    int pos[kTokens / kThreads], page[kTokens / kThreads], *fresh[kTokens / kThreads];
#pragma unroll
    for (int i = 0; i < kTokens / kThreads; ++i) {
      const int t = lo + i * kThreads;
      pos[i] = page[i] = -1;
      fresh[i] = nullptr;
      if (t >= hi) continue;
      const int r = find_row(c, rows, t);
      if (c.first[r] < 0) continue;
      const int held = blocks_of(c.ctx[r], sh);
      pos[i] = c.ctx[r] + (t - c.place[r]);
      const int j = pos[i] >> sh;
      int *entry = a.block_table + static_cast<size_t>(base + r) * a.max_blocks + j;
      page[i] = j < held ? *entry : a.free_pages[F - 1 - (c.first[r] + j - held)];
      if (j >= held && (pos[i] & (a.bs - 1)) == 0) fresh[i] = entry;  // the new block's first token
    }
#pragma unroll
    for (int i = 0; i < kTokens / kThreads; ++i) {
      const int t = lo + i * kThreads;
      if (t >= hi) continue;
      if (pos[i] >= 0 && (page[i] < 0 || page[i] >= a.num_pages)) {
        flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
        page[i] = -1;
      }
      if (fresh[i] != nullptr) *fresh[i] = page[i];
      a.slots[t] =
          page[i] < 0 ? -1LL : (static_cast<long long>(page[i]) << sh) + (pos[i] & (a.bs - 1));
      a.positions[t] = pos[i];
    }
    if (base + kChunk < a.B) __syncthreads();  // the chunk is read before the next one fills it
  }
  if (base >= a.B) {  // every row seen: what lies behind them is padding
    for (int t = max(t0, tokens) + threadIdx.x; t < t1; t += kThreads) {
      a.slots[t] = -1;
      a.positions[t] = -1;
    }
  }
  if (!last_cta(a.counter, &flag)) return;
  // this CTA may have stopped early, and a chunk at a time is held: scan again where needed
  int taken = 0;
  const bool held = base >= a.B && a.B <= kChunk;
  tokens = pages = 0;
  for (base = 0; base < a.B; base += kChunk) {
    __syncthreads();
    if (!held) rows = scan_assign(a, base, F, c, scratch, tokens, pages, false);
    for (int r = threadIdx.x; r < rows; r += kThreads) {
      const int len = c.len[r];
      a.seq_lens[base + r] = len;
      taken += blocks_of(len, sh) - blocks_of(c.ctx[r], sh);
    }
  }
  int zero = 0, total, tz;
  block_scan2(taken, zero, total, tz, scratch);
  if (threadIdx.x == 0) *a.num_free_out = F - total;
}

// Scans rows [base, base + kChunk): the blocks each released row gives back.
__device__ __forceinline__ int scan_release(const ReleaseArgs &a, int base, Chunk &c,
                                            int2 *scratch, int &blocks, bool report) {
  const int rows = min(kChunk, a.B - base), sh = __ffs(a.bs) - 1;
  int n[kRowsPerThread], sn = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int r = threadIdx.x * kRowsPerThread + i;
    n[i] = 0;
    if (r < rows && a.done[base + r] != 0) {
      const int L = a.seq_lens[base + r], Lc = min(max(L, 0), a.T);
      if (report && L != Lc) flag_status(a.status, KSA_FLAG_SEQ_LEN_CLAMPED);
      n[i] = blocks_of(Lc, sh);
    }
    sn += n[i];
  }
  int en = sn, zero = 0, tn, tz;
  block_scan2(en, zero, tn, tz, scratch);
  en += blocks;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int r = threadIdx.x * kRowsPerThread + i;
    if (r < rows) c.place[r] = en;
    en += n[i];
  }
  blocks += tn;
  if (threadIdx.x == 0) c.place[rows] = blocks;
  __syncthreads();
  return rows;
}

__global__ void __launch_bounds__(kThreads) release_pages_kernel(const ReleaseArgs a) {
  __shared__ Chunk c;
  __shared__ int2 scratch[kThreads / 32];
  __shared__ int flag;
  pdl_wait();
  pdl_launch_dependents();
  const bool reporter = blockIdx.x == 0;
  const int F0 = *a.num_free, F = min(max(F0, 0), a.num_pages);
  if (reporter && threadIdx.x == 0 && F != F0) flag_status(a.status, KSA_FLAG_NO_PAGE);
  // the stack's order needs the total before any page moves
  int total = 0, rows = 0;
  for (int base = 0; base < a.B; base += kChunk) {
    if (base > 0) __syncthreads();
    rows = scan_release(a, base, c, scratch, total, reporter);
  }
  if (reporter && threadIdx.x == 0 && total > a.num_pages - F)
    flag_status(a.status, KSA_FLAG_NO_PAGE);
  int blocks = 0;
  for (int base = 0; base < a.B; base += kChunk) {
    const int before = blocks;
    if (a.B > kChunk) {
      __syncthreads();
      rows = scan_release(a, base, c, scratch, blocks, false);
    } else {
      blocks = total;
    }
    // places are shared out CTA by CTA: e = blockIdx.x * kPages + ..., then a grid further
    for (long long e0 = static_cast<long long>(blockIdx.x) * kPages; e0 < blocks;
         e0 += static_cast<long long>(gridDim.x) * kPages) {
      const int end = static_cast<int>(min(e0 + kPages, static_cast<long long>(blocks)));
      const int lo = max(static_cast<int>(e0), before) + threadIdx.x;
      int *entry[kPages / kThreads], page[kPages / kThreads];
#pragma unroll
      for (int i = 0; i < kPages / kThreads; ++i) {
        const int e = lo + i * kThreads;
        entry[i] = nullptr;
        if (e >= end) continue;
        const int r = find_row(c, rows, e);
        entry[i] = a.block_table + static_cast<size_t>(base + r) * a.max_blocks + (e - c.place[r]);
        page[i] = *entry[i];
      }
#pragma unroll
      for (int i = 0; i < kPages / kThreads; ++i) {
        if (entry[i] == nullptr) continue;
        *entry[i] = -1;
        if (page[i] < 0 || page[i] >= a.num_pages) {
          flag_status(a.status, KSA_FLAG_INDEX_SKIPPED);
          page[i] = -1;
        }
        const int above = total - 1 - (lo + i * kThreads);  // the top; F + above may pass 2^31
        if (above < a.num_pages - F) a.free_pages[F + above] = page[i];
      }
    }
  }
  if (!last_cta(a.counter, &flag)) return;
  for (int b = threadIdx.x; b < a.B; b += kThreads)
    if (a.done[b] != 0) a.seq_lens[b] = 0;
  if (threadIdx.x == 0) *a.num_free = F + min(total, a.num_pages - F);
}

}  // namespace

cudaError_t launch_assign_pages(const AssignArgs &a, cudaStream_t stream) {
  const int ctas = a.N > kTokens ? (a.N + kTokens - 1) / kTokens : 1;
  return launch_pdl(assign_pages_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0,
                    stream, a);
}

cudaError_t launch_release_pages(const ReleaseArgs &a, int num_sms, cudaStream_t stream) {
  const long long most = static_cast<long long>(a.B) * a.max_blocks;  // blocks released at most
  long long ctas = (most + kPages - 1) / kPages;
  if (ctas > 2LL * num_sms) ctas = 2LL * num_sms;
  return launch_pdl(release_pages_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0,
                    stream, a);
}

}  // namespace ksa
