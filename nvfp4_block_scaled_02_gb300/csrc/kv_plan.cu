// kv_plan.cu -- block tables and slot maps of a paged cache from request
// lengths, in one launch.
//
// Two prefix sums over the requests (new tokens, new pages) fix everything:
// token t belongs to the request whose token range holds it, page j of the
// ones taken to the request whose page range holds it. Every CTA runs both
// scans over all requests by itself (1024 at a time, 8 bytes each, out of L2)
// instead of waiting for another CTA or a second launch, and fills in the
// blocks of 1024 tokens and pages that fall to it, looking the owner up by
// bisection in the scans' shared-memory copy. A new token in a new page takes
// the page from the free list directly, so no CTA reads a table entry that
// another one writes.
//
// Bound by latency (a few KB to a few MB move): 5.0 us for 64 requests with one new
// token each, 7.8 us for 1500 requests (two passes of 1024) and 2.7 MB of results.
#include "kv.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Largest i in [0, kThreads) with start[i] <= x.
__device__ __forceinline__ int owner(const int64_t* start, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (start[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const KvPlanParams p) {
  pdl_begin();
  __shared__ int64_t s_tok[kThreads], s_page[kThreads];  // exclusive prefix sums
  __shared__ int32_t s_len[kThreads];
  __shared__ int64_t w_tok[kWarps], w_page[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t tok0 = 0, page0 = 0;  // tokens and pages of the requests before this chunk

  for (int64_t c0 = 0; c0 < p.B; c0 += kThreads) {
    const int64_t b = c0 + tid;
    int32_t c = 0, n = 0;
    if (b < p.B) {
      c = p.cached[b];
      n = p.fresh[b];
    }
    bool bad = c < 0 || n < 0;
    c = max(c, 0);
    n = max(n, 0);
    if ((int64_t)c + n > INT32_MAX) bad = true, n = 0;
    const int32_t held = (int32_t)fastdiv((uint32_t)c + p.P - 1, p.by_page);
    int32_t total = (int32_t)fastdiv((uint32_t)c + (uint32_t)n + p.P - 1, p.by_page);
    if (total > p.cols) bad = true, total = p.cols;
    const int32_t need = max(total - held, 0);
    if (bad && blockIdx.x == 0) flag(p.status, kDevBadIndex);

    int64_t it = warp_scan(n, lane), ip = warp_scan(need, lane);
    if (lane == 31) {
      w_tok[warp] = it;
      w_page[warp] = ip;
    }
    __syncthreads();
    if (warp == 0) {
      const int64_t a = w_tok[lane], e = w_page[lane];
      w_tok[lane] = warp_scan(a, lane);
      w_page[lane] = warp_scan(e, lane);
    }
    __syncthreads();
    if (warp > 0) {
      it += w_tok[warp - 1];
      ip += w_page[warp - 1];
    }
    const int64_t tok1 = tok0 + w_tok[kWarps - 1], page1 = page0 + w_page[kWarps - 1];
    s_tok[tid] = tok0 + it - n;
    s_page[tid] = page0 + ip - need;
    s_len[tid] = c;
    __syncthreads();
    if (b < p.B && (c0 / kThreads) % gridDim.x == blockIdx.x) {
      p.q_start[b] = (int32_t)min(tok0 + it - n, (int64_t)p.T);
      p.seq_len[b] = c + n;
    }

    // tokens of this chunk's requests, in this CTA's blocks of 1024
    const int64_t tend = min(tok1, (int64_t)p.T);
    if (tok0 < tend) {
      int64_t tb = tok0 / kThreads;
      tb += (blockIdx.x + gridDim.x - tb % gridDim.x) % gridDim.x;
      for (; tb * kThreads < tend; tb += gridDim.x) {
        const int64_t t = tb * kThreads + tid;
        if (t < tok0 || t >= tend) continue;
        const int i = owner(s_tok, t);
        const int32_t cl = s_len[i], pos = cl + (int32_t)(t - s_tok[i]);
        const int32_t hp = (int32_t)fastdiv((uint32_t)cl + p.P - 1, p.by_page);
        const int32_t pg = (int32_t)fastdiv((uint32_t)pos, p.by_page);
        int64_t page = -1;
        if (pg < p.cols) {
          if (pg < hp) {
            page = p.table[(c0 + i) * p.cols + pg];
          } else {
            const int64_t j = s_page[i] + pg - hp;
            if (j < p.n_free) page = p.free_pages[j];
          }
        }
        p.positions[t] = pos;
        p.slots[t] = page < 0 ? -1 : page * p.P + (pos - pg * p.P);
      }
    }
    // table entries of the pages taken
    if (page0 < page1) {
      int64_t pb = page0 / kThreads;
      pb += (blockIdx.x + gridDim.x - pb % gridDim.x) % gridDim.x;
      for (; pb * kThreads < page1; pb += gridDim.x) {
        const int64_t j = pb * kThreads + tid;
        if (j < page0 || j >= page1) continue;
        const int i = owner(s_page, j);
        const int32_t hp = (int32_t)fastdiv((uint32_t)s_len[i] + p.P - 1, p.by_page);
        p.table[(c0 + i) * p.cols + hp + (j - s_page[i])] = j < p.n_free ? p.free_pages[j] : -1;
      }
    }
    tok0 = tok1;
    page0 = page1;
    __syncthreads();  // the scans' copies are rewritten by the next chunk
  }

  // rows past the last new token
  int64_t tb = tok0 / kThreads;
  tb += (blockIdx.x + gridDim.x - tb % gridDim.x) % gridDim.x;
  for (; tb * kThreads < p.T; tb += gridDim.x) {
    const int64_t t = tb * kThreads + tid;
    if (t < tok0 || t >= p.T) continue;
    p.positions[t] = 0;
    p.slots[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.q_start[p.B] = (int32_t)min(tok0, (int64_t)p.T);
    p.used[0] = (int32_t)min(page0, (int64_t)p.n_free);
    if (tok0 > p.T) flag(p.status, kDevBadIndex);
    if (page0 > p.n_free) flag(p.status, kDevNoPages);
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t st) {
  // enough CTAs for the tokens' and requests' blocks; pages are fewer than tokens
  const int64_t want = ((int64_t)p.T + p.B) / kThreads + 1;
  return launch_pdl(kv_plan_kernel, dim3((unsigned)std::min<int64_t>(want, sm_count())),
                    dim3(kThreads), st, p);
}

}  // namespace nvfp4
