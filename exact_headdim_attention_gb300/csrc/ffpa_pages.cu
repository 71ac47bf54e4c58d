// The page plan of one step: pages for the new tokens of each request, the
// slot and position of every token, cumulative and new lengths.
//
// Request b holds seq_lens[b] tokens and gets new_lens[b] more.  Its pages
// beyond those it has come off the end of the free list, in the order of the
// requests and then of their pages, so that every page number is a closed form of two
// prefix sums (tokens and pages): no block waits for another, and a
// second call with the same inputs writes the same values.  The work is a few
// integers a token; latency is the bound.
//
// A warp takes one request (and, with long prompts, a stretch of its tokens:
// grid.y); every block sums the requests before its own by itself.
#include "ffpa_paged.cuh"

namespace ffpa {
namespace {

constexpr int PLAN_WARPS = 8;
constexpr int PLAN_STRETCH = 512;    // tokens of a request that one warp writes

struct PlanParams {
  int32_t* table;
  const int32_t *seq_lens, *new_lens, *free_pages, *free_count;
  int64_t* slots;
  int32_t *positions, *cu_seqlens, *lens_out, *count_out;
  int* err;
  int64_t table_str;
  int B, max_pages, page_size, n_free, tokens;
};

struct Grow {
  unsigned old, add, before, need;   // tokens held and added, pages held and needed
  bool bad;
};

// (32-bit arithmetic: max_pages * page_size is at most 0x7fff0000.)
__device__ __forceinline__ Grow grow(const PlanParams& P, int b) {
  Grow g;
  const int o = P.seq_lens[b], a = P.new_lens[b];
  const unsigned cap = (unsigned)P.max_pages * P.page_size, page = P.page_size;
  g.old = o < 0 ? 0 : min((unsigned)o, cap);
  g.add = a < 0 ? 0 : a;
  // Tokens past the end of the request's row of the table get no page.
  const unsigned fit = min(cap - g.old, g.add);
  g.before = (g.old + page - 1) / page;
  g.need = (g.old + fit + page - 1) / page - g.before;
  g.bad = o != (int)g.old || a < 0 || fit != g.add;
  return g;
}

__global__ void __launch_bounds__(PLAN_WARPS * 32) plan_kernel(const PlanParams P) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int first = blockIdx.x * PLAN_WARPS;
  __shared__ long long sums[PLAN_WARPS][4];
  __shared__ uint4 mine[PLAN_WARPS];
  // Later stretches exist for long prompts only.
  if (blockIdx.y > 0) {
    const int b = first + lane;
    const int add = lane < PLAN_WARPS && b < P.B ? P.new_lens[b] : 0;
    if (!__any_sync(~0u, add > (int)blockIdx.y * PLAN_STRETCH)) return;
  }
  // Tokens and pages before this block's requests, and of all of them.
  long long before_t = 0, before_p = 0, all_t = 0, all_p = 0;
  bool bad = false;
  for (int b = tid; b < P.B; b += PLAN_WARPS * 32) {
    const Grow g = grow(P, b);
    bad |= g.bad;
    all_t += g.add;
    all_p += g.need;
    if (b < first) {
      before_t += g.add;
      before_p += g.need;
    } else if (b < first + PLAN_WARPS) {
      mine[b - first] = make_uint4(g.old, g.add, g.before, g.need);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before_t += __shfl_xor_sync(~0u, before_t, d);
    before_p += __shfl_xor_sync(~0u, before_p, d);
    all_t += __shfl_xor_sync(~0u, all_t, d);
    all_p += __shfl_xor_sync(~0u, all_p, d);
  }
  if (lane == 0) {
    sums[warp][0] = before_t;
    sums[warp][1] = before_p;
    sums[warp][2] = all_t;
    sums[warp][3] = all_p;
  }
  __syncthreads();
  before_t = before_p = all_t = all_p = 0;
  for (int w = 0; w < PLAN_WARPS; ++w) {
    before_t += sums[w][0];
    before_p += sums[w][1];
    all_t += sums[w][2];
    all_p += sums[w][3];
  }
  const int given = P.free_count[0];
  const int count = given < 0 ? 0 : given > P.n_free ? P.n_free : given;
  if (bad || given != count || all_p > count || all_t > P.tokens) report_invalid(P.err);
  const bool lead = blockIdx.x == 0 && blockIdx.y == 0;
  if (lead && tid == 0) {
    P.count_out[0] = all_p > count ? 0 : (int)(count - all_p);
    P.cu_seqlens[P.B] = (int)(all_t < P.tokens ? all_t : P.tokens);
  }
  // Entries behind the last token belong to none.
  if (blockIdx.y == 0)
    for (long long t = all_t + (long long)blockIdx.x * blockDim.x + tid; t < P.tokens; t += (long long)gridDim.x * blockDim.x) {
      P.slots[t] = -1;
      P.positions[t] = 0;
    }
  const int b = first + warp;
  if (b >= P.B) return;
  for (int w = 0; w < warp; ++w) {
    before_t += mine[w].y;
    before_p += mine[w].w;
  }
  const unsigned old = mine[warp].x, add = mine[warp].y, held = mine[warp].z, need = mine[warp].w;
  const unsigned page_size = P.page_size;
  // Pages of this request that the free list still has.
  const long long left = count - before_p;
  const unsigned got = left <= 0 ? 0 : left < need ? (unsigned)left : need;
  int32_t* table = P.table + b * P.table_str;
  const unsigned room = min((unsigned long long)(held + got) * page_size, ~0ull >> 32);   // tokens that have a page
  if (blockIdx.y == 0 && lane == 0) {
    P.cu_seqlens[b] = (int)(before_t < P.tokens ? before_t : P.tokens);
    P.lens_out[b] = (int)max(old, min(old + add, room));
  }
  // New page j: the free list's entry, or -1 when the list has run out.  A page
  // number is never negative, in the list and in what the table holds.
  auto fresh = [&](unsigned j) { return j - held < got ? P.free_pages[count - 1 - (before_p + (j - held))] : -1; };
  // This warp's stretch of the request's new tokens that have a row, and the pages that begin in it.
  const long long rows = P.tokens - before_t;
  const unsigned end = rows <= 0 ? 0 : rows < add ? (unsigned)rows : add, step = gridDim.y * PLAN_STRETCH;
  for (unsigned from = blockIdx.y * PLAN_STRETCH; from < end; from += step) {
    const unsigned to = min(from + PLAN_STRETCH, end);
    for (unsigned i = from + lane; i < to; i += 32) {
      const unsigned pos = old + i, j = pos / page_size, in = pos - j * page_size;
      const long long at = before_t + i;
      int page = -1;
      if (j < held)
        page = table[j];
      else if (j < held + need) {
        page = fresh(j);
        if (in == 0) table[j] = page;
      }
      if (page < 0) report_invalid(P.err);
      P.slots[at] = page < 0 ? -1 : (long long)page * page_size + in;
      P.positions[at] = (int)pos;
    }
  }
  // Pages that begin behind the last row (the call is reported): as many as the table takes,
  // however many tokens the lengths name.
  if (blockIdx.y == 0 && end < add) {
    const unsigned next = old + end, j0 = next / page_size + (next % page_size != 0);
    for (unsigned j = max(held, j0) + lane; j < held + need; j += 32) table[j] = fresh(j);
  }
}

}  // namespace
}  // namespace ffpa

extern "C" ffpa_status ffpa_page_plan(int32_t* block_table, int64_t table_str, int B, int max_pages,
                                      const int32_t* seq_lens, const int32_t* new_lens, const int32_t* free_pages,
                                      int n_free, const int32_t* free_count, int page_size, int tokens,
                                      int64_t* slots, int32_t* positions, int32_t* cu_seqlens,
                                      int32_t* seq_lens_out, int32_t* free_count_out, ffpa_stream_t stream,
                                      const ffpa_options* options) {
  using namespace ffpa;
  if (B < 1 || max_pages < 1 || n_free < 0 || page_size < 1 || tokens < 0) return FFPA_ERR_INVALID;
  if ((long long)max_pages * page_size > 0x7fff0000LL) return FFPA_ERR_INVALID;
  if (B > 1 && table_str < max_pages) return FFPA_ERR_INVALID;
  if (!block_table || !seq_lens || !new_lens || !free_count || !cu_seqlens || !seq_lens_out || !free_count_out)
    return FFPA_ERR_INVALID;
  if ((n_free > 0 && !free_pages) || (tokens > 0 && (!slots || !positions))) return FFPA_ERR_INVALID;
  for (const void* p : {(const void*)block_table, (const void*)seq_lens, (const void*)new_lens, (const void*)free_pages,
                        (const void*)free_count, (const void*)positions, (const void*)cu_seqlens,
                        (const void*)seq_lens_out, (const void*)free_count_out})
    if (!on_boundary(p, 4)) return FFPA_ERR_INVALID;
  // Blocks read the old values while others write the new ones.
  if (seq_lens_out == seq_lens || seq_lens_out == new_lens || free_count_out == free_count) return FFPA_ERR_INVALID;
  if (!on_boundary(slots, 8)) return FFPA_ERR_INVALID;
  int dev = 0;
  ffpa_status st = call_device({block_table, seq_lens, new_lens, n_free > 0 ? free_pages : nullptr, free_count,
                                tokens > 0 ? slots : nullptr, tokens > 0 ? positions : nullptr, cu_seqlens,
                                seq_lens_out, free_count_out},
                               &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  PlanParams P{};
  int sms = 0;
  if ((st = call_status(dev, options, &P.err, &sms)) != FFPA_OK) return st;
  P.table = block_table;
  P.seq_lens = seq_lens;
  P.new_lens = new_lens;
  P.free_pages = free_pages;
  P.free_count = free_count;
  P.slots = slots;
  P.positions = positions;
  P.cu_seqlens = cu_seqlens;
  P.lens_out = seq_lens_out;
  P.count_out = free_count_out;
  P.table_str = table_str;
  P.B = B;
  P.max_pages = max_pages;
  P.page_size = page_size;
  P.n_free = n_free;
  P.tokens = tokens;
  const int gx = (B + PLAN_WARPS - 1) / PLAN_WARPS;
  int gy = (tokens - 1) / PLAN_STRETCH + 1;              // a request may have all the tokens
  const int most = gx < 2048 ? 2048 / gx : 1;
  gy = gy < 1 ? 1 : gy > most ? most : gy;
  plan_kernel<<<dim3(gx, gy), PLAN_WARPS * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}
