// mla_tables.cu - block tables, slot map and causal lengths of one step, built
// on the GPU from the requests' lengths (mla_tables_step).
//
// The mathematics are three prefix sums over the requests in row order: pages
// given back, pages taken, tokens appended.  With have_r = ceil(len_r / page)
// and need_r = ceil((len_r + new_r) / page), request r's pages are the
// need_r - have_r entries below the top of the free stack that start at the
// exclusive sum of its predecessors' counts, and its tokens start at cu_r.
// A request fits while the inclusive sums stay within the pages at hand and
// the token capacity; both sums only grow, so from the first that does not
// fit on, none does, and no second pass is needed.
//
// What bounds it is latency: a decode step moves a few KiB.  So it is one
// launch of one thread-block cluster: every CTA scans all requests (at most
// 4096, four a thread, redundantly: a scan costs less than handing its result
// over), pushes its share of the released pages, and after the one cluster
// barrier pops pages and writes its share of the outputs.  The barrier is also
// what lets lens_out and free_count_out alias their inputs: every CTA has read
// them by then.  A token finds its request by bisecting the token offsets in
// shared memory.
#include "../../include/mla_query.h"
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kTabRowsPerThread = 4;
constexpr int kTabCluster = 8;  // CTAs of a large step (portable cluster size)

constexpr int kGiveNone = -1, kGiveNothing = -2;

struct TabSmem {  // per request; sized by rows
  int32_t* cu;     // inclusive token offsets of the admitted requests
  int32_t* have;   // pages held before the step
  int32_t* give;   // first stack place of the released pages above free_count;
                   // kGiveNone: not released, kGiveNothing: released, held no page
  int32_t* take;   // pages taken
  int32_t* first;  // pages taken by the requests before
  int32_t* len;    // length before
};

// Inclusive block-wide sums of two 64-bit values; returns this thread's
// inclusive prefix in a, b and the totals in ta, tb.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb,
                                            int64_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, a, o), y = __shfl_up_sync(0xFFFFFFFFu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    red[warp] = a;
    red[32 + warp] = b;
  }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = 0;
  tb = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) {
      pa = ta;
      pb = tb;
    }
    ta += red[w];
    tb += red[32 + w];
  }
  a += pa;
  b += pb;
}

__global__ void __launch_bounds__(1024) mla_tables_kernel(const TableArgs t) {
  extern __shared__ int32_t tab_smem[];
  __shared__ int64_t red[64];
  __shared__ int fail_row;
  const int R = t.rows;
  const TabSmem s{tab_smem, tab_smem + R, tab_smem + 2 * R, tab_smem + 3 * R, tab_smem + 4 * R,
                  tab_smem + 5 * R};
  const int tid = threadIdx.x, nt = blockDim.x;
  const int rank = blockIdx.x, ctas = gridDim.x;
  const int64_t ps = t.page_size;
  if (tid == 0) fail_row = R;
  pdl_launch_dependents();
  pdl_wait();

  // ---- this thread's requests 4 tid .. 4 tid + 3
  const int r0 = tid * kTabRowsPerThread;
  int64_t have[kTabRowsPerThread], freed[kTabRowsPerThread], take[kTabRowsPerThread],
      toks[kTabRowsPerThread];
  bool released[kTabRowsPerThread];
  bool refused = false;
  int64_t sum_f = 0, sum_p = 0, sum_t = 0, unused = 0;
#pragma unroll
  for (int i = 0; i < kTabRowsPerThread; ++i) {
    have[i] = freed[i] = take[i] = toks[i] = 0;
    released[i] = false;
    const int r = r0 + i;
    if (r < R) {
      const int64_t len = t.lens[r], nw = t.new_tokens[r];
      const bool sound = len >= 0 && (len + ps - 1) / ps <= t.bt_stride;
      if (sound) {
        have[i] = (len + ps - 1) / ps;
        if (nw < 0) {
          freed[i] = have[i];
          released[i] = true;
        } else if (nw > 0) {
          const int64_t need = (len + nw + ps - 1) / ps;
          if (need <= t.bt_stride && len + nw <= 0x7FFFFFFF) {
            take[i] = need - have[i];
            toks[i] = nw;
          } else {
            refused = true;  // its row of the block table cannot hold it
          }
        }
      } else {
        refused = true;
      }
    }
    sum_f += freed[i];
    sum_p += take[i];
    sum_t += toks[i];
  }
  int64_t in_f = sum_f, in_p = sum_p, in_t = sum_t, tot_f, tot_p, tot_t, zero;
  block_scan2(in_p, in_t, tot_p, tot_t, red);
  block_scan2(in_f, unused, tot_f, zero, red);
  int64_t count = *t.free_count;
  if (count < 0 || count > t.num_pages) {
    count = 0;
    refused = true;
  }
  // stack places that the array cannot hold are left out (more pages given
  // back than exist)
  const int64_t avail = min(count + tot_f, t.num_pages);
  if (count + tot_f > t.num_pages) refused = true;

  // ---- who fits; the first that does not
  int64_t ex_f = in_f - sum_f, ex_p = in_p - sum_p, ex_t = in_t - sum_t;
  {
    int64_t p = ex_p, k = ex_t;
#pragma unroll
    for (int i = 0; i < kTabRowsPerThread; ++i) {
      p += take[i];
      k += toks[i];
      if (toks[i] > 0 && (p > avail || k > t.max_tokens)) {
        atomicMin(&fail_row, r0 + i);
        break;
      }
    }
  }
  __syncthreads();
  const int stop = fail_row;
  if (stop < R && tid == 0) refused = true;
  {
    int64_t f = ex_f, p = ex_p, k = ex_t;
#pragma unroll
    for (int i = 0; i < kTabRowsPerThread; ++i) {
      const int r = r0 + i;
      if (r < R) {
        const bool in = toks[i] > 0 && r < stop;
        s.len[r] = t.lens[r];
        s.have[r] = (int32_t)have[i];
        s.give[r] = !released[i] ? kGiveNone : freed[i] > 0 ? (int32_t)f : kGiveNothing;
        s.take[r] = in ? (int32_t)take[i] : 0;
        s.first[r] = (int32_t)min(p, (int64_t)0x7FFFFFFF);
        k += toks[i];
        s.cu[r] = r < stop ? (int32_t)k : -1;  // -1: the admitted total, below
        f += freed[i];
        p += take[i];
      }
    }
  }
  __syncthreads();
  // admitted totals: the inclusive sums of the last request before `stop`
  const int32_t all_tokens = stop > 0 ? s.cu[stop - 1] : 0;
  int64_t taken = 0;
  if (stop > 0) taken = (int64_t)s.first[stop - 1] + s.take[stop - 1];
  __syncthreads();
  for (int r = tid; r < R; r += nt)
    if (r >= stop) s.cu[r] = all_tokens;

  // ---- released pages onto the stack, a warp a request
  const int lane = tid & 31;
  const int gw = rank * (nt >> 5) + (tid >> 5), warps = ctas * (nt >> 5);
  if (tot_f > 0)
    for (int r = gw; r < R; r += warps)
      if (s.give[r] >= 0)
        for (int j = lane; j < s.have[r]; j += 32) {
          const int64_t at = count + s.give[r] + j;
          if (at < t.num_pages) t.free_pages[at] = t.block_table[(int64_t)r * t.bt_stride + j];
        }
  if (refused && rank == 0 && t.flags != nullptr) atomicOr(t.flags, MLA_DEVERR_REFUSED);
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();

  // ---- pages taken, lengths, offsets
  for (int r = gw; r < R; r += warps) {
    const int n = s.take[r];
    for (int j = lane; j < n; j += 32)
      t.block_table[(int64_t)r * t.bt_stride + s.have[r] + j] =
          t.free_pages[avail - 1 - s.first[r] - j];
  }
  for (int r = rank * nt + tid; r < R; r += ctas * nt) {
    const int32_t before = r > 0 ? s.cu[r - 1] : 0;
    t.lens_out[r] = s.give[r] != kGiveNone ? 0 : s.len[r] + (s.cu[r] - before);
    t.cu_tokens[r + 1] = s.cu[r];
  }
  if (rank == 0 && tid == 0) {
    t.cu_tokens[0] = 0;
    *t.free_count_out = (int32_t)(avail - taken);
  }

  // ---- the tokens, padded behind the last
  for (int64_t k = (int64_t)rank * nt + tid; k < t.max_tokens; k += (int64_t)ctas * nt) {
    int64_t slot = -1;
    int32_t row = -1, len = 0;
    if (k < all_tokens) {
      int lo = 0, hi = R - 1;  // the first request whose inclusive offset passes k
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.cu[mid] > k)
          hi = mid;
        else
          lo = mid + 1;
      }
      row = lo;
      const int32_t pos = s.len[row] + (int32_t)(k - (row > 0 ? s.cu[row - 1] : 0));
      const int32_t j = pos / t.page_size;
      const int64_t page =
          j >= s.have[row] ? t.free_pages[avail - 1 - s.first[row] - (j - s.have[row])]
                           : t.block_table[(int64_t)row * t.bt_stride + j];
      if (page >= 0 && page < t.num_pages)
        slot = page * ps + pos % t.page_size;
      else if (t.flags != nullptr)
        atomicOr(t.flags, MLA_DEVERR_BAD_SLOT);
      len = pos + 1;
    }
    t.slot_mapping[k] = slot;
    t.token_row[k] = row;
    t.token_len[k] = len;
  }
}

}  // namespace

cudaError_t launch_tables(const TableArgs& t, cudaStream_t stream) {
  // One CTA of 256 threads serves a decode step; a step with many requests or
  // tokens takes a cluster of eight CTAs of 1024.
  const bool large = t.rows > 512 || t.max_tokens > 2048;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(large ? kTabCluster : 1, 1, 1);
  cfg.blockDim = dim3(large ? 1024 : 256, 1, 1);
  cfg.dynamicSmemBytes = 6 * (size_t)t.rows * sizeof(int32_t);
  if (cfg.dynamicSmemBytes > 40 * 1024) {  // beyond the default limit, on the device in use
    const cudaError_t e =
        cudaFuncSetAttribute(mla_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             6 * MLA_MAX_TABLE_ROWS * (int)sizeof(int32_t));
    if (e != cudaSuccess) return e;
  }
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = large ? kTabCluster : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mla_tables_kernel, t);
}

}  // namespace mla
