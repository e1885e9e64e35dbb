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
// 4096, redundantly: a scan costs less than handing its result
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

struct Sum3 {
  int64_t f, p, t;  // pages given back, pages taken, tokens
};
__device__ __forceinline__ Sum3 warp_scan(Sum3 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t f = __shfl_up_sync(0xFFFFFFFFu, v.f, o), p = __shfl_up_sync(0xFFFFFFFFu, v.p, o),
                  t = __shfl_up_sync(0xFFFFFFFFu, v.t, o);
    if (lane >= o) {
      v.f += f;
      v.p += p;
      v.t += t;
    }
  }
  return v;
}

// Inclusive block-wide sums (the warps' totals are summed by every warp for
// itself); returns the block's total too.
__device__ __forceinline__ Sum3 block_scan(Sum3 v, Sum3* total, Sum3* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_scan(v, lane);
  if (lane == 31) red[warp] = v;
  __syncthreads();
  const Sum3 w = warp_scan(lane < nw ? red[lane] : Sum3{0, 0, 0}, lane);
  const int before = warp > 0 ? warp - 1 : 0;
  const int64_t f = __shfl_sync(0xFFFFFFFFu, w.f, before), p = __shfl_sync(0xFFFFFFFFu, w.p, before),
                t = __shfl_sync(0xFFFFFFFFu, w.t, before);
  if (warp > 0) {
    v.f += f;
    v.p += p;
    v.t += t;
  }
  total->f = __shfl_sync(0xFFFFFFFFu, w.f, 31);
  total->p = __shfl_sync(0xFFFFFFFFu, w.p, 31);
  total->t = __shfl_sync(0xFFFFFFFFu, w.t, 31);
  return v;
}

// Blocks that v positions fill (v up to 2^32 - 2).
__device__ __forceinline__ uint32_t blocks_of(uint32_t v, uint32_t page_size) {
  const uint32_t q = v / page_size;
  return q + (v - q * page_size != 0);
}

// RPT: consecutive requests a thread has; kDeep: consecutive tokens.
template <int RPT, int kDeep>
__global__ void __launch_bounds__(1024) mla_tables_kernel(const TableArgs t) {
  extern __shared__ int32_t tab_smem[];
  __shared__ Sum3 red[32];
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

  // ---- this thread's requests
  const int r0 = tid * RPT;
  int32_t len[RPT], have[RPT], take[RPT], toks[RPT];
  bool released[RPT];
  bool refused = false;
  Sum3 sum{0, 0, 0};
  int32_t count = *t.free_count;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    len[i] = have[i] = take[i] = toks[i] = 0;
    released[i] = false;
    const int r = r0 + i;
    if (r < R) {
      const int32_t ln = t.lens[r], nw = t.new_tokens[r];
      len[i] = ln;
      const uint32_t held = blocks_of((uint32_t)max(ln, 0), (uint32_t)t.page_size);
      if (ln >= 0 && held <= t.bt_stride) {
        have[i] = (int32_t)held;
        if (nw < 0) {
          released[i] = true;
          sum.f += held;
        } else if (nw > 0) {
          const uint32_t after = (uint32_t)ln + (uint32_t)nw;
          const uint32_t need = blocks_of(after, (uint32_t)t.page_size);
          if (need <= t.bt_stride && after <= 0x7FFFFFFFu) {
            take[i] = (int32_t)(need - held);
            toks[i] = nw;
          } else {
            refused = true;  // its row of the block table cannot hold it
          }
        }
      } else {
        refused = true;
      }
    }
    sum.p += take[i];
    sum.t += toks[i];
  }
  Sum3 all;
  const Sum3 in = block_scan(sum, &all, red);
  if (count < 0 || count > t.num_pages) {
    count = 0;
    refused = true;
  }
  // stack places that the array cannot hold are left out (more pages given
  // back than exist)
  const int64_t tot_f = all.f;
  const int64_t avail = min(count + tot_f, t.num_pages);
  if (count + tot_f > t.num_pages) refused = true;

  // ---- who fits; the first that does not
  const int64_t ex_f = in.f - sum.f, ex_p = in.p - sum.p, ex_t = in.t - sum.t;
  {
    int64_t p = ex_p, k = ex_t;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
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
    for (int i = 0; i < RPT; ++i) {
      const int r = r0 + i;
      if (r < R) {
        const bool in_step = toks[i] > 0 && r < stop;
        s.len[r] = len[i];
        s.have[r] = have[i];
        // (a place that 32 bits do not hold lies behind the stack's end)
        s.give[r] = !released[i] ? kGiveNone : have[i] > 0 ? (int32_t)min(f, (int64_t)0x7FFFFFFF) : kGiveNothing;
        s.take[r] = in_step ? take[i] : 0;
        s.first[r] = (int32_t)min(p, (int64_t)0x7FFFFFFF);
        k += toks[i];
        s.cu[r] = (int32_t)min(k, (int64_t)0x7FFFFFFF);  // from `stop` on: the admitted total, below
        if (released[i]) f += have[i];
        p += take[i];
      }
    }
  }
  __syncthreads();
  // admitted totals: the inclusive sums of the last request before `stop`
  const int32_t all_tokens = stop > 0 ? s.cu[stop - 1] : 0;
  int64_t taken = 0;
  if (stop > 0) taken = (int64_t)s.first[stop - 1] + s.take[stop - 1];
  if (stop < R) {
    __syncthreads();
    for (int r = stop + tid; r < R; r += nt) s.cu[r] = all_tokens;
  }

  // ---- released pages onto the stack, a warp a request
  const int lane = tid & 31;
  const int gw = rank * (nt >> 5) + (tid >> 5), warps = ctas * (nt >> 5);
  if (tot_f > 0)
    for (int r = gw; r < R; r += warps)
      if (s.give[r] >= 0)
        for (int j = lane; j < s.have[r]; j += 32) {
          const int64_t at = (int64_t)count + s.give[r] + j;
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

  // ---- the tokens, padded behind the last, kDeep side by side a thread: one
  // bisection, one division unless the request changes, and with four whole
  // 16-byte stores where the arrays allow them
  const bool vec = kDeep == 4 && ((reinterpret_cast<uintptr_t>(t.slot_mapping) | reinterpret_cast<uintptr_t>(t.token_row) |
                     reinterpret_cast<uintptr_t>(t.token_len)) & 15u) == 0;
  for (int64_t k0 = kDeep * ((int64_t)rank * nt + tid); k0 < t.max_tokens; k0 += kDeep * (int64_t)ctas * nt) {
    int32_t row[kDeep], pos[kDeep], off[kDeep], page[kDeep];
    int lo = 0, j = 0;
    if (k0 < all_tokens) {
      int hi = R - 1;  // the first request whose inclusive offset passes k0
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.cu[mid] > k0)
          hi = mid;
        else
          lo = mid + 1;
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t k = k0 + d;
      row[d] = pos[d] = page[d] = -1;
      off[d] = 0;
      if (k < all_tokens) {
        const int was = lo;
        while (s.cu[lo] <= k) ++lo;
        row[d] = lo;
        if (d == 0 || lo != was) {
          pos[d] = s.len[lo] + (int32_t)(k - (lo > 0 ? s.cu[lo - 1] : 0));
          j = pos[d] / t.page_size;
          off[d] = pos[d] - j * t.page_size;
        } else {
          pos[d] = pos[d - 1] + 1;
          off[d] = off[d - 1] + 1;
          if (off[d] == t.page_size) {
            off[d] = 0;
            ++j;
          }
        }
        const int32_t* from = j >= s.have[lo]
                                  ? t.free_pages + (avail - 1 - s.first[lo] - (j - s.have[lo]))
                                  : t.block_table + (int64_t)lo * t.bt_stride + j;
        page[d] = *from;
      }
    }
    int64_t slot[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      slot[d] = -1;
      if (row[d] >= 0) {
        if (page[d] >= 0 && page[d] < t.num_pages)
          slot[d] = page[d] * ps + off[d];
        else if (t.flags != nullptr)
          atomicOr(t.flags, MLA_DEVERR_BAD_SLOT);
      }
    }
    bool stored = false;
    const bool whole = vec && k0 + kDeep <= t.max_tokens;
    if constexpr (kDeep == 4) {
      if (whole) {
        longlong2* at = reinterpret_cast<longlong2*>(t.slot_mapping + k0);
        at[0] = make_longlong2(slot[0], slot[1]);
        at[1] = make_longlong2(slot[2], slot[3]);
        *reinterpret_cast<int4*>(t.token_row + k0) = make_int4(row[0], row[1], row[2], row[3]);
        *reinterpret_cast<int4*>(t.token_len + k0) = make_int4(pos[0] + 1, pos[1] + 1, pos[2] + 1, pos[3] + 1);
      }
    }
    if (!whole) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        if (k0 + d >= t.max_tokens) break;
        t.slot_mapping[k0 + d] = slot[d];
        t.token_row[k0 + d] = row[d];
        t.token_len[k0 + d] = pos[d] + 1;
      }
    }
  }
}

}  // namespace

cudaError_t launch_tables(const TableArgs& t, cudaStream_t stream) {
  // One CTA of 256 threads serves a decode step; a step with many requests or
  // tokens takes a cluster of eight CTAs of 1024 threads.
  const bool large = t.rows > 256 || t.max_tokens > 2048;
  // Four tokens a thread where there are more than one for each (256 requests,
  // 32,768 token places: 8.8 us with one at a time, now 7.3); a decode step's
  // few go to a thread each (64 requests: 4.2 us, by fours 5.3).
  auto kernel = t.rows > 1024       ? mla_tables_kernel<4, 4>
                : t.max_tokens > 256 ? mla_tables_kernel<1, 4>
                                     : mla_tables_kernel<1, 1>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(large ? kTabCluster : 1, 1, 1);
  cfg.blockDim = dim3(large ? 1024 : 256, 1, 1);
  cfg.dynamicSmemBytes = 6 * (size_t)t.rows * sizeof(int32_t);
  if (cfg.dynamicSmemBytes > 40 * 1024) {  // beyond the default limit, on the device in use
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  return cudaLaunchKernelEx(&cfg, kernel, t);
}

}  // namespace mla
