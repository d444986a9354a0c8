// Page tables and row maps of a step from the requests' lengths (kvr_page_plan).
//
// held_b = ceil(len_b / 64), need_b = ceil((keep_b + add_b) / 64), and three
// running sums over the sequences: rows, released pages, taken pages.  With
// them every released page, taken page and row finds its place on its own (a
// binary search for its sequence), so the three lists are written in parallel
// and in a fixed order.
//
// A few hundred KB of reads and writes at most: bound by latency, not by
// bytes.  One cluster of 8 CTAs, each of which forms the sums itself (a few
// integers per sequence from L2) rather than waiting for another CTA's; a
// single CTA where there is little to write.  The sums come before any change,
// so that a plan that cannot be carried out changes nothing.  8 sequences: 4.7 us
// a plan in a graph, 512 of up to 8192 tokens, an eighth of them new: 7.8 us; the
// host's side of a call takes as long.
#include <cooperative_groups.h>

#include "kvr_pages.cuh"

namespace cg = cooperative_groups;

namespace kvr {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = kPageMaxSeqs / kThreads;
constexpr int kCluster = 8;
// rows up to which one CTA does it all
constexpr int kOneCta = 1024;

struct Sums {
  int rows, rel, take;
};
__device__ __forceinline__ Sums add(Sums a, Sums b) { return {a.rows + b.rows, a.rel + b.rel, a.take + b.take}; }
__device__ __forceinline__ Sums shfl_up(Sums a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.rows, d), __shfl_up_sync(0xffffffffu, a.rel, d),
          __shfl_up_sync(0xffffffffu, a.take, d)};
}

// last b in [0, n) with off[b] <= x (off non-decreasing, off[0] = 0)
__device__ __forceinline__ int owner(const int* off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1)
page_plan_kernel(const PagesDev p, int n, const int32_t* keep, const int32_t* add_rows, int rows, int max_add) {
  // per sequence: first row, first released and first taken page, kept tokens,
  // pages held and needed
  extern __shared__ int sm[];
  int* s_cu = sm;
  int* s_rel = s_cu + n;
  int* s_take = s_rel + n;
  int* s_keep = s_take + n;
  int* s_held = s_keep + n;
  int* s_need = s_held + n;
  __shared__ Sums warp_sum[kWarps];
  __shared__ int bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int gtid = (int)blockIdx.x * kThreads + tid, gthreads = (int)gridDim.x * kThreads;
  dev::pdl_trigger();
  if (tid == 0) bad = 0;
  __syncthreads();
  dev::pdl_wait();

  const int free_count = *p.count;
  // sums of this thread's consecutive sequences, each value checked first (a
  // bad one counts as nothing; max_add <= rows <= 2^22, so that 32 threads'
  // rows stay below 2^31 and the total is formed in 64 bits)
  const int per = (n + kThreads - 1) / kThreads;
  Sums mine = {0, 0, 0};
  int keep_r[kPerThread], add_r[kPerThread], held_r[kPerThread], need_r[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    keep_r[k] = add_r[k] = held_r[k] = need_r[k] = 0;
    if (k >= per || b >= n) continue;
    const int kp = keep[b], ad = add_rows[b], len = p.lens[b];
    const bool ok = kp >= 0 && kp <= len && ad >= 0 && ad <= max_add && (long long)kp + ad <= p.max_len;
    if (!ok) bad = 1;
    keep_r[k] = ok ? kp : 0;
    add_r[k] = ok ? ad : 0;
    held_r[k] = (len + kPage - 1) / kPage;
    need_r[k] = (keep_r[k] + add_r[k] + kPage - 1) / kPage;
    mine.rows += add_r[k];
    mine.rel += max(0, held_r[k] - need_r[k]);
    mine.take += max(0, need_r[k] - held_r[k]);
  }
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(inc, d);
    if (lane >= d) inc = add(inc, o);
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Sums before = {0, 0, 0}, total = {0, 0, 0};
  long long all_rows = 0;
#pragma unroll 8
  for (int w = 0; w < kWarps; ++w) {
    const Sums s = warp_sum[w];
    if (w < warp) before = add(before, s);
    total = add(total, s);
    all_rows += s.rows;
  }
  const bool invalid = bad != 0 || all_rows > rows;
  const bool full = !invalid && total.take > free_count + total.rel;
  // every CTA of the cluster takes the same decision from the same values;
  // nothing is written before all of them have read theirs
  if (invalid || full) {
    cluster.sync();
    for (int r = gtid; r < rows; r += gthreads) p.row_seq[r] = p.row_pos[r] = p.row_slot[r] = -1;
    for (int b = gtid; b <= n; b += gthreads) p.cu[b] = 0;
    if (gtid == 0) {
      p.info[0] = n;
      p.info[1] = 0;
      if (*p.refused == 0) *p.refused = full ? KVR_ERR_CAPACITY : KVR_ERR_ARG;
    }
    return;
  }
  Sums at = add(before, {inc.rows - mine.rows, inc.rel - mine.rel, inc.take - mine.take});
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= n) continue;
    s_cu[b] = at.rows;
    s_rel[b] = at.rel;
    s_take[b] = at.take;
    s_keep[b] = keep_r[k];
    s_held[b] = held_r[k];
    s_need[b] = need_r[k];
    at.rows += add_r[k];
    at.rel += max(0, held_r[k] - need_r[k]);
    at.take += max(0, need_r[k] - held_r[k]);
  }
  cluster.sync();   // every CTA has read the lengths and the count
  if (blockIdx.x == gridDim.x - 1) {
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int b = tid * per + k;
      if (k >= per || b >= n) continue;
      p.lens[b] = keep_r[k] + add_r[k];
      p.cu[b] = s_cu[b];
    }
    if (tid == 0) {
      p.cu[n] = total.rows;
      p.info[0] = n;
      p.info[1] = total.rows;
      *p.count = free_count + total.rel - total.take;
    }
  }
  const int top = free_count + total.rel;
  for (int r = gtid; r < total.rel; r += gthreads) {
    const int b = owner(s_rel, n, r);
    int32_t* e = p.table + (long long)b * p.width + s_need[b] + (r - s_rel[b]);
    p.free_list[top - 1 - r] = *e;
    *e = -1;
  }
  if (total.rel > 0) cluster.sync();
  for (int t = gtid; t < total.take; t += gthreads) {
    const int b = owner(s_take, n, t);
    p.table[(long long)b * p.width + s_held[b] + (t - s_take[b])] = __ldcg(p.free_list + (top - 1 - t));
  }
  if (total.take > 0) cluster.sync();
  for (int r = gtid; r < rows; r += gthreads) {
    int seq = -1, pos = -1, slot = -1;
    if (r < total.rows) {
      seq = owner(s_cu, n, r);
      pos = s_keep[seq] + r - s_cu[seq];
      slot = __ldcg(p.table + (long long)seq * p.width + pos / kPage) * kPage + pos % kPage;
    }
    p.row_seq[r] = seq;
    p.row_pos[r] = pos;
    p.row_slot[r] = slot;
  }
}

__global__ void page_init_kernel(PagesDev p) {
  const int i = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  if (i < p.n_pages) p.free_list[i] = p.n_pages - 1 - i;
  if (i == 0) *p.count = p.n_pages;
}

// cos and sin of pos * theta^(-2j/d), in double, rounded once to float, and the
// rest of each (at most 2^-25) times 2^24
__global__ void page_rope_kernel(RopeFreq fr, int max_len, int half, float2* table, __half2* rest) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)max_len * half) return;
  double s, c;
  sincos((double)(i / half) * fr.inv[i % half], &s, &c);
  const float2 v = make_float2((float)c, (float)s);
  table[i] = v;
  rest[i] = __floats2half2_rn((float)((c - v.x) * 16777216.0), (float)((s - v.y) * 16777216.0));
}

}  // namespace

cudaError_t page_plan_setup() {
  return cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              6 * kPageMaxSeqs * (int)sizeof(int));
}

cudaError_t launch_page_init(const PagesDev& p, cudaStream_t st) {
  page_init_kernel<<<(p.n_pages + 255) / 256, 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_page_rope(const RopeFreq& fr, int max_len, int d, float2* table, __half2* rest, cudaStream_t st) {
  const long long n = (long long)max_len * (d / 2);
  page_rope_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(fr, max_len, d / 2, table, rest);
  return cudaGetLastError();
}

cudaError_t launch_page_plan(const PagesDev& p, int n_seq, const int32_t* keep, const int32_t* add, int rows,
                             int max_add, cudaStream_t st) {
  const int ctas = rows <= kOneCta ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)6 * n_seq * sizeof(int);
  cfg.stream = st;
  // (a launch of one CTA is a cluster of one without being told so)
  cudaLaunchAttribute attr[2];
  int n_attr = 0;
  if (pdl_enabled()) {
    attr[n_attr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n_attr++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (ctas > 1) {
    attr[n_attr].id = cudaLaunchAttributeClusterDimension;
    attr[n_attr].val.clusterDim.x = ctas;
    attr[n_attr].val.clusterDim.y = attr[n_attr].val.clusterDim.z = 1;
    ++n_attr;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n_attr;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, p, n_seq, keep, add, rows, max_add);
}

}  // namespace kvr
