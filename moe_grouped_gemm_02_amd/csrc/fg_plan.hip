// fg_plan.hip -- the sort of a batch's (token, choice) slots by expert into the
// row layouts of the grouped GEMMs: a stable counting sort, so that equal
// experts keep their tokens' order and the result never depends on timing.
//
//   contiguous  row = offsets[g] + rank, offsets[g + 1] = offsets[g] + count_g
//               rounded up to `align` rows
//   masked      row = g * M_max + rank for rank < M_max, else the slot has none
//
// with rank the number of earlier slots of the same expert. Slots whose id is
// outside [0, G) have no row.
//
// Ranks come from wave-wide matching: one ballot per bit of the id gives each
// lane the mask of lanes with its id; the lanes below it in that mask are its
// rank inside the batch of 64, and the lowest of them adds the batch's count to
// the wave's histogram in LDS. Each wave owns consecutive slots, so scanning
// the waves' histograms in order makes the ranks of a workgroup's chunk.
//
// What a workgroup needs of the others is counts alone: of each expert's slots
// before its chunk and in the whole batch. Up to kRecount slots every workgroup
// counts the batch itself (whole-number LDS atomics, a few microseconds at most),
// which saves a launch; beyond, a first launch leaves each chunk's histogram in the
// workspace, and where those are many (kSumEntries) a second one makes their prefixes.
// One or two launches are bound by latency: 131072 slots are 2 MB of ids, rows, slots
// and experts, under a microsecond of traffic. In a graph, G 64, contiguous, the one
// launch takes 5.2 / 5.8 / 7.0 / 9.5 us at 2048 / 8192 / 16384 / 32768 slots, two
// launches 8.6 / 9.0 / 9.5 / 9.6 us; at 131072 it is 24.9 against 10.4 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"

namespace {

using namespace fg;

constexpr int kThreads = 512, kPlanWaves = kThreads / 64;
constexpr int kMaxGroups = 1024;
constexpr int kRecount = 32768;    // slots up to which every workgroup counts them all
constexpr int kBatches = 4;        // batches of 64 slots per wave beyond that
constexpr int kChunk = kThreads * kBatches;
// Histogram entries (experts x chunks) up to which every placing workgroup sums all of
// them, work that grows with the square of the slots; beyond, a launch of its own leaves
// each chunk's prefix and the totals. Summed / with that launch, in a graph, us: 256
// experts, 65536 slots (8192 entries) 12.8 / 13.5, 131072 14.7 / 14.1, 1048576 111 / 25,
// 4194304 1400 / 81; 1024 experts, 40960 (20480) 17.3 / 16.3, 4194304 5535 / 139; 64
// experts, 131072 (4096) 10.4 / 12.1, 262144 (8192) 13.4 / 13.0, 4194304 370 / 56.
constexpr long kSumEntries = 8192;
constexpr int kFillRows = 1024;    // rows of the layout per workgroup, where that needs more of them

struct PlanArgs {
  const int32_t* ids;
  int32_t *rows, *slots, *m_indices, *offsets, *masked_m;
  const int32_t* hist;   // [G][chunks_up4], null: count here
  const int32_t* total;  // [G], hist holds prefixes; null: counts
  int S, G, align, M_max, cap, bits, chunks, chunks_up4;
};

// Inclusive sum over the workgroup's threads in thread order.
__device__ __forceinline__ int block_scan(int v, int* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  if (lane == 63) part[wave] = v;
  __syncthreads();
  for (int i = 0; i < wave; ++i) v += part[i];
  __syncthreads();
  return v;
}

__global__ __launch_bounds__(kThreads) void plan_count(const int32_t* __restrict__ ids, int32_t* __restrict__ hist,
                                                       int S, int G, int chunks_up4) {
  __shared__ int n[kMaxGroups];
  for (int g = threadIdx.x; g < G; g += kThreads) n[g] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * kChunk;
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) {
    const int s = s0 + i * kThreads + threadIdx.x;
    const int id = s < S ? ids[s] : -1;
    if (id >= 0 && id < G) atomicAdd(&n[id], 1);   // whole numbers: any order gives the same count
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += kThreads) hist[(long)g * chunks_up4 + blockIdx.x] = n[g];
}

// Each expert's counts become the sums of the chunks before, and their total: a wave
// per expert, 256 chunks at a time.
__global__ __launch_bounds__(256) void plan_prefix(int32_t* __restrict__ hist, int32_t* __restrict__ total, int G,
                                                   int chunks, int chunks_up4) {
  const int lane = threadIdx.x & 63, g = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (g >= G) return;
  int carry = 0;
  for (int c0 = 0; c0 < chunks; c0 += 256) {
    const int c = c0 + 4 * lane;
    int4* at = (int4*)(hist + (long)g * chunks_up4 + (c < chunks_up4 ? c : 0));
    const int4 n = *at;
    const int n0 = c < chunks ? n.x : 0, n1 = c + 1 < chunks ? n.y : 0, n2 = c + 2 < chunks ? n.z : 0,
              n3 = c + 3 < chunks ? n.w : 0, sum = n0 + n1 + n2 + n3;
    int end = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(end, d, 64);
      if (lane >= d) end += u;
    }
    const int before = carry + end - sum;
    if (c < chunks_up4) *at = make_int4(before, before + n0, before + n0 + n1, before + n0 + n1 + n2);
    carry += __shfl(end, 63, 64);
  }
  if (lane == 0) total[g] = carry;
}

// NB: batches of 64 slots per wave.
template <int NB>
__global__ __launch_bounds__(kThreads) void plan_place(PlanArgs p) {
  extern __shared__ int lds[];
  const int G = p.G, GS = G + 1;               // bin G: slots without an expert here
  int* hist = lds;                             // [kPlanWaves][GS]
  int* total = hist + kPlanWaves * GS;         // [G] slots of each expert in the whole batch
  int* base = total + G;                       // [G] of those, in earlier chunks
  int* start = base + G;                       // [G + 1] first row of each expert
  int* part = start + GS;                      // [kPlanWaves]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kPlanWaves * GS; i += kThreads) hist[i] = 0;
  for (int i = tid; i < 2 * G; i += kThreads) total[i] = 0;   // total and base
  __syncthreads();

  const int s0 = (blockIdx.x * kPlanWaves + wave) * (64 * NB);
  int id[NB], rank[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int s = s0 + b * 64 + lane;
    const int v = s < p.S ? p.ids[s] : -1;
    id[b] = v >= 0 && v < G ? v : G;
  }
  volatile int* mine = hist + wave * GS;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    unsigned long long same = ~0ull;
    for (int i = 0; i < p.bits; ++i) {
      const bool one = (id[b] >> i) & 1;
      const unsigned long long v = __ballot(one);
      same &= one ? v : ~v;
    }
    const int below = __popcll(same & ((1ull << lane) - 1ull));
    rank[b] = mine[id[b]] + below;
    // every lane of the wave has read the bins before the lowest ones add to them
    __builtin_amdgcn_wave_barrier();
    if (below == 0) mine[id[b]] = rank[b] + __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  // total and base, in whole numbers (any order of additions gives the same)
  if (p.total) {
    for (int g = tid; g < G; g += kThreads) {
      total[g] = p.total[g];
      // workgroups past the last chunk have no slots
      base[g] = (int)blockIdx.x < p.chunks ? p.hist[(long)g * p.chunks_up4 + blockIdx.x] : 0;
    }
  } else if (p.hist) {
    // threads take (expert, four chunks) pairs
    const int quads = p.chunks_up4 / 4;
    for (int i = tid; i < G * quads; i += kThreads) {
      const int g = i / quads, c = 4 * (i - g * quads);
      const int4 n = *(const int4*)(p.hist + (long)g * p.chunks_up4 + c);
      const int v[4] = {n.x, n.y, n.z, n.w};
      int before = 0, all = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = c + u < p.chunks ? v[u] : 0;
        all += k;
        before += c + u < (int)blockIdx.x ? k : 0;
      }
      if (all) atomicAdd(&total[g], all);
      if (before) atomicAdd(&base[g], before);
    }
  } else if (gridDim.x > 1) {
    const int first = (int)blockIdx.x * (kThreads * NB);
    for (int s1 = 0; s1 < p.S; s1 += 8 * kThreads) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s1 + u * kThreads + tid;
        v[u] = p.ids[s < p.S ? s : p.S - 1];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s1 + u * kThreads + tid;
        if (s < p.S && v[u] >= 0 && v[u] < G) atomicAdd(s < first ? &base[v[u]] : &total[v[u]], 1);
      }
    }
    __syncthreads();
    for (int g = tid; g < G; g += kThreads) total[g] += base[g];
  }
  __syncthreads();
  // each wave's first rank inside the chunk; one workgroup: the chunk is the batch
  for (int g = tid; g < G; g += kThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w * GS + g];
      hist[w * GS + g] = n;
      n += c;
    }
    if (gridDim.x == 1) total[g] = n;
  }
  __syncthreads();
  // first rows of the experts
  const bool masked = p.M_max > 0;
  int carry = 0;
  for (int g0 = 0; g0 < G; g0 += kThreads) {
    const int g = g0 + tid;
    const int n = g < G ? total[g] : 0;
    const int padded = masked ? (g < G ? p.M_max : 0) : (n + p.align - 1) / p.align * p.align;
    const int end = block_scan(padded, part) + carry;
    if (g < G) start[g + 1] = end;
    if (tid == kThreads - 1) part[0] = end;
    __syncthreads();
    carry = part[0];
    __syncthreads();
  }
  if (tid == 0) start[0] = 0;
  __syncthreads();

#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int s = s0 + b * 64 + lane;
    if (s < p.S) {
      int row = -1;
      const int g = id[b];
      if (g < G) {
        const int r = base[g] + hist[wave * GS + g] + rank[b];
        if (!masked || r < p.M_max) {
          row = start[g] + r;
          p.slots[row] = s;
          if (!masked) p.m_indices[row] = g;
        }
      }
      p.rows[s] = row;
    }
  }
  // rows without a slot: behind each expert's last one, a wave per expert, and behind
  // the last expert, all waves
  const int nw = gridDim.x * kPlanWaves, me = blockIdx.x * kPlanWaves + wave;
  for (int g = me; g < G; g += nw) {
    const int n = total[g], to = start[g + 1];
    for (int r = start[g] + (masked && n > p.M_max ? p.M_max : n) + lane; r < to; r += 64) {
      p.slots[r] = -1;
      if (!masked) p.m_indices[r] = -1;
    }
  }
  for (long r = (long)start[G] + 64L * me + lane; r < p.cap; r += 64L * nw) {
    p.slots[r] = -1;
    if (!masked) p.m_indices[r] = -1;
  }
  if (blockIdx.x == 0) {
    for (int g = tid; g <= G; g += kThreads) {
      if (!masked) p.offsets[g] = start[g];
      else if (g < G) p.masked_m[g] = total[g] < p.M_max ? total[g] : p.M_max;
    }
  }
}

bool sizes_ok(int T, int k, int G) {
  return T >= 0 && k >= 1 && G >= 1 && G <= kMaxGroups && (long long)T * k <= 0x7fffffffLL - kChunk;
}

long long capacity(int T, int k, int G, int align) {
  const long long S = (long long)T * k, used = S < G ? S : G;
  return (S + used * (align - 1) + align - 1) / align * align;
}

int chunks_of(int S) { return (int)(((long long)S + kChunk - 1) / kChunk); }
int up4(int n) { return (n + 3) / 4 * 4; }

int plan(PlanArgs p, void* ws, hipStream_t stream) {
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  p.bits = 32 - __builtin_clz((unsigned)p.G);   // ids 0 .. G
  const size_t lds = sizeof(int) * ((size_t)(kPlanWaves + 1) * (p.G + 1) + 2 * p.G + kPlanWaves);
  // enough workgroups for the slots, and for the rows without one
  const int fill = p.cap / kFillRows < 256 ? p.cap / kFillRows : 256;
  if (p.S > kRecount) {
    if (!ws || !aligned(ws, 16)) return FG_EINVAL;
    int32_t* hist = static_cast<int32_t*>(ws);
    p.chunks = chunks_of(p.S);
    p.chunks_up4 = up4(p.chunks);
    hipLaunchKernelGGL(plan_count, dim3(p.chunks), dim3(kThreads), 0, stream, p.ids, hist, p.S, p.G, p.chunks_up4);
    if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
    p.hist = hist;
    if ((long)p.G * p.chunks > kSumEntries) {
      int32_t* total = hist + (long)p.G * p.chunks_up4;
      hipLaunchKernelGGL(plan_prefix, dim3((p.G + 3) / 4), dim3(256), 0, stream, hist, total, p.G, p.chunks, p.chunks_up4);
      if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
      p.total = total;
    }
    const int grid = fill > p.chunks ? fill : p.chunks;
    hipLaunchKernelGGL((plan_place<kBatches>), dim3(grid), dim3(kThreads), lds, stream, p);
  } else {
    const int chunks = (p.S + kThreads - 1) / kThreads, most = fill > chunks ? fill : chunks;
    hipLaunchKernelGGL((plan_place<1>), dim3(most > 1 ? most : 1), dim3(kThreads), lds, stream, p);
  }
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}

}  // namespace

extern "C" {

int fg_plan_capacity(int T, int k, int G, int align, int* rows) {
  if (!sizes_ok(T, k, G) || align < 1 || align > 65536 || !rows) return FG_EINVAL;
  const long long cap = capacity(T, k, G, align);
  if (cap > 0x7fffffffLL) return FG_EINVAL;
  *rows = (int)cap;
  return FG_OK;
}

int fg_plan_workspace(int T, int k, int G, size_t* bytes) {
  if (!sizes_ok(T, k, G) || !bytes) return FG_EINVAL;
  const int S = T * k;
  *bytes = S <= kRecount ? 0 : ((size_t)up4(chunks_of(S)) + 1) * G * sizeof(int32_t);
  return FG_OK;
}

int fg_plan_contiguous(const int32_t* ids, int32_t* rows, int32_t* slots, int32_t* m_indices, int32_t* offsets,
                       void* ws, int T, int k, int G, int align, hipStream_t stream) {
  int cap = 0;
  const int rc = fg_plan_capacity(T, k, G, align, &cap);
  if (rc != FG_OK) return rc;
  if (!offsets || !aligned(offsets, 4)) return FG_EINVAL;
  if (T > 0 && (!ids || !rows || !slots || !m_indices)) return FG_EINVAL;
  if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(m_indices, 4)) return FG_EINVAL;
  PlanArgs p = {};
  p.ids = ids;
  p.rows = rows;
  p.slots = slots;
  p.m_indices = m_indices;
  p.offsets = offsets;
  p.S = T * k;
  p.G = G;
  p.align = align;
  p.cap = cap;
  return plan(p, ws, stream);
}

int fg_plan_masked(const int32_t* ids, int32_t* rows, int32_t* slots, int32_t* masked_m, void* ws, int T, int k,
                   int G, int M_max, hipStream_t stream) {
  if (!sizes_ok(T, k, G) || M_max < 1 || (long long)G * M_max > 0x7fffffffLL) return FG_EINVAL;
  if (!slots || !masked_m || (T > 0 && (!ids || !rows))) return FG_EINVAL;
  if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(masked_m, 4)) return FG_EINVAL;
  PlanArgs p = {};
  p.ids = ids;
  p.rows = rows;
  p.slots = slots;
  p.masked_m = masked_m;
  p.S = T * k;
  p.G = G;
  p.align = 1;
  p.M_max = M_max;
  p.cap = G * M_max;
  return plan(p, ws, stream);
}

}  // extern "C"
