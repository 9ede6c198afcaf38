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
// the waves' histograms in order makes the ranks of a whole chunk; no atomics.
//
// A batch of at most kOneBlock slots is sorted by one workgroup in one launch.
// A larger one is cut into chunks: a first launch writes each chunk's
// histogram to the workspace, a second one lets every chunk sum the histograms
// before its own (its base) and all of them (the segments), and place its slots.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"

namespace {

using namespace fg;

constexpr int kThreads = 512, kPlanWaves = kThreads / 64;
constexpr int kMaxGroups = 1024;
constexpr int kOneBlock = 4096;    // slots one workgroup sorts alone
constexpr int kChunk = 2048;       // slots per workgroup otherwise

struct PlanArgs {
  const int32_t* ids;
  int32_t *rows, *slots, *m_indices, *offsets, *masked_m;
  const int32_t* hist;   // [chunks][G], null: a single workgroup
  int S, G, align, M_max, cap, bits;
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
                                                       int S, int G) {
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
  for (int g = threadIdx.x; g < G; g += kThreads) hist[(long)blockIdx.x * G + g] = n[g];
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
  if (p.hist) {
    // threads take (expert, every parts-th chunk) pairs; whole-number sums
    const int chunks = gridDim.x;
    const int parts = kThreads / G > 1 ? kThreads / G : 1;
    for (int i = tid; i < parts * G; i += kThreads) {
      const int g = i % G;
      int before = 0, all = 0;
      for (int c0 = i / G; c0 < chunks; c0 += 8 * parts) {
        int n[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int c = c0 + u * parts;
          n[u] = c < chunks ? p.hist[(long)c * G + g] : 0;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          all += n[u];
          before += c0 + u * parts < (int)blockIdx.x ? n[u] : 0;
        }
      }
      atomicAdd(&total[g], all);
      atomicAdd(&base[g], before);
    }
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
    if (!p.hist) total[g] = n;
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
  // rows without a slot: behind each expert's last one, and behind the last expert
  const int nw = gridDim.x * kPlanWaves;
  for (int g = blockIdx.x * kPlanWaves + wave; g <= G; g += nw) {
    int from = start[g], to = p.cap;
    if (g < G) {
      const int n = total[g];
      from += masked && n > p.M_max ? p.M_max : n;
      to = start[g + 1];
    }
    for (int r = from + lane; r < to; r += 64) {
      p.slots[r] = -1;
      if (!masked) p.m_indices[r] = -1;
    }
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

int plan(PlanArgs p, void* ws, hipStream_t stream) {
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  p.bits = 32 - __builtin_clz((unsigned)p.G);   // ids 0 .. G
  const int chunks = p.S <= kOneBlock ? 1 : chunks_of(p.S);
  const size_t lds = sizeof(int) * ((size_t)(kPlanWaves + 1) * (p.G + 1) + 2 * p.G + kPlanWaves);
  if (chunks > 1) {
    if (!ws || !aligned(ws, 4)) return FG_EINVAL;
    int32_t* hist = static_cast<int32_t*>(ws);
    hipLaunchKernelGGL(plan_count, dim3(chunks), dim3(kThreads), 0, stream, p.ids, hist, p.S, p.G);
    if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
    p.hist = hist;
    hipLaunchKernelGGL((plan_place<kChunk / kThreads>), dim3(chunks), dim3(kThreads), lds, stream, p);
  } else {
    p.hist = nullptr;
    if (p.S <= kThreads) hipLaunchKernelGGL((plan_place<1>), dim3(1), dim3(kThreads), lds, stream, p);
    else if (p.S <= 4 * kThreads) hipLaunchKernelGGL((plan_place<4>), dim3(1), dim3(kThreads), lds, stream, p);
    else hipLaunchKernelGGL((plan_place<kOneBlock / kThreads>), dim3(1), dim3(kThreads), lds, stream, p);
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
  *bytes = S <= kOneBlock ? 0 : (size_t)chunks_of(S) * G * sizeof(int32_t);
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
