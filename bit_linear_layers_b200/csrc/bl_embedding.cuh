// Embedding lookup with a scale, and the gradient of the table.
//
//   y_t = scale * E[id_t]              dE_v = scale * sum_{t: id_t = v} dy_t
//
// The gradient adds rows of dy that share a token. Adding them with atomics
// would make the order, and so the rounding, of frequent tokens' sums differ
// from run to run; here the tokens are first sorted by id (stable: the rows of
// a token are added in the order of their positions), then the sorted list is
// cut into chunks of 32 positions and one warp per (chunk, 256 columns) adds
// up the segments that start in its chunk. A segment that ends in the next
// chunk is finished by the warp that began it (at most 63 rows); a longer one
// is summed chunk by chunk into fp32 partial rows that a last kernel adds up
// in order, so a token that fills the batch is as parallel as any other. Rows
// of the table that no token names are zero-filled by the same launch as the
// sums: each element of dE is written once.
#pragma once

#include "bl_elem.cuh"

namespace bl {

// an id in [0, V) as a row index, or -1 (recorded) where it is outside
template <typename TI>
__device__ __forceinline__ int64_t embed_row(const TI* ids, int64_t t, int64_t V) {
  const int64_t id = static_cast<int64_t>(ids[t]);
  return id >= 0 && id < V ? id : -1;
}

constexpr int kEmbThreads = 256;

// One CTA per token (grid-stride); a token outside the table gets a row of zeros.
template <typename TI, typename TT, typename TY, int E>
__global__ void __launch_bounds__(kEmbThreads)
    embedding_kernel(const TI* __restrict__ ids, const TT* __restrict__ table, TY* __restrict__ y, int64_t T,
                     int64_t V, int64_t D, float scale) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int64_t row = embed_row(ids, t, V);
    if (row < 0 && threadIdx.x == 0) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingId);
    for (int64_t k = static_cast<int64_t>(threadIdx.x) * E; k < D; k += kEmbThreads * E) {
      float f[E];
      if (row >= 0) {
        Elem<TT, E>::load(table + row * D + k, f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] *= scale;
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = 0.f;
      }
      Elem<TY, E>::store(y + t * D + k, f);
    }
  }
}

// ---------------------------------------------------------------------------
// The sort: one cluster of 8 CTAs, a stable radix sort of (id, position) by
// digits of up to 8 bits, ping-pong through the workspace (it stays in L2).
// CTA r of the cluster owns the r-th eighth of the positions and each of its
// warps a contiguous run of that, so that counting in order gives stability.
// Tokens that take no part (padding, ids outside the table) get the key V,
// sort behind all others and are skipped.
constexpr int kEsCluster = 8;
constexpr int kEsThreads = 1024;
constexpr int kEsWarps = kEsThreads / 32;
constexpr int kEsBins = 256;
constexpr int kEgChunk = 32;  // sorted positions per warp of the sums

struct EmbedHeavy {
  uint32_t first, last;  // the chunks in which a long segment starts and ends
};

struct EmbedSort {
  uint32_t* key[2];
  uint32_t* val[2];
  uint32_t* touched;    // bit v: some token names row v
  uint32_t* num_heavy;
  EmbedHeavy* heavy;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::
          : "memory");
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t smem_addr, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <typename TI>
__global__ void __cluster_dims__(kEsCluster, 1, 1) __launch_bounds__(kEsThreads)
    embed_sort_kernel(const TI* __restrict__ ids, uint32_t T, uint32_t V, int64_t padding_id, int passes, int digit_bits,
                      EmbedSort p) {
  __shared__ uint32_t hist[kEsWarps][kEsBins];  // counts, then next output positions
  __shared__ uint32_t tot[kEsBins];             // this CTA's counts, read by the cluster
  __shared__ uint32_t wsum[kEsBins / 32];
  const uint32_t rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t gtid = rank * kEsThreads + tid;
  constexpr uint32_t kAll = kEsCluster * kEsThreads;
  // whole warps of positions: a warp's run, then a CTA's
  const uint32_t run = ((T + kAll - 1) / kAll) * 32;
  const uint32_t w0 = min(T, (rank * kEsWarps + warp) * run), w1 = min(T, w0 + run);
  for (uint32_t i = gtid; i < (V + 31) / 32; i += kAll) p.touched[i] = 0u;
  if (gtid == 0) *p.num_heavy = 0u;
  const uint32_t mask = (1u << digit_bits) - 1u;

  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * digit_bits;
    const uint32_t* kin = p.key[(pass + 1) & 1];
    const uint32_t* vin = p.val[(pass + 1) & 1];
    uint32_t* kout = p.key[pass & 1];
    uint32_t* vout = p.val[pass & 1];
    auto key_at = [&](uint32_t i) -> uint32_t {
      if (pass > 0) return __ldcg(kin + i);
      const int64_t id = static_cast<int64_t>(ids[i]);
      return id >= 0 && id < V && id != padding_id ? static_cast<uint32_t>(id) : V;
    };
    for (int d = lane; d < kEsBins; d += 32) hist[warp][d] = 0u;
    __syncwarp();
    for (uint32_t i = w0 + lane; i < w1; i += 32) atomicAdd(&hist[warp][(key_at(i) >> shift) & mask], 1u);
    __syncthreads();
    // digit d: counts of the warps ahead, this CTA's total
    if (tid < kEsBins) {
      uint32_t t = 0;
      for (int w = 0; w < kEsWarps; ++w) {
        const uint32_t c = hist[w][tid];
        hist[w][tid] = t;
        t += c;
      }
      tot[tid] = t;
    }
    cluster_barrier();
    uint32_t below = 0, all = 0;
    if (tid < kEsBins) {
      for (uint32_t r = 0; r < kEsCluster; ++r) {
        const uint32_t c = ld_cluster_u32(smem_u32(&tot[tid]), r);
        below += r < rank ? c : 0u;
        all += c;
      }
      // exclusive sum of `all` over the digits
      uint32_t inc = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= static_cast<uint32_t>(o)) inc += u;
      }
      if (lane == 31) wsum[warp] = inc;
      below += inc - all;
    }
    __syncthreads();
    if (tid < kEsBins) {
      for (uint32_t w = 0; w < warp; ++w) below += wsum[w];
      for (int w = 0; w < kEsWarps; ++w) hist[w][tid] += below;
    }
    __syncthreads();
    for (uint32_t i0 = w0; i0 < w1; i0 += 32) {
      const uint32_t i = i0 + lane;
      const bool live = i < w1;
      uint32_t key = 0, val = 0, d = kEsBins;
      if (live) {
        key = key_at(i);
        val = pass > 0 ? __ldcg(vin + i) : i;
        d = (key >> shift) & mask;
        if (pass == 0 && key < V) atomicOr(&p.touched[key >> 5], 1u << (key & 31));
        if (pass == 0 && key == V) {
          const int64_t id = static_cast<int64_t>(ids[i]);
          if (id < 0 || id >= V) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingGradId);
        }
      }
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const uint32_t before = __popc(same & ((1u << lane) - 1u));
      uint32_t at = 0;
      if (live) at = hist[warp][d] + before;
      __syncwarp();
      if (live && before == 0) hist[warp][d] += __popc(same);
      __syncwarp();
      if (live) {
        kout[at] = key;
        vout[at] = val;
      }
    }
    cluster_barrier();  // the sorted list, and `tot` read by everyone
  }

  // list the segments that reach past the chunk after the one they start in
  const uint32_t* key = p.key[(passes + 1) & 1];
  const uint32_t chunks = (T + kEgChunk - 1) / kEgChunk;
  for (uint32_t c = gtid; c + 2 < chunks; c += kAll) {
    const uint32_t h = __ldcg(key + (c + 1) * kEgChunk - 1);
    if (h == V || __ldcg(key + (c + 2) * kEgChunk) != h) continue;
    if (c > 0 && __ldcg(key + c * kEgChunk - 1) == h) continue;  // it started earlier
    uint32_t lo = c + 2, hi = chunks;  // chunk lo starts with h, chunk hi does not
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (__ldcg(key + mid * kEgChunk) == h)
        lo = mid;
      else
        hi = mid;
    }
    p.heavy[atomicAdd(p.num_heavy, 1u)] = EmbedHeavy{c, lo};
  }
}

// ---------------------------------------------------------------------------
// The sums. Warp (chunk c, column tile): the segments that start in chunk c,
// and chunk c's share of the long ones. part: fp32 rows, [2 c] for a long
// segment that began in an earlier chunk, [2 c + 1] for one that begins here.
constexpr int kEgWarps = 8;
constexpr int kEgCols = 256;  // columns per warp
constexpr int kEgBatch = 8;   // rows of dy in flight per warp

template <typename TG, typename TT, int E, bool ACC>
__global__ void __launch_bounds__(kEgWarps * 32)
    embed_grad_kernel(const uint32_t* __restrict__ key, const uint32_t* __restrict__ val,
                      const uint32_t* __restrict__ touched, const TG* __restrict__ dy, TT* __restrict__ dtable,
                      float* __restrict__ part, uint32_t T, uint32_t V, int64_t D, float scale, uint32_t sum_blocks) {
  constexpr int NC = kEgCols / (32 * E);  // accesses per lane
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles = static_cast<uint32_t>((D + kEgCols - 1) / kEgCols);
  if (blockIdx.x >= sum_blocks) {
    // zero rows: 32 rows of the table per warp and step
    if constexpr (!ACC) {
      const uint64_t nw = static_cast<uint64_t>(gridDim.x - sum_blocks) * kEgWarps;
      const float z[E] = {};
      for (uint64_t v = static_cast<uint64_t>(blockIdx.x - sum_blocks) * kEgWarps + warp; v < V; v += nw) {
        if ((touched[v >> 5] >> (v & 31)) & 1u) continue;
        for (int64_t k = static_cast<int64_t>(lane) * E; k < D; k += 32 * E)
          Elem<TT, E>::store(dtable + static_cast<int64_t>(v) * D + k, z);
      }
    }
    return;
  }
  const uint64_t item = static_cast<uint64_t>(blockIdx.x) * kEgWarps + warp;
  const uint32_t c = static_cast<uint32_t>(item / tiles);
  const int64_t col = static_cast<int64_t>(item % tiles) * kEgCols + lane * E;
  const uint32_t p0 = c * kEgChunk;
  if (p0 >= T) return;

  const uint32_t ka = p0 + lane < T ? key[p0 + lane] : V;
  if (__shfl_sync(0xffffffffu, ka, 0) == V) return;  // nothing but tokens that take no part
  const uint32_t q = p0 + kEgChunk;
  const uint32_t kb = q + lane < T ? key[q + lane] : V;
  const uint32_t va = ka != V ? val[p0 + lane] : 0u, vb = kb != V ? val[q + lane] : 0u;
  const uint32_t next = q + kEgChunk < T ? key[q + kEgChunk] : V;  // the first key two chunks on
  const uint32_t first = __shfl_sync(0xffffffffu, ka, 0), last = __shfl_sync(0xffffffffu, ka, 31);
  const uint32_t after = __shfl_sync(0xffffffffu, kb, 0);
  const bool goes_on = last != V && after == last;

  uint32_t begin = 0;  // positions within [chunk | next chunk]
  bool head = false;   // the first segment belongs to partial row 2 c
  if (p0 > 0 && key[p0 - 1] == first) {
    const bool whole = first == last;
    head = (whole && goes_on) || (p0 > kEgChunk && key[p0 - kEgChunk - 1] == first);
    // otherwise the warp of the chunk before finishes this segment
    if (!head) begin = __popc(__ballot_sync(0xffffffffu, ka == first));
  }
  uint32_t end = __popc(__ballot_sync(0xffffffffu, ka != V));
  bool tail = false;  // the last segment belongs to partial row 2 c + 1
  if (goes_on && !(head && first == last)) {
    tail = next == last;
    if (!tail && begin < 32) end += __popc(__ballot_sync(0xffffffffu, kb == last));
  }
  if (begin >= end) return;

  auto key_of = [&](uint32_t i) { return __shfl_sync(0xffffffffu, i < 32 ? ka : kb, i & 31); };
  auto val_of = [&](uint32_t i) { return __shfl_sync(0xffffffffu, i < 32 ? va : vb, i & 31); };
  float acc[NC][E] = {};
  uint32_t cur = key_of(begin);
  auto flush = [&](float* prow) {
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int64_t k = col + u * 32 * E;
      if (k < D) {
        if (prow) {
          Elem<float, E>::store(prow + k, acc[u]);
        } else {
          TT* out = dtable + static_cast<int64_t>(cur) * D + k;
          float o[E];
          if constexpr (ACC) Elem<TT, E>::load(out, o);
#pragma unroll
          for (int j = 0; j < E; ++j) o[j] = ACC ? fmaf(acc[u][j], scale, o[j]) : acc[u][j] * scale;
          Elem<TT, E>::store(out, o);
        }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) acc[u][j] = 0.f;
    }
  };
  float* head_row = part + (2 * static_cast<int64_t>(c)) * D;
  for (uint32_t i0 = begin; i0 < end; i0 += kEgBatch) {
    float f[kEgBatch][NC][E];
#pragma unroll
    for (int b = 0; b < kEgBatch; ++b) {
      const uint32_t t = val_of(min(i0 + b, end - 1));
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const int64_t k = col + u * 32 * E;
        if (i0 + b < end && k < D) Elem<TG, E>::load(dy + static_cast<int64_t>(t) * D + k, f[b][u]);
      }
    }
#pragma unroll
    for (int b = 0; b < kEgBatch; ++b) {
      if (i0 + b >= end) break;
      const uint32_t kk = key_of(i0 + b);
      if (kk != cur) {
        flush(head ? head_row : nullptr);
        head = false;
        cur = kk;
      }
#pragma unroll
      for (int u = 0; u < NC; ++u)
#pragma unroll
        for (int j = 0; j < E; ++j) acc[u][j] += f[b][u][j];
    }
  }
  flush(head ? head_row : tail ? head_row + D : nullptr);
}

// One CTA per (long segment, 32 columns), grid-stride: its partial rows added
// in order, the warps taking contiguous shares.
template <typename TT, bool ACC>
__global__ void __launch_bounds__(kEgWarps * 32)
    embed_grad_heavy_kernel(const uint32_t* __restrict__ key, const uint32_t* __restrict__ num_heavy,
                            const EmbedHeavy* __restrict__ heavy, const float* __restrict__ part,
                            TT* __restrict__ dtable, int64_t D, float scale) {
  __shared__ float sh[kEgWarps][32];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles = static_cast<uint32_t>((D + 31) / 32);
  const uint64_t items = static_cast<uint64_t>(*num_heavy) * tiles;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const EmbedHeavy s = heavy[it / tiles];
    const int64_t k = static_cast<int64_t>(it % tiles) * 32 + lane;
    const uint32_t n = s.last - s.first + 1, per = (n + kEgWarps - 1) / kEgWarps;
    const uint32_t a = s.first + min(n, warp * per), b = s.first + min(n, (warp + 1) * per);
    float t = 0.f;
    if (k < D)
      for (uint32_t c = a; c < b; ++c) t += part[(2 * static_cast<int64_t>(c) + (c == s.first ? 1 : 0)) * D + k];
    __syncthreads();  // sh is still read from the item before
    sh[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && k < D) {
      t = 0.f;
#pragma unroll
      for (int w = 0; w < kEgWarps; ++w) t += sh[w][lane];
      TT* out = dtable + static_cast<int64_t>(key[s.last * kEgChunk]) * D + k;
      float o[1] = {0.f};
      if constexpr (ACC) Elem<TT, 1>::load(out, o);
      o[0] = ACC ? fmaf(t, scale, o[0]) : t * scale;
      Elem<TT, 1>::store(out, o);
    }
  }
}

}  // namespace bl
