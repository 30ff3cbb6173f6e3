// Embedding lookup with a scale, and the gradient of the table.
//
//   y_t = scale * E[id_t]              dE_v = scale * sum_{t: id_t = v} dy_t
//
// The gradient adds rows of dy that share a token. Adding them with atomics
// would make the order, and so the rounding, of frequent tokens' sums differ
// from run to run; here the tokens are first put in order of their ids (stable:
// the rows of a token are added in the order of their positions), then the list is
// cut into chunks of 32 positions (8 in a short list) and one warp per (chunk,
// 256 columns) adds up the segments that start in its chunk. A segment that ends
// in the next chunk is finished by the warp that began it; a longer one is
// summed chunk by chunk into fp32 partial rows that a last kernel adds up in
// order, so a token that fills the batch is as parallel as any other.
// Most of the table's rows have no token, and zero-filling them is most of the
// traffic: the first CTAs of the second kernel write zeros to the rows that no
// token names while the list is made, the others wait for it
// and add up rows beside them. Each element of dE is written once.
#pragma once

#include <type_traits>

#include "bl_elem.cuh"

namespace bl {

// an id in [0, V) as a row index, or -1 where it is outside
template <typename TI>
__device__ __forceinline__ int64_t embed_row(const TI* ids, int64_t t, int64_t V) {
  const int64_t id = static_cast<int64_t>(ids[t]);
  return id >= 0 && id < V ? id : -1;
}

constexpr int kEmbThreads = 256;
constexpr int emb_batch(int E) { return E == 1 ? 16 : E == 2 ? 8 : 4; }  // accesses in flight per lane

// One warp per token and up to 512 columns (1024 in accesses of eight); a token outside
// the table gets a row of zeros. Bound by memory: 16384 rows of 2048 from fp32 to
// bf16 17.4 us (97% of the copy rate; 24 us with a CTA per token and one access in
// flight), 16 rows of 4096 1.5 us.
template <typename TI, typename TT, typename TY, int E>
__global__ void __launch_bounds__(kEmbThreads)
    embedding_kernel(const TI* __restrict__ ids, const TT* __restrict__ table, TY* __restrict__ y, uint32_t T,
                     int64_t V, int64_t D, uint32_t tiles, float scale) {
  const uint32_t item = blockIdx.x * (kEmbThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t t = item / tiles, tile = item % tiles;
  grid_begin();
  if (t >= T) return;
  const int64_t row = embed_row(ids, t, V);
  if (row < 0 && lane == 0 && tile == 0) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingId);
  constexpr int BATCH = emb_batch(E), STEP = 32 * E;
  const int64_t base = static_cast<int64_t>(tile) * (BATCH * STEP), k0 = base + lane * E;
  const TT* src = table + (row < 0 ? 0 : row) * D;
  TY* out = y + static_cast<int64_t>(t) * D + k0;
  // columns that are all there need no check and one address
  auto copy = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
    float f[BATCH][E];
    // from valid places all of them, so that nothing stands between the loads
#pragma unroll
    for (int u = 0; u < BATCH; ++u) Elem<TT, E>::load(ALL || k0 + u * STEP < D ? src + k0 + u * STEP : src + D - E, f[u]);
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (ALL || k0 + u * STEP < D) {
#pragma unroll
        for (int j = 0; j < E; ++j) f[u][j] = row < 0 ? 0.f : f[u][j] * scale;
        Elem<TY, E>::store(out + u * STEP, f[u]);
      }
  };
  if (base + BATCH * STEP <= D)
    copy(std::true_type{});
  else
    copy(std::false_type{});
}

// Rows of few columns: the output as one run of accesses, `n` to a row, so that
// no lane is without one (65536 rows of 128 columns: 6.3 us, 14.6 us with a warp
// to each).
template <typename TI, typename TT, typename TY, int E>
__global__ void __launch_bounds__(kEmbThreads)
    embedding_narrow_kernel(const TI* __restrict__ ids, const TT* __restrict__ table, TY* __restrict__ y, uint32_t items,
                            uint32_t n, int64_t V, int64_t D, float scale) {
  constexpr int BATCH = 4;
  grid_begin();
  const uint32_t i0 = blockIdx.x * (kEmbThreads * BATCH) + threadIdx.x;
  float f[BATCH][E];
  int64_t row[BATCH];
  uint32_t t[BATCH], k[BATCH];
#pragma unroll
  for (int u = 0; u < BATCH; ++u) {
    const uint32_t i = min(i0 + u * kEmbThreads, items - 1);
    t[u] = i / n;
    k[u] = (i - t[u] * n) * E;
    row[u] = embed_row(ids, t[u], V);
  }
#pragma unroll
  for (int u = 0; u < BATCH; ++u) Elem<TT, E>::load(table + (row[u] < 0 ? 0 : row[u]) * D + k[u], f[u]);
#pragma unroll
  for (int u = 0; u < BATCH; ++u) {
    if (i0 + u * kEmbThreads >= items) break;
    if (row[u] < 0 && k[u] == 0) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingId);
#pragma unroll
    for (int j = 0; j < E; ++j) f[u][j] = row[u] < 0 ? 0.f : f[u][j] * scale;
    Elem<TY, E>::store(y + static_cast<int64_t>(t[u]) * D + k[u], f[u]);
  }
}

// ---------------------------------------------------------------------------
// A long list is sorted by one cluster of 8 CTAs, a stable radix sort of (id, position) by
// digits of up to 8 bits, ping-pong through the workspace (it stays in L2).
// CTA r of the cluster owns the r-th eighth of the positions and each of its
// warps a contiguous run of that, so that counting in order gives stability.
// Tokens that take no part (padding, ids outside the table) get the key V,
// sort behind all others and are skipped. 65536 tokens take 30 us, longer lists in
// proportion, bound by the scattered stores of the pairs; beside the zeros that is
// hidden where the table is large.
constexpr int kEsCluster = 8;
constexpr int kEsThreads = 1024;
constexpr int kEsWarps = kEsThreads / 32;
constexpr int kEsBins = 256;
constexpr uint32_t kEhFew = 16;  // a long segment's partial rows that one warp adds up
constexpr int kEsHold = 8;    // positions per lane that are held between counting and placing

struct EmbedHeavy {
  uint32_t first, last;  // the chunks in which a long segment starts and ends
};

struct EmbedSort {
  uint2* list[2];       // (id, position), in one store: scattered stores are what bounds a pass
  uint32_t* num_heavy;  // [0]: listed from the front, [1]: those over more than kEhFew chunks, from the back
  EmbedHeavy* heavy;
  uint32_t room;        // entries of the list: chunks
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

__device__ __forceinline__ uint32_t embed_key_of(int64_t id, uint32_t V, int64_t padding_id) {
  return id >= 0 && id < V && id != padding_id ? static_cast<uint32_t>(id) : V;
}
template <typename TI>
__device__ __forceinline__ uint32_t embed_key(const TI* ids, uint32_t i, uint32_t V, int64_t padding_id) {
  return embed_key_of(static_cast<int64_t>(ids[i]), V, padding_id);
}

template <typename TI>
__global__ void __cluster_dims__(kEsCluster, 1, 1) __launch_bounds__(kEsThreads)
    embed_sort_kernel(const TI* __restrict__ ids, uint32_t T, uint32_t V, int64_t padding_id, int passes, int digit_bits,
                      EmbedSort p) {
  __shared__ uint32_t hist[kEsWarps][kEsBins];  // counts, then next output positions
  __shared__ uint32_t tot[kEsBins];         // this CTA's counts, read by the cluster
  __shared__ uint32_t quarter[4][kEsBins];  // of eight warps each
  __shared__ uint32_t wsum[kEsBins / 32];
  const uint32_t rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint32_t kAll = kEsCluster * kEsThreads;
  grid_begin();  // what follows writes zeros meanwhile; its sums wait for this grid
  // whole warps of positions: a warp's run, then a CTA's
  const uint32_t run = ((T + kAll - 1) / kAll) * 32;
  const uint32_t w0 = min(T, (rank * kEsWarps + warp) * run), w1 = min(T, w0 + run);
  const bool hold = run <= kEsHold * 32;
  if (rank == 0 && tid < 2) p.num_heavy[tid] = 0u;
  const uint32_t mask = (1u << digit_bits) - 1u;

  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * digit_bits;
    const uint2* in = p.list[(pass + 1) & 1];
    uint2* out = p.list[pass & 1];
    uint32_t kh[kEsHold], vh[kEsHold];
    // the block of positions b0 + 32 u + lane (key V + 1: none)
    auto load = [&](uint32_t b0) {
#pragma unroll
      for (int u = 0; u < kEsHold; ++u) {
        const uint32_t i = b0 + 32 * u + lane;
        kh[u] = V + 1;
        if (i < w1) {
          const uint2 kv = pass > 0 ? __ldcg(in + i) : make_uint2(embed_key(ids, i, V, padding_id), i);
          kh[u] = kv.x;
          vh[u] = kv.y;
        }
      }
    };
    for (int d = lane; d < kEsBins; d += 32) hist[warp][d] = 0u;
    __syncwarp();
    for (uint32_t b0 = w0; b0 < w1; b0 += kEsHold * 32) {
      load(b0);
#pragma unroll
      for (int u = 0; u < kEsHold; ++u)
        if (kh[u] <= V) atomicAdd(&hist[warp][(kh[u] >> shift) & mask], 1u);
    }
    __syncthreads();
    // digit d: counts of the warps ahead, this CTA's total
    const uint32_t d = tid & (kEsBins - 1), q = tid / kEsBins;
    uint32_t c[kEsWarps / 4], sum = 0;
#pragma unroll
    for (int w = 0; w < kEsWarps / 4; ++w) c[w] = hist[q * (kEsWarps / 4) + w][d];
#pragma unroll
    for (int w = 0; w < kEsWarps / 4; ++w) {
      const uint32_t x = c[w];
      c[w] = sum;
      sum += x;
    }
    quarter[q][d] = sum;
    __syncthreads();
    uint32_t ahead = 0, all4 = 0;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t x = quarter[i][d];
      ahead += i < q ? x : 0u;
      all4 += x;
    }
    if (q == 0) tot[d] = all4;
    cluster_barrier();
    uint32_t x[kEsCluster], below = 0, all = 0;
#pragma unroll
    for (uint32_t r = 0; r < kEsCluster; ++r) x[r] = ld_cluster_u32(smem_u32(&tot[d]), r);
#pragma unroll
    for (uint32_t r = 0; r < kEsCluster; ++r) {
      below += r < rank ? x[r] : 0u;
      all += x[r];
    }
    // exclusive sum of `all` over the digits (the four quarters of the threads do the same)
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= static_cast<uint32_t>(o)) inc += u;
    }
    if (q == 0 && lane == 31) wsum[d / 32] = inc;
    __syncthreads();
    uint32_t base = below + inc - all + ahead;
#pragma unroll
    for (uint32_t w = 0; w < kEsBins / 32; ++w) base += w < d / 32 ? wsum[w] : 0u;
#pragma unroll
    for (int w = 0; w < kEsWarps / 4; ++w) hist[q * (kEsWarps / 4) + w][d] = c[w] + base;
    __syncthreads();
    for (uint32_t b0 = w0; b0 < w1; b0 += kEsHold * 32) {
      if (!hold) load(b0);
#pragma unroll
      for (int u = 0; u < kEsHold; ++u) {
        if (b0 + 32 * u >= w1) break;  // uniform over the warp
        const bool live = kh[u] <= V;
        const uint32_t dig = (kh[u] >> shift) & mask;
        if (pass == 0 && kh[u] == V) {
          const int64_t id = static_cast<int64_t>(ids[vh[u]]);
          if (id < 0 || id >= V) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingGradId);
        }
        // lanes with the same digit, one vote per bit
        uint32_t same = __ballot_sync(0xffffffffu, live);
        for (int b = 0; b < digit_bits; ++b) {
          const bool bit = (dig >> b) & 1u;
          const uint32_t votes = __ballot_sync(0xffffffffu, bit);
          same &= bit ? votes : ~votes;
        }
        const uint32_t before = __popc(same & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (live) at = hist[warp][dig] + before;
        __syncwarp();
        if (live && before == 0) hist[warp][dig] += __popc(same);
        __syncwarp();
        if (live) out[at] = make_uint2(kh[u], vh[u]);
      }
    }
    cluster_barrier();  // the sorted list, and `tot` read by everyone
  }
}

// A short list: a position's place is the number of positions ahead of it in the
// order, counted outright by the whole GPU, 32 positions to a CTA: every warp
// compares them, one to a lane, with its share of the keys, a comparison and an
// addition for each pair. Up to one CTA per SM it takes less than the sort's
// barriers and digits (4096 tokens into 1000 rows of 128 columns: 11.4 us with
// all three kernels, sorted 17 us; 6000 tokens 17.6 and 17.2 us).
constexpr int kErThreads = 1024;
constexpr int kErMost = 148 * 32;

template <typename TI>
__global__ void __launch_bounds__(kErThreads)
    embed_rank_kernel(const TI* __restrict__ ids, uint32_t T, uint32_t V, int64_t padding_id, EmbedSort p) {
  __shared__ __align__(16) uint32_t keys[kErMost];
  __shared__ uint32_t count[32];
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, base = blockIdx.x * 32;
  // a warp's share, whole groups of four; behind the list keys that are ahead of none
  constexpr uint32_t kWarps = kErThreads / 32;
  const uint32_t share = (T + 4 * kWarps - 1) / (4 * kWarps) * 4;
  if (tid < 32) count[tid] = 0u;
  grid_begin();
  if (blockIdx.x == 0 && tid < 2) p.num_heavy[tid] = 0u;
  for (uint32_t i = tid; i < share * kWarps; i += kErThreads) keys[i] = i < T ? embed_key(ids, i, V, padding_id) : V + 1;
  __syncthreads();
  const uint32_t mine = keys[base + lane];
  uint32_t n = 0u;
  const uint32_t j0 = warp * share, j1 = j0 + share;
  // ahead: smaller keys, and equal ones of earlier positions
  auto add = [&](uint32_t a, uint32_t b, uint32_t m) {
#pragma unroll 4
    for (uint32_t j = a; j < b; j += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
      n += (k.x < m ? 1u : 0u) + (k.y < m ? 1u : 0u) + (k.z < m ? 1u : 0u) + (k.w < m ? 1u : 0u);
    }
  };
  const uint32_t a = max(j0, min(j1, base)), b = max(j0, min(j1, base + 32));
  add(j0, a, mine + 1);
  for (uint32_t j = a; j < b; ++j) n += keys[j] < mine + (j < base + lane ? 1u : 0u) ? 1u : 0u;
  add(b, j1, mine);
  atomicAdd(&count[lane], n);
  __syncthreads();
  const uint32_t i = base + tid;
  if (tid < 32 && i < T) {
    if (keys[i] == V) {
      const int64_t id = static_cast<int64_t>(ids[i]);
      if (id < 0 || id >= V) record_error(BL_ERR_INVALID_ARG, kWhereEmbeddingGradId);
    }
    p.list[0][count[tid]] = make_uint2(keys[i], i);
  }
}

// Zeros in the rows of the table that no token names: CTA z of nz takes a
// contiguous range of rows, whose bits it sets from the whole list of tokens. It
// uses nothing of the ordering, and runs ahead of its caller's wait for it: it
// reads the ids (from L2, where the kernels ahead have left them) and writes rows
// of the table, neither of which the ordering writes. 253 MB of zeros take about
// 44 us (5.8 TB/s).
constexpr int kEgThreads = 256;
constexpr int kEgWarps = kEgThreads / 32;
constexpr int kEzRows = 4096 * 32;  // rows of the table whose bits are held at a time

template <typename TT, int E>
__device__ __forceinline__ void embed_zero(uint32_t* bits, const void* __restrict__ ids, bool ids64, uint32_t T,
                                           uint32_t V, int64_t padding_id, TT* __restrict__ dtable, int64_t D,
                                           uint64_t z, uint64_t nz) {
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t v_end = static_cast<uint32_t>(V * (z + 1) / nz);
  for (uint32_t v0 = static_cast<uint32_t>(V * z / nz); v0 < v_end; v0 += kEzRows) {
    const uint32_t rows = min(v_end - v0, static_cast<uint32_t>(kEzRows));
    for (uint32_t i = tid; i < (rows + 31) / 32; i += kEgThreads) bits[i] = 0u;
    __syncthreads();
    auto mark = [&](const auto* id) {
#pragma unroll 8
      for (uint32_t i = tid; i < T; i += kEgThreads) {
        const uint32_t k = embed_key_of(__ldcg(id + i), V, padding_id) - v0;
        if (k < rows) atomicOr(&bits[k >> 5], 1u << (k & 31));
      }
    };
    if (ids64)
      mark(static_cast<const int64_t*>(ids));
    else
      mark(static_cast<const int32_t*>(ids));
    __syncthreads();
    const float zero[E] = {};
    for (uint32_t r = warp; r < rows; r += kEgWarps) {
      if ((bits[r >> 5] >> (r & 31)) & 1u) continue;
      TT* row = dtable + static_cast<int64_t>(v0 + r) * D;
      if constexpr (E > 1) {
#pragma unroll 4
        for (int64_t k = static_cast<int64_t>(lane) * E; k < D; k += 32 * E) Elem<TT, E>::store(row + k, zero);
      } else {
        // 16 bytes at a time between the row's first and last whole pieces, its ends one by one
        const uintptr_t a = reinterpret_cast<uintptr_t>(row), end = a + static_cast<uintptr_t>(D) * sizeof(TT);
        const uintptr_t a16 = min((a + 15) & ~uintptr_t(15), end), e16 = max(end & ~uintptr_t(15), a16);
#pragma unroll 4
        for (uintptr_t i = a16 + lane * 16; i < e16; i += 512) *reinterpret_cast<uint4*>(i) = make_uint4(0u, 0u, 0u, 0u);
        const uintptr_t head = a + lane * sizeof(TT), tail = e16 + lane * sizeof(TT);
        if (head < a16) Elem<TT, 1>::store(reinterpret_cast<TT*>(head), zero);
        if (tail < end) Elem<TT, 1>::store(reinterpret_cast<TT*>(tail), zero);
      }
    }
    __syncthreads();  // the bits are read
  }
}

// ---------------------------------------------------------------------------
// The sums. Warp (chunk c, column tile): the segments that start in chunk c,
// and chunk c's share of the long ones. part: fp32 rows, [2 c] for a long
// segment that began in an earlier chunk, [2 c + 1] for one that begins here.
// Rows of dy are read as they come in the list, 4 KB of them in flight per warp,
// kept packed until they are added (unpacked, 128 registers left 16 warps per SM
// and the sums of 32768 x 4096 took 110 us; so they take 62). With the sort, the
// zeros and the long segments: 32768 tokens of 4096 columns into 32000 fp32 rows
// 139 us (82% of the copy rate), 2048 x 2048 49 us (84%).
constexpr int kEgCols = 256;   // columns per warp
constexpr int kEgChunk = 32;   // sorted positions per warp
constexpr int kEgShort = 8;    // ... of a list so short that chunks of 32 leave SMs without work

// the row as loaded, unpacked when it is added; always loaded from valid places
// (behind the last column from it; ALL: there is none), so that nothing stands
// between the loads
template <typename T, int E>
struct EgRow {
  static constexpr int NC = kEgCols / (32 * E);
  float f[NC][E];
  template <bool ALL>
  __device__ __forceinline__ void load(const T* row, int64_t col, int64_t D) {
#pragma unroll
    for (int u = 0; u < NC; ++u) Elem<T, E>::load(row + (ALL ? col + u * 32 * E : min(col + u * 32 * E, D - E)), f[u]);
  }
  __device__ __forceinline__ void add(float (&acc)[NC][E]) const {
#pragma unroll
    for (int u = 0; u < NC; ++u)
#pragma unroll
      for (int j = 0; j < E; ++j) acc[u][j] += f[u][j];
  }
};
template <>
struct EgRow<uint16_t, 8> {
  uint4 v;
  template <bool ALL>
  __device__ __forceinline__ void load(const uint16_t* row, int64_t col, int64_t D) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(row + min(col, D - 8)));
  }
  __device__ __forceinline__ void add(float (&acc)[1][8]) const {
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[0][2 * j] += __uint_as_float(h[j] << 16);
      acc[0][2 * j + 1] += __uint_as_float(h[j] & 0xFFFF0000u);
    }
  }
};

// The first `zero_ctas` CTAs write zeros, while the list is ordered. What allows
// that: this grid is scheduled once every CTA of the kernel ahead has let it be,
// which each does after its own wait (grid_begin), so whatever was enqueued
// before the two is complete by then, its results are in L2, and nothing reads
// the table's old rows any more; the kernel ahead writes only the workspace. The
// CTAs that use its list wait for it first, the others before they end: the grid
// is complete only after the one ahead, for the kernels that wait for this one
// (the next may be scheduled at once, and does).
// (With every zero behind a wait, half of them written by CTAs of the ordering's own
// grid: 2048 tokens x 2048 columns 49 -> 55 us, 16384 x 2048 65 -> 78 us.)
template <typename TG, typename TT, int E, int CH, bool ACC>
__global__ void __launch_bounds__(kEgThreads, 3)
    embed_grad_kernel(const void* __restrict__ ids, bool ids64, int64_t padding_id, uint32_t zero_ctas,
                      const uint2* __restrict__ list, const TG* __restrict__ dy, TT* __restrict__ dtable, float* __restrict__ part,
                      uint32_t* __restrict__ num_heavy, EmbedHeavy* __restrict__ heavy, uint32_t room, uint32_t T,
                      uint32_t V, int64_t D, float scale) {
  grid_dependents_launch();
  if constexpr (!ACC) {
    __shared__ uint32_t bits[kEzRows / 32];
    if (blockIdx.x < zero_ctas) {
      embed_zero<TT, E == 8 ? 8 : 1>(bits, ids, ids64, T, V, padding_id, dtable, D, blockIdx.x, zero_ctas);
      grid_dependency_wait();
      return;
    }
  }
  constexpr int NC = kEgCols / (32 * E);  // accesses per lane
  constexpr uint32_t BATCH = E == 8 && sizeof(TG) == 2 ? 8 : 4;  // rows in flight
  constexpr uint32_t kAll = 0xffffffffu;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles = static_cast<uint32_t>((D + kEgCols - 1) / kEgCols);
  grid_dependency_wait();
  const uint32_t item = (blockIdx.x - zero_ctas) * kEgWarps + warp, c = item / tiles;
  const int64_t col = static_cast<int64_t>(item % tiles) * kEgCols + lane * E;
  const uint32_t p0 = c * CH;
  if (p0 >= T) return;

  // lanes 0 .. CH - 1: the chunk's positions (ka, va) and the next chunk's (kb, vb)
  const uint32_t q = p0 + CH;
  const bool in_a = lane < CH && p0 + lane < T, in_b = lane < CH && q + lane < T;
  const uint2 none = make_uint2(V, 0u), pa = in_a ? list[p0 + lane] : none, pb = in_b ? list[q + lane] : none;
  const uint32_t ka = pa.x, va = pa.y, kb = pb.x, vb = pb.y;
  const uint32_t next = q + CH < T ? list[q + CH].x : V;       // the first key two chunks on
  const uint32_t before = p0 > 0 ? list[p0 - 1].x : V;         // the last key of the chunk before
  const uint32_t before2 = p0 > CH ? list[p0 - CH - 1].x : V;  // ... and of the one before that
  const uint32_t first = __shfl_sync(kAll, ka, 0), last = __shfl_sync(kAll, ka, CH - 1);
  if (first == V) return;  // nothing but tokens that take no part
  const bool goes_on = last != V && __shfl_sync(kAll, kb, 0) == last;

  uint32_t begin = 0;  // positions within [chunk | next chunk]
  bool head = false;   // the first segment belongs to partial row 2 c
  if (before == first) {
    head = (first == last && goes_on) || before2 == first;
    // otherwise the warp of the chunk before finishes this segment
    if (!head) begin = __popc(__ballot_sync(kAll, in_a && ka == first));
  }
  uint32_t end = __popc(__ballot_sync(kAll, in_a && ka != V));
  bool tail = false;  // the last segment belongs to partial row 2 c + 1
  if (goes_on && !(head && first == last)) {
    tail = next == last;
    if (!tail) end += __popc(__ballot_sync(kAll, in_b && kb == last));
    if (tail && item % tiles == 0) {  // list it: chunk lo starts with it, chunk hi does not
      uint32_t lo = c + 2, hi = room;
      while (hi - lo > 1) {
        const uint32_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const uint32_t n = __popc(__ballot_sync(kAll, at < hi && list[static_cast<uint64_t>(at) * CH].x == last));
        hi = min(hi, lo + (n + 1) * step);
        lo += n * step;
      }
      if (lane == 0) {
        const bool few = lo - c < kEhFew;
        const uint32_t at = atomicAdd(num_heavy + (few ? 0 : 1), 1u);
        heavy[few ? at : room - 1 - at] = EmbedHeavy{c, lo};
      }
    }
  }
  if (begin >= end) return;

  auto key_of = [&](uint32_t i) { return __shfl_sync(kAll, i < CH ? ka : kb, i < CH ? i : i - CH); };
  auto val_of = [&](uint32_t i) { return __shfl_sync(kAll, i < CH ? va : vb, i < CH ? i : i - CH); };
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
  auto sums = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
    for (uint32_t i0 = begin; i0 < end; i0 += BATCH) {
      EgRow<TG, E> row[BATCH];
#pragma unroll
      for (uint32_t b = 0; b < BATCH; ++b) {
        const uint32_t t = val_of(min(i0 + b, end - 1));
        row[b].template load<ALL>(dy + static_cast<int64_t>(t) * D, col, D);
      }
#pragma unroll
      for (uint32_t b = 0; b < BATCH; ++b) {
        if (i0 + b >= end) break;
        const uint32_t kk = key_of(i0 + b);
        if (kk != cur) {
          flush(head ? head_row : nullptr);
          head = false;
          cur = kk;
        }
        row[b].add(acc);
      }
    }
  };
  // narrow accesses of columns that are all there need one address per row (4788 x 4095: 51 us, 53 us without)
  if (E < 8 && static_cast<int64_t>(item % tiles + 1) * kEgCols <= D)
    sums(std::bool_constant<E < 8>{});
  else
    sums(std::false_type{});
  flush(head ? head_row : tail ? head_row + D : nullptr);
}

// The long segments' partial rows added in order: a warp per (segment, 32 E
// columns) for those over few chunks, a CTA for the others, each of its warps a
// contiguous share.
constexpr int kEhWarps = 8;

template <typename TT, int E, bool ACC>
__global__ void __launch_bounds__(kEhWarps * 32)
    embed_grad_heavy_kernel(const uint2* __restrict__ list, const uint32_t* __restrict__ num_heavy,
                            const EmbedHeavy* __restrict__ heavy, uint32_t room, const float* __restrict__ part,
                            TT* __restrict__ dtable, uint32_t chunk, int64_t D, float scale) {
  __shared__ float sh[kEhWarps][32 * E];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tiles = static_cast<uint32_t>((D + 32 * E - 1) / (32 * E));
  grid_begin();
  const uint64_t few = static_cast<uint64_t>(num_heavy[0]) * tiles, many = static_cast<uint64_t>(num_heavy[1]) * tiles;
  // sum of partial rows a .. b - 1 of a segment that began in chunk `first`
  auto add_rows = [&](uint32_t first, uint32_t a, uint32_t b, int64_t k, float(&t)[E]) {
#pragma unroll
    for (int j = 0; j < E; ++j) t[j] = 0.f;
    if (k >= D) return;
    for (uint32_t c0 = a; c0 < b; c0 += 8) {
      float f[8][E];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t c = c0 + i;
#pragma unroll
        for (int j = 0; j < E; ++j) f[i][j] = 0.f;
        if (c < b) Elem<float, E>::load(part + (2 * static_cast<int64_t>(c) + (c == first ? 1 : 0)) * D + k, f[i]);
      }
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) t[j] += f[i][j];
    }
  };
  auto write = [&](const EmbedHeavy& s, int64_t k, const float(&t)[E]) {
    if (k >= D) return;
    TT* out = dtable + static_cast<int64_t>(list[static_cast<uint64_t>(s.last) * chunk].x) * D + k;
    float o[E];
    if constexpr (ACC) Elem<TT, E>::load(out, o);
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = ACC ? fmaf(t[j], scale, o[j]) : t[j] * scale;
    Elem<TT, E>::store(out, o);
  };
  float t[E];
  for (uint64_t it = blockIdx.x; it < many; it += gridDim.x) {
    const EmbedHeavy s = heavy[room - 1 - it / tiles];
    const int64_t k = static_cast<int64_t>(it % tiles) * (32 * E) + lane * E;
    const uint32_t m = s.last - s.first + 1, per = (m + kEhWarps - 1) / kEhWarps;
    add_rows(s.first, s.first + min(m, warp * per), s.first + min(m, (warp + 1) * per), k, t);
    __syncthreads();  // sh is still read from the item before
#pragma unroll
    for (int j = 0; j < E; ++j) sh[warp][j * 32 + lane] = t[j];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        t[j] = 0.f;
#pragma unroll
        for (int w = 0; w < kEhWarps; ++w) t[j] += sh[w][j * 32 + lane];
      }
      write(s, k, t);
    }
  }
  // from the last CTA down: the first ones have the long segments
  const uint64_t me = static_cast<uint64_t>(gridDim.x - 1 - blockIdx.x) * kEhWarps + warp;
  for (uint64_t it = me; it < few; it += static_cast<uint64_t>(gridDim.x) * kEhWarps) {
    const EmbedHeavy s = heavy[it / tiles];
    const int64_t k = static_cast<int64_t>(it % tiles) * (32 * E) + lane * E;
    add_rows(s.first, s.first, s.last + 1, k, t);
    write(s, k, t);
  }
}

}  // namespace bl
