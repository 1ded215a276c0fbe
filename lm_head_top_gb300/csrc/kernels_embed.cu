// Rows of an embedding table, and the table's gradient.
//
//   Y[t] = s W[ids[t]],    dW[v] = s sum over t with ids[t] = v of dY[t]
//
// Forward: a copy of rows by index, one read and one write of DRAM; warps take
// slices of rows, eight elements a lane at a time.
//
// Backward: the (id, token) pairs are sorted by id, stably, so that an id's tokens
// lie together in their order. A warp then takes a piece of 32 sorted tokens and a
// slab of 256 columns: lane i holds the piece's i-th pair, so where an id ends is a
// ballot, and every lane adds up 8 columns of the tokens' rows, which come through
// shared memory, 24 to 32 of them always under way (16 KB a warp; read when they were
// needed, 8 at a time, they kept DRAM at 60 %). A row of dY is read once and a row of dW
// written once (or added to once: a reduction in L2, of which every element gets one,
// and nothing comes back to be waited for). Sums of ids that run past a piece's ends
// are left in the workspace and added up in a last launch, in their order. Where dW is
// overwritten, the sort notes the ids it meets in a bitmap, and the same warps then
// write zeros to the other rows: a row of dW is written once, and not cleared before.
// No atomics whose order could change a sum.
//
// The sort. Up to EMBED_RANKED tokens: every token's place is counted, the ids
// below its own and the equal ones before it: T^2 comparisons, spread over the
// whole GPU in one launch. Above: a stable sort by 9 bits at a time; up to
// CLUSTER_SORTED tokens in the shared memory of one cluster, in one launch, beyond
// in two launches each (counts of every tile, then each tile's places, for which every
// block adds up the tiles' counts itself: at most EMBED_TILES of them). Tokens that do not
// count get the id V and go last.
#include <algorithm>
#include <atomic>

#include "kdkl_body.h"
#include "rows.cuh"
#include "tc_primitives.cuh"

namespace kdkl {

namespace {

constexpr int kMaxDevices = 64;
constexpr int EMBED_THREADS = 256;
constexpr int EMBED_CHECK = 32768;  // ids that one block checks beside the copies
constexpr int FORWARD_VECTORS = 4;
constexpr int EMBED_RANKED = 8192;
constexpr int CLUSTER_BLOCKS = 8, CLUSTER_MOST = 16, CLUSTER_THREADS = 1024;
constexpr int CLUSTER_SORTED = 65536;
constexpr int RANK_LANES = 8;   // threads that count for one token
constexpr int EMBED_TILES = 256;
constexpr int EMBED_TILE_MIN = 1024;
constexpr int DIGIT_BITS = 9;
constexpr int DIGITS = 1 << DIGIT_BITS;
constexpr int SORT_WARPS = EMBED_THREADS / 32;
constexpr int SUM_THREADS = 128;
constexpr int SLAB = 256;    // columns of a warp
constexpr int FILL_ROWS = 8;  // of dW that a warp clears at a time
constexpr int BATCH = 8;     // rows of dY that are copied, or partial sums that are read, together
constexpr int GROUPS = EMBED_PIECE / BATCH;
static_assert(EMBED_PIECE == 32, "a lane for each token of a piece");

// A slab of a row in shared memory, and room for where it starts within 16 bytes.
template <typename TY>
__host__ __device__ constexpr int place_bytes() {
  return SLAB * (int)sizeof(TY) + 16;
}
// Groups of rows that a warp has there: 16 KB of either type, and three blocks on an SM (with 32
// KB and one block, fp32 rows and dW's other rows both took longer).
template <typename TY>
__host__ __device__ constexpr int ring_groups() {
  return sizeof(TY) == 2 ? GROUPS : GROUPS / 2;
}
template <typename TY>
__host__ __device__ constexpr int ring_bytes() {
  return ring_groups<TY>() * BATCH * place_bytes<TY>();
}

__device__ __forceinline__ void cp_async_16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The first n bytes of 16; nothing after them is read.
__device__ __forceinline__ void cp_async_16_of(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n)
               : "memory");
}

template <typename TW, typename TY, int VEC>
__global__ void __launch_bounds__(EMBED_THREADS)
    embedding_forward_kernel(const EmbedArgs a, int slices, int per_slice, int check) {
  grid_dependents_go();
  grid_dependency_wait();
  if (check && blockIdx.x == 0) {  // the status word, and nothing else
    int bad = 0;
    for (int t = threadIdx.x; t < a.T; t += EMBED_THREADS)
      if (!a.mask || a.mask[t]) bad |= (unsigned)a.ids[t] >= (unsigned)a.V;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = bad ? DEV_ERR_INDEX_RANGE : DEV_OK;
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long item = (long long)(blockIdx.x - (check ? 1 : 0)) * SORT_WARPS + (threadIdx.x >> 5);
  const long long t = item / slices;
  if (t >= a.T) return;
  const int c0 = (int)(item - t * slices) * per_slice, c1 = min(a.d, c0 + per_slice);
  long long id = -1;
  if (!a.mask || a.mask[t]) {
    id = a.ids[t];
    if (id < 0 || id >= a.V) {
      id = -1;
      if (!check && lane == 0 && c0 == 0) record_error(a.status, DEV_ERR_INDEX_RANGE);
    }
  }
  TY* y = static_cast<TY*>(a.Y) + t * a.d;
  const TW* w = static_cast<const TW*>(a.W) + id * a.d;
#pragma unroll 4
  for (int c = c0 + lane * VEC; c < c1; c += 32 * VEC) {
    float v[VEC] = {};
    if (id >= 0) {
      RowVec<TW, VEC> r;
      r.load(w + c);
      r.get(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] *= a.scale;
    }
    RowVec<TY, VEC> o;
    o.set(v);
    o.store(y + c);
  }
}

// The id of token t as it is sorted.
__device__ __forceinline__ int sort_key(const EmbedArgs& a, int t, bool report) {
  const int id = a.ids[t];  // read beside the mask, not after it
  if (a.mask && !a.mask[t]) return a.V;
  if ((unsigned)id < (unsigned)a.V) return id;
  if (report) record_error(a.status, DEV_ERR_INDEX_RANGE);
  return a.V;
}

// Notes in the bitmap that id is met.
__device__ __forceinline__ void note_id(const EmbedArgs& a, int id) {
  if (a.met && id < a.V) atomicOr(&a.met[id >> 5], 1u << (id & 31));
}

// One launch for up to EMBED_RANKED tokens: RANK_LANES threads count for one token.
__global__ void __launch_bounds__(EMBED_THREADS) embedding_rank_kernel(const EmbedArgs a) {
  extern __shared__ int4 rank_keys[];
  int* keys = reinterpret_cast<int*>(rank_keys);
  grid_dependents_go();
  grid_dependency_wait();
  const int padded = (a.T + 3) & ~3;
  for (int t = threadIdx.x; t < padded; t += EMBED_THREADS)
    keys[t] = t < a.T ? sort_key(a, t, blockIdx.x == 0) : 0x7fffffff;
  __syncthreads();
  const int t = (int)(blockIdx.x * EMBED_THREADS + threadIdx.x) / RANK_LANES;
  const int part = threadIdx.x % RANK_LANES;
  const int mine = t < a.T ? keys[t] : 0;
  int rank = 0;
  if (t < a.T) {
    for (int q = part; q < padded / 4; q += RANK_LANES) {
      const int4 k = rank_keys[q];
      const int j = 4 * q;
      // equal ids count where their token is earlier
      rank += k.x < mine + (j < t) ? 1 : 0;
      rank += k.y < mine + (j + 1 < t) ? 1 : 0;
      rank += k.z < mine + (j + 2 < t) ? 1 : 0;
      rank += k.w < mine + (j + 3 < t) ? 1 : 0;
    }
  }
#pragma unroll
  for (int o = RANK_LANES / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (t < a.T && part == 0) {
    a.pairs[0][rank] = make_int2(mine, t);
    note_id(a, mine);
  }
}

// One launch for up to CLUSTER_SORTED tokens: a cluster of blocks holds all pairs in its shared
// memory, `share` of them a block, in their order; every 9 bits they move to their places in the
// other buffer, in whichever block that is, and after the last ones to memory. A warp has
// consecutive pairs and ranks equal digits by a match; blocks read one another's counts. What
// takes its time is a chain of waits: for the blocks' counts and barriers, the matches, the
// scattered stores: 32,768 tokens take 18 us, 21 with cold caches. 16 blocks are faster than 8
// (21 and 27 us when pairs were matched twice).
__global__ void __launch_bounds__(CLUSTER_THREADS)
    embedding_cluster_sort_kernel(const EmbedArgs a, const int share, const int blocks) {
  extern __shared__ uint4 cluster_smem[];
  constexpr int WARPS = CLUSTER_THREADS / 32;
  constexpr int ROUNDS = CLUSTER_SORTED / CLUSTER_BLOCKS / CLUSTER_THREADS;  // of a warp, at most
  static_assert(DIGITS <= CLUSTER_THREADS, "a thread for each digit");
  uint2* buf = reinterpret_cast<uint2*>(cluster_smem);                          // [2][share]
  uint32_t* total = reinterpret_cast<uint32_t*>(buf + 2 * share);               // [DIGITS]
  uint32_t* base = total + DIGITS;                                              // [DIGITS]
  unsigned short* count = reinterpret_cast<unsigned short*>(base + DIGITS);     // [WARPS][DIGITS]
  __shared__ uint32_t warp_sum[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  const uint32_t rank = cluster_ctarank();
  const int mine = share / WARPS, mine0 = warp * mine;  // of a warp: a multiple of 32
  unsigned short* my_count = count + warp * DIGITS;
  grid_dependents_go();
  grid_dependency_wait();
#pragma unroll 4
  for (int i = threadIdx.x; i < share; i += CLUSTER_THREADS) {
    const int t = (int)rank * share + i;
    const int key = t < a.T ? sort_key(a, t, true) : a.V;
    if (t < a.T) note_id(a, key);
    buf[i] = make_uint2((uint32_t)key, (uint32_t)t);
  }
  int from = 0;
  for (int shift = 0; shift < 31 && (a.V >> shift); shift += DIGIT_BITS, from ^= 1) {
    const bool last = shift + DIGIT_BITS >= 31 || !(a.V >> (shift + DIGIT_BITS));
    const uint2* in = buf + from * share;
    for (int i = threadIdx.x; i < WARPS * DIGITS / 8; i += CLUSTER_THREADS)
      reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    unsigned short nth[ROUNDS];  // of each of this lane's pairs among the warp's of its digit
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (32 * r >= mine) break;
      const int digit = (int)(in[mine0 + 32 * r + lane].x >> shift) & (DIGITS - 1);
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      nth[r] = (unsigned short)(my_count[digit] + __popc(same & below));
      __syncwarp();
      if ((same & below) == 0) my_count[digit] += (unsigned short)__popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < DIGITS) {
      unsigned short n[WARPS];
#pragma unroll
      for (int w = 0; w < WARPS; ++w) n[w] = count[w * DIGITS + threadIdx.x];
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {  // each warp's start among the block's
        count[w * DIGITS + threadIdx.x] = (unsigned short)sum;
        sum += n[w];
      }
      total[threadIdx.x] = sum;
    }
    cluster_sync_all();
    uint32_t all = 0, before = 0;
    if (threadIdx.x < DIGITS) {
      const uint32_t at = smem_u32(total + threadIdx.x);
      uint32_t n[CLUSTER_MOST];
#pragma unroll
      for (int r = 0; r < CLUSTER_MOST; ++r)  // all of them under way together
        asm volatile("ld.shared::cluster.b32 %0, [%1];"
                     : "=r"(n[r])
                     : "r"(mapa_shared(at, (uint32_t)min(r, blocks - 1)))
                     : "memory");
#pragma unroll
      for (int r = 0; r < CLUSTER_MOST; ++r) {
        all += r < blocks ? n[r] : 0;
        before += r < (int)rank ? n[r] : 0;
      }
    }
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (threadIdx.x < DIGITS) {
      const uint32_t sum = lane < warp ? warp_sum[lane] : 0;
      base[threadIdx.x] = inc - all + before + __reduce_add_sync(0xffffffffu, sum);
    }
    __syncthreads();
    const uint32_t to0 = smem_u32(buf + (from ^ 1) * share);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (32 * r >= mine) break;
      const uint2 pair = in[mine0 + 32 * r + lane];
      const int digit = (int)(pair.x >> shift) & (DIGITS - 1);
      const uint32_t to = base[digit] + my_count[digit] + nth[r];
      if (last) {
        if (to < (uint32_t)a.T)  // pairs past the end are last
          a.pairs[0][to] = make_int2((int)pair.x, (int)pair.y);
      } else {
        const uint32_t block = to / (uint32_t)share;
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(
                         mapa_shared(to0 + (to - block * share) * 8, block)),
                     "r"(pair.x), "r"(pair.y)
                     : "memory");
      }
    }
    cluster_sync_all();  // the pairs have moved, and all have read the counts
  }
}

struct SortPass {
  const int2* in;  // null: the ids themselves, in their order
  int2* out;
  int tile, tiles, shift;
};

__device__ __forceinline__ int2 pass_pair(const EmbedArgs& a, const SortPass& p, int i,
                                          bool report) {
  return p.in ? p.in[i] : make_int2(sort_key(a, i, report), i);
}

// hist[tile][digit]; the first pass notes the ids
__global__ void __launch_bounds__(EMBED_THREADS)
    embedding_count_kernel(const EmbedArgs a, const SortPass p) {
  __shared__ unsigned count[DIGITS];
  for (int i = threadIdx.x; i < DIGITS; i += EMBED_THREADS) count[i] = 0;
  __syncthreads();
  grid_dependents_go();
  grid_dependency_wait();
  const long long begin = (long long)blockIdx.x * p.tile;
  const int end = (int)min((long long)a.T, begin + p.tile);
  for (int i = (int)begin + threadIdx.x; i < end; i += EMBED_THREADS) {
    const int key = pass_pair(a, p, i, true).x;
    atomicAdd(&count[(key >> p.shift) & (DIGITS - 1)], 1u);
    if (!p.in) note_id(a, key);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < DIGITS; i += EMBED_THREADS)
    a.hist[(long long)blockIdx.x * DIGITS + i] = count[i];
}

// The pairs of one tile to their places: by digit, then by tile, then by warp (each has
// a consecutive share of the tile), then in their order.
__global__ void __launch_bounds__(EMBED_THREADS)
    embedding_place_kernel(const EmbedArgs a, const SortPass p) {
  __shared__ unsigned place[SORT_WARPS][DIGITS];
  __shared__ unsigned total[DIGITS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < SORT_WARPS * DIGITS; i += EMBED_THREADS) (&place[0][0])[i] = 0;
  __syncthreads();
  grid_dependents_go();
  grid_dependency_wait();
  const long long tile0 = (long long)blockIdx.x * p.tile;
  const int share = p.tile / SORT_WARPS;  // a multiple of 32
  const long long begin = tile0 + (long long)warp * share;
  const int end = (int)min((long long)a.T, begin + share);
  for (long long i = begin + lane; i < end; i += 32)
    atomicAdd(&place[warp][(pass_pair(a, p, (int)i, false).x >> p.shift) & (DIGITS - 1)], 1u);
  // this tile's start within every digit, and the digits' totals
  __shared__ unsigned before[DIGITS];
  for (int digit = threadIdx.x; digit < DIGITS; digit += EMBED_THREADS) {
    unsigned all = 0, mine = 0;
#pragma unroll 16
    for (int t = 0; t < p.tiles; ++t) {
      const unsigned n = a.hist[(long long)t * DIGITS + digit];
      all += n;
      mine += t < (int)blockIdx.x ? n : 0;
    }
    total[digit] = all;
    before[digit] = mine;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the digits
    unsigned carry = 0;
    for (int d0 = 0; d0 < DIGITS; d0 += 32) {
      const unsigned n = total[d0 + lane];
      unsigned inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      total[d0 + lane] = carry + inc - n;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  for (int digit = threadIdx.x; digit < DIGITS; digit += EMBED_THREADS) {
    unsigned at = total[digit] + before[digit];
    for (int w = 0; w < SORT_WARPS; ++w) {
      const unsigned n = place[w][digit];
      place[w][digit] = at;
      at += n;
    }
  }
  __syncthreads();
  for (long long i0 = begin; i0 < end; i0 += 32) {
    const long long i = i0 + lane;
    const bool here = i < end;
    const unsigned live = __ballot_sync(0xffffffffu, here);
    if (here) {
      const int2 pair = pass_pair(a, p, (int)i, false);
      const int digit = (pair.x >> p.shift) & (DIGITS - 1);
      const unsigned same = __match_any_sync(live, digit);
      const unsigned rank = __popc(same & ((1u << lane) - 1u));
      const unsigned at = place[warp][digit] + rank;
      __syncwarp(live);
      if (rank == 0) place[warp][digit] += __popc(same);
      p.out[at] = pair;
    }
    __syncwarp();
  }
}

// dW's row of `id`, columns from c, gets v (times the scale).
template <int VEC>
__device__ __forceinline__ void hand_over(const EmbedArgs& a, int id, int c, const float (&v)[VEC]) {
  float* to = a.dW + (long long)id * a.d + c;
  float o[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) o[j] = v[j] * a.scale;
  if (a.accumulate) {
    if constexpr (VEC == 4) {
      red_add_f32x4(to, make_float4(o[0], o[1], o[2], o[3]));
    } else {
      atomicAdd(to, o[0]);  // one for each element
    }
    return;
  }
  RowVec<float, VEC> r;
  r.set(o);
  r.store(to);
}

// A lane's 8 columns of a slab: where rows lie on vectors two times 4, so that a warp's
// reductions are whole sectors of L2 (two halves of a sector cost it two operations: 54 us of
// 175 for 19,000 rows of 2880); else every 32nd.
template <bool ODD>
__device__ __forceinline__ int slab_column(int lane, int k) {
  return ODD ? lane + 32 * k : (k >> 2) * (SLAB / 2) + lane * 4 + (k & 3);
}

// A piece's sum of a slab, to dW's row `id` or (part not null) to the workspace.
template <bool ODD>
__device__ __forceinline__ void put_sum(const EmbedArgs& a, int id, float* part, int c0, int lane,
                                        const float (&acc)[8]) {
  constexpr int N = ODD ? 1 : 4;
#pragma unroll
  for (int k = 0; k < 8; k += N) {
    const int c = c0 + slab_column<ODD>(lane, k);
    if (c >= a.d) continue;
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = acc[k + j];
    if (part) {
      RowVec<float, N> o;
      o.set(v);
      o.store(part + c);
    } else {
      hand_over<N>(a, id, c, v);
    }
  }
}

// What a warp holds of a piece and a slab.
struct SumItem {
  int key, pos;    // of this lane's pair
  int n;           // pairs that count
  unsigned ends;   // after which of them an id's sum ends
  int head;        // the first sum continues one of the piece before
  int piece, c0;
};

__device__ __forceinline__ SumItem sum_item(const EmbedArgs& a, const int2* __restrict__ pairs,
                                            long long item, long long items, int slabs) {
  SumItem x;
  x.n = 0;
  if (item >= items) return x;
  const int lane = threadIdx.x & 31;
  x.piece = (int)(item / slabs);
  x.c0 = (int)(item - (long long)x.piece * slabs) * SLAB;
  const int begin = x.piece * EMBED_PIECE;
  // pairs past the end, and those that do not count (they are last), are left out
  const int2 pair = begin + lane < a.T ? pairs[begin + lane] : make_int2(a.V, 0);
  x.key = pair.x;
  x.pos = pair.y;
  int edge = a.V;  // lane 0: the pair before the piece, lane 31: the one after it
  if (lane == 0 && begin > 0) edge = pairs[begin - 1].x;
  if (lane == 31 && begin + EMBED_PIECE < a.T) edge = pairs[begin + EMBED_PIECE].x;
  x.n = __popc(__ballot_sync(0xffffffffu, x.key < a.V));
  int next = __shfl_down_sync(0xffffffffu, x.key, 1);
  if (lane == 31) next = edge;
  x.ends = __ballot_sync(0xffffffffu, x.key != next);
  x.head = __shfl_sync(0xffffffffu, edge == x.key, 0);
  return x;
}

// Rows of a piece's group, a slab of each, on their way to the group's places of the warp's
// ring (a group of copies, empty past the piece's end).
template <typename TY, bool ODD>
__device__ __forceinline__ void fetch_rows(const EmbedArgs& a, const SumItem& x, int group,
                                           uint32_t ring) {
  const int lane = threadIdx.x & 31, j0 = group * BATCH;
  const uint32_t places = ring + group % ring_groups<TY>() * BATCH * place_bytes<TY>();
  const TY* dY = static_cast<const TY*>(a.dY);
#pragma unroll
  for (int j = 0; j < BATCH; ++j) {
    if (j0 + j >= x.n) break;
    const int t = __shfl_sync(0xffffffffu, x.pos, j0 + j);
    const uint32_t to = places + j * place_bytes<TY>();
    const TY* from = dY + (long long)t * a.d + x.c0;
    if constexpr (!ODD) {
      constexpr int UNIT = 16 / (int)sizeof(TY);
#pragma unroll
      for (int c = lane * UNIT; c < SLAB; c += 32 * UNIT)
        if (x.c0 + c < a.d) cp_async_16(to + c * (int)sizeof(TY), from + c);
    } else {
      // the 16-byte pieces that hold the slab, as they lie; of the last what is the row's
      const uintptr_t first = (uintptr_t)from & ~(uintptr_t)15;
      const uintptr_t end = (uintptr_t)(from + min(SLAB, a.d - x.c0));
      for (uintptr_t at = first + lane * 16; at < end; at += 512) {
        if (at < (uintptr_t)dY) {  // dY itself starts inside this piece
          for (uintptr_t b = (uintptr_t)dY; b < min(end, at + 16); b += sizeof(TY)) {
            const uint32_t sh = to + (uint32_t)(b - first);
            if constexpr (sizeof(TY) == 2)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(sh),
                           "h"(*reinterpret_cast<const unsigned short*>(b))
                           : "memory");
            else
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(sh),
                           "r"(*reinterpret_cast<const uint32_t*>(b))
                           : "memory");
          }
        } else {
          cp_async_16_of(to + (uint32_t)(at - first), reinterpret_cast<const void*>(at),
                         (int)min((uintptr_t)16, end - at));
        }
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Persistent warps: pieces and slabs in turn, BATCH rows' copies at a time and a ring of them
// under way, across pieces too. Then (where dW is overwritten) its rows that no token names.
template <typename TY, bool ODD>
__global__ void __launch_bounds__(SUM_THREADS)
    embedding_sum_kernel(const EmbedArgs a, const int2* __restrict__ pairs, int pieces,
                         int slabs) {
  extern __shared__ uint4 sum_places[];
  grid_dependents_go();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int RING = ring_groups<TY>();
  static_assert(GROUPS % RING == 0, "a piece's groups have the same places in every turn");
  const uint32_t ring = smem_u32(sum_places) + warp * ring_bytes<TY>();
  const long long items = (long long)pieces * slabs;
  const long long warps = (long long)gridDim.x * (SUM_THREADS / 32);
  long long item = (long long)blockIdx.x * (SUM_THREADS / 32) + warp;
  SumItem x = sum_item(a, pairs, item, items, slabs);
#pragma unroll
  for (int g = 0; g < RING - 1; ++g) fetch_rows<TY, ODD>(a, x, g, ring);
  for (; item < items; item += warps) {
    const SumItem y = sum_item(a, pairs, item + warps, items, slabs);
    float* part = a.part + (long long)x.piece * 2 * a.d;
    bool first = x.head;
    float acc[8] = {};
#pragma unroll 1
    for (int g = 0; g < GROUPS; ++g) {
      const int j0 = g * BATCH;
      __syncwarp();  // the place that is filled has been read
      if (g + RING - 1 < GROUPS)
        fetch_rows<TY, ODD>(a, x, g + RING - 1, ring);
      else
        fetch_rows<TY, ODD>(a, y, g + RING - 1 - GROUPS, ring);
      asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
      __syncwarp();  // others copied what this lane reads
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (j0 + j >= x.n) break;
        const uint32_t at = ring + (g % RING * BATCH + j) * place_bytes<TY>();
        float v[8];
        if constexpr (!ODD) {
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const uint32_t e = at + slab_column<ODD>(lane, k) * (int)sizeof(TY);
            if constexpr (sizeof(TY) == 2) {
              uint32_t w[2];
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                           : "=r"(w[0]), "=r"(w[1])
                           : "r"(e)
                           : "memory");
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                v[k + 2 * i] = __uint_as_float(w[i] << 16);
                v[k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
              }
            } else {
              const uint4 w = ld_shared_v4(e);
              v[k] = __uint_as_float(w.x), v[k + 1] = __uint_as_float(w.y);
              v[k + 2] = __uint_as_float(w.z), v[k + 3] = __uint_as_float(w.w);
            }
          }
        } else {
          const int t = __shfl_sync(0xffffffffu, x.pos, j0 + j);
          const TY* from = static_cast<const TY*>(a.dY) + (long long)t * a.d + x.c0;
          const uint32_t row = at + (uint32_t)((uintptr_t)from & 15);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t e = row + slab_column<ODD>(lane, k) * (int)sizeof(TY);
            if constexpr (sizeof(TY) == 2) {
              unsigned short h;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(e) : "memory");
              v[k] = __uint_as_float((uint32_t)h << 16);
            } else {
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[k]) : "r"(e) : "memory");
            }
          }
        }
        row_add(acc, acc, v);
        if (x.ends >> (j0 + j) & 1u) {
          const int id = __shfl_sync(0xffffffffu, x.key, j0 + j);
          put_sum<ODD>(a, id, first ? part : nullptr, x.c0, lane, acc);
          first = false;
          row_fill(acc, 0.f);
        }
      }
    }
    if (x.n > 0 && !(x.ends >> (x.n - 1) & 1u))  // first half: continued, second: begun here
      put_sum<ODD>(a, 0, part + (first ? 0 : a.d), x.c0, lane, acc);
    x = y;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!a.met) return;
  const long long fills = ((long long)a.V + FILL_ROWS - 1) / FILL_ROWS;
  long long f = (long long)blockIdx.x * (SUM_THREADS / 32) + warp;
  unsigned word = f < fills ? a.met[f * FILL_ROWS / 32] : 0u;
  for (; f < fills; f += warps) {
    const unsigned met = word >> (f * FILL_ROWS % 32);
    if (f + warps < fills) word = a.met[(f + warps) * FILL_ROWS / 32];
#pragma unroll 1
    for (int r = 0; r < FILL_ROWS; ++r) {
      const long long row = f * FILL_ROWS + r;
      if ((met >> r & 1u) || row >= a.V) continue;
      float* to = a.dW + row * a.d;
      if constexpr (ODD) {
        for (int c = lane; c < a.d; c += 32) to[c] = 0.f;
      } else {
        for (int c = lane * 4; c < a.d; c += 128)
          *reinterpret_cast<float4*>(to + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
}

// The sums that were begun in one piece and continued in others, in their order: a warp for a
// slab of columns of a piece that begins one. So its time goes by the longest id: of 32,768 tokens of
// d = 2880, 14 us where ids repeat as words do, 44 where one has a third of the places (a padding
// id that no mask leaves out: 341 pieces, 8 of them read at a time), 90 where it has them all.
template <int VEC>
__global__ void __launch_bounds__(EMBED_THREADS)
    embedding_join_kernel(const EmbedArgs a, const int2* __restrict__ pairs, int pieces,
                          int slabs) {
  grid_dependents_go();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * SORT_WARPS + (threadIdx.x >> 5);
  const int piece = (int)(item / slabs);
  if (piece >= pieces - 1) return;
  const int begin = piece * EMBED_PIECE, end = begin + EMBED_PIECE;  // < T: a piece follows
  const int id = pairs[end - 1].x, after = pairs[end].x, front = pairs[begin].x;
  const int before = begin > 0 ? pairs[begin - 1].x : -1;
  if (id >= a.V || after != id) return;
  if (front == id && before == id) return;  // it fills the piece, and was begun earlier
  const int c = ((int)(item - (long long)piece * slabs) * 32 + lane) * VEC;
  const bool col_ok = c < a.d;
  const float* part = a.part + (long long)piece * 2 * a.d + c;
  RowVec<float, VEC> r;
  float acc[VEC] = {}, v[VEC];
  if (col_ok) {
    r.load(part + a.d);
    r.get(acc);
  }
  // 32 pieces' first ids at a time: the first that is another's ends the sum
  for (int p0 = piece + 1; p0 < pieces; p0 += 32) {
    const int p = p0 + lane;
    const unsigned same =
        __ballot_sync(0xffffffffu, p < pieces && pairs[(long long)p * EMBED_PIECE].x == id);
    const int n = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
    for (int j0 = 0; j0 < n; j0 += BATCH) {
      RowVec<float, VEC> q[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (j0 + j < n && col_ok) q[j].load(a.part + (long long)(p0 + j0 + j) * 2 * a.d + c);
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (j0 + j < n && col_ok) {
          q[j].get(v);
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] += v[k];
        }
    }
    if (n < 32) break;
  }
  if (col_ok) hand_over<VEC>(a, id, c, acc);
}

int blocks_of(long long items, int per_block) {
  return (int)((items + per_block - 1) / per_block);
}

int sort_tile(int T) {  // a multiple of 32 for every warp
  const long long per = ((long long)T + EMBED_TILES - 1) / EMBED_TILES;
  const long long unit = SORT_WARPS * 32;
  return (int)std::max<long long>(EMBED_TILE_MIN, (per + unit - 1) / unit * unit);
}

template <typename TW, typename TY, int VEC>
cudaError_t forward(const EmbedArgs& a, cudaStream_t stream) {
  // slices of at most FORWARD_VECTORS a lane: a block's last warp ends soon after its first
  const int vectors = (a.d + 32 * VEC - 1) / (32 * VEC);
  const int per_slice = std::min(vectors, FORWARD_VECTORS) * 32 * VEC;
  const int slices = (a.d + per_slice - 1) / per_slice;
  const int check = a.status && a.T <= EMBED_CHECK ? 1 : 0;
  if (a.status && !check) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int), stream);
    if (e != cudaSuccess) return e;
  }
  const long long blocks = ((long long)a.T * slices + SORT_WARPS - 1) / SORT_WARPS + check;
  return launch_kernel_early("embedding_forward", embedding_forward_kernel<TW, TY, VEC>,
                             dim3((unsigned)blocks), dim3(EMBED_THREADS), 0, stream, a, slices,
                             per_slice, check);
}

// Pairs twice, totals, starts, the warps' counts.
constexpr int sort_smem_bytes(int share) {
  return 2 * share * 8 + 2 * DIGITS * 4 + CLUSTER_THREADS / 32 * DIGITS * 2;
}
static_assert(sort_smem_bytes(CLUSTER_SORTED / CLUSTER_BLOCKS) <= 216 * 1024, "shared memory");

// Blocks of the sort's cluster: 16 where the device can run that many together, else 8, which any
// can. Found once for a device; concurrent first calls find the same.
cudaError_t cluster_blocks(int dev, int* blocks) {
  static std::atomic<int> known[kMaxDevices] = {};
  if ((*blocks = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  auto kern = embedding_cluster_sort_kernel;
  constexpr int smem = sort_smem_bytes(CLUSTER_SORTED / CLUSTER_BLOCKS);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CLUSTER_MOST);
  cfg.blockDim = dim3(CLUSTER_THREADS);
  cfg.dynamicSmemBytes = sort_smem_bytes(CLUSTER_SORTED / CLUSTER_MOST);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CLUSTER_MOST;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  known[dev].store(*blocks = n > 0 ? CLUSTER_MOST : CLUSTER_BLOCKS, std::memory_order_release);
  return cudaSuccess;
}

template <typename TY, int VEC>
cudaError_t backward(const EmbedArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(a.status, 0, a.clear_bytes, stream);
  if (e != cudaSuccess) return e;
  const int2* pairs = a.pairs[0];
  int dev = 0, per_sm = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (a.T <= EMBED_RANKED) {
    e = launch_kernel_early("embedding_rank", embedding_rank_kernel,
                            dim3(blocks_of((long long)a.T * RANK_LANES, EMBED_THREADS)),
                            dim3(EMBED_THREADS), (size_t)((a.T + 3) / 4) * 16, stream, a);
    if (e != cudaSuccess) return e;
  } else if (a.T <= CLUSTER_SORTED) {
    int blocks = 0;
    if ((e = cluster_blocks(dev, &blocks)) != cudaSuccess) return e;
    const int unit = blocks * CLUSTER_THREADS;
    const int share = (a.T + unit - 1) / unit * CLUSTER_THREADS;
    e = launch_kernel_cluster("embedding_sort", embedding_cluster_sort_kernel, dim3(blocks),
                              dim3(CLUSTER_THREADS), (size_t)sort_smem_bytes(share), stream,
                              (unsigned)blocks, true, a, share, blocks);
    if (e != cudaSuccess) return e;
  } else {
    SortPass p{};
    p.tile = sort_tile(a.T);
    p.tiles = blocks_of(a.T, p.tile);
    for (int turn = 0; p.shift < 31 && (a.V >> p.shift); ++turn, p.shift += DIGIT_BITS) {
      p.out = a.pairs[turn & 1];
      e = launch_kernel_early("embedding_count", embedding_count_kernel, dim3(p.tiles),
                              dim3(EMBED_THREADS), 0, stream, a, p);
      if (e != cudaSuccess) return e;
      e = launch_kernel_early("embedding_place", embedding_place_kernel, dim3(p.tiles),
                              dim3(EMBED_THREADS), 0, stream, a, p);
      if (e != cudaSuccess) return e;
      pairs = p.in = p.out;
    }
  }
  const int pieces = blocks_of(a.T, EMBED_PIECE);
  const long long items = (long long)pieces * blocks_of(a.d, SLAB);
  const long long fills = a.accumulate ? 0 : ((long long)a.V + FILL_ROWS - 1) / FILL_ROWS;
  auto kern = embedding_sum_kernel<TY, VEC == 1>;
  constexpr int smem = SUM_THREADS / 32 * ring_bytes<TY>();
  static std::atomic<int> known[kMaxDevices] = {};  // blocks that an SM holds
  if ((per_sm = known[dev].load(std::memory_order_acquire)) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, SUM_THREADS, smem);
    if (e != cudaSuccess) return e;
    known[dev].store(per_sm = std::max(1, per_sm), std::memory_order_release);
  }
  const long long most = (std::max(items, fills) + SUM_THREADS / 32 - 1) / (SUM_THREADS / 32);
  e = launch_kernel_early("embedding_sum", kern,
                          dim3((unsigned)std::min<long long>(most, per_sm * num_sms)),
                          dim3(SUM_THREADS), (size_t)smem, stream, a, pairs, pieces,
                          blocks_of(a.d, SLAB));
  if (e != cudaSuccess || pieces < 2) return e;
  constexpr int JOIN = VEC == 1 ? 1 : 4;
  const int slabs = blocks_of(a.d, 32 * JOIN);
  return launch_kernel_early("embedding_join", embedding_join_kernel<JOIN>,
                             dim3((unsigned)(((long long)pieces * slabs + SORT_WARPS - 1) / SORT_WARPS)),
                             dim3(EMBED_THREADS), 0, stream, a, pairs, pieces, slabs);
}

}  // namespace

size_t embed_sort_bytes(int T) {
  if (T <= CLUSTER_SORTED) return 0;
  return (size_t)DIGITS * blocks_of(T, sort_tile(T)) * 4;
}

cudaError_t launch_embedding_forward(const EmbedArgs& a, bool table_bf16, bool rows_bf16,
                                     cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (a.vec) {
    if (table_bf16)
      return rows_bf16 ? forward<bf16, bf16, 8>(a, stream)
                       : forward<bf16, float, 8>(a, stream);
    return rows_bf16 ? forward<float, bf16, 8>(a, stream)
                     : forward<float, float, 8>(a, stream);
  }
  if (table_bf16)
    return rows_bf16 ? forward<bf16, bf16, 1>(a, stream)
                     : forward<bf16, float, 1>(a, stream);
  return rows_bf16 ? forward<float, bf16, 1>(a, stream)
                   : forward<float, float, 1>(a, stream);
}

cudaError_t launch_embedding_backward(const EmbedArgs& a, bool rows_bf16, int num_sms,
                                      cudaStream_t stream) {
  if (a.vec)
    return rows_bf16 ? backward<__nv_bfloat16, 8>(a, num_sms, stream)
                     : backward<float, 8>(a, num_sms, stream);
  return rows_bf16 ? backward<__nv_bfloat16, 1>(a, num_sms, stream)
                   : backward<float, 1>(a, num_sms, stream);
}

}  // namespace kdkl
