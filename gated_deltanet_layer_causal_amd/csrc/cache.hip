// Upkeep of a cache of states: copying, taking, counting and compacting
// slots.  What is decided (which slots are free, who moves where) is decided
// by one workgroup that leaves a list of moves in the workspace; a second
// launch carries the moves out, HBM-bound, over the whole chip.
#include "chunk_stream.h"
#include "launch.h"

namespace gdn {

constexpr int PLAN_THREADS = 1024;
constexpr int PIECE = 4096;    // bytes one workgroup copies at a time: 16 a thread

// Exclusive rank of this thread's flag among the workgroup's, in thread
// order; *total receives the count.  Ends with a barrier.
__device__ __forceinline__ int flag_rank(bool flag, int* wsum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned long long m = __ballot(flag);
  if (lane == 0) wsum[wave] = __popcll(m);
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < PLAN_THREADS / 64; ++w) {
    if (w < wave) before += wsum[w];
    total += wsum[w];
  }
  __syncthreads();
  return before + __popcll(m & ((1ull << lane) - 1));
}

// The move list: moves[0] = count, then `room` sources, then `room` targets.
__device__ __forceinline__ int32_t* list_src(int32_t* moves) { return moves + 4; }
__device__ __forceinline__ int32_t* list_dst(int32_t* moves, int64_t room) { return moves + 4 + room; }

// Fork: the r-th valid request takes the r-th free slot, so the list of free
// slots in order is the list of the moves' targets.
__global__ void __launch_bounds__(PLAN_THREADS) fork_plan_kernel(
    int32_t* __restrict__ refs, int n_slots, const int32_t* src, int n, int32_t* dst,
    int32_t* __restrict__ moves, int64_t room) {
  __shared__ int wsum[PLAN_THREADS / 64];
  const int tid = threadIdx.x;
  int32_t *msrc = list_src(moves), *mdst = list_dst(moves, room);
  int n_free = 0;
  for (int64_t base = 0; base < n_slots && n_free < n; base += PLAN_THREADS) {
    const int64_t i = base + tid;
    const bool f = i < n_slots && refs[i] <= 0;
    int total;
    const int r = n_free + flag_rank(f, wsum, total);
    if (f && r < n) mdst[r] = (int32_t)i;
    n_free += total;
  }
  __syncthreads();
  int asked = 0;
  for (int64_t base = 0; base < n; base += PLAN_THREADS) {
    const int64_t i = base + tid;
    const int s = i < n ? src[i] : -2;
    const bool valid = s == -1 || (s >= 0 && s < n_slots && refs[s] > 0);
    int total;
    const int r = asked + flag_rank(valid, wsum, total);
    if (i < n) {
      const bool given = valid && r < n_free;
      if (given) msrc[r] = s;
      dst[i] = given ? mdst[r] : -1;
    }
    asked += total;
  }
  const int count = asked < n_free ? asked : n_free;
  __syncthreads();
  for (int r = tid; r < count; r += PLAN_THREADS) refs[mdst[r]] = 1;
  if (tid == 0) moves[0] = count;
}

// Compact: with L live slots, the m-th live slot at or behind L moves into
// the m-th free slot before L (there are as many of the one as of the other).
__global__ void __launch_bounds__(PLAN_THREADS) compact_plan_kernel(
    int32_t* __restrict__ refs, int n_slots, int32_t* __restrict__ remap,
    int32_t* __restrict__ table, int n_table, int32_t* __restrict__ moves, int64_t room) {
  __shared__ int wsum[PLAN_THREADS / 64];
  const int tid = threadIdx.x;
  int32_t *msrc = list_src(moves), *mdst = list_dst(moves, room);
  int L = 0;
  for (int64_t base = 0; base < n_slots; base += PLAN_THREADS) {
    const int64_t i = base + tid;
    int total;
    flag_rank(i < n_slots && refs[i] > 0, wsum, total);
    L += total;
  }
  int holes = 0, movers = 0;
  for (int64_t base = 0; base < n_slots; base += PLAN_THREADS) {
    const int64_t i = base + tid;
    const bool live = i < n_slots && refs[i] > 0;
    const bool hole = i < L && !live, mover = live && i >= L;
    int th, tm;
    const int rh = holes + flag_rank(hole, wsum, th);
    const int rm = movers + flag_rank(mover, wsum, tm);
    if (hole) mdst[rh] = (int32_t)i;
    if (mover) msrc[rm] = (int32_t)i;
    if (i < n_slots && !mover) remap[i] = live ? (int32_t)i : -1;
    holes += th;
    movers += tm;
  }
  __syncthreads();
  for (int m = tid; m < movers; m += PLAN_THREADS) {
    const int s = msrc[m], d = mdst[m];
    remap[s] = d;
    refs[d] = refs[s];
    refs[s] = 0;
  }
  if (tid == 0) moves[0] = movers;
  __syncthreads();
  for (int64_t i = tid; i < n_table; i += PLAN_THREADS) {
    const int s = table[i];
    if (s >= 0 && s < n_slots) table[i] = remap[s];
  }
}

// One piece of one slot's copy; without a source (nullptr) the word `fill`
// throughout.  One 16-byte word a thread in workgroups that follow each other
// through memory, non-temporal and written through: the fewer bytes are under
// way at once, the more of them share DRAM pages (49 slots of 9.6 MB: 171 us
// with 64 bytes a thread and plain accesses, 156 us with 16 and non-temporal,
// 151 us written through as well).
__device__ __forceinline__ void copy_piece(const char* src, uint32_t fill, char* dst, int64_t at,
                                           int64_t bytes) {
  const uint32_t left = bytes - at < PIECE ? (uint32_t)(bytes - at) : PIECE, o = threadIdx.x * 16;
  u32x4 v = {fill, fill, fill, fill};
  if (src)   // past the slot's end: reads zero, stores nothing
    v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buffer_of(src + at, left), o, 0, CACHE_NT));
  __builtin_amdgcn_raw_buffer_store_b128(v, buffer_of(dst + at, left), o, 0, CACHE_NT | CACHE_SC1);
}

__global__ void __launch_bounds__(256) cache_move_kernel(char* base, int64_t stride,
                                                         const int32_t* __restrict__ moves,
                                                         int64_t room) {
  const int64_t pieces = (stride + PIECE - 1) / PIECE, total = moves[0] * pieces;
  const int32_t *msrc = moves + 4, *mdst = moves + 4 + room;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t m = w / pieces;
    const int s = __builtin_amdgcn_readfirstlane(msrc[m]), d = __builtin_amdgcn_readfirstlane(mdst[m]);
    copy_piece(s < 0 ? nullptr : base + s * stride, 0, base + d * stride, (w - m * pieces) * PIECE, stride);
  }
}

__global__ void __launch_bounds__(256) cache_copy_kernel(const char* src, int64_t src_stride,
                                                         int n_src, const int32_t* src_idx,
                                                         char* dst, int64_t dst_stride, int n_dst,
                                                         const int32_t* dst_idx, int64_t bytes,
                                                         int n) {
  const int64_t pieces = (bytes + PIECE - 1) / PIECE, total = n * pieces;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t m = w / pieces;
    const int s = __builtin_amdgcn_readfirstlane(src_idx ? src_idx[m] : (int)m);
    const int d = __builtin_amdgcn_readfirstlane(dst_idx ? dst_idx[m] : (int)m);
    if (d < 0 || d >= n_dst) continue;
    // a source outside the cache leaves all bits set: NaN in every storage type
    copy_piece(s < 0 || s >= n_src ? nullptr : src + s * src_stride, s < 0 ? 0 : ~0u,
               dst + d * dst_stride, (w - m * pieces) * PIECE, bytes);
  }
}

// Counts are whole numbers and each change is a single compare-and-swap that
// depends on the count alone, so the order does not matter.
__global__ void __launch_bounds__(256) cache_count_kernel(int32_t* refs, int n_slots,
                                                          const int32_t* __restrict__ slots, int n,
                                                          int delta) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int s = slots[i];
  if (s < 0 || s >= n_slots) return;
  int32_t have = refs[s];
  while (have > 0 && !(delta > 0 && have == 0x7fffffff)) {   // free slots, and a full count, stay
    const int32_t was = atomicCAS(&refs[s], have, have + delta);
    if (was == have) break;
    have = was;
  }
}

// Workgroups for n slots: one a piece (1 GiB: 6.9 TB/s; 6.1 TB/s where each
// of 65536 workgroups takes four), up to `most`, which then take several.
static unsigned copy_grid(int64_t n, int64_t bytes, int64_t most = 1 << 22) {
  const int64_t total = n * ((bytes + PIECE - 1) / PIECE);
  return (unsigned)(total < most ? total : most);
}

hipError_t launch_cache_copy(const void* src, int64_t src_stride, int32_t n_src,
                             const int32_t* src_idx, void* dst, int64_t dst_stride, int32_t n_dst,
                             const int32_t* dst_idx, int64_t bytes, int32_t n, hipStream_t st) {
  if (n == 0 || bytes == 0) return hipSuccess;
  hipLaunchKernelGGL(cache_copy_kernel, dim3(copy_grid(n, bytes)), dim3(256), 0, st,
                     (const char*)src, src_stride, n_src, src_idx, (char*)dst, dst_stride, n_dst,
                     dst_idx, bytes, n);
  return hipGetLastError();
}

hipError_t launch_cache_fork(void* base, int64_t stride, int32_t n_slots, int32_t* refs,
                             const int32_t* src, int32_t n, int32_t* dst, void* ws,
                             hipStream_t st) {
  if (n == 0) return hipSuccess;
  const int64_t room = cache_room(n_slots);
  hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, refs, n_slots, src, n,
                     dst, (int32_t*)ws, room);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int32_t most = n < n_slots ? n : n_slots;
  hipLaunchKernelGGL(cache_move_kernel, dim3(copy_grid(most, stride)), dim3(256), 0, st,
                     (char*)base, stride, (const int32_t*)ws, room);
  return hipGetLastError();
}

hipError_t launch_cache_count(int32_t* refs, int32_t n_slots, const int32_t* slots, int32_t n,
                              int delta, hipStream_t st) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(cache_count_kernel, dim3((unsigned)((n + 255LL) / 256)), dim3(256), 0, st,
                     refs, n_slots, slots, n, delta);
  return hipGetLastError();
}

hipError_t launch_cache_compact(void* base, int64_t stride, int32_t n_slots, int32_t* refs,
                                int32_t* remap, int32_t* table, int32_t n_table, void* ws,
                                hipStream_t st) {
  const int64_t room = cache_room(n_slots);
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, refs, n_slots, remap,
                     table, n_table, (int32_t*)ws, room);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || n_slots < 2) return e;
  // up to half of the slots move, usually far fewer: 60 of up to 100 slots of
  // 6.4 MB take 120 us with 131072 workgroups, 126 us with one for every
  // piece that could have to move
  hipLaunchKernelGGL(cache_move_kernel, dim3(copy_grid(n_slots / 2, stride, 1 << 17)), dim3(256), 0, st,
                     (char*)base, stride, (const int32_t*)ws, room);
  return hipGetLastError();
}

}  // namespace gdn
