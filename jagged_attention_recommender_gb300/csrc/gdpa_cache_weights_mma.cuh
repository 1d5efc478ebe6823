// gdpa_cache_weights_mma.cuh -- pieces of the kernel of the stored keys' weight on
// the 5th-generation tensor cores.
#pragma once

#include "gdpa_cache_tile.cuh"
#include "gdpa_cache_weights.cuh"

namespace gdpa {

namespace ptx {

// 3-D tiled bulk tensor load global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrives on `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 consecutive 32-bit columns of the warp's 32 lanes, there when the call is
// over: the load and its wait in one, since a wait that names the registers
// again, to keep their uses behind it, has the compiler copy them.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// The rest of a wait for `bar` that was not over at once: one copy of it, since
// the roles of a kernel share the instruction caches.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort, int idle) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (idle) __nanosleep(100);
    if (idle ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// mbar_wait with its loop out of line ...
__device__ __forceinline__ bool mbar_wait_near(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort) {
  return mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_on(bar, parity, limit_ns, abort, 0);
}

// ... and for roles that are far ahead: a warp that waits sleeps between its
// looks, so that it takes no issue slots from those that compute.
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort) {
  return mbar_test_wait(bar, parity) || wait_on(bar, parity, limit_ns, abort, 1);
}

}  // namespace ptx

// A place in a ring of stages, and the parity of its present turn.
struct StageRing {
  uint32_t at = 0, turn = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++at == stages) at = 0, turn ^= 1;
  }
};

// What goes with a tile of 128 keys, by blocks of 16: the first one's row of the
// cache (-1: no page), the word with its scale's code; and earlier weights.
struct alignas(16) KeyNotes {
  int64_t row[8];
  uint32_t word[8];
  float old[128];
  __device__ __forceinline__ float scale(int key) const {  // its block's
    return sf_value(word[key >> 4] >> static_cast<int>((row[key >> 4] >> 4) & 3) * 8 & 0xff);
  }
};

// How many blocks the copy of a lane brings, of a tile's blocks that lie behind each
// other in a page (a bulk copy takes its warp about 75 cycles, whatever its size);
// 0 where another lane does, or where there is none.  `there`: a bit for each lane's block.
__device__ __forceinline__ int blocks_of_copy(const CacheWeightsParams& w, uint32_t there) {
  const int lane = threadIdx.x & 31, per = 1 << min(w.cache.lp - 4, 3);
  return (lane & (per - 1)) == 0 ? __popc(there >> lane & ((1u << per) - 1)) : 0;
}

// Brings the notes of one or two tiles, by a whole warp; lane i below 8 * tiles
// knows its block's row (the others -1) and its tile's stage.  `full` takes 9 arrivals:
// eight that stand for asynchronous copies alone, and one that releases the rows of all
// eight lanes, which the warp's barrier in front of it puts before it.
__device__ __forceinline__ void bring_notes(const CacheWeightsParams& w, KeyNotes& note, uint64_t* full, int64_t row, int tiles) {
  const int lane = threadIdx.x & 31, block = lane & 7;
  const bool mine = lane < 8 * tiles;
  const int64_t sf_bytes = static_cast<int64_t>(w.cache.num_pages) * w.cache.H << (w.cache.lp - 4);
  if (mine) {
    note.row[block] = row;
    if (row >= 0) {
      const int64_t word = (row >> 4) & ~(int64_t)3;
      split::cp_async4(ptx::smem_u32(&note.word[block]), w.cache.k_sf + word,
                       static_cast<int>(min((int64_t)4, sf_bytes - word)));
    }
    ptx::copies_arrive(full);
  }
  __syncwarp();
  const uint32_t there = w.w_in ? __ballot_sync(0xffffffffu, row >= 0) : 0;
  if (mine && block == 0) ptx::mbar_arrive_expect_tx(full, __popc(there >> lane & 0xff) * 64);
  __syncwarp();
  if (const int n = blocks_of_copy(w, there)) ptx::bulk_load(ptx::smem_u32(&note.old[block * 16]), w.w_in + row, n * 64, full);
}

// Brings the codes of one or two tiles, likewise.  (A block that is not there
// keeps what the stage held: no other key's score depends on it.)
template <int D>
__device__ __forceinline__ void bring_codes(const CacheWeightsParams& w, uint32_t raw, uint64_t* full, int64_t row, int tiles) {
  const int lane = threadIdx.x & 31, block = lane & 7;
  const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
  if (lane < 8 * tiles && block == 0) ptx::mbar_arrive_expect_tx(full, __popc(there >> lane & 0xff) * 16 * D);
  __syncwarp();
  if (const int n = blocks_of_copy(w, there)) ptx::bulk_load(raw + block * 16 * D, w.cache.k + row * D, n * 16 * D, full);
}

// Waits for the last turns of `stages` stages of which `count` were filled, `at`
// being the next one's place: no copy may land behind a CTA's end.
__device__ __forceinline__ void drain_stages(uint64_t* full, StageRing at, uint32_t stages, uint32_t count) {
  for (uint32_t i = 0; i < min(count, stages); ++i) {
    const int never = 0;
    if (at.at == 0) at.turn ^= 1;
    at.at = (at.at == 0 ? stages : at.at) - 1;
    ptx::mbar_wait(&full[at.at], at.turn, 100000000ull, &never);
  }
}

}  // namespace gdpa
