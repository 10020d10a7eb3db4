// tc_device.cuh -- what the tensor-core kernels share: mbarrier waits, TMA
// loads, descriptors, TMEM reads, the persistent tile order and the host's
// tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "mx_device.cuh"

namespace mxnorm {
namespace tc {

constexpr unsigned long long kWaitNs = 2000000000ull;  // limit of every mbarrier wait, drills apart

__device__ __forceinline__ uint32_t saddr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ unsigned long long gtimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// A waiting thread sleeps in try_wait until the phase completes or this
// hint runs out, instead of spinning: the eight epilogue warps wait through
// every tile's main loop, and spinning cost issue slots and power (8.7 %
// slower at the power cap, about 3 % in short runs).  The single-thread
// roles sleep too: letting them spin measured 11 % slower.
constexpr uint32_t kSuspendHintNs = 1000000u;

// CLUSTER: for arrivals of the peer CTA's threads.  Relaxed: the tcgen05
// fences (arrive_remote) or acquire_shared_cluster (arrive_remote_release)
// order what lies around it.
template <bool CLUSTER = false>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
  return ok != 0u;
}

// Bounded wait (limit_ns by %globaltimer); false (and bit 0 of *error set) on
// timeout.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, unsigned int* error,
                                             unsigned long long limit_ns = kWaitNs) {
  if (try_wait<CLUSTER>(bar, parity)) return true;
  const unsigned long long t0 = gtimer();
  while (!try_wait<CLUSTER>(bar, parity)) {
    if (gtimer() - t0 > limit_ns) {
      atomicOr(error, 1u);
      return false;
    }
  }
  return true;
}

// One lane of a converged warp, the same one every time.  A role whose whole
// warp runs its loop and whose elected lane alone issues keeps addresses and
// descriptors in uniform registers, which the tcgen05 and TMA instructions
// read; under a branch on the lane number each operand moves there first.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}

// The wait of a whole warp: true in every lane, or false in every lane.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, unsigned int* error,
                                          unsigned long long limit_ns = kWaitNs) {
  return __all_sync(0xFFFFFFFFu, wait_bounded<CLUSTER>(bar, parity, error, limit_ns));
}

// A walk over a ring of DEPTH slots: slot and phase parity (a 64-bit stage
// count with its divisions costs more than the rest of a role's loop).
template <int DEPTH>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  bool first = true;  // first round: the slots are free
  __device__ __forceinline__ void next() {
    if (++s == DEPTH) {
      s = 0;
      phase ^= 1u;
      first = false;
    }
  }
  // Parity of slot j's last fill; false if it was never filled.
  __device__ __forceinline__ bool last(int j, uint32_t& ph) const {
    ph = j < s ? phase : phase ^ 1u;
    return j < s || !first;
  }
};

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrive on an mbarrier of either CTA, once TMEM has been read: the
// accumulators' hand-back, after tcgen05.wait::ld, tcgen05.fence::before_thread_sync
// and a __syncwarp.  All that the waiter's MMAs need ordered is that tcgen05
// work, which the fences at both ends order, so the arrival itself is relaxed
// (at cluster scope: the waiter may be in the other CTA).  A release here,
// which waits for the epilogue's global stores, costs microseconds per arrival.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Arrive on an mbarrier of either CTA, handing over what this warp wrote to
// shared memory with ordinary stores (each lane's fence.proxy.async and a
// __syncwarp before it; at the other end try_wait<true>, then
// acquire_shared_cluster).  The writes are made in one CTA and read by MMAs
// that the other issues, so release and acquire have cluster scope; they are
// restricted to shared memory, since a full release and acquire, which order
// global memory too, took 0.4 us a stage (the weight gradient at 4096 x 2048 x
// 2048: 54.6 us, 28.6 restricted).
__device__ __forceinline__ void arrive_remote_release(uint32_t cluster_addr) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  arrive_remote(cluster_addr);
}
__device__ __forceinline__ void acquire_shared_cluster() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// All threads of both CTAs (per-thread form: callers may arrive diverged).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// K-major operand tile with 128-byte swizzle: 8-row atoms of 1024 bytes,
// leading offset unused, stride 1024 bytes, descriptor version 1.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// A 512-byte scale atom as a plain 32-row x 16-byte matrix (8-row groups
// 128 bytes apart) for tcgen05.cp.
__device__ __forceinline__ uint64_t desc_atom(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// 2-D tiled TMA load into this CTA's shared memory, completing on an
// mbarrier of either CTA of the pair (bar: a shared::cluster address), so
// the peer's loads count towards the leader's stage barrier directly.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// Persistent tile order: groups of kGroupM 256-row tiles walk the column
// tiles together (row tile fastest inside a group), so the pairs running at
// one time share both their x and w tiles in L2.
constexpr int kGroupM = 16;
__device__ __forceinline__ void tile_coords(int64_t tile, int64_t num_m, int num_n, int64_t& mt, int& nt) {
  const int64_t per_group = (int64_t)kGroupM * num_n;
  const int64_t g = tile / per_group;
  const int64_t in = tile - g * per_group;
  const int64_t rows_here = min((int64_t)kGroupM, num_m - g * kGroupM);
  mt = g * kGroupM + in % rows_here;
  nt = (int)(in / rows_here);
}

// 32 bytes of an output tile, as one store (V8: the address is 32-byte
// aligned) or two.  They bypass L1: lanes store rows far apart, and lines
// allocated for them cost the loads and copies beside them (1024 x 4096 x 4096
// of the weight gradient: 33.1 us, 29.7 without allocation; the NVFP4 product
// at 4096 x 4096 x 4096 29.6 and 29.0).
template <bool V8>
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  if constexpr (V8) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(static_cast<uint32_t*>(dst) + i),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3])
                   : "memory");
  }
}

// One lane's 128 consecutive bf16 outputs (64 packed words) to global
// memory: 32-byte stores (whole sectors) when the row start allows, else
// 16-byte ones.
template <bool kV8>
__device__ __forceinline__ void store_row128(uint16_t* dst, const uint32_t (&o)[64]) {
#pragma unroll
  for (int q = 0; q < 64; q += 8) {
    if constexpr (kV8) {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 2 * q), "r"(o[q]), "r"(o[q + 1]),
                   "r"(o[q + 2]), "r"(o[q + 3]), "r"(o[q + 4]), "r"(o[q + 5]), "r"(o[q + 6]), "r"(o[q + 7])
                   : "memory");
    } else {
      asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(dst + 2 * q), "r"(o[q]), "r"(o[q + 1]), "r"(o[q + 2]),
                   "r"(o[q + 3])
                   : "memory");
      asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(dst + 2 * q + 8), "r"(o[q + 4]), "r"(o[q + 5]),
                   "r"(o[q + 6]), "r"(o[q + 7])
                   : "memory");
    }
  }
}

// 64 TMEM columns of this warp's 32 lanes (two 32-column loads, completed
// by the caller's tcgen05.wait::ld).
__device__ __forceinline__ void tmem_load64(uint32_t taddr, uint32_t (&v)[64]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t* w = v + 32 * q;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]), "=r"(w[8]),
          "=r"(w[9]), "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]), "=r"(w[14]), "=r"(w[15]), "=r"(w[16]),
          "=r"(w[17]), "=r"(w[18]), "=r"(w[19]), "=r"(w[20]), "=r"(w[21]), "=r"(w[22]), "=r"(w[23]), "=r"(w[24]),
          "=r"(w[25]), "=r"(w[26]), "=r"(w[27]), "=r"(w[28]), "=r"(w[29]), "=r"(w[30]), "=r"(w[31])
        : "r"(taddr + (uint32_t)(32 * q)));
  }
}

// v * r in fp32 (IEEE products), rounded to bf16 and packed in pairs.
__device__ __forceinline__ void scale_pack64(const uint32_t (&v)[64], float r, uint32_t* o) {
  const unsigned long long rr = f2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), rr), lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// --------------------------------------------------------------- host side
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace tc
}  // namespace mxnorm
