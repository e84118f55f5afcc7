// Streaming products for few tokens (skinny.hip, moe.hip): each wavefront runs
// its own stream of slabs from global memory through a ring in LDS, with no
// barrier, so that the loads of the slabs ahead are always in flight.
//
// A slab is 128 bytes of K of 16 rows, of weights or of tokens, copied by buffer
// loads that write LDS: 8 rows of 128 bytes (whole cache lines) an instruction, no
// registers held.  Row r keeps
// chunk c (16 bytes) at position c ^ (r / 2 % 8), so the fragment reads are free
// of bank conflicts; a chunk past the end of K is read out of the buffer's
// range, which gives zeros.
//
// This pattern alone, without the tokens and the products, streams 235 MB of
// 8 KB rows in 38.4 us (6.1 TB/s); the best plain register stream of the same
// bytes takes 34.9 (6.7 TB/s).
#pragma once

#include "ffn_tile.h"
#include "lanes.h"

namespace dyra {

// This lane's part of the copies of 16 rows: row 8 q + lane / 8, q = 0, 1, and
// the chunk (byte offset) that the swizzle puts at its place.
__device__ __forceinline__ int slab_row(int q) { return 8 * q + ((threadIdx.x & 63) >> 3); }
__device__ __forceinline__ uint32_t slab_chunk(int q) {
    const int lane = threadIdx.x & 63;
    return 16u * (((lane & 7) ^ (lane >> 4)) ^ (4 * q));
}
// Where 16 rows lie: the buffer of rows 8 q .. and this lane's offset in it.
struct SlabRows {
    __amdgpu_buffer_rsrc_t buf[2];
    uint32_t off[2];
};

// Fragments of one slab: 128 bytes of K are STEPS steps of 32 elements.
template <typename E> struct SlabFrag {
    static constexpr int STEPS = 128 / (32 * (int)sizeof(E));
    typename Frag<E>::type f[STEPS];
};
__device__ __forceinline__ f32x4 slab_product(f32x4 acc, const SlabFrag<bf16> &w, const SlabFrag<bf16> &x) {
    return mma32(mma32(acc, w.f[0], x.f[0]), w.f[1], x.f[1]);
}
__device__ __forceinline__ f32x4 slab_product(f32x4 acc, const SlabFrag<float> &w, const SlabFrag<float> &x) {
    return mma32(acc, w.f[0], x.f[0]);
}
// The fragments of row `lane % ROWS` of a slab in LDS.
template <typename E, int ROWS> __device__ __forceinline__ SlabFrag<E> slab_read(const char *slab) {
    const int lane = threadIdx.x & 63, r16 = lane & (ROWS - 1), g = lane >> 4, sw = r16 >> 1;
    const char *p = slab + r16 * 128;
    SlabFrag<E> r;
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r.f[h] = *reinterpret_cast<const bf16x8 *>(p + (((4 * h + g) ^ sw) << 4));
    } else {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(p + (((2 * g) ^ sw) << 4));
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(p + (((2 * g + 1) ^ sw) << 4));
        r.f[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}
constexpr int kRingBytes = 16384;  // of LDS for each wavefront's ring

// One wavefront's ring of slabs: WROWS rows of weights and XROWS of tokens (16
// or 8 each, XROWS also 0; with 8, rows 8 .. 15 of the fragments repeat them).
template <typename E, int WROWS, int XROWS> struct SlabRing {
    static constexpr int WBYTES = 128 * WROWS, SLAB = WBYTES + 128 * XROWS;
    static constexpr int DEPTH = kRingBytes / SLAB, COPIES = (WROWS + XROWS) / 8;
    char *ring;            // this wavefront's kRingBytes of LDS
    int ahead = 0;             // slabs issued and not consumed
    int put = 0, got = 0;      // places of the next slab to issue and to consume

    template <int ROWS> __device__ __forceinline__ void copy(const SlabRows &r, uint32_t k, int left, char *dst) {
#pragma unroll
        for (int q = 0; q < ROWS / 8; ++q)
            buffer_to_lds16(r.buf[q], (int)slab_chunk(q) < left ? r.off[q] : kOutside, k, dst + 1024 * q);
    }
    // Copies one slab at byte `k` of the rows; `left` bytes of the rows are left.
    __device__ __forceinline__ void issue(const SlabRows &w, uint32_t k, int left) { issue(w, w, k, left); }
    __device__ __forceinline__ void issue(const SlabRows &w, const SlabRows &x, uint32_t k, int left) {
        char *dst = ring + put * SLAB;
        copy<WROWS>(w, k, left, dst);
        if constexpr (XROWS > 0) copy<XROWS>(x, k, left, dst + WBYTES);
        put = put + 1 == DEPTH ? 0 : put + 1;
        ++ahead;
    }
    // Waits for the oldest slab and reads its fragments; its place is then free.
    __device__ __forceinline__ void take(SlabFrag<E> &w) {
        SlabFrag<E> none;
        take(w, none);
    }
    __device__ __forceinline__ void take(SlabFrag<E> &w, SlabFrag<E> &x) {
        // (stores issued in between only make the wait stricter)
        if (ahead == DEPTH) wait_vmcnt<(DEPTH - 1) * COPIES>();
        else wait_vmcnt<0>();
        // the copies write LDS behind the compiler's back: no read may move above the wait
        asm volatile("" ::: "memory");
        const char *slab = ring + got * SLAB;
        w = slab_read<E, WROWS>(slab);
        if constexpr (XROWS > 0) x = slab_read<E, XROWS>(slab + WBYTES);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the fragments are in registers
        asm volatile("" ::: "memory");
        got = got + 1 == DEPTH ? 0 : got + 1;
        --ahead;
    }
};

// The products of a sequence of positions: position p multiplies 16 weight rows
// with one or two blocks of 16 tokens.  The workgroup's eight wavefronts split K,
// each running its part of every position through one ring without a break.  The
// tokens' fragments come through the same ring, ahead of the weights that they
// meet, and stay in registers (SLABS slabs of K, TB blocks) until a position with
// other tokens; where a wavefront has more than SLABS slabs they pass anew for
// every position.  The wavefronts' sums meet in LDS, added in their order.
//
// A Positions type gives: count; weights(p, SlabRows &); new_tokens(p), whether
// p's differ from p - 1's; tokens(p, SlabRows (&)[TB]); blocks(p), 1 .. TB;
// finish(p, sums, thread), called by all threads with sums of 16 tokens x 16
// rows per block and wavefront.  All but finish must give wave-uniform answers.
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kBlockSums = 256;  // floats of a block's sums: token, then row
// The sum over the wavefronts of row r of a block's token i.
__device__ __forceinline__ float joined(const float *block, int i, int r) {
    float z = 0.f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) z += block[v * kBlockSums + i * 16 + r];
    return z;
}
// One variable, so that the compiler sees no separate objects whose accesses it
// would hold back for copies still in flight.
template <int TB> struct StreamLds {
    char ring[kWaves * kRingBytes];
    float sums[2][kWaves][kBlockSums];
};

template <typename E, int SLABS, int TB, class Positions>
__device__ __forceinline__ void stream_products(const Positions &P, int row_bytes, StreamLds<TB> &lds) {
    static_assert(TB == 1 || TB == 2, "token blocks");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slabs = (row_bytes + 127) / 128, per = (slabs + kWaves - 1) / kWaves;
    const int s0 = min(slabs, wave * per), s1 = min(slabs, s0 + per);  // this wavefront's slabs
    const bool parts = s1 - s0 > SLABS;  // the tokens do not stay

    // the stream: position, slabs from `in_base` on; tokens first where they are due
    SlabRing<E, 16, 0> ring{lds.ring + wave * kRingBytes};
    SlabRows w, x[TB];
    int in_pos = s0 == s1 ? P.count : 0, in_base = s0, in_slab = 0, in_block = 0, in_blocks = 0;
    auto aim = [&]() __attribute__((always_inline)) {
        P.weights(in_pos, w);
        if (parts || P.new_tokens(in_pos)) {
            P.tokens(in_pos, x);
            in_blocks = P.blocks(in_pos);
        }
    };
    auto ahead = [&]() __attribute__((always_inline)) {
        if (in_pos == P.count) return;
        const int n = min(SLABS, s1 - in_base), s = in_base + in_slab;
        const uint32_t k = 128u * (uint32_t)s;
        const int left = row_bytes - 128 * s;
        const bool last = ++in_slab == n;
        if (last) in_slab = 0;
        if (in_block < in_blocks) {
            ring.issue(TB == 2 && in_block == 1 ? x[TB - 1] : x[0], k, left);
            if (last) ++in_block;
        } else {
            ring.issue(w, k, left);
            if (last) {
                in_block = 0;
                in_base += SLABS;
                if (in_base >= s1) {
                    in_base = s0;
                    in_blocks = 0;
                    if (++in_pos < P.count) aim();
                }
            }
        }
    };
    if (in_pos < P.count) aim();
#pragma unroll 1
    for (int q = 0; q < ring.DEPTH; ++q) ahead();

    SlabFrag<E> fx[TB][SLABS];
    int set = 1, begin = 0;
    bool was_two = false;
    for (int p = 0; p < P.count; ++p) {
        const bool two = TB == 2 && P.blocks(p) == 2;
        f32x4 acc[TB] = {};
        for (int base = s0; base < s1; base += SLABS) {
            if (parts || P.new_tokens(p)) {
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    if (t == 0 || two) unroll_seq<SLABS>([&](auto j) __attribute__((always_inline)) {
                        if (base + (int)j >= s1) return;
                        ring.take(fx[t][j]);
                        ahead();
                    });
            }
            unroll_seq<SLABS>([&](auto j) __attribute__((always_inline)) {
                if (base + (int)j >= s1) return;
                SlabFrag<E> fw;
                ring.take(fw);
                ahead();
                acc[0] = slab_product(acc[0], fw, fx[0][j]);
                if (TB == 2 && two) acc[TB - 1] = slab_product(acc[TB - 1], fw, fx[TB - 1][j]);
            });
        }
        // One block takes one of the two sets of sums, in turn, so that one is read
        // while the next position's is written; two take both, once the position
        // before has been read.
        if (two || was_two) __syncthreads();
        was_two = two;
        set = two ? 0 : set ^ 1;
        float *mine = &lds.sums[set][wave][(lane & 15) * 16 + 4 * (lane >> 4)];
        *reinterpret_cast<f32x4 *>(mine) = acc[0];
        if (two) *reinterpret_cast<f32x4 *>(mine + kWaves * kBlockSums) = acc[TB - 1];
        __syncthreads();
        P.finish(p, &lds.sums[set][0][0], (tid - begin) & (kThreads - 1));
        begin += Positions::kFinishers;  // other wavefronts finish the next one
    }
}

}  // namespace dyra
