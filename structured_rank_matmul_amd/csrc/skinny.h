// Streaming products for few tokens (skinny.hip, moe.hip): each wavefront runs
// its own stream of slabs from global memory through a ring in LDS, with no
// barrier, so that the loads of the slabs ahead are always in flight.
//
// A slab is 128 bytes of K of 16 rows, of weights or of tokens, copied by buffer
// loads that write LDS: 8 rows of 128 bytes (whole cache lines) an instruction, no
// registers held.  Row r keeps
// chunk c (16 bytes) at position c ^ r % 8; a chunk past the end of K is read out of
// the buffer's range, which gives zeros.  A 16-byte LDS read serves 16 lanes at a
// time, lanes 0 .. 3, 12 .. 15 and 20 .. 27 (of rows 0 .. 3, 12 .. 15 and 4 .. 11, two
// chunks) first: these positions fall on distinct banks, of 16 rows and of 8.  The
// conflicts that the counters show in skinny_kernel, skinny_ring_kernel and
// moe_up_kernel (15 to 43 % of LDS cycles) are those of the wavefronts' sums, which
// are written 16 bytes a lane.
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
__device__ __forceinline__ uint32_t slab_chunk() {
    const int lane = threadIdx.x & 63;
    return 16u * ((lane & 7) ^ (lane >> 3));
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
    const int lane = threadIdx.x & 63, r16 = lane & (ROWS - 1), g = lane >> 4, sw = r16 & 7;
    const char *p = slab + r16 * 128;
    SlabFrag<E> r;
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r.f[h] = *reinterpret_cast<const bf16x8 *>(p + (((4 * h + g) ^ sw) << 4));
    } else {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(p + ((g ^ sw) << 4));
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(p + (((4 + g) ^ sw) << 4));
        r.f[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}
// The same fragments from global memory: `row` this lane's row's offset in the
// buffer (kOutside: zeros), `k` the slab's first byte, `left` the bytes of the rows
// from there on.
template <typename E> __device__ __forceinline__ SlabFrag<E> slab_load(__amdgpu_buffer_rsrc_t buf, uint32_t row, uint32_t k,
                                                                      int left) {
    const uint32_t g = (threadIdx.x & 63) >> 4;
    SlabFrag<E> r;
    auto chunk = [&](uint32_t c) -> u32x4 {
        return __builtin_amdgcn_raw_buffer_load_b128(buf, (int)(16 * c) < left ? row + 16 * c : kOutside, (int)k, 0);
    };
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r.f[h] = __builtin_bit_cast(bf16x8, chunk(4 * h + g));
    } else {
        const f32x4 lo = __builtin_bit_cast(f32x4, chunk(g)), hi = __builtin_bit_cast(f32x4, chunk(4 + g));
        r.f[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}

constexpr int kRingBytes = 16384;  // of LDS for each wavefront's ring

// One wavefront's ring of slabs, always full: DEPTH slabs are issued at first and
// one more after each is taken, past the end of the stream slabs of nothing (no
// byte left: zeros, no memory is read), so that one wait fits every take.  The
// copies left over have to land before the workgroup ends.  WROWS rows of
// weights and XROWS of tokens a slab (16 or 8 each, XROWS also 0 or 32; with 8, rows
// 8 .. 15 of the fragments repeat them, with 32 there are two fragments of 16).  The
// tokens' rows may lie anywhere: their slab is at byte `kx` of them.
template <typename E, int WROWS, int XROWS> struct SlabRing {
    static constexpr int WBYTES = 128 * WROWS, SLAB = WBYTES + 128 * XROWS;
    static constexpr int DEPTH = kRingBytes / SLAB, COPIES = (WROWS + XROWS) / 8;
    char *ring;            // this wavefront's kRingBytes of LDS
    int at = 0;            // place of the oldest slab, and of the next to issue

    template <int ROWS> __device__ __forceinline__ void copy(const SlabRows &r, uint32_t k, int left, char *dst) {
#pragma unroll
        for (int q = 0; q < ROWS / 8; ++q)
            buffer_to_lds16(r.buf[q], (int)slab_chunk() < left ? r.off[q] : kOutside, k, dst + 1024 * q);
    }
    // Copies one slab at byte `k` of the rows; `left` bytes of the rows are left.
    __device__ __forceinline__ void issue(const SlabRows &w, uint32_t k, int left) { issue(w, w, k, left); }
    __device__ __forceinline__ void issue(const SlabRows &w, const SlabRows &x, uint32_t k, int left) {
        issue(w, x, x, k, k, left);
    }
    __device__ __forceinline__ void issue(const SlabRows &w, const SlabRows &x, const SlabRows &x2, uint32_t k, uint32_t kx,
                                          int left) {
        char *dst = ring + at * SLAB;
        if (left <= 0) k = kx = 0;  // past a short buffer's end the range check could wrap
        copy<WROWS>(w, k, left, dst);
        if constexpr (XROWS > 0) copy<(XROWS < 16 ? XROWS : 16)>(x, kx, left, dst + WBYTES);
        if constexpr (XROWS == 32) copy<16>(x2, kx, left, dst + WBYTES + 16 * 128);
        at = at + 1 == DEPTH ? 0 : at + 1;
    }
    // Waits for the oldest slab and reads its fragments; the next issue has to
    // follow, into its place.
    __device__ __forceinline__ void take(SlabFrag<E> &w) {
        SlabFrag<E> none;
        take(w, none);
    }
    __device__ __forceinline__ void take(SlabFrag<E> &w, SlabFrag<E> &x) {
        SlabFrag<E> none;
        take(w, x, none);
    }
    __device__ __forceinline__ void take(SlabFrag<E> &w, SlabFrag<E> &x, SlabFrag<E> &x2) {
        // (stores issued in between only make the wait stricter)
        wait_vmcnt<(DEPTH - 1) * COPIES>();
        // the copies write LDS behind the compiler's back: no read may move above the wait
        asm volatile("" ::: "memory");
        const char *slab = ring + at * SLAB;
        w = slab_read<E, WROWS>(slab);
        if constexpr (XROWS > 0) x = slab_read<E, (XROWS < 16 ? XROWS : 16)>(slab + WBYTES);
        if constexpr (XROWS == 32) x2 = slab_read<E, 16>(slab + WBYTES + 16 * 128);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the fragments are in registers
        asm volatile("" ::: "memory");
    }
};

// The products of a sequence of positions: a position multiplies 16 weight rows
// with one or two blocks of 16 tokens.  The workgroup's eight wavefronts split K,
// each running its part of every position through one ring without a break.  The
// tokens' fragments stay in registers (SLABS slabs of K, TB blocks) until a
// position with other tokens; where a wavefront has more than SLABS slabs they are
// loaded anew for every position, and the ring drains each time.  The wavefronts'
// sums meet in LDS, added in their order.
//
// A Position type stands at one of the sequence and gives: left, the positions
// from it on; advance(); weights(SlabRows &), with `fresh` set the rows' offsets
// too (they are the same at every position); new_tokens(), whether its tokens
// differ from those of the position before; blocks(), 1 .. TB; tokens(), their
// buffer; token_row(t), this lane's row (lane % 16) of block t in it; finish(sums,
// thread), called by all threads with sums of 16 tokens x 16 rows per block and
// wavefront.  All but token_row and finish give wave-uniform answers.
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

template <typename E, int SLABS, int TB, class Position>
__device__ __forceinline__ void stream_products(const Position &start, int row_bytes, StreamLds<TB> &lds) {
    static_assert(TB == 1 || TB == 2, "token blocks");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slabs = (row_bytes + 127) / 128, per = (slabs + kWaves - 1) / kWaves;
    const int s0 = min(slabs, wave * per), s1 = min(slabs, s0 + per);  // this wavefront's slabs
    const bool parts = s1 - s0 > SLABS;  // the tokens do not stay

    SlabFrag<E> fx[TB][SLABS];
    auto load_tokens = [&](const Position &at, int base) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t buf = at.tokens();
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const uint32_t row = at.token_row(t);
            if (t > 0 && at.blocks() == 1) continue;
#pragma unroll
            for (int j = 0; j < SLABS; ++j)  // slabs past s1 are not used
                fx[t][j] = slab_load<E>(buf, row, 128u * (uint32_t)(base + j), row != kOutside ? row_bytes - 128 * (base + j) : 0);
        }
    };
    // loads return in order: with the tokens first, the first slab is multiplied
    // as soon as it lands
    load_tokens(start, s0);
    asm volatile("" ::: "memory");

    // the stream of weights: slabs s0 .. s1 of position after position
    SlabRing<E, 16, 0> ring{lds.ring + wave * kRingBytes};
    SlabRows w;
    Position in = start;
    int in_slab = s0;
    if (s0 == s1) in.left = 0;
    in.weights(w, true);
    auto ahead = [&]() __attribute__((always_inline)) {
        ring.issue(w, 128u * (uint32_t)in_slab, in.left > 0 ? row_bytes - 128 * in_slab : 0);
        if (++in_slab >= s1) {
            in_slab = s0;
            if (--in.left > 0) {
                in.advance();
                in.weights(w, false);
            }
        }
    };
#pragma unroll
    for (int q = 0; q < ring.DEPTH; ++q) ahead();
    // said to the compiler as well: the tokens are in their registers, and no wait
    // for them stands between the products
    wait_vmcnt<ring.DEPTH * ring.COPIES>();

    int set = 1, begin = 0;
    bool was_two = false, stale = parts;
    for (Position at = start; at.left > 0; --at.left) {
        if (at.left != start.left) {
            at.advance();
            stale = parts || at.new_tokens();
        }
        const bool two = TB == 2 && at.blocks() == 2;
        f32x4 acc[TB] = {};
        for (int base = s0; base < s1; base += SLABS) {
            if (stale) {
                load_tokens(at, base);
                wait_vmcnt<0>();
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
        at.finish(&lds.sums[set][0][0], (tid - begin) & (kThreads - 1));
        begin += Position::kFinishers;  // other wavefronts finish the next one
    }
    wait_vmcnt<0>();
}

}  // namespace dyra
