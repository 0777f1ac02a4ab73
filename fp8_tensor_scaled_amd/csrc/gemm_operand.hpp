// Operand tiles of the LDS-tiled fp8 GEMM kernels: the LDS layouts and their
// swizzles, the global -> LDS loads and the fragment reads (gemm_tiled.hip's
// header describes them; the block-scaled kernels use them too).
#pragma once

#include "common.hpp"

namespace fp8lin {

constexpr int kSub = 64;  // k per MFMA substep
typedef __attribute__((address_space(3))) void lds_void;

// vmcnt-only wait (gfx9 encoding: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] |
// vmcnt[5:4] at [15:14]; expcnt and lgkmcnt left at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// lgkmcnt(0) only (LDS reads of this wave complete).
__device__ __forceinline__ void wait_lgkmcnt0() {
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
}

// Chunk swizzle of a K-major tile row r (BK/16 chunks of 16 B per row).  A
// ds_read_b128 phase reads one chunk column of 16 consecutive rows.
// 128-byte rows: rows 2i and 2i+1 differ in the bank half and (r/2) % 8
// spreads the 8 row pairs over the 8 chunk positions.  64-byte rows: 4 rows
// share a 256-byte bank line, (r/2) % 4 and r/8 spread the rest.  Either way
// the 16 reads hit 16 distinct bank groups.  Only bits 1..3 of r are used.
template <int BK>
__device__ __forceinline__ int swz_kmajor(int r) {
    if constexpr (BK == 128) return (r >> 1) & 7;
    else return ((r >> 1) & 3) ^ ((r >> 3) & 1);
}

// Chunk swizzle of an MN-major tile row k (R / 16 chunks per row): even
// values, so the two 16-lane groups of a transposed-read phase (adjacent
// chunks, same rows) never share a bank group.  Depends on k % 8 only
// through the bits used, so rows k and k + 8q share it.
template <int R>
__device__ __forceinline__ int swz_mnmajor(int k) {
    if constexpr (R >= 256) return (k & 7) << 1;
    else if constexpr (R == 128) return ((k >> 1) & 3) << 1;
    else return ((k >> 2) & 1) << 1;
}

constexpr uint32_t kOOB = 0x80000000u;  // beyond every buffer range -> zeros

// Buffer descriptor (raw, 4 dwords): base address, no stride, the largest
// record count (offsets past it, such as kOOB, read as zero), and the
// default data format.  The base is uniform; readfirstlane says so to the
// compiler, so the descriptor lives in SGPRs.
__device__ __forceinline__ v4i make_rsrc(const void* base) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    v4i r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    r[2] = 0x7fffffff;
    r[3] = 0x00020000;
    return r;
}

// One buffer_load_dwordx4 ... lds: lane l fetches 16 bytes at descriptor base
// + voff and the hardware writes them to LDS at M0 + 16*l.  Written as
// inline asm so that the compiler does not track these LDS writes: its own
// tracking merges them at the k-loop back edge and then waits for every load
// in flight before the next fragment read, which drains the prefetch ring.
// The ring's waits are explicit here (wait_vmcnt), and nothing else in the
// k loop uses the vector memory counter.  The instruction has no output
// register; the s_nop covers the M0-write-to-LDS-DMA hazard.
__device__ __forceinline__ void dma16(const v4i& rsrc, uint32_t lds_addr, uint32_t voff) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(lds_addr));
}

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)p);
}

template <bool MN, int R, int NW, int BK>
struct Operand {
    static_assert(R == 64 || R == 128 || R == 256, "tile rows");
    static_assert(BK == 64 || BK == 128, "stage depth");
    static constexpr int kInstr = R * BK / 1024;  // 1 KB DMA instructions per stage
    static_assert(kInstr % NW == 0, "instructions per wave");
    static constexpr int kPerWave = kInstr / NW;

    // Lane layout of DMA instruction j of this wave: the tile row (K-major:
    // 1024/BK rows x BK bytes per instruction) or k row (MN-major: 1024/R
    // rows x R bytes) and the 16-byte chunk it fetches.
    __device__ static void slot(int j, int wave, int lane, int& row, int& chunk) {
        const int i = wave + j * NW;
        if constexpr (!MN) {
            constexpr int kLanesPerRow = BK / 16;
            row = (64 / kLanesPerRow) * i + lane / kLanesPerRow;
            chunk = (lane % kLanesPerRow) ^ swz_kmajor<BK>(row);
        } else {
            constexpr int kRowsPer = 1024 / R;
            constexpr int kChunks = R / 16;
            row = kRowsPer * i + lane / kChunks;
            chunk = (lane % kChunks) ^ swz_mnmajor<R>(row);
        }
    }

    // Instruction j of a wave covers the rows of instruction 0 shifted by
    // j*NW instructions; the swizzle of those rows is the same (the shift is
    // a multiple of 16 rows for K-major, of 8 k rows for MN-major), so the
    // offset of instruction j is that of instruction 0 plus a uniform stride.
    static constexpr int kRowStep = NW * (MN ? 1024 / R : 1024 / BK);  // rows per j
    static_assert(NW % 2 == 0, "row shift keeps the swizzle");

    // Per-lane byte offset of instruction 0 at k = 0.  MN-major: kOOB when
    // the lane's 16 columns lie outside the matrix (the same for every j).
    // `rows_left` = extent of the operand along m (A) or n (B) from this
    // tile's origin.
    __device__ static uint32_t init(uint32_t ld, int64_t rows_left, int wave, int lane) {
        int row, c;
        slot(0, wave, lane, row, c);
        if constexpr (!MN) return (uint32_t)row * ld + 16 * c;
        else return 16 * c < rows_left ? (uint32_t)row * ld + 16 * c : kOOB;
    }

    // Issue this wave's DMA loads of the stage starting at k0 into `lds`.
    // All offsets are 32-bit (the host only takes this path when every
    // operand slice is addressable that way; kOOB plus any in-range offset
    // stays below 2^32 and beyond the range).  `full_rows`: every tile row
    // exists (uniform), else K-major rows past the edge read zeros.
    __device__ static void issue(const v4i& rs, uint8_t* lds, uint32_t base, uint32_t ld, int k0,
                                 int kdim, bool full_rows, int64_t rows_left, int wave, int lane) {
        const uint32_t delta = MN ? (uint32_t)k0 * ld : (uint32_t)k0;
        const uint32_t jstride = (uint32_t)kRowStep * ld;
        const bool full = k0 + BK <= kdim;  // uniform: no k tail in this stage
#pragma unroll
        for (int j = 0; j < kPerWave; ++j) {
            uint32_t off = base + delta + j * jstride;
            if (!full || (!MN && !full_rows)) {
                int row, c;
                slot(j, wave, lane, row, c);
                const int gk = MN ? k0 + row : k0 + 16 * c;
                if (gk >= kdim) off = kOOB;
                if (!MN && row >= rows_left) off = kOOB;
            }
            dma16(rs, lds_addr(lds + 1024 * (wave + j * NW)), off);
        }
    }

    // Offset of this lane for DMA instruction j of the stage at k0 (kOOB past
    // the matrix), and the LDS address instruction j writes.
    __device__ static uint32_t off_of(uint32_t base, uint32_t ld, int k0, int kdim,
                                      bool full_rows, int64_t rows_left, int j, int wave,
                                      int lane) {
        const uint32_t delta = MN ? (uint32_t)k0 * ld : (uint32_t)k0;
        uint32_t off = base + delta + j * ((uint32_t)kRowStep * ld);
        if (!(k0 + BK <= kdim) || (!MN && !full_rows)) {
            int row, c;
            slot(j, wave, lane, row, c);
            const int gk = MN ? k0 + row : k0 + 16 * c;
            if (gk >= kdim) off = kOOB;
            if (!MN && row >= rows_left) off = kOOB;
        }
        return off;
    }
    __device__ static uint32_t lds_of(uint8_t* lds, int j, int wave) {
        return lds_addr(lds + 1024 * (wave + j * NW));
    }

    // Fragment addressing.  The MFMA operand of the 32 tile rows starting at
    // rf, substep h, gives lane l row rf + l%32 and k = 64h + 32*(l/32) ..
    // +31 of the stage.  The lane-dependent part of each address is computed
    // once (frag_off); the rest is a compile-time constant or a fixed XOR.
    //
    // K-major: rf is a multiple of 32, so the swizzle depends on the lane
    // only and rf adds rf*128.  The 16-byte pieces wanted are chunks
    // 4h + 2*(l/32) + e (e = 0, 1); their bits are disjoint, so the swizzled
    // chunk is (2*(l/32) ^ swizzle) ^ 4h ^ e, i.e. the substep and the half
    // flip bits 6 and 4 of the lane's offset.
    // MN-major (ds_read_b64_tr_b8): within each 16-lane group, lane p names
    // the 8 bytes at (k = kb + 8q + p/2, m = mb + 8*(p%2)) and lane p of the
    // group receives m = mb + p for k = kb+8q .. +7 (q = 0..3), with kb =
    // 64h + 32*(group/2).  The swizzle of row k depends on p only, so h and
    // q add (64h + 8q)*R; the chunk (mb/16) ^ swizzle stays per fragment.
    __device__ static uint32_t frag_off(int rf, int lane) {
        if constexpr (!MN) {
            const int row = lane & 31;  // rf*128 is added as a constant
            const int c = (2 * (lane >> 5)) ^ swz_kmajor<BK>(row);
            (void)rf;
            return (uint32_t)(row * BK + (c << 4));
        } else {
            const int g = lane >> 4, p = lane & 15;
            const int mb = rf + 16 * (g & 1);
            const int kr = 32 * (g >> 1) + (p >> 1);
            return (uint32_t)(kr * R + (((mb >> 4) ^ swz_mnmajor<R>(kr)) << 4) + 8 * (p & 1));
        }
    }

    // Reads the substep-H fragment: `lds` = stage start (K-major: plus
    // rf*BK), `off` = frag_off(rf, lane).
    template <int H>
    __device__ static v8i frag(const uint8_t* lds, uint32_t off) {
        v8i v;
        if constexpr (!MN) {
            const v4i lo = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
                (lds_void*)(lds + (off ^ (64u * H))));
            const v4i hi = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
                (lds_void*)(lds + (off ^ (64u * H + 16u))));
            v[0] = lo[0]; v[1] = lo[1]; v[2] = lo[2]; v[3] = lo[3];
            v[4] = hi[0]; v[5] = hi[1]; v[6] = hi[2]; v[7] = hi[3];
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v2i t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) v2i*)(lds + off + (kSub * H + 8 * q) * R));
                v[2 * q] = t[0];
                v[2 * q + 1] = t[1];
            }
        }
        return v;
    }
};

}  // namespace fp8lin
