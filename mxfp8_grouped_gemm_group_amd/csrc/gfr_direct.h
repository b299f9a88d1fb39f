// The run of a block through its tiles of a 16-bit product, operands straight to LDS:
// the core of gfr_grouped.hip's direct kernel and of gfr_lora.hip's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gfr_device.h"
#include "gfr_tile.h"

namespace gfr {
namespace {

#define GFR_INLINE __attribute__((always_inline))
template <int N>
using Int = std::integral_constant<int, N>;

// 16 bytes a lane from memory straight to LDS, 1024 consecutive bytes from `lds` on.
// (Assembly, because behind the builtin the compiler waits for all of them ahead of
// every later LDS read.  It writes no register but m0, which the compiler keeps for single
// instructions and does not take as a clobber; direct_wait is its wait.  A vector access has
// to be five wait states behind a vector instruction that wrote a scalar register it reads,
// which the compiler does not see to in here: the buffer's size and `off` come by
// v_readfirstlane, or by v_readlane where they were spilled.)
__device__ __forceinline__ void load_lds(rsrc_t r, int lane_off, int off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(lane_off), "s"(r), "s"(off) : "memory");
}
// All but this wave's N latest loads and stores are through; then the same of the
// block's other waves.
template <int N>
__device__ __forceinline__ void direct_wait() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(N) : "memory");
}
// This wave's LDS accesses are through, then the other waves' too.
__device__ __forceinline__ void lds_wait() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One operand's loads of a step, straight to LDS, for rows of whole pieces (row
// lengths multiples of 8).  A load takes 1024 bytes of the tile; its lanes choose
// their piece by the layout's swizzle.  Pieces behind the summed index's end are
// zeros (their offsets lie behind the buffer's end), and so is all of a step behind
// it; what lies behind the last line belongs to lines that are not stored.
template <bool LINE, int BX, int WAVES>
struct Direct {
    static constexpr int kLoads = BX / 8 / WAVES;      // a wave's, per step
    static constexpr int kRows = LINE ? 512 / BX : 8;  // of the tile in a load
    static_assert(WAVES % 2 == 0 && (!LINE || kRows >= 2), "a wave's loads share their swizzle");
    const char *base;
    int64_t bytes;                 // from base to the end of what may be read
    rsrc_t r;
    int row_bytes, stride;         // stride: bytes between a wave's loads
    int first;                     // the wave's first row times row_bytes, less one stride
    int offs, now;                 // the lane's place in a load; in the step's loads
    int piece_k;                   // k-major: first k of the lane's piece
    int K, off, loads;             // loads: those that hold any line of the tile
    int turn;                      // k-major: the step of K that comes first
    int thrice;                    // k-major: pieces of a row whose pairs come three times

    // Rows of `ld` elements.  Load i takes the tile's rows from (WAVES i + wave) kRows on.
    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
        row_bytes = static_cast<int>(2 * ld);
        stride = WAVES * kRows * row_bytes;
        first = wave * kRows * row_bytes - stride;
        if (LINE) {
            constexpr int kLanes = 64 / kRows;
            const int row = lane / kLanes, k = (wave * kRows + row) & 3;
            offs = now = row * row_bytes + 16 * ((lane % kLanes) ^ (4 * k));
        } else {
            const int row = lane >> 3, piece = (lane & 7) ^ ((wave * 8 + row) >> 1 & 7);
            piece_k = 8 * piece;
            offs = row * row_bytes + 16 * piece;
        }
    }
    // The tile whose first line begins at `from` (line-major: at k = 0), with `bytes_`
    // from there to the end of what may be read (0: no tile) and K_ to sum over.
    __device__ __forceinline__ void tile(const uint16_t *from, int64_t bytes_, int K_, int lines,
                                         int turn_ = 0, int thrice_ = 0) {
        turn = turn_;
        thrice = thrice_;
        base = reinterpret_cast<const char *>(from);
        bytes = bytes_;
        K = K_;
        // (of a line-major step every load holds some of the lines)
        loads = LINE ? kLoads : uniform((lines + 8 * WAVES - 1) / (8 * WAVES));
        if (!LINE) r = uniform_buffer(base, bytes);
    }
    // Ahead of a step's loads (THRICE: of tiles that may have it; up to 96 pieces in all).
    template <bool THRICE>
    __device__ __forceinline__ void at(int step) {
        if (LINE) {
            const int64_t gone = static_cast<int64_t>(step) * 64 * row_bytes;
            r = uniform_buffer(base + gone, bytes > gone ? bytes - gone : 0);
            off = first;
        } else {
            step += turn;
            if (64 * step >= K && turn > 0) step -= (K + 63) / 64;
            off = first + 128 * step;
            now = offs;
            if (THRICE && thrice > 0) {
                const int p = 8 * step + (piece_k >> 3), pair = p * 43 >> 8;       // p / 6
                const int second = 2 * pair + 1 < thrice ? p - 6 * pair & 1 : 0;
                off = first;
                now += 16 * (2 * pair + second) - 2 * piece_k;
            }
            if (64 * step + piece_k >= K) now = kPast;
        }
    }
    // Load i, all in turn.  `off` goes on to it in two of load_lds's five states, all of which
    // cost 1 % where the matrix cores bound it (32768 rows over 32 experts of 4096 x 7168 1787
    // -> 1810 us; 1816 with the sums ahead of load_lds, and twice the scalar spills).
    __device__ __forceinline__ void load(int i, uint32_t tile) {
        asm volatile("s_add_u32 %0, %0, %3\n\ts_add_u32 m0, %4, %5\n\ts_nop 2\n\t"
                     "buffer_load_dwordx4 %1, %2, %0 offen lds"
                     : "+&s"(off)
                     : "v"(now), "s"(r), "s"(stride), "s"(tile), "i"(WAVES * 1024 * i)
                     : "memory", "scc");
    }
};

// The kernel's first argument, read where this is called: kept over the run of tiles its
// many words took the scalar registers that the run's loops need.
template <class Params>
__device__ __forceinline__ Params fresh() {
    typedef const __attribute__((address_space(4))) Params *at_t;
    at_t at = (at_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *(const Params *)at;
}

// n / d for 0 <= n < 2^31 by d's reciprocal in FP32, which is off by a few for the largest
// quotients, and corrected.
struct Divisor {
    int d;
    float inverse;
    __device__ __forceinline__ explicit Divisor(int d_) : d(d_), inverse(1.0f / d_) {}
    __device__ __forceinline__ int of(int n) const {
        int q = static_cast<int>(static_cast<float>(n) * inverse);
        int rest = n - q * d;
        while (uniform(rest) < 0) --q, rest += d;
        while (uniform(rest) >= d) ++q, rest -= d;
        return uniform(q);
    }
};

constexpr int kMaxLds = 159 << 10;          // of kernels that have no static LDS
constexpr int kTile = 256, kWaves = 4;
constexpr int kStage = 2 * kTile * 8;       // pieces: an operand's 256 lines, the other's

// A tile: `rows` rows from m0 on, columns from n0 on, of the group e's product; steps of
// the summed index.
//
// Tiles of a kernel with kExtra end with `extra` steps whose products only some of the
// 32-row fragments take: byte i of `masks` says which ones take the i-th run of
// `extra_run` steps.
struct TileAt {
    int e, m0, n0, rows, steps;
    int extra, extra_run;
    uint64_t masks;
};

// 256 x 256 tiles of four waves, one block to a CU, which goes through its tiles'
// steps (64 of the summed index) as one run: two LDS stages, filled straight from
// memory two steps ahead, also over the end of a tile.  A step is four parts of 16;
// each part's fragments have registers of their own, so that a stage is read within
// three parts and filled in the other five of its two steps:
//
//   part 0   reads the step's last fragments; then a barrier: the stage is free
//   part 1   begins the loads of the step after next; then a barrier: the next stage
//            has landed
//   part 2   reads the next step's fragments 0 and 1, goes on loading
//   part 3   reads fragment 2, goes on loading
//
// (One barrier a step, and all loads behind it, took 400 clocks of 2048 more: a CU's
// loads take 16 clocks each, 64 a step.)  A tile of fewer rows takes less
// time: up to 128 of them split their columns over the waves, up to 192 go as 256.
//
// Tiles: at(id), the tile, for ids begin, begin + stride, ... below end; next(cursor, da,
// db, wave, lane), the operands of the next run of steps and their number, 0 behind the
// last tile.  Finish: tile<FM, FN>(t, acc, wm, wn, lane) takes a
// wave's results (32 FM x 32 FN of them from wm, wn on) and returns how many stores it
// has issued at least (kLong: it needs many registers); clear(t) a tile without a sum.
template <bool F16, bool ALINE, bool BLINE, class Tiles, class Finish>
__device__ __forceinline__ void run_tiles(u4_t *lds, const Tiles &tiles, const Finish &finish,
                                          int64_t lda, int64_t ldb) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    // The loads' place: the operands of a tile, its next step.
    Direct<ALINE, kTile, kWaves> da;
    Direct<BLINE, kTile, kWaves> db;
    da.init(lda, wave, lane);
    db.init(ldb, wave, lane);
    const int stride = tiles.stride, end = uniform(tiles.end);
    int id = uniform(tiles.begin);
    if (id >= end) return;
    int load_step = 0, load_steps = 0;
    typename Tiles::Cursor cursor(id - stride);
    auto next_loads = [&]() GFR_INLINE {
        load_step = uniform(load_step + 1);
        if (load_step < uniform(load_steps)) return;
        load_step = 0;
        load_steps = tiles.next(cursor, da, db, wave, lane);
        if (load_steps == 0) {
            load_steps = 0x7fffffff;             // no tile left: zeros
            da.tile(nullptr, 0, 0, 0);
            db.tile(nullptr, 0, 0, 0);
        }
    };
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) void *)lds)) + wave * 1024;
    constexpr int kB = decltype(db)::kLoads, kLoads = kB + decltype(da)::kLoads;
    // (B's first: their number does not depend on the tile's rows)
    auto load = [&](int i, int stage) GFR_INLINE {
        const uint32_t to = lds0 + stage * kStage * 16;
        if (i < kB) db.load(i, to + kTile * 128);
        else if (ALINE || i - kB < da.loads) da.load(i - kB, to);
    };
    int now = 0;                              // the stage of the step that is multiplied
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        next_loads();
        da.template at<false>(load_step);
        db.template at<Tiles::kExtra>(load_step);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load(j, i);
    }
    direct_wait<kB>();
    int stores = 0;                           // of this wave, behind its latest loads

    // A tile in waves of 32 FM x 32 FN, kWaves / COLS by COLS of them.
    auto run_tile = [&](const TileAt &t, auto fm, auto fn, auto cols) GFR_INLINE {
        constexpr int FM = fm, FN = fn, COLS = cols;
        constexpr int kGets = FM + FN, kMfmas = FM * FN;
        const int wm = wave / COLS * (32 * FM), wn = wave % COLS * (32 * FN);
        // (opaque: the shapes' fragment addresses are not kept over all tiles, which took
        // the registers that loops then missed)
        int line = lane;
        asm volatile("" : "+v"(line));
        u4_t a[4][FM], b[4][FN];
        auto get = [&](int part, int stage, int i) GFR_INLINE {
            const u4_t *tile = lds + stage * kStage;
            if (i < FM)
                a[part][i] = fragment<ALINE, kTile>(tile, wm + 32 * i, part, line);
            else
                b[part][i - FM] =
                    fragment<BLINE, kTile>(tile + kTile * 8, wn + 32 * (i - FM), part, line);
        };
        f16_t acc[FM][FN] = {};
        // A part: its MFMAs, and between them `gets` fragments from part `first` on
        // of a stage, and loads [from, to).
        auto run_part = [&](auto masked, int mask, auto part, auto gets, auto first, int stage,
                            auto from, auto to, int into) GFR_INLINE {
            constexpr int kG = (gets + kMfmas - 1) / kMfmas;
            constexpr int kL = (to - from + kMfmas - 1) / kMfmas;
#pragma unroll
            for (int m = 0; m < kMfmas; ++m) {
#pragma unroll
                for (int h = 0; h < kG; ++h)
                    if (const int i = m * kG + h; i < gets)
                        get(first + i / kGets, stage, i % kGets);
#pragma unroll
                for (int h = 0; h < kL; ++h)
                    if (const int i = from + m * kL + h; i < to) load(i, into);
                if (!masked || (mask >> m / FN & 1))
                    acc[m / FN][m % FN] = mfma32<F16>(b[part][m % FN], a[part][m / FN],
                                                      acc[m / FN][m % FN]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
#pragma unroll
        for (int i = 0; i < 3 * kGets; ++i) get(i / kGets, now, i % kGets);
        constexpr int kFirst = (kLoads + 2) / 3, kSecond = kFirst + (kLoads - kFirst + 1) / 2;
        static_assert(kFirst <= kB, "part 1 begins the same number of loads in every tile");
        auto run_step = [&](auto masked, int mask) GFR_INLINE {
            run_part(masked, mask, Int<0>{}, Int<kGets>{}, Int<3>{}, now, Int<0>{}, Int<0>{}, 0);
            lds_wait();
            next_loads();
            da.template at<false>(load_step);
            db.template at<Tiles::kExtra>(load_step);
            run_part(masked, mask, Int<1>{}, Int<0>{}, Int<0>{}, 0, Int<0>{}, Int<kFirst>{}, now);
            // (the last tile's results may still be on their way)
            if (stores < 16) direct_wait<kFirst>();
            else if (stores < 32) direct_wait<kFirst + 16>();
            else direct_wait<kFirst + 32>();
            stores = 0;
            run_part(masked, mask, Int<2>{}, Int<2 * kGets>{}, Int<0>{}, now ^ 1, Int<kFirst>{},
                     Int<kSecond>{}, now);
            run_part(masked, mask, Int<3>{}, Int<kGets>{}, Int<2>{}, now ^ 1, Int<kSecond>{},
                     Int<kLoads>{}, now);
            now ^= 1;
        };
        const int all = Tiles::kExtra ? t.steps - t.extra : t.steps;
        for (int step = 0; step < all; ++step) run_step(Int<0>{}, 0);
        if (Tiles::kExtra) {
            uint64_t masks = t.masks;
            for (int step = 0, run = 0; step < t.extra; ++step) {
                run_step(Int<1>{}, static_cast<int>(masks & 0xff) >> (wm / 32));
                if (++run == t.extra_run) run = 0, masks >>= 8;
            }
        }
        // (what a long finish needs registers for is not taken from the loop's sums, of which
        // one went to memory and back every step; a short one is better off without: 8192
        // rows over 64 experts of 2048 x 1536 145 us with it, 132 without)
        if (Finish::kLong && FM * FN == 16)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
        stores = finish.template tile<FM, FN>(t, acc, wm, wn, line);
    };
    for (; id < end; id += stride) {
        const TileAt t = tiles.at(id);
        if (t.steps == 0) {
            finish.clear(t);
            continue;
        }
        if (t.rows > 192) run_tile(t, Int<4>{}, Int<4>{}, Int<2>{});
        else if (t.rows > 128) run_tile(t, Int<3>{}, Int<4>{}, Int<2>{});
        else if (t.rows > 64) run_tile(t, Int<4>{}, Int<2>{}, Int<4>{});
        else if (t.rows > 32) run_tile(t, Int<2>{}, Int<2>{}, Int<4>{});
        else run_tile(t, Int<1>{}, Int<2>{}, Int<4>{});
    }
    // (no load may be on its way to LDS when the block ends)
    direct_wait<0>();
}

}  // namespace
}  // namespace gfr
