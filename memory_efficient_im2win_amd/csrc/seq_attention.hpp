// Pieces that the window attention kernels share: which keys a run of rows
// sees, and the copy of key and row tiles into LDS.
#pragma once

#include "seq_common.hpp"
#include "seq_kernels.hpp"

namespace im2win {
namespace seq {

constexpr int kKeyTile = 64;

// Lengths of sequence b, cut to the tensors' extents; off = position of
// query 0.
struct Span {
    int nq, nk, off;
    __device__ __forceinline__ Span(const AttnParams& a, int b)
    {
        nq = a.q_lens ? min(max(a.q_lens[b], 0), a.Lq) : a.Lq;
        nk = a.kv_lens ? min(max(a.kv_lens[b], 0), a.Lk) : a.Lk;
        nq = uniform(nq);
        nk = uniform(nk);
        off = nk - nq;
    }
};

// The key tiles that queries i0..i1 see: tiles of sinks that lie before the
// window's first tile, then the window's tiles in order.
struct KeyTiles {
    int lo, hi;          // first key of the union of windows, last key
    int far, first, n;   // sink tiles in front, first window tile, tiles in all
    __device__ __forceinline__ KeyTiles(const AttnParams& a, const Span& s, int i0, int i1)
    {
        hi = s.off + i1;
        lo = max(0, s.off + i0 - a.window + 1);
        far = first = n = 0;
        if (i0 > i1 || hi < 0) return;
        first = lo / kKeyTile;
        far = min((min(a.sinks, hi + 1) + kKeyTile - 1) / kKeyTile, first);
        n = far + hi / kKeyTile - first + 1;
    }
    __device__ __forceinline__ int at(int i) const { return i < far ? i : first + i - far; }
};

// Whether the query at position p sees key k0 + i, for constants i: compares
// with three numbers of the block. (Opaque: the compiler would otherwise keep
// p - i for every i of a walk in registers.)
struct Mask {
    int near, edge, sink;
    __device__ __forceinline__ Mask(int p, int k0, const AttnParams& a)
        : near(p - k0), edge(near - a.window), sink(a.sinks - k0)
    {
        asm("" : "+v"(near), "+v"(edge), "+v"(sink));
    }
    __device__ __forceinline__ bool operator()(int i) const { return i <= near && (i > edge || i < sink); }
};

// Copies tiles of 64 keys or values into LDS, by NW waves of which the caller
// is number `wave`. Keys that no row of the workgroup sees arrive as zeros, so
// what they hold in memory does not matter; those of a page outside the pool as
// NaN. Chunks past the head size are not written: clear() zeroes them once.
template <int LP, int NW, bool PAGED>
struct KeyStage {
    static constexpr int CH = LP / 8, RPI = 64 / CH, N = kKeyTile / RPI / NW, TILE = kKeyTile * LP * 2;
    struct Pages {
        int id[N];
    };
    const AttnParams& a;
    const KeyTiles& kt;
    int b, hk, lane, wave;

    __device__ __forceinline__ KeyStage(const AttnParams& a_, const KeyTiles& kt_, int b_, int hk_, int wave_)
        : a(a_), kt(kt_), b(b_), hk(hk_), lane(threadIdx.x & 63), wave(wave_)
    {
    }
    __device__ __forceinline__ u32 row(int j) const { return (j * NW + wave) * RPI + lane / CH; }
    __device__ __forceinline__ u32 chunk(int j) const { return (lane % CH) ^ swz<LP>(row(j)); }

    __device__ __forceinline__ static void clear(u32 lds, int bytes, int D)
    {
        if (D == LP) return;
        for (int at = threadIdx.x * 16; at < bytes; at += blockDim.x * 16) lds_write16(lds + at, (u32x4_t)(0u));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }

    // Looks up tile t's pages, a tile ahead of their use. Where the rows of a
    // copy lie in one page, lane j looks up the j-th copy's (id[0]); else every
    // lane that of its row of each copy.
    __device__ __forceinline__ bool even() const { return a.by_page.d % RPI == 0; }
    __device__ __forceinline__ int lane_row() const { return ((lane & (N - 1)) * NW + wave) * RPI; }
    __device__ __forceinline__ void look_up(int t, Pages& p) const
    {
        if (!PAGED) return;
        // The same loads either way: with a branch the compiler moved what they
        // load, and waited for it and the copies before, at once (108 -> 117 us,
        // a token each of 64 sequences of up to 8192 keys).
        const int32_t* const table = a.table + b * a.table_stride;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int key = t * kKeyTile + (even() ? lane_row() : (int)row(j));
            p.id[j] = table[a.by_page.div(min(key, kt.hi))];
        }
    }

    // Tiles t of k and of v.
    __device__ __forceinline__ void copy_both(int t, const Pages& p, u32 lds) const
    {
        const int k0 = t * kKeyTile;
        const bool whole = k0 + kKeyTile - 1 <= kt.hi && (k0 >= kt.lo || k0 + kKeyTile <= a.sinks);
        if constexpr (!PAGED) {
            copy_run(a.k, whole, a.k.p + b * a.k.sb + hk * a.k.sh + (k0 + wave * RPI) * a.k.sl, k0, lds);
            copy_run(a.v, whole, a.v.p + b * a.v.sb + hk * a.v.sh + (k0 + wave * RPI) * a.v.sl, k0, lds + TILE);
            return;
        }
        // Waits for what was looked up, before copies are under way that a wait
        // would also wait for.
        settle_loads();
        if (a.by_page.d % kKeyTile == 0) {  // the tile is in one page: as in a whole sequence
            const int id = uniform(p.id[0]);
            const bool bad = (u32)id >= (u32)a.pages;
            const auto run = [&](const Tensor& x, u32 to) {
                const unsigned char* const page = x.p + hk * x.sh + (uint32_t)id * (uint64_t)x.sb;
                copy_rows(x, whole && !bad, k0, to, [&](int j) {
                    const int row = k0 + (j * NW + wave) * RPI, at = row - (int)a.by_page.div(row) * (int)a.by_page.d;
                    return bad ? (const unsigned char*)nullptr : page + at * x.sl;
                });
            };
            run(a.k, lds);
            run(a.v, lds + TILE);
            return;
        }
        if (!even()) {
            copy_odd(a.k, k0, p, lds);
            copy_odd(a.v, k0, p, lds + TILE);
            return;
        }
        // Every copy's offset at once, one a lane. (With a copy's address in
        // scalar arithmetic, a tile of 16-token pages took 0.5 us more.)
        const int id = p.id[0], key = k0 + lane_row(), at = key - (int)a.by_page.div(key) * (int)a.by_page.d;
        const bool bad = (u32)id >= (u32)a.pages;
        const int64_t to_k = id * a.k.sb + at * a.k.sl;
        const int64_t to_v = a.k.sb == a.v.sb && a.k.sl == a.v.sl ? to_k : id * a.v.sb + at * a.v.sl;
        const uint64_t bad_ones = __ballot(bad);
        const auto from = [&](const Tensor& x, int64_t off, int j) {
            const u32 lo = __builtin_amdgcn_readlane((int)off, j), hi = __builtin_amdgcn_readlane((int)(off >> 32), j);
            return bad_ones >> j & 1 ? (const unsigned char*)nullptr : x.p + hk * x.sh + (int64_t)((uint64_t)hi << 32 | lo);
        };
        copy_rows(a.k, whole && !bad_ones, k0, lds, [&](int j) { return from(a.k, to_k, j); });
        copy_rows(a.v, whole && !bad_ones, k0, lds + TILE, [&](int j) { return from(a.v, to_v, j); });
    }

private:
    // The tile's rows of x, one after another in memory from `first` (this wave's).
    __device__ __forceinline__ void copy_run(const Tensor& x, bool plain, const unsigned char* first, int k0, u32 lds) const
    {
        const int64_t step = NW * RPI * x.sl;
        copy_rows(x, plain, k0, lds, [&](int) {
            const unsigned char* const r = first;
            first += step;
            return r;
        });
    }

    // The tile's rows of x, from(j) the address of the j-th copy's first row (null:
    // a page outside the pool). plain: all rows are there.
    template <typename F>
    __device__ __forceinline__ void copy_rows(const Tensor& x, bool plain, int k0, u32 lds, F from) const
    {
        const u32 row_at = (lane / CH) * (u32)x.sl;
        if (plain) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const unsigned char* first = from(j);
                if ((int)chunk(j) * 8 < a.D) dma16(first, row_at + chunk(j) * 16, lds + (j * NW + wave) * 1024);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned char* first = from(j);
            const int key = k0 + (int)row(j);
            const bool there = key <= kt.hi && (key >= kt.lo || key < a.sinks);
            const unsigned char* e = first ? first + row_at + chunk(j) * 16 : (const unsigned char*)kAbsent.nan;
            if (!there) e = (const unsigned char*)kAbsent.zero;
            if ((int)chunk(j) * 8 < a.D) dma16(e, lds + (j * NW + wave) * 1024);
        }
    }

    // The same where pages end inside a copy: every lane's own address.
    __device__ __forceinline__ void copy_odd(const Tensor& x, int k0, const Pages& p, u32 lds) const
    {
        const unsigned char* const head = x.p + hk * x.sh;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int key = k0 + (int)row(j), at = key - (int)a.by_page.div(key) * (int)a.by_page.d;
            const unsigned char* e = head + p.id[j] * x.sb + at * x.sl + chunk(j) * 16;
            if ((u32)p.id[j] >= (u32)a.pages) e = (const unsigned char*)kAbsent.nan;
            if (!(key <= kt.hi && (key >= kt.lo || key < a.sinks))) e = (const unsigned char*)kAbsent.zero;
            if ((int)chunk(j) * 8 < a.D) dma16(e, lds + (j * NW + wave) * 1024);
        }
    }
};

// The 16 bytes at column c of flattened row r of x, zeros past the sequence.
__device__ __forceinline__ const unsigned char* row_ptr(const AttnParams& a, const Tensor& x, int b, int hk,
                                                        int r, int r_end, int c)
{
    if (r >= r_end || c >= a.D) return (const unsigned char*)kAbsent.zero;
    const int i = a.by_group.div(r), g = r - i * a.G;
    return x.p + b * x.sb + i * x.sl + (int64_t)(hk * a.G + g) * x.sh + c * 2;
}

}  // namespace seq
}  // namespace im2win
