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

    // Looks up tile t's pages, a tile ahead of their use.
    __device__ __forceinline__ void look_up(int t, Pages& p) const
    {
        if (!PAGED) return;
#pragma unroll
        for (int j = 0; j < N; ++j)
            p.id[j] = a.table[b * a.table_stride + a.by_page.div(min(t * kKeyTile + (int)row(j), kt.hi))];
    }

    // Tiles t of k and of v. The pages that were looked up are waited for once,
    // before copies are under way that a wait for one of them would also wait for.
    __device__ __forceinline__ void copy_both(int t, const Pages& p, u32 lds) const
    {
        if (PAGED) settle_loads();
        copy(a.k, t, p, lds);
        copy(a.v, t, p, lds + TILE);
    }

    // Tile t of x (k or v).
    __device__ __forceinline__ void copy(const Tensor& x, int t, const Pages& p, u32 lds) const
    {
        const int k0 = t * kKeyTile;
        const unsigned char* const zero = (const unsigned char*)kAbsent.zero;
        if constexpr (!PAGED) {
            const unsigned char* from = x.p + b * x.sb + hk * x.sh + (k0 + wave * RPI) * x.sl;
            const u32 row_at = (lane / CH) * (u32)x.sl;
            if (k0 + kKeyTile - 1 <= kt.hi && (k0 >= kt.lo || k0 + kKeyTile <= a.sinks)) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if ((int)chunk(j) * 8 < a.D)
                        dma16(from + j * NW * RPI * x.sl, row_at + chunk(j) * 16, lds + (j * NW + wave) * 1024);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int key = k0 + (int)row(j);
                    const bool there = key <= kt.hi && (key >= kt.lo || key < a.sinks);
                    if ((int)chunk(j) * 8 < a.D)
                        dma16(there ? from + j * NW * RPI * x.sl + row_at + chunk(j) * 16 : zero,
                              lds + (j * NW + wave) * 1024);
                }
            }
            return;
        }
        const unsigned char* from = x.p + hk * x.sh;
        const bool whole = k0 + kKeyTile - 1 <= kt.hi && (k0 >= kt.lo || k0 + kKeyTile <= a.sinks);
        if (a.by_page.d % RPI == 0) {
            // The rows of one copy lie in one page: its address is the same for the wave.
            const u32 row_at = (lane / CH) * (u32)x.sl;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int id = uniform(p.id[j]), first = k0 + (j * NW + wave) * RPI;
                const int at = first - (int)a.by_page.div(first) * (int)a.by_page.d;
                const unsigned char* page = from + id * x.sb + at * x.sl;
                const bool bad = (u32)id >= (u32)a.pages;
                if ((int)chunk(j) * 8 >= a.D) continue;
                if (whole && !bad) {
                    dma16(page, row_at + chunk(j) * 16, lds + (j * NW + wave) * 1024);
                } else {
                    const int key = k0 + (int)row(j);
                    const bool there = key <= kt.hi && (key >= kt.lo || key < a.sinks);
                    const unsigned char* const e = bad ? (const unsigned char*)kAbsent.nan : page + row_at + chunk(j) * 16;
                    dma16(there ? e : zero, lds + (j * NW + wave) * 1024);
                }
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int key = k0 + (int)row(j), at = key - (int)a.by_page.div(key) * (int)a.by_page.d;
            const unsigned char* e = from + p.id[j] * x.sb + at * x.sl + chunk(j) * 16;
            if (p.id[j] < 0 || p.id[j] >= a.pages) e = (const unsigned char*)kAbsent.nan;
            if (!(key <= kt.hi && (key >= kt.lo || key < a.sinks))) e = zero;
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
