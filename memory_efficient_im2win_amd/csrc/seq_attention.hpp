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

// Copies tiles of 64 keys and values into LDS (k at `lds`, v a tile later).
// Keys that no row of the workgroup sees arrive as zeros, so what they hold in
// memory does not matter; those of a page outside the pool as NaN. Chunks past
// the head size are not written: clear() zeroes them once.
template <int LP, int NW>
struct KeyStage {
    static constexpr int CH = LP / 8, RPI = 64 / CH, N = kKeyTile / RPI / NW, TILE = kKeyTile * LP * 2;
    const AttnParams& a;
    const KeyTiles& kt;
    int b, hk, lane, wave;
    u32 ok, ov;     // lane offsets of the plain copy
    int page[N];    // the next tile's pages (or the sequence)

    __device__ __forceinline__ KeyStage(const AttnParams& a_, const KeyTiles& kt_, int b_, int hk_)
        : a(a_), kt(kt_), b(b_), hk(hk_), lane(threadIdx.x & 63), wave(uniform(threadIdx.x >> 6))
    {
        ok = (lane / CH) * (u32)a.k.sl;
        ov = (lane / CH) * (u32)a.v.sl;
    }
    __device__ __forceinline__ u32 row(int j) const { return (j * NW + wave) * RPI + lane / CH; }
    __device__ __forceinline__ u32 chunk(int j) const { return (lane % CH) ^ swz<LP>(row(j)); }

    __device__ __forceinline__ static void clear(u32 lds, int bytes, int D)
    {
        if (D == LP) return;
        for (int at = threadIdx.x * 16; at < bytes; at += NW * 1024) lds_write16(lds + at, (u32x4_t)(0u));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }

    // Looks up tile t's pages, a tile ahead of their use.
    __device__ __forceinline__ void look_up(int t)
    {
        if (!a.table) return;
#pragma unroll
        for (int j = 0; j < N; ++j)
            page[j] = a.table[b * a.table_stride + a.by_page.div(min(t * kKeyTile + (int)row(j), kt.hi))];
    }

    __device__ __forceinline__ void copy(int t, u32 lds)
    {
        const int k0 = t * kKeyTile;
        if (!a.table && a.short_rows && k0 + kKeyTile - 1 <= kt.hi && (k0 >= kt.lo || k0 + kKeyTile <= a.sinks)) {
            const unsigned char* pk = a.k.p + b * a.k.sb + hk * a.k.sh + (int64_t)k0 * a.k.sl;
            const unsigned char* pv = a.v.p + b * a.v.sb + hk * a.v.sh + (int64_t)k0 * a.v.sl;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int part = j * NW + wave;
                if ((int)chunk(j) * 8 < a.D) {
                    dma16(pk + part * RPI * a.k.sl, ok + chunk(j) * 16, lds + part * 1024);
                    dma16(pv + part * RPI * a.v.sl, ov + chunk(j) * 16, lds + TILE + part * 1024);
                }
            }
            return;
        }
        // All pages at once, before copies are under way that a wait for one
        // of them would also wait for.
        if (a.table) settle_loads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int part = j * NW + wave, key = k0 + (int)row(j);
            const unsigned char *pk = (const unsigned char*)kAbsent.zero, *pv = pk;
            if (key <= kt.hi && (key >= kt.lo || key < a.sinks)) {
                int at = key, pg = b;
                if (a.table) {
                    pg = page[j];
                    at = key - (int)a.by_page.div(key) * (int)a.by_page.d;
                }
                if (a.table && (pg < 0 || pg >= a.pages)) {
                    pk = pv = (const unsigned char*)kAbsent.nan;
                } else {
                    const int64_t in = (int64_t)hk * a.k.sh + chunk(j) * 16;
                    pk = a.k.p + pg * a.k.sb + at * a.k.sl + in;
                    pv = a.v.p + (a.same_kv ? pg * a.k.sb + at * a.k.sl + in
                                            : pg * a.v.sb + at * a.v.sl + (int64_t)hk * a.v.sh + chunk(j) * 16);
                }
            }
            if ((int)chunk(j) * 8 < a.D) {
                dma16(pk, lds + part * 1024);
                dma16(pv, lds + TILE + part * 1024);
            }
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
