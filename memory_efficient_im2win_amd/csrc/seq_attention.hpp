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

// Copies keys 64*t .. 64*t+63 of x (k or v) into the LDS tile at `lds`. Keys
// that no row of the tile sees arrive as zeros, so what they hold in memory
// does not matter; those of a page outside the pool as NaN.
template <int LP, int NW>
__device__ __forceinline__ void stage_keys(const AttnParams& a, const Tensor& k, const Tensor& v, int b,
                                           int hk, const KeyTiles& kt, int t, u32 lds_k, u32 lds_v)
{
    constexpr int CH = LP / 8, RPI = 64 / CH, N = kKeyTile / RPI / NW;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int part = j * NW + wave;
        const u32 row = part * RPI + lane / CH;
        const u32 c = (lane % CH) ^ swz<LP>(row);
        const int key = t * kKeyTile + (int)row;
        const unsigned char *pk = (const unsigned char*)kAbsent.zero, *pv = pk;
        if (key <= kt.hi && (key >= kt.lo || key < a.sinks) && (int)c * 8 < a.D) {
            int64_t ok, ov;
            bool good = true;
            if (a.table) {
                const u32 in = a.by_page.div(key);
                const int page = a.table[b * a.table_stride + in];
                const int at = key - in * a.by_page.d;
                good = page >= 0 && page < a.pages;
                ok = page * k.sb + at * k.sl;
                ov = page * v.sb + at * v.sl;
            } else {
                ok = b * k.sb + key * k.sl;
                ov = b * v.sb + key * v.sl;
            }
            pk = good ? k.p + ok + hk * k.sh + c * 16 : (const unsigned char*)kAbsent.nan;
            pv = good ? v.p + ov + hk * v.sh + c * 16 : (const unsigned char*)kAbsent.nan;
        }
        dma16(pk, lds_k + part * 1024);
        dma16(pv, lds_v + part * 1024);
    }
}

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
