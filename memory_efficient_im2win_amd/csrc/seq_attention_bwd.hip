// Window attention, backward. With P = exp(S - lse) and D_i = dout_i . out_i,
//     dS = P o (dout V^T - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dout.
//
// Three kernels: the row statistics; dK and dV with a wave owning 32 keys and
// walking the rows that see them (the heads of a group are rows of one walk,
// so shared heads are summed in registers, in a fixed order); dQ with a wave
// owning 32 rows and walking their keys, as the forward pass does. P and dS
// are formed in both (7 products in place of 5), which needs no sums across
// workgroups. P and dS are rounded to the element type as operands, half a step
// each, independent from pair to pair. In fp16 they carry powers of two that
// keep them inside the type's range, taken out of the fp32 sums: 2^14 for P,
// and for dS one for each column of the result (a lane's key or row), chosen
// from the largest |dP - D| so far, as P is at most 1.
//
// Keys below `sinks` are seen by every later row. Their tiles' rows past the
// window are split into chunks of their own, whose sums join in fp32.
#include "seq_attention.hpp"

namespace im2win {
namespace seq {
namespace {

constexpr int kRowTile = 64, kKeysPerGroup = 128;

// The factor that dS carries in a column. Its first value and, when the
// products outgrow it, its next one bring the largest to 2^13 .. 2^14; they
// stay below 2^15 in between. bf16 has the range of fp32 and needs none.
template <bool BF>
struct Lift {
    float f = 0;  // 0: none chosen yet
    // top: this lane's largest |dP - D| of the tile. Scales acc with it.
    template <int MT>
    __device__ __forceinline__ void update(float top, floatx16_t (&acc)[MT])
    {
        if (BF) return;
        if (!__ballot(f == 0 ? top > 0 : top * f > 32768.0f)) return;
        const float most = half_max(top);
        if (f == 0 ? !(most > 0) : !(most * f > 32768.0f)) return;
        const int e = min(max(__builtin_amdgcn_frexp_expf(most), -100), 100);  // most < 2^e
        const float f1 = __builtin_amdgcn_ldexpf(1.0f, 14 - e);
        const float r = f == 0 ? 0.0f : f1 / f;
        f = f1;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt] *= r;
    }
    __device__ __forceinline__ float in() const { return BF ? 1.0f : f; }
    __device__ __forceinline__ float out() const { return BF || f == 0 ? 1.0f : 1.0f / f; }
};

// Row statistics: lse in log2 units (+infinity where a row sees nothing or is
// padding, so that its P is 0) and D. 16 lanes a row.
template <bool BF>
__global__ __launch_bounds__(256) void attn_stat_kernel(const AttnParams a)
{
    const int64_t row = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    const int bh = (int)(row / a.stat_rows), r = (int)(row % a.stat_rows), lane = threadIdx.x & 15;
    if (bh >= a.B * a.Hkv) return;
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const Span s(a, b);
    const int i = a.by_group.div(r), g = r - i * a.G;
    float lse = INFINITY, d = 0;
    if (r < a.rows && i < s.nq && s.off + i >= 0) {
        for (int c = lane * 8; c < a.D; c += 128) {
            const u32x4_t x = *(const u32x4_t*)row_ptr(a, a.out, b, hk, r, a.rows, c);
            const u32x4_t y = *(const u32x4_t*)row_ptr(a, a.dout, b, hk, r, a.rows, c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const floatx2_t u = unpack2<BF>(x[j]), v = unpack2<BF>(y[j]);
                d = fmaf(u[0], v[0], d);
                d = fmaf(u[1], v[1], d);
            }
        }
        const float v = a.lse[((int64_t)b * a.Hq + hk * a.G + g) * a.Lq + i];
        lse = v == -INFINITY ? INFINITY : v * kLog2e;
    }
#pragma unroll
    for (int k = 8; k; k >>= 1) d += __shfl_xor(d, k, 16);
    if (lane == 0) {
        a.stat_lse[row] = lse;
        a.stat_delta[row] = d;
    }
}

// Copies rows rt .. rt+63 of q and dout and their statistics into LDS.
template <int LP>
__device__ __forceinline__ void stage_rows(const AttnParams& a, int b, int hk, int bh, int rt, int r_end,
                                           u32 lds_q, u32 lds_d, u32 lds_s)
{
    constexpr int CH = LP / 8, RPI = 64 / CH, N = kRowTile / RPI / 4;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int part = j * 4 + wave;
        const u32 row = part * RPI + lane / CH;
        const u32 c = (lane % CH) ^ swz<LP>(row);
        dma16(row_ptr(a, a.q, b, hk, rt + row, r_end, c * 8), lds_q + part * 1024);
        dma16(row_ptr(a, a.dout, b, hk, rt + row, r_end, c * 8), lds_d + part * 1024);
    }
    if (wave == 0) {
        // Lanes 0-15: 64 values of lse, 16-31: of D; the rest copy zeros.
        const int64_t at = (int64_t)bh * a.stat_rows + rt + (lane & 15) * 4;
        const void* src = lane < 16 ? (const void*)(a.stat_lse + at)
                        : lane < 32 ? (const void*)(a.stat_delta + at) : (const void*)kAbsent.zero;
        dma16(src, lds_s);
    }
}

// dK and dV of 128 keys, 32 a wave. Workgroups past the key tiles take the
// chunks of sink rows.
template <bool BF, int DP>
__global__ __launch_bounds__(256, 1) void attn_dkv_kernel(const AttnParams a)
{
    constexpr int LP = row_pitch(DP), KS = DP / 16, MT = DP / 32, TILE = kRowTile * LP * 2, STAT = 1024;
    __shared__ __align__(1024) unsigned char smem[4 * TILE + 2 * STAT];
    const u32 lds = (u32)(uintptr_t)(lds_byte*)smem;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;

    const int items = a.key_tiles + a.sink_tiles * a.chunks;
    const int id = (int)xcd_tile(blockIdx.x, gridDim.x, true);
    const int item = id % items, bh = id / items, b = bh / a.Hkv, hk = bh % a.Hkv;
    const bool extra = item >= a.key_tiles;
    const int tile = extra ? (item - a.key_tiles) / a.chunks : item;
    const int chunk = extra ? (item - a.key_tiles) % a.chunks : -1;
    const Span s(a, b);
    const int kg = tile * kKeysPerGroup, kw = kg + wave * 32, key = kw + (lane & 31);

    // Rows of this walk: positions p0 .. p1.
    const int last = min(kg + kKeysPerGroup, s.nk) - 1;
    int p0 = kg, p1 = (int)min((int64_t)last + a.window - 1, (int64_t)s.nk - 1);
    if (extra) {
        p0 = (int)min((int64_t)kg + kKeysPerGroup - 1 + a.window + (int64_t)chunk * a.chunk_len, (int64_t)s.nk);
        p1 = (int)min((int64_t)p0 + a.chunk_len - 1, (int64_t)s.nk - 1);
    }
    const int i0 = max(0, p0 - s.off), i1 = p1 - s.off;
    // First row down to a multiple of 4: the statistics' copies are 16 bytes.
    // The up to 3 rows before i0 are masked by position.
    const int r_first = i0 * a.G, rt0 = r_first & ~3;
    const int r_end = last < kg || i1 < i0 ? 0 : (i1 + 1) * a.G;
    const int n = r_end > rt0 ? (r_end - rt0 + kRowTile - 1) / kRowTile : 0;

    if (n > 0) stage_rows<LP>(a, b, hk, bh, rt0, r_end, lds, lds + TILE, lds + 4 * TILE);

    u32x4_t kf[KS], vf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const int d = ks * 16 + h * 8;
        const bool in = key < s.nk && d < a.D;
        kf[ks] = *(const u32x4_t*)(in ? a.k.p + b * a.k.sb + key * a.k.sl + hk * a.k.sh + d * 2
                                      : (const unsigned char*)kAbsent.zero);
        vf[ks] = *(const u32x4_t*)(in ? a.v.p + b * a.v.sb + key * a.v.sl + hk * a.v.sh + d * 2
                                      : (const unsigned char*)kAbsent.zero);
    }
    const float c = a.scale * kLog2e;
    constexpr float kLift = BF ? 0.0f : 14.0f;  // log2 of P's factor
    Lift<BF> lift;
    floatx16_t dk[MT] = {}, dv[MT] = {};
    for (int t = 0; t < n; ++t) {
        const int rt = rt0 + t * kRowTile;
        const u32 bq = lds + (t & 1) * (2 * TILE), bd = bq + TILE, bs = lds + 4 * TILE + (t & 1) * STAT;
        sync_all();
        if (t + 1 < n) {
            const u32 nq = lds + ((t + 1) & 1) * (2 * TILE);
            stage_rows<LP>(a, b, hk, bh, rt + kRowTile, r_end, nq, nq + TILE, lds + 4 * TILE + ((t + 1) & 1) * STAT);
        }
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            const int ra = rt + sb * 32, rb = min(ra + 31, r_end - 1);
            if (ra >= r_end) continue;
            const int pa = s.off + (int)a.by_group.div(ra), pb = s.off + (int)a.by_group.div(rb);
            // Nothing here is seen by this wave's keys.
            if (pb < kw || (pa - (kw + 31) >= a.window && kw >= a.sinks)) continue;
            floatx16_t sc = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                sc = mfma<BF>(read_rows<LP>(bq, sb * 32 + (lane & 31), ks * 16 + h * 8), kf[ks], sc);
                dp = mfma<BF>(read_rows<LP>(bd, sb * 32 + (lane & 31), ks * 16 + h * 8), vf[ks], dp);
            }
            floatx4_t l2[4], dl[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const u32 at = bs + (sb * 32 + 8 * g + 4 * h) * 4;
                l2[g] = __builtin_bit_cast(floatx4_t, lds_read16(at));
                dl[g] = __builtin_bit_cast(floatx4_t, lds_read16(at + 256));
            }
            const bool whole = pa >= kw + 31 && pb - kw < a.window && ra >= r_first && ra + 31 < r_end;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = ra + 8 * (i / 4) + 4 * h + i % 4, p = s.off + (int)a.by_group.div(r);
                    const bool seen = r >= r_first && r < r_end && key <= p &&
                                      (p - key < a.window || key < a.sinks);
                    l2[i / 4][i % 4] = seen ? l2[i / 4][i % 4] : INFINITY;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] -= dl[i / 4][i % 4];
            if (!BF) {
                float top = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(dp[i]));
                lift.update(top, dk);
            }
            const float ld = BF ? 1.0f : lift.in() * 0x1p-14f;
            u32x4_t pr[2], ds[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float e[2], f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(fmaf(sc[i + j], c, kLift - l2[i / 4][i % 4 + j]));
                    f[j] = e[j] * (BF ? dp[i + j] : dp[i + j] * ld);
                }
                pr[i / 8][i % 8 / 2] = pack2<BF>(e[0], e[1]);
                ds[i / 8][i % 8 / 2] = pack2<BF>(f[0], f[1]);
            }
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    dv[mt] = mfma<BF>(read_cols<LP>(bd, sb * 32 + s2 * 16, mt * 32), pr[s2], dv[mt]);
                    dk[mt] = mfma<BF>(read_cols<LP>(bq, sb * 32 + s2 * 16, mt * 32), ds[s2], dk[mt]);
                }
        }
    }

    if (!BF) {
        const float f = lift.out();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            dk[mt] *= f;
            dv[mt] *= 0x1p-14f;
        }
    }
    if (tile < a.sink_tiles) {
        // [sequence and head][sink tile][1 + chunks][dk, dv][key][D]
        float* w = a.part + ((((int64_t)bh * a.sink_tiles + tile) * (a.chunks + 1) + chunk + 1) * 2 * kKeysPerGroup +
                             wave * 32 + (lane & 31)) * a.D;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const int d = mt * 32 + 8 * (j / 4) + 4 * h;
                if (d >= a.D) continue;
                const floatx4_t x = {dk[mt][j], dk[mt][j + 1], dk[mt][j + 2], dk[mt][j + 3]};
                const floatx4_t y = {dv[mt][j], dv[mt][j + 1], dv[mt][j + 2], dv[mt][j + 3]};
                *(floatx4_t*)(w + d) = x;
                *(floatx4_t*)(w + kKeysPerGroup * a.D + d) = y;
            }
        return;
    }
    if (key >= a.Lk) return;
    unsigned char* ok = a.dk.p + b * a.dk.sb + key * a.dk.sl + hk * a.dk.sh;
    unsigned char* ov = a.dv.p + b * a.dv.sb + key * a.dv.sl + hk * a.dv.sh;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const int d = mt * 32 + 8 * (j / 4) + 4 * h;
            if (d >= a.D) continue;
            const u32x2_t x = {pack2<BF>(dk[mt][j] * a.scale, dk[mt][j + 1] * a.scale),
                               pack2<BF>(dk[mt][j + 2] * a.scale, dk[mt][j + 3] * a.scale)};
            const u32x2_t y = {pack2<BF>(dv[mt][j], dv[mt][j + 1]), pack2<BF>(dv[mt][j + 2], dv[mt][j + 3])};
            *(u32x2_t*)(ok + d * 2) = x;
            *(u32x2_t*)(ov + d * 2) = y;
        }
}

// Sums a sink tile's parts in order. A quarter of D lanes hold a key.
template <bool BF>
__global__ __launch_bounds__(256) void attn_sink_join_kernel(const AttnParams a, int lanes)
{
    const int per = 256 / lanes, sub = threadIdx.x / lanes, d = threadIdx.x % lanes * 4;
    const int64_t at = (int64_t)blockIdx.x * per + sub;
    const int which = (int)(at & 1), k = (int)(at >> 1) % kKeysPerGroup;
    const int64_t bt = (at >> 1) / kKeysPerGroup;
    const int tile = (int)(bt % a.sink_tiles);
    const int64_t bh = bt / a.sink_tiles;
    const int key = tile * kKeysPerGroup + k;
    if (sub >= per || bh >= (int64_t)a.B * a.Hkv || d >= a.D || key >= a.Lk) return;
    const int b = (int)(bh / a.Hkv), hk = (int)(bh % a.Hkv);
    floatx4_t x = {0, 0, 0, 0};
    for (int c = 0; c <= a.chunks; ++c)
        x += *(const floatx4_t*)(a.part + (((bt * (a.chunks + 1) + c) * 2 + which) * kKeysPerGroup + k) * a.D + d);
    if (!which) x *= a.scale;
    const Tensor& t = which ? a.dv : a.dk;
    const u32x2_t w = {pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3])};
    *(u32x2_t*)(t.p + b * t.sb + key * t.sl + hk * t.sh + d * 2) = w;
}

// dQ of 128 flattened rows, 32 a wave.
template <bool BF, int DP>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(const AttnParams a)
{
    constexpr int NW = 4, LP = row_pitch(DP), KS = DP / 16, MT = DP / 32, TILE = kKeyTile * LP * 2;
    __shared__ __align__(1024) unsigned char smem[4 * TILE];
    const u32 lds = (u32)(uintptr_t)(lds_byte*)smem;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), h = lane >> 5;

    const int id = (int)xcd_tile(blockIdx.x, gridDim.x, true);
    const int tile = id % a.tiles, bh = id / a.tiles, b = bh / a.Hkv, hk = bh % a.Hkv;
    const Span s(a, b);
    const int r0 = tile * (NW * 32), rw = r0 + wave * 32, r = rw + (lane & 31), r_end = s.nq * a.G;
    const int i0 = a.by_group.div(r0), i1 = min((int)a.by_group.div(min(r0 + NW * 32, a.rows) - 1), s.nq - 1);
    const KeyTiles kt(a, s, i0, i1);
    const int pw_lo = s.off + (int)a.by_group.div(rw), pw_hi = s.off + min((int)a.by_group.div(rw + 31), s.nq - 1);
    const int p = s.off + (int)a.by_group.div(r);

    if (kt.n > 0) stage_keys<LP, NW>(a, a.k, a.v, b, hk, kt, kt.at(0), lds, lds + TILE);

    u32x4_t q[KS], dout[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        q[ks] = *(const u32x4_t*)row_ptr(a, a.q, b, hk, r, r_end, ks * 16 + h * 8);
        dout[ks] = *(const u32x4_t*)row_ptr(a, a.dout, b, hk, r, r_end, ks * 16 + h * 8);
    }
    float l2 = INFINITY, delta = 0;
    if (r < a.rows) {
        l2 = a.stat_lse[(int64_t)bh * a.stat_rows + r];
        delta = a.stat_delta[(int64_t)bh * a.stat_rows + r];
    }
    const float c = a.scale * kLog2e;

    Lift<BF> lift;
    floatx16_t dq[MT] = {};
    for (int it = 0; it < kt.n; ++it) {
        const u32 buf = lds + (it & 1) * (2 * TILE), nbuf = lds + ((it + 1) & 1) * (2 * TILE);
        sync_all();
        if (it + 1 < kt.n) stage_keys<LP, NW>(a, a.k, a.v, b, hk, kt, kt.at(it + 1), nbuf, nbuf + TILE);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int k0 = kt.at(it) * kKeyTile + kb * 32;
            if (rw >= r_end || k0 > pw_hi || (k0 + 31 <= pw_lo - a.window && k0 >= a.sinks)) continue;
            floatx16_t sc = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                sc = mfma<BF>(read_rows<LP>(buf, kb * 32 + (lane & 31), ks * 16 + h * 8), q[ks], sc);
                dp = mfma<BF>(read_rows<LP>(buf + TILE, kb * 32 + (lane & 31), ks * 16 + h * 8), dout[ks], dp);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = fmaf(sc[i], c, -l2);
            if (k0 + 31 > pw_lo || k0 <= pw_hi - a.window) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int j = k0 + 8 * (i / 4) + 4 * h + i % 4;
                    const bool seen = j <= p && (j > p - a.window || j < a.sinks);
                    sc[i] = seen ? sc[i] : -INFINITY;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] -= delta;
            if (!BF) {
                float top = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(dp[i]));
                lift.update(top, dq);
            }
            const float ld = lift.in();
            u32x4_t ds[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float e0 = __builtin_amdgcn_exp2f(sc[i]), e1 = __builtin_amdgcn_exp2f(sc[i + 1]);
                ds[i / 8][i % 8 / 2] = BF ? pack2<BF>(e0 * dp[i], e1 * dp[i + 1])
                                          : pack2<BF>(e0 * (dp[i] * ld), e1 * (dp[i + 1] * ld));
            }
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    dq[mt] = mfma<BF>(read_cols<LP>(buf, kb * 32 + s2 * 16, mt * 32), ds[s2], dq[mt]);
        }
    }
    if (r >= a.rows) return;
    const float back = a.scale * lift.out();
    const int i = a.by_group.div(r), g = r - i * a.G;
    unsigned char* out = a.dq.p + b * a.dq.sb + i * a.dq.sl + (int64_t)(hk * a.G + g) * a.dq.sh;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const int d = mt * 32 + 8 * (j / 4) + 4 * h;
            u32x2_t w = {pack2<BF>(dq[mt][j] * back, dq[mt][j + 1] * back),
                         pack2<BF>(dq[mt][j + 2] * back, dq[mt][j + 3] * back)};
            if (r >= r_end) w = (u32x2_t)(0u);
            if (d < a.D) *(u32x2_t*)(out + d * 2) = w;
        }
}

template <bool BF>
int run(AttnParams a, hipStream_t st)
{
    const int64_t heads = (int64_t)a.B * a.Hkv;
    attn_stat_kernel<BF><<<(unsigned)((heads * a.stat_rows + 15) / 16), 256, 0, st>>>(a);
    int rc = launch_status();
    if (rc != 0) return rc;
    a.tiles = ceil_div(a.rows, 128);
    rc = with_head(a.D, [&](auto DP) {
        const int items = a.key_tiles + a.sink_tiles * a.chunks;
        if (items) attn_dkv_kernel<BF, DP.value><<<(unsigned)(heads * items), 256, 0, st>>>(a);
        if (a.tiles) attn_dq_kernel<BF, DP.value><<<(unsigned)(heads * a.tiles), 256, 0, st>>>(a);
        return launch_status();
    });
    if (rc != 0 || a.sink_tiles == 0) return rc;
    const int lanes = a.D / 4, per = 256 / lanes;
    const int64_t all = heads * a.sink_tiles * kKeysPerGroup * 2;
    attn_sink_join_kernel<BF><<<(unsigned)((all + per - 1) / per), 256, 0, st>>>(a, lanes);
    return launch_status();
}

}  // namespace

// Sink keys' rows past the window are cut into chunks as long as the window's
// own walk, so that no workgroup walks much longer than the others.
AttnBwdPlan attn_bwd_plan(const AttnParams& a)
{
    AttnBwdPlan p{};
    p.stat_rows = ceil_div(a.rows, kRowTile) * kRowTile + kRowTile;
    p.key_tiles = ceil_div(a.Lk, kKeysPerGroup);
    p.chunk_len = (int)std::min<int64_t>((int64_t)a.window + kKeysPerGroup, a.Lk);
    // Positions past the first key tile's window, if any key there is a sink.
    const int64_t past = (int64_t)a.Lk - (kKeysPerGroup - 1) - a.window;
    if (a.sinks > 0 && past > 0) {
        p.sink_tiles = ceil_div(std::min(a.sinks, a.Lk), kKeysPerGroup);
        p.chunks = (int)((past + p.chunk_len - 1) / p.chunk_len);
    }
    const size_t heads = (size_t)a.B * a.Hkv;
    p.stat_bytes = heads * p.stat_rows * 4;
    p.ws_bytes = 2 * p.stat_bytes +
                 heads * p.sink_tiles * (p.chunks + 1) * 2 * kKeysPerGroup * (size_t)a.D * 4;
    return p;
}

int launch_attn_bwd(AttnParams a, const AttnBwdPlan& p, void* ws, bool bf, hipStream_t st)
{
    unsigned char* w = static_cast<unsigned char*>(ws);
    a.stat_lse = reinterpret_cast<float*>(w);
    a.stat_delta = reinterpret_cast<float*>(w + p.stat_bytes);
    a.part = reinterpret_cast<float*>(w + 2 * p.stat_bytes);
    a.stat_rows = p.stat_rows;
    a.key_tiles = p.key_tiles;
    a.sink_tiles = p.sink_tiles;
    a.chunks = p.chunks;
    a.chunk_len = p.chunk_len;
    return bf ? run<true>(a, st) : run<false>(a, st);
}

}  // namespace seq
}  // namespace im2win
