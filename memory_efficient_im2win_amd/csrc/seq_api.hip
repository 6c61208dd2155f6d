// C ABI of the sequence operators: argument checks, workspaces and dispatch.
// The contract is in include/im2win_seq.h. Nothing here allocates or throws.
#include <math.h>

#include "im2win.h"
#include "im2win_seq.h"
#include "seq_kernels.hpp"

namespace {

using im2win::FastDiv;
using im2win::seq::AttnBwdPlan;
using im2win::seq::AttnParams;
using im2win::seq::AttnPlan;
using im2win::seq::LinJob;
using im2win::seq::LinParams;
using im2win::seq::LinPlan;
using im2win::seq::Tensor;

constexpr int kMost = 1 << 30;         // tokens, flattened rows
constexpr int64_t kGrid = 0x7fffffff;  // workgroups of a launch

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A 16-bit tensor of `elems` elements: strides and base fit 16-byte accesses,
// and 32-bit offsets reach across a tile of tokens.
bool good(const seq_tensor& t, int64_t elems)
{
    if (elems == 0) return true;
    return t.p && aligned(t.p, 16) && t.stride_b >= 0 && t.stride_l >= 0 && t.stride_h >= 0 && t.stride_b % 8 == 0 &&
           t.stride_l % 8 == 0 && t.stride_h % 8 == 0 && t.stride_l < (1 << 24);
}

bool good_head(int d) { return d >= 8 && d <= 128 && d % 8 == 0; }

Tensor tensor(const seq_tensor& t)
{
    return Tensor{static_cast<unsigned char*>(t.p), t.stride_b * 2, t.stride_l * 2, t.stride_h * 2};
}

int status_of(int rc) { return rc == 0 ? IM2WIN_OK : IM2WIN_ELAUNCH; }

int check_ws(const void* ws, size_t have, size_t need)
{
    if (have < need || (!ws && (need || have))) return IM2WIN_EWORKSPACE;
    return aligned(ws, 16) ? IM2WIN_OK : IM2WIN_EINVAL;
}

// Sizes only; fills what the plans need.
bool attn_sizes(const seq_attention* a, AttnParams* p)
{
    if (!a || (a->dtype != 0 && a->dtype != 1)) return false;
    if (a->B < 0 || a->Lq < 0 || a->Lk < 0 || a->Lq > kMost || a->Lk > kMost) return false;
    if (a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv || !good_head(a->D)) return false;
    if (a->window < 1 || a->sinks < 0 || !isfinite(a->scale)) return false;
    if (a->page_table ? a->page < 1 || a->pages < 0 : a->page != 0 || a->pages != 0) return false;
    const int G = a->Hq / a->Hkv;
    if ((int64_t)a->Lq * G > kMost) return false;
    // Row and key tiles of every launch, with the most splits a plan makes.
    if ((int64_t)a->B * a->Hkv * ((int64_t)a->Lq * G / 32 + 1) * 2 > kGrid - 1024) return false;
    if ((int64_t)a->B * a->Hkv * (a->Lk / 64 + 2) > kGrid / 4) return false;
    AttnParams z{};
    *p = z;
    p->B = a->B, p->Lq = a->Lq, p->Lk = a->Lk, p->Hq = a->Hq, p->Hkv = a->Hkv, p->D = a->D;
    p->G = G;
    p->rows = a->Lq * G;
    p->pages = a->pages;
    p->window = a->window < a->Lk ? a->window : (a->Lk > 1 ? a->Lk : 1);
    p->sinks = a->sinks < a->Lk ? a->sinks : a->Lk;
    p->scale = a->scale;
    p->by_group = FastDiv((uint32_t)G);
    p->by_page = FastDiv((uint32_t)(a->page_table ? a->page : 1));
    return true;
}

bool attn_params(const seq_attention* a, AttnParams* p)
{
    if (!attn_sizes(a, p)) return false;
    const int64_t nq = (int64_t)a->B * a->Lq;
    const int64_t nk = a->page_table ? (int64_t)a->pages : (int64_t)a->B * a->Lk;
    if (!good(a->q, nq) || !good(a->out, nq) || !good(a->k, nk) || !good(a->v, nk)) return false;
    if (!aligned(a->lse, 4) || !aligned(a->q_lens, 4) || !aligned(a->kv_lens, 4) || !aligned(a->page_table, 4))
        return false;
    p->q = tensor(a->q), p->k = tensor(a->k), p->v = tensor(a->v), p->out = tensor(a->out);
    p->lse = a->lse, p->q_lens = a->q_lens, p->kv_lens = a->kv_lens;
    p->table = a->page_table, p->table_stride = a->table_stride;
    return true;
}

bool linear_sizes(const seq_linear* a)
{
    if (!a || (a->dtype != 0 && a->dtype != 1)) return false;
    if (a->B < 0 || a->L < 0 || a->L > kMost || a->H < 1 || !good_head(a->Dk) || !good_head(a->Dv)) return false;
    if (!isfinite(a->scale)) return false;
    return (int64_t)a->B * a->H * 2 * ((int64_t)a->L / 64 + 64) <= kGrid;
}

bool linear_args(const seq_linear* a)
{
    if (!linear_sizes(a)) return false;
    const int64_t n = (int64_t)a->B * a->L;
    if (!good(a->q, n) || !good(a->k, n) || !good(a->v, n)) return false;
    if (!a->log_decay || !aligned(a->log_decay, 4) || !aligned(a->lens, 4)) return false;
    return aligned(a->state_in, 16) && aligned(a->state_out, 16);
}

LinParams linear_params(const seq_linear* a, int jobs, const LinPlan& plan)
{
    LinParams p{};
    p.log_decay = a->log_decay;
    p.lens = a->lens;
    p.jobs = jobs, p.B = a->B, p.L = a->L, p.H = a->H;
    p.nseg = plan.nseg, p.seg_len = plan.seg_len;
    return p;
}

// The recurrences of a backward call: dq on its own; dk and dv over the same
// tensors together where both heads pad to one size, else dk beside dq, whose
// states are dv x dk too, and dv on its own.
struct BackwardPlan {
    bool pair;
    LinPlan dq, dk, dv;
    size_t dq_bytes, dk_bytes, ws_bytes;
};

BackwardPlan backward_plan(const seq_linear* a)
{
    BackwardPlan p{};
    p.pair = im2win::seq::padded_head(a->Dk) == im2win::seq::padded_head(a->Dv);
    p.dq = im2win::seq::lin_plan(p.pair ? 1 : 2, a->B, a->L, a->H);
    p.dv = im2win::seq::lin_plan(p.pair ? 2 : 1, a->B, a->L, a->H);
    p.dk = p.pair ? p.dv : p.dq;
    p.dq_bytes = im2win::seq::lin_seg_bytes(p.dq, a->B, a->H, a->Dv, a->Dk);
    p.dk_bytes = im2win::seq::lin_seg_bytes(p.dk, a->B, a->H, a->Dv, a->Dk);
    p.ws_bytes = p.dq_bytes + p.dk_bytes + im2win::seq::lin_seg_bytes(p.dv, a->B, a->H, a->Dk, a->Dv);
    return p;
}

}  // namespace

extern "C" {

size_t im2win_seq_attention_workspace_bytes(const seq_attention* a)
{
    AttnParams p;
    if (!attn_sizes(a, &p) || p.B == 0 || p.Lq == 0) return 0;
    return im2win::seq::attn_plan(p).ws_bytes;
}

int im2win_seq_attention(const seq_attention* a, void* ws, size_t ws_bytes, void* stream)
{
    AttnParams p;
    if (!attn_params(a, &p)) return IM2WIN_EINVAL;
    if (p.B == 0 || p.Lq == 0) return IM2WIN_OK;
    const AttnPlan plan = im2win::seq::attn_plan(p);
    const int st = check_ws(ws, ws_bytes, plan.ws_bytes);
    if (st != IM2WIN_OK) return st;
    p.part = static_cast<float*>(ws);
    return status_of(im2win::seq::launch_attn_fwd(p, plan, a->dtype == 1, static_cast<hipStream_t>(stream)));
}

size_t im2win_seq_attention_backward_workspace_bytes(const seq_attention* a)
{
    AttnParams p;
    if (!attn_sizes(a, &p) || p.B == 0 || a->page_table) return 0;
    return im2win::seq::attn_bwd_plan(p).ws_bytes;
}

int im2win_seq_attention_backward(const seq_attention* a, void* ws, size_t ws_bytes, void* stream)
{
    AttnParams p;
    if (!attn_params(a, &p) || a->page_table) return IM2WIN_EINVAL;
    const int64_t nq = (int64_t)a->B * a->Lq, nk = (int64_t)a->B * a->Lk;
    if (!good(a->dout, nq) || !good(a->dq, nq) || !good(a->dk, nk) || !good(a->dv, nk)) return IM2WIN_EINVAL;
    if (nq && !a->lse) return IM2WIN_EINVAL;
    if (p.B == 0 || (p.Lq == 0 && p.Lk == 0)) return IM2WIN_OK;
    const AttnBwdPlan plan = im2win::seq::attn_bwd_plan(p);
    const int st = check_ws(ws, ws_bytes, plan.ws_bytes);
    if (st != IM2WIN_OK) return st;
    p.dout = tensor(a->dout), p.dq = tensor(a->dq), p.dk = tensor(a->dk), p.dv = tensor(a->dv);
    return status_of(im2win::seq::launch_attn_bwd(p, plan, ws, a->dtype == 1, static_cast<hipStream_t>(stream)));
}

size_t im2win_seq_linear_workspace_bytes(const seq_linear* a)
{
    if (!linear_sizes(a) || a->B == 0) return 0;
    const LinPlan plan = im2win::seq::lin_plan(1, a->B, a->L, a->H);
    return im2win::seq::lin_seg_bytes(plan, a->B, a->H, a->Dk, a->Dv);
}

int im2win_seq_linear(const seq_linear* a, void* ws, size_t ws_bytes, void* stream)
{
    if (!linear_args(a) || !good(a->out, (int64_t)a->B * a->L)) return IM2WIN_EINVAL;
    if (a->B == 0) return IM2WIN_OK;
    const LinPlan plan = im2win::seq::lin_plan(1, a->B, a->L, a->H);
    const int st = check_ws(ws, ws_bytes, im2win::seq::lin_seg_bytes(plan, a->B, a->H, a->Dk, a->Dv));
    if (st != IM2WIN_OK) return st;
    LinParams p = linear_params(a, 1, plan);
    p.job[0] = LinJob{tensor(a->q), tensor(a->k), tensor(a->v), tensor(a->out), a->state_in, a->state_out,
                      a->Dv, 1, a->Dk, a->Dv, 0, 1, a->scale, a->scale, 1.0f, static_cast<float*>(ws)};
    return status_of(im2win::seq::launch_linear(p, false, a->dtype == 1, static_cast<hipStream_t>(stream)));
}

int im2win_seq_linear_step(const seq_linear* a, void* stream)
{
    if (!linear_args(a) || a->L != 1 || a->lens || !good(a->out, a->B)) return IM2WIN_EINVAL;
    if (!a->state_in || a->state_in != a->state_out) return IM2WIN_EINVAL;
    if (a->B == 0) return IM2WIN_OK;
    const im2win::seq::LinStep p{tensor(a->q), tensor(a->k), tensor(a->v), tensor(a->out), a->log_decay, a->state_out,
                                 a->B, a->H, a->Dk, a->Dv, a->scale};
    return status_of(im2win::seq::launch_linear_step(p, a->dtype == 1, static_cast<hipStream_t>(stream)));
}

size_t im2win_seq_linear_backward_workspace_bytes(const seq_linear* a)
{
    if (!linear_sizes(a) || a->B == 0) return 0;
    return backward_plan(a).ws_bytes;
}

int im2win_seq_linear_backward(const seq_linear* a, void* ws, size_t ws_bytes, void* stream)
{
    const int64_t n = a ? (int64_t)a->B * a->L : 0;
    if (!linear_args(a) || !good(a->dout, n) || !good(a->dq, n) || !good(a->dk, n) || !good(a->dv, n))
        return IM2WIN_EINVAL;
    if (!aligned(a->dstate_out, 16) || !aligned(a->dstate_in, 16)) return IM2WIN_EINVAL;
    if (a->B == 0) return IM2WIN_OK;
    const BackwardPlan plan = backward_plan(a);
    const int st = check_ws(ws, ws_bytes, plan.ws_bytes);
    if (st != IM2WIN_OK) return st;
    unsigned char* w = static_cast<unsigned char*>(ws);
    const bool bf = a->dtype == 1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Tensor q = tensor(a->q), k = tensor(a->k), v = tensor(a->v), dout = tensor(a->dout);
    // The states are transposed (rows dv, columns dk) for dq and dk.
    const LinJob dq{dout, v, k, tensor(a->dq), a->state_in, nullptr, 1, a->Dv, a->Dv, a->Dk, 0, 1,
                    a->scale, a->scale, 1.0f, reinterpret_cast<float*>(w)};
    const LinJob dk{v, dout, q, tensor(a->dk), a->dstate_out, nullptr, 1, a->Dv, a->Dv, a->Dk, 1, 0,
                    a->scale, 1.0f, a->scale, reinterpret_cast<float*>(w + plan.dq_bytes)};
    const LinJob dv{k, q, dout, tensor(a->dv), a->dstate_out, a->dstate_in, a->Dv, 1, a->Dk, a->Dv, 1, 0,
                    a->scale, 1.0f, a->scale, reinterpret_cast<float*>(w + plan.dq_bytes + plan.dk_bytes)};
    LinParams p = linear_params(a, plan.pair ? 1 : 2, plan.dq);
    p.job[0] = dq;
    p.job[1] = dk;
    const int rc = im2win::seq::launch_linear(p, false, bf, s);
    if (rc != 0) return status_of(rc);
    p = linear_params(a, plan.pair ? 2 : 1, plan.dv);
    p.job[0] = plan.pair ? dk : dv;
    p.job[1] = dv;
    return status_of(im2win::seq::launch_linear(p, plan.pair, bf, s));
}

}  // extern "C"
