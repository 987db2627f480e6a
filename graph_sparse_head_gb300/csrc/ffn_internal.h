// Declarations shared by the feed-forward block's translation units.
#pragma once

#include <algorithm>

#include "pmha_internal.h"

namespace pmha {

// Tensor-core products of the bf16 block (ffn_tc.cu). Row-major operands with
// 16-byte row pitches (E and F multiples of 8; E of 16 for E4M3 tokens).
struct FfnTc {
    int64_t E, F;
    pmha_act act;
    const void *bg, *bu, *bd;  // (F), (F), (E) bf16 or null
};
// h (M, F) = act(x Wg^T + bg) * (x Wu^T + bu); with q8 x, wg, wu are E4M3
// with scales a row.
struct FfnUpArgs {
    const void *x, *wg, *wu;
    const float *x_scale, *wg_scale, *wu_scale;  // null for bf16 operands
    int64_t M;
    void *h;
};
pmha_status ffn_tc_up(const FfnTc &f, const FfnUpArgs &a, cudaStream_t s);
// out (M, E) = h Wd^T + bd + residual
pmha_status ffn_tc_down(const FfnTc &f, const void *h, const void *wd, const void *residual, int64_t M, void *out,
                        cudaStream_t s);
// The whole forward in one kernel, the hidden rows on the chip (ffn_fused.cu).
bool ffn_fused_supported(int64_t E, int64_t F);
pmha_status ffn_fused_forward(const FfnTc &f, const FfnUpArgs &a, const void *wd, const void *residual, void *out,
                              cudaStream_t s);
// The same for a few tokens, on the CUDA cores (ffn_small.cu); any widths, float32 too.
bool ffn_small_supported(int64_t E, int64_t M, int token_bytes);
pmha_status ffn_small_forward(const FfnTc &f, bool f32, const FfnUpArgs &a, const void *wd, const void *residual,
                              void *out, cudaStream_t s);
// h, dg, du (M, F): the hidden row and the gradients of gate and up, from x,
// dout and wd_t (F, E) = Wd transposed
struct FfnHiddenArgs {
    const void *x, *dy, *wg, *wu, *wd_t;
    int64_t M;
    void *h, *dg, *du;
    // null, or ffn_hidden_parts() rows of [2][F] partial column sums of dg and du, added to (zero before the first)
    float *sums;
};
int64_t ffn_hidden_parts(int64_t M, int64_t F);
pmha_status ffn_tc_hidden(const FfnTc &f, const FfnHiddenArgs &a, cudaStream_t s);
// The same from one kernel that keeps the tokens on the chip and, where
// ffn_fused_dx(E), forms dx (M, E) too.
bool ffn_fused_dx(int64_t E);
pmha_status ffn_fused_backward(const FfnTc &f, const FfnHiddenArgs &a, const void *wg_t, const void *wu_t, void *dx,
                               cudaStream_t s);
// dx (M, E) = dg Wg + du Wu from the transposed weights (E, F)
pmha_status ffn_tc_dx(const FfnTc &f, const void *dg, const void *du, const void *wg_t, const void *wu_t, int64_t M,
                      void *dx, cudaStream_t s);
// Partial weight gradients over the M rows, all three as (F, E) float32:
// part[split][0..2] (+)= dg^T x, du^T x, h^T dy; the row range is cut into
// ffn_dw_splits() pieces. `accumulate` adds to what part holds. sums, where not
// null, takes column sums of dy, (split, E).
struct FfnDwArgs {
    const void *dg, *du, *h, *x, *dy;
    int64_t M;
    float *part, *sums;
    bool gate_up, down;  // which of the products are wanted
    bool accumulate;
    int splits;
};
int ffn_dw_splits(int64_t E, int64_t F, int64_t rows_per_block);
pmha_status ffn_tc_dw(const FfnTc &f, const FfnDwArgs &a, cudaStream_t s);

// Products of a float32 block (ffn_f32.cu), over M rows.
struct FfnF32Args {
    const float *x, *dy, *wg, *wu, *wd, *bg, *bu, *bd, *res;
    float *h, *dg, *du, *out;
    int64_t M, E, F;
};
pmha_status ffn_f32_hidden(pmha_act act, const FfnF32Args &a, bool backward, cudaStream_t s);
pmha_status ffn_f32_down(const FfnF32Args &a, cudaStream_t s);
// dx, or with parts > 1 as many arrays (M, E), one after the other, that add up to it
int ffn_f32_dx_parts(int64_t E, int64_t F, int64_t rows);
pmha_status ffn_f32_dx(const FfnF32Args &a, int parts, cudaStream_t s);
int ffn_f32_splits(int64_t E, int64_t F, int64_t rows);
pmha_status ffn_f32_dw(const FfnF32Args &a, float *part, int splits, bool accumulate, cudaStream_t s);

}  // namespace pmha
