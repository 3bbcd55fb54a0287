/*
 * fp64 CPU oracle for the RWKV-4 WKV operator and the token-shift lerp.
 *
 * TEST INFRASTRUCTURE.  Only the test suite, the smoke check and the
 * benchmark's CPU-baseline leg may load or run this code.  The CUDA library
 * never links, includes or calls it, and the two share no code, headers,
 * tables or constants.  Plain, slow and obviously correct on purpose: every
 * loop follows the formula it cites, term by term, in double precision.
 * OpenMP only distributes independent channels over threads; it changes no
 * arithmetic.
 *
 * Sources (web pages on RWKV; cited by page and section):
 *   [MATH]  "RWKV" transformer-math page (aicassindra.com, tm_rwkv_math):
 *           section "The WKV operator: attention with a fixed decay" (the
 *           wkv_t equation, w = exp(omega) > 0, u the current-token bonus);
 *           section "Why it collapses into a recurrence" (the a_t, b_t
 *           recurrence with a_0 = b_0 = 0); section "Numerical stability:
 *           carry the exponent" (the (p, a, b) form); section "Token shift:
 *           a two-tap causal convolution" (the lerp).
 *   [WIKI]  "RWKV" (aiwiki.thehackersbrain.dev): eq. 1 and the one-token
 *           decode step in the stabilised form.
 *           Also section "Receptance: the gate on the way out" (the output is
 *           sigma(r) times wkv, channel by channel) and, in section "Token shift",
 *           the separate mu_r, mu_k, mu_v of the three projections.
 *   [VANOS] "RWKV (Attention-RNN Hybrid)" (vanos001.github.io): section
 *           "Versions: RWKV-4 -> Eagle -> Finch" (the Eagle matrix-state
 *           recurrence S_t = diag(d) S_{t-1} + k_t v_t^T read out as
 *           y_t = r_t^T S_t, one 64 x 64 state per head) and section
 *           "O(N) Inference Characteristics" (decode is one matrix-vector
 *           product against the state).
 *   [MULTI] "RWKV and Recurrent Models With Transformer Quality"
 *           (multigrid.ai): section "Prefill, decode, and where each form is
 *           used" (prefill yields the state after the last prompt token;
 *           decode steps from it).
 *
 * Indexing: 0-based t in [0, T).  eq. 1 at position t sums the past i < t with
 * weight exp(-(t-1-i) w + k_i) and the current token with exp(u + k_t); the
 * most recent past token (i = t-1) is not decayed.
 *
 * Layouts: k, v, y, s are [B][T][C] row-major; w, u are [C]; a state is
 * [3][B][C] holding (a, b, p) with true accumulators A = a e^p, B = b e^p.
 *
 * Every function also returns the "magnitude scale" s: the same weighted
 * average with |v| in place of v.  It is what the tests divide errors by
 * (|y| can be near zero while the terms that produced it are not).
 */
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>
#ifdef _OPENMP
#include <omp.h>
#endif

/* Initial running maximum for an empty state: finite, so p - w never forms
 * inf - inf, and far below any exponent the data can produce. */
#define ORACLE_P_EMPTY (-1e38)

static inline size_t at3(int64_t b, int64_t t, int64_t c, int64_t T, int64_t C)
{
    return ((size_t)b * (size_t)T + (size_t)t) * (size_t)C + (size_t)c;
}

int oracle_num_threads(void)
{
#ifdef _OPENMP
    return omp_get_max_threads();
#else
    return 1;
#endif
}

/* Threads for the parallel loops that follow (timing only: every loop distributes independent
 * channels, so the results do not depend on it). */
void oracle_set_num_threads(int n)
{
#ifdef _OPENMP
    if (n > 0) omp_set_num_threads(n);
#else
    (void)n;
#endif
}

/*
 * Direct evaluation of the wkv_t equation ([MATH] "The WKV operator: attention
 * with a fixed decay"; [WIKI] eq. 1), O(T^2) per channel, no stabilisation.
 * Valid while every exponent -(t-1-i) w + k_i and u + k_t stays below ~709.
 *   y[b,t,c] = (sum_{i<t} e^{-(t-1-i)w + k_i} v_i + e^{u + k_t} v_t)
 *            / (sum_{i<t} e^{-(t-1-i)w + k_i}     + e^{u + k_t})
 * s (may be NULL) is the same ratio with |v| in place of v.
 */
void oracle_wkv_direct(int64_t B, int64_t T, int64_t C, const double* w, const double* u,
                       const double* k, const double* v, double* y, double* s)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t c = 0; c < C; ++c)
            for (int64_t t = 0; t < T; ++t) {
                double num = 0.0, den = 0.0, mag = 0.0;
                for (int64_t i = 0; i < t; ++i) {
                    double e = exp(-(double)(t - 1 - i) * w[c] + k[at3(b, i, c, T, C)]);
                    num += e * v[at3(b, i, c, T, C)];
                    mag += e * fabs(v[at3(b, i, c, T, C)]);
                    den += e;
                }
                double e = exp(u[c] + k[at3(b, t, c, T, C)]);
                num += e * v[at3(b, t, c, T, C)];
                mag += e * fabs(v[at3(b, t, c, T, C)]);
                den += e;
                y[at3(b, t, c, T, C)] = num / den;
                if (s) s[at3(b, t, c, T, C)] = mag / den;
            }
}

/*
 * The running-maximum form ([MATH] "Numerical stability: carry the exponent";
 * [WIKI] decode step), applied token after token.  Per channel, with state
 * (a, b, p):
 *   output:  q = max(p, u + k_t)
 *            y_t = (e^{p-q} a + e^{u+k_t-q} v_t) / (e^{p-q} b + e^{u+k_t-q})
 *   update:  p' = max(p - w, k_t)
 *            a' = e^{p-w-p'} a + e^{k_t-p'} v_t
 *            b' = e^{p-w-p'} b + e^{k_t-p'}
 * The empty state is a = b = 0 with p = ORACLE_P_EMPTY.
 *
 * state_in  [3][B][C] (a, b, p) or NULL for the empty state.
 * sacc_in   [B][C] magnitude accumulator (a with |v|) or NULL for zeros.
 * y, s      [B][T][C]; s may be NULL.
 * state_out [3][B][C] or NULL; sacc_out [B][C] or NULL.
 * T may be 0 (state is copied through).  With T = 1 this is exactly one decode
 * step from a given state ([MULTI] "Prefill, decode, and where each form is
 * used").
 */
void oracle_wkv_recurrent(int64_t B, int64_t T, int64_t C, const double* w, const double* u,
                          const double* k, const double* v, const double* state_in,
                          const double* sacc_in, double* y, double* s, double* state_out,
                          double* sacc_out)
{
    const size_t BC = (size_t)B * (size_t)C;
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t c = 0; c < C; ++c) {
            size_t bc = (size_t)b * (size_t)C + (size_t)c;
            double a = 0.0, bb = 0.0, p = ORACLE_P_EMPTY, sa = 0.0;
            if (state_in) {
                a = state_in[bc];
                bb = state_in[BC + bc];
                p = state_in[2 * BC + bc];
            }
            if (sacc_in) sa = sacc_in[bc];
            for (int64_t t = 0; t < T; ++t) {
                double kt = k[at3(b, t, c, T, C)];
                double vt = v[at3(b, t, c, T, C)];
                /* output */
                double q = fmax(p, u[c] + kt);
                double w_past = exp(p - q);         /* weight of the carried history */
                double w_now = exp(u[c] + kt - q);  /* weight of the current token */
                double den = w_past * bb + w_now;
                y[at3(b, t, c, T, C)] = (w_past * a + w_now * vt) / den;
                if (s) s[at3(b, t, c, T, C)] = (w_past * sa + w_now * fabs(vt)) / den;
                /* update */
                double p_new = fmax(p - w[c], kt);
                double keep = exp(p - w[c] - p_new); /* decayed history, rescaled */
                double add = exp(kt - p_new);        /* the new token, rescaled */
                a = keep * a + add * vt;
                bb = keep * bb + add;
                sa = keep * sa + add * fabs(vt);
                p = p_new;
            }
            if (state_out) {
                state_out[bc] = a;
                state_out[BC + bc] = bb;
                state_out[2 * BC + bc] = p;
            }
            if (sacc_out) sacc_out[bc] = sa;
        }
}

/*
 * The plain two-accumulator recurrence ([MATH] "Why it collapses into a
 * recurrence"), no exponent carried:
 *   y_t = (a_{t-1} + e^{u+k_t} v_t) / (b_{t-1} + e^{u+k_t})
 *   a_t = e^{-w} a_{t-1} + e^{k_t} v_t,   b_t = e^{-w} b_{t-1} + e^{k_t},   a = b = 0 at start.
 * Overflows for large keys; used only as an in-range cross-check.
 */
void oracle_wkv_naive(int64_t B, int64_t T, int64_t C, const double* w, const double* u,
                      const double* k, const double* v, double* y)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t c = 0; c < C; ++c) {
            double a = 0.0, bb = 0.0;
            double decay = exp(-w[c]);
            for (int64_t t = 0; t < T; ++t) {
                double kt = k[at3(b, t, c, T, C)];
                double vt = v[at3(b, t, c, T, C)];
                double cur = exp(u[c] + kt);
                y[at3(b, t, c, T, C)] = (a + cur * vt) / (bb + cur);
                a = decay * a + exp(kt) * vt;
                bb = decay * bb + exp(kt);
            }
        }
}

/*
 * Token shift ([MATH] "Token shift: a two-tap causal convolution"):
 *   xbar_t = mu * x_t + (1 - mu) * x_{t-1},  per channel.
 * x [B][T][C], mu [C], x_last [B][C] is the token before t = 0 (NULL: zeros,
 * the causal zero padding), xbar [B][T][C].  With T = 1 and x_last the
 * previous token this is the single decode-step lerp.
 */
void oracle_token_shift(int64_t B, int64_t T, int64_t C, const double* mu, const double* x,
                        const double* x_last, double* xbar)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t t = 0; t < T; ++t)
            for (int64_t c = 0; c < C; ++c) {
                double prev;
                if (t > 0)
                    prev = x[at3(b, t - 1, c, T, C)];
                else
                    prev = x_last ? x_last[(size_t)b * (size_t)C + (size_t)c] : 0.0;
                xbar[at3(b, t, c, T, C)] = mu[c] * x[at3(b, t, c, T, C)] + (1.0 - mu[c]) * prev;
            }
}

/*
 * Receptance gate ([MATH] "Receptance: the gate on the way out"): each channel of
 * wkv_t passes through the logistic sigmoid of r_t,
 *   out[i] = wkv[i] * sigma(r[i]),   sigma(r) = 1 / (1 + e^{-r}),
 * elementwise over n values (the W_o projection that follows is not part of it).
 * For r -> -inf, e^{-r} overflows to +inf and the quotient is the limit 0.
 */
void oracle_gate(int64_t n, const double* r, const double* wkv, double* out)
{
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        const double sigma = 1.0 / (1.0 + exp(-r[i]));
        out[i] = wkv[i] * sigma;
    }
}

/*
 * Gradient of the wkv_t equation ([MATH] "The WKV operator: attention with a fixed decay";
 * [WIKI] eq. 1), differentiated as written; the pages give no gradient.  For a loss
 * L = sum_{b,t,c} gy[b,t,c] * y[b,t,c], with y_t = N_t / D_t,
 *   N_t = sum_{i<t} beta_{t,i} v_i + alpha_t v_t,   D_t = sum_{i<t} beta_{t,i} + alpha_t,
 *   beta_{t,i} = e^{-(t-1-i) w + k_i},   alpha_t = e^{u + k_t},
 * each term contributes (dy_t/dN_t = 1/D_t, dy_t/dD_t = -y_t/D_t):
 *   current token:  dy_t/dv_t = alpha_t / D_t;   dy_t/dk_t = dy_t/du = alpha_t (v_t - y_t) / D_t
 *   past token i:   dy_t/dv_i = beta_{t,i} / D_t;  dy_t/dk_i = beta_{t,i} (v_i - y_t) / D_t;
 *                   dy_t/dw  += -(t-1-i) beta_{t,i} (v_i - y_t) / D_t
 * gk, gv are [B][T][C]; gw, gu are [C], summed over b and t.  O(T^2) per channel, valid
 * while every exponent stays below ~709.  The optional s* outputs add up the same terms'
 * magnitudes with |gy| in place of gy and |v| + |y| in place of v - y: the scales the tests
 * divide by (y_t is only known to its own rounding, so v - y_t is only known to within a
 * fraction of |v| + |y_t|, whatever the arithmetic that follows).
 */
void oracle_wkv_backward_direct(int64_t B, int64_t T, int64_t C, const double* w, const double* u,
                                const double* k, const double* v, const double* gy, double* gk, double* gv,
                                double* gw, double* gu, double* sk, double* sv, double* sw, double* su)
{
#pragma omp parallel for schedule(static)
    for (int64_t c = 0; c < C; ++c) {
        double gwc = 0.0, guc = 0.0, swc = 0.0, suc = 0.0;
        for (int64_t b = 0; b < B; ++b) {
            for (int64_t t = 0; t < T; ++t) {
                gk[at3(b, t, c, T, C)] = 0.0;
                gv[at3(b, t, c, T, C)] = 0.0;
                if (sk) sk[at3(b, t, c, T, C)] = 0.0;
                if (sv) sv[at3(b, t, c, T, C)] = 0.0;
            }
            for (int64_t t = 0; t < T; ++t) {
                /* forward value of position t */
                double num = 0.0, den = 0.0;
                for (int64_t i = 0; i < t; ++i) {
                    double beta = exp(-(double)(t - 1 - i) * w[c] + k[at3(b, i, c, T, C)]);
                    num += beta * v[at3(b, i, c, T, C)];
                    den += beta;
                }
                double alpha = exp(u[c] + k[at3(b, t, c, T, C)]);
                num += alpha * v[at3(b, t, c, T, C)];
                den += alpha;
                double yt = num / den;
                double g = gy[at3(b, t, c, T, C)] / den;
                double gm = fabs(gy[at3(b, t, c, T, C)]) / den;
                /* current token */
                double vt = v[at3(b, t, c, T, C)];
                gv[at3(b, t, c, T, C)] += g * alpha;
                gk[at3(b, t, c, T, C)] += g * alpha * (vt - yt);
                guc += g * alpha * (vt - yt);
                if (sv) sv[at3(b, t, c, T, C)] += gm * alpha;
                if (sk) sk[at3(b, t, c, T, C)] += gm * alpha * (fabs(vt) + fabs(yt));
                suc += gm * alpha * (fabs(vt) + fabs(yt));
                /* past tokens */
                for (int64_t i = 0; i < t; ++i) {
                    double beta = exp(-(double)(t - 1 - i) * w[c] + k[at3(b, i, c, T, C)]);
                    double vi = v[at3(b, i, c, T, C)];
                    gv[at3(b, i, c, T, C)] += g * beta;
                    gk[at3(b, i, c, T, C)] += g * beta * (vi - yt);
                    gwc += -g * (double)(t - 1 - i) * beta * (vi - yt);
                    if (sv) sv[at3(b, i, c, T, C)] += gm * beta;
                    if (sk) sk[at3(b, i, c, T, C)] += gm * beta * (fabs(vi) + fabs(yt));
                    swc += gm * (double)(t - 1 - i) * beta * (fabs(vi) + fabs(yt));
                }
            }
        }
        gw[c] = gwc;
        gu[c] = guc;
        if (sw) sw[c] = swc;
        if (su) su[c] = suc;
    }
}

/*
 * Eagle (RWKV-5) matrix-state WKV ([VANOS] "Versions: RWKV-4 -> Eagle -> Finch"),
 * per sequence b and head h of N channels, token after token:
 *   S_t = diag(d) S_{t-1} + k_t v_t^T     S is N x N: row m a key channel, column j a value channel
 *   y_t = r_t^T S_t                       y_t[j] = sum_m r_t[m] S_t[m][j]
 * with d[m] = exp(-w[h N + m]) (w > 0: the per-channel decay rate, as in RWKV-4)
 * and S_{-1} = state_in (zero when NULL).
 *
 * r, k, v, y, s: [B][T][C] with C = H N, head h owning channels h N .. h N + N - 1.
 * w: [C].  state_in, state_out: [B][H][N][N] (m, j), either may be NULL.
 * s (may be NULL): the same read-out with |r|, |k|, |v| and |state_in|, the
 * magnitude scale that errors are measured against.
 * With T = 1 this is one decode step from the given state ([VANOS] "O(N) Inference
 * Characteristics").
 */
void oracle_eagle_recurrent(int64_t B, int64_t T, int64_t H, int64_t N, const double* w,
                            const double* r, const double* k, const double* v,
                            const double* state_in, double* y, double* s, double* state_out)
{
    const int64_t C = H * N;
    const size_t NN = (size_t)N * (size_t)N;
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t h = 0; h < H; ++h) {
            const size_t sb = ((size_t)b * (size_t)H + (size_t)h) * NN;
            double* S = (double*)malloc(NN * sizeof(double));
            double* Sa = (double*)malloc(NN * sizeof(double));
            for (size_t e = 0; e < NN; ++e) {
                S[e] = state_in ? state_in[sb + e] : 0.0;
                Sa[e] = fabs(S[e]);
            }
            for (int64_t t = 0; t < T; ++t) {
                /* update: S <- diag(d) S + k_t v_t^T */
                for (int64_t m = 0; m < N; ++m) {
                    const double d = exp(-w[h * N + m]);
                    const double km = k[at3(b, t, h * N + m, T, C)];
                    for (int64_t j = 0; j < N; ++j) {
                        const double vj = v[at3(b, t, h * N + j, T, C)];
                        S[m * N + j] = d * S[m * N + j] + km * vj;
                        Sa[m * N + j] = d * Sa[m * N + j] + fabs(km) * fabs(vj);
                    }
                }
                /* read-out: y_t = r_t^T S_t */
                for (int64_t j = 0; j < N; ++j) {
                    double acc = 0.0, acc_s = 0.0;
                    for (int64_t m = 0; m < N; ++m) {
                        const double rm = r[at3(b, t, h * N + m, T, C)];
                        acc += rm * S[m * N + j];
                        acc_s += fabs(rm) * Sa[m * N + j];
                    }
                    y[at3(b, t, h * N + j, T, C)] = acc;
                    if (s) s[at3(b, t, h * N + j, T, C)] = acc_s;
                }
            }
            if (state_out)
                for (size_t e = 0; e < NN; ++e) state_out[sb + e] = S[e];
            free(S);
            free(Sa);
        }
}

/*
 * The same outputs summed directly instead of carried: unrolling the recurrence gives
 * S_t = sum_{i<=t} diag(d)^{t-i} k_i v_i^T + diag(d)^{t+1} S_{-1}, so
 *   y_t[j] = sum_{i<=t} sum_m r_t[m] exp(-(t-i) w[m]) k_i[m] v_i[j]
 *          + sum_m r_t[m] exp(-(t+1) w[m]) state_in[m][j].
 * O(T^2 N^2) per head: for small cases only.
 */
void oracle_eagle_direct(int64_t B, int64_t T, int64_t H, int64_t N, const double* w,
                         const double* r, const double* k, const double* v,
                         const double* state_in, double* y)
{
    const int64_t C = H * N;
    const size_t NN = (size_t)N * (size_t)N;
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t h = 0; h < H; ++h) {
            const size_t sb = ((size_t)b * (size_t)H + (size_t)h) * NN;
            for (int64_t t = 0; t < T; ++t)
                for (int64_t j = 0; j < N; ++j) {
                    double acc = 0.0;
                    for (int64_t m = 0; m < N; ++m) {
                        const double rm = r[at3(b, t, h * N + m, T, C)];
                        for (int64_t i = 0; i <= t; ++i)
                            acc += rm * exp(-(double)(t - i) * w[h * N + m]) * k[at3(b, i, h * N + m, T, C)] *
                                   v[at3(b, i, h * N + j, T, C)];
                        if (state_in) acc += rm * exp(-(double)(t + 1) * w[h * N + m]) * state_in[sb + m * N + j];
                    }
                    y[at3(b, t, h * N + j, T, C)] = acc;
                }
        }
}

/*
 * Gated linear recurrence, token after token: f = 1 / (1 + e^{-g}), i = 1 / (1 + e^g) = 1 - f,
 *   h_t = f_t h_{t-1} + i_t x_t,  y_t = h_t,  h_{-1} = state_in ([B][C], NULL: zeros).
 * s, s_out: the same recurrence on |x| and |state_in| (every value's magnitude scale).
 */
void oracle_gated_scan(int64_t B, int64_t T, int64_t C, const double* g, const double* x,
                       const double* state_in, double* y, double* s, double* state_out, double* s_out)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t c = 0; c < C; ++c) {
            double h = state_in ? state_in[b * C + c] : 0.0, m = fabs(h);
            for (int64_t t = 0; t < T; ++t) {
                const size_t e = at3(b, t, c, T, C);
                const double f = 1.0 / (1.0 + exp(-g[e])), i = 1.0 / (1.0 + exp(g[e]));
                h = f * h + i * x[e];
                m = f * m + i * fabs(x[e]);
                y[e] = h;
                s[e] = m;
            }
            state_out[b * C + c] = h;
            s_out[b * C + c] = m;
        }
}

/*
 * Its gradients for a loss with dL/dy = gy and dL/dstate_out = gs ([B][C], NULL: zeros): lam_t
 * the gradient of h_t over all later tokens,
 *   lam_t = gy_t + f_{t+1} lam_{t+1} (gs after the last),  gx_t = i_t lam_t,
 *   gg_t = f_t i_t (h_{t-1} - x_t) lam_t,  gstate_in = f_0 lam_0.
 * sg, sx, ss: the same with |gy|, |gs|, and the magnitude scale of h plus |x| for h - x.
 * y, s: what oracle_gated_scan gives for these inputs.
 */
void oracle_gated_scan_backward(int64_t B, int64_t T, int64_t C, const double* g, const double* x,
                                const double* state_in, const double* y, const double* s, const double* gy,
                                const double* gs, double* gg, double* gx, double* gstate_in, double* sg,
                                double* sx, double* ss)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t b = 0; b < B; ++b)
        for (int64_t c = 0; c < C; ++c) {
            double m = gs ? gs[b * C + c] : 0.0, ms = fabs(m);
            for (int64_t t = T - 1; t >= 0; --t) {
                const size_t e = at3(b, t, c, T, C);
                const double f = 1.0 / (1.0 + exp(-g[e])), i = 1.0 / (1.0 + exp(g[e]));
                const double h0 = state_in ? state_in[b * C + c] : 0.0;
                const double before = t > 0 ? y[at3(b, t - 1, c, T, C)] : h0;
                const double mag = t > 0 ? s[at3(b, t - 1, c, T, C)] : fabs(h0);
                const double lam = gy[e] + m, lams = fabs(gy[e]) + ms;
                gx[e] = i * lam;
                sx[e] = i * lams;
                gg[e] = f * i * (before - x[e]) * lam;
                sg[e] = f * i * (mag + fabs(x[e])) * lams;
                m = f * lam;
                ms = f * lams;
            }
            gstate_in[b * C + c] = m;
            ss[b * C + c] = ms;
        }
}

/*
 * Gated group norm over each row's C = G * D channels.  act: 0 none, 1 SiLU, 2 sigma; z, weight,
 * bias may be NULL (no gate; 1; 0).  Per row and group of D adjacent channels
 *   n = (x - mean) / sqrt(var + eps), var about the mean;  a = n weight + bias;
 *   y = a act(z), or act(a) without z.
 * s: the magnitude scale of y, with sn = max|x| / sqrt(var + eps) + |n| in place of |n| (the
 * difference x - mean carries the rounding of the group's largest value):
 *   sa = |weight| sn + |bias|;  s = sa |act(z)|, or 1.1 sa + |act(a)| (|act'| <= 1.1).
 */
static double oracle_act(int act, double v)
{
    const double p = 1.0 / (1.0 + exp(-v));
    return act == 0 ? v : act == 1 ? v * p : p;
}

static void oracle_norm_row(int64_t D, double eps, const double* x, double* n, double* sn, double* rstd)
{
    double mean = 0.0, var = 0.0, top = 0.0;
    for (int64_t i = 0; i < D; ++i) mean += x[i];
    mean /= (double)D;
    for (int64_t i = 0; i < D; ++i) {
        var += (x[i] - mean) * (x[i] - mean);
        if (fabs(x[i]) > top) top = fabs(x[i]);
    }
    *rstd = 1.0 / sqrt(var / (double)D + eps);
    for (int64_t i = 0; i < D; ++i) {
        n[i] = (x[i] - mean) * *rstd;
        sn[i] = top * *rstd + fabs(n[i]);
    }
}

void oracle_group_norm_gated(int64_t rows, int64_t G, int64_t D, double eps, int act, const double* x,
                             const double* z, const double* weight, const double* bias, double* y, double* s)
{
#pragma omp parallel for collapse(2) schedule(static)
    for (int64_t r = 0; r < rows; ++r)
        for (int64_t g = 0; g < G; ++g) {
            const size_t at = ((size_t)r * (size_t)G + (size_t)g) * (size_t)D;
            double* n = (double*)malloc(2 * (size_t)D * sizeof(double));
            double rstd;
            oracle_norm_row(D, eps, x + at, n, n + D, &rstd);
            for (int64_t i = 0; i < D; ++i) {
                const double w = weight ? weight[g * D + i] : 1.0, b = bias ? bias[g * D + i] : 0.0;
                const double a = n[i] * w + b, sa = fabs(w) * n[D + i] + fabs(b);
                if (z) {
                    const double u = oracle_act(act, z[at + i]);
                    y[at + i] = a * u;
                    s[at + i] = sa * fabs(u);
                } else {
                    y[at + i] = oracle_act(act, a);
                    s[at + i] = 1.1 * sa + fabs(y[at + i]);
                }
            }
            free(n);
        }
}

/*
 * Its gradients for dL/dy = gy:  ga = gy act(z) and gz = gy a act'(z), or ga = gy act'(a);
 * gbias = sum ga, gweight = sum ga n (over rows), gn = ga weight,
 * gx = (gn - mean gn - n mean(gn n)) / sqrt(var + eps).
 * Scales: every product with its factors' magnitudes (sn, sa above; act' of SiLU with its two
 * terms' magnitudes; without a gate ga's scale adds |gy| sa / 2, |act''| <= 1/2), every sum of the
 * terms' scales.
 */
void oracle_group_norm_gated_backward(int64_t rows, int64_t G, int64_t D, double eps, int act, const double* x,
                                      const double* z, const double* weight, const double* bias, const double* gy,
                                      double* gx, double* gz, double* gweight, double* gbias, double* sx, double* sz,
                                      double* sw, double* sb)
{
    for (int64_t c = 0; c < G * D; ++c) gweight[c] = gbias[c] = sw[c] = sb[c] = 0.0;
#pragma omp parallel for schedule(static)
    for (int64_t g = 0; g < G; ++g) {
        double* n = (double*)malloc(4 * (size_t)D * sizeof(double));
        double *sn = n + D, *gn = n + 2 * D, *sgn = n + 3 * D;
        for (int64_t r = 0; r < rows; ++r) {
            const size_t at = ((size_t)r * (size_t)G + (size_t)g) * (size_t)D;
            double rstd, m1 = 0.0, m2 = 0.0, sm1 = 0.0, sm2 = 0.0;
            oracle_norm_row(D, eps, x + at, n, sn, &rstd);
            for (int64_t i = 0; i < D; ++i) {
                const int64_t c = g * D + i;
                const double w = weight ? weight[c] : 1.0, b = bias ? bias[c] : 0.0;
                const double a = n[i] * w + b, sa = fabs(w) * sn[i] + fabs(b);
                const double v = z ? z[at + i] : a, p = 1.0 / (1.0 + exp(-v)), q = 1.0 / (1.0 + exp(v));
                const double d = act == 0 ? 1.0 : act == 1 ? p + v * p * q : p * q;
                const double ds = act == 0 ? 1.0 : act == 1 ? p + fabs(v) * p * q : p * q;
                double ga, sga;
                if (z) {
                    ga = gy[at + i] * oracle_act(act, v);
                    sga = fabs(ga);
                    gz[at + i] = gy[at + i] * a * d;
                    sz[at + i] = fabs(gy[at + i]) * sa * ds;
                } else {
                    ga = gy[at + i] * d;
                    sga = fabs(gy[at + i]) * (ds + (act == 0 ? 0.0 : 0.5 * sa));
                }
                gbias[c] += ga;
                sb[c] += sga;
                gweight[c] += ga * n[i];
                sw[c] += sga * sn[i];
                gn[i] = ga * w;
                sgn[i] = sga * fabs(w);
                m1 += gn[i] / (double)D;
                m2 += gn[i] * n[i] / (double)D;
                sm1 += sgn[i] / (double)D;
                sm2 += sgn[i] * sn[i] / (double)D;
            }
            for (int64_t i = 0; i < D; ++i) {
                gx[at + i] = rstd * (gn[i] - m1 - n[i] * m2);
                sx[at + i] = rstd * (sgn[i] + sm1 + sn[i] * sm2);
            }
        }
        free(n);
    }
}
