// Training-step operators of libscopt: arguments and launchers shared by their kernels
// (tile_product.hip, few_tokens.hip, xent.hip, token_loss.hip, act.hip, layernorm.hip, clip.hip, embed.hip) and
// their C entries (train_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "scopt.h"

namespace scopt {

// What TP_STATS keeps of a piece's logits.
enum TpKeep {
    TP_KEEP_NONE = 0,   // nothing
    TP_KEEP_EXP = 1,    // 2^(s log2(e) - ref) in 16 bits (tp_pack_unit), ref the tile's row
                        // maximum in powers of two, rounded up: a later change of reference
                        // by a power of two is exact
    TP_KEEP_LOGIT = 2,  // the logits in float32
};

// How the `tiles` whole tiles of a product of `total` turns of k go to `slots` workgroups (TP_TAIL): the first
// `full` one after the other, in whole rounds, and of the others (`rest`) each in `splits` parts of k.
struct TpTail {
    int full, rest, splits;
};
// What that depends on: sizes, one of them bounded by the live tokens, and the tile's times (tp_plan).
struct TpTailQuery {
    int M = 0, K = 0, live_k = 0;  // live_k: the tokens are k, else the rows
    int bm = 1, turn_k = 1, tiles_n = 0, nseg = 1, slots = 1;
    int turn_ns = 0, tile_ns = 0, join_ns = 0;
    int pass_ns = 0;  // of the weights or their gradient through memory
    int most = 0;     // parts that there is room for
    __host__ __device__ int tiles(int live) const { return ((live_k || M < live ? M : live) + bm - 1) / bm * tiles_n; }
    __host__ __device__ int total(int live) const {
        const int k = live_k && live < K ? live : K;
        return (k > 0 ? (k + turn_k - 1) / turn_k : 1) * nseg;
    }
    // time of the last of the rounds of `tiles` in s parts, their sums and join included; the largest number where
    // that is not to be
    __host__ __device__ int ns(int tiles, int total, int s) const {
        const int rest = tiles % slots;
        if (s > 1 && (rest * s > most || total < 2 * s)) return 0x7fffffff;
        const int ns = (rest * s + slots - 1) / slots * ((total + s - 1) / s * turn_ns + tile_ns);
        const int least = tiles < slots ? pass_ns : 0;  // where the last round is all there is
        return (ns > least ? ns : least) + (s > 1 ? 4000 + rest * s * join_ns : 0);
    }
};

// One tiled product (tile_product.hpp).  An operand's rows are readable up to the next
// multiple of 8 elements; with k contiguous, what lies between K and there is finite where
// the other operand's rows beyond K do not exist (they count as zeros), else zero.
struct TpArgs {
    const uint16_t* A = nullptr;  // planes of [M][K] or [K][M]
    const uint16_t* B = nullptr;  // planes of [N][K] or [K][N]
    int64_t lda = 0, ldb = 0;     // row strides (elements, multiples of 8)
    int64_t a_plane = 0, b_plane = 0;  // elements between planes
    int M = 0, N = 0, K = 0;
    int nseg = 1;       // segments of k
    uint64_t segs = 0;  // 4 bits a segment: plane of A, plane of B << 2
    int tiles_m = 0, tiles_n = 0, splits = 1;
    // TP_STORE, and the reduction of TP_PART's splits
    void* C = nullptr;
    int64_t ldc = 0;
    int c_bf16 = 0;
    const float* alpha = nullptr;  // device scalar (NULL: 1); TP_GRAD: a factor of the values
    const void* gain = nullptr;    // column factors (NULL: 1)
    int gain_bf16 = 0;
    float* part = nullptr;
    // TP_STATS, TP_GRAD
    const int64_t* targets = nullptr;
    int64_t vocab = 0;
    int64_t n_first = 0;  // the vocabulary row of column 0
    int keep = 0;
    void* P = nullptr;
    int64_t ldp = 0;         // row stride of P; its rows hold whole tiles
    int64_t p_plane = 0;     // TP_GRAD: elements between planes
    int p_planes = 1;        // TP_GRAD: 1 or 3
    float* target_logit = nullptr;
    float* stat_max = nullptr;  // [tile of columns][M]
    float* stat_sum = nullptr;
    int64_t stat_first = 0;
    const float* lse = nullptr;
    // TP_GRAD: a factor of each row's values, in place of alpha; with coef_zeros only its zeros count, and
    // the others' factor is 1.  TP_TAIL: a factor of each row of C (NULL: 1)
    const float* coef = nullptr;
    int coef_zeros = 0;
    // Only the first *live tokens exist (NULL: all).  Tokens are the rows of the logits and of the
    // states' gradients, and k of the weights'.
    const int* live = nullptr;
    int live_rows = 0;          // set by the launch: live counts the rows of C
    const int* rows = nullptr;  // TP_TAIL, reduction: row m is stored as row rows[m] (NULL: m)
    const TpTail* tail = nullptr;  // TP_TAIL: on the device
    // Operands in float16: row m of A stands for 2^a_exp[m] times its planes, row n of B for 2^b_exp[n] times
    // (16-byte aligned, readable to the end of the last tile)
    const int *a_exp = nullptr, *b_exp = nullptr;
    // The live logits' statistics with TP_KEEP_EXP: a power of two for each row (its exponent, or NULL).  A tile's row
    // is kept relative to it, in bfloat16, where tp_by_row says so.
    const float* row_ref = nullptr;
};

// The product's operand layouts and what is done with its sums.
enum TpKind {
    TPK_LOGIT_STATS,  // A [M][K], B [N][K]
    TPK_LOGIT_GRAD,   // A [M][K], B [N][K]
    TPK_STATES,       // A [M][K], B [K][N]: store, or partial sums when splits > 1
    TPK_WEIGHTS,      // A [K][M], B [K][N]: likewise
    // as the ones above, for sizes that are only known on the device: the tiles that do not fill a round of
    // workgroups are cut along k there
    TPK_LOGIT_STATS_LIVE,
    TPK_STATES_LIVE,
    TPK_WEIGHTS_LIVE,
};

// Tile shapes, and the choice between them for an M x N product of `steps` 64-deep steps.
struct TpPlan {
    int shape = 0;  // index of the tile shape
    int bm = 0, bn = 0;
    int tiles_m = 0, tiles_n = 0;
    int splits = 1;
    int64_t part_bytes = 0;  // float32 partial sums (splits > 1; tp_plan_live: the most there can be)
};
// Row stride of an operand that the library lays out itself
inline int64_t tp_pad(int64_t cols) { return cols % 512 == 0 ? cols + 64 : cols; }
TpPlan tp_plan(int M, int N, int K, int nseg, bool may_split);
// For the kinds of live tokens: M, N, K are the most there can be.  The parts of the last round's tiles are at most
// two rounds of them (64 MiB each with the largest tile), of the logits one.
TpPlan tp_plan_live(TpKind kind, int M, int N, int K, int nseg, TpTailQuery& tail);
// A product whose sums join others (TPK_STATES, TPK_WEIGHTS): acc is added before the store;
// with out_acc the float32 sum goes there and C is not written.  Either asks for args.part
// also without splits.
struct TpSum {
    const float* acc = nullptr;
    float* out_acc = nullptr;
};
hipError_t launch_tile_product(TpKind kind, const TpPlan& plan, TpArgs args, const TpSum& sum, hipStream_t st);

// dW[v][n] = sum over the first *live of T <= kFewTokens tokens of d[t][v] h[t][n], bfloat16 (few_tokens.hip): d
// [T][ldd], h [T][ldh] as operands of a product, dW [V][N]
constexpr int64_t kFewTokens = 128;
hipError_t launch_few_tokens(const uint16_t* d, int64_t ldd, const uint16_t* h, int64_t ldh, int T, const int* live,
                             int V, int N, uint16_t* dW, hipStream_t st);

// `bytes` (even) zeros
hipError_t launch_zero(void* p, int64_t bytes, hipStream_t st);

// planes[p][r][c] of a float32 (three planes) or bfloat16 (one plane) matrix, zero in the
// columns from `cols` to ld and, with targets, in the rows whose target is not in [0, vocab).  With
// `place` row r goes to row place[r], and one with a negative place clears its row of `cleared`
// ([rows][cols] of src's type, or NULL) instead.
hipError_t launch_to_planes(bool bf16, const void* src, int64_t rows, int64_t cols, uint16_t* dst, int64_t ld,
                            int64_t plane, const int64_t* targets, int64_t vocab, hipStream_t st,
                            const int* place = nullptr, void* cleared = nullptr);

// Rows of a float32 matrix [rows][cols] as operands of a product of live tokens: two float16 planes half[2][rows][ld] of
// each row times a power of two (its exponent's negative is `exps`), and with `planes` the three bfloat16 ones too
// ([3][rows][ld]).  place, cleared: as launch_to_planes.
hipError_t launch_half_rows(const float* src, int64_t rows, int64_t cols, int64_t ld, uint16_t* half, int* exps,
                            uint16_t* planes, hipStream_t st, const int* place = nullptr, float* cleared = nullptr);

// ---- losses over a large vocabulary (xent.hip, token_loss.hip) -------------------------
struct XentPlan {
    bool bf16, planes;         // planes: W is copied into planes (float32, or H % 8), as h always is
    int64_t T, V, H, Hp, Hh;   // columns of W's operand (H, or padded when planes) and of h's
    int64_t piece;             // vocabulary rows of a piece
    int pieces;
    bool keep;                 // one piece whose probabilities are kept between the passes
    int64_t ldp;               // columns of P
    int64_t stat_tiles;        // tiles of a row
    TpPlan logits, logits_last, dh, dw, dw_last;
    TpTailQuery tails[5];      // of live tokens: dh, dw, dw_last, logits, logits_last
    bool half;                 // live tokens in float32: the logits' operands are float16 planes
    bool by_row;               // kept exponentials of live tokens are relative to a reference of their row
    // offsets into the workspace
    int64_t o_factors, o_h, o_scaled, o_w, o_s, o_p, o_tl, o_lse, o_smax, o_ssum, o_part, o_dh, o_tails, o_factor, o_ref;
    int64_t o_half_h, o_half_w, o_exp_h, o_exp_w, bytes;
};
// limit: bytes that the kept probabilities (or a piece's) may take; gradients = false: only the logits'
// statistics are taken, and there is room for nothing else
// live: the counted tokens' rows are put together (XentRun::rows)
XentPlan xent_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit, bool gradients = true,
                   bool live = false);

// What a row's log-sum-exp is formed from: its tiles' references (powers of two with pow2) and sums, [tile][T],
// and its target's logit; and where it goes
struct LogSums {
    const float *smax, *ssum;
    int tiles, pow2;
    const float* target_logit;
    float* lse;
    int64_t T;
};

// One call's buffers, and the steps that the losses share.  Without `rows` the rows of h are the tokens; with
// them only the counted ones, in order: row c is token rows[c], *live of them exist, and `targets`, lse
// and coef go by c.
struct XentRun {
    const XentPlan* p = nullptr;
    const void *h = nullptr, *W = nullptr;
    const int64_t* targets = nullptr;
    char* ws = nullptr;
    const int *live = nullptr, *rows = nullptr, *place = nullptr;  // place[t]: token t's row, or -1
    // The logit gradients are (softmax - onehot) times coef[row].  In bfloat16 the matrix keeps softmax - onehot, or
    // with by_row that times a power of two of the row, and coef joins dh's rows as they are stored and the rows of h
    // that dW reads, times what makes the target's entry exact (factor): the target's share of the gradients is the
    // largest, and one coefficient for all of a sequence's tokens would be rounded the same way in all of them.
    // Without coef the factor is factors[1], and the stores of dh and dW multiply by factors[0].
    const float* coef = nullptr;
    bool gradients_follow = true;
    hipStream_t st = nullptr;

    template <typename E> E* at(int64_t offset) const { return (E*)(ws + offset); }
    // h and, where it needs planes, W as operands.  dh: its rows of tokens that are not counted are cleared
    // (with rows; else NULL)
    hipError_t h_operand(void* dh) const;
    hipError_t w_planes() const;
    hipError_t row_references() const;
    hipError_t logits() const;                       // row statistics, and what is kept
    LogSums sums() const;
    hipError_t log_sums(float* loss, float* logp) const;  // lse; the tokens' losses, or with rows their negative
    hipError_t gradients(void* dh, void* dW) const;

private:
    TpArgs logit_args(int piece) const;
    const uint16_t* w_operand() const { return p->planes ? at<uint16_t>(p->o_w) : (const uint16_t*)W; }
    uint64_t segments() const;
};
hipError_t launch_xent(const XentPlan& p, const void* h, const void* W, const int64_t* targets, float* loss,
                       float* mean, void* dh, void* dW, void* workspace, hipStream_t st);

struct TokenLossPlan {
    XentPlan x;
    int64_t o_live, o_rows, o_place, o_targets, o_coef, bytes;
};
TokenLossPlan token_loss_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit, bool gradients);
hipError_t launch_token_logp(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                             float* logp, void* workspace, hipStream_t st);
struct PolicyArgs {
    const float *old_logp, *advantages, *ref_logp, *weights;  // [T]; ref_logp, weights or NULL
    double lo, hi;                                            // the ratio is clipped to [lo, hi]
    float kl;
    float *loss, *total, *kl_mean, *clipped, *logp;
};
hipError_t launch_policy_loss(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                              const PolicyArgs& a, void* dh, void* dW, void* workspace, hipStream_t st);
struct PreferenceArgs {
    const int64_t* starts;  // [2 pairs + 1]
    const float* ref_logp;  // [T] or NULL
    int64_t pairs;
    float beta, margin, smoothing;
    int average;
    float *loss, *mean, *rewards, *logp;
};
hipError_t launch_preference_loss(const TokenLossPlan& p, const void* h, const void* W, const int64_t* targets,
                                  const PreferenceArgs& a, void* dh, void* dW, void* workspace, hipStream_t st);

// ---- 8-bit activation checkpoints and the residual norm (act.hip) ----------------------
hipError_t launch_act_pack(bool bf16, const void* x, int64_t T, int H, int8_t* q, uint8_t* e, hipStream_t st);
hipError_t launch_act_unpack(bool bf16, const int8_t* q, const uint8_t* e, int64_t T, int H, void* x,
                             hipStream_t st);
hipError_t launch_rmsnorm(bool bf16, const void* x, const void* residual, const void* gain, float eps, int64_t T,
                          int H, void* h, void* y, float* rstd, int8_t* q, uint8_t* e, hipStream_t st);
int64_t rmsnorm_grad_parts(int64_t T, int H);
hipError_t launch_rmsnorm_grad(bool bf16, const void* dy, const void* gain, const float* rstd, const int8_t* q,
                               const uint8_t* e, const void* dh, int64_t T, int H, void* dx, float* dgain,
                               float* partial, hipStream_t st);

// ---- layer norm (layernorm.hip) ----------------------------------------------------------
hipError_t launch_layernorm(bool bf16, const void* x, const void* residual, const void* gain, const void* bias,
                            float eps, int64_t T, int H, void* h, void* y, float* mean, float* rstd, int8_t* q,
                            uint8_t* e, hipStream_t st);
int64_t layernorm_grad_parts(int64_t T, int H);  // rows of 2 H float32 of `partial`
hipError_t launch_layernorm_grad(bool bf16, const void* dy, const void* gain, const float* rstd, const float* mean,
                                 const int8_t* q, const uint8_t* e, const void* h, const void* dh, int64_t T, int H,
                                 void* dx, float* dgain, float* dbias, float* partial, hipStream_t st);

// ---- global gradient norm (clip.hip) -----------------------------------------------------
struct GradTensors {  // host arrays
    int n;
    const sc_dtype* dtypes;
    const int64_t* sizes;
    const void* const* src;
    void* const* dst;  // NULL where only the norm is taken
};
int64_t grad_sumsq_parts(const GradTensors& g);  // float64 partial sums
hipError_t launch_grad_sumsq(const GradTensors& g, double* sumsq, double* part, hipStream_t st);
// both: the norm of the gradients, and what it makes of them
hipError_t launch_clip_norm(const GradTensors& g, float max_norm, float* norm, float* scale, double* part,
                            hipStream_t st);
// sumsq: its value, or some parts of it (as many as launch_clip_norm leaves)
hipError_t launch_clip(const GradTensors& g, const double* sumsq, int parts, float max_norm, float* norm, float* scale,
                       hipStream_t st);

struct WgradPlan {
    bool bf16, planes;  // planes: dy is copied into planes (float32, or N % 8)
    int64_t T, N, H, Np, Hp;
    TpPlan prod;
    int64_t o_dy, o_n, o_part, bytes;
};
WgradPlan wgrad_plan(bool bf16, int64_t T, int64_t N, int64_t H);
hipError_t launch_act_wgrad(const WgradPlan& p, const void* dy, const int8_t* q, const uint8_t* e, const void* gain,
                            void* dW, void* workspace, hipStream_t st);

// ---- embedding (embed.hip) -------------------------------------------------------------
hipError_t launch_embed(bool bf16, const void* table, const int64_t* ids, int64_t T, int64_t V, int H, float scale,
                        void* out, hipStream_t st);
struct EmbedGradPlan {
    int64_t T, V, H;
    int shift, bins;     // ids of 2^shift rows share a bin
    int64_t per_block, blocks;  // tokens of a block, blocks
    int len;                    // sorted tokens of a stretch
    int64_t runs;               // stretches
    int64_t slabs;              // of 512 columns
    int64_t tasks;              // wavefronts of embed_sum: stretches and eights of table rows, times slabs
    int64_t o_counts, o_bin, o_key, o_pos, o_id, o_spos, o_start, o_part, bytes;
};
EmbedGradPlan embed_grad_plan(int64_t T, int64_t V, int64_t H);
hipError_t launch_embed_grad(const EmbedGradPlan& p, bool bf16, const void* dy, const int64_t* ids, float scale,
                             void* dW, void* workspace, hipStream_t st);

}  // namespace scopt
