// Training-step operators of libscopt: arguments and launchers shared by their kernels
// (tile_product.hip, xent.hip, act.hip, embed.hip) and their C entries (train_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace scopt {

// What TP_STATS keeps of a piece's logits.
enum TpKeep {
    TP_KEEP_NONE = 0,   // nothing
    TP_KEEP_EXP = 1,    // 2^(s log2(e) - ref) in 16 bits (tp_pack_unit), ref the tile's row
                        // maximum in powers of two, rounded up: a later change of reference
                        // by a power of two is exact
    TP_KEEP_LOGIT = 2,  // the logits in float32
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
};

// The product's operand layouts and what is done with its sums.
enum TpKind {
    TPK_LOGIT_STATS,  // A [M][K], B [N][K]
    TPK_LOGIT_GRAD,   // A [M][K], B [N][K]
    TPK_STATES,       // A [M][K], B [K][N]: store, or partial sums when splits > 1
    TPK_WEIGHTS,      // A [K][M], B [K][N]: likewise
};

// Tile shapes, and the choice between them for an M x N product of `steps` 64-deep steps.
struct TpPlan {
    int shape = 0;  // index of the tile shape
    int bm = 0, bn = 0;
    int tiles_m = 0, tiles_n = 0;
    int splits = 1;
    int64_t part_bytes = 0;  // float32 partial sums (splits > 1)
};
// Row stride of an operand that the library lays out itself
inline int64_t tp_pad(int64_t cols) { return cols % 512 == 0 ? cols + 64 : cols; }
TpPlan tp_plan(int M, int N, int K, int nseg, bool may_split);
// A product whose sums join others (TPK_STATES, TPK_WEIGHTS): acc is added before the store;
// with out_acc the float32 sum goes there and C is not written.  Either asks for args.part
// also without splits.
struct TpSum {
    const float* acc = nullptr;
    float* out_acc = nullptr;
};
hipError_t launch_tile_product(TpKind kind, const TpPlan& plan, TpArgs args, const TpSum& sum, hipStream_t st);

// `bytes` (even) zeros
hipError_t launch_zero(void* p, int64_t bytes, hipStream_t st);

// planes[p][r][c] of a float32 (three planes) or bfloat16 (one plane) matrix, zero in the
// columns from `cols` to ld and, with targets, in the rows whose target is not in [0, vocab)
hipError_t launch_to_planes(bool bf16, const void* src, int64_t rows, int64_t cols, uint16_t* dst, int64_t ld,
                            int64_t plane, const int64_t* targets, int64_t vocab, hipStream_t st);

// ---- cross entropy (xent.hip) --------------------------------------------------------
struct XentPlan {
    bool bf16, planes;         // planes: W is copied into planes (float32, or H % 8), as h always is
    int64_t T, V, H, Hp, Hh;   // columns of W's operand (H, or padded when planes) and of h's
    int64_t piece;             // vocabulary rows of a piece
    int pieces;
    bool keep;                 // one piece whose probabilities are kept between the passes
    int64_t ldp;               // columns of P
    int64_t stat_tiles;        // tiles of a row
    TpPlan logits, logits_last, dh, dw, dw_last;
    // offsets into the workspace
    int64_t o_factors, o_h, o_w, o_s, o_p, o_tl, o_lse, o_smax, o_ssum, o_part, o_dh, bytes;
};
// limit: bytes that the kept probabilities (or a piece's) may take
XentPlan xent_plan(bool bf16, int64_t T, int64_t V, int64_t H, int64_t limit);
hipError_t launch_xent(const XentPlan& p, const void* h, const void* W, const int64_t* targets, float* loss,
                       float* mean, void* dh, void* dW, void* workspace, hipStream_t st);

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
