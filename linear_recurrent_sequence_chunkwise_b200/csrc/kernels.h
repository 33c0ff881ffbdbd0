// kernels.h -- internal launch functions behind the C ABI.  Each returns
// RET_OK after enqueueing, RET_ERR_UNSUPPORTED if the shape does not fit the
// kernel (nothing launched), or RET_ERR_CUDA if the launch failed.  Argument
// validation has already happened in ret_api.cu.
#pragma once

#include "common.cuh"

namespace ret {

struct RetArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* final_state;          // may be null
    const float* initial_state;  // may be null (zero state); workspace path only
    // Workspace path only: elements between consecutive (token, head) rows of
    // q and of k (0: dk, i.e. contiguous), so that a column slice of a wider
    // tensor can serve as q or k; accumulate = 1 adds the result into an
    // fp32 out instead of storing it; out_rev = 1 writes the output of token n
    // to row N-1-n.
    int q_ld, k_ld, accumulate, out_rev;
    // Workspace path only: fp32 [B, N, H] factors the output row of each
    // (token, head) is multiplied by (the score normalizations), or null.
    const float* rowscale;
    // Workspace path only: the caller's d_k when it is below the tensor-core
    // kernel's (0: dk).  The rows are then zero-padded to dk in the
    // workspace, the rotation uses dk_real, and the states have dk_real rows.
    int dk_real;
    int B, N, H, dk, dv, chunk;
    ret_dtype in_dt, out_dt;
    int xpos;
    long long pos_offset;
    double theta_base;
    HeadConsts hc;
    double gamma[kMaxHeads];
};

// inverse: turn by -angle (the transpose of each rotation).
ret_status launch_xpos_rotate(void* x, ret_dtype dt, int B, int N, int H, int d, long long pos_offset,
                              double theta_base, cudaStream_t s, bool inverse = false);
ret_status launch_chunkwise_simt(const RetArgs& a, cudaStream_t s);
ret_status launch_parallel_simt(const RetArgs& a, cudaStream_t s);
// untaken_only: only the heads the tensor-core kernels leave out (anchor -1).
ret_status launch_recurrent_simt(const RetArgs& a, cudaStream_t s, bool untaken_only = false);
ret_status launch_decode(const void* q, const void* k, const void* v, const HeadConsts& hc, float* state,
                         void* out, int B, int H, int dk, int dv, ret_dtype in_dt, ret_dtype out_dt,
                         cudaStream_t s);


// Workspace path: prep kernel (rotation + zeta scaling into the workspace)
// and the warp-specialized tensor-core kernel.  The shape check alone; the
// number of heads whose anchor (HeadConsts) is below min_anchor (0: heads the
// kernel does not take; kChunkAnchorFull: heads not on the plain factors);
// and both together (shape on the path, every head taken).
bool chunkwise_ws_shape_ok(const RetArgs& a);
int chunkwise_heads_below(const RetArgs& a, int min_anchor);
bool chunkwise_ws_supported(const RetArgs& a);
size_t chunkwise_ws_bytes(const RetArgs& a);
ret_status launch_chunkwise_ws(const RetArgs& a, void* ws, cudaStream_t s);
// Its two halves: the prep pass alone, and the tensor-core kernel on a
// workspace the prep pass has filled (a.initial_state honoured).
ret_status launch_chunkwise_prep(const RetArgs& a, void* ws, cudaStream_t s);
ret_status launch_chunkwise_prepared(const RetArgs& a, void* ws, cudaStream_t s);
// The scores form: a tensor-core pass that rotates q and k, scales the keys
// and computes the masked intra-chunk scores P of every (b, h, chunk), then
// the warp-specialized kernel on those (read-out, P V, state update).  `ws`
// holds chunkwise_scores_bytes (256-byte aligned).  The pooled form takes it
// from a stream-ordered pool of the library.
size_t chunkwise_scores_bytes(const RetArgs& a);
ret_status launch_chunkwise_scores(const RetArgs& a, void* ws, cudaStream_t s);
// Its two passes on their own (the second honours a.initial_state).
ret_status launch_chunkwise_scores_pass1(const RetArgs& a, void* ws, cudaStream_t s);
ret_status launch_chunkwise_scores_pass2(const RetArgs& a, void* ws, cudaStream_t s);
ret_status launch_chunkwise_scores_pooled(const RetArgs& a, cudaStream_t s);
// The workspace path on the library's fixed device array (no allocation).
size_t chunkwise_static_ws_bytes();
ret_status launch_chunkwise_static(const RetArgs& a, cudaStream_t s);
// Score normalizations 2 and 3 on the workspace path: flags bit 0 divides
// row n of the decay matrix by sqrt(sum_i D_ni), bit 1 the scores by
// max(|sum_i R_ni|, 1); z0 / z1 the decayed key sum before / after the
// call ([B, H, dk] fp32, either may be null).
constexpr int kNormDecay = RET_NORM_DECAY, kNormScore = RET_NORM_SCORE;
size_t normalized_ws_bytes(const RetArgs& a);
ret_status launch_chunkwise_normalized(const RetArgs& a, int flags, const float* z0, float* z1, void* ws,
                                       cudaStream_t s);
// Options of the decode step: the xPos rotation of q and k and the score
// normalizations at each sequence's position (positions[b] on the device, or
// pos for all when positions is null); z [B, H, dk] updated in place (needed
// with kNormScore).
struct DecodeOpts {
    float* z;
    const long long* positions;
    long long pos;
    int flags;
    int xpos;
    double log2base;
};
ret_status launch_decode_ex(const void* q, const void* k, const void* v, const HeadConsts& hc, float* state,
                            void* out, int B, int H, int dk, int dv, ret_dtype in_dt, ret_dtype out_dt,
                            const DecodeOpts& o, cudaStream_t s);

// One thread waits on a barrier nothing arrives on (bounded), then sets the
// device error word: the timeout path without a hang or a fault.
ret_status launch_wait_selftest(uint32_t polls, cudaStream_t s);

// The tensor-core kernel alone, on prepared q_rot (or q) and k' (zeta-scaled keys).
// q_rot: [B, N, H, dk] rows q_pitch elements apart.
ret_status launch_chunkwise_main(const RetArgs& a, const void* q_rot, int q_pitch, const void* k_prime,
                                 cudaStream_t s);

// Gradients of chunkwise retention (k_backward.cu): bf16 q, k, v, dout
// [B, N, H, d], fp32 dq, dk, dv.
struct BwdArgs {
    const void *q, *k, *v, *dout;
    float *dq, *dkk, *dvv;
    int B, N, H, dk, dv, chunk;
    int xpos;
    long long pos_offset;
    double theta_base;
    HeadConsts hc;
    void* workspace;
};
bool backward_supported(const BwdArgs& a);
size_t backward_ws_bytes(const BwdArgs& a);
ret_status launch_backward(const BwdArgs& a, cudaStream_t s);

struct MsrArgs {
    const void *X, *Wq, *Wk, *Wv, *Wg, *Wo;
    int B, N, dmodel, H, dk, dv, chunk;
    double k_scale, eps;
    int xpos;
    long long pos_offset;
    double theta_base;
    HeadConsts hc;
    void* out;
    ret_dtype out_dt;
    void* workspace;
    const void* residual;  // bf16 [B*N, dmodel] added to the output, or null
};
size_t msr_workspace_bytes(int B, int N, int dmodel, int H, int dk, int dv);
ret_status launch_msr(const MsrArgs& m, cudaStream_t s);
ret_status launch_linear(const void* X, const void* W, void* Y, int M, int N, int K, ret_dtype out_dt, cudaStream_t s);

// One pre-norm RetNet block: Y = MSR(LN1(X)) + X, out = gelu(LN2(Y) W1) W2 + Y.
struct BlockArgs {
    MsrArgs msr;            // X, the MSR weights and shapes; out / residual / workspace unused
    const void *ln1_g, *ln1_b, *ln2_g, *ln2_b;  // bf16 [dmodel] each, or null (gain 1, bias 0)
    const void *W1, *W2;    // bf16 [dmodel, dff], [dff, dmodel]
    int dff;
    double ln_eps;
    void* out;
    ret_dtype out_dt;
    void* workspace;
};
size_t block_workspace_bytes(int B, int N, int dmodel, int H, int dk, int dv, int dff);
ret_status launch_block(const BlockArgs& a, cudaStream_t s);
// LayerNorm of the rows of x [M, d] (bf16) into y (bf16).
ret_status launch_layernorm(const void* x, const void* gain, const void* bias, void* y, int M, int d, double eps,
                            cudaStream_t s);

// Rotary positions (k_rotary.cu).  A view of [B, N, heads, d] with element
// strides of batch, token and head; components are consecutive.
constexpr int kMaxRotaryDim = 512;
struct RotaryView {
    void* p;
    long long sb, sn, sh;
};
struct RotaryArgs {
    RotaryView q, k, qo, ko;      // k, ko unused when Hk is 0
    const long long* positions;   // device [B, N], or null (pos_offset + n)
    long long pos_offset;
    int B, N, H, Hk, d, rotary_dim;
    int half;                     // pairs (p, p + rotary_dim / 2) instead of (2p, 2p + 1)
    int inverse;                  // turn by the negative angle (the transpose)
    float scale;
    ret_dtype dt;
};
// freqs: host, rotary_dim / 2 angles per position.
ret_status launch_rotary(const RotaryArgs& a, const double* freqs, cudaStream_t s);

// Layer norm and its gradients (k_layernorm.cu), rows of d <= kLayerNormMaxDim.
constexpr int kLayerNormMaxDim = 8192;
struct LayerNormArgs {
    const void *x, *gain, *bias, *dy;  // gain, bias may be null
    void *y, *dx;
    float *mean, *rstd;                // written by the forward (may be null), read by the backward
    float *dgain, *dbias;              // may be null
    void* workspace;
    long long rows;
    int d;
    double eps;
    ret_dtype dt, w_dt;                // of x, dy, y, dx; of gain, bias
};
size_t layernorm_bwd_workspace_bytes(long long rows, int d);
ret_status launch_layernorm_forward(const LayerNormArgs& a, cudaStream_t s);
ret_status launch_layernorm_backward(const LayerNormArgs& a, cudaStream_t s);

// The gated delta rule (k_delta_step.cu, k_delta_prep.cu, k_delta_chunk.cu,
// k_delta_backward.cu).
// Value head h reads key head h / (H / Hk).
constexpr int kDeltaMaxDk = 256;
struct DeltaArgs {
    const void *q, *k, *v;        // [B, N, Hk, dk] twice, [B, N, H, dv]
    const float *g, *beta;        // [B, N, H]
    const int* lengths;           // device [B] (clamped to [0, N]), or null
    const float* initial_state;   // [B, H, dk, dv], or null
    float* final_state;           // or null
    void* out;
    // backward
    const void* dout;
    const float* dfinal_state;    // or null
    void *dq, *dkk, *dvv;         // of dtype grad_dt
    float *dg, *dbeta, *dinitial_state;  // dinitial_state may be null
    ret_dtype grad_dt;
    int B, N, Hk, H, dk, dv;
    ret_dtype in_dt, out_dt;
};
ret_status launch_delta_step(const DeltaArgs& a, float* state, cudaStream_t s);
// The whole sequence token by token (any dk <= kDeltaMaxDk, any dv).
ret_status launch_delta_recurrent(const DeltaArgs& a, cudaStream_t s);
// The chunkwise tensor-core path: bf16, dk 64, 128 or 256, dv a multiple of 8.
bool delta_chunk_shape_ok(const DeltaArgs& a);
size_t delta_forward_ws_bytes(const DeltaArgs& a);
ret_status launch_delta_forward(const DeltaArgs& a, void* ws, cudaStream_t s);
size_t delta_backward_ws_bytes(const DeltaArgs& a);
ret_status launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t s);

}  // namespace ret
