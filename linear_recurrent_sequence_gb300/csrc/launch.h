// Internal launchers shared between the kernel files and the C ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>
#include <utility>

#include "common.cuh"

namespace ret {

// Launch with programmatic stream serialization when pdl is set: the kernel
// may then start while the previous kernel on the stream still runs, so it
// must call pdl_wait() before it touches global memory that an earlier
// kernel may write or read (common.cuh).
template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                     bool pdl, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// SMs of the current device (asked once per device).
int device_sms();

// Lets a kernel use all of an SM's shared memory a CTA can have (once per
// kernel and device).
cudaError_t allow_big_smem(const void *kern, std::atomic<unsigned> &done);

enum ScaleMode { kScaleNone = 0, kScaleArray = 1, kScaleXi = 2, kScaleZeta = 3 };

// rotate.cu
cudaError_t launch_rotate(const KParams &p, const void *x, const long long s[3], int d,
                          void *out, int out_bf16, const float *scale, int mode,
                          cudaStream_t st);

// Per-(batch*head, chunk) record of the tensor-core path's fp16 operands,
// written by the prologue and copied into shared memory with each chunk.
struct ChunkMeta {
  int qexp, kexp;    // Q', K' are stored as fp16 * 2^-exp
  float qmax, kmax;  // largest pair norm of the rotated q / k rows before the decays
};

// Rotate-and-scale prologue of the tensor-core path (bf16 q, k; chunk 64):
// Q' = xi (.) rot(q), K' = zeta (.) rot(k) as contiguous fp16 [B*H][N][d_k]
// with per-chunk exponents, magnitudes and (if colsum) key column sums.
// keys_only: rotate k alone (q is not read; Q' and the query fields of meta
// are left as they are).
cudaError_t launch_rotate_qk(const KParams &p, const void *q, const void *k, __half *Qp,
                             __half *Kp, ChunkMeta *meta, float *colsum, cudaStream_t st,
                             bool keys_only = false);

// chunk_simt.cu: fp32 CUDA-core forms writing unnormalised rows + row factors.
// Qr, Kr: rotated contiguous fp32 [B,H,N,dk]; Oraw: fp32 [B,H,N,dv];
// F: fp32 [B,H,N] (row factor f = s(n) r(n)).
cudaError_t launch_chunk_simt(const KParams &p, const float *Qr, const float *Kr,
                              const void *v, const float *S_in, const float *z_in,
                              float *S_out, float *z_out, float *Oraw, float *F,
                              cudaStream_t st);
cudaError_t launch_parallel_simt(const KParams &p, const float *Qr, const float *Kr,
                                 const void *v, float *Oraw, float *F, cudaStream_t st);

// chunk_tc.cu: tensor-core chunkwise kernel (chunk 64, d_k in 64..256 step
// 64, d_v multiple of 128 up to 1024, bf16 inputs, gamma^64 >= 2^-16).
// Qp, Kp: contiguous fp16 [B,H,N,d_k] from the rotate-and-scale prologue
// (xi-scaled queries, zeta-scaled keys) with per-chunk records meta
// ([B*H][chunks]) and key column sums ksum ([B*H][chunks][d_k]).
bool chunk_tc_supported(const KParams &p, const void *v, const long long sv[3]);

// groupnorm.cu: o = GroupNorm(F * Oraw), written through so[]; and
// y <- y * swish(g) elementwise over n bf16 values (the MSR layer's gate).
cudaError_t launch_groupnorm(const KParams &p, const float *Oraw, const float *F,
                             void *o, cudaStream_t st);
cudaError_t launch_swish_gate(void *y, const void *g, long long n, cudaStream_t st);

// Sequence segments of the tensor-core chunk kernel.  P segments of seg_len
// chunks run as separate CTA groups; the entry state of segment k > 0 is
// assembled from the partial states of the npieces pieces (piece_len whole
// chunks each, covering chunks [0, (P-1) seg_len)) that state_tc writes.
struct SegPlan {
  int P = 1, seg_len = 0, npieces = 0, piece_len = 1;
  float *Part = nullptr, *zPart = nullptr;  // [piece][B*H][d_k][d_v], [piece][B*H][d_k]
};

cudaError_t launch_chunk_tc(const KParams &p, const void *Qp, const void *Kp, const void *v,
                            const ChunkMeta *meta, const float *ksum, const float *S_in,
                            const float *z_in, float *S_out, float *z_out, void *o,
                            int need_z, const SegPlan &seg, cudaStream_t st);

// state_tc.cu: partial states of the pieces of a SegPlan (tensor cores).
// Piece i covers chunks [i piece_len, min((i+1) piece_len, chunks)).
cudaError_t launch_state_tc(const KParams &p, const void *Kp, const void *v,
                            const ChunkMeta *meta, const float *ksum, int npieces,
                            int piece_len, float *Part, float *zPart, int need_z,
                            cudaStream_t st);

// state_combine.cu: S_out = sum_i gamma_h^(t_i) S_i over the parts (null
// entries skipped), z likewise; either output may be null and may alias a
// part.  States fp32 [B*H][d_k][d_v], z fp32 [B*H][d_k].
constexpr int kMaxCombineParts = 64;
struct CombineParts {
  int count = 0;
  const float *S[kMaxCombineParts] = {};
  const float *z[kMaxCombineParts] = {};
  long long t[kMaxCombineParts] = {};
};
cudaError_t launch_state_combine(const KParams &p, const CombineParts &parts, float *S_out,
                                 float *z_out, cudaStream_t st);
// The state after the call's tokens on CUDA cores: Kr rotated keys fp32
// [B*H][N][d_k], v through sv[]; S_out/z_out may alias S_in/z_in; either
// output may be null.
cudaError_t launch_state_simt(const KParams &p, const float *Kr, const void *v,
                              const float *S_in, const float *z_in, float *S_out, float *z_out,
                              cudaStream_t st);

// recurrent.cu: one decode step, state in place.  gate (optional, bf16
// [B][H][d_v]): the output is multiplied by swish(gate) after its bf16
// rounding, as the MSR layer's gate pass would.
cudaError_t launch_recurrent_step(const KParams &p, const void *q, const void *k,
                                  const void *v, float *S, float *z, void *o,
                                  cudaStream_t st, const void *gate = nullptr);

// gemm_tc.cu: tensor-core C[M,N] = A[M,K] B[K,N] (bf16 row-major, fp32
// accumulate); N % 256, K % 64 == 0 (any M >= 1) and 16-byte aligned pointers.
bool gemm_tc_supported(const void *A, const void *Bm, const void *C, int M, int N, int K);
// gate: C <- swish(A B) (.) C (bf16 C read and rewritten in the epilogue).
cudaError_t launch_gemm_tc(const void *A, const void *Bm, void *C, int M, int N, int K,
                           unsigned *status, cudaStream_t st, bool gate = false);
// Up to four B matrices of one A (same K), split over K: fp32 partials
// P[ks][M][sum N_i] (matrix i at its column offset), added by the skinny
// reduce (launch_skinny_reduce_split).  gemm_tc_split: the K split for a
// shape (about two work items per SM, partials at most 1/4 of B's bytes).
constexpr int kGemmJobMax = 4;
struct GemmJob {
  CUtensorMap tmB[kGemmJobMax];
  int count = 0, ldc = 0, ksplit = 1;
  int ntile0[kGemmJobMax + 1] = {}, col0[kGemmJobMax] = {};
  __nv_bfloat16 *C = nullptr;
  float *P = nullptr;
  int early_b = 0;  // B tiles of the first stages loaded before pdl_wait (as for the skinny job)
};
int gemm_tc_split(int M, int Ntot, int K);
cudaError_t launch_gemm_tc_partials(const void *A, int count, const void *const *Bs,
                                    const int *Ns, int M, int K, float *P, int ksplit,
                                    unsigned *status, cudaStream_t st, bool early_b = false);

// gemm_simt.cu: C[M,N] = A[M,K] B[K,N], bf16 in (row-major), fp32 accumulate.
cudaError_t launch_gemm_bf16(const void *A, const void *Bm, void *C, int M, int N,
                             int K, int out_bf16, cudaStream_t st);

// backward.cu: gradients on CUDA cores (fp32).  Z, Qr, Kr: rotated
// contiguous fp32 [B*H][N][d_k]; dO through so[] (out dtype); row outputs
// fp32 [B*H][N][d_k]; dv through sv[] (in dtype); states fp32 [B*H][d_k][d_v].
// rev = false: dQ' from S_in (T0) and K' (Z); rev = true: dK' from dS_out
// (T0) and Q' (Z).
cudaError_t launch_bwd_rows(const KParams &p, bool rev, const float *Z, const void *v,
                            const void *dO, const float *T0, float *out, cudaStream_t st);
cudaError_t launch_bwd_values(const KParams &p, const float *Qr, const float *Kr,
                              const void *dO, const float *dS_out, void *dv, float *dS_in,
                              cudaStream_t st);
// x (contiguous fp32 [B*H][N][d_k]) turned by e^{-i t theta} into out (strides s).
cudaError_t launch_unrotate(const KParams &p, const float *x, const long long s[3], void *out,
                            int out_bf16, cudaStream_t st);

// parallel_tc.cu: the parallel form on the tensor cores.  Qp, Kp and meta
// from launch_rotate_qk (64-token chunks).  d_v <= 256 (one CTA per row):
// writes o itself (*fused = true).  Wider: writes the raw rows Oraw [B*H][N]
// [d_v] and the row factors F [B*H][N] that launch_groupnorm turns into o.
// d_k a multiple of 64 up to 256, d_v a multiple of 128 up to 1024.
cudaError_t launch_parallel_tc(const KParams &p, const __half *Qp, const __half *Kp, const void *v,
                               const ChunkMeta *meta, float *Oraw, float *F, void *o,
                               bool *fused, cudaStream_t st);

// backward_tc.cu: operands of the tensor-core backward's forward runs.
// A prep job reads rows of src (strides s, bf16 or fp32, row width d, a
// multiple of 8), optionally rotates them (+t theta) and scales them by the
// first two normalisations' row factor, and writes bf16 rows to fwd[bh][t]
// and/or rev[bh][N-1-t] (contiguous [B*H][N][d], 16-byte aligned).
struct BwdPrepJob {
  const void *src = nullptr;
  long long s[3] = {};
  int bf16 = 1, d = 0, rotate = 0, rowscale = 0, vec = 0;
  __nv_bfloat16 *fwd = nullptr, *rev = nullptr;
};
constexpr int kBwdPrepMax = 4;
struct BwdPrepJobs {
  int count = 0;
  BwdPrepJob job[kBwdPrepMax];
};
cudaError_t launch_bwd_prep(const KParams &p, BwdPrepJobs jobs, cudaStream_t st);
// T_j[bh][e][a] = S[bh][a][j w + e]: the column blocks of width w transposed.
cudaError_t launch_bwd_transpose(const float *S, int BH, int dk, int dv, int w, float *T,
                                 cudaStream_t st);
// out (strides s, dtype) at t = the sum of n_in fp32 [B*H][N][d] inputs at
// row (reverse ? N-1-t : t), times the row factor when rowscale is set,
// turned back by -t theta when unrotate is set.
constexpr int kBwdFinishMax = 8;
struct BwdFinish {
  const float *x[kBwdFinishMax] = {};
  int n_in = 0, d = 0, reverse = 0, rowscale = 0, unrotate = 0, out_bf16 = 1, vec = 0;
  long long s[3] = {};
  void *out = nullptr;
};
cudaError_t launch_bwd_finish(const KParams &p, BwdFinish F, cudaStream_t st);

// block.cu: the RetNet block's LayerNorm (bf16 rows of d, fp32 gain and
// bias), skip connection y <- y + r and in-place GELU (bf16, n values).
// pdl = false: the kernel starts only once everything before it on the
// stream is complete (the first kernel of a chain whose later kernels read
// data before their pdl_wait, see launch_gemm_skinny_job).
cudaError_t launch_layernorm(const void *x, const float *w, const float *b, void *y, long long rows,
                             int d, float eps, cudaStream_t st, bool pdl = true);
cudaError_t launch_residual_add(void *y, const void *r, long long n, cudaStream_t st);
cudaError_t launch_gelu(void *y, long long n, cudaStream_t st);

// Rows (i, j) of a strided matrix, i < n0, j < n1, numbered r = i n1 + j:
// row r starts at element i s0 + j s1, its values are contiguous.
struct RowSet {
  long long n0 = 1, n1 = 0, s0 = 0, s1 = 0;
};

// layernorm.cu: LayerNorm and its gradients over `rows` rows of d values.
// Forward: x -> out = y, mean and rstd written where not null.  Backward:
// x, dy, mean, rstd -> out = dx and, per CTA, partial sums of dw and db
// (part [groups][2][d], null = not wanted) that launch_layernorm_bwd_sum
// adds.  A two-pass plan (rows too long for registers) first writes stat
// [rows][2].  out may be x or dy themselves.
struct LnArgs {
  const void *x = nullptr, *dy = nullptr;
  void *out = nullptr;
  const float *w = nullptr, *b = nullptr;
  float *mean = nullptr, *rstd = nullptr;
  RowSet sx, sg, so;
  long long rows = 0;
  int d = 0;
  float eps = 0.f;
};
struct LnBwdPlan {
  bool vec = false, narrow = false, wide = false, two_pass = false;
  int tpr = 0, threads = 0, groups = 0;  // threads a row, of a CTA; CTAs
};
cudaError_t launch_layernorm_rows(const LnArgs &a, int bf16, cudaStream_t st);
LnBwdPlan layernorm_bwd_plan(const LnArgs &a, int bf16);
size_t layernorm_bwd_bytes(long long rows, int d);  // stat and part
cudaError_t launch_layernorm_bwd_stat(const LnArgs &a, int bf16, const LnBwdPlan &pl, float *stat,
                                      cudaStream_t st);
cudaError_t launch_layernorm_bwd(const LnArgs &a, int bf16, const LnBwdPlan &pl, const float *stat,
                                 float *part, cudaStream_t st);
cudaError_t launch_layernorm_bwd_sum(const float *part, int groups, int d, float *dw, float *db,
                                     cudaStream_t st);

// logits.cu: one pass over each row of logits [rows][V] (bf16 or fp32).
struct LogprobArgs {
  const void *x = nullptr;
  RowSet sx;
  long long rows = 0;
  int V = 0, top = 0, id64 = 1;
  float inv_t = 1.f, scale = 1.f;  // 1 / temperature, log2(e) / temperature
  const void *tokens = nullptr;    // [rows] int32 / int64, null = none
  float *logprob = nullptr, *entropy = nullptr, *top_logprob = nullptr;
  long long *top_id = nullptr;
};
cudaError_t launch_token_logprobs(const LogprobArgs &a, int bf16, cudaStream_t st);

// distill.cu: the loss against a teacher's list and its gradient.
enum { kDistillFwd = 1, kDistillBwd = 2, kDistillStep = 3 };
struct DistillArgs {
  const void *x = nullptr;
  void *dx = nullptr;
  RowSet sx, sd;
  long long rows = 0;
  int V = 0, top = 0, id64 = 1, tail = 0;
  float inv_t = 1.f, scale = 1.f, t = 1.f;
  const void *ids = nullptr;       // [rows][top]
  const float *values = nullptr;   // [rows][top]
  const float *weight = nullptr;   // [rows], null = 1
  float *loss = nullptr, *stats = nullptr;  // [rows], [rows][2]
};
cudaError_t launch_distill(const DistillArgs &a, int bf16, int what, cudaStream_t st);

// scan_fwd.cu, scan_bwd.cu: the selective scan over [B][N][E] channels with S
// states each, and its gradients.  Strides in elements: (batch, token) of the
// channels' tensors, (batch, token, group) of B and C.  A [E][S], states
// [B][E][S], D, bias [E]: contiguous fp32.
struct ScanArgs {
  int B = 0, N = 0, E = 0, S = 0, G = 1, softplus = 1;
  const void *x = nullptr, *dt = nullptr, *z = nullptr, *Bm = nullptr, *Cm = nullptr, *dy = nullptr;
  const float *A = nullptr, *D = nullptr, *bias = nullptr, *h_in = nullptr, *dh_out = nullptr;
  const void *lengths = nullptr;  // [B] int32 / int64, null = N
  int len64 = 0;
  void *y = nullptr, *dx = nullptr, *ddt = nullptr, *dz = nullptr, *dBm = nullptr, *dCm = nullptr;
  float *h_out = nullptr, *dA = nullptr, *dD = nullptr, *dbias = nullptr, *dh_in = nullptr;
  long long sx[2] = {}, sdt[2] = {}, sz[2] = {}, sdy[2] = {}, sy[2] = {}, sdx[2] = {}, sddt[2] = {},
            sdz[2] = {}, sB[3] = {}, sC[3] = {};
  int pair_y = 0;  // y's rows begin on a pair's boundary (set by the launcher)
};
// Segments of a sequence that run at once; loc [count-1][B][E][S]: the state
// that each segment but the last leaves behind from a zero state, sum
// [count-1][B][E]: its step sizes added up.
struct ScanSegs {
  int count = 1, len = 0;
  float *loc = nullptr, *sum = nullptr;
};
ScanSegs scan_fwd_plan(const ScanArgs &a);
size_t scan_fwd_bytes(const ScanArgs &a);  // loc and sum
cudaError_t launch_scan_states(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st);
cudaError_t launch_scan_fwd(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st);
// Gradients, in chunks of `chunk` tokens that run on their own once the states
// at their ends are known.  h, g [chunks][B][E][S]: first what a chunk alone
// adds to the state after it (h) and to the state's gradient before it (g),
// then the state before it and the gradient that arrives behind it; dA's
// partial sums take h's place.  sum [chunks][B][E]: step sizes added up.
// bc [blocks][B][N][G][2][S]: a channel block's share of dB and dC.  dd
// [2][chunks][B][E]: partial sums of dD and dbias.
struct ScanBwdPlan {
  int chunk = 0, chunks = 0, blocks = 0;
  size_t g = 0, sum = 0, bc = 0, dd = 0, total = 0;  // offsets in floats (h at 0)
};
ScanBwdPlan scan_bwd_plan(const ScanArgs &a);
cudaError_t launch_scan_bwd_chunks(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st);
cudaError_t launch_scan_bwd_carry(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st);
cudaError_t launch_scan_bwd_bc(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, const float *ws, cudaStream_t st);

// colsum.cu: out[c] = sum_p part[p * stride + c], p < count, in a fixed order.
// Up to three such sums of one count in a launch (out null = none).
struct ColSum {
  const float *part[3] = {};
  long long stride[3] = {};
  int cols[3] = {}, count = 0;
  float *out[3] = {};
};
cudaError_t launch_colsum(const ColSum &c, cudaStream_t st);

// One token: x, dt, z, y [B][E], B, C [B][G][S]; h_out may be h_in.
cudaError_t launch_scan_step(const ScanArgs &a, int bf16, cudaStream_t st);

// conv.cu: the short causal convolution over [B][N][E], W taps (2 to 4), and
// its gradients.  w [E][W], b [E] fp32; states [B][W-1][E] contiguous in the
// tensors' type, null = zeros / not wanted.
struct ConvArgs {
  int B = 0, N = 0, E = 0, W = 0, silu = 1;
  const void *x = nullptr, *dy = nullptr, *state_in = nullptr, *dstate_out = nullptr;
  const float *w = nullptr, *b = nullptr;
  const void *lengths = nullptr;
  int len64 = 0;
  void *out = nullptr, *state_out = nullptr, *dstate_in = nullptr;  // out: y or dx
  long long sx[2] = {}, sg[2] = {}, so[2] = {};                    // of x, dy, out: (batch, token)
};
cudaError_t launch_conv_fwd(const ConvArgs &a, int bf16, cudaStream_t st);
// Partial sums of dw and db: part [runs][E][W] and then [runs][E], a run of
// tokens each (null = not wanted).
int conv_bwd_runs(const ConvArgs &a);
cudaError_t launch_conv_bwd(const ConvArgs &a, int bf16, float *part, cudaStream_t st);

// rmsnorm.cu: h = x + r (r null: x), y = h rstd w over rows of d values.
struct RmsArgs {
  const void *x = nullptr, *r = nullptr, *dy = nullptr, *dh = nullptr;
  void *h = nullptr, *out = nullptr;  // out: y, e4m3 values or dx
  const float *w = nullptr;
  float *rstd = nullptr, *scales = nullptr;
  RowSet sx, sr, sh, sg, sdh, so;
  long long rows = 0;
  int d = 0, group = 0, groups = 1, shift = -1;  // group: columns of a scale; 2^shift of them (launcher)
  float eps = 0.f;
};
cudaError_t launch_rmsnorm_fwd(const RmsArgs &a, int bf16, cudaStream_t st);
cudaError_t launch_rmsnorm_quant(const RmsArgs &a, int bf16, cudaStream_t st);
// x holds h.  dw's partial sums: part [groups][d]; stat [rows] for rows too
// long for registers.
struct RmsBwdPlan {
  bool vec = false, two_pass = false;
  int values = 0, tpr = 0, groups = 0;  // values a thread, threads a row; CTAs
};
RmsBwdPlan rmsnorm_bwd_plan(const RmsArgs &a, int bf16);
size_t rmsnorm_bwd_bytes(long long rows, int d, int bf16);  // part and stat
cudaError_t launch_rmsnorm_bwd_stat(const RmsArgs &a, int bf16, const RmsBwdPlan &pl, float *stat, cudaStream_t st);
cudaError_t launch_rmsnorm_bwd(const RmsArgs &a, int bf16, const RmsBwdPlan &pl, const float *stat, float *part,
                               cudaStream_t st);

// gemm_skinny.cu: C[M,N] = A[M,K] B[K,N] for M <= 16 rows (bf16 row-major,
// fp32 accumulation), split over K into fp32 partials [split][M][N] that
// launch_skinny_reduce adds in order into bf16 C.  Needs N % 8 == 0 and a
// 16-byte aligned B.
bool gemm_skinny_supported(const void *A, const void *Bm, const void *C, int M, int N, int K);
size_t gemm_skinny_partial_bytes(int M, int N, int K);
cudaError_t launch_gemm_skinny(const void *A, const void *Bm, int M, int N, int K,
                               float *partial, cudaStream_t st);
cudaError_t launch_skinny_reduce(const float *partial, void *C, int M, int N, int K,
                                 cudaStream_t st);
// Up to four weight matrices with the same K read in one launch (their
// columns side by side in the partials), and the reduce's epilogue: none,
// GELU, or a skip connection (one matrix; C = sum + R, R [M][N] bf16).
constexpr int kSkMaxMats = 4;
enum { kSkEpNone = 0, kSkEpGelu = 1, kSkEpResidual = 2 };
struct SkinnyJob {
  int count = 0, Ntot = 0, epi = kSkEpNone;
  const __nv_bfloat16 *B[kSkMaxMats] = {};
  __nv_bfloat16 *C[kSkMaxMats] = {};
  int N[kSkMaxMats] = {}, col0[kSkMaxMats] = {}, blk0[kSkMaxMats + 1] = {};
  const __nv_bfloat16 *R = nullptr;
};
bool skinny_job_init(SkinnyJob &job, int count, const void *const *Bs, void *const *Cs,
                     const int *Ns, int epi, const void *R);
// early_b: the first rows of the weights are copied before the kernel's
// pdl_wait, overlapping the kernel before it.  Only for callers that know
// no kernel that may still run writes the weights: every kernel launched
// since the last launch without programmatic serialization.
cudaError_t launch_gemm_skinny_job(const void *A, const SkinnyJob &job, int M, int K,
                                   float *partial, cudaStream_t st, bool early_b = false);
cudaError_t launch_skinny_reduce_job(const float *partial, const SkinnyJob &job, int M, int K,
                                     cudaStream_t st);
// The same reduce over `split` given slices (the tensor-core GEMM's partials).
cudaError_t launch_skinny_reduce_split(const float *partial, const SkinnyJob &job, int M,
                                       int split, cudaStream_t st);

}  // namespace ret
