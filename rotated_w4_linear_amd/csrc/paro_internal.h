// Internal declarations shared by the host library and the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

#include "../../include/paro.h"

namespace paro {

// ---------------------------------------------------------------------------
// Rotation schedule for the activation kernel.
//
// The d channels are cut into segments of 128 channels (groups of 64 or 128:
// one or two groups per segment) or 256 channels (group 256). One wavefront
// processes one segment of a token: "virtual lane" v (0 .. SEG/2-1) holds two
// channels, in registers X and Y; with 256-channel segments a hardware lane
// holds two virtual lanes (v = lane and v = lane + 64).
//
// Between two consecutive pairings (the natural pairing {2v, 2v+1} before
// stage 0 and after stage K-1, and the K stages in between) every virtual
// lane keeps one of its two channels (in X) and fetches the other member of
// its next pair from the Y register of another virtual lane, through a
// per-wave LDS tile. The two pairings together form disjoint even cycles, so
// a "keep one, fetch one" assignment always exists.
//
// Table image per segment: NW fields (padded with zero words to a multiple of
// four) for each of NV virtual lanes, four fields interleaved per lane so that
// a lane loads four consecutive fields with one 16-byte load and a wavefront's
// load is one contiguous 1 KB: field f of virtual lane v is word
// ((f / 4) * NV + v) * 4 + f % 4 of the segment. Field order:
//   0                 load selector (v_perm byte selector putting the kept
//                     channel of the natural pair in the low half)
//   1 + 2*tau         LDS byte offset the lane writes its Y to, tau = 0..K
//   2 + 2*tau         LDS byte offset the lane reads its fetched value from
//   3 + 2*K + c*t + e stage t coefficient e (c = 2 for the factored form,
//                     4 for the general 2x2 form)
//   then              final scale of X, final scale of the fetched value,
//                     store byte offset of the natural pair, store selector.
// After all segments' images: the store permutation, [segs][NV][2] words.
// Virtual lane v ends the last exchange holding the natural pair q(v) (the
// pair at the store byte offset above); word 0 of lane v is the LDS byte
// offset it writes its packed output word to, word 1 the offset virtual lane
// v reads natural pair v from (slots planned like an exchange's).
// ---------------------------------------------------------------------------
struct RotPlanLayout {
  int seg_ch = 128;      // channels per segment
  int ppl = 1;           // virtual lanes per hardware lane
  int nv = 64;           // virtual lanes per segment
  int coef = 2;          // coefficients per stage (2 factored, 4 general)
  int words = 0;         // words per virtual lane (fields rounded up to four)
  int stages = 0;        // stages the activation schedule executes (<= K)
  bool fast = true;      // factored two-FMA stage form
};

inline int rot_field_count(int K, int coef) { return 1 + 2 * (K + 1) + coef * K + 4; }
// words per virtual lane in the image: the field count rounded up to four
inline int rot_words(int K, int coef) { return (rot_field_count(K, coef) + 3) & ~3; }

// first word of the store permutation, and the whole image, in words
inline size_t rot_perm_base(int64_t segs, const RotPlanLayout& lay) { return (size_t)segs * lay.words * lay.nv; }
inline size_t rot_table_words(int64_t segs, const RotPlanLayout& lay) {
  return rot_perm_base(segs, lay) + (size_t)segs * lay.nv * 2;
}

struct RotPlanHost {
  RotPlanLayout lay;
  std::vector<uint32_t> table;  // [segs][words / 4][nv][4], then [segs][nv][2]
  // canonical fp32 tables for the weight transform, per group, stage, pair:
  // local (i | j << 16), c bits, s bits
  std::vector<uint32_t> wt_pairs;  // [groups][K][G/2]
  std::vector<float> wt_c, wt_s;   // [groups][K][G/2]
  std::vector<float> alpha;        // [d]
  // gradient kernel: per segment, stage, lane slot: (i | j << 16, c bits,
  // s bits, flat pair index)
  std::vector<uint32_t> bw;        // [segs][K][seg_ch / 2][4]
};

// Validates arguments and builds the schedule. Returns a paro_status.
int build_rotation_plan(int64_t d, int32_t group, int32_t K, const int32_t* pairs,
                        const float* theta, const float* alpha, RotPlanHost* out);

void set_error(const std::string& msg);

// Gradients of the transform (activation side: X' = X T^-1; weight side:
// rows of T W). part is scratch of rotate_backward_scratch_bytes(r, M).
size_t rotate_backward_scratch_bytes(const paro_rotation* r, int64_t M);
hipError_t launch_rotate_backward(const paro_rotation* r, int weight_side, const uint16_t* x,
                                  const float* gy, float* gx, float* dtheta, float* dalpha,
                                  int64_t M, void* part, hipStream_t stream);

// Layer-wise output loss and its straight-through angle/scale gradients
// (layer_loss.hip): scratch bytes, the whole computation, and a zero fill.
size_t layer_loss_scratch_bytes(const paro_rotation* r, int64_t M, int64_t N, int64_t d, bool grad);
int run_layer_loss(const paro_rotation* r, const uint16_t* x, const uint16_t* w, const uint8_t* qw,
                   const uint16_t* sc, const uint8_t* zr, int64_t M, int64_t N, int64_t d, int group,
                   float* loss, float* dtheta, float* dalpha, void* ws, hipStream_t stream);
hipError_t launch_fill_zero(float* a, int64_t n, hipStream_t stream);

}  // namespace paro

struct paro_rotation {
  int64_t d;
  int32_t group;
  int32_t K;
  int device;
  paro::RotPlanLayout lay;
  uint32_t* d_table;    // device copy of RotPlanHost::table
  uint32_t* d_wt_pairs; // device canonical weight-transform tables
  float* d_wt_c;
  float* d_wt_s;
  float* d_alpha;
  uint32_t* d_bw;       // device copy of RotPlanHost::bw
};

namespace paro {
// Kernel launchers (defined in the .hip files). Return hipError_t of the launch.
hipError_t launch_rotate(const paro_rotation* r, const uint16_t* x, uint16_t* y, int64_t M,
                         hipStream_t stream);
// err (NULL or 4-byte aligned): also writes the quantization error
// E = W_hat - T W [N][d] (W_hat = (q - z) s, T W in the canonical fp32 order)
// rounded to fp16
hipError_t launch_quantize(const paro_rotation* r, const uint16_t* w, int64_t N, int64_t d,
                           int group, uint8_t* qweight, uint16_t* scales, uint8_t* zeros,
                           int* d_flag, hipStream_t stream, uint16_t* err = nullptr);
// Dense fp16 "NT" products (dense_gemm.hip), C[m][n] = sum_k A[m][k] B[n][k]
// with fp32 accumulation; K % 64 == 0, row strides in elements, 16-byte
// aligned rows.
//  * launch_nt_gemm_f32: C fp32 [M][ldc].
//  * launch_nt_gemm_loss: A = x [M][d], B = w [N][d]; part[nt_tiles(M, N)]
//    receives the per-tile sums of (yq - x w^T)^2 (yq fp16 [M][N]) and, with dy
//    != NULL, dy [M][ldd] = fp16(2 (yq - x w^T)), zero in columns N .. ldd - 1.
//  * launch_transpose_pad: out [C][ldo] = in^T for in fp16 [R][C] (C even,
//    ldo even, ldo >= R), zero in columns R .. ldo - 1.
int nt_tiles(int64_t M, int64_t N);
// Plain device copy (copy.hip): bytes % 16 == 0, 16-byte aligned pointers.
hipError_t launch_stream_copy(const void* src, void* dst, size_t bytes, int blocks, hipStream_t stream);
hipError_t launch_mfma_loop(const void* src, int64_t n8, float* out, int blocks, int iters, hipStream_t stream);
hipError_t launch_nt_gemm_f32(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb,
                              int64_t M, int64_t N, int64_t K, float* c, int64_t ldc,
                              hipStream_t stream);
hipError_t launch_nt_gemm_loss(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N, int64_t d,
                               const uint16_t* yq, uint16_t* dy, int64_t ldd, float* part,
                               hipStream_t stream);
hipError_t launch_transpose_pad(const uint16_t* in, int64_t R, int64_t C, uint16_t* out, int64_t ldo,
                                hipStream_t stream);
// Large-batch linear (M > 16) on already transformed activations. The plan
// says whether the 256 x 256-tile kernel runs, and whether stream-K (the
// tiles' k-tiles shared out among the workgroups); a stream-K run needs the
// arrival counters (zero between calls) and partial_bytes of fp32 partial
// tiles, and without them (NULL) the layer takes the smaller-tile kernel.
struct GemmPlan {
  bool wide = false;
  bool sk = false;
  int sk_slots = 0;  // stream-K workgroups per XCD
  int nsplit = 1;    // smaller-tile kernel: workgroups per tile along k
  size_t partial_bytes = 0;
};
GemmPlan plan_w4_gemm(int64_t M, int64_t N, int64_t d);
hipError_t launch_w4_gemm(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                          const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                          int64_t N, int64_t d, int group, uint32_t* cnt, float* part, hipStream_t stream);
// What an epilogue of the W4 products needs beside the bias: aux, the residual
// (may be NULL) or dy, fp16 [M][N]; act, a paro_activation.
struct W4Epilogue {
  const uint16_t* aux = nullptr;
  int32_t act = 0;
};
// Whether paro_device_init found workgroup b running on XCD b % 8.
bool xcd_dispatch_is_round_robin();

// Small-batch linear (M <= kDecodeMaxM). With r != NULL the activation transform runs
// inside the kernel (requires decode_fuses_rotation(r)); ws is the workspace:
// kDecodeCounterBytes of arrival counters (zero between calls), then the fp32
// partial sums [ceil(d / 512)][M][N].
constexpr size_t kDecodeCounterBytes = 16384;
constexpr int64_t kDecodeMaxM = 64;
bool decode_fuses_rotation(const paro_rotation* r);
// whether the small-batch call with these sizes fuses it (else the transform
// runs first, into the workspace)
bool decode_fuses_rotation(const paro_rotation* r, int64_t M, int64_t N, int64_t d);
// Devices the library keeps per-device state for (device ordinals below this).
constexpr int kMaxDevices = 64;
// Runs the XCD dispatch probe on device dev (current) once and records the
// result; allocates, launches and synchronizes. Returns a paro_status.
int xcd_dispatch_probe(int dev);

// Static device scratch of paro_w4_linear_noalloc (noalloc.hip): its size,
// the once-per-device look-up of its address (with dev current; clears the
// arrival counters and synchronizes) and the recorded address (NULL before
// set-up).
constexpr size_t kNoallocScratchBytes = (size_t(64) << 20) + kDecodeCounterBytes;
int noalloc_scratch_setup(int dev);
void* noalloc_scratch(int dev);
hipError_t launch_w4_decode(const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                            const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                            int64_t N, int64_t d, int group, const paro_rotation* r, void* ws,
                            hipStream_t stream);
// The same kernels with an epilogue (w4_epilogue.h). N: output channels; the
// gated ones take a weight block of 2 N rows, and launch_w4_gemm_gated_grad
// writes [M][2 N].
hipError_t launch_w4_gemm_act(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    uint32_t* cnt, float* part, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_gemm_gated(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    uint32_t* cnt, float* part, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_gemm_act_grad(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    uint32_t* cnt, float* part, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_gemm_gated_grad(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    uint32_t* cnt, float* part, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_decode_act(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    const paro_rotation* r, void* ws, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_decode_gated(
    const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
    const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d, int group,
    const paro_rotation* r, void* ws, const W4Epilogue& ep, hipStream_t stream);

// The act and gated products on at most kRowsMaxM tokens whose activations are
// transformed already (decode_rows.hip); no workspace.
constexpr int64_t kRowsMaxM = 16;
hipError_t launch_w4_rows(bool gated, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                          const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d,
                          int group, const W4Epilogue& ep, hipStream_t stream);
// The products with an epilogue (any but kEpiPlain) in small tiles, k inside the
// workgroup (w4_tiles.hip); no workspace. N: output channels, P: weight rows.
// w4_tiles_fit: whether they are taken before the kernels of w4_gemm_kernels.h.
bool w4_tiles_fit(int64_t M, int64_t P, int64_t d);
hipError_t launch_w4_tiles(int epi, const uint16_t* x, const uint8_t* qweight, const uint16_t* scales,
                           const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t d,
                           int group, const W4Epilogue& ep, hipStream_t stream);

// Gradient of a W4 product at its input (w4_input_grad.hip): dx fp16 [M][d] =
// dz [M][P] W_hat, P the rows of the weight block (a multiple of 16); cnt are
// arrival counters (zero between calls), ws holds input_grad_scratch_bytes(M, P, d).
size_t input_grad_scratch_bytes(int64_t M, int64_t P, int64_t d);
hipError_t launch_w4_input_grad(const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                                const uint8_t* zeros, uint16_t* dx, int64_t M, int64_t P, int64_t d, int group,
                                uint32_t* cnt, void* ws, hipStream_t stream);
// The same for few tokens, straight from the codes (w4_input_grad_rows.hip);
// scratch holds input_grad_rows_bytes. input_grad_rows_fit: whether
// launch_w4_input_grad takes it.
bool input_grad_rows_fit(int64_t M);
size_t input_grad_rows_bytes(int64_t M, int64_t P, int64_t d);
hipError_t launch_w4_input_grad_rows(const uint16_t* dz, const uint8_t* qweight, const uint16_t* scales,
                                     const uint8_t* zeros, uint16_t* dx, int64_t M, int64_t P, int64_t d, int group,
                                     void* scratch, hipStream_t stream);

// One launch of the AdamW step (adamw.hip). Every tensor is cut into chunks of
// kAdamChunk values; chunk0 is its first chunk of the launch, block0 its first
// block of 256 moments. Up to kAdamTensors tensors travel as kernel arguments
// (AdamwLaunch), more of them as a table in device memory (AdamwTable: the
// tensors, and the tensor of each chunk).
constexpr int kAdamTensors = 120;
constexpr int kAdamChunk = 2048;
struct AdamwTensor {
  void* p;
  const void* g;
  int64_t n;
  uint32_t chunk0, block0;
};
struct AdamwScalars {
  void *m, *v;
  float *ms, *vs;
  float b1, c1, b2, c2;          // b, 1 - b
  float keep, rate, root, eps;   // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};
struct AdamwLaunch {
  AdamwScalars s;
  int32_t count;
  AdamwTensor t[kAdamTensors];
};
struct AdamwTable {
  AdamwScalars s;
  const AdamwTensor* t;
  const uint32_t* of_chunk;
};
hipError_t launch_adamw(const AdamwLaunch& a, uint32_t chunks, int param_type, int grad_type, bool eight,
                        hipStream_t stream);
hipError_t launch_adamw(const AdamwTable& a, uint32_t chunks, int param_type, int grad_type, bool eight,
                        hipStream_t stream);

// Mixture of experts. The limits of a routing, and its tables as the kernels take
// them: R = M k pairs, rows in expert order.
constexpr int kExpertsMax = 1024, kExpertsMaxK = 16;
struct ExpertRouting {
  int M, E, k, R;
  const int *ids, *offsets, *order, *place;
  const float* weights;
};
// Most blocks of at most bm rows of one expert that R rows in E experts make.
inline int64_t expert_blocks(const ExpertRouting& t, int bm) {
  const int64_t full = t.R / bm, used = t.E < t.R ? t.E : t.R;
  return full + used < t.R ? full + used : t.R;
}
// The router (logits NULL: the tables of given ids) and its gradient
// (experts_route.hip); scratch holds experts_route_scratch(M, E, k) bytes.
size_t experts_route_scratch(int64_t M, int E, int k);
hipError_t launch_experts_route(const void* logits, int type, int64_t M, int E, int k, int normalize, int* ids,
                                float* weights, int* offsets, int* order, int* place, void* scratch,
                                hipStream_t stream);
hipError_t launch_experts_route_backward(const void* logits, int type, int64_t M, int E, int k, int normalize,
                                         const int* ids, const float* weights, const float* dweights, void* dlogits,
                                         hipStream_t stream);
// The experts' products: epi kEpiGated and kEpiGatedGrad on tokens x, kEpiShare on rows
// x in expert order; y by row. For few pairs in all (decode_rows.hip).
hipError_t launch_w4_experts_rows(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                  const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                  int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream);
// The same for up to some hundred rows of an expert (w4_experts_mid.hip).
hipError_t launch_w4_experts_mid(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                 const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                 int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream);
// The same in 256 x 256 tiles (w4_experts_wide.hip), and whichever fits.
hipError_t launch_w4_experts_wide(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                                  const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y,
                                  int64_t N, int64_t d, int group, const W4Epilogue& ep, hipStream_t stream);
hipError_t launch_w4_experts(int epi, const ExpertRouting& t, const uint16_t* x, const uint8_t* qweight,
                             const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, void* y, int64_t N,
                             int64_t d, int group, const W4Epilogue& ep, hipStream_t stream);
// part [splits][R][d] = dz W_hat of each row's expert, in pieces of the
// contraction (w4_input_grad_rows.hip); gather: dz by token, else by row.
int experts_grad_rows_splits(const ExpertRouting& t, int64_t P, int64_t d);
// Row counts R up to which (one at least of each pair of choices) the rules above and
// those of the large tiles choose alike: more rows can need less room behind one.
void experts_grad_rows_steps(int64_t E, int64_t d, std::vector<int64_t>& rows);
void experts_grad_wide_steps(int64_t E, int64_t d, std::vector<int64_t>& rows);
hipError_t launch_w4_experts_grad_rows(const ExpertRouting& t, bool gather, const uint16_t* dz,
                                       const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                                       float* part, int64_t P, int64_t d, int group, hipStream_t stream);
// The same in large tiles for experts of many rows (w4_experts_grad.hip): part
// [experts_grad_splits][R][d] (dz by row), or dh = w U and the partial dots U . h (dy by token).
bool experts_grad_wide_fit(const ExpertRouting& t, int64_t P, int64_t d, bool share);
int experts_grad_splits(const ExpertRouting& t, int64_t P, int64_t d);
size_t experts_grad_dots(const ExpertRouting& t, int64_t d);
hipError_t launch_w4_experts_grad_part(const ExpertRouting& t, const uint16_t* dz, const uint8_t* qweight,
                                       const uint16_t* scales, const uint8_t* zeros, float* part, int64_t P, int64_t d,
                                       int group, hipStream_t stream);
hipError_t launch_w4_experts_grad_share(const ExpertRouting& t, const uint16_t* dy, const uint8_t* qweight,
                                        const uint16_t* scales, const uint8_t* zeros, float* dots, const uint16_t* h,
                                        uint16_t* dh, int64_t P, int64_t d, int group, hipStream_t stream);
// Sums over a token's experts and the weights' gradients (experts_sum.hip):
//   y[m] = residual[m] + sum_s sum_p part[p][place[m][s]]  (fp16 [M][N]);
//   dh[r] = w U[r], dw[p] = U[r] . h[r] + dy[m] . bias[e], U = sum_p part[p].
hipError_t launch_experts_sum(const ExpertRouting& t, const float* part, int splits, const uint16_t* residual,
                              uint16_t* y, int64_t N, hipStream_t stream);
hipError_t launch_experts_share_grad(const ExpertRouting& t, const float* part, int splits, const uint16_t* h,
                                     const uint16_t* dy, const uint16_t* bias, uint16_t* dh, float* dweights,
                                     int64_t N, int64_t d, hipStream_t stream);
//   dw[p] = the pair's partial dots [count][R] + dy[m] . bias[e]
hipError_t launch_experts_dots(const ExpertRouting& t, const float* dots, int count, const uint16_t* dy,
                               const uint16_t* bias, float* dweights, int64_t N, hipStream_t stream);

// Distillation from a teacher's top logits (distill.hip).
struct DistillArgs {
  const void* z;          // [M][V]
  const void* values;     // [M][K]
  const int* index;       // [M][K]
  const float* lse;       // [M] or NULL
  const float* weight;    // [M] or NULL
  float* loss;            // [M]
  void* dz;               // [M][V] or NULL
  int64_t M;
  int V, K;
  float temperature, grad_scale;
};
hipError_t launch_distill(const DistillArgs& a, int z_type, int value_type, hipStream_t stream);

// Shared by the products' entry points (api.cpp): the argument checks (N: rows
// of the weight block; *noop set when M == 0), the smallest workspace, and the
// launches of the product with epilogue epi on a checked workspace.
int check_w4_linear(const char* fn, const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                    const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, const uint16_t* y, int64_t M,
                    int64_t N, int64_t d, int32_t group, bool* noop);
size_t w4_linear_min_workspace(const paro_rotation* r, int64_t M, int64_t N, int64_t d);
int run_w4_product(int epi, const W4Epilogue& ep, const paro_rotation* r, const uint16_t* x, const uint8_t* qweight,
                   const uint16_t* scales, const uint8_t* zeros, const uint16_t* bias, uint16_t* y, int64_t M,
                   int64_t N, int64_t d, int32_t group, char* ws, size_t ws_bytes, hipStream_t stream);
}  // namespace paro
