/*
 * fa.h -- C ABI of the fused exact attention forward library (libfa.so) for
 * NVIDIA GB300 (sm_103a).
 *
 * Operation.  Exact scaled-dot-product attention, forward pass:
 *     S = scale * Q K^T,   P = softmax(S) row-wise,   O = P V,
 *     LSE_i = ln sum_j exp(S_ij)
 * (definition: wmrh.cn FlashAttention V3 article, sec. 1.1 "self-attention
 * and the O(N^2) problem").  The kernels stream K/V tiles through shared
 * memory and run the online-softmax recurrence -- running row max m, running
 * row sum l, rescaled accumulator o, initially -inf, 0, 0, output o/l after
 * the last tile (same article, sec. 2.1; "FlashAttention-3: async pipelines
 * on Hopper" (charlestar.github.io), section "Online Softmax is still the
 * core of exact merging") -- so the N x N score matrix never reaches HBM.
 * Causal attention keeps the lower triangle, key j <= query i, and skips the
 * key tiles above the diagonal ("FlashAttention-3: async pipelines on
 * Hopper", section "why causal shapes are harder to schedule").  The LSE
 * output is not defined on the pages; here it is the natural log of the sum
 * of exponentials of the scaled, masked scores, in fp32.
 *
 * Conventions shared by every entry point
 *   - Tensors are contiguous row-major [B, H, N, d] (PyTorch SDPA order,
 *     wmrh.cn article sec. 6.4); LSE is [B, H, N] fp32.
 *   - Every tensor pointer is a DEVICE pointer on the current CUDA device,
 *     16-byte aligned, owned by the caller.  Inputs are only read; outputs are
 *     fully overwritten.  The library allocates no memory in these calls.
 *   - Work is enqueued on `stream` and the call returns without waiting.
 *     A launch error is reported as FA_ERR_CUDA; errors found by the kernels
 *     (a pipeline wait that ran out of time) are reported later by
 *     fa_check_device_error().
 *   - B*H*N == 0 is valid and does nothing.
 *   - Head dimension d must be 64, 128 or 256.  The library runs only on
 *     compute capability 10.3 (sm_103a); anything else is FA_ERR_UNSUPPORTED.
 *     There is no fallback path.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, negative size, non-finite scale, bad dtype */
    FA_ERR_UNSUPPORTED = 2,   /* head dimension or device not supported                            */
    FA_ERR_CUDA = 3,          /* a CUDA runtime/driver call or kernel launch failed                 */
    FA_ERR_TIMEOUT = 4,       /* a kernel's pipeline wait ran out of time (see fa_check_device_error) */
    FA_ERR_SCRATCH_LIMIT = 5, /* problem larger than the library's static scratch (no-allocation entry point) */
    FA_ERR_INDEX = 6          /* a length, position or page number read from device memory was out of range
                                 (see fa_check_device_error)                                                 */
} fa_status;

typedef enum {
    FA_DTYPE_BF16 = 0,
    FA_DTYPE_FP16 = 1
} fa_dtype;

/* Maximum number of rows per FP8 quantisation block (one scale per block). */
#define FA_FP8_BLOCK_ROWS 128

/*
 * fa_fwd -- BF16 / FP16 attention forward.
 *   q, k, v  [B, H, N, d] of `dtype` (device, read only)
 *   o        [B, H, N, d] of `dtype` (device, written), rounded to nearest even
 *   lse      [B, H, N] fp32 (device, written)
 *   causal   0: every key visible; 1: key j visible to query i iff j <= i
 *   scale    multiplies Q K^T before the softmax (usually 1/sqrt(d)); finite
 *   dtype    FA_DTYPE_BF16 or FA_DTYPE_FP16
 * Softmax statistics and accumulation are fp32; P is rounded to `dtype`
 * before the P V product ("FlashAttention-3: async pipelines on Hopper",
 * section "Online Softmax is still the core of exact merging": FP16/BF16
 * keep the rescaling and accumulation state in FP32).
 * Non-finite inputs are not checked.  A NaN in a query row makes that row's
 * O and LSE NaN; a NaN in key row j makes NaN every row that sees key j.  A
 * NaN or infinity in element (j, c) of V reaches column c of O in every row
 * that sees key j and also, with causal = 1, in the rows of j's 128-row tile
 * that precede j (P V multiplies their P = 0 by it); rows of earlier tiles,
 * the other columns and LSE are unaffected.
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int64_t B, int64_t H, int64_t N, int64_t d,
                 int causal, float scale, int dtype, cudaStream_t stream);

/*
 * fa_fwd_fp8 -- FP8 E4M3 attention forward with per-block scales.
 *   q8, k8, v8  [B, H, N, d] E4M3 codes (device, read only), as written by
 *               fa_quant_fp8; real value = decode(code) * descale of its block
 *   q_descale, k_descale, v_descale
 *               [B, H, ceil(N/128)] fp32 (device): one scale per 128-row block
 *               ("FlashAttention-3: async pipelines on Hopper", section "why
 *               block quantization beats a per-tensor scale": the Q/K block
 *               scales are restored on each score tile, the V block scale is
 *               applied with the P V product)
 *   o           [B, H, N, d] bf16 (device, written);  lse [B, H, N] fp32
 *   causal, scale as in fa_fwd.
 * Q K^T and P V run on the FP8 tensor cores with fp32 accumulation; the
 * softmax state is fp32 ("FlashAttention-3: async pipelines on Hopper",
 * section "FP8 attention is still not FP8 end to end").  If Q and K were
 * rotated by the same orthogonal matrix (fa_quant_fp8 with signs), the
 * scores are unchanged and O needs no correction; V is never rotated.
 */
fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* v8, void* o, float* lse,
                     int64_t B, int64_t H, int64_t N, int64_t d,
                     int causal, float scale,
                     const float* q_descale, const float* k_descale, const float* v_descale,
                     cudaStream_t stream);

/*
 * fa_fwd_gqa -- fa_fwd for grouped-query / multi-query attention and for
 * different query and key lengths ("FlashAttention-3: async pipelines on
 * Hopper", section "how GQA/MQA changes the kernel's task count": several
 * query heads share one K/V head through the head index, K/V are never
 * copied in HBM).
 *   q    [B, Hq, Nq, d];  k, v [B, Hkv, Nk, d];  o [B, Hq, Nq, d];  lse [B, Hq, Nq]
 *   Hq must be a multiple of Hkv (>= 1); query head h reads K/V head
 *   h / (Hq / Hkv).  Nk >= 1 when Nq >= 1.
 *   causal: key j is visible to query i iff j <= i + (Nk - Nq) (the mask is
 *   aligned at the bottom right; for Nq == Nk this is j <= i).  A query row
 *   that sees no key (causal with Nq > Nk) gets O = 0 and LSE = -inf.
 * fa_fwd(q, k, v, o, lse, B, H, N, d, ...) equals
 * fa_fwd_gqa(q, k, v, o, lse, B, H, H, N, N, d, ...).
 */
fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                     int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                     int causal, float scale, int dtype, cudaStream_t stream);

/*
 * fa_fwd_fp8_gqa -- fa_fwd_fp8 with the head and length conventions of
 * fa_fwd_gqa: q8 [B, Hq, Nq, d], q_descale [B, Hq, ceil(Nq/128)];
 * k8, v8 [B, Hkv, Nk, d], k_descale, v_descale [B, Hkv, ceil(Nk/128)].
 */
fa_status fa_fwd_fp8_gqa(const void* q8, const void* k8, const void* v8, void* o, float* lse,
                         int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                         int causal, float scale,
                         const float* q_descale, const float* k_descale, const float* v_descale,
                         cudaStream_t stream);

/*
 * fa_fwd_host -- fa_fwd_gqa on HOST buffers: the call copies q, k, v to the
 * device, runs the attention kernel and copies o and lse back, in chunks of
 * whole key/value heads (each with its query heads), so that the copies of
 * one chunk overlap the kernel of the previous one and the copies back of
 * the one before (4 chunks, or up to 16 when each still holds a wave of
 * work units; two host->device streams, two compute streams that
 * consecutive chunks alternate between, and a device->host stream, created
 * once per device and joined to `stream` with events; nothing is allocated
 * per call).
 *   q_host, o_host  [B, Hq, Nq, d]   bf16 or fp16 (dtype), HOST memory
 *   k_host, v_host  [B, Hkv, Nk, d]  same dtype, HOST memory
 *   lse_host        [B, Hq, Nq] fp32, HOST memory
 *                   Page-locked memory (cudaHostAlloc / cudaHostRegister)
 *                   lets the copies run asynchronously and overlap; with
 *                   pageable memory the results are the same but the copies
 *                   do not overlap.
 *   workspace       DEVICE pointer, 256-byte aligned, owned by the caller,
 *                   at least fa_fwd_host_workspace_bytes(...) bytes (device
 *                   copies of q, o, k, v, lse); overwritten
 * Asynchronous on `stream` like cudaMemcpyAsync: o_host and lse_host hold
 * the results once `stream` has synchronised; the host buffers must stay
 * valid until then.  Results are bit-identical to fa_fwd_gqa on device
 * copies of the same inputs.  Errors: as fa_fwd_gqa (host pointers need no
 * alignment), plus FA_ERR_INVALID_ARG for a missing, misaligned or too
 * small workspace.
 */
fa_status fa_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* o_host, float* lse_host,
                      int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                      int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream);

/*
 * fa_fwd_host_workspace_bytes -- device workspace fa_fwd_host needs:
 * 2*B*Hq*Nq*d*2 + 2*B*Hkv*Nk*d*2 + B*Hq*Nq*4 bytes, each part rounded up to
 * 256.  Writes *bytes (0 for an empty batch).  Same size checks as
 * fa_fwd_host.
 */
fa_status fa_fwd_host_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                                      size_t* bytes);

/*
 * fa_fwd_splitkv -- the forward pass of fa_fwd_gqa for decode-like shapes
 * (few query rows against a long key/value sequence), where batch x heads x
 * query tiles leave most SMs idle ("FlashAttention-3: async pipelines on
 * Hopper", sections "why GQA/MQA changes the kernel's task count" and
 * "prefill, decode and training gain differently": decode needs split-KV
 * and GQA packing to produce enough parallelism).
 *   Same inputs, outputs, layouts and masking as fa_fwd_gqa (q [B, Hq, Nq, d],
 *   k/v [B, Hkv, Nk, d], bf16 or fp16; causal masks bottom-right aligned).
 *   The Hq / Hkv query heads sharing a key/value head are processed as one
 *   head of (Hq / Hkv) * Nq rows, so every key/value byte is read once per
 *   group; each row's keys are split into num_splits runs processed in
 *   parallel, whose partial results (O normalised per run, fp32, and the
 *   run's LSE) go to `workspace` and are merged by LSE weights in a second
 *   kernel on the same stream.  The merge is exact in real arithmetic.
 *   num_splits   0: chosen for the current device (about eight work units
 *                per SM, at least 8 key tiles of 128 per run); else the
 *                requested count, capped at the number of 128-key tiles
 *                (runs are never empty).
 *   workspace    DEVICE pointer, 256-byte aligned, owned by the caller, at
 *                least the size fa_splitkv_workspace_bytes reports for the
 *                same shape and num_splits on the same device (NULL allowed
 *                when that size is 0: a single run writes O directly);
 *                overwritten; calls sharing it must not overlap on the GPU.
 * Errors: as fa_fwd_gqa, plus FA_ERR_INVALID_ARG for num_splits < 0 or a
 * missing, misaligned or too small workspace.
 */
fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                         int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                         int causal, float scale, int dtype, int num_splits,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_splitkv_workspace_bytes -- bytes of device workspace fa_fwd_splitkv
 * needs for this shape and num_splits on the current device (0 when the
 * keys are not split).  Writes *bytes; same argument checks as
 * fa_fwd_splitkv (no pointers besides bytes).
 */
fa_status fa_splitkv_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                                     int num_splits, size_t* bytes);

/*
 * fa_bwd -- gradients of the loss sum(dout * O) for O = fa_fwd_gqa(q, k, v):
 * dq, dk, dv (the pages list the backward pass dQ, dK, dV among the paths a
 * test must cover and compare its speed with FA2: "FlashAttention-3: async
 * pipelines on Hopper", sections "correctness validation must cover
 * asynchronous boundaries" and "how to read the paper's performance
 * numbers").  With P = softmax(scale q k^T) recomputed from the forward's
 * LSE, dP = dout v^T, D_i = dout_i . o_i and dS = P * (dP - D):
 *   dv = P^T dout,   dk = scale dS^T q,   dq = scale dS k,
 * dk and dv summed over the query heads of each key/value group.
 *   q, dout, o, dq  [B, Hq, Nq, d]   bf16 or fp16 (dtype), device
 *   k, v, dk, dv    [B, Hkv, Nk, d]  same dtype, device
 *   lse             [B, Hq, Nq] fp32, the natural-log LSE fa_fwd_gqa wrote
 *                   for the same q, k, v, causal and scale (-inf: a row that
 *                   sees no key; it gets dq = 0 and adds nothing)
 *   causal          0 / 1, masks aligned at the bottom right as in fa_fwd_gqa
 *   workspace       DEVICE pointer, 256-byte aligned, owned by the caller, at
 *                   least fa_bwd_workspace_bytes(B, Hq, Nq, d) bytes (an fp32
 *                   dQ accumulator and two floats per query row); overwritten;
 *                   calls sharing it must not overlap on the GPU
 * q, k, v, o, lse, dout are read only; dq, dk, dv are fully overwritten.
 * All pointers 16-byte aligned.  Asynchronous on `stream` (four kernels:
 * D and accumulator clear, the fused gradient kernel, dQ conversion), no
 * host synchronisation, no allocation.  dq is accumulated across key tiles
 * with fp32 reduce-adds, so its rounding may differ between runs.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment, sizes, dtype,
 * causal flag, scale or workspace; FA_ERR_UNSUPPORTED for d = 256 (the
 * backward kernel covers d = 64 and 128) or a device other than sm_103;
 * FA_ERR_CUDA for a launch failure; a pipeline timeout is reported by
 * fa_check_device_error.  B*Hq = 0 is a no-op; Nq = 0 writes dk = dv = 0.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dout, void* dq, void* dk, void* dv,
                 int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                 int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream);

/*
 * fa_bwd_workspace_bytes -- bytes of device workspace fa_bwd needs:
 * B*Hq*Nq*d*4 (fp32 dQ accumulator, rounded up to 256) + B*Hq*R*512 with R
 * the 64-row records per head: ceil(Nq/64) for d = 128, 2*ceil(Nq/128) for
 * d = 64 (the kernel's step is 128 query rows there); each record holds
 * its rows' log-sum-exp and D terms.  Writes *bytes.  FA_ERR_INVALID_ARG for negative sizes or a null
 * `bytes`, FA_ERR_UNSUPPORTED for d not in {64, 128, 256}.
 */
fa_status fa_bwd_workspace_bytes(int64_t B, int64_t Hq, int64_t Nq, int64_t d, size_t* bytes);

/*
 * fa_quant_fp8 -- quantise fp32 [B, H, N, d] to E4M3 with one scale per
 * 128-row block (per_tensor = 0) or one scale for the whole tensor
 * (per_tensor = 1, the baseline), optionally after the incoherent-processing
 * rotation x -> x diag(signs) H_d / sqrt(d) ("FlashAttention-3: async
 * pipelines on Hopper", section "how incoherent processing flattens
 * outliers": a random +-1 diagonal combined with a Hadamard matrix, applied
 * to both Q and K, never to V).
 *   x              [B, H, N, d] fp32 (device, read only)
 *   x8             [B, H, N, d] E4M3 codes (device, written)
 *   descale        [B, H, ceil(N/128)] fp32 (device, written): the value to
 *                  multiply a code by; scale = amax/448 of the (rotated) block
 *                  (wmrh.cn article sec. 3.3: 448 is the E4M3 maximum), 1 for
 *                  an all-zero block, times 1/sqrt(d) when rotating
 *   hadamard_signs HOST pointer to d int8 entries of +1/-1, or NULL for no
 *                  rotation; read during the call only
 *   per_tensor     0 or 1
 *   workspace      per_tensor = 1: DEVICE pointer to one float of scratch
 *                  (overwritten; calls sharing it must not overlap on the GPU);
 *                  per_tensor = 0: ignored, may be NULL
 * The rotated value y is fp32 (sign flip, then the Walsh-Hadamard butterfly
 * with strides 1, 2, 4, ...), scale = amax(y) / 448 rounded to fp32, and each
 * code is the E4M3 value nearest to the exact quotient y / scale (ties to
 * even, saturated at 448): a single rounding, decided exactly.
 * Errors: FA_ERR_INVALID_ARG for negative sizes, null or misaligned pointers
 * (x, x8 16-byte aligned), signs other than +-1, per_tensor not 0 / 1 or a
 * missing workspace; FA_ERR_UNSUPPORTED for d not in {64, 128, 256}, more
 * than 2^31 - 1 blocks, or a device other than sm_103; FA_ERR_CUDA for a
 * launch error.  B*H*N = 0 is a no-op.  A bounded wait inside the kernel that
 * runs out (about 2 s) sets the library's error word (fa_check_device_error
 * then returns FA_ERR_TIMEOUT) and marks the blocks it could not finish with
 * a NaN descale (per-tensor mode: an infinite scale) instead of leaving old
 * values.
 */
fa_status fa_quant_fp8(const float* x, void* x8, float* descale,
                       int64_t B, int64_t H, int64_t N, int64_t d,
                       const int8_t* hadamard_signs, int per_tensor, float* workspace,
                       cudaStream_t stream);

/*
 * fa_quant_fp8_qkv -- the FP8 inputs of one attention call in one call: Q and
 * K with block scales after the rotation (when hadamard_signs is not NULL),
 * V with block scales and no rotation (the pages rotate Q and K only, with
 * the same signs, so that Q K^T is unchanged).  Each result is exactly what
 * fa_quant_fp8(x, ..., per_tensor = 0) gives for that tensor.  The three
 * quantisations run on internal streams forked from `stream` and joined back
 * into it, so that each launch's CTAs start on the SMs the others' last CTAs
 * leave free (at B=4 H=16 N=4096 d=128: 95 us against 107 us for three
 * calls in a row); work enqueued on `stream` afterwards runs after all three.
 *   q, k, v        [B, Hq, Nq, d], [B, Hkv, Nk, d], [B, Hkv, Nk, d] fp32 (device, read only)
 *   q8, k8, v8     E4M3 codes of the same shapes (device, written)
 *   q_descale      [B, Hq, ceil(Nq/128)] fp32 (device, written); k_descale and
 *   v_descale      [B, Hkv, ceil(Nk/128)], as fa_quant_fp8's descale
 *   hadamard_signs as fa_quant_fp8 (applied to Q and K)
 * Errors: as fa_quant_fp8 for any of the three tensors, checked before
 * anything is launched; FA_ERR_CUDA if the internal streams cannot be
 * created.  A tensor with no element is skipped.  Calls on one device share
 * the internal streams (serialised by a lock; the launches of consecutive
 * calls still run in order on each of them).
 */
fa_status fa_quant_fp8_qkv(const float* q, const float* k, const float* v, void* q8, void* k8, void* v8,
                           float* q_descale, float* k_descale, float* v_descale,
                           int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                           const int8_t* hadamard_signs, cudaStream_t stream);

/*
 * fa_quant_fp8_rope -- fa_quant_fp8 with a rotary position embedding applied
 * to every row first, in the same pass ("FlashAttention-3: async pipelines on
 * Hopper", sections "why block quantization beats a per-tensor scale" and
 * "how incoherent processing flattens outliers": the block scales and the
 * Hadamard rotation can share one pass with a preceding RoPE).  The pages fix
 * no RoPE convention, so the angles come from the caller and both usual
 * channel pairings are offered:
 *   FA_ROPE_INTERLEAVED  pairs (2i, 2i+1), i < d/2
 *   FA_ROPE_HALF         pairs (i, i + d/2), i < d/2
 * Pair (a, b) of row n becomes (a*c - b*s, a*s + b*c) with c = rope_cos[n][i],
 * s = rope_sin[n][i], in fp32 with each product rounded before the sum; then
 * the optional rotation and the quantisation proceed as in fa_quant_fp8.
 *   rope_cos, rope_sin  [N, d/2] fp32 (device, read only, 16-byte aligned),
 *                       shared by every (b, h): row n is position n of each
 *                       sequence (offset positions by offsetting the tables)
 *   rope_layout         FA_ROPE_INTERLEAVED or FA_ROPE_HALF
 *   other arguments as for fa_quant_fp8.
 * Errors: FA_ERR_INVALID_ARG for a null or misaligned table or an unknown
 * layout, otherwise as fa_quant_fp8.
 */
#define FA_ROPE_INTERLEAVED 1
#define FA_ROPE_HALF 2
fa_status fa_quant_fp8_rope(const float* x, void* x8, float* descale,
                            int64_t B, int64_t H, int64_t N, int64_t d,
                            const float* rope_cos, const float* rope_sin, int rope_layout,
                            const int8_t* hadamard_signs, int per_tensor, float* workspace,
                            cudaStream_t stream);

/*
 * fa_quant_fp8_per_tensor_noalloc -- the per-tensor mode of fa_quant_fp8
 * (per_tensor = 1) for callers that cannot allocate device memory.  The
 * pages have no counterpart; it exists for the library's users.
 *
 * fa_quant_fp8 needs one float of device scratch from the caller in
 * per-tensor mode.  Callers that cannot allocate -- code running under a
 * framework that owns every device buffer, plug-ins whose host forbids
 * cudaMalloc (which may also synchronise the device), runtimes with a fixed
 * memory budget -- use this entry point instead: it takes the same inputs
 * and outputs but keeps its scratch in a device array compiled into the
 * library (about 256 KiB, held by every GPU that loads the library until
 * the process exits).  It calls no allocator.
 *   x, x8, descale, B, H, N, d, hadamard_signs: as for fa_quant_fp8; the
 *   output equals fa_quant_fp8 with per_tensor = 1 bit for bit.
 *   Limit: B * H * ceil(N / 128) <= FA_QUANT_NOALLOC_MAX_BLOCKS, else
 *   FA_ERR_SCRATCH_LIMIT and nothing is launched.
 *   The first call on each device looks up the scratch array's device
 *   address (with that device current); make that first call before any
 *   stream capture.
 *   All calls share the one scratch array and it keeps the last call's
 *   contents (each call writes every entry it reads, so nothing needs
 *   clearing; a block whose input load timed out writes +inf and sets the
 *   library's error word, see fa_check_device_error): calls that overlap on
 *   the GPU -- other streams, other host threads on the same device -- race
 *   and can produce wrong scales.
 *   Errors: as fa_quant_fp8 (per_tensor = 1), plus FA_ERR_SCRATCH_LIMIT.
 */
#define FA_QUANT_NOALLOC_MAX_BLOCKS 65536
fa_status fa_quant_fp8_per_tensor_noalloc(const float* x, void* x8, float* descale,
                                          int64_t B, int64_t H, int64_t N, int64_t d,
                                          const int8_t* hadamard_signs, cudaStream_t stream);

/*
 * ---- sliding window with sinks, and the paged key/value cache ----
 *
 * Visibility.  A query at position p of its sequence sees key j iff
 *     j <= p  and  (j > p - window  or  j < sinks):
 * the last `window` keys up to its own, and the first `sinks` keys of the
 * sequence.  window >= 1 (any value of at least the sequence length makes the
 * mask plain causal), sinks >= 0.  Key tiles without a visible key are
 * neither read nor multiplied.  A query that sees no key gets O = 0 and
 * LSE = -inf.
 */

/*
 * fa_fwd_window -- fa_fwd_gqa under a sliding window with sinks.
 *   q [B, Hq, Nq, d], k, v [B, Hkv, Nk, d], o [B, Hq, Nq, d], lse [B, Hq, Nq]
 *   as fa_fwd_gqa (contiguous, bf16 or fp16, Hq a multiple of Hkv).  Query i
 *   sits at position p = i + Nk - Nq (the sequence ends with the last query).
 * Numerics, ownership and non-finite inputs as fa_fwd: a NaN or infinity in
 * element (j, c) of V may also reach column c of rows that do not see key j
 * but share its 128-key tile with rows that do.
 * Errors: as fa_fwd_gqa, FA_ERR_INVALID_ARG also for window < 1 or sinks < 0,
 * FA_ERR_UNSUPPORTED also for Nq or Nk above 2^30.
 */
fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse,
                        int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                        int64_t window, int64_t sinks, float scale, int dtype, cudaStream_t stream);

/*
 * fa_bwd_window -- gradients of sum(dout * O) for O = fa_fwd_window(q, k, v)
 * with the same window, sinks and scale: fa_bwd's arguments, formulas and
 * layouts (d 64 or 128) with P restricted to the visible keys.  Rows that see
 * at most 32 keys take D = sum_j P_j dP_j over them in fp32 in place of
 * dO . O, whose rounded O few keys do not average out (with one key dS must
 * vanish).  But for these rows a window of at least Nk without sinks runs as
 * fa_bwd's causal kernel, with the same bits of dK and dV (so with its key
 * tiles whole: with few key/value heads a shorter window, whose tiles are shared
 * out over the GPU, can take less time).
 *   lse        [B, Hq, Nq] fp32 as fa_fwd_window wrote it
 *   workspace  at least fa_bwd_window_workspace_bytes(...) bytes, 256-byte
 *              aligned; overwritten; calls sharing it must not overlap
 * dk and dv are the same from run to run; dq, as in fa_bwd, is accumulated
 * across key tiles with fp32 reduce-adds whose order may change its rounding.
 * Errors: as fa_bwd, FA_ERR_INVALID_ARG also for window < 1 or sinks < 0,
 * FA_ERR_UNSUPPORTED also for Nq or Nk above 2^30.
 */
fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                        const void* dout, void* dq, void* dk, void* dv,
                        int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                        int64_t window, int64_t sinks, float scale, int dtype,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_bwd_window_workspace_bytes -- bytes of device workspace fa_bwd_window
 * needs: fa_bwd's, and fp32 dK and dV parts of the key tiles whose queries are
 * shared out (at most 256 MiB at d = 128).  Same checks as fa_bwd_window.  The
 * size depends on the arguments alone, not on a device (none is needed to ask).
 */
fa_status fa_bwd_window_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t Nk, int64_t d,
                                        int64_t window, int64_t sinks, size_t* bytes);

/*
 * A paged key/value cache: num_pages pages of page_size tokens for each of
 * `heads` key/value heads.  Element (page, head, token, c) of k (and of v)
 * lies at k + page * page_stride + head * head_stride + token * token_stride
 * + c, strides in elements: [pages, heads, page_size, d] and [pages,
 * page_size, heads, d] are both such layouts, as are k and v interleaved in
 * one allocation.
 *   k, v       DEVICE pointers, 16-byte aligned, owned by the caller
 *   page_size  a power of two, 16 to 1024;  d 64, 128 or 256
 *   strides    multiples of 8 and at least d (a stride whose size is 1 is not
 *              looked at)
 */
typedef struct {
    void* k;
    void* v;
    int64_t num_pages, page_size, heads, d;
    int64_t page_stride, head_stride, token_stride;
    int dtype;
} fa_kv_cache;

/*
 * A ragged batch over a cache, as fa_fwd_paged and fa_cache_append take it.
 * Sequence b brings the new tokens cu_q[b] .. cu_q[b + 1] - 1 of the packed
 * token arrays and has seq_k[b] keys, those of its new tokens included and
 * last: new token i of n sits at position seq_k[b] - n + i.  Key j lies at
 * row j % page_size of page block_table[b * table_stride + j / page_size].
 *   block_table  [B, max_pages] int32 (device), rows table_stride apart; only
 *                the entries of pages with a visible key (fa_fwd_paged) or a
 *                new token (fa_cache_append) are read
 *   cu_q         [B + 1] int32 (device), not decreasing, cu_q[B] <= T.  Rows
 *                of the packed arrays outside every sequence are neither
 *                written nor used
 *   seq_k        [B] int32 (device)
 * All three are device data, read by the kernels when they run, so a captured
 * graph follows their contents.  The host cannot refuse what they hold; the
 * kernels do: a token range is cut to the T rows there are (by both calls
 * alike), a number of keys to the table (fa_fwd_paged), a page number out of
 * range reads as zeros (fa_fwd_paged) or drops the token (fa_cache_append),
 * nothing out of bounds is touched, and fa_check_device_error then returns
 * FA_ERR_INDEX.  (Ranges that go back overlap others: which of them a shared
 * row follows is not defined, and fa_fwd_paged writes nothing at all where
 * their work passes the most that T, B and max_pages allow without.)
 */

/*
 * fa_fwd_paged -- attention of the new tokens of a ragged batch (one token or
 * a chunk per sequence, mixed freely) over a paged cache that already holds
 * their keys and values, under a sliding window with sinks.
 *   q          [T, Hq, d] of the cache's dtype (device), tokens q_stride
 *              elements apart (a multiple of 8, at least Hq * d), heads d apart
 *   o          [T, Hq, d] contiguous (device, written);  lse [T, Hq] fp32
 *   Hq         a multiple of cache->heads, at most 128 query heads to each
 *   max_q      the most new tokens any sequence brings, 0 if not known.  A
 *              hint: it sizes the query tiles; results are right for any value
 *              (of finite inputs: see below)
 *   window, sinks, scale  as fa_fwd_window (pages that left every query's
 *              window, sinks apart, may be freed: they are not read)
 *   workspace  DEVICE pointer, 256-byte aligned, owned by the caller, at least
 *              fa_paged_workspace_bytes(d) bytes; overwritten; calls sharing
 *              it must not overlap on the GPU (two captured graphs included)
 * Rows of the cache behind a sequence's end, and pages it does not see, may
 * hold anything (NaN included).  A NaN or infinity in a value row that a new
 * token of the sequence sees may also reach its column of O, as NaN, in those
 * of its tokens that do not see it, and an infinity as NaN in those that do:
 * which of them depends on the rest of the batch and on max_q, as these pick
 * the form of the kernel.  Two kernels on `stream`, no allocation.  The
 * result of one sequence may differ in its last bits with the rest of the
 * batch (the work is cut evenly over the GPU and the pieces are joined), but
 * is the same from run to run.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment, sizes, strides,
 * window, sinks, scale or workspace; FA_ERR_UNSUPPORTED for d, page_size or
 * head counts outside the above, more than 2^24 sequences, lengths above
 * 2^30, work that could pass 2^30 key tiles by the host's sizes (T, B,
 * max_pages, window), or a device other than sm_103.  B * T * Hq = 0 is a no-op.
 */
fa_status fa_fwd_paged(const void* q, const fa_kv_cache* cache, void* o, float* lse,
                       const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                       const int32_t* cu_q, const int32_t* seq_k,
                       int64_t B, int64_t T, int64_t Hq, int64_t q_stride, int64_t max_q,
                       int64_t window, int64_t sinks, float scale,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * fa_paged_workspace_bytes -- bytes of device workspace fa_fwd_paged needs on
 * the current device for head dimension d, whatever the batch: two partial
 * results of 256 query rows (d = 256: 128) per SM, about 40 MB at d = 128.
 */
fa_status fa_paged_workspace_bytes(int64_t d, size_t* bytes);

/*
 * fa_cache_append -- writes the new tokens' keys and values of a ragged batch
 * into their pages, after a rotary position embedding of the keys, and
 * rotates the new tokens' queries by the same angles: the step before
 * fa_fwd_paged.
 *   k, v       [T, heads, d] of the cache's dtype (device, read only), tokens
 *              k_stride / v_stride elements apart (multiples of 8, at least
 *              heads * d): slices of one fused projection are such arrays
 *   q          [T, Hq, d] likewise (q_stride), or NULL with Hq = 0
 *   q_out      [T, Hq, d] contiguous (device, written).  q_out = q is allowed
 *              when q is contiguous; any other overlap of an input with an
 *              output is not
 *   rope_cos, rope_sin  [rope_len, d/2] fp32 (device, read only, 16-byte
 *              aligned); row p holds the angles of position p
 *   rope_layout  0: no rotation (keys and queries are copied), or
 *              FA_ROPE_INTERLEAVED / FA_ROPE_HALF as in fa_quant_fp8_rope:
 *              pair (a, b) becomes (a*c - b*s, a*s + b*c), each product
 *              rounded to fp32 before the sum, the sum once to the dtype
 * A token whose position is negative, behind its table row or the angle
 * tables, or whose page is out of range, is dropped (no key, value or query
 * of it is written) and reported by fa_check_device_error as FA_ERR_INDEX.
 * If two tokens share a cache row, which of them it holds is not defined.
 * Errors: as fa_fwd_paged, FA_ERR_INVALID_ARG also for a missing or
 * misaligned table or an unknown layout.  B * T = 0 is a no-op.
 */
fa_status fa_cache_append(const fa_kv_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride,
                          const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                          const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T, int64_t Hq,
                          const float* rope_cos, const float* rope_sin, int64_t rope_len, int rope_layout,
                          cudaStream_t stream);

/*
 * fa_cache_append_at -- fa_cache_append with the rotation's positions given, and
 * of part of the head:
 *   positions  [T] int32 (device): token t is turned by the angles of
 *              positions[t]; where its key and value are written follows from cu_q
 *              and seq_k all the same.  (The nodes of a tree of drafted tokens
 *              lie one behind the other in the cache, but at positions by their
 *              depth: see fa_tree_plan.)  NULL: by where it is written
 *   rope_dim   the rotated columns, a multiple of 16 up to d; the tables are
 *              [rope_len, rope_dim/2].  The columns behind them are copied
 * fa_cache_append is this call with positions = NULL and rope_dim = d.  A token
 * whose position lies outside the tables is dropped and reported.
 * Errors: as fa_cache_append, FA_ERR_UNSUPPORTED also for another rope_dim
 * (which is not looked at with rope_layout 0, nor are the positions).
 */
fa_status fa_cache_append_at(const fa_kv_cache* cache, const void* q, const void* k, const void* v, void* q_out,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                             const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T, int64_t Hq,
                             const float* rope_cos, const float* rope_sin, int64_t rope_len, int64_t rope_dim,
                             int rope_layout, const int32_t* positions, cudaStream_t stream);

/*
 * ---- trees of drafted tokens ----
 *
 * A sequence of the ragged batch brings the nodes of a tree (or several) in
 * place of consecutive tokens: continuations that are tried at once, of which one
 * path will be kept.  Node i's parent is an earlier node of its sequence, or none:
 * then it follows the cached tokens.  Nodes lie in the cache one behind the other,
 * node i at position seq_k[b] - n + i as any new token, but sit in their sequence
 * at the position that their depth gives them: seq_k[b] - n + (nodes above it).
 * The steps of one round: fa_tree_plan (under a window fa_tree_plan_window, with the
 * layers' own) once; in each layer fa_cache_append_at with
 * its positions, and fa_fwd_tree; then fa_cache_compact keeps the accepted path.
 */

/*
 * fa_tree_plan -- mask rows and positions of the nodes.
 *   parents    [T] int32 (device): the parent's number within its sequence, below
 *              the node's own, or -1
 *   cu_q, seq_k, B, T  the batch, as in fa_fwd_paged
 *   mask       [T, words] uint32 (device, written): bit k of word w of a node's
 *              row says that node 32 w + k of its sequence is the node itself or
 *              above it
 *   words      1 to 32.  A sequence of more than 32 * words tokens is a plain chunk
 *              (of a prompt): the parent of its token i has to be i - 1, and the rows
 *              get what words bits there are
 *   positions  [T] int32 (device, written)
 * Rows outside every sequence are not written.  A parent that is out of range
 * counts as -1, and it or a chunk that is not one is reported by
 * fa_check_device_error as FA_ERR_INDEX.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment or sizes;
 * FA_ERR_UNSUPPORTED for words above 32, B above 2^24, T above 2^30, or a device
 * other than sm_103.  B * T = 0 is a no-op.
 */
fa_status fa_tree_plan(const int32_t* parents, const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T,
                       uint32_t* mask, int64_t words, int32_t* positions, cudaStream_t stream);

/*
 * fa_tree_plan_window -- fa_tree_plan under a sliding window with sinks: a node
 * at position p keeps the bits of those nodes above it that sit at a position j >
 * p - window or j < sinks, as it would see them if its path were decoded token by
 * token with fa_fwd_paged.  (The rows of a chunk are fa_tree_plan's: fa_fwd_tree
 * does not look at them.)
 * A round under a window takes its plan from this call, with the window and sinks
 * that fa_fwd_tree gets.  fa_tree_plan is this call without a window.
 * Errors: as fa_tree_plan, FA_ERR_INVALID_ARG also for window < 1 or sinks < 0.
 */
fa_status fa_tree_plan_window(const int32_t* parents, const int32_t* cu_q, const int32_t* seq_k, int64_t B, int64_t T,
                              uint32_t* mask, int64_t words, int32_t* positions, int64_t window, int64_t sinks,
                              cudaStream_t stream);

/*
 * fa_fwd_tree -- fa_fwd_paged where the new tokens of a sequence are a tree's
 * nodes.  Node i, at position p, sees
 *   the cached keys j < seq_k[b] - n with j > p - window or j < sinks, and
 *   new token k <= i iff bit k of its mask row is set (the window does not apply
 *   to these: fa_tree_plan_window leaves out the bits of nodes that have left it; a
 *   row without any bit and any cached key gets O = 0 and LSE = -inf).
 *   mask       [T, words] uint32 (device), as fa_tree_plan and fa_tree_plan_window
 *              write it, or any other
 *              (bits behind a token's own are not looked at)
 *   words      1 to 32.  Sequences of more than 32 * words new tokens attend as in
 *              fa_fwd_paged, whatever their mask rows hold
 *   positions  [T] int32 (device), as fa_tree_plan writes them: between seq_k[b] -
 *              n and where the token lies.  NULL: where the tokens lie.  They are
 *              looked at under a window shorter than the sequence alone; others are
 *              then cut to the above and reported by fa_check_device_error as
 *              FA_ERR_INDEX
 * Everything else as in fa_fwd_paged, its workspace included.  Pages that hold
 * no key from position seq_k[b] - n - window + 1 on, nor a sink, are not read.
 * (Any entry of block_table's [B, max_pages] may be, to see which rows share pages;
 * it then changes what stays in the GPU's cache, and no result.)
 * For what a NaN or an infinity in a value row reaches, the new tokens' rows and
 * the cached ones from that position on count as seen.
 */
fa_status fa_fwd_tree(const void* q, const fa_kv_cache* cache, void* o, float* lse,
                      const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                      const int32_t* cu_q, const int32_t* seq_k, const uint32_t* mask, int64_t words,
                      const int32_t* positions, int64_t B, int64_t T, int64_t Hq, int64_t q_stride, int64_t max_q,
                      int64_t window, int64_t sinks, float scale, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream);

/*
 * ---- rotary positions ----
 *
 * Pair (a, b) of a row at position p becomes (a*c - b*s, a*s + b*c) with c =
 * rope_cos[p][i], s = rope_sin[p][i], each product rounded to fp32 before the
 * sum, the sum once to the element type.  The first rope_dim columns of a row
 * are rotated -- pairs (2i, 2i+1) (FA_ROPE_INTERLEAVED) or (i, i + rope_dim/2)
 * (FA_ROPE_HALF), i < rope_dim/2 -- and the columns behind them are copied.
 */

/*
 * How a table's frequencies are scaled for contexts longer than a model was
 * trained on.  With f_i = theta^(-2i/rope_dim) the unscaled angle per position
 * of pair i, s = factor, and keep clamped to 0..1:
 *   FA_ROPE_SCALE_NONE    f_i
 *   FA_ROPE_SCALE_LINEAR  f_i / s
 *   FA_ROPE_SCALE_BASE    f_i of theta * s^(rope_dim / (rope_dim - 2))
 *   FA_ROPE_SCALE_TURNS   (1 - keep) f_i / s + keep f_i, with keep = (w_i - low)
 *                         / (high - low) of the turns w_i = original f_i / 2 pi
 *                         that the pair makes over the original length
 *   FA_ROPE_SCALE_INDEX   the same with keep = 1 - (i - a) / max(b - a, 0.001)
 *                         between the pairs a = max(0, floor(i(high))) and b =
 *                         min(rope_dim - 1, ceil(i(low))), i(w) = rope_dim ln(original
 *                         / (2 pi w)) / (2 ln theta) the (fractional) pair of w turns
 * amplitude multiplies cosines and sines (with every kind; usually 1).
 */
enum {
    FA_ROPE_SCALE_NONE = 0,
    FA_ROPE_SCALE_LINEAR = 1,
    FA_ROPE_SCALE_BASE = 2,
    FA_ROPE_SCALE_TURNS = 3,
    FA_ROPE_SCALE_INDEX = 4
};
typedef struct {
    int kind;
    double factor;      /* at least 1 */
    double original;    /* TURNS, INDEX: the original length, at least 1 */
    double low, high;   /* TURNS, INDEX: 0 <= low < high (INDEX: 0 < low) */
    double amplitude;   /* within fp32's range */
} fa_rope_scaling;

/*
 * fa_rope_table -- cosines and sines of the positions start .. start + n - 1,
 * the tables that fa_rope, fa_cache_append, fa_cache_append_at and
 * fa_quant_fp8_rope take.
 *   rope_cos, rope_sin  [n, rope_dim/2] fp32 (device, written, 16-byte aligned)
 *   rope_dim            a multiple of 16, at most 256
 *   theta               above 1
 *   scaling             as above (HOST pointer, read during the call), or NULL
 * A frequency is kept to 2^-65 of a turn, and its product with the position is
 * reduced exactly: a value at position p is within two units of its own last fp32
 * place, and amplitude * (p + 128) * 2^-62 beside them, of the exact one.  (The
 * latter is less than a unit for every value above 2^-18 up to position 2^20, and
 * above 2^-7 at any.)
 * Errors: FA_ERR_INVALID_ARG for negative sizes, bad pointers, theta or scaling;
 * FA_ERR_UNSUPPORTED for another rope_dim, n or start above 2^30, or a device
 * other than sm_103.  n = 0 is a no-op.
 */
fa_status fa_rope_table(float* rope_cos, float* rope_sin, int64_t n, int64_t rope_dim, double theta, int64_t start,
                        const fa_rope_scaling* scaling, cudaStream_t stream);

/*
 * One array that fa_rope turns: element (b, h, n, c) lies at x + b * x_batch +
 * h * x_head + n * x_token + c, of the result at y + b * y_batch + ... (strides
 * in elements, multiples of 8, of y at least d; one whose size is 1 is not
 * looked at).  [B, heads, N, d], [N, heads, d] with B = 1, and slices of a fused
 * projection are such arrays.  y = x with the same strides turns in place (and
 * leaves the columns behind rope_dim alone); no other overlap is allowed.
 */
typedef struct {
    const void* x;      /* device, 16-byte aligned */
    void* y;            /* device, 16-byte aligned */
    int64_t heads;
    int64_t x_batch, x_head, x_token;
    int64_t y_batch, y_head, y_token;
} fa_rope_array;

/*
 * fa_rope -- rotates one or two arrays (a layer's queries and keys) by their
 * positions, or back by them.
 *   arrays, count  HOST array of 1 or 2 (read during the call); both have B
 *                  batch entries of N tokens, and their own numbers of heads
 *   positions      int32 (device): token n of entry b is at positions[b *
 *                  pos_stride + n] (pos_stride 0: the same in every entry); or
 *                  NULL: at offset + n
 *   rope_cos, rope_sin  [rope_len, rope_dim/2] fp32 (device, 16-byte aligned)
 *   rope_dim       a multiple of 16, at most d (64, 128 or 256)
 *   inverse        1: sines negated, the transposed matrix.  It undoes the
 *                  rotation, and it is its gradient: of sum(dy * rope(x)) by x
 *   dtype          FA_DTYPE_BF16 or FA_DTYPE_FP16
 * A row whose position from device memory lies outside the tables is not
 * written, and reported by fa_check_device_error as FA_ERR_INDEX.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment, sizes, strides,
 * layout, flags, or offset + N above rope_len without positions;
 * FA_ERR_UNSUPPORTED for d, rope_dim or sizes outside the above (N, B, rope_len
 * and offset at most 2^30, heads 2^20) or a device other than sm_103.
 * B * N * heads = 0 is a no-op.
 */
fa_status fa_rope(const fa_rope_array* arrays, int64_t count, int64_t B, int64_t N, int64_t d, const int32_t* positions,
                  int64_t pos_stride, int64_t offset, const float* rope_cos, const float* rope_sin, int64_t rope_len,
                  int64_t rope_dim, int rope_layout, int inverse, int dtype, cudaStream_t stream);

/*
 * ---- the pages of a cache ----
 *
 * A pool of pages is its reference counts: refs[p], int32 (device, 16-byte
 * aligned), is how many rows of the block table hold page p, 0 for a free page.
 * Row r of the table holds the pages of its first seq_k[r] tokens, one entry for
 * each page begun; entries behind them are -1 or not looked at.  The calls below
 * keep the three in step, on the device and in stream order, so a captured graph
 * can hold them; a free page is always handed out lowest number first, so that
 * results do not depend on timing.  Calls that change one pool must not overlap
 * on the GPU.
 *
 * fa_pages_fork, fa_cache_copy and fa_cache_compact move keys and values in all
 * layers of a cache at once: `cache` describes the first, and layer l lies l *
 * layer_stride elements behind it (a multiple of 8; not looked at for one layer),
 * at most 32767.
 */

/*
 * fa_pages_resize -- rows of a block table shrink or grow.  Rows with want[r] <
 * seq_k[r] give back the pages that want[r] tokens do not need (want 0: all);
 * then rows with want[r] > seq_k[r] get pages, the lowest-numbered free ones, in
 * the order of rows.  Entries given back become -1.
 *   refs         [num_pages] int32 (device, read and written)
 *   page_size    a power of two, 16 to 1024
 *   block_table  [B, max_pages] int32 (device, read and written), rows
 *                table_stride apart
 *   seq_k        [B] int32 (device, read and written): afterwards want[r], or if
 *                the pages ran out as many tokens as the row has pages for
 *                (its entries that got none are -1)
 *   want         [B] int32 (device, read only)
 * Pages are not written: new ones hold what they held.  A page that several rows
 * share is free once the last of them has given it back.  A row that is cut to a
 * length within a page it shares must not be written to from there on, as the
 * others hold those tokens (a fork of it may: fa_pages_fork copies such a page).
 * Lengths below 0 or above max_pages * page_size are cut, page numbers outside
 * the pool and pages that nobody held are passed over, and both are reported by
 * fa_check_device_error as FA_ERR_INDEX.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment or sizes;
 * FA_ERR_UNSUPPORTED for page_size outside the above, B above 49152, max_pages
 * above 2^30 or a device other than sm_103.  B = 0 is a no-op.
 */
fa_status fa_pages_resize(int32_t* refs, int64_t num_pages, int64_t page_size, int32_t* block_table, int64_t table_stride,
                          int64_t max_pages, int32_t* seq_k, const int32_t* want, int64_t B, cudaStream_t stream);

/*
 * fa_pages_fork -- row dst[i] becomes a second copy of the sequence in row
 * src[i]: it shares the source's full pages, and gets the lowest-numbered free
 * page for a last page that is partly filled, whose rows are copied.  (So pages
 * that are shared are full, and both sequences go on without writing into them.)
 *   refs         [cache->num_pages] int32 (device, read and written)
 *   block_table  [rows, max_pages] int32 (device, read and written)
 *   seq_k        [rows] int32 (device, read and written)
 *   src, dst     [n] int32 (device, read only).  A source may be given several
 *                times.  A row dst[i] holds no tokens (seq_k 0: give its pages back
 *                first), and is neither given twice nor a source
 *   fresh        [n] int32 (device, written): the page that the fork got, -1 if
 *                it needed none, -2 if it was refused, -3 if no page was left
 * Forks take their pages in the order of i.  One that breaks the above, or whose
 * source has a bad length or last page, is refused as a whole and reported by
 * fa_check_device_error as FA_ERR_INDEX; one without a page is not done, and not
 * reported.
 * Errors: FA_ERR_INVALID_ARG for bad pointers, alignment, sizes or strides;
 * FA_ERR_UNSUPPORTED for a cache outside fa_kv_cache's limits, rows above 2^18, n
 * above 16384, a page of one layer's keys above 32 GiB, or a device other than
 * sm_103.  n = 0 is a no-op.
 */
fa_status fa_pages_fork(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, int32_t* refs, int32_t* block_table,
                        int64_t table_stride, int64_t max_pages, int32_t* seq_k, int64_t rows, const int32_t* src,
                        const int32_t* dst, int32_t* fresh, int64_t n, cudaStream_t stream);

/*
 * fa_cache_copy -- copies page src[i] to page dst[i], keys and values of all
 * layers, i < n (both [n] int32, device).  No page may be given twice in dst, or
 * in both (their contents are then not defined).  A pair with a page number
 * outside the cache is passed over and reported by fa_check_device_error as
 * FA_ERR_INDEX.  Errors: as fa_pages_fork.  n * layers = 0 is a no-op.
 */
fa_status fa_cache_copy(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, const int32_t* src, const int32_t* dst,
                        int64_t n, cudaStream_t stream);

/*
 * fa_cache_compact -- moves the tokens of each sequence that are kept together:
 * for i < keep_n[b], the keys and values at position keep[b][i] of sequence b go
 * to position first[b] + i, as if all were read before one is written.  With
 * first = the cached tokens before a step it keeps the accepted ones of the
 * step's drafted tokens; with first = 0 it evicts tokens from a cache.
 *   block_table  [B, max_pages] int32 (device, read only)
 *   first        [B] int32 (device, read only)
 *   keep         [B, max_keep] int32 (device, read only), rows keep_stride apart;
 *                keep[b][i] >= first[b] + i, as in any ascending list of positions
 *                from first[b] on
 *   keep_n       [B] int32 (device, read only)
 *   seq_k_out    [B] int32 (device, written): first[b] + keep_n[b].  Not one of
 *                the inputs
 * The table is not changed: fa_pages_resize gives back the pages behind the new
 * lengths.  Pages that are written to must not be shared with another sequence.
 * Counts are cut to max_keep, and positions that are out of range, lead to no
 * page or break the above are passed over; both are reported by
 * fa_check_device_error as FA_ERR_INDEX.
 * Errors: as fa_pages_fork, FA_ERR_UNSUPPORTED for B above 2^24 or B * heads
 * above 2^29.  B = 0 is a no-op.
 */
fa_status fa_cache_compact(const fa_kv_cache* cache, int64_t layers, int64_t layer_stride, const int32_t* block_table,
                           int64_t table_stride, int64_t max_pages, const int32_t* first, const int32_t* keep,
                           int64_t keep_stride, int64_t max_keep, const int32_t* keep_n, int32_t* seq_k_out, int64_t B,
                           cudaStream_t stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* fa_status_string(fa_status status);

/*
 * fa_check_device_error -- synchronises `stream`, then reports and clears the
 * library's device error word on the current device: FA_ERR_TIMEOUT if a
 * kernel gave up on a pipeline wait since that was last reported, else
 * FA_ERR_INDEX if a kernel met an index out of range in device memory
 * (fa_fwd_paged and the calls on trees, positions and pages) since that was,
 * FA_ERR_CUDA if the
 * synchronisation itself failed, else FA_OK.  One error is reported per call:
 * after both kinds the next call reports the second.
 */
fa_status fa_check_device_error(cudaStream_t stream);

/*
 * fa_debug_inject -- TEST HOOK for the failure path; not for production use.
 * flags bit 0: the next fa_fwd / fa_fwd_fp8 / fa_fwd_window / fa_fwd_paged /
 * fa_fwd_tree launch has its first CTA leave one K/V ring slot unfilled (the next fa_bwd
 * or fa_bwd_window launch: one Q/dO stage of its first CTA's second step), so the bounded waits on it run out (about 2 s):
 * the kernel then stops every role, frees its tensor memory and ends, and
 * fa_check_device_error() returns FA_ERR_TIMEOUT.  The output of that
 * launch is incomplete.  The flag is consumed by the next fa_fwd*,
 * fa_fwd_fp8* or fa_bwd* call.
 * flags bit 1: the same for the next quantiser call (fa_quant_fp8,
 * fa_quant_fp8_rope or fa_quant_fp8_per_tensor_noalloc): the first CTA of its
 * first launch leaves one input slot unfilled; the blocks it cannot finish
 * get a NaN descale (per-tensor: an infinite maximum) and the error word is
 * set.
 * flags = 0 clears pending injections.  Values outside 0..3:
 * FA_ERR_INVALID_ARG.
 */
fa_status fa_debug_inject(int flags);

/*
 * fa_debug_exp2 -- TEST HOOK: evaluates, element by element, y[i] = 2^x[i]
 * the ways the forward kernels can compute the exponentials of P: method 0
 * with the special-function unit's ex2 as the shipped kernels do
 * (approximate, subnormal results flushed to zero), method 3 or 4 with the
 * FMA-pipe polynomial of that degree that the ablation variant 64 of
 * fa_ablate.h uses for a share of P (range
 * reduction x = n + f, |f| <= 1/2, minimax polynomial for 2^f; relative
 * error at most 7.5e-5 (degree 3) or 2.6e-6 (degree 4) for -125 <= x <= 127;
 * x below -126 gives a result of at most 2^-125.5; NaN gives NaN).  x, y:
 * device arrays of n fp32 values (y may equal x).  Asynchronous on `stream`.
 * FA_ERR_INVALID_ARG for n < 0, a null pointer with n > 0 or another method.
 */
fa_status fa_debug_exp2(const float* x, float* y, int64_t n, int method, cudaStream_t stream);

/* Library version, major * 10000 + minor * 100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */
