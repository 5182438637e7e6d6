/*
 * dc1d.h -- C ABI of libdc1d, the MI355X (gfx950) forward pass of 1D
 * deformable convolution with an optional modulation mask.
 *
 * The operation (restated from the pages; each part cited by page and
 * section):
 *
 *   out[b, co, l] = bias[co]
 *       + sum_{ci in co's group} sum_{k < K} weight[co, ci_local, k] * S[b, ci, k, l]
 *
 *   S[b, ci, k, l] = m * ( (1 - f) * x~(i0) + f * x~(i0 + 1) )
 *       i0 = l*stride - padding + k*dilation + floor(o),   f = o - floor(o)
 *       o  = offsets[b, g, l, k],   g = ci / (C_in / offset_groups)
 *       m  = mask[b, g, l, k], or 1 when no mask is given
 *       x~(i) = x[b, ci, i] for 0 <= i < L_in, else 0
 *
 *   - The sum and its grid position l*stride - padding + k*dilation are the
 *     conv1d cross-correlation (conv1d operator page, section Description);
 *     the offset moves each tap's sampling point (dilated/deformable
 *     convolution article, section Deformable Convolution, the y(p0)
 *     formula, and its Step 2 / Step 3 workflow: sample, then weigh).
 *   - Sampling between integer positions is linear (dc1d page, section Demo
 *     notebook: integer offsets shift exactly, fractional ones interpolate
 *     linearly); samples off either end read zero (torchvision issue on the
 *     deform_conv2d offset layout, its printed demo output).
 *   - Offsets are [B, offset_groups, L_out, K] with offset_groups dividing
 *     C_in (dc1d page, section Usage / DeformConv1d); the mask has the same
 *     shape and is applied as given, no sigmoid inside (dc1d page, section
 *     Modulation (DCNv2)).
 *   - groups split channels into contiguous independent blocks, weight is
 *     [C_out, C_in/groups, K], bias [C_out] (conv1d operator page, sections
 *     Arguments and Axis convention).
 *   - L_out = floor((L_in + 2*padding - dilation*(K-1) - 1)/stride + 1)
 *     (conv1d operator page, section Shape).
 *
 * Layout: every tensor is dense, contiguous, row-major, channels-first
 * ([B, C, L], conv1d operator page, section Axis convention).  All tensors of
 * one call share one dtype; the output has the input's dtype (conv1d page:
 * the computation stays in the input dtype).  Arithmetic is fp32 inside the
 * kernels (bf16 values are widened exactly; a bf16 output is rounded once,
 * to nearest even).
 *
 * Ownership: the caller owns every buffer (device memory for tensors and the
 * workspace).  The library allocates nothing, keeps no pointer after a call
 * returns, and has no mutable global state other than a per-device
 * capability cache filled once.  Work is enqueued on the given HIP stream and
 * the call returns without synchronising; buffers must stay alive until that
 * stream's work is done (of a call captured into a graph: as long as the graph
 * is replayed).  Calls are re-entrant; calls that share a workspace
 * must be ordered on one stream.
 *
 * Logging: with the environment variable DC1D_LOG set to a non-zero value
 * (read once, at the first call that launches work), each such call writes
 * one line to stderr naming the entry, the shapes, the dtype, the kernel
 * chosen, its grid and split count and the workspace bytes.
 *
 * Errors: every entry returns a dc1d_status.  Errors detected on the host
 * return before any device work and write nothing.  Faults inside a kernel
 * surface at the caller's next synchronisation.  No C++ exception crosses
 * this boundary.
 */
#ifndef DC1D_H
#define DC1D_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage dtypes. */
typedef enum dc1d_dtype {
    DC1D_F32 = 0,  /* IEEE binary32 */
    DC1D_BF16 = 1, /* bfloat16 (upper half of a binary32) */
    DC1D_I32 = 2   /* 32-bit integers: positions and lengths of the sequence operators only */
} dc1d_dtype;

typedef enum dc1d_status {
    DC1D_OK = 0,
    DC1D_ERR_NULL_PTR = 1,  /* a required descriptor or data pointer is NULL */
    DC1D_ERR_BAD_ARG = 2,   /* stride/padding/dilation/groups/offset_groups/K out of range,
                               groups or offset_groups not dividing the channels,
                               offset_groups disagreeing with offsets->shape[1] */
    DC1D_ERR_BAD_SHAPE = 3, /* a tensor's rank or shape disagrees, L_out <= 0, or a size
                               beyond the supported limits (see dc1d_forward) */
    DC1D_ERR_BAD_DTYPE = 4, /* unsupported dtype, or dtypes mixed within a call */
    DC1D_ERR_ALIAS = 5,     /* out overlaps an input */
    DC1D_ERR_WORKSPACE = 6, /* workspace NULL, smaller than dc1d_workspace_bytes(), or not
                               256-byte aligned */
    DC1D_ERR_DEVICE = 7,    /* no current HIP device, or it is not a gfx950 */
    DC1D_ERR_LAUNCH = 8     /* the kernel launch reported an error */
} dc1d_status;

/* A dense, contiguous tensor in device memory.  shape[i] for i >= ndim is
 * ignored.  data may be NULL only when the tensor has no elements. */
typedef struct dc1d_tensor {
    void *data;
    int32_t dtype; /* a dc1d_dtype */
    int32_t ndim;
    int64_t shape[4];
} dc1d_tensor;

/*
 * conv1d output length (conv1d operator page, section Shape):
 *   floor((L_in + 2*padding - dilation*(K-1) - 1)/stride + 1).
 * Returns -1 when an argument is out of range (L_in < 0, K < 1, stride < 1,
 * padding < 0, dilation < 1) or the result is not positive.  Host only.
 */
int64_t dc1d_output_length(int64_t L_in, int64_t K, int64_t stride, int64_t padding,
                           int64_t dilation);

/*
 * Bytes of device workspace that dc1d_forward needs for these arguments on
 * the current device (0 when the chosen kernels need none).  Only the
 * descriptors' dtype, ndim and shape are read; data pointers may be NULL.
 * The same validation as dc1d_forward applies (except pointers and
 * aliasing).  What the workspace holds is described at dc1d_forward.
 */
int dc1d_workspace_bytes(const dc1d_tensor *x, const dc1d_tensor *offsets,
                         const dc1d_tensor *mask_or_null, const dc1d_tensor *weight,
                         const dc1d_tensor *bias_or_null, int64_t stride, int64_t padding,
                         int64_t dilation, int64_t groups, int64_t offset_groups,
                         size_t *bytes_out);

/*
 * Forward pass.  Overwrites all of out; never accumulates into it.
 *
 *   x       [B, C_in, L_in]
 *   offsets [B, offset_groups, L_out, K]     (K fastest)
 *   mask    [B, offset_groups, L_out, K] or NULL (NULL means a mask of ones;
 *           an all-ones mask gives bit-identical results)
 *   weight  [C_out, C_in/groups, K]
 *   bias    [C_out] or NULL (NULL means zero)
 *   out     [B, C_out, L_out]
 *
 * offset_groups must equal offsets->shape[1] (a double entry, checked).
 * stream is a hipStream_t (NULL: the null stream).
 *
 * workspace: device memory of at least dc1d_workspace_bytes() bytes, aligned
 * to 256 bytes, or NULL with workspace_bytes 0 when that is 0.  It holds the
 * weights rearranged into the kernel's reduction order (written by a first
 * kernel of the call) and the fp32 partial sums of a split reduction, passed
 * from the main kernel to a last one on the same stream; it needs no
 * initialisation and holds nothing between calls.  Calls in flight at the
 * same time must not share a workspace.
 *
 * An empty input sequence (L_in == 0) is rejected with DC1D_ERR_BAD_SHAPE
 * even when the padding would give L_out >= 1 (as conv1d rejects it).
 *
 * Limits (DC1D_ERR_BAD_SHAPE beyond them): L_in + padding <= 2^29,
 * dilation*(K-1) <= 2^29, L_out*stride <= 2^30, C_in*K <= 2^30,
 * C_out <= 2^30.  Offsets whose magnitude exceeds 2^29 are clamped to
 * +-2^29, which under these limits only moves a sample that already reads
 * zero.  Non-finite offsets or masks are outside the contract: the kernels
 * stay memory-safe but the values are unspecified.
 *
 * B == 0 is a valid no-op.  The call is asynchronous.
 */
int dc1d_forward(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
                 const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, const dc1d_tensor *out,
                 int64_t stride, int64_t padding, int64_t dilation, int64_t groups,
                 int64_t offset_groups, void *workspace, size_t workspace_bytes, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * forward as dc1d_forward (same kernels, same results bit for bit), with
 * its workspace taken from a scratch array that the library keeps in device
 * memory, one per device, of dc1d_noalloc_scratch_bytes() bytes (64 MiB),
 * held from the library's first use on that device until the process ends.
 * The call allocates nothing (no hipMalloc, no allocating library routine);
 * the caller still passes inputs and out.  Returns DC1D_ERR_WORKSPACE,
 * before any device work, when dc1d_workspace_bytes() for these arguments
 * exceeds the scratch size; DC1D_ERR_DEVICE if the scratch address cannot
 * be looked up.  Every call on one device shares that device's scratch
 * (it needs no initialisation and holds nothing useful between calls):
 * calls that may run at the same time on one device (different streams
 * without an ordering between them) race on it and must be serialised by
 * the caller.  Other arguments and errors as dc1d_forward.
 */
int dc1d_forward_noalloc(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
                         const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, const dc1d_tensor *out,
                         int64_t stride, int64_t padding, int64_t dilation, int64_t groups,
                         int64_t offset_groups, void *stream);

/* Size in bytes of the per-device scratch array dc1d_forward_noalloc uses. */
size_t dc1d_noalloc_scratch_bytes(void);

/*
 * Profiling aid.  While set, every forward call made on the calling thread
 * (dc1d_forward, dc1d_forward_constrained, dc1d_forward_noalloc) records
 * start_event on its stream immediately before it launches its dominant
 * kernel (the fused sampling + MFMA kernel, or the depthwise or direct
 * kernel) and stop_event immediately after, so that the elapsed time
 * between them is that kernel's alone, without the small kernels the call
 * may also enqueue (the weight rearrangement before it, the split
 * reduction after it).  Both are hipEvent_t handles owned by the caller,
 * passed as void*; (NULL, NULL) turns the hook off.  The setting is
 * per thread and changes no result.  Returns DC1D_ERR_NULL_PTR when exactly
 * one of the two is NULL.
 */
int dc1d_set_kernel_events(void *start_event, void *stop_event);

/*
 * Constrained mode: dc1d_forward with every tap kept inside its receptive
 * field (the dc1d page's default, section Usage / DeformConv1d: each kernel
 * tap is constrained to its own receptive field unless the layer is made
 * unconstrained).  The page does not give the rule; this library reads the
 * receptive field as the undeformed kernel's window of the output,
 * [l*stride - padding, l*stride - padding + (K-1)*dilation], so tap k's
 * offset is clamped to [-k*dilation, (K-1-k)*dilation] before the position
 * is split; positions in the window outside [0, L_in) still read zero.
 * Same arguments, workspace and errors as dc1d_forward, plus
 * DC1D_ERR_BAD_ARG when (K-1)*dilation >= 2^24.
 */
int dc1d_forward_constrained(const dc1d_tensor *x, const dc1d_tensor *offsets,
                             const dc1d_tensor *mask_or_null, const dc1d_tensor *weight,
                             const dc1d_tensor *bias_or_null, const dc1d_tensor *out, int64_t stride,
                             int64_t padding, int64_t dilation, int64_t groups, int64_t offset_groups,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward (fp32 or bf16 storage; every gradient has its input's dtype, and
 * grad_out the inputs' dtype).  For
 * grad_out = dL/d(out) [B, C_out, L_out], writes the gradients of
 * L = sum(grad_out * out) with respect to the inputs of dc1d_forward, each
 * into a caller buffer shaped like that input (NULL: not computed):
 *
 *   dS[b,ci,k,l]    = sum over co's group of weight[co,ci_local,k] * grad_out[b,co,l]
 *   grad_x[b,ci,i0] += dS*m*(1-f);  grad_x[b,ci,i0+1] += dS*m*f  (indices inside [0, L_in))
 *   grad_offsets[b,g,l,k] = sum over ci in g of dS*m*(x~(i0+1) - x~(i0))
 *   grad_mask[b,g,l,k]    = sum over ci in g of dS*((1-f)*x~(i0) + f*x~(i0+1))
 *   grad_weight[co,cl,k]  = sum over (b,l) of grad_out[b,co,l] * S[b,ci,k,l]
 *   grad_bias[co]         = sum over (b,l) of grad_out[b,co,l]
 *
 * with i0, f, m, x~ and S as in dc1d_forward: the derivatives of the
 * forward's definition term by term (the dc1d page trains the offsets and
 * checks their gradient against a finite difference, section Demo
 * notebook).  The offset gradient is that of the interpolation formula with
 * i0 held fixed, i.e. the right derivative at integer offsets.  Every
 * requested gradient is overwritten.  grad_x is gathered (each position's
 * sum formed by one thread in a fixed order) when the shape's gather arrays
 * fit in LDS, samples moved more than 16 positions then added with atomics;
 * otherwise it is cleared and accumulated with atomics.  grad_bias and, for
 * some shapes, the other gradients are accumulated with atomics.  Where
 * atomics are used the last bits may differ between runs.  grad_mask needs
 * a mask.  Gradients must not overlap the inputs, each other or the
 * workspace.
 *
 * bf16 storage: the inputs are widened exactly into fp32 copies in the
 * workspace, the fp32 kernels compute every gradient there (fp32
 * arithmetic, as above), and each requested gradient is rounded once, to
 * nearest even, into its bf16 buffer (the dc1d page trains the layer with
 * torch.autograd, whose gradients keep the input dtype; intro and section
 * Demo notebook).
 *
 * workspace: at least dc1d_backward_workspace_bytes() bytes, 256-byte
 * aligned, when that is not 0 (for bf16 it first holds the fp32 copies of
 * the inputs and the fp32 gradients; then dS = the gradient of the samples,
 * the transposed weight and the samples for the weight gradient, split
 * partial sums, and the grad_x gather's flag, depending on the shape;
 * depthwise shapes need only the flag, or nothing); no initialisation;
 * nothing kept.
 */
int dc1d_backward_workspace_bytes(const dc1d_tensor *x, const dc1d_tensor *offsets,
                                  const dc1d_tensor *mask_or_null, const dc1d_tensor *weight,
                                  const dc1d_tensor *grad_out, int want_grad_weight, int64_t stride,
                                  int64_t padding, int64_t dilation, int64_t groups,
                                  int64_t offset_groups, size_t *bytes_out);

int dc1d_backward(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
                  const dc1d_tensor *weight, const dc1d_tensor *grad_out,
                  const dc1d_tensor *grad_x_or_null, const dc1d_tensor *grad_offsets_or_null,
                  const dc1d_tensor *grad_mask_or_null, const dc1d_tensor *grad_weight_or_null,
                  const dc1d_tensor *grad_bias_or_null, int64_t stride, int64_t padding,
                  int64_t dilation, int64_t groups, int64_t offset_groups, void *workspace,
                  size_t workspace_bytes, void *stream);

/*
 * The packed layer (fp32 or bf16 storage, one dtype for every tensor of the
 * call): the layer computes its own offsets, and optionally its mask, from its input,
 * then runs the forward above with them (dc1d page, section
 * PackedDeformConv1d: offsets from a depthwise-separable convolutional
 * block; section Modulation (DCNv2): a second pointwise branch off the same
 * depthwise trunk, ending in a sigmoid, predicts the mask).  The block's
 * layers are only sketched there; this library reads them as:
 *
 *   t[b,c,l]          = trunk_bias[c] + sum_k trunk_weight[c,0,k] * x~[b,c, l*stride - padding + k*dilation]
 *   offsets[b,g,l,k]  = off_bias[g*K+k] + sum_c off_weight[g*K+k, c, 0] * t[b,c,l]
 *   mask[b,g,l,k]     = sigmoid(mask_bias[g*K+k] + sum_c mask_weight[g*K+k, c, 0] * t[b,c,l])
 *   out               = dc1d_forward(x, offsets, mask or none, weight, bias)
 *
 * i.e. a depthwise conv1d with the layer's K, stride, padding and dilation
 * (so it yields L_out columns), no activation, then pointwise convs whose
 * output channel g*K + k is tap k of offset group g; sigmoid(z) =
 * 1 / (1 + exp(-z)).  Shapes: x [B, C_in, L_in]; trunk_weight [C_in, 1, K];
 * trunk_bias [C_in]; off_weight and mask_weight [G*K, C_in, 1] (G = offset
 * groups, dividing C_in, implied by the shape); off_bias and mask_bias
 * [G*K]; weight, bias, out as in dc1d_forward; offsets_out and mask_out
 * [B, G, L_out, K].  Biases may be NULL (zero); mask_weight NULL means no
 * mask (then mask_bias and mask_out must be NULL too).  offsets_out /
 * mask_out, when given, receive the generated offsets / mask (the layer's
 * with_offsets output); otherwise they live in the workspace.  Outputs
 * must not overlap the inputs, each other or the workspace.
 * B * L_out must be below 2^31.
 *
 * bf16 storage: the generator (trunk and heads) runs in fp32 on the input
 * and on its parameters widened exactly; the offsets and mask it produces
 * are rounded once (to nearest even) to bf16, and the bf16 forward reads
 * those, as a layer computing in its input dtype does (conv1d operator
 * page: the computation stays in the input dtype).
 *
 * workspace: at least dc1d_packed_workspace_bytes() bytes, 256-byte
 * aligned, when that is not 0 (the trunk [B, C_in, L_out], the offsets and
 * mask in fp32, for bf16 also the widened parameters and the bf16 offsets
 * and mask, and the forward's own workspace); no initialisation; nothing
 * kept.
 */
int dc1d_packed_workspace_bytes(const dc1d_tensor *x, const dc1d_tensor *trunk_weight,
                                const dc1d_tensor *off_weight, const dc1d_tensor *mask_weight_or_null,
                                const dc1d_tensor *weight, int64_t stride, int64_t padding,
                                int64_t dilation, int64_t groups, size_t *bytes_out);

int dc1d_packed_forward(const dc1d_tensor *x, const dc1d_tensor *trunk_weight,
                        const dc1d_tensor *trunk_bias_or_null, const dc1d_tensor *off_weight,
                        const dc1d_tensor *off_bias_or_null, const dc1d_tensor *mask_weight_or_null,
                        const dc1d_tensor *mask_bias_or_null, const dc1d_tensor *weight,
                        const dc1d_tensor *bias_or_null, const dc1d_tensor *out,
                        const dc1d_tensor *offsets_out_or_null, const dc1d_tensor *mask_out_or_null,
                        int64_t stride, int64_t padding, int64_t dilation, int64_t groups,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * dc1d_packed_forward_constrained: the packed layer with the forward in the
 * constrained mode of dc1d_forward_constrained (each tap's offset clamped
 * to its window before the split).  The generated offsets, and the offsets
 * output, are the heads' own (unclamped).  Same arguments, workspace and
 * errors as dc1d_packed_forward, plus DC1D_ERR_BAD_ARG when
 * (K-1)*dilation >= 2^24.
 */
int dc1d_packed_forward_constrained(const dc1d_tensor *x, const dc1d_tensor *trunk_weight,
                        const dc1d_tensor *trunk_bias_or_null, const dc1d_tensor *off_weight,
                        const dc1d_tensor *off_bias_or_null, const dc1d_tensor *mask_weight_or_null,
                        const dc1d_tensor *mask_bias_or_null, const dc1d_tensor *weight,
                        const dc1d_tensor *bias_or_null, const dc1d_tensor *out,
                        const dc1d_tensor *offsets_out_or_null, const dc1d_tensor *mask_out_or_null,
                        int64_t stride, int64_t padding, int64_t dilation, int64_t groups,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward of dc1d_forward_constrained: the gradients above at the clamped
 * offsets, with grad_offsets multiplied by the clamp's right derivative
 * (1 for an offset in [-k*dilation, (K-1-k)*dilation), 0 otherwise: a tap
 * held at its window's edge does not move).  Same arguments, workspace and
 * errors as dc1d_backward.
 */
int dc1d_backward_constrained(const dc1d_tensor *x, const dc1d_tensor *offsets,
                              const dc1d_tensor *mask_or_null, const dc1d_tensor *weight,
                              const dc1d_tensor *grad_out, const dc1d_tensor *grad_x_or_null,
                              const dc1d_tensor *grad_offsets_or_null, const dc1d_tensor *grad_mask_or_null,
                              const dc1d_tensor *grad_weight_or_null, const dc1d_tensor *grad_bias_or_null,
                              int64_t stride, int64_t padding, int64_t dilation, int64_t groups,
                              int64_t offset_groups, void *workspace, size_t workspace_bytes, void *stream);

/*
 * 2D modulated deformable convolution (DCNv2), the variant the deformable
 * convolution article describes (section Deformable Convolution: every tap
 * of a 2D kernel moved by its own offset, Step 2 bilinear sampling between
 * the four surrounding pixels, Step 3 the weighted sum), with the offset
 * layout of torchvision's deform_conv2d as its documentation issue settles
 * it:
 *
 *   x        [B, C_in, H, W]
 *   offsets  [B, 2*G*kh*kw, H_out, W_out]: channel 2*((g*kh + i)*kw + j) is
 *            the row (height) offset of kernel tap (i, j) for offset group g,
 *            the next channel its column (width) offset
 *   mask     [B, G*kh*kw, H_out, W_out] or NULL (channel (g*kh + i)*kw + j),
 *            multiplied as given
 *   weight   [C_out, C_in/groups, kh, kw];  bias [C_out] or NULL
 *   out      [B, C_out, H_out, W_out], overwritten
 *
 *   out[b,co,oh,ow] = bias[co] + sum over the group's ci and taps (i, j) of
 *       weight[co,ci_local,i,j] * m * bilinear(x[b,ci], oh*stride_h - pad_h +
 *       i*dil_h + dy, ow*stride_w - pad_w + j*dil_w + dx)
 *
 * with channel ci in offset group ci / (C_in/G); each coordinate split as
 * in the 1D forward (integer grid term plus the floor of the offset);
 * bilinear weights (1-fy)(1-fx), (1-fy)fx, fy(1-fx), fy fx on the four
 * neighbours, a neighbour outside the image reading 0.  H_out and W_out
 * follow dc1d_output_length per axis.  Storage fp32 or bf16 (one dtype per
 * call; fp32 arithmetic, bf16 samples rounded once for the bf16 MFMA).
 * Limits (DC1D_ERR_BAD_SHAPE beyond them): H >= 1 and W >= 1 (an empty
 * image is rejected even when the padding would give outputs), H*W < 2^31, B <= 65535,
 * B*H_out*W_out < 2^31, G*kh*kw <= 2^24, and the 1D position limits per
 * axis.  workspace: at least dc2d_workspace_bytes() bytes, 256-byte aligned,
 * when that is not 0 (the sampled matrix [B, C_in*kh*kw, H_out*W_out] in the
 * storage dtype and split partial sums; dense layers only); no
 * initialisation; nothing kept.  Errors as dc1d_forward.
 */
int dc2d_workspace_bytes(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
                         const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, int64_t stride_h,
                         int64_t stride_w, int64_t pad_h, int64_t pad_w, int64_t dil_h, int64_t dil_w,
                         int64_t groups, int64_t offset_groups, size_t *bytes_out);

int dc2d_forward(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
                 const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, const dc1d_tensor *out,
                 int64_t stride_h, int64_t stride_w, int64_t pad_h, int64_t pad_w, int64_t dil_h, int64_t dil_w,
                 int64_t groups, int64_t offset_groups, void *workspace, size_t workspace_bytes, void *stream);

/* Which path dc2d_forward takes ("im2col2d_gemm_f32", "im2col2d_gemm_bf16",
 * "direct2d"); same validation as dc2d_workspace_bytes, no device query. */
int dc2d_plan(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
              const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, int64_t stride_h, int64_t stride_w,
              int64_t pad_h, int64_t pad_w, int64_t dil_h, int64_t dil_w, int64_t groups, int64_t offset_groups,
              const char **kernel_name);

/*
 * Test aid: the sampling positions the forward kernels use, from the same
 * device function.  For every (b, g, l, k) of offsets [B, G, L_out, K]
 * (K = offsets->shape[3]; L_out must equal dc1d_output_length(L_in, K, ...)):
 *   i0[idx]    = l*stride - padding + k*dilation + floor(o)   (int32, exact)
 *   frac[idx]  = o - floor(o)                                 (fp32)
 *   valid[idx] = (0 <= i0 < L_in) | (0 <= i0+1 < L_in) << 1
 * i0, frac and valid are device buffers of B*G*L_out*K elements each.
 */
int dc1d_debug_positions(const dc1d_tensor *offsets, int64_t L_in, int64_t stride,
                         int64_t padding, int64_t dilation, int32_t *i0, float *frac,
                         uint8_t *valid, void *stream);

/*
 * Which kernel dc1d_forward would launch for these arguments on the
 * current device, as a short static string ("mfma_f32", "mfma_bf16",
 * "depthwise", "direct", ...), and its launch shape.  Same validation as
 * dc1d_workspace_bytes.  For logging, tests and profiling.
 */
int dc1d_plan(const dc1d_tensor *x, const dc1d_tensor *offsets, const dc1d_tensor *mask_or_null,
              const dc1d_tensor *weight, const dc1d_tensor *bias_or_null, int64_t stride,
              int64_t padding, int64_t dilation, int64_t groups, int64_t offset_groups,
              const char **kernel_name, int64_t *grid_blocks, int32_t *block_threads,
              int32_t *splits);

/* ---- sequence operators ------------------------------------------------------
 *
 * What a sequence or image model puts next to a deformable convolution:
 * layer norm over the channels, rotary positions with several axes,
 * attention, group norm, and a gated linear recurrence, each with its
 * gradient.  fp32 or bf16 storage (one dtype per
 * call for the data tensors); sums, statistics and softmax are held in fp32
 * and each result is rounded once, to nearest even; probabilities and score
 * gradients of bf16 calls are rounded to bf16 as operands of the matrix
 * instructions.  Every result is summed in a fixed order without atomics:
 * the same call gives the same bits.  Ownership, streams, workspaces,
 * logging and errors are those of the calls above.
 */

/* A tensor in device memory with a stride (in elements) for each dimension.
 * Strides are not negative and the last dimension is contiguous (stride 1,
 * any where its size is 1); a stride of 0 repeats an input.  An output's
 * elements must not share memory, and an output must not overlap another
 * tensor of the call: tensors whose ranges of memory meet are taken as apart
 * where they are slices of one buffer at the same strides, along any
 * dimension, that share no element (q, k and v packed in [B, L, 3, H, D], say),
 * or slices of its heads. */
typedef struct dc1d_strided {
    void *data;
    int32_t dtype; /* a dc1d_dtype */
    int32_t ndim;
    int64_t shape[4];
    int64_t stride[4];
} dc1d_strided;

/*
 * Layer norm over axis 1:
 *
 *   mean = mean_c x,  rstd = 1 / sqrt(mean_c (x - mean)^2 + eps)
 *   y    = (x - mean) * rstd * weight + bias
 *
 *   x, y       [N, C], [B, C, L] or [B, C, H, W]   (axis 1 normalised)
 *   weight, bias  [C], x's dtype, or NULL (ones, zeros)
 *   mean, rstd  x's shape without axis 1, fp32, or NULL (not wanted)
 *
 * y may be x itself (in place); otherwise outputs must not overlap the
 * inputs or each other.  eps is finite and not negative.  C >= 1; an empty
 * x is a no-op.  Limits: C <= 2^24, fewer than 2^31 positions.
 */
int dc1d_layer_norm(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                    const dc1d_tensor *y, const dc1d_tensor *mean_or_null, const dc1d_tensor *rstd_or_null, double eps,
                    void *stream);

/*
 * Gradients of sum(grad_out * y) with respect to x, weight and bias, from
 * the forward's x, mean and rstd (NULL: not computed):
 *
 *   grad_x = rstd * (u - mean_c u - xh * mean_c(u * xh)),
 *            u = grad_out * weight,  xh = (x - mean) * rstd
 *   grad_weight[c] = sum grad_out * xh,   grad_bias[c] = sum grad_out
 *
 * in their inputs' shapes and dtype.  grad_x may be grad_out itself.  An
 * empty x gives zero grad_weight and grad_bias.  workspace: at least
 * dc1d_layer_norm_backward_workspace_bytes() bytes, 256-byte aligned, when
 * that is not 0 (the parameter gradients' partial sums).
 */
int dc1d_layer_norm_backward_workspace_bytes(const dc1d_tensor *x, int want_params, size_t *bytes_out);

int dc1d_layer_norm_backward(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *grad_out,
                             const dc1d_tensor *mean, const dc1d_tensor *rstd, const dc1d_tensor *grad_x_or_null,
                             const dc1d_tensor *grad_weight_or_null, const dc1d_tensor *grad_bias_or_null,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary positions with up to four axes (one for sequences, rows and columns
 * for images, time, rows and columns for video).  Every head of D elements
 * holds R pairs, 2 R <= D; pair i belongs to the axis whose section it is in
 * (axis 0 the first sections[0] pairs, and so on; the sections add up to R)
 * and turns by the tables' angle of that axis' position:
 *
 *   (a, b) -> (a c - b s, a s + b c),  c = cos[p][i], s = sin[p][i],
 *   p = positions[b][l][axis(i)]
 *
 * The pair is elements (i, R + i) of the head, or (2i, 2i + 1) where
 * interleaved is not 0; elements past 2 R are copied.  inverse not 0 turns
 * the other way: the backward pass (apply it to the output's gradient).
 *
 *   q, q_out   [B, L, Hq, D], k, k_out [B, L, Hkv, D] (both NULL: queries only)
 *   cos, sin   [P, R] fp32
 *   positions  [B, L, A] or [1, L, A] (shared) int32, A = n_axes
 *   sections   n_axes host integers, each >= 0, R = their sum >= 1
 *
 * Positions outside [0, P) are taken as the nearest end of the tables.  An
 * output may be its own input (in place); otherwise it must not overlap any
 * input or the other output.  Limits: B * L < 2^31, (Hq + Hkv) * D < 2^30,
 * B * L * (Hq + Hkv) * D < 2^40.
 */
int dc1d_rotary(const dc1d_strided *q, const dc1d_strided *k_or_null, const dc1d_tensor *cos, const dc1d_tensor *sin,
                const dc1d_tensor *positions, const dc1d_strided *q_out, const dc1d_strided *k_out_or_null,
                const int64_t *sections, int32_t n_axes, int interleaved, int inverse, void *stream);

/*
 * Attention.  Query i of batch b stands at position p = q_start[b] + i and
 * sees the keys j with
 *
 *   j < kv_lens[b],   j <= p where causal,   |p - j| < window where window > 0
 *
 *   out[b,i,h] = sum_j P_ij v[b,j,h'],   P_ij = exp(s_ij - lse[b,h,i]),
 *   s_ij = scale * q[b,i,h] . k[b,j,h'],   lse = log sum_j exp s_ij,
 *
 * h' = h / (Hq / Hkv): neighbouring query heads share a key head.  A query
 * that sees no key gives out 0 and lse -infinity.  Keys and values that no
 * query of the batch sees (at and past kv_lens[b], past the last query where
 * causal, ahead of the first one's window) are never used, whatever they hold;
 * those that one query sees should be finite for the sake of the others, too.
 *
 *   q, out    [B, Lq, Hq, D], k, v [B, Lk, Hkv, D], Hkv dividing Hq, D <= 128
 *   kv_lens   [B] int32, clamped to [0, Lk], or NULL (Lk)
 *   q_start   [B] int32, or NULL (Lk - Lq: the last query at the last key);
 *             for a cache of ragged lengths, kv_lens - Lq
 *   lse       [B, Hq, Lq] fp32, or NULL (not wanted)
 *   scale     finite, > 0 (usually 1 / sqrt(D));  window >= 0, 0: none
 *
 * Strides are free, so q, k, v and out may be slices of larger buffers; out
 * must not overlap the inputs.
 * |q_start| and window are clamped to 2^29.  workspace: at least
 * dc1d_attention_workspace_bytes() bytes, 256-byte aligned, when that is not
 * 0 (few queries over many keys: the partial results of parts of the keys).
 * Limits: Lq, Lk <= 2^29, B * Hkv < 2^24, B * Lq * Hq < 2^29, B * Lk * Hkv < 2^31.
 */
int dc1d_attention_workspace_bytes(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                                   size_t *bytes_out);

int dc1d_attention(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                   const dc1d_tensor *kv_lens_or_null, const dc1d_tensor *q_start_or_null, const dc1d_strided *out,
                   const dc1d_tensor *lse_or_null, int causal, int64_t window, double scale, void *workspace,
                   size_t workspace_bytes, void *stream);

/* Which kernel dc1d_attention would use ("attention_rows", "attention_keys"),
 * its workgroups, and into how many parts it splits the keys, where no window
 * narrows them. */
int dc1d_attention_plan(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v, const char **kernel_name,
                        int64_t *grid_blocks, int32_t *splits);

/*
 * Gradients of sum(grad_out * out) with respect to q, k and v, from the
 * forward's inputs, out and lse (the probabilities are formed again):
 *
 *   dS = P * (grad_out . v - grad_out . out),
 *   grad_q = scale * dS k,  grad_k = scale * dS^T q,  grad_v = P^T grad_out,
 *
 * grad_k and grad_v summed over the query heads that share a key head.
 * Keys that no query sees get zeros, and so do queries that see no key; what
 * those hold, and their grad_out, reaches no gradient.  NULL gradients are not
 * computed.  The other arguments are the forward's; gradients must not overlap
 * the inputs or each other.
 * workspace: at least dc1d_attention_backward_workspace_bytes() bytes, 256-byte
 * aligned, when that is not 0.
 */
int dc1d_attention_backward_workspace_bytes(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                                            size_t *bytes_out);

int dc1d_attention_backward(const dc1d_strided *q, const dc1d_strided *k, const dc1d_strided *v,
                            const dc1d_tensor *kv_lens_or_null, const dc1d_tensor *q_start_or_null,
                            const dc1d_strided *out, const dc1d_tensor *lse, const dc1d_strided *grad_out,
                            const dc1d_strided *grad_q_or_null, const dc1d_strided *grad_k_or_null,
                            const dc1d_strided *grad_v_or_null, int causal, int64_t window, double scale,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Group norm over positions in channels-last order, with an activation:
 *
 *   mean, rstd  of the n[b] * D elements of group k of sample b: its first
 *               n[b] positions and the D = C / groups channels k D ... k D + D - 1,
 *               rstd = 1 / sqrt(mean of (x - mean)^2 + eps)
 *   z = (x - mean) * rstd * weight + bias
 *   y = z, max(z, 0) or z / (1 + exp(-z))
 *
 *   x, y       [N, C] (one position each), [B, L, C] or [B, H, W, C]
 *   weight, bias  [C], x's dtype, or NULL (ones, zeros)
 *   lens       [B] int32, clamped to [0, L], or NULL (L); with [B, L, C] only
 *   mean, rstd  [B, groups] fp32, or NULL (not wanted)
 *   activation  a dc1d_activation
 *
 * Positions past a sample's length give 0, whatever they hold; a sample of
 * length 0 has mean 0 and rstd 0.  Squares past fp32's range make the variance
 * infinite and rstd 0.  y may be x itself (in place); otherwise
 * outputs must not overlap the inputs or each other.  eps is finite and not
 * negative; groups divides C.  An empty x is a no-op (with L = 0, mean and rstd
 * are 0).  workspace: at least dc1d_group_norm_workspace_bytes() bytes, 256-byte
 * aligned, when that is not 0 (the partial statistics of samples that one
 * workgroup does not hold).  Limits: C <= 2^24, fewer than 2^31 positions,
 * B * groups < 2^31.
 */
typedef enum dc1d_activation { DC1D_ACT_NONE = 0, DC1D_ACT_RELU = 1, DC1D_ACT_SILU = 2 } dc1d_activation;

int dc1d_group_norm_workspace_bytes(const dc1d_tensor *x, int64_t groups, size_t *bytes_out);

int dc1d_group_norm(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                    const dc1d_tensor *lens_or_null, const dc1d_tensor *y, const dc1d_tensor *mean_or_null,
                    const dc1d_tensor *rstd_or_null, int64_t groups, double eps, int activation, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * Gradients of sum(grad_out * y) with respect to x, weight and bias, from
 * the forward's x, mean and rstd (NULL: not computed):
 *
 *   g = grad_out * (the activation's derivative at z),  u = g * weight,
 *   xh = (x - mean) * rstd,
 *   grad_x = rstd * (u - mean of u - xh * mean of (u * xh)),  the means over the group
 *   grad_weight[c] = sum of g * xh,   grad_bias[c] = sum of g
 *
 * in their inputs' shapes and dtype.  The derivative of relu at 0 is 0.  bias
 * is read where there is an activation.  Positions past a sample's length get
 * zeros, and nothing that they or their grad_out hold reaches a gradient.
 * grad_x may be grad_out itself.  An empty x gives zero grad_weight and
 * grad_bias.  workspace: at least dc1d_group_norm_backward_workspace_bytes()
 * bytes, 256-byte aligned, when that is not 0 (partial sums; 8 bytes for every
 * element of [N, C] where a group has more than 2048 fp32 or 4096 bf16 channels).
 */
int dc1d_group_norm_backward_workspace_bytes(const dc1d_tensor *x, int64_t groups, int want_params, size_t *bytes_out);

int dc1d_group_norm_backward(const dc1d_tensor *x, const dc1d_tensor *weight_or_null, const dc1d_tensor *bias_or_null,
                             const dc1d_tensor *lens_or_null, const dc1d_tensor *grad_out, const dc1d_tensor *mean,
                             const dc1d_tensor *rstd, const dc1d_tensor *grad_x_or_null,
                             const dc1d_tensor *grad_weight_or_null, const dc1d_tensor *grad_bias_or_null,
                             int64_t groups, int activation, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A gated linear recurrence along the positions of x [B, L, C], every channel
 * on its own:
 *
 *   a_t = sigmoid(gate_t),   h_t = a_t * h_{t-1} + u_t,   y_t = h_t,
 *   u_t = x_t,  or (1 - a_t) * x_t where blend is not 0,
 *
 * over t = 0 ... n - 1, or n - 1 ... 0 where reverse is not 0, n = lens[b]; the
 * state ahead of the first one is state[b].
 *
 *   x, gate, y  [B, L, C], any strides over contiguous channels (rank 3 of
 *               dc1d_strided); a gate that is the same for all batches or
 *               positions has stride 0 there
 *   state, last [B, C] fp32: the states ahead of the first position (NULL:
 *               zeros) and after the last one (NULL: not wanted); last may be
 *               state itself, for one position at a time
 *   lens        [B] int32, clamped to [0, L], or NULL (L)
 *   states      [B, ceil(L / 64), C] fp32: the state ahead of every 64th position
 *               in the recurrence's order, from the first on, which the backward
 *               pass starts from (past the length: the last state), or NULL
 *
 * The state is held in fp32 throughout.  A gate of -infinity starts anew
 * (a = 0), one of +infinity holds the state (a = 1).  A NaN, or an infinite x
 * or state, reaches its channel's later states only, which are then infinite or
 * NaN, also behind a gate of -infinity (0 times either is NaN).  Positions past a
 * sequence's length give 0, whatever they hold; an empty one leaves its state.
 * y may be x itself (in place); otherwise outputs must not overlap the inputs
 * or each other.  workspace: at least dc1d_gated_recurrence_workspace_bytes()
 * bytes, 256-byte aligned, when that is not 0 (long sequences of few channels:
 * what its parts do to a state).  Limits: L <= 2^29, C <= 2^24, B * L < 2^31,
 * B * C < 2^31.
 */
int dc1d_gated_recurrence_workspace_bytes(const dc1d_strided *x, size_t *bytes_out);

int dc1d_gated_recurrence(const dc1d_strided *x, const dc1d_strided *gate, const dc1d_tensor *state_or_null,
                          const dc1d_tensor *lens_or_null, const dc1d_strided *y, const dc1d_tensor *last_or_null,
                          const dc1d_tensor *states_or_null, int blend, int reverse, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * Gradients of sum(grad_out * y) + sum(grad_last * last) with respect to x,
 * gate and state, from the forward's x, gate and states (NULL: not computed;
 * grad_last NULL: zeros).  In the recurrence's order:
 *
 *   r_t = grad_out_t + a_{t+1} * r_{t+1},   r_n = grad_last (with a_n = 1),
 *   grad_x = r,              grad_gate = r * h_{t-1} * a * (1 - a),
 *   or r * (1 - a),          or r * (h_{t-1} - x) * a * (1 - a) where blend,
 *   grad_state = a_0 * r_0
 *
 * The states between those given are formed again in fp32.  Positions past a
 * sequence's length get zeros, and nothing that they hold reaches a gradient.
 * grad_x and grad_gate may have any strides over contiguous channels; each is
 * the gradient of one element of the full [B, L, C].  grad_x may be grad_out
 * itself.  Gradients must not overlap the inputs or each other otherwise;
 * grad_state may be grad_last itself.
 */
int dc1d_gated_recurrence_backward_workspace_bytes(const dc1d_strided *x, size_t *bytes_out);

int dc1d_gated_recurrence_backward(const dc1d_strided *x, const dc1d_strided *gate, const dc1d_tensor *states,
                                   const dc1d_tensor *lens_or_null, const dc1d_strided *grad_out,
                                   const dc1d_tensor *grad_last_or_null, const dc1d_strided *grad_x_or_null,
                                   const dc1d_strided *grad_gate_or_null, const dc1d_tensor *grad_state_or_null,
                                   int blend, int reverse, void *workspace, size_t workspace_bytes, void *stream);

/* A static, NUL-terminated description of a status code. */
const char *dc1d_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* DC1D_H */
