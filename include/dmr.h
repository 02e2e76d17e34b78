/*
 * dmr.h - C ABI of the MI355X (gfx950) K-nearest-face mesh rasterizer.
 *
 * Entry points: the rasterizer's forward and backward passes
 * (rasterize_meshes_fwd, rasterize_meshes_fwd_ex with settings,
 * rasterize_meshes_fwd_noalloc for callers that cannot allocate,
 * rasterize_meshes_bwd) and their workspace helpers; the second stage that
 * fuses each pixel's K faces (dmr_blend_fwd / dmr_blend_bwd); point clouds
 * (rasterize_points_fwd / rasterize_points_bwd); the upstream projection
 * from world space (dmr_project_fwd / dmr_project_bwd); linear layers with
 * one weight per mesh (dmr_grouped_linear_fwd / dmr_grouped_linear_bwd) and
 * the orthogonalised update of such weights (dmr_orthogonalize); status
 * strings and optional per-kernel timing.
 *
 * The main operation is the face-selection stage of the two-stage rasterizer of
 * "Accelerating 3D Deep Learning with PyTorch3D": for every pixel, select the
 * faces that influence it and keep the K nearest (gptget.net summary,
 * "Methodology": stage one selects the faces affecting each pixel; nubint.ai
 * review, "Proposed method": per-pixel K nearest faces), over a batch of
 * meshes of different sizes (rocketrecap summary, "1:00 Heterogeneous
 * Batching"), with per-pixel intermediates returned so that shading can be
 * composed on top and differentiated (nubint.ai review, "Proposed method";
 * rocketrecap summary, "3:52 Differentiable Renderer").
 *
 * Conventions (the pages fix none of them; these are the library's):
 *   pixel (i, j) of an H x W image has its centre at
 *       x = fl(fl((2j+1)/W) - 1),  y = fl(fl((2i+1)/H) - 1)   (binary32, no flip);
 *   a face is a candidate for a pixel when the centre is strictly inside it
 *   (all barycentrics > 0, centre in the face's closed bounding box) or its
 *   squared 2D distance to the face's edges is below blur_radius, it is not
 *   degenerate (doubled area A != 0) and its depth z at the pixel, from
 *   barycentrics clipped to [0,1] and renormalised, is > 0;
 *   each pixel keeps its K candidates of smallest (z, global face index);
 *   all decisions and values are binary32, evaluated in one fixed operation
 *   order with no fused multiply-add, so results are reproducible bit for bit.
 * Rasterizer settings (rocketrecap summary, "32:56 Technical Bug Fix", names
 * a perspective_correct setting; the pages define none of them), bits of the
 * `flags` of rasterize_meshes_fwd_ex and rasterize_meshes_bwd:
 *   DMR_RASTER_PERSPECTIVE_CORRECT  a face is a candidate only if its three
 *       vertex depths are > 0; the clipped barycentrics c are weighted as
 *       n_k = (c_k z_{k+1}) z_{k+2} (the inverse depths, scaled), normalised
 *       by n0 + n1 + n2 in place of c0 + c1 + c2, and z = sum of the weighted
 *       barycentrics times the vertex depths (1/z linear in screen space);
 *   DMR_RASTER_CULL_BACKFACES  faces with A > 0 are skipped: A is the depth
 *       component of the normal (v1 - v0) x (v2 - v0), so their normal points
 *       away from the viewer;
 *   DMR_RASTER_UNCLIPPED_BARY  bary returns the barycentrics before clipping
 *       (perspective-weighted the same way with the setting above); depth,
 *       inclusion and order do not change.
 *
 * Memory: every pointer argument is a device pointer on the device the
 * stream belongs to (the default device for the null stream); arrays are
 * row-major, contiguous and must not alias. The library keeps no pointer
 * after a call returns and owns no device memory. Calls are asynchronous and
 * ordered on `stream`; results are valid once the stream reaches them.
 * Calls on different streams may run concurrently if they use different
 * workspaces.
 *
 * Errors: every entry point validates its scalar arguments and pointers on
 * the host before it launches anything and returns a status; no exception
 * crosses the ABI. Device data (indices, offsets) is not read on the host:
 * a vertex index outside [0, V) makes its face a non-candidate and sets
 * DMR_FLAG_BAD_VERTEX_INDEX in the workspace statistics; offsets that are not
 * non-decreasing from 0 to F give unspecified (but memory-safe) results.
 * Non-finite vertex coordinates give unspecified outputs.
 */
#ifndef DMR_H
#define DMR_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dmr_status {
    DMR_SUCCESS = 0,
    DMR_ERROR_INVALID_VALUE = 1,        /* a size, pointer or scalar argument is invalid */
    DMR_ERROR_WORKSPACE_TOO_SMALL = 2,  /* below dmr_workspace_min_size() */
    DMR_ERROR_HIP = 3,                  /* a HIP runtime call failed (launch, event, copy) */
    DMR_ERROR_UNSUPPORTED = 4           /* K > DMR_MAX_K, or a size beyond the index limits */
} dmr_status;

#define DMR_MAX_K 64
#define DMR_MAX_IMAGE_SIDE 32767
#define DMR_FLAG_BAD_VERTEX_INDEX 0x1u

#define DMR_RASTER_PERSPECTIVE_CORRECT 0x2u
#define DMR_RASTER_CULL_BACKFACES 0x4u
#define DMR_RASTER_UNCLIPPED_BARY 0x8u
#define DMR_RASTER_SETTINGS (DMR_RASTER_PERSPECTIVE_CORRECT | DMR_RASTER_CULL_BACKFACES | DMR_RASTER_UNCLIPPED_BARY)

/*
 * Forward pass: K nearest faces per pixel.
 *
 *   verts      [V,3] float32  x, y in normalised device coordinates, z = view
 *                             depth; the vertices of all meshes, packed.
 *   faces      [F,3] int64    vertex indices into verts (global), packed.
 *   mesh_face_offsets [N+1] int64  mesh n owns faces [off[n], off[n+1]);
 *                             off[0] = 0, non-decreasing, off[N] = F. Empty
 *                             meshes are allowed and give all-padding images.
 *   H, W       image size, 1..DMR_MAX_IMAGE_SIDE.
 *   K          faces kept per pixel, 1..DMR_MAX_K.
 *   blur_radius squared NDC distance; finite and >= 0.
 *   pix_to_face [N,H,W,K] int64  global face index, ascending (z, face); -1 pads.
 *   zbuf       [N,H,W,K]   float32  depth at the pixel; -1 on padding.
 *   bary       [N,H,W,K,3] float32  clipped, renormalised barycentrics; -1 pads.
 *   dists      [N,H,W,K]   float32  signed squared distance to the face's
 *                                   edges (< 0 inside); -1 on padding.
 *   workspace  device scratch of workspace_bytes >= dmr_workspace_min_size(),
 *              16-byte aligned (else DMR_ERROR_INVALID_VALUE; hipMalloc and
 *              torch allocations are); dmr_workspace_size_hint() gives a
 *              size that normally holds the per-bin face lists. Results do
 *              not depend on the size: bins
 *              whose list does not fit are rasterised from their mesh's full
 *              face range instead (exact, slower), and the size that would
 *              have held every list is recorded (dmr_workspace_stats).
 * All outputs are fully overwritten, padding included. Returns DMR_SUCCESS
 * without launching anything when N*H*W == 0.
 */
dmr_status rasterize_meshes_fwd(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                const int64_t* mesh_face_offsets, int64_t N,
                                int32_t H, int32_t W, int32_t K, float blur_radius,
                                int64_t* pix_to_face, float* zbuf, float* bary, float* dists,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The forward pass with rasterizer settings: flags is a mask of the
 * DMR_RASTER_* bits (any other bit: DMR_ERROR_INVALID_VALUE); flags = 0 is
 * rasterize_meshes_fwd. A backward pass of its outputs takes the same bits. */
dmr_status rasterize_meshes_fwd_ex(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                   const int64_t* mesh_face_offsets, int64_t N,
                                   int32_t H, int32_t W, int32_t K, float blur_radius,
                                   int64_t* pix_to_face, float* zbuf, float* bary, float* dists,
                                   void* workspace, size_t workspace_bytes, uint32_t flags, hipStream_t stream);

/*
 * Allocation-free forward pass, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): rasterize_meshes_fwd with the workspace replaced by a
 * device array of DMR_NOALLOC_SCRATCH_BYTES that the library holds on each
 * device it runs on until the process ends. Arguments and results are those
 * of rasterize_meshes_fwd (settings 0); the call allocates nothing.
 *   Sizes whose face records and bin tables (dmr_workspace_min_size) exceed
 *   DMR_NOALLOC_SCRATCH_BYTES give DMR_ERROR_UNSUPPORTED before anything is
 *   launched; bin lists that do not fit in the rest of the array take the
 *   exact full-face-range path, so results never depend on the size.
 *   Every call on a device shares that device's array: calls that overlap on
 *   one device (different streams, or host threads) race and give undefined
 *   results; calls ordered on one stream are safe. A backward pass of these
 *   outputs runs without the forward's workspace (flags without
 *   DMR_BWD_REUSE_FORWARD_WORKSPACE), which allocates nothing either.
 */
#define DMR_NOALLOC_SCRATCH_BYTES (128u << 20)
dmr_status rasterize_meshes_fwd_noalloc(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                        const int64_t* mesh_face_offsets, int64_t N,
                                        int32_t H, int32_t W, int32_t K, float blur_radius,
                                        int64_t* pix_to_face, float* zbuf, float* bary, float* dists,
                                        hipStream_t stream);

/*
 * Backward pass: maps the gradients of zbuf, bary and dists to vertex
 * positions (rocketrecap summary, "3:52 Differentiable Renderer": gradients
 * flow from image pixels back to the 3D parameters).
 *
 *   verts, faces, mesh_face_offsets, N, H, W, K, blur_radius: as given to the
 *              forward pass that produced pix_to_face.
 *   pix_to_face [N,H,W,K] int64: that forward pass's output.
 *   grad_zbuf [N,H,W,K], grad_bary [N,H,W,K,3], grad_dists [N,H,W,K] float32:
 *              upstream gradients; any of them may be NULL (= zero). Values on
 *              padded slots are ignored.
 *   grad_verts [V,3] float32: overwritten (not accumulated) with dL/dverts.
 *   flags      the DMR_RASTER_* bits the forward pass was given, plus
 *              optionally DMR_BWD_REUSE_FORWARD_WORKSPACE (any other bit:
 *              DMR_ERROR_INVALID_VALUE).
 *   workspace  With DMR_BWD_REUSE_FORWARD_WORKSPACE, `workspace` is the
 *              forward pass's workspace for these same inputs, unmodified
 *              since that call (workspace_bytes as given to it); its per-face
 *              records replace recomputing each face's data from verts and
 *              faces, and its bin order and counts schedule the tiles (bins
 *              without faces are skipped). The caller guarantees this; it is
 *              not checked (only its size and 16-byte alignment are), and any
 *              other content gives wrong gradients. The call only reads the
 *              workspace. Without that bit the workspace is not used and may
 *              be NULL.
 * Contributions are summed per 16x16 tile and vertex in LDS, in 64-bit fixed
 * point relative to each sum's own scale (units of 2^-30 of the largest
 * partial of the slot that started it), so the accuracy does not depend on
 * the scale of the upstream gradients; the tile sums are then added to
 * grad_verts with float32 atomics, so the rounding of grad_verts may differ
 * between runs.
 */
#define DMR_BWD_REUSE_FORWARD_WORKSPACE 0x1u
dmr_status rasterize_meshes_bwd(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                const int64_t* mesh_face_offsets, int64_t N,
                                int32_t H, int32_t W, int32_t K, float blur_radius,
                                const int64_t* pix_to_face,
                                const float* grad_zbuf, const float* grad_bary, const float* grad_dists,
                                float* grad_verts,
                                void* workspace, size_t workspace_bytes, uint32_t flags, hipStream_t stream);

/*
 * Second stage: fusing each pixel's kept faces (gptget.net summary,
 * "Methodology": the second stage merges the influence of the several faces
 * of a pixel, easing the discontinuity of rasterization; nubint.ai review,
 * "Proposed method": per-pixel K-nearest-face influence). The pages give no
 * formula; the library's reading, per pixel over its filled slots k
 * (pix_to_face in [0, F)), is
 *     p_k = 1 / (1 + exp(dists_k / sigma)),      alpha = 1 - prod_k (1 - p_k)
 *     zeta_k = (zfar - zbuf_k) / (zfar - znear), zeta_max = max_k zeta_k
 *     w_k = p_k exp((zeta_k - zeta_max) / gamma), w_bg = exp((eps - zeta_max) / gamma)
 *     rgb = (sum_k w_k color[pix_to_face_k] + w_bg background) / (sum_k w_k + w_bg)
 * and (background, 0) for a pixel without filled slots.
 */
typedef struct dmr_blend_params {
    float sigma;          /* > 0, squared NDC units: sharpness of the coverage */
    float gamma;          /* > 0: depth softness of the colour weights */
    float znear, zfar;    /* zfar > znear: depth range of the normalised inverse depth */
    float eps;            /* offset of the background weight */
    float background[3];  /* RGB of uncovered pixels */
} dmr_blend_params;

/*   pix_to_face [P,K] int64, zbuf [P,K] float32, dists [P,K] float32: the
 *              forward pass's outputs (P = N*H*W pixels, K slots each);
 *              indices outside [0, F) count as empty slots.
 *   face_colors [F,3] float32 RGB per face.
 *   params     host pointer, read during the call; finite values, sigma > 0,
 *              gamma > 0, zfar > znear (else DMR_ERROR_INVALID_VALUE).
 *   rgba       [P,4] float32, 16-byte aligned, overwritten.
 * K above DMR_MAX_K, F above INT32_MAX or P above 64 * INT32_MAX give
 * DMR_ERROR_UNSUPPORTED. Computed in binary32 with the device exp; P == 0
 * launches nothing. */
dmr_status dmr_blend_fwd(const int64_t* pix_to_face, const float* zbuf, const float* dists, int64_t P, int32_t K,
                         const float* face_colors, int64_t F, const dmr_blend_params* params, float* rgba,
                         hipStream_t stream);

/* Backward of dmr_blend_fwd for the same inputs: grad_rgba [P,4] float32
 * (16-byte aligned) in,
 * grad_zbuf [P,K] and grad_dists [P,K] float32 out (overwritten; 0 on empty
 * slots). zeta_max is held fixed (rgb does not depend on it); no gradient
 * flows to the colours or parameters. */
dmr_status dmr_blend_bwd(const int64_t* pix_to_face, const float* zbuf, const float* dists, int64_t P, int32_t K,
                         const float* face_colors, int64_t F, const dmr_blend_params* params,
                         const float* grad_rgba, float* grad_zbuf, float* grad_dists, hipStream_t stream);

/*
 * Upstream projection: world-space vertices to the screen space the
 * rasterizer takes, so that gradients reach 3D parameters (rocketrecap
 * summary, "3:52 Differentiable Renderer": gradients flow from image pixels
 * back to the 3D model parameters; "22:00 2D-to-3D Reconstruction": several
 * viewpoints per object). The pages give no camera model; the library's
 * reading: mesh n is seen through one 4x4 matrix M_n, and a vertex X of mesh
 * n maps to
 *     h = M_n (X, 1),   (x, y, z) = (h0 / h3, h1 / h3, h2)
 * (x, y perspective-divided NDC; the third row gives the depth, e.g. the
 * view depth for a pinhole camera). Binary32; each h_r is the left-to-right
 * sum M_r0 X + M_r1 Y + M_r2 Z + M_r3, and both divisions are correctly
 * rounded. A vertex with h3 == 0 (on the camera plane) gets non-finite x, y,
 * as the definition does.
 *
 *   verts_world [V,3] float32; mesh_vert_offsets [N+1] int64: mesh n owns
 *              vertices [off[n], off[n+1]) (off[0] = 0, non-decreasing,
 *              off[N] = V; other offsets give unspecified, memory-safe
 *              results); N >= 1 when V > 0.
 *   cameras    [N,4,4] float32, row-major.
 *   verts_ndc  [V,3] float32, overwritten; must not alias verts_world.
 * Errors: negative sizes, missing pointers or N == 0 with V > 0:
 * DMR_ERROR_INVALID_VALUE; V above 256 * (2^32 - 1) or N above (2^32 - 1) / 16:
 * DMR_ERROR_UNSUPPORTED. V == 0
 * launches nothing.
 */
dmr_status dmr_project_fwd(const float* verts_world, int64_t V, const int64_t* mesh_vert_offsets, int64_t N,
                           const float* cameras, float* verts_ndc, hipStream_t stream);

/* Backward of dmr_project_fwd for the same inputs: grad_verts_ndc [V,3] in,
 * grad_verts_world [V,3] out (overwritten) and, if grad_cameras is not NULL,
 * grad_cameras [N,4,4] (overwritten; summed over each mesh's vertices with
 * float32 atomics, so its rounding may differ between runs). */
dmr_status dmr_project_bwd(const float* verts_world, int64_t V, const int64_t* mesh_vert_offsets, int64_t N,
                           const float* cameras, const float* grad_verts_ndc, float* grad_verts_world,
                           float* grad_cameras, hipStream_t stream);

/*
 * Point clouds: for every pixel, the K nearest points of its own cloud
 * within a radius (rocketrecap summary, "2:02 Data Structures and I/O":
 * point clouds beside meshes; gptget.net summary, "Methodology": per-pixel
 * selection over heterogeneous batches). The pages give no formula; the
 * library's reading: a point q with z_q > 0 is a candidate for pixel (i, j)
 * (centre (x, y) as for meshes) when d2 = (x - x_q)^2 + (y - y_q)^2 <
 * radius * radius (binary32, that order, strict); each pixel keeps the K
 * candidates of smallest (z_q, q).
 *
 *   points     [P,3] float32 x, y NDC, z depth; cloud_offsets [N+1] int64:
 *              cloud n owns points [off[n], off[n+1]) (as mesh_face_offsets).
 *   radius     NDC units; finite and >= 0.
 *   idx [N,H,W,K] int64 global point index (-1 pads); zbuf [N,H,W,K] float32
 *              z_q (-1 pads); dists [N,H,W,K] float32 d2 (-1 pads).
 *   workspace  as for meshes, sized by dmr_points_workspace_size_hint();
 *              too small a workspace keeps the results exact (slow path).
 * Errors as for rasterize_meshes_fwd; P above INT32_MAX - 1 or more than
 * 256 * (2^32 - 1) slots: DMR_ERROR_UNSUPPORTED.
 */
dmr_status rasterize_points_fwd(const float* points, int64_t P, const int64_t* cloud_offsets, int64_t N,
                                int32_t H, int32_t W, int32_t K, float radius,
                                int64_t* idx, float* zbuf, float* dists,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Backward of rasterize_points_fwd: grad_points [P,3] (overwritten) from the
 * gradients of zbuf and dists (each may be NULL), for the idx that pass
 * returned: dL/dz_q += g_z, dL/d(x_q, y_q) += -2 (x - x_q, y - y_q) g_d per
 * slot, summed with float32 atomics (rounding may differ between runs). */
dmr_status rasterize_points_bwd(const float* points, int64_t P, const int64_t* cloud_offsets, int64_t N,
                                int32_t H, int32_t W, int32_t K, const int64_t* idx,
                                const float* grad_zbuf, const float* grad_dists, float* grad_points,
                                hipStream_t stream);

/* Workspace of the point rasterizer: minimum (records and bin tables) and
 * suggested (with room for the per-bin point lists) sizes; 0 on invalid
 * arguments. */
size_t dmr_points_workspace_min_size(int64_t N, int64_t P, int32_t H, int32_t W);
size_t dmr_points_workspace_size_hint(int64_t N, int64_t P, int32_t H, int32_t W, int32_t K, float radius);

/* Smallest forward workspace (bytes) for these sizes: face records and bin
 * tables, with room for no per-bin face list. 0 on invalid arguments. */
size_t dmr_workspace_min_size(int64_t N, int64_t F, int32_t H, int32_t W);

/* Suggested forward workspace (bytes): the minimum plus an estimate of the
 * per-bin face lists from F, the image size and blur_radius. 0 on invalid
 * arguments. */
size_t dmr_workspace_size_hint(int64_t N, int64_t F, int32_t H, int32_t W, int32_t K, float blur_radius);

/*
 * Linear layers of a packed batch, one weight per group: the decoders and
 * shading layers that a model of each mesh (or material, or view) learns
 * from the rasterizer's gradients. Rows of all groups are packed one after
 * another, as vertices are for dmr_project_fwd, and for the rows r of group n
 *     y_r = W_n x_r + b_n.
 *
 *   x          [R, in_features]; y [R, out_features], overwritten.
 *   row_offsets [N+1] int64: group n owns rows [off[n], off[n+1]) (off[0] =
 *              0, non-decreasing, off[N] = R; other offsets give unspecified,
 *              memory-safe results). Empty groups and groups of one row are
 *              allowed; N >= 1 when R > 0.
 *   weight     [N, out_features, in_features]; bias [N, out_features] or NULL.
 *   dtype      of x, weight, bias, y and all gradients. Sums are float32
 *              (float32 products too), rounded once.
 * A row depends on no other row; infinities and NaN propagate as in the
 * formula. Arrays with 16-byte aligned start and widths that are multiples
 * of 16 bytes take wide loads; others are as exact, and slower.
 * Errors: negative sizes, widths below 1, missing pointers, an unknown dtype
 * or N == 0 with R > 0: DMR_ERROR_INVALID_VALUE; widths above
 * DMR_MAX_LINEAR_WIDTH or more output tiles than a launch can hold:
 * DMR_ERROR_UNSUPPORTED. R == 0 launches nothing.
 */
typedef enum dmr_dtype {
    DMR_FLOAT32 = 0,
    DMR_FLOAT16 = 1,
    DMR_BFLOAT16 = 2
} dmr_dtype;
#define DMR_MAX_LINEAR_WIDTH (1 << 20)
dmr_status dmr_grouped_linear_fwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                  const void* weight, const void* bias, int32_t out_features, dmr_dtype dtype, void* y,
                                  hipStream_t stream);

/* Backward of dmr_grouped_linear_fwd for the same inputs, from grad_y
 * [R, out_features]; each result is overwritten and may be NULL:
 *     grad_x_r = W_n^T g_r,  grad_weight_n = sum_r g_r x_r^T,
 *     grad_bias_n = sum_r g_r   (zero for an empty group).
 * weight is read only for grad_x, x only for grad_weight and grad_bias.
 * Long sums over rows are cut into pieces that `workspace` holds (16-byte
 * aligned, of dmr_grouped_linear_workspace_size() bytes; not used without
 * grad_weight and grad_bias) and added in a fixed order: results are the
 * same on every run. */
dmr_status dmr_grouped_linear_bwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                  const void* weight, int32_t out_features, dmr_dtype dtype, const void* grad_y,
                                  void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);
/* Workspace of dmr_grouped_linear_bwd in bytes; 0 on invalid arguments. */
size_t dmr_grouped_linear_workspace_size(int64_t R, int64_t N, int32_t in_features, int32_t out_features, dmr_dtype dtype);

/* What calls of these sizes are computed by (for measurement and tests; the
 * results do not depend on it but for the order of sums): the tile of y and of
 * grad_x, in columns and rows, the side of the weight gradient's tile, the
 * most rows of one of its pieces, and whether both gradients are computed in
 * one launch (by tiles of at most 64 x 128 then). aligned: the arrays start
 * on 16 bytes. */
typedef struct dmr_linear_plan {
    int32_t y_columns, y_rows, grad_x_columns, grad_x_rows, grad_weight_side, piece_rows, together;
} dmr_linear_plan;
dmr_status dmr_grouped_linear_plan(int64_t R, int64_t N, int32_t in_features, int32_t out_features, dmr_dtype dtype,
                                   int32_t aligned, dmr_linear_plan* out);

/*
 * Orthogonalised updates of B weight matrices (an optimiser's step for the
 * layers above): with U a matrix [m, n] of the batch,
 *     X_0 = U / (|U|_F + eps),  X_{k+1} = a X_k + (b A_k + c A_k A_k) X_k,
 *     A_k = X_k X_k^T (of the shorter side; X_k^T X_k gives the same),
 *     (a, b, c) = (3.4445, -4.7750, 2.0315),
 * `steps` times: the singular vectors of U with singular values pushed
 * towards 1 (within about 0.7 to 1.2 after five steps).
 *
 *   update, out [B, m, n] of dtype; out is overwritten and may not alias.
 *   steps      1..DMR_MAX_ORTHOGONALIZE_STEPS; eps finite and > 0.
 *   workspace  16-byte aligned, of dmr_orthogonalize_workspace_size() bytes.
 * Every type is computed to float32 accuracy and rounded once. A matrix of
 * zeros gives zeros; one with an infinity or NaN gives NaN throughout, and
 * leaves the others as they are.
 * Errors: negative sizes, sides below 1, missing pointers, an unknown dtype,
 * steps below 1, eps not > 0 and finite: DMR_ERROR_INVALID_VALUE; steps above
 * the limit, sides above DMR_MAX_LINEAR_WIDTH or beyond what a launch can
 * hold: DMR_ERROR_UNSUPPORTED. B == 0 launches nothing.
 */
#define DMR_MAX_ORTHOGONALIZE_STEPS 64
dmr_status dmr_orthogonalize(const void* update, int64_t B, int32_t m, int32_t n, dmr_dtype dtype, int32_t steps, float eps,
                             void* out, void* workspace, size_t workspace_bytes, hipStream_t stream);
/* The side of the tiles that X is computed by: 64, 128 or 256; 0: each matrix
 * by one workgroup; -1 on invalid arguments. For measurement and tests. */
int32_t dmr_orthogonalize_tile(int64_t B, int32_t m, int32_t n);
/* Workspace of dmr_orthogonalize in bytes; 0 on invalid arguments. */
size_t dmr_orthogonalize_workspace_size(int64_t B, int32_t m, int32_t n, dmr_dtype dtype);

/* What the last forward call on `workspace` recorded. Copies the workspace
 * header to the host and synchronises `stream`. */
typedef struct dmr_stats {
    int64_t required_bytes;   /* workspace that holds every bin list */
    int64_t bin_entries;      /* face entries over all bins */
    int64_t bin_capacity;     /* entries the given workspace could hold */
    int64_t bins;             /* number of bins (N * ceil(H/16) * ceil(W/16)) */
    int64_t overflow_bins;    /* bins rasterised from the full face range */
    int64_t live_faces;       /* faces that survived culling */
    uint32_t flags;           /* DMR_FLAG_* */
    uint32_t reserved;
} dmr_stats;
dmr_status dmr_workspace_stats(const void* workspace, dmr_stats* out, hipStream_t stream);

/* Static description of a status code; never NULL. */
const char* dmr_status_string(dmr_status s);

/*
 * Optional per-kernel timing for measurement. When enabled, every launch of
 * kernel `id` (0 .. dmr_kernel_count()-1) is bracketed with HIP events on
 * the stream it runs on; dmr_kernel_timing() synchronises on the recorded
 * events and returns the summed duration (ms) and number of launches since
 * the last reset. Disabled by default; timing is process-wide. Launches
 * from several host threads are recorded safely (the bookkeeping is
 * serialised), but a kernel launched concurrently on two streams pairs its
 * start and stop events per launch only when the launches do not overlap.
 */
int32_t dmr_kernel_count(void);
const char* dmr_kernel_name(int32_t id);
dmr_status dmr_set_kernel_timing(int32_t enable);
/* Times only the kernels whose id bit is set in mask (bit i = kernel i);
 * DMR_ERROR_INVALID_VALUE for bits at or above dmr_kernel_count(). */
dmr_status dmr_set_kernel_timing_mask(uint32_t mask);
dmr_status dmr_kernel_timing(int32_t id, double* total_ms, int64_t* launches);
dmr_status dmr_reset_kernel_timing(void);

#ifdef __cplusplus
}
#endif

#endif /* DMR_H */
