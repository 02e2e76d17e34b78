// C ABI of libdmr (include/dmr.h): host-side validation, workspace layout,
// launch sequencing and optional per-kernel event timing.
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "dmr_internal.h"

namespace dmr {

// ---------------------------------------------------------------------------
// per-kernel event timing
// ---------------------------------------------------------------------------
namespace {

struct Pending {
    hipEvent_t start, stop;
};

struct Timing {
    std::vector<Pending> pending[kKernelCount];
    std::vector<hipEvent_t> pool;
    double total_ms[kKernelCount] = {};
    int64_t launches[kKernelCount] = {};
    hipEvent_t open_start[kKernelCount] = {};
};

// The bookkeeping below is shared by every host thread that launches
// kernels: it is only touched under g_timing_mu. The mask (bit id set:
// kernel id is timed) is read without the lock on every launch.
Timing g_timing;
std::mutex g_timing_mu;
std::atomic<uint32_t> g_timing_mask{0};

const char* const kKernelNames[kKernelCount] = {
    "zero_fwd", "face_setup_count", "bin_scan", "bin_fill", "bin_sort", "fine_raster", "zero_grad", "backward_slots",
    "blend_fwd", "blend_bwd", "project_fwd", "project_bwd", "point_setup", "point_raster", "point_bwd",
    "grouped_linear_fwd", "grouped_linear_bwd", "orthogonalize", "grouped_layer_norm_fwd", "grouped_layer_norm_bwd",
    "clip_norm", "grouped_gated_linear_fwd", "grouped_gated_linear_bwd",
};

hipEvent_t take_event() {
    if (!g_timing.pool.empty()) {
        hipEvent_t e = g_timing.pool.back();
        g_timing.pool.pop_back();
        return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
}

hipError_t drain(int id) {
    for (auto& p : g_timing.pending[id]) {
        hipError_t err = hipEventSynchronize(p.stop);
        if (err != hipSuccess) return err;
        float ms = 0.0f;
        err = hipEventElapsedTime(&ms, p.start, p.stop);
        if (err != hipSuccess) return err;
        g_timing.total_ms[id] += ms;
        g_timing.launches[id] += 1;
        g_timing.pool.push_back(p.start);
        g_timing.pool.push_back(p.stop);
    }
    g_timing.pending[id].clear();
    return hipSuccess;
}

}  // namespace

void timing_begin(KernelId id, hipStream_t s) {
    if (!(g_timing_mask.load(std::memory_order_relaxed) >> id & 1u)) return;
    std::lock_guard<std::mutex> lk(g_timing_mu);
    hipEvent_t e = take_event();
    if (e && hipEventRecord(e, s) == hipSuccess) g_timing.open_start[id] = e;
}

void timing_end(KernelId id, hipStream_t s) {
    if (!(g_timing_mask.load(std::memory_order_relaxed) >> id & 1u)) return;
    std::lock_guard<std::mutex> lk(g_timing_mu);
    if (!g_timing.open_start[id]) return;
    hipEvent_t e = take_event();
    if (e && hipEventRecord(e, s) == hipSuccess) g_timing.pending[id].push_back({g_timing.open_start[id], e});
    g_timing.open_start[id] = nullptr;
}

}  // namespace dmr

using namespace dmr;

namespace {

bool mul_overflows(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return true;
    if (a != 0 && b > INT64_MAX / a) return true;
    *out = a * b;
    return false;
}

// Shared validation of the geometry arguments. Returns DMR_SUCCESS or the
// status to report.
dmr_status check_geometry(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                          const int64_t* off, int64_t N, int32_t H, int32_t W, int32_t K,
                          int64_t* slots_out) {
    if (V < 0 || F < 0 || N < 0) return DMR_ERROR_INVALID_VALUE;
    if (H < 1 || W < 1 || K < 1) return DMR_ERROR_INVALID_VALUE;
    if (H > DMR_MAX_IMAGE_SIDE || W > DMR_MAX_IMAGE_SIDE || K > DMR_MAX_K) return DMR_ERROR_UNSUPPORTED;
    if (F > (int64_t)INT32_MAX - 1) return DMR_ERROR_UNSUPPORTED;  // face ids are 32-bit inside
    if (V > INT64_MAX / 3) return DMR_ERROR_UNSUPPORTED;
    int64_t pix, slots, slots3;
    if (mul_overflows(N, (int64_t)H * W, &pix)) return DMR_ERROR_UNSUPPORTED;
    if (mul_overflows(pix, K, &slots)) return DMR_ERROR_UNSUPPORTED;
    if (mul_overflows(slots, 3, &slots3)) return DMR_ERROR_UNSUPPORTED;
    if (F > 0 && faces == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (V > 0 && verts == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (N > 0 && off == nullptr) return DMR_ERROR_INVALID_VALUE;
    *slots_out = slots;
    return DMR_SUCCESS;
}

}  // namespace

// The kernels read the workspace's per-face records and bin tables with
// 16-byte vector accesses at 256-byte aligned offsets from its start.
static bool ws_aligned(const void* workspace) {
    return (reinterpret_cast<uintptr_t>(workspace) & 15) == 0;
}

extern "C" {

const char* dmr_status_string(dmr_status s) {
    switch (s) {
        case DMR_SUCCESS: return "success";
        case DMR_ERROR_INVALID_VALUE: return "invalid argument";
        case DMR_ERROR_WORKSPACE_TOO_SMALL: return "workspace too small";
        case DMR_ERROR_HIP: return "HIP runtime error";
        case DMR_ERROR_UNSUPPORTED: return "unsupported size or parameter";
    }
    return "unknown status";
}

size_t dmr_workspace_min_size(int64_t N, int64_t F, int32_t H, int32_t W) {
    if (N < 0 || F < 0 || H < 1 || W < 1 || H > DMR_MAX_IMAGE_SIDE || W > DMR_MAX_IMAGE_SIDE) return 0;
    return fwd_layout(N, F, H, W).min_bytes;
}

size_t dmr_workspace_size_hint(int64_t N, int64_t F, int32_t H, int32_t W, int32_t K, float blur_radius) {
    (void)K;
    size_t base = dmr_workspace_min_size(N, F, H, W);
    if (base == 0 || !(blur_radius >= 0.0f) || !isfinite(blur_radius)) return 0;
    FwdLayout L = fwd_layout(N, F, H, W);
    // Face boxes grow by the blur radius (in pixels: sqrt(blur) * side / 2);
    // allow each face the bins of a box one blur diameter wider than a bin.
    double rpx = sqrt((double)blur_radius) * 0.5 * (double)(H > W ? H : W);
    double per_face = (1.0 + (2.0 * rpx + 2.0) / kBin) * (1.0 + (2.0 * rpx + 2.0) / kBin);
    double entries = 2.0 * per_face * (double)F + 4.0 * (double)L.bins + 1024.0;
    if (entries > (double)INT32_MAX) entries = (double)INT32_MAX;
    return align_up(base + (size_t)entries * sizeof(int32_t), 256);
}

dmr_status rasterize_meshes_fwd(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                const int64_t* mesh_face_offsets, int64_t N, int32_t H, int32_t W, int32_t K,
                                float blur_radius, int64_t* pix_to_face, float* zbuf, float* bary,
                                float* dists, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return rasterize_meshes_fwd_ex(verts, V, faces, F, mesh_face_offsets, N, H, W, K, blur_radius, pix_to_face, zbuf,
                                   bary, dists, workspace, workspace_bytes, 0u, stream);
}

dmr_status rasterize_meshes_fwd_ex(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                   const int64_t* mesh_face_offsets, int64_t N, int32_t H, int32_t W, int32_t K,
                                   float blur_radius, int64_t* pix_to_face, float* zbuf, float* bary,
                                   float* dists, void* workspace, size_t workspace_bytes, uint32_t flags,
                                   hipStream_t stream) {
    int64_t slots = 0;
    dmr_status st = check_geometry(verts, V, faces, F, mesh_face_offsets, N, H, W, K, &slots);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(blur_radius) || blur_radius < 0.0f) return DMR_ERROR_INVALID_VALUE;
    if ((flags & ~(uint32_t)DMR_RASTER_SETTINGS) != 0) return DMR_ERROR_INVALID_VALUE;
    if (slots == 0) return DMR_SUCCESS;
    if (!pix_to_face || !zbuf || !bary || !dists) return DMR_ERROR_INVALID_VALUE;
    FwdLayout L = fwd_layout(N, F, H, W);
    // work items of the fine pass are bin << 3 | part in 32 bits, four per bin at most
    if (L.bins >= ((int64_t)1 << 28)) return DMR_ERROR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < L.min_bytes) return DMR_ERROR_WORKSPACE_TOO_SMALL;
    if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    int64_t cap = (int64_t)((workspace_bytes - L.min_bytes) / sizeof(int32_t));
    if (cap > (int64_t)INT32_MAX) cap = INT32_MAX;

    FwdArgs a;
    a.verts = verts; a.V = V; a.faces = faces; a.F = F; a.off = mesh_face_offsets; a.N = N;
    a.H = H; a.W = W; a.K = K; a.blur = blur_radius; a.settings = flags;
    a.points = nullptr; a.radius = 0.0f;
    a.pix_to_face = pix_to_face; a.zbuf = zbuf; a.bary = bary; a.dists = dists;
    a.ws = static_cast<char*>(workspace); a.ws_bytes = workspace_bytes;
    a.L = L; a.capacity = cap; a.stream = stream;
    return launch_forward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// allocation-free forward: its workspace is a file-scope device array
// ---------------------------------------------------------------------------
// Every device the library runs on holds its own copy of `scratch` until the
// process ends. Host code never passes the array's name to a kernel or a
// copy (on the host it only stands for the symbol): the device address is
// looked up once per device with hipGetSymbolAddress and used from then on.
static __device__ __align__(256) unsigned char scratch[DMR_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxScratchDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxScratchDevices] = {};

// This device's `scratch`: the device of `stream` (the current device for
// the null stream), looked up on first use with that device current.
dmr_status scratch_for(hipStream_t stream, void** out) {
    int dev = 0;
    if (stream == nullptr) {
        if (hipGetDevice(&dev) != hipSuccess) return DMR_ERROR_HIP;
    } else if (hipStreamGetDevice(stream, &dev) != hipSuccess) {
        return DMR_ERROR_HIP;
    }
    if (dev < 0 || dev >= kMaxScratchDevices) return DMR_ERROR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        int cur = 0;
        if (hipGetDevice(&cur) != hipSuccess) return DMR_ERROR_HIP;
        if (cur != dev && hipSetDevice(dev) != hipSuccess) return DMR_ERROR_HIP;
        void* p = nullptr;
        const hipError_t err = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (cur != dev && hipSetDevice(cur) != hipSuccess) return DMR_ERROR_HIP;
        if (err != hipSuccess || p == nullptr) return DMR_ERROR_HIP;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return DMR_SUCCESS;
}

}  // namespace

extern "C" {

dmr_status rasterize_meshes_fwd_noalloc(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                        const int64_t* mesh_face_offsets, int64_t N, int32_t H, int32_t W,
                                        int32_t K, float blur_radius, int64_t* pix_to_face, float* zbuf, float* bary,
                                        float* dists, hipStream_t stream) {
    int64_t slots = 0;
    dmr_status st = check_geometry(verts, V, faces, F, mesh_face_offsets, N, H, W, K, &slots);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(blur_radius) || blur_radius < 0.0f) return DMR_ERROR_INVALID_VALUE;
    if (slots == 0) return DMR_SUCCESS;
    if (!pix_to_face || !zbuf || !bary || !dists) return DMR_ERROR_INVALID_VALUE;
    // face records and bin tables must fit; bin lists that do not fit take
    // the exact full-face-range path, as with any small workspace
    if (fwd_layout(N, F, H, W).min_bytes > (size_t)DMR_NOALLOC_SCRATCH_BYTES) return DMR_ERROR_UNSUPPORTED;
    void* ws = nullptr;
    st = scratch_for(stream, &ws);
    if (st != DMR_SUCCESS) return st;
    return rasterize_meshes_fwd_ex(verts, V, faces, F, mesh_face_offsets, N, H, W, K, blur_radius, pix_to_face,
                                   zbuf, bary, dists, ws, (size_t)DMR_NOALLOC_SCRATCH_BYTES, 0u, stream);
}

dmr_status rasterize_meshes_bwd(const float* verts, int64_t V, const int64_t* faces, int64_t F,
                                const int64_t* mesh_face_offsets, int64_t N, int32_t H, int32_t W, int32_t K,
                                float blur_radius, const int64_t* pix_to_face, const float* grad_zbuf,
                                const float* grad_bary, const float* grad_dists, float* grad_verts, void* workspace,
                                size_t workspace_bytes, uint32_t flags, hipStream_t stream) {
    int64_t slots = 0;
    dmr_status st = check_geometry(verts, V, faces, F, mesh_face_offsets, N, H, W, K, &slots);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(blur_radius) || blur_radius < 0.0f) return DMR_ERROR_INVALID_VALUE;
    if ((flags & ~(uint32_t)(DMR_BWD_REUSE_FORWARD_WORKSPACE | DMR_RASTER_SETTINGS)) != 0)
        return DMR_ERROR_INVALID_VALUE;
    if (V > 0 && grad_verts == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (slots > 0 && pix_to_face == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (V == 0) return DMR_SUCCESS;
    FwdLayout L = fwd_layout(N, F, H, W);
    if (L.bins >= ((int64_t)1 << 28)) return DMR_ERROR_UNSUPPORTED;  // as in the forward pass
    const bool reuse = (flags & DMR_BWD_REUSE_FORWARD_WORKSPACE) != 0;
    if (reuse && slots > 0 && (workspace == nullptr || workspace_bytes < L.min_bytes))
        return DMR_ERROR_WORKSPACE_TOO_SMALL;
    if (reuse && slots > 0 && !ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    int64_t cap = (reuse && slots > 0) ? (int64_t)((workspace_bytes - L.min_bytes) / sizeof(int32_t)) : 0;
    if (cap > (int64_t)INT32_MAX) cap = INT32_MAX;
    BwdArgs a;
    a.verts = verts; a.V = V; a.faces = faces; a.F = F; a.off = mesh_face_offsets; a.N = N;
    a.H = H; a.W = W; a.K = K; a.blur = blur_radius; a.settings = flags & DMR_RASTER_SETTINGS;
    a.pix_to_face = pix_to_face;
    a.gz = grad_zbuf; a.gb = grad_bary; a.gd = grad_dists; a.grad_verts = grad_verts;
    a.ws = static_cast<char*>(workspace); a.ws_bytes = workspace_bytes; a.L = L; a.capacity = cap;
    a.reuse_forward = reuse;
    a.stream = stream;
    return launch_backward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_blend(const int64_t* pix_to_face, const float* zbuf, const float* dists, int64_t P, int32_t K,
                       const float* colors, int64_t F, const dmr_blend_params* params) {
    if (P < 0 || F < 0 || K < 1 || params == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (K > DMR_MAX_K) return DMR_ERROR_UNSUPPORTED;
    // face indices are staged as int32; one 64-pixel workgroup per grid entry
    if (F > INT32_MAX || P > (int64_t)INT32_MAX * 64) return DMR_ERROR_UNSUPPORTED;
    int64_t slots = 0;
    if (mul_overflows(P, K, &slots) || slots > INT64_MAX / 3) return DMR_ERROR_UNSUPPORTED;
    const dmr_blend_params& p = *params;
    if (!(p.sigma > 0.0f) || !isfinite(p.sigma) || !(p.gamma > 0.0f) || !isfinite(p.gamma)) return DMR_ERROR_INVALID_VALUE;
    if (!isfinite(p.znear) || !isfinite(p.zfar) || !(p.zfar > p.znear) || !isfinite(p.eps)) return DMR_ERROR_INVALID_VALUE;
    for (int c = 0; c < 3; ++c)
        if (!isfinite(p.background[c])) return DMR_ERROR_INVALID_VALUE;
    if (P > 0 && (!pix_to_face || !zbuf || !dists)) return DMR_ERROR_INVALID_VALUE;
    if (F > 0 && !colors) return DMR_ERROR_INVALID_VALUE;
    return DMR_SUCCESS;
}

}  // namespace

dmr_status dmr_blend_fwd(const int64_t* pix_to_face, const float* zbuf, const float* dists, int64_t P, int32_t K,
                         const float* face_colors, int64_t F, const dmr_blend_params* params, float* rgba,
                         hipStream_t stream) {
    dmr_status st = check_blend(pix_to_face, zbuf, dists, P, K, face_colors, F, params);
    if (st != DMR_SUCCESS) return st;
    if (P == 0) return DMR_SUCCESS;
    if (!rgba || reinterpret_cast<uintptr_t>(rgba) % 16 != 0) return DMR_ERROR_INVALID_VALUE;
    BlendArgs a{};
    a.pix_to_face = pix_to_face; a.zbuf = zbuf; a.dists = dists; a.P = P; a.K = K;
    a.colors = face_colors; a.F = F; a.prm = *params; a.rgba = rgba; a.stream = stream;
    return launch_blend_forward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

dmr_status dmr_blend_bwd(const int64_t* pix_to_face, const float* zbuf, const float* dists, int64_t P, int32_t K,
                         const float* face_colors, int64_t F, const dmr_blend_params* params,
                         const float* grad_rgba, float* grad_zbuf, float* grad_dists, hipStream_t stream) {
    dmr_status st = check_blend(pix_to_face, zbuf, dists, P, K, face_colors, F, params);
    if (st != DMR_SUCCESS) return st;
    if (P == 0) return DMR_SUCCESS;
    if (!grad_rgba || !grad_zbuf || !grad_dists || reinterpret_cast<uintptr_t>(grad_rgba) % 16 != 0)
        return DMR_ERROR_INVALID_VALUE;
    BlendArgs a{};
    a.pix_to_face = pix_to_face; a.zbuf = zbuf; a.dists = dists; a.P = P; a.K = K;
    a.colors = face_colors; a.F = F; a.prm = *params; a.grad_rgba = grad_rgba; a.grad_zbuf = grad_zbuf;
    a.grad_dists = grad_dists; a.stream = stream;
    return launch_blend_backward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_project(const float* verts, int64_t V, const int64_t* off, int64_t N, const float* cameras) {
    if (V < 0 || N < 0) return DMR_ERROR_INVALID_VALUE;
    if (V > INT64_MAX / 3 || N > INT64_MAX / 16) return DMR_ERROR_UNSUPPORTED;
    // one 256-vertex workgroup per grid entry
    if (V > (int64_t)UINT32_MAX * 256) return DMR_ERROR_UNSUPPORTED;
    // the camera gradient takes 16 workgroups per mesh
    if (N > (int64_t)(UINT32_MAX / 16)) return DMR_ERROR_UNSUPPORTED;
    if (V > 0 && (N == 0 || !verts || !off || !cameras)) return DMR_ERROR_INVALID_VALUE;
    return DMR_SUCCESS;
}

}  // namespace

dmr_status dmr_project_fwd(const float* verts_world, int64_t V, const int64_t* mesh_vert_offsets, int64_t N,
                           const float* cameras, float* verts_ndc, hipStream_t stream) {
    dmr_status st = check_project(verts_world, V, mesh_vert_offsets, N, cameras);
    if (st != DMR_SUCCESS) return st;
    if (V == 0) return DMR_SUCCESS;
    if (!verts_ndc) return DMR_ERROR_INVALID_VALUE;
    ProjectArgs a{};
    a.verts = verts_world; a.V = V; a.off = mesh_vert_offsets; a.N = N; a.cameras = cameras; a.out = verts_ndc;
    a.stream = stream;
    return launch_project_forward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

dmr_status dmr_project_bwd(const float* verts_world, int64_t V, const int64_t* mesh_vert_offsets, int64_t N,
                           const float* cameras, const float* grad_verts_ndc, float* grad_verts_world,
                           float* grad_cameras, hipStream_t stream) {
    dmr_status st = check_project(verts_world, V, mesh_vert_offsets, N, cameras);
    if (st != DMR_SUCCESS) return st;
    if (V > 0 && (!grad_verts_ndc || !grad_verts_world)) return DMR_ERROR_INVALID_VALUE;
    if (V == 0 && (N == 0 || grad_cameras == nullptr)) return DMR_SUCCESS;
    ProjectArgs a{};
    a.verts = verts_world; a.V = V; a.off = mesh_vert_offsets; a.N = N; a.cameras = cameras;
    a.grad_out = grad_verts_ndc; a.grad_verts = grad_verts_world; a.grad_cameras = grad_cameras;
    a.stream = stream;
    return launch_project_backward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

size_t dmr_points_workspace_min_size(int64_t N, int64_t P, int32_t H, int32_t W) {
    if (N < 0 || P < 0 || H < 1 || W < 1 || H > DMR_MAX_IMAGE_SIDE || W > DMR_MAX_IMAGE_SIDE) return 0;
    return fwd_layout(N, P, H, W, sizeof(PointRec)).min_bytes;
}

size_t dmr_points_workspace_size_hint(int64_t N, int64_t P, int32_t H, int32_t W, int32_t K, float radius) {
    (void)K;
    size_t base = dmr_points_workspace_min_size(N, P, H, W);
    if (base == 0 || !(radius >= 0.0f) || !isfinite(radius)) return 0;
    FwdLayout L = fwd_layout(N, P, H, W, sizeof(PointRec));
    // a point's box is 2 radius wide: the bins of a box one bin wider than that
    double rpx = (double)radius * 0.5 * (double)(H > W ? H : W);
    double per_point = (1.0 + (2.0 * rpx + 2.0) / kBin) * (1.0 + (2.0 * rpx + 2.0) / kBin);
    double entries = 2.0 * per_point * (double)P + 4.0 * (double)L.bins + 1024.0;
    if (entries > (double)INT32_MAX) entries = (double)INT32_MAX;
    return align_up(base + (size_t)entries * sizeof(int32_t), 256);
}

namespace {

dmr_status check_points(const float* points, int64_t P, const int64_t* off, int64_t N, int32_t H, int32_t W,
                        int32_t K, int64_t* slots_out) {
    if (P < 0 || N < 0 || H < 1 || W < 1 || K < 1) return DMR_ERROR_INVALID_VALUE;
    if (H > DMR_MAX_IMAGE_SIDE || W > DMR_MAX_IMAGE_SIDE || K > DMR_MAX_K) return DMR_ERROR_UNSUPPORTED;
    if (P > (int64_t)INT32_MAX - 1) return DMR_ERROR_UNSUPPORTED;   // point ids are 32-bit inside
    int64_t pix, slots;
    if (mul_overflows(N, (int64_t)H * W, &pix) || mul_overflows(pix, K, &slots)) return DMR_ERROR_UNSUPPORTED;
    if (slots > (int64_t)UINT32_MAX * 256) return DMR_ERROR_UNSUPPORTED;
    if (P > 0 && points == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (N > 0 && off == nullptr) return DMR_ERROR_INVALID_VALUE;
    *slots_out = slots;
    return DMR_SUCCESS;
}

}  // namespace

dmr_status rasterize_points_fwd(const float* points, int64_t P, const int64_t* cloud_offsets, int64_t N, int32_t H,
                                int32_t W, int32_t K, float radius, int64_t* idx, float* zbuf, float* dists,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int64_t slots = 0;
    dmr_status st = check_points(points, P, cloud_offsets, N, H, W, K, &slots);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(radius) || radius < 0.0f) return DMR_ERROR_INVALID_VALUE;
    if (slots == 0) return DMR_SUCCESS;
    if (!idx || !zbuf || !dists) return DMR_ERROR_INVALID_VALUE;
    FwdLayout L = fwd_layout(N, P, H, W, sizeof(PointRec));
    if (L.bins >= ((int64_t)1 << 28)) return DMR_ERROR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < L.min_bytes) return DMR_ERROR_WORKSPACE_TOO_SMALL;
    if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    int64_t cap = (int64_t)((workspace_bytes - L.min_bytes) / sizeof(int32_t));
    if (cap > (int64_t)INT32_MAX) cap = INT32_MAX;
    FwdArgs a{};
    a.verts = nullptr; a.V = 0; a.faces = nullptr; a.F = P; a.off = cloud_offsets; a.N = N;
    a.H = H; a.W = W; a.K = K; a.blur = 0.0f; a.settings = 0u;
    a.points = points; a.radius = radius;
    a.pix_to_face = idx; a.zbuf = zbuf; a.bary = nullptr; a.dists = dists;
    a.ws = static_cast<char*>(workspace); a.ws_bytes = workspace_bytes;
    a.L = L; a.capacity = cap; a.stream = stream;
    return launch_points_forward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

dmr_status rasterize_points_bwd(const float* points, int64_t P, const int64_t* cloud_offsets, int64_t N, int32_t H,
                                int32_t W, int32_t K, const int64_t* idx, const float* grad_zbuf,
                                const float* grad_dists, float* grad_points, hipStream_t stream) {
    int64_t slots = 0;
    dmr_status st = check_points(points, P, cloud_offsets, N, H, W, K, &slots);
    if (st != DMR_SUCCESS) return st;
    if (P > 0 && grad_points == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (slots > 0 && idx == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (P == 0) return DMR_SUCCESS;
    if (fwd_layout(N, P, H, W, sizeof(PointRec)).bins >= ((int64_t)1 << 28)) return DMR_ERROR_UNSUPPORTED;
    PointBwdArgs a{};
    a.points = points; a.P = P; a.N = N; a.H = H; a.W = W; a.K = K;
    a.idx = idx; a.gz = grad_zbuf; a.gd = grad_dists; a.grad_points = grad_points; a.stream = stream;
    return launch_points_backward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_grouped(int64_t R, int32_t cin, int64_t N, int32_t cout, dmr_dtype dtype, const int64_t* off) {
    if (R < 0 || N < 0 || cin < 1 || cout < 1) return DMR_ERROR_INVALID_VALUE;
    if (dtype != DMR_FLOAT32 && dtype != DMR_FLOAT16 && dtype != DMR_BFLOAT16) return DMR_ERROR_INVALID_VALUE;
    if (cin > DMR_MAX_LINEAR_WIDTH || cout > DMR_MAX_LINEAR_WIDTH) return DMR_ERROR_UNSUPPORTED;
    // tiles are counted in 32 bits (at least 16 rows a tile, and one for each group)
    const int64_t columns = (int64_t)(cin > cout ? cin : cout) / 16 + 1;
    const int64_t weight_tiles = ((int64_t)cin / 32 + 1) * ((int64_t)cout / 32 + 1);
    const int64_t most = (int64_t)INT32_MAX - 1024;
    if (R > INT64_MAX / ((int64_t)DMR_MAX_LINEAR_WIDTH * 4)) return DMR_ERROR_UNSUPPORTED;
    if (N > most / 64 || N > most / columns || N > most / weight_tiles) return DMR_ERROR_UNSUPPORTED;
    if (R / 16 + N > most / columns || R / 512 + N > most / weight_tiles) return DMR_ERROR_UNSUPPORTED;
    if (N > 0 && off == nullptr) return DMR_ERROR_INVALID_VALUE;
    if (R > 0 && N == 0) return DMR_ERROR_INVALID_VALUE;
    return DMR_SUCCESS;
}

}  // namespace

dmr_status dmr_grouped_linear_fwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                  const void* weight, const void* bias, int32_t out_features, dmr_dtype dtype, void* y,
                                  hipStream_t stream) {
    dmr_status st = check_grouped(R, in_features, N, out_features, dtype, row_offsets);
    if (st != DMR_SUCCESS) return st;
    if (R == 0) return DMR_SUCCESS;
    if (!x || !weight || !y) return DMR_ERROR_INVALID_VALUE;
    GroupedLinearArgs a{};
    a.x = x; a.R = R; a.cin = in_features; a.off = row_offsets; a.N = N; a.weight = weight; a.bias = bias;
    a.cout = out_features; a.dtype = dtype; a.y = y; a.stream = stream;
    return launch_grouped_linear_forward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

size_t dmr_grouped_linear_workspace_size(int64_t R, int64_t N, int32_t in_features, int32_t out_features, dmr_dtype dtype) {
    static const int64_t none = 0;
    if (check_grouped(R, in_features, N, out_features, dtype, &none) != DMR_SUCCESS ||
        !grouped_sums_fit(R, N, in_features, out_features, dtype != DMR_FLOAT32))
        return 0;
    const int64_t slots = grouped_pieces(R, N, in_features, out_features, dtype != DMR_FLOAT32).slots;
    return align_up((size_t)(slots * grouped_piece_values(in_features, out_features)) * sizeof(float) + 256, 256);
}

dmr_status dmr_grouped_linear_plan(int64_t R, int64_t N, int32_t in_features, int32_t out_features, dmr_dtype dtype,
                                   int32_t aligned, dmr_linear_plan* out) {
    static const int64_t none = 0;
    if (out == nullptr) return DMR_ERROR_INVALID_VALUE;
    const dmr_status st = check_grouped(R, in_features, N, out_features, dtype, &none);
    if (st != DMR_SUCCESS) return st;
    const bool half = dtype != DMR_FLOAT32;
    const int whole = half ? 8 : 4;
    const bool vec = aligned && in_features % whole == 0 && out_features % whole == 0;
    const RowsTile y = grouped_rows_tile(R, N, out_features, half, false, aligned && in_features % whole == 0);
    const RowsTile gx = grouped_rows_tile(R, N, in_features, half, true, vec);
    const GroupedPieces p = grouped_pieces(R, N, in_features, out_features, half);
    *out = {y.columns, y.rows, gx.columns, gx.rows, grouped_weight_side(p, vec), p.rows,
            grouped_together(R, N, in_features, out_features, half)};
    return DMR_SUCCESS;
}

dmr_status dmr_grouped_linear_bwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                  const void* weight, int32_t out_features, dmr_dtype dtype, const void* grad_y,
                                  void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
    dmr_status st = check_grouped(R, in_features, N, out_features, dtype, row_offsets);
    if (st != DMR_SUCCESS) return st;
    const bool sums = grad_weight || grad_bias;
    if (R > 0 && !grad_y) return DMR_ERROR_INVALID_VALUE;
    if (R > 0 && ((grad_x && !weight) || (sums && !x))) return DMR_ERROR_INVALID_VALUE;
    if (N == 0 || !(grad_x || sums)) return DMR_SUCCESS;
    if (sums) {
        if (!grouped_sums_fit(R, N, in_features, out_features, dtype != DMR_FLOAT32)) return DMR_ERROR_UNSUPPORTED;
        if (workspace == nullptr ||
            workspace_bytes < dmr_grouped_linear_workspace_size(R, N, in_features, out_features, dtype))
            return DMR_ERROR_WORKSPACE_TOO_SMALL;
        if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    }
    GroupedLinearArgs a{};
    a.x = x; a.R = R; a.cin = in_features; a.off = row_offsets; a.N = N; a.weight = weight; a.cout = out_features;
    a.dtype = dtype; a.grad_y = grad_y; a.grad_x = grad_x; a.grad_weight = grad_weight; a.grad_bias = grad_bias;
    a.workspace = static_cast<float*>(workspace); a.stream = stream;
    return launch_grouped_linear_backward(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_orthogonalize(int64_t B, int32_t m, int32_t n, dmr_dtype dtype) {
    if (B < 0 || m < 1 || n < 1) return DMR_ERROR_INVALID_VALUE;
    if (dtype != DMR_FLOAT32 && dtype != DMR_FLOAT16 && dtype != DMR_BFLOAT16) return DMR_ERROR_INVALID_VALUE;
    if (m > DMR_MAX_LINEAR_WIDTH || n > DMR_MAX_LINEAR_WIDTH) return DMR_ERROR_UNSUPPORTED;
    if (B > 0 && orthogonalize_workspace(B, m, n) == 0) return DMR_ERROR_UNSUPPORTED;
    return DMR_SUCCESS;
}

}  // namespace

size_t dmr_orthogonalize_workspace_size(int64_t B, int32_t m, int32_t n, dmr_dtype dtype) {
    if (check_orthogonalize(B, m, n, dtype) != DMR_SUCCESS) return 0;
    return B > 0 ? orthogonalize_workspace(B, m, n) : 256;
}

int32_t dmr_orthogonalize_tile(int64_t B, int32_t m, int32_t n) {
    if (B < 1 || check_orthogonalize(B, m, n, DMR_FLOAT32) != DMR_SUCCESS) return -1;
    return orthogonalize_tile(B, m, n);
}

dmr_status dmr_orthogonalize(const void* update, int64_t B, int32_t m, int32_t n, dmr_dtype dtype, int32_t steps, float eps,
                             void* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    dmr_status st = check_orthogonalize(B, m, n, dtype);
    if (st != DMR_SUCCESS) return st;
    if (steps < 1 || !isfinite(eps) || !(eps > 0.0f)) return DMR_ERROR_INVALID_VALUE;
    if (steps > DMR_MAX_ORTHOGONALIZE_STEPS) return DMR_ERROR_UNSUPPORTED;
    if (B == 0) return DMR_SUCCESS;
    if (!update || !out) return DMR_ERROR_INVALID_VALUE;
    if (workspace == nullptr || workspace_bytes < orthogonalize_workspace(B, m, n))
        return DMR_ERROR_WORKSPACE_TOO_SMALL;
    if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    OrthogonalizeArgs a{};
    a.update = update; a.B = B; a.m = m; a.n = n; a.dtype = dtype; a.steps = steps; a.eps = eps; a.out = out;
    a.workspace = static_cast<char*>(workspace); a.stream = stream;
    return launch_orthogonalize(a) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_layer_norm(int64_t R, int32_t C, int64_t N, dmr_dtype dtype) {
    if (R < 0 || N < 0 || C < 1) return DMR_ERROR_INVALID_VALUE;
    if (dtype != DMR_FLOAT32 && dtype != DMR_FLOAT16 && dtype != DMR_BFLOAT16) return DMR_ERROR_INVALID_VALUE;
    if (C > DMR_MAX_LINEAR_WIDTH) return DMR_ERROR_UNSUPPORTED;
    if (R > INT64_MAX / ((int64_t)DMR_MAX_LINEAR_WIDTH * 64)) return DMR_ERROR_UNSUPPORTED;
    // the sums over rows take a workgroup of 1024 for each group and 64 of its values
    if (N > kMaxWorkItems / 1024 / (2 * (int64_t)C / 64 + 1)) return DMR_ERROR_UNSUPPORTED;
    if (R > 0 && N == 0) return DMR_ERROR_INVALID_VALUE;
    return DMR_SUCCESS;
}

}  // namespace

dmr_status dmr_grouped_layer_norm_fwd(const void* x, int64_t R, int32_t features, const int64_t* row_offsets, int64_t N,
                                      const void* weight, const void* bias, float eps, dmr_dtype dtype, void* y,
                                      hipStream_t stream) {
    dmr_status st = check_layer_norm(R, features, N, dtype);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(eps) || !(eps > 0.0f) || (N > 0 && row_offsets == nullptr)) return DMR_ERROR_INVALID_VALUE;
    if (R == 0) return DMR_SUCCESS;
    if (!x || !y) return DMR_ERROR_INVALID_VALUE;
    LayerNormArgs a{};
    a.x = x; a.R = R; a.C = features; a.off = row_offsets; a.N = N; a.weight = weight; a.bias = bias; a.eps = eps;
    a.dtype = dtype; a.y = y; a.stream = stream;
    return launch_layer_norm(a, false) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

size_t dmr_grouped_layer_norm_workspace_size(int64_t R, int64_t N, int32_t features, dmr_dtype dtype) {
    if (check_layer_norm(R, features, N, dtype) != DMR_SUCCESS) return 0;
    return align_up(layer_norm_plan(R, N, features, dtype != DMR_FLOAT32, true).workspace + 256, 256);
}

dmr_status dmr_grouped_layer_norm_bwd(const void* x, int64_t R, int32_t features, const int64_t* row_offsets, int64_t N,
                                      const void* weight, float eps, dmr_dtype dtype, const void* grad_y, void* grad_x,
                                      void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    dmr_status st = check_layer_norm(R, features, N, dtype);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(eps) || !(eps > 0.0f) || (N > 0 && row_offsets == nullptr)) return DMR_ERROR_INVALID_VALUE;
    const bool sums = grad_weight || grad_bias;
    if (R > 0 && (!x || !grad_y)) return DMR_ERROR_INVALID_VALUE;
    if (N == 0 || !(grad_x || sums) || (R == 0 && !sums)) return DMR_SUCCESS;
    if (sums) {
        if (workspace == nullptr || workspace_bytes < dmr_grouped_layer_norm_workspace_size(R, N, features, dtype))
            return DMR_ERROR_WORKSPACE_TOO_SMALL;
        if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    }
    LayerNormArgs a{};
    a.x = x; a.R = R; a.C = features; a.off = row_offsets; a.N = N; a.weight = weight; a.eps = eps; a.dtype = dtype;
    a.grad_y = grad_y; a.grad_x = grad_x; a.grad_weight = grad_weight; a.grad_bias = grad_bias;
    a.workspace = static_cast<float*>(workspace); a.stream = stream;
    return launch_layer_norm(a, true) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

// Also as a linear layer of 2 F outputs, which the backward pass is.
dmr_status check_gated(int64_t R, int32_t C, int64_t N, int32_t F, int32_t act, dmr_dtype dtype, const int64_t* off) {
    if (F < 1 || act < DMR_SILU || act > DMR_SIGMOID) return DMR_ERROR_INVALID_VALUE;
    if (F > DMR_MAX_LINEAR_WIDTH / 2) return DMR_ERROR_UNSUPPORTED;
    return check_grouped(R, C, N, 2 * F, dtype, off);
}

}  // namespace

dmr_status dmr_grouped_gated_linear_fwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                        const void* weight, const void* bias, int32_t out_features, dmr_activation activation,
                                        dmr_dtype dtype, void* y, hipStream_t stream) {
    const dmr_status st = check_gated(R, in_features, N, out_features, activation, dtype, row_offsets);
    if (st != DMR_SUCCESS) return st;
    if (R == 0) return DMR_SUCCESS;
    if (!x || !weight || !y) return DMR_ERROR_INVALID_VALUE;
    GatedArgs a{};
    a.x = x; a.R = R; a.C = in_features; a.off = row_offsets; a.N = N; a.weight = weight; a.bias = bias; a.F = out_features;
    a.act = activation; a.dtype = dtype; a.y = y; a.stream = stream;
    return launch_gated(a, false) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

size_t dmr_grouped_gated_linear_workspace_size(int64_t R, int64_t N, int32_t in_features, int32_t out_features,
                                               dmr_dtype dtype) {
    static const int64_t none = 0;
    if (check_gated(R, in_features, N, out_features, DMR_SILU, dtype, &none) != DMR_SUCCESS) return 0;
    if (!gated_fits(R, N, in_features, out_features, dtype != DMR_FLOAT32)) return 0;
    return gated_workspace(R, N, in_features, out_features, dtype);
}

dmr_status dmr_grouped_gated_linear_plan(int64_t R, int64_t N, int32_t in_features, int32_t out_features, dmr_dtype dtype,
                                         int32_t aligned, dmr_gated_plan* out) {
    static const int64_t none = 0;
    if (out == nullptr) return DMR_ERROR_INVALID_VALUE;
    const dmr_status st = check_gated(R, in_features, N, out_features, DMR_SILU, dtype, &none);
    if (st != DMR_SUCCESS) return st;
    const bool half = dtype != DMR_FLOAT32;
    const RowsTile t = gated_tile(R, N, out_features, half, aligned && in_features % (half ? 8 : 4) == 0);
    const GroupedPieces p = gated_pieces(R, N, in_features, out_features, half);
    *out = {t.columns, t.rows, gated_narrow(in_features, out_features), p.rows};
    return DMR_SUCCESS;
}

dmr_status dmr_grouped_gated_linear_bwd(const void* x, int64_t R, int32_t in_features, const int64_t* row_offsets, int64_t N,
                                        const void* weight, const void* bias, int32_t out_features, dmr_activation activation,
                                        dmr_dtype dtype, const void* grad_y, void* grad_x, void* grad_weight, void* grad_bias,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const dmr_status st = check_gated(R, in_features, N, out_features, activation, dtype, row_offsets);
    if (st != DMR_SUCCESS) return st;
    const bool sums = grad_weight || grad_bias;
    if (R > 0 && (!x || !weight || !grad_y)) return DMR_ERROR_INVALID_VALUE;
    if (N == 0 || !(grad_x || sums) || (R == 0 && !sums)) return DMR_SUCCESS;
    if (!gated_fits(R, N, in_features, out_features, dtype != DMR_FLOAT32)) return DMR_ERROR_UNSUPPORTED;
    if (workspace == nullptr ||
        workspace_bytes < dmr_grouped_gated_linear_workspace_size(R, N, in_features, out_features, dtype))
        return DMR_ERROR_WORKSPACE_TOO_SMALL;
    if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    GatedArgs a{};
    a.x = x; a.R = R; a.C = in_features; a.off = row_offsets; a.N = N; a.weight = weight; a.bias = bias; a.F = out_features;
    a.act = activation; a.dtype = dtype; a.grad_y = grad_y; a.grad_x = grad_x; a.grad_weight = grad_weight;
    a.grad_bias = grad_bias; a.workspace = static_cast<char*>(workspace); a.stream = stream;
    return launch_gated(a, true) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

namespace {

dmr_status check_clip(const dmr_tensor_span* tensors, int32_t count, int64_t groups, ClipPlan* plan) {
    if (count < 0 || groups < 0 || (count > 0 && tensors == nullptr)) return DMR_ERROR_INVALID_VALUE;
    int64_t all = 0;
    for (int32_t k = 0; k < count; ++k) {
        const dmr_dtype t = tensors[k].dtype;
        if (tensors[k].values < 0 || (t != DMR_FLOAT32 && t != DMR_FLOAT16 && t != DMR_BFLOAT16)) return DMR_ERROR_INVALID_VALUE;
        if (tensors[k].values > (INT64_MAX / 8 - all) / (groups > 0 ? groups : 1)) return DMR_ERROR_UNSUPPORTED;
        all += tensors[k].values * groups;
    }
    *plan = clip_plan(tensors, count, groups);
    return plan->fits ? DMR_SUCCESS : DMR_ERROR_UNSUPPORTED;
}

size_t clip_workspace(const ClipPlan& p, int64_t groups) {
    return align_up((p.small ? 0 : (size_t)(p.chunks * groups) * sizeof(double)) + 256, 256);
}

}  // namespace

size_t dmr_clip_norm_workspace_size(const dmr_tensor_span* tensors, int32_t count, int64_t groups) {
    ClipPlan p{};
    return check_clip(tensors, count, groups, &p) == DMR_SUCCESS ? clip_workspace(p, groups) : 0;
}

dmr_status dmr_clip_norm(const dmr_tensor_span* tensors, int32_t count, int64_t groups, float max_norm, float eps,
                         float* norms, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    ClipPlan p{};
    const dmr_status st = check_clip(tensors, count, groups, &p);
    if (st != DMR_SUCCESS) return st;
    if (!isfinite(max_norm) || !(max_norm >= 0.0f) || !isfinite(eps) || !(eps >= 0.0f)) return DMR_ERROR_INVALID_VALUE;
    if (groups == 0) return DMR_SUCCESS;
    if (norms == nullptr) return DMR_ERROR_INVALID_VALUE;
    for (int32_t k = 0; k < count; ++k)
        if (tensors[k].values > 0 && (!tensors[k].in || !tensors[k].out)) return DMR_ERROR_INVALID_VALUE;
    if (!p.small) {
        if (workspace == nullptr || workspace_bytes < clip_workspace(p, groups)) return DMR_ERROR_WORKSPACE_TOO_SMALL;
        if (!ws_aligned(workspace)) return DMR_ERROR_INVALID_VALUE;
    }
    ClipArgs a{};
    a.tensors = tensors; a.count = count; a.groups = groups; a.max_norm = max_norm; a.eps = eps; a.norms = norms;
    a.workspace = static_cast<double*>(workspace); a.stream = stream;
    return launch_clip(a, p) == hipSuccess ? DMR_SUCCESS : DMR_ERROR_HIP;
}

dmr_status dmr_workspace_stats(const void* workspace, dmr_stats* out, hipStream_t stream) {
    if (workspace == nullptr || out == nullptr) return DMR_ERROR_INVALID_VALUE;
    WsHeader h;
    if (hipMemcpyAsync(&h, workspace, sizeof(h), hipMemcpyDeviceToHost, stream) != hipSuccess)
        return DMR_ERROR_HIP;
    if (hipStreamSynchronize(stream) != hipSuccess) return DMR_ERROR_HIP;
    out->required_bytes = h.required_bytes;
    out->bin_entries = h.bin_entries;
    out->bin_capacity = h.bin_capacity;
    out->bins = h.bins;
    out->overflow_bins = h.overflow_bins;
    out->live_faces = h.live_faces;
    out->flags = h.flags;
    out->reserved = 0;
    return DMR_SUCCESS;
}

int32_t dmr_kernel_count(void) { return kKernelCount; }

const char* dmr_kernel_name(int32_t id) {
    if (id < 0 || id >= kKernelCount) return "";
    return kKernelNames[id];
}

dmr_status dmr_set_kernel_timing(int32_t enable) {
    std::lock_guard<std::mutex> lk(g_timing_mu);
    g_timing_mask.store(enable != 0 ? (1u << kKernelCount) - 1u : 0u);
    return DMR_SUCCESS;
}

dmr_status dmr_set_kernel_timing_mask(uint32_t mask) {
    if (mask >> kKernelCount) return DMR_ERROR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_timing_mu);
    g_timing_mask.store(mask);
    return DMR_SUCCESS;
}

dmr_status dmr_kernel_timing(int32_t id, double* total_ms, int64_t* launches) {
    if (id < 0 || id >= kKernelCount || !total_ms || !launches) return DMR_ERROR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_timing_mu);
    if (drain(id) != hipSuccess) return DMR_ERROR_HIP;
    *total_ms = g_timing.total_ms[id];
    *launches = g_timing.launches[id];
    return DMR_SUCCESS;
}

dmr_status dmr_reset_kernel_timing(void) {
    std::lock_guard<std::mutex> lk(g_timing_mu);
    for (int id = 0; id < kKernelCount; ++id) {
        if (drain(id) != hipSuccess) return DMR_ERROR_HIP;
        g_timing.total_ms[id] = 0.0;
        g_timing.launches[id] = 0;
    }
    return DMR_SUCCESS;
}

}  // extern "C"
