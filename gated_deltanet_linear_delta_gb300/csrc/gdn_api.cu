// gdn_api.cu -- the exported C ABI: argument checks, the device status word,
// and dispatch to the kernels. Every check runs before any device work is
// queued; a failed check returns its gdn_status and touches nothing.
#include <stdint.h>

#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "gdn.h"
#include "gdn_internal.h"

namespace {

// Device-side consistency flag, one per device (a __device__ variable has one
// instance per device context). Kernels set it with atomicExch; the host reads
// and clears it in gdn_get_device_status.
__device__ int g_device_status = 0;
__device__ int g_status_taken = 0;  // where the read-and-clear kernel leaves the old value

// Read and clear the status word in one atomic step, so a flag raised by a kernel on another
// stream between a read and a separate clear cannot be lost.
__global__ void take_status_kernel(int *status, int *taken) { *taken = atomicExch(status, 0); }

constexpr int kMaxDevices = 64;
int *g_status_ptr[kMaxDevices] = {nullptr};
int *g_taken_ptr[kMaxDevices] = {nullptr};

std::mutex g_status_mu;  // first use on a device may come from several host threads

int *status_ptr() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_status_mu);
    if (!g_status_ptr[dev]) {
        void *p = nullptr, *t = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
        if (cudaGetSymbolAddress(&t, g_status_taken) != cudaSuccess) return nullptr;
        g_taken_ptr[dev] = static_cast<int *>(t);
        g_status_ptr[dev] = static_cast<int *>(p);
    }
    return g_status_ptr[dev];
}

int *taken_ptr() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    if (!status_ptr()) return nullptr;
    std::lock_guard<std::mutex> lock(g_status_mu);
    return g_taken_ptr[dev];
}

// gdn_prefill's own workspace for the kernels that need one: one per device, allocated on the
// first call that needs it (and grown when a call needs more). Calls on different streams are
// ordered on the GPU through an event, so they never use it at the same time; inside a stream
// capture the workspace must already be large enough (no allocation, no cross-stream wait).
struct DeviceWorkspace {
    std::mutex mu;
    void *ptr = nullptr;
    size_t bytes = 0;
    cudaEvent_t last = nullptr;   // recorded after the last call that used the workspace
    cudaStream_t last_stream = nullptr;
    bool used = false;
};
DeviceWorkspace g_ws[kMaxDevices];

bool stream_capturing(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) return true;
    return st != cudaStreamCaptureStatusNone;
}

bool force_cluster_kernel() {
    const char *env = getenv("GDN_PREFILL_KERNEL");
    return env && strcmp(env, "cluster") == 0;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool chunk_ok(int c) { return c == 16 || c == 32 || c == 64; }

int common_checks(int Hk, int Hv, int dk, int dv, int dtype) {
    if (Hk <= 0 || Hv <= 0 || Hv % Hk != 0 || Hv > 65535) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    if (!dim_ok(dk) || !dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int prefill_checks(const void *q, const void *k, const void *v, const void *g, const void *b,
                   const float *state_in, const float *state_out, const void *out,
                   const int32_t *cu, int B, int T, int Hk, int Hv, int dk, int dv, int chunk,
                   int dtype) {
    if (B < 0 || T < 0 || B > 65535) return GDN_ERR_INVALID_ARG;
    int rc = common_checks(Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK) return rc;
    if (!chunk_ok(chunk)) return GDN_ERR_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    const long long Ttot = cu ? (long long)T : (long long)B * T;
    if (Ttot > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if (!state_out) return GDN_ERR_INVALID_ARG;
    if (Ttot > 0 && (!q || !k || !v || !g || !b || !out)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, b, state_in, state_out, out, cu};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// What the three paged cache calls share. Sizes first (a call with no tokens touches no pointer),
// then the pointers that every call reads.
int kv_checks(int B, int T, const int32_t *cu, int Hq, int Hkv, int d, int num_pages, int page_size, int max_pages,
              int dtype, int cache_dtype, int64_t stride_a, int64_t stride_b) {
    if (B < 0 || T < 0 || B > 65535 || num_pages < 0 || max_pages < 0) return GDN_ERR_INVALID_ARG;
    if (Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || Hq > 65535) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    if (cache_dtype != dtype && cache_dtype != GDN_FP8 && cache_dtype != GDN_INT8) return GDN_ERR_UNSUPPORTED;
    if (d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return GDN_ERR_UNSUPPORTED;
    if (Hq / Hkv > 64) return GDN_ERR_UNSUPPORTED;
    const long long Ttot = cu ? (long long)T : (long long)B * T;
    if (Ttot * Hq > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv > 0x7fffffffLL || (long long)max_pages * page_size > (1LL << 30))
        return GDN_ERR_INVALID_ARG;
    const int64_t vec = dtype == GDN_BF16 ? 8 : 4;  // 16 bytes
    if (stride_a < (int64_t)Hq * d || stride_a % vec || stride_b < (int64_t)Hkv * d || stride_b % vec)
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

int kv_pointers(const void *k_cache, const void *v_cache, const void *k_scale, const void *v_scale,
                const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu, int num_pages, int max_pages,
                int dtype, int cache_dtype, const void *a, const void *b) {
    const bool codes = cache_dtype != dtype;
    if (!a || !b || !aligned16(a) || !aligned16(b)) return GDN_ERR_INVALID_ARG;
    // lengths and tables may be slices of a larger batch's
    if (!kv_lens || ((reinterpret_cast<uintptr_t>(kv_lens) | reinterpret_cast<uintptr_t>(block_table)) & 3u))
        return GDN_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_cache || !v_cache || (codes && (!k_scale || !v_scale)))) return GDN_ERR_INVALID_ARG;
    if (max_pages > 0 && !block_table) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {k_cache, v_cache, k_scale, v_scale, cu};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn::KvPages kv_pages(const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu, int B, int T, int Hkv,
                      int d, int num_pages, int page_size, int max_pages, int dtype, int cache_dtype, int *status) {
    gdn::KvPages p{};
    p.table = block_table;
    p.kv_lens = kv_lens;
    p.cu = cu;
    p.B = B;
    p.T = T;
    p.Ttot = cu ? (long)T : (long)B * T;
    p.Hkv = Hkv;
    p.d = d;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.dtype = dtype;
    p.cache_dtype = cache_dtype;
    p.status = status;
    return p;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sequences of a call on trees: nodes per sequence (or packed), and the accepted paths' rows where there are any.
int tree_checks(int B, int T, const int32_t *cu, const int32_t *a, const int32_t *b, const int32_t *c) {
    if (B < 0 || T < 0 || B > 65535) return GDN_ERR_INVALID_ARG;
    if (!cu && T > gdn::kTreeMax) return GDN_ERR_UNSUPPORTED;
    if (!aligned16(cu) || !aligned4(a) || !aligned4(b) || !aligned4(c)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// The states of a call on trees (in and out the same where they are only read), if any are used.
int state_checks(bool used, const float *in, const float *out, const int32_t *slots, int B, int T, const int32_t *cu, int num_slots,
                 int Hk, int Hv, int dk, int dv, int dtype) {
    const int rc = common_checks(Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK) return rc;
    const long long states = slots ? (long long)num_slots : (long long)B;
    if (num_slots < 0 || states * Hv * dv * dk > (1LL << 40)) return GDN_ERR_INVALID_ARG;
    if ((long long)B * Hv > 0x7fffffffLL || (cu ? (long long)T : (long long)B * T) > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if (B > 0 && states > 0 && used && (!in || !out || !aligned16(in) || !aligned16(out))) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

void tree_sizes(gdn::TreeArgs &a, const int32_t *cu, int B, int T, int num_slots, int Hk, int Hv, int dk, int dv, int dtype,
                int *status) {
    a.cu = cu;
    a.B = B;
    a.T = T;
    a.Ttot = cu ? (long)T : (long)B * T;
    a.num_slots = num_slots;
    a.Hk = Hk;
    a.Hv = Hv;
    a.dk = dk;
    a.dv = dv;
    a.dtype = dtype;
    a.status = status;
}

int paged_attn(const void *q, const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
               const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens, const int32_t *parents,
               void *out, int B, int T, int Hq, int Hkv, int d, int num_pages, int page_size, int max_pages,
               int64_t q_stride, float scale, int dtype, int cache_dtype, void *workspace, size_t workspace_bytes,
               void *stream) {
    int rc = kv_checks(B, T, cu_seqlens, Hq, Hkv, d, num_pages, page_size, max_pages, dtype, cache_dtype, q_stride,
                       (int64_t)Hkv * d);
    if (rc != GDN_OK || B == 0 || T == 0) return rc;
    if (num_pages == 0 || max_pages == 0 || !std::isfinite(scale)) return GDN_ERR_INVALID_ARG;
    rc = kv_pointers(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, num_pages, max_pages, dtype,
                     cache_dtype, q, out);
    if (rc != GDN_OK) return rc;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < gdn::attn_workspace(T, Hq / Hkv, d))
        return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::AttnArgs a{};
    a.pg = kv_pages(block_table, kv_lens, cu_seqlens, B, T, Hkv, d, num_pages, page_size, max_pages, dtype,
                    cache_dtype, status);
    a.parents = parents;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.out = out;
    a.Hq = Hq;
    a.q_stride = (long)q_stride;
    a.scale = scale;
    a.ws = workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype != GDN_BF16 ? gdn::launch_attn_simt(a, s)
                          : gdn::attn_rows_supported(a) ? gdn::launch_attn_rows(a, s)
                                                        : gdn::launch_attn_tc(a, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

extern "C" {

const char *gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "GDN_OK";
        case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG";
        case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED";
        case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
        case GDN_ERR_DEVICE_CHECK: return "GDN_ERR_DEVICE_CHECK";
    }
    return "GDN_UNKNOWN_STATUS";
}

int gdn_prefill_path(int B, int T, int Hk, int Hv, int dk, int dv, int chunk, int dtype) {
    // a dummy aligned address stands in for every pointer: only sizes are checked
    static __align__(16) char dummy[16];
    const void *p = dummy;
    int rc = prefill_checks(p, p, p, p, p, nullptr, (const float *)p, p, nullptr, B, T, Hk, Hv, dk,
                            dv, chunk, dtype);
    if (rc != GDN_OK) return rc;
    gdn::PrefillArgs a{};
    a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.chunk = chunk; a.dtype = dtype;
    if (gdn::prefill_scan_supported(a)) return 2;
    return gdn::prefill_tc_supported(a) || gdn::prefill_ring_supported(a) ? 1 : 0;
}

// Workspace the tensor-core kernel needs for these sizes, whether or not cu_seqlens is given
// (with cu_seqlens NULL and T <= 8 the token scan runs instead and uses none of it).
size_t gdn_prefill_workspace_size(int B, int T, int Hk, int Hv, int dk, int dv, int chunk, int dtype) {
    static __align__(16) char dummy[16];
    const void *p = dummy;
    if (prefill_checks(p, p, p, p, p, nullptr, (const float *)p, p, nullptr, B, T, Hk, Hv, dk, dv, chunk,
                       dtype) != GDN_OK || B == 0)
        return 0;
    gdn::PrefillArgs a{};
    a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.chunk = chunk; a.dtype = dtype;
    if (!gdn::prefill_ring_supported(a)) return 0;
    return gdn::prefill_ring_workspace(a);
}

int gdn_prefill_ws(const void *q, const void *k, const void *v, const void *g, const void *b,
                   const float *state_in, float *state_out, void *out, const int32_t *cu_seqlens,
                   int B, int T, int Hk, int Hv, int dk, int dv, int chunk, int dtype, void *workspace,
                   size_t workspace_bytes, void *stream) {
    int rc = prefill_checks(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk,
                            dv, chunk, dtype);
    if (rc != GDN_OK) return rc;
    if (B == 0) return GDN_OK;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::PrefillArgs a{q, k, v, g, b, state_in, state_out, out, cu_seqlens,
                       B, T, Hk, Hv, dk, dv, chunk, dtype, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (gdn::prefill_scan_supported(a)) {
        e = gdn::launch_prefill_scan(a, s);
    } else if (gdn::prefill_ring_supported(a) && !force_cluster_kernel()) {
        const size_t need = gdn::prefill_ring_workspace(a);
        if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
            return GDN_ERR_INVALID_ARG;
        e = gdn::launch_prefill_ring(a, workspace, workspace_bytes, s);
    } else {
        e = gdn::prefill_tc_supported(a) ? gdn::launch_prefill_tc(a, s) : gdn::launch_prefill_simt(a, s);
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_prefill_static(const void *q, const void *k, const void *v, const void *g, const void *b,
                       const float *state_in, float *state_out, void *out, const int32_t *cu_seqlens,
                       int B, int T, int Hk, int Hv, int dk, int dv, int chunk, int dtype, void *stream) {
    int rc = prefill_checks(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk,
                            dv, chunk, dtype);
    if (rc != GDN_OK) return rc;
    if (B == 0) return GDN_OK;
    gdn::PrefillArgs a{q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, dtype,
                       nullptr};
    // sizes whose kernels take no scratch: the same kernels as gdn_prefill, nothing allocated
    if (gdn::prefill_scan_supported(a) || !gdn::prefill_ring_supported(a))
        return gdn_prefill_ws(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                              dtype, nullptr, 0, stream);
    const size_t need = gdn::prefill_ring_workspace(a, gdn::kStaticChainCtas);
    if (need == 0 || need > gdn::kStaticScratchBytes) return GDN_ERR_UNSUPPORTED;
    void *scratch = gdn::static_scratch();
    a.status = status_ptr();
    if (!scratch || !a.status) return GDN_ERR_CUDA;
    const cudaError_t e = gdn::launch_prefill_ring(a, scratch, gdn::kStaticScratchBytes,
                                                   static_cast<cudaStream_t>(stream), gdn::kStaticChainCtas);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_prefill(const void *q, const void *k, const void *v, const void *g, const void *b,
                const float *state_in, float *state_out, void *out, const int32_t *cu_seqlens,
                int B, int T, int Hk, int Hv, int dk, int dv, int chunk, int dtype, void *stream) {
    int rc = prefill_checks(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk,
                            dv, chunk, dtype);
    if (rc != GDN_OK) return rc;
    if (B == 0) return GDN_OK;
    gdn::PrefillArgs probe{q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, dtype,
                           nullptr};
    const bool ring = !force_cluster_kernel() && !gdn::prefill_scan_supported(probe) && gdn::prefill_ring_supported(probe);
    const size_t need = ring ? gdn::prefill_ring_workspace(probe) : 0;
    if (need == 0)
        return gdn_prefill_ws(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                              dtype, nullptr, 0, stream);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GDN_ERR_CUDA;
    DeviceWorkspace &w = g_ws[dev];
    std::lock_guard<std::mutex> lock(w.mu);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool capturing = stream_capturing(s);
    if (w.bytes < need) {
        if (capturing) return GDN_ERR_CUDA;  // first use (or growth) must happen outside a capture
        if (w.ptr) {  // the old buffer may still be in use by queued work
            if (w.used && cudaEventSynchronize(w.last) != cudaSuccess) return GDN_ERR_CUDA;
            cudaFree(w.ptr);
            w.ptr = nullptr;
            w.bytes = 0;
        }
        const size_t bytes = (need + (1u << 20) - 1) & ~(size_t)((1u << 20) - 1);
        if (cudaMalloc(&w.ptr, bytes) != cudaSuccess) return GDN_ERR_CUDA;
        w.bytes = bytes;
        if (!w.last && cudaEventCreateWithFlags(&w.last, cudaEventDisableTiming) != cudaSuccess) return GDN_ERR_CUDA;
    }
    if (w.used && !capturing && w.last_stream != s && cudaStreamWaitEvent(s, w.last, 0) != cudaSuccess)
        return GDN_ERR_CUDA;
    rc = gdn_prefill_ws(q, k, v, g, b, state_in, state_out, out, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, dtype,
                        w.ptr, w.bytes, stream);
    if (rc == GDN_OK && !capturing) {
        if (cudaEventRecord(w.last, s) != cudaSuccess) return GDN_ERR_CUDA;
        w.last_stream = s;
        w.used = true;
    }
    return rc;
}

int gdn_decode_step(const void *q, const void *k, const void *v, const void *g, const void *b,
                    float *state, void *out, int N, int Hk, int Hv, int dk, int dv, int dtype,
                    void *stream) {
    if (N < 0) return GDN_ERR_INVALID_ARG;
    int rc = common_checks(Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK) return rc;
    if (N == 0) return GDN_OK;
    if ((long long)N * Hv * dv * dk > (1LL << 40)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, b, state, out};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
    gdn::DecodeArgs a{q, k, v, g, b, state, out, N, Hk, Hv, dk, dv, dtype};
    return gdn::launch_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                   : GDN_ERR_CUDA;
}

int gdn_decode_step_slots(const void *q, const void *k, const void *v, const void *g, const void *b,
                          float *state_pool, const int32_t *slots, void *out, int N, int num_slots,
                          int Hk, int Hv, int dk, int dv, int dtype, void *stream) {
    if (N < 0 || num_slots < 0) return GDN_ERR_INVALID_ARG;
    int rc = common_checks(Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK) return rc;
    if (N == 0) return GDN_OK;
    if ((long long)num_slots * Hv * dv * dk > (1LL << 40)) return GDN_ERR_INVALID_ARG;
    if (num_slots > 0 && (!state_pool || !aligned16(state_pool))) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, b, slots, out};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::DecodeArgs a{q, k, v, g, b, state_pool, out, N, Hk, Hv, dk, dv, dtype};
    a.slots = slots;
    a.num_slots = num_slots;
    a.status = status;
    return gdn::launch_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                   : GDN_ERR_CUDA;
}

int gdn_prepass(const void *q, const void *k, const void *g, const void *b,
                const int32_t *cu_seqlens, int B, int T, int Hk, int Hv, int dk, int chunk,
                int dtype, float *rq, float *rk, float *beta, float *gcum, void *stream) {
    if (B < 0 || T < 0 || B > 65535) return GDN_ERR_INVALID_ARG;
    int rc = common_checks(Hk, Hv, dk, 32, dtype);
    if (rc != GDN_OK) return rc;
    if (!chunk_ok(chunk)) return GDN_ERR_UNSUPPORTED;
    const long long Ttot = cu_seqlens ? (long long)T : (long long)B * T;
    if (Ttot > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    if (B == 0 || Ttot == 0) return GDN_OK;
    const void *ptrs[] = {q, k, g, b, rq, rk, beta, gcum};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
    if (cu_seqlens && !aligned16(cu_seqlens)) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::PrepassArgs a{q, k, g, b, cu_seqlens, B, T, Hk, Hv, dk, chunk, dtype, rq, rk, beta, gcum,
                       status};
    return gdn::launch_prepass(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                     : GDN_ERR_CUDA;
}

int gdn_kv_write(const void *k, const void *v, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                 const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens, int B, int T,
                 int Hkv, int d, int num_pages, int page_size, int max_pages, int64_t k_stride, int64_t v_stride,
                 int dtype, int cache_dtype, void *stream) {
    int rc = kv_checks(B, T, cu_seqlens, Hkv, Hkv, d, num_pages, page_size, max_pages, dtype, cache_dtype, k_stride,
                       v_stride);
    if (rc != GDN_OK || B == 0 || T == 0) return rc;
    rc = kv_pointers(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, num_pages, max_pages, dtype,
                     cache_dtype, k, v);
    if (rc != GDN_OK) return rc;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::KvArgs a{kv_pages(block_table, kv_lens, cu_seqlens, B, T, Hkv, d, num_pages, page_size, max_pages, dtype,
                           cache_dtype, status),
                  const_cast<void *>(k), const_cast<void *>(v), k_cache, v_cache, k_scale, v_scale, (long)k_stride,
                  (long)v_stride};
    return gdn::launch_kv_write(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_kv_read(const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens, void *k, void *v,
                int B, int T, int Hkv, int d, int num_pages, int page_size, int max_pages, int64_t k_stride,
                int64_t v_stride, int dtype, int cache_dtype, void *stream) {
    int rc = kv_checks(B, T, cu_seqlens, Hkv, Hkv, d, num_pages, page_size, max_pages, dtype, cache_dtype, k_stride,
                       v_stride);
    if (rc != GDN_OK || B == 0 || T == 0) return rc;
    rc = kv_pointers(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, num_pages, max_pages, dtype,
                     cache_dtype, k, v);
    if (rc != GDN_OK) return rc;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::KvArgs a{kv_pages(block_table, kv_lens, cu_seqlens, B, T, Hkv, d, num_pages, page_size, max_pages, dtype,
                           cache_dtype, status),
                  k, v, const_cast<void *>(k_cache), const_cast<void *>(v_cache), const_cast<float *>(k_scale),
                  const_cast<float *>(v_scale), (long)k_stride, (long)v_stride};
    return gdn::launch_kv_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_paged_attn_workspace_size(int B, int T, int packed, int Hq, int Hkv, int d) {
    static const int32_t some = 0;
    const int32_t *cu = packed ? &some : nullptr;
    if (kv_checks(B, T, cu, Hq, Hkv, d, 1, 16, 1, GDN_BF16, GDN_BF16, (int64_t)Hq * d, (int64_t)Hkv * d) != GDN_OK ||
        B == 0 || T == 0)
        return 0;
    return gdn::attn_workspace(T, Hq / Hkv, d);
}

int gdn_paged_attn(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                   const float *v_scale, const int32_t *block_table, const int32_t *kv_lens,
                   const int32_t *cu_seqlens, void *out, int B, int T, int Hq, int Hkv, int d, int num_pages,
                   int page_size, int max_pages, int64_t q_stride, float scale, int dtype, int cache_dtype,
                   void *workspace, size_t workspace_bytes, void *stream) {
    return paged_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, nullptr, out, B, T, Hq, Hkv,
                      d, num_pages, page_size, max_pages, q_stride, scale, dtype, cache_dtype, workspace, workspace_bytes,
                      stream);
}

int gdn_tree_attn(const void *q, const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                  const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens,
                  const int32_t *parents, void *out, int B, int T, int Hq, int Hkv, int d, int num_pages,
                  int page_size, int max_pages, int64_t q_stride, float scale, int dtype, int cache_dtype,
                  void *workspace, size_t workspace_bytes, void *stream) {
    const int rc = tree_checks(B, T, cu_seqlens, parents, nullptr, nullptr);
    if (rc != GDN_OK) return rc;
    if (B > 0 && T > 0 && !parents) return GDN_ERR_INVALID_ARG;
    return paged_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, parents, out, B, T, Hq, Hkv,
                      d, num_pages, page_size, max_pages, q_stride, scale, dtype, cache_dtype, workspace, workspace_bytes,
                      stream);
}

int gdn_kv_keep(void *k_cache, void *v_cache, float *k_scale, float *v_scale, const int32_t *block_table,
                const int32_t *kv_lens, const int32_t *cu_seqlens, const int32_t *path, const int32_t *counts, int B,
                int T, int path_stride, int Hkv, int d, int num_pages, int page_size, int max_pages, int cache_dtype,
                void *stream) {
    if (cu_seqlens) T = 1;  // (says nothing)
    int rc = tree_checks(B, T, cu_seqlens, path, counts, nullptr);
    if (rc != GDN_OK) return rc;
    const int dtype = cache_dtype == GDN_F32 ? GDN_F32 : GDN_BF16;
    rc = kv_checks(B, T, cu_seqlens, Hkv, Hkv, d, num_pages, page_size, max_pages, dtype, cache_dtype, (int64_t)Hkv * d,
                   (int64_t)Hkv * d);
    if (rc != GDN_OK) return rc;
    if (path_stride < 0) return GDN_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return GDN_OK;
    static const int32_t __attribute__((aligned(16))) some[4] = {0};  // (no rows come with this call)
    rc = kv_pointers(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, num_pages, max_pages, dtype,
                     cache_dtype, some, some);
    if (rc != GDN_OK) return rc;
    if ((!path && path_stride > 0) || !counts) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::KeepArgs a{kv_pages(block_table, kv_lens, cu_seqlens, B, T, Hkv, d, num_pages, page_size, max_pages, dtype,
                             cache_dtype, status),
                    k_cache, v_cache, k_scale, v_scale, path, counts, path_stride};
    return gdn::launch_kv_keep(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_tree_scan(const void *q, const void *k, const void *v, const void *g, const void *b, const float *state,
                  const int32_t *slots, const int32_t *parents, const int32_t *cu_seqlens, void *out, int B, int T,
                  int num_slots, int Hk, int Hv, int dk, int dv, int dtype, void *stream) {
    gdn::TreeArgs a{};
    int rc = tree_checks(B, T, cu_seqlens, slots, parents, nullptr);
    if (rc == GDN_OK) rc = state_checks(T > 0, state, state, slots, B, T, cu_seqlens, num_slots, Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK || B == 0 || T == 0) return rc;
    const void *ptrs[] = {q, k, v, g, b, out};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
    if (!parents) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.b = b;
    a.state_in = state;
    a.out = out;
    a.slots = slots;
    a.parents = parents;
    tree_sizes(a, cu_seqlens, B, T, num_slots, Hk, Hv, dk, dv, dtype, status);
    return gdn::launch_tree_scan(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_tree_advance(const void *k, const void *v, const void *g, const void *b, const float *state_in,
                     float *state_out, const int32_t *slots, const int32_t *path, const int32_t *counts,
                     const int32_t *cu_seqlens, int B, int T, int path_stride, int num_slots, int Hk, int Hv, int dk,
                     int dv, int dtype, void *stream) {
    gdn::TreeArgs a{};
    int rc = tree_checks(B, T, cu_seqlens, slots, path, counts);
    if (rc == GDN_OK) rc = state_checks(true, state_in, state_out, slots, B, T, cu_seqlens, num_slots, Hk, Hv, dk, dv, dtype);
    if (rc != GDN_OK) return rc;
    if (path_stride < 0) return GDN_ERR_INVALID_ARG;
    if (B == 0) return GDN_OK;
    const void *ptrs[] = {k, v, g, b};
    for (const void *p : ptrs)
        if (T > 0 && (!p || !aligned16(p))) return GDN_ERR_INVALID_ARG;
    if ((!path && path_stride > 0) || !counts) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    a.k = k;
    a.v = v;
    a.g = g;
    a.b = b;
    a.state_in = state_in;
    a.state_out = state_out;
    a.slots = slots;
    a.path = path;
    a.counts = counts;
    a.path_stride = path_stride;
    tree_sizes(a, cu_seqlens, B, T, num_slots, Hk, Hv, dk, dv, dtype, status);
    return gdn::launch_tree_advance(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_tree_verify(const float *target_probs, const float *draft_probs, const int32_t *tokens, const int32_t *parents,
                    const float *r, const float *r_last, const int32_t *cu_seqlens, int32_t *path, int32_t *counts,
                    int32_t *next, int B, int T, int V, int64_t target_stride, int64_t draft_stride, int path_stride,
                    void *stream) {
    int rc = tree_checks(B, T, cu_seqlens, tokens, parents, path);
    if (rc != GDN_OK) return rc;
    if (V < 1) return GDN_ERR_INVALID_ARG;
    if (V > gdn::kVerMaxVocab) return GDN_ERR_UNSUPPORTED;
    if (target_stride < V || (draft_probs && draft_stride < V)) return GDN_ERR_INVALID_ARG;
    if (path_stride < 0 || path_stride > (1 << 20) || (!cu_seqlens && path_stride < T)) return GDN_ERR_INVALID_ARG;
    const long long tokens_all = cu_seqlens ? (long long)T : (long long)B * T;
    const int64_t widest = draft_probs && draft_stride > target_stride ? draft_stride : target_stride;
    if (widest > (1LL << 40) || tokens_all * (widest >> 8) > (1LL << 40)) return GDN_ERR_INVALID_ARG;
    if (B == 0) return GDN_OK;
    if (!aligned4(counts) || !aligned4(next) || !aligned4(r) || !aligned4(r_last)) return GDN_ERR_INVALID_ARG;
    if (!counts || !next || !r_last || (!path && path_stride > 0)) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!target_probs || !tokens || !parents || !r)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(target_probs) || !aligned16(draft_probs)) return GDN_ERR_INVALID_ARG;
    int *status = status_ptr();
    if (!status) return GDN_ERR_CUDA;
    gdn::VerifyArgs a{};
    a.target = target_probs;
    a.draft = draft_probs;
    a.tokens = tokens;
    a.parents = parents;
    a.cu = cu_seqlens;
    a.r = r;
    a.r_last = r_last;
    a.path = path;
    a.counts = counts;
    a.next = next;
    a.B = B;
    a.T = T;
    a.Ttot = (long)tokens_all;
    a.V = V;
    a.target_stride = (long)target_stride;
    a.draft_stride = (long)draft_stride;
    a.path_stride = path_stride;
    a.status = status;
    return gdn::launch_tree_verify(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_get_device_status(void *stream) {
    int *status = status_ptr();
    int *taken = taken_ptr();
    if (!status || !taken) return GDN_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
    take_status_kernel<<<1, 1, 0, s>>>(status, taken);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    int host = 0;
    if (cudaMemcpyAsync(&host, taken, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
    return host == 0 ? GDN_OK : GDN_ERR_DEVICE_CHECK;
}

}  // extern "C"
