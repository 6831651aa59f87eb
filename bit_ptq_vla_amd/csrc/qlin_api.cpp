// Host side of the qlin C ABI: argument validation (before any HIP call),
// device check, launch, and HIP error mapping.  Declarations and the meaning
// of every argument are in include/qlin.h.

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/qlin.h"
#include "qlin_internal.h"

namespace {

constexpr int kMaxDevices = 64;
// 0 = unchecked, 1 = gfx950, 2 = other device
int g_device_ok[kMaxDevices] = {0};
std::mutex g_device_mu;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t dtype_size(qlin_dtype d) {
    switch (d) {
        case QLIN_F16: case QLIN_BF16: return 2;
        case QLIN_F32: case QLIN_I32: return 4;
    }
    return 0;
}

bool is_float_in(qlin_dtype d) { return d == QLIN_F16 || d == QLIN_BF16 || d == QLIN_F32; }

bool pow2_block_ok(int32_t b) { return b == 0 || b == 1 || (b > 1 && b <= 256 && (b & (b - 1)) == 0); }

struct Span {
    const void* p;
    int64_t bytes;
};

bool overlap(Span a, Span b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

bool any_overlap(const Span* outs, int nout, const Span* ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

// Checks (once per device, cached) that the current device is a gfx950.
qlin_status check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return QLIN_ERR_DEVICE;
    if (dev >= kMaxDevices) return QLIN_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(g_device_mu);
    if (g_device_ok[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return QLIN_ERR_DEVICE;
        g_device_ok[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    }
    return g_device_ok[dev] == 1 ? QLIN_OK : QLIN_ERR_DEVICE;
}

qlin_status map_err(hipError_t e) {
    if (e == hipSuccess) return QLIN_OK;
    if (e == hipErrorStreamCaptureUnsupported) return QLIN_ERR_CAPTURE;
    return QLIN_ERR_LAUNCH;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// Largest k the activation / weight row kernel holds in registers:
// 256 lanes x 16 chunks x 8 values.
constexpr int64_t kMaxRowK = 32768;

// GEMM k bound (exclusive): 2^17.
constexpr int64_t kMaxGemmK = 131072;

// Code widths of the quantizers: int8, packed int4, or int4 codes in E2M3
// storage (k a multiple of 128 there, the GEMM's stage).
bool bits_ok(int32_t bits) { return bits == 4 || bits == 8 || bits == QLIN_BITS_E2M3; }
bool bits_k_ok(int32_t bits, int64_t k) { return bits != QLIN_BITS_E2M3 || k % 128 == 0; }
int64_t code_bytes(int64_t rows, int64_t k, int32_t bits) {
    if (bits == 8) return rows * k;
    if (bits == 4) return rows * (k / 2);
    return rows * (k / 4 * 3);
}

// Step of k the GEMM schemes take: 64 (W8A8, and W4A4, whose last 64-byte
// stage of 128 codes may then be half full), 128 for W4A8 (a stage holds
// 128 k of both operands) and E2M3 (128 codes per 96-byte stage).
int64_t gemm_k_step(bool int4, bool a8, bool f6) { return (f6 || (int4 && a8)) ? 128 : 64; }

// Shape checks of the integer GEMM schemes (before any pointer check).
bool gemm_shape_ok(int64_t m, int64_t n, int64_t k, int64_t kstep) {
    if (m < 0 || n < 1 || k < kstep || (k % kstep) != 0) return false;
    // k < 2^17: the accumulator, 256 * acc for W4A4 and 16 * acc for W4A8,
    // stays below 2^31 in magnitude for any codes (|code| <= 8 int4, 128 int8)
    if (k >= kMaxGemmK) return false;
    return m <= 0x7FFFFFFF && n <= 0x7FFFFFFF;
}

// Split-K partial bytes of the plan a call with a workspace takes (0: no split).
int64_t gemm_ws_need(int64_t m, int64_t n, int64_t k, bool int4, bool a8, bool f6) {
    if (f6) return 0;                                     // the E2M3 kernels never split
    if (m == 0 || m <= qlin::kSkinnyIntMaxM) return 0;   // the small-M kernel never splits
    return qlin::plan_gemm(m, n, k, int4, a8, true).ws_bytes;
}

// Split-K scratch of a GEMM call: none (no split), the caller's workspace, or
// the library's static device array.
enum class Scratch { None, Caller, Static };

qlin_status gemm_common(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                        int64_t m, int64_t n, int64_t k, void* y, qlin_dtype y_dtype, Scratch mode, void* ws,
                        int64_t ws_bytes, void* stream, bool int4, bool a8, bool f6) {
    const bool use_static = mode == Scratch::Static;
    if (!xq && m > 0) return QLIN_ERR_NULL;
    if (!wq || !y) return QLIN_ERR_NULL;
    if (y_dtype != QLIN_I32 && ((!x_scale && m > 0) || !w_scale)) return QLIN_ERR_NULL;
    if (y_dtype != QLIN_F16 && y_dtype != QLIN_BF16 && y_dtype != QLIN_F32 && y_dtype != QLIN_I32)
        return QLIN_ERR_DTYPE;
    if (!gemm_shape_ok(m, n, k, gemm_k_step(int4, a8, f6))) return QLIN_ERR_SHAPE;
    if (ws_bytes < 0) return QLIN_ERR_SHAPE;
    if (!ws && ws_bytes > 0) return QLIN_ERR_NULL;
    if (!aligned16(xq) || !aligned16(wq) || !aligned16(y) || !aligned16(x_scale) || !aligned16(w_scale) ||
        !aligned16(ws))
        return QLIN_ERR_ALIGN;
    const int64_t need = ws ? gemm_ws_need(m, n, k, int4, a8, f6) : 0;
    if (ws && ws_bytes < need) return QLIN_ERR_WORKSPACE;
    const int64_t kb = f6 ? k / 4 * 3 : int4 ? k / 2 : k;
    const int64_t ka = f6 ? k / 4 * 3 : (int4 && !a8) ? k / 2 : k;
    const Span outs[2] = {{y, m * n * dtype_size(y_dtype)}, {ws, ws ? ws_bytes : 0}};
    const Span ins[4] = {{xq, m * ka}, {wq, n * kb}, {x_scale, m * 4}, {w_scale, n * 4}};
    if (any_overlap(outs, 2, ins, 4)) return QLIN_ERR_ALIAS;
    if (use_static && gemm_ws_need(m, n, k, int4, a8, f6) > QLIN_STATIC_SCRATCH_BYTES) return QLIN_ERR_WORKSPACE;
    if (m == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    hipStream_t s = as_stream(stream);
    if (f6)
        return map_err(qlin::launch_gemm_f6(qlin::plan_gemm_f6(m, n, k, false), xq, x_scale, wq, w_scale, m, n, k,
                                            y, y_dtype, false, s));
    if (m <= qlin::kSkinnyIntMaxM)
        return map_err(qlin::launch_skinny_int(xq, x_scale, wq, w_scale, m, n, k, int4, a8, y, y_dtype, s));
    if (use_static) {
        int32_t* scratch_dev = nullptr;
        if (qlin::static_scratch(&scratch_dev) != hipSuccess) return QLIN_ERR_DEVICE;
        const qlin::GemmPlan plan = qlin::plan_gemm(m, n, k, int4, a8, true);
        return map_err(qlin::launch_gemm(plan, xq, x_scale, wq, w_scale, m, n, k, int4, a8, y, y_dtype,
                                         scratch_dev, s));
    }
    const qlin::GemmPlan plan = qlin::plan_gemm(m, n, k, int4, a8, ws != nullptr);
    return map_err(qlin::launch_gemm(plan, xq, x_scale, wq, w_scale, m, n, k, int4, a8, y, y_dtype,
                                     static_cast<int32_t*>(ws), s));
}

bool scheme_flags(qlin_scheme scheme, bool* int4, bool* a8, bool* f6) {
    *f6 = false;
    switch (scheme) {
        case QLIN_W4A4: *int4 = true; *a8 = false; return true;
        case QLIN_W8A8: *int4 = false; *a8 = false; return true;
        case QLIN_W4A8: *int4 = true; *a8 = true; return true;
        case QLIN_W4A4_E2M3: *int4 = true; *a8 = false; *f6 = true; return true;
    }
    return false;
}

// Shared checks of the per-step table entry points (rows of k values, no pre-op).
qlin_status table_rows_check(const void* x, qlin_dtype dt, int64_t rows, int64_t k, int64_t ldx,
                             const float* fold, int32_t had_block, int32_t bits, const void* table) {
    if (!table) return QLIN_ERR_NULL;
    if (rows > 0 && !x) return QLIN_ERR_NULL;
    if (!is_float_in(dt)) return QLIN_ERR_DTYPE;
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!pow2_block_ok(had_block)) return QLIN_ERR_UNSUPPORTED;
    if (rows < 0 || k < 8 || (k % 8) != 0 || (ldx % 8) != 0 || ldx < k) return QLIN_ERR_SHAPE;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (had_block > 1 && (k % had_block) != 0) return QLIN_ERR_SHAPE;
    if (k > kMaxRowK) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(fold) || !aligned16(table)) return QLIN_ERR_ALIGN;
    return QLIN_OK;
}

// Shared checks of the composite-rotation entry points.
qlin_status composite_check(const void* x, qlin_dtype dt, int64_t rows, int64_t k, int64_t ldx, int32_t b) {
    if (rows > 0 && !x) return QLIN_ERR_NULL;
    if (!is_float_in(dt)) return QLIN_ERR_DTYPE;
    if (b != 16 && b != 32 && b != 64 && b != 128) return QLIN_ERR_UNSUPPORTED;
    if (rows < 0 || k < b || (k % b) != 0 || (k % 8) != 0 || (ldx % 8) != 0 || ldx < k) return QLIN_ERR_SHAPE;
    if (k > kMaxRowK) return QLIN_ERR_SHAPE;
    return QLIN_OK;
}

// The rotated rows (fp32 [rows][k]) go through the caller's workspace.
qlin_status composite_run(const void* x, qlin_dtype dt, int64_t rows, int64_t k, int64_t ldx, const float* mult,
                          const int32_t* perm, const float* rot, int32_t b, int32_t bits, void* q, float* scale,
                          float* work, void* stream) {
    return map_err(qlin::launch_composite_quant(x, dt, rows, k, ldx, mult, perm, rot, b, bits, q, scale, work,
                                                as_stream(stream)));
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shared checks of the calls on a paged cache.
qlin_status kv_check(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t tokens, int32_t heads_q) {
    if (!c || !b) return QLIN_ERR_NULL;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return QLIN_ERR_NULL;
    if (b->batch > 0 && (!b->page_table || !b->q_start || !b->kv_len)) return QLIN_ERR_NULL;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64) return QLIN_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QLIN_ERR_UNSUPPORTED;
    if (c->pages < 1 || c->pages > 0x7FFFFFFF || c->heads < 1 || c->heads > 4096) return QLIN_ERR_SHAPE;
    if (heads_q < 1 || heads_q > 65536 || heads_q % c->heads != 0) return QLIN_ERR_SHAPE;
    if (tokens < 0 || tokens > 0x7FFFFFFF || b->batch < 0 || b->max_q < 0 || b->max_kv < 0) return QLIN_ERR_SHAPE;
    if (b->table_ld < (static_cast<int64_t>(b->max_kv) + c->page_size - 1) / c->page_size) return QLIN_ERR_SHAPE;
    // positions and (token, head) rows are 32-bit integers in the kernels
    if (b->table_ld > 0x7FFFFFFF || b->max_kv > (1 << 30)) return QLIN_ERR_SHAPE;
    if (static_cast<int64_t>(b->max_q) * (heads_q / c->heads) > (1LL << 30)) return QLIN_ERR_SHAPE;
    if (static_cast<int64_t>(b->batch) * c->heads > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale)) return QLIN_ERR_ALIGN;
    if (!aligned4(b->page_table) || !aligned4(b->q_start) || !aligned4(b->kv_len) || !aligned4(b->prefix_len))
        return QLIN_ERR_ALIGN;
    return QLIN_OK;
}

// Blocks of 512 threads that a launch (of 2^32 threads) holds.
constexpr int64_t kMaxAttnBlocks = (1 << 23) - 1;

// The call's index arrays as spans (4 of them).
void kv_index_spans(const qlin_kv_cache* c, const qlin_kv_batch* b, Span* s) {
    const int64_t n = b->batch, used = (static_cast<int64_t>(b->max_kv) + c->page_size - 1) / c->page_size;
    s[0] = {b->page_table, n > 0 ? ((n - 1) * b->table_ld + used) * 4 : 0};
    s[1] = {b->q_start, n > 0 ? (n + 1) * 4 : 0};
    s[2] = {b->kv_len, n * 4};
    s[3] = {b->prefix_len, n * 4};
}

qlin::KvIndex kv_index(const qlin_kv_cache* c, const qlin_kv_batch* b, int64_t tokens) {
    return {b->page_table, b->table_ld, b->q_start, b->kv_len, b->prefix_len, tokens, c->pages, b->batch, b->max_q,
            b->max_kv, c->page_size};
}

static_assert(QLIN_MAX_TREE_NODES == qlin::kMaxTreeNodes && QLIN_MAX_POOL_ROWS == qlin::kMaxPoolRows, "bounds of the header");

// Rows of qlin_sample (a block of 512 threads each, of the 2^32 a launch holds).
constexpr int64_t kMaxSampleRows = 1 << 21;

// Shared checks of the tree calls, which read a batch's lengths only.
qlin_status tree_check(const qlin_kv_batch* b, int64_t tokens) {
    if (!b) return QLIN_ERR_NULL;
    if (b->batch > 0 && (!b->q_start || !b->kv_len)) return QLIN_ERR_NULL;
    if (tokens < 0 || tokens > 0x7FFFFFFF || b->batch < 0 || b->batch > (1 << 23) || b->max_q < 0 || b->max_kv < 0 ||
        b->max_kv > (1 << 30) || b->max_q > qlin::kMaxTreeNodes)
        return QLIN_ERR_SHAPE;
    return aligned4(b->q_start) && aligned4(b->kv_len) ? QLIN_OK : QLIN_ERR_ALIGN;
}

qlin::KvIndex tree_index(const qlin_kv_batch* b, int64_t tokens) {
    return {nullptr, 0, b->q_start, b->kv_len, nullptr, tokens, 0, b->batch, b->max_q, b->max_kv, 16};
}

qlin_status pool_check(const qlin_kv_pool* p) {
    if (!p || !p->refs || !p->free_bits) return QLIN_ERR_NULL;
    if (p->pages < 1 || p->pages > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    return aligned16(p->refs) && aligned16(p->free_bits) ? QLIN_OK : QLIN_ERR_ALIGN;
}

qlin_status table_check(int32_t page_size, const int32_t* table, int64_t ld, int64_t cols, int64_t rows) {
    if (rows > 0 && !table) return QLIN_ERR_NULL;
    if (page_size != 16 && page_size != 32 && page_size != 64) return QLIN_ERR_UNSUPPORTED;
    if (rows < 0 || rows > 0x7FFFFFFF || cols < 0 || cols > (1 << 24) || ld < cols || ld > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    return aligned4(table) ? QLIN_OK : QLIN_ERR_ALIGN;
}

// A stack of layers' caches: each complete, all of one shape, none twice.
qlin_status stack_check(const qlin_kv_cache* c, int32_t layers) {
    if (!c) return QLIN_ERR_NULL;
    if (layers < 1 || layers > 4096) return QLIN_ERR_SHAPE;
    for (int32_t i = 0; i < layers; ++i)
        if (!c[i].k || !c[i].v || !c[i].k_scale || !c[i].v_scale) return QLIN_ERR_NULL;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64) return QLIN_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QLIN_ERR_UNSUPPORTED;
    if (c->pages < 1 || c->pages > 0x7FFFFFFF || c->heads < 1 || c->heads > 4096) return QLIN_ERR_SHAPE;
    for (int32_t i = 0; i < layers; ++i) {
        if (c[i].pages != c->pages || c[i].page_size != c->page_size || c[i].heads != c->heads ||
            c[i].head_dim != c->head_dim)
            return QLIN_ERR_SHAPE;
        if (!aligned16(c[i].k) || !aligned16(c[i].v) || !aligned16(c[i].k_scale) || !aligned16(c[i].v_scale))
            return QLIN_ERR_ALIGN;
        for (int32_t j = 0; j < i; ++j)
            if (c[i].k == c[j].k || c[i].v == c[j].v || c[i].k_scale == c[j].k_scale || c[i].v_scale == c[j].v_scale)
                return QLIN_ERR_ALIAS;
    }
    return QLIN_OK;
}

bool stack_overlaps(const qlin_kv_cache* c, int32_t layers, const Span* s, int n) {
    for (int32_t i = 0; i < layers; ++i) {
        const int64_t scales = c[i].pages * c[i].heads * 4, codes = scales / 4 * c[i].page_size * c[i].head_dim;
        const Span own[4] = {{c[i].k, codes}, {c[i].v, codes}, {c[i].k_scale, scales}, {c[i].v_scale, scales}};
        for (const Span& o : own)
            for (int j = 0; j < n; ++j)
                if (overlap(o, s[j])) return true;
    }
    return false;
}

// The layers from `at` on that one launch takes.
qlin::KvStackArgs stack_args(const qlin_kv_cache* c, int32_t layers, int32_t at) {
    qlin::KvStackArgs a{};
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.heads = c->heads;
    a.head_dim = c->head_dim;
    a.layers = layers - at < qlin::kMaxStackLayers ? layers - at : qlin::kMaxStackLayers;
    for (int i = 0; i < a.layers; ++i) a.layer[i] = {c[at + i].k, c[at + i].v, c[at + i].k_scale, c[at + i].v_scale};
    return a;
}

// Checks and launch of the two attention entry points (tree: with a mask, null where no
// sequence has a new token).
int64_t attention_bytes(int32_t heads_q, const qlin_kv_cache* cache, const qlin_kv_batch* batch, bool tree) {
    if (kv_check(cache, batch, 0, heads_q) != QLIN_OK) return -1;
    const qlin::KvAttnPlan plan = (tree ? qlin::plan_kv_attention_tree : qlin::plan_kv_attention)(
        batch->batch, batch->max_q, batch->max_kv, heads_q, cache->heads, cache->head_dim, true);
    return plan.blocks > kMaxAttnBlocks ? -1 : plan.ws_bytes;
}

qlin_status attention(const void* q, qlin_dtype dtype, int64_t tokens, int64_t ldq, int32_t heads_q,
                      const qlin_kv_cache* cache, const qlin_kv_batch* batch, bool tree, const uint32_t* mask,
                      int64_t mask_ld, float sm_scale, float softcap, void* out, int64_t ldo, void* workspace,
                      int64_t workspace_bytes, void* stream) {
    qlin_status st = kv_check(cache, batch, tokens, heads_q);
    if (st != QLIN_OK) return st;
    if (tokens > 0 && (!q || !out)) return QLIN_ERR_NULL;
    if (dtype != QLIN_F16 && dtype != QLIN_BF16) return QLIN_ERR_DTYPE;
    constexpr float kMax = 3.402823466e38f;
    if (!(sm_scale >= -kMax && sm_scale <= kMax)) return QLIN_ERR_UNSUPPORTED;
    // (a capped score is off by 2^-21 of the cap; 2 / cap must stay in range)
    if (softcap != 0.f && !(softcap >= 0x1p-20f && softcap <= 4096.f)) return QLIN_ERR_UNSUPPORTED;
    const int64_t wide = static_cast<int64_t>(heads_q) * cache->head_dim;
    if (ldq % 8 != 0 || ldq < wide || ldo % 8 != 0 || ldo < wide || workspace_bytes < 0) return QLIN_ERR_SHAPE;
    if (!workspace && workspace_bytes > 0) return QLIN_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return QLIN_ERR_ALIGN;
    const qlin::KvAttnPlan plan = (tree ? qlin::plan_kv_attention_tree : qlin::plan_kv_attention)(
        batch->batch, batch->max_q, batch->max_kv, heads_q, cache->heads, cache->head_dim, workspace != nullptr);
    if (plan.blocks > kMaxAttnBlocks) return QLIN_ERR_SHAPE;
    if (workspace && workspace_bytes < plan.ws_bytes) return QLIN_ERR_WORKSPACE;
    const int64_t codes = cache->pages * cache->heads * cache->page_size * cache->head_dim;
    const int64_t scales = cache->pages * cache->heads * 4;
    const Span outs[2] = {{out, tokens > 0 ? ((tokens - 1) * ldo + wide) * 2 : 0}, {workspace, workspace_bytes}};
    Span ins[10] = {{q, tokens > 0 ? ((tokens - 1) * ldq + wide) * 2 : 0}, {cache->k, codes}, {cache->v, codes},
                   {cache->k_scale, scales}, {cache->v_scale, scales},
                   {mask, tree && tokens > 0 ? ((tokens - 1) * mask_ld + (static_cast<int64_t>(batch->max_q) + 31) / 32) * 4 : 0}};
    kv_index_spans(cache, batch, ins + 6);
    if (any_overlap(outs, 2, ins, 10)) return QLIN_ERR_ALIAS;
    if (tokens == 0 || batch->batch == 0 || batch->max_q == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    if (tree)
        return map_err(qlin::launch_kv_attention_tree(plan, q, dtype, ldq, heads_q, kv_index(cache, batch, tokens),
                                                      cache->k, cache->v, cache->k_scale, cache->v_scale, cache->heads,
                                                      cache->head_dim, sm_scale, softcap, mask, mask_ld, out, ldo,
                                                      workspace, as_stream(stream)));
    return map_err(qlin::launch_kv_attention(plan, q, dtype, ldq, heads_q, kv_index(cache, batch, tokens), cache->k,
                                             cache->v, cache->k_scale, cache->v_scale, cache->heads, cache->head_dim,
                                             sm_scale, softcap, out, ldo, workspace, as_stream(stream)));
}

// Checks and launch of the two residual + RMS norm entry points (bits 0: the
// float output, no scale).
qlin_status add_rmsnorm(const void* x, qlin_dtype dt, int64_t m, int64_t k, int64_t ldx, const void* res, int64_t ldr,
                        const float* w, float eps, int32_t had_block, int32_t bits, void* res_out, void* q,
                        float* scale, void* stream) {
    if (m > 0 && (!x || !q || (bits && !scale))) return QLIN_ERR_NULL;
    if (!w) return QLIN_ERR_NULL;
    if (!is_float_in(dt)) return QLIN_ERR_DTYPE;
    if (bits && !bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!pow2_block_ok(had_block)) return QLIN_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || eps > 3.402823466e38f) return QLIN_ERR_UNSUPPORTED;
    if (m < 0 || m > 0x7FFFFFFF || k < 8 || (k % 8) != 0 || k > kMaxRowK) return QLIN_ERR_SHAPE;
    if ((ldx % 8) != 0 || ldx < k) return QLIN_ERR_SHAPE;
    if ((res || res_out) && ((ldr % 8) != 0 || ldr < k)) return QLIN_ERR_SHAPE;
    int64_t row_threads = 32;      // of the 2^32 a launch holds
    while (row_threads < 1024 && row_threads * 8 < k) row_threads *= 2;
    if (m * row_threads > 0xFFFFFFFFLL) return QLIN_ERR_SHAPE;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (had_block > 1 && (k % had_block) != 0) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(res) || !aligned16(res_out) || !aligned16(w) || !aligned16(q) || !aligned16(scale))
        return QLIN_ERR_ALIGN;
    const int64_t es = dtype_size(dt);
    const int64_t xb = m > 0 ? ((m - 1) * ldx + k) * es : 0, rb = m > 0 ? ((m - 1) * ldr + k) * es : 0;
    const Span outs[2] = {{q, bits ? code_bytes(m, k, bits) : m * k * es}, {scale, m * 4}};
    const Span ins[4] = {{x, xb}, {res, rb}, {w, k * 4}, {res_out, rb}};
    if (any_overlap(outs, 2, ins, 4)) return QLIN_ERR_ALIAS;
    // r may replace the residual or x where it covers the same rows
    const Span r = {res_out, rb};
    if (overlap(r, ins[2])) return QLIN_ERR_ALIAS;
    if (res_out != res && overlap(r, ins[1])) return QLIN_ERR_ALIAS;
    if (!(res_out == x && ldx == ldr) && overlap(r, ins[0])) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_add_rmsnorm(x, dt, m, k, ldx, res, ldr, w, eps, had_block, bits, res_out, q, scale,
                                            as_stream(stream)));
}

}  // namespace

extern "C" {

int32_t qlin_abi_version(void) { return QLIN_ABI_VERSION; }

const char* qlin_status_string(qlin_status s) {
    switch (s) {
        case QLIN_OK: return "ok";
        case QLIN_ERR_NULL: return "null pointer";
        case QLIN_ERR_SHAPE: return "invalid shape";
        case QLIN_ERR_DTYPE: return "unsupported dtype";
        case QLIN_ERR_ALIGN: return "pointer or row pitch not 16-byte aligned";
        case QLIN_ERR_UNSUPPORTED: return "unsupported bits, block, group or pre-op";
        case QLIN_ERR_DEVICE: return "no usable gfx950 device or HIP runtime error";
        case QLIN_ERR_LAUNCH: return "kernel launch failed";
        case QLIN_ERR_ALIAS: return "output overlaps an input";
        case QLIN_ERR_CAPTURE: return "first use of a lookup table inside stream capture";
        case QLIN_ERR_WORKSPACE: return "workspace smaller than the call needs";
    }
    return "unknown status";
}

qlin_status qlin_calibrate_fold(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                                qlin_preop pre, const void* w, qlin_dtype w_dtype, int64_t n, float* s,
                                float* inv_s, void* stream) {
    if (!x || !w || !s || !inv_s) return QLIN_ERR_NULL;
    if (!is_float_in(x_dtype) || !is_float_in(w_dtype)) return QLIN_ERR_DTYPE;
    if (pre != QLIN_PRE_NONE && pre != QLIN_PRE_GEGLU) return QLIN_ERR_UNSUPPORTED;
    const int64_t width = (pre == QLIN_PRE_GEGLU) ? 2 * k : k;
    if (m < 1 || n < 1 || k < 8 || (k % 8) != 0 || (ldx % 8) != 0 || ldx < width) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(w) || !aligned16(s) || !aligned16(inv_s)) return QLIN_ERR_ALIGN;
    const Span outs[2] = {{s, k * 4}, {inv_s, k * 4}};
    const Span ins[2] = {{x, ((m - 1) * ldx + width) * dtype_size(x_dtype)}, {w, n * k * dtype_size(w_dtype)}};
    if (any_overlap(outs, 2, ins, 2)) return QLIN_ERR_ALIAS;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_calibrate_fold(x, x_dtype, m, k, ldx, pre == QLIN_PRE_GEGLU, w, w_dtype,
                                               n, s, inv_s, as_stream(stream)));
}

qlin_status qlin_quantize_weights(const void* w, qlin_dtype w_dtype, int64_t n, int64_t k,
                                  const float* fold_s, int32_t had_block, int32_t bits, int32_t group,
                                  void* wq, void* w_scale, void* stream) {
    if (!w || !wq || !w_scale) return QLIN_ERR_NULL;
    if (!is_float_in(w_dtype)) return QLIN_ERR_DTYPE;
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!pow2_block_ok(had_block)) return QLIN_ERR_UNSUPPORTED;
    if (group != 0 && group != 128) return QLIN_ERR_UNSUPPORTED;
    if (group == 128 && (bits != 4 || fold_s != nullptr || had_block > 1)) return QLIN_ERR_UNSUPPORTED;
    if (n < 1 || k < 8 || (k % 8) != 0) return QLIN_ERR_SHAPE;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (group && (k % group) != 0) return QLIN_ERR_SHAPE;
    if (had_block > 1 && (k % had_block) != 0) return QLIN_ERR_SHAPE;
    if (!group && k > kMaxRowK) return QLIN_ERR_SHAPE;
    if (!aligned16(w) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(fold_s)) return QLIN_ERR_ALIGN;
    const int64_t scale_bytes = group ? n * (k / group) * 2 : n * 4;
    const Span outs[2] = {{wq, code_bytes(n, k, bits)}, {w_scale, scale_bytes}};
    const Span ins[2] = {{w, n * k * dtype_size(w_dtype)}, {fold_s, fold_s ? k * 4 : 0}};
    if (any_overlap(outs, 2, ins, 2)) return QLIN_ERR_ALIAS;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    hipStream_t s = as_stream(stream);
    if (group) return map_err(qlin::launch_quant_groups_w4(w, w_dtype, n, k, wq, w_scale, s));
    return map_err(qlin::launch_rotate_quant(w, w_dtype, n, k, k, false, fold_s, had_block, bits, wq,
                                             static_cast<float*>(w_scale), s));
}

qlin_status qlin_rotate_quant_act(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                                  qlin_preop pre, const float* fold_inv_s, int32_t had_block, int32_t bits,
                                  void* xq, float* x_scale, void* stream) {
    if (m > 0 && (!x || !xq || !x_scale)) return QLIN_ERR_NULL;
    if (!is_float_in(x_dtype)) return QLIN_ERR_DTYPE;
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!pow2_block_ok(had_block)) return QLIN_ERR_UNSUPPORTED;
    if (pre != QLIN_PRE_NONE && pre != QLIN_PRE_GEGLU) return QLIN_ERR_UNSUPPORTED;
    const int64_t width = (pre == QLIN_PRE_GEGLU) ? 2 * k : k;
    if (m < 0 || k < 8 || (k % 8) != 0 || (ldx % 8) != 0 || ldx < width) return QLIN_ERR_SHAPE;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (had_block > 1 && (k % had_block) != 0) return QLIN_ERR_SHAPE;
    if (k > kMaxRowK) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(x_scale) || !aligned16(fold_inv_s)) return QLIN_ERR_ALIGN;
    const Span outs[2] = {{xq, code_bytes(m, k, bits)}, {x_scale, m * 4}};
    const Span ins[2] = {{x, m > 0 ? ((m - 1) * ldx + width) * dtype_size(x_dtype) : 0},
                         {fold_inv_s, fold_inv_s ? k * 4 : 0}};
    if (any_overlap(outs, 2, ins, 2)) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_rotate_quant(x, x_dtype, m, k, ldx, pre == QLIN_PRE_GEGLU, fold_inv_s,
                                             had_block, bits, xq, x_scale, as_stream(stream)));
}

qlin_status qlin_add_rmsnorm_quant(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                                   const void* residual, int64_t ldr, const float* weight, float eps,
                                   int32_t had_block, int32_t bits, void* residual_out, void* xq, float* x_scale,
                                   void* stream) {
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    return add_rmsnorm(x, x_dtype, m, k, ldx, residual, ldr, weight, eps, had_block, bits, residual_out, xq, x_scale,
                       stream);
}

qlin_status qlin_add_rmsnorm(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                             const void* residual, int64_t ldr, const float* weight, float eps, void* residual_out,
                             void* y, void* stream) {
    return add_rmsnorm(x, x_dtype, m, k, ldx, residual, ldr, weight, eps, 0, 0, residual_out, y, nullptr, stream);
}

qlin_status qlin_calibrate_step_scales(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                                       const float* fold_inv_s, int32_t had_block, int32_t bits,
                                       float* table, void* stream) {
    qlin_status st = table_rows_check(x, x_dtype, m, k, ldx, fold_inv_s, had_block, bits, table);
    if (st != QLIN_OK) return st;
    if (m < 1) return QLIN_ERR_SHAPE;
    const Span outs[1] = {{table, k * 4}};
    const Span ins[2] = {{x, ((m - 1) * ldx + k) * dtype_size(x_dtype)}, {fold_inv_s, fold_inv_s ? k * 4 : 0}};
    if (any_overlap(outs, 1, ins, 2)) return QLIN_ERR_ALIAS;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_calibrate_step_scales(x, x_dtype, m, k, ldx, fold_inv_s, had_block, bits,
                                                      table, as_stream(stream)));
}

qlin_status qlin_rotate_quant_act_static(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k, int64_t ldx,
                                         const float* fold_inv_s, int32_t had_block, int32_t bits,
                                         const float* table, void* xq, void* stream) {
    qlin_status st = table_rows_check(x, x_dtype, m, k, ldx, fold_inv_s, had_block, bits, table);
    if (st != QLIN_OK) return st;
    if (m > 0 && !xq) return QLIN_ERR_NULL;
    if (!aligned16(xq)) return QLIN_ERR_ALIGN;
    const Span outs[1] = {{xq, code_bytes(m, k, bits)}};
    const Span ins[3] = {{x, m > 0 ? ((m - 1) * ldx + k) * dtype_size(x_dtype) : 0},
                         {fold_inv_s, fold_inv_s ? k * 4 : 0}, {table, k * 4}};
    if (any_overlap(outs, 1, ins, 3)) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_rotate_quant_table(x, x_dtype, m, k, ldx, fold_inv_s, had_block, bits, table,
                                                   false, xq, nullptr, as_stream(stream)));
}

qlin_status qlin_quantize_weights_step(const void* w, qlin_dtype w_dtype, int64_t n, int64_t k,
                                       const float* fold_s, int32_t had_block, int32_t bits,
                                       const float* table, void* wq, float* w_scale, void* stream) {
    qlin_status st = table_rows_check(w, w_dtype, n, k, k, fold_s, had_block, bits, table);
    if (st != QLIN_OK) return st;
    if (!wq || !w_scale) return QLIN_ERR_NULL;
    if (n < 1) return QLIN_ERR_SHAPE;
    if (!aligned16(wq) || !aligned16(w_scale)) return QLIN_ERR_ALIGN;
    const Span outs[2] = {{wq, code_bytes(n, k, bits)}, {w_scale, n * 4}};
    const Span ins[3] = {{w, n * k * dtype_size(w_dtype)}, {fold_s, fold_s ? k * 4 : 0}, {table, k * 4}};
    if (any_overlap(outs, 2, ins, 3)) return QLIN_ERR_ALIAS;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_rotate_quant_table(w, w_dtype, n, k, k, fold_s, had_block, bits, table, true,
                                                   wq, w_scale, as_stream(stream)));
}

int64_t qlin_calibrate_composite_work_bytes(int64_t n, int64_t k, int32_t had_block) {
    if (n < 1 || k < 1 || (had_block != 16 && had_block != 32 && had_block != 64 && had_block != 128) ||
        k % had_block != 0 || k > kMaxRowK)
        return -1;
    return qlin::composite_calib_work_bytes(n, k, had_block);
}

qlin_status qlin_calibrate_composite(const void* w, qlin_dtype w_dtype, int64_t n, int64_t k,
                                     const float* fold_s, int32_t had_block, int32_t* perm, float* rot,
                                     void* work, int64_t work_bytes, void* stream) {
    qlin_status st = composite_check(w, w_dtype, n, k, k, had_block);
    if (st != QLIN_OK) return st;
    if (!w || !perm || !rot || !work) return QLIN_ERR_NULL;
    if (n < 1) return QLIN_ERR_SHAPE;
    if (!aligned16(w) || !aligned16(fold_s) || !aligned16(perm) || !aligned16(rot) || !aligned16(work))
        return QLIN_ERR_ALIGN;
    if (work_bytes < qlin::composite_calib_work_bytes(n, k, had_block)) return QLIN_ERR_WORKSPACE;
    const Span outs[3] = {{perm, k * 4}, {rot, k * had_block * 4}, {work, work_bytes}};
    const Span ins[2] = {{w, n * k * dtype_size(w_dtype)}, {fold_s, fold_s ? k * 4 : 0}};
    if (any_overlap(outs, 3, ins, 2)) return QLIN_ERR_ALIAS;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_calibrate_composite(w, w_dtype, n, k, fold_s, had_block, perm, rot, work,
                                                    as_stream(stream)));
}

qlin_status qlin_rotate_quant_act_composite(const void* x, qlin_dtype x_dtype, int64_t m, int64_t k,
                                            int64_t ldx, const float* fold_inv_s, const int32_t* perm,
                                            const float* rot, int32_t had_block, int32_t bits, void* xq,
                                            float* x_scale, float* work, void* stream) {
    qlin_status st = composite_check(x, x_dtype, m, k, ldx, had_block);
    if (st != QLIN_OK) return st;
    if (!perm || !rot) return QLIN_ERR_NULL;
    if (m > 0 && (!xq || !x_scale || !work)) return QLIN_ERR_NULL;
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(fold_inv_s) || !aligned16(perm) || !aligned16(rot) || !aligned16(xq) ||
        !aligned16(x_scale) || !aligned16(work))
        return QLIN_ERR_ALIGN;
    const Span outs[3] = {{xq, code_bytes(m, k, bits)}, {x_scale, m * 4}, {work, m * k * 4}};
    const Span ins[4] = {{x, m > 0 ? ((m - 1) * ldx + k) * dtype_size(x_dtype) : 0},
                         {fold_inv_s, fold_inv_s ? k * 4 : 0}, {perm, k * 4}, {rot, k * had_block * 4}};
    if (any_overlap(outs, 3, ins, 4)) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return composite_run(x, x_dtype, m, k, ldx, fold_inv_s, perm, rot, had_block, bits, xq, x_scale, work, stream);
}

qlin_status qlin_quantize_weights_composite(const void* w, qlin_dtype w_dtype, int64_t n, int64_t k,
                                            const float* fold_s, const int32_t* perm, const float* rot,
                                            int32_t had_block, int32_t bits, void* wq, float* w_scale,
                                            float* work, void* stream) {
    qlin_status st = composite_check(w, w_dtype, n, k, k, had_block);
    if (st != QLIN_OK) return st;
    if (!w || !perm || !rot || !wq || !w_scale || !work) return QLIN_ERR_NULL;
    if (n < 1) return QLIN_ERR_SHAPE;
    if (!bits_ok(bits)) return QLIN_ERR_UNSUPPORTED;
    if (!bits_k_ok(bits, k)) return QLIN_ERR_SHAPE;
    if (!aligned16(w) || !aligned16(fold_s) || !aligned16(perm) || !aligned16(rot) || !aligned16(wq) ||
        !aligned16(w_scale) || !aligned16(work))
        return QLIN_ERR_ALIGN;
    const Span outs[3] = {{wq, code_bytes(n, k, bits)}, {w_scale, n * 4}, {work, n * k * 4}};
    const Span ins[4] = {{w, n * k * dtype_size(w_dtype)}, {fold_s, fold_s ? k * 4 : 0}, {perm, k * 4},
                         {rot, k * had_block * 4}};
    if (any_overlap(outs, 3, ins, 4)) return QLIN_ERR_ALIAS;
    st = check_device();
    if (st != QLIN_OK) return st;
    return composite_run(w, w_dtype, n, k, k, fold_s, perm, rot, had_block, bits, wq, w_scale, work, stream);
}

qlin_status qlin_gemm_w4a4(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                           int64_t m, int64_t n, int64_t k, void* y, qlin_dtype y_dtype, void* stream) {
    return gemm_common(xq, x_scale, wq, w_scale, m, n, k, y, y_dtype, Scratch::None, nullptr, 0, stream, true, false,
                       false);
}

qlin_status qlin_gemm_w8a8(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                           int64_t m, int64_t n, int64_t k, void* y, qlin_dtype y_dtype, void* stream) {
    return gemm_common(xq, x_scale, wq, w_scale, m, n, k, y, y_dtype, Scratch::None, nullptr, 0, stream, false,
                       false, false);
}

qlin_status qlin_gemm_w4a8(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                           int64_t m, int64_t n, int64_t k, void* y, qlin_dtype y_dtype, void* stream) {
    return gemm_common(xq, x_scale, wq, w_scale, m, n, k, y, y_dtype, Scratch::None, nullptr, 0, stream, true, true,
                       false);
}

int64_t qlin_gemm_workspace_bytes(qlin_scheme scheme, int64_t m, int64_t n, int64_t k) {
    bool int4 = false, a8 = false, f6 = false;
    if (!scheme_flags(scheme, &int4, &a8, &f6)) return -1;
    if (!gemm_shape_ok(m, n, k, gemm_k_step(int4, a8, f6))) return -1;
    return gemm_ws_need(m, n, k, int4, a8, f6);
}

qlin_status qlin_gemm_ws(qlin_scheme scheme, const void* xq, const float* x_scale, const void* wq,
                         const float* w_scale, int64_t m, int64_t n, int64_t k, void* y, qlin_dtype y_dtype,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    bool int4 = false, a8 = false, f6 = false;
    if (!scheme_flags(scheme, &int4, &a8, &f6)) return QLIN_ERR_UNSUPPORTED;
    return gemm_common(xq, x_scale, wq, w_scale, m, n, k, y, y_dtype, Scratch::Caller, workspace, workspace_bytes,
                       stream, int4, a8, f6);
}

qlin_status qlin_gemm_w4a4_geglu(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                                 int64_t m, int64_t n2, int64_t k, void* h, qlin_dtype h_dtype, void* stream) {
    return qlin_gemm_geglu(QLIN_W4A4, xq, x_scale, wq, w_scale, m, n2, k, h, h_dtype, stream);
}

qlin_status qlin_gemm_geglu(qlin_scheme scheme, const void* xq, const float* x_scale, const void* wq,
                            const float* w_scale, int64_t m, int64_t n2, int64_t k, void* h, qlin_dtype h_dtype,
                            void* stream) {
    if (scheme != QLIN_W4A4 && scheme != QLIN_W4A4_E2M3) return QLIN_ERR_UNSUPPORTED;
    const bool f6 = scheme == QLIN_W4A4_E2M3;
    if (!xq && m > 0) return QLIN_ERR_NULL;
    if (!wq || !h || !w_scale || (!x_scale && m > 0)) return QLIN_ERR_NULL;
    if (h_dtype != QLIN_F16 && h_dtype != QLIN_BF16 && h_dtype != QLIN_F32) return QLIN_ERR_DTYPE;
    const int64_t kstep = gemm_k_step(true, false, f6);
    if (m < 0 || n2 < 64 || (n2 % 64) != 0 || k < kstep || (k % kstep) != 0 || k >= kMaxGemmK) return QLIN_ERR_SHAPE;
    if (m > 0x7FFFFFFF || n2 > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    if (!aligned16(xq) || !aligned16(wq) || !aligned16(h) || !aligned16(x_scale) || !aligned16(w_scale))
        return QLIN_ERR_ALIGN;
    const int64_t kb = f6 ? k / 4 * 3 : k / 2;
    const Span outs[1] = {{h, m * (n2 / 2) * dtype_size(h_dtype)}};
    const Span ins[4] = {{xq, m * kb}, {wq, n2 * kb}, {x_scale, m * 4}, {w_scale, n2 * 4}};
    if (any_overlap(outs, 1, ins, 4)) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    hipStream_t s = as_stream(stream);
    if (f6)
        return map_err(qlin::launch_gemm_f6(qlin::plan_gemm_f6(m, n2, k, true), xq, x_scale, wq, w_scale, m, n2, k,
                                            h, h_dtype, true, s));
    return map_err(qlin::launch_gemm_geglu(xq, x_scale, wq, w_scale, m, n2, k, true, h, h_dtype, s));
}

qlin_status qlin_gemv_w4a16(const void* x, const void* wq, const void* w_scale, int64_t m, int64_t n,
                            int64_t k, int32_t group, void* y, void* stream) {
    if (m > 0 && (!x || !y)) return QLIN_ERR_NULL;
    if (!wq || !w_scale) return QLIN_ERR_NULL;
    if (group != 128) return QLIN_ERR_UNSUPPORTED;
    if (m < 0 || m > 64 || n < 1 || k < group || (k % group) != 0 || k > 32768) return QLIN_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y)) return QLIN_ERR_ALIGN;
    const Span outs[1] = {{y, m * n * 2}};
    const Span ins[3] = {{x, m * k * 2}, {wq, n * k / 2}, {w_scale, n * (k / group) * 2}};
    if (any_overlap(outs, 1, ins, 3)) return QLIN_ERR_ALIAS;
    if (m == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_gemv_w4a16(x, wq, w_scale, m, n, k, group, y, as_stream(stream)));
}

qlin_status qlin_rope_append_kv(const void* qkv, qlin_dtype dtype, int64_t tokens, int64_t ld, int32_t heads_q,
                                const float* rope, int64_t rope_len, int32_t rot_dim, int32_t interleaved,
                                const int32_t* positions, const qlin_kv_cache* cache, const qlin_kv_batch* batch,
                                void* q_out, int64_t ldq, void* stream) {
    qlin_status st = kv_check(cache, batch, tokens, heads_q);
    if (st != QLIN_OK) return st;
    if (tokens > 0 && (!qkv || !q_out)) return QLIN_ERR_NULL;
    if (rot_dim > 0 && !rope) return QLIN_ERR_NULL;
    if (dtype != QLIN_F16 && dtype != QLIN_BF16) return QLIN_ERR_DTYPE;
    if (interleaved != 0 && interleaved != 1) return QLIN_ERR_UNSUPPORTED;
    const int64_t d = cache->head_dim, wide = (static_cast<int64_t>(heads_q) + 2 * cache->heads) * d;
    if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0 || (rot_dim > 0 && rope_len < 1)) return QLIN_ERR_SHAPE;
    if (ld % 8 != 0 || ld < wide || ldq % 8 != 0 || ldq < heads_q * d) return QLIN_ERR_SHAPE;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(rope)) return QLIN_ERR_ALIGN;
    if (!aligned4(positions)) return QLIN_ERR_ALIGN;
    // one block per (page, head) of k and of v, then the q heads
    const int64_t touched = qlin::kv_max_touched(batch->max_q, cache->page_size);
    if (touched > 0 && static_cast<int64_t>(batch->batch) * cache->heads > (1LL << 29) / touched) return QLIN_ERR_SHAPE;
    const int64_t q_tasks = static_cast<int64_t>(batch->max_q) * heads_q * (d / 16);
    if (q_tasks > (1LL << 31)) return QLIN_ERR_SHAPE;
    // (a launch holds 2^32 threads, and a block at most 256)
    const int64_t threads = touched * cache->heads * 2 * 256 + q_tasks + 256;
    if (batch->batch > 0 && threads > 0xFFFFFFFFLL / batch->batch) return QLIN_ERR_SHAPE;
    const int64_t codes = cache->pages * cache->heads * cache->page_size * d, scales = cache->pages * cache->heads * 4;
    const Span outs[5] = {{cache->k, codes}, {cache->v, codes}, {cache->k_scale, scales}, {cache->v_scale, scales},
                          {q_out, tokens > 0 ? ((tokens - 1) * ldq + heads_q * d) * 2 : 0}};
    Span ins[7] = {{qkv, tokens > 0 ? ((tokens - 1) * ld + wide) * 2 : 0}, {rope, rope_len * rot_dim * 4},
                   {positions, tokens * 4}};
    kv_index_spans(cache, batch, ins + 3);
    if (any_overlap(outs, 5, ins, 7)) return QLIN_ERR_ALIAS;
    if (tokens == 0 || batch->batch == 0 || batch->max_q == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_rope_append(qkv, dtype, ld, heads_q, rope, rope_len, rot_dim, interleaved, positions,
                                            kv_index(cache, batch, tokens), cache->k, cache->v, cache->k_scale,
                                            cache->v_scale, cache->heads, cache->head_dim, q_out, ldq,
                                            as_stream(stream)));
}

int64_t qlin_kv_attention_workspace_bytes(int32_t heads_q, const qlin_kv_cache* cache, const qlin_kv_batch* batch) {
    return attention_bytes(heads_q, cache, batch, false);
}

qlin_status qlin_kv_attention(const void* q, qlin_dtype dtype, int64_t tokens, int64_t ldq, int32_t heads_q,
                              const qlin_kv_cache* cache, const qlin_kv_batch* batch, float sm_scale, float softcap,
                              void* out, int64_t ldo, void* workspace, int64_t workspace_bytes, void* stream) {
    return attention(q, dtype, tokens, ldq, heads_q, cache, batch, false, nullptr, 0, sm_scale, softcap, out, ldo, workspace,
                     workspace_bytes, stream);
}

int64_t qlin_kv_attention_tree_workspace_bytes(int32_t heads_q, const qlin_kv_cache* cache,
                                               const qlin_kv_batch* batch) {
    if (!batch || batch->prefix_len || batch->max_q > qlin::kMaxTreeNodes) return -1;
    return attention_bytes(heads_q, cache, batch, true);
}

qlin_status qlin_kv_attention_tree(const void* q, qlin_dtype dtype, int64_t tokens, int64_t ldq, int32_t heads_q,
                                   const qlin_kv_cache* cache, const qlin_kv_batch* batch, const uint32_t* mask,
                                   int64_t mask_ld, float sm_scale, float softcap, void* out, int64_t ldo,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
    if (!batch || (tokens > 0 && batch->max_q > 0 && !mask)) return QLIN_ERR_NULL;
    if (batch->prefix_len) return QLIN_ERR_UNSUPPORTED;
    if (batch->max_q > qlin::kMaxTreeNodes || mask_ld < (static_cast<int64_t>(batch->max_q) + 31) / 32 ||
        mask_ld > 0x7FFFFFFF)
        return QLIN_ERR_SHAPE;
    if (!aligned4(mask)) return QLIN_ERR_ALIGN;
    return attention(q, dtype, tokens, ldq, heads_q, cache, batch, true, mask, mask_ld, sm_scale, softcap, out, ldo,
                     workspace, workspace_bytes, stream);
}

qlin_status qlin_rope_table(float* table, int64_t positions, int32_t rot_dim, double base, double stretch,
                            void* stream) {
    if (!table) return QLIN_ERR_NULL;
    if (!(base > 0.0) || !(base < 1e300) || !(stretch > 0.0) || !(stretch < 1e300)) return QLIN_ERR_UNSUPPORTED;
    if (positions < 0 || positions > 0x7FFFFFFF || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 1024 ||
        positions * (rot_dim / 2) > 0xFFFFFF00LL)
        return QLIN_ERR_SHAPE;
    if (!aligned16(table)) return QLIN_ERR_ALIGN;
    if (positions == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_rope_table(table, positions, rot_dim, base, stretch, as_stream(stream)));
}

qlin_status qlin_tree_plan(const int32_t* parents, int64_t tokens, const qlin_kv_batch* batch, uint32_t* mask,
                           int64_t mask_ld, int32_t* positions, void* stream) {
    qlin_status st = tree_check(batch, tokens);
    if (st != QLIN_OK) return st;
    if (tokens > 0 && (!parents || (batch->max_q > 0 && !mask) || !positions)) return QLIN_ERR_NULL;
    const int64_t words = (static_cast<int64_t>(batch->max_q) + 31) / 32;
    if (mask_ld < words || mask_ld > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    if (!aligned4(parents) || !aligned4(mask) || !aligned4(positions)) return QLIN_ERR_ALIGN;
    const Span outs[2] = {{mask, tokens > 0 ? ((tokens - 1) * mask_ld + words) * 4 : 0}, {positions, tokens * 4}};
    const Span ins[3] = {{parents, tokens * 4}, {batch->q_start, (batch->batch + 1LL) * 4},
                         {batch->kv_len, batch->batch * 4LL}};
    if (any_overlap(outs, 2, ins, 3)) return QLIN_ERR_ALIAS;
    if (tokens == 0 || batch->batch == 0 || batch->max_q == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_tree_plan(tree_index(batch, tokens), parents, mask, mask_ld, positions, as_stream(stream)));
}

qlin_status qlin_tree_accept(const int32_t* parents, const int32_t* draft, const int32_t* sampled, int64_t tokens,
                             const qlin_kv_batch* batch, int32_t* path, int64_t path_ld, int32_t* count,
                             int32_t* token, void* stream) {
    qlin_status st = tree_check(batch, tokens);
    if (st != QLIN_OK) return st;
    if (tokens > 0 && (!parents || !draft || !sampled)) return QLIN_ERR_NULL;
    const int64_t n = batch->batch;
    if (n > 0 && ((batch->max_q > 0 && !path) || !count || !token)) return QLIN_ERR_NULL;
    if (path_ld < batch->max_q || path_ld > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    if (!aligned4(parents) || !aligned4(draft) || !aligned4(sampled) || !aligned4(path) || !aligned4(count) ||
        !aligned4(token))
        return QLIN_ERR_ALIGN;
    const Span outs[3] = {{path, n > 0 ? ((n - 1) * path_ld + batch->max_q) * 4 : 0}, {count, n * 4}, {token, n * 4}};
    const Span ins[5] = {{parents, tokens * 4}, {draft, tokens * 4}, {sampled, tokens * 4},
                         {batch->q_start, (n + 1) * 4}, {batch->kv_len, n * 4}};
    if (any_overlap(outs, 3, ins, 5)) return QLIN_ERR_ALIAS;
    if (n == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_tree_accept(tree_index(batch, tokens), parents, draft, sampled, path, path_ld, count,
                                            token, as_stream(stream)));
}

int64_t qlin_sample_workspace_bytes(int64_t rows, int64_t vocab) {
    if (rows < 0 || rows > kMaxSampleRows || vocab < 1 || vocab > qlin::kMaxVocab) return -1;
    return qlin::plan_sample(rows, vocab, true).ws_bytes;
}

qlin_status qlin_sample(const void* logits, qlin_dtype dtype, int64_t rows, int64_t vocab, int64_t ld, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                        int32_t* token, float* logprob, void* workspace, int64_t workspace_bytes, void* stream) {
    if (rows > 0 && (!logits || !u || !token)) return QLIN_ERR_NULL;
    if (!is_float_in(dtype)) return QLIN_ERR_DTYPE;
    if (rows < 0 || rows > kMaxSampleRows || vocab < 1 || vocab > qlin::kMaxVocab) return QLIN_ERR_SHAPE;
    const int64_t size = dtype_size(dtype);
    if (ld < vocab || ld > 0x7FFFFFFF || (ld * size) % 16 != 0 || workspace_bytes < 0) return QLIN_ERR_SHAPE;
    if (!workspace && workspace_bytes > 0) return QLIN_ERR_NULL;
    if (!aligned16(logits) || !aligned16(workspace)) return QLIN_ERR_ALIGN;
    if (!aligned4(u) || !aligned4(temperature) || !aligned4(top_k) || !aligned4(top_p) || !aligned4(min_p) ||
        !aligned4(token) || !aligned4(logprob))
        return QLIN_ERR_ALIGN;
    if (workspace && workspace_bytes < qlin::plan_sample(rows, vocab, true).ws_bytes) return QLIN_ERR_WORKSPACE;
    const Span outs[3] = {{token, rows * 4}, {logprob, rows * 4}, {workspace, workspace_bytes}};
    const Span ins[6] = {{logits, rows > 0 ? ((rows - 1) * ld + vocab) * size : 0}, {u, rows * 4},
                         {temperature, rows * 4}, {top_k, rows * 4}, {top_p, rows * 4}, {min_p, rows * 4}};
    if (any_overlap(outs, 3, ins, 6)) return QLIN_ERR_ALIAS;
    if (rows == 0) return QLIN_OK;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    const qlin::SampleArgs a{logits, ld, static_cast<int>(rows), static_cast<int>(vocab), u, temperature, top_k, top_p,
                             min_p, token, logprob};
    return map_err(qlin::launch_sample(a, dtype, workspace, as_stream(stream)));
}

qlin_status qlin_kv_pool_init(const qlin_kv_pool* pool, void* stream) {
    qlin_status st = pool_check(pool);
    if (st != QLIN_OK) return st;
    const Span outs[2] = {{pool->refs, pool->pages * 4}, {pool->free_bits, (pool->pages + 31) / 32 * 4}};
    if (any_overlap(outs, 2, nullptr, 0)) return QLIN_ERR_ALIAS;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_pool_init({pool->refs, pool->free_bits, pool->pages}, as_stream(stream)));
}

qlin_status qlin_kv_resize(const qlin_kv_pool* pool, const qlin_kv_cache* caches, int32_t layers, int32_t page_size,
                           int32_t* page_table, int64_t table_ld, int64_t table_cols, int64_t rows,
                           const int32_t* old_len, const int32_t* new_len, int32_t* len_out, int32_t* moved,
                           void* stream) {
    qlin_status st = pool_check(pool);
    if (st != QLIN_OK) return st;
    st = table_check(page_size, page_table, table_ld, table_cols, rows);
    if (st != QLIN_OK) return st;
    if (layers < 0 || rows > qlin::kMaxPoolRows) return QLIN_ERR_SHAPE;
    if (layers > 0) {
        st = stack_check(caches, layers);
        if (st != QLIN_OK) return st;
        if (caches[0].page_size != page_size || caches[0].pages != pool->pages) return QLIN_ERR_SHAPE;
    }
    if (rows > 0 && (!old_len || !new_len || !len_out || !moved)) return QLIN_ERR_NULL;
    if (!aligned4(old_len) || !aligned4(new_len) || !aligned4(len_out) || !aligned4(moved)) return QLIN_ERR_ALIGN;
    const Span outs[5] = {{pool->refs, pool->pages * 4}, {pool->free_bits, (pool->pages + 31) / 32 * 4},
                          {page_table, rows > 0 ? ((rows - 1) * table_ld + table_cols) * 4 : 0},
                          {len_out, rows * 4}, {moved, rows * 8}};
    const Span ins[2] = {{old_len, rows * 4}, {new_len, rows * 4}};
    if (any_overlap(outs, 5, ins, 2)) return QLIN_ERR_ALIAS;
    if (stack_overlaps(caches, layers, outs, 5) || stack_overlaps(caches, layers, ins, 2)) return QLIN_ERR_ALIAS;
    if (rows == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    st = map_err(qlin::launch_kv_resize({pool->refs, pool->free_bits, pool->pages}, page_table, table_ld,
                                        static_cast<int>(table_cols), static_cast<int>(rows), page_size, old_len,
                                        new_len, len_out, moved, as_stream(stream)));
    for (int32_t at = 0; st == QLIN_OK && at < layers; at += qlin::kMaxStackLayers)
        st = map_err(qlin::launch_kv_copy_pages(stack_args(caches, layers, at), moved, rows, as_stream(stream)));
    return st;
}

qlin_status qlin_kv_fork(const qlin_kv_pool* pool, int32_t page_size, int32_t* page_table, int64_t table_ld,
                         int64_t table_cols, int64_t rows, const int32_t* src, const int32_t* dst,
                         const int32_t* len, int64_t n, void* stream) {
    qlin_status st = pool_check(pool);
    if (st != QLIN_OK) return st;
    st = table_check(page_size, page_table, table_ld, table_cols, rows);
    if (st != QLIN_OK) return st;
    if (n < 0 || n > (1 << 20)) return QLIN_ERR_SHAPE;
    if (n > 0 && (!src || !dst || !len)) return QLIN_ERR_NULL;
    if (!aligned4(src) || !aligned4(dst) || !aligned4(len)) return QLIN_ERR_ALIGN;
    const Span outs[2] = {{pool->refs, pool->pages * 4},
                          {page_table, rows > 0 ? ((rows - 1) * table_ld + table_cols) * 4 : 0}};
    const Span ins[3] = {{src, n * 4}, {dst, n * 4}, {len, n * 4}};
    if (any_overlap(outs, 2, ins, 3)) return QLIN_ERR_ALIAS;
    if (n == 0 || rows == 0) return QLIN_OK;
    st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_kv_fork({pool->refs, pool->free_bits, pool->pages}, page_table, table_ld,
                                        static_cast<int>(table_cols), static_cast<int>(rows), page_size, src, dst, len,
                                        static_cast<int>(n), as_stream(stream)));
}

qlin_status qlin_kv_copy_pages(const qlin_kv_cache* caches, int32_t layers, const int32_t* pairs, int64_t n,
                               void* stream) {
    qlin_status st = stack_check(caches, layers);
    if (st != QLIN_OK) return st;
    if (n < 0 || n > (1 << 24)) return QLIN_ERR_SHAPE;
    if (n > 0 && !pairs) return QLIN_ERR_NULL;
    if (!aligned4(pairs)) return QLIN_ERR_ALIGN;
    const Span ins[1] = {{pairs, n * 8}};
    if (stack_overlaps(caches, layers, ins, 1)) return QLIN_ERR_ALIAS;
    if (n == 0) return QLIN_OK;
    st = check_device();
    for (int32_t at = 0; st == QLIN_OK && at < layers; at += qlin::kMaxStackLayers)
        st = map_err(qlin::launch_kv_copy_pages(stack_args(caches, layers, at), pairs, n, as_stream(stream)));
    return st;
}

qlin_status qlin_kv_compact(const qlin_kv_cache* caches, int32_t layers, const qlin_kv_batch* batch,
                            const int32_t* path, int64_t path_ld, const int32_t* count, int32_t* kv_len_out,
                            void* stream) {
    if (!batch) return QLIN_ERR_NULL;
    qlin_status st = stack_check(caches, layers);
    if (st != QLIN_OK) return st;
    st = kv_check(&caches[0], batch, 0, caches[0].heads);
    if (st != QLIN_OK) return st;
    const int64_t n = batch->batch;
    if (n > 0 && ((batch->max_q > 0 && !path) || !count)) return QLIN_ERR_NULL;
    if (batch->max_q > qlin::kMaxTreeNodes || path_ld < batch->max_q || path_ld > 0x7FFFFFFF) return QLIN_ERR_SHAPE;
    const int64_t wide = layers < qlin::kMaxStackLayers ? layers : qlin::kMaxStackLayers;
    if (n * wide * caches[0].heads > kMaxAttnBlocks) return QLIN_ERR_SHAPE;
    if (!aligned4(path) || !aligned4(count) || !aligned4(kv_len_out)) return QLIN_ERR_ALIGN;
    const Span outs[1] = {{kv_len_out, n * 4}};
    Span ins[6] = {{path, n > 0 ? ((n - 1) * path_ld + batch->max_q) * 4 : 0}, {count, n * 4}};
    kv_index_spans(&caches[0], batch, ins + 2);
    if (any_overlap(outs, 1, ins, 6) || stack_overlaps(caches, layers, ins, 6) || stack_overlaps(caches, layers, outs, 1))
        return QLIN_ERR_ALIAS;
    if (n == 0) return QLIN_OK;
    st = check_device();
    const qlin::KvIndex ix = kv_index(&caches[0], batch, 0x7FFFFFFF);
    for (int32_t at = 0; st == QLIN_OK && at < layers; at += qlin::kMaxStackLayers)
        st = map_err(qlin::launch_kv_compact(ix, stack_args(caches, layers, at), path, path_ld, count,
                                             at == 0 ? kv_len_out : nullptr, as_stream(stream)));
    return st;
}

qlin_status qlin_stream_read(const void* src, int64_t bytes, uint32_t* sink, void* stream) {
    if (!src || !sink) return QLIN_ERR_NULL;
    if (bytes < 16 || (bytes % 16) != 0) return QLIN_ERR_SHAPE;
    if (!aligned16(src) || !aligned16(sink)) return QLIN_ERR_ALIGN;
    const Span outs[1] = {{sink, QLIN_STREAM_READ_SINK_WORDS * 4}};
    const Span ins[1] = {{src, bytes}};
    if (any_overlap(outs, 1, ins, 1)) return QLIN_ERR_ALIAS;
    qlin_status st = check_device();
    if (st != QLIN_OK) return st;
    return map_err(qlin::launch_stream_read(src, bytes, sink, QLIN_STREAM_READ_SINK_WORDS, as_stream(stream)));
}

qlin_status qlin_gemm_static_ws(qlin_scheme scheme, const void* xq, const float* x_scale, const void* wq,
                                const float* w_scale, int64_t m, int64_t n, int64_t k, void* y,
                                qlin_dtype y_dtype, void* stream) {
    bool int4 = false, a8 = false, f6 = false;
    if (!scheme_flags(scheme, &int4, &a8, &f6)) return QLIN_ERR_UNSUPPORTED;
    return gemm_common(xq, x_scale, wq, w_scale, m, n, k, y, y_dtype, Scratch::Static, nullptr, 0, stream, int4,
                       a8, f6);
}

}  // extern "C"
