// fa_kv4.cu -- C-ABI entry points of the quantised K/V cache and of the rotary
// positions (declared in include/fa_gb300.h): argument validation, kernel
// choice and launch.  No device memory is allocated and nothing is
// synchronised.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_gb300.h"
#include "fa_kv4_status.h"
#include "kv4_cache.cuh"
#include "kv4_decode.cuh"
#include "kv4_prompt.cuh"
#include "rotary.cuh"

static_assert(kv4::kStatusTimeout == FA_ERR_TIMEOUT && kv4::kStatusBadSeqlens == FA_ERR_BAD_SEQLENS &&
                  kv4::kStatusBadPages == FA_ERR_BAD_PAGES && rot::kStatusBadAxis == FA_ERR_BAD_AXIS,
              "device status codes");

namespace {

constexpr int kMaxDevices = 64;

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Checks of what every call shares; fills the kernels' description of it.
int check_cache(const fa_kv4_cache_t* d, int dtype, kv4::Cache* c) {
    if (d == nullptr || d->codes == nullptr || d->scales == nullptr || d->page_table == nullptr ||
        d->seq_lens == nullptr)
        return FA_ERR_INVALID_ARG;
    if (d->B < 1 || d->max_seqlen < 1 || d->H_kv < 1 || d->pages < 1 || d->max_pages < 1 || d->page_size < 1)
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    long long total = d->total;
    if (d->cu_seqlens == nullptr) {
        total = static_cast<long long>(d->B) * d->max_seqlen;
        if (d->total != 0 && d->total != total) return FA_ERR_INVALID_ARG;
    } else if (d->total < 1) {
        return FA_ERR_INVALID_ARG;
    }
    if (d->D < kv4::kGroup || d->D > 8 * kv4::kGroup || d->D % kv4::kGroup != 0) return FA_ERR_UNSUPPORTED;
    if (d->page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
    // rows, tokens of the cache and tokens of a sequence are numbered with an int
    // (and a few tiles past the last token are looked at)
    if (total > 0x7fffffffLL - 4 || static_cast<long long>(d->pages) * d->page_size > 0x7fffffffLL ||
        static_cast<long long>(d->max_pages) * d->page_size > 0x7fffffffLL - 4096)
        return FA_ERR_UNSUPPORTED;
    if (misaligned(d->codes, 16) || misaligned(d->scales, 16) || misaligned(d->page_table, 4) ||
        misaligned(d->seq_lens, 4) || misaligned(d->cu_seqlens, 4))
        return FA_ERR_UNSUPPORTED;
    c->codes = static_cast<uint8_t*>(d->codes);
    c->scales = static_cast<uint16_t*>(d->scales);
    c->table = d->page_table;
    c->lens = d->seq_lens;
    c->cu = d->cu_seqlens;
    c->B = d->B;
    c->S = d->max_seqlen;
    c->total = static_cast<int>(total);
    c->pages = d->pages;
    c->max_pages = d->max_pages;
    c->P = d->page_size;
    c->Hkv = d->H_kv;
    return FA_OK;
}

// Strides (in elements) of a 16-bit tensor [batch, row, head, D] whose last
// axis is contiguous, against the accesses of `unit` elements.
bool bad_strides(const long long* s, int unit) {
    return s[0] % unit != 0 || s[1] % unit != 0 || s[2] % unit != 0;
}

// Blocks of a launch over the call's rows, K and V of every head (0: too
// many), and how many of a token's rows a warp takes: one while that does not fill
// the GPU (16 warps an SM; a step of 64 tokens, 16 rows each: 8.2 us with four
// rows a warp, one after the other, 3.1 us with one), up to kRows where the
// search for the token's place is to be shared.
template <int NG, int LANES>
unsigned row_blocks(const kv4::Cache& c, int* per) {
    constexpr int TOK = 32 / LANES;
    const long long groups = (static_cast<long long>(c.total) + TOK - 1) / TOK, rows = 2LL * c.Hkv;
    *per = static_cast<int>(std::max<long long>(1, std::min<long long>(kv4::kRows<NG, LANES>, groups * rows / (152 * 16))));
    const long long warps = groups * ((rows + *per - 1) / *per);
    const long long blocks = (warps + kv4::kRowThreads / 32 - 1) / (kv4::kRowThreads / 32);
    return blocks > 0x7fffffffLL ? 0u : static_cast<unsigned>(blocks);
}

int launched() { return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// SMs of the current device and how many CTAs of `kernel` one holds, looked
// up once for each device; some launches may take `smem_more` bytes besides.
struct Resident {
    std::once_flag once[kMaxDevices];
    int sms[kMaxDevices] = {}, ctas[kMaxDevices] = {};
};

template <typename Kernel>
bool resident(Resident& r, Kernel* kernel, int threads, int smem, int* sms, int* ctas, int smem_more = 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::call_once(r.once[dev], [&] {
        int n = 0, k = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + smem_more) != cudaSuccess) return;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, kernel, threads, smem) != cudaSuccess) return;
        r.sms[dev] = n;
        r.ctas[dev] = k;
    });
    *sms = r.sms[dev];
    *ctas = r.ctas[dev];
    return *sms > 0 && *ctas > 0;
}

// How a call of the attention is laid out over the GPU.
struct DecodePlan {
    int grid = 0;
    int items_most = 0;      // of a sequence
    size_t bytes = 0;        // workspace
};

template <int NG, int NT, bool BF16>
int decode(const kv4::Cache& c, kv4::Attend a, void* ws, size_t ws_bytes, DecodePlan* only_plan, cudaStream_t st) {
    constexpr int R = 8 * NT, D = NG * kv4::kGroup;
    static Resident res;
    auto* kernel = kv4::decode_kernel<NG, NT, BF16>;
    constexpr int smem = kv4::kDecodeSmem<NG, NT>;
    int sms = 0, ctas = 0;
    if (!resident(res, kernel, kv4::kThreads, smem, &sms, &ctas, kv4::kClusterSmem<NG, NT>)) return FA_ERR_CUDA;
    DecodePlan plan;
    const long long items = (static_cast<long long>(c.S) * a.G + R - 1) / R * c.Hkv;
    const long long blocks = (static_cast<long long>(c.max_pages) * c.P + 2 * kv4::kBlock - 1) / kv4::kBlock;
    // items of a call, and blocks of a sequence, are numbered with an int
    if (items * c.B > 0x7fffffffLL || items * blocks > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    plan.items_most = static_cast<int>(items);
    // Contexts of at most kWholeBlocks blocks for each CTA of a cluster, where
    // the clusters take no more than two rounds of the GPU: a cluster an item.
    // Else the blocks are cut into ranges and a second launch joins the parts.
    int cluster = 1;
    while (cluster < kv4::kMaxCluster && blocks > static_cast<long long>(kv4::kWholeBlocks) * cluster + 1) cluster *= 2;
    const bool whole = blocks <= static_cast<long long>(kv4::kWholeBlocks) * cluster + 1 &&
                       (cluster == 1 || items * c.B * cluster <= 2LL * sms * ctas);
    if (whole && items * c.B * cluster > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const long long most = whole ? items * c.B * cluster : (items * c.B * blocks + kv4::kWarps - 1) / kv4::kWarps;
    plan.grid = static_cast<int>(whole ? most : std::min<long long>(most, static_cast<long long>(sms) * ctas));
    const size_t slots = whole ? 0 : static_cast<size_t>(plan.grid) * 2 * R;
    plan.bytes = slots * (D * sizeof(float) + sizeof(float2));
    if (only_plan != nullptr) {
        *only_plan = plan;
        return FA_OK;
    }
    if (plan.bytes > 0 && (ws == nullptr || ws_bytes < plan.bytes)) return FA_ERR_INVALID_ARG;
    if (misaligned(ws, 16)) return FA_ERR_UNSUPPORTED;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + slots * D);
    a.grid = plan.grid;
    a.whole = whole ? plan.items_most : 0;
    a.cluster = whole ? cluster : 1;
    if (whole && cluster > 1) {
        cudaLaunchAttribute dim[1];
        dim[0].id = cudaLaunchAttributeClusterDimension;
        dim[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        dim[0].val.clusterDim.y = dim[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
        cfg.blockDim = dim3(kv4::kThreads);
        cfg.dynamicSmemBytes = smem + kv4::kClusterSmem<NG, NT>;
        cfg.stream = st;
        cfg.attrs = dim;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, c, a) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    kernel<<<plan.grid, kv4::kThreads, smem, st>>>(c, a);
    if (launched() != FA_OK) return FA_ERR_CUDA;
    if (whole) return FA_OK;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.items_most) * c.B);
    cfg.blockDim = dim3(kv4::kJoinWarps * 32);
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4::combine_kernel<NG, NT, BF16>, c, a, plan.items_most) == cudaSuccess
               ? FA_OK : FA_ERR_CUDA;
}

// Query rows a K/V head (the group's heads times the call's tokens) up to
// which decode_kernel takes a call: it reads the cache once for every 8 or 16
// rows, prompt_kernel once for 128 or 256, for the price of that many.  us at 32 /
// 64 rows, decode against prompt: 16 x 8192 keys, 8 heads, D = 64 84 / 150
// against 131, D = 128 113 / 199 against 139, D = 256 236 / 449 against 318; 64 x 2048
// keys, D = 128 117 / 192 against 106.
constexpr int kDecodeRows = 32;

template <int NG, bool BF16>
int prompt(const kv4::Cache& c, kv4::Attend a, void* ws, size_t ws_bytes, DecodePlan* only_plan, cudaStream_t st) {
    using L = kv4::Prompt<NG>;
    constexpr int R = L::TILES * kv4::kRowTile;
    static Resident res;
    auto* kernel = kv4::prompt_kernel<NG, BF16>;
    int sms = 0, ctas = 0;
    if (!resident(res, kernel, L::kThreads, L::kSmem, &sms, &ctas)) return FA_ERR_CUDA;
    kv4::PromptPlan plan;
    const long long tiles = (static_cast<long long>(c.S) * a.G + R - 1) / R, items = tiles * c.Hkv * c.B;
    const long long keys = (static_cast<long long>(c.max_pages) * c.P + L::kGroupKeys - 1) / L::kGroupKeys;   // groups
    plan.tiles_most = static_cast<int>(tiles);
    // The items behind the last whole wave of CTAs share their keys out so that
    // the SMs end together: s CTAs an item, each with its share of the groups of
    // keys (4 at least) and about three groups' time to start and end, and a second launch.
    const long long whole = items / sms * sms, rest = items - whole;
    long long best = rest > 0 ? keys + 3 : 0;
    plan.whole = static_cast<int>(std::min<long long>(items, 0x7fffffff));
    plan.splits = 1;
    for (long long s = 2; s <= std::min<long long>(sms, keys / 4) && rest > 0; ++s) {
        const long long cost = (rest * s + sms - 1) / sms * ((keys + s - 1) / s + 3) + 4;
        if (cost < best) {
            best = cost;
            plan.whole = static_cast<int>(whole);
            plan.splits = static_cast<int>(s);
        }
    }
    const long long split_items = plan.splits > 1 ? rest : 0;
    const long long grid = items - split_items + split_items * plan.splits;
    if (grid > 0x7fffffffLL || items * L::TILES * NG > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const size_t slots = static_cast<size_t>(split_items) * plan.splits * R;
    DecodePlan sizes;
    sizes.bytes = slots * (L::D * sizeof(float) + sizeof(float2));
    if (only_plan != nullptr) {
        *only_plan = sizes;
        return FA_OK;
    }
    if (sizes.bytes > 0 && (ws == nullptr || ws_bytes < sizes.bytes)) return FA_ERR_INVALID_ARG;
    if (misaligned(ws, 16)) return FA_ERR_UNSUPPORTED;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + slots * L::D);
    kernel<<<static_cast<unsigned>(grid), L::kThreads, L::kSmem, st>>>(c, a, plan);
    if (launched() != FA_OK) return FA_ERR_CUDA;
    if (plan.splits == 1) return FA_OK;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split_items * L::TILES * NG));
    cfg.blockDim = dim3(kv4::kRowTile);
    cfg.stream = st;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4::prompt_combine_kernel<NG, BF16>, c, a, plan) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// <groups of a row, tiles of 8 query rows, bf16>
// Tiles of 16 rows are for D <= 128 only: with D = 256 the accumulators of 16
// rows would not fit the registers beside the rest.
int decode_any(int D, bool bf16, const kv4::Cache& c, const kv4::Attend& a, void* ws, size_t ws_bytes,
               DecodePlan* only_plan, cudaStream_t st) {
    const long long rows = static_cast<long long>(c.S) * a.G;   // numbered with an int
    if (rows > 0x7fffffffLL - 1024) return FA_ERR_UNSUPPORTED;
    if (rows > kDecodeRows) {
#define KV4_ONE(NG_)                                                                              \
    case NG_:                                                                                     \
        return bf16 ? prompt<NG_, true>(c, a, ws, ws_bytes, only_plan, st)                        \
                    : prompt<NG_, false>(c, a, ws, ws_bytes, only_plan, st)
        switch (D / kv4::kGroup) {
            KV4_ONE(1); KV4_ONE(2); KV4_ONE(3); KV4_ONE(4); KV4_ONE(5); KV4_ONE(6); KV4_ONE(7); KV4_ONE(8);
            default: return FA_ERR_UNSUPPORTED;
        }
#undef KV4_ONE
    }
    const bool wide = rows > 8;
#define KV4_TWO(NG_)                                                                              \
    case NG_:                                                                                     \
        if (wide && bf16) return decode<NG_, 2, true>(c, a, ws, ws_bytes, only_plan, st);         \
        if (wide) return decode<NG_, 2, false>(c, a, ws, ws_bytes, only_plan, st);                \
        return bf16 ? decode<NG_, 1, true>(c, a, ws, ws_bytes, only_plan, st)                     \
                    : decode<NG_, 1, false>(c, a, ws, ws_bytes, only_plan, st)
#define KV4_ONE(NG_)                                                                              \
    case NG_:                                                                                     \
        return bf16 ? decode<NG_, 1, true>(c, a, ws, ws_bytes, only_plan, st)                     \
                    : decode<NG_, 1, false>(c, a, ws, ws_bytes, only_plan, st)
    switch (D / kv4::kGroup) {
        KV4_TWO(1); KV4_TWO(2); KV4_TWO(3); KV4_TWO(4); KV4_ONE(5); KV4_ONE(6); KV4_ONE(7); KV4_ONE(8);
        default: return FA_ERR_UNSUPPORTED;
    }
#undef KV4_ONE
#undef KV4_TWO
}

template <int NG>
int write(const kv4::Cache& c, kv4::RowIo io, bool bf16, cudaStream_t st) {
    const unsigned blocks = row_blocks<NG, kv4::kWriteLanes>(c, &io.per);
    if (blocks == 0) return FA_ERR_UNSUPPORTED;
    const bool values = io.k_out != nullptr;
    if (bf16) {
        if (values) kv4::write_kernel<NG, true, true><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
        else kv4::write_kernel<NG, true, false><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
    } else {
        if (values) kv4::write_kernel<NG, false, true><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
        else kv4::write_kernel<NG, false, false><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
    }
    return launched();
}

template <int NG>
int read(const kv4::Cache& c, kv4::RowIo io, bool bf16, cudaStream_t st) {
    const unsigned blocks = row_blocks<NG, kv4::kReadLanes>(c, &io.per);
    if (blocks == 0) return FA_ERR_UNSUPPORTED;
    if (bf16) kv4::read_kernel<NG, true><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
    else kv4::read_kernel<NG, false><<<blocks, kv4::kRowThreads, 0, st>>>(c, io);
    return launched();
}

template <int VEC, bool INTER>
int rotate(const rot::Rotary& p, bool bf16, unsigned blocks, size_t smem, cudaStream_t st) {
    if (bf16) rot::rotary_kernel<VEC, INTER, true><<<blocks, rot::kThreads, smem, st>>>(p);
    else rot::rotary_kernel<VEC, INTER, false><<<blocks, rot::kThreads, smem, st>>>(p);
    return launched();
}

}  // namespace

extern "C" {

int fa_kv4_write(const fa_kv4_cache_t* cache, const void* K, const void* V, const long long* k_strides,
                 const long long* v_strides, void* K_out, void* V_out, int dtype, fa_stream_t stream) {
    kv4::Cache c;
    const int v = check_cache(cache, dtype, &c);
    if (v != FA_OK) return v;
    if (K == nullptr || V == nullptr || k_strides == nullptr || v_strides == nullptr ||
        (K_out == nullptr) != (V_out == nullptr))
        return FA_ERR_INVALID_ARG;
    if (misaligned(K, 8) || misaligned(V, 8) || misaligned(K_out, 8) || misaligned(V_out, 8) ||
        bad_strides(k_strides, 4) || bad_strides(v_strides, 4))
        return FA_ERR_UNSUPPORTED;
    const kv4::RowIo io = {K, V, k_strides[0], k_strides[1], k_strides[2], v_strides[0], v_strides[1],
                           v_strides[2], K_out, V_out,
                           !misaligned(K, 16) && !misaligned(V, 16) && !misaligned(K_out, 16) && !misaligned(V_out, 16) &&
                               !bad_strides(k_strides, 8) && !bad_strides(v_strides, 8),
                           1};
#define KV4_ONE(NG_) case NG_: return write<NG_>(c, io, dtype == FA_BF16, reinterpret_cast<cudaStream_t>(stream))
    switch (cache->D / kv4::kGroup) {
        KV4_ONE(1); KV4_ONE(2); KV4_ONE(3); KV4_ONE(4); KV4_ONE(5); KV4_ONE(6); KV4_ONE(7); KV4_ONE(8);
        default: return FA_ERR_UNSUPPORTED;
    }
#undef KV4_ONE
}

int fa_kv4_read(const fa_kv4_cache_t* cache, void* K, void* V, int dtype, fa_stream_t stream) {
    kv4::Cache c;
    const int v = check_cache(cache, dtype, &c);
    if (v != FA_OK) return v;
    if (K == nullptr || V == nullptr) return FA_ERR_INVALID_ARG;
    if (misaligned(K, 16) || misaligned(V, 16)) return FA_ERR_UNSUPPORTED;
    kv4::RowIo io = {};
    io.k_out = K;
    io.v_out = V;
#define KV4_ONE(NG_) case NG_: return read<NG_>(c, io, dtype == FA_BF16, reinterpret_cast<cudaStream_t>(stream))
    switch (cache->D / kv4::kGroup) {
        KV4_ONE(1); KV4_ONE(2); KV4_ONE(3); KV4_ONE(4); KV4_ONE(5); KV4_ONE(6); KV4_ONE(7); KV4_ONE(8);
        default: return FA_ERR_UNSUPPORTED;
    }
#undef KV4_ONE
}

int fa_kv4_attention_workspace_size(const fa_kv4_cache_t* cache, int H, int dtype, size_t* bytes) {
    kv4::Cache c;
    const int v = check_cache(cache, dtype, &c);
    if (v != FA_OK) return v;
    if (bytes == nullptr || H < 1 || H % c.Hkv != 0) return FA_ERR_INVALID_ARG;
    kv4::Attend a = {};
    a.H = H;
    a.G = H / c.Hkv;
    DecodePlan plan;
    const int rc = decode_any(cache->D, dtype == FA_BF16, c, a, nullptr, 0, &plan, nullptr);
    *bytes = plan.bytes;
    return rc;
}

int fa_kv4_attention(const fa_kv4_cache_t* cache, const void* Q, const long long* q_strides, void* O, float* LSE,
                     int H, int window_left, float scale, int dtype, void* workspace, size_t workspace_bytes,
                     fa_stream_t stream) {
    kv4::Cache c;
    const int v = check_cache(cache, dtype, &c);
    if (v != FA_OK) return v;
    if (Q == nullptr || O == nullptr || q_strides == nullptr || H < 1 || H % c.Hkv != 0 || window_left < -1 ||
        !std::isfinite(scale) || !(scale > 0.f))
        return FA_ERR_INVALID_ARG;
    if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(LSE, 4) || bad_strides(q_strides, 8))
        return FA_ERR_UNSUPPORTED;
    kv4::Attend a = {};
    a.q = Q;
    a.q_batch = q_strides[0];
    a.q_row = q_strides[1];
    a.q_head = q_strides[2];
    a.o = O;
    a.lse = LSE;
    a.lse_batch = c.cu != nullptr ? 0 : static_cast<long long>(H) * c.S;
    a.lse_head = c.cu != nullptr ? c.total : c.S;
    a.scale = scale;
    a.H = H;
    a.G = H / c.Hkv;
    a.window = window_left;
    return decode_any(cache->D, dtype == FA_BF16, c, a, workspace, workspace_bytes, nullptr,
                      reinterpret_cast<cudaStream_t>(stream));
}

int fa_rotary(const void* X, const long long* x_strides, void* Y, const long long* y_strides, int H,
              const void* X2, const long long* x2_strides, void* Y2, const long long* y2_strides, int H2,
              const int* positions, const double* inv_freq, const int* axes, int T, int n_axes, int n_freq, int D,
              int interleaved, int inverse, int dtype, fa_stream_t stream) {
    if (X == nullptr || Y == nullptr || x_strides == nullptr || y_strides == nullptr || positions == nullptr ||
        inv_freq == nullptr || axes == nullptr)
        return FA_ERR_INVALID_ARG;
    if (T < 1 || H < 1 || H2 < 0 || n_axes < 1 || n_freq < 1 || D < 1 || 2LL * n_freq > D) return FA_ERR_INVALID_ARG;
    if (H2 > 0 && (X2 == nullptr || Y2 == nullptr || x2_strides == nullptr || y2_strides == nullptr))
        return FA_ERR_INVALID_ARG;
    if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (n_freq > rot::kMaxFreqs || D > 2 * rot::kMaxFreqs || H > 65535 || H2 > 65535) return FA_ERR_UNSUPPORTED;
    if (misaligned(X, 2) || misaligned(Y, 2) || misaligned(X2, 2) || misaligned(Y2, 2) || misaligned(positions, 4) ||
        misaligned(inv_freq, 8) || misaligned(axes, 4))
        return FA_ERR_UNSUPPORTED;
    rot::Rotary p = {};
    p.x[0] = X;
    p.y[0] = Y;
    p.x_row[0] = x_strides[0];
    p.x_head[0] = x_strides[1];
    p.y_row[0] = y_strides[0];
    p.y_head[0] = y_strides[1];
    p.heads[0] = H;
    bool wide = n_freq % 8 == 0 && D % 8 == 0 && !misaligned(X, 16) && !misaligned(Y, 16) &&
                (x_strides[0] | x_strides[1] | y_strides[0] | y_strides[1]) % 8 == 0;
    if (H2 > 0) {
        p.x[1] = X2;
        p.y[1] = Y2;
        p.x_row[1] = x2_strides[0];
        p.x_head[1] = x2_strides[1];
        p.y_row[1] = y2_strides[0];
        p.y_head[1] = y2_strides[1];
        p.heads[1] = H2;
        wide = wide && !misaligned(X2, 16) && !misaligned(Y2, 16) &&
               (x2_strides[0] | x2_strides[1] | y2_strides[0] | y2_strides[1]) % 8 == 0;
    }
    p.pos = positions;
    p.inv_freq = inv_freq;
    p.axes = axes;
    p.T = T;
    p.A = n_axes;
    p.F = n_freq;
    p.D = D;
    p.inverse = inverse != 0;
    // enough tokens a CTA to give every thread units, while the CTAs
    // still fill the GPU (152 SMs, 8 CTAs each)
    const int vec = wide ? 8 : 1;
    const int per_token = (H + H2 + rot::kUnroll - 1) / rot::kUnroll * (n_freq / vec + (D - 2 * n_freq + 2 * vec - 1) / (2 * vec));
    int tokens = rot::kThreads / per_token;
    tokens = std::min(tokens, T / (152 * 8));
    p.tokens = std::max(1, std::min(tokens, rot::kMaxAngles / n_freq));
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(T) + p.tokens - 1) / p.tokens);
    const size_t smem = static_cast<size_t>(p.tokens + 1) * n_freq * sizeof(float2);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == FA_BF16;
    if (wide) return interleaved ? rotate<8, true>(p, bf16, blocks, smem, st) : rotate<8, false>(p, bf16, blocks, smem, st);
    return interleaved ? rotate<1, true>(p, bf16, blocks, smem, st) : rotate<1, false>(p, bf16, blocks, smem, st);
}

}  // extern "C"

// ---- the status word, for fa_device_status and fa_last_device_status
int fa_kv4_status_read(int clear, int* value) {
    if (cudaMemcpyFromSymbol(value, kv4::g_kv4_status, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
    const int zero = 0;
    if (clear && cudaMemcpyToSymbol(kv4::g_kv4_status, &zero, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
}

int fa_kv4_status_read_async(int* value, fa_stream_t stream) {
    return cudaMemcpyFromSymbolAsync(value, kv4::g_kv4_status, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                     reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK : FA_ERR_CUDA;
}
