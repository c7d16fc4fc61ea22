// jamba_ssm_serve.cu -- host side of the C ABI declared in
// include/jamba_ssm_serve.h: argument validation and the launches of the 8-bit
// product's and the batch maps' kernels.  Built as its own library, so its
// kernels and status word form a module of their own.  Nothing here allocates
// device memory.
#include "jamba_ssm_serve.h"

#include "batch_maps.cuh"
#include "host_utils.h"
#include "i8_proj.cuh"
#include "i8_quant.cuh"

#define JSSM_SERVE_API extern "C" __attribute__((visibility("default")))

using namespace jssm_host;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - (int64_t(1) << 16);
constexpr uint64_t kDefaultTimeoutCycles = 4000000000ull;  // about 2 s

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn(jamba_ssm_status *st) {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (err == cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else if (err == cudaSuccess)
            err = cudaErrorSymbolNotFound;
    });
    if (!fn) *st = cuda_fail(err);
    return fn;
}

// Map over [rows][pitch] bytes, box of 128 bytes x box_rows, 128-byte swizzle,
// zeros outside the tensor.
bool encode_bytes(EncodeTiledFn fn, CUtensorMap *map, const void *ptr, int64_t pitch, int64_t rows,
                  int box_rows) {
    cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Kernel {
    const void *fn;
    int smem, threads;
};

// Raises a kernel's dynamic shared-memory limit, once per kernel and device.
cudaError_t raise_smem(const Kernel &k, int dev) {
    static std::mutex mutex;
    static const void *done[kMaxDevices][16];
    std::lock_guard<std::mutex> lock(mutex);
    for (const void *&slot : done[dev]) {
        if (slot == k.fn) return cudaSuccess;
        if (slot == nullptr) {
            const cudaError_t e =
                cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
            if (e == cudaSuccess) slot = k.fn;
            return e;
        }
    }
    return cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
}

template <typename T, int LANES> const void *quant_kernel_l(bool vec) {
    return vec ? (const void *)&jssm::i8_quant_kernel<T, LANES, true>
               : (const void *)&jssm::i8_quant_kernel<T, LANES, false>;
}
template <typename T> const void *quant_kernel(int lanes, bool vec) {
    return lanes == 32 ? quant_kernel_l<T, 32>(vec)
         : lanes == 128 ? quant_kernel_l<T, 128>(vec)
                        : quant_kernel_l<T, 256>(vec);
}

template <typename T> Kernel split_kernel(int nt) {
    switch (nt) {
        case 16: return {(const void *)&jssm::i8_proj_split_kernel<T, 16>, jssm::I8SplitCfg<16>::kSmem, 192};
        case 32: return {(const void *)&jssm::i8_proj_split_kernel<T, 32>, jssm::I8SplitCfg<32>::kSmem, 192};
        case 64: return {(const void *)&jssm::i8_proj_split_kernel<T, 64>, jssm::I8SplitCfg<64>::kSmem, 192};
        default: return {(const void *)&jssm::i8_proj_split_kernel<T, 128>, jssm::I8SplitCfg<128>::kSmem, 192};
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of a tile and CTAs to a tile's K; nt = 0: the pairs' kernel.
struct ProjCut {
    int nt, ks;
    int64_t tiles;
};

// The cut that should take the least time.  Measured, in us: a 128-byte block of
// K takes a CTA 0.3 whatever the tokens (its 128 rows of the weight come from
// HBM as single lines); a tile's start, first copy and outputs 2 + nt / 64; the
// exchange of a split K 1.3; the pairs' kernel 5 once and a round of its tiles
// 0.26 a block, or 3.5 where the outputs take longer.  A wave is as many CTAs as
// run at once, with clusters of 4 and 8 fewer than the SMs, whose groups they
// leave partly empty (128 x 1024 x 1024 in 8 ways: 9.6 us for 128 tokens, one
// wave, 17 for 200, two).  E.g. 200 tokens, K 1024, 1024 channels: 64-token
// tiles in 4 ways 7.5, 128-token tiles in 4 and 8 ways 9.1 and 14, pairs 10.
ProjCut choose_proj(int64_t ntok, int64_t n_out, int kblocks, int sms) {
    ProjCut best{0, 1, ceil_div(n_out, 256) * ceil_div(ntok, 256)};
    const double round = 0.26 * kblocks > 3.5 ? 0.26 * kblocks : 3.5;
    double least = ntok <= 64 ? 1e30 : 5.0 + double(ceil_div(best.tiles, sms / 2)) * round;
    for (int nt : {16, 32, 64, 128}) {
        if (nt < 64 && ntok > nt) continue;  // 16 and 32 for that few tokens only
        const int64_t tiles = ceil_div(n_out, 128) * ceil_div(ntok, nt);
        for (int ks = 1; ks <= jssm::kI8MaxSplit && ks <= kblocks; ks *= 2) {
            const int64_t at_once = ks == 8 ? sms * 3 / 4 : ks == 4 ? sms * 15 / 16 : sms;
            const double us = double(ceil_div(tiles * ks, at_once)) *
                              (2.0 + nt / 64.0 + 0.3 * double(ceil_div(kblocks, ks)) + (ks > 1 ? 1.3 : 0.0));
            if (us < least) {
                least = us;
                best = {nt, ks, tiles};
            }
        }
        if (ntok <= nt) break;  // more columns would be empty
    }
    return best;
}

bool io_dtype(int32_t d) { return d == JAMBA_SSM_BF16 || d == JAMBA_SSM_F32; }

}  // namespace

JSSM_SERVE_API jamba_ssm_status jamba_ssm_i8_quant(const jamba_ssm_i8_quant_params *pin, void *stream) {
    jamba_ssm_i8_quant_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.rows < 0 || p.k < 1 || p.reserved != 0 || !io_dtype(p.x_dtype)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.x_stride == 0) p.x_stride = p.k;
    if (p.x_stride < p.k) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.rows > kMaxRows || p.k > JAMBA_SSM_I8_MAX_K || p.x_stride > (int64_t(1) << 31))
        return JAMBA_SSM_ERR_UNSUPPORTED;
    if (p.rows == 0) return JAMBA_SSM_OK;  // no work; the pointers are not used
    if (!p.x || !p.q || !p.scale) return JAMBA_SSM_ERR_INVALID_ARG;
    const int es = p.x_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p.x, es) || !aligned(p.q, 16) || !aligned(p.scale, 4)) return JAMBA_SSM_ERR_MISALIGNED;
    const int64_t pitch = JAMBA_SSM_I8_PITCH(p.k);
    const Range ins[] = {{p.x, size_t((p.rows - 1) * p.x_stride + p.k) * es}};
    const Range outs[] = {{p.q, size_t(p.rows) * pitch}, {p.scale, size_t(p.rows) * 4}};
    if (any_overlap(outs, 2, ins, 1)) return JAMBA_SSM_ERR_INVALID_ARG;
    jamba_ssm_status st;
    if (!current_device(&st)) return st;
    jssm::I8QuantArgs a{};
    a.x = p.x;
    a.xs = p.x_stride;
    a.q = p.q;
    a.scale = p.scale;
    a.rows = p.rows;
    a.k = static_cast<int>(p.k);
    a.pitch = static_cast<int>(pitch);
    void *args[] = {&a};
    // the fewest threads that keep the whole row in registers
    const int per = 8 * jssm::kQuantKept;
    const int lanes = p.k <= 32 * per ? 32 : p.k <= 128 * per ? 128 : 256;
    const bool vec = aligned(p.x, 16) && p.x_stride * es % 16 == 0;
    const void *k = p.x_dtype == JAMBA_SSM_BF16 ? quant_kernel<__nv_bfloat16>(lanes, vec)
                                                : quant_kernel<float>(lanes, vec);
    st = launch_early(k, dim3(unsigned(ceil_div(p.rows, jssm::kQuantThreads / lanes))),
                      jssm::kQuantThreads, 0, 1, args, stream);
    return st != JAMBA_SSM_OK ? st : finish_launch(stream, nullptr);
}

JSSM_SERVE_API jamba_ssm_status jamba_ssm_i8_proj(const jamba_ssm_i8_proj_params *pin, void *stream) {
    jamba_ssm_i8_proj_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.ntok < 0 || p.k < 1 || p.n_out < 1 || p.reserved != 0 || !io_dtype(p.out_dtype))
        return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.ntok > kMaxRows || p.k > JAMBA_SSM_I8_MAX_K || p.n_out > (int64_t(1) << 24))
        return JAMBA_SSM_ERR_UNSUPPORTED;
    if (p.ntok == 0) return JAMBA_SSM_OK;  // no work; the pointers are not used
    if (!p.q || !p.q_scale || !p.w || !p.w_scale || !p.out) return JAMBA_SSM_ERR_INVALID_ARG;
    const int es = p.out_dtype == JAMBA_SSM_BF16 ? 2 : 4;
    if (!aligned(p.q, 16) || !aligned(p.w, 16) || !aligned(p.q_scale, 4) || !aligned(p.w_scale, 4) ||
        !aligned(p.bias, 4) || !aligned(p.out, es))
        return JAMBA_SSM_ERR_MISALIGNED;
    const int64_t pitch = JAMBA_SSM_I8_PITCH(p.k);
    const Range ins[] = {{p.q, size_t(p.ntok) * pitch},
                         {p.w, size_t(p.n_out) * pitch},
                         {p.q_scale, size_t(p.ntok) * 4},
                         {p.w_scale, size_t(p.n_out) * 4},
                         {p.bias, size_t(p.n_out) * 4}};
    const Range outs[] = {{p.out, size_t(p.ntok) * p.n_out * es}};
    if (any_overlap(outs, 1, ins, 5)) return JAMBA_SSM_ERR_INVALID_ARG;
    jamba_ssm_status st;
    const DeviceInfo *dev = current_device(&st);
    if (!dev) return st;
    EncodeTiledFn fn = encode_fn(&st);
    if (!fn) return st;
    jssm::I8ProjArgs a{};
    a.qs = p.q_scale;
    a.ws = p.w_scale;
    a.bias = p.bias;
    a.out = p.out;
    a.ntok = static_cast<int>(p.ntok);
    a.n = static_cast<int>(p.n_out);
    a.kblocks = static_cast<int>(ceil_div(pitch, 128));
    a.limit = p.timeout_cycles ? p.timeout_cycles : kDefaultTimeoutCycles;
    a.withhold = (p.debug_flags & 1u) ? 0xffu : 0u;
    const bool bf = p.out_dtype == JAMBA_SSM_BF16;
    a.pairs = bf && p.n_out % 2 == 0 && aligned(p.out, 4);
    CUtensorMap map_w, map_q;
    if (!encode_bytes(fn, &map_w, p.w, pitch, p.n_out, 128)) return cuda_fail(cudaErrorInvalidValue);

    Kernel k;
    int64_t grid;
    const ProjCut cut = choose_proj(p.ntok, p.n_out, a.kblocks, dev->sms);
    if (cut.nt == 0) {
        if (!encode_bytes(fn, &map_q, p.q, pitch, p.ntok, 128)) return cuda_fail(cudaErrorInvalidValue);
        k = bf ? Kernel{(const void *)&jssm::i8_proj_pair_kernel<__nv_bfloat16>, jssm::I8PairCfg::kSmem,
                        jssm::I8PairCfg::kThreads}
               : Kernel{(const void *)&jssm::i8_proj_pair_kernel<float>, jssm::I8PairCfg::kSmem,
                        jssm::I8PairCfg::kThreads};
        grid = 2 * (cut.tiles < dev->sms / 2 ? cut.tiles : dev->sms / 2);
    } else {
        if (!encode_bytes(fn, &map_q, p.q, pitch, p.ntok, cut.nt)) return cuda_fail(cudaErrorInvalidValue);
        k = bf ? split_kernel<__nv_bfloat16>(cut.nt) : split_kernel<float>(cut.nt);
        if (p.debug_flags & 2u) a.withhold |= 1u;
        grid = cut.tiles * cut.ks;
        if (grid > 0x7fffffff) return JAMBA_SSM_ERR_UNSUPPORTED;
    }
    a.ks = cut.ks;  // 1 for the pairs' kernel, which has its own cluster of 2
    const cudaError_t e = raise_smem(k, dev->id);
    if (e != cudaSuccess) return cuda_fail(e);
    void *args[] = {&map_w, &map_q, &a};
    st = launch_early(k.fn, dim3(unsigned(grid)), unsigned(k.threads), k.smem, a.ks, args, stream);
    return st != JAMBA_SSM_OK ? st : finish_launch(stream, nullptr);
}

JSSM_SERVE_API jamba_ssm_status jamba_ssm_batch_maps(const jamba_ssm_batch_maps_params *pin, void *stream) {
    jamba_ssm_batch_maps_params p;
    if (!read_params(pin, &p)) return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.requests < 0 || p.max_tokens < 0 || p.max_blocks < 1 || p.block_size < 1 ||
        p.num_free_blocks < 0 || p.num_free_slots < 0)
        return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.requests > (int64_t(1) << 20) || p.max_tokens > (int64_t(1) << 30) ||
        p.max_blocks > (int64_t(1) << 24) || p.block_size > (int64_t(1) << 20) ||
        p.num_free_blocks > 0x7fffffff || p.num_free_slots > 0x7fffffff)
        return JAMBA_SSM_ERR_UNSUPPORTED;
    if (!p.cu_seqlens || !p.counts || (p.num_free_blocks > 0 && !p.free_blocks) ||
        (p.num_free_slots > 0 && !p.free_slots))
        return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.requests > 0 && (!p.new_lens || !p.block_tables || !p.request_slots || !p.state_indices ||
                           !p.initial_indices))
        return JAMBA_SSM_ERR_INVALID_ARG;
    if (p.max_tokens > 0 && (!p.positions || !p.token_request || !p.slot_map))
        return JAMBA_SSM_ERR_INVALID_ARG;
    for (const void *q : {(const void *)p.new_lens, (const void *)p.ctx_lens, (const void *)p.free_blocks,
                          (const void *)p.free_slots, (const void *)p.block_tables,
                          (const void *)p.request_slots, (const void *)p.cu_seqlens,
                          (const void *)p.positions, (const void *)p.token_request,
                          (const void *)p.state_indices, (const void *)p.initial_indices,
                          (const void *)p.counts})
        if (!aligned(q, 4)) return JAMBA_SSM_ERR_MISALIGNED;
    if (!aligned(p.slot_map, 8)) return JAMBA_SSM_ERR_MISALIGNED;
    const size_t r = size_t(p.requests), t = size_t(p.max_tokens);
    const Range ins[] = {{p.new_lens, r * 4},
                         {p.ctx_lens, r * 4},
                         {p.free_blocks, size_t(p.num_free_blocks) * 4},
                         {p.free_slots, size_t(p.num_free_slots) * 4}};
    const Range outs[] = {{p.block_tables, r * size_t(p.max_blocks) * 4},
                          {p.request_slots, r * 4},
                          {p.cu_seqlens, (r + 1) * 4},
                          {p.positions, t * 4},
                          {p.token_request, t * 4},
                          {p.slot_map, t * 8},
                          {p.state_indices, r * 4},
                          {p.initial_indices, r * 4},
                          {p.counts, 16}};
    if (any_overlap(outs, 9, ins, 4)) return JAMBA_SSM_ERR_INVALID_ARG;
    jamba_ssm_status st;
    if (!current_device(&st)) return st;
    jssm::BatchMapsArgs a{};
    a.requests = static_cast<int>(p.requests);
    a.max_tokens = static_cast<int>(p.max_tokens);
    a.max_blocks = static_cast<int>(p.max_blocks);
    a.block_size = static_cast<int>(p.block_size);
    a.new_lens = p.new_lens;
    a.ctx_lens = p.ctx_lens;
    a.free_blocks = p.free_blocks;
    a.free_slots = p.free_slots;
    a.num_free_blocks = static_cast<int>(p.num_free_blocks);
    a.num_free_slots = static_cast<int>(p.num_free_slots);
    a.block_tables = p.block_tables;
    a.request_slots = p.request_slots;
    a.cu_seqlens = p.cu_seqlens;
    a.positions = p.positions;
    a.token_request = p.token_request;
    a.slot_map = p.slot_map;
    a.state_indices = p.state_indices;
    a.initial_indices = p.initial_indices;
    a.counts = p.counts;
    a.wide = aligned(p.positions, 16) && aligned(p.token_request, 16) && aligned(p.slot_map, 16);
    void *args[] = {&a};
    const unsigned ctas =
        unsigned(ceil_div(p.max_tokens, int64_t(jssm::kMapsThreads) * jssm::kMapsTokens));
    if (p.requests <= jssm::kMapsFused) {
        const void *k = p.requests <= jssm::kMapsThreads ? (const void *)&jssm::batch_maps_kernel<1>
                        : p.requests <= 4 * jssm::kMapsThreads ? (const void *)&jssm::batch_maps_kernel<4>
                                                               : (const void *)&jssm::batch_maps_kernel<8>;
        st = launch_early(k, dim3(ctas > 0 ? ctas : 1), jssm::kMapsThreads, 0, 1, args, stream);
    } else {
        st = launch_early((const void *)&jssm::batch_maps_requests_kernel, dim3(1),
                          jssm::kMapsManyThreads, 0, 1, args, stream);
        if (st == JAMBA_SSM_OK && ctas > 0)
            st = launch_early((const void *)&jssm::batch_maps_tokens_kernel, dim3(ctas),
                              jssm::kMapsThreads, 0, 1, args, stream);
    }
    return st != JAMBA_SSM_OK ? st : finish_launch(stream, nullptr);
}

JSSM_SERVE_API jamba_ssm_status jamba_ssm_serve_get_status(void *stream) {
    return read_status(nullptr, stream);
}
JSSM_SERVE_API int jamba_ssm_serve_last_cuda_error(void) { return t_last_cuda_error; }
JSSM_SERVE_API int jamba_ssm_serve_abi_version(void) { return JAMBA_SSM_SERVE_ABI_VERSION; }
